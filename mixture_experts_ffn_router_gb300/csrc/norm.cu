// norm.cu — the norms after one block and before the next, with the gated residual between them.
//
//   y = scale * (x + gate * N(block; post)),  n = N(y; pre),  N(v; w) = v / sqrt(mean(v^2) + eps) * (1 + w)
//
// 8 to 10 bytes per value meet a dozen operations, so HBM bounds it, or the launch where tokens are few. A CTA takes
// one row, whose values stay in its registers from the only load to the stores: a thread holds up to kMaxVecs vectors
// of eight of x, block and gate, all loaded before the first is used. The two sums of squares are a reduction over
// the CTA each. The row's statistics and y are fp32; y and n are rounded once.
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "moe_ffn.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxVecs = 4;

struct NormParams {
  const uint16_t* x;
  const uint16_t* block;
  const uint16_t* gate;
  const float* post;
  const float* pre;
  uint16_t* y;
  uint16_t* n;
  long long x_stride, block_stride, gate_stride, y_stride, n_stride;
  float scale, eps;
  int hidden;
};

__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// The sum over the CTA, in every thread. `sums` holds a float per warp and is not used again before the next barrier.
__device__ __forceinline__ float cta_sum(float v, float* sums) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  v = lane < warps ? sums[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Multiplies by (1 + w) of eight features.
__device__ __forceinline__ void weighted(float (&f)[8], const float* w, float r) {
  const float4 a = *reinterpret_cast<const float4*>(w), b = *reinterpret_cast<const float4*>(w + 4);
  const float g[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = f[i] * r * (1.0f + g[i]);
}

template <int VECS>
__global__ void __launch_bounds__(kMaxThreads) block_norm_kernel(const NormParams p) {
  __shared__ float sums[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const long long row = blockIdx.x;
  const int vecs = p.hidden / 8;
  uint4 xv[VECS], bv[VECS], gv[VECS];
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    const int at = (j * blockDim.x + threadIdx.x) * 8;
    xv[j] = bv[j] = gv[j] = make_uint4(0u, 0u, 0u, 0u);
    if (at >= p.hidden) continue;
    xv[j] = *reinterpret_cast<const uint4*>(p.x + row * p.x_stride + at);
    if (p.block) bv[j] = *reinterpret_cast<const uint4*>(p.block + row * p.block_stride + at);
    if (p.gate) gv[j] = *reinterpret_cast<const uint4*>(p.gate + row * p.gate_stride + at);
  }
  float f[VECS][8];
  float r = 1.0f;
  if (p.post) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      unpack(bv[j], f[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(f[j][i], f[j][i], sum);
    }
    r = rsqrtf(cta_sum(sum, sums[0]) / static_cast<float>(p.hidden) + p.eps);
  }
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    const int v = j * blockDim.x + threadIdx.x;
    if (v >= vecs) continue;
    float x[8];
    unpack(xv[j], x);
    if (p.block) {
      unpack(bv[j], f[j]);
      if (p.post) weighted(f[j], p.post + v * 8, r);
      if (p.gate) {
        float g[8];
        unpack(gv[j], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[j][i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] += f[j][i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[j][i] = x[i] * p.scale;
      sum = fmaf(f[j][i], f[j][i], sum);
    }
    if (p.y) *reinterpret_cast<uint4*>(p.y + row * p.y_stride + v * 8) = pack(f[j]);
  }
  if (!p.n) return;
  r = rsqrtf(cta_sum(sum, sums[1]) / static_cast<float>(p.hidden) + p.eps);
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    const int v = j * blockDim.x + threadIdx.x;
    if (v >= vecs) continue;
    weighted(f[j], p.pre + v * 8, r);
    *reinterpret_cast<uint4*>(p.n + row * p.n_stride + v * 8) = pack(f[j]);
  }
}

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// Whether rows of `bytes` bytes at a, and others at b, have a byte in common. Rows that interleave at one stride do
// not, if they fit between each other.
bool rows_meet(const void* a, long long sa, const void* b, long long sb, long long rows, long long bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  if (x >= y + (rows - 1) * sb + bytes || y >= x + (rows - 1) * sa + bytes) return false;
  if (sa != sb || sa < 2 * bytes) return true;
  const long long d = static_cast<long long>((y > x ? y - x : x - y) % sa);
  return d < bytes || sa - d < bytes;
}

}  // namespace

}  // namespace moe

extern "C" int moe_ffn_block_norm(const moe_ffn_norm* a, void* stream) {
  using namespace moe;
  if (!a || a->tokens < 0 || a->hidden < 8 || a->hidden > MOE_FFN_NORM_MAX_HIDDEN || a->hidden % 8 != 0)
    return MOE_FFN_EINVAL;
  if (!(a->eps > 0.0f) || !std::isfinite(a->eps) || !std::isfinite(a->scale)) return MOE_FFN_EINVAL;
  if (a->x_stride < 0 || a->block_stride < 0 || a->gate_stride < 0) return MOE_FFN_EINVAL;
  if (a->tokens == 0) return MOE_FFN_OK;
  if (!a->x || (!a->y && !a->n) || !a->n != !a->pre || (!a->block && (a->gate || a->post))) return MOE_FFN_EINVAL;
  if ((a->y && a->y_stride < a->hidden) || (a->n && a->n_stride < a->hidden)) return MOE_FFN_EINVAL;
  const void* pointers[] = {a->x, a->block, a->gate, a->post, a->pre, a->y, a->n};
  for (const void* p : pointers)
    if (off16(p)) return MOE_FFN_EALIGN;
  const long long strides[] = {a->x_stride, a->block ? a->block_stride : 0, a->gate ? a->gate_stride : 0,
                               a->y ? a->y_stride : 0, a->n ? a->n_stride : 0};
  for (long long s : strides)
    if (s % 8 != 0) return MOE_FFN_EALIGN;
  const long long rows = a->tokens, bytes = 2LL * a->hidden;
  struct { const void* p; long long stride; } outs[] = {{a->y, 2 * a->y_stride}, {a->n, 2 * a->n_stride}},
                                              ins[] = {{a->x, 2 * a->x_stride}, {a->block, 2 * a->block_stride}};
  for (const auto& o : outs) {
    if (!o.p) continue;
    for (const auto& i : ins)
      if (i.p && !(i.p == o.p && (i.stride == o.stride || rows == 1)) && rows_meet(o.p, o.stride, i.p, i.stride, rows, bytes))
        return MOE_FFN_EINVAL;
    if (a->gate && rows_meet(o.p, o.stride, a->gate, 2 * a->gate_stride, rows, bytes)) return MOE_FFN_EINVAL;
    const float* weights[] = {a->post, a->pre};
    for (const float* w : weights)
      if (w && (rows_meet(o.p, o.stride, w, 0, rows, bytes) || rows_meet(o.p, o.stride, w + a->hidden / 2, 0, rows, bytes)))
        return MOE_FFN_EINVAL;
  }
  if (a->y && a->n && rows_meet(a->y, 2 * a->y_stride, a->n, 2 * a->n_stride, rows, bytes)) return MOE_FFN_EINVAL;
  NormParams p;
  p.x = static_cast<const uint16_t*>(a->x);
  p.block = static_cast<const uint16_t*>(a->block);
  p.gate = static_cast<const uint16_t*>(a->gate);
  p.post = a->post;
  p.pre = a->pre;
  p.y = static_cast<uint16_t*>(a->y);
  p.n = static_cast<uint16_t*>(a->n);
  p.x_stride = a->x_stride;
  p.block_stride = a->block_stride;
  p.gate_stride = a->gate_stride;
  p.y_stride = a->y_stride;
  p.n_stride = a->n_stride;
  p.scale = a->scale;
  p.eps = a->eps;
  p.hidden = a->hidden;
  // As few vectors to a thread as the block's limit allows.
  const int vecs = a->hidden / 8, per = (vecs + kMaxThreads - 1) / kMaxThreads;
  const dim3 grid(a->tokens), block(((vecs + per - 1) / per + 31) / 32 * 32);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (per) {
    case 1: e = launch_pdl(block_norm_kernel<1>, grid, block, 0, s, p); break;
    case 2: e = launch_pdl(block_norm_kernel<2>, grid, block, 0, s, p); break;
    case 3: e = launch_pdl(block_norm_kernel<3>, grid, block, 0, s, p); break;
    default: e = launch_pdl(block_norm_kernel<kMaxVecs>, grid, block, 0, s, p); break;
  }
  return e == cudaSuccess ? MOE_FFN_OK : MOE_FFN_ECUDA;
}
