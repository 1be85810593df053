// norm.cu — the norms after one block and before the next, with the gated residual between them.
//
//   y = scale * (x + gate * N(block; post)),  n = N(y; pre),  N(v; w) = v / sqrt(mean(v^2) + eps) * (1 + w)
//
// 8 to 10 bytes per value meet a dozen operations, so HBM bounds it, or the launch where tokens are few. A CTA takes
// a row at a time, whose values stay in its registers from the only load to the stores: a thread holds up to kMaxVecs
// vectors of eight of x, block and gate. The two sums of squares are a reduction over the CTA each. The row's statistics
// and y are fp32; y and n are rounded once. 8192 rows of 2816 with a gate take 38.1 us, 91% of the copy rate; 64 rows 2.4
// in a graph (from Python the call itself takes 11 to 16).
//
// Narrow rows: a warp for each, whose sums need no barrier. Others, where they are few or very wide: a CTA for each, all its
// loads before the first use. Many rows: CTAs that stay, each with every gridDim-th row, the weights in registers and the
// next kAhead rows on their way into shared memory (a thread copies what it will read itself, so no barrier is needed for
// that).
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "moe_ffn.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxVecs = 4;
constexpr int kRowWarps = 8;    // of a CTA, where a row is a warp's

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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The sum over the CTA, in every thread. `sums` holds a float per warp and is not used again before the next barrier.
__device__ __forceinline__ float cta_sum(float v, float* sums) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  return warp_sum(lane < warps ? sums[lane] : 0.0f);
}

// Multiplies by (1 + w) of eight features.
__device__ __forceinline__ void weighted(float (&f)[8], const float* w, float r) {
  const float4 a = *reinterpret_cast<const float4*>(w), b = *reinterpret_cast<const float4*>(w + 4);
  const float g[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = f[i] * r * (1.0f + g[i]);
}

// WARP: a row to a warp, else to a CTA.
template <int VECS, bool WARP>
__global__ void __launch_bounds__(WARP ? kRowWarps * 32 : kMaxThreads) block_norm_kernel(const NormParams p, int tokens) {
  __shared__ float sums[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const long long row = WARP ? static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= tokens) return;
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, n = WARP ? 32 : blockDim.x;
  const int vecs = p.hidden / 8;
  auto row_sum = [&](float v, float* to) { return WARP ? warp_sum(v) : cta_sum(v, to); };
  uint4 xv[VECS], bv[VECS], gv[VECS];
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    const int at = (j * n + tid) * 8;
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
    r = rsqrtf(row_sum(sum, sums[0]) / static_cast<float>(p.hidden) + p.eps);
  }
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    const int v = j * n + tid;
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
  r = rsqrtf(row_sum(sum, sums[1]) / static_cast<float>(p.hidden) + p.eps);
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    const int v = j * n + tid;
    if (v >= vecs) continue;
    weighted(f[j], p.pre + v * 8, r);
    *reinterpret_cast<uint4*>(p.n + row * p.n_stride + v * 8) = pack(f[j]);
  }
}

constexpr int kAhead = 3;
constexpr int kSms = 152;

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// Rows of up to 8 * THREADS values, a vector of eight to a thread. `parts`: 1, and 1 for a block and for a gate each.
template <int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) block_norm_rows_kernel(const NormParams p, int tokens, int parts) {
  extern __shared__ uint4 ring[];  // [kAhead + 1][parts][blockDim.x]
  __shared__ float sums[2][2][32];
  const int tid = threadIdx.x, n = blockDim.x, at = tid * 8;
  const bool live = at < p.hidden;
  pdl_wait();
  pdl_launch_dependents();
  auto fetch = [&](long long row, int slot) {
    if (live && row < tokens) {
      const uint32_t to = smem_u32(ring + slot * parts * n + tid);
      copy16(to, p.x + row * p.x_stride + at);
      if (p.block) copy16(to + 16 * n, p.block + row * p.block_stride + at);
      if (p.gate) copy16(to + 32 * n, p.gate + row * p.gate_stride + at);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(blockIdx.x + static_cast<long long>(i) * gridDim.x, i);
  float post[8], pre[8];  // 1 + w
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    post[i] = live && p.post ? 1.0f + p.post[at + i] : 1.0f;
    pre[i] = live && p.pre ? 1.0f + p.pre[at + i] : 1.0f;
  }
  const float inv = 1.0f / static_cast<float>(p.hidden);
  int slot = 0;
  for (long long row = blockIdx.x, k = 0; row < tokens; row += gridDim.x, ++k) {
    fetch(row + static_cast<long long>(kAhead) * gridDim.x, slot == 0 ? kAhead : slot - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
    const uint4* mine = ring + slot * parts * n + tid;
    if (++slot > kAhead) slot = 0;
    float f[8], x[8];
    unpack(live ? mine[0] : make_uint4(0u, 0u, 0u, 0u), x);
    if (p.block) {
      unpack(live ? mine[n] : make_uint4(0u, 0u, 0u, 0u), f);
      if (p.post) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], sum);
        // (Two sets of sums: a warp may be a row ahead of one that still reads.)
        const float r = rsqrtf(cta_sum(sum, sums[k & 1][0]) * inv + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * r * post[i];
      }
      if (p.gate) {
        float g[8];
        unpack(live ? mine[2 * n] : make_uint4(0u, 0u, 0u, 0u), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] += f[i];
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] *= p.scale;
      sum = fmaf(x[i], x[i], sum);
    }
    if (p.y && live) *reinterpret_cast<uint4*>(p.y + row * p.y_stride + at) = pack(x);
    if (!p.n) continue;
    const float r = rsqrtf(cta_sum(sum, sums[k & 1][1]) * inv + p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * pre[i];
    if (live) *reinterpret_cast<uint4*>(p.n + row * p.n_stride + at) = pack(x);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// CTAS of THREADS to an SM, or more of fewer.
template <int THREADS, int CTAS>
cudaError_t launch_rows(const NormParams& p, int tokens, int parts, dim3 block, int smem, cudaStream_t s) {
  const auto kernel = block_norm_rows_kernel<THREADS, CTAS>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (kAhead + 1) * 3 * 16 * THREADS);
  return e == cudaSuccess ? launch_pdl(kernel, dim3(THREADS * CTAS / block.x * kSms), block, smem, s, p, tokens, parts) : e;
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
  // Which of the three, in us of two inputs without a gate. A warp to a row or a CTA: 40000 rows of 264 24 and 41, of 512 29 and
  // 42; of 1024 the warp's loads are too few (8192 rows: 17 and 15). CTAs that stay, or one a row: 8192 rows of 2816 35 and
  // 40, of 4096 46 and 56, of 2048 26 and 28; of 1536 21 and 21, and narrower ones with a gate lose (40000 of 768: 55 and
  // 50). Below about eight rows to each they lose too (2000 rows of 2816: 11.6 and 10.7). Above 4096 a CTA for each row is all
  // there is: 8192 rows of 4104 60 us, of 5376 84, of 8192 104, of 16384 256 (1.5, 1.6, 1.3 and 1.6 times the bytes).
  if (vecs <= 64) {
    const dim3 rows((a->tokens + kRowWarps - 1) / kRowWarps), warps(kRowWarps * 32);
    e = vecs <= 32 ? launch_pdl(block_norm_kernel<1, true>, rows, warps, 0, s, p, a->tokens)
                   : launch_pdl(block_norm_kernel<2, true>, rows, warps, 0, s, p, a->tokens);
  } else if (per == 1 && block.x >= 224 && static_cast<long long>(a->tokens) * block.x >= 8LL * kSms * 1152) {
    const int parts = 1 + (a->block ? 1 : 0) + (a->gate ? 1 : 0), smem = (kAhead + 1) * parts * 16 * static_cast<int>(block.x);
    e = block.x <= 384 ? launch_rows<384, 3>(p, a->tokens, parts, block, smem, s) : launch_rows<512, 2>(p, a->tokens, parts, block, smem, s);
  } else {
    switch (per) {
      case 1: e = launch_pdl(block_norm_kernel<1, false>, grid, block, 0, s, p, a->tokens); break;
      case 2: e = launch_pdl(block_norm_kernel<2, false>, grid, block, 0, s, p, a->tokens); break;
      case 3: e = launch_pdl(block_norm_kernel<3, false>, grid, block, 0, s, p, a->tokens); break;
      default: e = launch_pdl(block_norm_kernel<kMaxVecs, false>, grid, block, 0, s, p, a->tokens); break;
    }
  }
  return e == cudaSuccess ? MOE_FFN_OK : MOE_FFN_ECUDA;
}
