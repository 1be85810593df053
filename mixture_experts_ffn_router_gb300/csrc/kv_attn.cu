// kv_attn.cu — attention of new tokens over the paged key/value cache.
//
// One warp per token and query head walks the visible positions once, with the running maximum m
// and sum l of the softmax: a key's score s moves m to m' = max(m, s), scales l and the output so
// far by exp(m - m') and adds exp(s - m') and exp(s - m') V. Lane i holds the dimensions i, i + 32, ...
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "kv.h"

namespace moe {

namespace {

constexpr int kWarps = 8;

template <int D, bool E4M3>
__device__ __forceinline__ float element(const uint8_t* base, long long i) {
  if constexpr (E4M3) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(base[i], __NV_E4M3)));
  } else {
    return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(base)[i]) << 16);
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) kv_attention_kernel(KvAttn a) {
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int row = static_cast<int>(w / a.q_heads), head = static_cast<int>(w % a.q_heads);
  if (row >= a.b.n_tokens) return;
  int seq = 0;
  while (seq + 1 < a.b.n_seqs && a.b.cu_q[seq + 1] <= row) ++seq;
  KvSeq s = {0, 0, 0};
  if (a.b.n_seqs > 0) s = kv_sequence(a.b, a.c, seq, a.status);
  const int p = row >= s.row0 && row < s.row0 + s.n ? s.len - s.n + (row - s.row0) : -1;
  float q[D / 32], o[D / 32];
  const uint16_t* qp = a.q.ptr + row * a.q.token_stride + head * a.q.head_stride;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    q[i] = __uint_as_float(static_cast<uint32_t>(qp[lane + 32 * i]) << 16) * a.scale;
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  const int kvh = head / a.group;
  const int lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
  for (int j = lo > 0 && a.sinks > 0 ? 0 : lo; j <= p; ++j) {
    if (j < lo && j >= a.sinks) j = lo;
    const int page = kv_page(a.b, a.c, seq, j >> a.c.page_log2, a.status);
    if (page < 0) break;
    const long long at =
        (((static_cast<long long>(page) * a.c.kv_heads + kvh) << a.c.page_log2) + (j & ((1 << a.c.page_log2) - 1)));
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) x += q[i] * element<D, E4M3>(a.c.k, at * D + lane + 32 * i);
#pragma unroll
    for (int t = 16; t > 0; t >>= 1) x += __shfl_xor_sync(0xffffffffu, x, t);
    float vs = 1.0f;
    if constexpr (E4M3) {
      x *= a.c.k_scale[at];
      vs = a.c.v_scale[at];
    }
    // The maximum drops a NaN: before any finite score it stays -inf, and 0 stands in for it below.
    const float m1 = fmaxf(m, x), base = m1 == -INFINITY ? 0.0f : m1;
    const float f = __expf(m - base), e = __expf(x - base);
    l = l * f + e;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = o[i] * f + e * vs * element<D, E4M3>(a.c.v, at * D + lane + 32 * i);
    m = m1;
  }
  const long long to = static_cast<long long>(row) * a.q_heads + head;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    a.out[to * D + lane + 32 * i] = __bfloat16_as_ushort(__float2bfloat16_rn(l == 0.0f ? 0.0f : o[i] / l));
  if (a.lse && lane == 0) a.lse[to] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_kv_attention(const KvAttn& a, cudaStream_t s) {
  const unsigned grid =
      static_cast<unsigned>((static_cast<long long>(a.b.n_tokens) * a.q_heads + kWarps - 1) / kWarps);
  switch (a.c.head_dim * 2 + a.c.e4m3) {
    case 256: kv_attention_kernel<128, false><<<grid, kWarps * 32, 0, s>>>(a); break;
    case 257: kv_attention_kernel<128, true><<<grid, kWarps * 32, 0, s>>>(a); break;
    case 512: kv_attention_kernel<256, false><<<grid, kWarps * 32, 0, s>>>(a); break;
    case 513: kv_attention_kernel<256, true><<<grid, kWarps * 32, 0, s>>>(a); break;
    case 1024: kv_attention_kernel<512, false><<<grid, kWarps * 32, 0, s>>>(a); break;
    default: kv_attention_kernel<512, true><<<grid, kWarps * 32, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace moe
