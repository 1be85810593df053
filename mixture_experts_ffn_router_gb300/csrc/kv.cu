// kv.cu — the paged key/value cache: the host side of its C ABI, and the kernels that write new
// tokens into it and read cached ones back.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cmath>
#include <new>

#include "internal.h"
#include "kv.h"
#include "moe_ffn.h"

namespace moe {

namespace {

// Writing and reading back. A row is one head's key or value of one token, D bf16 values in
// registers as 16-byte vectors, D / 8 lanes (or D / 16 with two vectors) to a row. A warp takes
// 2 KB of one token's keys, or of its values: four loads per lane in flight before the first is used,
// and enough warps for a single decode step's tokens to spread over the SMs.
constexpr int kMoveWarps = 8;
constexpr int kVecs = 4;  // 16-byte bf16 vectors per lane

// The sequence a token row belongs to, found by the whole warp: 32 probes per step, so two steps for
// up to 1023 sequences instead of ten of a binary search, each a dependent load.
__device__ __forceinline__ int find_sequence(const KvBatch& b, int row, int lane) {
  int lo = 0, hi = b.n_seqs;  // the answer's last sequence with cu_q <= row is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && b.cu_q[min(at, hi - 1)] <= row);
    const int last = 31 - __clz(le | 1u);
    lo += last * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Where token row `row` is kept: {page, slot}, page -1 if nowhere.
__device__ __forceinline__ int2 find_place(const KvBatch& b, const KvCache& c, int row, int lane,
                                           unsigned int* status) {
  if (b.n_seqs == 0) return make_int2(-1, 0);
  const int seq = find_sequence(b, row, lane);
  const KvSeq s = kv_sequence(b, c, seq, status);
  const int i = row - s.row0;
  if (i < 0 || i >= s.n) return make_int2(-1, 0);
  const int pos = s.len - s.n + i;
  if (pos < 0) return make_int2(-1, 0);
  return make_int2(kv_page(b, c, seq, pos >> c.page_log2, status), pos & ((1 << c.page_log2) - 1));
}

// The e4m3 codes of x / s, each quotient correctly rounded in fp32 first, of two bf16 numbers whose negated
// values are the halves of `neg`. From the correctly rounded reciprocal of s: a quotient, its exact
// remainder by fma, and one correction (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990), two at a time; of the signs, the negated value is what keeps a -0. Far
// from the ends of the exponent range only; a remainder that underflows belongs to a quotient that
// rounds to the code 0 anyway. (A division per value bounded the kernel: 102 us for 317 MB.)
__device__ __forceinline__ uint32_t quotient_codes(uint32_t neg, unsigned long long s2, unsigned long long nr2) {
  unsigned long long nx, q, rem;
  asm("mov.b64 %0, {%1, %2};" : "=l"(nx) : "r"(neg << 16), "r"(neg & 0xFFFF0000u));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(nx), "l"(nr2));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(rem) : "l"(q), "l"(s2), "l"(nx));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(rem), "l"(nr2), "l"(q));
  float2 y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(q));
  return __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ unsigned long long twice(float x) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
  return r;
}

// How a warp's lanes lie over its rows: kRows rows of each group of kLanes lanes, kVecs vectors each.
template <int D>
struct Move {
  static constexpr int kLanes = D / 8 < 32 ? D / 8 : 32;  // lanes of a row
  static constexpr int kRowVecs = D / 8 / kLanes;         // vectors of a row per lane
  static constexpr int kRows = kVecs / kRowVecs;          // rows per lane
  static constexpr int kGroups = 32 / kLanes;             // rows side by side
  static constexpr int kWarpRows = kRows * kGroups;
};

// The same of eight numbers by divisions, out of line; of a row of zeros or with a value that is not finite
// codes 0.
__device__ __noinline__ uint2 divided_codes(uint4 x, float s) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  uint32_t code[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    code[q] = s > 0.0f ? __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(__uint_as_float(u[q] << 16), s),
                                                              __fdiv_rn(__uint_as_float(u[q] & 0xFFFF0000u), s)),
                                                  __NV_SATFINITE, __NV_E4M3)
                       : 0u;
  return make_uint2(__byte_perm(code[0], code[1], 0x5410), __byte_perm(code[2], code[3], 0x5410));
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kMoveWarps * 32)
    kv_write_kernel(KvBatch b, KvCache c, KvRows k, KvRows v, unsigned int* status) {
  using M = Move<D>;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
  if (row >= b.n_tokens) return;
  const bool value = blockIdx.z != 0;
  const int sub = lane % M::kLanes, h0 = blockIdx.y * M::kWarpRows + lane / M::kLanes;
  const long long head_stride = value ? v.head_stride : k.head_stride;
  const uint16_t* src = (value ? v.ptr : k.ptr) + row * (value ? v.token_stride : k.token_stride) + h0 * head_stride + sub * 8;
  uint4 x[M::kRows][M::kRowVecs];
#pragma unroll
  for (int i = 0; i < M::kRows; ++i) {
    if (h0 + i * M::kGroups >= c.kv_heads) continue;
#pragma unroll
    for (int j = 0; j < M::kRowVecs; ++j)
      x[i][j] = *reinterpret_cast<const uint4*>(src + i * M::kGroups * head_stride + j * M::kLanes * 8);
  }
  const int2 at = find_place(b, c, row, lane, status);
  if (at.x < 0) return;
  const long long to = ((static_cast<long long>(at.x) * c.kv_heads + h0) << c.page_log2) + at.y;  // the lane's first row
  const long long step = static_cast<long long>(M::kGroups) << c.page_log2;
  if constexpr (!E4M3) {
    uint16_t* dst = reinterpret_cast<uint16_t*>(value ? c.v : c.k) + to * D + sub * 8;
#pragma unroll
    for (int i = 0; i < M::kRows; ++i) {
      if (h0 + i * M::kGroups >= c.kv_heads) continue;
#pragma unroll
      for (int j = 0; j < M::kRowVecs; ++j)
        *reinterpret_cast<uint4*>(dst + i * step * D + j * M::kLanes * 8) = x[i][j];
    }
  } else {
    // Each row's largest magnitude, on the bits: they order as the values do, with infinities and NaNs
    // (which fmaxf would drop) above every finite one. Two at a time, as 16-bit numbers; in the first steps
    // lanes trade rows, so that a lane ends with one row's.
    uint32_t top[M::kRows];
#pragma unroll
    for (int i = 0; i < M::kRows; ++i) {
      top[i] = 0;
      if (h0 + i * M::kGroups < c.kv_heads) {
#pragma unroll
        for (int j = 0; j < M::kRowVecs; ++j)
          top[i] = __vmaxu2(top[i], __vmaxu2(__vmaxu2(x[i][j].x & 0x7fff7fffu, x[i][j].y & 0x7fff7fffu),
                                             __vmaxu2(x[i][j].z & 0x7fff7fffu, x[i][j].w & 0x7fff7fffu)));
      }
    }
    int d = M::kLanes / 2;
#pragma unroll
    for (int half = M::kRows / 2; half > 0; half >>= 1, d >>= 1) {
      const bool up = lane & d;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? top[i] : top[i + half], d);
        top[i] = __vmaxu2(up ? top[i + half] : top[i], got);
      }
    }
#pragma unroll
    for (; d > 0; d >>= 1) top[0] = __vmaxu2(top[0], __shfl_xor_sync(0xffffffffu, top[0], d));
    // Row i's is in the lanes whose highest bits (within the row's lanes) are i; one division and one
    // reciprocal per lane serve all rows.
    const uint32_t mine = max(top[0] << 16, top[0] & 0xffff0000u);
    const float scale = mine < 0x7f800000u ? __fdiv_rn(__uint_as_float(mine), 448.0f) : __uint_as_float(0x7fffffffu);
    const float recip = __frcp_rn(scale);
    const int my_row = sub / (M::kLanes / M::kRows);
    if (sub % (M::kLanes / M::kRows) == 0 && h0 + my_row * M::kGroups < c.kv_heads)
      (value ? c.v_scale : c.k_scale)[to + my_row * step] = scale;
    uint8_t* dst = (value ? c.v : c.k) + to * D + sub * 8;
#pragma unroll
    for (int i = 0; i < M::kRows; ++i) {
      const int from = (lane & ~(M::kLanes - 1)) + i * (M::kLanes / M::kRows);
      const float s = __shfl_sync(0xffffffffu, scale, from), r_s = __shfl_sync(0xffffffffu, recip, from);
      if (h0 + i * M::kGroups >= c.kv_heads) continue;
      const bool fast = s > 0x1p-90f && s < 0x1p90f;
      const unsigned long long s2 = twice(s), nr2 = twice(-r_s);
#pragma unroll
      for (int j = 0; j < M::kRowVecs; ++j) {
        uint2 codes;
        if (__builtin_expect(fast, 1)) {
          const uint32_t u[4] = {x[i][j].x, x[i][j].y, x[i][j].z, x[i][j].w};
          uint32_t code[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) code[q] = quotient_codes(u[q] ^ 0x80008000u, s2, nr2);
          codes = make_uint2(__byte_perm(code[0], code[1], 0x5410), __byte_perm(code[2], code[3], 0x5410));
        } else {
          codes = divided_codes(x[i][j], s);
        }
        *reinterpret_cast<uint2*>(dst + i * step * D + j * M::kLanes * 8) = codes;
      }
    }
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kMoveWarps * 32)
    kv_read_kernel(KvBatch b, KvCache c, uint16_t* k_out, uint16_t* v_out, unsigned int* status) {
  using M = Move<D>;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
  if (row >= b.n_tokens) return;
  const bool value = blockIdx.z != 0;
  const int sub = lane % M::kLanes, h0 = blockIdx.y * M::kWarpRows + lane / M::kLanes;
  const int2 at = find_place(b, c, row, lane, status);
  const long long from = ((static_cast<long long>(max(at.x, 0)) * c.kv_heads + h0) << c.page_log2) + at.y;
  const long long step = static_cast<long long>(M::kGroups) << c.page_log2;
  const uint8_t* src = (value ? c.v : c.k) + (from * D + sub * 8) * (E4M3 ? 1 : 2);
  uint4 x[M::kRows][M::kRowVecs];
  float s[M::kRows];
#pragma unroll
  for (int i = 0; i < M::kRows; ++i) {
    s[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < M::kRowVecs; ++j) x[i][j] = make_uint4(0u, 0u, 0u, 0u);
    if (h0 + i * M::kGroups >= c.kv_heads || at.x < 0) continue;
#pragma unroll
    for (int j = 0; j < M::kRowVecs; ++j) {
      const uint8_t* p = src + (i * step * D + j * M::kLanes * 8) * (E4M3 ? 1 : 2);
      if constexpr (E4M3) {
        const uint2 code = *reinterpret_cast<const uint2*>(p);
        x[i][j].x = code.x;
        x[i][j].y = code.y;
      } else {
        x[i][j] = *reinterpret_cast<const uint4*>(p);
      }
    }
    if constexpr (E4M3) s[i] = (value ? c.v_scale : c.k_scale)[from + i * step];
  }
  uint16_t* dst = (value ? v_out : k_out) + (static_cast<long long>(row) * c.kv_heads + h0) * D + sub * 8;
#pragma unroll
  for (int i = 0; i < M::kRows; ++i) {
    if (h0 + i * M::kGroups >= c.kv_heads) continue;
#pragma unroll
    for (int j = 0; j < M::kRowVecs; ++j) {
      uint4 y = x[i][j];
      if constexpr (E4M3) {
        const uint32_t code[2] = {x[i][j].x, x[i][j].y};
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const __half2_raw hr =
              __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(code[q >> 1] >> (16 * (q & 1))), __NV_E4M3);
          const float2 f = __half22float2(__half2(hr));
          const __nv_bfloat162 p = __floats2bfloat162_rn(f.x * s[i], f.y * s[i]);
          o[q] = *reinterpret_cast<const uint32_t*>(&p);
        }
        y = make_uint4(o[0], o[1], o[2], o[3]);
      }
      *reinterpret_cast<uint4*>(dst + (i * M::kGroups * D + j * M::kLanes * 8)) = y;
    }
  }
}

// Eight tokens to a block, 2 KB of each token's keys or values to a warp. (All of a token's rows to a warp,
// so that its place is found once, was slower: 97 us against 80 for 317 MB.)
dim3 move_grid(const KvBatch& b, const KvCache& c) {
  return dim3((b.n_tokens + kMoveWarps - 1) / kMoveWarps, (c.kv_heads * c.head_dim + 1023) / 1024, 2);
}

}  // namespace

cudaError_t launch_kv_write(const KvBatch& b, const KvCache& c, const KvRows& k, const KvRows& v, unsigned int* status,
                            cudaStream_t s) {
  const dim3 grid = move_grid(b, c), block(kMoveWarps * 32);
  switch (c.head_dim * 2 + c.e4m3) {
    case 256: kv_write_kernel<128, false><<<grid, block, 0, s>>>(b, c, k, v, status); break;
    case 257: kv_write_kernel<128, true><<<grid, block, 0, s>>>(b, c, k, v, status); break;
    case 512: kv_write_kernel<256, false><<<grid, block, 0, s>>>(b, c, k, v, status); break;
    case 513: kv_write_kernel<256, true><<<grid, block, 0, s>>>(b, c, k, v, status); break;
    case 1024: kv_write_kernel<512, false><<<grid, block, 0, s>>>(b, c, k, v, status); break;
    default: kv_write_kernel<512, true><<<grid, block, 0, s>>>(b, c, k, v, status); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvBatch& b, const KvCache& c, uint16_t* k_out, uint16_t* v_out, unsigned int* status,
                           cudaStream_t s) {
  const dim3 grid = move_grid(b, c), block(kMoveWarps * 32);
  switch (c.head_dim * 2 + c.e4m3) {
    case 256: kv_read_kernel<128, false><<<grid, block, 0, s>>>(b, c, k_out, v_out, status); break;
    case 257: kv_read_kernel<128, true><<<grid, block, 0, s>>>(b, c, k_out, v_out, status); break;
    case 512: kv_read_kernel<256, false><<<grid, block, 0, s>>>(b, c, k_out, v_out, status); break;
    case 513: kv_read_kernel<256, true><<<grid, block, 0, s>>>(b, c, k_out, v_out, status); break;
    case 1024: kv_read_kernel<512, false><<<grid, block, 0, s>>>(b, c, k_out, v_out, status); break;
    default: kv_read_kernel<512, true><<<grid, block, 0, s>>>(b, c, k_out, v_out, status); break;
  }
  return cudaGetLastError();
}

}  // namespace moe

// ------------------------------------------------------------------ the C ABI

using namespace moe;

struct moe_ffn_kv {
  moe_ffn_kv_config cfg;
  int device;
  int num_sms;
  uint8_t* ws;
  size_t ws_bytes;
  unsigned int* status;
  int* counters;
  int* counters_in;
  float* partial;
  KvChunkList list;
  float* chunk_partial;
  int chunk_pairs;  // SM pairs of the kernel for chunks
};

namespace {

bool kv_config_ok(const moe_ffn_kv_config* c) {
  return c && c->kv_heads >= 1 && c->kv_heads <= 1024 && c->q_heads >= c->kv_heads && c->q_heads % c->kv_heads == 0 &&
         c->q_heads / c->kv_heads <= 64 && (c->head_dim == 128 || c->head_dim == 256 || c->head_dim == 512) &&
         (c->page_size == 16 || c->page_size == 32 || c->page_size == 64 || c->page_size == 128) && c->n_pages >= 1 &&
         static_cast<long long>(c->n_pages) * c->kv_heads * c->page_size < (1LL << 31) &&
         (c->format == MOE_FFN_KV_BF16 || c->format == MOE_FFN_KV_E4M3) && c->max_tokens >= 1 &&
         c->max_tokens <= MOE_FFN_KV_MAX_TOKENS_LIMIT && c->max_seqs >= 1 && c->max_seqs <= MOE_FFN_KV_MAX_SEQS_LIMIT;
}

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

bool meet(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

// Checks a call's cache and batch and gives them in the kernels' form. Returns MOE_FFN_OK, an error,
// or 1 if there is nothing to do.
int kv_arguments(const moe_ffn_kv* kv, const moe_ffn_kv_cache* cache, const moe_ffn_kv_batch* batch, KvBatch* b,
                 KvCache* c) {
  if (!kv || !cache || !batch) return MOE_FFN_EINVAL;
  if (batch->n_tokens < 0 || batch->n_seqs < 0 || batch->pages_cols < 0 || batch->max_new < 0 ||
      batch->pages_stride < batch->pages_cols)
    return MOE_FFN_EINVAL;
  if (batch->n_tokens > kv->cfg.max_tokens || batch->n_seqs > kv->cfg.max_seqs) return MOE_FFN_ETOOBIG;
  if (batch->n_tokens == 0) return 1;
  const bool q8 = kv->cfg.format == MOE_FFN_KV_E4M3;
  if (!cache->k || !cache->v || (q8 && (!cache->k_scale || !cache->v_scale))) return MOE_FFN_EINVAL;
  if (batch->n_seqs > 0 && (!batch->cu_q || !batch->kv_len || (batch->pages_cols > 0 && !batch->pages)))
    return MOE_FFN_EINVAL;
  if (off16(cache->k) || off16(cache->v) || (q8 && (off16(cache->k_scale) || off16(cache->v_scale))) ||
      off4(batch->cu_q) || off4(batch->kv_len) || off4(batch->pages))
    return MOE_FFN_EALIGN;
  b->cu_q = batch->cu_q;
  b->kv_len = batch->kv_len;
  b->pages = batch->pages;
  b->pages_stride = batch->pages_stride;
  b->pages_cols = batch->pages_cols;
  b->n_seqs = batch->n_seqs;
  b->n_tokens = batch->n_tokens;
  b->max_new = batch->max_new;
  c->k = static_cast<uint8_t*>(cache->k);
  c->v = static_cast<uint8_t*>(cache->v);
  c->k_scale = cache->k_scale;
  c->v_scale = cache->v_scale;
  c->n_pages = kv->cfg.n_pages;
  c->kv_heads = kv->cfg.kv_heads;
  c->page_log2 = kv->cfg.page_size == 16 ? 4 : kv->cfg.page_size == 32 ? 5 : kv->cfg.page_size == 64 ? 6 : 7;
  c->head_dim = kv->cfg.head_dim;
  c->e4m3 = q8 ? 1 : 0;
  return MOE_FFN_OK;
}

int kv_rows(const moe_ffn_kv_rows* r, KvRows* o) {
  if (!r || !r->ptr || r->token_stride < 0 || r->head_stride < 0) return MOE_FFN_EINVAL;
  if (off16(r->ptr) || r->token_stride % 8 != 0 || r->head_stride % 8 != 0) return MOE_FFN_EALIGN;
  o->ptr = static_cast<const uint16_t*>(r->ptr);
  o->token_stride = r->token_stride;
  o->head_stride = r->head_stride;
  return MOE_FFN_OK;
}

size_t kv_rows_bytes(const KvRows& r, int tokens, int heads, int d) {
  return static_cast<size_t>((tokens - 1) * r.token_stride + (heads - 1) * r.head_stride + d) * 2;
}

// Whether an output would meet the cache that the call reads.
bool meets_cache(const void* p, size_t bytes, const KvCache& c) {
  const size_t rows = (static_cast<size_t>(c.n_pages) * c.kv_heads) << c.page_log2, values = rows * c.head_dim * (c.e4m3 ? 1 : 2);
  return meet(p, bytes, c.k, values) || meet(p, bytes, c.v, values) ||
         (c.e4m3 && (meet(p, bytes, c.k_scale, rows * 4) || meet(p, bytes, c.v_scale, rows * 4)));
}

// The workspace: control words (zeroed when the handle is made), then the kernels' pieces.
struct KvLayout {
  size_t status, counters, counters_in, n_tiles, partial, first_tile, tiles, first_unit, shares, joins, chunk_partial,
      total;
};

size_t max_row_tiles(const moe_ffn_kv_config& c) {
  return static_cast<size_t>(c.max_tokens) / chunk_tokens(c.q_heads / c.kv_heads) + c.max_seqs;
}

KvLayout make_kv_layout(const moe_ffn_kv_config& c) {
  KvLayout l;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  l.status = take(4);
  l.counters = take(static_cast<size_t>(c.max_seqs) * c.kv_heads * 4);
  l.counters_in = take(2 * kDecodeMaxCtas * 4);
  l.n_tiles = take(4);
  l.partial = take(static_cast<size_t>(2 * kDecodeMaxCtas * decode_piece_floats(c.head_dim)) * 4);
  const size_t tiles = max_row_tiles(c);
  l.first_tile = take(static_cast<size_t>(c.max_seqs) * 4);
  l.tiles = take(tiles * sizeof(KvRowTile));
  l.first_unit = take(tiles * 8);
  l.shares = take(kChunkMaxPairs * sizeof(KvShare));
  l.joins = take(kChunkMaxPairs * sizeof(KvJoin));
  l.chunk_partial = take(static_cast<size_t>(2 * kChunkMaxPairs * kChunkPieceFloats) * 4);
  l.total = o;
  return l;
}

int on_device(const moe_ffn_kv* kv) {
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) return MOE_FFN_ECUDA;
  return cur == kv->device || cudaSetDevice(kv->device) == cudaSuccess ? MOE_FFN_OK : MOE_FFN_ECUDA;
}

}  // namespace

extern "C" {

size_t moe_ffn_kv_workspace_bytes(const moe_ffn_kv_config* cfg) {
  if (!kv_config_ok(cfg)) return 0;
  return make_kv_layout(*cfg).total;
}

int moe_ffn_kv_init(moe_ffn_kv** out, const moe_ffn_kv_config* cfg, void* workspace, size_t workspace_bytes,
                    int device) {
  if (!out) return MOE_FFN_EINVAL;
  *out = nullptr;
  if (!kv_config_ok(cfg) || !workspace) return MOE_FFN_EINVAL;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return MOE_FFN_EALIGN;
  const KvLayout l = make_kv_layout(*cfg);
  if (workspace_bytes < l.total) return MOE_FFN_ETOOBIG;
  if (cudaSetDevice(device) != cudaSuccess) return MOE_FFN_ECUDA;
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return MOE_FFN_ECUDA;
  if (major != 10 || minor != 3) return MOE_FFN_EARCH;
  moe_ffn_kv* kv = new (std::nothrow) moe_ffn_kv();
  if (!kv) return MOE_FFN_ECUDA;
  kv->cfg = *cfg;
  kv->device = device;
  kv->num_sms = sms;
  kv->ws = static_cast<uint8_t*>(workspace);
  kv->ws_bytes = workspace_bytes;
  kv->status = reinterpret_cast<unsigned int*>(kv->ws + l.status);
  kv->counters = reinterpret_cast<int*>(kv->ws + l.counters);
  kv->counters_in = reinterpret_cast<int*>(kv->ws + l.counters_in);
  kv->partial = reinterpret_cast<float*>(kv->ws + l.partial);
  kv->list.first_tile = reinterpret_cast<int*>(kv->ws + l.first_tile);
  kv->list.tiles = reinterpret_cast<KvRowTile*>(kv->ws + l.tiles);
  kv->list.first_unit = reinterpret_cast<long long*>(kv->ws + l.first_unit);
  kv->list.n_tiles = reinterpret_cast<int*>(kv->ws + l.n_tiles);
  kv->list.shares = reinterpret_cast<KvShare*>(kv->ws + l.shares);
  kv->list.joins = reinterpret_cast<KvJoin*>(kv->ws + l.joins);
  kv->list.max_tiles = static_cast<int>(max_row_tiles(*cfg));
  kv->chunk_partial = reinterpret_cast<float*>(kv->ws + l.chunk_partial);
  // The workspace may be memory that work still queued on some stream writes: that ends before the control words
  // are cleared, and the clearing before any call.
  if (kv_decode_setup() != cudaSuccess || kv_chunk_setup(&kv->chunk_pairs) != cudaSuccess ||
      cudaDeviceSynchronize() != cudaSuccess || cudaMemset(kv->ws, 0, l.partial) != cudaSuccess ||
      cudaDeviceSynchronize() != cudaSuccess) {
    delete kv;
    return MOE_FFN_ECUDA;
  }
  *out = kv;
  return MOE_FFN_OK;
}

int moe_ffn_kv_write(moe_ffn_kv* kv, const moe_ffn_kv_cache* cache, const moe_ffn_kv_batch* batch,
                     const moe_ffn_kv_rows* k, const moe_ffn_kv_rows* v, void* stream) {
  KvBatch b;
  KvCache c;
  KvRows kr, vr;
  int rc = kv_arguments(kv, cache, batch, &b, &c);
  if (rc != MOE_FFN_OK) return rc > 0 ? MOE_FFN_OK : rc;
  if ((rc = kv_rows(k, &kr)) != MOE_FFN_OK || (rc = kv_rows(v, &vr)) != MOE_FFN_OK) return rc;
  if ((rc = on_device(kv)) != MOE_FFN_OK) return rc;
  return launch_kv_write(b, c, kr, vr, kv->status, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_FFN_OK
                                                                                                     : MOE_FFN_ECUDA;
}

int moe_ffn_kv_read(moe_ffn_kv* kv, const moe_ffn_kv_cache* cache, const moe_ffn_kv_batch* batch, void* k_out,
                    void* v_out, void* stream) {
  KvBatch b;
  KvCache c;
  int rc = kv_arguments(kv, cache, batch, &b, &c);
  if (rc != MOE_FFN_OK) return rc > 0 ? MOE_FFN_OK : rc;
  if (!k_out || !v_out) return MOE_FFN_EINVAL;
  if (off16(k_out) || off16(v_out)) return MOE_FFN_EALIGN;
  const size_t bytes = static_cast<size_t>(b.n_tokens) * c.kv_heads * c.head_dim * 2;
  if (meet(k_out, bytes, v_out, bytes) || meet(k_out, bytes, kv->ws, kv->ws_bytes) ||
      meet(v_out, bytes, kv->ws, kv->ws_bytes) || meets_cache(k_out, bytes, c) || meets_cache(v_out, bytes, c))
    return MOE_FFN_EINVAL;
  if ((rc = on_device(kv)) != MOE_FFN_OK) return rc;
  return launch_kv_read(b, c, static_cast<uint16_t*>(k_out), static_cast<uint16_t*>(v_out), kv->status,
                        static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_FFN_OK
             : MOE_FFN_ECUDA;
}

int moe_ffn_kv_attention(moe_ffn_kv* kv, const moe_ffn_kv_cache* cache, const moe_ffn_kv_batch* batch,
                         const moe_ffn_kv_rows* q, float scale, int window, int sinks, void* out, float* lse,
                         void* stream) {
  KvAttn a;
  int rc = kv_arguments(kv, cache, batch, &a.b, &a.c);
  if (rc < 0) return rc;
  if (!(scale > 0.0f) || !std::isfinite(scale) || window < 0 || sinks < 0) return MOE_FFN_EINVAL;
  if (rc > 0) return MOE_FFN_OK;
  if ((rc = kv_rows(q, &a.q)) != MOE_FFN_OK) return rc;
  if (!out) return MOE_FFN_EINVAL;
  if (off16(out) || off4(lse)) return MOE_FFN_EALIGN;
  const moe_ffn_kv_config& f = kv->cfg;
  const size_t rows = static_cast<size_t>(a.b.n_tokens) * f.q_heads, bytes = rows * f.head_dim * 2;
  const size_t q_bytes = kv_rows_bytes(a.q, a.b.n_tokens, f.q_heads, f.head_dim);
  if (meet(out, bytes, a.q.ptr, q_bytes) || meet(out, bytes, kv->ws, kv->ws_bytes) || meets_cache(out, bytes, a.c) ||
      (lse && (meet(lse, rows * 4, out, bytes) || meet(lse, rows * 4, kv->ws, kv->ws_bytes) ||
               meet(lse, rows * 4, a.q.ptr, q_bytes) || meets_cache(lse, rows * 4, a.c))))
    return MOE_FFN_EINVAL;
  a.group = f.q_heads / f.kv_heads;
  a.q_heads = f.q_heads;
  a.scale = scale;
  a.window = window;
  a.sinks = sinks;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = kv->status;
  a.counters = kv->counters;
  a.counters_in = kv->counters_in;
  a.partial = kv->partial;
  a.list = kv->list;
  // One cost per format, of 2 to 6 tiles. Prompts of 1500 to 4100 tokens of width 256 take 196 us in bf16 with 3
  // (206 with 2, 202 with 4, 206 with 5); in e4m3, where the queries are split on the way, 279 with 4 (302
  // with 3, 275 with 5, 280 with 6). Of the other widths in e4m3, 128 takes 210 with 4 and 216 with 5, 512 672 and
  // 651, and a mixed batch 130 and 135 (width 128), 196 and 186 (512).
  a.item_cost = a.c.e4m3 ? 4 : 3;
  a.chunk_partial = kv->chunk_partial;
  if ((rc = on_device(kv)) != MOE_FFN_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int ctas = 2 * kv->num_sms < kDecodeMaxCtas ? 2 * kv->num_sms : kDecodeMaxCtas;
  // A single token of up to kDecodeHeads heads per kv head fills an item of the decode kernel; the chunk
  // kernel computes tiles of 256 rows of which it would fill `group`. Single tokens through the one and the other:
  // one short sequence 14 and 20 us, 64 e4m3 sequences (width 512) 78 and 226, 256 windows 217 and 360,
  // one long bf16 sequence 96 and 124.
  const cudaError_t e = a.b.max_new <= 1 && a.group <= kDecodeHeads ? launch_kv_decode(a, ctas, s)
                                                                    : launch_kv_chunk(a, kv->chunk_pairs, s);
  return e == cudaSuccess ? MOE_FFN_OK : MOE_FFN_ECUDA;
}

int moe_ffn_kv_device_status(moe_ffn_kv* kv, void* stream, uint32_t* word) {
  if (!kv) return MOE_FFN_EINVAL;
  if (cudaSetDevice(kv->device) != cudaSuccess) return MOE_FFN_ECUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return MOE_FFN_ECUDA;
  uint32_t v = 0;
  if (cudaMemcpy(&v, kv->status, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return MOE_FFN_ECUDA;
  // (Done before this returns: a clearing that lands later could take the next call's report with it.)
  if (v != 0 && (cudaMemsetAsync(kv->status, 0, 4, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess))
    return MOE_FFN_ECUDA;
  if (word) *word = v;
  return v ? MOE_FFN_EDEVICE : MOE_FFN_OK;
}

void moe_ffn_kv_destroy(moe_ffn_kv* kv) { delete kv; }

}  // extern "C"
