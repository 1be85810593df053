// kv_decode.cu — attention of single tokens (one new token per sequence, at most eight query heads per
// kv head) over the paged cache.
//
// With a row or a few per kv head, every cached byte meets a handful of multiplications: HBM bounds the
// kernel, and all it has to do is keep loads in flight and let no key wait for another CTA's length.
//
// Work. An item is one sequence's kv head; its visible keys fall into tiles of KT positions. The tiles of
// all items, one after the other, are shared out evenly over the CTAs, two to an SM, so ragged lengths
// and single long sequences alike end together. An item that several CTAs share is joined by the one
// that finishes it last, from fp32 pieces (unnormalised output, maximum, sum) in the order of the tiles:
// whichever CTA that is, the sums are the same.
//
// A CTA: warp 4 loads, TMA boxes of one page's rows (128-byte swizzle) into a ring of units, one unit the
// keys or the values of a tile; warps 0..3 compute with mma.sync, the keys as the rows of the products
// (S^T = K Q^T, then O^T = V^T P^T), so the eight heads are the narrow side and nothing is padded to
// 16 query rows. Each warp takes S of its own keys (of half the width where a tile has only 32 or the
// width is 512), all exchange S through shared memory, and each forms all of P in the layout the second
// product reads, and multiplies its own quarter of V's width: one barrier per tile, no output to be
// joined between warps, and P^T needs no transpose.
//
// Softmax: one pass, running maximum m and sum l in fp32 and base 2; P is rounded to bf16 for the product
// with V (half a step is 2^-8 of each weight; l adds the unrounded ones).
//
// e4m3: the keys meet the queries as e4m3, each query value as the sum of two e4m3 numbers (its leading
// and next four bits; the row is scaled by a power of two to at most 256, so what two numbers lose lies
// 2^-18 below the row's largest magnitude). The key's scale multiplies S, the value's scale P. Value codes
// become bf16 by moving their bits and a multiplication by 2^120, exactly.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "kv.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kComputeWarps = 4;
constexpr int kThreads = (kComputeWarps + 1) * 32;

template <int D, bool E4M3>
struct Dec {
  static constexpr int kRow = D * (E4M3 ? 1 : 2);                    // bytes of a cached row
  // Positions per tile: a unit of 32 KB (16 KB for e4m3 rows of 128), three of them (six) per CTA, so
  // that 64 KB and more per CTA are on their way while a tile is computed.
  static constexpr int KT = E4M3 ? (D == 512 ? 64 : 128) : 16384 / D;
  static constexpr int KG = D == 512 ? 2 : 4;                        // warps along the keys, for S
  static constexpr int DS = kComputeWarps / KG;                      // warps along the width, for S
  static constexpr int MT = KT / (16 * KG);                          // 16-key blocks per warp, for S
  static constexpr int kUnit = KT * kRow;
  static constexpr int kUnits = 98304 / kUnit;
  static constexpr int kSteps = kRow / 32 / DS;                      // 32-byte steps of a key row per warp
  static constexpr int kQRegs = kSteps * 2 * (E4M3 ? 2 : 1);
  static constexpr int VT = D / 64;                                  // 16-wide blocks of V per warp
  static constexpr int SP = KT + 4;                                  // row pitch of S, in floats
  static constexpr int kSBytes = 2 * DS * kDecodeHeads * SP * 4;
  static constexpr int kScaleBytes = E4M3 ? kUnits * KT * 4 : 0;
  static constexpr int kSmem = 1024 + kUnits * kUnit + kSBytes + kScaleBytes + 256;
  static_assert(kSmem <= 115712, "two CTAs to an SM");
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Two e4m3 codes in the high bytes of w's halves, as bf16: sign, exponent and fraction move to bf16's
// fields, where the exponent reads 120 too low.
__device__ __forceinline__ uint32_t widen_e4m3(uint32_t w) {
  const uint32_t t = ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
  __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&t);
  const uint32_t f = 0x7b807b80u;  // 2^120
  v = __hmul2(v, *reinterpret_cast<const __nv_bfloat162*>(&f));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The leading (or, with the leading part taken off, the next) e4m3 parts of four values.
__device__ __forceinline__ uint32_t e4m3_part(float (&x)[4]) {
  uint32_t codes = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * j], x[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
    codes |= static_cast<uint32_t>(c) << (16 * j);
    const float2 back = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
    x[2 * j] -= back.x;
    x[2 * j + 1] -= back.y;
  }
  return codes;
}

// The four computing warps.
__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

constexpr int kJoin = 24;  // pieces joined at once, at most 32

// Where a CTA's share of the tiles begins, and how a sequence's tiles lie.
struct SeqTiles {
  int row;     // the token's row
  KvSpan span;
  int front;   // tiles of the sinks, before the window's
  int skip;    // tiles between the two
  int count;
};

template <int KT>
__device__ __forceinline__ SeqTiles seq_tiles(const KvAttn& a, int seq) {
  const KvSeq s = kv_sequence(a.b, a.c, seq, a.status);
  SeqTiles t;
  t.row = s.row0;
  t.span = kv_span(s.n > 0 ? s.len - 1 : -1, a.window, a.sinks);
  t.count = 0;
  t.front = t.skip = 0;
  if (t.span.p < 0) return t;
  const int first = t.span.lo / KT;
  t.front = min((t.span.sinks + KT - 1) / KT, first);
  t.skip = first - t.front;
  t.count = t.span.p / KT + 1 - t.skip;
  return t;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 2)
    kv_decode_kernel(const KvAttn a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using C = Dec<D, E4M3>;
  constexpr int KT = C::KT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* s_buf = reinterpret_cast<float*>(ring + C::kUnits * C::kUnit);
  float* scale_buf = s_buf + C::kSBytes / 4;
  uint64_t* full = reinterpret_cast<uint64_t*>(scale_buf + C::kScaleBytes / 4);
  uint64_t* empty = full + C::kUnits;
  __shared__ volatile int abort_flag;
  __shared__ int s_last;
  __shared__ float s_weight[kDecodeHeads][32], s_join[kDecodeHeads][2];
  __shared__ long long s_sum[kThreads / 32], s_total, s_before;
  __shared__ int s_seq;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    abort_flag = 0;
    for (int u = 0; u < C::kUnits; ++u) {
      mbar_init(&full[u], 1);
      mbar_init(&empty[u], kComputeWarps);
    }
    fence_barrier_init();
  }
  if (warp == kComputeWarps && lane == 0) {
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  pdl_wait();
  pdl_launch_dependents();

  // The tiles of all sequences, and the sequence this CTA's share begins in.
  const int heads = a.c.kv_heads, n_seqs = a.b.n_seqs;
  auto block_sum = [&](long long v) {  // inclusive sum over the threads; s_total: over the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += up;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = v;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp; ++w) before += s_sum[w];
    if (tid == kThreads - 1) s_total = before + v;
    __syncthreads();
    return before + v;
  };
  int own = 0;  // tiles of sequence tid
  long long mine = 0;
  for (int b = tid; b < n_seqs; b += kThreads) {
    const SeqTiles t = seq_tiles<KT>(a, b);
    if (b == tid) own = t.count;
    mine += t.count;
    if (t.span.p < 0 && b % gridDim.x == blockIdx.x && t.row < a.b.n_tokens && a.b.cu_q[b + 1] > t.row) {
      // A token that sees nothing.
      for (int h = 0; h < a.q_heads; ++h) {
        const long long to = static_cast<long long>(t.row) * a.q_heads + h;
        for (int i = 0; i < D; i += 8) *reinterpret_cast<uint4*>(a.out + to * D + i) = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse) a.lse[to] = -INFINITY;
      }
    }
  }
  {  // Rows of no sequence.
    const int used = n_seqs > 0 ? min(max(a.b.cu_q[n_seqs], 0), a.b.n_tokens) : 0;
    const long long n = static_cast<long long>(a.b.n_tokens - used) * a.q_heads;
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + tid; i < n; i += static_cast<long long>(gridDim.x) * kThreads) {
      const long long to = static_cast<long long>(used) * a.q_heads + i;
      for (int j = 0; j < D; j += 8) *reinterpret_cast<uint4*>(a.out + to * D + j) = make_uint4(0u, 0u, 0u, 0u);
      if (a.lse) a.lse[to] = -INFINITY;
    }
  }
  long long upto = block_sum(mine);
  const long long total = s_total * heads;
  // A share is at least two tiles: below that the joining of pieces costs more than the tiles.
  const long long ctas = min(static_cast<long long>(gridDim.x), (total + 1) / 2);
  if (blockIdx.x >= ctas) return;
  const long long begin = blockIdx.x * total / ctas, end = (blockIdx.x + 1) * total / ctas;
  for (int base = 0;; base += kThreads) {
    // One block of sequences after the other; the first block's counts are at hand.
    long long before = 0;
    if (base == 0 && n_seqs <= kThreads) {
      before = 0;
    } else {
      if (base > 0) own = base + tid < n_seqs ? seq_tiles<KT>(a, base + tid).count : 0;
      if (tid == 0 && base == 0) s_before = 0;
      upto = block_sum(own);
      before = s_before;
    }
    const long long lo = (before + upto - own) * heads, hi = (before + upto) * heads;
    if (begin >= lo && begin < hi) {
      s_seq = base + tid;
      s_sum[0] = lo;
    }
    const bool here = __syncthreads_or(begin >= lo && begin < hi);
    if (here || base + kThreads >= n_seqs) break;
    if (tid == 0) s_before = before + s_total;
    __syncthreads();
  }
  int seq = s_seq;
  const long long seq_start = s_sum[0];
  SeqTiles t = seq_tiles<KT>(a, seq);
  int head = static_cast<int>((begin - seq_start) / t.count);
  int i0 = static_cast<int>((begin - seq_start) % t.count);

  const int rows_log2 = min(a.c.page_log2, KT == 128 ? 7 : KT == 64 ? 6 : 5);
  const int R = 1 << rows_log2;  // rows of a box
  int unit = 0;
  uint32_t phase = 0;
  auto next_unit = [&] {
    if (++unit == C::kUnits) {
      unit = 0;
      phase ^= 1;
    }
  };
  // Goes on to the next item, of the same sequence or of the next that has tiles.
  auto next_item = [&] {
    i0 = 0;
    if (++head < heads) return;
    head = 0;
    do t = seq_tiles<KT>(a, ++seq);
    while (t.count == 0);
  };

  if (warp == kComputeWarps) {
    // ---------------------------------------------------------------- loads
    const uint64_t policy = policy_evict_first();
    bool alive = true;
    int issued = 0;
    for (long long pos = begin; pos < end && alive;) {
      const int n = static_cast<int>(min(static_cast<long long>(t.count - i0), end - pos));
      for (int i = i0; i < i0 + n && alive; ++i) {
        const int tile = i < t.front ? i : i + t.skip;
        const int p0 = tile * KT + (lane << rows_log2);  // the first position of this lane's page part
        const bool need = lane < (KT >> rows_log2) && p0 <= t.span.p && (p0 + R - 1 >= t.span.lo || p0 < t.span.sinks);
        int page = -1;
        if (need) page = kv_page(a.b, a.c, seq, p0 >> a.c.page_log2, a.status);
        const int row = page < 0 ? 0
                                 : ((page * heads + head) << a.c.page_log2) + (p0 & ((1 << a.c.page_log2) - 1));
        const unsigned who = __ballot_sync(0xffffffffu, page >= 0);
        const uint32_t bytes = __popc(who) * static_cast<uint32_t>(R * (C::kRow + (E4M3 ? 4 : 0)));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (issued >= C::kUnits) {
            bool ok = true;
            if (lane == 0) ok = mbar_wait_bounded(&empty[unit], phase ^ 1, &abort_flag, a.status, kStatusWaitEmpty);
            alive = alive && __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          }
          if (!alive) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[unit], bytes);
          __syncwarp();
          if (page >= 0) {
            uint8_t* dst = ring + unit * C::kUnit + (lane << rows_log2) * C::kRow;
            asm volatile(
                "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
                " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
                "l"(reinterpret_cast<uint64_t>(kv ? &map_v : &map_k)), "r"(0), "r"(row), "r"(0),
                "r"(smem_u32(&full[unit])), "l"(policy)
                : "memory");
            if constexpr (E4M3) {
              asm volatile(
                  "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                      smem_u32(scale_buf + unit * KT + (lane << rows_log2))),
                  "l"(reinterpret_cast<uint64_t>((kv ? a.c.v_scale : a.c.k_scale) + row)), "r"(R * 4),
                  "r"(smem_u32(&full[unit]))
                  : "memory");
            }
          }
          ++issued;
          next_unit();
        }
      }
      pos += n;
      if (pos < end) next_item();
    }
    if (!alive && lane == 0) {
      // Given up: the copies on their way land before the CTA's shared memory goes.
      for (int u = 0; u < min(issued, C::kUnits); ++u) {
        if (unit == 0) {
          unit = C::kUnits;
          phase ^= 1;
        }
        --unit;
        mbar_wait_timeout(&full[unit], phase, 1000000ull, a.status);
      }
    }
    return;
  }

  // ------------------------------------------------------------------ compute
  const int kg = warp % C::KG, ds = warp / C::KG;
  const int c4 = lane & 3, r8 = lane >> 2;
  int flip = 0;
  for (long long pos = begin; pos < end;) {
    const int n = static_cast<int>(min(static_cast<long long>(t.count - i0), end - pos));
    // The queries as the second operand of S^T = K Q^T: lane holds head r8.
    uint32_t q[C::kQRegs];
    float qs[2];  // what S of heads 2 c4 and 2 c4 + 1 is multiplied by
    {
      const uint16_t* qp = a.q.ptr + t.row * a.q.token_stride + (head * a.group + min(r8, a.group - 1)) * a.q.head_stride +
                           ds * (D / C::DS);
      const float in_log2 = a.scale * 1.44269504f;
      if constexpr (!E4M3) {
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) {
          q[2 * s] = *reinterpret_cast<const uint32_t*>(qp + 16 * s + 2 * c4);
          q[2 * s + 1] = *reinterpret_cast<const uint32_t*>(qp + 16 * s + 8 + 2 * c4);
        }
        qs[0] = qs[1] = in_log2;
      } else {
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < 2 * C::kSteps; ++s) {
          const uint2 w = *reinterpret_cast<const uint2*>(qp + 16 * s + 4 * c4);
          top = max(top, max(max(w.x << 16 & 0x7fffffffu, w.x & 0x7fffffffu), max(w.y << 16 & 0x7fffffffu, w.y & 0x7fffffffu)));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // A power of two that brings the largest magnitude into [128, 256); NaN for a row with one.
        const int e = static_cast<int>(top >> 23);
        const float up = e == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float(static_cast<uint32_t>(min(261 - e, 254)) << 23);
        const float down = in_log2 * (e == 255 ? up : __uint_as_float(static_cast<uint32_t>(max(e - 7, 0)) << 23));
        const float undo = e < 8 ? in_log2 / up : down;
#pragma unroll
        for (int s = 0; s < 2 * C::kSteps; ++s) {
          const uint2 w = *reinterpret_cast<const uint2*>(qp + 16 * s + 4 * c4);
          float x[4] = {__uint_as_float(w.x << 16) * up, __uint_as_float(w.x & 0xffff0000u) * up,
                        __uint_as_float(w.y << 16) * up, __uint_as_float(w.y & 0xffff0000u) * up};
          q[s] = e4m3_part(x);
          q[2 * C::kSteps + s] = e4m3_part(x);
        }
        qs[0] = __shfl_sync(0xffffffffu, undo, 8 * c4);
        qs[1] = __shfl_sync(0xffffffffu, undo, 8 * c4 + 4);
      }
    }
    float o[C::VT][4];
#pragma unroll
    for (int v = 0; v < C::VT; ++v) o[v][0] = o[v][1] = o[v][2] = o[v][3] = 0.0f;
    float m = -INFINITY, l = 0.0f;  // of head r8; l of this lane's keys

    for (int i = i0; i < i0 + n; ++i) {
      const int tile = i < t.front ? i : i + t.skip;
      const bool masked = !(tile * KT + KT - 1 <= t.span.p &&
                            (tile * KT >= t.span.lo || tile * KT + KT <= t.span.sinks));
      // S^T of this warp's keys.
      float s[C::MT][2][4];
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[mt][0][x] = s[mt][1][x] = 0.0f;
      mbar_wait_bounded(&full[unit], phase, &abort_flag, a.status, kStatusWaitFull);
      {
        const uint32_t base = smem_u32(ring + unit * C::kUnit);
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
          const int key = (kg * C::MT + mt) * 16 + (lane & 15);
          const uint32_t row = base + (key >> rows_log2) * (C::kRow << rows_log2) + (key & (R - 1)) * 128;
          const uint32_t swz = (key & 7) << 4;
#pragma unroll
          for (int st = 0; st < C::kSteps; ++st) {
            const uint32_t x = ds * (C::kRow / C::DS) + st * 32;
            uint32_t f[4];
            ldsm4(row + ((x >> 7) << (7 + rows_log2)) + (((x & 127) + ((lane >> 4) << 4)) ^ swz), f);
            if constexpr (E4M3) {
              mma_e4m3(s[mt][0], f, q[2 * st], q[2 * st + 1]);
              mma_e4m3(s[mt][1], f, q[2 * C::kSteps + 2 * st], q[2 * C::kSteps + 2 * st + 1]);
            } else {
              mma_bf16(s[mt][st & 1], f, q[2 * st], q[2 * st + 1]);
            }
          }
        }
      }
      float* sb = s_buf + flip * (C::DS * kDecodeHeads * C::SP);
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt) {
        const int key = (kg * C::MT + mt) * 16 + r8;
        float f0 = 1.0f, f1 = 1.0f;
        if constexpr (E4M3) {
          f0 = scale_buf[unit * KT + key];
          f1 = scale_buf[unit * KT + key + 8];
        }
        float* to = sb + (ds * kDecodeHeads + 2 * c4) * C::SP + key;
        to[0] = (s[mt][0][0] + s[mt][1][0]) * (qs[0] * f0);
        to[C::SP] = (s[mt][0][1] + s[mt][1][1]) * (qs[1] * f0);
        to[8] = (s[mt][0][2] + s[mt][1][2]) * (qs[0] * f1);
        to[C::SP + 8] = (s[mt][0][3] + s[mt][1][3]) * (qs[1] * f1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[unit]);
      next_unit();
      compute_sync();

      // P of every key, for head r8: this lane the keys 16 k + 2 c4 + {0, 1, 8, 9}.
      float p[KT / 16][4];
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < KT / 16; ++k) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float* from = sb + r8 * C::SP + 16 * k + 8 * half + 2 * c4;
          float2 v = *reinterpret_cast<const float2*>(from);
          if constexpr (C::DS == 2) {
            const float2 w = *reinterpret_cast<const float2*>(from + kDecodeHeads * C::SP);
            v.x += w.x;
            v.y += w.y;
          }
          if (masked) {
            const int at = tile * KT + 16 * k + 8 * half + 2 * c4;
            if (at > t.span.p || (at < t.span.lo && at >= t.span.sinks)) v.x = -INFINITY;
            if (at + 1 > t.span.p || (at + 1 < t.span.lo && at + 1 >= t.span.sinks)) v.y = -INFINITY;
          }
          p[k][2 * half] = v.x;
          p[k][2 * half + 1] = v.y;
          mx = fmaxf(mx, fmaxf(v.x, v.y));
        }
      }
      flip ^= 1;
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // The maximum drops a NaN, and stays -inf where no score is a number yet; 0 stands in for it.
      const float m1 = fmaxf(m, mx), base = m1 == -INFINITY ? 0.0f : m1;
      const float f = exp2_approx(m - base);
      m = m1;
      l *= f;
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < KT / 16; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          p[k][x] = exp2_approx(p[k][x] - base);
          sum += p[k][x];
        }
      l += sum;
      if (__any_sync(0xffffffffu, f != 1.0f)) {
        const float f0 = __shfl_sync(0xffffffffu, f, 8 * c4), f1 = __shfl_sync(0xffffffffu, f, 8 * c4 + 4);
#pragma unroll
        for (int v = 0; v < C::VT; ++v) {
          o[v][0] *= f0;
          o[v][1] *= f1;
          o[v][2] *= f0;
          o[v][3] *= f1;
        }
      }

      // O^T += V^T P^T over this warp's quarter of the width.
      mbar_wait_bounded(&full[unit], phase, &abort_flag, a.status, kStatusWaitFull);
      const uint32_t vbase = smem_u32(ring + unit * C::kUnit);
#pragma unroll
      for (int k = 0; k < KT / 16; ++k) {
        uint32_t b0, b1, keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if constexpr (E4M3) {
          const float* vs = scale_buf + unit * KT + 16 * k + 2 * c4;
          // Hidden keys: a weight of 0 whatever the scale that lies there.
          float w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) w[x] = p[k][x] == 0.0f ? 0.0f : p[k][x] * vs[(x & 1) + 8 * (x >> 1)];
          b0 = pack_bf16(w[0], w[1]);
          b1 = pack_bf16(w[2], w[3]);
        } else {
          b0 = pack_bf16(p[k][0], p[k][1]);
          b1 = pack_bf16(p[k][2], p[k][3]);
          if (masked) {
            // Hidden values may be anything, NaN included: they become 0.
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int at = tile * KT + 16 * k + 2 * c4 + (x & 1) + 8 * (x >> 1);
              const uint32_t gone = at > t.span.p || (at < t.span.lo && at >= t.span.sinks) ? 0xffffu << (16 * (x & 1)) : 0u;
              if (x < 2) keep0 &= ~gone;
              else keep1 &= ~gone;
            }
          }
        }
        const int key = 16 * k + (lane & 7) + (E4M3 ? (lane & 8) : (lane & 16) >> 1);
        const uint32_t row = vbase + (key >> rows_log2) * (C::kRow << rows_log2) + (key & (R - 1)) * 128;
        const uint32_t swz = (key & 7) << 4;
        if constexpr (E4M3) {
          // A 16-byte piece is 16 dimensions; as 16-bit pairs the transposed load gives a lane the
          // dimensions 2 r8 and 2 r8 + 1, which become the rows r8 and r8 + 8 of the block.
#pragma unroll
          for (int v = 0; v < C::VT; v += 2) {
            const uint32_t x = warp * (D / 4) + v * 16;
            uint32_t w[4];
            ldsm4_trans(row + ((x >> 7) << (7 + rows_log2)) + (((x & 127) + (lane & 16)) ^ swz), w);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t fr[4] = {widen_e4m3(w[2 * y] << 8), widen_e4m3(w[2 * y]), widen_e4m3(w[2 * y + 1] << 8),
                                      widen_e4m3(w[2 * y + 1])};
              mma_bf16(o[v + y], fr, b0, b1);
            }
          }
        } else {
#pragma unroll
          for (int v = 0; v < C::VT; ++v) {
            const uint32_t x = (warp * (D / 4) + v * 16) * 2;
            uint32_t w[4];
            ldsm4_trans(row + ((x >> 7) << (7 + rows_log2)) + (((x & 127) + ((lane & 8) << 1)) ^ swz), w);
            if (masked) {
              w[0] &= keep0;
              w[1] &= keep0;
              w[2] &= keep1;
              w[3] &= keep1;
            }
            mma_bf16(o[v], w, b0, b1);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[unit]);
      next_unit();
    }

    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const long long item_start = pos - i0;
    const long long to = static_cast<long long>(t.row) * a.q_heads + head * a.group;  // the first head's output row
    const int h0 = 2 * c4, h1 = h0 + 1;
    // The dimension of o[v][0]; o[v][2] is `apart` further.
    constexpr int apart = E4M3 ? 1 : 8;
    const int dim0 = warp * (D / 4) + (E4M3 ? 2 * r8 : r8);
    if (i0 == 0 && n == t.count) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const float f0 = __shfl_sync(0xffffffffu, inv, 4 * h0), f1 = __shfl_sync(0xffffffffu, inv, 4 * h1);
#pragma unroll
      for (int v = 0; v < C::VT; ++v)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int h = x & 1 ? h1 : h0;
          if (h < a.group)
            a.out[(to + h) * D + dim0 + v * 16 + (x >> 1) * apart] = f32_to_bf16_rn(o[v][x] * (x & 1 ? f1 : f0));
        }
      if (a.lse && warp == 0 && c4 == 0 && r8 < a.group)
        a.lse[to + r8] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147181f;
    } else {
      // A piece. Its place is this CTA's first if the item began before the CTA's share or with it, as
      // it did for all of the item's CTAs but its first.
      const int first = static_cast<int>(((item_start + 1) * ctas - 1) / total);
      const int count = static_cast<int>(((item_start + t.count) * ctas - 1) / total) - first + 1;
      const int first_place = 2 * first + (first * total / ctas >= item_start ? 0 : 1);
      auto place = [&](int x) { return x == 0 ? first_place : 2 * (first + x); };  // of the item's piece x
      constexpr long long piece_floats = decode_piece_floats(D);
      const int me = static_cast<int>(blockIdx.x) - first;
      {
        float* piece = a.partial + place(me) * piece_floats;
#pragma unroll
        for (int v = 0; v < C::VT; ++v)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int h = x & 1 ? h1 : h0;
            if (h < a.group) piece[h * D + dim0 + v * 16 + (x >> 1) * apart] = o[v][x];
          }
        if (warp == 0 && c4 == 0) {
          piece[kDecodeHeads * D + r8] = m;
          piece[kDecodeHeads * D + kDecodeHeads + r8] = l;
        }
      }
      // Up to kJoin pieces are joined at once; more in groups first, by each group's last CTA into the
      // group's first piece, and then the groups: 152 pieces in one go were 25 us at the end of a
      // long sequence's 80.
      const int span = count <= kJoin ? count : static_cast<int>(ceilf(sqrtf(static_cast<float>(count))));
      const int groups = (count + span - 1) / span;
      int from = me / span * span, n_in = min(span, count - from), apart_in = 1;
      int* counter = groups == 1 ? a.counters + static_cast<long long>(seq) * heads + head : a.counters_in + place(from);
      for (;;) {
        __threadfence();
        compute_sync();
        if (tid == 0) {
          const int done = atomicAdd(counter, 1);
          s_last = done == n_in - 1;
          if (done == n_in - 1) *counter = 0;
        }
        compute_sync();
        if (!s_last) break;
        __threadfence();
        const bool final = apart_in > 1 || groups == 1;
        // The pieces' weights, a warp for every other head, a lane for each piece.
        for (int h = warp; h < a.group; h += kComputeWarps) {
          const float* at = a.partial + place(from + min(lane, n_in - 1) * apart_in) * piece_floats + kDecodeHeads * D + h;
          const float pm = lane < n_in ? __ldcg(at) : -INFINITY;
          float top = pm;
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          const float w = lane < n_in ? exp2_approx(pm - (top == -INFINITY ? 0.0f : top)) : 0.0f;
          float sum = lane < n_in ? w * __ldcg(at + kDecodeHeads) : 0.0f;
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          s_weight[h][lane] = w;
          if (lane == 0) {
            s_join[h][0] = top;
            s_join[h][1] = sum;
          }
        }
        compute_sync();
        constexpr int kE = kDecodeHeads * D / 4 / (kComputeWarps * 32);
        float4 acc[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
        for (int x = 0; x < n_in; ++x) {
          const float* at = a.partial + place(from + x * apart_in) * piece_floats;
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            const int i = tid + e * kComputeWarps * 32, h = i / (D / 4);
            if (h >= a.group) continue;
            const float4 y = __ldcg(reinterpret_cast<const float4*>(at + 4 * i));
            const float w = s_weight[h][x];
            acc[e].x = fmaf(w, y.x, acc[e].x);
            acc[e].y = fmaf(w, y.y, acc[e].y);
            acc[e].z = fmaf(w, y.z, acc[e].z);
            acc[e].w = fmaf(w, y.w, acc[e].w);
          }
        }
        float* group_piece = a.partial + place(from) * piece_floats;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const int i = tid + e * kComputeWarps * 32, h = i / (D / 4);
          if (h >= a.group) continue;
          if (final) {
            const float sum = s_join[h][1], inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            *reinterpret_cast<uint2*>(a.out + to * D + 4 * i) = make_uint2(
                pack_bf16(acc[e].x * inv, acc[e].y * inv), pack_bf16(acc[e].z * inv, acc[e].w * inv));
          } else {
            *reinterpret_cast<float4*>(group_piece + 4 * i) = acc[e];
          }
        }
        if (tid < a.group) {
          const float top = s_join[tid][0], sum = s_join[tid][1];
          if (!final) {
            group_piece[kDecodeHeads * D + tid] = top;
            group_piece[kDecodeHeads * D + kDecodeHeads + tid] = sum;
          } else if (a.lse) {
            a.lse[to + tid] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.693147181f;
          }
        }
        compute_sync();
        if (final) break;
        counter = a.counters + static_cast<long long>(seq) * heads + head;
        from = 0;
        n_in = groups;
        apart_in = span;
      }
    }
    pos += n;
    if (pos < end) next_item();
  }
}

template <int D, bool E4M3>
cudaError_t launch(const KvAttn& a, int ctas, cudaStream_t s) {
  using C = Dec<D, E4M3>;
  CUtensorMap mk, mv;
  const uint64_t rows = (static_cast<uint64_t>(a.c.n_pages) * a.c.kv_heads) << a.c.page_log2;
  const uint32_t box = (1 << a.c.page_log2) < C::KT ? 1 << a.c.page_log2 : C::KT;
  if (!encode_row_chunks(&mk, a.c.k, rows, C::kRow, box, C::kRow / 128) ||
      !encode_row_chunks(&mv, a.c.v, rows, C::kRow, box, C::kRow / 128))
    return cudaErrorInvalidValue;
  return launch_pdl(kv_decode_kernel<D, E4M3>, dim3(ctas), dim3(kThreads), C::kSmem, s, a, mk, mv);
}

template <int D, bool E4M3>
cudaError_t setup() {
  return cudaFuncSetAttribute(kv_decode_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Dec<D, E4M3>::kSmem);
}

}  // namespace

cudaError_t kv_decode_setup() {
  cudaError_t e = setup<128, false>();
  if (e == cudaSuccess) e = setup<128, true>();
  if (e == cudaSuccess) e = setup<256, false>();
  if (e == cudaSuccess) e = setup<256, true>();
  if (e == cudaSuccess) e = setup<512, false>();
  if (e == cudaSuccess) e = setup<512, true>();
  return e;
}

cudaError_t launch_kv_decode(const KvAttn& a, int ctas, cudaStream_t s) {
  switch (a.c.head_dim * 2 + a.c.e4m3) {
    case 256: return launch<128, false>(a, ctas, s);
    case 257: return launch<128, true>(a, ctas, s);
    case 512: return launch<256, false>(a, ctas, s);
    case 513: return launch<256, true>(a, ctas, s);
    case 1024: return launch<512, false>(a, ctas, s);
    default: return launch<512, true>(a, ctas, s);
  }
}

}  // namespace moe
