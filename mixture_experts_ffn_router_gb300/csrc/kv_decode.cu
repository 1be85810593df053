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
// A CTA: warp 8 loads, TMA boxes of one page's rows (128-byte swizzle) into a ring of units, one unit the
// keys or the values of a tile; warps 0..7 compute with mma.sync, the keys as the rows of the products
// (S^T = K Q^T, then O^T = V^T P^T), so the eight heads are the narrow side and nothing is padded to
// 16 query rows. For S the tile's keys are shared out over the warps, 16 to a warp; where a tile has
// fewer than 128, several warps take a part of the width each and add their S in shared memory. P goes
// through shared memory to all warps, each of which multiplies its own eighth of V's width: no output
// is joined between warps.
//
// Softmax: one pass in base 2 (M. Milakov and N. Gimelshein, "Online normalizer calculation for softmax", 2018).
// The weights are exp2(s - M) with a reference M that all warps share and
// that moves (to the maximum so far, with the outputs and sums rescaled) only when a score passes it
// by more than 8: a tile then costs one barrier, which also tells every warp whether a score did.
// Weights are so at most 2^8, kept in fp32 for the sum l, and rounded to 16 bits for the product with V.
//
// e4m3: codes are exact in fp16, so both products run in fp16. A row of queries is scaled by a power of
// two to at most 2^15, where fp16 holds all of bf16's bits down to 2^-29 below the row's largest
// magnitude; the key's scale multiplies S. The weights carry the value's scale in their exponent,
// exp2(s + log2(scale) - R) with a reference R of their own that keeps the largest between 2^7 and 2^15:
// fp16's half step (2^-11) holds down to 2^-21 below that, and what is lost under it is at most 2^-32 of
// the largest per key. (mma.sync on e4m3 itself, with queries split in two e4m3 parts, was slower: 883 us
// against 772 for 64 sequences of 16384 tokens, 8 heads of width 256.)
//
// Measured: 64 sequences of 16384 tokens, beside the 6.70 TB/s of a copy: bf16 7.1, 7.2 and 7.0 TB/s (8 heads of
// width 128, 8 of 256, 2 of 512); e4m3 6.7, 6.8 and 6.5 (there a tile's chain of widened products, weights and
// barriers is as long as its loads, with 42% of the issue slots busy). A call takes about 6 us
// beside its loads: 3 to find its work and load its queries, the rest to join pieces.
#include "kv_mma.cuh"

namespace moe {

namespace {

constexpr int kThreads = (kComputeWarps + 1) * 32;

template <int D, bool E4M3>
struct Dec {
  static constexpr int kRow = D * (E4M3 ? 1 : 2);                    // bytes of a cached row
  // Positions per tile: a unit of 32 KB (16 KB for e4m3 rows of 128), three of them (six) per CTA, so
  // that 64 KB and more per CTA are on their way while a tile is computed.
  static constexpr int KT = E4M3 ? (D == 512 ? 64 : 128) : 16384 / D;
  static constexpr int KG = KT / 16 < kComputeWarps ? KT / 16 : kComputeWarps;  // warps along the keys, for S
  static constexpr int DS = kComputeWarps / KG;                      // warps along the width, for S
  static constexpr int kUnit = KT * kRow;
  static constexpr int kUnits = 98304 / kUnit;
  static constexpr int kSteps = kRow / 32 / DS;                      // 32-byte steps of a key row per warp
  static constexpr int kQRegs = D / DS / 8;
  static constexpr int VT = D / (16 * kComputeWarps);                // 16-wide blocks of V per warp
  // Of the steps of 32 keys through V, those unrolled. A CTA's two warps per scheduler execute the tile
  // in step and wait for its instructions: 64 sequences of 16384 e4m3 tokens take 333 us with 1 and 419 with
  // 2 at width 512, 637 and 640 at 256; at 128, whose steps are short, 337 with 1 and 324 with all 4.
  static constexpr int kVUnroll = D == 128 ? 4 : 1;
  static constexpr int SP = KT + 4;                                  // row pitch of S, in floats
  static constexpr int PP = KT + 8;                                  // row pitch of P, in 16-bit values
  static constexpr int kSBytes = DS > 1 ? DS * kDecodeHeads * SP * 4 : 0;
  static constexpr int kPBytes = 2 * kDecodeHeads * PP * 2;
  static constexpr int kScaleBytes = E4M3 ? kUnits * KT * 4 : 0;
  static constexpr int kSmem = 1024 + kUnits * kUnit + kSBytes + kPBytes + kScaleBytes + 256;
  static_assert(kSmem <= 115712, "two CTAs to an SM");
};

// What an item costs beside its tiles (its queries, its end), in tiles: shares are equal in units, an
// item being kItemCost units and one for each tile. (Equal in tiles, a batch of 64 ragged sequences took
// 95 us instead of 85: the CTAs with its short ones came last.) And what joining pieces costs.
constexpr int kItemCost = 2, kJoinCost = 4;

constexpr int kJoin = 24;  // pieces joined at once, at most 32

// How a sequence's tiles lie.
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
  if (a.tree && s.len < s.n) atomicOr(a.status, kStatusBadIndex);  // a drafted token that the cache does not hold
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
  uint16_t* p_buf = reinterpret_cast<uint16_t*>(s_buf + C::kSBytes / 4);
  float* scale_buf = reinterpret_cast<float*>(p_buf + C::kPBytes / 2);
  uint64_t* full = reinterpret_cast<uint64_t*>(scale_buf + C::kScaleBytes / 4);
  uint64_t* empty = full + C::kUnits;
  __shared__ volatile int abort_flag;
  __shared__ int s_last;
  __shared__ float s_top[kComputeWarps][kDecodeHeads], s_vtop[kComputeWarps][kDecodeHeads];
  __shared__ float s_weight[kDecodeHeads][32], s_join[kDecodeHeads][2];
  __shared__ long long s_units[2][kThreads / 32], s_total, s_begin;
  __shared__ int s_items[2][kThreads / 32], s_most[2][kThreads / 32];
  __shared__ struct {
    SeqTiles t;
    int seq, head, u0;
  } s_first;

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
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();

  // The units of all sequences, and the sequence this CTA's share begins in. A thread looks at a sequence
  // at a time, kThreads of them in a round; most batches take one round, whose counts then stay at hand.
  const int heads = a.c.kv_heads, n_seqs = a.b.n_seqs;
  const int rounds = (n_seqs + kThreads - 1) / kThreads;
  SeqTiles t = {};
  long long all = 0, some = 0;  // units and items of every head, before this round
  int most = 0;
  long long units_to = 0, items_to = 0;  // of the round's sequences up to this thread's
  auto look = [&](int round, bool clear) {
    const int b = round * kThreads + tid;
    t.count = 0;
    if (b < n_seqs) {
      t = seq_tiles<KT>(a, b);
      if (clear && t.span.p < 0 && b % gridDim.x == blockIdx.x && t.row < a.b.n_tokens && a.b.cu_q[b + 1] > t.row)
        clear_rows<D>(a, static_cast<long long>(t.row) * a.q_heads, a.q_heads, 0, 1);  // a token that sees nothing
    }
    units_to = t.count > 0 ? t.count + kItemCost : 0;
    items_to = t.count > 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, units_to, o), i = __shfl_up_sync(0xffffffffu, items_to, o);
      if (lane >= o) {
        units_to += u;
        items_to += i;
      }
    }
    const int top = __reduce_max_sync(0xffffffffu, t.count);
    const int at = round & 1;  // (a round's sums are read before the round after the next writes them)
    if (lane == 31) {
      s_units[at][warp] = units_to;
      s_items[at][warp] = static_cast<int>(items_to);
      s_most[at][warp] = top;
    }
    __syncthreads();
    long long units = 0, items = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w == warp) {
        units_to += units;
        items_to += items;
      }
      units += s_units[at][w];
      items += s_items[at][w];
      most = max(most, s_most[at][w]);
    }
    units_to += all;
    items_to += some;
    all += units;
    some += items;
  };
  for (int r = 0; r < max(rounds, 1); ++r) look(r, true);
  {  // Rows of no sequence.
    const KvNoRows none = kv_no_rows(a.b);
    const long long id = static_cast<long long>(blockIdx.x) * kThreads + tid, of = static_cast<long long>(gridDim.x) * kThreads;
    clear_rows<D>(a, static_cast<long long>(none.after) * a.q_heads,
                  static_cast<long long>(a.b.n_tokens - none.after) * a.q_heads, id, of);
    if (none.before > 0) clear_rows<D>(a, 0, static_cast<long long>(none.before) * a.q_heads, id, of);
  }
  // A share is at least one item of one tile: below that pieces cost more than they save. And where items
  // one by one end no later than equal shares and their joins would, nothing is cut and items are counted.
  const bool whole =
      (some * heads + gridDim.x - 1) / gridDim.x * (most + kItemCost) <= all * heads / gridDim.x + kJoinCost;
  const long long total = (whole ? some : all) * heads;
  const int least = whole ? 1 : kItemCost + 1;
  const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), (total + least - 1) / least));
  if (blockIdx.x >= ctas) return;
  const long long begin = decode_share(blockIdx.x, total, ctas);
  if (rounds > 1) {
    all = some = 0;
    __syncthreads();
  }
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) look(r, false);
    const int own = t.count > 0 ? (whole ? 1 : t.count + kItemCost) : 0;
    const long long hi = (whole ? items_to : units_to) * heads, lo = hi - static_cast<long long>(own) * heads;
    if (begin >= lo && begin < hi) {
      s_first.t = t;
      s_first.seq = r * kThreads + tid;
      s_first.head = static_cast<int>((begin - lo) / own);
      s_first.u0 = static_cast<int>((begin - lo) % own);
    }
  }
  if (tid == 0) {
    s_total = total;
    s_begin = begin;
  }
  __syncthreads();
  t = s_first.t;
  int seq = s_first.seq, head = s_first.head, u0 = s_first.u0;  // u0: where the item goes on, in units
  int left = static_cast<int>(decode_share(blockIdx.x + 1, total, ctas) - begin);  // units of the share
  const int cost = whole ? 0 : kItemCost;
  // Units of the item in hand, tiles of it in the share, and the first of these.
  int un, i0, n;
  auto take = [&] {
    un = min((whole ? 1 : t.count + cost) - u0, left);
    i0 = whole ? 0 : max(u0 - cost, 0);
    n = whole ? t.count : max(u0 + un - cost, 0) - i0;
  };

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
    u0 = 0;
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
    while (left > 0 && alive) {
      take();
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
      left -= un;
      if (left > 0) next_item();
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
  // Where 16 keys begin in a unit, and this lane's swizzled places in them: for S rows of keys, four
  // 32-byte steps of a 128-byte chunk; for P V its pieces of V's rows.
  auto block = [&](int k) {
    return static_cast<uint32_t>(((16 * k) >> rows_log2) * (C::kRow << rows_log2) + ((16 * k) & (R - 1)) * 128);
  };
  constexpr int kVLoads = E4M3 && C::VT > 1 ? C::VT / 2 : C::VT;
  uint32_t koff[4], voff[kVLoads];
#pragma unroll
  for (int x = 0; x < 4; ++x)
    koff[x] = block(kg) + ((ds * (C::kSteps / 4)) << (7 + rows_log2)) + (lane & 15) * 128 +
              ((x * 32 + ((lane >> 4) << 4)) ^ ((lane & 7) << 4));
#pragma unroll
  for (int v = 0; v < kVLoads; ++v) {
    const int byte = warp * (C::kRow / kComputeWarps) + v * 32;
    const int key = (lane & 7) + (E4M3 ? lane & 8 : (lane & 16) >> 1);
    const int piece = E4M3 ? (C::VT > 1 ? lane & 16 : 0) : (lane & 8) << 1;
    voff[v] = ((byte >> 7) << (7 + rows_log2)) + key * 128 + (((byte & 127) + piece) ^ ((lane & 7) << 4));
  }
  int taken = 0;  // units of the share before the item
  while (left > 0) {
    take();
    if (n == 0) break;  // the share ends in front of the item's first tile
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
        // A power of two that brings the largest magnitude into [2^14, 2^15); NaN for a row with one.
        const int e = static_cast<int>(top >> 23);
        const float up = e == 255 ? __uint_as_float(0x7fffffffu)
                                  : __uint_as_float(static_cast<uint32_t>(min(268 - e, 254)) << 23);
        const float undo = in_log2 / up;
        // The products' 16 dimensions per step: this lane's four in a row, as a key's bytes are loaded.
#pragma unroll
        for (int s = 0; s < 2 * C::kSteps; ++s) {
          const uint2 w = *reinterpret_cast<const uint2*>(qp + 16 * s + 4 * c4);
          q[2 * s] = pack_f16(__uint_as_float(w.x << 16) * up, __uint_as_float(w.x & 0xffff0000u) * up);
          q[2 * s + 1] = pack_f16(__uint_as_float(w.y << 16) * up, __uint_as_float(w.y & 0xffff0000u) * up);
        }
        qs[0] = __shfl_sync(0xffffffffu, undo, 8 * c4);
        qs[1] = __shfl_sync(0xffffffffu, undo, 8 * c4 + 4);
      }
    }
    float o[C::VT][4];
#pragma unroll
    for (int v = 0; v < C::VT; ++v) o[v][0] = o[v][1] = o[v][2] = o[v][3] = 0.0f;
    // Of heads 2 c4 and 2 c4 + 1: the references, and this lane's part of the sums.
    float ref[2] = {-INFINITY, -INFINITY}, vref[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    for (int i = i0; i < i0 + n; ++i) {
      const int tile = i < t.front ? i : i + t.skip;
      const bool masked = !(tile * KT + KT - 1 <= t.span.p &&
                            (tile * KT >= t.span.lo || tile * KT + KT <= t.span.sinks));
      // S^T of this warp's 16 keys, over its part of the width.
      float s[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
      mbar_wait_bounded(&full[unit], phase, &abort_flag, a.status, kStatusWaitFull);
      {
        const uint32_t base = smem_u32(ring + unit * C::kUnit);
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st) {
          uint32_t f[4];
          ldsm4(base + ((st >> 2) << (7 + rows_log2)) + koff[st & 3], f);
          if constexpr (E4M3) {
            uint32_t f0[4], f1[4];
            widen_e4m3(f[0], f0[0], f0[2]);
            widen_e4m3(f[1], f0[1], f0[3]);
            widen_e4m3(f[2], f1[0], f1[2]);
            widen_e4m3(f[3], f1[1], f1[3]);
            mma_f16(s[0], f0, q[4 * st], q[4 * st + 1]);
            mma_f16(s[1], f1, q[4 * st + 2], q[4 * st + 3]);
          } else {
            mma_bf16(s[st & 1], f, q[2 * st], q[2 * st + 1]);
          }
        }
      }
      // The scores this lane weighs: of two heads, keys k0 and k0 + 8, or k0 alone where S is joined.
      constexpr int kMine = C::DS > 1 ? 1 : 2;
      const int k0 = C::DS > 1 ? warp * 8 + r8 : kg * 16 + r8;
      const bool active = C::DS == 1 || warp * 8 < KT;
      float f0 = 1.0f, f1 = 1.0f;
      if constexpr (E4M3) {
        f0 = scale_buf[unit * KT + kg * 16 + r8];
        f1 = scale_buf[unit * KT + kg * 16 + r8 + 8];
      }
      float x[kMine][2];  // scores in base 2
      const float x00 = (s[0][0] + s[1][0]) * (qs[0] * f0), x01 = (s[0][1] + s[1][1]) * (qs[1] * f0);
      const float x10 = (s[0][2] + s[1][2]) * (qs[0] * f1), x11 = (s[0][3] + s[1][3]) * (qs[1] * f1);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[unit]);
      next_unit();
      if constexpr (C::DS > 1) {
        float* to = s_buf + (ds * kDecodeHeads + 2 * c4) * C::SP + kg * 16 + r8;
        to[0] = x00;
        to[C::SP] = x01;
        to[8] = x10;
        to[C::SP + 8] = x11;
        compute_sync();
        x[0][0] = x[0][1] = 0.0f;
        if (active) {
#pragma unroll
          for (int part = 0; part < C::DS; ++part) {
            x[0][0] += s_buf[(part * kDecodeHeads + 2 * c4) * C::SP + k0];
            x[0][1] += s_buf[(part * kDecodeHeads + 2 * c4 + 1) * C::SP + k0];
          }
        }
      } else {
        x[0][0] = x00;
        x[0][1] = x01;
        x[1][0] = x10;
        x[1][1] = x11;
      }
      // The values' scales, in base 2.
      float lv[kMine];
      if constexpr (E4M3) {
        mbar_wait_bounded(&full[unit], phase, &abort_flag, a.status, kStatusWaitFull);
#pragma unroll
        for (int r = 0; r < kMine; ++r) lv[r] = active ? log2f(scale_buf[unit * KT + k0 + 8 * r]) : 0.0f;
      }
      bool hidden[kMine];
#pragma unroll
      for (int r = 0; r < kMine; ++r) {
        const int at = tile * KT + k0 + 8 * r;
        hidden[r] = !active || (masked && (at > t.span.p || (at < t.span.lo && at >= t.span.sinks)));
        if (hidden[r]) x[r][0] = x[r][1] = -INFINITY;
        if (E4M3 && hidden[r]) lv[r] = 0.0f;
      }
      uint16_t* pb = p_buf + flip * (kDecodeHeads * C::PP);
      flip ^= 1;
      // A reference of -inf (nothing but NaN or -inf so far) counts as 0.
      auto weigh = [&](float (&sum)[2]) {
        const float base[2] = {ref[0] == -INFINITY ? 0.0f : ref[0], ref[1] == -INFINITY ? 0.0f : ref[1]};
        const float vbase[2] = {vref[0] == -INFINITY ? 0.0f : vref[0], vref[1] == -INFINITY ? 0.0f : vref[1]};
        sum[0] = sum[1] = 0.0f;
#pragma unroll
        for (int r = 0; r < kMine; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float w = exp2_approx(x[r][h] - base[h]);
            sum[h] += w;
            uint16_t bits;
            if constexpr (E4M3) bits = __half_as_ushort(__float2half_rn(exp2_approx(x[r][h] + lv[r] - vbase[h])));
            else bits = f32_to_bf16_rn(w);
            if (active) pb[(2 * c4 + h) * C::PP + k0 + 8 * r] = bits;
          }
      };
      bool over = false;
#pragma unroll
      for (int r = 0; r < kMine; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          over |= x[r][h] > ref[h] + 8.0f;
          if constexpr (E4M3) over |= x[r][h] + lv[r] > vref[h] + 15.0f;
        }
      float sum[2];
      weigh(sum);
      if (compute_sync_or(over)) {
        float top[2] = {x[0][0], x[0][1]}, vtop[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (kMine > 1) top[h] = fmaxf(top[h], x[kMine - 1][h]);
          if constexpr (E4M3)
#pragma unroll
            for (int r = 0; r < kMine; ++r) vtop[h] = fmaxf(vtop[h], x[r][h] + lv[r]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], d));
            if constexpr (E4M3) vtop[h] = fmaxf(vtop[h], __shfl_xor_sync(0xffffffffu, vtop[h], d));
          }
          if (r8 == 0) {
            s_top[warp][2 * c4 + h] = top[h];
            if constexpr (E4M3) s_vtop[warp][2 * c4 + h] = vtop[h];
          }
        }
        compute_sync();
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float m = ref[h], vm = vref[h] + 7.0f;
          for (int w = 0; w < kComputeWarps; ++w) {
            m = fmaxf(m, s_top[w][2 * c4 + h]);
            if constexpr (E4M3) vm = fmaxf(vm, s_vtop[w][2 * c4 + h]);
          }
          f[h] = exp2_approx(ref[h] - (m == -INFINITY ? 0.0f : m));
          l[h] *= f[h];
          ref[h] = m;
          if constexpr (E4M3) {
            vm -= 7.0f;
            f[h] = exp2_approx(vref[h] - (vm == -INFINITY ? 0.0f : vm));
            vref[h] = vm;
          }
        }
#pragma unroll
        for (int v = 0; v < C::VT; ++v) {
          o[v][0] *= f[0];
          o[v][1] *= f[1];
          o[v][2] *= f[0];
          o[v][3] *= f[1];
        }
        weigh(sum);
        compute_sync();
      }
      l[0] += sum[0];
      l[1] += sum[1];

      // O^T += V^T P^T over this warp's part of the width.
      if constexpr (!E4M3) mbar_wait_bounded(&full[unit], phase, &abort_flag, a.status, kStatusWaitFull);
      const uint32_t vbase = smem_u32(ring + unit * C::kUnit);
      const uint32_t paddr = smem_u32(pb) + ((lane & 7) * C::PP + (lane >> 3) * 8) * 2;
      auto products = [&](bool hide) {  // inlined with either value
#pragma unroll(C::kVUnroll)
        for (int k2 = 0; k2 < KT / 32; ++k2) {
          uint32_t pr[4];
          ldsm4(paddr + k2 * 64, pr);
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            const int k = 2 * k2 + kk;
            const uint32_t b0 = pr[2 * kk], b1 = pr[2 * kk + 1];
            uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
            if (hide) {
              // Hidden values may be anything, NaN included: they become 0.
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int at = tile * KT + 16 * k + 2 * c4 + (y & 1) + 8 * (y >> 1);
                const uint32_t gone = at > t.span.p || (at < t.span.lo && at >= t.span.sinks) ? 0xffffu << (16 * (y & 1)) : 0u;
                if (y < 2) keep0 &= ~gone;
                else keep1 &= ~gone;
              }
            }
            const uint32_t vk = vbase + block(k);
            if constexpr (E4M3) {
              // A 16-byte piece is 16 dimensions; as 16-bit pairs the transposed load gives a lane the
              // dimensions 2 r8 and 2 r8 + 1, which become the rows r8 and r8 + 8 of the block.
#pragma unroll
              for (int v = 0; v < C::VT; v += 2) {
                uint32_t w[4];
                if constexpr (C::VT > 1) ldsm4_trans(vk + voff[v / 2], w);
                else ldsm2_trans(vk + voff[0], w[0], w[1]);
#pragma unroll
                for (int y = 0; y < (C::VT > 1 ? 2 : 1); ++y) {
                  uint32_t fr[4];
                  // Bytes: d and d + 1 of one key, then of the next.
                  widen_e4m3(__byte_perm(w[2 * y], 0, 0x3120), fr[0], fr[1]);
                  widen_e4m3(__byte_perm(w[2 * y + 1], 0, 0x3120), fr[2], fr[3]);
                  if (hide) {
                    fr[0] &= keep0;
                    fr[1] &= keep0;
                    fr[2] &= keep1;
                    fr[3] &= keep1;
                  }
                  mma_f16(o[v + y], fr, b0, b1);
                }
              }
            } else {
#pragma unroll
              for (int v = 0; v < C::VT; ++v) {
                uint32_t w[4];
                ldsm4_trans(vk + voff[v], w);
                if (hide) {
                  w[0] &= keep0;
                  w[1] &= keep0;
                  w[2] &= keep1;
                  w[3] &= keep1;
                }
                mma_bf16(o[v], w, b0, b1);
              }
            }
          }
        }
      };
      if (masked) products(true);
      else products(false);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[unit]);
      next_unit();
    }

    // The sums of all lanes and warps, and the outputs relative to the scores' reference.
    float m[2] = {ref[0], ref[1]};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], d);
      if (r8 == 0) s_top[warp][2 * c4 + h] = l[h];
    }
    compute_sync();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] = 0.0f;
      for (int w = 0; w < kComputeWarps; ++w) l[h] += s_top[w][2 * c4 + h];
      if constexpr (E4M3) {
        const float f = vref[h] == -INFINITY ? 1.0f : exp2f(vref[h] - (m[h] == -INFINITY ? 0.0f : m[h]));
#pragma unroll
        for (int v = 0; v < C::VT; ++v) {
          o[v][h] *= f;
          o[v][2 + h] *= f;
        }
      }
    }
    compute_sync();
    const long long to = static_cast<long long>(t.row) * a.q_heads + head * a.group;  // the first head's output row
    const int h0 = 2 * c4, h1 = h0 + 1;
    // The dimension of o[v][0]; o[v][2] is `apart` further.
    constexpr int apart = E4M3 ? 1 : 8;
    const int dim0 = warp * (D / kComputeWarps) + (E4M3 ? 2 * r8 : r8);
    if (i0 == 0 && n == t.count) {
      const float f0 = l[0] == 0.0f ? 0.0f : 1.0f / l[0], f1 = l[1] == 0.0f ? 0.0f : 1.0f / l[1];
#pragma unroll
      for (int v = 0; v < C::VT; ++v)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int h = x & 1 ? h1 : h0;
          if (h < a.group)
            a.out[(to + h) * D + dim0 + v * 16 + (x >> 1) * apart] = f32_to_bf16_rn(o[v][x] * (x & 1 ? f1 : f0));
        }
      if (a.lse && warp == 0 && r8 == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (h0 + h < a.group) a.lse[to + h0 + h] = l[h] == 0.0f ? -INFINITY : (m[h] + log2f(l[h])) * 0.693147181f;
      }
    } else {
      // A piece. Its place is this CTA's first if the item began before the CTA's share or with it, as
      // it did for all of the item's CTAs but its first.
      const long long all_units = s_total, item_start = s_begin + taken - u0;
      const int first = decode_owner(item_start + cost, all_units, ctas);
      const int count = decode_owner(item_start + cost + t.count - 1, all_units, ctas) - first + 1;
      const int first_place = 2 * first + (decode_share(first, all_units, ctas) >= item_start ? 0 : 1);
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
        if (warp == 0 && r8 == 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            piece[kDecodeHeads * D + h0 + h] = m[h];
            piece[kDecodeHeads * D + kDecodeHeads + h0 + h] = l[h];
          }
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
    taken += un;
    left -= un;
    if (left > 0) next_item();
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
