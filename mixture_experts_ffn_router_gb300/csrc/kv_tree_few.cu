// kv_tree_few.cu — attention of small trees of drafted tokens over an e4m3 paged cache: up to 16 rows, (node, query head), to
// each kv head.
//
// The kernel for chunks takes the same time for a tile of keys however few of its 256 rows there are, and over e4m3 that time
// is three to five times the tile's bytes'. Here the keys are the wide side, as for single tokens (kv_decode.cu, which
// explains the ring of units, the shares and their joins, the softmax against a reference per row and the scales of both
// formats): S^T = K Q^T and O^T = V^T P^T by mma.sync, with the rows as two blocks of the narrow side. A warp has 16 keys of
// a tile for S, and an eighth of V's width; codes are widened to fp16 once for both blocks. The queries, scaled and in the
// order of the products' second operand, lie in shared memory, as registers hold the outputs of 16 rows.
//
// What a row sees: in tiles with nodes, or where windows begin, a word of bits per node and 64 keys (tree_seen), in shared
// memory; elsewhere every row sees every key. A tile's values that no row sees are cleared, whatever they are.
//
// Measured, in a graph, against the kernel for chunks, trees of 4 nodes, 16 heads on 8 of width 256: 64 sequences
// of 1000 to 4000 tokens 118 and 262 us (the bytes 87.5), of 250 to 1000 51 and 120 (22.5), 1 of 4000 23 and 28; 16 heads
// on 4 of width 128: 56 and 112 us (22.4), 30 and 53 (5.9), 19 and 23. A chain of barriers per tile bounds it, as for single
// tokens, and a tile of width 128 has the same chain for half the bytes. Tiles of 64 keys, which leave room
// for more of them on their way but double the barriers, took 144 us for the first. With 32 rows, four blocks, the outputs
// and references no longer fit two CTAs' registers: 98 us against 127 for 64 sequences of 1000, but 45 against 27 for one of
// 4000, so these stay with the kernel for chunks.
#include "kv_mma.cuh"
#include "kv_tree.cuh"

namespace moe {

namespace {

constexpr int kThreads = (kComputeWarps + 1) * 32;
constexpr int kItemCost = 2, kJoinCost = 4, kJoin = 24;  // as for single tokens

constexpr int NB = 2;      // blocks of eight rows
constexpr int R = 8 * NB;
constexpr int KT = 128;    // keys of a tile, 16 to a warp
static_assert(R == kFewRows && KT == 16 * kComputeWarps, "rows and keys");

template <int D>
struct Few {
  static constexpr int kUnit = KT * D;
  static constexpr int kUnits = D == 256 ? 2 : 5;
  static constexpr int kSteps = D / 32;                // 32-byte steps of a key row
  static constexpr int VT = D / (16 * kComputeWarps);  // 16-wide blocks of V per warp
  static constexpr int PP = KT + 8;                    // row pitch of P, in 16-bit values
  static constexpr int kPBytes = 2 * R * PP * 2;
  static constexpr int kScaleBytes = kUnits * KT * 4;
  static constexpr int kQBytes = R * D * 2;
  static constexpr int kSmem = 1024 + kUnits * kUnit + kPBytes + kScaleBytes + kQBytes + 16 * kUnits;
  static constexpr long long kPiece = static_cast<long long>(R) * D + 2 * R;  // floats: outputs, maxima, sums
  static_assert(R * 34 * 4 <= kPBytes, "the joins' weights lie where P was");
  static_assert(2 * kDecodeMaxCtas * kPiece <= 2 * kChunkMaxPairs * kChunkPieceFloats, "room for the pieces");
  static_assert(kSmem <= 111616, "two CTAs to an SM");
};

// A sequence's tree, and how the tiles of its keys lie. keys.p0 is the context's last position.
struct TreeTiles {
  KvRowTile keys;
  int last;   // the last key that a node may see, below 0: none
  int lo;     // the first one that is not hidden to all by their windows, but for sinks
  int sinks;
};

__device__ __forceinline__ TreeTiles tree_tiles(const KvAttn& a, int seq) {
  const KvSeq s = kv_sequence(a.b, a.c, seq, a.status);
  TreeTiles t = {};
  t.keys.seq = seq;
  t.keys.row0 = s.row0;
  t.keys.nt = s.n;
  t.keys.p0 = s.len - s.n - 1;
  t.last = -1;
  if (s.n == 0) return t;
  if (s.len < s.n) {
    atomicOr(a.status, kStatusBadIndex);
    return t;
  }
  t.last = s.len - 1;
  const KvSpan span = kv_span(t.keys.p0 + 1, a.window, a.sinks);
  t.lo = span.lo;
  t.sinks = span.sinks;
  const int first = span.lo / KT;
  t.keys.front = min((span.sinks + KT - 1) / KT, first);
  t.keys.skip = first - t.keys.front;
  t.keys.count = t.last / KT + 1 - t.keys.skip;
  return t;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    kv_tree_few_kernel(const KvAttn a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using C = Few<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint2* q_buf = reinterpret_cast<uint2*>(ring + C::kUnits * C::kUnit);  // [D / 16][NB][32 lanes]
  uint16_t* p_buf = reinterpret_cast<uint16_t*>(q_buf + C::kQBytes / 8);
  float* scale_buf = reinterpret_cast<float*>(p_buf + C::kPBytes / 2);
  uint64_t* full = reinterpret_cast<uint64_t*>(scale_buf + C::kScaleBytes / 4);
  uint64_t* empty = full + C::kUnits;
  __shared__ volatile int abort_flag;
  __shared__ int s_last;
  __shared__ float s_top[kComputeWarps][R], s_vtop[kComputeWarps][R], s_undo[R];
  __shared__ unsigned long long s_seen[2][R][KT / 64], s_any[2][KT / 64];
  __shared__ long long s_units[2][kThreads / 32], s_total, s_begin;
  __shared__ int s_items[2][kThreads / 32], s_most[2][kThreads / 32];
  __shared__ struct {
    TreeTiles t;
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

  // The units of all sequences, and the sequence this CTA's share begins in: as for single tokens.
  const int heads = a.c.kv_heads, n_seqs = a.b.n_seqs;
  const int rounds = (n_seqs + kThreads - 1) / kThreads;
  TreeTiles t = {};
  long long all = 0, some = 0;  // units and items of every head, before this round
  int most = 0;
  long long units_to = 0, items_to = 0;  // of the round's sequences up to this thread's
  auto look = [&](int round, bool clear) {
    const int b = round * kThreads + tid;
    t.keys.count = 0;
    if (b < n_seqs) {
      t = tree_tiles(a, b);
      if (clear && t.last < 0 && t.keys.nt > 0 && b % gridDim.x == blockIdx.x)  // nodes that see nothing
        clear_rows<D>(a, static_cast<long long>(t.keys.row0) * a.q_heads, static_cast<long long>(t.keys.nt) * a.q_heads, 0, 1);
    }
    units_to = t.keys.count > 0 ? t.keys.count + kItemCost : 0;
    items_to = t.keys.count > 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, units_to, o), i = __shfl_up_sync(0xffffffffu, items_to, o);
      if (lane >= o) {
        units_to += u;
        items_to += i;
      }
    }
    const int top = __reduce_max_sync(0xffffffffu, t.keys.count);
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
    const int own = t.keys.count > 0 ? (whole ? 1 : t.keys.count + kItemCost) : 0;
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
    un = min((whole ? 1 : t.keys.count + cost) - u0, left);
    i0 = whole ? 0 : max(u0 - cost, 0);
    n = whole ? t.keys.count : max(u0 + un - cost, 0) - i0;
  };

  const int rows_log2 = min(a.c.page_log2, 7);
  const int box = 1 << rows_log2;  // rows of a box
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
    do t = tree_tiles(a, ++seq);
    while (t.keys.count == 0);
  };

  if (warp == kComputeWarps) {
    // ---------------------------------------------------------------- loads
    const uint64_t policy = policy_evict_first();
    bool alive = true;
    int issued = 0;
    while (left > 0 && alive) {
      take();
      for (int i = i0; i < i0 + n && alive; ++i) {
        const int tile = i < t.keys.front ? i : i + t.keys.skip;
        const int p0 = tile * KT + (lane << rows_log2);  // the first position of this lane's page part
        const bool need = lane < (KT >> rows_log2) && p0 <= t.last && (p0 + box - 1 >= t.lo || p0 < t.sinks);
        int page = -1;
        if (need) page = kv_page(a.b, a.c, seq, p0 >> a.c.page_log2, a.status);
        const int row = page < 0 ? 0
                                 : ((page * heads + head) << a.c.page_log2) + (p0 & ((1 << a.c.page_log2) - 1));
        const unsigned who = __ballot_sync(0xffffffffu, page >= 0);
        const uint32_t bytes = __popc(who) * static_cast<uint32_t>(box * (D + 4));
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
            uint8_t* dst = ring + unit * C::kUnit + (lane << rows_log2) * D;
            asm volatile(
                "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
                " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
                "l"(reinterpret_cast<uint64_t>(kv ? &map_v : &map_k)), "r"(0), "r"(row), "r"(0),
                "r"(smem_u32(&full[unit])), "l"(policy)
                : "memory");
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                    smem_u32(scale_buf + unit * KT + (lane << rows_log2))),
                "l"(reinterpret_cast<uint64_t>((kv ? a.c.v_scale : a.c.k_scale) + row)), "r"(box * 4),
                "r"(smem_u32(&full[unit]))
                : "memory");
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
  const int c4 = lane & 3, r8 = lane >> 2;
  int flip = 0;
  // Where 16 keys begin in a unit, and this lane's swizzled places in them: for S rows of keys, four
  // 32-byte steps of a 128-byte chunk; for P V its pieces of V's rows.
  auto block = [&](int k) {
    return static_cast<uint32_t>(((16 * k) >> rows_log2) * (D << rows_log2) + ((16 * k) & (box - 1)) * 128);
  };
  uint32_t koff[4], voff;
#pragma unroll
  for (int x = 0; x < 4; ++x)
    koff[x] = block(warp) + (lane & 15) * 128 + ((x * 32 + ((lane >> 4) << 4)) ^ ((lane & 7) << 4));
  {
    const int byte = warp * (D / kComputeWarps);
    const int key = (lane & 7) + (lane & 8);
    const int piece = C::VT > 1 ? lane & 16 : 0;
    voff = ((byte >> 7) << (7 + rows_log2)) + key * 128 + (((byte & 127) + piece) ^ ((lane & 7) << 4));
  }
  int taken = 0;  // units of the share before the item
  while (left > 0) {
    take();
    if (n == 0) break;  // the share ends in front of the item's first tile
    const int rows = t.keys.nt * a.group;  // (those after them are copies of the last)
    // The queries, a row to a warp at a time: brought by a power of two into [2^14, 2^15), as fp16; a lane of the products'
    // second operand has row r8 of a block, and of 16 dimensions four in a row, as a key's bytes are loaded.
#pragma unroll 1
    for (int nb = 0; nb < NB; ++nb) {
      const int r = nb * 8 + warp, tok = min(r, rows - 1) / a.group, h = min(r, rows - 1) % a.group;
      const uint16_t* qp = a.q.ptr + (t.keys.row0 + tok) * a.q.token_stride + (head * a.group + h) * a.q.head_stride;
      constexpr int kMine = D / 32 / 4;  // of four dimensions
      uint2 w[kMine];
      uint32_t top = 0;
#pragma unroll
      for (int x = 0; x < kMine; ++x) {
        w[x] = *reinterpret_cast<const uint2*>(qp + 4 * (lane + 32 * x));
        top = max(top, max(max(w[x].x << 16 & 0x7fffffffu, w[x].x & 0x7fffffffu),
                           max(w[x].y << 16 & 0x7fffffffu, w[x].y & 0x7fffffffu)));
      }
      top = __reduce_max_sync(0xffffffffu, top);
      const int e = static_cast<int>(top >> 23);  // (NaN for a row with one, or an infinity)
      const float up = e == 255 ? __uint_as_float(0x7fffffffu)
                                : __uint_as_float(static_cast<uint32_t>(min(268 - e, 254)) << 23);
      if (lane == 0) s_undo[r] = a.scale * 1.44269504f / up;
#pragma unroll
      for (int x = 0; x < kMine; ++x) {
        const int four = lane + 32 * x;
        q_buf[((four >> 2) * NB + nb) * 32 + warp * 4 + (four & 3)] =
            make_uint2(pack_f16(__uint_as_float(w[x].x << 16) * up, __uint_as_float(w[x].x & 0xffff0000u) * up),
                       pack_f16(__uint_as_float(w[x].y << 16) * up, __uint_as_float(w[x].y & 0xffff0000u) * up));
      }
    }
    compute_sync();
    float o[NB][C::VT][4];
    // Of rows 2 c4 and 2 c4 + 1 of each block: the references, and this lane's part of the sums.
    float ref[NB][2], vref[NB][2], l[NB][2];
    int node[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int v = 0; v < C::VT; ++v) o[nb][v][0] = o[nb][v][1] = o[nb][v][2] = o[nb][v][3] = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ref[nb][h] = vref[nb][h] = -INFINITY;
        l[nb][h] = 0.0f;
        node[nb][h] = min(nb * 8 + 2 * c4 + h, rows - 1) / a.group;
      }
    }

    for (int i = i0; i < i0 + n; ++i) {
      const int tile = i < t.keys.front ? i : i + t.keys.skip;
      // Whether each row sees each key: no node among them, and the window of the deepest that there could be.
      const bool masked = !(tile * KT + KT - 1 <= t.keys.p0 &&
                            (a.window == 0 || tile * KT > t.last - a.window || tile * KT + KT <= a.sinks));
      unsigned long long (&seen)[R][KT / 64] = s_seen[i & 1];
      if (masked) {
        if (warp < KT / 64) {
          const unsigned long long bits = tree_seen(a, t.keys, lane, tile * KT + 64 * warp);
          if (lane < R) seen[lane][warp] = bits;
          const uint32_t lo = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(bits));
          const uint32_t hi = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(bits >> 32));
          if (lane == 0) s_any[i & 1][warp] = lo | static_cast<unsigned long long>(hi) << 32;
        }
        compute_sync();
      }
      // S^T of this warp's 16 keys.
      float s[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.0f;
      mbar_wait_bounded(&full[unit], phase, &abort_flag, a.status, kStatusWaitFull);
      {
        const uint32_t base = smem_u32(ring + unit * C::kUnit);
        const uint2* qf = q_buf + lane;
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st) {
          uint32_t f[4], f0[4], f1[4];
          ldsm4(base + ((st >> 2) << (7 + rows_log2)) + koff[st & 3], f);
          widen_e4m3(f[0], f0[0], f0[2]);
          widen_e4m3(f[1], f0[1], f0[3]);
          widen_e4m3(f[2], f1[0], f1[2]);
          widen_e4m3(f[3], f1[1], f1[3]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint2 q0 = qf[(2 * st * NB + nb) * 32], q1 = qf[((2 * st + 1) * NB + nb) * 32];
            mma_f16(s[nb], f0, q0.x, q0.y);
            mma_f16(s[nb], f1, q1.x, q1.y);
          }
        }
      }
      // The scores this lane weighs: of two rows of each block, keys k0 and k0 + 8.
      const int k0 = warp * 16 + r8;
      const float f0 = scale_buf[unit * KT + k0], f1 = scale_buf[unit * KT + k0 + 8];
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[unit]);
      next_unit();
      float x[NB][2][2];  // scores in base 2
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float u0 = s_undo[nb * 8 + 2 * c4], u1 = s_undo[nb * 8 + 2 * c4 + 1];
        x[nb][0][0] = s[nb][0] * (u0 * f0);
        x[nb][0][1] = s[nb][1] * (u1 * f0);
        x[nb][1][0] = s[nb][2] * (u0 * f1);
        x[nb][1][1] = s[nb][3] * (u1 * f1);
      }
      // The values' scales, in base 2.
      float lv[2];
      mbar_wait_bounded(&full[unit], phase, &abort_flag, a.status, kStatusWaitFull);
#pragma unroll
      for (int r = 0; r < 2; ++r) lv[r] = log2f(scale_buf[unit * KT + k0 + 8 * r]);
      // Bits of what is hidden: 4 nb + 2 r + h.
      uint32_t hidden = 0;
      if (masked) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int k = k0 + 8 * r;
              if (seen[node[nb][h]][k >> 6] >> (k & 63) & 1ull) continue;
              hidden |= 1u << (4 * nb + 2 * r + h);
              x[nb][r][h] = -INFINITY;
            }
      }
      uint16_t* pb = p_buf + flip * (R * C::PP);
      flip ^= 1;
      // A reference of -inf (nothing but NaN or -inf so far) counts as 0.
      auto weigh = [&](float (&sum)[NB][2]) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float base = ref[nb][h] == -INFINITY ? 0.0f : ref[nb][h];
            const float vbase = vref[nb][h] == -INFINITY ? 0.0f : vref[nb][h];
            sum[nb][h] = 0.0f;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              sum[nb][h] += exp2_approx(x[nb][r][h] - base);
              // (A hidden key's scale may be anything.)
              const float weight = hidden >> (4 * nb + 2 * r + h) & 1u ? 0.0f : exp2_approx(x[nb][r][h] + lv[r] - vbase);
              pb[(nb * 8 + 2 * c4 + h) * C::PP + k0 + 8 * r] = __half_as_ushort(__float2half_rn(weight));
            }
          }
      };
      bool over = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (hidden >> (4 * nb + 2 * r + h) & 1u) continue;
            over |= x[nb][r][h] > ref[nb][h] + 8.0f || x[nb][r][h] + lv[r] > vref[nb][h] + 15.0f;
          }
      float sum[NB][2];
      weigh(sum);
      if (compute_sync_or(over)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float top = -INFINITY, vtop = -INFINITY;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if (hidden >> (4 * nb + 2 * r + h) & 1u) continue;
              top = fmaxf(top, x[nb][r][h]);
              vtop = fmaxf(vtop, x[nb][r][h] + lv[r]);
            }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
              vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, d));
            }
            if (r8 == 0) {
              s_top[warp][nb * 8 + 2 * c4 + h] = top;
              s_vtop[warp][nb * 8 + 2 * c4 + h] = vtop;
            }
          }
        compute_sync();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float f[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float m = ref[nb][h], vm = vref[nb][h] + 7.0f;
            for (int w = 0; w < kComputeWarps; ++w) {
              m = fmaxf(m, s_top[w][nb * 8 + 2 * c4 + h]);
              vm = fmaxf(vm, s_vtop[w][nb * 8 + 2 * c4 + h]);
            }
            l[nb][h] *= exp2_approx(ref[nb][h] - (m == -INFINITY ? 0.0f : m));
            ref[nb][h] = m;
            vm -= 7.0f;
            f[h] = exp2_approx(vref[nb][h] - (vm == -INFINITY ? 0.0f : vm));
            vref[nb][h] = vm;
          }
#pragma unroll
          for (int v = 0; v < C::VT; ++v) {
            o[nb][v][0] *= f[0];
            o[nb][v][1] *= f[1];
            o[nb][v][2] *= f[0];
            o[nb][v][3] *= f[1];
          }
        }
        weigh(sum);
        compute_sync();
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        l[nb][0] += sum[nb][0];
        l[nb][1] += sum[nb][1];
      }

      // O^T += V^T P^T over this warp's part of the width.
      const uint32_t vbase = smem_u32(ring + unit * C::kUnit);
      const uint32_t paddr = smem_u32(pb) + ((lane & 7) * C::PP + (lane >> 3) * 8) * 2;
      auto products = [&](bool hide) {  // inlined with either value
#pragma unroll 1
        for (int k2 = 0; k2 < KT / 32; ++k2) {
          uint32_t pr[NB][4];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) ldsm4(paddr + nb * (8 * C::PP * 2) + k2 * 64, pr[nb]);
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            const int k = 2 * k2 + kk;
            uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
            if (hide) {
              // Values that no row sees may be anything, NaN included: they become 0.
              const uint32_t any = static_cast<uint32_t>(s_any[i & 1][k >> 2] >> (16 * (k & 3))) >> (2 * c4);
              keep0 = (any & 1u ? 0xffffu : 0u) | (any & 2u ? 0xffff0000u : 0u);
              keep1 = (any & 0x100u ? 0xffffu : 0u) | (any & 0x200u ? 0xffff0000u : 0u);
            }
            // A 16-byte piece is 16 dimensions; as 16-bit pairs the transposed load gives a lane the
            // dimensions 2 r8 and 2 r8 + 1, which become the rows r8 and r8 + 8 of the block.
            uint32_t w[4];
            if constexpr (C::VT > 1) ldsm4_trans(vbase + block(k) + voff, w);
            else ldsm2_trans(vbase + block(k) + voff, w[0], w[1]);
#pragma unroll
            for (int y = 0; y < C::VT; ++y) {
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
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma_f16(o[nb][y], fr, pr[nb][2 * kk], pr[nb][2 * kk + 1]);
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
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nb][h] += __shfl_xor_sync(0xffffffffu, l[nb][h], d);
        if (r8 == 0) s_top[warp][nb * 8 + 2 * c4 + h] = l[nb][h];
      }
    compute_sync();
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[nb][h] = 0.0f;
        for (int w = 0; w < kComputeWarps; ++w) l[nb][h] += s_top[w][nb * 8 + 2 * c4 + h];
        const float f =
            vref[nb][h] == -INFINITY ? 1.0f : exp2f(vref[nb][h] - (ref[nb][h] == -INFINITY ? 0.0f : ref[nb][h]));
#pragma unroll
        for (int v = 0; v < C::VT; ++v) {
          o[nb][v][h] *= f;
          o[nb][v][2 + h] *= f;
        }
      }
    compute_sync();
    // A row's place among all tokens' heads.
    auto row_of = [&](int r) {
      const int tok = r / a.group;
      return (static_cast<long long>(t.keys.row0) + tok) * a.q_heads + head * a.group + (r - tok * a.group);
    };
    const int dim0 = warp * (D / kComputeWarps) + 2 * r8;  // of o[..][0][0]; o[..][0][2] is the next
    if (i0 == 0 && n == t.keys.count) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = nb * 8 + 2 * c4 + h;
          if (r >= rows) continue;
          const long long to = row_of(r);
          const float f = l[nb][h] == 0.0f ? 0.0f : 1.0f / l[nb][h];
#pragma unroll
          for (int v = 0; v < C::VT; ++v)
            *reinterpret_cast<uint32_t*>(a.out + to * D + dim0 + v * 16) = pack_bf16(o[nb][v][h] * f, o[nb][v][2 + h] * f);
          if (a.lse && warp == 0 && r8 == 0)
            a.lse[to] = l[nb][h] == 0.0f ? -INFINITY : (ref[nb][h] + log2f(l[nb][h])) * 0.693147181f;
        }
    } else {
      // A piece: as for single tokens.
      const long long all_units = s_total, item_start = s_begin + taken - u0;
      const int first = decode_owner(item_start + cost, all_units, ctas);
      const int count = decode_owner(item_start + cost + t.keys.count - 1, all_units, ctas) - first + 1;
      const int first_place = 2 * first + (decode_share(first, all_units, ctas) >= item_start ? 0 : 1);
      auto place = [&](int x) { return x == 0 ? first_place : 2 * (first + x); };  // of the item's piece x
      const int me = static_cast<int>(blockIdx.x) - first;
      {
        float* piece = a.chunk_partial + place(me) * C::kPiece;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = nb * 8 + 2 * c4 + h;
            if (r >= rows) continue;
#pragma unroll
            for (int v = 0; v < C::VT; ++v)
              *reinterpret_cast<float2*>(piece + r * D + dim0 + v * 16) = make_float2(o[nb][v][h], o[nb][v][2 + h]);
            if (warp == 0 && r8 == 0) {
              piece[R * D + r] = ref[nb][h];
              piece[R * D + R + r] = l[nb][h];
            }
          }
      }
      float* weights = reinterpret_cast<float*>(p_buf);  // [R][32], then [R][2]: P is done with
      float* joined = weights + R * 32;
      // Up to kJoin pieces are joined at once; more in groups first.
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
        // The pieces' weights, a warp to a row, a lane for each piece.
        for (int r = warp; r < rows; r += kComputeWarps) {
          const float* at = a.chunk_partial + place(from + min(lane, n_in - 1) * apart_in) * C::kPiece + R * D + r;
          const float pm = lane < n_in ? __ldcg(at) : -INFINITY;
          float top = pm;
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          const float w = lane < n_in ? exp2_approx(pm - (top == -INFINITY ? 0.0f : top)) : 0.0f;
          float sum = lane < n_in ? w * __ldcg(at + R) : 0.0f;
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          weights[r * 32 + lane] = w;
          if (lane == 0) {
            joined[2 * r] = top;
            joined[2 * r + 1] = sum;
          }
        }
        compute_sync();
        float* group_piece = a.chunk_partial + place(from) * C::kPiece;
#pragma unroll 1
        for (int i = tid; i < rows * (D / 4); i += kComputeWarps * 32) {
          const int r = i / (D / 4);
          float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
          for (int x = 0; x < n_in; ++x) {
            const float4 y =
                __ldcg(reinterpret_cast<const float4*>(a.chunk_partial + place(from + x * apart_in) * C::kPiece + 4 * i));
            const float w = weights[r * 32 + x];
            acc.x = fmaf(w, y.x, acc.x);
            acc.y = fmaf(w, y.y, acc.y);
            acc.z = fmaf(w, y.z, acc.z);
            acc.w = fmaf(w, y.w, acc.w);
          }
          if (final) {
            const float sum = joined[2 * r + 1], inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            *reinterpret_cast<uint2*>(a.out + row_of(r) * D + 4 * (i - r * (D / 4))) =
                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
          } else {
            *reinterpret_cast<float4*>(group_piece + 4 * i) = acc;
          }
        }
        if (tid < rows) {
          const float top = joined[2 * tid], sum = joined[2 * tid + 1];
          if (!final) {
            group_piece[R * D + tid] = top;
            group_piece[R * D + R + tid] = sum;
          } else if (a.lse) {
            a.lse[row_of(tid)] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.693147181f;
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

template <int D>
cudaError_t launch(const KvAttn& a, int ctas, cudaStream_t s) {
  using C = Few<D>;
  CUtensorMap mk, mv;
  const uint64_t rows = (static_cast<uint64_t>(a.c.n_pages) * a.c.kv_heads) << a.c.page_log2;
  const uint32_t box = 1 << a.c.page_log2;  // (at most 128: no page is larger)
  if (!encode_row_chunks(&mk, a.c.k, rows, D, box, D / 128) || !encode_row_chunks(&mv, a.c.v, rows, D, box, D / 128))
    return cudaErrorInvalidValue;
  return launch_pdl(kv_tree_few_kernel<D>, dim3(ctas), dim3(kThreads), C::kSmem, s, a, mk, mv);
}

template <int D>
cudaError_t setup() {
  return cudaFuncSetAttribute(kv_tree_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<D>::kSmem);
}

}  // namespace

cudaError_t kv_tree_few_setup() {
  const cudaError_t e = setup<128>();
  return e == cudaSuccess ? setup<256>() : e;
}

cudaError_t launch_kv_tree_few(const KvAttn& a, int ctas, cudaStream_t s) {
  return a.c.head_dim == 128 ? launch<128>(a, ctas, s) : launch<256>(a, ctas, s);
}

}  // namespace moe
