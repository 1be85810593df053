// kv_chunk.cu — attention of chunks of new tokens over the paged cache, on the 5th-generation tensor
// cores (tcgen05).
//
// A row tile is up to 128 (token, query head) rows of one sequence that share a kv head: the group's
// heads of a token lie next to each other, so a tile of keys and values read once serves all of them.
// Its keys fall into tiles of 128 positions. For each:
//   S = Q K^T    128 x 128 x D, operands in shared memory, fp32 accumulator in TMEM (two of them);
//   P = exp2(scaled S - M) by eight warps, written over S in TMEM with 16 bits;
//   O += P V     128 x 128 x (width), P from TMEM, V as it lies in the cache (its width is the
//                contiguous dimension, which the MMA reads transposed), accumulator in TMEM.
// S of the next tile is issued before P V of this one, so the tensor cores work while the softmax does.
// O takes 256 TMEM columns beside the two S, so a head of width 512 is two items that each take
// half of V's width and form S for themselves (1.5 times the products of one pass).
//
// Softmax: one pass in base 2, against a reference M per row that moves (with O and the sum rescaled)
// only when a score passes it by more than 8, so O is almost never read back: P is at most 2^8, summed
// in fp32 and rounded to bf16 (2^-8 of each weight) for the product with V.
//
// Work. An item is a row tile, a kv head and a half of V's width where it has two. The key tiles of all
// items, one after the other with kItemCost more for each item, are shared out evenly over one CTA per
// SM, so that ragged batches, causal triangles and a few rows over a long cache all end together. Items
// cut by the shares leave fp32 pieces (unnormalised output, maximum, sum) that kv_chunk_join_kernel
// adds in the order of the tiles.
//
// Warps: 0 loads K and V by TMA (boxes of one page's rows, 128-byte swizzle), 1 issues the MMAs, 4..11
// are the softmax (two warps per 32 rows, each half the columns) and write the output, 12..15 bring
// the queries into shared memory, gathered by row.
//
// Hidden values. P is 0 for a key a row does not see, but 0 times a NaN or an infinity is not 0, so in
// key tiles with hidden keys the softmax warps clear V's rows that no row of the tile sees, and
// non-finite values that only some rows see; the rows that do see them get them back at the end.
//
// e4m3: S is formed by e4m3 products at twice the rate, each query value being the sum of two e4m3
// numbers (its leading and next four bits; rows are scaled by a power of two to at most 256, so what
// two numbers lose lies 2^-18 below the row's largest magnitude), which needs no widened copy of K.
// The keys' scales multiply S. V's codes are widened to fp16, exactly, by warps 12..15 on the way to
// the tensor cores. The values' scales multiply P before it is rounded to fp16, relative to the
// largest scale so far and 2^7 up: P is then at most 2^15, and what is lost under fp16's smallest
// number is 2^-32 of a weight of 1 per key.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "kv.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 512;
constexpr int kRows = 128;   // rows of a row tile
constexpr int KT = 128;      // positions of a key tile
constexpr int kChunk = 16384;  // 128 rows of 128 bytes
constexpr int kSoftmaxWarp0 = 4, kSoftmaxWarps = 8, kAuxWarp0 = 12, kAuxWarps = 4;
// What an item costs beside its key tiles, in key tiles.
constexpr int kItemCost = 2;

template <int D, bool E4M3>
struct Chk {
  static constexpr int kRow = D * (E4M3 ? 1 : 2);
  static constexpr int DV = D < 256 ? D : 256;            // V's width of an item
  static constexpr int kHalves = D / DV;
  static constexpr int kQBytes = kRows * D * 2;           // bf16, or two e4m3 parts
  static constexpr int kKStages = D / 128;                // stages of a key tile's K
  static constexpr int kVStages = DV / 128;               // and V
  static constexpr int kStage = E4M3 ? kChunk : 2 * kChunk;  // 128 dimensions of 128 rows
  static constexpr int kStages = E4M3 ? (D == 512 ? 2 : D == 256 ? 5 : 6) : (D == 512 ? 3 : D == 256 ? 5 : 6);
  static constexpr int kWide = E4M3 ? (D == 128 ? 3 : 2) : 0;    // stages of widened V, 32 KB each
  static constexpr int kScaleBytes = E4M3 ? 2 * 2 * KT * 4 : 0;
  static constexpr int kBarBytes = 384;
  static constexpr int kSmem = kQBytes + kStages * kStage + kWide * 2 * kChunk + kScaleBytes + kRows * 4 + kBarBytes;
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(8 * (2 * kStages + 2 * kWide + 2 + 2 + 8) + 40 + 64 <= kBarBytes, "barriers");
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
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

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 operands, both K-major, 32 K elements.
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Shared-memory descriptor of V as the transposed operand: rows (keys) of 64 dimensions, 128-byte
// swizzle; eight keys 1024 bytes apart (stride byte offset), the next 64 dimensions one chunk further
// (leading byte offset).
__device__ __forceinline__ uint64_t smem_desc_v(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(kChunk >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// fp32 accumulator; a and b formats of kind::f16 (0 fp16, 1 bf16) or kind::f8f6f4 (0 e4m3).
__host__ __device__ constexpr uint32_t idesc_of(uint32_t format, bool b_transposed, int M, int N) {
  return (1u << 4) | (format << 7) | (format << 10) | (b_transposed ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// The two warps of 32 rows: a barrier, and one with the disjunction of a condition.
__device__ __forceinline__ void pair_sync(int pair) { asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory"); }
__device__ __forceinline__ bool pair_sync_or(int pair, bool c) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbar.red.or.pred q, %2, 64, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(c ? 1 : 0), "r"(1 + pair)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 5, 256;" ::: "memory"); }
__device__ __forceinline__ void aux_sync() { asm volatile("bar.sync 6, 128;" ::: "memory"); }

// ------------------------------------------------------------------ the list of row tiles

// What the tokens [i0, i0 + nt) of a sequence see together.
__device__ __forceinline__ KvRowTile row_tile(const KvAttn& a, int seq, const KvSeq& s, int i0, int tokens) {
  KvRowTile t;
  t.seq = seq;
  t.row0 = s.row0 + i0;
  t.nt = min(tokens, s.n - i0);
  t.p0 = s.len - s.n + i0;
  t.front = t.skip = t.count = 0;
  const int p1 = t.p0 + t.nt - 1;
  if (p1 < 0) return t;
  const KvSpan span = kv_span(max(t.p0, 0), a.window, a.sinks);
  const int first = span.lo / KT;
  t.front = min((span.sinks + KT - 1) / KT, first);
  t.skip = first - t.front;
  t.count = p1 / KT + 1 - t.skip;
  return t;
}

constexpr int kListThreads = 1024;

__device__ long long block_scan(long long v, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += up;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[31];
  return v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

__global__ void __launch_bounds__(kListThreads) kv_chunk_list_kernel(const KvAttn a, int tokens) {
  __shared__ long long sums[32];
  pdl_wait();
  pdl_launch_dependents();
  const KvChunkList& l = a.list;
  long long before = 0, total;
  for (int base = 0; base < a.b.n_seqs; base += kListThreads) {
    const int b = base + threadIdx.x;
    long long n = 0;
    if (b < a.b.n_seqs) n = (kv_sequence(a.b, a.c, b, a.status).n + tokens - 1) / tokens;
    const long long upto = block_scan(n, sums, &total);
    if (b < a.b.n_seqs) l.first_tile[b] = static_cast<int>(min(before + upto - n, 0x7fffffffLL));
    before += total;
  }
  // (More than the list holds only where the sequences' rows overlap, which kv_sequence reports.)
  const int n_tiles = static_cast<int>(min(before, static_cast<long long>(l.max_tiles)));
  __syncthreads();
  before = 0;
  for (int base = 0; base < n_tiles; base += kListThreads) {
    const int e = base + threadIdx.x;
    long long units = 0;
    if (e < n_tiles) {
      int lo = 0, hi = a.b.n_seqs;  // the last sequence with first_tile <= e
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (l.first_tile[mid] <= e) lo = mid;
        else hi = mid;
      }
      const KvRowTile t = row_tile(a, lo, kv_sequence(a.b, a.c, lo, a.status), (e - l.first_tile[lo]) * tokens, tokens);
      l.tiles[e] = t;
      units = t.count > 0 ? t.count + kItemCost : 0;
    }
    const long long upto = block_scan(units, sums, &total);
    if (e < n_tiles) l.first_unit[e] = before + upto - units;
    before += total;
  }
  if (threadIdx.x == 0) {
    l.first_unit[n_tiles] = before;
    *l.n_tiles = n_tiles;
  }
}

// The row tile whose units (times `parts`) hold unit `at`.
__device__ __forceinline__ int find_tile(const KvChunkList& l, int n_tiles, long long at, int parts) {
  int lo = 0, hi = n_tiles;  // the last with first_unit * parts <= at that has units
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (l.first_unit[mid] * parts <= at) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ the attention

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1)
    kv_chunk_kernel(const KvAttn a, int tokens, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v) {
  using C = Chk<D, E4M3>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sq = smem;
  uint8_t* ring = sq + C::kQBytes;
  uint8_t* wide = ring + C::kStages * C::kStage;
  float* scales = reinterpret_cast<float*>(wide + C::kWide * 2 * kChunk);  // [2][2][KT]
  float* exch = scales + C::kScaleBytes / 4;                              // [kRows]
  uint64_t* full = reinterpret_cast<uint64_t*>(exch + kRows);
  uint64_t* empty = full + C::kStages;
  uint64_t* wide_full = empty + C::kStages;
  uint64_t* wide_empty = wide_full + C::kWide;
  uint64_t* s_full = wide_empty + C::kWide;  // [2]
  uint64_t* scale_full = s_full + 2;         // [2]
  uint64_t* p_ready = scale_full + 2;        // [2]: a fast pair of warps may be a tile ahead of a slow one
  uint64_t* o_done = p_ready + 2;
  uint64_t* o_free = o_done + 1;
  uint64_t* q_full = o_free + 1;
  uint64_t* q_free = q_full + 1;
  uint64_t* v_loaded = q_free + 1;
  uint64_t* drain = v_loaded + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* scale_step = reinterpret_cast<float*>(tmem_slot + 2);  // [2] what O is multiplied by before a tile
  float* scale_ref = scale_step + 2;  // [2] what the values' scales of a tile are relative to
  uint32_t* aux_top = tmem_slot + 6;  // [4]
  uint32_t* odd = tmem_slot + 10;     // [2][8] keys with values that were cleared, of alternate items

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((smem_u32(smem) & 1023u) != 0) {  // what the swizzle's address bits and the descriptors rely on
    if (tid == 0) atomicOr(a.status, kStatusBadSchedule);
    return;
  }
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::kWide; ++s) {
      mbar_init(&wide_full[s], kAuxWarps);
      mbar_init(&wide_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&scale_full[s], kAuxWarps);
      mbar_init(&p_ready[s], kSoftmaxWarps);
    }
    mbar_init(o_done, 1);
    mbar_init(o_free, kSoftmaxWarps);
    mbar_init(q_full, kAuxWarps);
    mbar_init(q_free, 1);
    mbar_init(v_loaded, 1);
    mbar_init(drain, 1);
    fence_barrier_init();
    for (int i = 0; i < 16; ++i) odd[i] = 0;
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t why) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    return mbar_wait_bounded(bar, parity, abort_flag, a.status, why);
  };

  const int n_tiles = *a.list.n_tiles;
  const int parts = a.c.kv_heads * C::kHalves;
  const long long total = a.list.first_unit[n_tiles] * parts;
  {  // Rows of no sequence, and of tokens that see nothing.
    const int used = a.b.n_seqs > 0 ? min(max(a.b.cu_q[a.b.n_seqs], 0), a.b.n_tokens) : 0;
    auto clear = [&](long long to) {
      for (int j = 0; j < D; j += 8) *reinterpret_cast<uint4*>(a.out + to * D + j) = make_uint4(0u, 0u, 0u, 0u);
      if (a.lse) a.lse[to] = -INFINITY;
    };
    const long long n = static_cast<long long>(a.b.n_tokens - used) * a.q_heads;
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + tid; i < n; i += static_cast<long long>(gridDim.x) * kThreads)
      clear(static_cast<long long>(used) * a.q_heads + i);
    for (int e = blockIdx.x; e < n_tiles; e += gridDim.x) {
      const KvRowTile t = a.list.tiles[e];
      if (t.count > 0) continue;
      for (int i = tid; i < t.nt * a.q_heads; i += kThreads) clear(static_cast<long long>(t.row0) * a.q_heads + i);
    }
  }
  constexpr int kShare = kItemCost + 1;
  const long long ctas = min(static_cast<long long>(gridDim.x), (total + kShare - 1) / kShare);
  const bool busy = blockIdx.x < ctas;
  const long long begin = busy ? blockIdx.x * total / ctas : 0, end = busy ? (blockIdx.x + 1) * total / ctas : 0;

  // The walk over this CTA's items, the same for every role.
  int entry = 0, part = 0, u0 = 0;
  long long pos = begin;
  KvRowTile t;
  int un = 0, i0 = 0, n = 0;  // of the item: units in the share, first key tile and key tiles
  auto look = [&] {
    const int units = t.count + kItemCost;
    un = static_cast<int>(min(static_cast<long long>(units - u0), end - pos));
    i0 = max(u0 - kItemCost, 0);
    n = max(u0 + un - kItemCost, 0) - i0;
  };
  auto start = [&] {
    if (!busy) return false;
    entry = find_tile(a.list, n_tiles, begin, parts);
    t = a.list.tiles[entry];
    const long long off = begin - a.list.first_unit[entry] * parts;
    part = static_cast<int>(off / (t.count + kItemCost));
    u0 = static_cast<int>(off % (t.count + kItemCost));
    look();
    return n > 0;
  };
  auto next = [&] {
    pos += un;
    if (pos >= end) return false;
    u0 = 0;
    if (++part == parts) {
      part = 0;
      do t = a.list.tiles[++entry];
      while (t.count == 0);
    }
    look();
    return n > 0;
  };
  const int R = 1 << a.c.page_log2;
  // Whether every row of the item sees every key of the tile.
  auto tile_at = [&](int i) { return i < t.front ? i : i + t.skip; };
  auto is_masked = [&](int tile) {
    const int k0 = tile * KT, k1 = k0 + KT - 1, p1 = t.p0 + t.nt - 1;
    return !(k1 <= t.p0 && (a.window == 0 || k0 > p1 - a.window || k1 < a.sinks));
  };
  // The keys that some row of the item sees.
  auto any_sees = [&](int j) {
    const int p1 = t.p0 + t.nt - 1;
    return j <= p1 && (a.window == 0 || j > max(t.p0, 0) - a.window || j < a.sinks);
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    const uint64_t policy = policy_evict_last();
    const int np = KT >> a.c.page_log2;  // pages of a tile
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool alive = true;
    for (bool more = start(); more && alive; more = next()) {
      const int head = part / C::kHalves, half = part % C::kHalves;
      // K of tile 0; then K of tile j + 1 and V of tile j.
      for (int step = 0; step < 2 * n && alive; ++step) {
        const bool is_v = step == 2 * n - 1 || (step > 0 && !(step & 1));
        const int j = is_v ? step / 2 - (step & 1 ? 0 : 1) : (step + 1) / 2;
        const int tile = tile_at(i0 + j);
        const int first = tile * KT + ((lane & (np - 1)) << a.c.page_log2);  // first position of this lane's page
        const bool need = lane < np && first <= t.p0 + t.nt - 1 &&
                          (a.window == 0 || first + R - 1 > max(t.p0, 0) - a.window || first < a.sinks);
        int page = -1;
        if (need) page = kv_page(a.b, a.c, t.seq, first >> a.c.page_log2, a.status);
        const unsigned who = __ballot_sync(0xffffffffu, page >= 0);
        const int row = page < 0 ? 0 : (page * a.c.kv_heads + head) << a.c.page_log2;
        constexpr int kBoxes = C::kStage / kChunk;  // chunks of a stage
        const int from = __shfl_sync(0xffffffffu, row, lane & (np - 1));
        const bool mine = lane < np * kBoxes && ((who >> (lane & (np - 1))) & 1);
        const int chunk = lane / np;
        const int stages = is_v ? C::kVStages : C::kKStages;
        for (int st = 0; st < stages && alive; ++st) {
          if (issued >= C::kStages) {
            bool ok = true;
            if (lane == 0) ok = wait(&empty[stage], phase ^ 1, kStatusWaitEmpty);
            alive = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (!alive) break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&full[stage], __popc(who) * static_cast<uint32_t>(R * 128 * kBoxes));
          __syncwarp();
          if (mine) {
            const int c = (is_v ? half * C::kVStages * kBoxes : 0) + st * kBoxes + chunk;
            asm volatile(
                "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
                " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(
                    smem_u32(ring + stage * C::kStage + chunk * kChunk + ((lane & (np - 1)) << a.c.page_log2) * 128)),
                "l"(reinterpret_cast<uint64_t>(is_v ? &map_v : &map_k)), "r"(0), "r"(from), "r"(c),
                "r"(smem_u32(&full[stage])), "l"(policy)
                : "memory");
          }
          ++issued;
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
    if (!alive && lane == 0) {
      for (int s = 0; s < min(issued, C::kStages); ++s) {
        if (stage == 0) {
          stage = C::kStages;
          phase ^= 1;
        }
        --stage;
        mbar_wait_timeout(&full[stage], phase, 1000000ull, a.status);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs
    if (lane == 0) {
      constexpr uint32_t kIdescS = idesc_of(E4M3 ? 0u : 1u, false, 128, KT);
      constexpr uint32_t kIdescV = idesc_of(E4M3 ? 0u : 1u, true, 128, 128);
      int stage = 0, w_stage = 0, tile_no = 0, item_no = 0;
      uint32_t phase = 0, w_phase = 0;
      bool alive = true;
      auto advance = [&] {
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1;
        }
      };
      auto scores = [&](int no) {  // S of the item's next tile, the CTA's tile `no`
        const uint32_t d = tmem + 256 + (no & 1) * KT;
        for (int st = 0; st < C::kKStages && alive; ++st) {
          alive = wait(&full[stage], phase, kStatusWaitFull);
          if (!alive) break;
          tc_fence_after();
          const uint64_t kb = smem_desc_sw128(smem_u32(ring + stage * C::kStage));
          if constexpr (E4M3) {
#pragma unroll
            for (int piece = 0; piece < 2; ++piece) {
              const uint64_t qb = smem_desc_sw128(smem_u32(sq + (piece * (D / 128) + st) * kChunk));
#pragma unroll
              for (int k = 0; k < 4; ++k) umma_e4m3(d, qb + 2 * k, kb + 2 * k, kIdescS, st > 0 || piece > 0 || k > 0);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint64_t qb = smem_desc_sw128(smem_u32(sq + (2 * st + c) * kChunk));
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_bf16(d, qb + 2 * k, kb + c * (kChunk >> 4) + 2 * k, kIdescS, st > 0 || c > 0 || k > 0);
            }
          }
          umma_commit(&empty[stage]);
          advance();
        }
        if (alive) umma_commit(&s_full[no & 1]);
      };
      for (bool more = start(); more && alive; more = next(), ++item_no) {
        alive = wait(q_full, item_no & 1, kStatusWaitItem);
        if (!alive) break;
        tc_fence_after();
        scores(tile_no);
        for (int j = 0; j < n && alive; ++j, ++tile_no) {
          if (j + 1 < n) scores(tile_no + 1);
          if (j + 1 >= n && alive) umma_commit(q_free);  // the item's last S has read the queries
          if (!alive) break;
          if (j == 0 && item_no > 0) alive = wait(o_free, (item_no - 1) & 1, kStatusWaitAccEmpty);
          if constexpr (!E4M3) {
            // The softmax may have to look at V first, and could not tell an earlier use of the ring's
            // stages from this one.
            for (int st = 0; st < C::kVStages && alive; ++st) {
              const int at = stage + st;
              alive = wait(&full[at < C::kStages ? at : at - C::kStages], at < C::kStages ? phase : phase ^ 1, kStatusWaitFull);
            }
            if (alive) mbar_arrive(v_loaded);
          }
          alive = alive && wait(&p_ready[tile_no & 1], (tile_no >> 1) & 1, kStatusWaitAccFull);
          if (!alive) break;
          tc_fence_after();
          const uint32_t p = tmem + 256 + (tile_no & 1) * KT;
          for (int st = 0; st < C::kVStages && alive; ++st) {
            alive = E4M3 ? wait(&wide_full[w_stage], w_phase, kStatusWaitFull) : wait(&full[stage], phase, kStatusWaitFull);
            if (!alive) break;
            tc_fence_after();
            const uint64_t vb = smem_desc_v(smem_u32(E4M3 ? wide + w_stage * 2 * kChunk : ring + stage * C::kStage));
#pragma unroll
            for (int k = 0; k < KT / 16; ++k)
              umma_bf16_ta(tmem + st * 128, p + 8 * k, vb + k * (2048 >> 4), kIdescV, j > 0 || k > 0);
            if constexpr (E4M3) {
              umma_commit(&wide_empty[w_stage]);
              if (++w_stage == C::kWide) {
                w_stage = 0;
                w_phase ^= 1;
              }
              advance();  // the raw stage, which the widening warps release
            } else {
              umma_commit(&empty[stage]);
              advance();
            }
          }
          if (alive) umma_commit(o_done);
        }
      }
      if (!alive) {
        umma_commit(drain);
        mbar_wait_timeout(drain, 0, 1000000ull, a.status);
      }
    }
  } else if (warp >= kSoftmaxWarp0 && warp < kSoftmaxWarp0 + kSoftmaxWarps) {
    // ---------------------------------------------------------------- softmax and output
    const int quarter = warp & 3, half = (warp - kSoftmaxWarp0) >> 2;  // 32 rows, 64 of the columns
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int r = quarter * 32 + lane;
    const int stid = tid - kSoftmaxWarp0 * 32;
    int tile_no = 0, item_no = 0, stage_no = 0;  // tiles, items and ring stages before this item
    for (bool more = start(); more; more = next(), ++item_no) {
      const int head = part / C::kHalves, vhalf = part % C::kHalves;
      const int tok = r / a.group;
      const bool live = tok < t.nt;
      const int p = live ? t.p0 + tok : -1;
      const int lo = a.window > 0 ? p - a.window + 1 : 0;  // first position in the window
      float qs = a.scale * 1.44269504f;
      if constexpr (E4M3) {
        wait(q_full, item_no & 1, kStatusWaitItem);
        qs *= exch[r];
        pair_sync(quarter);  // exch is used for more below
      }
      float ref = -INFINITY, l = 0.0f, vref = 0.0f;
      // P V of the tile before is complete.
      auto wait_pv = [&] {
        if (tile_no > 0) wait(o_done, (tile_no - 1) & 1, kStatusWaitAccFull);
      };
      for (int j = 0; j < n; ++j, ++tile_no) {
        const int tile = tile_at(i0 + j);
        const bool masked = is_masked(tile);
        const float* sk = scales + (tile_no & 1) * 2 * KT + half * 64;
        wait(&s_full[tile_no & 1], (tile_no >> 1) & 1, kStatusWaitAccFull);
        tc_fence_after();
        const uint32_t s_at = tmem + lanes + 256 + (tile_no & 1) * KT;
        float y[64];
        {
          uint32_t b0[32], b1[32];
          tmem_ld32_nowait(s_at + half * 64, b0);
          tmem_ld32_nowait(s_at + half * 64 + 32, b1);
          tmem_wait_ld();
          reg_fence32(b0);
          reg_fence32(b1);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            y[i] = __uint_as_float(b0[i]);
            y[32 + i] = __uint_as_float(b1[i]);
          }
        }
        float step = 1.0f;
        if constexpr (E4M3) {
          wait(&scale_full[tile_no & 1], (tile_no >> 1) & 1, kStatusWaitFull);
          step = scale_step[tile_no & 1];
          vref = scale_ref[tile_no & 1];
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(sk + i);
            y[i] *= f.x;
            y[i + 1] *= f.y;
            y[i + 2] *= f.z;
            y[i + 3] *= f.w;
          }
        }
        if (masked) {
          const int k0 = tile * KT + half * 64;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (k0 + i > p || (k0 + i < lo && k0 + i >= a.sinks)) y[i] = -INFINITY;
        }
        float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          top0 = fmaxf(top0, fmaxf(y[i], y[i + 1]));
          top1 = fmaxf(top1, fmaxf(y[i + 2], y[i + 3]));
        }
        // (A row scale that is NaN makes no maximum.)
        float top = fmaxf(top0, top1) * qs;
        if (pair_sync_or(quarter, top > ref + 8.0f || step != 1.0f)) {
          // The reference moves to the maximum so far, of both halves.
          if (half == 1) exch[r] = top;
          pair_sync(quarter);
          if (half == 0) {
            top = fmaxf(top, exch[r]);
            exch[r] = top;
          }
          pair_sync(quarter);
          top = fmaxf(ref, exch[r]);
          const float f = exp2_approx(ref - (top == -INFINITY ? 0.0f : top));
          ref = top;
          l *= f;
          if (j > 0) {
            const float of = f * step;
            wait_pv();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < C::DV / 2; c += 32) {
              uint32_t o[32];
              const uint32_t at = tmem + lanes + half * (C::DV / 2) + c;
              tmem_ld32_nowait(at, o);
              tmem_wait_ld();
              reg_fence32(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * of);
              tmem_st32(at, o);
            }
            tmem_wait_st();
          }
        }
        const float base = ref == -INFINITY ? 0.0f : ref;
        float sum0 = 0.0f, sum1 = 0.0f;
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float e0 = exp2_approx(fmaf(y[2 * i], qs, -base)), e1 = exp2_approx(fmaf(y[2 * i + 1], qs, -base));
          sum0 += e0;
          sum1 += e1;
          if constexpr (E4M3) {
            const float2 v = *reinterpret_cast<const float2*>(sk + KT + 2 * i);
            if (masked) {  // a hidden key's scale may be anything
              e0 = e0 == 0.0f ? 0.0f : e0 * v.x;
              e1 = e1 == 0.0f ? 0.0f : e1 * v.y;
            } else {
              e0 *= v.x;
              e1 *= v.y;
            }
            w[i] = pack_f16(e0, e1);
          } else {
            w[i] = pack_bf16(e0, e1);
          }
        }
        l += sum0 + sum1;
        tmem_st32(s_at + half * 32, w);
        if constexpr (!E4M3) {
          if (masked) {
            // V's rows that no row sees, and non-finite values that only some rows see.
            const int p1 = t.p0 + t.nt - 1;
            wait_pv();  // (the barrier's phase of the tile before is over)
            wait(v_loaded, tile_no & 1, kStatusWaitFull);
            const int v_no = stage_no + min(j + 2, n) * C::kKStages + j * C::kVStages;
            for (int st = 0; st < C::kVStages; ++st) {
              const int sno = v_no + st;
              wait(&full[sno % C::kStages], (sno / C::kStages) & 1, kStatusWaitFull);
              uint8_t* v = ring + sno % C::kStages * C::kStage;
              for (int i = stid; i < C::kStage / 16; i += kSoftmaxWarps * 32) {
                const int key = tile * KT + ((i >> 3) & (KT - 1));
                const bool all = key <= t.p0 && (a.window == 0 || key > p1 - a.window || key < a.sinks);
                if (all) continue;
                uint4* at = reinterpret_cast<uint4*>(v) + i;
                if (!any_sees(key)) {
                  *at = make_uint4(0u, 0u, 0u, 0u);
                  continue;
                }
                const uint4 x = *at;
                uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                bool found = false;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  if ((xs[q] & 0x7f80u) == 0x7f80u) xs[q] &= 0xffff0000u, found = true;
                  if ((xs[q] & 0x7f800000u) == 0x7f800000u) xs[q] &= 0xffffu, found = true;
                }
                if (found) {
                  *at = make_uint4(xs[0], xs[1], xs[2], xs[3]);
                  // Keys only some rows see: after the first token, or leaving the first tokens' windows.
                  const int bit = key > t.p0 ? key - t.p0 - 1 : 128 + key - (max(t.p0, 0) - a.window + 1);
                  atomicOr(&odd[(item_no & 1) * 8 + (bit >> 5)], 1u << (bit & 31));
                }
              }
            }
            fence_proxy_async_shared();
          }
        }
        wait_pv();  // a barrier's phases are told apart by their parity: none may be passed over
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[tile_no & 1]);
      }
      stage_no += n * (C::kKStages + C::kVStages);

      // The item's output: its row sums, then O.
      pair_sync(quarter);  // (exch may still be read for the last tile's reference)
      if (half == 1) exch[r] = l;
      pair_sync(quarter);
      if (half == 0) {
        l += exch[r];
        exch[r] = l;
      }
      pair_sync(quarter);
      l = exch[r];
      if constexpr (!E4M3) {
        if (stid < 8) odd[((item_no + 1) & 1) * 8 + stid] = 0;
      }
      wait(o_done, (tile_no - 1) & 1, kStatusWaitAccFull);
      tc_fence_after();
      softmax_sync();
      uint32_t cleared = 0;
      if constexpr (!E4M3) {
        for (int i = 0; i < 8; ++i) cleared |= odd[(item_no & 1) * 8 + i];
      }
      const bool whole = i0 == 0 && n == t.count;
      float vs = 1.0f;
      if constexpr (E4M3) vs = vref * 0.0078125f;
      const float f = whole ? (l == 0.0f ? 0.0f : vs / l) : vs;
      const long long row = static_cast<long long>(t.row0 + tok) * a.q_heads + head * a.group + r % a.group;
      const long long item_start = pos - u0;
      // A piece's place: this CTA's first if the item began before the CTA's share or with it.
      float* piece = a.chunk_partial + (2LL * blockIdx.x + (begin >= item_start ? 0 : 1)) * kChunkPieceFloats;
#pragma unroll 1
      for (int c = 0; c < C::DV / 2; c += 32) {
        uint32_t o[32];
        const int col = half * (C::DV / 2) + c;
        tmem_ld32_nowait(tmem + lanes + col, o);
        tmem_wait_ld();
        reg_fence32(o);
        if constexpr (!E4M3) {
          if (cleared) {
            for (int b = 0; b < 256; ++b) {
              if (!(odd[(item_no & 1) * 8 + (b >> 5)] >> (b & 31) & 1)) continue;
              const int key = b < 128 ? t.p0 + 1 + b : max(t.p0, 0) - a.window + 1 + b - 128;
              if (key > p || (key < lo && key >= a.sinks)) continue;
              const int page = kv_page(a.b, a.c, t.seq, key >> a.c.page_log2, a.status);
              if (page < 0) continue;
              const uint16_t* v = reinterpret_cast<const uint16_t*>(a.c.v) +
                                  ((((static_cast<long long>(page) * a.c.kv_heads + head) << a.c.page_log2) + (key & (R - 1))) * D +
                                   vhalf * C::DV + col);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const uint32_t x = static_cast<uint32_t>(v[i]) << 16;
                if ((x & 0x7f800000u) == 0x7f800000u) o[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(x));
              }
            }
          }
        }
        if (whole) {
          if (live) {
            uint4* to = reinterpret_cast<uint4*>(a.out + row * D + vhalf * C::DV + col);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              to[i] = make_uint4(pack_bf16(__uint_as_float(o[8 * i]) * f, __uint_as_float(o[8 * i + 1]) * f),
                                 pack_bf16(__uint_as_float(o[8 * i + 2]) * f, __uint_as_float(o[8 * i + 3]) * f),
                                 pack_bf16(__uint_as_float(o[8 * i + 4]) * f, __uint_as_float(o[8 * i + 5]) * f),
                                 pack_bf16(__uint_as_float(o[8 * i + 6]) * f, __uint_as_float(o[8 * i + 7]) * f));
          }
        } else if (live) {
          float4* to = reinterpret_cast<float4*>(piece + r * C::DV + col);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            to[i] = make_float4(__uint_as_float(o[4 * i]) * f, __uint_as_float(o[4 * i + 1]) * f,
                                __uint_as_float(o[4 * i + 2]) * f, __uint_as_float(o[4 * i + 3]) * f);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
      if (half == 0) {
        if (!whole) {
          piece[kRows * 256 + r] = ref;
          piece[kRows * 257 + r] = l;
        } else if (live && a.lse && vhalf == 0) {
          a.lse[row] = l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.693147181f;
        }
      }
    }
  } else if (warp >= kAuxWarp0) {
    // ---------------------------------------------------------------- queries; e4m3: V and the scales
    const int awarp = warp - kAuxWarp0;
    int item_no = 0;
    for (bool more = start(); more; more = next(), ++item_no) {
      const int head = part / C::kHalves;
      if (item_no > 0) wait(q_free, (item_no - 1) & 1, kStatusWaitEmpty);
      // A warp takes 32 rows, four at a time; a lane 16 bytes of a row and every 512 bytes on.
      constexpr int kVecs = D / 8 < 32 ? 1 : D / 256;            // 16-byte vectors of a row per lane
      constexpr int kLanes = D / 8 < 32 ? D / 8 : 32;            // lanes of a row
      constexpr int kRowsAtOnce = 32 / kLanes;
      constexpr int kBatch = 8 / kVecs;
#pragma unroll 1
      for (int g = 0; g < 32; g += kBatch * kRowsAtOnce) {
        uint4 x[kBatch][kVecs];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int r = awarp * 32 + g + b * kRowsAtOnce + lane / kLanes;
          const int tok = r / a.group;
#pragma unroll
          for (int v = 0; v < kVecs; ++v) {
            x[b][v] = make_uint4(0u, 0u, 0u, 0u);
            if (tok < t.nt)
              x[b][v] = *reinterpret_cast<const uint4*>(a.q.ptr + static_cast<long long>(t.row0 + tok) * a.q.token_stride +
                                                        (head * a.group + r % a.group) * a.q.head_stride +
                                                        (lane % kLanes + v * 32) * 8);
          }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int r = awarp * 32 + g + b * kRowsAtOnce + lane / kLanes;
          const uint32_t swz = (r & 7) << 4;
#pragma unroll
          for (int v = 0; v < kVecs; ++v) {
            const uint32_t byte = (lane % kLanes + v * 32) * 16;
            *reinterpret_cast<uint4*>(sq + (byte >> 7) * kChunk + r * 128 + ((byte & 127) ^ swz)) = x[b][v];
          }
        }
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ joining an item's pieces

// A block for each place where a share begins (x) and each 8 rows: if that is the first cut in an item,
// a warp joins a row of the item's pieces.
template <int D>
__global__ void __launch_bounds__(256) kv_chunk_join_kernel(const KvAttn a, int tokens, int grid) {
  constexpr int DV = D < 256 ? D : 256, kHalves = D / DV;
  pdl_wait();
  pdl_launch_dependents();
  const int n_tiles = *a.list.n_tiles;
  const int parts = a.c.kv_heads * kHalves;
  const long long total = a.list.first_unit[n_tiles] * parts;
  constexpr int kShare = kItemCost + 1;
  const long long ctas = min(static_cast<long long>(grid), (total + kShare - 1) / kShare);
  const long long x = blockIdx.x + 1;
  if (x >= ctas) return;
  const long long cut = x * total / ctas;
  const int entry = find_tile(a.list, n_tiles, cut, parts);
  const KvRowTile t = a.list.tiles[entry];
  const int units = t.count + kItemCost;
  const long long off = cut - a.list.first_unit[entry] * parts;
  const int part = static_cast<int>(off / units);
  const long long item_start = cut - off % units;
  // The CTAs with the item's first and last key tiles.
  const long long first = ((item_start + kItemCost + 1) * ctas - 1) / total;
  const long long last = ((item_start + units) * ctas - 1) / total;
  if (first == last || first + 1 != x) return;
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int tok = r / a.group;
  if (tok >= t.nt) return;
  auto place = [&](long long c) {
    return a.chunk_partial + (2 * c + (c > first || c * total / ctas >= item_start ? 0 : 1)) * kChunkPieceFloats;
  };
  float top = -INFINITY;
  for (long long c = first; c <= last; ++c) top = fmaxf(top, __ldcg(place(c) + kRows * 256 + r));
  const float base = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  float4 acc[DV / 128];
#pragma unroll
  for (int v = 0; v < DV / 128; ++v) acc[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (long long c = first; c <= last; ++c) {
    const float* from = place(c);
    const float w = exp2_approx(__ldcg(from + kRows * 256 + r) - base);
    sum = fmaf(w, __ldcg(from + kRows * 257 + r), sum);
#pragma unroll
    for (int v = 0; v < DV / 128; ++v) {
      const float4 y = __ldcg(reinterpret_cast<const float4*>(from + r * DV + v * 128 + lane * 4));
      acc[v].x = fmaf(w, y.x, acc[v].x);
      acc[v].y = fmaf(w, y.y, acc[v].y);
      acc[v].z = fmaf(w, y.z, acc[v].z);
      acc[v].w = fmaf(w, y.w, acc[v].w);
    }
  }
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
  const long long row = static_cast<long long>(t.row0 + tok) * a.q_heads + part / kHalves * a.group + r % a.group;
#pragma unroll
  for (int v = 0; v < DV / 128; ++v)
    *reinterpret_cast<uint2*>(a.out + row * D + part % kHalves * DV + v * 128 + lane * 4) =
        make_uint2(pack_bf16(acc[v].x * f, acc[v].y * f), pack_bf16(acc[v].z * f, acc[v].w * f));
  if (a.lse && lane == 0 && part % kHalves == 0)
    a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.693147181f;
}

template <int D, bool E4M3>
cudaError_t launch(const KvAttn& a, int ctas, cudaStream_t s) {
  using C = Chk<D, E4M3>;
  CUtensorMap mk, mv;
  const uint64_t rows = (static_cast<uint64_t>(a.c.n_pages) * a.c.kv_heads) << a.c.page_log2;
  const uint32_t box = 1u << a.c.page_log2;
  if (!encode_row_chunks(&mk, a.c.k, rows, C::kRow, box, 1) || !encode_row_chunks(&mv, a.c.v, rows, C::kRow, box, 1))
    return cudaErrorInvalidValue;
  const int tokens = chunk_tokens(a.group);
  cudaError_t e = launch_pdl(kv_chunk_list_kernel, dim3(1), dim3(kListThreads), 0, s, a, tokens);
  if (e == cudaSuccess) e = launch_pdl(kv_chunk_kernel<D, E4M3>, dim3(ctas), dim3(kThreads), C::kSmem, s, a, tokens, mk, mv);
  if (e == cudaSuccess && ctas > 1)
    e = launch_pdl(kv_chunk_join_kernel<D>, dim3(ctas - 1, kRows / 8), dim3(256), 0, s, a, tokens, ctas);
  return e;
}

template <int D, bool E4M3>
cudaError_t setup() {
  return cudaFuncSetAttribute(kv_chunk_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, Chk<D, E4M3>::kSmem);
}

}  // namespace

cudaError_t kv_chunk_setup() {
  cudaError_t e = setup<128, false>();
  if (e == cudaSuccess) e = setup<256, false>();
  if (e == cudaSuccess) e = setup<512, false>();
  return e;
}

cudaError_t launch_kv_chunk(const KvAttn& a, int ctas, cudaStream_t s) {
  switch (a.c.head_dim) {
    case 128: return launch<128, false>(a, ctas, s);
    case 256: return launch<256, false>(a, ctas, s);
    default: return launch<512, false>(a, ctas, s);
  }
}

}  // namespace moe
