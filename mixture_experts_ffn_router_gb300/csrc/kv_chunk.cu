// kv_chunk.cu — attention of chunks of new tokens over the paged cache, on the 5th-generation tensor
// cores (tcgen05).
//
// A row tile is up to 256 (token, query head) rows of one sequence that share a kv head: the group's
// heads of a token lie next to each other, so a tile of keys and values read once serves all of them.
// A cluster of two CTAs works on it as an SM pair (cta_group::2), 128 rows each; a key tile, 128
// positions, is loaded by halves: each CTA holds 64 keys of K and half of the width of V, so the pair
// reads it once, and a ring of the same shared memory holds twice the tiles. For each key tile:
//   S = Q K^T    256 x 128 x D, operands in shared memory, fp32 accumulator in TMEM (two of them);
//   P = exp2(scaled S - M) by eight warps of each CTA, written over S in TMEM with 16 bits;
//   O += P V     256 x (width) x 128, P from TMEM, V as it lies in the cache (its width is the
//                contiguous dimension, which the MMA reads transposed), accumulator in TMEM.
// S of the next tile is issued before P V of this one, so the tensor cores work while the softmax does.
// O takes 256 TMEM columns beside the two S, so a head of width 512 is two items that each take
// half of V's width and form S for themselves (1.5 times the products of one pass).
//
// Softmax: one pass in base 2 (M. Milakov and N. Gimelshein, "Online normalizer calculation for softmax", 2018),
// against a reference M per row instead of the running maximum. M moves, with O and the sum rescaled, only
// when half a row's weights in a tile sum to more than 2^9, so O is almost never read back and no maximum
// is taken: weights are at most 2^9, summed in fp32 and rounded to bf16 (half a step is 2^-8 of each) for
// the product with V.
//
// Work. An item is a row tile, a kv head and a half of V's width where it has two. The key tiles of all
// items, one after the other with item_cost more for each item, are shared out evenly over the pairs
// of SMs, so that ragged batches, causal triangles and a few rows over a long cache all end together. Items
// cut by the shares leave fp32 pieces (unnormalised output, maximum, sum) that kv_chunk_join_kernel
// adds in the order of the tiles.
//
// Warps: 0 loads K and V by TMA (boxes of one page's rows, 128-byte swizzle), 1 issues the MMAs (in the
// pair's first CTA), 4..11 are the softmax (two warps per 32 rows, each half the columns), 12..15 bring
// the queries into shared memory, gathered by row, and write an item's output while the next one is under
// way. What the MMA thread waits for is counted on barriers of the first CTA, which the other's warps and
// copies reach over the cluster.
//
// What bounds it. Prompts of 4096 tokens, 16 heads on 8: width 256 1.54 PFLOP/s, width 512 1.14 (1.71 with
// the second S), of 1.91 measured for a burst and 1.72 sustained; at these the power limit holds the
// clock. A key tile takes about 2400 cycles where its products are 2048 (width 256): the softmax's chain,
// from S to P, is nearly as long. Width 128 (products 1024) and e4m3, whose softmax multiplies by two
// scales per key and shares its SM's issue slots with the widening, are bound by that chain: about 1800, and
// 2400 and 3200 (e4m3, widths 128 and 256). Much of the chain is instructions on their way: see wait_slow.
// Measured and not kept: the softmax warps in two groups that take turns at whole tiles (width 256 430 us
// against 376, with two S to work from a group's turn waits for the other's products), V looked through by
// warps 12..15 (385), S loaded before what else there is to know of the tile (width 128 293 against 283), more
// registers for the softmax by setmaxnreg (width 256 1% less, width 512 5% more, e4m3 3% more).
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
// largest scale so far and 2^6 up: P is then at most 2^15, and what is lost under fp16's smallest
// number is 2^-31 of a weight of 1 per key of that scale. (A NaN among the codes, which moe_ffn_kv_write does not make,
// may reach rows that do not see it; a NaN scale does not.)
//
// Scales far apart. A reference that all rows of an item share would take the values of a row that does not
// see the largest scale (or hardly weighs it) out of fp16. So where an item's scales span more than kFarScales,
// zeros among them, its further tiles go through far_weights: P = exp2(s + log2(scale) - R) with a reference R
// per row, over the keys that the row sees, rounded to bf16 (as over a bf16 cache, half a step is 2^-8), which
// holds 2^-133 of the largest term; V's codes are widened to bf16 there, exactly too. Up to there a shared
// reference loses at most 2^-19 per key of the row's largest term.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "kv.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 512;
constexpr int kRows = 128;   // rows of a row tile in a CTA
constexpr int KT = 128;      // positions of a key tile
constexpr int kHalfKeys = 64;  // of which a CTA holds the keys of 64
constexpr int kChunk = 16384;  // 128 rows of 128 bytes
constexpr int kSoftmaxWarp0 = 4, kSoftmaxWarps = 8, kAuxWarp0 = 12, kAuxWarps = 4;

template <int D, bool E4M3>
struct Chk {
  static constexpr int kRow = D * (E4M3 ? 1 : 2);
  static constexpr int DV = D < 256 ? D : 256;            // V's width of an item
  static constexpr int kHalves = D / DV;
  static constexpr int kQBytes = kRows * D * 2;           // bf16, or two e4m3 parts
  // K: stages of up to two chunks of 64 rows of 128 bytes.
  static constexpr int kKChunks = kRow == 128 || (E4M3 && D == 512) ? 1 : 2;
  static constexpr int kKStage = kKChunks * kHalfKeys * 128;
  static constexpr int kKTile = kRow / 128 / kKChunks;    // stages of a key tile
  static constexpr int NK = E4M3 ? (D == 128 ? 6 : D == 256 ? 3 : 5) : (D == 512 ? 4 : 6);
  // V: 128 rows of this CTA's half of the width, a slot for a key tile. bf16: chunks of 64 dimensions;
  // e4m3: rows of codes, as they lie where they are narrower than 128 bytes, and slots of widened ones.
  static constexpr int kVTile = DV / 128;                 // chunks of 64 dimensions
  static constexpr int kVBytes = E4M3 ? DV / 2 : 128;     // bytes of a loaded row (of a chunk)
  static constexpr int kVLoads = E4M3 ? 1 : kVTile;
  static constexpr int kVSlot = kVLoads * KT * kVBytes;
  static constexpr int kWSlot = kVTile * kChunk;
  static constexpr int NV = E4M3 ? (D == 128 ? 4 : D == 256 ? 2 : 1) : (D == 512 ? 1 : D == 256 ? 2 : 6);
  static constexpr int NW = E4M3 ? (D == 128 ? 4 : D == 256 ? 2 : 1) : 0;
  // Of a thread's pieces of V to widen, those unrolled: prompts of 1500 to 4100 tokens take 210 us with 1
  // and 213 with 4 at width 128 (fewer instructions to fetch), but 291 and 279 at width 256, 687 and 672 at 512.
  static constexpr int kWUnroll = D == 128 ? 1 : 4;
  static constexpr int kScaleBytes = E4M3 ? 2 * 2 * KT * 4 : 0;
  static constexpr int kBarBytes = (8 * (2 * NK + 2 * NV + 2 * NW + 18) + 32 + (E4M3 ? 48 : 96) + 15) / 16 * 16;
  static constexpr int kSmem =
      kQBytes + NK * kKStage + NV * kVSlot + NW * kWSlot + kScaleBytes + (E4M3 ? 5 : 4) * kRows * 4 + (E4M3 ? 2 * kRows : 0) + kBarBytes;
  static_assert(kSmem <= 232448, "shared memory");
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// To 2^-22 of the result, or outside (1/2, 2) of its size: 2^-15 of a weight at the ends of the range.
__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 numbers in a register pair, and operations on both at once.
__device__ __forceinline__ unsigned long long two(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(unsigned long long v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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

// The MMA warp issues with all its lanes together, one of them elected per instruction: what the
// instructions take (descriptors, addresses) then stays in uniform registers. Under a branch on the
// lane, moving it there for every instruction took about 100 cycles where an MMA takes 64.

// D (both CTAs' TMEM) (+)= A * B^T, A and B in shared memory, K-major: 16 K elements of bf16, or 32 of e4m3.
template <bool E4M3>
__device__ __forceinline__ void umma_pair_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  if constexpr (E4M3) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// The same over 16 K elements of 16 bits, A in each CTA's TMEM.
__device__ __forceinline__ void umma_ta_pair_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                   uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives on `bar` of both CTAs when the MMAs issued before have completed.
__device__ __forceinline__ void commit_pair_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// A box of one 128-byte (or narrower) chunk of rows into this CTA's shared memory, counted on the
// barrier at shared::cluster address `bar`, which may be the other CTA's.
__device__ __forceinline__ void tma_rows_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int row,
                                              int chunk) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(chunk), "r"(bar)
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

// Whether the phase of the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// The lowest n bits, of all n below 0 or above 64 too.
__device__ __forceinline__ unsigned long long low_bits(int n) {
  return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull;
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
// Arrives on a barrier at a shared::cluster address. What the arrival announces lies in this CTA's own
// TMEM and shared memory, for its own tensor core, so nothing is released to the cluster: with
// .release.cluster the arrival took 1200 cycles of a key tile's 3500.
__device__ __forceinline__ void arrive_at(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// Sets bits at a shared::cluster address.
__device__ __forceinline__ void or_shared(uint32_t addr, uint32_t bits) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(bits) : "memory");
}

// Warps 12..15: the same two.
__device__ __forceinline__ void aux_sync() { asm volatile("bar.sync 6, 128;" ::: "memory"); }
__device__ __forceinline__ bool aux_sync_or(bool c) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbar.red.or.pred q, 6, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(c ? 1 : 0)
      : "memory");
  return r != 0;
}

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

__global__ void __launch_bounds__(kListThreads) kv_chunk_list_kernel(const KvAttn a, int tokens, int parts, int max_pairs) {
  constexpr int kNear = 1024;  // row tiles whose first units are at hand in shared memory
  __shared__ long long near_unit[kNear];
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
      units = t.count > 0 ? t.count + a.item_cost : 0;
    }
    const long long upto = block_scan(units, sums, &total);
    if (e < n_tiles) l.first_unit[e] = before + upto - units;
    if (e < min(n_tiles, kNear)) near_unit[e] = before + upto - units;
    before += total;
  }
  if (threadIdx.x == 0) *l.n_tiles = n_tiles;
  __syncthreads();
  // Where each pair's share begins, and the item it begins in if others have part in it: the first cut in
  // an item stands for the item's join.
  const int x = threadIdx.x;
  if (x >= max_pairs) return;
  const long long all = before * parts;
  const int share = a.item_cost + 1;
  const long long pairs = min(static_cast<long long>(max_pairs), (all + share - 1) / share);
  KvShare s = {};
  KvJoin j = {};
  if (x < pairs) {
    s.begin = x * all / pairs;
    s.end = (x + 1) * all / pairs;
    int lo = 0, hi = n_tiles;  // the last row tile with first unit * parts <= begin
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if ((mid < kNear ? near_unit[mid] : l.first_unit[mid]) * parts <= s.begin) lo = mid;
      else hi = mid;
    }
    const KvRowTile t = l.tiles[lo];
    const int units = t.count + a.item_cost;
    const long long off = s.begin - (lo < kNear ? near_unit[lo] : l.first_unit[lo]) * parts;
    s.entry = lo;
    s.part = static_cast<int>(off / units);
    s.u0 = static_cast<int>(off % units);
    const long long item_start = s.begin - s.u0;
    const long long first = ((item_start + share) * pairs - 1) / all, last = ((item_start + units) * pairs - 1) / all;
    if (first + 1 == x && last > first) {
      j.row0 = t.row0;
      j.nt = t.nt;
      j.part = s.part;
      j.first = static_cast<int>(first);
      j.count = static_cast<int>(last - first) + 1;
      j.first_place = 2 * j.first + (first * all / pairs >= item_start ? 0 : 1);
    }
  }
  l.shares[x] = s;
  l.joins[x] = j;
}

// ------------------------------------------------------------------ the attention

// mbar_wait_bounded out of line. Inlined, the loops of the kernel's many waits lay between the instructions
// that every tile executes, and fetching those cost 5 to 8%: prompts of 4096 tokens of width 128 took 285 us
// instead of 270, 2048 rows of width 512 on 16384 tokens 975 instead of 897. (The branches that few tiles
// take are marked for the same reason.)
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* status, uint32_t why) {
  if (*abort) return false;
  return mbar_wait_bounded(bar, parity, abort, status, why);
}

// The weights of a tile whose values' scales are far from others of the item (e4m3): as the kernel's own code
// for a tile's weights, with a reference of the row's own for P, in base 2 like the scores, that moves when a
// term passes it by more than 2^15 and then leaves the largest term at 2^7. The maximum moves in every such tile.
// Few caches have such tiles: what is theirs lies out of line and takes its time (one prompt of 4096 tokens,
// 16 heads on 8 of width 256: 281 us with a large scale at its start, 147 without; to find out costs the others
// 0 to 2.5%).
constexpr float kFarScales = 4096.0f;

struct FarRow {
  float ref, l;  // maximum of the scores, and this half row's sum
  float vref;    // reference of P
};

// s_at, o_at: TMEM of the row's S (and P) and of this half of its O; sk: this half's key scales, the values'
// scales' logarithms KT further.
template <int kCols>
__device__ __noinline__ FarRow far_weights(FarRow row, uint32_t s_at, uint32_t o_at, const float* sk, unsigned long long seen,
                                           float qs, float* top_at, float* vtop_at, int half, int quarter, bool first) {
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
  // (The scales of hidden keys may be anything; what becomes of -inf and a logarithm of infinity or NaN makes no
  // maximum.)
  float top = -INFINITY, vtop = -INFINITY;
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    y[i] = seen >> i & 1ull ? y[i] * sk[i] * qs : -INFINITY;
    top = fmaxf(top, y[i]);
    vtop = fmaxf(vtop, y[i] + sk[KT + i]);
  }
  if (half == 1) {
    *top_at = top;
    *vtop_at = vtop;
  }
  pair_sync(quarter);
  if (half == 0) {
    *top_at = fmaxf(top, *top_at);
    *vtop_at = fmaxf(vtop, *vtop_at);
  }
  pair_sync(quarter);
  top = fmaxf(row.ref, *top_at);
  vtop = *vtop_at;
  pair_sync(quarter);  // (the next tile's may follow)
  const float base = top == -INFINITY ? 0.0f : top;
  row.l *= exp2_approx(row.ref - base);
  row.ref = top;
  const bool move = vtop > row.vref + 15.0f;
  const float vref = move ? vtop - 7.0f : row.vref;
  const float vbase = vref == -INFINITY ? 0.0f : vref;
  if (!first && __any_sync(0xffffffffu, move)) {
    const float f = move ? exp2_approx(row.vref - vbase) : 1.0f;
#pragma unroll 1
    for (int c = 0; c < kCols; c += 32) {
      uint32_t o[32];
      tmem_ld32_nowait(o_at + c, o);
      tmem_wait_ld();
      reg_fence32(o);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
      tmem_st32(o_at + c, o);
    }
  }
  row.vref = vref;
  float sum = 0.0f;
  uint32_t w[32];
#pragma unroll
  for (int i = 0; i < 64; i += 2) {
    sum += exp2_approx(y[i] - base) + exp2_approx(y[i + 1] - base);
    w[i / 2] = pack_bf16(exp2_approx(y[i] + sk[KT + i] - vbase), exp2_approx(y[i + 1] + sk[KT + i + 1] - vbase));
    const uint32_t bits = static_cast<uint32_t>(seen >> i) & 3u;
    w[i / 2] &= (bits & 1u ? 0xffffu : 0u) | (bits & 2u ? 0xffff0000u : 0u);
  }
  row.l += sum;
  tmem_st32(s_at + half * 32, w);
  return row;
}

// A widened tile's values from fp16 to bf16, by warps 12..15.
__device__ __noinline__ void far_values(uint32_t* w, int pairs) {
  aux_sync();
  for (int i = threadIdx.x - kAuxWarp0 * 32; i < pairs; i += kAuxWarps * 32) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(w + i));
    w[i] = pack_bf16(f.x, f.y);
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1)
    kv_chunk_kernel(const KvAttn a, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v) {
  using C = Chk<D, E4M3>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sq = smem;
  uint8_t* k_ring = sq + C::kQBytes;
  uint8_t* v_ring = k_ring + C::NK * C::kKStage;
  uint8_t* w_ring = v_ring + C::NV * C::kVSlot;
  float* scales = reinterpret_cast<float*>(w_ring + C::NW * C::kWSlot);  // [2][2][KT]
  float* exch = scales + C::kScaleBytes / 4;                          // [kRows] maxima of a tile
  float* row_sums = exch + kRows;  // [kRows] an item's sums
  float* vexch = row_sums + kRows;  // [kRows] (e4m3) as exch, with the values' scales
  float* fin = vexch + (E4M3 ? kRows : 0);  // [2][kRows] what an item's O is multiplied by, of alternate items
  uint8_t* q_exp = reinterpret_cast<uint8_t*>(fin + 2 * kRows);          // [2][kRows] (e4m3), of alternate items
  uint64_t* full_k = reinterpret_cast<uint64_t*>(q_exp + (E4M3 ? 2 * kRows : 0));  // first CTA's: both CTAs' keys
  uint64_t* empty_k = full_k + C::NK;
  uint64_t* full_v = empty_k + C::NK;    // this CTA's part
  uint64_t* empty_v = full_v + C::NV;
  uint64_t* full_w = empty_v + C::NV;
  uint64_t* empty_w = full_w + C::NW;
  uint64_t* s_full = empty_w + C::NW;    // [2]
  uint64_t* scale_full = s_full + 2;     // [2]
  uint64_t* scale_free = scale_full + 2;  // [2]
  uint64_t* p_ready = scale_free + 2;    // [2], first CTA's: a fast pair of warps may be a tile ahead of a slow one
  uint64_t* o_done = p_ready + 2;
  uint64_t* o_free = o_done + 1;         // first CTA's
  uint64_t* q_full = o_free + 1;         // first CTA's
  uint64_t* q_free = q_full + 1;
  uint64_t* q_scaled = q_free + 1;       // [2]: the softmax may be an item behind the queries
  uint64_t* o_full = q_scaled + 2;       // an item's last P V is complete
  uint64_t* fin_full = o_full + 1;       // [2]
  uint64_t* drain = fin_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* scale_step = reinterpret_cast<float*>(tmem_slot + 2);  // [2] what O is multiplied by before a tile
  float* scale_ref = scale_step + 2;  // [2] what the values' scales of a tile are relative to; 0: far apart
  uint32_t* aux_top = tmem_slot + 8;  // [2][4] (at a multiple of 16 bytes), the tile's largest scale by warps
  uint32_t* w_far = aux_top + 8;      // [NW] whether a widened tile is bf16
  uint32_t* odd = aux_top;            // [3][8] (bf16) keys with values that either CTA cleared, of items in turn

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  // What the swizzle's address bits and the descriptors rely on (the same in both CTAs).
  const bool aligned = (smem_u32(smem) & 1023u) == 0;
  if (!aligned) {
    if (tid == 0) atomicOr(a.status, kStatusBadSchedule);
    return;
  }
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < C::NK; ++s) {
      mbar_init(&full_k[s], 1);
      mbar_init(&empty_k[s], 1);
    }
    for (int s = 0; s < C::NV; ++s) {
      mbar_init(&full_v[s], 1);
      mbar_init(&empty_v[s], E4M3 ? kAuxWarps : 1);
    }
    for (int s = 0; s < C::NW; ++s) {
      mbar_init(&full_w[s], kAuxWarps);
      mbar_init(&empty_w[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&scale_full[s], kAuxWarps);
      mbar_init(&scale_free[s], kSoftmaxWarps);
      mbar_init(&q_scaled[s], kAuxWarps);
      mbar_init(&p_ready[s], 2 * kSoftmaxWarps);
    }
    mbar_init(o_done, 1);
    mbar_init(o_free, 2 * kAuxWarps);
    mbar_init(o_full, 1);
    mbar_init(&fin_full[0], kSoftmaxWarps / 2);
    mbar_init(&fin_full[1], kSoftmaxWarps / 2);
    mbar_init(q_full, 2 * kAuxWarps);
    mbar_init(q_free, 1);
    mbar_init(drain, 1);
    fence_barrier_init_cluster();
    for (int i = 0; i < (E4M3 ? 8 : 24); ++i) odd[i] = 0;
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  // Waits that have to wait look at the CTA's flag first, so that all of them end soon after one has given up.
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t why) {
    if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
    return wait_slow(bar, parity, abort_flag, a.status, why);
  };
  auto arrive_first = [&](uint64_t* bar) { arrive_at(mapa_shared(smem_u32(bar), 0)); };

  const int n_tiles = *a.list.n_tiles;
  const int parts = a.c.kv_heads * C::kHalves;
  {  // Rows of no sequence, and of tokens that see nothing.
    const KvNoRows none = kv_no_rows(a.b);
    auto clear = [&](long long to) {
      for (int j = 0; j < D; j += 8) *reinterpret_cast<uint4*>(a.out + to * D + j) = make_uint4(0u, 0u, 0u, 0u);
      if (a.lse) a.lse[to] = -INFINITY;
    };
    const long long before = static_cast<long long>(none.before) * a.q_heads;
    const long long n = before + static_cast<long long>(a.b.n_tokens - none.after) * a.q_heads;
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + tid; i < n; i += static_cast<long long>(gridDim.x) * kThreads)
      clear(i < before ? i : static_cast<long long>(none.after) * a.q_heads + i - before);
    for (int e = blockIdx.x; e < n_tiles; e += gridDim.x) {
      const KvRowTile t = a.list.tiles[e];
      if (t.count > 0) continue;
      for (int i = tid; i < t.nt * a.q_heads; i += kThreads) clear(static_cast<long long>(t.row0) * a.q_heads + i);
    }
  }
  const int me = blockIdx.x / 2;
  const KvShare my_share = a.list.shares[me];
  const long long begin = my_share.begin, end = my_share.end;

  // The walk over this pair's items, the same for every role.
  int entry = 0, part = 0, u0 = 0;
  long long pos = begin;
  KvRowTile t;
  int un = 0, i0 = 0, n = 0;  // of the item: units in the share, first key tile and key tiles
  auto look = [&] {
    const int units = t.count + a.item_cost;
    un = static_cast<int>(min(static_cast<long long>(units - u0), end - pos));
    i0 = max(u0 - a.item_cost, 0);
    n = max(u0 + un - a.item_cost, 0) - i0;
  };
  auto start = [&] {
    if (begin >= end) return false;
    entry = my_share.entry;
    part = my_share.part;
    u0 = my_share.u0;
    t = a.list.tiles[entry];
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
  // An item's piece: this pair's first if the item began before the pair's share or with it.
  auto piece_of = [&](long long item_start) {
    return a.chunk_partial + (2LL * me + (begin >= item_start ? 0 : 1)) * kChunkPieceFloats;
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

  // Adds the values that were cleared of V (bf16) back to 32 columns of the row of the token at p.
  auto put_back = [&](const KvRowTile& it, int head, int col, int p, int no, uint32_t (&o)[32]) {
    const int p1 = it.p0 + it.nt - 1, lo = a.window > 0 ? p - a.window + 1 : 0;
    // Each set bit stands for up to two keys; a key that every row of the tile sees was not cleared.
    for (int b = 0; b < 512; ++b) {
      if (!(odd[no % 3 * 8 + ((b & 255) >> 5)] >> (b & 31) & 1)) continue;
      const int key = b < 256 ? it.p0 + 1 + b : max(it.p0, 0) - a.window + 1 + b - 256;
      if (b >= 256 && (a.window == 0 || key > it.p0)) continue;
      if (key < 0 || key > p || (key < lo && key >= a.sinks)) continue;
      if (key <= it.p0 && (a.window == 0 || key > p1 - a.window || key < a.sinks)) continue;
      const int page = kv_page(a.b, a.c, it.seq, key >> a.c.page_log2, a.status);
      if (page < 0) continue;
      const uint16_t* v =
          reinterpret_cast<const uint16_t*>(a.c.v) +
          ((((static_cast<long long>(page) * a.c.kv_heads + head) << a.c.page_log2) + (key & (R - 1))) * D + col);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const uint32_t x = static_cast<uint32_t>(v[i]) << 16;
        if ((x & 0x7f800000u) == 0x7f800000u) o[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(x));
      }
    }
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    // Boxes are one page's rows, or 64 of them: lane i holds the cache row of the tile's box i (and of
    // box i - boxes, ...). A tile's page ids are fetched a tile ahead, and serve its K and then its V.
    const int rows_log2 = min(a.c.page_log2, 6);
    const int boxes = KT >> rows_log2;
    const int box = lane & (boxes - 1);
    const int own = boxes / 2;  // boxes of this CTA's keys
    const int chunk = lane / boxes;
    const bool k_lane = box / own == static_cast<int>(rank) && chunk < C::kKChunks, v_lane = lane < boxes;
    const uint32_t full_k0 = mapa_shared(smem_u32(&full_k[0]), 0);
    const uint32_t k_to = smem_u32(k_ring) + chunk * (kHalfKeys * 128) + (((box % own) << rows_log2) * 128);
    const uint32_t v_to = smem_u32(v_ring) + (box << rows_log2) * C::kVBytes;
    int ks = 0, vs = 0, k_issued = 0, v_issued = 0;
    uint32_t k_phase = 0, v_phase = 0;
    bool alive = true;
    struct Boxes {
      int row;       // of this lane's box
      unsigned who;  // boxes to load
    };
    for (bool more = start(); more && alive; more = next()) {
      const int head = part / C::kHalves, half = part % C::kHalves;
      // The position a box begins at, -1 if no row sees any of it, and the page table's entry of it.
      auto fetch = [&](int j, int& first) {
        first = j < n ? tile_at(i0 + j) * KT + (box << rows_log2) : 0x7fffffff;
        const bool need = first <= t.p0 + t.nt - 1 &&
                          (a.window == 0 || first + (1 << rows_log2) - 1 > max(t.p0, 0) - a.window || first < a.sinks);
        if (!need) first = -1;
        return need ? a.b.pages[t.seq * a.b.pages_stride + (first >> a.c.page_log2)] : -1;
      };
      auto boxes_of = [&](int page, int first) {
        const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(a.c.n_pages);
        if (first >= 0 && !ok) atomicOr(a.status, kStatusBadIndex);
        Boxes o;
        o.who = __ballot_sync(0xffffffffu, ok) & ((1u << boxes) - 1);
        o.row = ok ? ((page * a.c.kv_heads + head) << a.c.page_log2) + (first & (R - 1)) : 0;
        return o;
      };
      int first;
      int page = fetch(0, first);
      Boxes cur = boxes_of(page, first), last = cur;
      page = fetch(1, first);
      // K of tile 0; then K of tile j + 1 and V of tile j.
      for (int j = -1; j < n && alive; ++j) {
        if (j + 1 < n) {
          if (j >= 0) {
            last = cur;
            cur = boxes_of(page, first);
            page = fetch(j + 2, first);
          }
          const bool mine = k_lane && ((cur.who >> box) & 1);
          const uint32_t bytes = __popc(cur.who) * static_cast<uint32_t>((128 << rows_log2) * C::kKChunks);
          for (int st = 0; st < C::kKTile && alive; ++st) {
            if (k_issued >= C::NK) alive = __all_sync(0xffffffffu, wait(&empty_k[ks], k_phase ^ 1, kStatusWaitEmpty));
            if (!alive) break;
            if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&full_k[ks], bytes);
            __syncwarp();
            if (mine) tma_rows_pair(k_to + ks * C::kKStage, &map_k, full_k0 + 8u * ks, 0, cur.row, st * C::kKChunks + chunk);
            ++k_issued;
            if (++ks == C::NK) {
              ks = 0;
              k_phase ^= 1;
            }
          }
        } else {
          last = cur;
        }
        if (j < 0 || !alive) continue;
        if (v_issued >= C::NV) alive = __all_sync(0xffffffffu, wait(&empty_v[vs], v_phase ^ 1, kStatusWaitEmpty));
        if (!alive) break;
        if (lane == 0)
          mbar_arrive_expect_tx(&full_v[vs], __popc(last.who) * static_cast<uint32_t>((C::kVBytes << rows_log2) * C::kVLoads));
        __syncwarp();
        if (v_lane && ((last.who >> box) & 1)) {
          // The CTA's half of the item's width begins at this byte of the row.
          const int byte = (half * C::DV + static_cast<int>(rank) * (C::DV / 2)) * (E4M3 ? 1 : 2);
          const uint32_t bar = mapa_shared(smem_u32(&full_v[vs]), rank);
#pragma unroll
          for (int c = 0; c < C::kVLoads; ++c)
            tma_rows_pair(v_to + vs * C::kVSlot + c * kChunk, &map_v, bar, byte & 127, last.row, (byte >> 7) + c);
        }
        ++v_issued;
        if (++vs == C::NV) {
          vs = 0;
          v_phase ^= 1;
        }
      }
    }
    if (!alive && lane == 0) {
      // Given up: the copies on their way land before the CTA's shared memory goes.
      for (int s = 0; s < min(v_issued, C::NV); ++s) {
        if (vs == 0) {
          vs = C::NV;
          v_phase ^= 1;
        }
        --vs;
        mbar_wait_timeout(&full_v[vs], v_phase, 1000000ull, a.status);
      }
      for (int s = 0; rank == 0 && s < min(k_issued, C::NK); ++s) {
        if (ks == 0) {
          ks = C::NK;
          k_phase ^= 1;
        }
        --ks;
        mbar_wait_timeout(&full_k[ks], k_phase, 1000000ull, a.status);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs
    if (rank == 0) {
      constexpr uint32_t kIdescS = idesc_of(E4M3 ? 0u : 1u, false, 256, KT);
      constexpr uint32_t kIdescV = idesc_of(E4M3 ? 0u : 1u, true, 256, C::DV);
      constexpr uint32_t kIdescFar = idesc_of(1u, true, 256, C::DV);
      constexpr int NVW = E4M3 ? C::NW : C::NV;
      uint8_t* const v_chunks = E4M3 ? w_ring : v_ring;
      uint64_t* const v_empty = E4M3 ? empty_w : empty_v;
      auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
      int ks = 0, vs = 0, tile_no = 0, item_no = 0;
      uint32_t k_phase = 0;
      bool alive = true;
      auto wait_all = [&](uint64_t* bar, uint32_t parity, uint32_t why) {
        alive = uniform(wait(bar, parity, why) ? 1 : 0) != 0 && alive;
        return alive;
      };
      auto scores = [&](int no) {  // S of the item's next tile, the pair's tile `no`
        const uint32_t d = tm + 256 + (uniform(no) & 1) * KT;
        for (int st = 0; st < C::kKTile; ++st) {
          if (!wait_all(&full_k[ks], k_phase, kStatusWaitFull)) return;
          tc_fence_after();
          const int u = uniform(ks);
          const uint64_t kb = smem_desc_sw128(smem_u32(k_ring) + u * C::kKStage);
#pragma unroll
          for (int c = 0; c < C::kKChunks; ++c) {
#pragma unroll
            for (int piece = 0; piece < (E4M3 ? 2 : 1); ++piece) {
              const uint64_t qb = smem_desc_sw128(smem_u32(sq) + (piece * (C::kRow / 128) + st * C::kKChunks + c) * kChunk);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_pair_elect<E4M3>(d, qb + 2 * k, kb + c * (kHalfKeys * 128 >> 4) + 2 * k, kIdescS,
                                      st > 0 || c > 0 || piece > 0 || k > 0);
            }
          }
          commit_pair_elect(&empty_k[u]);
          if (++ks == C::NK) {
            ks = 0;
            k_phase ^= 1;
          }
        }
        commit_pair_elect(&s_full[no & 1]);
      };
      for (bool more = start(); more && alive; more = next(), ++item_no) {
        const int tiles = uniform(n);
        if (!wait_all(q_full, item_no & 1, kStatusWaitItem)) break;
        tc_fence_after();
        for (int j = -1; j < tiles && alive; ++j) {
          if (j + 1 < tiles) scores(tile_no + (j < 0 ? 0 : 1));
          if (!alive) break;
          if (j < 0) continue;
          if (j + 1 >= tiles) commit_pair_elect(q_free);  // the item's last S has read the queries
          if (j == 0 && item_no > 0) wait_all(o_free, (item_no - 1) & 1, kStatusWaitAccEmpty);
          // (The softmax has seen V's arrival.)
          if (!alive || !wait_all(&p_ready[tile_no & 1], (tile_no >> 1) & 1, kStatusWaitAccFull)) break;
          tc_fence_after();
          const uint32_t p = tm + 256 + (uniform(tile_no) & 1) * KT;
          const int u = uniform(vs);
          const uint64_t vb = smem_desc_v(smem_u32(v_chunks) + u * (E4M3 ? C::kWSlot : C::kVSlot));
          const uint32_t add = uniform(j > 0 ? 1 : 0);
          uint32_t idesc = kIdescV;
          if constexpr (E4M3) {
            if (__builtin_expect(__any_sync(0xffffffffu, w_far[vs] != 0), 0)) idesc = kIdescFar;
          }
#pragma unroll
          for (int k = 0; k < KT / 16; ++k)
            umma_ta_pair_elect(tm, p + 8 * k, vb + k * (2048 >> 4), idesc, k > 0 ? 1u : add);
          commit_pair_elect(&v_empty[u]);
          if (++vs == NVW) vs = 0;
          commit_pair_elect(o_done);
          if (j + 1 >= tiles) commit_pair_elect(o_full);
          ++tile_no;
        }
      }
      if (!alive) {
        commit_pair_elect(drain);
        mbar_wait_timeout(drain, 0, 1000000ull, a.status);
      }
    }
  } else if (warp >= kSoftmaxWarp0 && warp < kSoftmaxWarp0 + kSoftmaxWarps) {
    // ---------------------------------------------------------------- softmax and output
    const int quarter = warp & 3, half = (warp - kSoftmaxWarp0) >> 2;  // 32 rows, 64 of the columns
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int r = quarter * 32 + lane;              // row of the CTA
    const int rr = static_cast<int>(rank) * kRows + r;  // and of the pair
    const int stid = tid - kSoftmaxWarp0 * 32;
    uint64_t* const v_full = E4M3 ? full_w : full_v;
    constexpr int NVW = E4M3 ? C::NW : C::NV;
    int tile_no = 0, item_no = 0, vs = 0;
    uint32_t v_phase = 0;
    for (bool more = start(); more; more = next(), ++item_no) {
      const int head = part / C::kHalves, vhalf = part % C::kHalves;
      const int tok = rr / a.group;
      const bool live = tok < t.nt;
      const int p = live ? t.p0 + tok : -1;
      const int lo = a.window > 0 ? p - a.window + 1 : 0;  // first position in the window
      float qs = a.scale * 1.44269504f;
      if constexpr (E4M3) {
        // The power of two that the row was multiplied by (a NaN for a row with one).
        wait(&q_scaled[item_no & 1], (item_no >> 1) & 1, kStatusWaitItem);
        const int e = q_exp[(item_no & 1) * kRows + r];
        if (p >= 0) qs = e == 255 ? __uint_as_float(0x7fffffffu) : qs / __uint_as_float(static_cast<uint32_t>(e) << 23);
      }
      float ref = -INFINITY, l = 0.0f;
      float vref = 0.0f;  // what the values' scales are relative to
      bool far = false;
      // P V of the tile before is complete.
      auto wait_pv = [&] {
        if (tile_no > 0) wait(o_done, (tile_no - 1) & 1, kStatusWaitAccFull);
      };
      int j = 0;
      for (; j < n; ++j, ++tile_no) {
        const int tile = tile_at(i0 + j);
        const bool masked = is_masked(tile);
        const float* sk = scales + (tile_no & 1) * 2 * KT + half * 64;
        wait(&s_full[tile_no & 1], (tile_no >> 1) & 1, kStatusWaitAccFull);
        tc_fence_after();
        float step = 1.0f;
        if constexpr (E4M3) {
          wait(&scale_full[tile_no & 1], (tile_no >> 1) & 1, kStatusWaitFull);
          step = scale_step[tile_no & 1];
          const float now = scale_ref[tile_no & 1];
          if (__builtin_expect(now == 0.0f, 0)) {
            far = true;
            break;
          }
          vref = now;
        }
        // What the end of the tile waits for has mostly happened by now.
        const bool v_here = mbar_test(&v_full[vs], v_phase), pv_done = tile_no == 0 || mbar_test(o_done, (tile_no - 1) & 1);
        const uint32_t s_at = tmem + lanes + 256 + (tile_no & 1) * KT;
        // The keys of this half that the row sees, by bits.
        unsigned long long seen = ~0ull;
        if (__builtin_expect(masked, 0)) {
          const int k0 = tile * KT + half * 64;
          seen = low_bits(p + 1 - k0) & ~(low_bits(lo - k0) & ~low_bits(a.sinks - k0));
        }
        bool move = j == 0 || step != 1.0f;  // the reference is to move
        uint32_t w[32];
        float sum;
        for (;;) {
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
          if constexpr (E4M3) {
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
              const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(sk + i);
              split(mul2(two(y[i], y[i + 1]), f.x), y[i], y[i + 1]);
              split(mul2(two(y[i + 2], y[i + 3]), f.y), y[i + 2], y[i + 3]);
            }
          }
          if (__builtin_expect(masked, 0)) {
            const uint32_t s0 = static_cast<uint32_t>(seen), s1 = static_cast<uint32_t>(seen >> 32);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (!(s0 >> i & 1u)) y[i] = -INFINITY;
              if (!(s1 >> i & 1u)) y[32 + i] = -INFINITY;
            }
          }
          if (__builtin_expect(move, 0)) {
            // The reference moves to the maximum so far, of both halves. (A row scale that is NaN makes no
            // maximum.)
            float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
              top0 = fmaxf(top0, fmaxf(y[i], y[i + 1]));
              top1 = fmaxf(top1, fmaxf(y[i + 2], y[i + 3]));
            }
            float top = fmaxf(top0, top1) * qs;
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
            step = 1.0f;
          }
          // A reference of -inf (nothing but hidden keys and NaN so far) counts as 0.
          const float base = ref == -INFINITY ? 0.0f : ref;
          const unsigned long long qs2 = two(qs, qs), base2 = two(-base, -base);
          unsigned long long sum2 = 0ull, sum3 = 0ull;  // two zeros each
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float e[4];
            split(fma2(two(y[2 * i], y[2 * i + 1]), qs2, base2), e[0], e[1]);
            split(fma2(two(y[2 * i + 2], y[2 * i + 3]), qs2, base2), e[2], e[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) e[k] = exp2_approx(e[k]);
            sum2 = add2(sum2, two(e[0], e[1]));
            sum3 = add2(sum3, two(e[2], e[3]));
            if constexpr (E4M3) {
              const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sk + KT + 2 * i);
              split(mul2(two(e[0], e[1]), v.x), e[0], e[1]);
              split(mul2(two(e[2], e[3]), v.y), e[2], e[3]);
              w[i] = pack_f16(e[0], e[1]);
              w[i + 1] = pack_f16(e[2], e[3]);
            } else {
              w[i] = pack_bf16(e[0], e[1]);
              w[i + 1] = pack_bf16(e[2], e[3]);
            }
          }
          float sums[4];
          split(sum2, sums[0], sums[1]);
          split(sum3, sums[2], sums[3]);
          sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
          // No weight is above the half row's sum, so a sum of at most 2^9 is all there is to check, once the
          // row has a reference (its first tiles may have shown it nothing). One move is enough.
          if (__builtin_expect(!pair_sync_or(quarter, !move && (sum > 512.0f || (ref == -INFINITY && seen != 0))), 1)) break;
          move = true;
        }
        l += sum;
        if constexpr (E4M3) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&scale_free[tile_no & 1]);
          if (__builtin_expect(masked, 0)) {
            // (A hidden key's scale may have been anything.)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const uint32_t bits = static_cast<uint32_t>(seen >> (2 * i)) & 3u;
              w[i] &= (bits & 1u ? 0xffffu : 0u) | (bits & 2u ? 0xffff0000u : 0u);
            }
          }
        }
        tmem_st32(s_at + half * 32, w);
        // V of this tile has arrived (what the MMA thread knows of it, it knows from here).
        if (__builtin_expect(!v_here, 0)) wait(&v_full[vs], v_phase, kStatusWaitFull);
        if constexpr (!E4M3) {
          if (__builtin_expect(masked, 0)) {
            // V's rows that no row sees, and non-finite values that only some rows see.
            const int p1 = t.p0 + t.nt - 1;
            // A thread's vectors are the same 16 bytes of four keys, in each chunk.
            uint4* v = reinterpret_cast<uint4*>(v_ring + vs * C::kVSlot) + stid;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const int key = tile * KT + (stid >> 3) + 32 * m;
              const bool all = key <= t.p0 && (a.window == 0 || key > p1 - a.window || key < a.sinks);
              if (all) continue;
              const bool none = !any_sees(key);
#pragma unroll
              for (int c = 0; c < C::kVTile; ++c) {
                uint4* at = v + m * 256 + c * (kChunk / 16);
                if (none) {
                  *at = make_uint4(0u, 0u, 0u, 0u);
                  continue;
                }
                const uint4 x = *at;
                // Whether some exponent is all ones: a carry out of its field after adding one to it.
                const uint32_t even = ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
                                      ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
                if ((even & 0x80008000u) == 0) continue;
                uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  if ((xs[q] & 0x7f80u) == 0x7f80u) xs[q] &= 0xffff0000u;
                  if ((xs[q] & 0x7f800000u) == 0x7f800000u) xs[q] &= 0xffffu;
                }
                *at = make_uint4(xs[0], xs[1], xs[2], xs[3]);
                // The pair's row tile has up to 256 tokens; keys only some of them see lie after the first
                // token, or leave the first tokens' windows: 256 bits by the distance, of either kind.
                const int bit = (key > t.p0 ? key - t.p0 - 1 : key - (max(t.p0, 0) - a.window + 1)) & 255;
                const uint32_t to = smem_u32(&odd[item_no % 3 * 8 + (bit >> 5)]), mark = 1u << (bit & 31);
                or_shared(mapa_shared(to, 0), mark);
                or_shared(mapa_shared(to, 1), mark);
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
              }
            }
            fence_proxy_async_shared();
          }
        }
        if (++vs == NVW) {
          vs = 0;
          v_phase ^= 1;
        }
        if (__builtin_expect(!pv_done, 0)) wait_pv();  // a barrier's phases are told apart by their parity: none may be passed over
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&p_ready[tile_no & 1]);
      }
      if constexpr (E4M3) {
        if (__builtin_expect(far, 0)) {
          // The tiles from the first whose scales are far from others on. The reference of P is the same number
          // until it moves.
          FarRow row = {ref, l, j == 0 || ref == -INFINITY ? -INFINITY : ref + log2f(vref) - 6.0f};
#pragma unroll 1
          for (; j < n; ++j, ++tile_no) {
            wait(&s_full[tile_no & 1], (tile_no >> 1) & 1, kStatusWaitAccFull);
            wait(&scale_full[tile_no & 1], (tile_no >> 1) & 1, kStatusWaitFull);
            wait_pv();
            tc_fence_after();
            const int k0 = tile_at(i0 + j) * KT + half * 64;
            const unsigned long long seen = low_bits(p + 1 - k0) & ~(low_bits(lo - k0) & ~low_bits(a.sinks - k0));
            row = far_weights<C::DV / 2>(row, tmem + lanes + 256 + (tile_no & 1) * KT, tmem + lanes + half * (C::DV / 2),
                                         scales + (tile_no & 1) * 2 * KT + half * 64, seen, qs, &exch[r], &vexch[r], half,
                                         quarter, j == 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&scale_free[tile_no & 1]);
            wait(&v_full[vs], v_phase, kStatusWaitFull);
            if (++vs == NVW) {
              vs = 0;
              v_phase ^= 1;
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_first(&p_ready[tile_no & 1]);
          }
          ref = row.ref;
          l = row.l;
          vref = row.vref == -INFINITY || ref == -INFINITY ? 64.0f : 64.0f * exp2f(row.vref - ref);
        }
      }

      // The rows' sums, and what the output is multiplied by; warps 12..15 write it.
      // One half's sum goes to the other through words of its own: in exch the next item's first maximum could
      // follow it before it is read. (It has been read before the next sum comes: each of an item's tiles
      // has a barrier.)
      if (half == 1) row_sums[r] = l;
      pair_sync(quarter);
      if (half == 0) {
        l += row_sums[r];
        const bool whole = i0 == 0 && n == t.count;
        float vs_f = 1.0f;
        if constexpr (E4M3) vs_f = vref * 0.015625f;
        fin[(item_no & 1) * kRows + r] = whole ? (l == 0.0f ? 0.0f : vs_f / l) : vs_f;
        __syncwarp();
        if (lane == 0) mbar_arrive(&fin_full[item_no & 1]);
        if (!whole) {
          float* piece = piece_of(pos - u0);
          piece[256 * 256 + rr] = ref;
          piece[256 * 257 + rr] = l;
        } else if (live && a.lse && vhalf == 0) {
          a.lse[static_cast<long long>(t.row0 + tok) * a.q_heads + head * a.group + rr % a.group] =
              l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.693147181f;
        }
      }
    }
  } else if (warp >= kAuxWarp0) {
    // ---------------------------------------------------------------- queries; e4m3: V and the scales
    const int awarp = warp - kAuxWarp0;
    int item_no = 0, tile_no = 0, vs = 0, ws = 0;
    uint32_t v_phase = 0, w_phase = 0;

    // The output of item `no`: lane by lane a row, 32 columns at a time.
    auto output = [&](const KvRowTile& it, int it_part, bool whole, long long item_start, int no) {
      const int head = it_part / C::kHalves, vhalf = it_part % C::kHalves;
      const int r = awarp * 32 + lane, rr = static_cast<int>(rank) * kRows + r;
      const int tok = rr / a.group;
      const bool live = tok < it.nt;
      const uint32_t at = tmem + (static_cast<uint32_t>(awarp * 32) << 16);
      const unsigned long long own =
          !live ? 0ull
          : whole
              ? reinterpret_cast<unsigned long long>(
                    a.out + (static_cast<long long>(it.row0 + tok) * a.q_heads + head * a.group + rr % a.group) * D + vhalf * C::DV)
              : reinterpret_cast<unsigned long long>(piece_of(item_start) + rr * C::DV);
      // Four lanes trade their rows' pieces, so that a store writes 64 bytes of a row from neighbouring
      // lanes (lane i of the four has piece i of each of their rows): a lane writing its own row alone
      // touches 32 lines per instruction, and took three times as long.
      unsigned long long to[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) to[k] = __shfl_sync(0xffffffffu, own, (lane & ~3) + k);
      auto trade = [&](uint32_t (&w)[16]) {
#pragma unroll
        for (int d = 1; d <= 2; d <<= 1) {
          const bool up = lane & d;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k & d) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t &lo_w = w[4 * k + i], &hi_w = w[4 * (k | d) + i];
              const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo_w : hi_w, d);
              if (up) lo_w = got;
              else hi_w = got;
            }
          }
        }
      };
      if constexpr (!E4M3) {
        // The marks of the item after the next (the softmax of either CTA may be in the next one already):
        // the last output is done with them, and that item is reached only through this one's o_free.
        aux_sync();
        if (awarp == 0 && lane < 8) odd[(no + 2) % 3 * 8 + lane] = 0;
        __syncwarp();
      }
      wait(&fin_full[no & 1], (no >> 1) & 1, kStatusWaitAccFull);
      const float f = fin[(no & 1) * kRows + r];
      wait(o_full, no & 1, kStatusWaitAccFull);
      tc_fence_after();
      uint32_t cleared = 0;
      if constexpr (!E4M3) {
        for (int i = 0; i < 8; ++i) cleared |= odd[no % 3 * 8 + i];
      }
#pragma unroll 1
      for (int col = 0; col < C::DV; col += 32) {
        uint32_t o[32];
        tmem_ld32_nowait(at + col, o);
        tmem_wait_ld();
        reg_fence32(o);
        if (col + 32 == C::DV) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_first(o_free);
        }
        if constexpr (!E4M3) {
          if (cleared && live) put_back(it, head, vhalf * C::DV + col, it.p0 + tok, no, o);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        if (whole) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack_bf16(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
          trade(w);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (to[k])
              *reinterpret_cast<uint4*>(to[k] + col * 2 + (lane & 3) * 16) =
                  make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = o[16 * h + i];
            trade(w);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (to[k])
                *reinterpret_cast<uint4*>(to[k] + (col + 16 * h) * 4 + (lane & 3) * 16) =
                    make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
          }
        }
      }
    };
    KvRowTile was = {};
    int was_part = 0;
    bool was_whole = false;
    long long was_start = 0;
    for (bool more = start(); more; more = next(), ++item_no) {
      const int head = part / C::kHalves;
      // e4m3: this thread's key of the item's tiles. Its page id is fetched two tiles ahead, its scales one.
      const int key = awarp * 32 + lane;
      auto page_of = [&](int j) {
        const int at = j < n ? tile_at(i0 + j) * KT + key : 0;
        return j < n && any_sees(at) ? a.b.pages[t.seq * a.b.pages_stride + (at >> a.c.page_log2)] : -1;
      };
      auto scales_of = [&](int j, int page) {
        float2 s = make_float2(0.0f, 0.0f);
        if (static_cast<unsigned>(page) < static_cast<unsigned>(a.c.n_pages)) {
          const int at = tile_at(i0 + j) * KT + key;
          const long long i = ((static_cast<long long>(page) * a.c.kv_heads + head) << a.c.page_log2) + (at & (R - 1));
          s = make_float2(a.c.k_scale[i], a.c.v_scale[i]);
        }
        return s;
      };
      int next_page = -1;
      float2 next_scales = make_float2(0.0f, 0.0f);
      bool next_seen = false;
      if constexpr (E4M3) {
        const int page = page_of(0);
        next_page = page_of(1);
        next_scales = scales_of(0, page);
        next_seen = page >= 0;
      }
      if (item_no > 0) wait(q_free, (item_no - 1) & 1, kStatusWaitEmpty);
      // A warp brings 32 rows; each lane knows where one of them is, or that there is none.
      constexpr int kVecs = D / 8 < 32 ? 1 : D / 256;            // 16-byte vectors of a row per lane
      constexpr int kLanes = D / 8 < 32 ? D / 8 : 32;            // lanes of a row
      constexpr int kRowsAtOnce = 32 / kLanes;
      const int rr = static_cast<int>(rank) * kRows + awarp * 32 + lane, tok = rr / a.group;
      const unsigned long long own_row =
          tok >= t.nt ? 0ull
                      : reinterpret_cast<unsigned long long>(a.q.ptr + static_cast<long long>(t.row0 + tok) * a.q.token_stride +
                                                             (head * a.group + rr % a.group) * a.q.head_stride);
      // Where 16 bytes of a row lie.
      auto place = [&](int r, int v) {
        const uint32_t byte = (lane % kLanes + v * 32) * 16;
        return (byte >> 7) * kChunk + r * 128 + ((byte & 127) ^ ((r & 7) << 4));
      };
#pragma unroll 8
      for (int g = 0; g < 32; g += kRowsAtOnce) {
        const unsigned long long from = __shfl_sync(0xffffffffu, own_row, g + lane / kLanes);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
          // (A row that is none reads nothing and leaves zeros; any address will do.)
          const unsigned long long at =
              from ? from + (lane % kLanes + v * 32) * 16 : reinterpret_cast<unsigned long long>(a.q.ptr);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           smem_u32(sq) + place(awarp * 32 + g + lane / kLanes, v)),
                       "l"(at), "r"(from ? 16 : 0)
                       : "memory");
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if constexpr (E4M3) {
        // A row's two parts take the place of its values: the warp that brought it reads it, then writes them.
        // (Through registers, eight rows at a time, each with a wait of its own for L2, an item cost 6 key
        // tiles instead of 4.)
        __syncwarp();
        constexpr int kBatch = 2 / kVecs;
#pragma unroll 1
        for (int g = 0; g < 32; g += kBatch * kRowsAtOnce) {
          uint4 x[kBatch][kVecs];
#pragma unroll
          for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
              x[b][v] = *reinterpret_cast<const uint4*>(sq + place(awarp * 32 + g + b * kRowsAtOnce + lane / kLanes, v));
          __syncwarp();
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int r = awarp * 32 + g + b * kRowsAtOnce + lane / kLanes;
            const uint32_t swz = (r & 7) << 4;
            // A power of two that brings the row's largest magnitude into [128, 256).
            uint32_t two_tops = 0;
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
              const uint32_t u[4] = {x[b][v].x, x[b][v].y, x[b][v].z, x[b][v].w};
#pragma unroll
              for (int q = 0; q < 4; ++q) two_tops = __vmaxu2(two_tops, u[q] & 0x7fff7fffu);
            }
            uint32_t top = max(two_tops << 16, two_tops & 0xffff0000u);
            if constexpr (kLanes == 32) {
              top = __reduce_max_sync(0xffffffffu, top);
            } else {
#pragma unroll
              for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
            const int e = static_cast<int>(top >> 23), up_exp = e == 255 ? 255 : min(261 - e, 254);
            const float up = e == 255 ? 1.0f : __uint_as_float(static_cast<uint32_t>(up_exp) << 23);
            if (lane % kLanes == 0) q_exp[(item_no & 1) * kRows + r] = static_cast<uint8_t>(up_exp);
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
              const uint32_t u[4] = {x[b][v].x, x[b][v].y, x[b][v].z, x[b][v].w};
              uint32_t hi[2], lo[2];
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                float f[4] = {__uint_as_float(u[2 * q] << 16) * up, __uint_as_float(u[2 * q] & 0xffff0000u) * up,
                              __uint_as_float(u[2 * q + 1] << 16) * up, __uint_as_float(u[2 * q + 1] & 0xffff0000u) * up};
                hi[q] = e4m3_part(f);
                lo[q] = e4m3_part(f);
              }
              const uint32_t byte = (lane % kLanes + v * 32) * 8;
              uint8_t* to = sq + (byte >> 7) * kChunk + r * 128 + ((byte & 127) ^ swz);
              *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
              *reinterpret_cast<uint2*>(to + (C::kRow / 128) * kChunk) = make_uint2(lo[0], lo[1]);
            }
          }
        }
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        arrive_first(q_full);
        if (E4M3) mbar_arrive(&q_scaled[item_no & 1]);
      }
      // The item before is written once this one's queries (and first V) are on their way.
      auto output_last = [&] {
        if (item_no > 0) output(was, was_part, was_whole, was_start, item_no - 1);
        was = t;
        was_part = part;
        was_whole = i0 == 0 && n == t.count;
        was_start = pos - u0;
      };
      if constexpr (!E4M3) output_last();
      if constexpr (E4M3) {
        float vref = __uint_as_float(0x00800000u);  // at least the values' largest scale so far, a power of two
        // The scales so far of keys that some row sees: the largest, and the smallest of this thread's.
        uint32_t largest = 0, smallest = 0x7f7fffffu;
        for (int j = 0; j < n; ++j, ++tile_no) {
          const int tile = tile_at(i0 + j);
          const bool masked = is_masked(tile);
          // The scales of this thread's key: for the keys as they are, for the values relative to vref.
          const float sk = next_scales.x, sv = next_scales.y;
          const bool counts = next_seen && __float_as_uint(sv) < 0x7f800000u;
          next_scales = scales_of(j + 1, next_page);
          next_seen = next_page >= 0;
          next_page = page_of(j + 2);
          const uint32_t top = __reduce_max_sync(0xffffffffu, counts ? __float_as_uint(sv) : 0u);
          if (counts) smallest = min(smallest, __float_as_uint(sv));
          if (lane == 0) aux_top[(tile_no & 1) * 4 + awarp] = top;
          aux_sync();
          const uint4 tops = *reinterpret_cast<const uint4*>(aux_top + (tile_no & 1) * 4);
          const uint32_t most = max(max(tops.x, tops.y), max(tops.z, tops.w));
          largest = max(largest, most);
          const bool far = aux_sync_or(__uint_as_float(smallest) * kFarScales < __uint_as_float(largest));
          const float want = __uint_as_float(min((most >> 23) + 1u, 254u) << 23);
          const float before = vref;
          if (most > 0) vref = fmaxf(vref, want);
          // 1 / vref, another power of two (of 2^127 a subnormal one): a product with it is the quotient.
          const uint32_t vexp = __float_as_uint(vref) >> 23;
          const float inv = __uint_as_float(vexp == 254 ? 0x00400000u : (254u - vexp) << 23);
          if (tile_no >= 2) wait(&scale_free[tile_no & 1], ((tile_no >> 1) - 1) & 1, kStatusWaitEmpty);
          float* to = scales + (tile_no & 1) * 2 * KT;
          to[key] = sk;
          to[KT + key] = far ? log2_approx(sv) : sv * inv * 64.0f;
          if (awarp == 0 && lane == 0) {
            scale_step[tile_no & 1] = j == 0 ? 1.0f : before * inv;
            scale_ref[tile_no & 1] = far ? 0.0f : vref;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&scale_full[tile_no & 1]);
          // V's codes to fp16, 16 at a time; rows no row sees to 0.
          wait(&full_v[vs], v_phase, kStatusWaitFull);
          if (tile_no >= C::NW) wait(&empty_w[ws], w_phase ^ 1, kStatusWaitEmpty);
          // Four lanes take the four pieces of a chunk's row, eight lanes two rows that are 5 apart: then the
          // swizzled places they read and write lie in different banks.
#pragma unroll(C::kWUnroll)
          for (int m = 0; m < KT * C::kVBytes / 16 / (kAuxWarps * 32); ++m) {
            const int i = m * (kAuxWarps * 32) + awarp * 32 + lane, piece = i & 3, c = i / (4 * KT);
            const int k = ((i >> 2) & (KT - 1)) ^ (i & 4 ? 4 : 0);
            const uint32_t from = C::kVBytes == 128 ? ((c * 64 + piece * 16) ^ ((k & 7) << 4)) : piece * 16;
            const uint4 x = *reinterpret_cast<const uint4*>(v_ring + vs * C::kVSlot + k * C::kVBytes + from);
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
            uint32_t w[8];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
                  "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
                  : "=r"(w[2 * q]), "=r"(w[2 * q + 1])
                  : "r"(u[q]));
            if (masked && !any_sees(tile * KT + k)) {
#pragma unroll
              for (int q = 0; q < 8; ++q) w[q] = 0;
            }
            uint8_t* to_w = w_ring + ws * C::kWSlot + c * kChunk + k * 128;
            const uint32_t byte = piece * 32, swz = (k & 7) << 4;
            *reinterpret_cast<uint4*>(to_w + (byte ^ swz)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(to_w + ((byte + 16) ^ swz)) = make_uint4(w[4], w[5], w[6], w[7]);
          }
          if (awarp == 0 && lane == 0) w_far[ws] = far ? 1 : 0;
          if (__builtin_expect(far, 0)) far_values(reinterpret_cast<uint32_t*>(w_ring + ws * C::kWSlot), C::kWSlot / 4);
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&empty_v[vs]);
            mbar_arrive(&full_w[ws]);
          }
          if (++vs == C::NV) {
            vs = 0;
            v_phase ^= 1;
          }
          if (++ws == C::NW) {
            ws = 0;
            w_phase ^= 1;
          }
          if (j == 0) output_last();
        }
      }
    }
    if (item_no > 0) output(was, was_part, was_whole, was_start, item_no - 1);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------------ joining an item's pieces

// A block for each place where a share begins and each 8 rows: if that is the first cut in an item, a warp
// joins a row of the item's pieces.
template <int D>
__global__ void __launch_bounds__(256) kv_chunk_join_kernel(const KvAttn a) {
  constexpr int DV = D < 256 ? D : 256, kHalves = D / DV;
  pdl_wait();
  pdl_launch_dependents();
  const KvJoin j = a.list.joins[blockIdx.x + 1];
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int tok = r / a.group;
  if (tok >= j.nt) return;
  auto place = [&](int c) {
    return a.chunk_partial + (c == 0 ? j.first_place : 2 * (j.first + c)) * kChunkPieceFloats;
  };
  float top = -INFINITY;
  for (int c = lane; c < j.count; c += 32) top = fmaxf(top, __ldcg(place(c) + 256 * 256 + r));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float base = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  float4 acc[DV / 128];
#pragma unroll
  for (int v = 0; v < DV / 128; ++v) acc[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int c = 0; c < j.count; ++c) {
    const float* from = place(c);
    const float w = exp2_approx(__ldcg(from + 256 * 256 + r) - base);
    sum = fmaf(w, __ldcg(from + 256 * 257 + r), sum);
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
  const long long row = static_cast<long long>(j.row0 + tok) * a.q_heads + j.part / kHalves * a.group + r % a.group;
#pragma unroll
  for (int v = 0; v < DV / 128; ++v)
    *reinterpret_cast<uint2*>(a.out + row * D + j.part % kHalves * DV + v * 128 + lane * 4) =
        make_uint2(pack_bf16(acc[v].x * f, acc[v].y * f), pack_bf16(acc[v].z * f, acc[v].w * f));
  if (a.lse && lane == 0 && j.part % kHalves == 0)
    a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.693147181f;
}

template <int D, bool E4M3>
cudaError_t launch(const KvAttn& a, int pairs, cudaStream_t s) {
  using C = Chk<D, E4M3>;
  CUtensorMap mk, mv;
  const uint64_t rows = (static_cast<uint64_t>(a.c.n_pages) * a.c.kv_heads) << a.c.page_log2;
  const uint32_t box = 1u << (a.c.page_log2 < 6 ? a.c.page_log2 : 6);
  if (!encode_row_chunks(&mk, a.c.k, rows, C::kRow, box, 1, 128, true) ||
      !encode_row_chunks(&mv, a.c.v, rows, C::kRow, box, 1, C::kVBytes, C::kVBytes == 128))
    return cudaErrorInvalidValue;
  const int tokens = chunk_tokens(a.group);
  cudaError_t e = launch_pdl(kv_chunk_list_kernel, dim3(1), dim3(kListThreads), 0, s, a, tokens, a.c.kv_heads * C::kHalves, pairs);
  if (e == cudaSuccess)
    e = launch_pdl_pair(kv_chunk_kernel<D, E4M3>, dim3(2 * pairs), dim3(kThreads), C::kSmem, s, a, mk, mv);
  if (e == cudaSuccess && pairs > 1)
    e = launch_pdl(kv_chunk_join_kernel<D>, dim3(pairs - 1, 256 / 8), dim3(256), 0, s, a);
  return e;
}

// Sets the shared memory limit and lowers *pairs to the pairs that can be resident at once.
template <int D, bool E4M3>
cudaError_t setup(int* pairs) {
  using C = Chk<D, E4M3>;
  cudaError_t e = cudaFuncSetAttribute(kv_chunk_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * kChunkMaxPairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, kv_chunk_kernel<D, E4M3>, &cfg);
  if (e == cudaSuccess && n < 1) e = cudaErrorInvalidConfiguration;
  if (e == cudaSuccess && n < *pairs) *pairs = n;
  return e;
}

}  // namespace

cudaError_t kv_chunk_setup(int* pairs) {
  *pairs = kChunkMaxPairs;
  cudaError_t e = setup<128, false>(pairs);
  if (e == cudaSuccess) e = setup<256, false>(pairs);
  if (e == cudaSuccess) e = setup<512, false>(pairs);
  if (e == cudaSuccess) e = setup<128, true>(pairs);
  if (e == cudaSuccess) e = setup<256, true>(pairs);
  if (e == cudaSuccess) e = setup<512, true>(pairs);
  return e;
}

cudaError_t launch_kv_chunk(const KvAttn& a, int pairs, cudaStream_t s) {
  switch (a.c.head_dim * 2 + a.c.e4m3) {
    case 256: return launch<128, false>(a, pairs, s);
    case 257: return launch<128, true>(a, pairs, s);
    case 512: return launch<256, false>(a, pairs, s);
    case 513: return launch<256, true>(a, pairs, s);
    case 1024: return launch<512, false>(a, pairs, s);
    default: return launch<512, true>(a, pairs, s);
  }
}

}  // namespace moe
