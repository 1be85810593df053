// beam.cu — the selection of a beam search over beams and vocabulary.
//
// A continuation's value is score + x - log sum exp(x) over its beam's logits x, so within a beam the order is the
// logits' own: one pass over a beam's logits yields both its sum of exponentials and its `count` largest, and a
// second kernel compares the beams' best. The logits are read once, two or four bytes for one exponential and
// half a dozen operations; HBM bounds it where there are many beams, the launches and the last steps where there are few.
//
// The pass. A row's logits are cut into equal parts, a CTA each, so that few beams fill the GPU too. A CTA takes
// tiles of 256 x 4 vectors, the next one's loads under way. The first tile gives a threshold that at least `count` of
// the 256 threads' maxima are above: nothing below it counts. A vector with something above it is noted, about `count`
// of each tile as a rule, without a barrier; at the end these are looked through, and what is above the threshold is
// ranked. Where that is more than the lists hold (logits that ascend, or many equal ones), the part is gone through again
// in steps that the list has room for: when it is long, it is cut to the `count` best, which raise the threshold.
//
// Sums. What is at most the threshold is added as exp(x - R) with R the first tile's maximum, by the hardware's
// 2^x, and sums of 16 go into a pair of fp32 numbers that keeps the rounding (D. E. Knuth, "The Art of Computer
// Programming" 2, 4.2.2, Theorem B). What is above it may outweigh all else: these terms are formed in such pairs, by the
// exponential's series, to 2^-30; the selected logits' are added in the order of their ranks, the others' as integers, whose
// sum does not depend on the order in which they were noted. So that few large logits are above it however few are asked
// for, the threshold is lowered to the kExact-th of the threads' maxima where `count` is less (and only what is above
// the count-th is ranked). (160 rows, the best 32.2 us, 30.0 without; with 16 of them instead of 8 33.5, and the 10 best
// 30.3 instead of 28.6.)
//   A term below the threshold is off by 2^-22 of itself, and by half a step of the exponent, log2 e of its distance from
// R. Over many different ones that averages out: log sum exp is good to about 1e-8, below which values of different
// beams seldom lie. Many equal ones are all off alike, by up to 2^-20 if it takes 10^5 of them to outweigh the
// largest. Equal rows have equal sums wherever they lie.
//
// fp64 is slow here (an operation takes a warp 16 cycles or more, and its result some 60): only the last comparisons
// are made in it.
//
// Times in a graph, 262144 bf16 logits to a row, each call's logits from HBM. 160 rows, the 10 best: 35.4 us, of which the
// bytes are 12.6. The same with 32 users of 5 beams of which a fifth has ended: 28.4 (10.2). There the pass takes 24 at
// 2.6 TB/s, a third of HBM's, with 54% of the issue slots busy, so neither bounds it: its parts run in one wave and in step,
// and HBM waits while all form their thresholds, and again while all list, rank and sum. The join is a chain of barriers and
// small steps of one CTA to a user. 4 rows, the 8 best: 10.1, of which the bytes are 0.3. 64 rows, the 64 best: 56.5 (5.0); in fp32, 180 rows of
// 116508, the 20 best: 30.2 (12.6). One token far above all others takes 41 for the 160 rows (73 if coarse distances were not cut
// again), -infinity in place of all but 0.1% of the logits 33. Where no threshold parts a row, because most logits are equal
// or are the type's lowest value, parts are gone through twice: equal rows take two to five times as long as others (160 rows
// 101 us, 64 rows and the 64 best 269), rows with 0.1% above the lowest value two to three times (83 and 140). The join in
// fp64 throughout took 40 us. A form that found its thresholds by bisection, a barrier for each step, and summed in fp64 took
// 136 for the 160 rows with ended ones and 44 for the 4.
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "moe_ffn.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;                     // 16-byte vectors of a thread in a tile
constexpr int kNoted = 1024;                 // vectors
constexpr int kList = 2560;
constexpr int kListLong = kList - kThreads * 8 - 32;  // what still has room for a vector of each thread, and the ends
constexpr int kMaxSplits = 64;
constexpr int kMaxCount = MOE_FFN_BEAM_MAX;
// As many of a part's largest logits at least have their terms formed in two numbers, as far as they lie within kNear of
// the first tile's maximum (one that is further weighs at most e^-4 of it, and 2^-22 of that is 4e-9), and unless there are more
// than kNearMost in the distance of the last (many like it: rather none of these, as there would be no room for them).
constexpr int kExact = 8, kNearMost = 48;
constexpr float kNear = 4.0f;
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinHeld = 2048;  // candidates
constexpr int kJoinList = 512;

struct BeamParams {
  const void* logits;
  long long stride;
  const float* scores;
  const uint8_t* finished;
  float* out_scores;
  int32_t* out_beams;
  int32_t* out_tokens;
  float2* part_sum;       // [rows, splits] sums in two numbers, in units of exp(part_ref)
  float* part_ref;
  float* part_x;          // [rows, splits, count] the part's largest logits, best first
  int32_t* part_token;    // and their tokens, -1 for none
  int end_token, beams, vocab, count, splits;
  int part;               // vectors of a part
};

// fp32 numbers in an order of unsigned integers.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ (u & 0x80000000u ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o ^ (o & 0x80000000u ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ unsigned long long ordered(double x) {
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
  return u ^ (u >> 63 ? ~0ull : 1ull << 63);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2eHigh = 1.44269502f;          // log2 e, and what fp32 leaves of it
constexpr float kLog2eLow = 1.92596303e-8f;

// exp(x - ref). (The small product first: the exponent is rounded once.)
__device__ __forceinline__ float term(float x, float ref) {
  const float d = __fsub_rn(x, ref);
  return exp2_approx(fmaf(d, kLog2eHigh, __fmul_rn(d, kLog2eLow)));
}

__device__ __forceinline__ unsigned long long two(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The same of eight numbers, two at a time.
__device__ __forceinline__ void terms(const float (&x)[8], float ref, float (&e)[8]) {
  const unsigned long long r2 = two(-ref, -ref), high = two(kLog2eHigh, kLog2eHigh), low = two(kLog2eLow, kLog2eLow);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const unsigned long long d = add2(two(x[i], x[i + 1]), r2);
    unsigned long long t;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(d), "l"(low));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(t) : "l"(d), "l"(high), "l"(t));
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(t));
    e[i] = exp2_approx(a);
    e[i + 1] = exp2_approx(b);
  }
}

// Distances below a maximum in 256 bins, eight to a factor of two, from 2^-20 to 2^12; NaN and what is further is in the last.
// Where one is far above all others these are coarse, and each is cut into 256 again.
constexpr int kBins = 256;
constexpr int kBinShift = 20, kBinFirst = (127 - 20) << 3;
constexpr int kFineShift = kBinShift - 8;
__device__ __forceinline__ int bin_of(float d) {
  return min(max(static_cast<int>(__float_as_uint(d) >> kBinShift) - kBinFirst, 0), kBins - 1);
}
// What all distances in bins up to b are below; infinity for the last.
__device__ __forceinline__ float bin_end(int b) {
  return b == kBins - 1 ? INFINITY : __uint_as_float(static_cast<uint32_t>(b + 1 + kBinFirst) << kBinShift);
}
// The first bin up to which there are at least `count`, or the last, and how many come before it; for a whole warp.
__device__ __forceinline__ int bin_reached(const int* bins, int count, int& before) {
  const int lane = threadIdx.x & 31;
  const int4 a = reinterpret_cast<const int4*>(bins)[2 * lane], b = reinterpret_cast<const int4*>(bins)[2 * lane + 1];
  const int n[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  int upto = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) upto += n[i];
  const int mine = upto;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += up;
  }
  int at = upto - mine, bin = 0;
  before = at;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    at += n[i];
    if (at >= count) continue;
    ++bin;
    before = at;
  }
  const unsigned reached = __ballot_sync(0xffffffffu, upto >= count);
  if (reached == 0) return kBins - 1;
  const int which = __ffs(reached) - 1;
  before = __shfl_sync(0xffffffffu, before, which);
  return __shfl_sync(0xffffffffu, 8 * lane + bin, which);
}
// What at least `count` of the CTA's distances are below, and no more than `room` where bins can tell them apart; infinity
// where there are fewer. each(f) calls f with each of a thread's. The bins are zero.
struct Bins {
  alignas(16) int coarse[kBins];
  alignas(16) int fine[kBins];
};
template <typename Each>
__device__ __forceinline__ float distance_reached(Bins& bins, int count, int room, Each each) {
  each([&](float d) { atomicAdd(&bins.coarse[bin_of(d)], 1); });
  __syncthreads();
  int before;
  const int b = bin_reached(bins.coarse, count, before);
  if (b == 0 || b == kBins - 1 || before + bins.coarse[b] <= room) return bin_end(b);
  each([&](float d) {
    if (bin_of(d) == b) atomicAdd(&bins.fine[__float_as_uint(d) >> kFineShift & (kBins - 1)], 1);
  });
  __syncthreads();
  int none;
  const uint32_t sub = static_cast<uint32_t>(bin_reached(bins.fine, count - before, none)) + 1;
  return __uint_as_float((static_cast<uint32_t>(b + kBinFirst) << kBinShift) + (sub << kFineShift));
}

// A number in two of fp32, the second what the first leaves of it; and operations that lose about 2^-46.
struct Sum {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float v) {
    const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b)));
    hi = s;
  }
  __device__ __forceinline__ void add(const Sum& o) {
    add(o.hi);
    lo = __fadd_rn(lo, o.lo);
  }
  // By a number near it in size, so that neither part is lost; and the first part the sum of both.
  __device__ __forceinline__ void times(const Sum& o) {
    const float h = __fmul_rn(hi, o.hi);
    lo = fmaf(hi, o.hi, -h) + fmaf(hi, o.lo, lo * o.hi);
    hi = h;
    settle();
  }
  __device__ __forceinline__ void settle() {
    const float s = __fadd_rn(hi, lo);
    lo = __fsub_rn(lo, __fsub_rn(s, hi));
    hi = s;
  }
};

__device__ __forceinline__ Sum difference(float a, float b) {
  Sum s;
  s.hi = __fsub_rn(a, b);
  const float t = __fsub_rn(a, s.hi);  // b, but for the rounding
  s.lo = __fadd_rn(__fsub_rn(t, b), __fsub_rn(a, __fadd_rn(s.hi, t)));
  return s;
}

// exp(d) to about 2^-30, of d up to 1 or so; below e^-87, 0. d less a multiple k of log 2 (W. J. Cody and W. Waite, "Software
// Manual for the Elementary Functions", 1980: the multiple of a constant of 16 bits is exact, the rest's is added),
// then the series, its first three terms in two numbers.
__device__ __forceinline__ Sum exp_pair(const Sum& d) {
  constexpr float kLn2High = 0.693145752f, kLn2Low = 1.42860677e-6f;
  if (!(d.hi > -87.0f)) return Sum{d.hi == d.hi ? 0.0f : d.hi, 0.0f};  // (NaN stays)
  const float k = rintf(d.hi * kLog2eHigh);
  Sum x;
  x.hi = fmaf(-k, kLn2High, d.hi);
  x.lo = fmaf(-k, kLn2Low, d.lo);
  x.settle();
  const float q = x.hi * x.hi;
  const float q_lo = fmaf(x.hi, x.hi, -q) + 2.0f * x.hi * x.lo;
  float r = fmaf(x.hi, 1.0f / 362880.0f, 1.0f / 40320.0f);
  r = fmaf(x.hi, r, 1.0f / 5040.0f);
  r = fmaf(x.hi, r, 1.0f / 720.0f);
  r = fmaf(x.hi, r, 1.0f / 120.0f);
  r = fmaf(x.hi, r, 1.0f / 24.0f);
  r = fmaf(x.hi, r, 1.0f / 6.0f);
  Sum e;
  e.hi = 1.0f;
  e.add(x.hi);
  e.add(0.5f * q);
  e.lo += fmaf(0.5f, q_lo, x.lo) + x.hi * q * r;
  e.settle();
  const float scale = __uint_as_float(static_cast<uint32_t>(static_cast<int>(k) + 127) << 23);
  e.hi *= scale;
  e.lo *= scale;
  return e;
}

// log(s) of s from about 1 to 2^60: from its fp32 value l, s exp(-l) is 1 + t, and log(1 + t) two terms of t.
__device__ __forceinline__ Sum log_pair(const Sum& s) {
  const float l = logf(s.hi);
  Sum minus;
  minus.hi = -l;
  Sum t = exp_pair(minus);
  t.times(s);
  t.add(-1.0f);
  t.settle();
  Sum r;
  r.hi = l;
  r.add(t.hi - 0.5f * t.hi * t.hi);
  r.lo += t.lo;
  r.settle();
  return s.hi > 0.0f && s.hi < INFINITY ? r : Sum{l, 0.0f};
}

template <typename T>
struct Logits;
template <>
struct Logits<uint16_t> {
  static constexpr int kVec = 8;
  __device__ static __forceinline__ void unpack(const uint4& v, float* f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  __device__ static __forceinline__ float value(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
  __device__ static __forceinline__ uint4 none() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
};
template <>
struct Logits<float> {
  static constexpr int kVec = 4;
  __device__ static __forceinline__ void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  __device__ static __forceinline__ float value(float x) { return x; }
  __device__ static __forceinline__ uint4 none() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
};

// A row's vectors begin at its first element, wherever that lies, so that equal rows have equal sums. Where that is no
// multiple of 16 bytes (SHIFTED: of some row), a vector is cut out of two aligned blocks. A row's first vector and its
// last one to two, whose blocks hold other bytes too, are taken element by element.
template <bool SHIFTED>
struct Raw;
template <>
struct Raw<false> {
  uint4 a;
};
template <>
struct Raw<true> {
  uint4 a, b;
};

// Vector v of the row whose first block is `blocks`, if it is one of [lo, hi); else -infinity.
template <typename T, bool SHIFTED>
__device__ __forceinline__ Raw<SHIFTED> load_vec(const uint4* blocks, int v, int lo, int hi) {
  Raw<SHIFTED> r;
  r.a = Logits<T>::none();
  if constexpr (SHIFTED) r.b = r.a;
  if (v >= lo && v < hi) {
    if constexpr (SHIFTED) {
      r.a = __ldg(blocks + v);
      r.b = __ldg(blocks + v + 1);
    } else {
      r.a = __ldcs(blocks + v);
    }
  }
  return r;
}

// The vector that begins `shift` bytes after its first block.
template <bool SHIFTED>
__device__ __forceinline__ uint4 cut(const Raw<SHIFTED>& r, int shift) {
  if constexpr (SHIFTED) {
    uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
    const int bits = (shift & 3) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                      __funnelshift_r(w[3], w[4], bits));
  } else {
    return r.a;
  }
}

// A list entry: by logit (-0 is 0), of equal ones by the lower token.
__device__ __forceinline__ unsigned long long entry(float x, int token) {
  return static_cast<unsigned long long>(ordered(x + 0.0f)) << 32 | (0xffffffffu - static_cast<uint32_t>(token));
}
__device__ __forceinline__ float entry_x(unsigned long long e) { return from_ordered(static_cast<uint32_t>(e >> 32)); }
__device__ __forceinline__ int entry_token(unsigned long long e) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(e)); }

struct Shared {
  unsigned long long list[kList];
  unsigned long long best[kMaxCount];
  unsigned long long warp_best[2][kWarps];
  uint4 noted[kNoted];
  int noted_at[kNoted];
  Bins bins;
  Sum warp_sum[kWarps];
  long long warp_fixed[kWarps];
  float warp_max[kWarps];
  int n_noted;
  int n;
};

__device__ __forceinline__ float cta_max(Shared& s, float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) s.warp_max[threadIdx.x >> 5] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v = fmaxf(v, s.warp_max[w]);
  return v;
}

// The `count` best of the first n entries of the list (fewer if there are fewer), best first, in s.best; their
// number. All entries differ. Few entries are ranked by comparing each with all; of more, those within a distance from the
// best that `count` are within, copied over the noted vectors, which are done with; of many such, the best is taken
// `count` times.
__device__ int select_best(Shared& s, int n, int count) {
  const int tid = threadIdx.x, found = min(n, count);
  auto rank_all = [&](const unsigned long long* from, int m) {
    const unsigned long long mine = tid < m ? from[tid] : 0ull;
    int rank = 0;
    if ((tid & ~31) < m)
      for (int i = 0; i < m; ++i) rank += from[i] > mine ? 1 : 0;
    if (tid < m && rank < count) s.best[rank] = mine;
    __syncthreads();
    return found;
  };
  if (n <= kThreads) return rank_all(s.list, n);
  constexpr int kOwn = kList / kThreads;
  unsigned long long own[kOwn], top = 0ull;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    own[i] = i * kThreads + tid < n ? s.list[i * kThreads + tid] : 0ull;
    top = max(top, own[i]);
  }
  // (No entry is NaN or -infinity; where one is +infinity there is no distance that says anything.)
  s.bins.coarse[tid] = s.bins.fine[tid] = 0;
  if (tid == 0) s.n_noted = 0;
  const float most = cta_max(s, entry_x(top));
  const float far = distance_reached(s.bins, count, kThreads, [&](auto&& take) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (own[i] != 0ull) take(most - entry_x(own[i]));
  });
  unsigned long long* close = reinterpret_cast<unsigned long long*>(s.noted);
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    if (own[i] == 0ull || far == INFINITY || !(most - entry_x(own[i]) < far)) continue;
    const int to = atomicAdd(&s.n_noted, 1);
    if (to < kThreads) close[to] = own[i];
  }
  __syncthreads();
  if (far < INFINITY && s.n_noted <= kThreads) return rank_all(close, s.n_noted);
  for (int c = 0; c < found; ++c) {
    unsigned long long m = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) s.warp_best[c & 1][tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = max(m, s.warp_best[c & 1][w]);
    if (top == m) {  // one thread's
      s.best[c] = m;
      top = 0ull;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        if (own[i] == m) own[i] = 0ull;
        top = max(top, own[i]);
      }
    }
  }
  __syncthreads();
  return found;
}

template <typename T, bool SHIFTED>
__global__ void __launch_bounds__(kThreads, SHIFTED ? 3 : 4) beam_part_kernel(const BeamParams p) {
  using L = Logits<T>;
  constexpr int N = L::kVec;
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int row = blockIdx.x / p.splits, split = blockIdx.x - row * p.splits;
  if (p.finished && p.finished[row]) return;
  const T* logits = static_cast<const T*>(p.logits) + row * p.stride;
  const int shift = SHIFTED ? static_cast<int>(reinterpret_cast<uintptr_t>(logits) & 15u) : 0;
  const uint4* blocks = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(logits) - shift);
  // The part's vectors, of the row's whole ones but the first and the last; the first part has the row's ends too, an
  // element to a thread.
  const int end = p.vocab / N - 1;
  const int lo = 1 + split * p.part, hi = max(lo, min(end, lo + p.part));
  const int tiles = (hi - lo + kThreads * kVecs - 1) / (kThreads * kVecs);
  const int head = end > 1 ? N : p.vocab;
  int side = -1;
  if (split == 0) side = tid < head ? tid : end > 1 && end * N + tid - head < p.vocab ? end * N + tid - head : -1;
  const float x_side = side < 0 ? -INFINITY : L::value(logits[side]);
  if (tid == 0) s.n = s.n_noted = 0;
  s.bins.coarse[tid] = s.bins.fine[tid] = 0;

  Raw<SHIFTED> v[kVecs];
#pragma unroll
  for (int u = 0; u < kVecs; ++u) v[u] = load_vec<T, SHIFTED>(blocks, lo + u * kThreads + tid, lo, hi);
  // The first tile's maximum (with the row's ends), and a value that at least `count` of the threads' maxima are above: from
  // the number of them at each distance from the maximum.
  float m = x_side;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    float f[N];
    L::unpack(cut<SHIFTED>(v[u], shift), f);
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, f[i]);
  }
  float ref = cta_max(s, m);
  // (Rounded down, and by more than the distances' rounding: what is in the bins is above it.) What may be selected is above
  // `listed`; what is above `above` alone has its term formed in two numbers.
  float above = -INFINITY, listed = -INFINITY;
  const float d = distance_reached(s.bins, p.count, p.count + p.count / 2 + 8, [&](auto&& take) { take(ref - m); });
  if (ref < INFINITY && d < INFINITY) {
    listed = above = __fsub_rd(ref, d * 1.000001f);
    if (p.count < kExact) {
      int less;
      const int b = bin_reached(s.bins.coarse, kExact, less);
      if (b > 0) above = fminf(above, __fsub_rd(ref, fminf(bin_end(less + s.bins.coarse[b] <= kNearMost ? b : b - 1), kNear)));
    }
  }
  float unit = ref == -INFINITY ? 0.0f : ref;

  Sum sum;
  if (side >= 0) {
    if (x_side > above) s.list[atomicAdd(&s.n, 1)] = entry(x_side, side);
    else sum.add(term(x_side, unit));
  }
  for (int t = 0; t < tiles; ++t) {
    const int at = lo + t * (kThreads * kVecs) + tid;  // this thread's first vector
    unsigned long long sum2 = 0ull;                    // of 16 numbers, two zeros
#pragma unroll
    for (int g = 0; g < kVecs * N / 8; ++g) {
      float f[8];
      uint4 now[8 / N];
#pragma unroll
      for (int k = 0; k < 8 / N; ++k) {
        const int u = g * (8 / N) + k;
        now[k] = cut<SHIFTED>(v[u], shift);
        L::unpack(now[k], f + k * N);
        v[u] = load_vec<T, SHIFTED>(blocks, at + (kVecs + u) * kThreads, lo, hi);  // the next tile's (none after the last)
      }
      float e[8];
      terms(f, unit, e);
      const float top = fmaxf(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])), fmaxf(fmaxf(f[4], f[5]), fmaxf(f[6], f[7])));
      if (__builtin_expect(top > above, 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = f[i] > above ? 0.0f : e[i];
#pragma unroll
        for (int k = 0; k < 8 / N; ++k) {
          if (N < 8 && !(fmaxf(fmaxf(f[k * N], f[k * N + 1]), fmaxf(f[k * N + 2], f[k * N + 3])) > above)) continue;
          const int to = atomicAdd(&s.n_noted, 1);
          if (to >= kNoted) continue;
          s.noted[to] = now[k];
          s.noted_at[to] = at + (g * (8 / N) + k) * kThreads;
        }
      }
      sum2 = add2(sum2, add2(add2(two(e[0], e[1]), two(e[2], e[3])), add2(two(e[4], e[5]), two(e[6], e[7]))));
      if (g & 1) {
        float a, b;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(sum2));
        sum.add(a + b);
        sum2 = 0ull;
      }
    }
  }
  __syncthreads();
  const int noted = s.n_noted;
  long long fixed = 0;
  // A logit that is too small to be selected, and the same of what is listed but not selected below: added in units of
  // 2^-36 exp(ref), as long as it is no more than e^10 of these.
  auto add_fixed = [&](float x) {
    const Sum t = exp_pair(difference(x, unit));
    fixed += __float2ll_rn(t.hi * 0x1p36f) + __float2ll_rn(t.lo * 0x1p36f);
  };
  for (int i = tid; i < min(noted, kNoted); i += kThreads) {
    const int at = s.noted_at[i];
    float f[N];
    L::unpack(s.noted[i], f);
    uint32_t near = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (!(f[k] > above)) continue;
      if (!(f[k] > listed)) {
        near |= 1u << k;
        continue;
      }
      const int to = atomicAdd(&s.n, 1);
      if (to < kList) s.list[to] = entry(f[k], at * N + k);
    }
#pragma unroll 1
    for (; near != 0u; near &= near - 1u) add_fixed(L::value(reinterpret_cast<const T*>(&s.noted[i])[__ffs(near) - 1]));
  }
  __syncthreads();
  int found = -1;
  if (__builtin_expect(noted <= kNoted && s.n <= kList, 1)) {
    // (Where there are more than `count` above e^10 of these: in the other way.)
    const int n = s.n;
    found = select_best(s, n, p.count);
    bool large = false;
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long e = s.list[i];
      if (e >= s.best[found - 1]) continue;
      const float x = entry_x(e);
      large |= x > ref + 10.0f;
      add_fixed(x);
    }
    if (__syncthreads_or(large)) found = -1;
  }
  if (found < 0) {
    const int exact = max(p.count, kExact);
    float m = x_side;
    for (int i = lo + tid; i < hi; i += kThreads) {
      float f[N];
      L::unpack(cut<SHIFTED>(load_vec<T, SHIFTED>(blocks, i, lo, hi), shift), f);
#pragma unroll
      for (int k = 0; k < N; ++k) m = fmaxf(m, f[k]);
    }
    __syncthreads();
    ref = cta_max(s, m);
    unit = ref == -INFINITY ? 0.0f : ref;
    above = -INFINITY;
    fixed = 0;
    sum = Sum();
    if (side >= 0) sum.add(term(x_side, unit));
    if (tid == 0) s.n = 0;
    for (int at = lo; at < hi; at += kThreads) {
      __syncthreads();
      const int n = s.n;
      __syncthreads();
      if (at == lo && side < head && x_side > above) s.list[atomicAdd(&s.n, 1)] = entry(x_side, side);
      if (n > kListLong) {
        const int best = select_best(s, n, exact);
        if (tid < best) s.list[tid] = s.best[tid];
        if (tid == 0) s.n = best;
        above = fmaxf(above, entry_x(s.best[best - 1]));  // (as many as are asked for: of equal ones the earlier win)
        __syncthreads();
      }
      if (at + tid >= hi) continue;
      float f[N];
      L::unpack(cut<SHIFTED>(load_vec<T, SHIFTED>(blocks, at + tid, lo, hi), shift), f);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        sum.add(term(f[k], unit));
        if (f[k] > above) s.list[atomicAdd(&s.n, 1)] = entry(f[k], (at + tid) * N + k);
      }
    }
    if (side >= head && x_side > above) s.list[atomicAdd(&s.n, 1)] = entry(x_side, side);
    __syncthreads();
    found = select_best(s, s.n, exact);
    // (These terms were added by the hardware's exponential.)
    if (tid < found) sum.add(-term(entry_x(s.best[tid]), unit));
    if (tid >= p.count && tid < found) sum.add(exp_pair(difference(entry_x(s.best[tid]), unit)));
    found = min(found, p.count);
  }
  // The sum in units of the largest logit's exponential: the selected ones' terms in the order of their ranks.
  const float most = found > 0 ? entry_x(s.best[0]) : ref;
  sum.settle();
  const Sum by = exp_pair(difference(ref, most));
  if (ref != most) sum.times(by);
  if (tid < found) sum.add(exp_pair(difference(entry_x(s.best[tid]), most)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sum other;
    other.hi = __shfl_xor_sync(0xffffffffu, sum.hi, o);
    other.lo = __shfl_xor_sync(0xffffffffu, sum.lo, o);
    fixed += __shfl_xor_sync(0xffffffffu, fixed, o);
    sum.add(other);
    sum.settle();
  }
  if (lane == 0) {
    s.warp_sum[warp] = sum;
    s.warp_fixed[warp] = fixed;
  }
  __syncthreads();
  const long long out = static_cast<long long>(row) * p.splits + split;
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) {
      sum.add(s.warp_sum[w]);
      fixed += s.warp_fixed[w];
    }
    // The integer, in two numbers.
    Sum whole;
    whole.hi = __ll2float_rn(fixed);
    whole.lo = __ll2float_rn(fixed - __float2ll_rn(whole.hi));
    whole.hi *= 0x1p-36f;
    whole.lo *= 0x1p-36f;
    if (ref != most) whole.times(by);
    sum.add(whole);
    sum.settle();
    p.part_sum[out] = make_float2(sum.hi, sum.lo);
    p.part_ref[out] = most;
  }
  if (tid < p.count) {
    p.part_x[out * p.count + tid] = tid < found ? entry_x(s.best[tid]) : -INFINITY;
    p.part_token[out * p.count + tid] = tid < found ? entry_token(s.best[tid]) : -1;
  }
}

// A candidate in the order of unsigned integers: its value in fp64; of equal ones the lower beam, then the larger logit (-0 is
// 0), then the lower token.
struct Candidate {
  unsigned long long value;  // 0: none
  unsigned long long place;  // beam << 56 | (complement of the logit's order) << 24 | token
};
static_assert(MOE_FFN_BEAM_MAX_VOCAB <= 1 << 24 && MOE_FFN_BEAM_MAX <= 1 << 8, "places");
__device__ __forceinline__ bool before(const Candidate& a, const Candidate& b) {
  return a.value > b.value || (a.value == b.value && a.place < b.place);
}

__device__ __forceinline__ double value_of(unsigned long long o) {
  return __longlong_as_double(static_cast<long long>(o ^ (o >> 63 ? 1ull << 63 : ~0ull)));
}

// A CTA per user: the beams' log sum exp, then the best of all parts' candidates, found as in a part: a distance from the
// largest value within which there are `count`, a list of these, and the order by comparing each with all. Candidates
// have their values formed in fp32 first, with a bound of what that loses. Where there are too many to be copied into shared
// memory, the first ones of each part, which is sorted, give a distance, and only the parts whose first one is within it are
// looked through. (64 beams, the 64 best, 832 parts of 64 candidates each: 38 us; 175 to look through 640 such parts.) Where
// more are close together than the list holds, equal ones for instance, the best of the parts' first ones is taken `count`
// times. Loops over candidates are not unrolled: fetching instructions costs more here (4 us more in all where they were).
__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const BeamParams p) {
  // A continuation's value is (x - ref) + shift: the sum of exp(x - ref) is what has been formed. NaN: none.
  __shared__ double shift[MOE_FFN_BEAM_MAX];
  __shared__ float rough_shift[MOE_FFN_BEAM_MAX], beam_ref[MOE_FFN_BEAM_MAX];
  __shared__ bool ended[MOE_FFN_BEAM_MAX];
  __shared__ float held_x[kJoinHeld];
  __shared__ int held_token[kJoinHeld];
  __shared__ Candidate list[kJoinList];
  __shared__ uint8_t taken[MOE_FFN_BEAM_MAX * kMaxSplits];  // of a part's candidates
  __shared__ float warp_top[kJoinWarps];
  __shared__ Bins bins;
  __shared__ int found, live;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, user = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const long long row0 = static_cast<long long>(user) * p.beams;
  const int n_parts = p.beams * p.splits, per_beam = p.splits * p.count, n = p.beams * per_beam;
  const float* xs = p.part_x + row0 * per_beam;
  const int32_t* tokens = p.part_token + row0 * per_beam;
  static_assert(kJoinThreads == kBins && kThreads == kBins, "a bin to a thread");
  bins.coarse[tid] = bins.fine[tid] = 0;
  if (tid == 0) found = live = 0;
  // The candidates are on their way while the sums are formed.
  const bool all = n <= kJoinHeld;
#pragma unroll
  for (int j = 0; j < kJoinHeld / kJoinThreads; ++j) {
    const int i = tid + j * kJoinThreads;
    if (!all || i >= n) break;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&held_x[i])), "l"(xs + i) : "memory");
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&held_token[i])), "l"(tokens + i) : "memory");
  }
  {
    // All beams at once, 4 to 32 lanes to each.
    static_assert(kJoinThreads >= 4 * MOE_FFN_BEAM_MAX, "lanes for all beams");
    const int lanes = p.beams <= kJoinThreads / 32 ? 32 : p.beams <= kJoinThreads / 16 ? 16 : p.beams <= kJoinThreads / 8 ? 8 : 4;
    const int k = tid / lanes, l = tid & (lanes - 1);
    const bool live_beam = k < p.beams;
    const long long row = row0 + (live_beam ? k : 0);
    const bool end = !live_beam || (p.finished && p.finished[row]);
    const float score = p.scores[row];
    const float* refs = p.part_ref + row * p.splits;
    const float2* sums = p.part_sum + row * p.splits;
    const int splits = end ? 0 : p.splits;
    float2 first = make_float2(0.0f, 0.0f);
    if (l < splits) first = sums[l];
    float top = -INFINITY;
    for (int i = l; i < splits; i += lanes) top = fmaxf(top, refs[i]);
    for (int o = lanes >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    Sum sum;
#pragma unroll 1
    for (int i = l; i < splits; i += lanes) {
      const float r = refs[i];
      const float2 part = i == l ? first : sums[i];
      Sum a;
      a.hi = part.x;
      a.lo = part.y;
      if (r != top) a.times(exp_pair(difference(r, top)));
      sum.add(a);
    }
#pragma unroll 1
    for (int o = lanes >> 1; o > 0; o >>= 1) {
      Sum other;
      other.hi = __shfl_xor_sync(0xffffffffu, sum.hi, o);
      other.lo = __shfl_xor_sync(0xffffffffu, sum.lo, o);
      sum.add(other);
      sum.settle();
    }
    const Sum log_sum = log_pair(sum);
    if (live_beam && l == 0) {
      ended[k] = end;
      beam_ref[k] = top;
      const double sh = end ? static_cast<double>(score)
                            : static_cast<double>(score) - (static_cast<double>(log_sum.hi) + static_cast<double>(log_sum.lo));
      shift[k] = sh;
      rough_shift[k] = static_cast<float>(sh);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  auto x_of = [&](int i) { return all ? held_x[i] : xs[i]; };
  auto token_of = [&](int i) { return all ? held_token[i] : tokens[i]; };
  const float per_beam_inv = 1.0f / static_cast<float>(per_beam);
  // (n is at most 2^18: the product is off by less than the distance of i + 1/2 from a multiple.)
  auto beam_of = [&](int i) { return static_cast<int>((static_cast<float>(i) + 0.5f) * per_beam_inv); };
  // A candidate's value in fp32 (-infinity or NaN: none), and what it may be off by: half a step of each of two operations
  // and of shift.
  auto rough = [&](int i, float& off) {
    const int k = beam_of(i);
    const float t = rough_shift[k];
    if (ended[k]) {
      off = 0x1p-22f * fabsf(t);
      return i == k * per_beam ? t : -INFINITY;
    }
    const float d = x_of(i) - beam_ref[k];
    off = 0x1p-22f * (fabsf(d) + fabsf(t));
    return token_of(i) >= 0 ? d + t : -INFINITY;
  };
  auto exact = [&](int i) {
    const int k = beam_of(i);
    double v = shift[k];
    float x = 0.0f;
    int token = p.end_token;
    if (!ended[k]) {
      x = x_of(i);
      v += static_cast<double>(x) - static_cast<double>(beam_ref[k]);
      token = token_of(i);
    } else if (i != k * per_beam) {
      token = -1;
    }
    Candidate c;
    c.value = token >= 0 && static_cast<float>(v) > -INFINITY ? ordered(v + 0.0) : 0ull;
    c.place = static_cast<unsigned long long>(k) << 56 | static_cast<unsigned long long>(~ordered(x + 0.0f)) << 24 |
              static_cast<unsigned long long>(token & 0xffffff);
    return c;
  };
  // The parts' first candidates: their largest value, and how many there are.
  float top = -INFINITY;
  int mine_live = 0;
#pragma unroll 1
  for (int i = tid; i < n_parts; i += kJoinThreads) {
    float off;
    const float v = rough(i * p.count, off);
    if (!(v > -INFINITY)) continue;
    ++mine_live;
    top = fmaxf(top, __fsub_rd(v, off));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    mine_live += __shfl_xor_sync(0xffffffffu, mine_live, o);
  }
  if (lane == 0) {
    warp_top[warp] = top;
    atomicAdd(&live, mine_live);
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, warp_top[w]);
  // What is looked through: all candidates, or first as many of each part that `count` of all can be among them, and then all of
  // the parts whose first one is near enough (what comes after it is no larger).
  uint16_t* near = reinterpret_cast<uint16_t*>(held_x);
  static_assert(sizeof(held_x) >= 2 * MOE_FFN_BEAM_MAX * kMaxSplits, "all parts");
  int per = all ? p.count : live > 0 ? (p.count + live - 1) / live : 1;
  int m = n_parts * per;
  bool last = all;
  float least = -INFINITY;
  auto at = [&](int h) {
    if (all) return h;
    const int part = h / per;
    return (last ? near[part] : part) * p.count + h - part * per;
  };
#pragma unroll 1
  for (;;) {
    const float d = distance_reached(bins, p.count, last ? kJoinList : p.count + p.count / 2 + 8, [&](auto&& take) {
#pragma unroll 1
      for (int h = tid; h < m; h += kJoinThreads) {
        float off;
        const float v = rough(at(h), off);
        if (v > -INFINITY) take(top - __fsub_rd(v, off));
      }
    });
    if (top < INFINITY && d < INFINITY) least = fmaxf(least, __fsub_rd(top, d * 1.000001f));
    if (!last && tid == 0) live = 0;
    if (!last) __syncthreads();
#pragma unroll 1
    for (int h = tid; h < m; h += kJoinThreads) {
      const int i = at(h);
      float off;
      const float v = rough(i, off);
      if (!(v > -INFINITY && __fadd_ru(v, off) >= least)) continue;
      if (last) {
        const int to = atomicAdd(&found, 1);
        if (to < kJoinList) list[to].place = static_cast<unsigned long long>(i);
      } else if (h % per == 0) {
        near[atomicAdd(&live, 1)] = static_cast<uint16_t>(h / per);
      }
    }
    if (last) break;
    __syncthreads();
    bins.coarse[tid] = bins.fine[tid] = 0;
    last = true;
    per = p.count;
    m = live * per;
    __syncthreads();
  }
  __syncthreads();
  auto answer = [&](int c, const Candidate& a) {
    const long long o = static_cast<long long>(user) * p.count + c;
    const unsigned long long u = a.value;
    const bool some = u != 0ull;
    p.out_scores[o] = some ? static_cast<float>(value_of(u)) : -INFINITY;
    p.out_beams[o] = some ? static_cast<int>(a.place >> 56) : -1;
    p.out_tokens[o] = some ? static_cast<int>(a.place & 0xffffffull) : -1;
  };
  const int have = found;
  if (have <= kJoinList) {
    for (int i = tid; i < have; i += kJoinThreads) list[i] = exact(static_cast<int>(list[i].place));
    __syncthreads();
    for (int i = tid; i < have; i += kJoinThreads) {
      const Candidate c = list[i];
      int rank = 0;
      for (int j = 0; j < have; ++j) rank += before(list[j], c) ? 1 : 0;
      if (rank < p.count) answer(rank, c);
    }
    for (int c = have + tid; c < p.count; c += kJoinThreads) answer(c, Candidate{0ull, 0u});
    return;
  }
  // A thread keeps the best that is left of its parts.
  for (int i = tid; i < n_parts; i += kJoinThreads) taken[i] = 0;
  Candidate mine;
  int mine_of = -1;
  auto look = [&] {
    mine = Candidate{0ull, ~0ull};
#pragma unroll 4
    for (int i = tid; i < n_parts; i += kJoinThreads) {
      if (taken[i] >= p.count) continue;
      const Candidate b = exact(i * p.count + taken[i]);
      if (b.value == 0ull || !before(b, mine)) continue;
      mine = b;
      mine_of = i;
    }
  };
  look();
  for (int c = 0; c < p.count; ++c) {
    Candidate a = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Candidate b = {__shfl_xor_sync(0xffffffffu, a.value, o), __shfl_xor_sync(0xffffffffu, a.place, o)};
      if (before(b, a)) a = b;
    }
    Candidate* best = list + (c & 1) * kJoinWarps;  // (a warp may be a step ahead of one that still reads)
    if (lane == 0) best[warp] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w)
      if (before(best[w], a)) a = best[w];
    if (tid == 0) answer(c, a);
    if (a.value != 0ull && a.value == mine.value && a.place == mine.place) {
      ++taken[mine_of];
      look();
    }
  }
}

// Parts of a row: as many as four CTAs on each SM, which run there at once, of a tile at least. Rounded up where a part is then
// still of eight tiles (160 rows of 262144: 30 us, 32 rounded down), else down, as a few CTAs more take as long as all before
// (64 rows of 128256, 9 parts or 10: 16 and 20 us). And small enough that the vectors that it notes, one or two times
// `count` of a tile, have room: of 400 rows of 262144, the 8 best take 61 us in 2 parts and 55 in 3; the 64 best of 32 rows 129
// in 8 and 51 in 10. (Tiles of bf16 logits, which have the larger ones: one workspace serves both types.)
int beam_splits(int rows, int vocab, int count) {
  constexpr int kTile = kThreads * kVecs * 8, kCtas = 4 * 152;
  const int tiles = (vocab + kTile - 1) / kTile;
  int splits = rows > 0 ? (kCtas + rows - 1) / rows : kCtas;
  if (rows <= kCtas && splits * rows > kCtas && tiles < 8 * splits) --splits;
  const int least = (tiles * (count > 13 ? count : 13) + 159) / 160;
  if (splits < least) splits = least;
  if (splits > tiles) splits = tiles;
  if (splits > kMaxSplits) splits = kMaxSplits;
  return splits;
}

bool sizes_ok(int users, int beams, int vocab, int count) {
  return users >= 0 && users <= MOE_FFN_BEAM_MAX_USERS && beams >= 1 && beams <= MOE_FFN_BEAM_MAX && vocab >= 1 &&
         vocab <= MOE_FFN_BEAM_MAX_VOCAB && count >= 1 && count <= kMaxCount;
}

struct BeamLayout {
  size_t sum, ref, x, token, total;
};

BeamLayout beam_layout(int users, int beams, int vocab, int count) {
  const size_t parts = static_cast<size_t>(users) * beams * beam_splits(users * beams, vocab, count);
  BeamLayout l;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  l.sum = take(parts * 8);
  l.ref = take(parts * 4);
  l.x = take(parts * count * 4);
  l.token = take(parts * count * 4);
  l.total = o > 0 ? o : 256;
  return l;
}

bool meet(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

}  // namespace

}  // namespace moe

extern "C" size_t moe_ffn_beam_workspace_bytes(int users, int beams, int vocab, int count) {
  return moe::sizes_ok(users, beams, vocab, count) ? moe::beam_layout(users, beams, vocab, count).total : 0;
}

extern "C" int moe_ffn_beam_select(const moe_ffn_beam* a, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace moe;
  if (!a || !sizes_ok(a->users, a->beams, a->vocab, a->count) || a->logits_stride < 0) return MOE_FFN_EINVAL;
  if (a->finished && (a->end_token < 0 || a->end_token >= a->vocab)) return MOE_FFN_EINVAL;
  if (a->users == 0) return MOE_FFN_OK;
  if (!a->logits || !a->scores || !a->out_scores || !a->out_beams || !a->out_tokens || !workspace) return MOE_FFN_EINVAL;
  const uintptr_t of4 = reinterpret_cast<uintptr_t>(a->scores) | reinterpret_cast<uintptr_t>(a->out_scores) |
                        reinterpret_cast<uintptr_t>(a->out_beams) | reinterpret_cast<uintptr_t>(a->out_tokens);
  const size_t element = a->logits_fp32 ? 4 : 2;
  if ((of4 & 3u) != 0 || reinterpret_cast<uintptr_t>(a->logits) % element != 0 ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return MOE_FFN_EALIGN;
  const BeamLayout l = beam_layout(a->users, a->beams, a->vocab, a->count);
  if (workspace_bytes < l.total) return MOE_FFN_ETOOBIG;
  const int rows = a->users * a->beams;
  const size_t out = static_cast<size_t>(a->users) * a->count * 4;
  struct { const void* p; size_t n; } outs[] = {{a->out_scores, out}, {a->out_beams, out}, {a->out_tokens, out}, {workspace, l.total}},
      ins[] = {{a->logits, ((rows - 1) * static_cast<size_t>(a->logits_stride) + a->vocab) * element},
               {a->scores, static_cast<size_t>(rows) * 4},
               {a->finished, a->finished ? static_cast<size_t>(rows) : 0}};
  for (int i = 0; i < 4; ++i) {
    for (const auto& in : ins)
      if (in.n && meet(outs[i].p, outs[i].n, in.p, in.n)) return MOE_FFN_EINVAL;
    for (int j = 0; j < i; ++j)
      if (meet(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return MOE_FFN_EINVAL;
  }
  BeamParams p;
  p.logits = a->logits;
  p.stride = a->logits_stride;
  p.scores = a->scores;
  p.finished = a->finished;
  p.out_scores = a->out_scores;
  p.out_beams = a->out_beams;
  p.out_tokens = a->out_tokens;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part_sum = reinterpret_cast<float2*>(ws + l.sum);
  p.part_ref = reinterpret_cast<float*>(ws + l.ref);
  p.part_x = reinterpret_cast<float*>(ws + l.x);
  p.part_token = reinterpret_cast<int32_t*>(ws + l.token);
  p.end_token = a->end_token;
  p.beams = a->beams;
  p.vocab = a->vocab;
  p.count = a->count;
  p.splits = beam_splits(rows, a->vocab, a->count);
  p.part = (a->vocab / static_cast<int>(16 / element) + p.splits - 1) / p.splits;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool shifted = reinterpret_cast<uintptr_t>(a->logits) % 16 != 0 || (rows > 1 && a->logits_stride * element % 16 != 0);
  const dim3 grid(p.splits * rows), block(kThreads);
  cudaError_t e;
  if (a->logits_fp32)
    e = shifted ? launch_pdl(beam_part_kernel<float, true>, grid, block, 0, s, p)
                : launch_pdl(beam_part_kernel<float, false>, grid, block, 0, s, p);
  else
    e = shifted ? launch_pdl(beam_part_kernel<uint16_t, true>, grid, block, 0, s, p)
                : launch_pdl(beam_part_kernel<uint16_t, false>, grid, block, 0, s, p);
  if (e == cudaSuccess) e = launch_pdl(beam_join_kernel, dim3(a->users), dim3(kJoinThreads), 0, s, p);
  return e == cudaSuccess ? MOE_FFN_OK : MOE_FFN_ECUDA;
}
