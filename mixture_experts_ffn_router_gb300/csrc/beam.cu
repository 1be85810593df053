// beam.cu — the selection of a beam search over beams and vocabulary.
//
// A continuation's value is score + x - log sum exp(x) over its beam's logits x, so within a beam the order is the
// logits' own: one pass over a beam's logits yields both its sum of exponentials and its `count` largest, and a
// second kernel compares the beams' best. The logits are read once, two or four bytes for one exponential and
// three operations; HBM bounds it where there are many beams, the launches and the last steps where there are few.
//
// The pass. A row's logits are cut into equal parts, a CTA each, so that few beams fill the GPU too. A CTA takes
// tiles of 256 x 32 logits, the next one's loads under way. The first tile gives a threshold: at least `count` of
// the 256 threads' maxima are not below it, so nothing below it counts, and what passes it later must be above it
// (of equal logits the lower token wins). What passes is put into a list in shared memory, a few times `count` as a
// rule; a list that grows long (logits that ascend, or many equal ones) is cut to the `count` best, which raise
// the threshold, and tiles that could overfill it go through in four steps.
//
// Sums. exp(x - R) = 2^((x - R) log2 e) with the first tile's maximum as R, and log2 e in two parts. Sums of eight
// go into a pair of fp32 numbers that keeps the rounding (D. E. Knuth, "The Art of Computer Programming" 2, 4.2.2,
// Theorem B). The hardware's exponential is off by up to 2^-22 of a term: that averages out over many, but not where
// one token holds most of the weight, so the selected logits' terms are exchanged for ones in fp64. log sum exp is
// then good to about 1e-8, below which values of different beams seldom lie.
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "moe_ffn.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPerThread = 32;               // logits of a tile
constexpr int kTile = kThreads * kPerThread;
constexpr int kSteps = 4;                    // of a tile that could overfill the list
constexpr int kList = 4096;
constexpr int kListLong = kList - kTile / kSteps;
constexpr int kMaxSplits = 64;
constexpr int kMaxCount = MOE_FFN_BEAM_MAX;
constexpr int kJoinThreads = 256;

struct BeamParams {
  const void* logits;
  long long stride;
  const float* scores;
  const uint8_t* finished;
  float* out_scores;
  int32_t* out_beams;
  int32_t* out_tokens;
  double* part_sum;       // [rows, splits] sums, in units of exp(part_ref)
  float* part_ref;
  float* part_x;          // [rows, splits, count] the part's largest logits, best first
  int32_t* part_token;    // and their tokens, -1 for none
  int end_token, beams, vocab, count, splits;
  int part;               // logits of a part, a multiple of 8
};

// fp32 numbers in an order of unsigned integers.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ (u & 0x80000000u ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o ^ (o & 0x80000000u ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2eHigh = 1.44269502f;          // log2 e, and what fp32 leaves of it
constexpr float kLog2eLow = 1.92596303e-8f;

// exp(x - ref).
__device__ __forceinline__ float term(float x, float ref) {
  const float d = __fsub_rn(x, ref);
  return exp2_approx(fmaf(d, kLog2eLow, __fmul_rn(d, kLog2eHigh)));
}

// A sum in two fp32 numbers.
struct Sum {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float v) {
    const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b)));
    hi = s;
  }
};

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
  __device__ static __forceinline__ uint4 none() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
};

// A vector of a row at virtual element v * kVec, where the row begins at virtual element `skip` (so that vectors are
// aligned) and ends before `end`; elements that are not the part's, [lo, hi), count as -infinity.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* base, int v, int lo, int hi) {
  constexpr int N = Logits<T>::kVec;
  const int e = v * N;
  if (e >= lo && e + N <= hi) return __ldcs(reinterpret_cast<const uint4*>(base + e));
  uint4 x = Logits<T>::none();
  if (e + N <= lo || e >= hi) return x;
  uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (e + i < lo || e + i >= hi) continue;
    if constexpr (N == 8) {
      const uint32_t s = base[e + i];
      u[i / 2] = i & 1 ? (u[i / 2] & 0xffffu) | (s << 16) : (u[i / 2] & 0xffff0000u) | s;
    } else {
      u[i] = __float_as_uint(base[e + i]);
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
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
  double warp_sum[kWarps];
  float warp_max[kWarps];
  int n;
  int unused;
};

// The `count` best of the first n entries of the list (fewer if there are fewer), best first, in s.best; their
// number. All entries differ. Few entries are ranked by comparing each with all; of many, the best is taken `count`
// times.
__device__ int select_best(Shared& s, int n, int count) {
  const int tid = threadIdx.x, found = min(n, count);
  if (n <= kThreads) {
    const unsigned long long mine = tid < n ? s.list[tid] : 0ull;
    int rank = 0;
    for (int i = 0; i < n; ++i) rank += s.list[i] > mine ? 1 : 0;
    if (tid < n && rank < count) s.best[rank] = mine;
    __syncthreads();
    return found;
  }
  constexpr int kOwn = kList / kThreads;
  unsigned long long own[kOwn], top = 0ull;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    own[i] = i * kThreads + tid < n ? s.list[i * kThreads + tid] : 0ull;
    top = max(top, own[i]);
  }
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

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) beam_part_kernel(const BeamParams p) {
  using L = Logits<T>;
  constexpr int N = L::kVec, kVecs = kPerThread / N;
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int row = blockIdx.x / p.splits, split = blockIdx.x - row * p.splits;
  if (p.finished && p.finished[row]) return;
  const T* logits = static_cast<const T*>(p.logits) + row * p.stride;
  const int skip = static_cast<int>((reinterpret_cast<uintptr_t>(logits) & 15u) / sizeof(T));
  const T* base = logits - skip;
  // The part, in elements from the aligned base.
  const int lo = max(skip, split * p.part);
  const int hi = static_cast<int>(min(static_cast<long long>(skip) + p.vocab, static_cast<long long>(split + 1) * p.part));
  const int first = split * p.part / N;
  const int tiles = hi > lo ? (hi - split * p.part + kTile - 1) / kTile : 0;
  if (tid == 0) s.n = 0;

  uint4 v[kVecs];
#pragma unroll
  for (int u = 0; u < kVecs; ++u) v[u] = load_vec(base, first + u * kThreads + tid, lo, hi);
  float f[kPerThread];
  float ref = -INFINITY;
  uint32_t bar = 0;        // what passes is above it, in the order of ordered()
  Sum sum;
  if (tiles > 0) {
    // The first tile's maximum, and a value that at least `count` of the threads' maxima reach: the upper 16 bits of
    // the largest such.
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      L::unpack(v[u], f + u * N);
#pragma unroll
      for (int i = 0; i < N; ++i) m = fmaxf(m, f[u * N + i]);
    }
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s.warp_max[warp] = top;
    const uint32_t mine = ordered(m + 0.0f) >> 16;
    uint32_t at = 0;
#pragma unroll
    for (int b = 15; b >= 0; --b) {
      const uint32_t probe = at | 1u << b;
      if (__syncthreads_count(mine >= probe) >= p.count) at = probe;
    }
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s.warp_max[w]);
    // (A maximum of infinity makes terms of NaN, which is what the sum is to be.)
    ref = top;
    bar = max(at << 16, ordered(-INFINITY) + 1u) - 1u;
    if (bar == ordered(-0.0f)) --bar;  // (0 and -0 both are above it)
  }
  float above = from_ordered(bar);
  for (int t = 0; t < tiles; ++t) {
    const int at = first + t * (kTile / N) + tid;  // this thread's first vector
#pragma unroll
    for (int u = 0; u < kVecs; ++u) L::unpack(v[u], f + u * N);
    if (t + 1 < tiles) {
#pragma unroll
      for (int u = 0; u < kVecs; ++u) v[u] = load_vec(base, at + kTile / N + u * kThreads, lo, hi);
    }
    float m[kVecs];
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      m[u] = f[u * N];
#pragma unroll
      for (int i = 1; i < N; ++i) m[u] = fmaxf(m[u], f[u * N + i]);
      top = fmaxf(top, m[u]);
    }
    if (__builtin_expect(top > ref + 30.0f, 0)) {  // far above the reference, or the first that is finite: it moves
      const float by = term(ref, top);
      sum.hi *= by;
      sum.lo *= by;
      ref = top;
    }
    const float unit = ref == -INFINITY ? 0.0f : ref;
#pragma unroll
    for (int g = 0; g < kPerThread / 8; ++g) {
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = term(f[g * 8 + i], unit);
      if (__builtin_expect(top > above, 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum.add(e[i]);
      } else {
        sum.add(((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7])));
      }
    }
    // (The barrier also has everybody know the list's length before anybody adds to it.)
    const int could = __syncthreads_count(top > above) * kPerThread;
    const int have = s.n;
    __syncthreads();
    if (have + could <= kList) {
      if (top > above) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
          if (!(m[u] > above)) continue;
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (f[u * N + i] > above) s.list[atomicAdd(&s.n, 1)] = entry(f[u * N + i], (at + u * kThreads) * N + i - skip);
        }
      }
    } else {
#pragma unroll
      for (int u0 = 0; u0 < kSteps; ++u0) {
        __syncthreads();
        const int n = s.n;
        if (n > kListLong) {
          const int found = select_best(s, n, p.count);
          if (tid < found) s.list[tid] = s.best[tid];
          if (tid == 0) s.n = found;
          if (found == p.count) {
            bar = max(bar, static_cast<uint32_t>(s.best[found - 1] >> 32));
            above = from_ordered(bar);
          }
          __syncthreads();
        } else {
          __syncthreads();
        }
#pragma unroll
        for (int u = u0 * kVecs / kSteps; u < (u0 + 1) * kVecs / kSteps; ++u) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (f[u * N + i] > above) s.list[atomicAdd(&s.n, 1)] = entry(f[u * N + i], (at + u * kThreads) * N + i - skip);
        }
      }
      __syncthreads();
    }
  }
  __syncthreads();
  const int found = select_best(s, s.n, p.count);
  // The CTA's largest reference, and the sum in its units.
  float most = ref;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) s.warp_max[warp] = most;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) most = fmaxf(most, s.warp_max[w]);
  double all = static_cast<double>(sum.hi) + static_cast<double>(sum.lo);
  if (ref != most) all *= exp(static_cast<double>(ref) - static_cast<double>(most));
  if (tid < found) {
    // (Where a thread's reference has moved, its term of x was a little different from this one.)
    const float x = entry_x(s.best[tid]);
    all += exp(static_cast<double>(x) - static_cast<double>(most)) - static_cast<double>(term(x, most));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  if (lane == 0) s.warp_sum[warp] = all;
  __syncthreads();
  const long long out = static_cast<long long>(row) * p.splits + split;
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) all += s.warp_sum[w];
    p.part_sum[out] = all;
    p.part_ref[out] = most;
  }
  if (tid < p.count) {
    p.part_x[out * p.count + tid] = tid < found ? entry_x(s.best[tid]) : -INFINITY;
    p.part_token[out * p.count + tid] = tid < found ? entry_token(s.best[tid]) : -1;
  }
}

// Whether (a, i) comes before (b, j): the larger value, of equal ones the lower place.
__device__ __forceinline__ bool before(double a, long long i, double b, long long j) { return a > b || (a == b && i < j); }

// A CTA per user: the beams' log sum exp, then the best of all parts' candidates, taken `count` times. A thread holds
// the best of its own candidates, which are those of some parts' ranks in turn.
__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const BeamParams p) {
  constexpr int kJoinWarps = kJoinThreads / 32;
  // A continuation's value is (x - ref) + shift: the sum of exp(x - ref) is what has been formed. NaN: none.
  __shared__ double shift[MOE_FFN_BEAM_MAX], beam_ref[MOE_FFN_BEAM_MAX];
  __shared__ double warp_value[2][kJoinWarps];
  __shared__ long long warp_place[2][kJoinWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, user = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const long long row0 = static_cast<long long>(user) * p.beams;
  for (int k = warp; k < p.beams; k += kJoinWarps) {
    const long long row = row0 + k;
    if (p.finished && p.finished[row]) continue;
    float top = -INFINITY;
    for (int i = lane; i < p.splits; i += 32) top = fmaxf(top, p.part_ref[row * p.splits + i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    double sum = 0.0;
    for (int i = lane; i < p.splits; i += 32)
      sum += p.part_sum[row * p.splits + i] * exp(static_cast<double>(p.part_ref[row * p.splits + i]) - static_cast<double>(top));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      shift[k] = static_cast<double>(p.scores[row]) - log(sum);
      beam_ref[k] = top;
    }
  }
  __syncthreads();
  const int per_beam = p.splits * p.count, n = p.beams * per_beam;
  // The best of this thread's candidates that come after (value, place).
  double best;
  long long place;
  auto look = [&](double after, long long after_place) {
    best = -INFINITY;
    place = 0x7fffffffffffffffLL;
    for (int i = tid; i < n; i += kJoinThreads) {
      const int k = i / per_beam;
      double v;
      long long at;
      if (p.finished && p.finished[row0 + k]) {
        if (i - k * per_beam != 0) continue;
        v = static_cast<double>(p.scores[row0 + k]);
        at = static_cast<long long>(k) * p.vocab + p.end_token;
      } else {
        const int token = p.part_token[row0 * per_beam + i];
        if (token < 0) continue;
        v = (static_cast<double>(p.part_x[row0 * per_beam + i]) - beam_ref[k]) + shift[k];
        at = static_cast<long long>(k) * p.vocab + token;
      }
      if (v > -INFINITY && before(after, after_place, v, at) && before(v, at, best, place)) {
        best = v;
        place = at;
      }
    }
  };
  look(INFINITY, -1);
  for (int c = 0; c < p.count; ++c) {
    double v = best;
    long long at = place;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double w = __shfl_xor_sync(0xffffffffu, v, o);
      const long long a = __shfl_xor_sync(0xffffffffu, at, o);
      if (before(w, a, v, at)) {
        v = w;
        at = a;
      }
    }
    if (lane == 0) {
      warp_value[c & 1][warp] = v;
      warp_place[c & 1][warp] = at;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      if (before(warp_value[c & 1][w], warp_place[c & 1][w], v, at)) {
        v = warp_value[c & 1][w];
        at = warp_place[c & 1][w];
      }
    }
    const bool some = v > -INFINITY;
    if (tid == 0) {
      const long long o = static_cast<long long>(user) * p.count + c;
      p.out_scores[o] = static_cast<float>(v);
      p.out_beams[o] = some ? static_cast<int>(at / p.vocab) : -1;
      p.out_tokens[o] = some ? static_cast<int>(at % p.vocab) : -1;
    }
    if (some && best == v && place == at) look(v, at);
  }
}

// Parts of a row: enough for three CTAs on each SM, of a tile at least, and few tiles where rows are long, so that
// the lists stay short.
int beam_splits(int rows, int vocab) {
  const int tiles = (vocab + 8 + kTile - 1) / kTile;
  int splits = (3 * 152 + rows - 1) / (rows > 0 ? rows : 1);
  const int least = (tiles + 15) / 16;
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
  const size_t parts = static_cast<size_t>(users) * beams * beam_splits(users * beams, vocab);
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
  p.part_sum = reinterpret_cast<double*>(ws + l.sum);
  p.part_ref = reinterpret_cast<float*>(ws + l.ref);
  p.part_x = reinterpret_cast<float*>(ws + l.x);
  p.part_token = reinterpret_cast<int32_t*>(ws + l.token);
  p.end_token = a->end_token;
  p.beams = a->beams;
  p.vocab = a->vocab;
  p.count = a->count;
  p.splits = beam_splits(rows, a->vocab);
  p.part = ((a->vocab + 8 + p.splits - 1) / p.splits + 7) / 8 * 8;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = a->logits_fp32 ? launch_pdl(beam_part_kernel<float>, dim3(p.splits * rows), dim3(kThreads), 0, s, p)
                                 : launch_pdl(beam_part_kernel<uint16_t>, dim3(p.splits * rows), dim3(kThreads), 0, s, p);
  if (e == cudaSuccess) e = launch_pdl(beam_join_kernel, dim3(a->users), dim3(kJoinThreads), 0, s, p);
  return e == cudaSuccess ? MOE_FFN_OK : MOE_FFN_ECUDA;
}
