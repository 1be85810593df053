// rotary.cu — rotary positions with one or several axes, on queries and keys in one launch.
//
// Pair i of a head turns by the angle positions[axis[i], token] * freq[i]. Each value is read and written once (4 bytes
// meet 3 operations), so HBM bounds it, or the launch where tokens are few. A CTA takes a token. A thread has the same
// two vectors of pairs in several heads: it loads those of its first heads, the CTA forms the token's cosines and
// sines, each once, while these are under way, and the thread keeps its own in registers for all its heads. (Read
// from shared memory for each head they bounded the kernel: 79 us for 9001 tokens of 18 heads of width 512. It is 52.7 now,
// 94% of the copy rate; interleaved 57, with 188 pairs, which go by 8 bytes, 55. Narrow heads are further from it: 9001
// tokens of 32 heads of width 72 take 17 us, where the bytes are 12.5.) 64 tokens of 24 heads take 2.3 us in a graph, and
// the call from Python 11 to 16.
//
// Angles. In fp32 a position of a million leaves a tenth of a radian unknown, and in fp64 an angle would cost more
// than the rest. Here a frequency is a fraction of a turn in 64-bit fixed point, rounded from the exact quotient (to 2^-65):
// its product with the position, modulo 2^64, is the angle modulo a turn to 2^-34, and its upper 32 bits, as a signed
// number and rounded to nearest (to 2^-33), the angle in (-1/2, 1/2] turns, which sincospif takes.
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "moe_ffn.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 128;   // at least, where heads are narrow
constexpr int kMaxThreads = 160;
constexpr int kAtOnce = 4;      // heads of a thread whose loads are under way together

struct Rows {
  const uint16_t* in;
  uint16_t* out;
  long long in_token, in_head, out_token, out_head;
};

struct RotaryParams {
  Rows q, k;
  const moe_ffn_rotary_pair* table;
  const int32_t* positions;
  long long positions_stride;
  float scale;
  float sign;
  int pairs, axes, head_dim, q_heads, k_heads;
  int copy;  // whether elements after the pairs are to be copied
};

template <int VEC>
struct Vec;
template <>
struct Vec<8> {
  using T = uint4;
};
template <>
struct Vec<4> {
  using T = uint2;
};

template <int VEC>
__device__ __forceinline__ void unpack(const typename Vec<VEC>::T& v, float (&f)[VEC]) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

template <int VEC>
__device__ __forceinline__ typename Vec<VEC>::T pack(const float (&f)[VEC]) {
  typename Vec<VEC>::T v;
  uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return v;
}

// VEC: bf16 values of a vector. Of a head, `turned` threads have the vector of first elements and the one of second
// elements (interleaved: two neighbouring vectors' worth of pairs) of VEC pairs each, the `per - turned` next ones two
// vectors of the elements after them each, where these go elsewhere. `across` heads are taken side by side.
template <int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kMaxThreads) rotary_kernel(const RotaryParams p, int turned, int per, int across) {
  using V = typename Vec<VEC>::T;
  __shared__ alignas(16) float2 cs[MOE_FFN_ROTARY_MAX_PAIRS];
  pdl_wait();
  pdl_launch_dependents();
  const long long token = blockIdx.x;
  const int first = threadIdx.x / per, i = threadIdx.x - first * per;
  const bool turns = i < turned, live = first < across;
  // Elements where the two vectors begin.
  int x, y;
  if (turns) {
    x = INTERLEAVED ? 2 * i * VEC : i * VEC;
    y = INTERLEAVED ? x + VEC : x + p.pairs;
  } else {
    x = 2 * p.pairs + 2 * (i - turned) * VEC;
    y = x + VEC;
  }
  const bool two = y + VEC <= p.head_dim;
  const int heads = live ? p.q_heads + p.k_heads : 0;
  const uint16_t* q_in = p.q.in + token * p.q.in_token;
  const uint16_t* k_in = p.k.in + token * p.k.in_token;
  uint16_t* q_out = p.q.out + token * p.q.out_token;
  uint16_t* k_out = p.k.out + token * p.k.out_token;
  V a[kAtOnce], b[kAtOnce];
  auto load = [&](int head0) {
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int head = head0 + j * across;
      if (head >= heads) continue;
      const uint16_t* from = head < p.q_heads ? q_in + head * p.q.in_head : k_in + (head - p.q_heads) * p.k.in_head;
      a[j] = *reinterpret_cast<const V*>(from + x);
      if (two) b[j] = *reinterpret_cast<const V*>(from + y);
    }
  };
  load(first);
  for (int k = threadIdx.x; k < p.pairs; k += blockDim.x) {
    const ulonglong2 e = *reinterpret_cast<const ulonglong2*>(p.table + k);
    const int axis = e.y < static_cast<unsigned long long>(p.axes) ? static_cast<int>(e.y) : 0;
    const long long pos = p.positions[axis * p.positions_stride + token];
    const unsigned long long turn = e.x * static_cast<unsigned long long>(pos);
    // The nearest number of 2^-32 turns; two of them to a half.
    const int near = static_cast<int>((turn + 0x80000000ull) >> 32);
    float s, c;
    sincospif(static_cast<float>(near) * 0x1p-31f, &s, &c);
    cs[k] = make_float2(c * p.scale, s * p.scale * p.sign);
  }
  __syncthreads();
  float2 u[VEC];
  if (live && turns) {
#pragma unroll
    for (int k = 0; k < VEC; k += 2) {
      const float4 w = *reinterpret_cast<const float4*>(&cs[i * VEC + k]);
      u[k] = make_float2(w.x, w.y);
      u[k + 1] = make_float2(w.z, w.w);
    }
  }
  for (int head0 = first; head0 < heads; head0 += kAtOnce * across) {
    if (head0 != first) load(head0);
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int head = head0 + j * across;
      if (head >= heads) continue;
      if (turns) {
        float f[VEC], g[VEC];
        unpack<VEC>(a[j], f);
        unpack<VEC>(b[j], g);
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int k = 0; k < VEC / 2; ++k) {
            const float2 v = u[k], w = u[VEC / 2 + k];
            const float f0 = f[2 * k], g0 = g[2 * k];
            f[2 * k] = f0 * v.x - f[2 * k + 1] * v.y;
            f[2 * k + 1] = f[2 * k + 1] * v.x + f0 * v.y;
            g[2 * k] = g0 * w.x - g[2 * k + 1] * w.y;
            g[2 * k + 1] = g[2 * k + 1] * w.x + g0 * w.y;
          }
        } else {
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            const float f0 = f[k];
            f[k] = f0 * u[k].x - g[k] * u[k].y;
            g[k] = g[k] * u[k].x + f0 * u[k].y;
          }
        }
        a[j] = pack<VEC>(f);
        b[j] = pack<VEC>(g);
      }
      uint16_t* to = head < p.q_heads ? q_out + head * p.q.out_head : k_out + (head - p.q_heads) * p.k.out_head;
      *reinterpret_cast<V*>(to + x) = a[j];
      if (two) *reinterpret_cast<V*>(to + y) = b[j];
    }
  }
}

template <int VEC, bool INTERLEAVED>
cudaError_t launch(const RotaryParams& p, int tokens, cudaStream_t s) {
  const int turned = p.pairs / VEC, rest = p.copy ? (p.head_dim - 2 * p.pairs) / VEC : 0;
  const int per = turned + (rest + 1) / 2;
  // As many heads side by side as a CTA of about kThreads threads has room for, and there are.
  const int heads = p.q_heads + p.k_heads;
  int across = per >= kThreads ? 1 : kThreads / per;
  if (across > heads) across = heads;
  const int threads = (per * across + 31) / 32 * 32;
  return launch_pdl(rotary_kernel<VEC, INTERLEAVED>, dim3(tokens), dim3(threads), 0, s, p, turned, per, across);
}

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// [tokens, heads, dim] bf16 values, in bytes.
struct Extent {
  uintptr_t at;
  long long token, head;
};

Extent extent(const moe_ffn_kv_rows& r, int tokens, int heads) {
  return {reinterpret_cast<uintptr_t>(r.ptr), tokens > 1 ? 2 * r.token_stride : 0, heads > 1 ? 2 * r.head_stride : 0};
}

bool apart_modulo(uintptr_t a, long long an, uintptr_t b, long long bn, long long s) {
  if (s < an + bn) return false;
  const long long d = a <= b ? static_cast<long long>((b - a) % s) : (s - static_cast<long long>((a - b) % s)) % s;
  return d >= an && s - d >= bn;
}

// Whether two tensors certainly have no byte in common: one lies before the other, or their tokens (or heads) lie
// between each other's, at one stride.
bool apart(const Extent& a, int a_heads, const Extent& b, int b_heads, int tokens, int dim) {
  const long long row = 2LL * dim;
  const long long an = (a_heads - 1) * a.head + row, bn = (b_heads - 1) * b.head + row;  // a token's
  const long long at = (tokens - 1) * a.token, bt = (tokens - 1) * b.token;
  if (a.at + at + an <= b.at || b.at + bt + bn <= a.at) return true;
  if (tokens > 1 && a.token == b.token && a.token > 0 && apart_modulo(a.at, an, b.at, bn, a.token)) return true;
  return a_heads > 1 && b_heads > 1 && a.head == b.head && a.head > 0 && apart_modulo(a.at, at + row, b.at, bt + row, a.head);
}

// 2 pi / 8 in binary, a fraction of 1280 bits, the highest word first.
constexpr uint64_t kEighthOfTurn[20] = {
    0xc90fdaa22168c234ull, 0xc4c6628b80dc1cd1ull, 0x29024e088a67cc74ull, 0x020bbea63b139b22ull,
    0x514a08798e3404ddull, 0xef9519b3cd3a431bull, 0x302b0a6df25f1437ull, 0x4fe1356d6d51c245ull,
    0xe485b576625e7ec6ull, 0xf44c42e9a637ed6bull, 0x0bff5cb6f406b7edull, 0xee386bfb5a899fa5ull,
    0xae9f24117c4b1fe6ull, 0x49286651ece45b3dull, 0xc2007cb8a163bf05ull, 0x98da48361c55d39aull,
    0x69163fa8fd24cf5full, 0x83655d23dca3ad96ull, 0x1c62f356208552bbull, 0x9ed529077096966dull};

// x / 2 pi modulo 1, times 2^64, of x >= 0, rounded to nearest: a long division, a bit at a time. (A quotient in fp64 is
// known to 2^-53 of itself, which a position of 2^31 makes 2^-25 turns at x = 1, and a large x a part of a turn.)
uint64_t turn_of(double x) {
  if (x == 0.0) return 0;
  int exponent;
  const double f = std::frexp(x, &exponent);  // [1/2, 1)
  const int last = exponent + 61;              // x / 2 pi 2^64 = f / (2 pi / 8) 2^last
  if (last < -1) return 0;
  // The divisor's words after these change the quotient by less than 2^-64 of its last bit.
  const int n = (last + 64) / 64 + 1;
  static_assert((1024 + 61 + 64) / 64 + 1 <= 20, "words");
  uint64_t r[20] = {static_cast<uint64_t>(std::ldexp(f, 64))}, q = 0;
  for (int bit = 0; bit <= last + 1; ++bit) {
    uint64_t carry = 0;
    if (bit > 0)
      for (int i = n - 1; i >= 0; --i) {
        const uint64_t out = r[i] >> 63;
        r[i] = r[i] << 1 | carry;
        carry = out;
      }
    bool less = false;
    if (carry == 0)
      for (int i = 0; i < n; ++i)
        if (r[i] != kEighthOfTurn[i]) {
          less = r[i] < kEighthOfTurn[i];
          break;
        }
    if (!less) {
      uint64_t borrow = 0;
      for (int i = n - 1; i >= 0; --i) {
        const uint64_t was = r[i], d = kEighthOfTurn[i];
        r[i] = was - d - borrow;
        borrow = was < d || (was == d && borrow != 0) ? 1 : 0;
      }
    }
    // The bits up to the last, as many as 64 hold, then the one that rounds.
    q = bit <= last ? q << 1 | (less ? 0 : 1) : q + (less ? 0 : 1);
  }
  return q;
}

bool own_rows_apart(const Extent& e, int tokens, int heads, int dim) {
  const long long row = 2LL * dim;
  if (heads > 1 && e.head < row) return false;
  if (tokens > 1 && e.token < row) return false;
  return heads <= 1 || tokens <= 1 || e.token >= (heads - 1) * e.head + row || e.head >= (tokens - 1) * e.token + row;
}

}  // namespace

}  // namespace moe

extern "C" int moe_ffn_rotary_table(const double* freq, const int* axis, int pairs, moe_ffn_rotary_pair* table) {
  if (!freq || !axis || !table || pairs < 1 || pairs > MOE_FFN_ROTARY_MAX_PAIRS) return MOE_FFN_EINVAL;
  for (int i = 0; i < pairs; ++i)
    if (!std::isfinite(freq[i]) || axis[i] < 0 || axis[i] >= MOE_FFN_ROTARY_MAX_AXES) return MOE_FFN_EINVAL;
  for (int i = 0; i < pairs; ++i) {
    const uint64_t t = moe::turn_of(std::fabs(freq[i]));
    table[i].turn = freq[i] < 0.0 ? 0 - t : t;
    table[i].axis = static_cast<uint64_t>(axis[i]);
  }
  return MOE_FFN_OK;
}

extern "C" int moe_ffn_rotary_apply(const moe_ffn_rotary* a, const moe_ffn_kv_rows* q, const moe_ffn_kv_rows* k,
                                    const moe_ffn_kv_rows* q_out, const moe_ffn_kv_rows* k_out, void* stream) {
  using namespace moe;
  if (!a || a->tokens < 0 || a->pairs < 4 || a->pairs > MOE_FFN_ROTARY_MAX_PAIRS || a->pairs % 4 != 0 ||
      a->head_dim < 8 || a->head_dim > 1024 || a->head_dim % 8 != 0 || 2 * a->pairs > a->head_dim || a->axes < 1 ||
      a->axes > MOE_FFN_ROTARY_MAX_AXES || a->q_heads < 0 || a->q_heads > 1024 || a->k_heads < 0 || a->k_heads > 1024 ||
      !std::isfinite(a->scale) || a->positions_stride < 0)
    return MOE_FFN_EINVAL;
  if (a->tokens == 0 || a->q_heads + a->k_heads == 0) return MOE_FFN_OK;
  if (!a->table || !a->positions) return MOE_FFN_EINVAL;
  if (off16(a->table) || (reinterpret_cast<uintptr_t>(a->positions) & 3u) != 0) return MOE_FFN_EALIGN;
  const moe_ffn_kv_rows* given[2][2] = {{q, q_out}, {k, k_out}};
  const int heads[2] = {a->q_heads, a->k_heads};
  Extent ins[2], outs[2];
  bool in_place[2] = {false, false};
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    for (const moe_ffn_kv_rows* r : given[i]) {
      if (!r || !r->ptr || r->token_stride < 0 || r->head_stride < 0) return MOE_FFN_EINVAL;
      if (off16(r->ptr) || r->token_stride % 8 != 0 || r->head_stride % 8 != 0) return MOE_FFN_EALIGN;
    }
    ins[i] = extent(*given[i][0], a->tokens, heads[i]);
    outs[i] = extent(*given[i][1], a->tokens, heads[i]);
    in_place[i] = ins[i].at == outs[i].at && ins[i].token == outs[i].token && ins[i].head == outs[i].head;
    if (!own_rows_apart(outs[i], a->tokens, heads[i], a->head_dim)) return MOE_FFN_EINVAL;
  }
  const size_t table_bytes = a->pairs * sizeof(moe_ffn_rotary_pair);
  const size_t positions_bytes = ((a->axes - 1) * a->positions_stride + a->tokens) * sizeof(int32_t);
  for (int o = 0; o < 2; ++o) {
    if (heads[o] == 0) continue;
    for (int i = 0; i < 2; ++i) {
      if (heads[i] == 0) continue;
      if (!(i == o && in_place[i]) && !apart(outs[o], heads[o], ins[i], heads[i], a->tokens, a->head_dim))
        return MOE_FFN_EINVAL;
      if (i != o && !apart(outs[o], heads[o], outs[i], heads[i], a->tokens, a->head_dim)) return MOE_FFN_EINVAL;
    }
    const uintptr_t end = outs[o].at + (a->tokens - 1) * outs[o].token + (heads[o] - 1) * outs[o].head + 2 * a->head_dim;
    const uintptr_t t = reinterpret_cast<uintptr_t>(a->table), x = reinterpret_cast<uintptr_t>(a->positions);
    if ((t < end && outs[o].at < t + table_bytes) || (x < end && outs[o].at < x + positions_bytes)) return MOE_FFN_EINVAL;
  }
  RotaryParams p = {};
  Rows* rows[2] = {&p.q, &p.k};
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    rows[i]->in = static_cast<const uint16_t*>(given[i][0]->ptr);
    rows[i]->out = static_cast<uint16_t*>(const_cast<void*>(given[i][1]->ptr));
    rows[i]->in_token = given[i][0]->token_stride;
    rows[i]->in_head = given[i][0]->head_stride;
    rows[i]->out_token = given[i][1]->token_stride;
    rows[i]->out_head = given[i][1]->head_stride;
    if (!in_place[i]) p.copy = 1;
  }
  p.table = a->table;
  p.positions = a->positions;
  p.positions_stride = a->positions_stride;
  p.scale = a->scale;
  p.sign = a->inverse ? -1.0f : 1.0f;
  p.pairs = a->pairs;
  p.axes = a->axes;
  p.head_dim = a->head_dim;
  p.q_heads = a->q_heads;
  p.k_heads = a->k_heads;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Vectors of 16 bytes where the second elements of the pairs begin at a multiple of that, of 8 else.
  cudaError_t e;
  if (a->pairs % 8 == 0) e = a->interleaved ? launch<8, true>(p, a->tokens, s) : launch<8, false>(p, a->tokens, s);
  else e = a->interleaved ? launch<4, true>(p, a->tokens, s) : launch<4, false>(p, a->tokens, s);
  return e == cudaSuccess ? MOE_FFN_OK : MOE_FFN_ECUDA;
}
