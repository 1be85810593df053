// kv_mma.cuh — what the kernels that keep few rows against many keys share: mma.sync with the keys as its rows, e4m3 codes
// widened on the way, and equal shares of the work.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "kv.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kComputeWarps = 8;

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

__device__ __forceinline__ void ldsm2_trans(uint32_t addr, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four e4m3 codes as two pairs of fp16, exactly.
__device__ __forceinline__ void widen_e4m3(uint32_t y, uint32_t& even, uint32_t& odd) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(even), "=r"(odd)
      : "r"(y));
}

// The computing warps.
__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The same, with the disjunction of a condition.
__device__ __forceinline__ bool compute_sync_or(bool c) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbar.red.or.pred q, 1, 256, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(c ? 1 : 0)
      : "memory");
  return r != 0;
}

// Where CTA x's share begins, and the CTA whose share holds a unit. (64-bit divisions are long; few batches
// need them.)
__device__ __forceinline__ long long decode_share(int x, long long total, int ctas) {
  if (total < (1 << 22)) return static_cast<unsigned>(x) * static_cast<unsigned>(total) / static_cast<unsigned>(ctas);
  return x * total / ctas;
}
__device__ __forceinline__ int decode_owner(long long unit, long long total, int ctas) {
  if (total < (1 << 22))
    return (static_cast<unsigned>(unit + 1) * static_cast<unsigned>(ctas) - 1) / static_cast<unsigned>(total);
  return static_cast<int>(((unit + 1) * ctas - 1) / total);
}

// Writes rows of zeros (and -infinity) for `rows` rows of one head from `first` on, of which the caller
// takes number `id` of every `of`.
template <int D>
__device__ __forceinline__ void clear_rows(const KvAttn& a, long long first, long long rows, long long id, long long of) {
  for (long long i = id; i < rows; i += of) {
    const long long to = first + i;
    for (int j = 0; j < D; j += 8) *reinterpret_cast<uint4*>(a.out + to * D + j) = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse) a.lse[to] = -INFINITY;
  }
}

}  // namespace

}  // namespace moe
