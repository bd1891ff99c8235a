// Device pieces that the paged kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "lf_device.cuh"
#include "lf_paged.h"
#include "longflow.h"

namespace lf {

constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes global -> shared, or 16 zero bytes when `valid` is 0 (nothing is read then).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int valid) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two floats as packed bf16 (x in the low half), rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}

// Shared-memory chunk of (row, 16-byte chunk c) in a tile of rows of NC chunks:
// the low bits of c are XORed with the row's place among the rows that share
// its banks, so that eight rows' equal chunks fall into eight bank groups.
template <int NC>
__device__ __forceinline__ int tile_chunk(int row, int c) {
  if constexpr (NC >= 8) return row * NC + (c ^ (row & 7));
  else return row * NC + (c ^ ((row / (8 / NC)) & (NC - 1)));
}

// Two floats in a register pair, for the instructions that take both at once.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float* x, float* y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*x), "=f"(*y) : "l"(p));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// The key tiles of `size` tokens that queries at positions p_lo .. p_hi visit: [0, sink)
// and [from, to).
struct Tiles {
  int sink, from, to;
  __device__ Tiles(const PagedPromptArgs& a, int p_lo, int p_hi, int size) : sink(0), from(0), to(0) {
    if (p_hi < 0) return;
    to = p_hi / size + 1;
    if (a.window > 0) {
      from = (int)max((int64_t)0, (int64_t)p_lo - a.window + 1) / size;
      sink = min((int)(((int64_t)a.sinks + size - 1) / size), from);
    }
  }
  __device__ int count() const { return sink + to - from; }
  __device__ int at(int j) const { return j < sink ? j : from + j - sink; }
};

// Does some query at positions p_lo .. p_hi not see some of the `size` keys from k0 on?
__device__ __forceinline__ bool some_hidden(const PagedPromptArgs& a, int p_lo, int p_hi, int k0, int size) {
  return k0 + size - 1 > p_lo ||
         (a.window > 0 && k0 + size > a.sinks && (int64_t)k0 <= (int64_t)p_hi - a.window);
}

// One row by the definition, a warp at a time: for CTAs whose tiles held values
// that are not finite where some row does not look (0 * NaN is NaN).
template <typename T, int D>
__device__ __noinline__ void row_by_hand(const PagedPromptArgs& a, int b, int g, int64_t row, int pos,
                                         int lane) {
  constexpr int E = D >= 32 ? D / 32 : 1;
  const bool mine = lane * E < D;   // lanes past a short row take nothing
  const T* q = reinterpret_cast<const T*>(a.q) + row * D + lane * E;
  float qv[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = mine ? to_f32(q[e]) : 0.f;
    acc[e] = 0.f;
  }
  float m = kNegInf, l = 0.f;
  for (int p = 0; p <= pos; ++p) {
    if (a.window > 0 && p >= a.sinks && p <= pos - a.window) p = pos - a.window + 1;
    int pi, slot;
    paged_split(a.pool, p, &pi, &slot);
    const int page = a.pool.table[(int64_t)b * a.pool.max_pages + pi];
    if (page < 0 || page >= a.pool.num_pages) continue;
    const int64_t off = page * a.pool.page_stride + slot * a.pool.token_stride + g * a.pool.head_stride;
    const T* k = reinterpret_cast<const T*>(a.pool.k + off) + lane * E;
    const T* v = reinterpret_cast<const T*>(a.pool.v + off) + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) if (mine) s = fmaf(qv[e], to_f32(k[e]), s);
    s = warp_sum(s) * a.scale_log2;
    const float mn = fmaxf(m, s), mu = mn == kNegInf ? 0.f : mn;
    const float f = ex2(m - mu), w = ex2(s - mu);
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < E; ++e) if (mine) acc[e] = acc[e] * f + w * to_f32(v[e]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = reinterpret_cast<T*>(a.out) + row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (mine) from_f32(l == 0.f ? 0.f : acc[e] * inv, out + e);
  if (lane == 0) {
    if (a.lse) a.lse[row] = l == 0.f ? kNegInf : (m + log2f(l)) * 0.6931471805599453f;
    if (a.pool.err && !(l <= 3.0e38f)) atomicOr(a.pool.err, LF_DEVERR_NONFINITE);
  }
}

}  // namespace lf
