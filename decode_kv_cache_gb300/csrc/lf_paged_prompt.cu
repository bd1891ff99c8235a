// Causal attention of the last tokens of every sequence over a paged key-value
// cache, with an optional sliding window and sinks: the CUDA-core kernel.
//
//   out_i = sum_j 2^(s_ij - m_i) v_j / sum_j 2^(s_ij - m_i),  s = q . k log2(e) / sqrt(d)
//
// over j <= i and (no window, or j > i - window, or j < sinks), in one pass over
// the keys with the running maximum m_i and sum of every row.
//
// A CTA takes 64 rows, (token, head of the group) pairs with the head inner: every
// key and value it loads serves all heads of the group.  Keys and values pass
// through shared memory in tiles of 64 tokens, gathered by page; key tiles that no
// row sees are not visited.  A thread holds a 4 x 4 piece of S and 4 rows x d/16
// columns of O.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "lf_device.cuh"
#include "lf_paged.h"
#include "longflow.h"

namespace lf {

namespace {

constexpr int kRows = 64, kKeys = 64, kThreadsP = 256;
constexpr float kNegInfP = -INFINITY;

__device__ __forceinline__ float ex2p(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T, int D>
constexpr int prompt_smem() {
  return (2 * 64 * (D + 4) + kKeys * (kRows + 4)) * 4;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsP) paged_prompt_simt_kernel(const __grid_constant__ PagedPromptArgs a) {
  constexpr int LD = D + 4;           // row stride in floats: eight rows' equal chunks differ in bank
  constexpr int CW = D / 16;          // columns of O per thread
  constexpr int VW = CW < 4 ? CW : 4; // .. in runs of
  constexpr int PER = 16 / sizeof(T); // elements of a 16-byte chunk
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;                     // [kRows][LD]
  float* skv = sm + kRows * LD;       // [kKeys][LD]
  float* sp = skv + kKeys * LD;       // [kKeys][kRows + 4], transposed weights
  __shared__ int64_t s_off[kKeys];

  const int b = blockIdx.z, g = blockIdx.y, tid = threadIdx.x;
  const int G = a.group;
  const int q0 = a.q_start[b], n = a.q_start[b + 1] - q0;
  const bool head_block = blockIdx.x == 0 && g == 0 && tid == 0;
  if (q0 < 0 || n < 0 || n > a.total_q - q0) {   // not rows of q
    if (head_block && a.pool.err) atomicOr(a.pool.err, LF_DEVERR_STATE);
    return;
  }
  const int len = paged_len(a.pool, b);
  if (head_block && a.pool.err && (n > a.max_q || len != a.pool.lens[b] || n > len))
    atomicOr(a.pool.err, LF_DEVERR_STATE);
  // The last rows see the most keys: they start first.
  const int64_t r0 = (int64_t)(gridDim.x - 1 - blockIdx.x) * kRows;
  const int64_t rows = (int64_t)n * G;
  if (r0 >= rows) return;
  const int first_pos = len - n;      // may be negative: those rows see nothing
  const int p_lo = first_pos + (int)(r0 / G);
  const int p_hi = first_pos + (int)((min(r0 + kRows, rows) - 1) / G);

  for (int i = tid; i < kRows * (D / PER); i += kThreadsP) {
    const int r = i / (D / PER), c = i - r * (D / PER);
    float x[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) x[e] = 0.f;
    if (r0 + r < rows) {
      const int64_t t = q0 + (r0 + r) / G, h = g * G + (r0 + r) % G;
      load16_f32(reinterpret_cast<const T*>(a.q) + (t * a.q_heads + h) * D + c * PER, x);
    }
#pragma unroll
    for (int e = 0; e < PER; e += 4)
      *reinterpret_cast<float4*>(sq + r * LD + c * PER + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
  }

  const int rg = tid >> 4, cg = tid & 15;
  int pos[4];
  float m[4], l[4], o[4][CW];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + rg * 4 + i;
    pos[i] = r < rows ? first_pos + (int)(r / G) : -1;
    m[i] = kNegInfP;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < CW; ++c) o[i][c] = 0.f;
  }
  auto load_rows = [&](const char* pool) {   // a tile of keys or values, zeros where nothing is read
    for (int i = tid; i < kKeys * (D / PER); i += kThreadsP) {
      const int r = i / (D / PER), c = i - r * (D / PER);
      float x[PER];
#pragma unroll
      for (int e = 0; e < PER; ++e) x[e] = 0.f;
      if (s_off[r] >= 0)
        load16_f32(reinterpret_cast<const T*>(pool + s_off[r] + g * a.pool.head_stride) + c * PER, x);
#pragma unroll
      for (int e = 0; e < PER; e += 4)
        *reinterpret_cast<float4*>(skv + r * LD + c * PER + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    }
  };

  for (int k0 = 0; k0 <= p_hi; k0 += kKeys) {
    if (a.window > 0 && k0 >= a.sinks) {   // past the sinks: on to the window of the first row
      const int64_t lo = (int64_t)p_lo - a.window + 1;
      if (lo > k0) k0 = max(k0, (int)lo / kKeys * kKeys);
    }
    __syncthreads();
    if (tid < kKeys) {
      const int p = k0 + tid;
      int64_t off = -1;
      if (p <= p_hi) {
        int pi, slot;
        paged_split(a.pool, p, &pi, &slot);
        const int page = a.pool.table[(int64_t)b * a.pool.max_pages + pi];
        if (page >= 0 && page < a.pool.num_pages)
          off = page * a.pool.page_stride + slot * a.pool.token_stride;
        else if (a.pool.err)
          atomicOr(a.pool.err, LF_DEVERR_STATE);
      }
      s_off[tid] = off;
    }
    __syncthreads();
    load_rows(a.pool.k);
    __syncthreads();
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(sq + (rg * 4 + i) * LD + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(skv + (cg + 16 * j) * LD + d);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
          s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
          s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
          s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = k0 + cg + 16 * j;
        const bool see = p <= pos[i] && (a.window == 0 || p > pos[i] - a.window || p < a.sinks);
        s[i][j] = see ? s[i][j] * a.scale_log2 : kNegInfP;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float mu = top == kNegInfP ? 0.f : top;
      const float f = ex2p(m[i] - mu);
      m[i] = top;
      l[i] *= f;
#pragma unroll
      for (int c = 0; c < CW; ++c) o[i][c] *= f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = ex2p(s[i][j] - mu);
        l[i] += s[i][j];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4*>(sp + (cg + 16 * j) * (kRows + 4) + rg * 4) =
          make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
    __syncthreads();
    load_rows(a.pool.v);
    __syncthreads();
    // Where some row does not see some key of the tile, a weight of zero takes
    // nothing of the value, which may hold anything there.
    const bool masked = k0 + kKeys - 1 > p_lo || p_lo < 0 ||
                        (a.window > 0 && k0 + kKeys > a.sinks && k0 <= p_hi - a.window);
    auto accumulate = [&](auto part) {
#pragma unroll 4
      for (int k = 0; k < kKeys; ++k) {
        const float4 p = *reinterpret_cast<const float4*>(sp + k * (kRows + 4) + rg * 4);
        const float pi[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int c = 0; c < CW; c += VW) {
          float v[VW];
          const float* src = skv + k * LD + (c / VW) * 16 * VW + cg * VW;
          if constexpr (VW == 4) load16_f32(src, v);
          else if constexpr (VW == 2) {
            const float2 t = *reinterpret_cast<const float2*>(src);
            v[0] = t.x;
            v[1] = t.y;
          } else v[0] = *src;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < VW; ++e)
              if (!part.value || pi[i] != 0.f) o[i][c + e] = fmaf(pi[i], v[e], o[i][c + e]);
        }
      }
    };
    if (masked) accumulate(std::true_type{});
    else accumulate(std::false_type{});
  }

#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float ls = l[i];
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
    const int64_t r = r0 + rg * 4 + i;
    if (r >= rows) continue;
    const float inv = ls == 0.f ? 0.f : 1.f / ls;
    const int64_t row = (q0 + r / G) * a.q_heads + g * G + r % G;
    T* out = reinterpret_cast<T*>(a.out) + row * D;
#pragma unroll
    for (int c = 0; c < CW; ++c)
      from_f32(o[i][c] * inv, out + (c / VW) * 16 * VW + cg * VW + c % VW);
    if (cg == 0) {
      if (a.lse) a.lse[row] = ls == 0.f ? kNegInfP : (m[i] + log2f(ls)) * 0.6931471805599453f;
      if (a.pool.err && !(ls <= 3.0e38f)) atomicOr(a.pool.err, LF_DEVERR_NONFINITE);
    }
  }
}

template <typename T, int D>
cudaError_t launch(const PagedPromptArgs& a, cudaStream_t stream) {
  constexpr int kSmem = prompt_smem<T, D>();
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(&paged_prompt_simt_kernel<T, D>), kSmem, done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((int64_t)a.max_q * a.group + kRows - 1) / kRows;
  paged_prompt_simt_kernel<T, D><<<dim3((unsigned)tiles, a.pool.kv_heads, a.pool.batch), kThreadsP, kSmem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_dim(const PagedPromptArgs& a, int head_dim, cudaStream_t stream) {
  switch (head_dim) {
    case 16: return launch<T, 16>(a, stream);
    case 32: return launch<T, 32>(a, stream);
    case 64: return launch<T, 64>(a, stream);
    default: return launch<T, 128>(a, stream);
  }
}

}  // namespace

cudaError_t paged_prompt_launch(const PagedPromptArgs& a, int elem, int head_dim, cudaStream_t stream) {
  cudaError_t e;
  if (elem == 2 && paged_prompt_tc_launch(a, head_dim, stream, &e)) return e;
  return elem == 2 ? launch_dim<__nv_bfloat16>(a, head_dim, stream) : launch_dim<float>(a, head_dim, stream);
}

}  // namespace lf
