// Attention of a piece of rows over a paged cache, in tiles of 64 keys: the kernels of bf16 caches whose heads or
// pages the tensor-core kernels do not take, and of fp32 caches.  What the rows are, what they see and where
// their results go is a Task's matter: PromptTask, the queries of a prompt (causal, lf_paged_prompt.cu), and
// SharedTask, the last tokens of a group of sequences before its shared prefix (lf_paged_shared.cu).
//
// A Task has its Args, and
//   take(a, per_piece, keys), take_level           the block's rows and its key tiles of `keys`; false: it has none
//   count(), at(j)                                 its key tiles
//   live(a, r), q_row(a, r), pos(a, r)             is there a row r, its row of q, the last position it may see (or -1)
//   offset<kSkip>(a, pos, behind), behind(a)       bytes in the pools of a position, -1: nothing to read (offset_of)
//   hidden(a, k0, keys), sees(a, pos, key)         does some row not see some of these keys; does this one see this one
//   parts(a), part<D>(a, .., r, m, l, first)       are the results shares of rows, and where row r's goes
//   out(a), stats(a, row, m, l)                    where whole rows go
//   by_hand<T, D>(a, ..)                           rows by the definition
//   finish()                                       at the kernel's end
#pragma once

#include <type_traits>

#include "lf_paged.cuh"

namespace lf {

namespace {

constexpr int kKeys = 64;

// ---- bf16: m16n8k16 ------------------------------------------------------------------
//
// Four warps of 16 rows, two stages of K and V tiles.  The queries stay in registers as
// A operands, S comes out as the C operand whose layout is the A operand of P.V, so P
// (rounded to bf16: half a step is 2^-8 of a weight) never leaves the registers either.
// Bound by these instructions' rate, 600 TFLOP/s here, and the softmax between them: 8192
// tokens in pages of 24, 32 / 8 heads of 128, 1.61 ms, 341 TFLOP/s; 2000 tokens, heads of 32, 43 us.

constexpr int kMmaThreads = 128, kMmaRows = 64;

// Three blocks of heads of 128 on an SM: a few registers more than that leaves make it two (pages of
// 24: 1.61 ms against 1.97 to 2.15).
template <class Task, int D>
__global__ void __launch_bounds__(kMmaThreads, D == 128 ? 3 : D >= 32 ? 4 : 5) paged_mma_kernel(const __grid_constant__ typename Task::Args a) {
  constexpr int NC = D / 8;                // 16-byte chunks of a row
  constexpr int kTileBytes = kKeys * NC * 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_off[2][kKeys];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Task task;
  if (!task.take(a, kMmaRows, kKeys)) return;
  const int nt = task.count();
  const uint32_t ring = smem_u32(smem);

  auto look_up = [&](int j) {
    if (tid < kKeys)
      s_off[j & 1][tid] = task.template offset<true>(a, task.at(j) * kKeys + tid, [&] { return task.behind(a); });
  };
  auto issue = [&](int j) {
    const uint32_t kd = ring + (j & 1) * 2 * kTileBytes, vd = kd + kTileBytes;
    constexpr int kStep = kMmaThreads / NC;   // rows that the block covers at once
    const int c = tid % NC;
#pragma unroll
    for (int i = 0; i < (kKeys + kStep - 1) / kStep; ++i) {
      const int r = i * kStep + tid / NC;
      if (kKeys % kStep == 0 || r < kKeys) {
        const int64_t off = s_off[j & 1][r];
        const uint32_t d = 16 * tile_chunk<NC>(r, c);
        cp_async16(kd + d, a.pool.k + (off >= 0 ? off + c * 16 : 0), off >= 0);
        cp_async16(vd + d, a.pool.v + (off >= 0 ? off + c * 16 : 0), off >= 0);
      }
    }
  };

  const int ra = warp * 16 + (lane >> 2);   // and ra + 8
  uint32_t qa[D / 16][4];
  int pos[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = ra + 8 * i;
    const bool live = task.live(a, r);
    pos[i] = task.pos(a, r);
    const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q) + (live ? task.q_row(a, r) * (D / 2) : 0) + (lane & 3);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qa[kk][i] = live ? q[8 * kk] : 0u;
      qa[kk][2 + i] = live ? q[8 * kk + 4] : 0u;
    }
  }
  float o[D / 8][4], m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
  __nv_bfloat162 bad = __float2bfloat162_rn(0.f);

  if (nt > 0) {
    look_up(0);
    __syncthreads();
    issue(0);
    cp_async_commit();
    if (nt > 1) look_up(1);
  }
#pragma unroll 1
  for (int j = 0; j < nt; ++j) {
    __syncthreads();   // the other stage has been read, its new offsets are there
    if (j + 1 < nt) issue(j + 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    if (j + 2 < nt) look_up(j + 2);
    const uint32_t ks = ring + (j & 1) * 2 * kTileBytes, vs = ks + kTileBytes;
    const int k0 = task.at(j) * kKeys;
    const bool hidden = task.hidden(a, k0, kKeys);
    if (hidden) {   // a weight of 0 must take nothing: are there values that are not finite?
      const uint4* v = reinterpret_cast<const uint4*>(smem + (j & 1) * 2 * kTileBytes + kTileBytes);
      const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
      for (int i = tid; i < kKeys * NC; i += kMmaThreads) {
        const uint4 x = v[i];
        bad = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.x), zero, bad);
        bad = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.y), zero, bad);
        bad = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.z), zero, bad);
        bad = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.w), zero, bad);
      }
    }
    float s[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      if constexpr (D >= 32) {
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          uint32_t kb[4];
          ldmatrix4(ks + 16 * tile_chunk<NC>(8 * n + (lane & 7), c + (lane >> 3)), kb);
          mma16816(s[n], qa[c / 2][0], qa[c / 2][1], qa[c / 2][2], qa[c / 2][3], kb[0], kb[1]);
          mma16816(s[n], qa[c / 2 + 1][0], qa[c / 2 + 1][1], qa[c / 2 + 1][2], qa[c / 2 + 1][3], kb[2], kb[3]);
        }
      } else if ((n & 1) == 0) {
        uint32_t kb[4];
        ldmatrix4(ks + 16 * tile_chunk<NC>(8 * n + (lane & 7) + 8 * (lane >> 4), (lane >> 3) & 1), kb);
        mma16816(s[n], qa[0][0], qa[0][1], qa[0][2], qa[0][3], kb[0], kb[1]);
        mma16816(s[n + 1], qa[0][0], qa[0][1], qa[0][2], qa[0][3], kb[2], kb[3]);
      }
    }
    if (hidden) {
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!task.sees(a, pos[i >> 1], k0 + 8 * n + 2 * (lane & 3) + (i & 1))) s[n][i] = kNegInf;
    }
    float top[2] = {kNegInf, kNegInf};
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) top[i >> 1] = fmaxf(top[i >> 1], s[n][i]);
    bool up = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2)) * a.scale_log2;
      up |= top[i] > m[i];
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mn = fmaxf(m[i], top[i]);
        const float f = mn == kNegInf ? 1.f : ex2(m[i] - mn);
        m[i] = mn;
        l[i] *= f;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          o[n][2 * i] *= f;
          o[n][2 * i + 1] *= f;
        }
      }
    }
    const float mu[2] = {m[0] == kNegInf ? 0.f : m[0], m[1] == kNegInf ? 0.f : m[1]};
    uint32_t pa[8][2];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float x = ex2(fmaf(s[n][2 * i], a.scale_log2, -mu[i]));
        const float y = ex2(fmaf(s[n][2 * i + 1], a.scale_log2, -mu[i]));
        l[i] += x + y;
        pa[n][i] = pack_bf16(x, y);
      }
#pragma unroll
    for (int kk = 0; kk < kKeys / 16; ++kk) {
      const int row = 16 * kk + (lane & 7) + 8 * ((lane >> 3) & 1);
#pragma unroll
      for (int c = 0; c < NC; c += 2) {
        uint32_t vb[4];
        ldmatrix4_trans(vs + 16 * tile_chunk<NC>(row, c + (lane >> 4)), vb);
        mma16816(o[c], pa[2 * kk][0], pa[2 * kk][1], pa[2 * kk + 1][0], pa[2 * kk + 1][1], vb[0], vb[1]);
        mma16816(o[c + 1], pa[2 * kk][0], pa[2 * kk][1], pa[2 * kk + 1][0], pa[2 * kk + 1][1], vb[2], vb[3]);
      }
    }
  }

  const float2 f = __bfloat1622float2(bad);
  if (__syncthreads_or(!(f.x == 0.f) || !(f.y == 0.f))) {
    task.template by_hand<__nv_bfloat16, D>(a, kKeys, kMmaRows, warp * 16, 16, lane);
    task.finish();
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float ls = l[i] + __shfl_xor_sync(0xffffffffu, l[i], 1);
    ls += __shfl_xor_sync(0xffffffffu, ls, 2);
    const int r = ra + 8 * i;
    if (!task.live(a, r)) continue;
    if (task.parts(a)) {
      float* part = task.template part<D>(a, kMmaRows, r, m[i], ls, (lane & 3) == 0) + 2 * (lane & 3);
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(part + 8 * n) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
      continue;
    }
    const float inv = ls == 0.f ? 0.f : 1.f / ls;
    const int64_t row = task.q_row(a, r);
    uint32_t* out = reinterpret_cast<uint32_t*>(task.out(a)) + row * (D / 2) + (lane & 3);
#pragma unroll
    for (int n = 0; n < D / 8; ++n) out[4 * n] = pack_bf16(o[n][2 * i] * inv, o[n][2 * i + 1] * inv);
    if ((lane & 3) == 0) task.stats(a, row, m[i], ls);
  }
  task.finish();
}

// ---- fp32: CUDA cores -----------------------------------------------------------------
//
// Two floats per multiply-add instruction.  A thread holds an M x 4 piece of S (sums over
// even and over odd columns of d) and M rows x d/16 columns of O.  V is on its way while S is computed.
// Bound by the multiply-adds (67 TFLOP/s in pairs) and, with few blocks, by the chain of a
// tile's steps: 4000 tokens, 32 / 8 heads of 128, 2.9 ms, 45 TFLOP/s; 2000 tokens, 8 heads of
// 64, 135 us, 30 TFLOP/s; three prompts of 500 to 1000 56 us.

// In blocks of 32 rows P has a place of its own, so that the next K can come in as soon
// as S is done; in those of 64 it goes where K was, which leaves room for two blocks.
template <int D, int R>
constexpr int fma_smem() {
  constexpr int LD = D + 4, LP = R + 4;   // eight rows' equal chunks fall into different banks
  return (R * LD + kKeys * (R == 32 ? LD + LP : LD > LP ? LD : LP) + kKeys * LD) * 4;
}

template <class Task, int D, int R, int M>
__global__ void __launch_bounds__(16 * R / M, D <= 64 ? 4 : 1) paged_fma_kernel(const __grid_constant__ typename Task::Args a) {
  constexpr int kThreads = 16 * R / M;
  static_assert(kThreads >= kKeys && M % 4 == 0, "one thread looks up a key");
  constexpr int LD = D + 4, LP = R + 4;
  constexpr int NC = D / 4;
  constexpr int CW = D / 16;            // columns of O per thread
  constexpr int VW = CW < 4 ? CW : 4;   // .. in runs of
  constexpr int CP = (CW + 1) / 2;      // .. in pairs
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;                                  // [R][LD]
  constexpr bool kOwnP = R == 32;
  float* sk = sm + R * LD;                         // [kKeys][LD]
  float* sv = sk + kKeys * (kOwnP || LD > LP ? LD : LP);   // [kKeys][LD]
  float* sp = kOwnP ? sv + kKeys * LD : sk;        // P^T [kKeys][LP]
  __shared__ int64_t s_off[kKeys];
  const int tid = threadIdx.x;
  Task task;
  if (!task.take_level(a, R, kKeys)) return;
  const int nt = task.count();

  // (From shared memory for an entry that is no page: worked out there from the piece it costs
  // the loop 2 to 5 % by its registers.  Every thread that looks up has written it.)
  __shared__ int s_behind;
  if (tid < kKeys) s_behind = task.behind(a);
  auto look_up = [&](int j) {
    if (tid < kKeys)
      s_off[tid] = task.template offset<false>(a, task.at(j) * kKeys + tid,
                                    [&] { return *const_cast<const volatile int*>(&s_behind); });
  };
  auto issue = [&](float* dst, const char* pool) {
#pragma unroll 4
    for (int i = tid; i < kKeys * NC; i += kThreads) {
      const int r = i / NC, c = i - r * NC;
      const int64_t off = s_off[r];
      cp_async16(smem_u32(dst + r * LD + c * 4), pool + (off >= 0 ? off + c * 16 : 0), off >= 0);
    }
    cp_async_commit();
  };
  if (nt > 0) look_up(0);
  for (int i = tid; i < R * NC; i += kThreads) {
    const int r = i / NC, c = i - r * NC;
    const bool live = task.live(a, r);
    const float* q = reinterpret_cast<const float*>(a.q) + (live ? task.q_row(a, r) * D + c * 4 : 0);
    *reinterpret_cast<float4*>(sq + r * LD + c * 4) =
        live ? *reinterpret_cast<const float4*>(q) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  if (nt > 0) issue(sk, a.pool.k);

  const int rg = tid >> 4, cg = tid & 15;
  int pos[M];
  float m[M], l[M];
  uint64_t o[M][CP];
#pragma unroll
  for (int i = 0; i < M; ++i) {
    pos[i] = task.pos(a, rg * M + i);
    m[i] = kNegInf;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < CP; ++c) o[i][c] = 0ull;
  }

#pragma unroll 1
  for (int j = 0; j < nt; ++j) {
    const int k0 = task.at(j) * kKeys;
    const bool hidden = task.hidden(a, k0, kKeys);
    issue(sv, a.pool.v);
    cp_async_wait<1>();
    __syncthreads();
    uint64_t s2[M][4];
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int n = 0; n < 4; ++n) s2[i][n] = 0ull;
#pragma unroll (M == 4 ? 4 : 2)
    for (int d = 0; d < D; d += 4) {
      ulonglong2 y[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) y[n] = *reinterpret_cast<const ulonglong2*>(sk + (cg + 16 * n) * LD + d);
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(sq + (rg * M + i) * LD + d);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          s2[i][n] = fma_pair(x.x, y[n].x, s2[i][n]);
          s2[i][n] = fma_pair(x.y, y[n].y, s2[i][n]);
        }
      }
    }
    float w[M][4];
#pragma unroll
    for (int i = 0; i < M; ++i) {
      float top = kNegInf;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        float x, y;
        unpair(s2[i][n], &x, &y);
        w[i][n] = x + y;
        if (hidden && !task.sees(a, pos[i], k0 + cg + 16 * n)) w[i][n] = kNegInf;
        top = fmaxf(top, w[i][n]);
      }
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      top = fmaxf(m[i], top * a.scale_log2);
      const float mu = top == kNegInf ? 0.f : top;
      const float f = ex2(m[i] - mu);
      m[i] = top;
      l[i] *= f;
#pragma unroll
      for (int c = 0; c < CP; ++c) o[i][c] = fma_pair(o[i][c], pair(f, f), 0ull);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        w[i][n] = ex2(fmaf(w[i][n], a.scale_log2, -mu));   // rounded as a difference, not at the logit's size
        l[i] += w[i][n];
      }
    }
    __syncthreads();   // K has been read
    if (kOwnP && j + 1 < nt) {   // and the offsets, by the copies of V
      look_up(j + 1);
      __syncthreads();
      issue(sk, a.pool.k);
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int i = 0; i < M; i += 4)
        *reinterpret_cast<float4*>(sp + (cg + 16 * n) * LP + rg * M + i) =
            make_float4(w[i][n], w[i + 1][n], w[i + 2][n], w[i + 3][n]);
    if (!kOwnP && j + 1 < nt) look_up(j + 1);
    if (kOwnP && j + 1 < nt) cp_async_wait<1>();   // V; K goes on
    else cp_async_wait<0>();
    __syncthreads();
    // Where some row does not see some key of the tile, a weight of zero takes
    // nothing of the value, which may hold anything there.
    auto accumulate = [&](auto part) {
#pragma unroll (M == 4 ? 8 : 2)
      for (int k = 0; k < kKeys; ++k) {
        float pi[M];
#pragma unroll
        for (int i = 0; i < M; i += 4) load16_f32(sp + k * LP + rg * M + i, pi + i);
        uint64_t v[CP];
#pragma unroll
        for (int c = 0; c < CW; c += VW) {
          const float* src = sv + k * LD + (c / VW) * 16 * VW + cg * VW;
          if constexpr (VW == 4) {
            const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(src);
            v[c / 2] = t.x;
            v[c / 2 + 1] = t.y;
          } else if constexpr (VW == 2) {
            v[0] = *reinterpret_cast<const uint64_t*>(src);
          } else {
            v[0] = pair(*src, 0.f);
          }
        }
#pragma unroll
        for (int i = 0; i < M; ++i) {
          if (part.value && pi[i] == 0.f) continue;
          const uint64_t pp = pair(pi[i], pi[i]);
#pragma unroll
          for (int c = 0; c < CP; ++c) o[i][c] = fma_pair(pp, v[c], o[i][c]);
        }
      }
    };
    if (hidden) accumulate(std::true_type{});
    else accumulate(std::false_type{});
    __syncthreads();   // P and V have been read
    if (!kOwnP && j + 1 < nt) issue(sk, a.pool.k);
  }

#pragma unroll
  for (int i = 0; i < M; ++i) {
    float ls = l[i];
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
    const int r = rg * M + i;
    if (!task.live(a, r)) continue;
    // the row's output, or its share of it
    const bool part = task.parts(a);
    const float inv = part ? 1.f : ls == 0.f ? 0.f : 1.f / ls;
    const int64_t row = task.q_row(a, r);
    float* out = part ? task.template part<D>(a, R, r, m[i], ls, cg == 0) : reinterpret_cast<float*>(task.out(a)) + row * D;
#pragma unroll
    for (int c = 0; c < CP; ++c) {
      float x, y;
      unpair(o[i][c], &x, &y);
      float* dst = out + (2 * c / VW) * 16 * VW + cg * VW + 2 * c % VW;
      if constexpr (VW >= 2) *reinterpret_cast<float2*>(dst) = make_float2(x * inv, y * inv);
      else *dst = x * inv;
    }
    if (cg == 0 && !part) task.stats(a, row, m[i], ls);
  }
  task.finish();
}

}  // namespace

}  // namespace lf
