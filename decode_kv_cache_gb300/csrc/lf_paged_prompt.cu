// Causal attention of the last tokens of every sequence over a paged key-value
// cache, with an optional sliding window and sinks:
//
//   out_i = sum_j 2^(s_ij - m_i) v_j / sum_j 2^(s_ij - m_i),  s = q . k log2(e) / sqrt(d)
//
// over j <= i and (no window, or j > i - window, or j < sinks), in one pass over
// the keys with the running maximum m_i and sum of every row.  bf16 with head_dim 64
// and 128 has a kernel of its own (lf_paged_prompt_tc.cu); here are the others:
//   - bf16 on the legacy matrix instructions, for short heads and for pages that a
//     tensor map's boxes do not divide into;
//   - fp32 on the CUDA cores: a tf32 product drops 13 bits of each factor, and three
//     of them in place of one lose to the tensor cores' truncating sums what fp32
//     callers keep.
// A CTA takes some rows of one KV head's queries, (token, head of the group) pairs
// with the head inner: every key and value it loads serves all heads of the group.
// Keys and values pass through shared memory in tiles of 64 tokens, 16-byte chunks
// gathered by page; key tiles that no row sees are not visited.  A sequence's
// last rows, which see the most keys, start first.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

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
template <int D>
__global__ void __launch_bounds__(kMmaThreads, D == 128 ? 3 : D >= 32 ? 4 : 5) paged_prompt_mma_kernel(const __grid_constant__ PagedPromptArgs a) {
  constexpr int NC = D / 8;                // 16-byte chunks of a row
  constexpr int kTileBytes = kKeys * NC * 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_off[2][kKeys];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int share = blockIdx.y;
  Piece p;
  int number;
  const int b = locate(a, blockIdx.x, &number);
  if (!take_piece(a, blockIdx.x, b, number, kMmaRows, tid == 0 && share == 0, &p)) return;
  const Tiles tiles(a, p.p_lo, p.p_hi, kKeys, share);
  const int nt = tiles.count();
  const uint32_t ring = smem_u32(smem);

  auto look_up = [&](int j) {
    if (tid < kKeys)
      s_off[j & 1][tid] = offset_of<true>(a, p, tiles.at(j) * kKeys + tid, [&] { return behind_window(a, p.p_lo); });
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

  const int64_t ra = p.r0 + warp * 16 + (lane >> 2);   // and ra + 8
  uint32_t qa[D / 16][4];
  int pos[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t r = ra + 8 * i;
    const bool live = r < p.rows;
    pos[i] = live ? p.first_pos + (int)(r / a.group) : -1;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q) + (live ? row_of(a, p, r) * (D / 2) : 0) + (lane & 3);
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
    const int k0 = tiles.at(j) * kKeys;
    const bool hidden = some_hidden(a, p.p_lo, p.p_hi, k0, kKeys);
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
          if (!sees(a, pos[i >> 1], k0 + 8 * n + 2 * (lane & 3) + (i & 1))) s[n][i] = kNegInf;
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
    rows_by_hand<__nv_bfloat16, D>(a, blockIdx.x, share, kKeys, kMmaRows, warp * 16, 16, lane);
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float ls = l[i] + __shfl_xor_sync(0xffffffffu, l[i], 1);
    ls += __shfl_xor_sync(0xffffffffu, ls, 2);
    const int64_t r = ra + 8 * i;
    if (r >= p.rows) continue;
    if (a.splits > 1) {
      float* part = part_row<D>(a, p.id, share, kMmaRows, (int)(r - p.r0), m[i], ls, (lane & 3) == 0) + 2 * (lane & 3);
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(part + 8 * n) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
      continue;
    }
    const float inv = ls == 0.f ? 0.f : 1.f / ls;
    const int64_t row = row_of(a, p, r);
    uint32_t* out = reinterpret_cast<uint32_t*>(a.out) + row * (D / 2) + (lane & 3);
#pragma unroll
    for (int n = 0; n < D / 8; ++n) out[4 * n] = pack_bf16(o[n][2 * i] * inv, o[n][2 * i + 1] * inv);
    if ((lane & 3) == 0) write_row_stats(a, row, m[i], ls);
  }
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

template <int D, int R, int M>
__global__ void __launch_bounds__(16 * R / M) paged_prompt_fma_kernel(const __grid_constant__ PagedPromptArgs a) {
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
  Piece p;
  const int share = blockIdx.y, heads = a.pool.batch * a.pool.kv_heads;
  const int id = gridDim.x - 1 - blockIdx.x, tile = id / heads;   // the last rows first
  if (!take_piece_level(a, id - tile * heads, tile, R, tid == 0 && share == 0, &p)) return;
  const Tiles tiles(a, p.p_lo, p.p_hi, kKeys, share);
  const int nt = tiles.count();

  // (From shared memory for an entry that is no page: worked out there from the piece it costs
  // the loop 2 to 5 % by its registers.  Every thread that looks up has written it.)
  __shared__ int s_behind;
  if (tid < kKeys) s_behind = behind_window(a, p.p_lo);
  auto look_up = [&](int j) {
    if (tid < kKeys)
      s_off[tid] = offset_of<false>(a, p, tiles.at(j) * kKeys + tid,
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
    const bool live = p.r0 + r < p.rows;
    const float* q = reinterpret_cast<const float*>(a.q) + (live ? row_of(a, p, p.r0 + r) * D + c * 4 : 0);
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
    const int64_t r = p.r0 + rg * M + i;
    pos[i] = r < p.rows ? p.first_pos + (int)(r / a.group) : -1;
    m[i] = kNegInf;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < CP; ++c) o[i][c] = 0ull;
  }

#pragma unroll 1
  for (int j = 0; j < nt; ++j) {
    const int k0 = tiles.at(j) * kKeys;
    const bool hidden = some_hidden(a, p.p_lo, p.p_hi, k0, kKeys);
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
        if (hidden && !sees(a, pos[i], k0 + cg + 16 * n)) w[i][n] = kNegInf;
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
    const int64_t r = p.r0 + rg * M + i;
    if (r >= p.rows) continue;
    // the row's output, or its share of it
    const float inv = a.splits > 1 ? 1.f : ls == 0.f ? 0.f : 1.f / ls;
    const int64_t row = row_of(a, p, r);
    float* out = a.splits > 1 ? part_row<D>(a, p.id, share, R, (int)(r - p.r0), m[i], ls, cg == 0)
                              : reinterpret_cast<float*>(a.out) + row * D;
#pragma unroll
    for (int c = 0; c < CP; ++c) {
      float x, y;
      unpair(o[i][c], &x, &y);
      float* dst = out + (2 * c / VW) * 16 * VW + cg * VW + 2 * c % VW;
      if constexpr (VW >= 2) *reinterpret_cast<float2*>(dst) = make_float2(x * inv, y * inv);
      else *dst = x * inv;
    }
    if (cg == 0 && a.splits == 1) write_row_stats(a, row, m[i], ls);
  }
}

// ---- joining the shares of rows whose keys several blocks took -----------------------
//
// A warp per row: lane i reads share i's maximum and sum, then all lanes add up the
// shares' outputs in their order.  Bound by latency, 4 us.
constexpr int kJoinWarps = 8, kMaxSplits = 32;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_prompt_join_kernel(const __grid_constant__ PagedPromptArgs a, int per_piece) {
  constexpr int E = D >= 32 ? D / 32 : 1;
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  const int rr = (int)(i % per_piece);
  Piece p;
  const unsigned id = (unsigned)(i / per_piece);
  int number;
  const int b = locate(a, id, &number);
  if (!take_piece(a, id, b, number, per_piece, false, &p) || p.r0 + rr >= p.rows) return;
  const int64_t part = p.id * a.splits * per_piece + rr;   // share s: + s * per_piece
  float m = kNegInf, l = 0.f;
  if (lane < a.splits) {
    m = a.part_ml[2 * (part + (int64_t)lane * per_piece)];
    l = a.part_ml[2 * (part + (int64_t)lane * per_piece) + 1];
  }
  const float top = warp_max(m), mu = top == kNegInf ? 0.f : top;
  const float f = ex2(m - mu);
  const float sum = warp_sum(l * f);
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  const int col = (lane * E) % D;
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const float fs = __shfl_sync(0xffffffffu, f, s);
    const float* o = a.part_o + (part + (int64_t)s * per_piece) * D + col;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(o[e], fs, acc[e]);
  }
  const int64_t row = row_of(a, p, p.r0 + rr);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* out = reinterpret_cast<T*>(a.out) + row * D;
  if (lane * E < D) {
#pragma unroll
    for (int e = 0; e < E; ++e) from_f32(sum == 0.f ? 0.f : acc[e] * inv, out + col + e);
  }
  if (lane == 0) write_row_stats(a, row, top, sum);
}

template <typename T, int D>
cudaError_t launch_join(const PagedPromptArgs& a, const PromptPlan& plan, cudaStream_t stream) {
  const int64_t rows = plan.pieces * plan.rows;   // few: splits are for few pieces
  paged_prompt_join_kernel<T, D><<<(unsigned)((rows + kJoinWarps - 1) / kJoinWarps), kJoinWarps * 32, 0, stream>>>(a, plan.rows);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_join_dim(const PagedPromptArgs& a, const PromptPlan& plan, int head_dim, cudaStream_t stream) {
  switch (head_dim) {
    case 16: return launch_join<T, 16>(a, plan, stream);
    case 32: return launch_join<T, 32>(a, plan, stream);
    case 64: return launch_join<T, 64>(a, plan, stream);
    default: return launch_join<T, 128>(a, plan, stream);
  }
}

template <int D>
cudaError_t launch_mma(const PagedPromptArgs& a, const PromptPlan& plan, cudaStream_t stream) {
  constexpr int kSmem = 4 * kKeys * D * 2;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(&paged_prompt_mma_kernel<D>), kSmem, done);
  if (e != cudaSuccess) return e;
  paged_prompt_mma_kernel<D><<<dim3((unsigned)plan.pieces, plan.splits), kMmaThreads, kSmem, stream>>>(a);
  return cudaGetLastError();
}

template <int D, int R, int M>
cudaError_t launch_fma(const PagedPromptArgs& a, const PromptPlan& plan, cudaStream_t stream) {
  constexpr int kSmem = fma_smem<D, R>();
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(&paged_prompt_fma_kernel<D, R, M>), kSmem, done);
  if (e != cudaSuccess) return e;
  paged_prompt_fma_kernel<D, R, M><<<dim3((unsigned)plan.pieces, plan.splits), 16 * R / M, kSmem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kernel(const PagedPromptArgs& a, const PromptPlan& plan, int head_dim, cudaStream_t stream) {
  if (plan.kernel == PromptPlan::kTensor) return paged_prompt_tc_launch(a, plan, head_dim, stream);
  if (plan.kernel == PromptPlan::kMatrix) {
    switch (head_dim) {
      case 16: return launch_mma<16>(a, plan, stream);
      case 32: return launch_mma<32>(a, plan, stream);
      case 64: return launch_mma<64>(a, plan, stream);
      default: return launch_mma<128>(a, plan, stream);
    }
  }
  switch (head_dim) {
    case 16: return launch_fma<16, 32, 4>(a, plan, stream);
    case 32: return launch_fma<32, 32, 4>(a, plan, stream);
    case 64: return launch_fma<64, 32, 4>(a, plan, stream);
    default: return plan.rows == 64 ? launch_fma<128, 64, 8>(a, plan, stream) : launch_fma<128, 32, 4>(a, plan, stream);
  }
}

}  // namespace

PromptPlan paged_prompt_plan(const PagedPool& pool, int elem, int head_dim, int group, int total_q, int max_q,
                             int window, int sinks, int sms) {
  PromptPlan plan;
  int keys = kKeys, room = 3 * sms;   // keys of a tile, blocks that run at once
  if (elem == 2 && paged_prompt_tc_takes(pool, head_dim)) {
    plan.kernel = PromptPlan::kTensor;
    plan.rows = 256;
    keys = 128;
    room = sms;
  } else if (elem == 2) {
    plan.kernel = PromptPlan::kMatrix;
    plan.rows = kMmaRows;
  } else {
    // Pieces of 32 rows in 4 x 4 shares: more blocks, each done sooner.  Heads of 128
    // read more per multiply-add than that feeds, so where the blocks fill the GPU all
    // the same they take 64 rows in 8 x 4 shares.  (Eight heads of 128: three prompts of
    // 500 to 1000 tokens 92 us against 130, three of 2000 tokens 722 against 636.
    // Shorter heads gain nothing from it: heads of 64, three of 2000 tokens, 362 against
    // 425.)
    plan.kernel = PromptPlan::kFma;
    const int64_t of64 = paged_prompt_pieces(pool, group, total_q, max_q, 64, false, &plan.tiles_per_seq);
    plan.rows = head_dim == 128 && of64 >= 4 * (int64_t)sms ? 64 : 32;
  }
  plan.pieces = paged_prompt_pieces(pool, group, total_q, max_q, plan.rows, elem == 2, &plan.tiles_per_seq);
  // Where the pieces leave half of the GPU idle and their keys may be many, several
  // blocks share a piece's keys: at least four tiles for each of them.  (32 / 8 heads of
  // 128, one to 64 tokens behind 8000: 93 us without, 26 us.)  fp32 pieces differ in
  // length and take long, so that there halves of twice as many even out, up to the blocks
  // that an SM holds at once.  (Eight heads of 64, one prompt of 2000 tokens: 180 us
  // without, 135 us; three of 500 to 1000: 67 us, 57 us.)  How many keys there may be follows the
  // table's width: a prompt of 300 tokens, 16 / 8 heads of 128, takes 12.4 us under a table of its own 19
  // pages and 22.7 under one of 8192, for shares that find no keys and their join.
  if (plan.kernel == PromptPlan::kFma && plan.pieces >= sms) room = (head_dim == 128 ? 4 : 8) * sms;
  const int64_t all = (int64_t)pool.max_pages * pool.page_size;
  const int64_t most = window > 0 ? (int64_t)window + sinks + plan.rows + 2 * keys : all;
  const int64_t tiles = ((most < all ? most : all) + keys - 1) / keys;
  int64_t splits = 1;
  if (plan.pieces <= room / 2 && tiles >= (plan.kernel == PromptPlan::kFma ? 8 : 16)) {
    splits = room / plan.pieces;
    if (splits > tiles / 4) splits = tiles / 4;
    if (splits > kMaxSplits) splits = kMaxSplits;
  }
  plan.splits = (int)splits;
  plan.off_ml = plan.bytes = 0;
  if (splits > 1) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    plan.off_ml = up((size_t)plan.pieces * splits * plan.rows * head_dim * 4);
    plan.bytes = plan.off_ml + up((size_t)plan.pieces * splits * plan.rows * 2 * 4);
  }
  return plan;
}

cudaError_t paged_prompt_launch(const PagedPromptArgs& a, const PromptPlan& plan, int elem, int head_dim,
                                cudaStream_t stream) {
  const cudaError_t e = launch_kernel(a, plan, head_dim, stream);
  if (e != cudaSuccess || plan.splits == 1) return e;
  return elem == 2 ? launch_join_dim<__nv_bfloat16>(a, plan, head_dim, stream)
                   : launch_join_dim<float>(a, plan, head_dim, stream);
}

}  // namespace lf
