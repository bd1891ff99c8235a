// Attention of one new token per sequence where groups of sequences share a prefix: the prefix's keys and
// values are read once for all of a group's sequences and heads, the rest as decode reads it.
//
//   out = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s,  m = max_s m_s
//
// over shares s of a row's keys, each with its maximum m_s (log2), sum l_s and output O_s (not normalised): shares of
// the prefix, and what lies behind it.  bf16 with heads of 64 and 128 has a kernel for both (lf_paged_shared_tc.cu).  Others take
// two launches:
//   - lf_paged_decode.cu's kernel walks every sequence from its prefix's end on;
//   - a kernel here takes up to 64 rows, (sequence, head of the group) pairs, of a KV head against a segment of the
//     prefix's keys.  It depends on nothing that the first one writes and is placed while that drains (programmatic
//     dependent launch); it ends behind it.
// The join, the last launch of either way, adds the shares up, in order of position.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "lf_paged_shared.cuh"

namespace lf {

namespace {

// A segment as its block's threads see it.
struct Block {
  Segment s;

  template <int kThreads>
  __device__ __forceinline__ bool take(const PagedSharedArgs& a, void* smem);
  __device__ __forceinline__ int count() const { return s.last - s.first; }
  __device__ __forceinline__ int at(int j) const { return s.first + j; }
  __device__ __forceinline__ bool live(const PagedSharedArgs& a, int r) const { return r < s.members * a.group; }
  // The last position that row r sees, -1: none, or no row.
  __device__ __forceinline__ int pos(const PagedSharedArgs& a, int r) const {
    return live(a, r) ? last_seen(a, s.prefix, s.b0 + r / a.group) : -1;
  }
  // Where row r's share goes.
  template <int D>
  __device__ __forceinline__ float* part(const PagedSharedArgs& a, int r, float m, float l, bool first) const {
    if (first) {
      a.part_ml[2 * (s.row + r)] = m;
      a.part_ml[2 * (s.row + r) + 1] = l;
    }
    return a.part_o + (s.row + r) * D;
  }
  // The kernel before this one ends before this one does, and with it before the join.
  __device__ __forceinline__ void finish() const {
    if (threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  }
};

constexpr int kKeys = 64;

// The groups that a block looks at together lie where its tiles will.
using Families = FamilyTable<kTableOther>;

template <int kThreads>
__device__ __forceinline__ bool Block::take(const PagedSharedArgs& a, void* smem) {
  const bool ok = take_segment<kThreads>(a, kKeys, *static_cast<Families*>(smem), &s);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!ok) finish();
  return ok;
}

// ---- bf16: m16n8k16 ------------------------------------------------------------------
//
// For short heads and for pages that a tensor map's boxes do not divide into.  Four warps of 16 rows, two stages of K and V
// tiles of 64 tokens, 16-byte chunks gathered by page.  The queries stay in registers as A operands, S comes out as the C operand
// whose layout is the A operand of P.V, so P (rounded to bf16: half a step is 2^-8 of a weight) never leaves the registers either.
// Bound by these instructions' rate and the softmax between them, and with few tiles by the launches' starts: 32 sequences
// behind 8192 in pages of 24, 32 / 8 heads of 128, 43 us with the rest and the join; four groups of eight behind 1000 to 2000, heads of
// 32, 16 us.

constexpr int kMmaThreads = 128, kMmaRows = 64;

// Three blocks of heads of 128 on an SM.
template <int D>
__global__ void __launch_bounds__(kMmaThreads, D == 128 ? 3 : D >= 32 ? 4 : 5) paged_shared_mma_kernel(const __grid_constant__ PagedSharedArgs a) {
  constexpr int NC = D / 8;                // 16-byte chunks of a row
  constexpr int kTileBytes = kKeys * NC * 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_off[2][kKeys];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Block block;
  static_assert(sizeof(Families) <= 4 * kTileBytes, "the groups fit where the tiles will lie");
  if (!block.take<kMmaThreads>(a, smem)) return;
  const int nt = block.count();
  const uint32_t ring = smem_u32(smem);

  auto look_up = [&](int j) {
    if (tid < kKeys)
      s_off[j & 1][tid] = shared_offset(a, block.s, block.at(j) * kKeys + tid);
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
    const bool live = block.live(a, r);
    pos[i] = block.pos(a, r);
    const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q) + (live ? shared_row(a, block.s, r) * (D / 2) : 0) + (lane & 3);
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
    const int k0 = block.at(j) * kKeys;
    const bool hidden = k0 + kKeys - 1 > block.s.p_lo;
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
          if (k0 + 8 * n + 2 * (lane & 3) + (i & 1) > pos[i >> 1]) s[n][i] = kNegInf;
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
    for (int r = warp * 16; r < warp * 16 + 16 && block.live(a, r); ++r)
      shared_row_by_hand<__nv_bfloat16, D>(a, block.s, kKeys, r, block.pos(a, r), lane);
    block.finish();
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float ls = l[i] + __shfl_xor_sync(0xffffffffu, l[i], 1);
    ls += __shfl_xor_sync(0xffffffffu, ls, 2);
    const int r = ra + 8 * i;
    if (!block.live(a, r)) continue;
    float* part = block.part<D>(a, r, m[i], ls, (lane & 3) == 0) + 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<float2*>(part + 8 * n) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
  }
  block.finish();
}

// ---- fp32: CUDA cores -----------------------------------------------------------------
//
// (A tf32 product drops 13 bits of each factor.)  Two floats per multiply-add instruction.  A thread holds an M x 4 piece of S
// (sums over even and over odd columns of d, two columns' products at a time: a chain of d / 4 roundings at the sum's size,
// where one product at a time has d / 2) and M rows x d/16 columns of O.  V is on its way while S is computed.  Bound by
// the chain of a tile's steps: a tile of 64 keys takes about 6 us.  24 sequences behind 3000, 8 heads of 64, 29 us with
// the rest and the join; 16 behind 4000, 32 / 8 heads of 128, 59 us; 64 behind 8192, 8 heads of 64, 60 us.

// In blocks of 32 rows P has a place of its own, so that the next K can come in as soon
// as S is done; in those of 64 it goes where K was, which leaves room for two blocks.
template <int D, int R>
constexpr int fma_smem() {
  constexpr int LD = D + 4, LP = R + 4;   // eight rows' equal chunks fall into different banks
  return (R * LD + kKeys * (R == 32 ? LD + LP : LD > LP ? LD : LP) + kKeys * LD) * 4;
}

template <int D, int R, int M>
__global__ void __launch_bounds__(16 * R / M, D <= 64 ? 4 : 1) paged_shared_fma_kernel(const __grid_constant__ PagedSharedArgs a) {
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
  Block block;
  if (!block.take<kThreads>(a, sm)) return;
  const int nt = block.count();

  auto look_up = [&](int j) {
    if (tid < kKeys) s_off[tid] = shared_offset(a, block.s, block.at(j) * kKeys + tid);
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
    const bool live = block.live(a, r);
    const float* q = reinterpret_cast<const float*>(a.q) + (live ? shared_row(a, block.s, r) * D + c * 4 : 0);
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
    pos[i] = block.pos(a, rg * M + i);
    m[i] = kNegInf;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < CP; ++c) o[i][c] = 0ull;
  }

#pragma unroll 1
  for (int j = 0; j < nt; ++j) {
    const int k0 = block.at(j) * kKeys;
    const bool hidden = k0 + kKeys - 1 > block.s.p_lo;
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
        for (int n = 0; n < 4; ++n) s2[i][n] = add_pair(s2[i][n], fma_pair(x.y, y[n].y, mul_pair(x.x, y[n].x)));
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
        if (hidden && k0 + cg + 16 * n > pos[i]) w[i][n] = kNegInf;
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
    if (!block.live(a, r)) continue;
    float* out = block.part<D>(a, r, m[i], ls, cg == 0);
#pragma unroll
    for (int c = 0; c < CP; ++c) {
      float x, y;
      unpair(o[i][c], &x, &y);
      float* dst = out + (2 * c / VW) * 16 * VW + cg * VW + 2 * c % VW;
      if constexpr (VW >= 2) *reinterpret_cast<float2*>(dst) = make_float2(x, y);
      else *dst = x;
    }
  }
  block.finish();
}

cudaError_t launch(const void* kernel, const PagedSharedArgs& a, int64_t grid, int threads, int smem,
                   std::atomic<uint64_t>& done, cudaStream_t stream) {
  cudaError_t e = allow_smem(kernel, smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[1] = {const_cast<PagedSharedArgs*>(&a)};
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

template <int D>
cudaError_t launch_mma(const PagedSharedArgs& a, int64_t grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  return launch(reinterpret_cast<const void*>(&paged_shared_mma_kernel<D>), a, grid, kMmaThreads,
                4 * kKeys * D * 2, done, stream);
}

template <int D, int R, int M>
cudaError_t launch_fma(const PagedSharedArgs& a, int64_t grid, cudaStream_t stream) {
  constexpr int kThreads = 16 * R / M;
  static_assert(sizeof(Families) <= fma_smem<D, R>(), "the groups fit where the tiles will lie");
  static std::atomic<uint64_t> done{0};
  return launch(reinterpret_cast<const void*>(&paged_shared_fma_kernel<D, R, M>), a, grid, kThreads,
                fma_smem<D, R>(), done, stream);
}

// ---- many groups ---------------------------------------------------------------------
//
// What the members of each group see of its prefix, a warp for each group, where the groups are more than the kernels' own
// tables hold.  Bound by its launch.

constexpr int kSeenWarps = 8;

__global__ void __launch_bounds__(kSeenWarps * 32) paged_shared_seen_kernel(const __grid_constant__ PagedSharedArgs a) {
  const int lane = threadIdx.x & 31, i = blockIdx.x * kSeenWarps + (threadIdx.x >> 5);
  if (i >= a.groups) return;
  const int start = a.group_start[i], end = a.group_start[i + 1];
  int most = 0;
  if (start >= 0 && end > start && end <= a.pool.batch) {
    for (int b = start + lane; b < end; b += 32)
      most = max(most, shared_len(a.prefix_lens[b], paged_len(a.pool, b), a.fresh != 0));
    most = __reduce_max_sync(0xffffffffu, most);
    most = min(most, max(a.prefix_lens[start], 0));
  }
  if (lane == 0) a.seen[i] = most;
}

// ---- the join --------------------------------------------------------------------------
//
// A block per sequence and KV head.  The rest's share is in its place, or in the parts of the CTAs whose ranges
// met it (lf_paged_decode.cu); the prefix's shares are rows that its blocks left.  Warps take a row of the group each, or
// every so many of its shares, and join through shared memory, in order of position.  Bound by latency: what the call was given is
// read while the kernel before drains, then come two reads that depend on each other, places and shares.
constexpr int kJoinBatch = 4;

// Shares i = 0 .. n - 1 of a row (maximum and sum at ml(i), output at o(i)[D]) joined in their order, kJoinBatch of
// them read at once: lane j holds columns E j .. E j + E - 1.
template <int D, class Ml, class O>
__device__ __forceinline__ void join_shares(int n, Ml ml, O o, int lane, float* m_out, float* l_out, float* acc) {
  constexpr int E = D >= 32 ? D / 32 : 1;
  const int col = (lane * E) % D;
  float m = kNegInf, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kJoinBatch) {
    float s[kJoinBatch], t[kJoinBatch], v[kJoinBatch][E];
    float top = m;
#pragma unroll
    for (int u = 0; u < kJoinBatch; ++u) {
      s[u] = kNegInf;
      if (i0 + u < n) {
        const float* p = ml(i0 + u);
        s[u] = p[0];
        t[u] = p[1];
        const float* x = o(i0 + u) + col;
#pragma unroll
        for (int e = 0; e < E; ++e) v[u][e] = x[e];
      } else {
        t[u] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[u][e] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kJoinBatch; ++u) top = fmaxf(top, s[u]);
    const float mu = top == kNegInf ? 0.f : top, f = ex2(m - mu);
    m = top;
    l *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f;
#pragma unroll
    for (int u = 0; u < kJoinBatch; ++u) {
      const float w = ex2(s[u] - mu);
      l = fmaf(t[u], w, l);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(v[u][e], w, acc[e]);
    }
  }
  *m_out = m;
  *l_out = l;
}

template <typename T, int D, int G, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_shared_join_kernel(const __grid_constant__ PagedSharedArgs a,
                                                                            const __grid_constant__ PagedDecodeArgs d,
                                                                            int ctas) {
  constexpr int E = D >= 32 ? D / 32 : 1;
  constexpr int kStripes = kJoinWarps / G;
  __shared__ float s_o[kJoinWarps][D];
  __shared__ float s_ml[kJoinWarps][2];
  __shared__ int s_first[kJoinWarps], s_count[kJoinWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / a.pool.kv_heads, g = blockIdx.x - b * a.pool.kv_heads;
  // The sequence's group: the last one that starts at or before it.
  int lo = 0, n = a.groups;
  do {
    const int step = (n + 31) / 32, i = lane * step;
    const int k = __popc(__ballot_sync(0xffffffffu, i < n && (lane == 0 || a.group_start[lo + i] <= b))) - 1;
    lo += k * step;
    n = min(step, n - k * step);
  } while (n > 1);
  const int start = a.group_start[lo], end = a.group_start[lo + 1];
  bool right = start >= 0 && b >= start && b < end && end <= a.pool.batch;
  if (right) right = a.prefix_lens[b] <= max(a.prefix_lens[start], 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!right) {   // of no group, or a longer prefix than its group's: left as it is
    if (tid == 0 && g == 0 && a.pool.err) atomicOr(a.pool.err, LF_DEVERR_STATE);
    return;
  }
  // The CTAs whose ranges start inside the rest of this unit; what the prefix's blocks say of the group.
  const int unit = b * a.pool.kv_heads + g;
  int segs = a.segments[lo];
  const int64_t group_first = a.first_row[lo];
  const unsigned range_ctas = a.ranges[0], places = a.ranges[1], in_front = a.ranges[2];
  int w0 = INT_MAX, count = 0;
  for (int i = tid; i < ctas; i += kJoinWarps * 32)
    if (d.part_unit[i] == unit) {
      w0 = min(w0, i);
      ++count;
    }
  w0 = __reduce_min_sync(0xffffffffu, w0);
  count = __reduce_add_sync(0xffffffffu, count);
  if (lane == 0) {
    s_first[warp] = w0;
    s_count[warp] = count;
  }
  // The prefix's shares: `segs` rows of part_o from `row`, `apart` rows apart.
  const int each = a.rows / G, piece = (b - start) / each, members = min(each, end - start - piece * each);
  int64_t row = 0, apart = (int64_t)members * G;
  bool room = true;
  if (segs > 0 && range_ctas > 0) {
    const Ranges ranges(places, range_ctas);
    const unsigned first = (unsigned)group_first + (unsigned)(piece * a.pool.kv_heads + g) * (segs + in_front) + in_front;
    const unsigned cta = ranges.owner(first);
    segs = ranges.owner(first + segs - 1) - cta + 1;
    apart = a.slot_rows;
    row = cta * apart + (int64_t)(start + piece * each) * a.q_heads + (int64_t)g * members * G + (b - start - piece * each) * G;
  } else if (segs > 0) {
    row = group_first + (int64_t)piece * each * a.q_heads * segs + g * segs * apart + (b - start - piece * each) * G;
  }
  if (segs != 0) room = segs > 0 && row >= 0 && row + (segs - 1) * apart + G <= a.part_rows;
  __syncthreads();
  w0 = INT_MAX;
  count = 0;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) {
    w0 = min(w0, s_first[i]);
    count += s_count[i];
  }
  const int w = w0, rest = count > 0 ? count + 1 : 1;
  const int parts = rest + (room ? segs : 0);
  const int h = warp % G, stripe = warp / G;
  const int64_t out_row = (int64_t)b * a.q_heads + g * G + h;
  auto slot = [&](int i) { return (i == 0 ? 2 * (int64_t)(w - 1) + 1 : 2 * (int64_t)(w - 1 + i)) * G + h; };
  auto ml = [&](int i) -> const float* {
    if (i >= rest) return a.part_ml + 2 * (row + (i - rest) * apart + h);
    return rest == 1 ? d.rest_ml + 2 * out_row : d.part_ml + 2 * slot(i);
  };
  auto o = [&](int i) -> const float* {
    if (i >= rest) return a.part_o + (row + (i - rest) * apart + h) * D;
    return rest == 1 ? d.rest_o + out_row * D : d.part_o + slot(i) * D;
  };
  const int mine = parts > stripe ? (parts - stripe + kStripes - 1) / kStripes : 0;
  float m, l, acc[E];
  join_shares<D>(
      mine, [&](int i) { return ml(stripe + i * kStripes); }, [&](int i) { return o(stripe + i * kStripes); }, lane, &m, &l,
      acc);
  if constexpr (kStripes > 1) {
    if (lane * E < D) {
#pragma unroll
      for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
    }
    if (lane == 0) {
      s_ml[warp][0] = m;
      s_ml[warp][1] = l;
    }
    __syncthreads();
    if (stripe > 0) return;
    join_shares<D>(
        min(parts, kStripes), [&](int i) { return s_ml[h + i * G]; }, [&](int i) { return s_o[h + i * G]; }, lane, &m, &l,
        acc);
  }
  const float inv = inverse_sum(l);
  T* out = reinterpret_cast<T*>(d.out) + out_row * D;
  if (lane * E < D) {
#pragma unroll
    for (int e = 0; e < E; ++e) from_f32(acc[e] * inv, out + lane * E + e);
  }
  if (lane == 0) {
    write_row_stats(d, out_row, m, l);
    if (!room && g == 0 && h == 0 && a.pool.err) atomicOr(a.pool.err, LF_DEVERR_STATE);
  }
}

template <typename T, int D, int G, int W>
cudaError_t launch_join_warps(const PagedSharedArgs& a, const PagedDecodeArgs& rest, int ctas, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.pool.batch * a.pool.kv_heads), 1, 1);
  cfg.blockDim = dim3(W * 32, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_shared_join_kernel<T, D, G, W>, a, rest, ctas);
}

template <typename T, int D, int G>
cudaError_t launch_join(const PagedSharedArgs& a, const PagedDecodeArgs& rest, int ctas, cudaStream_t stream) {
  // Few units: more warps for each.  (8 behind 2000, 64 units: 16 warps 17.0 us, 8 17.8, 4 19.1; 32 behind 60000, 256 units: 68.8,
  // 70.5, 73.7; 64 behind 8192, 512: 53.1, 52.9, 52.4; 256 in 16 groups, 1944: 126, 117, 112.  A number that the
  // kernel is told of and not built with costs registers: 114 and 72.8.)
  if ((int64_t)a.pool.batch * a.pool.kv_heads <= 2 * (int64_t)ctas) return launch_join_warps<T, D, G, 16>(a, rest, ctas, stream);
  return launch_join_warps<T, D, G, (G > 4 ? G : 4)>(a, rest, ctas, stream);
}

template <typename T, int D>
cudaError_t join_group(const PagedSharedArgs& a, const PagedDecodeArgs& rest, int ctas, cudaStream_t stream) {
  switch (a.group) {
    case 1: return launch_join<T, D, 1>(a, rest, ctas, stream);
    case 2: return launch_join<T, D, 2>(a, rest, ctas, stream);
    case 4: return launch_join<T, D, 4>(a, rest, ctas, stream);
    default: return launch_join<T, D, 8>(a, rest, ctas, stream);
  }
}

template <typename T>
cudaError_t join_dim(const PagedSharedArgs& a, const PagedDecodeArgs& rest, int head_dim, int ctas, cudaStream_t stream) {
  switch (head_dim) {
    case 16: return join_group<T, 16>(a, rest, ctas, stream);
    case 32: return join_group<T, 32>(a, rest, ctas, stream);
    case 64: return join_group<T, 64>(a, rest, ctas, stream);
    default: return join_group<T, 128>(a, rest, ctas, stream);
  }
}

}  // namespace

cudaError_t paged_shared_seen_launch(const PagedSharedArgs& a, cudaStream_t stream) {
  paged_shared_seen_kernel<<<(a.groups + kSeenWarps - 1) / kSeenWarps, kSeenWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

SharedPlan paged_shared_plan(const PagedPool& pool, int elem, int head_dim, int group, int groups, int sms) {
  SharedPlan p;
  p.keys = kKeys;
  p.least = 1;
  p.table = kTableOther;
  if (elem == 2 && paged_prompt_tc_takes(pool, head_dim)) {
    p.kernel = PromptPlan::kTensor;
    p.table = kTableTensor;
    p.rows = 256;
    p.keys = 128;
    p.slots = sms;
  } else if (elem == 2) {
    // Shares of three tiles or more: of one they are as much as its keys (four groups of eight behind 1000 to 2000 tokens, heads
    // of 32, 16.2 us, of one tile 21.0).  A tile of fp32 takes longer than a block's start (24 behind 3000, heads of
    // 64, shares of one tile 30 us, of two 36).
    p.kernel = PromptPlan::kMatrix;
    p.least = 3;
    p.rows = kMmaRows;
    p.slots = sms * (head_dim == 128 ? 3 : head_dim >= 32 ? 4 : 5);
  } else {
    p.kernel = PromptPlan::kFma;
    // Blocks of 64 rows read a key half as often as those of 32 and take each tile longer: for groups of 256 rows on average
    // (heads of 128; 8 KV heads, 256 rows behind 4000: 160 us, in blocks of 32 174; 2 KV heads behind 16000: 130, 142, but behind
    // 2000: 47, 43).  Of fewer rows blocks of 32 are as fast or faster (8 KV heads behind 4000, 192 rows: 148 us, of 64 148; 128: 112,
    // 110; 96: 91, 104; 64: 66, 68; one: 33, 48; 2 KV heads, 64 behind 2000: 29, 39).
    p.rows = head_dim == 128 && (int64_t)pool.batch * group >= 256ll * groups ? 64 : 32;
    p.slots = sms * (head_dim == 128 ? 2 : 4);
  }
  // Pieces of groups that sum to the batch: the most there can be.
  const int64_t each = p.rows / group;
  const int64_t pieces = ((int64_t)pool.batch + groups * (each - 1)) / each;
  const int64_t units = (pieces < pool.batch ? pieces : pool.batch) * pool.kv_heads;
  p.slot_rows = (int)((int64_t)pool.batch * group < p.rows ? (int64_t)pool.batch * group : p.rows);
  if (p.kernel == PromptPlan::kTensor) {   // ranges: a slot for each CTA, and a unit's own rows
    const int64_t tiles = ((int64_t)pool.max_pages * pool.page_size + p.keys - 1) / p.keys;
    p.grid = sms;
    p.rounds = 1;
    p.part_rows = (int64_t)sms * p.slot_rows + (int64_t)pool.batch * group * pool.kv_heads;
    p.fits = units * (tiles + 8) <= INT_MAX;
    return p;
  }
  p.rounds = 2 * units <= p.slots ? 1 : (int)(units / p.slots) + 2;
  p.grid = (int64_t)p.rounds * p.slots;
  // A unit of c-tile segments has at most one more than its share of the room (segment_tiles).
  p.part_rows = (int64_t)p.slot_rows * 2 * p.slots + (int64_t)pool.batch * group * pool.kv_heads;
  p.fits = p.grid <= INT_MAX;
  return p;
}

cudaError_t paged_shared_launch(const PagedSharedArgs& a, const SharedPlan& plan, int head_dim, cudaStream_t stream) {
  if (plan.kernel == PromptPlan::kMatrix) {
    switch (head_dim) {
      case 16: return launch_mma<16>(a, plan.grid, stream);
      case 32: return launch_mma<32>(a, plan.grid, stream);
      case 64: return launch_mma<64>(a, plan.grid, stream);
      default: return launch_mma<128>(a, plan.grid, stream);
    }
  }
  switch (head_dim) {
    case 16: return launch_fma<16, 32, 4>(a, plan.grid, stream);
    case 32: return launch_fma<32, 32, 4>(a, plan.grid, stream);
    case 64: return launch_fma<64, 32, 4>(a, plan.grid, stream);
    default: return plan.rows == 64 ? launch_fma<128, 64, 8>(a, plan.grid, stream) : launch_fma<128, 32, 4>(a, plan.grid, stream);
  }
}

cudaError_t paged_shared_join_launch(const PagedSharedArgs& a, const PagedDecodeArgs& rest, int elem, int head_dim,
                                     int ctas, cudaStream_t stream) {
  return elem == 2 ? join_dim<__nv_bfloat16>(a, rest, head_dim, ctas, stream) : join_dim<float>(a, rest, head_dim, ctas, stream);
}

}  // namespace lf
