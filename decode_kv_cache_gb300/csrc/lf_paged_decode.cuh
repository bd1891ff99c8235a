// The walk of the paged decode kernel: what it does and why stands in lf_paged_decode.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "lf_paged.cuh"
#include "longflow.h"

namespace lf {

namespace {

// ---- what one warp does with a tile ------------------------------------------
//
// The exponent of a weight, s log2(e) / sqrt(d) - m, is one multiply-add: its only rounding is that
// of the difference, and that m itself is rounded drops out.  (A scaled logit that is rounded before
// m is taken from it is off by 2^-24 of its own size, however near m it is.)
//
// A consumer holds a warp's running maximum (in units of log2), sum and output
// of one unit: begin(unit's queries), tile(...), and store(m, l, O) of G heads.

// bf16: legacy matrix instructions (m16n8k16), which leave the tile in shared
// memory layouts that any page gathers into; the tensor rate is not what bounds
// this kernel (32 of them per 16 tokens of 8 KB).  A's 16 rows are the heads:
// rows 0-7 take the group's queries, zero behind them.  For P.V rows 0-7 hold
// bf16(p) and rows 8-15 bf16(p - bf16(p)), so p keeps 16 bits at no cost: O is
// the sum of the two halves.
template <int D, int G, int Warps, int Stages>
struct MmaWalk {
  using T = __nv_bfloat16;
  static constexpr int kTokens = D == 128 ? 16 : D == 64 ? 32 : 64;
  static constexpr int kWarps = Warps, kStages = Stages, kExtra = 0;
  static constexpr int NC = D / 8;  // 16-byte chunks of a row
  uint32_t qa[D / 16][2];
  float o[D / 8][4];
  float m, l;  // of head lane / 4; l: this lane's columns only

  __device__ __forceinline__ void begin(const PagedDecodeArgs& a, int b, int g, float*) {
    const int lane = threadIdx.x & 31, r = lane >> 2;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q) +
                        (((int64_t)b * a.q_heads + (int64_t)g * G + r) * D) / 2 + (lane & 3);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qa[kk][0] = r < G ? q[kk * 8] : 0u;
      qa[kk][1] = r < G ? q[kk * 8 + 4] : 0u;
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
    m = kNegInf;
    l = 0.f;
  }

  __device__ __forceinline__ void tile(const PagedDecodeArgs& a, uint32_t ks, uint32_t vs, int valid,
                                       float*) {
    constexpr int NT = kTokens / 8;
    const int lane = threadIdx.x & 31;
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
    // S = q . K^T
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (D >= 32) {
#pragma unroll
        for (int c = 0; c < NC; c += 4) {  // four chunks: two steps of 16 along d
          uint32_t kb[4];
          ldmatrix4(ks + 16 * tile_chunk<NC>(8 * n + (lane & 7), c + (lane >> 3)), kb);
          mma16816(s[n], qa[c / 2][0], 0u, qa[c / 2][1], 0u, kb[0], kb[1]);
          mma16816(s[n], qa[c / 2 + 1][0], 0u, qa[c / 2 + 1][1], 0u, kb[2], kb[3]);
        }
      } else if ((n & 1) == 0) {  // d = 16: one step along d, two groups of eight tokens
        uint32_t kb[4];
        ldmatrix4(ks + 16 * tile_chunk<NC>(8 * n + (lane & 7) + 8 * (lane >> 4), (lane >> 3) & 1), kb);
        mma16816(s[n], qa[0][0], 0u, qa[0][1], 0u, kb[0], kb[1]);
        mma16816(s[n + 1], qa[0][0], 0u, qa[0][1], 0u, kb[2], kb[3]);
      }
    }
    float top = kNegInf;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = 8 * n + 2 * (lane & 3) + i;
        if (j >= valid) s[n][i] = kNegInf;
        top = fmaxf(top, s[n][i]);
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)) * a.scale_log2;
    if (__any_sync(0xffffffffu, top > m)) {
      const float mn = fmaxf(m, top);
      const float f = mn == kNegInf ? 1.f : ex2(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][i] *= f;
    }
    const float mu = m == kNegInf ? 0.f : m;
    uint32_t hi[NT], lo[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float p0 = ex2(fmaf(s[n][0], a.scale_log2, -mu)), p1 = ex2(fmaf(s[n][1], a.scale_log2, -mu));
      l += p0 + p1;
      hi[n] = pack_bf16(p0, p1);
      const float2 h = bf2_to_f2(hi[n]);
      lo[n] = pack_bf16(p0 - h.x, p1 - h.y);
    }
    // O += P . V
#pragma unroll
    for (int kk = 0; kk < kTokens / 16; ++kk) {
      const int row = 16 * kk + (lane & 7) + 8 * ((lane >> 3) & 1);
#pragma unroll
      for (int c = 0; c < NC; c += 2) {
        uint32_t vb[4];
        ldmatrix4_trans(vs + 16 * tile_chunk<NC>(row, c + (lane >> 4)), vb);
        mma16816(o[c], hi[2 * kk], lo[2 * kk], hi[2 * kk + 1], lo[2 * kk + 1], vb[0], vb[1]);
        mma16816(o[c + 1], hi[2 * kk], lo[2 * kk], hi[2 * kk + 1], lo[2 * kk + 1], vb[2], vb[3]);
      }
    }
  }

  // The whole unit's output rows, first row `row`.
  template <bool kBehind>
  __device__ __forceinline__ void write(const PagedDecodeArgs& a, int64_t row) {
    if constexpr (kBehind) return store(a.rest_o + row * D, a.rest_ml + row * 2);
    const int lane = threadIdx.x & 31, r = lane >> 2;
    float ls = l + __shfl_xor_sync(0xffffffffu, l, 1);
    ls += __shfl_xor_sync(0xffffffffu, ls, 2);
    if (r >= G) return;
    const float inv = inverse_sum(ls);
    uint32_t* out = reinterpret_cast<uint32_t*>(a.out) + ((row + r) * D) / 2 + (lane & 3);
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      out[4 * n] = pack_bf16((o[n][0] + o[n][2]) * inv, (o[n][1] + o[n][3]) * inv);
    if ((lane & 3) == 0) write_row_stats(a, row + r, m, ls);
  }

  // The unit's maximum, sum and output (not normalised) into po [G][D], pml [G][2].
  __device__ __forceinline__ void store(float* po, float* pml) {
    const int lane = threadIdx.x & 31, r = lane >> 2;
    float ls = l + __shfl_xor_sync(0xffffffffu, l, 1);
    ls += __shfl_xor_sync(0xffffffffu, ls, 2);
    if (r < G) {
      if ((lane & 3) == 0) {
        pml[2 * r] = m;
        pml[2 * r + 1] = ls;
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(po + r * D + 8 * n + 2 * (lane & 3)) =
            make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3]);
    }
  }
};

template <int D, int G>
struct MmaTile : MmaWalk<D, G, 8, 3> {};

// fp32: multiply-adds on the CUDA cores (tf32 would drop 13 bits of every
// factor).  For the logits a lane takes a token and a share of d; for P.V it
// takes four columns of O and a share of the tokens.  Each key and value is read
// from shared memory once for all G heads.  Extra shared memory of a warp: the
// group's queries [G][D], then the tile's weights [kTokens][G].
template <int D, int G>
struct SimtTile {
  using T = float;
  static constexpr int kTokens = D == 128 ? 8 : D == 64 ? 16 : 32;
  static constexpr int kWarps = 7, kStages = 3, kExtra = (G * D + kTokens * G) * 4;
  static constexpr int NC = D / 4;
  static constexpr int kShare = 32 / kTokens;   // lanes that share a token's dot product
  static constexpr int kRows = 32 / NC;         // tokens that P.V takes at once
  float o[G][4];
  float m[G], l[G];

  __device__ __forceinline__ void begin(const PagedDecodeArgs& a, int b, int g, float* extra) {
    const int lane = threadIdx.x & 31;
    const float* q = reinterpret_cast<const float*>(a.q) +
                     ((int64_t)b * a.q_heads + (int64_t)g * G) * D;
    __syncwarp();
    for (int i = lane; i < G * D / 4; i += 32)
      reinterpret_cast<float4*>(extra)[i] = reinterpret_cast<const float4*>(q)[i];
    __syncwarp();
#pragma unroll
    for (int h = 0; h < G; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[h][i] = 0.f;
      m[h] = kNegInf;
      l[h] = 0.f;
    }
  }

  __device__ __forceinline__ void tile(const PagedDecodeArgs& a, uint32_t ks, uint32_t vs, int valid,
                                       float* extra) {
    const int lane = threadIdx.x & 31;
    const ulonglong2* q4 = reinterpret_cast<const ulonglong2*>(extra);
    float* ps = extra + G * D;
    const int tok = lane % kTokens, part = lane / kTokens;
    // Four sums of a share's products, by column modulo 4 and in pairs: one alone would be a chain of 32
    // roundings, these are of at most 8.
    float s[G];
    uint64_t s2[G][2];
#pragma unroll
    for (int h = 0; h < G; ++h) s2[h][0] = s2[h][1] = 0ull;
#pragma unroll
    for (int i = 0; i < NC / kShare; ++i) {
      const int c = i * kShare + part;
      ulonglong2 k;
      asm volatile("ld.shared.v2.b64 {%0,%1}, [%2];"
                   : "=l"(k.x), "=l"(k.y)
                   : "r"(ks + 16 * tile_chunk<NC>(tok, c)));
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const ulonglong2 q = q4[h * NC + c];
        s2[h][0] = fma_pair(q.x, k.x, s2[h][0]);
        s2[h][1] = fma_pair(q.y, k.y, s2[h][1]);
      }
    }
    bool up = false;
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float x0, x1;
      unpair(add_pair(s2[h][0], s2[h][1]), &x0, &x1);
      s[h] = x0 + x1;
#pragma unroll
      for (int x = kTokens; x < 32; x <<= 1) s[h] += __shfl_xor_sync(0xffffffffu, s[h], x);
      if (tok >= valid) s[h] = kNegInf;
      up |= s[h] * a.scale_log2 > m[h];
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float mn = fmaxf(m[h], warp_max(s[h]) * a.scale_log2);
        const float f = mn == kNegInf ? 1.f : ex2(m[h] - mn);
        m[h] = mn;
        l[h] *= f;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[h][i] *= f;
      }
    }
    __syncwarp();  // the last tile's weights have been read
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float p = ex2(fmaf(s[h], a.scale_log2, m[h] == kNegInf ? 0.f : -m[h]));
      if (part == 0) {
        l[h] += p;
        ps[tok * G + h] = p;
      }
    }
    __syncwarp();
    const int c = lane % NC, r0 = lane / NC;
#pragma unroll
    for (int t = 0; t < kTokens; t += kRows) {
      float4 v;
      asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                   : "r"(vs + 16 * tile_chunk<NC>(t + r0, c)));
      const float* p = ps + (t + r0) * G;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float w = p[h];
        o[h][0] = fmaf(w, v.x, o[h][0]);
        o[h][1] = fmaf(w, v.y, o[h][1]);
        o[h][2] = fmaf(w, v.z, o[h][2]);
        o[h][3] = fmaf(w, v.w, o[h][3]);
      }
    }
  }

  // Sums over the lanes that hold shares of the same value.
  __device__ __forceinline__ void join_lanes() {
#pragma unroll
    for (int h = 0; h < G; ++h) {
      l[h] = warp_sum(l[h]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = NC; x < 32; x <<= 1) o[h][i] += __shfl_xor_sync(0xffffffffu, o[h][i], x);
    }
  }

  template <bool kBehind>
  __device__ __forceinline__ void write(const PagedDecodeArgs& a, int64_t row) {
    if constexpr (kBehind) return store(a.rest_o + row * D, a.rest_ml + row * 2);
    const int lane = threadIdx.x & 31;
    join_lanes();
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float inv = inverse_sum(l[h]);
      if (lane < NC)
        reinterpret_cast<float4*>(a.out)[(row + h) * NC + lane] =
            make_float4(o[h][0] * inv, o[h][1] * inv, o[h][2] * inv, o[h][3] * inv);
      if (lane == 0) write_row_stats(a, row + h, m[h], l[h]);
    }
  }

  __device__ __forceinline__ void store(float* po, float* pml) {
    const int lane = threadIdx.x & 31;
    join_lanes();
#pragma unroll
    for (int h = 0; h < G; ++h) {
      if (lane == 0) {
        pml[2 * h] = m[h];
        pml[2 * h + 1] = l[h];
      }
      if (lane < NC)
        *reinterpret_cast<float4*>(po + h * D + 4 * lane) =
            make_float4(o[h][0], o[h][1], o[h][2], o[h][3]);
    }
  }
};

// ---- the list of tiles ----------------------------------------------------------

// Positions that sequence b's query sees, numbered 0 .. seen - 1: number i is
// position i below `sinks`, else i + gap.
struct Seen {
  int len, seen, gap, tiles;
  bool right;   // the length fits the sequence's row of the page table
};

// kBehind: behind a shared prefix, whose positions are not seen here, and without a window.  (Known when the kernel is built:
// asked for at each place it cost a short decode 1 %, one sequence of 300 tokens 8.43 us, 8.37, and the walk beside prefixes
// more, 64 sequences behind 8192 51.2, 49.8.)
template <int TT, bool kBehind>
__device__ __forceinline__ Seen seen_of(const PagedDecodeArgs& a, int b) {
  Seen s;
  s.len = paged_len(a.pool, b);
  s.right = s.len == a.pool.lens[b];
  s.seen = s.len;
  if constexpr (kBehind) {
    s.seen = s.len - shared_len(a.prefix_lens[b], s.len, a.k_new != nullptr);
  } else if (a.window > 0) {
    const int64_t w = (int64_t)a.window + a.sinks;
    if (w < s.len) s.seen = (int)w;
  }
  s.gap = s.len - s.seen;
  s.tiles = (int)(((unsigned)s.seen + TT - 1) / TT);
  return s;
}

// A place in the list: tile t of (sequence b, KV head g).
struct Place {
  int b, g, t;
  Seen s;
};

// One step along the list, over empty sequences; past the end b is the batch.
template <int TT, bool kBehind>
__device__ __forceinline__ void step(const PagedDecodeArgs& a, Place& p) {
  if (++p.t < p.s.tiles) return;
  p.t = 0;
  if (++p.g < a.pool.kv_heads) return;
  p.g = 0;
  do {
    if (++p.b >= a.pool.batch) return;
    p.s = seen_of<TT, kBehind>(a, p.b);
  } while (p.s.tiles == 0);
}

template <typename T, int D, bool kBehind>
__device__ __forceinline__ void write_row(const PagedDecodeArgs& a, int64_t row, int lane, float m,
                                          float l, const float* acc) {
  constexpr int E = D >= 32 ? D / 32 : 1;
  if constexpr (kBehind) {
    if (lane * E < D) {
#pragma unroll
      for (int i = 0; i < E; ++i) a.rest_o[row * D + lane * E + i] = acc[i];
    }
    if (lane == 0) {
      a.rest_ml[row * 2] = m;
      a.rest_ml[row * 2 + 1] = l;
    }
    return;
  }
  const float inv = inverse_sum(l);
  T* out = reinterpret_cast<T*>(a.out) + row * D;
  if (lane * E < D) {
#pragma unroll
    for (int i = 0; i < E; ++i) from_f32(acc[i] * inv, out + lane * E + i);
  }
  if (lane == 0) write_row_stats(a, row, m, l);
}

// A warp's part of a unit that it does not take whole.
struct Part {
  int unit;            // b * kv_heads + g, or -1: no part
  int whole_start, whole_end;
};

// Shared memory of a warp: its ring, the consumer's own, a part; whole 128-byte lines.
template <class C, int D, int G>
__host__ __device__ constexpr int warp_bytes() {
  static_assert(C::kExtra % 16 == 0, "the part behind it starts on 16 bytes");
  return (C::kStages * 2 * C::kTokens * C::NC * 16 + C::kExtra + G * (D + 2) * 4 + 127) / 128 * 128;
}

// What a CTA does, as number `cta` of `ctas` that take the list together: its first kWarps warps, with kWarps * warp_bytes
// of shared memory, and `sync` among them.
template <class C, int D, int G, bool kBehind, class Sync>
__device__ __forceinline__ void decode_walk(const PagedDecodeArgs& a, unsigned char* smem, int cta, int ctas, Sync sync) {
  using T = typename C::T;
  constexpr int TT = C::kTokens, NC = C::NC, W = C::kWarps, S = C::kStages;
  constexpr int kTile = TT * NC * 16;       // bytes of a tile's keys (and of its values)
  constexpr int kPart = G * (D + 2);        // floats of a part: G outputs, then G maxima and sums
  constexpr int kRing = S * 2 * kTile;
  constexpr int kWarpBytes = warp_bytes<C, D, G>();
  static_assert(kPart * 4 <= kRing, "a part fits where the ring was");
  __shared__ Part s_part[2 * W];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = a.pool.kv_heads;

  // ---- this warp's range of the list: `left` tiles from place `at` -----------------
  Place at;
  long long left = 0;
  if (!kBehind && a.whole_units) {
    at.b = cta / H;
    at.g = cta - at.b * H;
    at.s = seen_of<TT, kBehind>(a, at.b);
    at.t = (int)((long long)at.s.tiles * warp / W);
    left = (int)((long long)at.s.tiles * (warp + 1) / W) - at.t;
  } else {
    // Tiles (of one head) before each thread's sequences, a scan over the CTA; it
    // borrows the rings' memory.
    long long* pre = reinterpret_cast<long long*>(smem);
    const int per = (a.pool.batch + W * 32 - 1) / (W * 32);
    long long sum = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b < a.pool.batch) sum += seen_of<TT, kBehind>(a, b).tiles;
    }
    long long x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) pre[W * 32 + 1 + warp] = x;
    sync();
    for (int w = 0; w < warp; ++w) x += pre[W * 32 + 1 + w];
    pre[tid + 1] = x;
    if (tid == 0) pre[0] = 0;
    sync();
    const long long total = pre[W * 32] * H;
    // Ranges of at least a tile per warp.
    const long long n = max(1ll, min((long long)ctas, (total + W - 1) / W));
    const long long i0 = min((long long)cta, n), i1 = min(cta + 1ll, n);
    const long long c0 = total * i0 / n, c1 = total * i1 / n;
    const long long x0 = c0 + (c1 - c0) * warp / W;
    left = c0 + (c1 - c0) * (warp + 1) / W - x0;
    auto place = [&](long long y, Place& p) {  // y < total
      int lo = 0, hi = W * 32;   // the last thread whose sequences start at or before y
      while (lo + 1 < hi) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] * H <= y) lo = mid;
        else hi = mid;
      }
      long long r = y - pre[lo] * H;
      p.b = lo * per;
      p.s = seen_of<TT, kBehind>(a, p.b);
      while (r >= (long long)p.s.tiles * H) {
        r -= (long long)p.s.tiles * H;
        p.s = seen_of<TT, kBehind>(a, ++p.b);
      }
      p.g = (int)(r / p.s.tiles);
      p.t = (int)(r - (long long)p.g * p.s.tiles);
    };
    if (left > 0 || (warp == 0 && c0 < c1)) place(x0, at);
    // For the join: the unit that this CTA's range starts inside.
    if (tid == 0) a.part_unit[cta] = c0 < c1 && at.t > 0 ? at.b * H + at.g : -1;
    sync();  // the scan's memory becomes the rings
  }

  // ---- the warp's walk ---------------------------------------------------------------
  unsigned char* wsm = smem + warp * kWarpBytes;
  const uint32_t ring = smem_u32(wsm);
  float* extra = reinterpret_cast<float*>(wsm + kRing);
  // A part that starts inside a unit is kept behind the ring, one that only ends
  // inside a unit (the range's last) where the ring was.
  float* const part_at[2] = {reinterpret_cast<float*>(wsm + kRing + C::kExtra),
                             reinterpret_cast<float*>(wsm)};
  if (lane < 2) s_part[2 * warp + lane].unit = -1;
  __syncwarp();

  // Copies of one tile.  Lane r looks up rows r, r + 32, ..; the lookups of the
  // tile after it are under way when its copies are issued.
  constexpr int RL = (TT + 31) / 32;
  Place ld = at;
  int64_t row_off[RL];   // byte offset of the row in the pools, -1: nothing to read
  auto look_up = [&]() {
#pragma unroll
    for (int i = 0; i < RL; ++i) {
      const int r = lane + 32 * i, j = ld.t * TT + r;
      row_off[i] = -1;
      if (r < TT && j < ld.s.seen) {
        const int pos = !kBehind && j < a.sinks ? j : j + ld.s.gap;
        int pi, slot;
        paged_split(a.pool, pos, &pi, &slot);
        const int page = __ldg(a.pool.table + (int64_t)ld.b * a.pool.max_pages + pi);
        if (page >= 0 && page < a.pool.num_pages)
          row_off[i] = page * a.pool.page_stride + slot * a.pool.token_stride;
        else if (a.pool.err)
          atomicOr(a.pool.err, LF_DEVERR_STATE);
      }
    }
  };
  auto issue = [&](int stage) {
    const uint32_t kd = ring + stage * 2 * kTile, vd = kd + kTile;
    // The new token's row comes from the call; the warp that meets it stores it.
    const int fresh = a.k_new && ld.s.right ? ld.s.seen - 1 - ld.t * TT : -1;
    const int64_t head = ld.g * a.pool.head_stride;
    const int64_t new_row = ((int64_t)ld.b * H + ld.g) * (NC * 16);
    constexpr int RPI = 32 / NC;   // rows that one instruction covers
    const int c = lane % NC;
#pragma unroll
    for (int i = 0; i < TT / RPI; ++i) {
      const int r = i * RPI + lane / NC;
      const int64_t off = __shfl_sync(0xffffffffu, row_off[(i * RPI) / 32], r & 31);
      const char* ks = a.pool.k + off + head + c * 16;
      const char* vs = a.pool.v + off + head + c * 16;
      bool ok = off >= 0;
      if (r == fresh) {
        ok = true;
        ks = a.k_new + new_row + c * 16;
        vs = a.v_new + new_row + c * 16;
      }
      const uint32_t d = 16 * tile_chunk<NC>(r, c);
      cp_async16(kd + d, ok ? ks : a.pool.k, ok);
      cp_async16(vd + d, ok ? vs : a.pool.v, ok);
    }
    if (fresh >= 0 && fresh < TT) {
      int64_t off = -1;
#pragma unroll
      for (int i = 0; i < RL; ++i) {
        const int64_t x = __shfl_sync(0xffffffffu, row_off[i], fresh & 31);
        if (fresh / 32 == i) off = x;
      }
      if (off >= 0 && lane < NC) {
        *reinterpret_cast<uint4*>(a.pool.k + off + head + lane * 16) =
            *reinterpret_cast<const uint4*>(a.k_new + new_row + lane * 16);
        *reinterpret_cast<uint4*>(a.pool.v + off + head + lane * 16) =
            *reinterpret_cast<const uint4*>(a.v_new + new_row + lane * 16);
      }
    }
  };
  long long to_load = left;
  if (to_load > 0) look_up();
  auto load_next = [&](int stage) {
    if (to_load > 0) {
      issue(stage);
      if (--to_load > 0) {
        step<TT, kBehind>(a, ld);
        look_up();
      }
    }
    cp_async_commit();   // a group per tile, empty ones at the end
  };
#pragma unroll
  for (int st = 0; st < S - 1; ++st) load_next(st);

  C c;
  int stage = 0;
  bool open = false, from_start = false;
#pragma unroll 1
  for (; left > 0; --left) {
    if (!open) {
      c.begin(a, at.b, at.g, extra);
      open = true;
      from_start = at.t == 0;
    }
    cp_async_wait<S - 2>();
    __syncwarp();
    const uint32_t kd = ring + stage * 2 * kTile;
    if constexpr (S == 2) load_next(stage ^ 1);   // on its way while this one is taken
    c.tile(a, kd, kd + kTile, min(TT, at.s.seen - at.t * TT), extra);
    __syncwarp();
    if constexpr (S > 2) load_next(stage == 0 ? S - 1 : stage - 1);
    stage = stage + 1 == S ? 0 : stage + 1;
    const bool unit_end = at.t + 1 == at.s.tiles;
    if (unit_end && from_start) {
      c.template write<kBehind>(a, (int64_t)at.b * a.q_heads + at.g * G);
      open = false;
    } else if (unit_end || left == 1) {
      const int k = from_start ? 1 : 0;
      if (k == 1) cp_async_wait<0>();   // the ring is done with
      __syncwarp();
      c.store(part_at[k], part_at[k] + G * D);
      if (lane == 0) s_part[2 * warp + k] = Part{at.b * H + at.g, from_start, unit_end};
      open = false;
    }
    step<TT, kBehind>(a, at);
  }
  cp_async_wait<0>();
  sync();

  // ---- sequences that see nothing have no tile and give zeros -----------------------------
  auto nothing_seen = [&](int b, int first_head, int heads) {
    const Seen s = seen_of<TT, kBehind>(a, b);
    const int64_t row = (int64_t)b * a.q_heads + first_head;
    if (s.tiles == 0 && kBehind) {
      for (int i = tid; i < heads * D; i += W * 32) a.rest_o[row * D + i] = 0.f;
      for (int i = tid; i < heads; i += W * 32) {
        a.rest_ml[(row + i) * 2] = kNegInf;
        a.rest_ml[(row + i) * 2 + 1] = 0.f;
      }
    } else if (s.tiles == 0) {
      T* out = reinterpret_cast<T*>(a.out) + row * D;
      for (int i = tid; i < heads * D; i += W * 32) from_f32(0.f, out + i);
      if (a.lse)
        for (int i = tid; i < heads; i += W * 32) a.lse[row + i] = kNegInf;
    }
    if (tid == 0 && first_head == 0 && a.pool.err && !s.right) atomicOr(a.pool.err, LF_DEVERR_STATE);
  };
  if (!kBehind && a.whole_units) {
    const int b = cta / H;
    nothing_seen(b, (cta - b * H) * G, G);
  } else {
    for (int b = cta; b < a.pool.batch; b += ctas) nothing_seen(b, 0, a.q_heads);
  }

  // ---- join the warps' parts -----------------------------------------------------------
  // In order of position the parts are warp 0's first and last, warp 1's, ..; a
  // unit's parts follow one another and start where one has whole_start, or at
  // the CTA's first part.  Warps take (unit, head) pairs in turn.
  int item = 0, p = 0;
  while (p < 2 * W) {
    if (s_part[p].unit < 0) {
      ++p;
      continue;
    }
    const int first = p, unit = s_part[p].unit;
    const bool starts = s_part[p].whole_start;
    bool ends = s_part[p].whole_end;
    for (++p; p < 2 * W && (s_part[p].unit < 0 || (s_part[p].unit == unit && !s_part[p].whole_start)); ++p)
      if (s_part[p].unit >= 0) ends = s_part[p].whole_end;
    for (int h = 0; h < G; ++h, ++item) {
      if (item % W != warp) continue;
      constexpr int E = D >= 32 ? D / 32 : 1;
      float m, l, acc[E];
      // parts without a unit count nothing: their place reads as the first part's,
      // with a maximum of -inf
      const float none[2] = {kNegInf, 0.f};
      auto base = [&](int i) {
        const int q = s_part[first + i].unit < 0 ? first : first + i;
        return reinterpret_cast<const float*>(smem + (q >> 1) * kWarpBytes +
                                              ((q & 1) ? 0 : kRing + C::kExtra));
      };
      join_parts<D>(
          p - first,
          [&](int i) { return s_part[first + i].unit < 0 ? none : base(i) + G * D + 2 * h; },
          [&](int i) { return base(i) + h * D; }, lane, &m, &l, acc);
      if (starts && ends) {
        const int b = unit / H;
        write_row<T, D, kBehind>(a, (int64_t)b * a.q_heads + (unit - b * H) * G + h, lane, m, l, acc);
      } else {
        const int64_t slot = 2 * (int64_t)cta + (starts ? 1 : 0);
        float* o = a.part_o + (slot * G + h) * D;
        if (lane * E < D) {
#pragma unroll
          for (int e = 0; e < E; ++e) o[lane * E + e] = acc[e];
        }
        if (lane == 0) {
          a.part_ml[(slot * G + h) * 2] = m;
          a.part_ml[(slot * G + h) * 2 + 1] = l;
        }
      }
    }
  }
}

// ---- the kernel and its launch --------------------------------------------------------

template <class C, int D, int G, bool kBehind>
__global__ void __launch_bounds__(C::kWarps * 32, 1) paged_decode_kernel(const __grid_constant__ PagedDecodeArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  // Everything below reads what earlier launches of the stream wrote.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  decode_walk<C, D, G, kBehind>(a, smem, blockIdx.x, gridDim.x, [] { __syncthreads(); });
}

// Launches that are placed while the one before them drains.
struct DrainConfig {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg;
  DrainConfig(dim3 grid, int threads, int smem, cudaStream_t stream) : cfg{} {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

template <class C, int D, int G, bool kBehind>
cudaError_t launch_walk(const PagedDecodeArgs& a, int grid, cudaStream_t stream) {
  constexpr int kSmem = C::kWarps * warp_bytes<C, D, G>();
  static_assert(kSmem + (2 * C::kWarps * (int)sizeof(Part) + 127) / 128 * 128 <= 232448, "shared memory of one CTA");
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(&paged_decode_kernel<C, D, G, kBehind>), kSmem, done);
  if (e != cudaSuccess) return e;
  const DrainConfig c(dim3(grid, 1, 1), C::kWarps * 32, kSmem, stream);
  return cudaLaunchKernelEx(&c.cfg, paged_decode_kernel<C, D, G, kBehind>, a);
}

// L::launch<C, D, G> for a call's heads.
template <class L, template <int, int> class C, int D>
cudaError_t by_group(const PagedDecodeArgs& a, int grid, cudaStream_t stream) {
  switch (a.group) {
    case 1: return L::template launch<C<D, 1>, D, 1>(a, grid, stream);
    case 2: return L::template launch<C<D, 2>, D, 2>(a, grid, stream);
    case 4: return L::template launch<C<D, 4>, D, 4>(a, grid, stream);
    default: return L::template launch<C<D, 8>, D, 8>(a, grid, stream);
  }
}

template <class L, template <int, int> class C>
cudaError_t by_dim(const PagedDecodeArgs& a, int head_dim, int grid, cudaStream_t stream) {
  switch (head_dim) {
    case 16: return by_group<L, C, 16>(a, grid, stream);
    case 32: return by_group<L, C, 32>(a, grid, stream);
    case 64: return by_group<L, C, 64>(a, grid, stream);
    default: return by_group<L, C, 128>(a, grid, stream);
  }
}

template <class L>
cudaError_t by_type(const PagedDecodeArgs& a, int elem, int head_dim, int grid, cudaStream_t stream) {
  return elem == 2 ? by_dim<L, MmaTile>(a, head_dim, grid, stream) : by_dim<L, SimtTile>(a, head_dim, grid, stream);
}

}  // namespace

}  // namespace lf
