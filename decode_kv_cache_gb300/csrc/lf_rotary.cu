// Rotary positions: rows of heads rotated where they lie or on their way to a paged cache
// (declarations and semantics: include/longflow.h).
//
//   (x_a, x_b) -> (x_a cos w - x_b sin w, x_b cos w + x_a sin w),  w = frequency_i * position
//
// for pair i of a row's first columns; the rest of a row, and values, are copied bit by bit.
//
// The angle.  fp32 holds w to 2^-24 of itself, which at position 100000 is 0.006 of a radian.  Only w modulo a
// turn counts, so a frequency is kept as a 64-bit fraction of a turn per position, and its
// product with the position modulo 2^64 IS the fraction of the turn: one integer multiplication, off by 2^-65
// of a turn for each position.  Its nearest quarter is taken off as an integer too, and sincospif gets the rest,
// at most an eighth of a turn, rounded to 2^-25 of itself.
//
// Work.  A row's eight columns and the eight that they turn with make an item, which one thread reads, turns
// and writes (so that a tensor may be rotated in place); its pairs' cosines and sines are the same for every head of the
// token and stay in its registers.  A warp takes a token, or a slice of the token's heads where there are
// few tokens: its lanes first ask for their first items, then look up where the token goes and what
// its position is, share the token's sines through shared memory, and go on.  Bound by HBM: every
// row is read and written once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "lf_device.cuh"
#include "lf_kernels.h"
#include "lf_paged.h"
#include "lf_paged_host.h"
#include "longflow.h"

namespace lf {

namespace {

constexpr int kWarps = 8;
constexpr int kMaxRow = 512;         // columns of a row: an item for each lane at most
constexpr int kMaxPairs = kMaxRow / 2;

struct RotaryRows {                  // strides in bytes
  const char* x;
  char* y;
  int heads;
  int64_t xs, xt, xh, ys, yt, yh;    // of sequences, tokens and heads
};

struct RotaryArgs {
  const uint64_t* turns;
  const int32_t* axis;               // may be null: axis 0
  const int32_t* positions;          // [axes][tokens], or null: the position in the cache
  int64_t axis_stride;
  int half, axes;
  float scale;
  int inverse;
  RotaryRows q, k;                   // either may have no heads
  const char* v;                     // paged: as k.x
  int items, heads_at_once;          // items of a row, heads that a warp's lanes cover
  int64_t tokens;
  int tokens_per_seq;                // not paged
  int slices, steps;                 // warps of a token, steps of heads_at_once heads in all
  PagedPool pool;                    // paged
  const int32_t* new_start;          // paged: [batch + 1], or null: one token per sequence
};

// The sequence that token t of a paged call belongs to and its place in the pools, for the whole warp together.
// *row: the token is one of a sequence's, *offset: where its rows go, -1: nowhere.
__device__ __forceinline__ void find_token(const RotaryArgs& a, int t, int lane, bool* row, int64_t* pos,
                                           int64_t* offset) {
  int b = t, first = t, end = t + 1;
  if (a.new_start) {
    int lo = 0, n = a.pool.batch;    // the last sequence of [lo, lo + n) that starts at or before t
    do {
      const int step = (n + 31) / 32, i = lane * step;
      const bool in = i < n;
      const int k = __popc(__ballot_sync(0xffffffffu, in && (lane == 0 || a.new_start[lo + i] <= t))) - 1;
      lo += k * step;
      n = min(step, n - k * step);
    } while (n > 1);
    b = lo;
    first = a.new_start[b];
    end = a.new_start[b + 1];
  }
  *offset = -1;
  *pos = 0;
  *row = first >= 0 && end >= first && end <= a.tokens && t >= first && t < end;
  if (!*row) return;
  *pos = (int64_t)a.pool.lens[b] - end + t;
  bool ok = *pos >= 0 && *pos < (int64_t)a.pool.max_pages * a.pool.page_size;
  if (ok) {
    int pi, slot;
    paged_split(a.pool, (int)*pos, &pi, &slot);
    const int page = a.pool.table[(int64_t)b * a.pool.max_pages + pi];
    ok = page >= 0 && page < a.pool.num_pages;
    if (ok) *offset = page * a.pool.page_stride + slot * a.pool.token_stride;
  }
  if (!ok && lane == 0 && a.pool.err) atomicOr(a.pool.err, LF_DEVERR_STATE);
}

// Cosine and sine of a position's angle, given as turns per position (2^-64 of a turn).
__device__ __forceinline__ float2 turn_of(uint64_t per_position, int64_t position) {
  const uint32_t w = (uint32_t)((per_position * (uint64_t)position) >> 32);   // modulo a turn, in 2^-32
  const uint32_t quarter = (w + 0x20000000u) >> 30;
  float s, c;
  sincospif((float)(int32_t)(w - (quarter << 30)) * 0x1p-31f, &s, &c);
  if (quarter & 1) {
    const float x = c;
    c = -s;
    s = x;
  }
  return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

__device__ __forceinline__ void unpack(const uint4 (&x)[1], float (&f)[8]) {
  const uint32_t w[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = bf2_to_f2(w[i]);
    f[2 * i] = y.x;
    f[2 * i + 1] = y.y;
  }
}
__device__ __forceinline__ void unpack(const uint4 (&x)[2], float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(x[i].x);
    f[4 * i + 1] = __uint_as_float(x[i].y);
    f[4 * i + 2] = __uint_as_float(x[i].z);
    f[4 * i + 3] = __uint_as_float(x[i].w);
  }
}
__device__ __forceinline__ uint32_t two_bf16(float x, float y) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
__device__ __forceinline__ void pack(const float (&f)[8], uint4 (&x)[1]) {
  x[0] = make_uint4(two_bf16(f[0], f[1]), two_bf16(f[2], f[3]), two_bf16(f[4], f[5]), two_bf16(f[6], f[7]));
}
__device__ __forceinline__ void pack(const float (&f)[8], uint4 (&x)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    x[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                      __float_as_uint(f[4 * i + 3]));
}

template <typename T, bool kPaged, bool kAdjacent>
__global__ void __launch_bounds__(kWarps * 32) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int W = sizeof(T) / 2;         // 16-byte words of eight columns
  constexpr int U = 4 / W;                 // items under way per thread
  __shared__ float2 s_turn[kWarps][kMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t id = (int64_t)blockIdx.x * kWarps + warp;
  if constexpr (kPaged) {
    if (a.new_start && a.pool.err)   // a sequence whose starts are wrong may have no token that finds it
      for (int64_t b = id * 32 + lane; b < a.pool.batch; b += (int64_t)gridDim.x * kWarps * 32) {
        const int first = a.new_start[b], end = a.new_start[b + 1];
        if (first < 0 || end < first || end > a.tokens) atomicOr(a.pool.err, LF_DEVERR_STATE);
      }
  }
  const int64_t t = id / a.slices;
  const int slice = (int)(id - t * a.slices);
  if (t >= a.tokens) return;
  const int from = (int)((int64_t)a.steps * slice / a.slices), to = (int)((int64_t)a.steps * (slice + 1) / a.slices);

  // This thread's item: eight columns at lo and eight at hi, in bytes.
  const int item = lane % a.items, first_head = lane / a.items;
  const int turning = a.half / 8;          // items that turn
  const bool turns = item < turning;
  int lo = 16 * item, hi = lo + 8;
  if (!kAdjacent && turns) {
    lo = 8 * item;
    hi = a.half + lo;
  }
  const int64_t seq = kPaged ? 0 : t / a.tokens_per_seq, ti = kPaged ? t : t - seq * a.tokens_per_seq;
  const char* qx = a.q.x + seq * a.q.xs + ti * a.q.xt;
  const char* kx = a.k.x + seq * a.k.xs + ti * a.k.xt;
  const char* vx = a.v + ti * a.k.xt;
  const int all = a.q.heads + a.k.heads * (kPaged ? 2 : 1);
  auto head_of = [&](int step) {           // of q, k and v in this order; -1: none
    const int h = step * a.heads_at_once + first_head;
    return first_head < a.heads_at_once && h < all ? h : -1;
  };
  uint4 xl[U][W], xh[U][W];
  auto load = [&](int step) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = step + u < to ? head_of(step + u) : -1, g = h - a.q.heads;
      if (h < 0) continue;
      const char* row = h < a.q.heads ? qx + h * a.q.xh : g < a.k.heads ? kx + g * a.k.xh : vx + (g - a.k.heads) * a.k.xh;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        xl[u][w] = __ldcs(reinterpret_cast<const uint4*>(row + lo * (int)sizeof(T)) + w);
        xh[u][w] = __ldcs(reinterpret_cast<const uint4*>(row + hi * (int)sizeof(T)) + w);
      }
    }
  };
  load(from);

  bool row = true;
  int64_t cache_pos = 0, offset = -1;
  if constexpr (kPaged) find_token(a, (int)t, lane, &row, &cache_pos, &offset);
  if (!row) return;                        // of no sequence: left as it is
  for (int i = lane; i < a.half; i += 32) {
    int64_t p = cache_pos;
    if (a.positions) {
      const int ax = a.axis ? min(max(a.axis[i], 0), a.axes - 1) : 0;
      p = a.positions[ax * a.axis_stride + t];
    }
    float2 y = turn_of(a.turns[i], a.inverse ? -p : p);
    y.x *= a.scale;
    y.y *= a.scale;
    s_turn[warp][i] = y;
  }
  __syncwarp();
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 y = turns ? s_turn[warp][8 * item + e] : make_float2(1.f, 0.f);
    c[e] = y.x;
    s[e] = y.y;
  }

  char* qy = a.q.y + seq * a.q.ys + ti * a.q.yt;
  char* ky = kPaged ? a.pool.k + offset : a.k.y + seq * a.k.ys + ti * a.k.yt;
  char* vy = kPaged ? a.pool.v + offset : nullptr;
  const int64_t kyh = kPaged ? a.pool.head_stride : a.k.yh;
  for (int step = from;;) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = step + u < to ? head_of(step + u) : -1, g = h - a.q.heads;
      if (h < 0 || (kPaged && g >= 0 && offset < 0)) continue;
      if (turns && g < a.k.heads) {
        float l[8], r[8], yl[8], yr[8];
        unpack(xl[u], l);
        unpack(xh[u], r);
        if constexpr (kAdjacent) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            yl[2 * e] = l[2 * e] * c[e] - l[2 * e + 1] * s[e];
            yl[2 * e + 1] = l[2 * e + 1] * c[e] + l[2 * e] * s[e];
            yr[2 * e] = r[2 * e] * c[4 + e] - r[2 * e + 1] * s[4 + e];
            yr[2 * e + 1] = r[2 * e + 1] * c[4 + e] + r[2 * e] * s[4 + e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            yl[e] = l[e] * c[e] - r[e] * s[e];
            yr[e] = r[e] * c[e] + l[e] * s[e];
          }
        }
        pack(yl, xl[u]);
        pack(yr, xh[u]);
      }
      char* out = h < a.q.heads ? qy + h * a.q.yh : g < a.k.heads ? ky + g * kyh : vy + (g - a.k.heads) * kyh;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        *(reinterpret_cast<uint4*>(out + lo * (int)sizeof(T)) + w) = xl[u][w];
        *(reinterpret_cast<uint4*>(out + hi * (int)sizeof(T)) + w) = xh[u][w];
      }
    }
    step += U;
    if (step >= to) break;
    load(step);
  }
}

template <typename T, bool kPaged>
cudaError_t launch(const RotaryArgs& a, int adjacent, cudaStream_t stream) {
  const unsigned grid = (unsigned)((a.tokens * a.slices + kWarps - 1) / kWarps);
  if (adjacent) rotary_kernel<T, kPaged, true><<<grid, kWarps * 32, 0, stream>>>(a);
  else rotary_kernel<T, kPaged, false><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

// Everything that does not depend on where the rows lie.
int take_rotary(const lf_rotary* r, int row_dim, const int32_t* positions, int64_t axis_stride, RotaryArgs* a) {
  if (!r) return fail(LF_ERR_ARG, "null rotary");
  if (r->rotary_dim < 16 || r->rotary_dim % 16 != 0 || r->rotary_dim > row_dim)
    return fail(LF_ERR_ARG, "rotary_dim (%d) must be a multiple of 16 and at most the rows' %d columns", r->rotary_dim,
                row_dim);
  if (r->axes < 1 || r->axes > LF_ROTARY_MAX_AXES)
    return fail(LF_ERR_ARG, "axes must be in [1, %d]", LF_ROTARY_MAX_AXES);
  if (r->adjacent != 0 && r->adjacent != 1) return fail(LF_ERR_ARG, "adjacent must be 0 or 1");
  if (!std::isfinite(r->scale)) return fail(LF_ERR_ARG, "scale must be finite");
  if (!r->turns || (reinterpret_cast<uintptr_t>(r->turns) & 7u) != 0)
    return fail(LF_ERR_ARG, "turns must be non-null and 8-byte aligned");
  if (!aligned4(r->axis) || !aligned4(positions)) return fail(LF_ERR_ARG, "axis and positions must be 4-byte aligned");
  if (axis_stride < 0) return fail(LF_ERR_ARG, "axis_stride must be >= 0 (0: every axis has the same positions)");
  a->turns = r->turns;
  a->axis = r->axes > 1 ? r->axis : nullptr;
  a->positions = positions;
  a->axis_stride = axis_stride;
  a->half = r->rotary_dim / 2;
  a->axes = r->axes;
  a->scale = r->scale;
  a->inverse = 0;
  a->q = a->k = RotaryRows{};
  a->v = nullptr;
  a->items = row_dim / 16;
  a->heads_at_once = 32 / a->items;
  a->pool = PagedPool{};
  a->new_start = nullptr;
  return LF_OK;
}

// Rows of lf_rotate; `rows` may be null for none.
int take_rows(const lf_rows* rows, const char* name, int elem, RotaryRows* out) {
  if (!rows) return LF_OK;
  if (rows->heads < 1 || rows->heads > 65535) return fail(LF_ERR_ARG, "%s: heads must be in [1, 65535]", name);
  if (!rows->x || !rows->y || !aligned16(rows->x) || !aligned16(rows->y))
    return fail(LF_ERR_ARG, "%s: x and y must be non-null and 16-byte aligned", name);
  const int64_t st[6] = {rows->x_seq, rows->x_token, rows->x_head, rows->y_seq, rows->y_token, rows->y_head};
  for (int64_t s : st)
    if (s < 0 || s > (int64_t)1 << 40 || (s * elem) % 16 != 0)
      return fail(LF_ERR_ARG, "%s: strides must be >= 0, at most 2^40 elements and whole multiples of 16 bytes", name);
  *out = RotaryRows{static_cast<const char*>(rows->x), static_cast<char*>(rows->y), rows->heads, st[0] * elem,
                    st[1] * elem, st[2] * elem, st[3] * elem, st[4] * elem, st[5] * elem};
  return LF_OK;
}

// How many warps a token gets: as many as it takes to fill the GPU with warps.
int take_slices(RotaryArgs* a, int heads) {
  int sms = 0;
  const int rc = sm_count(&sms);
  if (rc != LF_OK) return rc;
  a->steps = (heads + a->heads_at_once - 1) / a->heads_at_once;
  const int64_t want = ((int64_t)sms * 32 + a->tokens - 1) / a->tokens;
  a->slices = (int)(want < a->steps ? want : a->steps);
  return LF_OK;
}

}  // namespace

}  // namespace lf

// ---- C ABI --------------------------------------------------------------------

using lf::aligned16;
using lf::aligned4;
using lf::cuda_fail;
using lf::fail;

extern "C" {

int lf_rotary_turns(const double* frequency, int pairs, uint64_t* turns) {
  lf::clear_last_error();
  if (!frequency || !turns || pairs < 0) return fail(LF_ERR_ARG, "null frequency or turns, or pairs < 0");
  // 1 / (2 pi) in 2^-192, 32 bits at a time from the lowest.
  static const uint32_t kInverse[6] = {0x4f10e410u, 0x36d8a566u, 0x4d4d3770u, 0x7f09d5f4u, 0x9391054au, 0x28be60dbu};
  for (int i = 0; i < pairs; ++i) {
    if (!std::isfinite(frequency[i]) || std::fabs(frequency[i]) > 1024.0)
      return fail(LF_ERR_ARG, "frequency %d must be finite and at most 1024 radians per position", i);
    int e;
    const uint64_t m = (uint64_t)std::ldexp(std::frexp(std::fabs(frequency[i]), &e), 53);
    e -= 53;   // |frequency| = m 2^e, e <= -42
    // m / (2 pi) in 2^-192, then the 64 bits from 2^-64 on of its product with 2^e, rounded
    uint32_t p[9] = {0};
    const uint64_t half[2] = {m & 0xffffffffu, m >> 32};
    for (int h = 0; h < 2; ++h) {
      uint64_t carry = 0;
      for (int j = 0; j < 6; ++j) {
        carry += half[h] * kInverse[j] + p[h + j];
        p[h + j] = (uint32_t)carry;
        carry >>= 32;
      }
      p[h + 6] += (uint32_t)carry;
    }
    const int shift = 128 - e;   // at least 170
    auto bit = [&](int n) { return n < 9 * 32 ? (uint64_t)(p[n >> 5] >> (n & 31) & 1u) : 0ull; };
    uint64_t t = bit(shift - 1);
    for (int j = 0; j < 64; ++j) t += bit(shift + j) << j;
    turns[i] = frequency[i] < 0 ? 0 - t : t;
  }
  return LF_OK;
}

int lf_rotate(const lf_rotary* rotary, int dtype, int row_dim, int seqs, int tokens, const lf_rows* q, const lf_rows* k,
              const int32_t* positions, int64_t axis_stride, int inverse, lf_stream_t stream) {
  lf::clear_last_error();
  if (dtype != LF_BF16 && dtype != LF_F32) return fail(LF_ERR_ARG, "dtype must be LF_BF16 or LF_F32");
  if (row_dim < 16 || row_dim % 16 != 0 || row_dim > lf::kMaxRow)
    return fail(LF_ERR_ARG, "row_dim (%d) must be a multiple of 16 in [16, %d]", row_dim, lf::kMaxRow);
  lf::RotaryArgs a;
  int rc = lf::take_rotary(rotary, row_dim, positions, axis_stride, &a);
  if (rc != LF_OK) return rc;
  if (seqs < 0 || tokens < 0 || (int64_t)seqs * tokens > INT_MAX)
    return fail(LF_ERR_ARG, "need seqs, tokens >= 0 and seqs * tokens below 2^31");
  if (inverse != 0 && inverse != 1) return fail(LF_ERR_ARG, "inverse must be 0 or 1");
  if (!q) return fail(LF_ERR_ARG, "null q");
  const int elem = dtype == LF_BF16 ? 2 : 4;
  if (seqs == 0 || tokens == 0) return LF_OK;
  if ((rc = lf::take_rows(q, "q", elem, &a.q)) != LF_OK || (rc = lf::take_rows(k, "k", elem, &a.k)) != LF_OK) return rc;
  if (!positions) return fail(LF_ERR_ARG, "null positions");
  a.inverse = inverse;
  a.tokens = (int64_t)seqs * tokens;
  a.tokens_per_seq = tokens;
  if ((rc = lf::take_slices(&a, a.q.heads + a.k.heads)) != LF_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = elem == 2 ? lf::launch<__nv_bfloat16, false>(a, rotary->adjacent, st)
                                  : lf::launch<float, false>(a, rotary->adjacent, st);
  return e == cudaSuccess ? LF_OK : cuda_fail(e, "rotate launch");
}

int lf_paged_append_rotated(const lf_pages* pages, int batch, const int32_t* page_table, int max_pages,
                            const int32_t* lens, const void* k_new, const void* v_new, const int32_t* new_start,
                            int total_new, const lf_rotary* rotary, const int32_t* positions, int64_t axis_stride,
                            int q_heads, const void* q, void* q_out, lf_stream_t stream) {
  lf::clear_last_error();
  lf::PagedPool pool;
  lf::RotaryArgs a;
  int rc = lf::take_pool(pages, batch, page_table, max_pages, lens, &pool);
  if (rc != LF_OK || (rc = lf::take_rotary(rotary, pages->head_dim, positions, axis_stride, &a)) != LF_OK) return rc;
  if (total_new < 0) return fail(LF_ERR_ARG, "total_new < 0");
  if (!new_start && total_new != batch)
    return fail(LF_ERR_ARG, "without new_start every sequence takes one token: total_new (%d) must "
                "be the batch (%d)", total_new, batch);
  if (!q != !q_out || (q && (q_heads < 1 || q_heads > 65535)))
    return fail(LF_ERR_ARG, "q and q_out come together (or both null), with q_heads in [1, 65535]");
  if (total_new == 0) return LF_OK;
  if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new) || !aligned16(q) || !aligned16(q_out))
    return fail(LF_ERR_ARG, "k_new and v_new must be non-null, and they, q and q_out 16-byte aligned");
  if (!aligned4(new_start)) return fail(LF_ERR_ARG, "new_start must be 4-byte aligned");
  const int64_t row = (int64_t)pages->head_dim * lf::elem_bytes(pages);
  if (q)
    a.q = lf::RotaryRows{static_cast<const char*>(q), static_cast<char*>(q_out), q_heads, 0, row * q_heads, row, 0,
                         row * q_heads, row};
  a.k = lf::RotaryRows{static_cast<const char*>(k_new), nullptr, pages->kv_heads, 0, row * pages->kv_heads, row, 0, 0, 0};
  a.v = static_cast<const char*>(v_new);
  a.pool = pool;
  a.new_start = new_start;
  a.tokens = total_new;
  a.tokens_per_seq = total_new;
  if ((rc = lf::take_slices(&a, a.q.heads + 2 * a.k.heads)) != LF_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = pages->dtype == LF_BF16 ? lf::launch<__nv_bfloat16, true>(a, rotary->adjacent, st)
                                                : lf::launch<float, true>(a, rotary->adjacent, st);
  return e == cudaSuccess ? LF_OK : cuda_fail(e, "paged append launch");
}

}  // extern "C"
