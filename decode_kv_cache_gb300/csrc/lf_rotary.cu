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
// of a turn for each position.  Its nearest quarter is taken off as an integer too, and sincospif gets the rest, at
// most an eighth of a turn, all 64 bits of it rounded once to a float, by 2^-24 of itself: sines of small angles are as
// exact as large ones, and opposite positions turn by opposite angles.
//
// Work.  Two 16-byte chunks of a row make an item, which one thread reads, turns and writes: those that turn with
// each other where pairs are half a row apart, so that a tensor may be rotated in place.  Neighbouring lanes take neighbouring
// chunks (with 32 bytes a lane fp32 read half sectors: 17 slab prompts 20 us instead of 12).  An item's cosines and sines are the
// same for every head of the token and stay in registers.  A warp takes a token, a slice of its heads where
// there are few tokens, or a few tokens where they are short.  Its lanes first ask for their first items (a ring of
// cp.async copies), then look up where the tokens go and what their positions are, share the sines through shared
// memory, and go on.  Warps that walked the whole call with such a ring were slower (32 prompts 129 us against 110):
// their lookups come one after another, those of fresh warps side by side.
//
// Bound by HBM: every row is read and written once.  Measured, other inputs every time, of a plain copy's 6.77 TB/s:
// 32 prompts, 34 thousand tokens of 48 rows of 128 bf16 columns, 110 us, 97 %, in fp32 215 us, 99 %; 16000 video tokens of 40 rows
// 52.6 us, 92 %; 17 slab prompts of 1000 fp32 tokens 12.3 us, 84 %; two prompts of 6000 video tokens 37.8 us, 77 % (start and end of two
// waves of warps); a step of 64 sequences 3.1 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "lf_kernels.h"
#include "lf_overlap.h"
#include "lf_paged.cuh"
#include "lf_paged_host.h"
#include "longflow.h"

namespace lf {

namespace {

constexpr int kWarps = 8;
constexpr int kMaxRowBytes = 1024;   // an item of 32 bytes for each lane at most
constexpr int kMaxPairs = kMaxRowBytes / 4;
constexpr int kMaxTokens = 4;        // of a warp: a lane for each position of each axis
constexpr int kDepth = 4;            // steps of a thread's ring; 6 and 8 were 0 to 6 % slower
constexpr int kFill = 16;            // warps of an SM that there should be

// Blocks on an SM: three leave bf16 85 registers a thread (32 prompts 110 us, four 113), fp32, which holds fewer
// cosines, does with 64 (17 slab prompts 12.1 us, three blocks 13.8).
template <typename T>
constexpr int blocks_of() { return sizeof(T) == 2 ? 3 : 4; }

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
  int slices, steps, per_warp;       // warps of a token, steps of heads_at_once heads in all; tokens of a warp
  PagedPool pool;                    // paged
  const int32_t* new_start;          // paged: [batch + 1], or null: one token per sequence
};

// The sequence whose rows token t of a paged call lies behind the start of, for the whole warp together.
__device__ __forceinline__ int find_sequence(const RotaryArgs& a, int t, int lane) {
  int lo = 0, n = a.pool.batch;    // the last sequence of [lo, lo + n) that starts at or before t
  do {
    const int step = (n + 31) / 32, i = lane * step;
    const bool in = i < n;
    const int k = __popc(__ballot_sync(0xffffffffu, in && (lane == 0 || a.new_start[lo + i] <= t))) - 1;
    lo += k * step;
    n = min(step, n - k * step);
  } while (n > 1);
  return lo;
}

// Cosine and sine of a position's angle, given as turns per position (2^-64 of a turn).
__device__ __forceinline__ float2 turn_of(uint64_t per_position, int64_t position) {
  const uint64_t w = per_position * (uint64_t)position;   // modulo a turn
  const uint64_t quarter = (w + (1ull << 61)) >> 62;
  float s, c;
  sincospif((float)(int64_t)(w - (quarter << 62)) * 0x1p-63f, &s, &c);
  if (quarter & 1) {
    const float x = c;
    c = -s;
    s = x;
  }
  return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

// A 16-byte chunk as floats, and back.
__device__ __forceinline__ void unpack(const uint4& x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = bf2_to_f2(w[i]);
    f[2 * i] = y.x;
    f[2 * i + 1] = y.y;
  }
}
__device__ __forceinline__ void unpack(const uint4& x, float (&f)[4]) {
  f[0] = __uint_as_float(x.x);
  f[1] = __uint_as_float(x.y);
  f[2] = __uint_as_float(x.z);
  f[3] = __uint_as_float(x.w);
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

template <typename T, bool kPaged, bool kAdjacent>
__global__ void __launch_bounds__(kWarps * 32, blocks_of<T>()) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int E = 16 / sizeof(T);        // columns of a chunk
  __shared__ float2 s_turn[kWarps][kMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned id = blockIdx.x * kWarps + warp;
  if constexpr (kPaged) {
    if (a.new_start && a.pool.err)   // a sequence whose starts are wrong may have no token that finds it
      for (int64_t b = (int64_t)id * 32 + lane; b < a.pool.batch; b += (int64_t)gridDim.x * kWarps * 32) {
        const int first = a.new_start[b], end = a.new_start[b + 1];
        if (first < 0 || end < first || end > a.tokens) atomicOr(a.pool.err, LF_DEVERR_STATE);
      }
  }
  // Tokens t0 .. t0 + nt - 1, of each a slice of the heads.
  const unsigned group = id / (unsigned)a.slices;
  const int slice = (int)(id - group * a.slices);
  const int64_t t0 = (int64_t)group * a.per_warp;
  if (t0 >= a.tokens) return;
  const int nt = (int)min((int64_t)a.per_warp, a.tokens - t0);
  const int from = a.steps * slice / a.slices, to = a.steps * (slice + 1) / a.slices;

  // This thread's item: the chunks at bytes `one` and `two` of a row.  Lanes take chunks in a row, so that what
  // an instruction reads or writes is whole sectors.
  const int item = lane % a.items, first_head = lane / a.items;
  const int turning = a.half / E;          // items that turn
  const bool turns = item < turning;
  const int at_one = turns ? item : turning + item, at_two = at_one + (turns ? turning : a.items - turning);
  const int one = 16 * at_one, two = 16 * at_two;
  const int all = a.q.heads + a.k.heads * (kPaged ? 2 : 1);
  auto head_of = [&](int step) {           // of q, k and v in this order; -1: none
    const int h = step * a.heads_at_once + first_head;
    return first_head < a.heads_at_once && h < all ? h : -1;
  };

  // A ring of kDepth steps, of which each thread reads only what it has copied itself.  It is filled before
  // the lookups and runs on from token to token.
  extern __shared__ uint4 s_ring[];
  uint4* ring = s_ring + warp * (kDepth * 2 * 32) + lane;
  int64_t seq = 0, ti = t0;
  if (!kPaged) {
    seq = (unsigned)t0 / (unsigned)a.tokens_per_seq;
    ti = t0 - seq * a.tokens_per_seq;
  }
  struct Cursor { int64_t seq, ti; };
  auto advance = [&](Cursor& c) {
    if (++c.ti == a.tokens_per_seq) {
      c.ti = 0;
      ++c.seq;
    }
  };
  Cursor in{seq, ti};
  int next = from, next_token = 0;
  const char *qx, *kx, *vx;
  auto open = [&]() {
    qx = a.q.x + in.seq * a.q.xs + in.ti * a.q.xt;
    kx = a.k.x + in.seq * a.k.xs + in.ti * a.k.xt;
    vx = a.v + in.ti * a.k.xt;
  };
  open();
  auto issue = [&](int stage) {
    if (next_token < nt) {
      const int h = head_of(next), g = h - a.q.heads;
      if (h >= 0) {
        const char* row = h < a.q.heads ? qx + h * a.q.xh : g < a.k.heads ? kx + g * a.k.xh : vx + (g - a.k.heads) * a.k.xh;
        cp_async16(smem_u32(ring + 64 * stage), row + one, 1);
        cp_async16(smem_u32(ring + 64 * stage + 32), row + two, 1);
      }
      if (++next == to) {
        next = from;
        ++next_token;
        advance(in);
        open();
      }
    }
    cp_async_commit();   // a group per step, empty ones at the end
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) issue(i);

  // Lane j looks up where token j goes, and lane axis * nt + j what its position on an axis is.
  bool mine = true;                        // of some sequence: others are left as they are
  int64_t offset = -1;                     // of its rows in the pools, -1: not stored
  int pos = 0;
  if constexpr (kPaged) {
    int b = (int)t0 + lane, first = b, end = b + 1;
    if (a.new_start) {
      int f = 0, e = 0, bs = 0;
      for (int j = 0; j < nt; ++j) {       // tokens in a row are most often of one sequence
        const int t = (int)t0 + j;
        if (j == 0 || t < f || t >= e) {
          bs = find_sequence(a, t, lane);
          f = a.new_start[bs];
          e = a.new_start[bs + 1];
        }
        if (lane == j) {
          b = bs;
          first = f;
          end = e;
        }
      }
    }
    const int t = (int)t0 + lane;
    mine = lane < nt && first >= 0 && end >= first && end <= a.tokens && t >= first && t < end;
    if (mine) {
      const int64_t at = (int64_t)a.pool.lens[b] - end + t;
      pos = (int)at;
      bool ok = at >= 0 && at < (int64_t)a.pool.max_pages * a.pool.page_size;
      if (ok) {
        int pi, slot;
        paged_split(a.pool, pos, &pi, &slot);
        const int page = a.pool.table[(int64_t)b * a.pool.max_pages + pi];
        ok = page >= 0 && page < a.pool.num_pages;
        if (ok) offset = page * a.pool.page_stride + slot * a.pool.token_stride;
      }
      if (!ok && a.pool.err) atomicOr(a.pool.err, LF_DEVERR_STATE);
    }
  }
  if (a.positions && lane < a.axes * nt) pos = a.positions[lane / nt * a.axis_stride + t0 + lane % nt];
  for (int i0 = 0; i0 < a.half; i0 += 32) {
    const int i = i0 + lane;
    const uint64_t per_position = i < a.half ? a.turns[i] : 0;
    int ax = 0;
    if (a.positions && a.axis && i < a.half) ax = min(max(a.axis[i], 0), a.axes - 1);
    for (int j = 0; j < nt; ++j) {
      const int64_t p = __shfl_sync(0xffffffffu, pos, ax * nt + j);
      if (i < a.half) {
        float2 y = turn_of(per_position, a.inverse ? -p : p);
        y.x *= a.scale;
        y.y *= a.scale;
        s_turn[warp][j * a.half + i] = y;
      }
    }
  }
  __syncwarp();

  Cursor at{seq, ti};
  int stage = 0;
#pragma unroll 1
  for (int j = 0; j < nt; ++j) {
    float c[E], s[E];                      // of the pairs of both chunks
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = !kAdjacent ? E * item + e : e < E / 2 ? E / 2 * at_one + e : E / 2 * at_two + e - E / 2;
      const float2 y = turns ? s_turn[warp][j * a.half + i] : make_float2(1.f, 0.f);
      c[e] = y.x;
      s[e] = y.y;
    }
    const int64_t off = kPaged ? __shfl_sync(0xffffffffu, offset, j) : 0;
    const bool row = kPaged ? __shfl_sync(0xffffffffu, (int)mine, j) != 0 : true;
    char* qy = a.q.y + at.seq * a.q.ys + at.ti * a.q.yt;
    char* ky = kPaged ? a.pool.k + off : a.k.y + at.seq * a.k.ys + at.ti * a.k.yt;
    char* vy = kPaged ? a.pool.v + off : nullptr;
    const int64_t kyh = kPaged ? a.pool.head_stride : a.k.yh;
#pragma unroll 1
    for (int step = from; step < to; ++step) {
      const int h = head_of(step), g = h - a.q.heads;
      cp_async_wait<kDepth - 1>();
      uint4 x = ring[64 * stage], y = ring[64 * stage + 32];
      if (turns && g < a.k.heads) {
        float p[E], q[E], u[E], v[E];
        unpack(x, p);
        unpack(y, q);
        if constexpr (kAdjacent) {
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            u[2 * e] = p[2 * e] * c[e] - p[2 * e + 1] * s[e];
            u[2 * e + 1] = p[2 * e + 1] * c[e] + p[2 * e] * s[e];
            v[2 * e] = q[2 * e] * c[E / 2 + e] - q[2 * e + 1] * s[E / 2 + e];
            v[2 * e + 1] = q[2 * e + 1] * c[E / 2 + e] + q[2 * e] * s[E / 2 + e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            u[e] = p[e] * c[e] - q[e] * s[e];
            v[e] = q[e] * c[e] + p[e] * s[e];
          }
        }
        x = pack(u);
        y = pack(v);
      }
      if (h >= 0 && row && !(kPaged && g >= 0 && off < 0)) {
        char* out = h < a.q.heads ? qy + h * a.q.yh : g < a.k.heads ? ky + g * kyh : vy + (g - a.k.heads) * kyh;
        *reinterpret_cast<uint4*>(out + one) = x;
        *reinterpret_cast<uint4*>(out + two) = y;
      }
      issue(stage);
      stage = stage + 1 == kDepth ? 0 : stage + 1;
    }
    advance(at);
  }
}

template <typename T, bool kPaged>
cudaError_t launch(const RotaryArgs& a, int adjacent, cudaStream_t stream) {
  constexpr int kSmem = kWarps * kDepth * 2 * 32 * 16;
  const int64_t warps = (a.tokens + a.per_warp - 1) / a.per_warp * a.slices;
  const unsigned grid = (unsigned)((warps + kWarps - 1) / kWarps);
  auto* kernel = adjacent ? &rotary_kernel<T, kPaged, true> : &rotary_kernel<T, kPaged, false>;
  static std::atomic<uint64_t> done[2];
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kSmem, done[adjacent]);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kWarps * 32, kSmem, stream>>>(a);
  return cudaGetLastError();
}

// Everything that does not depend on where the rows lie.
int take_rotary(const lf_rotary* r, int row_dim, int elem, const int32_t* positions, int64_t axis_stride, RotaryArgs* a) {
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
  a->items = row_dim * elem / 32;
  a->heads_at_once = 32 / a->items;
  a->pool = PagedPool{};
  a->new_start = nullptr;
  return LF_OK;
}

// Rows of lf_rotate; `rows` may be null for none.
int rows_to_turn(const lf_rows* rows, const char* name, int elem, RotaryRows* out) {
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

// What a call writes, and all that it reads: rows are read a few steps ahead of the writes (the ring), so that an output
// may be its own input and otherwise shares no memory with what is read or written.  A layout whose rows lie in each
// other in no order of strides, and would take long to tell apart, counts as one that does.
int apart(const RotaryArgs& a, int seqs, int tokens, int64_t row_bytes) {
  const RotaryRows* rows[2] = {&a.q, &a.k};
  static const char* const names[2] = {"q", "k"};
  auto in = [&](const RotaryRows& r) {
    return RowSet{reinterpret_cast<uintptr_t>(r.x), {seqs, tokens, r.heads}, {r.xs, r.xt, r.xh}, row_bytes};
  };
  auto out = [&](const RotaryRows& r) {
    return RowSet{reinterpret_cast<uintptr_t>(r.y), {seqs, tokens, r.heads}, {r.ys, r.yt, r.yh}, row_bytes};
  };
  for (int i = 0; i < 2; ++i) {
    if (rows[i]->heads == 0) continue;
    const RowSet y = out(*rows[i]);
    if (rows_overlap_themselves(y) != Overlap::kNo)
      return fail(LF_ERR_ARG, "%s: rows of y overlap one another", names[i]);
    for (int j = 0; j < 2; ++j) {
      if (rows[j]->heads == 0) continue;
      const RowSet x = in(*rows[j]);
      if (rows_overlap(y, x) != Overlap::kNo && !(i == j && same_rows(y, x)))
        return fail(LF_ERR_ARG, "%s: y overlaps %s's x, and is not the same rows", names[i], names[j]);
    }
  }
  if (a.k.heads > 0 && rows_overlap(out(a.q), out(a.k)) != Overlap::kNo)
    return fail(LF_ERR_ARG, "k: y overlaps q's y");
  return LF_OK;
}

// How many warps a token gets, or how many tokens a warp: enough warps to fill the GPU, and then, where a token has
// few steps, several tokens that look things up together (17 slab prompts of 1000 fp32 tokens, two steps each: four
// tokens 12.1 us, one 14.2; two video prompts of 6000, eight steps: two tokens 37.5, one 37.9).
int take_slices(RotaryArgs* a, int heads) {
  int sms = 0;
  const int rc = sm_count(&sms);
  if (rc != LF_OK) return rc;
  const int64_t warps = (int64_t)sms * kFill;
  a->steps = (heads + a->heads_at_once - 1) / a->heads_at_once;
  const int64_t want = (warps + a->tokens - 1) / a->tokens;
  a->slices = (int)(want < a->steps ? want : a->steps);
  a->per_warp = 1;
  while (a->slices == 1 && 2 * a->per_warp <= kMaxTokens && 2 * a->per_warp * a->steps <= 16 &&
         2 * a->per_warp * a->half <= kMaxPairs && a->tokens >= warps * 2 * a->per_warp)
    a->per_warp *= 2;
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
  static const uint32_t kInverse[6] = {0x4f10e410u, 0x36d8a566u, 0x7d4d3770u, 0x7f09d5f4u, 0x9391054au, 0x28be60dbu};
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
  const int elem = dtype == LF_BF16 ? 2 : 4;
  if (row_dim < 16 || row_dim % 16 != 0 || row_dim * (int64_t)elem > lf::kMaxRowBytes)
    return fail(LF_ERR_ARG, "row_dim (%d) must be a multiple of 16 in [16, %d]", row_dim, lf::kMaxRowBytes / elem);
  lf::RotaryArgs a;
  int rc = lf::take_rotary(rotary, row_dim, elem, positions, axis_stride, &a);
  if (rc != LF_OK) return rc;
  if (seqs < 0 || tokens < 0 || (int64_t)seqs * tokens > INT_MAX)
    return fail(LF_ERR_ARG, "need seqs, tokens >= 0 and seqs * tokens below 2^31");
  if (inverse != 0 && inverse != 1) return fail(LF_ERR_ARG, "inverse must be 0 or 1");
  if (!q) return fail(LF_ERR_ARG, "null q");
  if (seqs == 0 || tokens == 0) return LF_OK;
  if ((rc = lf::rows_to_turn(q, "q", elem, &a.q)) != LF_OK || (rc = lf::rows_to_turn(k, "k", elem, &a.k)) != LF_OK) return rc;
  if (!positions) return fail(LF_ERR_ARG, "null positions");
  if ((rc = lf::apart(a, seqs, tokens, (int64_t)row_dim * elem)) != LF_OK) return rc;
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
  if (rc != LF_OK || (rc = lf::take_rotary(rotary, pages->head_dim, lf::elem_bytes(pages), positions, axis_stride, &a)) != LF_OK) return rc;
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
  if (q) {
    const uintptr_t y = reinterpret_cast<uintptr_t>(q_out);
    const uint64_t y_bytes = (uint64_t)row * q_heads * total_new, k_bytes = (uint64_t)row * pages->kv_heads * total_new;
    auto overlaps = [&](const void* x, uint64_t bytes) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(x);
      return at < y + y_bytes && y < at + bytes;
    };
    if ((q != q_out && overlaps(q, y_bytes)) || overlaps(k_new, k_bytes) || overlaps(v_new, k_bytes))
      return fail(LF_ERR_ARG, "q_out may be q, and overlaps neither a part of it nor k_new and v_new");
  }
  if ((rc = lf::take_slices(&a, a.q.heads + 2 * a.k.heads)) != LF_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = pages->dtype == LF_BF16 ? lf::launch<__nv_bfloat16, true>(a, rotary->adjacent, st)
                                                : lf::launch<float, true>(a, rotary->adjacent, st);
  return e == cudaSuccess ? LF_OK : cuda_fail(e, "paged append launch");
}

}  // extern "C"
