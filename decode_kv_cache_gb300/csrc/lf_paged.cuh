// Device pieces that the paged kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

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

// A finished row's log-sum-exp, and the error word if its sum is not finite (Args: of decode or prompt).
template <class Args>
__device__ __forceinline__ void write_row_stats(const Args& a, int64_t row, float m, float l) {
  if (a.lse) a.lse[row] = l == 0.f ? kNegInf : (m + log2f(l)) * 0.6931471805599453f;
  if (a.pool.err && !(l <= 3.0e38f)) atomicOr(a.pool.err, LF_DEVERR_NONFINITE);
}

// A piece of work: rows r0 .. of `rows` of a sequence's queries, and what they see.
struct Piece {
  int b, g, q0, first_pos, p_lo, p_hi;
  int64_t r0, rows, id;
};

// With numbers that follow the rows (tiles_per_seq = 0): sequence b's first one.  Starts
// outside the rows count as their ends, so that other sequences keep their numbers.
__device__ __forceinline__ unsigned first_number(const PagedPromptArgs& a, int b, int start) {
  return ((unsigned)min(max(start, 0), a.total_q) >> a.piece_shift) + (unsigned)b;
}

// The sequence that piece number `id` belongs to, and which of its numbers that is (where they
// follow the rows), for the whole warp together.
//
// Up to 32 sequences have a lane each, and their pieces are numbered in the order of their
// lengths, the longest first and without gaps: a lane adds up the pieces before its own.
// (24 sequences, chunks of 1 to 512 behind up to 2048, 32 / 8 heads of 128, bf16: 132 us, in the
// sequences' own order 139; 8 such sequences 54, 69; one prompt of 8192 behind single
// tokens 532, 517.)  Of more sequences the lanes look at 32 at a time for the last one that
// starts at or before the number.
__device__ __forceinline__ int locate(const PagedPromptArgs& a, unsigned id, int* number) {
  const unsigned j = id / (unsigned)a.pool.kv_heads;
  *number = 0;
  if (a.tiles_per_seq > 0) return (int)(j % (unsigned)a.pool.batch);
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.pool.batch;
  if (n <= 32) {
    int len = -1;
    unsigned pieces = 0, before = 0;
    if (lane < n) {
      const int q0 = min(max(a.q_start[lane], 0), a.total_q), q1 = min(max(a.q_start[lane + 1], 0), a.total_q);
      len = a.pool.lens[lane];
      pieces = (unsigned)(max(q1 - q0, 0) + (1 << a.piece_shift) - 1) >> a.piece_shift;
    }
#pragma unroll 4
    for (int c = 0; c < n; ++c) {
      const int len_c = __shfl_sync(0xffffffffu, len, c);
      const unsigned pieces_c = __shfl_sync(0xffffffffu, pieces, c);
      if (len_c > len || (len_c == len && c < lane)) before += pieces_c;
    }
    const unsigned m = __ballot_sync(0xffffffffu, lane < n && j >= before && j - before < pieces);
    lo = m ? __ffs(m) - 1 : 0;
    *number = __shfl_sync(0xffffffffu, m ? (int)(j - before) : INT_MAX, lo);   // none: behind its rows
    return __shfl_sync(0xffffffffu, lo, 0);   // uniform for the compiler too
  }
  do {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const bool in = lane * step < n;
    // (starts that decrease may give any lane, but one that is `in`)
    const int k =
        __popc(__ballot_sync(0xffffffffu, in && (lane == 0 || first_number(a, i, a.q_start[i]) <= j))) - 1;
    lo += k * step;
    n = min(step, n - k * step);
  } while (n > 1);
  *number = (int)(j - first_number(a, lo, a.q_start[lo]));
  return __shfl_sync(0xffffffffu, lo, 0);
}

// Is something wrong with a sequence's rows or its length?
__device__ __forceinline__ bool wrong_sequence(const PagedPromptArgs& a, int b, int q0, int n) {
  const int len = paged_len(a.pool, b);
  return q0 < 0 || n < 0 || n > a.total_q - q0 || n > a.max_q || len != a.pool.lens[b] || n > len;
}

// Rows from piece `tile` of a sequence on, and what they see; false: it has none.
__device__ __forceinline__ bool take_rows(const PagedPromptArgs& a, int tile, int per_piece, int n, Piece* p) {
  const int len = paged_len(a.pool, p->b);
  p->r0 = (int64_t)tile * per_piece;
  p->rows = (int64_t)n * a.group;
  if (n > a.max_q) p->rows = (int64_t)a.max_q * a.group;   // the rest is left
  if (p->r0 >= p->rows) return false;
  p->first_pos = len - n;      // may be negative: those rows see nothing
  p->p_lo = p->first_pos + (int)(p->r0 / a.group);
  p->p_hi = p->first_pos + (int)((min(p->r0 + per_piece, p->rows) - 1) / a.group);
  return true;
}

// Piece number `id`, which is sequence b's and its `number` (locate); false: it has no rows.  The last
// rows, which see the most keys, come first.  `tell`: this thread reports what is wrong with
// sequence `id`, of the first `batch` blocks.
__device__ __forceinline__ bool take_piece(const PagedPromptArgs& a, unsigned id, int b, int number, int per_piece,
                                           bool tell, Piece* p) {
  if (tell && (int)id < a.pool.batch && a.pool.err) {
    const int q0 = a.q_start[id];
    if (wrong_sequence(a, (int)id, q0, a.q_start[id + 1] - q0)) atomicOr(a.pool.err, LF_DEVERR_STATE);
  }
  p->id = id;
  p->b = b;
  p->g = (int)(id % (unsigned)a.pool.kv_heads);
  p->q0 = a.q_start[b];
  const int n = a.q_start[b + 1] - p->q0;
  if (p->q0 < 0 || n < 0 || n > a.total_q - p->q0) return false;   // not rows of q
  const unsigned j = id / (unsigned)a.pool.kv_heads;
  int tile;
  if (a.tiles_per_seq > 0) {
    tile = a.tiles_per_seq - 1 - (int)(j / (unsigned)a.pool.batch);
  } else {
    tile = (int)(((int64_t)n * a.group + per_piece - 1) / per_piece) - 1 - number;
    if (tile < 0 || (int64_t)tile * per_piece >= (int64_t)a.max_q * a.group) return false;
  }
  return take_rows(a, tile, per_piece, n, p);
}

// The same where every sequence has as many numbers (tiles_per_seq > 0), for the fp32 kernel,
// which the search before its loop makes slower (8 heads of 64, one prompt of 2000 tokens: 135 us,
// with it 143; 24 prompts of 1 to 200: 29, 35).
__device__ __forceinline__ bool take_piece_level(const PagedPromptArgs& a, int head, int tile, int per_piece, bool tell,
                                                 Piece* p) {
  p->id = (int64_t)(a.tiles_per_seq - 1 - tile) * a.pool.batch * a.pool.kv_heads + head;
  p->b = head / a.pool.kv_heads;
  p->g = head - p->b * a.pool.kv_heads;
  p->q0 = a.q_start[p->b];
  const int n = a.q_start[p->b + 1] - p->q0;
  if (tell && tile == 0 && p->g == 0 && a.pool.err && wrong_sequence(a, p->b, p->q0, n))
    atomicOr(a.pool.err, LF_DEVERR_STATE);
  if (p->q0 < 0 || n < 0 || n > a.total_q - p->q0) return false;   // not rows of q
  return take_rows(a, tile, per_piece, n, p);
}

// Row r (of the sequence's token and head pairs) as a row of q and out.
__device__ __forceinline__ int64_t row_of(const PagedPromptArgs& a, const Piece& p, int64_t r) {
  return (p.q0 + r / a.group) * a.q_heads + p.g * a.group + r % a.group;
}

// Positions `sinks` .. this - 1 lie behind the window of every query from p_lo on: nothing there
// reaches an output, and the caller may have given the pages back.
__device__ __forceinline__ int behind_window(const PagedPromptArgs& a, int p_lo) {
  return a.window > 0 ? max(p_lo, 0) - a.window + 1 : 0;
}

// Byte offset in the pools of the piece's position `pos`, -1: nothing to read.  kSkip: nor where no
// row of the piece sees it (from `sinks` to behind() - 1), for the kernel that would find what is not
// finite there; others ask only before they report an entry that is no page.
template <bool kSkip, class Behind>
__device__ __forceinline__ int64_t offset_of(const PagedPromptArgs& a, const Piece& p, int pos, Behind behind) {
  if (pos > p.p_hi) return -1;
  int pi, slot;
  paged_split(a.pool, pos, &pi, &slot);
  const int page = a.pool.table[(int64_t)p.b * a.pool.max_pages + pi];
  auto unseen = [&] { return pos >= a.sinks && pos < behind(); };
  if (page >= 0 && page < a.pool.num_pages && !(kSkip && unseen()))
    return page * a.pool.page_stride + slot * a.pool.token_stride + p.g * a.pool.head_stride;
  if (a.pool.err && !unseen()) atomicOr(a.pool.err, LF_DEVERR_STATE);
  return -1;
}

__device__ __forceinline__ bool sees(const PagedPromptArgs& a, int pos, int key) {
  return key <= pos && (a.window == 0 || key > pos - a.window || key < a.sinks);
}

// The key tiles of `size` tokens that queries at positions p_lo .. p_hi visit: [0, sink)
// and [from, to); with splits, a block takes its share of them.
struct Tiles {
  int sink, gap, first, last;   // tile j of them is number j below `sink`, else j + gap
  __device__ Tiles(const PagedPromptArgs& a, int p_lo, int p_hi, int size, int share)
      : sink(0), gap(0), first(0), last(0) {
    if (p_hi < 0) return;
    last = p_hi / size + 1;
    if (a.window > 0) {
      const int from = (int)max((int64_t)0, (int64_t)p_lo - a.window + 1) / size;
      sink = min((int)(((int64_t)a.sinks + size - 1) / size), from);
      gap = from - sink;
      last -= gap;
    }
    if (a.splits > 1) {   // this block's share
      const unsigned n = last;
      first = n * (unsigned)share / (unsigned)a.splits;
      last = n * (unsigned)(share + 1) / (unsigned)a.splits;
    }
  }
  __device__ int count() const { return last - first; }
  __device__ int at(int j) const { return first + j < sink ? first + j : first + j + gap; }
};

// Does some query at positions p_lo .. p_hi not see some of the `size` keys from k0 on?
__device__ __forceinline__ bool some_hidden(const PagedPromptArgs& a, int p_lo, int p_hi, int k0, int size) {
  return k0 + size - 1 > p_lo ||
         (a.window > 0 && k0 + size > a.sinks && (int64_t)k0 <= (int64_t)p_hi - a.window);
}

// Where a block puts row rr of its piece when its keys are a share of the row's.
template <int D>
__device__ __forceinline__ float* part_row(const PagedPromptArgs& a, int64_t id, int share, int per_piece, int rr,
                                           float m, float l, bool write_ml) {
  const int64_t i = (id * a.splits + share) * per_piece + rr;
  if (write_ml) {
    a.part_ml[2 * i] = m;
    a.part_ml[2 * i + 1] = l;
  }
  return a.part_o + i * D;
}

// Row rr of a piece by the definition, a warp at a time: for blocks whose tiles held
// values that are not finite where some row does not look (0 * NaN is NaN).
template <typename T, int D>
__device__ __forceinline__ void row_by_hand(const PagedPromptArgs& a, const Piece& p, const Tiles& tiles, int share,
                                            int size, int per_piece, int rr, int lane) {
  constexpr int E = D >= 32 ? D / 32 : 1;
  const bool mine = lane * E < D;   // lanes past a short row take nothing
  const int64_t row = row_of(a, p, p.r0 + rr);
  const int pos = p.first_pos + (int)((p.r0 + rr) / a.group);
  const T* q = reinterpret_cast<const T*>(a.q) + row * D + lane * E;
  float qv[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = mine ? to_f32(q[e]) : 0.f;
    acc[e] = 0.f;
  }
  float m = kNegInf, l = 0.f;
  const int n = tiles.count();
  for (int j = 0; j < n; ++j) {
    const int k0 = tiles.at(j) * size;
    for (int key = k0; key < k0 + size; ++key) {
      if (!sees(a, pos, key)) continue;
      const int64_t off = offset_of<false>(a, p, key, [] { return 0; });
      if (off < 0) continue;
      const T* k = reinterpret_cast<const T*>(a.pool.k + off) + lane * E;
      const T* v = reinterpret_cast<const T*>(a.pool.v + off) + lane * E;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (mine) s = fmaf(qv[e], to_f32(k[e]), s);
      s = warp_sum(s);
      const float mn = fmaxf(m, s * a.scale_log2), mu = mn == kNegInf ? 0.f : mn;
      const float f = ex2(m - mu), w = ex2(fmaf(s, a.scale_log2, -mu));
      m = mn;
      l = l * f + w;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (mine) acc[e] = acc[e] * f + w * to_f32(v[e]);
    }
  }
  if (a.splits > 1) {
    float* o = part_row<D>(a, p.id, share, per_piece, rr, m, l, lane == 0) + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (mine) o[e] = acc[e];
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = reinterpret_cast<T*>(a.out) + row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (mine) from_f32(l == 0.f ? 0.f : acc[e] * inv, out + e);
  if (lane == 0) write_row_stats(a, row, m, l);
}

// Rows rr .. rr + n - 1 of a piece, for the whole warp together.  What describes it is
// worked out again, so that the usual path keeps none of it in registers for this one.  (A call here
// instead of its code slows the tensor-core kernel: 8192 tokens, 32 / 8 heads, 354 -> 414 us.)
template <typename T, int D>
__device__ __forceinline__ void rows_by_hand(const PagedPromptArgs& a, unsigned id, int share, int size, int per_piece,
                                          int rr, int n, int lane) {
  Piece p;
  int number;
  const int b = locate(a, id, &number);
  if (!take_piece(a, id, b, number, per_piece, false, &p)) return;
  const Tiles tiles(a, p.p_lo, p.p_hi, size, share);
  for (int i = rr; i < rr + n && p.r0 + i < p.rows; ++i)
    row_by_hand<T, D>(a, p, tiles, share, size, per_piece, i, lane);
}

}  // namespace lf
