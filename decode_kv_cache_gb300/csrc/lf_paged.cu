// C ABI of the paged key-value cache (declarations and semantics:
// include/longflow.h) and the append kernel.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "lf_device.cuh"
#include "lf_kernels.h"
#include "lf_paged.h"
#include "lf_paged_host.h"
#include "longflow.h"

namespace lf {

namespace {

// ---- append -----------------------------------------------------------------
//
// K[page(b, p)][g][slot(p)] = k_new[i], and V alike, for every token i of the
// call: a scatter of rows, one read and one write of each.  Bound by HBM.  A
// block takes `tokens_per_block` consecutive tokens: one warp's lanes look up
// where each goes (sequence by a search of new_start, page, slot), then all
// threads copy 16-byte chunks, K and V of the same chunk together, four chunks
// of each in flight per thread (also of tokens that are not stored: the loads do not
// wait for the lookup).  Tokens find their sequence by starts in order, and one whose
// starts are wrong may have no token that finds it, so that the first threads of the
// grid look at the sequences themselves.  (8 x 128 bf16: 32 prompts, 324 MB moved, 53.5 us, 6.05 TB/s,
// 90 % of a plain copy's rate; one token of 64 sequences 5 us on the device.)

constexpr int kAppendThreads = 256;
constexpr int kAppendMaxTokens = 32;

// Are a sequence's rows not rows of the call?
__device__ __forceinline__ bool wrong_starts(const PagedAppendArgs& a, int first, int end) {
  return first < 0 || end < first || end > a.total_new;
}

__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
  __shared__ int64_t dst[kAppendMaxTokens];  // byte offset of the token's rows, -1: not stored
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * a.tokens_per_block;
  const int nt = min(a.tokens_per_block, a.total_new - t0);
  if (tid < nt) {
    const int t = t0 + tid;
    int b = t, first = t, n = 1;
    bool mine = true;
    if (a.new_start) {
      int lo = 0, hi = a.pool.batch;  // the last b with new_start[b] <= t
      while (lo + 1 < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.new_start[mid] <= t) lo = mid;
        else hi = mid;
      }
      b = lo;
      first = a.new_start[b];
      const int end = a.new_start[b + 1];
      // rows behind the last sequence belong to none, and those of wrong starts are left out
      mine = !wrong_starts(a, first, end) && t >= first && t < end;
      n = mine ? end - first : 0;
    }
    int64_t off = -1;
    if (mine) {
      const int64_t pos = (int64_t)a.pool.lens[b] - n + (t - first);
      bool ok = pos >= 0 && pos < (int64_t)a.pool.max_pages * a.pool.page_size;
      if (ok) {
        int pi, slot;
        paged_split(a.pool, (int)pos, &pi, &slot);
        const int page = a.pool.table[(int64_t)b * a.pool.max_pages + pi];
        ok = page >= 0 && page < a.pool.num_pages;
        off = page * a.pool.page_stride + slot * a.pool.token_stride;
      }
      if (!ok) {
        off = -1;
        if (a.pool.err) atomicOr(a.pool.err, LF_DEVERR_STATE);
      }
    }
    dst[tid] = off;
  }
  if (a.new_start && a.pool.err)
    for (int64_t b = (int64_t)blockIdx.x * kAppendThreads + tid; b < a.pool.batch; b += (int64_t)gridDim.x * kAppendThreads)
      if (wrong_starts(a, a.new_start[b], a.new_start[b + 1])) atomicOr(a.pool.err, LF_DEVERR_STATE);
  __syncthreads();
  const unsigned per_head = (unsigned)a.row_bytes >> 4;
  const unsigned per_token = per_head * a.pool.kv_heads;
  const unsigned total = per_token * nt;
  const char* ks = a.k_new + (int64_t)t0 * per_token * 16;
  const char* vs = a.v_new + (int64_t)t0 * per_token * 16;
  constexpr int U = 4;
  for (unsigned i0 = tid; i0 < total; i0 += U * kAppendThreads) {
    uint4 kx[U], vx[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned i = i0 + u * kAppendThreads;
      if (i < total) {
        kx[u] = __ldcs(reinterpret_cast<const uint4*>(ks) + i);
        vx[u] = __ldcs(reinterpret_cast<const uint4*>(vs) + i);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned i = i0 + u * kAppendThreads;
      if (i < total) {
        const unsigned tl = i / per_token, c = i - tl * per_token;
        const unsigned g = c / per_head, ch = c - g * per_head;
        const int64_t off = dst[tl];
        if (off >= 0) {
          const int64_t o = off + g * a.pool.head_stride + ch * 16;
          *reinterpret_cast<uint4*>(a.pool.k + o) = kx[u];
          *reinterpret_cast<uint4*>(a.pool.v + o) = vx[u];
        }
      }
    }
  }
}

// ---- the error word ------------------------------------------------------------
//
// Read and cleared in one step: bits that another stream sets meanwhile stay or are taken,
// but are not lost.  One thread; bound by its launch.
__global__ void paged_take_errors_kernel(int32_t* err, int32_t* taken) { *taken = atomicExch(err, 0); }

}  // namespace

cudaError_t paged_take_errors_launch(int32_t* err, int32_t* taken, cudaStream_t stream) {
  paged_take_errors_kernel<<<1, 1, 0, stream>>>(err, taken);
  return cudaGetLastError();
}

cudaError_t paged_append_launch(const PagedAppendArgs& a, cudaStream_t stream) {
  const int blocks = (int)(((int64_t)a.total_new + a.tokens_per_block - 1) / a.tokens_per_block);
  paged_append_kernel<<<blocks, kAppendThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace lf

// ---- checks that the paged entry points share (lf_paged_host.h) ----------------

namespace lf {

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(code, buf);
  return code;
}

int cuda_fail(cudaError_t e, const char* what) {
  (void)cudaGetLastError();
  return fail(e == cudaErrorMemoryAllocation ? LF_ERR_OOM : LF_ERR_CUDA, "%s: %s", what,
              cudaGetErrorString(e));
}

// The pools, the page table and the lengths of a call, checked, as the kernels take them.
int take_pool(const lf_pages* p, int batch, const int32_t* table, int max_pages,
              const int32_t* lens, PagedPool* out) {
  if (!p) return fail(LF_ERR_ARG, "null pages");
  if (p->dtype != LF_BF16 && p->dtype != LF_F32)
    return fail(LF_ERR_ARG, "dtype must be LF_BF16 or LF_F32");
  if (p->head_dim != 16 && p->head_dim != 32 && p->head_dim != 64 && p->head_dim != 128)
    return fail(LF_ERR_UNSUPPORTED, "no paged kernel for head_dim %d (built: 16/32/64/128)",
                p->head_dim);
  if (p->kv_heads < 1 || p->kv_heads > 65535 || p->page_size < 1 || p->num_pages < 1)
    return fail(LF_ERR_ARG, "kv_heads must be in [1, 65535], page_size and num_pages >= 1");
  if (!p->k || !p->v || !aligned16(p->k) || !aligned16(p->v))
    return fail(LF_ERR_ARG, "the K and V pools must be non-null and 16-byte aligned");
  const int e = elem_bytes(p);
  const int64_t strides[3] = {p->page_stride, p->head_stride, p->token_stride};
  for (int64_t s : strides)
    if (s < 0 || s > (int64_t)1 << 40 || (s * e) % 16 != 0)
      return fail(LF_ERR_ARG, "page, head and token strides must be >= 0, at most 2^40 elements "
                  "and whole multiples of 16 bytes");
  if (batch < 1 || batch > 65535) return fail(LF_ERR_ARG, "batch must be in [1, 65535]");
  if ((int64_t)batch * p->kv_heads > INT_MAX)
    return fail(LF_ERR_ARG, "batch * kv_heads must be below 2^31");
  if (max_pages < 1 || (int64_t)max_pages * p->page_size > INT_MAX - 256)
    return fail(LF_ERR_ARG, "max_pages must be >= 1 and max_pages * page_size below 2^31 - 256");
  if (!table || !lens) return fail(LF_ERR_ARG, "null page_table or lens");
  if (!aligned4(table) || !aligned4(lens) || !aligned4(p->err))
    return fail(LF_ERR_ARG, "page_table, lens and the error word must be 4-byte aligned");
  out->k = static_cast<char*>(p->k);
  out->v = static_cast<char*>(p->v);
  out->page_stride = p->page_stride * e;
  out->head_stride = p->head_stride * e;
  out->token_stride = p->token_stride * e;
  out->page_size = p->page_size;
  out->page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (p->page_size == 1 << s) out->page_shift = s;
  out->num_pages = p->num_pages;
  out->kv_heads = p->kv_heads;
  out->table = table;
  out->lens = lens;
  out->batch = batch;
  out->max_pages = max_pages;
  out->err = p->err;
  return LF_OK;
}

int take_heads(const lf_pages* p, int q_heads, int* group) {
  if (q_heads < 1 || q_heads % p->kv_heads != 0)
    return fail(LF_ERR_ARG, "q_heads (%d) must be a multiple of kv_heads (%d)", q_heads,
                p->kv_heads);
  *group = q_heads / p->kv_heads;
  if (*group != 1 && *group != 2 && *group != 4 && *group != 8)
    return fail(LF_ERR_UNSUPPORTED, "no paged kernel for group size %d (built: 1/2/4/8)", *group);
  return LF_OK;
}

// Streaming multiprocessors of the current device.
int sm_count(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? LF_OK : cuda_fail(e, "device attributes");
}

}  // namespace lf

// ---- C ABI --------------------------------------------------------------------

namespace {

using lf::aligned16;
using lf::aligned4;
using lf::cuda_fail;
using lf::elem_bytes;
using lf::fail;
using lf::sm_count;
using lf::take_heads;
using lf::take_pool;

// The window as the kernels take it: one that covers every position a table can
// hold is none.
int take_window(const lf::PagedPool& p, int window, int sinks, int* w, int* s) {
  if (window < 0 || sinks < 0) return fail(LF_ERR_ARG, "window and sinks must be >= 0");
  if (sinks > 0 && window == 0)
    return fail(LF_ERR_ARG, "sinks need a window: without one every position is seen");
  const bool all = (int64_t)window + sinks >= (int64_t)p.max_pages * p.page_size;
  *w = all ? 0 : window;
  *s = all ? 0 : sinks;
  return LF_OK;
}

// The rows of a prompt call; their pieces, of 32 rows or more, fit a grid.
int take_rows(const lf::PagedPool& p, int group, int total_q, int max_q) {
  if (total_q < 0 || max_q < 0 || max_q > total_q) return fail(LF_ERR_ARG, "need 0 <= max_q <= total_q");
  int tiles;
  if (lf::paged_prompt_pieces(p, group, total_q, max_q, 32, false, &tiles) > INT_MAX)
    return fail(LF_ERR_ARG, "max_q * group / 32 * batch * kv_heads must be below 2^31");
  return LF_OK;
}

// How a decode call is spread over the GPU, and its workspace: the parts that
// its CTAs leave to be joined (outputs, maxima and sums, units), each piece
// 256-byte aligned.
struct DecodeShape {
  int whole_units, grid;
  size_t off_ml, off_unit, bytes;
};

// Either a CTA takes a whole unit (one sequence's KV head) and no second launch is needed,
// or every SM takes an equal range of all units' tokens and the units that were cut are
// joined.  A range costs its share of the work and the join, a whole unit all of its own
// tokens: the SMs that units leave idle cost a whole unit's time times (sms - units) / sms,
// and that may be four sweeps of a CTA's warps, about what the join costs.  Nearly as many
// units as SMs could be as long as they like if they were equally long; twelve sweeps where
// they are a quarter to all of it.  (bf16, 32 / 8 heads of 128, whole against cut, a sweep
// being 128 tokens: 8 units of 4 sweeps 10.0 us, 10.6, of 8 sweeps 14.9, 11.3; 64 units of
// 4 sweeps 11.2, 14.4, of 8 sweeps 15.7, 17.2, of 16 sweeps 25.3, 21.9; 136 units of 8
// sweeps 18.5, 23.7, of 16 sweeps 30.1, 35.3, but ragged 27.7, 30.1, of 32 sweeps ragged
// 44.8, 41.7.  Heads of 64 and fp32 cross over at the same numbers of sweeps.)  The bounds are on
// the careful side: 64 units of 8 sweeps and 136 of 16 are cut, though whole ones were faster.
// Lengths are known here by the table's width: short sequences under a wide table are cut too (one of
// 300 tokens under 8192 pages 10.3 us, 8.3 under its own 19; 17 fp32 ones of 1000 16.5, 13.6).
// Behind a prefix the table's width says nothing of what is left: ranges, and the join takes them as they are.
int decode_shape(const lf_pages* p, const lf::PagedPool& pool, int group, int window, int sinks,
                 DecodeShape* s, bool behind = false) {
  const int64_t most = window > 0 ? (int64_t)window + sinks : (int64_t)pool.max_pages * pool.page_size;
  const int64_t units = (int64_t)pool.batch * pool.kv_heads;
  int sms = 0;
  const int rc = sm_count(&sms);
  if (rc != LF_OK) return rc;
  const int64_t sweep = lf::paged_decode_sweep(elem_bytes(p), p->head_dim);
  s->whole_units = !behind && units <= sms && most * (sms - units) <= 4 * sms * sweep && most <= 12 * sweep;
  s->grid = s->whole_units ? (int)units : sms;
  s->off_ml = s->off_unit = s->bytes = 0;
  if (s->whole_units) return LF_OK;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  s->off_ml = up((size_t)s->grid * 2 * group * p->head_dim * 4);
  s->off_unit = s->off_ml + up((size_t)s->grid * 2 * group * 2 * 4);
  s->bytes = s->off_unit + up((size_t)s->grid * 4);
  return LF_OK;
}

// A call behind shared prefixes: the rest's shape, the prefixes' plan, and the workspace, each piece 256-byte aligned.
struct SharedShape {
  DecodeShape rest;
  lf::SharedPlan plan;
  size_t off_rest_o, off_rest_ml, off_part_o, off_part_ml, off_segments, off_first, off_ranges, off_seen, bytes;
};

int shared_shape(const lf_pages* p, const lf::PagedPool& pool, int group, int groups, SharedShape* s) {
  if (groups < 1 || groups > pool.batch) return fail(LF_ERR_ARG, "groups must be in [1, batch]");
  int sms = 0;
  int rc = sm_count(&sms);
  if (rc != LF_OK || (rc = decode_shape(p, pool, group, 0, 0, &s->rest, true)) != LF_OK) return rc;
  s->plan = lf::paged_shared_plan(pool, elem_bytes(p), p->head_dim, group, groups, sms);
  if (!s->plan.fits) return fail(LF_ERR_ARG, "batch * kv_heads * max_pages * page_size is too large for one call");
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = (size_t)pool.batch * pool.kv_heads * group, d = p->head_dim;
  s->off_rest_o = up(s->rest.bytes);
  s->off_rest_ml = s->off_rest_o + up(rows * d * 4);
  s->off_part_o = s->off_rest_ml + up(rows * 2 * 4);
  s->off_part_ml = s->off_part_o + up((size_t)s->plan.part_rows * d * 4);
  s->off_segments = s->off_part_ml + up((size_t)s->plan.part_rows * 2 * 4);
  s->off_first = s->off_segments + up((size_t)groups * 4);
  s->off_ranges = s->off_first + up((size_t)groups * 8);
  s->off_seen = s->off_ranges + up(3 * 4);
  const size_t sets = groups > s->plan.table ? 1 : s->plan.kernel == lf::PromptPlan::kTensor ? s->rest.grid : 0;
  s->bytes = s->off_seen + up(sets * groups * 4);
  return LF_OK;
}

}  // namespace

extern "C" {

int lf_paged_append(const lf_pages* pages, int batch, const int32_t* page_table, int max_pages,
                    const int32_t* lens, const void* k_new, const void* v_new,
                    const int32_t* new_start, int total_new, lf_stream_t stream) {
  lf::clear_last_error();
  lf::PagedAppendArgs a;
  int rc = take_pool(pages, batch, page_table, max_pages, lens, &a.pool);
  if (rc != LF_OK) return rc;
  if (total_new < 0) return fail(LF_ERR_ARG, "total_new < 0");
  if (!new_start && total_new != batch)
    return fail(LF_ERR_ARG, "without new_start every sequence takes one token: total_new (%d) must "
                "be the batch (%d)", total_new, batch);
  if (total_new == 0) return LF_OK;
  if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new))
    return fail(LF_ERR_ARG, "k_new and v_new must be non-null and 16-byte aligned");
  if (!aligned4(new_start)) return fail(LF_ERR_ARG, "new_start must be 4-byte aligned");
  a.k_new = static_cast<const char*>(k_new);
  a.v_new = static_cast<const char*>(v_new);
  a.new_start = new_start;
  a.total_new = total_new;
  a.row_bytes = pages->head_dim * elem_bytes(pages);
  a.tokens_per_block = 8;
  const cudaError_t e = lf::paged_append_launch(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LF_OK : cuda_fail(e, "paged append launch");
}

int lf_paged_decode_workspace(const lf_pages* pages, int batch, int max_pages, int q_heads,
                              int window, int sinks, size_t* bytes) {
  lf::clear_last_error();
  if (!pages || !bytes) return fail(LF_ERR_ARG, "null pages or bytes");
  lf::PagedPool pool;
  static const int32_t any = 0;  // only the shape counts here
  int group = 0;
  DecodeShape shape;
  int rc = take_pool(pages, batch, &any, max_pages, &any, &pool);
  if (rc != LF_OK || (rc = take_heads(pages, q_heads, &group)) != LF_OK ||
      (rc = take_window(pool, window, sinks, &window, &sinks)) != LF_OK ||
      (rc = decode_shape(pages, pool, group, window, sinks, &shape)) != LF_OK)
    return rc;
  *bytes = shape.bytes;
  return LF_OK;
}

int lf_paged_decode(const lf_pages* pages, int batch, const int32_t* page_table, int max_pages,
                    const int32_t* lens, int q_heads, const void* q, const void* k_new,
                    const void* v_new, void* out, float* lse, int window, int sinks,
                    void* workspace, size_t workspace_bytes, lf_stream_t stream) {
  lf::clear_last_error();
  lf::PagedDecodeArgs a;
  int rc = take_pool(pages, batch, page_table, max_pages, lens, &a.pool);
  if (rc != LF_OK || (rc = take_heads(pages, q_heads, &a.group)) != LF_OK ||
      (rc = take_window(a.pool, window, sinks, &a.window, &a.sinks)) != LF_OK)
    return rc;
  if (!q || !out || !aligned16(q) || !aligned16(out))
    return fail(LF_ERR_ARG, "q and out must be non-null and 16-byte aligned");
  if (!k_new != !v_new || !aligned16(k_new) || !aligned16(v_new))
    return fail(LF_ERR_ARG, "k_new and v_new come together, 16-byte aligned (or both null)");
  if (!aligned4(lse)) return fail(LF_ERR_ARG, "lse must be 4-byte aligned");
  a.q = q;
  a.k_new = static_cast<const char*>(k_new);
  a.v_new = static_cast<const char*>(v_new);
  a.out = out;
  a.lse = lse;
  a.q_heads = q_heads;
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)pages->head_dim));
  DecodeShape shape;
  if ((rc = decode_shape(pages, a.pool, a.group, a.window, a.sinks, &shape)) != LF_OK) return rc;
  a.whole_units = shape.whole_units;
  a.prefix_lens = nullptr;
  a.rest_o = a.rest_ml = nullptr;
  a.part_o = a.part_ml = nullptr;
  a.part_unit = nullptr;
  if (shape.bytes > 0) {
    if (!workspace || !aligned16(workspace) || workspace_bytes < shape.bytes)
      return fail(LF_ERR_ARG, "workspace: need %zu bytes, 16-byte aligned "
                  "(lf_paged_decode_workspace), got %zu", shape.bytes, workspace_bytes);
    char* w = static_cast<char*>(workspace);
    a.part_o = reinterpret_cast<float*>(w);
    a.part_ml = reinterpret_cast<float*>(w + shape.off_ml);
    a.part_unit = reinterpret_cast<int32_t*>(w + shape.off_unit);
  }
  const cudaError_t e = lf::paged_decode_launch(a, elem_bytes(pages), pages->head_dim, shape.grid,
                                                static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LF_OK : cuda_fail(e, "paged decode launch");
}

int lf_paged_decode_shared_workspace(const lf_pages* pages, int batch, int max_pages, int q_heads, int groups,
                                     size_t* bytes) {
  lf::clear_last_error();
  if (!pages || !bytes) return fail(LF_ERR_ARG, "null pages or bytes");
  lf::PagedPool pool;
  static const int32_t any = 0;  // only the shape counts here
  int group = 0;
  SharedShape shape;
  int rc = take_pool(pages, batch, &any, max_pages, &any, &pool);
  if (rc != LF_OK || (rc = take_heads(pages, q_heads, &group)) != LF_OK ||
      (rc = shared_shape(pages, pool, group, groups, &shape)) != LF_OK)
    return rc;
  *bytes = shape.bytes;
  return LF_OK;
}

int lf_paged_decode_shared(const lf_pages* pages, int batch, const int32_t* page_table, int max_pages,
                           const int32_t* lens, int q_heads, const void* q, const int32_t* group_start, int groups,
                           const int32_t* prefix_lens, const void* k_new, const void* v_new, void* out, float* lse,
                           void* workspace, size_t workspace_bytes, lf_stream_t stream) {
  lf::clear_last_error();
  lf::PagedDecodeArgs d = {};
  int rc = take_pool(pages, batch, page_table, max_pages, lens, &d.pool);
  if (rc != LF_OK || (rc = take_heads(pages, q_heads, &d.group)) != LF_OK) return rc;
  if (!q || !out || !aligned16(q) || !aligned16(out))
    return fail(LF_ERR_ARG, "q and out must be non-null and 16-byte aligned");
  if (!group_start || !prefix_lens || !aligned4(group_start) || !aligned4(prefix_lens))
    return fail(LF_ERR_ARG, "group_start and prefix_lens must be non-null and 4-byte aligned");
  if (!k_new != !v_new || !aligned16(k_new) || !aligned16(v_new))
    return fail(LF_ERR_ARG, "k_new and v_new come together, 16-byte aligned (or both null)");
  if (!aligned4(lse)) return fail(LF_ERR_ARG, "lse must be 4-byte aligned");
  if (groups < 1 || groups > batch) return fail(LF_ERR_ARG, "groups must be in [1, batch]");
  SharedShape shape;
  if ((rc = shared_shape(pages, d.pool, d.group, groups, &shape)) != LF_OK) return rc;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0 || workspace_bytes < shape.bytes)
    return fail(LF_ERR_ARG, "workspace: need %zu bytes, 16-byte aligned "
                "(lf_paged_decode_shared_workspace), got %zu", shape.bytes, workspace_bytes);
  char* w = static_cast<char*>(workspace);
  auto floats = [&](size_t off) { return reinterpret_cast<float*>(w + off); };
  d.q = q;
  d.k_new = static_cast<const char*>(k_new);
  d.v_new = static_cast<const char*>(v_new);
  d.out = out;
  d.lse = lse;
  d.q_heads = q_heads;
  d.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)pages->head_dim));
  d.part_o = floats(0);
  d.part_ml = floats(shape.rest.off_ml);
  d.part_unit = reinterpret_cast<int32_t*>(w + shape.rest.off_unit);
  d.prefix_lens = prefix_lens;
  d.rest_o = floats(shape.off_rest_o);
  d.rest_ml = floats(shape.off_rest_ml);
  lf::PagedSharedArgs a = {};
  a.pool = d.pool;
  a.q = q;
  a.group_start = group_start;
  a.prefix_lens = prefix_lens;
  a.groups = groups;
  a.q_heads = q_heads;
  a.group = d.group;
  a.fresh = k_new != nullptr;
  a.rows = shape.plan.rows;
  a.slots = shape.plan.slots;
  a.rounds = shape.plan.rounds;
  a.least = shape.plan.least;
  a.scale_log2 = d.scale_log2;
  a.part_rows = shape.plan.part_rows;
  a.part_o = floats(shape.off_part_o);
  a.part_ml = floats(shape.off_part_ml);
  a.segments = reinterpret_cast<int32_t*>(w + shape.off_segments);
  a.first_row = reinterpret_cast<int64_t*>(w + shape.off_first);
  a.ranges = reinterpret_cast<int32_t*>(w + shape.off_ranges);
  a.slot_rows = shape.plan.slot_rows;
  a.seen = reinterpret_cast<int32_t*>(w + shape.off_seen);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int e = elem_bytes(pages);
  const int ctas = shape.rest.grid;
  cudaError_t err = cudaSuccess;
  if (groups > shape.plan.table) err = lf::paged_shared_seen_launch(a, st);
  if (err == cudaSuccess && shape.plan.kernel == lf::PromptPlan::kTensor) {
    err = lf::paged_shared_tc_launch(a, d, pages->head_dim, ctas, st);
  } else if (err == cudaSuccess) {
    err = lf::paged_decode_behind_launch(d, e, pages->head_dim, ctas, st);
    if (err == cudaSuccess) err = lf::paged_shared_launch(a, shape.plan, pages->head_dim, st);
  }
  if (err == cudaSuccess) err = lf::paged_shared_join_launch(a, d, e, pages->head_dim, ctas, st);
  return err == cudaSuccess ? LF_OK : cuda_fail(err, "paged shared decode launch");
}

int lf_paged_prompt_workspace(const lf_pages* pages, int batch, int max_pages, int q_heads, int total_q,
                              int max_q, int window, int sinks, size_t* bytes) {
  lf::clear_last_error();
  if (!pages || !bytes) return fail(LF_ERR_ARG, "null pages or bytes");
  lf::PagedPool pool;
  static const int32_t any = 0;  // only the shape counts here
  int group = 0, sms = 0;
  int rc = take_pool(pages, batch, &any, max_pages, &any, &pool);
  if (rc != LF_OK || (rc = take_heads(pages, q_heads, &group)) != LF_OK ||
      (rc = take_window(pool, window, sinks, &window, &sinks)) != LF_OK ||
      (rc = take_rows(pool, group, total_q, max_q)) != LF_OK)
    return rc;
  *bytes = 0;
  if (max_q == 0) return LF_OK;
  if ((rc = sm_count(&sms)) != LF_OK) return rc;
  *bytes = lf::paged_prompt_plan(pool, elem_bytes(pages), pages->head_dim, group, total_q, max_q, window, sinks,
                                 sms)
               .bytes;
  return LF_OK;
}

int lf_paged_prompt(const lf_pages* pages, int batch, const int32_t* page_table, int max_pages,
                    const int32_t* lens, int q_heads, const void* q, const int32_t* q_start,
                    int total_q, int max_q, void* out, float* lse, int window, int sinks,
                    void* workspace, size_t workspace_bytes, lf_stream_t stream) {
  lf::clear_last_error();
  lf::PagedPromptArgs a;
  int rc = take_pool(pages, batch, page_table, max_pages, lens, &a.pool);
  if (rc != LF_OK || (rc = take_heads(pages, q_heads, &a.group)) != LF_OK ||
      (rc = take_window(a.pool, window, sinks, &a.window, &a.sinks)) != LF_OK)
    return rc;
  if ((rc = take_rows(a.pool, a.group, total_q, max_q)) != LF_OK) return rc;
  if (!q_start) return fail(LF_ERR_ARG, "null q_start");
  if (total_q == 0 || max_q == 0) return LF_OK;
  if (!q || !out || !aligned16(q) || !aligned16(out))
    return fail(LF_ERR_ARG, "q and out must be non-null and 16-byte aligned");
  if (!aligned4(q_start) || !aligned4(lse)) return fail(LF_ERR_ARG, "q_start and lse must be 4-byte aligned");
  a.q = q;
  a.q_start = q_start;
  a.out = out;
  a.lse = lse;
  a.q_heads = q_heads;
  a.total_q = total_q;
  a.max_q = max_q;
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)pages->head_dim));
  int sms = 0;
  if ((rc = sm_count(&sms)) != LF_OK) return rc;
  const lf::PromptPlan plan =
      lf::paged_prompt_plan(a.pool, elem_bytes(pages), pages->head_dim, a.group, total_q, max_q, a.window,
                            a.sinks, sms);
  a.tiles_per_seq = plan.tiles_per_seq;
  a.piece_shift = 0;
  while (a.group << a.piece_shift < plan.rows) ++a.piece_shift;
  a.splits = plan.splits;
  a.part_o = a.part_ml = nullptr;
  if (plan.bytes > 0) {
    if (!workspace || !aligned16(workspace) || workspace_bytes < plan.bytes)
      return fail(LF_ERR_ARG, "workspace: need %zu bytes, 16-byte aligned "
                  "(lf_paged_prompt_workspace), got %zu", plan.bytes, workspace_bytes);
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.off_ml);
  }
  const cudaError_t e = lf::paged_prompt_launch(a, plan, elem_bytes(pages), pages->head_dim,
                                                static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LF_OK : cuda_fail(e, "paged prompt launch");
}

int lf_paged_take_errors(const lf_pages* pages, int32_t* taken, lf_stream_t stream) {
  lf::clear_last_error();
  if (!pages || !pages->err || !taken) return fail(LF_ERR_ARG, "null pages, error word or taken");
  if (!aligned4(pages->err) || !aligned4(taken))
    return fail(LF_ERR_ARG, "the error word and taken must be 4-byte aligned");
  const cudaError_t e = lf::paged_take_errors_launch(pages->err, taken, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? LF_OK : cuda_fail(e, "paged take errors launch");
}

}  // extern "C"
