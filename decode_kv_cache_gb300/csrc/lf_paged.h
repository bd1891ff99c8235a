// Paged key-value cache: the arguments its kernels share and their lookup.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace lf {

// The pools of one layer and one call's page table.  Strides are in bytes.
struct PagedPool {
  char* k;
  char* v;
  int64_t page_stride, head_stride, token_stride;
  int page_size, page_shift;  // page_shift: log2(page_size), or -1 when it is no power of two
  int num_pages, kv_heads;
  const int32_t* table;       // [batch][max_pages]
  const int32_t* lens;        // [batch]
  int batch, max_pages;
  int32_t* err;               // may be null
};

struct PagedAppendArgs {
  PagedPool pool;
  const char* k_new;
  const char* v_new;
  const int32_t* new_start;   // [batch + 1], or null: one token per sequence
  int total_new, tokens_per_block, row_bytes;  // row_bytes: one head's row
};

struct PagedDecodeArgs {
  PagedPool pool;
  const void* q;
  const char* k_new;          // null: the new token is in the pages already
  const char* v_new;
  void* out;
  float* lse;                 // may be null
  int q_heads, group, window, sinks;
  float scale_log2;           // log2(e) / sqrt(head_dim)
  int whole_units;            // 1: CTA i takes unit i alone (no join); 0: level ranges
  float* part_o;              // level ranges: [2 grid][group][head_dim] partial outputs
  float* part_ml;             // [2 grid][group][2] their max and sum
  int32_t* part_unit;         // [grid] the unit a CTA's range starts inside, or -1
  // Behind a shared prefix (else null): the positions below it are left to PagedSharedArgs' kernel, and whole
  // units go to rest_o, rest_ml as parts do.
  const int32_t* prefix_lens; // [batch]
  float* rest_o;              // [batch][q_heads][head_dim]
  float* rest_ml;             // [batch][q_heads][2]
};

struct PagedPromptArgs {
  PagedPool pool;
  const void* q;
  const int32_t* q_start;     // [batch + 1]
  void* out;
  float* lse;                 // may be null
  int q_heads, group, window, sinks, total_q, max_q;
  float scale_log2;
  int tiles_per_seq;          // pieces that each sequence has numbers for, or 0 (PromptPlan)
  int piece_shift;            // log2 of a piece's tokens
  int splits;                 // blocks that share a piece's keys; 1: no join
  float* part_o;              // [pieces][splits][rows][head_dim] partial outputs
  float* part_ml;             // [pieces][splits][rows][2] their max and sum
};

// How a prompt call is spread over the GPU.  A piece of work is `rows` rows (token and
// head of the group) of one KV head's queries of one sequence.  The host knows neither
// the sequences' rows nor their sum, only bounds, so that some numbers name no piece and
// their blocks end at once: either every sequence has as many as max_q rows need
// (tiles_per_seq), or the numbers follow the rows (locate), with at most one more than pieces
// for each sequence.
struct PromptPlan {
  enum Kernel { kTensor, kMatrix, kFma } kernel;
  int rows, splits, tiles_per_seq;
  int64_t pieces;             // numbers of pieces, of all KV heads
  size_t off_ml, bytes;       // workspace: part_o, part_ml
};
PromptPlan paged_prompt_plan(const PagedPool& pool, int elem, int head_dim, int group, int total_q, int max_q,
                             int window, int sinks, int sms);

// The last tokens of groups of sequences before the prefix that each group shares.  A piece is
// up to `rows` rows (sequence and head of the group) of one KV head, a unit a piece of one KV head; a unit's
// key tiles are cut into segments of `chunk`, one block each.
struct PagedSharedArgs {
  PagedPool pool;
  const void* q;
  const int32_t* group_start; // [groups + 1]
  const int32_t* prefix_lens; // [batch]
  int groups, q_heads, group;
  int fresh;                  // 1: the last token comes with the call, and is no part of a prefix
  int rows;
  int slots, rounds, least;   // blocks that run at once; rounds of them that the grid has room for; tiles of a segment at least
  float scale_log2;
  int64_t part_rows;          // rows that part_o and part_ml have
  float* part_o;              // [part_rows][head_dim] partial outputs
  float* part_ml;             // [part_rows][2] their max and sum
  // For the join, of every group.  Blocks of a segment each: segments of a unit, first row of the group in part_o.
  // Ranges (ranges[0] > 0 CTAs of ranges[1] places, ranges[2] in front of a unit; slot_rows rows of part_o per CTA):
  // tiles of a unit, the group's first place.
  int32_t* segments;          // [groups]
  int64_t* first_row;         // [groups]
  int32_t* ranges;            // [3]
  int slot_rows;
  int32_t* seen;              // what a group's members see of its prefix: [groups], or, ranges of few groups, [CTAs][groups]
};

// Its kernel by type, heads and pages, and the rows of a piece.
struct SharedPlan {
  PromptPlan::Kernel kernel;
  int rows, keys, slots, rounds, least, slot_rows;
  int64_t grid, part_rows;
  int table;                  // groups that the kernel looks at in its own memory; of more another launch comes ahead
  bool fits;                  // the kernels' numbers hold such a call
};
constexpr int kTableTensor = 2048, kTableOther = 512;
SharedPlan paged_shared_plan(const PagedPool& pool, int elem, int head_dim, int group, int groups, int sms);

// Occupied tokens of sequence b, kept inside its row of the page table.
__device__ __forceinline__ int paged_len(const PagedPool& p, int b) {
  const int n = p.lens[b];
  const int64_t most = (int64_t)p.max_pages * p.page_size;
  return n < 0 ? 0 : (n > most ? (int)most : n);
}

// Page index in the row and slot in the page of a position.
__device__ __forceinline__ void paged_split(const PagedPool& p, int pos, int* page, int* slot) {
  if (p.page_shift >= 0) {
    *page = pos >> p.page_shift;
    *slot = pos & (p.page_size - 1);
  } else {
    *page = (int)((unsigned)pos / (unsigned)p.page_size);
    *slot = pos - *page * p.page_size;
  }
}

// Opt-in shared memory of a kernel, asked for once per device: `done` has a bit per
// device (the first 64; further ones ask each time).
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Numbers of the pieces of `rows` rows, of all KV heads; *tiles_per_seq as in PromptPlan.
// Numbers that follow the rows need a search of the row starts, and a sequence's pieces come
// together instead of all sequences' last ones first, so they have to be a third fewer.
// (32 / 8 heads of 128, bf16, each against following: one chunk of 512 among 255 single
// tokens behind 1000, 412 us, 285; one prompt of 8192 among 31, 795, 517; chunks of 1 to 512
// behind up to 2048, 153, 139; three fp32 prompts of 500 to 1000, 61, 67.)
inline int64_t paged_prompt_pieces(const PagedPool& pool, int group, int total_q, int max_q, int rows,
                                   bool may_follow, int* tiles_per_seq) {
  auto pieces = [&](int64_t tokens) { return (tokens * group + rows - 1) / rows; };
  const int64_t each = pieces(max_q) * pool.batch, all = pieces(total_q) + pool.batch - 1;
  const bool level = !may_follow || 2 * each <= 3 * all;
  *tiles_per_seq = level ? (int)pieces(max_q) : 0;
  return (level ? each : all) * pool.kv_heads;
}

// Launches (one translation unit each).  They return the launch's error.
cudaError_t paged_take_errors_launch(int32_t* err, int32_t* taken, cudaStream_t stream);
cudaError_t paged_append_launch(const PagedAppendArgs& a, cudaStream_t stream);
// elem: bytes of an element (2 bf16, 4 fp32).  `grid`: CTAs of the attention kernel.
cudaError_t paged_decode_launch(const PagedDecodeArgs& a, int elem, int head_dim, int grid,
                                cudaStream_t stream);
// The same behind shared prefixes, whole units and parts left to paged_shared_join_launch.
cudaError_t paged_decode_behind_launch(const PagedDecodeArgs& a, int elem, int head_dim, int grid, cudaStream_t stream);
cudaError_t paged_prompt_launch(const PagedPromptArgs& a, const PromptPlan& plan, int elem, int head_dim,
                                cudaStream_t stream);
// Its tensor-core kernel: whether that takes such a cache, and its launch.
bool paged_prompt_tc_takes(const PagedPool& pool, int head_dim);
cudaError_t paged_prompt_tc_launch(const PagedPromptArgs& a, const PromptPlan& plan, int head_dim,
                                   cudaStream_t stream);

// What the members of each group see of its prefix, to a.seen.
cudaError_t paged_shared_seen_launch(const PagedSharedArgs& a, cudaStream_t stream);

// A decode call behind prefixes, and the join of its shares; `ctas`: those that the rest's walk may have had.  On the
// tensor cores prefixes and rest are one launch of `ctas` CTAs.  Otherwise the prefixes follow the rest's launch, placed while
// that drains (it has waited for what came before it).
cudaError_t paged_shared_tc_launch(const PagedSharedArgs& a, const PagedDecodeArgs& rest, int head_dim, int ctas,
                                   cudaStream_t stream);
cudaError_t paged_shared_launch(const PagedSharedArgs& a, const SharedPlan& plan, int head_dim, cudaStream_t stream);
cudaError_t paged_shared_join_launch(const PagedSharedArgs& a, const PagedDecodeArgs& rest, int elem, int head_dim,
                                     int ctas, cudaStream_t stream);

// Tokens that one CTA of the decode kernel takes in one sweep of its warps.
int paged_decode_sweep(int elem, int head_dim);

}  // namespace lf
