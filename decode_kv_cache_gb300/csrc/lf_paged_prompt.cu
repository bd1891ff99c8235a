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

#include "lf_paged_generic.cuh"

namespace lf {

namespace {

// The rows of a prompt as the kernels of lf_paged_generic.cuh take them.
struct PromptTask {
  using Args = PagedPromptArgs;
  Piece p;
  Tiles tiles;
  int share;

  __device__ __forceinline__ bool take(const Args& a, int per_piece, int keys) {
    share = blockIdx.y;
    int number;
    const int b = locate(a, blockIdx.x, &number);
    if (!take_piece(a, blockIdx.x, b, number, per_piece, threadIdx.x == 0 && share == 0, &p)) return false;
    tiles = Tiles(a, p.p_lo, p.p_hi, keys, share);
    return true;
  }
  // Where every sequence has as many numbers.
  __device__ __forceinline__ bool take_level(const Args& a, int per_piece, int keys) {
    share = blockIdx.y;
    const int heads = a.pool.batch * a.pool.kv_heads;
    const int id = gridDim.x - 1 - blockIdx.x, tile = id / heads;   // the last rows first
    if (!take_piece_level(a, id - tile * heads, tile, per_piece, threadIdx.x == 0 && share == 0, &p)) return false;
    tiles = Tiles(a, p.p_lo, p.p_hi, keys, share);
    return true;
  }
  __device__ __forceinline__ int count() const { return tiles.count(); }
  __device__ __forceinline__ int at(int j) const { return tiles.at(j); }
  __device__ __forceinline__ bool live(const Args&, int r) const { return p.r0 + r < p.rows; }
  __device__ __forceinline__ int pos(const Args& a, int r) const {
    return live(a, r) ? p.first_pos + (int)((p.r0 + r) / a.group) : -1;
  }
  __device__ __forceinline__ int64_t q_row(const Args& a, int r) const { return row_of(a, p, p.r0 + r); }
  __device__ __forceinline__ int behind(const Args& a) const { return behind_window(a, p.p_lo); }
  template <bool kSkip, class Behind>
  __device__ __forceinline__ int64_t offset(const Args& a, int pos, Behind b) const {
    return offset_of<kSkip>(a, p, pos, b);
  }
  __device__ __forceinline__ bool hidden(const Args& a, int k0, int keys) const {
    return some_hidden(a, p.p_lo, p.p_hi, k0, keys);
  }
  __device__ __forceinline__ bool sees(const Args& a, int pos, int key) const { return lf::sees(a, pos, key); }
  __device__ __forceinline__ bool parts(const Args& a) const { return a.splits > 1; }
  template <int D>
  __device__ __forceinline__ float* part(const Args& a, int per_piece, int r, float m, float l, bool first) const {
    return part_row<D>(a, p.id, share, per_piece, r, m, l, first);
  }
  __device__ __forceinline__ void* out(const Args& a) const { return a.out; }
  __device__ __forceinline__ void stats(const Args& a, int64_t row, float m, float l) const { write_row_stats(a, row, m, l); }
  template <typename T, int D>
  __device__ __forceinline__ void by_hand(const Args& a, int keys, int per_piece, int r, int n, int lane) const {
    rows_by_hand<T, D>(a, blockIdx.x, share, keys, per_piece, r, n, lane);
  }
  __device__ __forceinline__ void finish() const {}
};

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
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(&paged_mma_kernel<PromptTask, D>), kSmem, done);
  if (e != cudaSuccess) return e;
  paged_mma_kernel<PromptTask, D><<<dim3((unsigned)plan.pieces, plan.splits), kMmaThreads, kSmem, stream>>>(a);
  return cudaGetLastError();
}

template <int D, int R, int M>
cudaError_t launch_fma(const PagedPromptArgs& a, const PromptPlan& plan, cudaStream_t stream) {
  constexpr int kSmem = fma_smem<D, R>();
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(&paged_fma_kernel<PromptTask, D, R, M>), kSmem, done);
  if (e != cudaSuccess) return e;
  paged_fma_kernel<PromptTask, D, R, M><<<dim3((unsigned)plan.pieces, plan.splits), 16 * R / M, kSmem, stream>>>(a);
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
