// Attention of one new token per sequence where groups of sequences share a prefix: the prefix's keys and
// values are read once for all of a group's sequences and heads, the rest as decode reads it.
//
//   out = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s,  m = max_s m_s
//
// over shares s of a row's keys, each with its maximum m_s (log2), sum l_s and output O_s (not normalised): shares of
// the prefix, and what lies behind it.  Three launches:
//   - lf_paged_decode.cu's kernel walks every sequence from its prefix's end on;
//   - the prefix's kernel (here or lf_paged_shared_tc.cu) takes up to 256 rows, (sequence, head of the group) pairs, of
//     a KV head against a segment of the prefix's keys, so that with G rows from each of n sequences a key is used n G
//     times.  It depends on nothing that the first one writes and is placed while that drains (programmatic
//     dependent launch); it ends behind it;
//   - the join below adds the shares up, in order of position.
// Bound by HBM while a KV head has fewer than about 500 rows, and by the matrix instructions above.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "lf_paged_generic.cuh"
#include "lf_paged_shared.cuh"

namespace lf {

namespace {

// A segment as the kernels of lf_paged_generic.cuh take it.
template <int kThreads>
struct SharedTask {
  using Args = PagedSharedArgs;
  Segment s;

  __device__ __forceinline__ bool take(const Args& a, int, int keys) {
    const bool ok = take_segment<kThreads>(a, keys, &s);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!ok) finish();
    return ok;
  }
  __device__ __forceinline__ bool take_level(const Args& a, int per_piece, int keys) { return take(a, per_piece, keys); }
  __device__ __forceinline__ int count() const { return s.last - s.first; }
  __device__ __forceinline__ int at(int j) const { return s.first + j; }
  __device__ __forceinline__ bool live(const Args& a, int r) const { return r < s.members * a.group; }
  __device__ __forceinline__ int pos(const Args& a, int r) const { return live(a, r) ? last_seen(a, s.prefix, s.b0 + r / a.group) : -1; }
  __device__ __forceinline__ int64_t q_row(const Args& a, int r) const { return shared_row(a, s, r); }
  __device__ __forceinline__ int behind(const Args&) const { return 0; }
  template <bool kSkip, class Behind>
  __device__ __forceinline__ int64_t offset(const Args& a, int pos, Behind) const { return shared_offset(a, s, pos); }
  __device__ __forceinline__ bool hidden(const Args&, int k0, int keys) const { return k0 + keys - 1 > s.p_lo; }
  __device__ __forceinline__ bool sees(const Args&, int pos, int key) const { return key <= pos; }
  __device__ __forceinline__ bool parts(const Args&) const { return true; }
  template <int D>
  __device__ __forceinline__ float* part(const Args& a, int, int r, float m, float l, bool first) const {
    if (first) {
      a.part_ml[2 * (s.row + r)] = m;
      a.part_ml[2 * (s.row + r) + 1] = l;
    }
    return a.part_o + (s.row + r) * D;
  }
  __device__ __forceinline__ void* out(const Args&) const { return nullptr; }
  __device__ __forceinline__ void stats(const Args&, int64_t, float, float) const {}
  template <typename T, int D>
  __device__ __forceinline__ void by_hand(const Args& a, int keys, int, int r, int n, int lane) const {
    for (int i = r; i < r + n && live(a, i); ++i) shared_row_by_hand<T, D>(a, s, keys, i, pos(a, i), lane);
  }
  // The kernel before this one ends before this one does, and with it before the join.
  __device__ __forceinline__ void finish() const {
    if (threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  }
};

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
  return launch(reinterpret_cast<const void*>(&paged_mma_kernel<SharedTask<kMmaThreads>, D>), a, grid, kMmaThreads,
                4 * kKeys * D * 2, done, stream);
}

template <int D, int R, int M>
cudaError_t launch_fma(const PagedSharedArgs& a, int64_t grid, cudaStream_t stream) {
  constexpr int kThreads = 16 * R / M;
  static std::atomic<uint64_t> done{0};
  return launch(reinterpret_cast<const void*>(&paged_fma_kernel<SharedTask<kThreads>, D, R, M>), a, grid, kThreads,
                fma_smem<D, R>(), done, stream);
}

// ---- the join --------------------------------------------------------------------------
//
// A block per sequence and KV head.  The rest's share is in its place, or in the parts of the CTAs whose ranges
// met it (lf_paged_decode.cu); the prefix's shares are rows that its blocks left.  Warps take a row of the group each, or
// every so many of its shares, and join through shared memory, in order of position.  Bound by latency: what the call was given is
// read while the kernel before drains, then come two reads that depend on each other, places and shares.
constexpr int kJoinWarps = 8, kJoinBatch = 4;

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

template <typename T, int D, int G>
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

template <typename T, int D, int G>
cudaError_t launch_join(const PagedSharedArgs& a, const PagedDecodeArgs& rest, int ctas, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.pool.batch * a.pool.kv_heads), 1, 1);
  cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_shared_join_kernel<T, D, G>, a, rest, ctas);
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

SharedPlan paged_shared_plan(const PagedPool& pool, int elem, int head_dim, int group, int groups, int sms) {
  SharedPlan p;
  p.keys = kKeys;
  p.least = 1;
  if (elem == 2 && paged_prompt_tc_takes(pool, head_dim)) {
    p.kernel = PromptPlan::kTensor;
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
    p.rows = head_dim == 128 && pool.batch * group >= 64 ? 64 : 32;
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
