// Attention of one new token per sequence over a paged key-value cache.
//
//   s_j = (q . k_j) / sqrt(d),  out = sum_j 2^(s_j' - m) v_j / sum_j 2^(s_j' - m)
//
// with s' = s log2(e) and m the running maximum, over the positions a query
// sees: all of the sequence, or the first `sinks` and the last `window` ones.
// These are numbered 0 .. seen - 1 without the gap between them, so that a
// window costs what its tokens cost and nothing else.
//
// Bound by HBM: every key and value is read once and used by the group's <= 8
// query heads (about 2 G flop per byte in bf16).  What follows from that:
//   - a warp is the worker.  It walks tiles of one KV head's tokens through a
//     ring of its own in shared memory (cp.async, 16-byte chunks gathered by
//     page, chunks of unseen tokens filled with zeros), and nothing but its own
//     copies makes it wait.  The ring runs on across the ends of sequences and
//     heads; the page indexes of a tile are fetched one tile ahead.
//   - the tiles of all sequences and KV heads are one list, cut into equal
//     ranges, one per CTA, and each CTA's range into one per warp.  Lengths are
//     read on the device, so a captured graph follows them.
//   - a warp's parts of a unit (sequence, KV head) are joined in shared memory
//     with those of its CTA's other warps, and parts of CTAs in a second, small
//     launch that is placed while the first one drains (programmatic dependent
//     launch).  Parts are joined in order of position: the result does not
//     depend on which finished first.
// Where a unit is too short for a cut to pay, a CTA takes a whole unit and there
// is no second launch.
//
// Measured, bf16, 32 / 8 heads of 128, and share of a plain copy's 6.69 TB/s: 64 sequences of
// 3276 tokens 138 us, 93 %; 256 of 64 to 3276 281 us, 93 %; two of 100 to 130 thousand 157 us,
// 95 %; a window of 1000 and 4 sinks of 64 sequences 53 us, 74 %: about 9 us of a launch are
// the first copies' latency and the last tiles, and the join, 5 us, waits for them.
// One sequence of 300 tokens takes 9 us on the device, most of it three round trips to
// memory: lengths, page indexes, keys.
#include "lf_paged_decode.cuh"

namespace lf {

namespace {

// ---- joining the CTAs' parts ---------------------------------------------------------
//
// Block (w, h) joins head h of the unit that CTA w + 1's range starts inside, if
// that is the first range that does: the last part of CTA w, then the first ones
// of CTAs w + 1, w + 2, .. while they start inside the same unit.  Its warps take
// the parts in turn and join through shared memory.  Bound by latency: 5 us, part of
// which passes while the first kernel drains.
constexpr int kJoinWarps = 8;

template <typename T, int D, int G>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_decode_join_kernel(const __grid_constant__ PagedDecodeArgs a, int ctas) {
  constexpr int E = D >= 32 ? D / 32 : 1;
  __shared__ float s_o[kJoinWarps][D];
  __shared__ float s_ml[kJoinWarps][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int w = blockIdx.x + 1, h = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int unit = a.part_unit[w];
  if (unit < 0 || a.part_unit[w - 1] == unit) return;
  int n = 1;  // parts: a unit's ranges are consecutive
  for (int i = w; i < ctas; i += kJoinWarps * 32) {
    const int c = __syncthreads_count(i + tid < ctas && a.part_unit[i + tid] == unit);
    n += c;
    if (c < kJoinWarps * 32) break;
  }
  auto slot = [&](int i) { return i == 0 ? 2 * (int64_t)(w - 1) + 1 : 2 * (int64_t)(w - 1 + i); };
  float m, l, acc[E];
  const int mine = n > warp ? (n - warp + kJoinWarps - 1) / kJoinWarps : 0;
  auto part = [&](int i) { return slot(warp + i * kJoinWarps) * G + h; };
  join_parts<D>(
      mine, [&](int i) { return a.part_ml + part(i) * 2; },
      [&](int i) { return a.part_o + part(i) * D; }, lane, &m, &l, acc);
  if (lane * E < D) {
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
  }
  if (lane == 0) {
    s_ml[warp][0] = m;
    s_ml[warp][1] = l;
  }
  __syncthreads();
  if (warp == 0) {
    join_parts<D>(
        min(n, kJoinWarps), [&](int i) { return s_ml[i]; }, [&](int i) { return s_o[i]; }, lane, &m,
        &l, acc);
    const int b = unit / a.pool.kv_heads;
    write_row<T, D, false>(a, (int64_t)b * a.q_heads + (unit - b * a.pool.kv_heads) * G + h, lane, m, l, acc);
  }
}

struct Decode {
  template <class C, int D, int G>
  static cudaError_t launch(const PagedDecodeArgs& a, int grid, cudaStream_t stream) {
    const cudaError_t e = launch_walk<C, D, G, false>(a, grid, stream);
    if (e != cudaSuccess || a.whole_units || grid < 2) return e;
    const DrainConfig c(dim3(grid - 1, G, 1), kJoinWarps * 32, 0, stream);
    return cudaLaunchKernelEx(&c.cfg, paged_decode_join_kernel<typename C::T, D, G>, a, grid);
  }
};

template <template <int, int> class C>
int sweep(int head_dim) {
  switch (head_dim) {
    case 16: return C<16, 1>::kTokens * C<16, 1>::kWarps;
    case 32: return C<32, 1>::kTokens * C<32, 1>::kWarps;
    case 64: return C<64, 1>::kTokens * C<64, 1>::kWarps;
    default: return C<128, 1>::kTokens * C<128, 1>::kWarps;
  }
}

}  // namespace

cudaError_t paged_decode_launch(const PagedDecodeArgs& a, int elem, int head_dim, int grid,
                                cudaStream_t stream) {
  return by_type<Decode>(a, elem, head_dim, grid, stream);
}

int paged_decode_sweep(int elem, int head_dim) {
  return elem == 2 ? sweep<MmaTile>(head_dim) : sweep<SimtTile>(head_dim);
}

}  // namespace lf
