// The decode kernel's walk behind shared prefixes: a launch of its own where lf_paged_shared.cu's kernels take the prefixes.
// Whole units go where that file's join looks for them, and so do the parts of others.  (lf_paged_decode.cu says what the walk
// does; its kernels for both uses are built side by side.)
#include "lf_paged_decode.cuh"

namespace lf {

namespace {

struct Behind {
  template <class C, int D, int G>
  static cudaError_t launch(const PagedDecodeArgs& a, int grid, cudaStream_t stream) {
    return launch_walk<C, D, G, true>(a, grid, stream);
  }
};

}  // namespace

cudaError_t paged_decode_behind_launch(const PagedDecodeArgs& a, int elem, int head_dim, int grid, cudaStream_t stream) {
  return by_type<Behind>(a, elem, head_dim, grid, stream);
}

}  // namespace lf
