// Equal ranges of a list of places (device code; plain C++ but for its qualifiers).
#pragma once

#include <stdint.h>

namespace lf {

// CTA i's range starts at place floor(places * i / ctas).  (Products that 32 bits do not hold are rare, and their divisions slow.)
struct Ranges {
  unsigned places, ctas;
  bool small;
  __device__ __forceinline__ Ranges(unsigned p, unsigned c) : places(p), ctas(c), small(p < 0xffffffffu / (c + 1)) {}
  __device__ __forceinline__ unsigned first(unsigned i) const {
    return small ? places * i / ctas : (unsigned)((uint64_t)places * i / ctas);
  }
  __device__ __forceinline__ unsigned owner(unsigned x) const {   // the last i with first(i) <= x
    return small ? ((x + 1) * ctas - 1) / places : (unsigned)((((uint64_t)x + 1) * ctas - 1) / places);
  }
};

}  // namespace lf
