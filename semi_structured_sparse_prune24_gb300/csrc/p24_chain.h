// p24_chain.h -- chains of list entries by index: head[] holds a chain's first entry, next[] the
// entry after each one, -1 the end. Host and device.
#pragma once

#ifdef __CUDACC__
#define P24_HD __host__ __device__ __forceinline__
#else
#define P24_HD inline
#endif

namespace p24 {

// f(entry) along the chain that begins with entry j, of at most `most` entries 0..most-1. A chain
// that entries were added to before it was used up, as may be left where a wait ran out, can be a
// cycle; the walk ends all the same.
template <typename F>
P24_HD void chain_walk(int j, const int* next, int most, F&& f) {
  for (int n = 0; n < most && static_cast<unsigned>(j) < static_cast<unsigned>(most); ++n) {
    const int then = next[j];
    f(j);
    j = then;
  }
}

}  // namespace p24
