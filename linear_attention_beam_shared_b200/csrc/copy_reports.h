// Which of a warp's items (tiles of a ring, numbered as they are issued) still
// have to be reported full by the warp itself: those brought in by its own
// asynchronous copies.  Items that come as TMA boxes report themselves.
#pragma once

#include <stdint.h>

#ifndef __CUDACC__
#define __host__
#define __device__
#define __forceinline__ inline
#endif

namespace onela {

struct CopyReports {
  // While pend is not 0: items below `told` are reported, and bit i mod 32 of
  // pend says that item i >= told waits to be.  The marks are told apart by
  // the index mod 32, so told has to start at the first of them and to keep
  // within 32 of the last: an item that is marked while nothing is pending
  // starts anew (told stood still since the last report, however many boxes
  // ago that was), and every item after it moves told along.
  uint32_t told = 0, pend = 0;

  // Item i is under way by asynchronous copies.
  __host__ __device__ __forceinline__ void mark(uint32_t i) {
    if (!pend) told = i;
    pend |= 1u << (i & 31);
  }
  // Is anything below `upto` to be looked at?
  __host__ __device__ __forceinline__ bool due(uint32_t upto) const { return pend && told < upto; }
  // The copies of all items below `upto` have landed: full(i) for each that waited.
  template <typename F>
  __host__ __device__ __forceinline__ void landed(uint32_t upto, F full) {
    for (; told < upto; ++told) {
      if ((pend >> (told & 31)) & 1) full(told);
      pend &= ~(1u << (told & 31));
    }
  }
};

}  // namespace onela
