// Reading what the previous kernel of a chain wrote.
#pragma once

#include "pdl.cuh"

namespace sana {

// griddep_wait(), then p as a pointer through which nothing can have been read
// before: loads through const __restrict__ parameters are free to move up past the
// wait, those through the result are not.
template <class T>
__device__ __forceinline__ const T* griddep_wait_for(const T* p) {
  griddep_wait();
  asm volatile("" : "+l"(p)::"memory");
  return p;
}

}  // namespace sana
