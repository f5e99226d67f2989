// One lane of a warp for the instructions that a single thread issues; internal.
#pragma once

#include <stdint.h>

namespace bconv {
namespace tcdev {

// True in one lane of the (converged) warp.  The compiler knows that a region behind this has one
// active thread and issues the MMA, commit and copy instructions of it, which take warp-uniform
// operands, directly; behind `lane == 0` each of them became a loop over the active lanes of some 90 cycles.
__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(pred));
  return pred != 0;
}

}  // namespace tcdev
}  // namespace bconv
