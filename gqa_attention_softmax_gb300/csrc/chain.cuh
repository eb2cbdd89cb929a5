// Device side of a chain of dependent launches (host side: internal.h).
#pragma once

namespace sinkattn {

// Waits until the launch this one programmatically depends on has completed
// and its writes are visible (immediate without one).
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Lets the next launch of the chain start as SMs have room (it still waits
// for this one where it has to).
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// A word that a launch further back in the chain wrote. The launch between has
// waited for that one, so the word is in L2; a launch that does not wait itself
// must not take it from its SM's L1.
__device__ __forceinline__ int32_t chain_load(const int32_t* p) { return __ldcg(p); }

}  // namespace sinkattn
