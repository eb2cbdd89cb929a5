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

}  // namespace sinkattn
