// Kernels of one call that follow each other are launched so that each sets up
// while the one before ends (programmatic launches): next_pass() lets the next
// one begin as soon as all of this one's CTAs have called it, last_pass() waits
// until the one before is done and its results can be read, past L1
// (__ldcg), which may hold older lines.  Both do nothing in ordinary launches.
#pragma once

namespace vrwkv {

__device__ __forceinline__ void next_pass() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void last_pass() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace vrwkv
