// pdl.cuh -- programmatic dependent launch: a kernel launched with the attribute
// may start while the kernel before it in the stream ends.  Nothing that depends
// on that kernel may be read, and nothing written, before grid_dependency_wait();
// every block calls it, also one without work, so that a grid's end implies the
// end of all before it.
// Nor may what that kernel can have written be read as read-only data (__ldg, const
// __restrict__): it changes while this kernel lives, and such reads may be moved before
// the wait or served from a copy made before the write.
#pragma once

namespace dg {
namespace pdl {

// All grids this one depends on have completed and their writes are visible.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The next grid may be scheduled once every block has called this (its first thread
// that does so counts) or ended.
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace pdl
}  // namespace dg
