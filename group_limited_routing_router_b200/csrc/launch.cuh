// Kernels that follow one another on a stream without the gap of a launch between them: the later one is launched
// (launch_after in ragged_api.cuh) while the earlier one still runs, and waits for it by itself.
#pragma once

namespace beam {

// First of all that touches global memory or TMEM, by every thread: returns when the stream's last kernel has
// completed and its writes are visible.  Nothing is read by non-coherent loads (ld.global.nc, __ldg, pointers to const
// __restrict__): they are for data that nobody writes while the kernel lives, which here includes the end of the one
// before.  A kernel that returns before the wait would let the next one overtake that kernel.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The next kernel may be launched once every block has come here.  For short kernels of small blocks: the next one's
// blocks take their places on the SMs meanwhile.
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace beam
