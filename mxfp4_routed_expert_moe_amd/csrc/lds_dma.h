// LDS-DMA loads of the attention-side kernels: memory to LDS, no registers in
// between.  A wave's 64 lanes give 64 source addresses; the bytes land one
// after the other from the (wave-uniform) LDS address on.
#pragma once

#include "moe_internal.h"

namespace moe {

// 16 bytes per lane from byte `offset` + `uniform` of a buffer resource.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t rsrc, int offset, int uniform, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, lds, 16, offset, uniform, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t rsrc, int offset, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, lds, 4, offset, 0, 0, 0);
}

// Barrier between the readers of an LDS stage and the DMA that refills it:
// the wave's LDS reads have returned; DMA in flight is left in flight.
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0), other counters untouched
  lds_barrier();
}

}  // namespace moe
