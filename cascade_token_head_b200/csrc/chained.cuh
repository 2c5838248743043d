// What the serving kernels share: launches that overlap the end of the kernel before, and wide stores.
#pragma once

#include "common.cuh"

namespace spt {

// Launch of a kernel that may start before the one ahead of it in the stream has ended (programmatic
// stream serialisation), in clusters of `cluster` CTAs.  Every thread of such a kernel calls
// grid_dep_wait() before it touches global memory or returns, so that what ran before is complete.
template <typename... P>
int32_t launch_chained(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, int cluster,
                       const P&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  SPT_CUDA(cudaLaunchKernelEx(&cfg, kernel, args...));
  return launch_status();
}

// Programmatic dependent launch: wait until the grids ahead have completed and their writes are visible;
// let the next grid's CTAs start once every CTA of this one has (or has ended).
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// 32 bytes to a 16-byte aligned address, in one piece where it is a multiple of 32 (whole sectors)
__device__ __forceinline__ void store32(void* p, const uint32_t* x) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]),
                 "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    static_cast<uint4*>(p)[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

}  // namespace spt
