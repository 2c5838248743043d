// Shared device/host helpers of libspatten (sm_100a).  Nothing here is specific to one kernel.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "spatten.h"

namespace spt {

// An NVTX range over one C-ABI call, named after the call: it shows the call's span (host
// enqueue) in profiler timelines; without a profiler attached the push and pop do nothing.
struct AbiRange {
  explicit AbiRange(const char* name) { nvtxRangePushA(name); }
  ~AbiRange() { nvtxRangePop(); }
  AbiRange(const AbiRange&) = delete;
  AbiRange& operator=(const AbiRange&) = delete;
};

// ----------------------------------------------------------------------------------------------
// host-side status helpers
// ----------------------------------------------------------------------------------------------
void record_cuda_error(cudaError_t e);                 // thread-local message for the ABI
int32_t launch_status();                               // cudaGetLastError -> status
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

#define SPT_TRY(expr)                                  \
  do {                                                 \
    int32_t _s = (expr);                               \
    if (_s != SPATTEN_OK) return _s;                   \
  } while (0)

#define SPT_CUDA(expr)                                 \
  do {                                                 \
    cudaError_t _e = (expr);                           \
    if (_e != cudaSuccess) {                           \
      ::spt::record_cuda_error(_e);                    \
      return SPATTEN_E_CUDA;                           \
    }                                                  \
  } while (0)

// Bump allocator over a caller-provided workspace (no device allocation).
struct WsCursor {
  char* base;
  size_t size;
  size_t used = 0;
  WsCursor(void* b, size_t s) : base(static_cast<char*>(b)), size(s) {}
  template <typename T>
  T* take(size_t count) {
    size_t off = align_up(used, 256);
    used = off + count * sizeof(T);
    return base ? reinterpret_cast<T*>(base + off) : nullptr;
  }
  bool fits() const { return used <= size; }
};

// Number of SMs of the current device (cached per device).
int sm_count();

// First-call set-up (kernel attributes, capability probes) once per device ordinal.  The first
// caller on a device runs `setup(dev)` under a lock; callers from other host threads wait for it,
// so no launch can run before its attributes are set.  A set-up that fails is tried again on the
// next call.  Returns the set-up's status (SPATTEN_OK once it has succeeded) and the device in *dev.
struct DeviceOnce {
  std::mutex mu;
  std::atomic<bool> done[64] = {};
};
template <typename F>
int32_t once_per_device(DeviceOnce& once, int* dev_out, F&& setup) {
  int dev = 0;
  SPT_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return SPATTEN_E_UNSUPPORTED;
  *dev_out = dev;
  if (once.done[dev].load(std::memory_order_acquire)) return SPATTEN_OK;
  std::lock_guard<std::mutex> lock(once.mu);
  if (once.done[dev].load(std::memory_order_relaxed)) return SPATTEN_OK;
  const int32_t s = setup(dev);
  if (s == SPATTEN_OK) once.done[dev].store(true, std::memory_order_release);
  return s;
}

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

// ----------------------------------------------------------------------------------------------
// device helpers
// ----------------------------------------------------------------------------------------------
// Programmatic dependent launch: wait until the grids ahead have completed and their writes are visible;
// let the next grid's CTAs start once every CTA of this one has (or has ended).
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void report(int32_t* st, int32_t code) {
  if (st) atomicCAS(st, 0, code);
}

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

__device__ __forceinline__ float ld_as_float(const float* p) { return *p; }
__device__ __forceinline__ float ld_as_float(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ void st_from_float(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_from_float(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 8 consecutive elements -> float[8] (16-byte or 32-byte aligned vector load)
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* f) {
  uint4 u = *reinterpret_cast<const uint4*>(p);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 t = __bfloat1622float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float* f) {
  float4 a = *reinterpret_cast<const float4*>(p);
  float4 b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ int warp_sum_int(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Order-preserving map float -> uint32 (larger float -> larger key); -0.0 maps like +0.0 (adding
// +0.0 turns -0.0 into +0.0 and leaves every other non-NaN value as it is).  Negative values take
// all bits flipped, the others the sign bit set.
__device__ __forceinline__ uint32_t float_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

}  // namespace spt
