// Launches that overlap their start with the end of the work before them.
//
// A kernel launched with `launch` may become resident while the stream's
// previous kernel still runs (programmatic dependent launch): it sets up its
// barriers and tensor memory, then waits in after_previous() until that kernel
// is complete and its writes are visible, and only then touches global memory.
// let_next_start() allows the following kernel the same; it is called once every
// block is past its start.  A kernel before it that never calls it simply
// completes first.
//
// Such a kernel lives while its predecessor still writes, so nothing that an earlier
// kernel may have written is constant for its lifetime: the read-only path (__ldg, or
// const __restrict__ pointers, which become it) is not allowed to it, and the compiler may
// move such loads above the wait.  Operands are read by the ld_* loads below, ordinary
// loads that stay behind after_previous().
//
// Measured on 8-bit products of one token (8192 x 8192): 15.5 us
// a pass without, 14.5 with; on one quantised row 2.85 and 1.75.
#pragma once

#include <initializer_list>
#include <utility>

#include "tcq_device.cuh"

namespace tcq {

__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ uint4 ld_u32x4(const void *p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_f32x4(const float *p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_u32(const void *p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float ld_f32(const float *p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint16_t ld_u16(const void *p) {
  uint16_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_u8(const void *p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

}  // namespace tcq

namespace tcq_host {

// What a call reads or writes.  `clash`: something written meets something read
// or something else written (an empty range or NULL meets nothing).
struct Range {
  const void *p;
  size_t n;
};
inline bool meet(const Range &a, const Range &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && a.n && b.n && x < y + b.n && y < x + a.n;
}
inline bool clash(std::initializer_list<Range> out, std::initializer_list<Range> in) {
  for (const Range *o = out.begin(); o != out.end(); ++o) {
    for (const Range *q = o + 1; q != out.end(); ++q)
      if (meet(*o, *q)) return true;
    for (const Range &i : in)
      if (meet(*o, i)) return true;
  }
  return false;
}

// A runtime call's status.  The runtime also keeps a failed call's error, which the next
// launch check of the library would take for its own: it is cleared here.
inline tcq_status_t status_of(cudaError_t e) {
  if (e == cudaSuccess) return TCQ_OK;
  (void)cudaGetLastError();
  return TCQ_ERR_CUDA;
}

// cluster: blocks of a cluster along x (0: the kernel's own attribute, or none)
template <typename... P, typename... A>
inline tcq_status_t launch(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster,
                           cudaStream_t stream, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster ? 2 : 1;
  return status_of(cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...));
}

}  // namespace tcq_host
