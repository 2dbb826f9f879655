// Launches that overlap their start with the end of the work before them.
//
// A kernel launched with `launch` may become resident while the stream's
// previous kernel still runs (programmatic dependent launch): it sets up its
// barriers and tensor memory, then waits in after_previous() until that kernel
// is complete and its writes are visible, and only then touches global memory.
// let_next_start() allows the following kernel the same; it is called once every
// block is past its start.  A kernel before it that never calls it simply
// completes first.  Measured on 8-bit products of one token (8192 x 8192): 15.5 us
// a pass without, 14.5 with; on one quantised row 2.85 and 1.75.
#pragma once

#include <initializer_list>
#include <utility>

#include "tcq_device.cuh"

namespace tcq {

__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...) == cudaSuccess ? TCQ_OK : TCQ_ERR_CUDA;
}

}  // namespace tcq_host
