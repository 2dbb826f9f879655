// The bounded waits of the matrix products, by themselves: a barrier that nothing
// arrives at, with a limit of milliseconds, and the accounting of the time.
#include "tcq_tensor.cuh"

using namespace tcq;

#define EXPORT extern "C" __attribute__((visibility("default")))

// Whether a wait that looks at the clock at these times is over at each of them.
EXPORT void waited(const unsigned long long *at, int n, unsigned long long limit, int *over) {
  Waited w(at[0]);
  for (int i = 1; i < n; ++i) over[i] = w.over(at[i], limit);
}

// Warp 0 waits for a barrier that nothing arrives at; warp 1 for another, with no limit to
// speak of: the block's flag ends it.  Warp 2's barrier is arrived at.
// out: for each warp, whether its wait was met, and how long it took; then the flag.
__global__ void wait_kernel(unsigned long long limit, unsigned long long *out) {
  __shared__ __align__(8) uint64_t bars[3];
  __shared__ volatile uint32_t stop;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    stop = 0;
    for (int i = 0; i < 3; ++i) mbar_init(smem_u32(bars + i), 1);
    mbar_init_fence();
  }
  __syncthreads();
  if (threadIdx.x == 64) mbar_expect(smem_u32(bars + 2), 0);
  if (threadIdx.x % 32 == 0) {
    const unsigned long long t0 = now_ns();
    out[2 * warp] = mbar_wait(smem_u32(bars + warp), 0, &stop, warp == 0 ? limit : kWaitNs);
    out[2 * warp + 1] = now_ns() - t0;
  }
  __syncthreads();
  if (threadIdx.x == 0) out[6] = stop;
}

EXPORT int wait_runs_out(unsigned long long limit, unsigned long long *out) {
  wait_kernel<<<1, 96>>>(limit, out);
  return (int)cudaDeviceSynchronize();
}

// A barrier that nothing arrives at, waited for as an aborted block does before it leaves.
__global__ void drain_kernel(unsigned long long *out) {
  __shared__ __align__(8) uint64_t bar;
  mbar_init(smem_u32(&bar), 1);
  mbar_init_fence();
  const unsigned long long t0 = now_ns();
  mbar_drain(smem_u32(&bar), 0);
  out[0] = now_ns() - t0;
}

EXPORT int drain_ends(unsigned long long *out) {
  drain_kernel<<<1, 1>>>(out);
  return (int)cudaDeviceSynchronize();
}

// A kernel that gave up says so, and what the next call sees: the count, whether there is
// a note, and whether there still is one.
__global__ void say_kernel(unsigned int *note) { say_gave_up(note); }

EXPORT int report(unsigned int *count, int *first, int *second) {
  unsigned int *const note = tcq_host::note_of_device();
  if (!note || tcq_host::take_note(note)) return -1;
  say_kernel<<<1, 1>>>(note);
  if (cudaDeviceSynchronize() != cudaSuccess) return -2;
  *first = tcq_host::take_note(note);
  *second = tcq_host::take_note(note);
  return (int)cudaMemcpyFromSymbol(count, g_gave_up, sizeof(unsigned));
}
