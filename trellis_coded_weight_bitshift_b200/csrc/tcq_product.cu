// Matrix products on decoded weights: int8 with token and channel scales, and
// the gated feed-forward block with its gradients.
//
// Plain tiles: a 256-thread block computes 32 x 32 results, four a thread,
// with 32-deep slices of both operands in shared memory.
#include <algorithm>
#include <cuda_bf16.h>

#include "tcq_activation.cuh"
#include "tcq_device.cuh"

namespace tcq {

template <typename T> struct Sum { typedef float type; };
template <> struct Sum<int8_t> { typedef int type; };
template <typename T> __device__ __forceinline__ typename Sum<T>::type widen(T v);
template <> __device__ __forceinline__ int widen<int8_t>(int8_t v) { return v; }
template <> __device__ __forceinline__ float widen<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// An operand's element (i, k) at p[i * si + k * sk].
template <typename T> struct Operand {
  const T *p;
  int64_t si, sk;
};

__device__ __forceinline__ void store(void *out, int64_t i, int dtype, float v) {
  if (dtype == TCQ_F16) ((__half *)out)[i] = __float2half_rn(v);
  else if (dtype == TCQ_BF16) ((__nv_bfloat16 *)out)[i] = __float2bfloat16_rn(v);
  else ((float *)out)[i] = v;
}

struct Out {
  void *out;
  int dtype, act;
  const float *a_scale, *s0, *s1, *bias;
  float *gate, *up;
};

// DUAL: both products share a0 and end in act(g) * u; else a1, b1 (if any) add
// to the same sums.
template <typename T, bool DUAL>
__global__ void __launch_bounds__(256) product_kernel(Operand<T> a0, Operand<T> b0, Operand<T> a1, Operand<T> b1,
                                                      int64_t M, int64_t N, int64_t K, Out o) {
  typedef typename Sum<T>::type S;
  __shared__ S as[32][33], bs[32][33], cs[32][33];
  const int64_t n0 = (int64_t)blockIdx.x * 32;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  for (int64_t m0 = (int64_t)blockIdx.y * 32; m0 < M; m0 += (int64_t)gridDim.y * 32) {
    S acc[4] = {}, acc2[4] = {};
    for (int seg = 0; seg < (!DUAL && b1.p ? 2 : 1); ++seg) {
      const Operand<T> a = seg ? a1 : a0, b = seg ? b1 : b0;
      for (int64_t k0 = 0; k0 < K; k0 += 32) {
        for (int r = ty; r < 32; r += 8) {
          const int64_t k = k0 + tx;
          as[r][tx] = m0 + r < M && k < K ? widen<T>(a.p[(m0 + r) * a.si + k * a.sk]) : S(0);
          bs[r][tx] = n0 + r < N && k < K ? widen<T>(b.p[(n0 + r) * b.si + k * b.sk]) : S(0);
          if (DUAL) cs[r][tx] = n0 + r < N && k < K ? widen<T>(b1.p[(n0 + r) * b1.si + k * b1.sk]) : S(0);
        }
        __syncthreads();
        for (int k = 0; k < 32; ++k)
          for (int j = 0; j < 4; ++j) {
            acc[j] += as[ty + 8 * j][k] * bs[tx][k];
            if (DUAL) acc2[j] += as[ty + 8 * j][k] * cs[tx][k];
          }
        __syncthreads();
      }
    }
    const int64_t n = n0 + tx;
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 8 * j;
      if (m >= M || n >= N) continue;
      float g = (float)acc[j], u = (float)acc2[j];
      if (o.a_scale) {
        g = g * o.a_scale[m] * o.s0[n];
        if (DUAL) u = u * o.a_scale[m] * o.s1[n];
      }
      if (o.bias) g = __fadd_rn(g, o.bias[n]);
      if (DUAL && o.gate) {
        o.gate[m * N + n] = g;
        o.up[m * N + n] = u;
      }
      store(o.out, m * N + n, o.dtype, DUAL ? activation(g, o.act) * u : g);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) gate_grad_kernel(const T *__restrict__ grad, const float *__restrict__ gate,
                                                        const float *__restrict__ up, int64_t n, int act,
                                                        T *__restrict__ dg, T *__restrict__ du) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    float a, d;
    activation_slope(gate[i], act, a, d);
    const float h = widen<T>(grad[i]);
    store(dg, i, sizeof(T) == 2 && std::is_same<T, __half>::value ? TCQ_F16 : TCQ_BF16, h * up[i] * d);
    store(du, i, sizeof(T) == 2 && std::is_same<T, __half>::value ? TCQ_F16 : TCQ_BF16, h * a);
  }
}

}  // namespace tcq

using namespace tcq;
using namespace tcq_host;

static bool size_ok(int64_t n) { return n < (1ll << 30); }

static bool aligned256(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

static tcq_status_t check_sizes(int64_t n_tok, int64_t n_out, int64_t n_in, int64_t most_in) {
  if (n_tok < 0 || n_out <= 0 || n_in <= 0) return TCQ_ERR_INVALID_ARG;
  if (!size_ok(n_tok) || !size_ok(n_out) || n_in > most_in) return TCQ_ERR_UNSUPPORTED;
  return TCQ_OK;
}

static bool bad_ptr(const void *p) { return !p || !aligned16(p); }

template <typename T, bool DUAL>
static tcq_status_t run_product(Operand<T> a0, Operand<T> b0, Operand<T> a1, Operand<T> b1, int64_t M, int64_t N,
                                int64_t K, const Out &o, cudaStream_t s) {
  const dim3 grid((unsigned)((N + 31) / 32), (unsigned)std::min<int64_t>((M + 31) / 32, 65535));
  product_kernel<T, DUAL><<<grid, 256, 0, s>>>(a0, b0, a1, b1, M, N, K, o);
  return launch_status();
}

extern "C" size_t tcq_int8_matmul_workspace_size(int64_t, int64_t, int64_t) { return 0; }
extern "C" size_t tcq_gated_ffn_workspace_size(int64_t, int64_t, int64_t) { return 0; }
extern "C" size_t tcq_int8_gated_ffn_workspace_size(int64_t, int64_t, int64_t) { return 0; }
extern "C" size_t tcq_gated_ffn_backward_workspace_size(int64_t n_tok, int64_t n_out, int64_t n_in) {
  if (check_sizes(n_tok, n_out, n_in, (1ll << 30) - 1) != TCQ_OK) return 0;
  return 2 * (((size_t)n_tok * n_out * 2 + 255) & ~(size_t)255);
}

extern "C" tcq_status_t tcq_int8_matmul(const int8_t *a, const float *a_scale, const int8_t *w, const float *w_scale,
                                        const float *bias, int64_t n_tok, int64_t n_out, int64_t n_in, void *out,
                                        int out_dtype, void *ws, size_t ws_bytes, void *stream) {
  if (out_dtype != TCQ_F16 && out_dtype != TCQ_BF16 && out_dtype != TCQ_F32) return TCQ_ERR_INVALID_ARG;
  tcq_status_t st = check_sizes(n_tok, n_out, n_in, 131071);
  if (st != TCQ_OK) return st;
  if (n_tok == 0) return TCQ_OK;
  if (bad_ptr(a) || bad_ptr(a_scale) || bad_ptr(w) || bad_ptr(w_scale) || bad_ptr(out) || !aligned16(bias))
    return TCQ_ERR_INVALID_ARG;
  Out o = {out, out_dtype, 0, a_scale, w_scale, nullptr, bias, nullptr, nullptr};
  Operand<int8_t> A = {a, n_in, 1}, W = {w, n_in, 1}, none = {nullptr, 0, 0};
  return run_product<int8_t, false>(A, W, none, none, n_tok, n_out, n_in, o, (cudaStream_t)stream);
}

extern "C" tcq_status_t tcq_int8_gated_ffn(const int8_t *a, const float *a_scale, const int8_t *w_gate,
                                           const float *w_gate_scale, const int8_t *w_up, const float *w_up_scale,
                                           int64_t n_tok, int64_t n_out, int64_t n_in, int act, void *h, int out_dtype,
                                           void *ws, size_t ws_bytes, void *stream) {
  if (out_dtype != TCQ_F16 && out_dtype != TCQ_BF16 && out_dtype != TCQ_F32) return TCQ_ERR_INVALID_ARG;
  if (act < TCQ_ACT_SILU || act > TCQ_ACT_RELU) return TCQ_ERR_INVALID_ARG;
  tcq_status_t st = check_sizes(n_tok, n_out, n_in, 131071);
  if (st != TCQ_OK) return st;
  if (n_tok == 0) return TCQ_OK;
  if (bad_ptr(a) || bad_ptr(a_scale) || bad_ptr(w_gate) || bad_ptr(w_gate_scale) || bad_ptr(w_up) ||
      bad_ptr(w_up_scale) || bad_ptr(h))
    return TCQ_ERR_INVALID_ARG;
  Out o = {h, out_dtype, act, a_scale, w_gate_scale, w_up_scale, nullptr, nullptr, nullptr};
  Operand<int8_t> A = {a, n_in, 1}, G = {w_gate, n_in, 1}, U = {w_up, n_in, 1};
  return run_product<int8_t, true>(A, G, A, U, n_tok, n_out, n_in, o, (cudaStream_t)stream);
}

template <typename T>
static tcq_status_t gated(const void *x, const void *wg, const void *wu, int dtype, int64_t M, int64_t F, int64_t K,
                          int act, void *h, float *gate, float *up, cudaStream_t s) {
  Out o = {h, dtype, act, nullptr, nullptr, nullptr, nullptr, gate, up};
  Operand<T> X = {(const T *)x, K, 1}, G = {(const T *)wg, K, 1}, U = {(const T *)wu, K, 1};
  return run_product<T, true>(X, G, X, U, M, F, K, o, s);
}

extern "C" tcq_status_t tcq_gated_ffn(const void *x, const void *w_gate, const void *w_up, int dtype, int64_t n_tok,
                                      int64_t n_out, int64_t n_in, int act, void *h, float *gate, float *up, void *ws,
                                      size_t ws_bytes, void *stream) {
  if (dtype != TCQ_F16 && dtype != TCQ_BF16) return TCQ_ERR_INVALID_ARG;
  if (act < TCQ_ACT_SILU || act > TCQ_ACT_RELU) return TCQ_ERR_INVALID_ARG;
  tcq_status_t st = check_sizes(n_tok, n_out, n_in, (1ll << 30) - 1);
  if (st != TCQ_OK) return st;
  if (!gate != !up) return TCQ_ERR_INVALID_ARG;
  if (n_tok == 0) return TCQ_OK;
  if (bad_ptr(x) || bad_ptr(w_gate) || bad_ptr(w_up) || bad_ptr(h) || !aligned16(gate) || !aligned16(up))
    return TCQ_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  return dtype == TCQ_F16 ? gated<__half>(x, w_gate, w_up, dtype, n_tok, n_out, n_in, act, h, gate, up, s)
                          : gated<__nv_bfloat16>(x, w_gate, w_up, dtype, n_tok, n_out, n_in, act, h, gate, up, s);
}

template <typename T>
static tcq_status_t gated_backward(const void *x, const void *wg, const void *wu, const float *gate, const float *up,
                                   const void *grad, int dtype, int64_t M, int64_t F, int64_t K, int act, void *gx,
                                   void *gwg, void *gwu, void *ws, cudaStream_t s) {
  T *dg = (T *)ws;
  T *du = (T *)((char *)ws + (((size_t)M * F * 2 + 255) & ~(size_t)255));
  const int64_t n = M * F;
  gate_grad_kernel<T><<<(unsigned)std::min<int64_t>((n + 255) / 256, (int64_t)sm_count() * 16), 256, 0, s>>>(
      (const T *)grad, gate, up, n, act, dg, du);
  tcq_status_t st = launch_status();
  if (st != TCQ_OK) return st;
  Out o = {nullptr, dtype, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
  const Operand<T> none = {nullptr, 0, 0};
  if (gx) {
    o.out = gx;
    Operand<T> A = {dg, F, 1}, B = {(const T *)wg, 1, K}, A2 = {du, F, 1}, B2 = {(const T *)wu, 1, K};
    st = run_product<T, false>(A, B, A2, B2, M, K, F, o, s);
  }
  for (int i = 0; i < 2 && st == TCQ_OK; ++i) {
    o.out = i ? gwu : gwg;
    if (!o.out) continue;
    Operand<T> A = {i ? du : dg, 1, F}, B = {(const T *)x, 1, K};
    st = run_product<T, false>(A, B, none, none, F, K, M, o, s);
  }
  return st;
}

extern "C" tcq_status_t tcq_gated_ffn_backward(const void *x, const void *w_gate, const void *w_up, const float *gate,
                                               const float *up, const void *grad_h, int dtype, int64_t n_tok,
                                               int64_t n_out, int64_t n_in, int act, void *grad_x, void *grad_w_gate,
                                               void *grad_w_up, void *ws, size_t ws_bytes, void *stream) {
  if (dtype != TCQ_F16 && dtype != TCQ_BF16) return TCQ_ERR_INVALID_ARG;
  if (act < TCQ_ACT_SILU || act > TCQ_ACT_RELU) return TCQ_ERR_INVALID_ARG;
  tcq_status_t st = check_sizes(n_tok, n_out, n_in, (1ll << 30) - 1);
  if (st != TCQ_OK) return st;
  if (!aligned16(grad_x) || !aligned16(grad_w_gate) || !aligned16(grad_w_up)) return TCQ_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (n_tok == 0) {                                   // no token: the weights' gradients are zero
    for (void *g : {grad_w_gate, grad_w_up})
      if (g && cudaMemsetAsync(g, 0, (size_t)n_out * n_in * 2, s) != cudaSuccess) return TCQ_ERR_CUDA;
    return TCQ_OK;
  }
  if (bad_ptr(x) || bad_ptr(w_gate) || bad_ptr(w_up) || bad_ptr(gate) || bad_ptr(up) || bad_ptr(grad_h))
    return TCQ_ERR_INVALID_ARG;
  if (!grad_x && !grad_w_gate && !grad_w_up) return TCQ_OK;
  if (!ws || !aligned256(ws) || ws_bytes < tcq_gated_ffn_backward_workspace_size(n_tok, n_out, n_in))
    return TCQ_ERR_WORKSPACE;
  return dtype == TCQ_F16 ? gated_backward<__half>(x, w_gate, w_up, gate, up, grad_h, dtype, n_tok, n_out, n_in, act,
                                                   grad_x, grad_w_gate, grad_w_up, ws, s)
                          : gated_backward<__nv_bfloat16>(x, w_gate, w_up, gate, up, grad_h, dtype, n_tok, n_out, n_in,
                                                          act, grad_x, grad_w_gate, grad_w_up, ws, s);
}
