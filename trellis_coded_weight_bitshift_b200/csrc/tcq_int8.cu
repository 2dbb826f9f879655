// Row-wise int8 quantisation and the sliding-window decode to int8.
//
// quantize_int8: scale = max|row| / 127, q = x / scale to the nearest integer,
// ties to even.  The rounding is decided exactly: with q0 the rounded
// x * (1 / scale), off by at most one, r = fma(-q0, scale, x) is exact (it is a
// multiple of half an ulp of scale, or finer with a smaller x, and at most
// about half of scale), and |r| against scale / 2 says whether q0 stays.
// Rows below 2^-60 are first multiplied by 2^64 (exact), so that neither
// 1 / scale nor scale / 2 leaves the normal range.
//
// decode_int8: the 1MAD code is (bytesum - 510) / 147.8 [QTIP blog, "The
// codebook is computed"]; its numerator is a whole number of at most 483 in
// size at L = 8, 12 and 16, and a quarter of it fits 8 bits.
#include <algorithm>
#include <cuda_bf16.h>

#include "tcq_device.cuh"

namespace tcq {

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

struct RowScale {
  float up;      // 1 or 2^64: what x is multiplied by first
  float scale;   // of the multiplied row
  float inv, half;
};

// x / scale to the nearest integer, ties to even, as the low byte of the
// result's bits (1.5 * 2^23 + q keeps q in two's complement there).
__device__ __forceinline__ uint32_t quantize_one(float x, const RowScale &s) {
  constexpr float kMagic = 12582912.0f;
  x *= s.up;
  float u = __fadd_rn(__fmul_rn(x, s.inv), kMagic);
  const float q = __fsub_rn(u, kMagic);
  const float r = __fmaf_rn(-q, s.scale, x);
  if (fabsf(r) >= s.half) {
    const bool odd = __float_as_uint(u) & 1u;
    if (fabsf(r) > s.half || odd) u = __fadd_rn(u, copysignf(1.0f, r));
  }
  return __float_as_uint(u);
}

template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const T *__restrict__ x, int64_t cols,
                                                            int8_t *__restrict__ q,
                                                            float *__restrict__ scale) {
  __shared__ uint32_t part[8];
  const T *row = x + (int64_t)blockIdx.x * cols;
  uint32_t top = 0;                                   // bits of the largest |x|; a NaN is above infinity
  for (int64_t i = threadIdx.x; i < cols; i += 256)
    top = max(top, __float_as_uint(to_f32<T>(row[i])) & 0x7FFFFFFFu);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  top = 0;
  for (int w = 0; w < 8; ++w) top = max(top, part[w]);
  const float amax = __uint_as_float(top);
  const float sc = __fdiv_rn(amax, 127.0f);
  if (threadIdx.x == 0) scale[blockIdx.x] = top < 0x7F800000u ? sc : __uint_as_float(0x7FC00000u);
  int8_t *out = q + (int64_t)blockIdx.x * cols;
  if (top >= 0x7F800000u || sc == 0.0f) {
    for (int64_t i = threadIdx.x; i < cols; i += 256) out[i] = 0;
    return;
  }
  RowScale s;
  s.up = amax < 0x1p-60f ? 0x1p64f : 1.0f;
  s.scale = sc * s.up;
  s.inv = 1.0f / s.scale;
  s.half = 0.5f * s.scale;
  for (int64_t i = threadIdx.x; i < cols; i += 256) out[i] = (int8_t)quantize_one(to_f32<T>(row[i]), s);
}

// One thread per weight.
template <int L>
__global__ void __launch_bounds__(256) decode_int8_kernel(const uint32_t *__restrict__ bits,
                                                          int64_t n_weights, int T, int layout,
                                                          int wps, int tiles_c, int8_t *__restrict__ out) {
  for (int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; g < n_weights;
       g += (int64_t)gridDim.x * blockDim.x) {
    const int64_t seq = g / T;
    const int t = (int)(g - seq * T);
    const uint32_t *src = bits + seq * wps;
    const int i = t >> 4, o = 2 * (t & 15);
    const int i1 = i + 1 < wps ? i + 1 : 0;
    const uint32_t lo = i + 1 < wps || layout == TCQ_TAILBITING ? src[i1] : 0u;
    const uint32_t state = __funnelshift_l(lo, src[i], o) >> (32 - L);
    const int k = (int)one_mad_bytesum(state) - 510;
    int64_t at = g;
    if (tiles_c > 0) {
      const int64_t tr = seq / tiles_c, tc = seq - tr * tiles_c;
      at = (tr * 16 + (t >> 4)) * ((int64_t)tiles_c * 16) + tc * 16 + (t & 15);
    }
    out[at] = (int8_t)__float2int_rn(0.25f * (float)k);
  }
}

}  // namespace tcq

using namespace tcq;
using namespace tcq_host;

static bool size_ok(int64_t n) { return n < (1ll << 30); }

extern "C" tcq_status_t tcq_quantize_int8(const void *x, int dtype, int64_t rows, int64_t cols, int8_t *q,
                                          float *scale, void *stream) {
  if (dtype != TCQ_F16 && dtype != TCQ_BF16 && dtype != TCQ_F32) return TCQ_ERR_INVALID_ARG;
  if (rows < 0 || cols <= 0) return TCQ_ERR_INVALID_ARG;
  if (!size_ok(rows) || !size_ok(cols)) return TCQ_ERR_UNSUPPORTED;
  if (rows == 0) return TCQ_OK;
  if (!x || !q || !scale || !aligned16(x) || !aligned16(q) || !aligned16(scale)) return TCQ_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const unsigned blocks = (unsigned)rows;
  if (dtype == TCQ_F16)
    quantize_rows_kernel<<<blocks, 256, 0, s>>>((const __half *)x, cols, q, scale);
  else if (dtype == TCQ_BF16)
    quantize_rows_kernel<<<blocks, 256, 0, s>>>((const __nv_bfloat16 *)x, cols, q, scale);
  else
    quantize_rows_kernel<<<blocks, 256, 0, s>>>((const float *)x, cols, q, scale);
  return launch_status();
}

extern "C" tcq_status_t tcq_decode_int8(const tcq_trellis_t *tr, const uint32_t *bits, int64_t n_seq, int layout,
                                        int out_layout, int64_t rows, int64_t cols, int8_t *out, void *stream) {
  tcq_status_t st = check_trellis(tr);
  if (st != TCQ_OK) return st;
  if (layout != TCQ_TAILBITING && layout != TCQ_FREE_START) return TCQ_ERR_INVALID_ARG;
  if (out_layout != TCQ_OUT_SEQ && out_layout != TCQ_OUT_TILE16) return TCQ_ERR_INVALID_ARG;
  if (n_seq < 0) return TCQ_ERR_INVALID_ARG;
  const size_t wps = tcq_stream_words(tr, layout);
  if (wps == 0) return TCQ_ERR_UNSUPPORTED;
  const bool tiles = out_layout == TCQ_OUT_TILE16;
  if (tiles) {
    if (tr->seq_len != 256) return TCQ_ERR_UNSUPPORTED;
    if (rows <= 0 || cols <= 0 || rows % 16 || cols % 16) return TCQ_ERR_INVALID_ARG;
    if (!size_ok(rows) || !size_ok(cols)) return TCQ_ERR_UNSUPPORTED;
    if ((rows / 16) * (cols / 16) != n_seq) return TCQ_ERR_INVALID_ARG;
  }
  if (n_seq == 0) return TCQ_OK;
  if (!bits || !out || !aligned16(bits) || !aligned16(out)) return TCQ_ERR_INVALID_ARG;
  const int64_t nw = n_seq * tr->seq_len;
  const unsigned blocks = (unsigned)std::min<int64_t>((nw + 255) / 256, (int64_t)sm_count() * 32);
  const int tc = tiles ? (int)(cols / 16) : 0;
  cudaStream_t s = (cudaStream_t)stream;
  switch (tr->L) {
    case 8: decode_int8_kernel<8><<<blocks, 256, 0, s>>>(bits, nw, tr->seq_len, layout, (int)wps, tc, out); break;
    case 12: decode_int8_kernel<12><<<blocks, 256, 0, s>>>(bits, nw, tr->seq_len, layout, (int)wps, tc, out); break;
    default: decode_int8_kernel<16><<<blocks, 256, 0, s>>>(bits, nw, tr->seq_len, layout, (int)wps, tc, out); break;
  }
  return launch_status();
}
