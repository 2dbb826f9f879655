// Row-wise int8 quantisation and the sliding-window decode to int8.
//
// quantize_int8: scale = max|row| / 127, q = x / scale to the nearest integer,
// ties to even.  The rounding is decided exactly: with q0 the rounded
// x * (1 / scale), off by at most one, r = fma(-q0, scale, x) is exact (it is a
// multiple of half an ulp of scale, or finer with a smaller x, and at most
// about half of scale), and |r| against scale / 2 says whether q0 stays.
// Rows below 2^-60 are first multiplied by 2^64 (exact), so that neither
// 1 / scale nor scale / 2 leaves the normal range.  Among them are rows whose scale is a
// subnormal of fewer than 127 units of 2^-149: rounding max / 127 to so few digits can leave
// x / scale at 127.5 and more (190 units: scale 1), which is then +-127.
//   A row is read once: up to 4,096 bytes by one warp, up to 16,384 by a block,
// into registers (16 bytes a load), its largest value is found, and it is
// written; longer rows are read a second time.  Rows that start anywhere go through
// shared memory, whole aligned units on both sides.  Bound by HBM traffic, then by
// issue: about five instructions a value (maximum, conversion, one fma, one
// subtraction, one fma and a maximum for the check, byte packing; pairs where the
// hardware has them).  Only where the check of eight values fails are they decided one by
// one: a value lies that close to a border about once in 10^5.
//
// decode_int8: the 1MAD code is (bytesum - 510) / 147.8 [QTIP blog, "The
// codebook is computed"]; its numerator is a whole number of at most 483 in
// size at L = 8, 12 and 16, and a quarter of it fits 8 bits.  The byte sum is
// taken into the mantissa of 2^21 + (sum + 514) / 4 (an ulp of 1/4), and adding
// 1.5 * 2^23 - 2^21 - 256 rounds the quarter to nearest even and leaves q in
// the low byte: two instructions for sum, centring, division and rounding.
#include <algorithm>
#include <cuda_bf16.h>
#include <type_traits>

#include "tcq_launch.cuh"

namespace tcq {

constexpr float kRound = 12582912.0f;                   // 1.5 * 2^23: adding it rounds to a whole number

// x / scale to the nearest integer, ties to even, in the low byte of the
// result's bits (kRound + q keeps q in two's complement there).
__device__ __forceinline__ uint32_t quantize_exactly(float x, float scale, float inv) {
  float u = __fmaf_rn(x, inv, kRound);
  const float r = __fmaf_rn(-__fsub_rn(u, kRound), scale, x), half = 0.5f * scale;
  if (fabsf(r) > half || (fabsf(r) == half && (__float_as_uint(u) & 1u))) u = __fadd_rn(u, copysignf(1.0f, r));
  return __float_as_uint(u);
}

// The same bits with the integer held to -127 .. 127.
__device__ __forceinline__ uint32_t within_127(uint32_t u) {
  return __float_as_uint(fminf(fmaxf(__uint_as_float(u), kRound - 127.0f), kRound + 127.0f));
}

// N values (1, 4 or 8) of one thread, as they are loaded: raw words of type T.
template <typename T, int N> struct Values {
  static constexpr int kWords = (N * (int)sizeof(T) + 3) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T *p) {
    if (N == 1) {
      w[0] = sizeof(T) == 4 ? ld_u32(p) : (uint32_t)ld_u16(p);
    } else {
      const uint4 v = ld_u32x4(p);
      w[0] = v.x; w[1 % kWords] = v.y; w[2 % kWords] = v.z; w[3 % kWords] = v.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // The largest |value|'s bits so far (16-bit types: one maximum for each half of the word; a NaN stays).
  __device__ __forceinline__ uint32_t top(uint32_t t) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if (sizeof(T) == 4)
        t = max(t, w[i] & 0x7FFFFFFFu);
      else if (std::is_same<T, __half>::value)
        asm("{.reg .b32 a;\n abs.f16x2 a, %1;\n max.NaN.f16x2 %0, %0, a;}" : "+r"(t) : "r"(w[i]));
      else
        asm("{.reg .b32 a;\n abs.bf16x2 a, %1;\n max.NaN.bf16x2 %0, %0, a;}" : "+r"(t) : "r"(w[i]));
    }
    return t;
  }
  __device__ __forceinline__ float get(int i) const {
    if (sizeof(T) == 4) return __uint_as_float(w[i % kWords]);
    const uint32_t h = w[(i >> 1) % kWords];
    if (std::is_same<T, __half>::value)
      return __half2float(__ushort_as_half((unsigned short)((i & 1) ? h >> 16 : h)));
    return __uint_as_float((i & 1) ? h & 0xFFFF0000u : h << 16);
  }
};

template <typename T>
__device__ __forceinline__ uint32_t top_as_f32(uint32_t t) {
  if (sizeof(T) == 4) return t;
  const unsigned short h = (unsigned short)max(t & 0xFFFFu, t >> 16);
  return std::is_same<T, __half>::value ? __float_as_uint(__half2float(__ushort_as_half(h))) : (uint32_t)h << 16;
}

// UP: the values are multiplied by 2^64 first, and the results held to +-127 (other rows'
// quotients are within 127 (1 + 2^-23)).
template <typename T, int N, bool UP>
__device__ __forceinline__ void quantize_store(const Values<T, N> &v, float scale, float inv, int8_t *q) {
  float x[N], worst = 0.0f;
  uint32_t u[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = UP ? v.get(i) * 0x1p64f : v.get(i);
  if (N == 1) {
    u[0] = quantize_exactly(x[0], scale, inv);
    q[0] = (int8_t)(UP ? within_127(u[0]) : u[0]);
    return;
  }
#pragma unroll
  for (int i = 0; i < (N + 1) / 2; ++i) {
    const f2_t xx = f2(x[2 * i], x[(2 * i + 1) % N]);
    const f2_t uu = f2fma(xx, f2(inv, inv), f2(kRound, kRound));
    const f2_t rr = f2fma(f2sub(f2(kRound, kRound), uu), f2(scale, scale), xx);
    asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(worst) : "f"(f2lo(rr)), "f"(f2hi(rr)));
    u[2 * i] = __float_as_uint(f2lo(uu));
    u[(2 * i + 1) % N] = __float_as_uint(f2hi(uu));
  }
  if (worst >= 0.5f * scale) {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = quantize_exactly(x[i], scale, inv);
  }
  if (UP) {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = within_127(u[i]);
  }
  uint32_t b[(N + 3) / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    b[i] = __byte_perm(__byte_perm(u[4 * i], u[(4 * i + 1) % N], 0x0040), __byte_perm(u[(4 * i + 2) % N], u[(4 * i + 3) % N], 0x0040),
                       0x5410);
  if (N == 4) *reinterpret_cast<uint32_t *>(q) = b[0];
  else *reinterpret_cast<uint2 *>(q) = make_uint2(b[0], b[(N + 3) / 4 - 1]);
}

// One row by TPR threads (32 or 256 of the block's 256), KEEP loads of N values
// a thread kept in registers; what a longer row has beyond them is read twice.
// Six blocks an SM keep enough loads in flight (4096 x 8192 bf16, GPU time: 17.8
// us with the compiler's own 48 registers, 17.0 with six blocks, 23.9 with eight,
// which spill; 16.7 since the maxima take packed and three-operand instructions).
template <typename T, int N, int TPR, int KEEP>
__global__ void __launch_bounds__(256, TPR == 256 ? 6 : 4) quantize_rows_kernel(const T *x, int64_t rows, int64_t cols,
                                                            int8_t *__restrict__ q, float *__restrict__ scale) {
  __shared__ uint32_t part[8];
  after_previous();
  let_next_start();
  const int t = threadIdx.x % TPR;
  const int64_t r = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  if (TPR == 32 && r >= rows) return;                   // whole warps: no block barrier follows
  const T *row = x + r * cols;
  int8_t *out = q + r * cols;
  Values<T, N> v[KEEP], w;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int64_t c = ((int64_t)i * TPR + t) * N;
    if (c < cols) v[i].load(row + c);
    else v[i].zero();
  }
#pragma unroll
  for (int i = 0; i < KEEP; ++i) top = v[i].top(top);
  for (int64_t c = ((int64_t)KEEP * TPR + t) * N; c < cols; c += (int64_t)TPR * N) {
    w.load(row + c);
    top = w.top(top);
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top_as_f32<T>(top));
  if (TPR > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
    top = __reduce_max_sync(0xFFFFFFFFu, part[threadIdx.x & 7]);
  }
  // an infinity or NaN in the row: a NaN scale and zeros; no scale: zeros (x * 0 = 0 for every finite x)
  const float amax = __uint_as_float(top), sc = __fdiv_rn(amax, 127.0f);
  const bool fine = top < 0x7F800000u;
  if (t == 0) scale[r] = fine ? sc : __uint_as_float(0x7FC00000u);
  const bool small = amax < 0x1p-60f;
  const float by = small ? sc * 0x1p64f : sc;
  const float inv = fine && by > 0.0f ? 1.0f / by : 0.0f;
  if (!(inv > 0.0f)) {
    for (int64_t c = t; c < cols; c += TPR) out[c] = 0;
    return;
  }
  const auto write = [&](auto up) {
    constexpr bool kUp = decltype(up)::value;
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
      const int64_t c = ((int64_t)i * TPR + t) * N;
      if (c < cols) quantize_store<T, N, kUp>(v[i], by, inv, out + c);
    }
    for (int64_t c = ((int64_t)KEEP * TPR + t) * N; c < cols; c += (int64_t)TPR * N) {
      w.load(row + c);
      quantize_store<T, N, kUp>(w, by, inv, out + c);
    }
  };
  if (small) write(std::true_type());
  else write(std::false_type());
}

// The same for rows that start anywhere, a block a row of up to kAnyCols values:
// the aligned 16-byte units that cover the row are read (what lies outside it
// cleared), quantised to shared memory where a unit's place is aligned too, and
// written in aligned units of the output, shifted as they are read back.  The two
// units at the row's ends go by bytes.
constexpr int kAnyCols = 8192;

template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_any_kernel(const T *x, int64_t rows, int cols,
                                                                int8_t *__restrict__ q, float *__restrict__ scale) {
  constexpr int N = 16 / (int)sizeof(T), KEEP = kAnyCols / (256 * N) + 1;
  __shared__ __align__(16) int8_t row8[kAnyCols + 32];
  __shared__ uint32_t part[8];
  after_previous();
  let_next_start();
  const int t = threadIdx.x;
  const T *row = x + (int64_t)blockIdx.x * cols, *end = x + rows * cols;
  const int mis = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T)), units = (mis + cols + N - 1) / N;
  const T *base = row - mis;
  Values<T, N> v[KEEP];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int u = i * 256 + t;
    v[i].zero();
    if (u >= units) continue;
    const T *at = base + (int64_t)u * N;
    if (u > 0 && u < units - 1) {
      v[i].load(at);
    } else {                                             // the row's ends: its own values only
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int e = u * N + k - mis;
        if (e >= 0 && e < cols) {
          Values<T, 1> one;
          one.load(at + k);
          v[i].w[k * (int)sizeof(T) / 4] |= one.w[0] << (sizeof(T) == 2 ? 16 * (k & 1) : 0);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < KEEP; ++i) top = v[i].top(top);
  top = __reduce_max_sync(0xFFFFFFFFu, top_as_f32<T>(top));
  if ((t & 31) == 0) part[t >> 5] = top;
  __syncthreads();
  top = __reduce_max_sync(0xFFFFFFFFu, part[t & 7]);
  const float amax = __uint_as_float(top), sc = __fdiv_rn(amax, 127.0f);
  const bool fine = top < 0x7F800000u, small = amax < 0x1p-60f;
  if (t == 0) scale[blockIdx.x] = fine ? sc : __uint_as_float(0x7FC00000u);
  const float by = small ? sc * 0x1p64f : sc;
  const float inv = fine && by > 0.0f ? 1.0f / by : 0.0f;
  int8_t *out = q + (int64_t)blockIdx.x * cols;
  if (!(inv > 0.0f)) {
    for (int c = t; c < cols; c += 256) out[c] = 0;
    return;
  }
  const auto write = [&](auto up) {
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      if (i * 256 + t < units)
        quantize_store<T, N, decltype(up)::value>(v[i], by, inv, row8 + (i * 256 + t) * N);
  };
  if (small) write(std::true_type());
  else write(std::false_type());
  __syncthreads();
  const int off = (int)(reinterpret_cast<uintptr_t>(out) & 15u);
  for (int w = t; 16 * w < off + cols; w += 256) {
    const int b = 16 * w - off, from = b + mis;
    if (b >= 0 && b + 16 <= cols) {
      const uint32_t *p = reinterpret_cast<const uint32_t *>(row8) + (from >> 2);
      const uint32_t sh = 8 * (from & 3);
      *reinterpret_cast<uint4 *>(out + b) =
          make_uint4(__funnelshift_r(p[0], p[1], sh), __funnelshift_r(p[1], p[2], sh), __funnelshift_r(p[2], p[3], sh),
                     __funnelshift_r(p[3], p[4], sh));
    } else {
      for (int k = max(0, -b); k < 16 && b + k < cols; ++k) out[b + k] = row8[from + k];
    }
  }
}

// Two states' quarter numerators, each in the low byte of its half (the comment
// at the top).
__device__ __forceinline__ f2_t quarter_codes(uint32_t state0, uint32_t state1) {
  const uint32_t m0 = __dp4a(state0 * kLcgMul + kLcgAdd, 0x01010101u, 0x4A000000u + 514u);
  const uint32_t m1 = __dp4a(state1 * kLcgMul + kLcgAdd, 0x01010101u, 0x4A000000u + 514u);
  constexpr float kCentre = 12582912.0f - 2097152.0f - 256.0f;
  return f2add(f2(__uint_as_float(m0), __uint_as_float(m1)), f2(kCentre, kCentre));
}

// The sixteen weights whose windows start in word `hi`.  The 32 bits from
// position o on hold the window at o in their top and the one at o + 16 in the
// lower half, so one funnel shift serves two weights: 4.7 instructions a weight
// where one shift each took 5.75, and issue, not memory, bounds an 8192 x 8192
// matrix (16.9 us a pass so, 15.4 this way).
template <int L>
__device__ __forceinline__ uint4 decode16(uint32_t hi, uint32_t lo) {
  uint32_t u[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t f = __funnelshift_l(lo, hi, 2 * i);
    const f2_t c = quarter_codes(f >> (32 - L), (f >> (16 - L)) & ((1u << L) - 1u));
    u[i] = __float_as_uint(f2lo(c));
    u[i + 8] = __float_as_uint(f2hi(c));
  }
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    b[i] = __byte_perm(__byte_perm(u[4 * i], u[4 * i + 1], 0x0040), __byte_perm(u[4 * i + 2], u[4 * i + 3], 0x0040),
                       0x5410);
  return make_uint4(b[0], b[1], b[2], b[3]);
}

// One thread per 16 x 16 tile: its stream in registers, a row of it in one
// 16-byte store; a warp's stores cover 512 neighbouring bytes.
template <int L, int LAYOUT>
__global__ void __launch_bounds__(128) decode_int8_tiles_kernel(const uint32_t *bits, int64_t n_seq,
                                                                int tiles_c, int wps, int8_t *__restrict__ out) {
  after_previous();
  let_next_start();
  const int64_t seq = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (seq >= n_seq) return;
  const uint32_t *src = bits + seq * wps;
  uint32_t w[17];
  if (LAYOUT == TCQ_TAILBITING) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = ld_u32x4(src + 4 * i);
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
    w[16] = w[0];
  } else {
#pragma unroll
    for (int i = 0; i < 17; ++i) w[i] = ld_u32(src + i);
  }
  const int64_t tr = seq / tiles_c, tc = seq - tr * tiles_c, cols = (int64_t)tiles_c * 16;
  int8_t *dst = out + tr * 16 * cols + tc * 16;
#pragma unroll
  for (int r = 0; r < 16; ++r) *reinterpret_cast<uint4 *>(dst + r * cols) = decode16<L>(w[r], w[r + 1]);
}

// One thread per word of the stream, sixteen weights in sequence order (T a
// multiple of 16: one 16-byte store), the last word's fewer.
template <int L>
__global__ void __launch_bounds__(256) decode_int8_seq_kernel(const uint32_t *bits, int64_t n_items,
                                                              int per_seq, int T, int layout, int wps,
                                                              int8_t *__restrict__ out) {
  after_previous();
  let_next_start();
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < n_items; g += (int64_t)gridDim.x * 256) {
    const int64_t seq = g / per_seq;
    const int i = (int)(g - seq * per_seq);
    const uint32_t *src = bits + seq * wps;
    const uint32_t lo = i + 1 < wps ? ld_u32(src + i + 1) : layout == TCQ_TAILBITING ? ld_u32(src) : 0u;
    const uint4 v = decode16<L>(ld_u32(src + i), lo);
    int8_t *dst = out + seq * T + 16 * i;
    if (T % 16 == 0) {
      *reinterpret_cast<uint4 *>(dst) = v;
    } else {
      const uint32_t b[4] = {v.x, v.y, v.z, v.w};
      const int n = min(16, T - 16 * i);
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (k < n) dst[k] = (int8_t)(b[k >> 2] >> (8 * (k & 3)));
    }
  }
}

}  // namespace tcq

using namespace tcq;
using namespace tcq_host;

static bool size_ok(int64_t n) { return n < (1ll << 30); }

template <typename T, int N, int TPR, int KEEP>
static tcq_status_t quantize_launch(const T *x, int64_t rows, int64_t cols, int8_t *q, float *scale, cudaStream_t s) {
  const unsigned blocks = (unsigned)((rows + 256 / TPR - 1) / (256 / TPR));
  return launch(quantize_rows_kernel<T, N, TPR, KEEP>, dim3(blocks), 256, 0, 0, s, x, rows, cols, q, scale);
}

// Whole 16-byte loads where every row starts on such a boundary (4096 rows of bf16:
// 8192 values 16.7 us).  Else the kernel for rows that start anywhere (8191 values
// 25.0 us, one at a time 40.6; 4095: 17.8 and 22.0), but one value at a time for rows
// of up to 2,048 (1023: 8.9 us, by that kernel 10.3) and those it does not hold.  A
// warp a row while the row fits its registers, else a block: 4096 rows of 512 values
// 2.4 us by warps, 5.6 by blocks; 2048 values 5.1 and 7.3; 4096 values 13.8 and 11.0.
// (Sixteen rows of 2048: 2.2 and 1.4.)
template <typename T>
static tcq_status_t quantize_any(const T *x, int64_t rows, int64_t cols, int8_t *q, float *scale, cudaStream_t s) {
  constexpr int N = 16 / (int)sizeof(T);
  if (cols % N) {
    if (cols <= 256) return quantize_launch<T, 1, 32, 8>(x, rows, cols, q, scale, s);
    if (cols > 2048 && cols <= kAnyCols)
      return launch(quantize_rows_any_kernel<T>, dim3((unsigned)rows), 256, 0, 0, s, x, rows, (int)cols, q, scale);
    return quantize_launch<T, 1, 256, 8>(x, rows, cols, q, scale, s);
  }
  const int64_t loads = cols / N;
  if (loads <= 64) return quantize_launch<T, N, 32, 2>(x, rows, cols, q, scale, s);
  if (loads <= 256) return quantize_launch<T, N, 32, 8>(x, rows, cols, q, scale, s);
  if (loads <= 512) return quantize_launch<T, N, 256, 2>(x, rows, cols, q, scale, s);
  return quantize_launch<T, N, 256, 4>(x, rows, cols, q, scale, s);
}

extern "C" tcq_status_t tcq_quantize_int8(const void *x, int dtype, int64_t rows, int64_t cols, int8_t *q,
                                          float *scale, void *stream) {
  if (dtype != TCQ_F16 && dtype != TCQ_BF16 && dtype != TCQ_F32) return TCQ_ERR_INVALID_ARG;
  if (rows < 0 || cols <= 0) return TCQ_ERR_INVALID_ARG;
  if (!size_ok(rows) || !size_ok(cols)) return TCQ_ERR_UNSUPPORTED;
  if (rows == 0) return TCQ_OK;
  if (!x || !q || !scale || !aligned16(x) || !aligned16(q) || !aligned16(scale)) return TCQ_ERR_INVALID_ARG;
  const size_t n = (size_t)rows * cols;
  if (clash({{q, n}, {scale, 4 * (size_t)rows}}, {{x, n * (dtype == TCQ_F32 ? 4 : 2)}})) return TCQ_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == TCQ_F16) return quantize_any((const __half *)x, rows, cols, q, scale, s);
  if (dtype == TCQ_BF16) return quantize_any((const __nv_bfloat16 *)x, rows, cols, q, scale, s);
  return quantize_any((const float *)x, rows, cols, q, scale, s);
}

template <int L>
static tcq_status_t decode_launch(const tcq_trellis_t *tr, const uint32_t *bits, int64_t n_seq, int layout,
                                  int64_t cols, int8_t *out, int wps, cudaStream_t s) {
  if (cols) {
    const unsigned blocks = (unsigned)((n_seq + 127) / 128);
    return launch(layout == TCQ_TAILBITING ? decode_int8_tiles_kernel<L, TCQ_TAILBITING>
                                           : decode_int8_tiles_kernel<L, TCQ_FREE_START>,
                  dim3(blocks), 128, 0, 0, s, bits, n_seq, (int)(cols / 16), wps, out);
  }
  const int per_seq = (tr->seq_len + 15) / 16;
  const int64_t n = n_seq * per_seq;
  const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 1 << 30);
  return launch(decode_int8_seq_kernel<L>, dim3(blocks), 256, 0, 0, s, bits, n, per_seq, (int)tr->seq_len, layout, wps,
                out);
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
    if (n_seq > (1ll << 37)) return TCQ_ERR_UNSUPPORTED;     // blocks of 128 tiles: a grid's most
  }
  if (n_seq == 0) return TCQ_OK;
  if (!bits || !out || !aligned16(bits) || !aligned16(out)) return TCQ_ERR_INVALID_ARG;
  if (clash({{out, (size_t)n_seq * tr->seq_len}}, {{bits, 4 * wps * (size_t)n_seq}})) return TCQ_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  switch (tr->L) {
    case 8: return decode_launch<8>(tr, bits, n_seq, layout, tiles ? cols : 0, out, (int)wps, s);
    case 12: return decode_launch<12>(tr, bits, n_seq, layout, tiles ? cols : 0, out, (int)wps, s);
    default: return decode_launch<16>(tr, bits, n_seq, layout, tiles ? cols : 0, out, (int)wps, s);
  }
}
