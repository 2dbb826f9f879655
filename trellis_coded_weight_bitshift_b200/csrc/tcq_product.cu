// Matrix products on decoded weights: int8 with token and channel scales, and
// the gated feed-forward block with its gradients.
//
// pair_kernel: persistent, two blocks of a cluster (two SMs) work on one tile
// of 256 x 256 results.  Each block loads its 128 rows of A and its half of B
// (128 rows) by tensor-map loads into a ring of 32 KB stages; one thread of the
// first block issues tcgen05.mma for the pair (M = 256, N = 256, 32 bytes of the
// contraction each); the sums stay in tensor memory, two tiles of them (2 x 256
// columns), so that eight warps a block write one tile out while the next is
// computed.  In the gated block the halves of B are 128 channels of Wg and the
// same 128 of Wu: both projections of a result lie in one thread's tensor-memory
// lane, and act(g) * u needs no exchange.
//
// Why this split: a 256 x 256 tile reads 64 KB of operands for each 64-deep
// 16-bit step (8 MFLOP), which neither the shared-memory port (64 of 128 bytes a
// clock) nor L2 limits; a 128 x 128 tile of one block would need all of the port.
//
// Measured (steady loop): int8 3001 x 8192 x 8192 151 us (2.66 POP/s), gated block
// 3001 x 2048 x 8192 bf16 152 us (1.33 PFLOP/s; the library's product of the same
// projections without the gate 162), the three gradients of 4096 x 2048 x 8192 374 us
// (1.47 PFLOP/s).  The tensor pipe is busy 89 to 95% of the active cycles (70% where a
// tile has only 16 steps) and the clock falls to 1.5 to 1.65 GHz: power bounds them.
#include <algorithm>
#include <cuda_bf16.h>

#include "tcq_activation.cuh"
#include "tcq_launch.cuh"
#include "tcq_tensor.cuh"

namespace tcq {

constexpr int kStages = 6, kStageBytes = 32768, kPairThreads = 320;
// the ring; for each of the eight epilogue warps 32 rows of 16 + 1 values and two
// scales (or a scale and a bias) for each of its 128 columns
constexpr int kStagePitch = 17, kWarpFloats = 32 * kStagePitch + 256;
constexpr int kPairSmem = kStages * kStageBytes + 8 * kWarpFloats * 4 + 1024;

// One product: sums over `segs` pairs of operands a[s], b[s] in turn, or (z > 1)
// z products with operands a[z] and the same b[0].
struct Job {
  CUtensorMap a[2], b[2], b_half[2];   // b_half: 64-row boxes, for narrow tiles of a K-major b
  void *out[2];
  int64_t M, N;        // results of one product
  int mt, nt;          // tiles of it
  int band;            // row tiles of a band
  int split;           // parts of the contraction; with more than one, raw sums go to `part`
  int planes;          // of `part`, [split][planes][M][pitch]: gate and up, or the z products
  int64_t pitch;
  float *part;
  int kb, segs;        // steps of one segment
  int z;
  int a_mn, b_mn;      // operand stored with its rows along the contraction
  int wide;            // bytes of a store: 32, 16 or one element
};

// Tiles [lo, hi) of a job, dealt in turn to clusters first .. first + n - 1.  A
// narrow share deals half tiles (256 x 128): lo and hi count those.
struct Share {
  int job, first, n, narrow;
  uint32_t lo, hi;
};

struct Epilogue {
  int dtype, act;
  const float *a_scale, *s0, *s1, *bias;
  float *gate, *up;
  int wide_save;
};

struct PairParams {
  Job job[2];
  Share share[5];
  int shares;
  int bf16;
  unsigned int *note;
  Epilogue e;
};

// The tiles of one cluster, in order.
struct Tiles {
  int s;
  uint32_t t;
  __device__ __forceinline__ Tiles() : s(-1), t(0) {}
  __device__ __forceinline__ bool next(const PairParams &p, int cluster) {
    if (s >= 0) {
      t += p.share[s].n;
      if (t < p.share[s].hi) return true;
    }
    while (++s < p.shares) {
      const int c = cluster - p.share[s].first;
      t = p.share[s].lo + (uint32_t)c;
      if (c >= 0 && c < p.share[s].n && t < p.share[s].hi) return true;
    }
    return false;
  }
};

// A tile: product z, row tile m, n half tiles of columns, steps [k0, k1) of the
// contraction as its part s.
struct Place {
  int z, m, n, s, k0, k1;
  // Tiles go by bands of rows, rows first, so that clusters at work share operands
  // in L2.  All in 32 bits (the host sees to it): 64-bit divisions took a
  // microsecond of every launch.
  __device__ __forceinline__ Place(const Job &j, uint32_t t, int narrow) {
    const uint32_t steps = (uint32_t)(j.kb * j.segs), split = (uint32_t)j.split;
    s = 0;
    k0 = 0;
    k1 = (int)steps;
    if (split > 1) {
      s = (int)(t % split);
      t /= split;
      k0 = (int)(steps * (uint32_t)s / split);
      k1 = (int)(steps * (uint32_t)(s + 1) / split);
    }
    uint32_t r = narrow ? t >> 1 : t;
    z = 0;
    if (j.z > 1 && r >= (uint32_t)(j.mt * j.nt)) {
      r -= (uint32_t)(j.mt * j.nt);
      z = 1;
    }
    const uint32_t per = (uint32_t)(j.band * j.nt), band = r / per, in = r - band * per;
    const uint32_t rows = min((uint32_t)j.band, (uint32_t)j.mt - band * j.band);
    m = (int)(band * j.band + in % rows);
    n = 2 * (int)(in / rows) + (narrow ? (int)(t & 1) : 0);
  }
};

__device__ __forceinline__ uint32_t pack2(float a, float b, int dtype) {
  if (dtype == TCQ_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void store32(void *p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ void store_words(char *p, const uint32_t (&v)[8], int wide) {
  if (wide == 32) {
    store32(p, v);
  } else {
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// Sixteen neighbouring results of one row (`wide` 16 or 32: bytes of a store).
__device__ __forceinline__ void store16(void *out, int64_t at, int dtype, const float (&v)[16], int wide) {
  uint32_t w[8];
  if (dtype == TCQ_F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * h + i]);
      store_words((char *)out + 4 * at + 32 * h, w, wide);
    }
    return;
  }
  if (dtype == TCQ_F16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack2(v[2 * i], v[2 * i + 1], TCQ_F16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack2(v[2 * i], v[2 * i + 1], TCQ_BF16);
  }
  store_words((char *)out + 2 * at, w, wide);
}

// The same for a whole warp's 32 rows where rows start anywhere or the matrix
// ends inside the sixteen: through shared memory, so that half a warp writes
// neighbouring values of one row (element stores of a lane's own row would touch
// 32 sectors each: the gated block 777 x 1024 x 2731 took 39.8 us so, 19.5 this way).
__device__ __noinline__ void store_rows(const float *buf, void *out, int64_t at, int rows, int64_t N, int valid,
                                        int dtype) {
  const int lane = threadIdx.x & 31, c = lane & 15;
  if (c >= valid) return;
#pragma unroll 4
  for (int r = lane >> 4; r < rows; r += 2) {
    const float x = buf[r * kStagePitch + c];
    const int64_t to = at + r * N + c;
    if (dtype == TCQ_F32) ((float *)out)[to] = x;
    else ((uint16_t *)out)[to] = (uint16_t)pack2(x, 0.0f, dtype);
  }
}
__device__ __forceinline__ void store16_staged(float *buf, void *out, int64_t row0, int64_t M, int64_t N, int64_t ch,
                                               int valid, int dtype, const float (&v)[16]) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 16; ++i) buf[(threadIdx.x & 31) * kStagePitch + i] = v[i];
  __syncwarp();
  store_rows(buf, out, row0 * N + ch, (int)max((int64_t)0, min((int64_t)32, M - row0)), N, valid, dtype);
}

// Int32 sums to fp32, times the token's scale and the channels' (sixteen floats in
// shared memory).
__device__ __forceinline__ void scale16(float (&v)[16], const float *c, float sa) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 q = *reinterpret_cast<const float4 *>(c + i);
    const f2_t r = f2mul(f2mul(f2((float)__float_as_int(v[i]), (float)__float_as_int(v[i + 1])), f2(sa, sa)), f2(q.x, q.y));
    const f2_t t = f2mul(f2mul(f2((float)__float_as_int(v[i + 2]), (float)__float_as_int(v[i + 3])), f2(sa, sa)), f2(q.z, q.w));
    v[i] = f2lo(r);
    v[i + 1] = f2hi(r);
    v[i + 2] = f2lo(t);
    v[i + 3] = f2hi(t);
  }
}

template <bool I8, bool DUAL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_kernel(const __grid_constant__ PairParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 4];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t stop;
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                 acc_empty = acc_full + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    stop = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, 16);                  // eight warps in each block
    }
    mbar_init_fence();
  }
  // An instruction of the pair needs both blocks there, from allocation to release: a block that
  // allocated before the other had started left that one waiting in its own allocation for good
  // (one training step in some thousands, behind the elementwise kernel, whose blocks delay one
  // of the two).
  __syncwarp();
  cluster_sync();
  if (warp == 1) tmem_alloc_pair(smem_u32(&tmem_slot), 512);
  tmem_fence_before_sync();
  __syncthreads();
  cluster_sync();
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  after_previous();
  let_next_start();

  if (warp == 0 && lane == 0) {
    // ---- loads: this block's rows of A and half of B, counted by the first block's barrier
    fence_before_loads();
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    Tiles it;
    while (ok && it.next(p, cluster)) {
      const int narrow = p.share[it.s].narrow;
      const Job &j = p.job[p.share[it.s].job];
      const Place at(j, it.t, narrow);
      const int row = at.m * 256 + (int)rank * 128;
      const int col = DUAL ? at.n * 64 : at.n * 128 + (int)rank * (narrow ? 64 : 128);
      const CUtensorMap *bs = narrow && !j.b_mn ? j.b_half : j.b;
      const uint32_t bytes = narrow ? 2 * kStageBytes - 16384 : 2 * kStageBytes;
      for (int kb = at.k0; kb < at.k1; ++kb) {
        if (!mbar_wait(empty + 8 * s, ph ^ 1, &stop)) { ok = false; break; }
        const int seg = kb >= j.kb ? 1 : 0;
        const int k = (kb - seg * j.kb) * (I8 ? 128 : 64);
        const uint32_t bar = map_to_rank(full + 8 * s, 0);
        const uint32_t a = ring + s * kStageBytes, b = a + 16384;
        if (rank == 0) mbar_expect(full + 8 * s, bytes);
        const CUtensorMap *am = &j.a[seg + at.z], *bm = bs + (DUAL ? rank : seg);
        if (!j.a_mn) {
          tma_load_pair(a, am, k, row, bar);
        } else {
          tma_load_pair(a, am, row, k, bar);
          tma_load_pair(a + 8192, am, row + 64, k, bar);
        }
        if (!j.b_mn) {
          tma_load_pair(b, bm, k, col, bar);
        } else {
          tma_load_pair(b, bm, col, k, bar);
          if (!narrow) tma_load_pair(b + 8192, bm, col + 64, k, bar);
        }
        if (++s == kStages) { s = 0; ph ^= 1; }
      }
    }
    if (ok) {
      // the last products' releases arrive while this block is still there
      for (int i = 0; i < kStages && ok; ++i) {
        ok = mbar_wait(empty + 8 * s, ph ^ 1, &stop);
        if (++s == kStages) { s = 0; ph ^= 1; }
      }
    } else if (rank == 0) {
      // gave up: the copies in flight land first (each wait limited)
      for (int i = 0; i < kStages; ++i) {
        s = s ? s - 1 : kStages - 1;
        if (s == kStages - 1) ph ^= 1;
        mbar_drain(full + 8 * s, ph);
      }
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- products
    int s = 0, n_acc = 0;
    uint32_t ph = 0;
    bool ok = true;
    Tiles it;
    while (ok && it.next(p, cluster)) {
      const Job &j = p.job[p.share[it.s].job];
      const int buf = n_acc & 1;
      if (!mbar_wait(acc_empty + 8 * buf, ((n_acc >> 1) & 1) ^ 1, &stop)) { ok = false; break; }
      tmem_fence_after_sync();
      const uint32_t d = tmem + buf * 256;
      const int w = p.share[it.s].narrow ? 128 : 256;
      const uint32_t instr = I8 ? instr_i8(256, w) : instr_f16(256, w, p.bf16, j.a_mn, j.b_mn);
      const uint32_t a_step = j.a_mn ? 2048 >> 4 : 32 >> 4, b_step = j.b_mn ? 2048 >> 4 : 32 >> 4;
      const Place place(j, it.t, p.share[it.s].narrow);
      for (int kb = place.k0; kb < place.k1; ++kb) {
        if (!mbar_wait(full + 8 * s, ph, &stop)) { ok = false; break; }
        tmem_fence_after_sync();
        const uint32_t at = ring + s * kStageBytes;
        uint64_t a = operand_desc(at, j.a_mn), b = operand_desc(at + 16384, j.b_mn);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mma<I8, true>(d, a, b, instr, kb > place.k0 || i > 0);
          a += a_step;
          b += b_step;
        }
        mma_commit_pair(empty + 8 * s);
        if (++s == kStages) { s = 0; ph ^= 1; }
      }
      mma_commit_pair(acc_full + 8 * buf);
      ++n_acc;
    }
    // gave up: the products issued so far end first (the last commit covers them all)
    if (!ok && n_acc > 0) mbar_drain(acc_full + 8 * ((n_acc - 1) & 1), ((n_acc - 1) >> 1) & 1);
  } else if (warp >= 2) {
    // ---- results: warp w reads the lanes of quarter w % 4, one half of the columns
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    float *scales = reinterpret_cast<float *>(raw + (ring - smem_u32(raw)) + kStages * kStageBytes) +
                    (warp - 2) * kWarpFloats, *stage = scales + 256;
    int n_acc = 0;
    Tiles it;
    while (it.next(p, cluster)) {
      const int narrow = p.share[it.s].narrow;
      const Job &j = p.job[p.share[it.s].job];
      const Place at(j, it.t, narrow);
      const int buf = n_acc & 1;
      const int64_t row = (int64_t)at.m * 256 + rank * 128 + quarter * 32 + lane;
      const bool in = row < j.M;
      const int chunks = (DUAL ? 4 : 8) >> narrow, col0 = half * chunks * 16, up0 = narrow ? 64 : 128;
      const int64_t n0 = (int64_t)at.n * (DUAL ? 64 : 128) + col0;
      const float sa = I8 && in ? ld_f32(p.e.a_scale + row) : 1.0f;
      if (I8) {
        // the columns' scales, while the products run: read chunk by chunk from L2 they took most of
        // the epilogue (8-bit gated block 2048 x 2048 x 8192: 61.1 us so, 58.7 this way)
        const float *second = DUAL ? p.e.s1 : p.e.bias;
        __syncwarp();
        for (int i = lane; i < 16 * chunks; i += 32) {
          const bool there = n0 + i < j.N;
          scales[i] = there ? ld_f32(p.e.s0 + n0 + i) : 0.0f;
          scales[128 + i] = there && second ? ld_f32(second + n0 + i) : 0.0f;
        }
      }
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(acc_full + 8 * buf, (n_acc >> 1) & 1, &stop))) break;
      tmem_fence_after_sync();
      const uint32_t t0 = tmem + buf * 256 + ((uint32_t)quarter << 21) + col0;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        float g[16], u[16];
        __syncwarp();                                    // rows past the end skipped the last stores
        tmem_ld16(t0 + 16 * c, g);
        if (DUAL) tmem_ld16(t0 + up0 + 16 * c, u);
        tmem_wait16(g);
        if (DUAL) tmem_wait16(u);
        if (c == chunks - 1) {                           // the tile's sums are in registers: the buffer is free
          tmem_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_at(acc_empty + 8 * buf, 0);
        }
        const int64_t ch = n0 + 16 * c;
        const int valid = (int)min((int64_t)16, j.N - ch);
        if (valid <= 0) continue;
        if (j.split > 1) {
          if (!in) continue;
          float *part = j.part + (((int64_t)at.s * j.planes + (DUAL ? 0 : at.z)) * j.M + row) * j.pitch + ch;
          store16(part, 0, TCQ_F32, g, 32);
          if (DUAL) store16(part + j.M * j.pitch, 0, TCQ_F32, u, 32);
          continue;
        }
        const int64_t to = row * j.N + ch, row0 = row - lane;
        if (I8) scale16(g, scales + 16 * c, sa);
        if (DUAL) {
          if (I8) scale16(u, scales + 128 + 16 * c, sa);
          if (!I8 && p.e.gate) {
            if (valid == 16 && p.e.wide_save >= 16) {
              if (in) {
                store16(p.e.gate, to, TCQ_F32, g, p.e.wide_save);
                store16(p.e.up, to, TCQ_F32, u, p.e.wide_save);
              }
            } else {
              store16_staged(stage, p.e.gate, row0, j.M, j.N, ch, valid, TCQ_F32, g);
              store16_staged(stage, p.e.up, row0, j.M, j.N, ch, valid, TCQ_F32, u);
            }
          }
          gate(g, u, p.e.act);
        } else if (I8 && p.e.bias) {
#pragma unroll
          for (int i = 0; i < 16; ++i) g[i] = __fadd_rn(g[i], scales[128 + 16 * c + i]);
        }
        if (valid == 16 && j.wide >= 16) {
          if (in) store16(j.out[at.z], to, p.e.dtype, g, j.wide);
        } else {
          store16_staged(stage, j.out[at.z], row0, j.M, j.N, ch, valid, p.e.dtype, g);
        }
      }
      ++n_acc;
    }
  }
  __syncwarp();
  tmem_fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
  __syncwarp();
  cluster_sync();                                        // neither leaves before both have released
  if (threadIdx.x == 0 && stop) say_gave_up(p.note);
}

// ---- few tokens: the weights on the M side
struct RowsParams {
  CUtensorMap w[2], x;
  int64_t M, N;
  int kb, bf16, wide4;
  void *out;
  unsigned int *note;
  Epilogue e;
};

template <bool DUAL, int NT> struct RowsShape {
  static constexpr int kWeightBytes = DUAL ? 32768 : 16384, kStage = kWeightBytes + NT * 128;
  // two blocks an SM where four stages and more fit twice (three of the dual ones), else one
  static constexpr int kDepth = DUAL ? (NT <= 32 ? 3 : 5) : (NT == 16 ? 6 : NT == 32 ? 5 : NT == 64 ? 4 : 3);
  static constexpr int kBlocksPerSm = DUAL && NT == 64 ? 1 : 2;
  static constexpr int kCols = DUAL ? 2 * NT : NT, kTmem = kCols < 32 ? 32 : kCols;
  static constexpr int kSmem = kDepth * kStage + 1024;
  static_assert(kCols * 512 <= kDepth * kStage, "the partial sums reuse the ring");
};

__device__ __forceinline__ void add4(float4 &s, const float4 &v, bool i8) {
  if (i8) {
    s.x = __int_as_float(__float_as_int(s.x) + __float_as_int(v.x));
    s.y = __int_as_float(__float_as_int(s.y) + __float_as_int(v.y));
    s.z = __int_as_float(__float_as_int(s.z) + __float_as_int(v.z));
    s.w = __int_as_float(__float_as_int(s.w) + __float_as_int(v.w));
  } else {
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
}

// Four neighbouring channels of a token: sums to results.  Scales that were read
// before come in `sa`, `c0` and `c1` (the up projection's, or the bias).
template <bool I8, bool DUAL>
__device__ __forceinline__ void finish4(const Epilogue &e, const float4 &g, const float4 &u, int64_t row, int64_t N,
                                        int64_t ch, int valid, bool wide, void *out, const float *sa,
                                        const float (&c0)[4], const float (&c1)[4]) {
  float gv[4] = {g.x, g.y, g.z, g.w}, uv[4] = {u.x, u.y, u.z, u.w};
  const int64_t at = row * N + ch;
  if (I8) {
    const float s = sa ? *sa : ld_f32(e.a_scale + row);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= valid) continue;
      gv[k] = (float)__float_as_int(gv[k]) * s * (sa ? c0[k] : ld_f32(e.s0 + ch + k));
      if (DUAL) uv[k] = (float)__float_as_int(uv[k]) * s * (sa ? c1[k] : ld_f32(e.s1 + ch + k));
      else if (e.bias) gv[k] = __fadd_rn(gv[k], sa ? c1[k] : ld_f32(e.bias + ch + k));
    }
  }
  if (DUAL) {
    if (!I8 && e.gate) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k >= valid) continue;
        e.gate[at + k] = gv[k];
        e.up[at + k] = uv[k];
      }
    }
    gate(gv, uv, e.act);
  }
  if (valid == 4 && wide) {
    if (e.dtype == TCQ_F32)
      *reinterpret_cast<float4 *>((float *)out + at) = make_float4(gv[0], gv[1], gv[2], gv[3]);
    else
      *reinterpret_cast<uint2 *>((uint16_t *)out + at) =
          make_uint2(pack2(gv[0], gv[1], e.dtype), pack2(gv[2], gv[3], e.dtype));
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= valid) continue;
      if (e.dtype == TCQ_F32) ((float *)out)[at + k] = gv[k];
      else ((uint16_t *)out)[at + k] = (uint16_t)pack2(gv[k], 0.0f, e.dtype);
    }
  }
}

// Adds the parts of a split product in order and finishes them, four channels a
// thread; blockIdx.z: the product.  The parts come from L2; about 3 us with its launch
// for a few MB of sums.
struct Join {
  const float *part;
  int split, planes, wide4;
  int64_t M, N, pitch;
  void *out[2];
  Epilogue e;
};

template <bool I8, bool DUAL>
__global__ void __launch_bounds__(256) join_kernel(const Join p) {
  after_previous();
  let_next_start();
  const int64_t quads = (p.N + 3) / 4;
  const int z = blockIdx.z;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.M * quads; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / quads, ch = (i - row * quads) * 4;
    float4 g = make_float4(0, 0, 0, 0), u = g;
    const float *at = p.part + ((int64_t)z * p.M + row) * p.pitch + ch;
    const int64_t plane = p.M * p.pitch, part = plane * p.planes;
    // four parts' loads at a time: one after the other their latencies would add up
    for (int s = 0; s < p.split; s += 4) {
      float4 a[4], b[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool there = s + k < p.split;
        a[k] = there ? ld_f32x4(at + (s + k) * part) : make_float4(0, 0, 0, 0);
        if (DUAL) b[k] = there ? ld_f32x4(at + (s + k) * part + plane) : make_float4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        add4(g, a[k], I8);
        if (DUAL) add4(u, b[k], I8);
      }
    }
    const float none[4] = {};
    finish4<I8, DUAL>(p.e, g, u, row, p.N, ch, (int)min((int64_t)4, p.N - ch), p.wide4, p.out[z], nullptr, none,
                      none);
  }
}

// y^T = W x^T for few tokens.  A cluster works on 128 channels (the products' M side,
// so that no lane of the tensor memory is idle with one token) by NT tokens; its blocks
// split the contraction and add their sums through distributed shared memory, in order.
// Bound by HBM: one int8 token against 8192 x 8192 takes 13.1 us, of which the 67 MB
// stream for 9.4 (7.1 TB/s); the first load's latency, the join and the launch are the
// rest.  Three blocks an SM with shallower rings: 13.7 to 13.9.
template <bool I8, bool DUAL, int NT>
__global__ void __launch_bounds__(192, RowsShape<DUAL, NT>::kBlocksPerSm)
    rows_kernel(const __grid_constant__ RowsParams p) {
  typedef RowsShape<DUAL, NT> Sh;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2 * Sh::kDepth + 1];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t stop;
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t full = smem_u32(bars), empty = full + 8 * Sh::kDepth, acc_full = empty + 8 * Sh::kDepth;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = (int)cluster_size(), rank = (int)cluster_rank();
  const int64_t n0 = (int64_t)(blockIdx.x / split) * 128, m0 = (int64_t)blockIdx.y * NT;
  const int kb0 = (int)((int64_t)p.kb * rank / split), kb1 = (int)((int64_t)p.kb * (rank + 1) / split);

  if (threadIdx.x == 0) {
    stop = 0;
    for (int i = 0; i < 2 * Sh::kDepth + 1; ++i) mbar_init(full + 8 * i, 1);
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(&tmem_slot, Sh::kTmem);
  const int ahead = min(Sh::kDepth, kb1 - kb0);          // the ring's first round needs no wait
  if (threadIdx.x == 64) {
    // its weights to L2 while the previous kernel ends (should that kernel write them, L2 stays coherent)
    for (int i = 0; i < ahead; ++i) {
      tma_prefetch(&p.w[0], (kb0 + i) * (I8 ? 128 : 64), (int)n0);
      if (DUAL) tma_prefetch(&p.w[1], (kb0 + i) * (I8 ? 128 : 64), (int)n0);
    }
  }
  after_previous();
  const auto load = [&](int kb, int s) {
    const uint32_t at = ring + s * Sh::kStage, bar = full + 8 * s;
    const int k = kb * (I8 ? 128 : 64);
    mbar_expect(bar, Sh::kStage);
    tma_load(at, &p.w[0], k, (int)n0, bar);
    if (DUAL) tma_load(at + 16384, &p.w[1], k, (int)n0, bar);
    tma_load(at + Sh::kWeightBytes, &p.x, k, (int)m0, bar);
  };
  if (threadIdx.x == 0) {
    fence_before_loads();
    for (int i = 0; i < ahead; ++i) load(kb0 + i, i);
  }
  // the scales of this thread's first results, while the operands stream
  const int quads = 32 / split, cols = (int)min((int64_t)NT, p.M - m0);
  float sa0 = 0.0f, s00[4] = {}, s10[4] = {};
  if (I8 && threadIdx.x < quads * cols) {
    const int64_t ch = n0 + 4 * (rank * quads + (int)threadIdx.x % quads);
    sa0 = ld_f32(p.e.a_scale + m0 + threadIdx.x / quads);
    const float *second = DUAL ? p.e.s1 : p.e.bias;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (ch + k >= p.N) continue;
      s00[k] = ld_f32(p.e.s0 + ch + k);
      if (second) s10[k] = ld_f32(second + ch + k);
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_slot;

  if (warp == 0 && lane == 0) {
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int kb = kb0 + ahead; kb < kb1; ++kb) {
      if (!mbar_wait(empty + 8 * s, ph ^ 1, &stop)) { ok = false; break; }
      load(kb, s);
      if (++s == Sh::kDepth) { s = 0; ph ^= 1; }
    }
    let_next_start();                                    // its blocks start while these finish
    if (!ok)                                             // gave up: the copies in flight land first
      for (int i = 0; i < Sh::kDepth; ++i) {
        s = s ? s - 1 : Sh::kDepth - 1;
        if (s == Sh::kDepth - 1) ph ^= 1;
        mbar_drain(full + 8 * s, ph);
      }
  } else if (warp == 1 && lane == 0) {
    const uint32_t instr = I8 ? instr_i8(128, NT) : instr_f16(128, NT, p.bf16, 0, 0);
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(full + 8 * s, ph, &stop)) { ok = false; break; }
      tmem_fence_after_sync();
      const uint32_t at = ring + s * Sh::kStage;
      const uint64_t w0 = operand_desc(at, false), w1 = operand_desc(at + 16384, false),
                     x = operand_desc(at + Sh::kWeightBytes, false);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mma<I8, false>(tmem, w0 + 2 * i, x + 2 * i, instr, kb > kb0 || i > 0);
        if (DUAL) mma<I8, false>(tmem + NT, w1 + 2 * i, x + 2 * i, instr, kb > kb0 || i > 0);
      }
      mma_commit(empty + 8 * s);
      if (++s == Sh::kDepth) { s = 0; ph ^= 1; }
    }
    mma_commit(acc_full);
    if (!ok) mbar_drain(acc_full, 0);                    // gave up: the products issued so far end first
  } else if (warp >= 2) {
    // sums to shared memory, [column][channel]: the ring is free once all products are done
    const int quarter = warp & 3;
    if (__all_sync(0xFFFFFFFFu, mbar_wait(acc_full, 0, &stop))) {
      tmem_fence_after_sync();
      const uint32_t ch = ring + 4 * (quarter * 32 + lane);
#pragma unroll 1
      for (int c = 0; c < Sh::kCols; c += 16) {
        const int left = cols - (c & (NT - 1));          // columns of tokens that exist
        if (left <= 0) continue;
        float v[16];
        tmem_ld16(tmem + ((uint32_t)quarter << 21) + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < left)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(ch + 512 * (c + i)), "f"(v[i]) : "memory");
      }
    }
  }
  __syncwarp();
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  cluster_sync();

  // each block finishes 128 / split of the channels, four a thread
  uint32_t peer[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) peer[r] = map_to_rank(ring, r < split ? r : rank);
  for (int i = threadIdx.x; i < quads * cols; i += 192) {
    const int q = rank * quads + i % quads, c = i / quads;
    const int64_t ch = n0 + 4 * q, row = m0 + c;
    const int valid = (int)min((int64_t)4, p.N - ch);
    if (valid <= 0) continue;
    const uint32_t off = 512 * c + 16 * q;
    float4 g = make_float4(0, 0, 0, 0), u = g;           // four zero bit patterns: int32 zeros too
    // four parts' loads at a time: one after the other their latencies would add up
#pragma unroll
    for (int r0 = 0; r0 < 8; r0 += 4) {
      if (r0 >= split) break;
      float4 a[4], b[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[k] = ld_cluster4(peer[r0 + k] + off);          // past the last part: the block's own sums, not added
        if (DUAL) b[k] = ld_cluster4(peer[r0 + k] + off + 512 * NT);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (r0 + k >= split) continue;
        add4(g, a[k], I8);
        if (DUAL) add4(u, b[k], I8);
      }
    }
    const bool first = i < 192;
    finish4<I8, DUAL>(p.e, g, u, row, p.N, ch, valid, p.wide4, p.out, first ? &sa0 : nullptr, s00, s10);
  }
  __syncwarp();
  if (warp == 1) tmem_dealloc(tmem, Sh::kTmem);
  cluster_sync();                                        // no block leaves while its sums are read
  if (threadIdx.x == 0 && stop) say_gave_up(p.note);
}

// Rows of `bytes` bytes, packed, to rows `pitch` bytes apart (a multiple of 16);
// blockIdx.y: the matrix.  A group of 2^lanes threads (32 at most) takes a row, 16
// bytes a thread at a time, read as two aligned units (the second is its
// neighbour's first) and shifted; units that the matrix ends in are read by bytes,
// so nothing past it is touched.  Bound by issue until rows were dealt to groups:
// a division for each unit took 8000 x 8191 bytes 40 us, now 28.
struct PitchCopies {
  struct {
    const uint8_t *src;
    int64_t rows, bytes, pitch;
    uint4 *dst;
    int lanes;
  } m[3];
  int n;
};

__device__ __noinline__ uint4 unit_before(const uint8_t *a, const uint8_t *end) {
  uint32_t w[4] = {};
  for (int q = 0; q < 16; ++q)
    if (a + q < end) w[q >> 2] |= ld_u8(a + q) << (8 * (q & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(256) pitch_rows_kernel(const PitchCopies p) {
  after_previous();
  let_next_start();
  const auto &m = p.m[blockIdx.y];
  const uint8_t *end = m.src + m.rows * m.bytes;
  const int lanes = 1 << m.lanes, per = (int)(m.pitch >> 4);
  const int64_t thread = (int64_t)blockIdx.x * 256 + threadIdx.x, step = ((int64_t)gridDim.x * 256) >> m.lanes;
  for (int64_t r = thread >> m.lanes; r < m.rows; r += step) {
    const uint8_t *at = m.src + r * m.bytes;
    const uint32_t mis = (uint32_t)reinterpret_cast<uintptr_t>(at) & 15u, sh = 8 * (mis & 3u);
    const uint8_t *base = at - mis;
    const bool safe = at + m.bytes + 32 <= end;          // every unit of the row lies inside the matrix
    uint4 *out = m.dst + r * per;
#pragma unroll 2
    for (int c = (int)thread & (lanes - 1); c < per; c += lanes) {
      const uint8_t *a = base + 16 * (int64_t)c;
      const int left = (int)min((int64_t)16, m.bytes - 16 * (int64_t)c);
      uint4 u, v = make_uint4(0, 0, 0, 0);
      u = safe || a + 16 <= end ? ld_u32x4(a) : unit_before(a, end);
      if (left + (int)mis > 16)
        v = safe || a + 32 <= end ? ld_u32x4(a + 16) : unit_before(a + 16, end);
      uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
      if (mis & 8u) {
#pragma unroll
        for (int q = 0; q < 6; ++q) w[q] = w[q + 2];
      }
      if (mis & 4u) {
#pragma unroll
        for (int q = 0; q < 5; ++q) w[q] = w[q + 1];
      }
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = __funnelshift_r(w[q], w[q + 1], sh);
      if (left < 16) {                                   // zeros past the row's end
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int here = left - 4 * q;
          if (here < 4) o[q] = here > 0 ? o[q] & ((1u << (8 * here)) - 1u) : 0u;
        }
      }
      out[c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <typename T> __device__ __forceinline__ float widen(T v);
template <> __device__ __forceinline__ float widen<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T narrow(float v);
template <> __device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// dg = grad u act'(g), du = grad act(g), in rows `pitch` elements apart; eight
// values a thread where rows start on 16-byte boundaries (N = 8), else one.  Both are rounded to
// 16 bits, as they are operands of a 16-bit product: with that a gradient's error is sqrt 2 of its
// last rounding's (0.0023 against 0.0017 in bf16); kept as two 16-bit parts each they would double
// the products.  Bound by HBM: 4096 x 8192 bf16, 470 MB in 65 us (7.2 TB/s).
template <typename T, int N>
__global__ void __launch_bounds__(256) gate_grad_kernel(const T *grad, const float *gate,
                                                        const float *up, int64_t rows, int64_t cols,
                                                        int64_t pitch, int act, T *__restrict__ dg,
                                                        T *__restrict__ du) {
  after_previous();
  let_next_start();
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * N;
  if (c >= cols) return;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const int64_t at = r * cols + c, to = r * pitch + c;
    if (N == 1) {
      float a, d;
      activation_slope(ld_f32(gate + at), act, a, d);
      const uint16_t bits = ld_u16(grad + at);
      const float h = widen<T>(*reinterpret_cast<const T *>(&bits));
      dg[to] = narrow<T>(h * ld_f32(up + at) * d);
      du[to] = narrow<T>(h * a);
    } else {
      const uint4 hv = ld_u32x4(grad + at);
      const float4 g0 = ld_f32x4(gate + at), g1 = ld_f32x4(gate + at + 4), u0 = ld_f32x4(up + at),
                   u1 = ld_f32x4(up + at + 4);
      const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
      const float u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
      const T *h = reinterpret_cast<const T *>(&hv);
      __align__(16) T og[8], ou[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float a, d;
        activation_slope(g[i], act, a, d);
        const float v = widen<T>(h[i]);
        og[i] = narrow<T>(v * u[i] * d);
        ou[i] = narrow<T>(v * a);
      }
      *reinterpret_cast<uint4 *>(dg + to) = *reinterpret_cast<const uint4 *>(og);
      *reinterpret_cast<uint4 *>(du + to) = *reinterpret_cast<const uint4 *>(ou);
    }
  }
}

}  // namespace tcq

using namespace tcq;
using namespace tcq_host;

namespace {

constexpr int64_t kMostIn8 = 131071, kMost = (1ll << 30) - 1;

tcq_status_t check_sizes(int64_t n_tok, int64_t n_out, int64_t n_in, int64_t most_in) {
  if (n_tok < 0 || n_out <= 0 || n_in <= 0) return TCQ_ERR_INVALID_ARG;
  if (n_tok > kMost || n_out > kMost || n_in > most_in) return TCQ_ERR_UNSUPPORTED;
  // tiles of 256 x 128, two products, halved: counted in 32 bits
  const int64_t t = (n_tok >> 8) + 1, o = (n_out >> 7) + 1, i = (n_in >> 7) + 1;
  if (t * o > kMost / 4 || t * i > kMost / 4 || o * i > kMost / 4) return TCQ_ERR_UNSUPPORTED;
  return TCQ_OK;
}

bool bad_ptr(const void *p) { return !p || !aligned16(p); }
bool bad_type(int t) { return t != TCQ_F16 && t != TCQ_BF16 && t != TCQ_F32; }
bool bad_act(int a) { return a < TCQ_ACT_SILU || a > TCQ_ACT_RELU; }
size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t tiles(int64_t n, int64_t by) { return (n + by - 1) / by; }
unsigned blocks_for(int64_t threads) {
  return (unsigned)std::min<int64_t>((threads + 255) / 256, (int64_t)sm_count() * 16);
}
int width(const void *p, int64_t cols, int size) {
  const uint64_t v = (uint64_t)reinterpret_cast<uintptr_t>(p) | (uint64_t)(cols * size);
  return v % 32 == 0 ? 32 : v % 16 == 0 ? 16 : size;
}
int type_size(int t) { return t == TCQ_F32 ? 4 : 2; }

// Whether a packed matrix of rows of `bytes` bytes has to be copied to an
// aligned pitch for tensor-map loads, and what the copy takes.
bool needs_pitch(int64_t rows, int64_t bytes) { return rows > 1 && bytes % 16 != 0; }
size_t pitch_bytes(int64_t rows, int64_t bytes) {
  return needs_pitch(rows, bytes) ? round256((size_t)rows * round_up(bytes, 16)) : 0;
}

// An operand ready for tensor-map loads: where it is and its pitch.
struct Operand {
  const void *p;
  int64_t rows, cols, pitch;
  int es;
};

struct Workspace {
  char *at;
  void *take(size_t n) {
    void *p = at;
    at += round256(n);
    return p;
  }
};

// Copies to an aligned pitch, collected and then made in one launch.
Operand ready(const void *p, int64_t rows, int64_t cols, int es, Workspace &ws, PitchCopies &todo) {
  Operand o = {p, rows, cols, round_up(cols * es, 16), es};
  if (!needs_pitch(rows, cols * es)) return o;
  uint4 *copy = (uint4 *)ws.take(pitch_bytes(rows, cols * es));
  int lanes = 0;
  while (lanes < 5 && (16 << lanes) < o.pitch) ++lanes;
  todo.m[todo.n++] = {(const uint8_t *)p, rows, cols * es, o.pitch, copy, lanes};
  o.p = copy;
  return o;
}

tcq_status_t make_copies(const PitchCopies &todo, cudaStream_t s) {
  if (todo.n == 0) return TCQ_OK;
  int64_t most = 0;
  for (int i = 0; i < todo.n; ++i) most = std::max(most, todo.m[i].rows * (todo.m[i].pitch / 16));
  const dim3 grid((unsigned)std::min<int64_t>((most + 511) / 512, (int64_t)sm_count() * 32), (unsigned)todo.n);
  return launch(pitch_rows_kernel, grid, 256, 0, 0, s, todo);
}

bool map_of(CUtensorMap *m, const Operand &o, int box_rows) {
  return make_map(m, o.p, o.es, o.rows, o.cols, o.pitch, box_rows);
}

// Row tiles of a band: the second operand is read from memory once for each
// band, so bands are as tall as leaves the first operand's rows (32 KB a step and
// tile) within 24 MB of the 126 MB L2, at least 8, and of equal height (gated block
// 3001 x 2048 x 8192: 155.0 us in bands of 8, 151.7 in one of 12; int8 3001 x 8192 x
// 8192 153.5 and 149.6).
int band_of(const Job &j) {
  const int64_t most = std::max<int64_t>(8, (24 << 20) / (32768ll * j.kb * j.segs));
  return (int)tiles(j.mt, tiles(j.mt, most));
}

// The tiles of one or two jobs, dealt to the clusters.  The job with the longer
// tiles goes first; clusters that its last round leaves idle take as many of the
// other's tiles as that round lasts; then the rest goes round.  What is left of
// the last round, if it occupies at most half of the clusters, is dealt in half
// tiles.  Measured: gradients of 4096 x 2048 x 8192 446 us for all three in one
// launch (elementwise pass counted), grad_x alone 272, the weights' two alone 280.
// Half tiles: int8 256 x 512 -> 2048 7.7 -> 6.3 us, gated block 100 x 1024 -> 2048
// 10.9 -> 9.2, 1024 x 1024 -> 8192 33.6 -> 32.1, training step 512 x 1024 x 2048 41.9
// -> 37.9; at 3001 x 2048 x 8192 (768 tiles, 74 clusters) nothing (power, not the
// idle SMs, sets the time there).
int clusters_of_gpu() { return std::max(1, sm_count() / 2); }

// Parts of the contraction for `count` tiles of `steps` steps whose sums are `sums`
// bytes: the number, of those that the clusters hold at once with eight steps or
// more each, that takes the least time by what was measured: 0.26 us a step while
// few clusters run, 3 us to join and the parts' sums twice through L2 at 6 TB/s.  Less
// than 15% to be had by that is none in fact, as the steps of a wide product take longer
// (int8 192 x 8192 x 8192, 32 tiles: whole 24.6, in two parts 29.3, by the formula 15.5 of 16.6).
// Measured (us, whole / best split): int8 512 x 8192 x 1024 25.8 / 16.9 (four
// parts), 1024 tokens 26.7 / 19.6 (four); 512 x 8192 x 2048 26.8 / 19.9 (four); int8
// gated block 129 x 8192 x 2048 26.4 / 19.5 (four); not split 512 x 2048 x 2048 11.1 /
// 15.0 (two), 1024 x 8192 x 2048 27.4 / 27.7 (two).
int parts_of(int64_t count, int64_t steps, double sums) {
  const int64_t most = std::min<int64_t>(clusters_of_gpu() / std::max<int64_t>(1, count), steps / 8);
  int best = 1;
  double least = 0.85 * 0.26 * (double)steps;
  for (int64_t s = 2; s <= most; ++s) {
    const double t = 0.26 * (double)steps / (double)s + 3.0 + 2.0 * (double)s * sums / 6e6;
    if (t < least) {
      least = t;
      best = (int)s;
    }
  }
  return best;
}

// A job's tiles and parts; what its parts' sums take in the workspace.
struct Plan {
  int mt, nt, split;
  int64_t pitch;
  size_t bytes;
};
Plan plan_of(int64_t M, int64_t N, int cols, int z, int planes, int64_t steps) {
  Plan l;
  l.mt = (int)tiles(M, 256);
  l.nt = (int)tiles(N, cols);
  l.pitch = round_up(N, 16);
  l.split = parts_of((int64_t)l.mt * l.nt * z, steps, 4.0 * planes * (double)M * (double)l.pitch);
  l.bytes = l.split > 1 ? round256((size_t)l.split * planes * M * l.pitch * 4) : 0;
  return l;
}

void lay_out(Job &j, const Plan &l, Workspace &w) {
  j.mt = l.mt;
  j.nt = l.nt;
  j.split = l.split;
  j.pitch = l.pitch;
  j.part = l.bytes ? (float *)w.take(l.bytes) : nullptr;
}

void deal(PairParams &p, int jobs, int clusters) {
  p.shares = 0;
  for (int i = 0; i < jobs; ++i) p.job[i].band = band_of(p.job[i]);
  const auto give = [&](int job, int64_t first, int64_t n, int narrow, int64_t lo, int64_t hi) {
    if (hi > lo) p.share[p.shares++] = {job, (int)first, (int)n, narrow, (uint32_t)lo, (uint32_t)hi};
  };
  const auto count = [&](int j) { return (int64_t)p.job[j].mt * p.job[j].nt * p.job[j].z * p.job[j].split; };
  const auto finish = [&](int j, int64_t lo) {
    const int64_t hi = count(j), rest = (hi - lo) % clusters;
    const bool halve = rest > 0 && 2 * rest <= clusters && p.job[j].split == 1;
    give(j, 0, clusters, 0, lo, halve ? hi - rest : hi);
    if (halve) give(j, 0, clusters, 1, 2 * (hi - rest), 2 * hi);
  };
  if (jobs == 1) return finish(0, 0);
  int64_t cost[2];
  for (int j = 0; j < 2; ++j)                            // a tile's write-out takes as long as eight steps
    cost[j] = p.job[j].kb * p.job[j].segs / p.job[j].split + 8;
  const int big = cost[0] >= cost[1] ? 0 : 1, small = 1 - big;
  int64_t t = count(big), c = cost[big];
  const bool halve = 2 * t <= clusters && p.job[big].split == 1;
  if (halve) {
    t *= 2;
    c = (c + 1) / 2;
  }
  give(big, 0, clusters, halve, 0, t);
  const int64_t used = t % clusters, idle = used ? clusters - used : 0;
  const int64_t fill = std::min(count(small), idle * ((c + cost[small] / 2) / cost[small]));
  give(small, used, idle, 0, 0, fill);
  if (fill < count(small)) finish(small, fill);
}

template <bool I8, bool DUAL>
tcq_status_t launch_pair(PairParams &p, int jobs, cudaStream_t s) {
  if (status_of(cudaFuncSetAttribute(pair_kernel<I8, DUAL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kPairSmem)) != TCQ_OK)
    return TCQ_ERR_CUDA;
  deal(p, jobs, clusters_of_gpu());
  int64_t grid = 0;                                      // clusters that get a tile
  for (int i = 0; i < p.shares; ++i)
    grid = std::max<int64_t>(grid, p.share[i].first + std::min<int64_t>(p.share[i].n, (int64_t)p.share[i].hi - p.share[i].lo));
  tcq_status_t st = launch(pair_kernel<I8, DUAL>, dim3(2 * (unsigned)grid), kPairThreads, kPairSmem, 0, s, p);
  for (int i = 0; i < jobs && st == TCQ_OK; ++i) {
    const Job &j = p.job[i];
    if (j.split == 1) continue;
    const Join q = {j.part, j.split, j.planes, j.N % 4 == 0, j.M, j.N, j.pitch, {j.out[0], j.out[1]}, p.e};
    st = launch(join_kernel<I8, DUAL>, dim3(blocks_for(j.M * tiles(j.N, 4)), 1, (unsigned)j.z), 256, 0, 0, s, q);
  }
  return st;
}

// Which kernel.  rows_kernel reads the weights once for each tile of tokens and then finishes
// 128 channels by its tile of tokens in each cluster: best for long sums of few tokens.  Of a
// short sum the finishing is most of it, and with two tiles of tokens and many channels the
// pairs' tiles fill the GPU and read less.  Measured, us, rows / pair, steps of 128 bytes of the
// contraction:
//   to 32 tokens: rows (20 tokens, 1024 channels, 4 steps, two projections 7.2 / 6.1 is its worst);
//   to 64, 4 steps: 9.2 / 6.0 (512 and 2048 channels), 9.4 / 7.0 (8192), two projections 11.4 / 6.1
//     (1024), 9.1 / 8.6 (8192, 16 bits; 40 tokens 7.5 / 8.5); 8 steps: 7.0 / 7.0 and 7.7 / 8.4, two projections 9.2 / 7.2
//     and 10.2 / 10.4, 16 bits 7.7 / 7.1 and 8.9 / 10.2; 16 steps of two, 8192: 13.2 / 13.6;
//   two projections of 96 tokens, bf16, 2048 -> 8192: 19.3 / 20.2, 128: 21.0 / 20.6, 1024 -> 2736 at 96
//     9.3 / 9.1;
//   to 128, one projection, 4 steps: 14.4 / 6.3, 8: 10.1 / 7.3, 12: 10.6 / 8.5, 64 (8192) 19.7 / 27.7;
//   to 256, 12 steps: 10.6 / 8.5; 16: 8.2 / 9.5 (2048), 10.0 / 9.6 (4096), 13.5 / 10.7 (8192); 32: 9.2 /
//     13.3, 11.7 / 14.2, 18.1 / 15.4; 64: 12.5 / 17.4, 15.8 / 20.4, 27.0 / 24.6.
template <bool DUAL>
bool few_tokens(int64_t M, int64_t N, int64_t steps) {
  if (M <= 32) return true;
  if (M <= 64) return steps > 4 || (DUAL && M <= 48 && N > 4096);
  return !DUAL && steps > 12 && (M <= 128 || (M <= 256 && N <= 4096));
}

template <bool I8, bool DUAL, int NT>
tcq_status_t launch_rows(const RowsParams &p, cudaStream_t s) {
  typedef RowsShape<DUAL, NT> Sh;
  if (status_of(cudaFuncSetAttribute(rows_kernel<I8, DUAL, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Sh::kSmem)) != TCQ_OK)
    return TCQ_ERR_CUDA;
  // Split the contraction while the clusters still fit the GPU at once (of 148 SMs, 132 hold clusters
  // of four blocks and 120 clusters of eight) and each block keeps four steps of it, eight in a cluster
  // of eight.  One int8 token, 8192 x 8192, in 1 / 2 / 4 / 8 parts: 21.4 / 15.6 / 15.5 / 20.7 us (the
  // last in two waves); 16 tokens, 8192 -> 2048: 18.8 / 11.1 / 7.5 / 6.9; bf16 gated block of 16 tokens,
  // 2048 -> 2048: 15.0 / 9.1 / 6.7 / 7.5 (four steps a block at eight parts), of 64 tokens, one block an
  // SM: 18.1 / 11.8 / 9.2 / 19.6 (two waves).
  const int64_t work = tiles(p.N, 128) * tiles(p.M, NT), sms = sm_count();
  const auto fits = [&](int parts) {
    const int64_t usable = parts == 8 ? sms * 13 / 16 : parts == 4 ? sms * 7 / 8 : sms;
    return work * parts <= usable * Sh::kBlocksPerSm && p.kb >= (parts == 8 ? 64 : 4 * parts);
  };
  int split = 1;
  while (split < 8 && fits(2 * split)) split *= 2;
  const int64_t nt = tiles(p.N, 128), mt = tiles(p.M, NT);
  return launch(rows_kernel<I8, DUAL, NT>, dim3((unsigned)(nt * split), (unsigned)mt), 192, Sh::kSmem, split, s, p);
}

}  // namespace

extern "C" tcq_status_t tcq_products_gave_up(unsigned int *count) {
  if (!count) return TCQ_ERR_INVALID_ARG;
  // the copy alone would not wait for non-blocking streams
  if (status_of(cudaDeviceSynchronize()) != TCQ_OK) return TCQ_ERR_CUDA;
  return status_of(cudaMemcpyFromSymbol(count, g_gave_up, sizeof(unsigned)));
}

// What a forward product needs: operands at an aligned pitch, the parts' sums.
template <bool DUAL>
static size_t product_bytes(int64_t M, int64_t N, int64_t K, int es) {
  return pitch_bytes(M, K * es) + (DUAL ? 2 : 1) * pitch_bytes(N, K * es) +
         (few_tokens<DUAL>(M, N, tiles(K * es, 128)) ? 0 : plan_of(M, N, DUAL ? 128 : 256, 1, DUAL ? 2 : 1, tiles(K * es, 128)).bytes);
}

extern "C" size_t tcq_int8_matmul_workspace_size(int64_t n_tok, int64_t n_out, int64_t n_in) {
  if (check_sizes(n_tok, n_out, n_in, kMostIn8) != TCQ_OK) return 0;
  return product_bytes<false>(n_tok, n_out, n_in, 1);
}

extern "C" size_t tcq_int8_gated_ffn_workspace_size(int64_t n_tok, int64_t n_out, int64_t n_in) {
  if (check_sizes(n_tok, n_out, n_in, kMostIn8) != TCQ_OK) return 0;
  return product_bytes<true>(n_tok, n_out, n_in, 1);
}

extern "C" size_t tcq_gated_ffn_workspace_size(int64_t n_tok, int64_t n_out, int64_t n_in) {
  if (check_sizes(n_tok, n_out, n_in, kMost) != TCQ_OK) return 0;
  return product_bytes<true>(n_tok, n_out, n_in, 2);
}

static Plan plan_grad_x(int64_t M, int64_t F, int64_t K) { return plan_of(M, K, 256, 1, 1, 2 * tiles(F, 64)); }
static Plan plan_grad_w(int64_t M, int64_t F, int64_t K, int z) { return plan_of(F, K, 256, z, z, tiles(M, 64)); }

// dg and du; x, Wg and Wu where their rows need an aligned pitch; the parts' sums
extern "C" size_t tcq_gated_ffn_backward_workspace_size(int64_t n_tok, int64_t n_out, int64_t n_in) {
  if (check_sizes(n_tok, n_out, n_in, kMost) != TCQ_OK) return 0;
  return 2 * round256((size_t)n_tok * round_up(2 * n_out, 16)) + pitch_bytes(n_tok, 2 * n_in) +
         2 * pitch_bytes(n_out, 2 * n_in) + plan_grad_x(n_tok, n_out, n_in).bytes +
         std::max(plan_grad_w(n_tok, n_out, n_in, 1).bytes, plan_grad_w(n_tok, n_out, n_in, 2).bytes);
}

static bool no_workspace(const void *ws, size_t have, size_t need) {
  return need && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || have < need);
}

// a x w0^T (and a x w1^T) on operands of `es` bytes.
template <bool I8, bool DUAL>
static tcq_status_t product(const void *a, const void *w0, const void *w1, int es, int bf16, int64_t M, int64_t N,
                            int64_t K, void *out, Epilogue e, void *ws, cudaStream_t s) {
  Workspace w = {(char *)ws};
  PitchCopies copies;
  copies.n = 0;
  unsigned int *const note = note_of_device();
  if (take_note(note)) return TCQ_ERR_TIMEOUT;
  Operand A = ready(a, M, K, es, w, copies), B[2];
  for (int i = 0; i < (DUAL ? 2 : 1); ++i) B[i] = ready(i ? w1 : w0, N, K, es, w, copies);
  tcq_status_t st = make_copies(copies, s);
  if (st != TCQ_OK) return st;
  if (few_tokens<DUAL>(M, N, tiles(K * es, 128))) {
    const int nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    RowsParams r;
    if (!map_of(&r.w[0], B[0], 128) || (DUAL && !map_of(&r.w[1], B[1], 128)) || !map_of(&r.x, A, nt))
      return TCQ_ERR_CUDA;
    r.M = M;
    r.N = N;
    r.kb = (int)tiles(K * es, 128);
    r.bf16 = bf16;
    r.wide4 = N % 4 == 0;
    r.out = out;
    r.note = note;
    r.e = e;
    return nt == 16   ? launch_rows<I8, DUAL, 16>(r, s)
           : nt == 32 ? launch_rows<I8, DUAL, 32>(r, s)
           : DUAL || nt == 64 ? launch_rows<I8, DUAL, 64>(r, s)
                              : launch_rows<I8, false, 128>(r, s);
  }
  PairParams p;
  p.bf16 = bf16;
  p.note = note;
  p.e = e;
  Job &j = p.job[0];
  if (!map_of(&j.a[0], A, 128)) return TCQ_ERR_CUDA;
  for (int i = 0; i < (DUAL ? 2 : 1); ++i)
    if (!map_of(&j.b[i], B[i], 128) || !map_of(&j.b_half[i], B[i], 64)) return TCQ_ERR_CUDA;
  j.out[0] = out;
  j.M = M;
  j.N = N;
  j.kb = (int)tiles(K * es, 128);
  j.planes = DUAL ? 2 : 1;
  lay_out(j, plan_of(M, N, DUAL ? 128 : 256, 1, j.planes, j.kb), w);
  j.segs = 1;
  j.z = 1;
  j.a_mn = j.b_mn = 0;
  j.wide = width(out, N, type_size(e.dtype));
  return launch_pair<I8, DUAL>(p, 1, s);
}

extern "C" tcq_status_t tcq_int8_matmul(const int8_t *a, const float *a_scale, const int8_t *w, const float *w_scale,
                                        const float *bias, int64_t n_tok, int64_t n_out, int64_t n_in, void *out,
                                        int out_dtype, void *ws, size_t ws_bytes, void *stream) {
  if (bad_type(out_dtype)) return TCQ_ERR_INVALID_ARG;
  tcq_status_t st = check_sizes(n_tok, n_out, n_in, kMostIn8);
  if (st != TCQ_OK) return st;
  if (n_tok == 0) return TCQ_OK;
  if (bad_ptr(a) || bad_ptr(a_scale) || bad_ptr(w) || bad_ptr(w_scale) || bad_ptr(out) || !aligned16(bias))
    return TCQ_ERR_INVALID_ARG;
  const size_t need = tcq_int8_matmul_workspace_size(n_tok, n_out, n_in), M = n_tok, N = n_out, K = n_in;
  if (no_workspace(ws, ws_bytes, need)) return TCQ_ERR_WORKSPACE;
  if (clash({{out, M * N * type_size(out_dtype)}, {ws, need}},
            {{a, M * K}, {a_scale, 4 * M}, {w, N * K}, {w_scale, 4 * N}, {bias, 4 * N}}))
    return TCQ_ERR_INVALID_ARG;
  const Epilogue e = {out_dtype, 0, a_scale, w_scale, nullptr, bias, nullptr, nullptr, 0};
  return product<true, false>(a, w, nullptr, 1, 0, n_tok, n_out, n_in, out, e, ws, (cudaStream_t)stream);
}

extern "C" tcq_status_t tcq_int8_gated_ffn(const int8_t *a, const float *a_scale, const int8_t *w_gate,
                                           const float *w_gate_scale, const int8_t *w_up, const float *w_up_scale,
                                           int64_t n_tok, int64_t n_out, int64_t n_in, int act, void *h, int out_dtype,
                                           void *ws, size_t ws_bytes, void *stream) {
  if (bad_type(out_dtype) || bad_act(act)) return TCQ_ERR_INVALID_ARG;
  tcq_status_t st = check_sizes(n_tok, n_out, n_in, kMostIn8);
  if (st != TCQ_OK) return st;
  if (n_tok == 0) return TCQ_OK;
  if (bad_ptr(a) || bad_ptr(a_scale) || bad_ptr(w_gate) || bad_ptr(w_gate_scale) || bad_ptr(w_up) ||
      bad_ptr(w_up_scale) || bad_ptr(h))
    return TCQ_ERR_INVALID_ARG;
  const size_t need = tcq_int8_gated_ffn_workspace_size(n_tok, n_out, n_in), M = n_tok, N = n_out, K = n_in;
  if (no_workspace(ws, ws_bytes, need)) return TCQ_ERR_WORKSPACE;
  if (clash({{h, M * N * type_size(out_dtype)}, {ws, need}},
            {{a, M * K}, {a_scale, 4 * M}, {w_gate, N * K}, {w_gate_scale, 4 * N}, {w_up, N * K}, {w_up_scale, 4 * N}}))
    return TCQ_ERR_INVALID_ARG;
  const Epilogue e = {out_dtype, act, a_scale, w_gate_scale, w_up_scale, nullptr, nullptr, nullptr, 0};
  return product<true, true>(a, w_gate, w_up, 1, 0, n_tok, n_out, n_in, h, e, ws, (cudaStream_t)stream);
}

extern "C" tcq_status_t tcq_gated_ffn(const void *x, const void *w_gate, const void *w_up, int dtype, int64_t n_tok,
                                      int64_t n_out, int64_t n_in, int act, void *h, float *gate, float *up, void *ws,
                                      size_t ws_bytes, void *stream) {
  if ((dtype != TCQ_F16 && dtype != TCQ_BF16) || bad_act(act)) return TCQ_ERR_INVALID_ARG;
  tcq_status_t st = check_sizes(n_tok, n_out, n_in, kMost);
  if (st != TCQ_OK) return st;
  if (!gate != !up) return TCQ_ERR_INVALID_ARG;
  if (n_tok == 0) return TCQ_OK;
  if (bad_ptr(x) || bad_ptr(w_gate) || bad_ptr(w_up) || bad_ptr(h) || !aligned16(gate) || !aligned16(up))
    return TCQ_ERR_INVALID_ARG;
  const size_t need = tcq_gated_ffn_workspace_size(n_tok, n_out, n_in), M = n_tok, N = n_out, K = n_in;
  if (no_workspace(ws, ws_bytes, need)) return TCQ_ERR_WORKSPACE;
  if (clash({{h, 2 * M * N}, {gate, 4 * M * N}, {up, 4 * M * N}, {ws, need}},
            {{x, 2 * M * K}, {w_gate, 2 * N * K}, {w_up, 2 * N * K}}))
    return TCQ_ERR_INVALID_ARG;
  Epilogue e = {dtype, act, nullptr, nullptr, nullptr, nullptr, gate, up, 0};
  e.wide_save = std::min(width(gate, n_out, 4), width(up, n_out, 4));
  return product<false, true>(x, w_gate, w_up, 2, dtype == TCQ_BF16, n_tok, n_out, n_in, h, e, ws,
                              (cudaStream_t)stream);
}

template <typename T>
static tcq_status_t gate_grads(const void *grad, const float *gate, const float *up, int64_t rows, int64_t cols,
                               int64_t pitch, int act, const void *dg, const void *du, cudaStream_t s) {
  const bool whole = cols % 8 == 0;
  const dim3 grid((unsigned)tiles(cols, whole ? 2048 : 256), (unsigned)std::min<int64_t>(rows, 65535));
  return launch(whole ? gate_grad_kernel<T, 8> : gate_grad_kernel<T, 1>, grid, 256, 0, 0, s, (const T *)grad, gate, up,
                rows, cols, pitch / 2, act, (T *)dg, (T *)du);
}

extern "C" tcq_status_t tcq_gated_ffn_backward(const void *x, const void *w_gate, const void *w_up, const float *gate,
                                               const float *up, const void *grad_h, int dtype, int64_t n_tok,
                                               int64_t n_out, int64_t n_in, int act, void *grad_x, void *grad_w_gate,
                                               void *grad_w_up, void *ws, size_t ws_bytes, void *stream) {
  if ((dtype != TCQ_F16 && dtype != TCQ_BF16) || bad_act(act)) return TCQ_ERR_INVALID_ARG;
  tcq_status_t st = check_sizes(n_tok, n_out, n_in, kMost);
  if (st != TCQ_OK) return st;
  if (!aligned16(grad_x) || !aligned16(grad_w_gate) || !aligned16(grad_w_up)) return TCQ_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (n_tok == 0) {                                      // no token: the weights' gradients are zero
    for (void *g : {grad_w_gate, grad_w_up})
      if (g && status_of(cudaMemsetAsync(g, 0, (size_t)n_out * n_in * 2, s)) != TCQ_OK) return TCQ_ERR_CUDA;
    return TCQ_OK;
  }
  if (bad_ptr(x) || bad_ptr(w_gate) || bad_ptr(w_up) || bad_ptr(gate) || bad_ptr(up) || bad_ptr(grad_h))
    return TCQ_ERR_INVALID_ARG;
  if (!grad_x && !grad_w_gate && !grad_w_up) return TCQ_OK;
  const size_t need = tcq_gated_ffn_backward_workspace_size(n_tok, n_out, n_in), M = n_tok, N = n_out, K = n_in;
  if (no_workspace(ws, ws_bytes, need)) return TCQ_ERR_WORKSPACE;
  if (clash({{grad_x, 2 * M * K}, {grad_w_gate, 2 * N * K}, {grad_w_up, 2 * N * K}, {ws, need}},
            {{x, 2 * M * K}, {w_gate, 2 * N * K}, {w_up, 2 * N * K}, {gate, 4 * M * N}, {up, 4 * M * N}, {grad_h, 2 * M * N}}))
    return TCQ_ERR_INVALID_ARG;

  unsigned int *const note = note_of_device();
  if (take_note(note)) return TCQ_ERR_TIMEOUT;
  Workspace w = {(char *)ws};
  const int64_t pitch = round_up(2 * n_out, 16);
  PitchCopies copies;
  copies.n = 0;
  Operand d[2];
  for (Operand &o : d) o = {w.take((size_t)n_tok * pitch), n_tok, n_out, pitch, 2};
  st = dtype == TCQ_F16 ? gate_grads<__half>(grad_h, gate, up, n_tok, n_out, pitch, act, d[0].p, d[1].p, s)
                        : gate_grads<__nv_bfloat16>(grad_h, gate, up, n_tok, n_out, pitch, act, d[0].p, d[1].p, s);
  if (st != TCQ_OK) return st;

  PairParams p;
  p.bf16 = dtype == TCQ_BF16;
  p.note = note;
  p.e = {dtype, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0};
  int jobs = 0;
  if (grad_x) {
    // one sum over both halves: dg Wg, then du Wu; the weights' rows run along it
    Job &j = p.job[jobs++];
    for (int i = 0; i < 2; ++i) {
      const Operand W = ready(i ? w_up : w_gate, n_out, n_in, 2, w, copies);
      if (!map_of(&j.a[i], d[i], 128) || !map_of(&j.b[i], W, 64)) return TCQ_ERR_CUDA;
    }
    j.out[0] = grad_x;
    j.M = n_tok;
    j.kb = (int)tiles(n_out, 64);
    j.segs = 2;
    j.z = 1;
    j.a_mn = 0;
    j.wide = width(grad_x, n_in, 2);
    j.planes = 1;
    lay_out(j, plan_grad_x(n_tok, n_out, n_in), w);
  }
  if (grad_w_gate || grad_w_up) {
    // dg^T x and du^T x: both operands' rows (tokens) run along the sum
    Job &j = p.job[jobs++];
    const Operand X = ready(x, n_tok, n_in, 2, w, copies);
    if (!map_of(&j.b[0], X, 64)) return TCQ_ERR_CUDA;
    j.z = 0;
    j.wide = 32;
    for (int i = 0; i < 2; ++i) {
      void *g = i ? grad_w_up : grad_w_gate;
      if (!g) continue;
      if (!map_of(&j.a[j.z], d[i], 64)) return TCQ_ERR_CUDA;
      j.out[j.z++] = g;
      j.wide = std::min(j.wide, width(g, n_in, 2));
    }
    j.M = n_out;
    j.kb = (int)tiles(n_tok, 64);
    j.segs = 1;
    j.a_mn = 1;
    j.planes = j.z;
    lay_out(j, plan_grad_w(n_tok, n_out, n_in, j.z), w);
  }
  for (int i = 0; i < jobs; ++i) {
    Job &j = p.job[i];
    j.N = n_in;
    j.b_mn = 1;
  }
  st = make_copies(copies, s);
  return st == TCQ_OK ? launch_pair<false, false>(p, jobs, s) : st;
}
