// 8-bit floating point (e4m3) with a scale for every 128 values: quantisation
// of rows and weight blocks, and the product of such operands on tcgen05.
//
//   s = max(amax / 448, 2^-126),  q = e4m3(x * (1 / s))   amax over 1 x 128 (rows)
//                                                         or 128 x 128 (weights)
//   out[t][n] = sum_g xs[t][g] ws[n / 128][g] (sum_{k in group g} xq[t][k] wq[n][k]) + bias[n]
//
// One e4m3 value of a group is its largest, so a group's inner sum needs no
// more than the tensor core's fp32; the groups' sums meet in fp32 registers,
// each multiplied by its own scales (the scales are arbitrary fp32 numbers, so
// they cannot ride in the MMA, which takes powers of two per 32 values).
#include <algorithm>

#include "e4m3.cuh"
#include "internal.h"
#include "tc.cuh"
#include "tma.cuh"

namespace dflash {

// ---------------------------------------------------------------------------
// Quantisation. Bound: one read and one write. A warp takes whole groups (16
// bytes a lane: two bf16 groups or one fp32 group at once), four at a time, and
// finds the largest magnitude by shuffles. Measured: 8190 x 20480 bf16 86 us (508
// MB, 0.87 of the copy bandwidth), 10 x 20480 2.0 us.
// ---------------------------------------------------------------------------
template <typename T> constexpr uint32_t kAbs = sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;
// NaN is passed over here and kept by the conversion.
template <typename T> __device__ __forceinline__ float vec_absmax(const uint4& u) {
  return vec_max<T>(make_uint4(u.x & kAbs<T>, u.y & kAbs<T>, u.z & kAbs<T>, u.w & kAbs<T>));
}
// The vector's values times 1 / scale (a division each would bound the kernel by
// its instructions: 138 us instead of 99 for 8190 x 20480 bf16), four e4m3 to a word.
template <typename T> __device__ __forceinline__ void f8_store(uint8_t* dst, const uint4& u, float r) {
  constexpr int N = VecTraits<T>::N;
  float f[N];
  unpack16<T>(u, f);
  uint32_t w[N / 4];
#pragma unroll
  for (int j = 0; j < N; j += 4) w[j / 4] = f8_pack4(f[j] * r, f[j + 1] * r, f[j + 2] * r, f[j + 3] * r);
  if constexpr (N == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(dst) = w[0];
}

// A warp's unit is U vectors a lane of one row, UNIT consecutive values.
template <typename T> struct QuantUnit {
  static constexpr int U = 2;
  static constexpr int VALUES = U * 32 * VecTraits<T>::N;
};

template <typename T>
__global__ void __launch_bounds__(256, 6)
f8_quant_rows_kernel(const T* x, uint8_t* q, float* scale, int T_rows, const int32_t* T_dev, int K) {
  wait_for_prior_grid();   // a dependent launch: the rows may come from the kernel before
  dependents_may_launch();
  constexpr int N = VecTraits<T>::N;
  constexpr int LPG = f8::G / N;           // lanes of a group
  constexpr int U = QuantUnit<T>::U, VALUES = QuantUnit<T>::VALUES;
  const unsigned rows = T_dev ? min(*T_dev, T_rows) : T_rows;
  const unsigned groups = (K + f8::G - 1) / f8::G, units = (K + VALUES - 1) / VALUES;
  const int lane = threadIdx.x & 31;
  const unsigned long warps = (unsigned long)gridDim.x * (blockDim.x >> 5), total = (unsigned long)rows * units;
  for (unsigned long w = (unsigned long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < total; w += warps) {
    // (rows * units fit 32 bits for all but the widest calls)
    const unsigned t = total >> 32 ? (unsigned)(w / units) : (unsigned)w / units;
    const int k0 = (int)(w - (unsigned long)t * units) * VALUES + lane * N;
    const T* src = x + (size_t)t * K;
    uint8_t* dst = q + (size_t)t * K;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 32 * N;       // K is a multiple of 16: a vector is inside or outside
      v[u] = k < K ? ld_once16(src + k) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 32 * N;
      float m = vec_absmax<T>(v[u]);
#pragma unroll
      for (int o = LPG / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float s = f8_scale(m);
      if (k < K) {
        f8_store<T>(dst + k, v[u], __frcp_rn(s));
        if (lane % LPG == 0) scale[(size_t)t * groups + k / f8::G] = s;
      }
    }
  }
}

// One CTA per 128 x 128 block (all in the grid's x: its y ends at 65535, below the
// row blocks and the groups that are allowed), a warp 16 of its rows, held in registers
// between the search for the largest magnitude and the conversion.
template <typename T>
__global__ void __launch_bounds__(256)
f8_quant_blocks_kernel(const T* x, uint8_t* q, float* scale, int T_rows, int K) {
  wait_for_prior_grid();   // a dependent launch
  dependents_may_launch();
  constexpr int N = VecTraits<T>::N;
  constexpr int LPG = f8::G / N, RPL = 32 / LPG;   // rows of a warp's load
  constexpr int L = 16 / RPL;
  __shared__ float s_max[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned groups = (K + f8::G - 1) / f8::G, row_block = blockIdx.x / groups;
  const int k = (int)(blockIdx.x - row_block * groups) * f8::G + (lane % LPG) * N;
  const int t0 = (int)row_block * f8::G + warp * 16 + lane / LPG;
  uint4 v[L];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int t = t0 + i * RPL;
    v[i] = t < T_rows && k < K ? ld_once16(x + (size_t)t * K + k) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < L; ++i) m = fmaxf(m, vec_absmax<T>(v[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, s_max[i]);
  const float s = f8_scale(m), r = __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int t = t0 + i * RPL;
    if (t < T_rows && k < K) f8_store<T>(q + (size_t)t * K + k, v[i], r);
  }
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
}

template <typename T>
static cudaError_t launch_f8_quant_t(const Fp8QuantArgs& a) {
  if (a.block_rows == f8::G) {
    const dim3 grid((unsigned)((a.K + f8::G - 1) / f8::G) * (unsigned)((a.T + f8::G - 1) / f8::G));
    return launch_dependent(f8_quant_blocks_kernel<T>, grid, dim3(256), 0, a.stream, (const T*)a.x, (uint8_t*)a.q,
                            a.scale, a.T, a.K);
  }
  // a warp per unit, up to what six CTAs an SM hold
  const long units = (long)a.T * ((a.K + QuantUnit<T>::VALUES - 1) / QuantUnit<T>::VALUES);
  const int grid = (int)std::max(1L, std::min((units + 7) / 8, 6L * 152));
  return launch_dependent(f8_quant_rows_kernel<T>, dim3(grid), dim3(256), 0, a.stream, (const T*)a.x, (uint8_t*)a.q,
                          a.scale, a.T, a.T_dev, a.K);
}

cudaError_t launch_fp8_quant(const Fp8QuantArgs& a) {
  return a.dtype == 0 ? launch_f8_quant_t<float>(a) : launch_f8_quant_t<bf16>(a);
}

// ---------------------------------------------------------------------------
// Product. A tile is 128 rows of x (the MMA's M, one TMEM lane each) by BN
// weight rows (N); a k-block is one group of 128 values, one 128-byte swizzle
// atom a row, and its four MMAs (K = 32 each) write a TMEM accumulator of their
// own. Sixteen warps take each accumulator out of TMEM and add it, times the
// group's scales, to the tile's sums in registers, while the MMAs of the next
// groups go on in the other accumulators. With the rows in the lanes a thread
// needs one scale a group (its row's times the weight block's), and the sums
// cost one multiply-add each.
//
// Few tiles (decode: the weights' bytes bound it) are split over K among the
// CTAs of a cluster of up to eight; each leaves its sums in its shared memory,
// and every CTA adds its part of the tile over the cluster in rank order
// (distributed shared memory: no workspace, no atomics, the same bits each
// time). Many tiles go round persistent CTAs, one per SM.
//
// Warps 0 - 15 sum, 16 and 17 issue the MMAs, 18 the TMA loads, and 19 brings the
// scales. Every wait is bounded as in the bf16 GEMM: one that gives up records a code,
// the CTA drains its copies and MMAs, frees its TMEM and returns.
//
// Shared memory begins at a constant address (aligned by its declaration, not by
// code), so that barriers and slots need no registers: 8 % at large sizes, where 64
// sums and 16 values on their way leave a thread little else. A group takes 240 ns
// (narrow; 255 where the CTAs' tiles go many rounds) or 425 (wide); the MMAs alone, 195
// and 335. Measured, bf16: 10 x 20480 x 4096 19.5 us (84 MB at 4.3 TB/s with the launch),
// 271 x 4096 x 10240 (fp32) 24, 8190 x 20480 x 4096 535 to 545 for a few calls (2.5
// PFLOP/s) and 610 to 625 in a long run, under the power cap (2.2).
// ---------------------------------------------------------------------------
namespace f8 {
constexpr int BM = 128;
constexpr int A_BYTES = BM * G;           // 16 KB
constexpr int RING_BYTES = 196608;        // 4 stages of 48 KB (BN = 256) or 6 of 32 KB
constexpr int SUM_WARPS = 16;
constexpr int MMA_WARPS = 2, TMA_WARPS = 2;
constexpr int THREADS = 32 * (SUM_WARPS + MMA_WARPS + TMA_WARPS);
constexpr int BUFS = 4, BUF_N = 128;      // TMEM accumulators of 128 columns
// Scales of the last groups, 128 of x, then the weight blocks'. They are written four
// groups at once when the first one's stage is free, up to STAGES + 3 groups ahead of
// the MMAs, which in turn run up to BUFS groups ahead of the sums.
constexpr int SCALE_SLOTS = 16, SCALE_LD = BM + 4;
constexpr int SMEM_BYTES = RING_BYTES + 4 * SCALE_SLOTS * SCALE_LD + 512;

template <int BN> struct Cfg {
  static constexpr int STAGE = A_BYTES + BN * G;
  static constexpr int STAGES = RING_BYTES / STAGE;
  static constexpr int PARTS = BN / BUF_N;   // accumulators that a k-block fills
  static constexpr int COLS = BN / 4;     // a summing thread's columns
  static constexpr int RED_LD = BN + 4;   // floats: a quarter warp's rows fall on distinct banks
  static_assert(STAGES + BUFS + 3 < SCALE_SLOTS, "scale slots");
  static constexpr int LD = PARTS > 1 ? 16 : 32;   // TMEM columns of a load: with 64 sums a thread has registers for 16
};

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
// Instruction descriptor, kind::f8f6f4: e4m3 A and B (format 0), fp32 D, both K-major.
__device__ __forceinline__ uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ uint32_t ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float4 ld_peer(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}
// Pairs of fp32 in a 64-bit register: one instruction multiplies and adds both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// The product of two scales may leave fp32's normal range where a term (the product
// times a group's sum, which is 0 or 2^-18 to 2^25 in magnitude) does not. Then the sums
// take the two scales in turn: the larger one first where the product is too small (the
// sum times it is not below the term), the smaller one where it is too large (not above
// it). A product with 0, NaN or infinity stays what it is either way.
__device__ __forceinline__ bool in_range(float f) {
  constexpr uint32_t kLow = 2u * 0x00800000u, kHigh = 2u * 0x7f800000u;   // 2^-126 and infinity, without a sign
  return 2u * __float_as_uint(f) - kLow < kHigh - kLow;
}
__device__ __forceinline__ float2 scales_in_turn(float xs, float ws) {
  const float a = fabsf(xs), b = fabsf(ws);
  if (in_range(xs * ws)) return make_float2(1.f, xs * ws);
  return (a > b) == (a * b < 1.f) ? make_float2(xs, ws) : make_float2(ws, xs);
}
__device__ __forceinline__ float4 four(uint64_t a, uint64_t b) {
  float4 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(a));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.z), "=f"(v.w) : "l"(b));
  return v;
}
// Scales kb .. kb + 3 of a row, 1 past the last group or row.
__device__ __forceinline__ float4 scale4(const float* scale, int row, int rows, int kb, int groups, int vec) {
  if (row >= rows || kb >= groups) return make_float4(1.f, 1.f, 1.f, 1.f);
  const float* s = scale + (size_t)row * groups + kb;
  if (vec) return *reinterpret_cast<const float4*>(s);
  return make_float4(s[0], kb + 1 < groups ? s[1] : 1.f, kb + 2 < groups ? s[2] : 1.f, kb + 3 < groups ? s[3] : 1.f);
}
__device__ __forceinline__ float of4(const float4& v, int i) { return i < 2 ? (i == 0 ? v.x : v.y) : (i == 2 ? v.z : v.w); }
// acc + bias for four columns from n on (8 or 16 aligned bytes, the same for all lanes).
template <typename O>
__device__ __forceinline__ void add_bias4(uint64_t* acc, const O* bias, int n) {
  float b[4];
  if constexpr (sizeof(O) == 4) {
    const float4 v = *reinterpret_cast<const float4*>(bias + n);
    b[0] = v.x; b[1] = v.y; b[2] = v.z; b[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(bias + n);
    b[0] = __uint_as_float(v.x << 16); b[1] = __uint_as_float(v.x & 0xffff0000u);
    b[2] = __uint_as_float(v.y << 16); b[3] = __uint_as_float(v.y & 0xffff0000u);
  }
  const float4 s = four(acc[0], acc[1]);
  acc[0] = pair(s.x + b[0], s.y + b[1]);
  acc[1] = pair(s.z + b[2], s.w + b[3]);
}
// A 32-byte sector of a row: 8 fp32 or 16 bf16 outputs.
template <typename O>
__device__ __forceinline__ void store_sector(O* dst, const uint64_t* acc) {
  constexpr int V = 32 / sizeof(O);
  float f[V];
#pragma unroll
  for (int j = 0; j < V; j += 4) {
    const float4 v = four(acc[j / 2], acc[j / 2 + 1]);
    f[j] = v.x; f[j + 1] = v.y; f[j + 2] = v.z; f[j + 3] = v.w;
  }
  uint32_t w[8];
  if constexpr (sizeof(O) == 4) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(f[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// Four consecutive outputs of a row from column n on.
template <typename O>
__device__ __forceinline__ void store_out4(O* row, int n, int N, float4 v, const O* bias, bool vec) {
  const float f[4] = {v.x, v.y, v.z, v.w};
  if (vec && n + 4 <= N) {
    float b[4] = {0.f, 0.f, 0.f, 0.f};
    if (bias) {
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = to_f32(bias[n + j]);
    }
    if constexpr (sizeof(O) == 4) {
      *reinterpret_cast<float4*>(row + n) = make_float4(f[0] + b[0], f[1] + b[1], f[2] + b[2], f[3] + b[3]);
    } else {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0] + b[0], f[1] + b[1]);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(f[2] + b[2], f[3] + b[3]);
      *reinterpret_cast<uint2*>(row + n) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n + j < N) row[n + j] = from_f32<O>(f[j] + (bias ? to_f32(bias[n + j]) : 0.f));
}
}  // namespace f8

struct Fp8GemmParams {
  const float* xs;        // [T, groups]
  const float* ws;        // [ceil(N / 128), groups]
  const void* bias;       // [N] or null
  void* out;              // [T, N]
  const int32_t* T_dev;   // or null
  int T, N, groups, splits, box_m, vec, wblocks;
  int vec_xs, vec_ws;     // rows of scales take 16-byte loads
  int vec32;              // rows of out take 32-byte stores, bias 16-byte loads
  int* err;
  unsigned long long wait_ns;
};

// SPLIT: the tile's K is divided among the CTAs of a cluster.
template <int BN, typename O, bool SPLIT>
__global__ void __launch_bounds__(f8::THREADS, 1)
f8_gemm_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
               const Fp8GemmParams p) {
  using namespace f8;
  using C = Cfg<BN>;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* scales = reinterpret_cast<float*>(smem + RING_BYTES);       // [SCALE_SLOTS][SCALE_LD]
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + SCALE_SLOTS * SCALE_LD);   // [STAGES]
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;    // [BUFS]
  uint64_t* tempty = tfull + BUFS;
  uint64_t* mma_done = tempty + BUFS;
  uint32_t* tmem_base_sm = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_sm + 1);
  int* groups_sent = reinterpret_cast<int*>(tmem_base_sm + 2);   // by the operands' and the scales' producer

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // A dependent launch (10 x 20480 x 4096 called in a row: 19.0 us, not 21.6): what
  // touches no memory of the caller's goes before the wait.
  // (TMEM does not: the kernel before may still be about to allocate its own.)
  if (warp == 1 && lane == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], TMA_WARPS);
      mbar_init(&empty[s], C::PARTS);
    }
    for (int a = 0; a < BUFS; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], SUM_WARPS / C::PARTS);
    }
    mbar_init(mma_done, MMA_WARPS);
    *abort_flag = 0;
    fence_barrier_init();
  } else if (warp >= SUM_WARPS + MMA_WARPS && lane == 0) {
    prefetch_tensor_map(warp == SUM_WARPS + MMA_WARPS ? &wmap : &xmap);
  }
  __syncwarp();
  wait_for_prior_grid();
  dependents_may_launch();

  const int T = p.T_dev ? min(*p.T_dev, p.T) : p.T;
  const int nt = (p.N + BN - 1) / BN;
  const int tiles = nt * ((T + BM - 1) / BM);
  const int S = SPLIT ? p.splits : 1;
  const int rank = SPLIT ? (int)ctarank() : 0;
  const int first = (int)blockIdx.x / S, step = (int)gridDim.x / S;
  if (first >= tiles) return;             // (every CTA of the cluster)
  const int kb0 = (int)((long)rank * p.groups / S), kb1 = (int)((long)(rank + 1) * p.groups / S);

  // The producers need the barriers alone: their first loads go out while TMEM is allocated.
  uint32_t tmem_base = 0;
  if (warp >= SUM_WARPS + MMA_WARPS) {
    named_sync(2, 32 * (TMA_WARPS + 1));
  } else {
    if (warp == 0) tmem_alloc(tmem_base_sm, 512);
    __syncwarp();
    if (warp == 1) named_sync(2, 32 * (TMA_WARPS + 1));
    tc_fence_before();
    named_sync(3, 32 * (SUM_WARPS + MMA_WARPS));
    tc_fence_after();
    tmem_base = *tmem_base_sm;
  }

  // The issuing warps run converged and let one lane issue: what the TMA and MMA
  // instructions take then sits in uniform registers. Barriers and commits cost an
  // MMA issuer some 400 cycles of latency a round all the same, as much as the tensor
  // core needs for an accumulator, so there are two. The scales have a warp of their
  // own: beside the rows' copies they held narrow tiles at 345 ns a group, not 240.
  if (warp >= SUM_WARPS + MMA_WARPS) {
    // ------------------------------ producers: operands (TMA), scales ------------------------------
    const bool leader = elect_one(), operands = warp == SUM_WARPS + MMA_WARPS;
    int stage = 0;
    int issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint32_t bytes = (uint32_t)((p.box_m + BN) * G);
    const uint64_t once = l2_policy_evict_first();
    const bool stream_w = T <= BM;          // each weight is read by one tile alone
    // Scales come four groups at a time (16 bytes a row; one group at a time, by every
    // summing warp, cost the L1 32 lines a warp and group and took longer than the
    // MMAs), read four groups ahead.
    float4 cur[5];                          // rows lane + 32 i; weight block `lane` of the tile
    for (int tile = first; ok && tile < tiles; tile += step) {
      const int m0 = tile / nt * BM, n0 = tile % nt * BN;
      auto fetch = [&](int kb) {            // groups kb .. kb + 3 (kb a multiple of 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) cur[i] = scale4(p.xs, m0 + 32 * i + lane, T, kb, p.groups, p.vec_xs);
        cur[4] = scale4(p.ws, lane < C::PARTS ? tile % nt * C::PARTS + lane : p.wblocks, p.wblocks, kb, p.groups, p.vec_ws);
      };
      if (!operands) fetch(kb0 & ~3);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait(&empty[stage], phase ^ 1u, abort_flag, p.err, 21, p.wait_ns)) { ok = false; break; }
        if (operands) {
          uint8_t* dst = smem + stage * C::STAGE;
          if (leader) {
            mbar_arrive_expect_tx(&full[stage], bytes);
            if (stream_w) tma_load_2d_hint(dst + A_BYTES, &wmap, &full[stage], kb * G, n0, once);
            else tma_load_2d(dst + A_BYTES, &wmap, &full[stage], kb * G, n0);
            tma_load_2d(dst, &xmap, &full[stage], kb * G, m0);
          }
        } else {
          if (kb == kb0 || kb % 4 == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {     // group kb - kb % 4 + j
              const int ahead = j - kb % 4;
              if (ahead < 0 || kb + ahead >= kb1) continue;
              float* sc = scales + (issued + ahead) % SCALE_SLOTS * SCALE_LD;
#pragma unroll
              for (int i = 0; i < 4; ++i) sc[32 * i + lane] = of4(cur[i], j);
              if (lane < C::PARTS) sc[BM + lane] = of4(cur[4], j);
            }
            __syncwarp();
            fetch((kb & ~3) + 4);
          }
          if (leader) mbar_arrive(&full[stage]);
        }
        ++issued;
        if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    if (lane == 0) groups_sent[operands ? 0 : 1] = issued;
    __syncwarp();
  } else if (warp >= SUM_WARPS) {
    // ------------------------------ MMA issuers ------------------------------
    // They take the accumulators in turn; each accumulator is filled by the MMAs of
    // one group alone, so these need no order among themselves.
    const bool leader = elect_one();
    bool ok = true;
    const uint32_t idesc = idesc_e4m3(BM, BUF_N);
    const uint64_t desc0 = sdesc_sw128(smem_u32(smem));
    int n = 0;                              // groups of all tiles so far
    for (int tile = first; ok && tile < tiles; tile += step)
      for (int kb = kb0; ok && kb < kb1; ++kb, ++n)
#pragma unroll
        for (int part = 0; part < C::PARTS; ++part) {
          const int u = n * C::PARTS + part;
          if (u % MMA_WARPS != warp - SUM_WARPS) continue;
          const int stage = n % C::STAGES, buf = u % BUFS;
          // (the address field counts 16 bytes, and the ring stays below its 2^14 of them)
          const uint64_t adesc = desc0 + (uint64_t)(stage * (C::STAGE / 16));
          const uint64_t bdesc = adesc + (A_BYTES + part * BUF_N * G) / 16;
          const uint32_t d_tmem = tmem_base + (uint32_t)(buf * BUF_N);
          // the operands are here before the accumulator is free
          if (!warp_wait(&full[stage], (uint32_t)(n / C::STAGES) & 1u, abort_flag, p.err, 23, p.wait_ns) ||
              !warp_wait(&tempty[buf], ((uint32_t)(u / BUFS) & 1u) ^ 1u, abort_flag, p.err, 22, p.wait_ns)) { ok = false; break; }
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int j = 0; j < G / 32; ++j)   // 32 bytes of K per instruction
              mma_e4m3(d_tmem, adesc + (uint64_t)(j * 2), bdesc + (uint64_t)(j * 2), idesc, j > 0 ? 1u : 0u);
            tc_commit(&tfull[buf]);
            tc_commit(&empty[stage]);
          }
        }
    // every MMA issued by this thread has completed before TMEM is released
    if (leader) tc_commit(mma_done);
    __syncwarp();
  } else {
    // ------------------------------ sums ------------------------------
    const int quarter = warp & 3, part = warp >> 2;   // TMEM lanes [32 q, 32 q + 32) belong to warp q mod 4
    constexpr int PER = BUF_N / C::COLS;              // summing threads across an accumulator
    int u = part / PER;                               // this thread's accumulators: every PARTS-th
    bool ok = true;
    for (int tile = first; ok && tile < tiles; tile += step) {
      // some lane's sums are wanted
      const bool warp_live = tile / nt * BM + quarter * 32 < T && tile % nt * BN + part * C::COLS < p.N;
      uint64_t acc[C::COLS / 2];                      // pairs of fp32 sums
#pragma unroll
      for (int c = 0; c < C::COLS / 2; ++c) acc[c] = 0;
      for (int kb = kb0; kb < kb1; ++kb, u += C::PARTS) {
        const int buf = u % BUFS;
        if (!warp_wait(&tfull[buf], (uint32_t)(u / BUFS) & 1u, abort_flag, p.err, 25, p.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float* sc = scales + u / C::PARTS % SCALE_SLOTS * SCALE_LD;
        const float xs = sc[quarter * 32 + lane], ws = sc[BM + part / PER];
        const float f = xs * ws;
        const uint64_t s = pair(f, f);
        bool apart = false;
        const uint32_t tbase = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * BUF_N + part % PER * C::COLS);
        auto release = [&]() {                        // the warp has read it out: the MMAs may have it
          tc_fence_before();
          if (lane == 0) mbar_arrive(&tempty[buf]);
        };
        if (warp_live) {
#pragma unroll
          for (int c0 = 0; c0 < C::COLS; c0 += C::LD) {
            uint32_t r[C::LD];
            if constexpr (C::LD == 32) tmem_ld32(tbase + (uint32_t)c0, r);
            else tmem_ld16(tbase + (uint32_t)c0, r);
            // Found while the first columns are on their way. Before them, each narrow tile's
            // group took 10 % longer and a wide one's 5; marked by the scales' producer instead,
            // 10 to 20 and none; so, 6 and none (2048 x 4096 x 10240 87 -> 93 us).
            if (c0 == 0) apart = __any_sync(0xffffffffu, !in_range(f));
            tmem_ld_wait();
            if (c0 + C::LD == C::COLS) release();
            if (apart) {
              const float2 t = scales_in_turn(xs, ws);
#pragma unroll
              for (int q = 0; q < C::LD; q += 2)
                acc[(c0 + q) / 2] = fma2(pair(__uint_as_float(r[q]) * t.x, __uint_as_float(r[q + 1]) * t.x), pair(t.y, t.y),
                                         acc[(c0 + q) / 2]);
            } else {
#pragma unroll
              for (int q = 0; q < C::LD; q += 2)
                acc[(c0 + q) / 2] = fma2(pair(__uint_as_float(r[q]), __uint_as_float(r[q + 1])), s, acc[(c0 + q) / 2]);
            }
          }
        }
        else release();
      }
      // a split tile's sums go to the ring, which the other half's MMAs may still read
      if (C::PARTS > 1 && SPLIT) named_sync(1, 32 * SUM_WARPS);
      if (!ok) break;
      int done = tile;                                // (opaque: the place of the tile is found anew,
      asm volatile("" : "+r"(done));                  //  not held in registers through the loop)
      const int row = done / nt * BM + quarter * 32 + lane, n0 = done % nt * BN + part * C::COLS;
      if (!SPLIT) {
        if (row < T && n0 < p.N) {
          O* o = (O*)p.out + (size_t)row * p.N;
          constexpr int V = 32 / sizeof(O);           // a whole 32-byte sector a store
          if (p.vec32 && n0 + C::COLS <= p.N) {
            if (p.bias) {
#pragma unroll
              for (int c = 0; c < C::COLS; c += 4) add_bias4<O>(acc + c / 2, (const O*)p.bias, n0 + c);
            }
#pragma unroll
            for (int c = 0; c < C::COLS; c += V) store_sector<O>(o + n0 + c, acc + c / 2);
          } else {
#pragma unroll
            for (int c = 0; c < C::COLS; c += 4)
              store_out4<O>(o, n0 + c, p.N, four(acc[c / 2], acc[c / 2 + 1]), (const O*)p.bias, p.vec != 0);
          }
        }
      } else if (row < T) {
        // the ring is idle: its last copies have been multiplied. The tile's sums go there
        float* red = reinterpret_cast<float*>(smem) + (size_t)(quarter * 32 + lane) * C::RED_LD + part * C::COLS;
#pragma unroll
        for (int c = 0; c < C::COLS; c += 4)
          *reinterpret_cast<float4*>(red + c) = four(acc[c / 2], acc[c / 2 + 1]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // After an abort copies may still be in flight: the last one of every stage is waited
  // for (bounded), so that none lands after the CTA has exited. No role issues any more,
  // and whichever gave up has set the flag before the barrier, also where all copies had
  // been issued before. A copy whose group the scales' producer has not arrived on gets
  // that arrival here: without it its stage would never complete. (It is at most STAGES
  // groups behind: a stage is filled again after its group has been multiplied.)
  if (warp == SUM_WARPS + MMA_WARPS && lane == 0 && *abort_flag) {
    const int issued = groups_sent[0], oldest = max(0, issued - C::STAGES);
    for (int i = max(oldest, groups_sent[1]); i < issued; ++i) mbar_arrive(&full[i % C::STAGES]);
    for (int i = oldest; i < issued; ++i)
      if (!mbar_wait_bounded(&full[i % C::STAGES], (uint32_t)((i / C::STAGES) & 1), p.err, 26)) break;
  }
  __syncwarp();
  if (SPLIT) {
    cluster_sync();
    const int m0 = first / nt * BM, n0 = first % nt * BN;   // a cluster has one tile
    const int rows = min(BM, T - m0), cells = rows * (BN / 4);
    const uint32_t red = smem_u32(smem);
    for (int i = rank * THREADS + (int)threadIdx.x; i < cells; i += S * THREADS) {
      const int r = i / (BN / 4), c = (i % (BN / 4)) * 4;
      if (n0 + c >= p.N) continue;
      const uint32_t at = red + (uint32_t)(r * C::RED_LD + c) * 4u;
      float4 v = ld_peer(at, 0);
      for (int k = 1; k < S; ++k) {
        const float4 y = ld_peer(at, (uint32_t)k);
        v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
      }
      store_out4<O>((O*)p.out + (size_t)(m0 + r) * p.N, n0 + c, p.N, v, (const O*)p.bias, p.vec != 0);
    }
    cluster_sync();                       // no CTA leaves while a peer reads its sums
  }
  // every accumulator has been read, or the CTA has given up: the MMAs end (bounded)
  // before TMEM is freed
  if (warp == 0) {
    if (lane == 0) mbar_wait_bounded(mma_done, 0, p.err, 24);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Tile width and split over K: the pair of least estimated time. A round of
// clusters takes, in nanoseconds, 280 a group for a narrow tile or 470 for a wide
// one, over the split, and for its start and end 5000 or 10500 whole, 6500 or 10000
// with the sum over the cluster; a GB300 holds 152, 76, 36 and 15 clusters of 1, 2,
// 4 and 8 CTAs, one an SM, at once. The constants are those of least loss over 90
// measured products of 1 to 2048 rows, 512 to 20480 values and 512 to 32000 columns:
// the choice is 0.3 % slower than the best of the eight in the mean and 7 % at most.
// Measured then (narrow against wide, us): 8190 x 20480 x 4096 615 against 531 whole, 400
// x 4096 x 10240 33 against 40; 10 x 4096 x 10240 13.4 whole, 15.5 wide in two parts.
struct Fp8Plan { int BN, S; };
static Fp8Plan fp8_plan(int T, int N, int groups) {
  static const int kSplit[4] = {1, 2, 4, 8}, kResident[4] = {152, 76, 36, 15};
  static const long kGroup[2] = {280, 470}, kEnds[2][2] = {{5000, 6500}, {10500, 10000}};
  const long mt = (T + f8::BM - 1) / f8::BM;
  Fp8Plan best{128, 1};
  long least = -1;
  for (int BN = 128; BN <= 256; BN += 128)
    for (int i = 0; i < 4; ++i) {
      const int S = kSplit[i];
      if (S > groups) break;
      const long rounds = (mt * ((N + BN - 1) / BN) + kResident[i] - 1) / kResident[i];
      const long ns = rounds * (kGroup[BN > 128] * ((groups + S - 1) / S) + kEnds[BN > 128][S > 1]);
      if (least < 0 || ns < least) {
        least = ns;
        best = Fp8Plan{BN, S};
      }
    }
  return best;
}

template <int BN, typename O, bool SPLIT>
static cudaError_t launch_f8_gemm_t(const Fp8GemmArgs& a, int S) {
  using namespace f8;
  Fp8GemmParams p{};
  p.xs = a.x_scale; p.ws = a.w_scale; p.bias = a.bias; p.out = a.out; p.T_dev = a.T_dev;
  p.T = a.T; p.N = a.N; p.groups = (a.K + G - 1) / G; p.splits = S;
  p.box_m = std::min(BM, (a.T + 7) / 8 * 8);
  auto aligned = [](const void* q, size_t n) { return reinterpret_cast<uintptr_t>(q) % n == 0; };
  p.vec = aligned(a.out, 16) && a.N % 4 == 0;
  p.vec32 = aligned(a.out, 32) && (size_t)a.N * sizeof(O) % 32 == 0 && aligned(a.bias, 16);
  p.wblocks = (a.N + G - 1) / G;
  p.vec_xs = p.groups % 4 == 0 && aligned(a.x_scale, 16);
  p.vec_ws = p.groups % 4 == 0 && aligned(a.w_scale, 16);
  p.err = a.err; p.wait_ns = wait_limit_ns();
  CUtensorMap xmap, wmap;
  const uint64_t xd[2] = {(uint64_t)a.K, (uint64_t)a.T}, wd[2] = {(uint64_t)a.K, (uint64_t)a.N};
  const uint64_t strides[1] = {(uint64_t)a.K};
  const uint32_t xb[2] = {G, (uint32_t)p.box_m}, wb[2] = {G, BN};
  if (!encode_tensor_map(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(a.x), xd, strides, xb,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tensor_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(a.w), wd, strides, wb,
                         CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorNotSupported;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.ensure(f8_gemm_kernel<BN, O, SPLIT>, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const long tiles = (long)((a.T + BM - 1) / BM) * ((a.N + BN - 1) / BN);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(S > 1 ? tiles * S : std::min(tiles, 152L)));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = a.stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = S;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, f8_gemm_kernel<BN, O, SPLIT>, xmap, wmap, p);
}

template <typename O>
static cudaError_t launch_f8_gemm_o(const Fp8GemmArgs& a) {
  const Fp8Plan plan = fp8_plan(a.T, a.N, (a.K + f8::G - 1) / f8::G);
  if (plan.BN == 256)
    return plan.S > 1 ? launch_f8_gemm_t<256, O, true>(a, plan.S) : launch_f8_gemm_t<256, O, false>(a, 1);
  return plan.S > 1 ? launch_f8_gemm_t<128, O, true>(a, plan.S) : launch_f8_gemm_t<128, O, false>(a, 1);
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a) {
  return a.out_dtype == 0 ? launch_f8_gemm_o<float>(a) : launch_f8_gemm_o<bf16>(a);
}

}  // namespace dflash
