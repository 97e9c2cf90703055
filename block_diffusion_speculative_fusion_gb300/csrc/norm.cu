// Root-mean-square norm of a sum with the residual, in the input's type, in e4m3 with
// a scale for every 128 values (the rows that the 8-bit product takes), or both.
//
//   s = x + r        y = s * rsqrt(mean(s^2) + eps) * w
//   scale = max(amax / 448, 2^-126),  q = e4m3(y * (1 / scale))   amax over 1 x 128
//
// One read of x and r, one write of each output: a row's sums stay in fp32 registers
// between the sum of squares and the outputs, so that what is normed and quantised
// is not rounded to the input's type on the way. Bound: those bytes (8,190 x 4,096 bf16 with
// residual, sum and e4m3 out 42 us, 5.5 TB/s).
#include <algorithm>

#include "e4m3.cuh"
#include "internal.h"

namespace dflash {

namespace norm {
constexpr int kThreads = 256;          // of a CTA whose rows are narrow: several rows side by side
constexpr int kMaxThreads = 1024;
constexpr int kSms = 152;
constexpr int kMaxVec = 4;             // 16-byte vectors of a row that one thread holds at most
}  // namespace norm

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A row belongs to `team` consecutive warps of the CTA: the sum (or maximum) of v over it.
// Every thread of the CTA takes part. Added in one order: the same bits each time.
template <bool MAX>
__device__ __forceinline__ float team_reduce(float v, int team, float* s_part) {
  v = MAX ? warp_max(v) : warp_sum(v);
  if (team == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();                     // the array may still be read from the call before
  if (lane == 0) s_part[warp] = v;
  __syncthreads();
  v = lane < team ? s_part[warp / team * team + lane] : 0.f;
  return MAX ? warp_max(v) : warp_sum(v);
}

// A sum of squares that overflows, or that has lost digits and is not small beside eps: the
// row is then taken times a power of two that brings its largest value near 1.
__device__ __forceinline__ bool out_of_range(float ssq, float eps) {
  return !(ssq <= 3e38f) || (ssq < 1e-30f && eps < 1e-16f);
}
__device__ __forceinline__ float row_factor(float amax, float eps) {
  const int e = (int)((__float_as_uint(amax) >> 23) & 0xff);
  // (nothing but zeros, or an infinity: as it is; NaN is passed over by the maximum)
  if (amax == 0.f || e == 255) return 1.f;
  const float f = __uint_as_float((uint32_t)min(max(254 - e, 1), 253) << 23);
  return eps * f * f > 1e30f ? 1.f : f;    // the squares are nothing beside eps
}

template <typename T>
struct Vec16 {
  static constexpr int N = VecTraits<T>::N;
  static __device__ __forceinline__ uint4 pack(const float* f) {
    if constexpr (N == 4) {
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
      uint4 u;
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      return u;
    }
  }
};

// A row in the registers of its team, V vectors a thread; the team's next row is on its way
// while this one is summed, normed and packed (8,190 rows of 4,096 bf16, sum and e4m3 out:
// 42 us; a CTA for each row 48).
template <typename T, int V>
__global__ void __launch_bounds__(norm::kMaxThreads)
rms_norm_kernel(const NormArgs a, int team) {
  wait_for_prior_grid();   // a dependent launch: the rows may come from the kernel before
  dependents_may_launch();
  constexpr int N = VecTraits<T>::N, LPG = f8::G / N;   // lanes of a group
  constexpr bool AHEAD = V < 4;   // (four vectors and the next four are too many registers: a CTA for each of its rows)
  constexpr bool HOLD = V == 1;   // the weights too (two vectors' spill; they come from L1)
  __shared__ float s_part[32];
  const int warps = (int)(blockDim.x >> 5), threads = team * 32, rows = warps / team;
  const int tid = (int)threadIdx.x % threads;
  const int groups = (a.d + f8::G - 1) / f8::G;
  uint4 xv[V], rv[V], wv;
  // a vector is inside or outside: d is a multiple of N
  auto load = [&](long t) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = (v * threads + tid) * N;
      const bool in = t < a.T && k < a.d;
      xv[v] = in ? ld_once16((const T*)a.x + t * a.d + k) : make_uint4(0, 0, 0, 0);
      rv[v] = in && a.residual ? ld_once16((const T*)a.residual + t * a.d + k) : make_uint4(0, 0, 0, 0);
    }
  };
  auto weight = [&](int v) {
    const int k = (v * threads + tid) * N;
    return k < a.d ? *reinterpret_cast<const uint4*>((const T*)a.weight + k) : make_uint4(0, 0, 0, 0);
  };
  const long step = (long)gridDim.x * rows;
  long t = (long)blockIdx.x * rows + (int)threadIdx.x / threads;
  load(t);
  if constexpr (HOLD) wv = weight(0);
  for (long t0 = (long)blockIdx.x * rows; t0 < a.T; t0 += step, t += step) {
    const bool live = t < a.T;
    float s[V][N], ssq = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[N];
      unpack16<T>(xv[v], s[v]);
      if (a.residual) {
        unpack16<T>(rv[v], f);
#pragma unroll
        for (int i = 0; i < N; ++i) s[v][i] += f[i];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) ssq = fmaf(s[v][i], s[v][i], ssq);
    }
    if constexpr (AHEAD) {
      if (t0 + step < a.T) load(t + step);
    }
    if (a.sum) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int k = (v * threads + tid) * N;
        if (live && k < a.d) *reinterpret_cast<uint4*>((T*)a.sum + t * a.d + k) = Vec16<T>::pack(s[v]);
      }
    }
    ssq = team_reduce<false>(ssq, team, s_part);
    float eps = a.eps;
    const bool far = live && out_of_range(ssq, eps);
    if (__syncthreads_or(far)) {
      float m = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(s[v][i]));
      m = team_reduce<true>(m, team, s_part);
      const float f = far ? row_factor(m, eps) : 1.f;
      ssq = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          s[v][i] *= f;
          ssq = fmaf(s[v][i], s[v][i], ssq);
        }
      ssq = team_reduce<false>(ssq, team, s_part);
      eps = eps * f * f;
    }
    const float inv = __frsqrt_rn(__fdiv_rn(ssq, (float)a.d) + eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = (v * threads + tid) * N;
      float w[N];
      if constexpr (HOLD)
        unpack16<T>(wv, w);
      else
        unpack16<T>(weight(v), w);
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s[v][i] = s[v][i] * inv * w[i];
        m = fmaxf(m, fabsf(s[v][i]));
      }
      const bool in = live && k < a.d;
      if (a.y && in) *reinterpret_cast<uint4*>((T*)a.y + t * a.d + k) = Vec16<T>::pack(s[v]);
      if (a.q) {
#pragma unroll
        for (int o = LPG / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float sc = f8_scale(m), rc = __frcp_rn(sc);
        if (in) {
          uint32_t* dst = reinterpret_cast<uint32_t*>((uint8_t*)a.q + t * a.d + k);
          const uint32_t q0 = f8_pack4(s[v][0] * rc, s[v][1] * rc, s[v][2] * rc, s[v][3] * rc);
          if constexpr (N == 8)
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(q0, f8_pack4(s[v][4] * rc, s[v][5] * rc, s[v][6] * rc, s[v][7] * rc));
          else
            *dst = q0;
          if ((tid & 31) % LPG == 0) a.scale[t * groups + k / f8::G] = sc;
        }
      }
    }
    if constexpr (!AHEAD) break;
  }
}

// Rows wider than a CTA's registers hold, or not made of whole aligned vectors: the row
// is read again for the outputs (from L2 where it fits), an element a thread: rows that the
// other kernel takes too cost it three to four times as much (8,190 x 4,096 137 us).
template <typename T>
__global__ void __launch_bounds__(norm::kThreads)
rms_norm_wide_kernel(const NormArgs a) {
  wait_for_prior_grid();   // a dependent launch
  dependents_may_launch();
  __shared__ float s_part[32];
  constexpr int team = norm::kThreads / 32;
  const int tid = threadIdx.x;
  const long t = blockIdx.x;
  const T* x = (const T*)a.x + t * a.d;
  const T* r = a.residual ? (const T*)a.residual + t * a.d : nullptr;
  auto value = [&](int k) { return to_f32(x[k]) + (r ? to_f32(r[k]) : 0.f); };
  float ssq = 0.f, m = 0.f, f = 1.f;
  for (int k = tid; k < a.d; k += norm::kThreads) {
    const float v = value(k);
    ssq = fmaf(v, v, ssq);
    m = fmaxf(m, fabsf(v));
  }
  ssq = team_reduce<false>(ssq, team, s_part);
  if (out_of_range(ssq, a.eps)) {          // the same for the whole CTA
    f = row_factor(team_reduce<true>(m, team, s_part), a.eps);
    ssq = 0.f;
    for (int k = tid; k < a.d; k += norm::kThreads) {
      const float v = value(k) * f;
      ssq = fmaf(v, v, ssq);
    }
    ssq = team_reduce<false>(ssq, team, s_part);
  }
  const float inv = __frsqrt_rn(__fdiv_rn(ssq, (float)a.d) + a.eps * f * f);
  const int groups = (a.d + f8::G - 1) / f8::G;
  for (int k0 = 0; k0 < a.d; k0 += norm::kThreads) {   // two groups at a time
    const int k = k0 + tid;
    const bool in = k < a.d;
    const float v = in ? value(k) : 0.f;
    const float y = in ? v * f * inv * to_f32(((const T*)a.weight)[k]) : 0.f;
    // (an output may stand where this very element was read)
    if (a.sum && in) ((T*)a.sum)[t * a.d + k] = from_f32<T>(v);
    if (a.y && in) ((T*)a.y)[t * a.d + k] = from_f32<T>(y);
    if (a.q) {
      const float sc = f8_scale(team_reduce<true>(fabsf(y) >= 0.f ? fabsf(y) : 0.f, f8::G / 32, s_part));
      if (in) {
        ((uint8_t*)a.q)[t * a.d + k] = __nv_cvt_float_to_fp8(y * __frcp_rn(sc), __NV_SATFINITE, __NV_E4M3);
        if (tid % f8::G == 0) a.scale[t * groups + k / f8::G] = sc;
      }
    }
  }
}

template <typename T>
static cudaError_t launch_rms_norm_t(const NormArgs& a) {
  using namespace norm;
  constexpr int N = VecTraits<T>::N;
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const bool vec = a.d % N == 0 && a.d <= N * kMaxVec * kMaxThreads && al(a.x) && al(a.residual) && al(a.weight) &&
                   al(a.sum) && al(a.y);
  if (!vec)
    return launch_dependent(rms_norm_wide_kernel<T>, dim3((unsigned)a.T), dim3(kThreads), 0, a.stream, a);
  const int n = a.d / N;
  // Vectors a thread: two (8,190 x 4,096: 42 us; one 48, four 43), or one where the rows are
  // too few to fill the SMs (10 x 4,096: 2.3 us; two 2.7, four 3.7).
  const int V = n > 2048 ? 4 : n > 1024 || a.T > kSms ? 2 : 1;
  const int team = ((n + V - 1) / V + 31) / 32;
  const int rows = std::max(1, kThreads / 32 / team);   // rows side by side in a CTA
  const int per_sm = std::max(1, kMaxThreads / (rows * team * 32));   // CTAs that an SM's registers hold
  const int all = (a.T + rows - 1) / rows;
  const dim3 grid((unsigned)(V < 4 ? std::min(all, kSms * per_sm) : all)), block(rows * team * 32);
  switch (V) {
    case 1: return launch_dependent(rms_norm_kernel<T, 1>, grid, block, 0, a.stream, a, team);
    case 2: return launch_dependent(rms_norm_kernel<T, 2>, grid, block, 0, a.stream, a, team);
    default: return launch_dependent(rms_norm_kernel<T, 4>, grid, block, 0, a.stream, a, team);
  }
}

cudaError_t launch_rms_norm(const NormArgs& a) {
  return a.dtype == 0 ? launch_rms_norm_t<float>(a) : launch_rms_norm_t<bf16>(a);
}

}  // namespace dflash
