// Rules on the logits of the verify rows: penalties for repeated tokens,
// sparse biases and grammar masks.
//
// Sequence b's row r holds the logits after the committed tokens and the
// candidates cand[b, 1 .. r], so its history is the committed one plus those.
// With c(v) the number of times token v occurs in the output (the history past
// the prompt, and the candidates up to r), and v "seen" when c(v) > 0 or v is
// in the prompt:
//   z <- seen ? (z > 0 ? z / repetition : z * repetition) : z
//   z <- z - frequency * c(v) - presence * [c(v) > 0] + bias(v)
//   z <- -inf where the mask's bit of v is 0
// in fp32, rounded to the I/O type once; a token that no rule touches keeps
// its bits.
//
// Bound: one read and one write of the rows. A CTA owns a chunk of the
// vocabulary of one sequence, for all its rows: it gathers the history's counts
// and the bias entries of its tokens once, in shared memory (one word a token),
// and streams the rows past them. Few tokens have a rule: one bit a token tells
// a 16-byte vector that none of its tokens has, and such a vector is copied. A
// vector that the mask forbids whole is written without being read; in place,
// a vector without a rule is neither read nor written.
#include "common.cuh"
#include "internal.h"

namespace dflash {

namespace rules {
constexpr int kThreads = 256;
// the word of a token in shared memory
constexpr uint32_t kCountMask = (1u << kRulesCountBits) - 1;            // occurrences in the output
constexpr int kBiasShift = kRulesCountBits;                             // last bias entry of the token, plus one
constexpr uint32_t kBiasMask = (1u << kRulesBiasBits) - 1;
constexpr uint32_t kCand = 1u << 30;                                    // the token is among the candidates
constexpr uint32_t kPrompt = 1u << 31;                                  // the token is in the prompt
static_assert(kRulesCountBits + kRulesBiasBits <= 30, "token word");
}  // namespace rules

struct RulesParams {
  int R, V, H, nb, W, chunk, in_place;
  const int64_t* cand;
  const int32_t* n_draft;
  const int64_t* hist;
  const int32_t* hist_len;
  const int32_t* prompt_len;
  const float* repetition;
  const float* presence;
  const float* frequency;
  const int64_t* bias_tok;
  const float* bias_val;
  const uint32_t* mask;
  const uint8_t* mask_on;
};

__device__ __forceinline__ uint4 ld_rows16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

// Element j (a run-time index) of a 16-byte vector, read and replaced.
__device__ __forceinline__ uint32_t vec_word(const uint4& u, int i) {
  return i < 2 ? (i == 0 ? u.x : u.y) : (i == 2 ? u.z : u.w);
}
__device__ __forceinline__ void set_vec_word(uint4& u, int i, uint32_t w) {
  u.x = i == 0 ? w : u.x;
  u.y = i == 1 ? w : u.y;
  u.z = i == 2 ? w : u.z;
  u.w = i == 3 ? w : u.w;
}
template <typename T> __device__ __forceinline__ float vec_get(const uint4& u, int j);
template <> __device__ __forceinline__ float vec_get<float>(const uint4& u, int j) { return __uint_as_float(vec_word(u, j)); }
template <> __device__ __forceinline__ float vec_get<bf16>(const uint4& u, int j) {
  const uint32_t w = vec_word(u, j >> 1);
  return (j & 1) ? bf16_hi(w) : bf16_lo(w);
}
template <typename T> __device__ __forceinline__ void vec_set(uint4& u, int j, float v);
template <> __device__ __forceinline__ void vec_set<float>(uint4& u, int j, float v) { set_vec_word(u, j, __float_as_uint(v)); }
template <> __device__ __forceinline__ void vec_set<bf16>(uint4& u, int j, float v) {
  const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rn(v)), w = vec_word(u, j >> 1);
  set_vec_word(u, j >> 1, (j & 1) ? (w & 0xffffu) | (h << 16) : (w & 0xffff0000u) | h);
}

// Element j of a 16-byte vector set to -inf where bit j of `ok` is 0.
template <typename T> __device__ __forceinline__ void forbid16(uint4& u, uint32_t ok);
template <> __device__ __forceinline__ void forbid16<float>(uint4& u, uint32_t ok) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (!((ok >> j) & 1)) w[j] = 0xff800000u;
}
template <> __device__ __forceinline__ void forbid16<bf16>(uint4& u, uint32_t ok) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (!((ok >> (2 * q)) & 1)) w[q] = (w[q] & 0xffff0000u) | 0xff80u;
    if (!((ok >> (2 * q + 1)) & 1)) w[q] = (w[q] & 0xffffu) | 0xff800000u;
  }
}

// n bits (n <= 8) of a bit array at bit `at`; `words` is its length in words.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* a, int at, int n, int words) {
  const int w = at >> 5, s = at & 31;
  uint32_t x = a[w] >> s;
  if (s + n > 32 && w + 1 < words) x |= a[w + 1] << (32 - s);
  return x & ((1u << n) - 1);
}

template <typename T>
__global__ void __launch_bounds__(rules::kThreads)
rules_kernel(const T* __restrict__ logits, T* __restrict__ out, const RulesParams p) {
  using namespace rules;
  constexpr int N = VecTraits<T>::N;
  constexpr uint32_t kAll = (1u << N) - 1;
  extern __shared__ uint32_t sm[];
  uint32_t* word = sm;                       // [chunk] what is known of each token
  uint32_t* rule = sm + p.chunk;             // [chunk / 32] bit: some row changes the token
  __shared__ int32_t s_cand[kRulesMaxRows];
  const int b = blockIdx.y, tid = threadIdx.x;
  const int c0 = blockIdx.x * p.chunk, c1 = min(p.V, c0 + p.chunk), len = c1 - c0;
  const int nd = p.n_draft ? min(max(p.n_draft[b], 0), p.R - 1) : p.R - 1;

  const float theta = p.repetition ? p.repetition[b] : 1.f;
  const float phi = p.frequency ? p.frequency[b] : 0.f;
  const float pi = p.presence ? p.presence[b] : 0.f;
  const bool penal = theta != 1.f || phi != 0.f || pi != 0.f;
  const bool any = penal || p.nb > 0;
  const bool masked = p.mask != nullptr && (p.mask_on == nullptr || p.mask_on[b] != 0);

  if (any) {
    for (int i = tid; i < p.chunk + p.chunk / 32; i += kThreads) sm[i] = 0;
    for (int i = tid; i < p.R; i += kThreads) {
      const int64_t t = (p.cand && penal && i >= 1 && i <= nd) ? p.cand[(size_t)b * p.R + i] : -1;
      s_cand[i] = t >= 0 && t < p.V ? (int32_t)t : -1;
    }
    __syncthreads();
    // the last entry of a token's biases counts
    for (int i = tid; i < p.nb; i += kThreads) {
      const int64_t t = p.bias_tok[(size_t)b * p.nb + i] - c0;
      if (t >= 0 && t < len) {
        atomicMax(&word[t], (uint32_t)(i + 1) << kBiasShift);
        atomicOr(&rule[t >> 5], 1u << (t & 31));
      }
    }
    __syncthreads();
    if (penal) {
      const int n = p.hist ? min(max(p.hist_len[b], 0), p.H) : 0;
      const int np = p.prompt_len ? min(max(p.prompt_len[b], 0), n) : 0;
      const int64_t* h = p.hist + (size_t)b * p.H;
      auto note = [&](int64_t tok, int i) {
        const int64_t t = tok - c0;
        if (t >= 0 && t < len) {
          if (i < np) atomicOr(&word[t], kPrompt);
          else atomicAdd(&word[t], 1u);
          atomicOr(&rule[t >> 5], 1u << (t & 31));
        }
      };
      for (int i = tid; i < n; i += kThreads) note(h[i], i);
      for (int i = 1 + tid; i <= nd; i += kThreads) {
        const int t = s_cand[i] - c0;
        if (t >= 0 && t < len) {
          atomicOr(&word[t], kCand);
          atomicOr(&rule[t >> 5], 1u << (t & 31));
        }
      }
    }
    __syncthreads();
  }

  // what row r makes of logit z of token e
  auto apply = [&](float z, int e, int r) -> float {
    const uint32_t w = word[e - c0];
    int c = (int)(w & kCountMask);
    if (w & kCand)
      for (int i = 1; i <= r; ++i) c += s_cand[i] == e ? 1 : 0;
    if (c > 0 || (w & kPrompt)) z = z > 0.f ? __fdiv_rn(z, theta) : z * theta;
    if (c > 0) z = __fsub_rn(__fsub_rn(z, __fmul_rn(phi, (float)c)), pi);
    const uint32_t j = (w >> kBiasShift) & kBiasMask;
    if (j) z += p.bias_val[(size_t)b * p.nb + j - 1];
    return z;
  };
  // whether row r changes token e at all (a candidate further on does not count yet)
  auto touched = [&](int e, int r) -> bool {
    const uint32_t w = word[e - c0];
    if (w & ~kCand) return true;
    for (int i = 1; i <= r; ++i)
      if (s_cand[i] == e) return true;
    return false;
  };

  constexpr int U = 4;
  for (int r = 0; r <= nd; ++r) {
    const size_t row = (size_t)b * p.R + r;
    const T* z = logits + row * p.V;
    T* o = out + row * p.V;
    const uint32_t* mk = masked ? p.mask + row * p.W : nullptr;
    auto one = [&](int e) {
      const bool ok = !mk || ((mk[e >> 5] >> (e & 31)) & 1);
      const bool rl = any && ((rule[(e - c0) >> 5] >> ((e - c0) & 31)) & 1);
      if (p.in_place && ok && !rl) return;
      T v = from_f32<T>(-CUDART_INF_F);
      if (ok) {
        v = z[e];
        if (rl && touched(e, r)) v = from_f32<T>(apply(to_f32(v), e, r));
      }
      o[e] = v;
    };
    // both rows have to start a vector at the same token
    const uintptr_t az = reinterpret_cast<uintptr_t>(z + c0), ao = reinterpret_cast<uintptr_t>(o + c0);
    int head = len, nvec = 0;
    if (((az ^ ao) & 15) == 0) {
      head = min(len, (int)(((16u - (unsigned)(az & 15u)) & 15u) / sizeof(T)));
      nvec = (len - head) / N;
    }
    const int a0 = c0 + head;
    for (int e = c0 + tid; e < a0; e += kThreads) one(e);
    for (int e = a0 + nvec * N + tid; e < c1; e += kThreads) one(e);
    for (int v0 = tid; v0 < nvec; v0 += U * kThreads) {
      uint32_t ok[U], rl[U];
      uint4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * kThreads, e = a0 + v * N;
        ok[u] = v >= nvec ? 0u : (mk ? bits_at(mk, e, N, p.W) : kAll);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * kThreads, e = a0 + v * N;
        rl[u] = any && v < nvec ? bits_at(rule, e - c0, N, p.chunk / 32) : 0u;
        x[u] = make_uint4(0, 0, 0, 0);
        if (ok[u] && !(p.in_place && ok[u] == kAll && !rl[u])) x[u] = ld_rows16(z + e);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * kThreads, e = a0 + v * N;
        if (v >= nvec || (p.in_place && ok[u] == kAll && !rl[u])) continue;
        uint32_t todo = rl[u] & ok[u];
        while (todo) {
          const int j = __ffs(todo) - 1;
          todo &= todo - 1;
          if (touched(e + j, r)) vec_set<T>(x[u], j, apply(vec_get<T>(x[u], j), e + j, r));
        }
        if (ok[u] != kAll) forbid16<T>(x[u], ok[u]);
        *reinterpret_cast<uint4*>(o + e) = x[u];
      }
    }
  }
}

template <typename T>
static cudaError_t launch_rules_t(const RulesArgs& a, int num_sms) {
  RulesParams p{};
  p.R = a.n_rows; p.V = a.V; p.H = a.hist_max; p.nb = a.n_bias; p.W = (a.V + 31) / 32;
  p.in_place = a.out == a.logits;
  p.cand = a.cand; p.n_draft = a.n_draft; p.hist = a.hist; p.hist_len = a.hist_len; p.prompt_len = a.prompt_len;
  p.repetition = a.repetition; p.presence = a.presence; p.frequency = a.frequency;
  p.bias_tok = a.bias_tok; p.bias_val = a.bias_val; p.mask = (const uint32_t*)a.mask; p.mask_on = a.mask_on;
  // the largest chunk that still gives every SM two CTAs: each chunk's CTA reads the whole history
  p.chunk = 8192;
  while (p.chunk > 1024 && (long)a.B * ((a.V + p.chunk - 1) / p.chunk) < 2L * num_sms) p.chunk /= 2;
  const size_t smem = (size_t)(p.chunk + p.chunk / 32) * sizeof(uint32_t);
  rules_kernel<T><<<dim3((a.V + p.chunk - 1) / p.chunk, a.B), rules::kThreads, smem, a.stream>>>(
      (const T*)a.logits, (T*)a.out, p);
  return cudaGetLastError();
}

cudaError_t launch_rules(const RulesArgs& a, int num_sms) {
  return a.dtype == 0 ? launch_rules_t<float>(a, num_sms) : launch_rules_t<bf16>(a, num_sms);
}

}  // namespace dflash
