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
// Bound: one read and one write of the rows. A CTA owns 2048 tokens of one
// sequence's vocabulary, a 16-byte vector a thread (bf16) or two (fp32), for all
// its rows. Without lists
// it streams them through registers, four rows in flight a thread, with the
// mask alone: a vector that the mask forbids whole is written without being
// read, and in place a vector without a masked token is neither read nor
// written. With lists the rows pass through shared memory, four at a time in
// two stages (cp.async keeps up to 32 KB a CTA in flight whatever the threads
// do); between a stage's arrival and its way out the CTA mends the tokens that
// have a rule, of which there are few: one (token, row) pair a thread, out of a
// list compacted in shared memory.
//
// What is known of the tokens, two words each, comes from the history, which
// the CTAs of a cluster of up to eight read once between them: each adds its
// part of it to the tokens' owners (distributed shared memory) while the first
// rows are on their way. (Three rows a stage and five CTAs an SM instead of four
// and four: 87 us, not 82, for the case below.)
//
// Measured, 64 sequences x 16 rows x 128256 bf16, histories up to 8192, 64 biases,
// half of the sequences masked: 84 us for 359 MB (0.63 of the copy bandwidth); the
// masks alone 66 us (0.80); in place 83, and 77 without masks (the first two stages
// are asked for before it is known which vectors have a rule). 8 x 10 rows x 100003
// fp32: 15.5 us, in place 15 (every vector of rows at any alignment is written back);
// one row: 4.7 us. Buffers whose vectors do not meet go token by token: 472 and 40 us.
#include <cstddef>

#include "common.cuh"
#include "internal.h"
#include "stream.cuh"
#include "tma.cuh"

namespace dflash {

namespace rules {
constexpr int kVecs = 256;               // threads
constexpr int kVecsInFlight = 4;         // vectors of a thread in a stage
constexpr int kStages = 2;
constexpr int kCtasPerSm = 4;            // 54 KB of shared memory each
constexpr int kHistAhead = 4;            // history tokens a thread asks for before the first wait
constexpr int kMaxCluster = 8;
// a token's word: occurrences in the output, and
constexpr uint32_t kCountMask = (1u << kRulesCountBits) - 1;
constexpr uint32_t kCand = 1u << 30;     // the token is among the candidates
constexpr uint32_t kPrompt = 1u << 31;   // the token is in the prompt
static_assert(kRulesCountBits <= 30, "token word");

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Address of this CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void red_add(uint32_t a, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void red_or(uint32_t a, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void red_max(uint32_t a, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
}  // namespace rules

struct RulesParams {
  int R, V, H, nb, W, in_place;
  int lists;   // penalties or biases are given
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
    // the two bits spread over their halves of the word
    const uint32_t lo = (uint32_t)((int)(ok << (31 - 2 * q)) >> 31), hi = (uint32_t)((int)(ok << (30 - 2 * q)) >> 31);
    const uint32_t m = __byte_perm(lo, hi, 0x7610);
    w[q] = (w[q] & m) | (0xff80ff80u & ~m);
  }
}

// Shared memory of a CTA: the stages, then what is known of the tokens.
template <typename T>
struct RulesSmem {
  static constexpr int VPT = 8 / VecTraits<T>::N;                  // vectors of a thread in a row
  static constexpr int UR = rules::kVecsInFlight / VPT;            // rows of a stage
  static constexpr int C = rules::kVecs * VPT * VecTraits<T>::N;   // tokens of a chunk
  // vectors start where the row's address is a multiple of 16 bytes, up to a
  // vector less one token past the chunk's start: the words reach that far
  static constexpr int CW = C + VecTraits<T>::N;
  uint4 stage[rules::kStages][rules::kVecsInFlight][rules::kVecs];   // [row, vector of the thread][thread]
  alignas(16) uint32_t word[CW];    // occurrences
  alignas(16) uint32_t entry[CW];   // the last bias entry plus one; then its value's bits
  uint16_t list[CW];       // the tokens that have a rule
  int32_t cand[kRulesMaxRows];
  int n;                   // length of list
};

// EVEN: logits and out start on 16 bytes and V is a multiple of a vector, so
// that every row's vectors start at the chunk's first token.
template <typename T, bool EVEN>
__global__ void __launch_bounds__(rules::kVecs, rules::kCtasPerSm)
rules_kernel(const T* logits, T* out, const RulesParams p) {
  using namespace rules;
  wait_for_prior_grid();                     // a dependent launch: its start overlaps the kernel before
  dependents_may_launch();
  constexpr int N = VecTraits<T>::N;
  constexpr int U = kVecsInFlight, VPT = RulesSmem<T>::VPT, UR = RulesSmem<T>::UR;
  constexpr uint32_t kAll = (1u << N) - 1;
  constexpr int C = RulesSmem<T>::C, CW = RulesSmem<T>::CW;
  extern __shared__ uint4 rules_smem[];
  RulesSmem<T>& sm = *reinterpret_cast<RulesSmem<T>*>(rules_smem);
  // clusters of low tokens, which text repeats most, start first: they mend most
  const int b = blockIdx.y, tid = threadIdx.x;
  const int chunk = blockIdx.z * gridDim.x + blockIdx.x;
  const int c0 = chunk * C;                  // past V in the CTAs that fill up a cluster
  if (p.lists) {
    static_assert(offsetof(RulesSmem<T>, entry) == offsetof(RulesSmem<T>, word) + 4 * CW && CW % 4 == 0, "words, then entries");
    for (int i = tid; i < CW / 2; i += kVecs) reinterpret_cast<uint4*>(sm.word)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) sm.n = 0;
    __syncthreads();
    cluster_arrive();                        // (with the wait below: the cluster's words are zero)
  }
  const int nd = p.n_draft ? min(max(p.n_draft[b], 0), p.R - 1) : p.R - 1;
  const float theta = p.repetition ? p.repetition[b] : 1.f;
  const float phi = p.frequency ? p.frequency[b] : 0.f;
  const float pi = p.presence ? p.presence[b] : 0.f;
  const int n_hist = p.hist ? min(max(p.hist_len[b], 0), p.H) : 0;
  const int n_prompt = p.prompt_len ? min(max(p.prompt_len[b], 0), n_hist) : 0;
  const bool penal = theta != 1.f || phi != 0.f || pi != 0.f;
  const bool any = penal || p.nb > 0;
  const bool masked = p.mask != nullptr && (p.mask_on == nullptr || p.mask_on[b] != 0);
  const T* z0 = logits + (size_t)b * p.R * p.V;
  T* o0 = out + (size_t)b * p.R * p.V;
  const uint32_t* m0 = masked ? p.mask + (size_t)b * p.R * p.W : nullptr;
  // both buffers' rows have to start their vectors at the same token
  const bool vec = EVEN || ((reinterpret_cast<uintptr_t>(z0) ^ reinterpret_cast<uintptr_t>(o0)) & 15) == 0;
  // tokens of row r before its first vector
  auto head = [&](int r) -> int {
    if (EVEN) return 0;
    return (int)(((16u - (unsigned)(reinterpret_cast<uintptr_t>(z0 + (size_t)r * p.V) & 15u)) & 15u) / sizeof(T));
  };
  // what row r makes of logit z of token c0 + i
  auto apply = [&](float z, int i, int r) -> float {
    const uint32_t w = sm.word[i];
    int c = (int)(w & kCountMask);
    if (w & kCand)                           // (a candidate further on does not count yet)
      for (int k = 1; k <= r; ++k) c += sm.cand[k] == c0 + i ? 1 : 0;
    if (c > 0 || (w & kPrompt)) z = z > 0.f ? __fdiv_rn(z, theta) : z * theta;
    if (c > 0) z = __fsub_rn(__fsub_rn(z, __fmul_rn(phi, (float)c)), pi);
    const uint32_t v = sm.entry[i];
    return v ? z + __uint_as_float(v) : z;
  };
  // a token that no vector holds: its logit if the mask allows it, then what becomes of it
  auto load_one = [&](int e, int r, bool* good) -> T {
    *good = !m0 || ((m0[(size_t)r * p.W + (e >> 5)] >> (e & 31)) & 1);
    return *good ? z0[(size_t)r * p.V + e] : from_f32<T>(-CUDART_INF_F);
  };
  auto store_one = [&](int e, int r, T z, bool good) {
    const int i = e - c0;
    const bool ruled = any && (sm.word[i] | sm.entry[i]) != 0;
    if (p.in_place && good && !ruled) return;
    o0[(size_t)r * p.V + e] = good && ruled ? from_f32<T>(apply(to_f32(z), i, r)) : z;
  };
  // The chunk's tokens of row r that no vector holds (EVEN: none): j < N before its
  // first one, j < 2 N after its last; -1 if there is no such token.
  auto edge = [&](int r, int j) -> int {
    const int h = min(head(r), p.V);
    if (j < N) return c0 == 0 && j < h ? j : -1;
    const int k = (p.V - h) / N, e = h + k * N + j - N;
    return k / (kVecs * VPT) == chunk && e < p.V ? e : -1;
  };
  // those of all rows from thread place `k` on, or every token where the buffers'
  // vectors do not meet
  auto edges = [&](int k) {
    if (EVEN) return;
    bool good;
    if (vec) {
      for (; k < 2 * N * (nd + 1); k += kVecs) {
        const int r = k / (2 * N), e = edge(r, k % (2 * N));
        if (e < 0) continue;
        const T z = load_one(e, r, &good);
        store_one(e, r, z, good);
      }
    } else {
      for (int r = 0; r <= nd; ++r)
#pragma unroll 4
        for (int e = c0 + tid; e < min(p.V, c0 + C); e += kVecs) {
          const T z = load_one(e, r, &good);
          store_one(e, r, z, good);
        }
    }
  };
  // The thread's U vectors of group g: slot u is vector u % VPT of row g * UR + u / VPT.
  auto row_of = [&](int g, int u) { return g * UR + u / VPT; };
  auto token_of = [&](int r, int u) { return head(r) + c0 + (tid + u % VPT * kVecs) * N; };   // its first
  auto has_vec = [&](int r, int u) { return r <= nd && vec && token_of(r, u) + N <= p.V; };
  // What the thread reads of row r's mask for slot u (one register, so that it can be on
  // its way for long), and the allowed bits of its vector, bit j for token j. EVEN: the
  // byte that holds them. Else a lane reads one of the N + 1 words under its warp's
  // vectors, and all lanes of the warp take part in handing them round (each lane
  // joining its own two words waited for them a stage early: 8 x 10 rows, 3 us).
  const int lane = tid & 31;
  auto mask_words = [&](int r, int u) -> uint32_t {
    if constexpr (EVEN) {
      if (!m0 || !has_vec(r, u)) return 0xffffffffu;
      return reinterpret_cast<const uint8_t*>(m0 + (size_t)r * p.W)[token_of(r, u) / 8];
    } else {
      if (!m0) return 0xffffffffu;
      const int w = ((token_of(r, u) - lane * N) >> 5) + lane;
      return r <= nd && lane <= N && w < p.W ? m0[(size_t)r * p.W + w] : 0u;
    }
  };
  auto allowed = [&](uint32_t words, int r, int u) -> uint32_t {
    if constexpr (EVEN) {
      words = N < 8 ? words >> (tid * N & 7) : words;
    } else {
      const int bit = ((token_of(r, u) - lane * N) & 31) + lane * N;
      words = __funnelshift_r(__shfl_sync(0xffffffffu, words, bit >> 5), __shfl_sync(0xffffffffu, words, (bit >> 5) + 1), bit);
    }
    return has_vec(r, u) ? words & kAll : 0u;
  };
  auto at_vec = [&](int r, int u) -> size_t { return (size_t)r * p.V + token_of(r, u); };

  if (!any) {
    if (p.lists) cluster_wait();
    if (c0 >= p.V) return;
    for (int g = 0; g * UR <= nd; ++g) {
      uint32_t ok[U];
      uint4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) ok[u] = mask_words(row_of(g, u), u);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = row_of(g, u);
        ok[u] = allowed(ok[u], r, u);
        if (ok[u] && !(p.in_place && ok[u] == kAll)) x[u] = ld_once16(z0 + at_vec(r, u));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = row_of(g, u);
        if (!has_vec(r, u) || (p.in_place && ok[u] == kAll)) continue;
        if (m0) forbid16<T>(x[u], ok[u]);
        *reinterpret_cast<uint4*>(o0 + at_vec(r, u)) = x[u];
      }
    }
    edges(tid);
    return;
  }

  // in place: bit j: the thread's vector j has no rule (once that is known)
  uint32_t plain = 0;
  // requests the thread's vectors of group g, whose mask words have been read
  // before; returns their allowed bits, a byte a vector
  auto read_mask = [&](int g, uint32_t* words) {
#pragma unroll
    for (int u = 0; u < U; ++u) words[u] = mask_words(row_of(g, u), u);
  };
  auto fetch = [&](int g, const uint32_t* words) -> uint32_t {
    uint32_t bits = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row_of(g, u);
      const uint32_t ok = allowed(words[u], r, u);
      bits |= ok << (8 * u);
      if (ok && !((plain >> (u % VPT) & 1) && ok == kAll)) cp_async16(&sm.stage[g % kStages][u][tid], z0 + at_vec(r, u));
    }
    cp_async_commit();
    return bits;
  };
  // everything that comes from memory is asked for before anything is waited for
  uint32_t cs;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(cs));
  const uint32_t rank = cluster_rank();
  const int step = (int)cs * kVecs, i0 = (int)rank * kVecs + tid;   // the thread's entries of the lists
  const int64_t* hist = p.hist + (size_t)b * p.H;
  uint32_t words[U], words1[U];
  read_mask(0, words);
  read_mask(1, words1);
  int64_t ahead[kHistAhead];
#pragma unroll
  for (int k = 0; k < kHistAhead; ++k) ahead[k] = penal && i0 + k * step < n_hist ? hist[i0 + k * step] : -1;
  for (int i = tid; i < p.R; i += kVecs) {
    const int64_t t = (p.cand && penal && i >= 1 && i <= nd) ? p.cand[(size_t)b * p.R + i] : -1;
    sm.cand[i] = t >= 0 && t < p.V ? (int32_t)t : -1;
  }
  // (row by row, a load at a time, the edges of 8 x 10 rows took 2 us longer)
  const int edge_r = tid / (2 * N), edge_e = !EVEN && vec && edge_r <= nd ? edge(edge_r, tid % (2 * N)) : -1;
  bool edge_good = false;
  T edge_z{};
  if (edge_e >= 0) edge_z = load_one(edge_e, edge_r, &edge_good);
  uint32_t ok_now = fetch(0, words);
  uint32_t ok_next = fetch(1, words1);
  read_mask(2, words);
  __syncthreads();
  cluster_wait();
  {
    const int64_t first = (int64_t)(chunk - (int)rank) * C;      // the cluster's first token
    const int span = (int)cs * C;
    // f at the token's word in its owner, and in the chunk before, whose vectors may reach it
    auto note = [&](int64_t tok, auto&& f) {
      const int64_t v = tok - first;
      if (tok < 0 || tok >= p.V || v < 0 || v >= span + N) return;
      const int owner = (int)v / C, off = (int)v % C;
      if (v < span) f((uint32_t)owner, off);
      if (!EVEN && off < N && owner >= 1) f((uint32_t)(owner - 1), off + C);
    };
    auto note_hist = [&](int64_t tok, int i) {
      note(tok, [&](uint32_t k, int off) {
        const uint32_t a = at_rank(&sm.word[off], k);
        if (i < n_prompt) red_or(a, kPrompt);
        else red_add(a, 1u);
      });
    };
    for (int i = i0; i < p.nb; i += step)    // the last entry of a token's biases counts
      note(p.bias_tok[(size_t)b * p.nb + i], [&](uint32_t k, int off) { red_max(at_rank(&sm.entry[off], k), (uint32_t)i + 1); });
    if (penal) {
#pragma unroll
      for (int k = 0; k < kHistAhead; ++k) note_hist(ahead[k], i0 + k * step);
#pragma unroll 4
      for (int i = i0 + kHistAhead * step; i < n_hist; i += step) note_hist(hist[i], i);
      for (int i = 1 + i0; i <= nd; i += step)
        note(sm.cand[i], [&](uint32_t k, int off) { red_or(at_rank(&sm.word[off], k), kCand); });
    }
  }
  cluster_arrive();
  cluster_wait();                            // every part of the lists is in
  if (c0 >= p.V) return;                     // (the whole CTA)
  // the list: eight tokens a thread (and one each of those past the chunk)
  {
    constexpr int TPT = C / kVecs;
    static_assert(TPT == 8, "tokens of a thread");
    auto ruled = [&](int i) -> bool {
      const uint32_t j = sm.entry[i];
      if (j) sm.entry[i] = __float_as_uint(p.bias_val[(size_t)b * p.nb + j - 1]);
      return (sm.word[i] | j) != 0;
    };
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < TPT / 4; ++q) {      // 16 bytes at once
      const uint4 w = reinterpret_cast<const uint4*>(sm.word)[tid * (TPT / 4) + q];
      const uint4 e = reinterpret_cast<const uint4*>(sm.entry)[tid * (TPT / 4) + q];
      m |= ((w.x | e.x ? 1u : 0u) | (w.y | e.y ? 2u : 0u) | (w.z | e.z ? 4u : 0u) | (w.w | e.w ? 8u : 0u)) << (4 * q);
      if (e.x | e.y | e.z | e.w)
        for (int j = 0; j < 4; ++j) ruled(tid * TPT + 4 * q + j);
    }
    if (!EVEN && tid < N && ruled(C + tid)) m |= 1u << TPT;
    int before = __popc(m);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    int at = 0;
    if (lane == 31 && before) at = atomicAdd(&sm.n, before);
    at = __shfl_sync(0xffffffffu, at, 31) + before - __popc(m);
    for (; m; m &= m - 1) {
      const int j = __ffs(m) - 1;
      sm.list[at++] = (uint16_t)(j < TPT ? tid * TPT + j : C + tid);
    }
  }
  __syncthreads();                           // the list is whole, every entry its value
  if (EVEN && p.in_place)
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      uint32_t any_rule = 0;
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const int i = (tid + j * kVecs) * N + q;
        any_rule |= sm.word[i] | sm.entry[i];   // (a value of 0 changes nothing)
      }
      plain |= any_rule ? 0u : 1u << j;
    }
  const int n = sm.n;
  if (edge_e >= 0) store_one(edge_e, edge_r, edge_z, edge_good);
  edges(tid + kVecs);

  // pairs (row, list entry) kVecs apart
  const int dr = n ? kVecs / n : 0, di = n ? kVecs % n : 0;
  const int r_first = n ? tid / n : 0, k_first = n ? tid % n : 0;
  for (int g = 0; g * UR <= nd; ++g) {
    cp_async_wait_one();                     // group g is here (group g + 1 may be on its way)
    __syncthreads();
    if (n) {
      const int rows = min(UR, nd + 1 - g * UR);
      for (int u = r_first, k = k_first; u < rows;) {
        const int i = sm.list[k], r = g * UR + u;
        // the token's place among the chunk's vectors; the tail of a row is in none
        const int off = i - head(r);
        if (EVEN || (vec && off >= 0 && off < C && c0 + i - off % N + N <= p.V)) {
          T* z = reinterpret_cast<T*>(sm.stage[g % kStages][u * VPT]) + off;
          *z = from_f32<T>(apply(to_f32(*z), i, r));
        }
        u += dr;
        k += di;
        if (k >= n) {
          k -= n;
          ++u;
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row_of(g, u);
      const uint32_t ok = (ok_now >> (8 * u)) & 0xffu;
      if (!has_vec(r, u) || ((plain >> (u % VPT) & 1) && ok == kAll)) continue;
      uint4 x = sm.stage[g % kStages][u][tid];
      if (m0) forbid16<T>(x, ok);
      *reinterpret_cast<uint4*>(o0 + at_vec(r, u)) = x;
    }
    ok_now = ok_next;
    ok_next = fetch(g + 2, words);
    read_mask(g + 3, words);
  }
  cp_async_wait_all();
}

template <typename T, bool EVEN>
static cudaError_t launch_rules_e(const RulesArgs& a, const RulesParams& p) {
  constexpr int C = RulesSmem<T>::C;
  const int nch = (a.V + C - 1) / C;
  // the largest cluster that the chunks fill; without lists there is nothing to share
  int cs = 1;
  if (p.lists)
    while (cs < rules::kMaxCluster && cs < nch) cs *= 2;
  const size_t smem = p.lists ? sizeof(RulesSmem<T>) : 0;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.ensure(rules_kernel<T, EVEN>, sizeof(RulesSmem<T>));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs, a.B, (nch + cs - 1) / cs);
  cfg.blockDim = dim3(rules::kVecs);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, rules_kernel<T, EVEN>, (const T*)a.logits, (T*)a.out, p);
}

template <typename T>
static cudaError_t launch_rules_t(const RulesArgs& a) {
  RulesParams p{};
  p.R = a.n_rows; p.V = a.V; p.H = a.hist_max; p.nb = a.n_bias; p.W = (a.V + 31) / 32;
  p.in_place = a.out == a.logits;
  p.lists = a.n_bias > 0 || a.repetition || a.presence || a.frequency;
  p.cand = a.cand; p.n_draft = a.n_draft; p.hist = a.hist; p.hist_len = a.hist_len; p.prompt_len = a.prompt_len;
  p.repetition = a.repetition; p.presence = a.presence; p.frequency = a.frequency;
  p.bias_tok = a.bias_tok; p.bias_val = a.bias_val; p.mask = (const uint32_t*)a.mask; p.mask_on = a.mask_on;
  auto aligned = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  const bool even = a.V % VecTraits<T>::N == 0 && aligned(a.logits) && aligned(a.out);
  return even ? launch_rules_e<T, true>(a, p) : launch_rules_e<T, false>(a, p);
}

cudaError_t launch_rules(const RulesArgs& a) { return a.dtype == 0 ? launch_rules_t<float>(a) : launch_rules_t<bf16>(a); }

}  // namespace dflash
