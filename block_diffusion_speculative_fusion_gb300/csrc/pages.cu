// Block tables and slot maps of the paged KV cache, built on the device from
// the sequences' lengths, so that a decode round's bookkeeping needs no host.
//   [SGLang] 5.1: KV headroom before the draft, given back after the verify;
//   req_to_token: logical position -> physical slot.
//
// Both operators are one launch in which every CTA forms the prefix sums over
// the sequences itself (a few KB of lengths, from L2), which costs less than a
// second launch or a wait between CTAs; the pages and rows are then divided
// among the CTAs. Both are dependent launches, whose start overlaps the end of the
// kernel before. Bound: the launch and two dependent loads for a decode
// round, the bytes written for a prefill's slot map. Measured: resize of 64
// sequences 3.8 us, of 1024 with a quarter admitted whole 8.0; slot map of 64 x 16
// rows 5.4 us, of 512 prompts (4.2 million rows, 67 MB stored) 14.6.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace dflash {

namespace pages {
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSegment = 128;            // pages that a warp moves at once
}  // namespace pages

// Exclusive prefix of one value per thread over the block, and the total.
__device__ __forceinline__ long long block_prefix(long long x, long long* total) {
  __shared__ long long s_w[pages::kWarps];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  long long in = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, in, o);
    if (l >= o) in += y;
  }
  __syncthreads();   // the array may still be read from the call before
  if (l == 31) s_w[w] = in;
  __syncthreads();
  long long base = 0, all = 0;
#pragma unroll
  for (int i = 0; i < pages::kWarps; ++i) {
    const long long v = s_w[i];
    base += i < w ? v : 0;
    all += v;
  }
  *total = all;
  return base + in - x;
}

// ---------------------------------------------------------------------------
// Block tables resized. The free list (a stack of n_free pages) is taken as
// extended by the pages given back, in sequence order; `pool` is its length
// then. Growing sequences take pages from its end, in sequence order; one whose
// pages, together with those asked for before it, exceed the pool gets none.
// Pages given back land at free_pages[n_free ..], which no CTA reads: a page
// taken from that part is looked up in the table row that gives it back (rows
// of shrinking sequences are not written), so no CTA waits for another, and
// the same inputs give the same outputs when the call is repeated.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(pages::kThreads)
pages_resize_kernel(const PagesArgs a) {
  using namespace pages;
  wait_for_prior_grid();
  dependents_may_launch();
  __shared__ int s_give[kPagesMaxB + 1];    // pages given back before sequence b
  __shared__ int s_want[kPagesMaxB + 1];    // pages asked for before sequence b
  const int tid = threadIdx.x, B = a.B;
  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  const int n_free = min(max(*a.n_free, 0), a.num_pages);
  auto held = [&](int b) { return min(max(a.n_pages[b], 0), a.max_pages); };
  // pages that the length takes; -1: more than a row of the table holds
  auto need = [&](int b) {
    const int n = max(a.length[b], 0);
    const int k = n / a.page_size + (n % a.page_size != 0);
    return k > a.max_pages ? -1 : k;
  };
  long long give = 0, want = 0;
  for (int b = b0; b < b1; ++b) {
    const int h = held(b), k = need(b);
    s_give[b] = k >= 0 ? max(h - k, 0) : 0;
    s_want[b] = k >= 0 ? max(k - h, 0) : 0;
    give += s_give[b];
    want += s_want[b];
  }
  // B * max_pages < 2^31: the sums fit an int
  long long all_give, all_want;
  int ge = (int)block_prefix(give, &all_give), we = (int)block_prefix(want, &all_want);
  for (int b = b0; b < b1; ++b) {
    const int g = s_give[b], w = s_want[b];
    s_give[b] = ge;
    s_want[b] = we;
    ge += g;
    we += w;
  }
  if (tid == 0) {
    s_give[B] = (int)all_give;
    s_want[B] = (int)all_want;
  }
  __syncthreads();
  const int pool = (int)min((long long)n_free + all_give, (long long)a.num_pages);
  // (more pages given back than the pool has: the surplus is dropped, not written)

  // a warp's unit is kSegment consecutive pages of one sequence, given back or
  // taken: all loads first (one by one, a whole prompt's 512 pages cost 16 round trips)
  const int lane = tid & 31, segs = (a.max_pages + kSegment - 1) / kSegment;
  const long units = (long)B * segs;
  for (long unit = (long)blockIdx.x * kWarps + (tid >> 5); unit < units; unit += (long)gridDim.x * kWarps) {
    const int b = (int)(unit / segs), i0 = (int)(unit - (long)b * segs) * kSegment + lane;
    const int h = held(b), k = need(b);
    const int g0 = s_give[b], g = s_give[b + 1] - g0;
    const int w0 = s_want[b], w = s_want[b + 1] - w0;
    int32_t* row = a.page_table + (size_t)b * a.max_pages;
    const bool granted = s_want[b + 1] <= pool;
    if (i0 == 0) {
      a.n_pages_out[b] = h - g + (granted ? w : 0);
      if (a.short_) a.short_[b] = k < 0 || (w > 0 && !granted);
    }
    const int n = granted ? w : 0;         // a sequence gives or takes, never both
    int page[kSegment / 32];
#pragma unroll
    for (int q = 0; q < kSegment / 32; ++q) {
      const int i = i0 + 32 * q;
      if (i < g) page[q] = row[k + i];
      if (i < n) {
        const int pos = pool - 1 - (w0 + i);
        if (pos < n_free) {
          page[q] = a.free_pages[pos];
        } else {
          // the last sequence whose pages start at or before this one
          const int f = pos - n_free;
          int lo = 0, hi = B - 1;
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_give[mid] <= f) lo = mid; else hi = mid - 1;
          }
          page[q] = a.page_table[(size_t)lo * a.max_pages + need(lo) + (f - s_give[lo])];
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kSegment / 32; ++q) {
      const int i = i0 + 32 * q;
      if (i < g && n_free + g0 + i < a.num_pages) a.free_pages[n_free + g0 + i] = page[q];
      if (i < n) row[h + i] = page[q];
    }
  }
  if (blockIdx.x == 0) {
    // granted sequences are those whose prefix fits: the largest prefix is what is taken
    long long taken = 0;
    for (int b = b0; b < b1; ++b)
      if (s_want[b + 1] <= pool) taken += s_want[b + 1] - s_want[b];
    long long total;
    block_prefix(taken, &total);
    if (tid == 0) *a.n_free_out = pool - (int)total;
  }
}

cudaError_t launch_pages_resize(const PagesArgs& a, int num_sms) {
  const long units = (long)a.B * ((a.max_pages + pages::kSegment - 1) / pages::kSegment);
  const int grid = (int)std::min((long)num_sms, (units + pages::kWarps - 1) / pages::kWarps);
  return launch_dependent(pages_resize_kernel, dim3(grid), dim3(pages::kThreads), 0, a.stream, a);
}

// ---------------------------------------------------------------------------
// Slot map of a ragged batch: the rows of all sequences, one after the other.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(pages::kThreads, 3)
slot_map_kernel(const SlotArgs a) {
  using namespace pages;
  wait_for_prior_grid();
  dependents_may_launch();
  constexpr int U = 4;                       // consecutive rows per thread: 16- and 32-byte stores
  extern __shared__ int slot_smem[];
  int* s_cu = slot_smem;                     // [B + 1] first row of each sequence
  int* s_off = slot_smem + a.B + 1;          // [B] position less row
  const int tid = threadIdx.x, B = a.B, T_max = a.rows_max;
  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  long long sum = 0, total;
  for (int b = b0; b < b1; ++b) sum += max(a.n_rows[b], 0);
  long long at = block_prefix(sum, &total);
  for (int b = b0; b < b1; ++b) {
    const int c = (int)min(at, (long long)T_max);
    s_cu[b] = c;
    s_off[b] = (int)((unsigned)a.start_pos[b] - (unsigned)c);
    if (blockIdx.x == 0) a.cu_rows[b] = c;
    at += max(a.n_rows[b], 0);
  }
  const int T = (int)min(total, (long long)T_max);
  if (tid == 0) {
    s_cu[B] = T;
    if (blockIdx.x == 0) a.cu_rows[B] = T;
  }
  __syncthreads();
  const int lane = tid & 31;
  for (long w0 = ((long)blockIdx.x * kThreads + tid - lane) * U; w0 < T_max; w0 += (long)gridDim.x * kThreads * U) {
    const long t0 = w0 + lane * U;
    // the last sequence that starts at or before the warp's first row, 32 ways at a
    // time; the lanes walk on from there
    int b = 0;
    if (w0 < T) {
      int lo = 0, n = B;                     // in [lo, lo + n), s_cu[lo] <= w0
      while (n > 1) {
        const int step = (n + 31) / 32, i = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, lane * step < n && s_cu[i] <= (int)w0);
        const int k = 31 - __clz((int)m);    // bit 0 is set
        n = min(step, n - k * step);
        lo += k * step;
      }
      b = lo;
    }
    int seq[U], pos[U];
    long long slot[U];
    // first slot of the page that position q of sequence b lies in, -1 without one
    auto page_slot = [&](int q, int lp) -> long long {
      if (q < 0 || lp >= a.max_pages) return -1;
      const int page = a.page_table[(size_t)b * a.max_pages + lp];
      return page >= 0 && page < a.num_pages ? (long long)page * a.page_size : -1;
    };
#pragma unroll
    for (int u = 0; u < U; ++u) seq[u] = pos[u] = -1, slot[u] = -1;
    if (t0 < T) {
      while (s_cu[b + 1] <= (int)t0) ++b;    // past the sequences that end before; t0 < T ends it
      const int q = (int)((unsigned)s_off[b] + (unsigned)t0), lp = q / a.page_size, in_page = q - lp * a.page_size;
      if ((unsigned)q <= (unsigned)(INT32_MAX - U) && (int)t0 + U <= s_cu[b + 1] && U <= a.page_size) {
        // the usual case: all U rows in one sequence, so in one page or two
        const long long base = page_slot(q, lp);
        const long long next = in_page + U > a.page_size ? page_slot(q, lp + 1) : -1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = in_page + u;
          const bool over = i >= a.page_size;
          const long long x = over ? next : base;
          seq[u] = b;
          pos[u] = q + u;
          slot[u] = x >= 0 ? x + (over ? i - a.page_size : i) : -1;
        }
      } else {
#pragma unroll 1
        for (int u = 0; u < U && t0 + u < T; ++u) {
          const int t = (int)t0 + u;
          while (s_cu[b + 1] <= t) ++b;
          const int v = (int)((unsigned)s_off[b] + (unsigned)t);
          const long long base = page_slot(v, v / a.page_size);
          const long long x = base >= 0 ? base + v % a.page_size : -1;
#pragma unroll
          for (int k = 0; k < U; ++k)
            if (k == u) seq[k] = b, pos[k] = v, slot[k] = x;
        }
      }
    }
    if (a.vec && t0 + U <= T_max) {
      *reinterpret_cast<int4*>(a.row_seq + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(a.slots + t0), "l"(slot[0]), "l"(slot[1]),
                   "l"(slot[2]), "l"(slot[3])
                   : "memory");
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t0 + u < T_max) {
          a.row_seq[t0 + u] = seq[u];
          a.positions[t0 + u] = pos[u];
          a.slots[t0 + u] = slot[u];
        }
    }
  }
}

cudaError_t launch_slot_map(const SlotArgs& args, int num_sms) {
  SlotArgs a = args;
  auto al = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  a.vec = al(a.row_seq, 16) && al(a.positions, 16) && al(a.slots, 32);
  const long need = ((long)a.rows_max + 4 * pages::kThreads - 1) / (4 * pages::kThreads);
  const int grid = (int)std::max(1L, std::min((long)num_sms * 3, need));
  return launch_dependent(slot_map_kernel, dim3(grid), dim3(pages::kThreads), (2 * (size_t)a.B + 1) * sizeof(int),
                          a.stream, a);
}

}  // namespace dflash
