// Block tables and slot map of one step, built on the GPU from the sequences'
// old and new lengths, in one launch.
//
// With pages(x) = ceil(x / P): three prefix sums over the sequences (new
// tokens, pages taken, pages returned) say where each one's rows, ring
// entries and returned pages begin; everything else follows element by
// element.  The free list is a ring: pages are taken from its front and
// returned behind its end, so the entries read and the entries written are
// disjoint and no CTA has to wait for another.
//
// The work is a few bytes a token: latency bounds it.  Every CTA therefore
// repeats the prefix sums (up to 8192 sequences: 96 KB of shared memory)
// instead of handing them over through memory, and then fills its own 512
// tokens and its own sequences' pages.  A token's path is a walk over parents,
// up to 256 dependent steps: they are staged in shared memory first (512
// sequences of up to 64 drafted tokens: 17 us with the walk in global memory
// and 2048 tokens a CTA, 8 us so).  Where a tenth of them shrinks, by 60 pages
// each, looking at the pages' numbers first takes 1.3 us more (2.8 with a search
// for each page's sequence behind the prefix sums).  The ring's new state is written by
// the last CTA to finish (a ticket), since the others read the old one, which
// may be the same two words.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.h"
#include "ptx.cuh"

namespace tpk {

constexpr int kTabThreads = 512;
constexpr int kTabTokens = 512;  // tokens of one CTA, one a thread

struct Scan3 {
  long long t, p, u;
};

// Exclusive prefix sums of v over the CTA's threads; *total gets the sums.
__device__ __forceinline__ Scan3 block_scan3(Scan3 v, Scan3* warp_sums, Scan3* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Scan3 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, x.t, o);
    const long long p = __shfl_up_sync(0xffffffffu, x.p, o);
    const long long u = __shfl_up_sync(0xffffffffu, x.u, o);
    if (lane >= o) { x.t += t; x.p += p; x.u += u; }
  }
  __syncthreads();  // the previous round's readers of warp_sums are done
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  Scan3 before = {0, 0, 0}, all = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < kTabThreads / 32; ++w) {
    const Scan3 s = warp_sums[w];
    if (w < warp) { before.t += s.t; before.p += s.p; before.u += s.u; }
    all.t += s.t; all.p += s.p; all.u += s.u;
  }
  *total = all;
  return {before.t + x.t - v.t, before.p + x.p - v.p, before.u + x.u - v.u};
}

// Whether a page that the warp's sequences give back has a number outside the
// cache, or other rows that hold it: `gone` pages of the lane's sequence, from `row` on.  Four sequences at
// a time, lane = page, eight look-ups in flight.  (Not inlined: steps that only
// grow do not fetch it.)
__device__ __noinline__ bool returns_bad_page(const int32_t* row, int gone, int n_pages,
                                              const int32_t* holders) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (unsigned left = __ballot_sync(0xffffffffu, gone > 0); left;) {
    const int32_t* src[4];
    int many[4], most = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = left ? __ffs(left) - 1 : 0;
      src[k] = reinterpret_cast<const int32_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), s));
      many[k] = __shfl_sync(0xffffffffu, gone, s);
      if (!left) many[k] = 0;
      most = max(most, many[k]);
      left &= left - 1;
    }
    for (int j = lane; j < most; j += 64) {
      int page[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = j + 32 * (k & 1);
        page[k] = i < many[k >> 1] ? src[k >> 1][i] : 0;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool out = (uint32_t)page[k] >= (uint32_t)n_pages;
        const bool mine = j + 32 * (k & 1) < many[k >> 1];
        bad |= out || (holders && mine && holders[page[k]] > 1);
      }
    }
  }
  return bad;
}

__global__ void __launch_bounds__(kTabThreads) step_tables_kernel(const StepTablesArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ Scan3 warp_sums[kTabThreads / 32];
  __shared__ int32_t parents[kMaxTreeTokens + kTabTokens];
  const int n = a.n_seqs, tid = threadIdx.x;
  int32_t* qs = sm;             // [n + 1] first token
  int32_t* pop = qs + n + 1;    // [n] first page taken
  int32_t* push = pop + n;      // [n] first page returned
  pdl_launch_dependents();
  pdl_wait();
  const int first = a.free_state[0], count = a.free_state[1];
  bool bad = first < 0 || first >= a.n_pages || count < 0 || count > a.n_pages;
  auto pages = [&](int len) { return (int)fast_div((uint32_t)len + a.page_size - 1, a.div_page); };
  Scan3 done = {0, 0, 0};
  for (int base = 0; base < n; base += kTabThreads) {
    const int b = base + tid;
    Scan3 v = {0, 0, 0};
    const int32_t* row = a.table;  // the first page that the sequence gives back
    if (b < n) {
      const int o = a.old_lens[b], w = a.new_lens[b];
      if (o < 0 || w < 0 || o > a.cap || w > a.cap || w - o > a.max_new) {
        bad = true;
      } else {
        const int have = pages(o), want = pages(w);
        v.t = max(w - o, 0);
        v.p = max(want - have, 0);
        v.u = max(have - want, 0);
        if (a.holders && w > o && o < have * a.page_size) {
          // the first new token goes to the sequence's last page
          const int page = row[(int64_t)b * a.ld_table + have - 1];
          if ((uint32_t)page < (uint32_t)a.n_pages && a.holders[page] > 1) bad = true;
        }
        row += (int64_t)b * a.ld_table + want;
      }
    }
    // A page number outside the cache in a row that shrinks must not get into
    // the ring, nor a page that other rows hold.  Every CTA looks at all pages given back (this launch writes none
    // of them), so that all come to the same verdict without waiting for others.
    if (__any_sync(0xffffffffu, v.u > 0) && returns_bad_page(row, (int)v.u, a.n_pages, a.holders)) bad = true;
    Scan3 total;
    const Scan3 e = block_scan3(v, warp_sums, &total);
    if (b < n) {
      qs[b] = (int32_t)(done.t + e.t);
      pop[b] = (int32_t)(done.p + e.p);
      push[b] = (int32_t)(done.u + e.u);
    }
    done.t += total.t; done.p += total.p; done.u += total.u;
  }
  bad = bad || done.t > a.n_tokens || done.p > count || count + done.u > a.n_pages;
  bad = __syncthreads_or(bad);
  const int tokens = bad ? 0 : (int)done.t;
  if (tid == 0) {
    qs[n] = tokens;
    if (bad && blockIdx.x == 0) record_status(a.status, kStatusTableRange);
  }
  __syncthreads();
  auto ring_at = [&](int i) {  // i <= n_pages
    i += first;
    return i >= a.n_pages ? i - a.n_pages : i;
  };

  if (blockIdx.x == 0)
    for (int b = tid; b <= n; b += kTabThreads) a.q_start[b] = bad ? 0 : qs[b];

  // this CTA's tokens
  const int t0 = blockIdx.x * kTabTokens;
  const int t1 = min(a.n_tokens, t0 + kTabTokens);
  const int p0 = max(0, t0 - kMaxTreeTokens);  // a path stays within its sequence's 256 tokens
  if (a.parents) {
    for (int t = p0 + tid; t < t1; t += kTabThreads) parents[t - p0] = a.parents[t];
    __syncthreads();
  }
  for (int t = t0 + tid; t < t1; t += kTabThreads) {
    int slot = -1, position = 0, seq = -1;
    uint64_t m[kMaxTreeWords] = {0, 0, 0, 0};
    if (t < tokens) {
      int lo = 0, hi = n;  // the last sequence that begins at or before t (empty ones precede it)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (qs[mid] <= t) lo = mid; else hi = mid;
      }
      seq = lo;
      const int q0 = qs[seq], i = t - q0, old = a.old_lens[seq], l = old + i;
      const int pg = (int)fast_div((uint32_t)l, a.div_page), have = pages(old);
      const int page = pg < have ? a.table[(int64_t)seq * a.ld_table + pg]
                                 : a.free_ring[ring_at(pop[seq] + pg - have)];
      if (page < 0 || page >= a.n_pages) record_status(a.status, kStatusTableRange);
      else slot = page * a.page_size + (l - pg * a.page_size);
      int depth = i;
      if (a.parents) {
        depth = 0;
        int p = i;
        while (true) {  // p falls with every step
#pragma unroll
          for (int w = 0; w < kMaxTreeWords; ++w)
            if ((p >> 6) == w) m[w] |= 1ull << (p & 63);
          const int q = parents[q0 + p - p0];
          if (q < -1 || q >= p) record_status(a.status, kStatusTableRange);
          if (q < 0 || q >= p) break;
          p = q;
          ++depth;
        }
      } else if (a.tree_mask) {
#pragma unroll
        for (int w = 0; w < kMaxTreeWords; ++w) {
          const int bits = i + 1 - 64 * w;
          m[w] = bits >= 64 ? ~0ull : (bits > 0 ? (1ull << bits) - 1 : 0);
        }
      }
      position = old + depth;
    }
    a.slots[t] = slot;
    a.positions[t] = position;
    a.token_seq[t] = seq;
    if (a.tree_mask) {
#pragma unroll
      for (int w = 0; w < kMaxTreeWords; ++w)
        if (w < a.tree_words) a.tree_mask[(int64_t)t * a.tree_words + w] = m[w];
    }
  }

  // pages taken and returned: a warp a sequence
  if (!bad) {
    const int lane = tid & 31, warps = gridDim.x * (kTabThreads / 32);
    for (int b = blockIdx.x * (kTabThreads / 32) + (tid >> 5); b < n; b += warps) {
      const int have = pages(a.old_lens[b]), want = pages(a.new_lens[b]);
      int32_t* row = a.table + (int64_t)b * a.ld_table;
      for (int j = have + lane; j < want; j += 32) row[j] = a.free_ring[ring_at(pop[b] + j - have)];
      for (int j = want + lane; j < have; j += 32)
        a.free_ring[ring_at(count + push[b] + j - want)] = row[j];
    }
  }

  // the ring's new state, once every CTA has read the old one
  __syncthreads();
  if (tid == 0) {
    bool last = gridDim.x == 1;
    if (!last) {
      fence_acq_rel_gpu();
      last = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
    }
    if (last) {
      if (gridDim.x > 1) *a.ticket = 0;
      a.free_next[0] = bad ? first : ring_at((int)done.p);
      a.free_next[1] = bad ? count : count - (int)done.p + (int)done.u;
    }
  }
}

cudaError_t launch_step_tables(const StepTablesArgs& a, cudaStream_t st) {
  const size_t smem = (size_t)(3 * a.n_seqs + 1) * sizeof(int32_t);
  if (smem > 40 * 1024) {
    // the largest size, whatever this call's: another thread's call may be about to launch
    constexpr int kMost = (3 * kMaxStepSeqs + 1) * (int)sizeof(int32_t);
    cudaError_t e = cudaFuncSetAttribute(step_tables_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  const int by_tokens = (int)(((int64_t)a.n_tokens + kTabTokens - 1) / kTabTokens);
  return launch_k(step_tables_kernel, dim3(by_tokens > 1 ? by_tokens : 1), dim3(kTabThreads), smem, st,
                  a);
}

}  // namespace tpk
