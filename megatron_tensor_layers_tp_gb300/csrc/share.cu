// Page tables whose rows share pages: forks (with rows shortened and freed by the
// same call) and compaction.
//
// Both count, for every page, the rows that hold it: from the tables themselves,
// so that no reference count has to be kept up elsewhere.  Then every page and
// every row follows from the counts and from prefix sums over pages and rows, in
// order, which makes the results independent of timing.
//
// One launch: the CTAs (at most one an SM, launched together) wait for each
// other between the passes.  A wait gives up after about 2 s and reports it.
// The counts lie in the workspace, zero between calls.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "paged.h"
#include "ptx.cuh"

namespace tpk {

constexpr int kShThreads = 512, kShWarps = kShThreads / 32;
constexpr int kShRows = 8;  // rows of a tile, 32 columns wide

// Sum of v over the CTA; all threads get it.
__device__ __forceinline__ int block_sum(int v) {
  __shared__ int sums[kShWarps];
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kShWarps; ++w) all += sums[w];
  return all;
}
// Threads before this one with the flag set; *total: those of the CTA.
__device__ __forceinline__ int block_rank(bool flag, int* total) {
  __shared__ int sums[kShWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned m = __ballot_sync(0xffffffffu, flag);
  __syncthreads();
  if (lane == 0) sums[warp] = __popc(m);
  __syncthreads();
  int before = __popc(m & ((1u << lane) - 1)), all = 0;
#pragma unroll
  for (int w = 0; w < kShWarps; ++w) {
    if (w < warp) before += sums[w];
    all += sums[w];
  }
  *total = all;
  return before;
}

// Every CTA waits for the others; what they wrote before is visible after.
// False when it gave up.
__device__ __forceinline__ bool grid_wait(ShareHeader* h, int which, int* status) {
  if (gridDim.x == 1) {
    __syncthreads();
    return true;
  }
  __shared__ int ok;
  __syncthreads();
  if (threadIdx.x == 0) {
    fence_acq_rel_gpu();
    atomicAdd(&h->arrived[which], 1u);
    ok = 1;
    volatile unsigned* p = &h->arrived[which];
    const long long t0 = clock64();
    while (*p < gridDim.x) {
      if (clock64() - t0 > kWaitLimitCycles) {
        record_status(status, kStatusTimeout);
        ok = 0;
        break;
      }
    }
    fence_acq_rel_gpu();
  }
  __syncthreads();
  return ok;
}

// The last CTA to come here clears the header.
__device__ __forceinline__ void leave(ShareHeader* h) {
  __syncthreads();
  if (threadIdx.x != 0) return;
  bool last = gridDim.x == 1;
  if (!last) {
    fence_acq_rel_gpu();
    last = atomicAdd(&h->done, 1u) == gridDim.x - 1;
  }
  if (last) {
    h->arrived[0] = h->arrived[1] = h->arrived[2] = h->arrived[3] = 0;
    h->done = h->bad = 0;
  }
}

// The CTA's share of n things: [first, end).
__device__ __forceinline__ void share_of(int n, int* first, int* end) {
  const int64_t G = gridDim.x, c = blockIdx.x;
  *first = (int)(c * n / G);
  *end = (int)((c + 1) * n / G);
}

// Adds what comes to the same page in consecutive calls in one go.
struct RefRun {
  int page;
  uint32_t refs;
  __device__ __forceinline__ void add(PageNote* notes, int p, uint32_t r) {
    if (p != page) {
      flush(notes);
      page = p;
    }
    refs += r;
  }
  __device__ __forceinline__ void flush(PageNote* notes) {
    if (refs) atomicAdd(&notes[page].refs, refs);
    refs = 0;
  }
};

// Row b of the fork: its source and the tokens it keeps; false: out of bounds.
__device__ __forceinline__ bool fork_row(const ForkArgs& a, int b, int* old, int* src, int* keep) {
  int o = a.old_lens[b], s = a.src[b], k = 0;
  bool ok = o >= 0 && o <= a.cap && s >= -1 && s < a.n_seqs;
  if (ok && s >= 0) {
    const int have = a.old_lens[s];
    k = a.keep_lens ? a.keep_lens[b] : have;
    ok = have >= 0 && have <= a.cap && k >= 0 && k <= have;
  }
  *old = ok ? o : 0;
  *src = ok ? s : -1;
  *keep = ok ? k : 0;
  return ok;
}

__global__ void __launch_bounds__(kShThreads) fork_pages_kernel(const ForkArgs a) {
  __shared__ uint32_t copied[kMaxStepSeqs / 32];  // the CTA's rows that take a page
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.n_seqs, P = a.page_size;
  const int first = a.free_state[0], count = a.free_state[1];
  auto pages = [&](int len) { return (int)fast_div((uint32_t)len + P - 1, a.div_page); };
  bool bad = first < 0 || first >= a.n_pages || count < 0 || count > a.n_pages;

  // Pass 1: references, and the new rows as if no page were copied.
  const int row_tiles = (n + kShRows - 1) / kShRows;
  const int col_tiles = max(1, (min(a.ld_table, pages(a.cap)) + 31) / 32);
  for (int64_t t = (int64_t)blockIdx.x * kShWarps + warp; t < (int64_t)row_tiles * col_tiles;
       t += (int64_t)gridDim.x * kShWarps) {
    const int b0 = (int)(t / col_tiles) * kShRows, col = (int)(t % col_tiles) * 32 + lane;
    int old = 0, src = -1, keep = 0;
    if (lane < kShRows && b0 + lane < n) bad |= !fork_row(a, b0 + lane, &old, &src, &keep);
    int was[kShRows], is[kShRows], part[kShRows];
#pragma unroll
    for (int r = 0; r < kShRows; ++r) {
      const int b = b0 + r, o = __shfl_sync(0xffffffffu, old, r), s = __shfl_sync(0xffffffffu, src, r);
      const int k = __shfl_sync(0xffffffffu, keep, r);
      was[r] = b < n && col < pages(o) ? a.table[(int64_t)b * a.ld_table + col] : -1;
      is[r] = s >= 0 && col < pages(k) ? a.table[(int64_t)s * a.ld_table + col] : -1;
      part[r] = (col + 1) * (int64_t)P > k;  // the row goes on writing to it
      bad |= (b < n && col < pages(o) && (uint32_t)was[r] >= (uint32_t)a.n_pages) ||
             (s >= 0 && col < pages(k) && (uint32_t)is[r] >= (uint32_t)a.n_pages);
    }
    RefRun before = {0, 0}, after = {0, 0};
#pragma unroll
    for (int r = 0; r < kShRows; ++r) {
      if ((uint32_t)was[r] < (uint32_t)a.n_pages) before.add(a.notes, was[r], 0x10000u);
      if ((uint32_t)is[r] < (uint32_t)a.n_pages) {
        a.table_out[(int64_t)(b0 + r) * a.ld_table + col] = is[r];
        if (part[r]) atomicMax(&a.notes[is[r]].first, (uint32_t)(n - b0 - r));
        else after.add(a.notes, is[r], 1u);
      }
    }
    before.flush(a.notes);
    after.flush(a.notes);
  }
  if (__syncthreads_or(bad) && tid == 0) atomicOr(&a.head->bad, 1u);
  if (!grid_wait(a.head, 0, a.status)) return;

  // Pass 2: pages that no row holds any more, rows that take a page.
  bad = *(volatile unsigned*)&a.head->bad;
  int p0, p1, b0, b1;
  share_of(a.n_pages, &p0, &p1);
  share_of(n, &b0, &b1);
  auto gone = [&](uint2 note) { return note.x >> 16 && !(note.x & 0xFFFF) && !note.y; };
  auto note_of = [&](int p) { return __ldcg(reinterpret_cast<const uint2*>(a.notes + p)); };
  // the page that row b goes on writing to, or -1
  auto open_page = [&](int b, int* keep, int* src) {
    int old;
    fork_row(a, b, &old, src, keep);
    const int full = (int)fast_div((uint32_t)*keep, a.div_page);
    if (*src < 0 || full * P == *keep) return -1;
    return a.table[(int64_t)*src * a.ld_table + full];
  };
  int freed = 0, taken = 0;
  if (!bad) {
    for (int p = p0 + tid; p < p1; p += kShThreads) freed += gone(note_of(p));
    for (int base = b0; base < b1; base += kShThreads) {
      const int b = base + tid;
      bool copy = false;
      if (b < b1) {
        int keep, src;
        const int p = open_page(b, &keep, &src);
        if (p >= 0) {
          const uint2 note = note_of(p);
          copy = (note.x & 0xFFFF) || note.y != (uint32_t)(n - b);
        }
      }
      const unsigned m = __ballot_sync(0xffffffffu, copy);
      if (lane == 0) copied[(base - b0) / 32 + warp] = m;
      taken += copy;
    }
  }
  freed = block_sum(freed);
  taken = block_sum(taken);
  if (tid == 0) {
    a.head->counts[0][blockIdx.x] = freed;
    a.head->counts[1][blockIdx.x] = taken;
  }
  if (!grid_wait(a.head, 1, a.status)) return;

  // Pass 3: the ring, the rows' own pages, the moves.
  int f_before = 0, f_all = 0, t_before = 0, t_all = 0;
  for (int c = tid; c < (int)gridDim.x; c += kShThreads) {
    const int f = __ldcg(&a.head->counts[0][c]), t = __ldcg(&a.head->counts[1][c]);
    f_all += f;
    t_all += t;
    if (c < (int)blockIdx.x) {
      f_before += f;
      t_before += t;
    }
  }
  f_all = block_sum(f_all);
  t_all = block_sum(t_all);
  f_before = block_sum(f_before);
  t_before = block_sum(t_before);
  bad = bad || t_all > count || count + f_all > a.n_pages;
  auto ring_at = [&](int i) {
    i += first;
    return i >= a.n_pages ? i - a.n_pages : i;
  };
  for (int base = p0; base < p1; base += kShThreads) {
    const int p = base + tid;
    uint2 note = make_uint2(0, 0);
    if (p < p1) {
      note = note_of(p);
      if (note.x || note.y) *reinterpret_cast<uint2*>(a.notes + p) = make_uint2(0, 0);
    }
    if (bad) continue;
    int many;
    const int at = f_before + block_rank(gone(note), &many);
    f_before += many;
    if (gone(note)) a.free_ring[ring_at(count + at)] = p;
    if (a.holders && (note.x || note.y)) {
      const int full = note.x & 0xFFFF;
      a.holders[p] = full ? full : note.y != 0;
    }
  }
  for (int base = b0; base < b1; base += kShThreads) {
    const int b = base + tid;
    const bool copy = !bad && b < b1 && (copied[(base - b0) / 32 + warp] >> lane & 1);
    int many;
    const int at = t_before + block_rank(copy, &many);
    t_before += many;
    if (b >= b1) continue;
    if (bad) {
      a.new_lens[b] = a.old_lens[b];
      continue;
    }
    int keep, src;
    const int p = open_page(b, &keep, &src);
    a.new_lens[b] = keep;
    if (copy) {
      const int full = (int)fast_div((uint32_t)keep, a.div_page), to = a.free_ring[ring_at(at)];
      const bool out = (uint32_t)to >= (uint32_t)a.n_pages;
      if (out) record_status(a.status, kStatusTableRange);
      a.table_out[(int64_t)b * a.ld_table + full] = to;
      if (a.holders && !out) a.holders[to] = 1;
      a.moves[3 * at] = p;
      a.moves[3 * at + 1] = to;
      a.moves[3 * at + 2] = keep - full * P;
    }
  }
  if (bad) {  // the old rows again
    const int64_t words = (int64_t)n * a.ld_table;
    for (int64_t i = (int64_t)blockIdx.x * kShThreads + tid; i < words; i += (int64_t)gridDim.x * kShThreads)
      a.table_out[i] = a.table[i];
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (bad) record_status(a.status, kStatusTableRange);
    a.free_next[0] = bad ? first : ring_at(t_all);
    a.free_next[1] = bad ? count : count - t_all + f_all;
    *a.n_moves = bad ? 0 : t_all;
  }
  leave(a.head);
}

__global__ void __launch_bounds__(kShThreads) compact_pages_kernel(const CompactArgs a) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.n_seqs, P = a.page_size;
  auto pages = [&](int len) { return (int)fast_div((uint32_t)len + P - 1, a.div_page); };
  const int first = a.free_state[0], count = a.free_state[1];
  bool bad = false;

  // Pass 1: references.
  const int row_tiles = (n + kShRows - 1) / kShRows;
  const int col_tiles = max(1, (min(a.ld_table, pages(a.cap)) + 31) / 32);
  auto for_tiles = [&](auto&& f) {
    for (int64_t t = (int64_t)blockIdx.x * kShWarps + warp; t < (int64_t)row_tiles * col_tiles;
         t += (int64_t)gridDim.x * kShWarps) {
      const int b0 = (int)(t / col_tiles) * kShRows, col = (int)(t % col_tiles) * 32 + lane;
      int len = 0;
      if (lane < kShRows && b0 + lane < n) {
        len = a.lens[b0 + lane];
        if (len < 0 || len > a.cap) {
          bad = true;
          len = 0;
        }
      }
      int page[kShRows];
#pragma unroll
      for (int r = 0; r < kShRows; ++r) {
        const bool held = col < pages(__shfl_sync(0xffffffffu, len, r));
        page[r] = held ? a.table[(int64_t)(b0 + r) * a.ld_table + col] : -1;
        if (held && (uint32_t)page[r] >= (uint32_t)a.n_pages) {
          bad = true;
          page[r] = -1;
        }
      }
      f(b0, col, page);
    }
  };
  for_tiles([&](int, int, const int(&page)[kShRows]) {
    RefRun run = {0, 0};
#pragma unroll
    for (int r = 0; r < kShRows; ++r)
      if (page[r] >= 0) run.add(a.notes, page[r], 1u);
    run.flush(a.notes);
  });
  if (__syncthreads_or(bad) && tid == 0) atomicOr(&a.head->bad, 1u);
  if (!grid_wait(a.head, 0, a.status)) return;

  // Pass 2: pages held, by share.
  bad = *(volatile unsigned*)&a.head->bad;
  int p0, p1;
  share_of(a.n_pages, &p0, &p1);
  int held = 0;
  for (int p = p0 + tid; p < p1; p += kShThreads) held += __ldcg(&a.notes[p].refs) != 0;
  held = block_sum(held);
  if (tid == 0) a.head->counts[0][blockIdx.x] = held;
  if (!grid_wait(a.head, 1, a.status)) return;

  // Pass 3: with h held pages below p, the free page p < U is the (p - h)-th hole, the
  // held page p >= U the (U - 1 - h)-th to move, from the highest on.
  int before = 0, used = 0;
  for (int c = tid; c < (int)gridDim.x; c += kShThreads) {
    const int h = __ldcg(&a.head->counts[0][c]);
    used += h;
    if (c < (int)blockIdx.x) before += h;
  }
  used = block_sum(used);
  before = block_sum(before);
  for (int base = p0; base < p1; base += kShThreads) {
    const int p = base + tid;
    uint32_t refs = 0;
    if (p < p1) {
      refs = __ldcg(&a.notes[p].refs);
      if (refs) a.notes[p].refs = 0;
    }
    int many;
    const int h = before + block_rank(refs != 0, &many);
    before += many;
    if (p >= p1) continue;
    if (bad) {
      if (a.ring_out != a.ring) a.ring_out[p] = a.ring[p];
      continue;
    }
    a.ring_out[p] = p;
    if (p == used - 1) *a.n_moves = p - h + (refs == 0);  // the holes
    if (p < used && !refs) {
      a.moves[3 * (p - h) + 1] = p;
      a.moves[3 * (p - h) + 2] = P;
    } else if (p >= used && refs) {
      const int move = used - 1 - h;
      a.moves[3 * move] = p;
      *reinterpret_cast<int2*>(&a.notes[p].move) = make_int2(move, (int)refs);
      if (a.holders) a.holders[p] = 0;
    } else if (p < used && a.holders) {
      a.holders[p] = (int)refs;
    } else if (a.holders) {
      a.holders[p] = 0;
    }
  }
  if (!grid_wait(a.head, 2, a.status)) return;

  // Pass 4: the rows' pages by their new names.
  if (bad) {
    if (a.table_out != a.table) {
      const int64_t words = (int64_t)n * a.ld_table;
      for (int64_t i = (int64_t)blockIdx.x * kShThreads + tid; i < words; i += (int64_t)gridDim.x * kShThreads)
        a.table_out[i] = a.table[i];
    }
  } else {
    for_tiles([&](int b0, int col, const int(&page)[kShRows]) {
#pragma unroll
      for (int r = 0; r < kShRows; ++r) {
        if (page[r] < 0) continue;
        int to = page[r];
        if (to >= used) {
          const int2 note = __ldcg(reinterpret_cast<const int2*>(&a.notes[to].move));
          to = __ldcg(&a.moves[3 * note.x + 1]);
          if (a.holders) a.holders[to] = note.y;  // (every row that holds it writes the same)
        }
        a.table_out[(int64_t)(b0 + r) * a.ld_table + col] = to;
      }
    });
  }
  if (blockIdx.x == 0) {
    if (tid == 0) {
      if (bad) record_status(a.status, kStatusTableRange);
      if (bad || used == 0) *a.n_moves = 0;
      a.free_next[0] = bad ? first : used == a.n_pages ? 0 : used;
      a.free_next[1] = bad ? count : a.n_pages - used;
    }
  }
  leave(a.head);
}

template <typename Args>
static cudaError_t launch_shared(void (*kernel)(Args), const Args& a, int64_t entries, int num_sms,
                                 cudaStream_t st) {
  const int64_t tiles = (entries + kShThreads * kShRows - 1) / (kShThreads * kShRows);
  const int64_t by_pages = (a.n_pages + 4095) / 4096;
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(std::max(tiles, by_pages), std::min(num_sms, kShareCtas)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kShThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = grid > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_fork_pages(const ForkArgs& a, int num_sms, cudaStream_t st) {
  const int64_t cols = std::min<int64_t>(a.ld_table, (a.cap + (int64_t)a.page_size - 1) / a.page_size);
  return launch_shared(fork_pages_kernel, a, cols * a.n_seqs, num_sms, st);
}

cudaError_t launch_compact_pages(const CompactArgs& a, int num_sms, cudaStream_t st) {
  const int64_t cols = std::min<int64_t>(a.ld_table, (a.cap + (int64_t)a.page_size - 1) / a.page_size);
  return launch_shared(compact_pages_kernel, a, cols * a.n_seqs, num_sms, st);
}

}  // namespace tpk
