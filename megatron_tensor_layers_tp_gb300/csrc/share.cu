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
//
// Latency bounds both: dependent look-ups (lengths, tables, counts), 1.5 us for a
// wait of 152 CTAs, and scattered atomics at one a cycle and SM.  128 requests of 8
// beams, up to 501 pages each, 165000 pages: the fork 11.4 to 11.7 us, of that two waits
// 3.  Measured before: shares by 64-bit divisions 12.5; waits by fences beside the atomics 13.1;
// with 125 CTAs 15.4, with 63 20.7; with the pages of a share looked up again in the last pass,
// sums over pages and rows one by one and a closing ticket 22.  The compaction of 800 such
// rows, 194000 pages: 13.8 to 14.1 us with three waits (14.5; 15.1); its tables' entries read twice
// instead of kept in registers, 98 CTAs: 25.7.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "paged.h"
#include "ptx.cuh"

namespace tpk {

constexpr int kShRows = 8;   // rows of a tile, 32 columns wide
constexpr int kShPages = 4;  // consecutive pages of a thread
constexpr unsigned kAll = 0xffffffffu;

// Two sums in one word: pages below, rows above.
__device__ __forceinline__ unsigned long long two(int pages, int rows) {
  return (unsigned long long)(unsigned)rows << 32 | (unsigned)pages;
}
// Sum of v over the CTA's threads before this one; *total: over all of them.
template <int kThreads>
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* total) {
  __shared__ unsigned long long sums[kThreads / 32];
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // (the sums of the scan before were read)
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  unsigned long long before = x - v, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
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
    red_add_release_gpu(&h->arrived[which], 1u);
    ok = 1;
    const long long t0 = clock64();
    while (ld_acquire_gpu(&h->arrived[which]) < gridDim.x) {
      if (clock64() - t0 > kWaitLimitCycles) {
        record_status(status, kStatusTimeout);
        ok = 0;
        break;
      }
    }
  }
  __syncthreads();
  return ok;
}

// The counters of the later barriers are made zero before the first one, that of the
// first (and the verdict) behind the second, when every CTA is through.
__device__ __forceinline__ void renew_later(ShareHeader* h) {
  if (blockIdx.x == 0 && threadIdx.x == 0) h->arrived[1] = h->arrived[2] = 0;
}
__device__ __forceinline__ void renew_first(ShareHeader* h) {
  if (blockIdx.x == 0 && threadIdx.x == 0) h->arrived[0] = h->bad = 0;
}

// The CTA's share of n things: [first, end), `share` (a multiple of four) for all but the last ones.
__device__ __forceinline__ void share_of(int n, int share, int* first, int* end) {
  *first = (int)min((int64_t)blockIdx.x * share, (int64_t)n);
  *end = (int)min((int64_t)*first + share, (int64_t)n);
}
// A tile's first row and column.
__device__ __forceinline__ int2 tile_at(int t, int col_tiles, const FastDiv& div_cols) {
  const int row = (int)fast_div((uint32_t)t, div_cols);
  return make_int2(row * kShRows, (t - row * col_tiles) * 32);
}

// What the CTAs before this one counted, and all of them.
template <int kThreads>
__device__ __forceinline__ unsigned long long before_this(const ShareHeader* h, unsigned long long* all) {
  __shared__ unsigned long long before;
  int2 c = {0, 0};
  if (threadIdx.x < gridDim.x) c = __ldcg(&h->counts[threadIdx.x]);  // (no more CTAs than threads)
  const unsigned long long x = block_scan<kThreads>(two(c.x, c.y), all);
  if (threadIdx.x == blockIdx.x) before = x;
  __syncthreads();
  return before;
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

__device__ __forceinline__ uint2 note_of(const PageNote* notes, int p) {
  return __ldcg(reinterpret_cast<const uint2*>(notes + p));
}

// The note of a page that a fork meets: how often rows name it afterwards as a full page (in 32
// bits: rows may name one page in many columns, as padding does), and the largest of 1 (rows held
// it before) and 1 + n - b (row b goes on writing to it).
__device__ __forceinline__ uint32_t held_mark() { return 1; }
__device__ __forceinline__ uint32_t open_mark(int n, int row) { return (uint32_t)(n - row) + 1; }
// The verdict on a fork: this, or n - i where entry i is the first of the free ones that names no
// page of the cache (it counts when rows take as many), or 0.
constexpr unsigned kRefused = 0x80000000u;
// A page that rows held before and none holds after.
__device__ __forceinline__ bool is_gone(uint2 note) { return !note.x && note.y == held_mark(); }
__device__ __forceinline__ int holders_of(uint2 note) {
  return note.x ? (int)min(note.x, (uint32_t)INT32_MAX) : note.y > held_mark();
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1) fork_pages_kernel(const ForkArgs a) {
  constexpr int kWarps = kThreads / 32;
  __shared__ uint32_t copied[kMaxStepSeqs / 32];  // the CTA's rows that take a page
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.n_seqs, P = a.page_size;
  pdl_launch_dependents();
  pdl_wait();
  const int first = a.free_state[0], count = a.free_state[1];
  renew_later(a.head);
  auto pages = [&](int len) { return (int)fast_div((uint32_t)len + P - 1, a.div_page); };
  bool bad = false;
  auto ring_at = [&](int i) {
    i += first;
    return i >= a.n_pages ? i - a.n_pages : i;
  };
  auto ring_is_bad = [&] { return first < 0 || first >= a.n_pages || count < 0 || count > a.n_pages; };

  // Pass 1: references, and the new rows as if no page were copied.
  const int row_tiles = (n + kShRows - 1) / kShRows;
  const int col_tiles = a.col_tiles;
  // (neighbouring tiles on different SMs: rows that share little take longest)
  for (int t = warp * gridDim.x + blockIdx.x; t < row_tiles * col_tiles; t += gridDim.x * kWarps) {
    const int2 at = tile_at(t, col_tiles, a.div_cols);
    const int b0 = at.x, col0 = at.y, col = col0 + lane;
    // the tile's rows, a lane each: tokens before, source, tokens kept
    const int row = b0 + lane;
    const bool mine = lane < kShRows && row < n;
    int old = 0, src = -1, keep = 0;
    if (mine) {
      old = a.old_lens[row];
      src = a.src[row];
      if (a.keep_lens) keep = a.keep_lens[row];
      if (old < 0 || old > a.cap || src < -1 || src >= n || (a.keep_lens && src >= 0 && (keep < 0 || keep > a.cap))) {
        bad = true;
        old = keep = 0;
        src = -1;
      }
    }
    // (with keep_lens the source's length is only looked at behind the tables)
    int have = src >= 0 ? a.old_lens[src] : 0;
    if (src < 0) keep = 0;
    if (!a.keep_lens) {
      keep = have;
      if (keep < 0 || keep > a.cap) {
        bad = true;
        keep = 0;
      }
    }
    int was[kShRows], is[kShRows], open = 0;
#pragma unroll
    for (int r = 0; r < kShRows; ++r) {
      const int o = pages(__shfl_sync(kAll, old, r)), s = __shfl_sync(kAll, src, r), k = __shfl_sync(kAll, keep, r);
      was[r] = col < o ? a.table[(int64_t)(b0 + r) * a.ld_table + col] : -1;
      is[r] = col < pages(k) ? a.table[(int64_t)s * a.ld_table + col] : -1;
      if (col < o && (uint32_t)was[r] >= (uint32_t)a.n_pages) {
        bad = true;
        was[r] = -1;
      }
      if (col < pages(k) && (uint32_t)is[r] >= (uint32_t)a.n_pages) {
        bad = true;
        is[r] = -1;
      }
      open |= (is[r] >= 0 && (int64_t)(col + 1) * P > k) << r;  // the row goes on writing to it
    }
    if (mine) {
      bad = bad || keep > have || have > a.cap;
      if (col0 == 0) {
        a.new_lens[row] = keep;
        if ((int)fast_div((uint32_t)keep, a.div_page) * P == keep) a.head->open[row] = -1;
      }
    }
    bool alike = true;  // all rows before and after hold one page, or none
#pragma unroll
    for (int r = 0; r < kShRows; ++r) {
      if (is[r] >= 0) a.table_out[(int64_t)(b0 + r) * a.ld_table + col] = is[r];
      if (open >> r & 1) {
        a.head->open[b0 + r] = is[r];
        atomicMax(&a.notes[is[r]].first, open_mark(n, b0 + r));
        is[r] = -1;  // (counted as full pages below)
      }
      alike = alike && was[r] == was[0] && is[r] == was[0];
    }
    if (__all_sync(kAll, alike)) {
      if (was[0] >= 0) atomicAdd(&a.notes[was[0]].refs, (uint32_t)kShRows);
    } else {  // each page of the tile once
      uint32_t done = 0;  // of `is`: counted with a page of `was`
#pragma unroll
      for (int r = 0; r < kShRows; ++r) {
        uint32_t refs = 0;
        bool again = was[r] < 0;
#pragma unroll
        for (int q = 0; q < kShRows; ++q) {
          if (q < r) again = again || was[q] == was[r];
          if (is[q] == was[r]) {
            refs += 1;
            done |= 1u << q;
          }
        }
        if (!again && refs) atomicAdd(&a.notes[was[r]].refs, refs);
        else if (!again) atomicMax(&a.notes[was[r]].first, held_mark());
      }
      RefRun after = {0, 0};
#pragma unroll
      for (int r = 0; r < kShRows; ++r)
        if (is[r] >= 0 && !(done >> r & 1)) after.add(a.notes, is[r], 1u);
      after.flush(a.notes);
    }
  }
  // The ring's entries that rows may take, one a row: how many they do take is known in pass 3 only.
  // The last warps begin, which mostly had no tile (1024 rows 11.4 us; by the first ones, before
  // their tiles, 11.9).
#pragma unroll 1
  for (int i = ((kWarps - 1 - warp) * gridDim.x + blockIdx.x) * 32 + lane; i < n; i += gridDim.x * kThreads)
    if (!ring_is_bad() && i < count && (uint32_t)a.free_ring[ring_at(i)] >= (uint32_t)a.n_pages)
      atomicMax(&a.head->bad, (unsigned)(n - i));
  bad = bad || ring_is_bad();
  if (__syncthreads_or(bad) && tid == 0) atomicMax(&a.head->bad, kRefused);
  if (!grid_wait(a.head, 0, a.status)) return;

  // Pass 2: pages that no row holds any more, rows that take a page.
  int p0, p1, b0, b1;
  share_of(a.n_pages, a.page_share, &p0, &p1);
  share_of(n, a.row_share, &b0, &b1);
  const unsigned verdict = __ldcg(&a.head->bad);
  bad = verdict == kRefused;
  // The thread's pages and row of the share's turn `at`; those of the first turn, mostly the only
  // one, stay in registers for pass 3.
  uint2 note[kShPages];
  int from, keep;  // the page that the row goes on writing to, or -1; its tokens
  const int turns = max((p1 - p0 + kShPages * kThreads - 1) / (kShPages * kThreads), (b1 - b0 + kThreads - 1) / kThreads);
  auto fetch = [&](int turn) {
    const int row = b0 + turn * kThreads + tid, page = p0 + (turn * kThreads + tid) * kShPages;
    from = row < b1 && !bad ? __ldcg(&a.head->open[row]) : -1;
    keep = row < b1 ? __ldcg(&a.new_lens[row]) : 0;
#pragma unroll
    for (int i = 0; i < kShPages; ++i) note[i] = page + i < p1 ? note_of(a.notes, page + i) : make_uint2(0, 0);
  };
  int freed = 0, taken = 0;
  for (int turn = turns - 1; turn >= 0; --turn) {
    fetch(turn);
    bool copy = false;
    if (from >= 0) {
      const uint2 x = note_of(a.notes, from);
      copy = x.x || x.y != open_mark(n, b0 + turn * kThreads + tid);
    }
    const unsigned m = __ballot_sync(kAll, copy);
    if (lane == 0 && b0 + turn * kThreads < b1) copied[turn * kWarps + warp] = m;
    taken += copy;
#pragma unroll
    for (int i = 0; i < kShPages; ++i) freed += is_gone(note[i]);
    if (a.old_holders) {  // (before the pages that rows take get theirs)
      const int page = p0 + (turn * kThreads + tid) * kShPages;
#pragma unroll
      for (int i = 0; i < kShPages; ++i)
        if (page + i < p1) a.holders[page + i] = holders_of(note[i]);
    }
  }
  unsigned long long all;
  block_scan<kThreads>(two(freed, taken), &all);
  if (tid == 0) a.head->counts[blockIdx.x] = make_int2((int)all, (int)(all >> 32));
  if (!grid_wait(a.head, 1, a.status)) return;

  // Pass 3: the ring, the rows' own pages, the moves.
  renew_first(a.head);
  unsigned long long before = before_this<kThreads>(a.head, &all);
  const int f_all = (int)all, t_all = (int)(all >> 32);
  bad = bad || t_all > count || t_all > n - (int)verdict || count + f_all > a.n_pages;
  for (int turn = 0; turn < turns; ++turn) {
    if (turn) fetch(turn);
    const int row = b0 + turn * kThreads + tid, page = p0 + (turn * kThreads + tid) * kShPages;
    const bool copy = !bad && row < b1 && (copied[turn * kWarps + warp] >> lane & 1);
    int gone = 0;
#pragma unroll
    for (int i = 0; i < kShPages; ++i) gone += is_gone(note[i]);
    unsigned long long here;
    const unsigned long long mine = before + block_scan<kThreads>(two(gone, copy), &here);
    before += here;
    int to_ring = (int)mine;
    const int move = (int)(mine >> 32), to = copy ? a.free_ring[ring_at(move)] : 0;
#pragma unroll
    for (int i = 0; i < kShPages; ++i) {
      const uint2 x = note[i];
      if (!x.x && !x.y) continue;  // (also what lies behind the share)
      *reinterpret_cast<uint2*>(a.notes + page + i) = make_uint2(0, 0);
      if (bad) continue;
      if (is_gone(x)) a.free_ring[ring_at(count + to_ring++)] = page + i;
      if (a.holders && !a.old_holders) a.holders[page + i] = holders_of(x);
    }
    if (copy) {
      const int full = (int)fast_div((uint32_t)keep, a.div_page);
      a.table_out[(int64_t)row * a.ld_table + full] = to;
      if (a.holders) a.holders[to] = 1;
      a.moves[3 * move] = from;
      a.moves[3 * move + 1] = to;
      a.moves[3 * move + 2] = keep - full * P;
    }
    if (bad && row < b1) a.new_lens[row] = a.old_lens[row];
  }
  if (bad) {  // the old rows again
    const int64_t words = (int64_t)n * a.ld_table;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < words; i += (int64_t)gridDim.x * kThreads)
      a.table_out[i] = a.table[i];
    if (a.old_holders)
      for (int p = p0 + tid; p < p1; p += kThreads) a.holders[p] = a.old_holders[p];
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (bad) record_status(a.status, kStatusTableRange);
    a.free_next[0] = bad ? first : ring_at(t_all);
    a.free_next[1] = bad ? count : count - t_all + f_all;
    *a.n_moves = bad ? 0 : t_all;
  }
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1) compact_pages_kernel(const CompactArgs a) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.n_seqs, P = a.page_size;
  pdl_launch_dependents();
  pdl_wait();
  auto pages = [&](int len) { return (int)fast_div((uint32_t)len + P - 1, a.div_page); };
  const int first = a.free_state[0], count = a.free_state[1];
  renew_later(a.head);
  bool bad = false;

  // A tile's pages, -1 where a row holds none.  The warp's first tile stays in registers.
  const int row_tiles = (n + kShRows - 1) / kShRows;
  const int col_tiles = a.col_tiles;
  const int tiles = row_tiles * col_tiles, tile0 = warp * gridDim.x + blockIdx.x;
  auto fetch = [&](int t, int (&page)[kShRows]) {
    const int2 at = tile_at(t, col_tiles, a.div_cols);
    const int b0 = at.x, col = at.y + lane;
    int len = 0;
    if (lane < kShRows && b0 + lane < n) {
      len = a.lens[b0 + lane];
      if (len < 0 || len > a.cap) {
        bad = true;
        len = 0;
      }
    }
#pragma unroll
    for (int r = 0; r < kShRows; ++r) {
      const bool held = col < pages(__shfl_sync(kAll, len, r));
      page[r] = held ? a.table[(int64_t)(b0 + r) * a.ld_table + col] : -1;
      if (held && (uint32_t)page[r] >= (uint32_t)a.n_pages) {
        bad = true;
        page[r] = -1;
      }
    }
  };
  // Pass 1: references.
  int kept[kShRows];
#pragma unroll
  for (int r = 0; r < kShRows; ++r) kept[r] = -1;
  auto refer = [&](const int (&page)[kShRows]) {
    RefRun run = {0, 0};
#pragma unroll
    for (int r = 0; r < kShRows; ++r)
      if (page[r] >= 0) run.add(a.notes, page[r], 1u);
    run.flush(a.notes);
  };
  if (tile0 < tiles) {
    fetch(tile0, kept);
    refer(kept);
  }
  for (int t = tile0 + gridDim.x * kWarps; t < tiles; t += gridDim.x * kWarps) {
    int page[kShRows];
    fetch(t, page);
    refer(page);
  }
  if (__syncthreads_or(bad) && tid == 0) atomicOr(&a.head->bad, 1u);
  if (!grid_wait(a.head, 0, a.status)) return;

  // Pass 2: pages held, by share.
  bad = __ldcg(&a.head->bad);
  int p0, p1;
  share_of(a.n_pages, a.page_share, &p0, &p1);
  uint32_t refs[kShPages];  // the thread's pages of a turn; the first turn's stay for pass 3
  const int turns = (p1 - p0 + kShPages * kThreads - 1) / (kShPages * kThreads);
  auto look = [&](int turn) {
    const int page = p0 + (turn * kThreads + tid) * kShPages;
#pragma unroll
    for (int i = 0; i < kShPages; ++i) refs[i] = page + i < p1 ? __ldcg(&a.notes[page + i].refs) : 0;
  };
  auto count_held = [&] {
    int many = 0;
#pragma unroll
    for (int i = 0; i < kShPages; ++i) many += refs[i] != 0;
    return many;
  };
  int held = 0;
  for (int turn = turns - 1; turn >= 0; --turn) {
    look(turn);
    held += count_held();
  }
  unsigned long long all;
  block_scan<kThreads>(two(held, 0), &all);
  if (tid == 0) a.head->counts[blockIdx.x] = make_int2((int)all, 0);
  if (!grid_wait(a.head, 1, a.status)) return;

  // Pass 3: with h held pages below p, the free page p < U is the (p - h)-th hole, the
  // held page p >= U the (U - 1 - h)-th to move, from the highest on.
  renew_first(a.head);
  unsigned long long before = before_this<kThreads>(a.head, &all);
  const int used = (int)all;
  for (int turn = 0; turn < turns; ++turn) {
    if (turn) look(turn);
    const int page = p0 + (turn * kThreads + tid) * kShPages;
    unsigned long long here;
    int h = (int)(before + block_scan<kThreads>(two(count_held(), 0), &here));
    before += here;
#pragma unroll
    for (int i = 0; i < kShPages; ++i) {
      const int p = page + i;
      if (p >= p1) break;
      if (refs[i]) a.notes[p].refs = 0;
      if (bad) {
        if (a.ring_out != a.ring) a.ring_out[p] = a.ring[p];
        if (a.old_holders) a.holders[p] = a.old_holders[p];
        continue;
      }
      a.ring_out[p] = p;
      if (p == used - 1) *a.n_moves = p - h + (refs[i] == 0);  // the holes
      if (a.holders) a.holders[p] = p < used ? (int)refs[i] : 0;  // (holes: when their pages come)
      if (p < used && !refs[i]) {
        a.moves[3 * (p - h) + 1] = p;
        a.moves[3 * (p - h) + 2] = P;
      } else if (p >= used && refs[i]) {
        const int move = used - 1 - h;
        a.moves[3 * move] = p;
        *reinterpret_cast<int2*>(&a.notes[p].move) = make_int2(move, (int)refs[i]);
      }
      h += refs[i] != 0;
    }
  }
  if (!grid_wait(a.head, 2, a.status)) return;

  // Pass 4: the rows' pages by their new names.
  if (bad) {
    if (a.table_out != a.table) {
      const int64_t words = (int64_t)n * a.ld_table;
      for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < words; i += (int64_t)gridDim.x * kThreads)
        a.table_out[i] = a.table[i];
    }
  } else {
    auto rename = [&](int t, int (&page)[kShRows]) {
      const int2 at = tile_at(t, col_tiles, a.div_cols);
      const int b0 = at.x, col = at.y + lane;
      int2 note[kShRows];
#pragma unroll
      for (int r = 0; r < kShRows; ++r)
        if (page[r] >= used) note[r] = __ldcg(reinterpret_cast<const int2*>(&a.notes[page[r]].move));
#pragma unroll
      for (int r = 0; r < kShRows; ++r)
        if (page[r] >= used) {
          page[r] = __ldcg(&a.moves[3 * note[r].x + 1]);
          if (a.holders) a.holders[page[r]] = note[r].y;  // (every row that holds it writes the same)
        }
#pragma unroll
      for (int r = 0; r < kShRows; ++r)
        if (page[r] >= 0) a.table_out[(int64_t)(b0 + r) * a.ld_table + col] = page[r];
    };
    if (tile0 < tiles) rename(tile0, kept);
    for (int t = tile0 + gridDim.x * kWarps; t < tiles; t += gridDim.x * kWarps) {
      int page[kShRows];
      fetch(t, page);
      rename(t, page);
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (bad) record_status(a.status, kStatusTableRange);
    if (bad || used == 0) *a.n_moves = 0;
    a.free_next[0] = bad ? first : used == a.n_pages ? 0 : used;
    a.free_next[1] = bad ? count : a.n_pages - used;
  }
}

// CTAs of 512 threads, one an SM at most; a single one has 256 (two requests of four beams:
// 6.5 us instead of 7.4, and 5.8 with the registers of a whole SM: more look-ups in flight; 5.9 with
// the ring's entries looked at).
constexpr int kMany = 512, kFew = 256;

static int share_size(int n, int ctas) { return ((n + ctas - 1) / ctas + 3) & ~3; }

template <typename Args>
static cudaError_t launch_shared(void (*many)(Args), void (*few)(Args), Args a, int num_sms,
                                 cudaStream_t st) {
  const int64_t cols = std::min<int64_t>(a.ld_table, (a.cap + (int64_t)a.page_size - 1) / a.page_size);
  const int64_t tiles = (cols * a.n_seqs + 2047) / 2048, by_pages = (a.n_pages + 2047) / 2048;
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(std::max(tiles, by_pages), std::min({num_sms, kShareCtas, kMany})));
  a.col_tiles = (int)std::max<int64_t>(1, (cols + 31) / 32);
  a.div_cols = make_fastdiv((uint32_t)a.col_tiles);
  a.page_share = share_size(a.n_pages, grid);
  a.row_share = share_size(a.n_seqs, grid);
  if (grid == 1) return launch_k(few, dim3(1), dim3(kFew), 0, st, a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kMany);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // all CTAs at once
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, many, a);
}

cudaError_t launch_fork_pages(const ForkArgs& a, int num_sms, cudaStream_t st) {
  return launch_shared(fork_pages_kernel<kMany>, fork_pages_kernel<kFew>, a, num_sms, st);
}

cudaError_t launch_compact_pages(const CompactArgs& a, int num_sms, cudaStream_t st) {
  return launch_shared(compact_pages_kernel<kMany>, compact_pages_kernel<kFew>, a, num_sms, st);
}

}  // namespace tpk
