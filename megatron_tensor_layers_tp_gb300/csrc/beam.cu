// Beam search's selection over beams and vocabulary, and the beams' texts.
//
// A continuation of row b by token v is worth s_b + (x_v - M) - log sum exp(x - M),
// M the row's largest logit.  Within a row the order is the logits', so the sum
// and the K best logits come out of one pass; a row is cut into parts, and the
// last CTA of a request's parts joins their sums and lists.
//
// The pass is bound by memory: 16 KB of a part at a time come by bulk copies into a
// ring in shared memory, and a thread takes 16-byte words of them into registers.
// The warps run through the ring without waiting for each other.
// The K best: a thread leaves the largest logit of each chunk in shared memory.
// Behind the last chunk the K-th largest of at least 2 K maxima (two to eight threads
// each) bounds the K-th largest logit from below, and the logits of the few cells (a
// thread's of a chunk) that reach the bound are read once more, from L2: what passes
// is the part's list.  Where more passes than the buffer holds (equal logits) the
// cells are gone through a warp a cell, as long as they can still count, and ranked in between.
//
// Sums: of 2^(x log2(e) - r), r the thread's largest x log2(e) so far, rounded to a whole
// number, so that sums are brought to one r exactly; added in fp32 (at most V / 256
// of them), the threads' sums as whole multiples of 2^-32, whose order does not
// matter: equal rows get equal sums.  What log2(e) in fp32 (c) is off by cancels, as x
// counts from M in the same units: M c - r.  Rows with NaN, and those whose largest
// logit is beyond 2^20, are summed once more, from M on.
//
// 64 requests of 4 rows of 128256 logits, bf16, K = 8: 18.5 us, 65.7 MB from memory (9.7 us at
// the copy rate).  The last logits are there after 11 to 12 us (a chunk takes a warp 240
// instructions, some 900 cycles, of which it waits 200 for logits); what follows is a chain of
// short steps, 6 us in all: the bound 0.9, the cells 0.7, the list 0.4, the ticket 0.8, the rows'
// sums 1.2, values 0.8, ranks 0.6, the next beams 0.3.  Code that a CTA runs once costs its way
// from L2: what is short wins there over what has more in flight.  The same rows of 128257 logits,
// off 16-byte boundaries: 20.5.  13 requests of 16 rows of 152064, fp32, K = 32: 27.8 us (114 MB:
// 16.8).  One request of 4 rows of 32000: 7.7 us, the chain alone.  All logits equal: 8 requests
// of 16 rows, K = 64, 0.17 ms.
// Measured before: what passes a running bound pushed to the buffer as it streams by, with a
// barrier a chunk: 25 and 43 us; the same by plain loads, two CTAs' widths in flight: 105 and
// 136.  A request's CTAs as a cluster that joins through distributed shared memory: 0.2 to
// 0.4 us less than a ticket between two fences, and as much as the ticket that has them in
// itself.  The next chunk's words ahead of this one's sums: 0.5 to 1 us more.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "paged.h"
#include "ptx.cuh"

namespace tpk {

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr int kSelVecs = 4;         // 16-byte words of a thread in a chunk
constexpr int kSelStages = 4;       // chunks in the ring, at most
// Of a thread: its largest logits, each of so many chunks: of one in parts of up to 40 (20 KB: what
// three CTAs an SM with three stages leave; 13 requests of 16 rows of 152064, fp32, 38 chunks a
// part: 29.0 us at the time, with 24 cells of two chunks 30.2).
constexpr int kSelCells = 40;
constexpr int kSelChunkBytes = kSelThreads * kSelVecs * 16;
constexpr int kSelStageBytes = kSelChunkBytes + 128;  // (rows off 16-byte boundaries look at a word more)
constexpr int kSelBuffer = 2 * kSelThreads - kMaxBeamCands;  // keys that may pass a bound
constexpr int kSelKeys = 2048;      // of a request's lists, at most
constexpr float kLog2e = 1.4426950408889634f;

// Bits whose order as whole numbers is that of the values (-0 as 0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_ordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ unsigned long long ordered(double x) {
  const long long b = __double_as_longlong(x);
  return (unsigned long long)(b ^ (b >> 63 | (long long)0x8000000000000000ull));
}
// Larger for larger logits, among equal ones for lower tokens; never 0.
__device__ __forceinline__ unsigned long long key_of(float x, int token) {
  return (unsigned long long)ordered(fminf(x, FLT_MAX)) << 32 | (uint32_t)~token;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, d;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 d, x, y;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, d;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 d, x, y, z;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {  // (NaN falls out)
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

constexpr float kFar = 1048576.f;  // logits beyond are summed from the largest on
__device__ __forceinline__ bool is_far(float top) { return !(fabsf(top) <= kFar); }
// r of a largest logit: whole, and exact in fp32
__device__ __forceinline__ float power_of(float top) {
  return rintf(fminf(fmaxf(top, -kFar), kFar) * kLog2e);
}

// The log of s * 2^(r - 32) - top * log2(e) * log(2), s >= 1, with log2(e) as the sums have it
// (kLog2e), to 10^-8: with s * 2^-32 = 2^k m, 2/3 < m <= 4/3, and z = (m - 1) / (m + 1), log m
// is 2 (z + z^3 / 3 + z^5 / 5 + ...); z in two fp32 numbers, the powers from its first.  (log
// in 64 bits took 2900 cycles, on the path of every request; 64-bit operations take 60 each.)
__device__ __forceinline__ double log_sum(unsigned long long s, int r, float top) {
  constexpr double kLn2 = 0.693147180559945309417;
  const int lead = __clzll((long long)s);
  const unsigned long long x = s << lead;
  float m = (float)(uint32_t)(x >> 40) * 0x1p-23f;             // in [1, 2), exact
  float ml = (float)(uint32_t)(x >> 8 & 0xFFFFFFFFu) * 0x1p-55f;  // the bits behind
  int k = 31 - lead;
  if (m > 1.3333333f) {
    m *= 0.5f;
    ml *= 0.5f;
    ++k;
  }
  const float a = m - 1.f, b = m + 1.f, bl = m - (b - 1.f) + ml;
  const float z = __fdividef(a, b);  // (what it is off by is in zl)
  const float zl = __fdividef(fmaf(-z, b, a) + ml - z * bl, b);
  const float y = z * z;
  float p = 1.f / 13.f;
  p = fmaf(p, y, 1.f / 11.f);
  p = fmaf(p, y, 1.f / 9.f);
  p = fmaf(p, y, 1.f / 7.f);
  p = fmaf(p, y, 1.f / 5.f);
  p = fmaf(p, y, 1.f / 3.f);
  return fma((double)(k + r), kLn2, fma((double)top, -(double)kLog2e * kLn2, (double)(2.f * z))) +
         (double)(2.f * fmaf(z * y, p, zl));
}

struct BoundSmem {
  __align__(16) uint32_t group[kSelThreads / 2];
  uint32_t bound;
};
struct SelectSmem {
  unsigned long long keys[kSelBuffer + kMaxBeamCands + 2];  // the best so far, then the buffer
  __align__(16) uint16_t cell[kSelThreads][kSelCells];  // bf16, rounded up
  uint64_t full[kSelStages], empty[kSelStages];
  int many;  // keys in the buffer, while cells are picked
  int hits;  // cells that reach the bound
  int picked, pick[kSelWarps];
  int warp_many[kSelWarps];
  int last;
  BoundSmem bound;
  uint32_t warp_top[kSelWarps];
  int warp_power[kSelWarps];
  unsigned long long warp_sum[kSelWarps];
};
struct JoinSmem {  // lies in the ring
  unsigned long long key[kSelKeys];    // of the lists
  float below[kSelKeys], near[kSelKeys];  // their values' parts: from the row's largest logit on; the row's
  uint32_t entry[kSelKeys];            // of those that may be among the K best: row << 16 | number
  // of those that are ranked at a time: values (bits in order) and keys, entries
  ulonglong2 ranked[kSelThreads];
  uint32_t its_entry[kSelThreads];
  unsigned long long best_value[kMaxBeamCands];
  int many;
  BoundSmem bound;
  double row_rest[kMaxBeams];  // score - log of the sum, from the largest logit on
  float row_top[kMaxBeams], row_near[kMaxBeams];  // the largest logit; row_rest (-infinity: not in use)
  int best_row[kMaxBeamCands], best_token[kMaxBeamCands];
  float best_score[kMaxBeamCands];
};
// How many threads count for one of m keys (as powers of two, here and below: divisions by
// other numbers are long).
__device__ __forceinline__ int log_threads_a_key(int m) { return m <= 32 ? 3 : m <= 64 ? 2 : m <= 128 ? 1 : 0; }

// The K-th largest of the threads' o, or of groups' largest where half as many groups are
// enough: at least K of the threads' values reach it.  All threads, together; .y: whether
// one of them has `flag`.
__device__ __forceinline__ int log_groups_of(int K) { return K > 32 ? 7 : K > 16 ? 6 : 5; }
constexpr int kLogThreads = 8;
static_assert(kSelThreads == 1 << kLogThreads, "");
__device__ __forceinline__ uint2 bound_of(BoundSmem& sm, uint32_t o, int K, bool flag) {
  const int log_size = kLogThreads - log_groups_of(K), size = 1 << log_size;
  const int mine = threadIdx.x >> log_size, turn = threadIdx.x & (size - 1);
  for (int q = 1; q < size; q <<= 1) o = max(o, __shfl_xor_sync(0xffffffffu, o, q));
  if (turn == 0) sm.group[mine] = o;
  const uint32_t any = __syncthreads_or(flag);
  int place = 0;
  const int share = kSelThreads >> 2 * log_size, j0 = turn * share, j1 = j0 + share;
#pragma unroll 4
  for (int j = j0; j < j1; j += 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(sm.group + j);
    place += (x.x > o || (x.x == o && j < mine)) + (x.y > o || (x.y == o && j + 1 < mine)) +
             (x.z > o || (x.z == o && j + 2 < mine)) + (x.w > o || (x.w == o && j + 3 < mine));
  }
  for (int q = 1; q < size; q <<= 1) place += __shfl_xor_sync(0xffffffffu, place, q);
  if (place == K - 1 && turn == 0) sm.bound = o;
  __syncthreads();
  return make_uint2(sm.bound, any);
}

// Ranks the keys, `best` sorted ones and n more, and keeps the K best: their
// number.  All threads, together; the keys are visible on entry and exit.
__device__ __noinline__ int rank_keys(SelectSmem& sm, int best, int n, int K) {
  const int m = best + n, tid = threadIdx.x, log_t = log_threads_a_key(m), T = 1 << log_t;
  constexpr int kMost = (kSelBuffer + kMaxBeamCands) / kSelThreads;
  unsigned long long key[kMost];
  int rank[kMost];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int at = (tid >> log_t) + i * kSelThreads;
    key[i] = at < m ? sm.keys[at] : 0;
    rank[i] = K;
    if (i * kSelThreads >= m) break;
    int r = 0;
#pragma unroll 4
    for (int j = tid & (T - 1); j < m; j += T) r += sm.keys[j] > key[i];
    for (int q = 1; q < T; q <<= 1) r += __shfl_xor_sync(0xffffffffu, r, q);
    if (at < m && (tid & (T - 1)) == 0) rank[i] = r;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMost; ++i)
    if (rank[i] < K) sm.keys[rank[i]] = key[i];
  if (tid == 0) sm.many = 0;
  __syncthreads();
  return min(m, K);
}

// The request's parts joined: its candidates and next beams.  All keys of its lists
// get their values in fp32, off by at most kNear of their parts; groups of threads bound the
// K-th value from below as they do among the logits, and what may reach it gets its value in
// 64 bits (of which the GPU does few at a time) and is ranked by counting.
constexpr float kNear = 0x1p-21f;
__device__ void join_request(const BeamSelectArgs& a, JoinSmem& sm, int req) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int W = a.width, K = a.n_cands, per_row = a.parts * a.list, N = W * per_row;
  const int row0 = req * W;
  const unsigned long long* keys = a.lists + (int64_t)row0 * per_row;
  // A thread's keys are one of each run of as many keys as there are groups, every run turned
  // further: a row's may be the best of all, and lists may be in order.  (The first are on their
  // way while the rows' sums are joined.)
  const int log_groups = log_groups_of(K), groups = 1 << log_groups, log_size = kLogThreads - log_groups;
  auto number = [&](int i) {
    const int run = (i << log_size) + (tid & ((1 << log_size) - 1));
    return (run << log_groups) + (((tid >> log_size) + 37 * run) & (groups - 1));
  };
  unsigned long long key[4];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) key[i] = number(i0 + i) < N ? keys[number(i0 + i)] : 0;
  };
  fetch(0);
  const int end = warp == 0 && lane < a.n_ends ? a.ends[lane] : -1;
  if (tid == 0) sm.many = 0;
  // A row a group of as many lanes as it has parts (up to 32, a power of two).
  const int log_group = a.parts > 16 ? 5 : a.parts > 8 ? 4 : a.parts > 4 ? 3 : a.parts > 2 ? 2 : a.parts - 1;
  const int group = 1 << log_group;
  const int of_row = tid & (group - 1);
  for (int w0 = 0; w0 < W; w0 += kSelThreads >> log_group) {
    const int w = w0 + (tid >> log_group);
    const float score = w < W ? a.scores[row0 + w] : -INFINITY;
    const BeamPart* p = a.sums + (int64_t)(row0 + min(w, W - 1)) * a.parts;
    const BeamPart own = of_row < a.parts ? p[of_row] : BeamPart{0, -INFINITY, INT_MIN};
    // the largest logit and power; parts far below the row's largest logit add nothing
    // (what stands for a row not in use may be anything)
    float top = own.top;
    for (int i = of_row + 32; i < a.parts; i += 32) top = fmaxf(top, p[i].top);
    for (int q = 1; q < group; q <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, q));
    const bool far = is_far(top);
    int r = is_far(own.top) ? INT_MIN : own.power;
    for (int i = of_row + 32; i < a.parts; i += 32)
      if (!is_far(p[i].top)) r = max(r, p[i].power);
    for (int q = 1; q < group; q <<= 1) r = max(r, __shfl_xor_sync(0xffffffffu, r, q));
    unsigned long long sum = 0;
    for (int i = of_row; i < a.parts; i += 32) {
      const BeamPart x = i == of_row ? own : p[i];
      if (!far && !is_far(x.top)) {
        sum += x.sum >> min(max(r - x.power, 0), 63);
      } else if (x.sum) {  // the row's, the part's or both sums count from the largest logit on
        const float d = !far ? fmaf(x.top, kLog2e, -(float)r)
                        : is_far(x.top) ? (x.top - top) * kLog2e : fmaf(-top, kLog2e, (float)x.power);
        sum += (unsigned long long)((double)x.sum * (double)ex2_approx(d));
      }
    }
    for (int q = 1; q < group; q <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, q);
    if (of_row == 0 && w < W) {
      const double rest = (double)score - log_sum(max(sum, 1ull), far ? 0 : r, far ? 0.f : top);
      sm.row_top[w] = top;
      sm.row_rest[w] = rest;
      sm.row_near[w] = isfinite(score) ? (float)rest : -INFINITY;
    }
  }
  __syncthreads();

  auto value = [](float below, float near, float side) { return below + near + side * (fabsf(below) + fabsf(near)); };
  float most = -INFINITY;
  for (int i0 = 0; i0 * kSelThreads < N; i0 += 4) {
    if (i0) fetch(i0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = number(i0 + i);
      if (e >= N) continue;
      const int w = (int)fast_div((uint32_t)e, a.div_row_keys);
      const float below = of_ordered((uint32_t)(key[i] >> 32)) - sm.row_top[w];
      const float near = key[i] ? sm.row_near[w] : -INFINITY;  // (-infinity: none)
      sm.key[e] = key[i];
      sm.below[e] = below, sm.near[e] = near;
      if (near > -INFINITY) most = fmaxf(most, value(below, near, -kNear));
    }
  }
  const uint32_t bound = max(bound_of(sm.bound, ordered(most), K, false).x, ordered(-INFINITY) + 1);
  for (int e = tid; e < N; e += kSelThreads) {
    const float below = sm.below[e], near = sm.near[e];
    if (near > -INFINITY && !(ordered(value(below, near, kNear)) < bound))
      sm.entry[atomicAdd(&sm.many, 1)] = fast_div((uint32_t)e, a.div_row_keys) << 16 | (uint32_t)e;
  }
  __syncthreads();
  const int many = sm.many, all = min(many, K);
  // As many as there are threads are ranked at a time (mostly all): the K best so far, in front,
  // and those from `next` on.  Equal values go by row, logit (different logits of a row can have
  // the same value in 64 bits) and token.
  for (int best = 0, next = 0; next < many;) {
    const int m = min(best + many - next, kSelThreads), log_t = log_threads_a_key(m), T = 1 << log_t;
    if (tid < m) {
      const uint32_t e = sm.entry[tid < best ? tid : tid - best + next];
      const unsigned long long k = sm.key[e & 0xFFFF];
      const double x = of_ordered((uint32_t)(k >> 32));
      sm.ranked[tid] = make_ulonglong2(
          tid < best ? sm.best_value[tid] : ordered(x - (double)sm.row_top[e >> 16] + sm.row_rest[e >> 16]), k);
      sm.its_entry[tid] = e;
    }
    __syncthreads();
    const int i = tid >> log_t;
    const ulonglong2 v = sm.ranked[i];
    const uint32_t e = sm.its_entry[i], w = e >> 16;
    int place = i < m ? 0 : K;
#pragma unroll 4
    for (int j = tid & (T - 1); j < m; j += T) {
      const ulonglong2 u = sm.ranked[j];
      const uint32_t row = sm.its_entry[j] >> 16;
      place += (u.x > v.x) | ((u.x == v.x) & ((row < w) | ((row == w) & (u.y > v.y))));
    }
    for (int q = 1; q < T; q <<= 1) place += __shfl_xor_sync(0xffffffffu, place, q);
    if ((tid & (T - 1)) == 0 && place < K) {
      sm.best_value[place] = v.x;
      sm.entry[place] = e;
    }
    __syncthreads();
    next += m - best;
    best = min(m, K);
  }
  if (tid < K) {
    const bool there = tid < all;
    const uint32_t e = there ? sm.entry[tid] : 0;
    const unsigned long long v = there ? sm.best_value[tid] : 0;
    const float score = there ? (float)__longlong_as_double((long long)(v >> 63 ? v ^ 0x8000000000000000ull : ~v)) : -INFINITY;
    const int from = there ? row0 + (int)(e >> 16) : -1, token = there ? (int)~(uint32_t)sm.key[e & 0xFFFF] : -1;
    a.cand_scores[req * K + tid] = sm.best_score[tid] = score;
    a.cand_rows[req * K + tid] = sm.best_row[tid] = from;
    a.cand_tokens[req * K + tid] = sm.best_token[tid] = token;
  }
  __syncthreads();
  // The next beams: the first W whose token ends no text.
  if (warp == 0) {
    int placed = 0;
    for (int base = 0; base < K; base += 32) {
      const int i = base + lane;
      bool goes = i < all;
      const int token = goes ? sm.best_token[i] : -1;
#pragma unroll 1
      for (int e = 0; e < a.n_ends; ++e) {
        const int x = __shfl_sync(0xffffffffu, end, e);
        goes = goes && token != x;
      }
      const unsigned m = __ballot_sync(0xffffffffu, goes);
      const int at = placed + __popc(m & ((1u << lane) - 1));
      if (goes && at < W) {
        a.next_scores[row0 + at] = sm.best_score[i];
        a.parents[row0 + at] = sm.best_row[i];
        a.tokens[row0 + at] = sm.best_token[i];
      }
      placed += __popc(m);
    }
    if (lane >= placed && lane < W) {
      a.next_scores[row0 + lane] = -INFINITY;
      a.parents[row0 + lane] = -1;
      a.tokens[row0 + lane] = 0;
    }
  }
}

// kStages: 4, for two CTAs an SM; 3, for three, where there are more CTAs than two an SM (their
// steps behind the stream then run beside others' streams; us, with four stages and with
// three: 800 rows of 128256, bf16: 47 and 43; 400: 31 and 24; 1024 rows of 8000, fp32: 23 and 19;
// 512 rows of 32000, K = 64: 28 and 29, before cells were collected by votes).
template <bool kFp32, int kStages>
__global__ void __launch_bounds__(kSelThreads, kStages == 4 ? 2 : 3) beam_select_kernel(const BeamSelectArgs a) {
  constexpr int kE = kFp32 ? 4 : 8;            // logits of a 16-byte word
  constexpr int kPer = kSelVecs * kE;          // of a thread in a chunk
  constexpr int kSize = kFp32 ? 4 : 2;
  constexpr int kChunk = kSelThreads * kPer;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) SelectSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = blockIdx.x, row = (int)fast_div((uint32_t)item, a.div_parts);
  const int part = item - row * a.parts, req = (int)fast_div((uint32_t)row, a.div_width);
  const int K = a.n_cands;
  if (tid == 0) {
    sm.many = sm.hits = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kSelWarps);
    }
    fence_barrier_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  if (isfinite(a.scores[row])) {
    const int begin = (int)min((int64_t)part * a.part_chunks * kChunk, (int64_t)a.vocab);
    const int end = (int)min((int64_t)begin + (int64_t)a.part_chunks * kChunk, (int64_t)a.vocab);
    const int chunks = (end - begin + kChunk - 1) / kChunk;
    const uint8_t* base = static_cast<const uint8_t*>(a.logits) + row * a.ld * kSize;
    const int off = (int)(reinterpret_cast<uintptr_t>(base) & 15);  // of every chunk's first logit
    // the row's 16-byte words that hold nothing else
    const uint8_t* inner0 = base + (-off & 15);
    const uint8_t* inner1 = base + (int64_t)a.vocab * kSize;
    inner1 -= reinterpret_cast<uintptr_t>(inner1) & 15;
    auto raw = [&](int v) {
      return kFp32 ? reinterpret_cast<const float*>(base)[v] : bf16_to_f(reinterpret_cast<const uint16_t*>(base)[v]);
    };
    auto issue = [&](int c, int slot) {
      const uint8_t* first = base + (begin + (int64_t)c * kChunk) * kSize - off;
      const uint8_t* last = base + min(begin + (int64_t)(c + 1) * kChunk, (int64_t)end) * kSize;
      last += -reinterpret_cast<uintptr_t>(last) & 15;
      const uint8_t *from = first < inner0 ? inner0 : first, *to = last > inner1 ? inner1 : last;
      if (to > from) {
        const uint32_t bytes = (uint32_t)(to - from);
        mbar_arrive_expect_tx(&sm.full[slot], bytes);
        bulk_load_plain(ring + slot * kSelStageBytes + (from - first), from, bytes, &sm.full[slot]);
      } else {
        mbar_arrive(&sm.full[slot]);
      }
    };
    if (tid == 0)
      for (int c = 0; c < min(chunks, kStages); ++c) issue(c, c);
    __syncthreads();

    float top = -INFINITY, power = power_of(-INFINITY), sum = 0.f, of_cell = -INFINITY;
    int slot = 0, cell = 0, in_cell = 0;
    uint32_t parity = 0;
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
      const int at = begin + c * kChunk;
      const int many = min(end - at, kChunk);
      const uint4* words = reinterpret_cast<const uint4*>(ring + slot * kSelStageBytes) + tid;
      ok = mbar_wait(&sm.full[slot], parity, a.status) && ok;
      // The thread's words; logits behind the part's last are -infinity.
      uint32_t w[4 * kSelVecs];
      if (off == 0 && many == kChunk) {
#pragma unroll
        for (int j = 0; j < kSelVecs; ++j) *reinterpret_cast<uint4*>(w + 4 * j) = words[j * kSelThreads];
      } else {
        // bytes off .. off + 15 of two words, from their 32-bit word `kFrom` on
        auto shift = [&](auto from) {
          constexpr int kFrom = decltype(from)::value;
#pragma unroll
          for (int j = 0; j < kSelVecs; ++j) {
            const uint4 u = words[j * kSelThreads], v = words[j * kSelThreads + 1];
            const uint32_t y[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) w[4 * j + i] = __funnelshift_r(y[kFrom + i], y[kFrom + i + 1], (off & 2) * 8);
          }
        };
        switch (off >> 2) {
          case 0: shift(std::integral_constant<int, 0>()); break;
          case 1: shift(std::integral_constant<int, 1>()); break;
          case 2: shift(std::integral_constant<int, 2>()); break;
          default: shift(std::integral_constant<int, 3>());
        }
        const uint8_t* at0 = base + (int64_t)at * kSize;
        if (many < kChunk || at0 < inner0 || at0 + kSelChunkBytes > inner1) {  // the edges of row and part
#pragma unroll
          for (int j = 0; j < kSelVecs; ++j) {
            const int e0 = (j * kSelThreads + tid) * kE;
            const uint8_t* p = at0 + e0 * kSize;
            if (e0 >= many) {
#pragma unroll
              for (int i = 0; i < 4; ++i) w[4 * j + i] = kFp32 ? 0xFF800000u : 0xFF80FF80u;
            } else if (p < inner0 || p + 16 > inner1 || e0 + kE > many) {
#pragma unroll
              for (int e = 0; e < kE; ++e) {
                const float x = e0 + e < many ? raw(at + e0 + e) : -INFINITY;
                if constexpr (kFp32) w[4 * j + e % 4] = __float_as_uint(x);
                else if (e & 1) w[4 * j + e / 2 % 4] |= __float_as_uint(x) & 0xFFFF0000u;
                else w[4 * j + e / 2 % 4] = __float_as_uint(x) >> 16;
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[slot]);

      // the largest (NaN falls out)
      uint32_t m = w[0];
      float mx;
      if constexpr (kFp32) {
#pragma unroll
        for (int i = 1; i < 4 * kSelVecs; ++i)
          m = __float_as_uint(fmaxf(__uint_as_float(m), __uint_as_float(w[i])));
        mx = fmaxf(__uint_as_float(m), -INFINITY);
      } else {
#pragma unroll
        for (int i = 1; i < 4 * kSelVecs; ++i) m = max_bf16x2(m, w[i]);
        mx = fmaxf(fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u)), -INFINITY);
      }
      top = fmaxf(top, mx);
      of_cell = fmaxf(of_cell, mx);
      if (++in_cell == a.per_cell || c + 1 == chunks) {
        sm.cell[tid][cell] = __bfloat16_as_ushort(__float2bfloat16_ru(of_cell));
        ++cell;
        in_cell = 0;
        of_cell = -INFINITY;
      }

      // the sum of exponentials
      const float r = fmaxf(power, power_of(mx));
      float2 s = {0.f, 0.f}, t = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) {
        const float2 x = kFp32 ? make_float2(__uint_as_float(w[2 * i % (4 * kSelVecs)]),
                                             __uint_as_float(w[(2 * i + 1) % (4 * kSelVecs)]))
                               : make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        const float2 q = fma2(x, make_float2(kLog2e, kLog2e), make_float2(-r, -r));
        const float2 e = make_float2(ex2_approx(q.x), ex2_approx(q.y));
        if (i & 1) t = add2(t, e); else s = add2(s, e);
      }
      s = add2(s, t);
      sum = fmaf(sum, ex2_approx(power - r), s.x + s.y);
      power = r;
      // the stage's next chunk, once every warp has taken this one; the warps in turn
      if (lane == 0 && warp == (c & (kSelWarps - 1)) && c + kStages < chunks) {
        ok = mbar_wait(&sm.empty[slot], parity, a.status) && ok;
        issue(c + kStages, slot);
      }
      if (++slot == kStages) {
        slot = 0;
        parity ^= 1;
      }
    }

    // What the warps know of the sum; the bound, and the cells that reach it.  (+infinity counts
    // as the largest number here already: a bound above it would pass over logits that are its
    // equals.)
    uint32_t o = ordered(fminf(top, FLT_MAX));
    const uint32_t warp_top = __reduce_max_sync(0xffffffffu, o);
    int r = __reduce_max_sync(0xffffffffu, (int)power);
    auto fixed_sum = [&](float x) {  // of the warp, in multiples of 2^(r - 32)
      const unsigned long long f = __float2ull_rn(x * 4294967296.f);  // < 2^62
      const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)f & 0x3FFFFFFu);
      const uint32_t mid = __reduce_add_sync(0xffffffffu, (uint32_t)(f >> 26) & 0x3FFFFFFu);
      const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(f >> 52));
      return ((unsigned long long)hi << 52) + ((unsigned long long)mid << 26) + lo;
    };
    unsigned long long fixed = fixed_sum(sum * ex2_approx(power - (float)r));
    if (lane == 0) {
      sm.warp_top[warp] = warp_top;
      sm.warp_power[warp] = r;
      sm.warp_sum[warp] = fixed;
    }
    const uint2 found = bound_of(sm.bound, o, K, !(sum < INFINITY));
    const bool bad = found.y;
    uint32_t v = found.x;
    o = sm.warp_top[0];
#pragma unroll
    for (int q = 1; q < kSelWarps; ++q) o = max(o, sm.warp_top[q]);
    const float most = of_ordered(o);  // the part's largest
    v = max(v, ordered(-INFINITY) + 1);  // (-infinity never passes)
    uint16_t* hit = reinterpret_cast<uint16_t*>(ring);  // (no copy is on its way any more)
    const float least = of_ordered(v);
#pragma unroll 1
    for (int c0 = 0; c0 < cell; c0 += 8) {  // the thread's cells that do
      const uint4 u = *reinterpret_cast<const uint4*>(sm.cell[tid] + c0);
      const uint32_t x[4] = {u.x, u.y, u.z, u.w};
      uint32_t reach = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        reach |= (uint32_t)(__uint_as_float(x[k] << 16) >= least) << 2 * k |
                 (uint32_t)(__uint_as_float(x[k] & 0xFFFF0000u) >= least) << (2 * k + 1);
      reach &= (1u << min(cell - c0, 8)) - 1;
      if (reach) {
        int to = atomicAdd(&sm.hits, __popc(reach));
        for (; reach; reach &= reach - 1) hit[to++] = (uint16_t)((c0 + __ffs(reach) - 1) * kSelThreads + tid);
      }
    }
    __syncthreads();
    // Logit i of those that a thread has in chunk d of a cell: its token, or -1.
    auto token_of = [&](int cell, int d, uint32_t i) {
      const int thread = cell & (kSelThreads - 1), in_thread = (int)(i / kE * kSelThreads * kE + i % kE);
      const int t = begin + ((cell >> kLogThreads) * a.per_cell + d) * kChunk + thread * kE + in_thread;
      return t < end ? t : -1;  // (in 32 bits: no more than 40 chunks past 2^30)
    };
    const int hits = sm.hits, items = hits * a.per_cell;  // an item: one chunk of a cell
    constexpr int kAtOnce = 4, kTogether = 32 / kPer;  // items that a warp reads at once, by one load
    const int once = hits <= kSelBuffer ? items : 0;  // (of more cells more would pass than there is room for)
    constexpr int kWarpKeys = 64;  // of a warp, behind the cells' numbers in the ring
    unsigned long long* mine_keys =
        reinterpret_cast<unsigned long long*>(ring + kSelCells * kSelThreads * 2) + warp * kWarpKeys;
    int mine_many = 0;
    for (int x0 = warp * kTogether; x0 < once; x0 += kAtOnce * kSelWarps * kTogether) {
      float x[kAtOnce];
      int t[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int item = x0 + i * kSelWarps * kTogether + lane / kPer;
        const int h = (int)fast_div((uint32_t)item, a.div_cell);
        t[i] = item < items ? token_of(hit[h], item - h * a.per_cell, lane % kPer) : -1;
        x[i] = raw(max(t[i], begin));
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const bool p = t[i] >= 0 && x[i] >= least;  // (not NaN)
        const unsigned m = __ballot_sync(0xffffffffu, p);
        const int to = mine_many + __popc(m & ((1u << lane) - 1));
        if (p && to < kWarpKeys) mine_keys[to] = key_of(x[i], t[i]);
        mine_many += __popc(m);
      }
    }
    if (lane == 0) sm.warp_many[warp] = mine_many;
    __syncthreads();
    int best = 0, n = 0, before = 0, longest = 0;
#pragma unroll
    for (int q = 0; q < kSelWarps; ++q) {
      if (q == warp) before = n;
      n += sm.warp_many[q];
      longest = max(longest, sm.warp_many[q]);
    }
    if (longest <= kWarpKeys && max(n, hits) <= kSelBuffer) {
      for (int l = lane; l < mine_many; l += 32) sm.keys[before + l] = mine_keys[l];
      __syncthreads();
    } else {  // a warp a cell, of those that can still count, until there are none
      n = 0;
      constexpr uint16_t kDone = 0xFFFF;
      while (true) {
        if (tid == 0) sm.picked = 0;
        __syncthreads();
        const unsigned long long worst = best == K ? sm.keys[K - 1] : 0;
        for (int h = tid; h < hits; h += kSelThreads) {
          const int c = hit[h];
          if (c == kDone) continue;
          const float most = bf16_to_f(sm.cell[c & (kSelThreads - 1)][c >> kLogThreads]);
          if (key_of(most, max(token_of(c, 0, 0), 0)) <= worst) {
            hit[h] = kDone;
            continue;
          }
          const int to = atomicAdd(&sm.picked, 1);
          if (to >= kSelWarps) break;
          sm.pick[to] = c;
          hit[h] = kDone;
        }
        __syncthreads();
        const int picked = min(sm.picked, kSelWarps);
        if (picked == 0) break;
        for (int d = 0; d < a.per_cell; ++d) {
          const int t = warp < picked && lane < kPer ? token_of(sm.pick[warp], d, lane) : -1;
          const float x = t >= 0 ? raw(t) : -INFINITY;
          const unsigned long long key = key_of(x, t);
          if (x >= least && (best < K || key > sm.keys[K - 1])) sm.keys[best + atomicAdd(&sm.many, 1)] = key;
          __syncthreads();
          const int n = sm.many;
          __syncthreads();
          if (n) best = rank_keys(sm, best, n, K);
        }
      }
    }

    // the part's list and sum
    if (n > a.list) best = rank_keys(sm, 0, n, K);
    else best += n;  // (in any order)
#pragma unroll
    for (int q = 0; q < kSelWarps; ++q) r = max(r, sm.warp_power[q]);
    if (bad || (is_far(most) && most > -INFINITY)) {  // once more, NaN left out
      sum = 0.f;
      for (int v = begin + tid; v < end; v += kSelThreads) {
        const float y = raw(v);
        if (y > -INFINITY)
          sum += ex2_approx(is_far(most) ? (fminf(y, FLT_MAX) - most) * kLog2e : fmaf(y, kLog2e, -(float)r));
      }
      fixed = fixed_sum(sum);
      __syncthreads();  // (what the warps left was read)
      if (lane == 0) {
        sm.warp_power[warp] = r;
        sm.warp_sum[warp] = fixed;
      }
      __syncthreads();
    }
    if (tid == 0) {
      fixed = 0;
#pragma unroll
      for (int q = 0; q < kSelWarps; ++q) fixed += sm.warp_sum[q] >> min(r - sm.warp_power[q], 63);
      a.sums[item] = {fixed, most, r};
    }
    if (tid < a.list) a.lists[(int64_t)item * a.list + tid] = tid < best && ok ? sm.keys[tid] : 0;
  }
  // The last of the request's CTAs joins them.
  __syncthreads();
  if (tid == 0) {
    sm.last = atomic_add_acq_rel_gpu(a.tickets + req, 1) == a.width * a.parts - 1;
    if (sm.last) a.tickets[req] = 0;
  }
  __syncthreads();
  if (sm.last) join_request(a, *reinterpret_cast<JoinSmem*>(ring), req);
}

// Parts of a row: as many as two CTAs an SM allow, and a request's lists have room.  (The two
// large cases above, us, at the time: 21.6 and 31.7 with two CTAs an SM and four stages; three and three
// 26.2 and 31.4; four and two 25.3 and 34.2.)
static int parts_most(int64_t rows, int width, int cands, int num_sms) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(2 * num_sms / rows, kSelKeys / (width * cands)));
}
int64_t beam_parts_all(int64_t rows, int num_sms) { return rows + 2 * num_sms; }
// What passes the bound is mostly less than twice K: it is not ranked then.
int beam_list_most(int cands) { return std::min(std::max(2 * cands, 32), kMaxBeamCands); }

template <bool kFp32, int kStages>
static cudaError_t launch_select(const BeamSelectArgs& a, int64_t ctas, cudaStream_t st) {
  const int smem = std::max(kStages * kSelStageBytes, (int)sizeof(JoinSmem));
  cudaError_t e = cudaFuncSetAttribute(beam_select_kernel<kFp32, kStages>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_k(beam_select_kernel<kFp32, kStages>, dim3((unsigned)ctas), dim3(kSelThreads), smem, st, a);
}

cudaError_t launch_beam_select(BeamSelectArgs a, int num_sms, cudaStream_t st) {
  const int chunk = kSelChunkBytes / (a.fp32 ? 4 : 2);
  const int chunks = (a.vocab + chunk - 1) / chunk;
  const int64_t rows = (int64_t)a.n_reqs * a.width;
  a.parts = std::min(chunks, parts_most(rows, a.width, a.n_cands, num_sms));
  a.part_chunks = (chunks + a.parts - 1) / a.parts;
  a.parts = (chunks + a.part_chunks - 1) / a.part_chunks;
  a.list = std::min(beam_list_most(a.n_cands), kSelKeys / (a.width * a.parts));
  a.per_cell = (a.part_chunks + kSelCells - 1) / kSelCells;
  a.div_cell = make_fastdiv((uint32_t)a.per_cell);
  a.div_parts = make_fastdiv((uint32_t)a.parts);
  a.div_width = make_fastdiv((uint32_t)a.width);
  a.div_row_keys = make_fastdiv((uint32_t)(a.parts * a.list));
  const int64_t ctas = rows * a.parts;
  if (ctas > 2 * num_sms) return a.fp32 ? launch_select<true, 3>(a, ctas, st) : launch_select<false, 3>(a, ctas, st);
  return a.fp32 ? launch_select<true, 4>(a, ctas, st) : launch_select<false, 4>(a, ctas, st);
}

// ---------------------------------------------------------------------------
// Texts behind their parents: bytes in, bytes out, a CTA 4096 ids of a row.
constexpr int kAdvThreads = 256;

__global__ void __launch_bounds__(kAdvThreads) beam_advance_kernel(const BeamAdvanceArgs a, int pieces,
                                                                  FastDiv div_pieces) {
  pdl_launch_dependents();
  pdl_wait();
  const int row = (int)fast_div(blockIdx.x, div_pieces), piece = blockIdx.x - row * pieces;
  const int tid = threadIdx.x;
  int p = a.parents[row];
  bool bad = p < -1 || p >= a.n_rows;
  if (bad) p = -1;
  int64_t n = 0;
  if (p >= 0) {
    n = a.lens[p];
    const int64_t most = min(a.room, a.room_out);
    if (n < 0 || n > most) {
      bad = true;
      n = max((int64_t)0, min(n, most));
    }
  }
  const bool room = p >= 0 && n < a.room_out;
  if (p >= 0 && !room) bad = true;
  int32_t* out = a.out + row * a.ld_out;
  if (piece == 0 && tid == 0) {
    a.lens_out[row] = (int)n + room;
    if (room) out[n] = a.tokens[row];
    if (bad) record_status(a.status, kStatusTableRange);
  }
  const int32_t* in = a.history + max(p, 0) * a.ld;
  const int64_t begin = (int64_t)piece * kAdvIds, end = min(n, begin + kAdvIds);
  if (((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0) {
    for (int64_t i = begin + 4 * tid; i < end; i += 4 * kAdvThreads) {
      if (i + 4 <= end) *reinterpret_cast<int4*>(out + i) = *reinterpret_cast<const int4*>(in + i);
      else for (int64_t j = i; j < end; ++j) out[j] = in[j];
    }
  } else {
    for (int64_t i = begin + tid; i < end; i += kAdvThreads) out[i] = in[i];
  }
}

cudaError_t launch_beam_advance(const BeamAdvanceArgs& a, cudaStream_t st) {
  const int pieces = (int)beam_advance_pieces(std::min(a.room, a.room_out));
  return launch_k(beam_advance_kernel, dim3((unsigned)((int64_t)a.n_rows * pieces)), dim3(kAdvThreads), 0, st, a,
                  pieces, make_fastdiv((uint32_t)pieces));
}

}  // namespace tpk
