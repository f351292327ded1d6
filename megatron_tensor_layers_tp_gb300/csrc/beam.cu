// Beam search's selection over beams and vocabulary, and the beams' texts.
//
// A continuation of row b by token v is worth s_b + (x_v - M) - log sum exp(x - M),
// M the row's largest logit.  Within a row the order is the logits', so the sum
// and the K best logits come out of one pass; a row is cut into parts, and the
// last CTA of a request's parts joins their sums and lists.
//
// The K best: a chunk of the part at a time in registers.  The K-th largest of
// 128 maxima (two threads each) of the first chunk bounds the K-th largest
// logit from below; what passes the bound goes to a buffer in shared memory, and
// the buffer, when it has many, is ranked by counting and cut to K, which
// raises the bound.  Later chunks' tokens have higher numbers, so that only
// what is larger than the bound can still count.  A chunk from which more passes
// than the buffer holds (rising or equal logits) is taken one logit of each
// thread at a time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "paged.h"
#include "ptx.cuh"

namespace tpk {

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr int kSelVecs = 4;         // 16-byte words of a thread in a chunk
constexpr int kSelBuffer = 512;     // keys that may pass a bound
constexpr int kSelRank = 192;       // from so many on they are ranked
constexpr int kSelLists = 512;      // parts of a request, at most
constexpr float kLog2e = 1.4426950408889634f;

// Bits whose order as whole numbers is that of the values (-0 as 0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_ordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
// Larger for larger logits, among equal ones for lower tokens; never 0.
__device__ __forceinline__ unsigned long long key_of(float x, int token) {
  return (unsigned long long)ordered(fminf(x, FLT_MAX)) << 32 | (uint32_t)~token;
}

struct SelectSmem {
  unsigned long long keys[kSelBuffer + kMaxBeamCands];  // the best so far, then the buffer
  float group[kSelThreads / 2];
  float bound;
  int many, valid;   // keys in the buffer; before the first that found no room
  int last;
  float warp_top[kSelWarps];
  double warp_sum[kSelWarps];
  // the join of a request's parts
  double row_top[kMaxBeams], row_log[kMaxBeams], row_score[kMaxBeams];
  double value[kSelWarps][kMaxBeamCands];
  unsigned long long key[kSelWarps][kMaxBeamCands];
  int row[kSelWarps][kMaxBeamCands];
  int found[kSelWarps];
  int best_row[kMaxBeamCands], best_token[kMaxBeamCands];
  float best_score[kMaxBeamCands];
};

// Ranks the keys, `best` sorted ones and n more, and keeps the K best: their
// number.  All threads, together; the keys are visible on entry and exit.
__device__ __forceinline__ int rank_keys(SelectSmem& sm, int best, int n, int K) {
  const int m = best + n, tid = threadIdx.x;
  constexpr int kMost = (kSelBuffer + kMaxBeamCands + kSelThreads - 1) / kSelThreads;
  unsigned long long key[kMost];
  int rank[kMost];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int at = tid + i * kSelThreads;
    if (at >= m) break;
    key[i] = sm.keys[at];
    int r = 0;
    for (int j = 0; j < m; ++j) r += sm.keys[j] > key[i];
    rank[i] = r;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    if (tid + i * kSelThreads >= m) break;
    if (rank[i] < K) sm.keys[rank[i]] = key[i];
  }
  if (tid == 0) sm.many = 0;
  __syncthreads();
  return min(m, K);
}

// A continuation: its value, row of the request and key; no row: none.
struct Candidate {
  double value;
  unsigned long long key;
  int row;
};
// The better value, equal ones by row, logit (different logits of a row can have the
// same value in 64 bits) and token.
__device__ __forceinline__ bool before(const Candidate& a, const Candidate& b) {
  if (a.value != b.value) return a.value > b.value;
  return a.row != b.row ? a.row < b.row : a.key > b.key;
}

// The request's parts joined: its candidates and next beams.
__device__ void join_request(const BeamSelectArgs& a, SelectSmem& sm, int req) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int W = a.width, K = a.n_cands, lists = W * a.parts;
  const int row0 = req * W;
  for (int w = warp; w < W; w += kSelWarps) {
    const float score = a.scores[row0 + w];
    const BeamPart* p = a.sums + (int64_t)(row0 + w) * a.parts;
    const bool used = isfinite(score);
    float top = -FLT_MAX;
    if (used)
      for (int i = lane; i < a.parts; i += 32) top = fmaxf(top, p[i].top);
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    double sum = 0.;
    if (used)
      for (int i = lane; i < a.parts; i += 32) sum += p[i].sum * exp((double)p[i].top - (double)top);
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      sm.row_top[w] = top;
      sm.row_log[w] = log(sum);
      sm.row_score[w] = used ? (double)score : -INFINITY;
    }
  }
  __syncthreads();

  // Each warp takes every eighth list, a lane up to two of them, and draws the
  // best head K times.
  constexpr int kOwn = kSelLists / kSelThreads;
  Candidate own[kOwn];
  int next[kOwn];
  auto head = [&](int i) {
    own[i] = {-INFINITY, 0, kMaxBeams};  // none: behind all others
    const int l = warp + kSelWarps * (lane + 32 * i);
    if (l >= lists || next[i] >= K) return;
    const int w = l / a.parts;
    if (sm.row_score[w] == -INFINITY) return;
    const unsigned long long key = a.lists[((int64_t)row0 * a.parts + l) * K + next[i]];
    if (key == 0) return;
    own[i] = {((double)of_ordered((uint32_t)(key >> 32)) - sm.row_top[w] - sm.row_log[w]) + sm.row_score[w], key, w};
  };
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    next[i] = 0;
    head(i);
  }
  int n = 0;
  for (; n < K; ++n) {
    Candidate c = own[0];
#pragma unroll
    for (int i = 1; i < kOwn; ++i)
      if (before(own[i], c)) c = own[i];
    for (int o = 16; o; o >>= 1) {
      const Candidate d = {__shfl_xor_sync(0xffffffffu, c.value, o), __shfl_xor_sync(0xffffffffu, c.key, o),
                           __shfl_xor_sync(0xffffffffu, c.row, o)};
      if (before(d, c)) c = d;
    }
    if (c.row == kMaxBeams) break;
    if (lane == 0) {
      sm.value[warp][n] = c.value;
      sm.key[warp][n] = c.key;
      sm.row[warp][n] = c.row;
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (own[i].row == c.row && own[i].key == c.key) {
        ++next[i];
        head(i);
      }
  }
  if (lane == 0) sm.found[warp] = n;
  __syncthreads();

  // A candidate's place: those before it in every warp's list.
  auto listed = [&](int q, int i) { return Candidate{sm.value[q][i], sm.key[q][i], sm.row[q][i]}; };
  int all = 0;
  for (int q = 0; q < kSelWarps; ++q) all += sm.found[q];
  all = min(all, K);
  for (int e = tid; e < kSelWarps * kMaxBeamCands; e += kSelThreads) {
    const int q = e / kMaxBeamCands, i = e % kMaxBeamCands;
    if (i >= sm.found[q]) continue;
    const Candidate c = listed(q, i);
    int place = i;
    for (int p = 0; p < kSelWarps; ++p) {
      if (p == q) continue;
      int lo = 0, hi = sm.found[p];
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (before(listed(p, mid), c)) lo = mid + 1; else hi = mid;
      }
      place += lo;
    }
    if (place < K) {
      sm.best_row[place] = row0 + c.row;
      sm.best_token[place] = (int)~(uint32_t)c.key;
      sm.best_score[place] = (float)c.value;
    }
  }
  __syncthreads();
  if (tid < K) {
    const bool there = tid < all;
    a.cand_scores[req * K + tid] = there ? sm.best_score[tid] : -INFINITY;
    a.cand_rows[req * K + tid] = there ? sm.best_row[tid] : -1;
    a.cand_tokens[req * K + tid] = there ? sm.best_token[tid] : -1;
  }
  // The next beams: the first W whose token ends no text.
  if (warp == 0) {
    int placed = 0;
    for (int base = 0; base < K; base += 32) {
      const int i = base + lane;
      bool goes = i < all;
      for (int e = 0; e < a.n_ends; ++e) goes = goes && sm.best_token[i] != a.ends[e];
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

template <bool kFp32>
__global__ void __launch_bounds__(kSelThreads) beam_select_kernel(const BeamSelectArgs a) {
  constexpr int kE = kFp32 ? 4 : 8;           // logits of a 16-byte word
  constexpr int kPer = kSelVecs * kE;         // of a thread in a chunk
  constexpr int kChunk = kSelThreads * kPer;
  __shared__ SelectSmem sm;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = blockIdx.x, row = (int)fast_div((uint32_t)item, a.div_parts);
  const int part = item - row * a.parts, req = (int)fast_div((uint32_t)row, a.div_width);
  const int K = a.n_cands;
  if (tid == 0) {
    sm.many = 0;
    sm.valid = kSelBuffer;
  }
  if (isfinite(a.scores[row])) {
    const int begin = (int)min((int64_t)part * a.part_chunks * kChunk, (int64_t)a.vocab);
    const int end = (int)min((int64_t)begin + (int64_t)a.part_chunks * kChunk, (int64_t)a.vocab);
    const uint8_t* base = static_cast<const uint8_t*>(a.logits) + row * a.ld * (kFp32 ? 4 : 2);
    const bool vec = (reinterpret_cast<uintptr_t>(base) & 15) == 0;
    float bound = -INFINITY, top = -FLT_MAX, sum = 0.f;
    int best = 0;
    for (int at = begin; at < end; at += kChunk) {
      float x[kPer];
#pragma unroll
      for (int j = 0; j < kSelVecs; ++j) {
        const int v = at + (j * kSelThreads + tid) * kE;
        if (vec && v + kE <= end) {
          const uint4 u = *reinterpret_cast<const uint4*>(base + (int64_t)v * (kFp32 ? 4 : 2));
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < kE; ++e)
            x[j * kE + e] = kFp32 ? __uint_as_float(w[e & 3])
                                  : __uint_as_float(e & 1 ? w[e / 2 & 3] & 0xFFFF0000u : w[e / 2 & 3] << 16);
        } else {
#pragma unroll
          for (int e = 0; e < kE; ++e)
            x[j * kE + e] = v + e >= end ? -INFINITY
                            : kFp32 ? reinterpret_cast<const float*>(base)[v + e]
                                    : bf16_to_f(reinterpret_cast<const uint16_t*>(base)[v + e]);
        }
      }
      auto token = [&](int i) { return at + (i / kE * kSelThreads + tid) * kE + i % kE; };
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < kPer; ++i) mx = fmaxf(mx, x[i]);  // (NaN falls out)

      // the sum of exponentials, from the thread's largest logit so far on
      {
        const float t = fmaxf(top, fminf(mx, FLT_MAX));
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) s += ex2_approx((x[i] - t) * kLog2e);
        if (!(s < INFINITY)) {  // infinities and NaN among them
          s = 0.f;
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (x[i] == x[i]) s += ex2_approx((fminf(x[i], FLT_MAX) - t) * kLog2e);
        }
        sum = sum * ex2_approx((top - t) * kLog2e) + s;
        top = t;
      }

      const bool first = at == begin;
      if (first) {
        const float g = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        if ((lane & 1) == 0) sm.group[tid >> 1] = g;
        __syncthreads();
        if (tid < kSelThreads / 2) {
          const float mine = sm.group[tid];
          int r = 0;
          for (int j = 0; j < kSelThreads / 2; ++j)
            r += sm.group[j] > mine || (sm.group[j] == mine && j < tid);
          if (r == K - 1) sm.bound = mine;
        }
        __syncthreads();
        bound = sm.bound;
      }
      auto passes = [&](float y) { return first ? y >= bound && y > -INFINITY : y > bound; };
      bool fails = false;
      if (first ? mx >= bound : mx > bound) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) n += passes(x[i]);
        if (n) {
          int to = atomicAdd(&sm.many, n);
          if (to + n <= kSelBuffer) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
              if (passes(x[i])) sm.keys[best + to++] = key_of(x[i], token(i));
          } else {
            atomicMin(&sm.valid, to);
            fails = true;
          }
        }
      }
      if (__syncthreads_or(fails)) {
        const int n = sm.valid;
        __syncthreads();
        if (tid == 0) sm.valid = kSelBuffer;
        best = rank_keys(sm, best, n, K);
#pragma unroll 1
        for (int i = 0; i < kPer; ++i) {
          float y = 0.f;
#pragma unroll
          for (int q = 0; q < kPer; ++q)
            if (q == i) y = x[q];
          const unsigned long long least = best == K ? sm.keys[K - 1] : 0;
          const unsigned long long key = key_of(y, token(i));
          if (fails && passes(y) && key > least) sm.keys[best + atomicAdd(&sm.many, 1)] = key;
          __syncthreads();
          const int more = sm.many;
          __syncthreads();
          if (more) best = rank_keys(sm, best, more, K);
        }
        if (best == K) bound = fmaxf(bound, of_ordered((uint32_t)(sm.keys[K - 1] >> 32)));
      } else if (sm.many > kSelRank) {
        const int n = sm.many;
        __syncthreads();
        best = rank_keys(sm, best, n, K);
        if (best == K) bound = fmaxf(bound, of_ordered((uint32_t)(sm.keys[K - 1] >> 32)));
      } else {
        __syncthreads();
      }
    }
    const int n = sm.many;
    __syncthreads();
    if (n) best = rank_keys(sm, best, n, K);

    // the part's list and sum
    float all = top;
    for (int o = 16; o; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
    if (lane == 0) sm.warp_top[warp] = all;
    __syncthreads();
    all = sm.warp_top[0];
#pragma unroll
    for (int q = 1; q < kSelWarps; ++q) all = fmaxf(all, sm.warp_top[q]);
    double d = (double)sum * (double)ex2_approx((top - all) * kLog2e);
    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) sm.warp_sum[warp] = d;
    __syncthreads();
    if (tid == 0) {
      d = 0.;
#pragma unroll
      for (int q = 0; q < kSelWarps; ++q) d += sm.warp_sum[q];
      a.sums[item] = {d, all};
    }
    if (tid < K) a.lists[(int64_t)item * K + tid] = tid < best ? sm.keys[tid] : 0;
  }
  // The last of the request's CTAs joins them.
  __syncthreads();
  if (tid == 0) {
    fence_acq_rel_gpu();
    sm.last = atomicAdd(a.tickets + req, 1) == a.width * a.parts - 1;
    if (sm.last) a.tickets[req] = 0;
    fence_acq_rel_gpu();
  }
  __syncthreads();
  if (sm.last) join_request(a, sm, req);
}

// Parts of a row: enough for two CTAs an SM.
static int parts_most(int64_t rows, int width, int num_sms) {
  const int64_t want = (2 * num_sms + rows - 1) / rows;
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, kSelLists / width));
}
int64_t beam_parts_all(int64_t rows, int num_sms) { return rows + 2 * num_sms; }

cudaError_t launch_beam_select(BeamSelectArgs a, int num_sms, cudaStream_t st) {
  const int chunk = kSelThreads * kSelVecs * (a.fp32 ? 4 : 8);
  const int chunks = (a.vocab + chunk - 1) / chunk;
  const int64_t rows = (int64_t)a.n_reqs * a.width;
  a.parts = std::min(chunks, parts_most(rows, a.width, num_sms));
  a.part_chunks = (chunks + a.parts - 1) / a.parts;
  a.parts = (chunks + a.part_chunks - 1) / a.part_chunks;
  a.div_parts = make_fastdiv((uint32_t)a.parts);
  a.div_width = make_fastdiv((uint32_t)a.width);
  return launch_k(a.fp32 ? beam_select_kernel<true> : beam_select_kernel<false>,
                  dim3((unsigned)(rows * a.parts)), dim3(kSelThreads), 0, st, a);
}

// ---------------------------------------------------------------------------
// Texts behind their parents: bytes in, bytes out, a CTA 4096 ids of a row.
constexpr int kAdvThreads = 256, kAdvIds = 4096;

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
    const int64_t most = min(a.ld, a.ld_out);
    if (n < 0 || n > most) {
      bad = true;
      n = max((int64_t)0, min(n, most));
    }
  }
  const bool room = p >= 0 && n < a.ld_out;
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

cudaError_t launch_beam_advance(const BeamAdvanceArgs& a, int num_sms, cudaStream_t st) {
  const int pieces = (int)std::max<int64_t>(1, (std::min(a.ld, a.ld_out) + kAdvIds - 1) / kAdvIds);
  return launch_k(beam_advance_kernel, dim3((unsigned)((int64_t)a.n_rows * pieces)), dim3(kAdvThreads), 0, st, a,
                  pieces, make_fastdiv((uint32_t)pieces));
}

}  // namespace tpk
