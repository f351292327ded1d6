// Penalties, biases and grammar masks on logits.
//
// x = logit; seen tokens: x > 0 ? x / repetition : x * repetition;
// x -= frequency * count; x -= presence * [count > 0]; x += bias; tokens not
// allowed: -infinity.  Counts come from the request's text and the drafted
// tokens on the row's path.
//
// Memory-bound: 2 bytes in, 2 or 4 out and a mask bit a token.  The vocabulary
// is cut into slices; a CTA takes one slice of some consecutive rows, the next
// row's logits, mask bits and path in flight while it works on this one.  A
// slice is every so-manieth block of 64 tokens: frequent tokens have
// neighbouring numbers, and runs of the vocabulary would give one CTA all of
// them (50 us instead of 47 for the rows below).
//
// What a request's text, biases and drafted path touch of a slice is little.
// All tokens stream through first, as copies with the mask applied, a few
// instructions each.  Meanwhile the CTA marks the touched tokens in shared memory
// (integer atomics: their order does not matter; 16 bits a token, or 32 where a
// text is long enough to overflow them) and lists them: once for as many rows as
// belong to the same request, a row's path added and taken out again.  The listed
// ones are then written over with the rules applied, one thread each, while their
// lines are still in the caches.  (In place the copies change only what is not
// allowed, so the listed tokens' logits are still there.)
//
// 256 rows (16 trees) of 152064 logits, texts of 1500 tokens, 300 biases, bf16:
// 45.5 us, 3.5 TB/s; the stream alone takes 29.  Measured before: marks before the
// stream: 47; the rules applied in the stream, a slice a CTA: 110 us; the touched
// tokens in a second kernel behind the stream: 55 us, since their lines come from
// memory again; rows through shared memory by asynchronous copies, three ahead: 63.
// 64 rows of 128256 with texts of 4096 tokens, fp32: 21 us, 2.3 TB/s (the stream
// alone 10.5); there the text's way into the marks binds.
//
// Slices have 4096 tokens; 2048 where there are too few rows to fill the GPU; 8192
// where the text buffer's rows have room for 2048 ids or more, since every slice
// reads the whole text.  That room stands in for the texts' lengths, which only the
// GPU knows.  Measured at texts of 300, 1500, 4000, 8000 ids (us, 8192 against 4096
// tokens a slice):
//   64 rows of as many requests, fp32        16.8 18.3 21.1 28.9   20.4 22.0 24.8 34.3
//   200 rows of as many requests, bf16       35.2 38.5 45.2 65.1   48.4 54.6 63.5 89.4
//   32 trees of 4, grammar                   22.4 23.1 25.1 32.1   27.0 27.9 30.0 36.4
//   16 trees of 16, grammar and 300 biases   81.0 81.4 84.0 103    44.8 45.5 47.1 51.5
// So the last kind pays for a buffer with that much room, whatever its texts are
// (16-bit marks, and 32-bit ones from 16128 ids on: 64 at 32768).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "paged.h"
#include "ptx.cuh"

namespace tpk {

// Marks of a token: bit 0 = in the prompt, bit 1 = has a bias, the rest = times
// written by the model.
constexpr uint32_t kMarkPrompt = 1, kMarkBias = 2, kMarkWritten = 4;
// the longest text (and path) whose counts fit 16-bit marks
constexpr int64_t kNarrowText = (1 << 14) - 1;

// The slice's marks; add and set return what the token had before.
template <bool kWide>
struct Marks {
  uint32_t* w;
  __device__ __forceinline__ uint32_t add(int v, uint32_t x) {
    if constexpr (kWide) return atomicAdd(w + v, x);
    else return atomicAdd(w + (v >> 1), x << (16 * (v & 1))) >> (16 * (v & 1)) & 0xFFFF;
  }
  __device__ __forceinline__ uint32_t set(int v, uint32_t x) {
    if constexpr (kWide) return atomicOr(w + v, x);
    else return atomicOr(w + (v >> 1), x << (16 * (v & 1))) >> (16 * (v & 1)) & 0xFFFF;
  }
  __device__ __forceinline__ uint32_t get(int v) const {
    if constexpr (kWide) return w[v];
    else return (w[v >> 1] >> (16 * (v & 1))) & 0xFFFF;
  }
};

// A thread's part of a row: its logits, which of them are allowed, and a token
// of the row's drafted path (-1: none).
template <int kPer>
struct RowPart {
  uint4 x[kPer / 8];
  uint32_t ok;
  int path;
};

// What a row's indices say, looked up once by the CTA: its request (-1: left
// alone), its grammar row (-1: none, -2: nothing is allowed), its path's first
// token and length.
struct RowInfo {
  int r, m, q0, T;
};
constexpr int kLogRows = 16;  // rows of a CTA, at most

// Two logits with those not allowed made -infinity (0xFF80).
__device__ __forceinline__ uint32_t allow2(uint32_t w, uint32_t ok) {
  if (!(ok & 1)) w = (w & 0xFFFF0000u) | 0xFF80u;
  if (!(ok & 2)) w = (w & 0x0000FFFFu) | 0xFF800000u;
  return w;
}

template <int kThreads, int kPer, bool kWide>
struct LogitsSmem {
  static constexpr int kSlice = kThreads * kPer;
  static constexpr int kMarks = 16 + kLogRows * sizeof(RowInfo);  // after the count and the rows
  static constexpr int kList = kMarks + kSlice * (kWide ? 4 : 2);
  static constexpr int kBias = kList + kSlice * 2;
  static constexpr int bytes(bool bias) { return kBias + (bias ? kSlice * 4 : 0); }
};

template <int kThreads, int kPer, bool kWide>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) process_logits_kernel(const LogitsArgs a, int slices, FastDiv div_slices,
                                                                  int rows) {
  using SM = LogitsSmem<kThreads, kPer, kWide>;
  constexpr int kSlice = SM::kSlice;
  extern __shared__ __align__(16) uint8_t smem[];
  int* listed = reinterpret_cast<int*>(smem);  // tokens in the list
  RowInfo* info = reinterpret_cast<RowInfo*>(smem + 16);
  Marks<kWide> marks{reinterpret_cast<uint32_t*>(smem + SM::kMarks)};
  uint16_t* list = reinterpret_cast<uint16_t*>(smem + SM::kList);
  float* bias = reinterpret_cast<float*>(smem + SM::kBias);      // with a.bias_start
  pdl_launch_dependents();
  pdl_wait();
  const int group = blockIdx.x / slices, slice = blockIdx.x - group * slices;
  const int tid = threadIdx.x;
  // place i of the slice <-> token
  auto token = [&](int i) { return ((i >> 6) * slices + slice) * 64 + (i & 63); };
  auto place = [&](int id) {  // -1: not a token of the slice
    if ((uint32_t)id >= (uint32_t)a.vocab) return -1;
    const int block = id >> 6, turn = (int)fast_div((uint32_t)block, div_slices);
    return block - turn * slices == slice ? turn * 64 + (id & 63) : -1;
  };
  const int row0 = group * rows, row1 = (int)min((int64_t)row0 + rows, (int64_t)a.S);
  auto in_of = [&](int row) { return a.logits + row * a.ld; };
  auto out_of = [&](int row) {
    return static_cast<uint8_t*>(a.out) + row * a.ld_out * (a.out_fp32 ? 4 : 2);
  };
  auto mask_of = [&](int m) {
    return reinterpret_cast<const uint8_t*>(a.allowed + m * a.ld_allowed);
  };

  // token t of the row's drafted path that lies in the slice, or -1
  auto path_token = [&](int row, const RowInfo& w, int t) {
    if (t >= w.T || !((a.tree_mask[(int64_t)row * a.tree_words + (t >> 6)] >> (t & 63)) & 1)) return -1;
    return place(a.draft_tokens[w.q0 + t]);
  };
  if (tid < row1 - row0) {
    const int row = row0 + tid;
    RowInfo w;
    w.r = a.row_req ? a.row_req[row] : row;
    w.m = a.allowed ? (a.allowed_row ? a.allowed_row[row] : row) : -1;
    w.q0 = w.T = 0;
    bool bad = false;
    if (w.r < 0 || w.r >= a.n_reqs) {
      bad = w.r != -1;
      w.r = w.m = -1;  // nothing of the row is looked up
    } else {
      if (a.allowed && (w.m < -1 || w.m >= a.n_allowed)) {
        bad = true;
        w.m = -2;
      }
      if (a.draft_tokens) {
        const int q0 = a.q_start[w.r];
        const int64_t T = (int64_t)a.q_start[w.r + 1] - q0;
        if (q0 < 0 || T < 0 || q0 + T > a.S) {
          bad = true;
        } else {
          w.q0 = q0;
          w.T = (int)min(T, (int64_t)64 * a.tree_words);
        }
      }
    }
    if (bad && slice == 0) record_status(a.status, kStatusTableRange);
    info[tid] = w;
  }
  __syncthreads();

  // The thread's tokens: runs of 8 where the rows allow 16-byte accesses, else
  // single ones a CTA's width apart.
  auto vec_row = [&](int row) {
    return ((reinterpret_cast<uintptr_t>(in_of(row)) | reinterpret_cast<uintptr_t>(out_of(row))) & 15) == 0;
  };
  auto fetch = [&](int row) {
    RowPart<kPer> p;
    const RowInfo w = info[row - row0];
    const uint16_t* in = in_of(row);
    p.ok = w.m == -2 ? 0 : 0xFFFFFFFFu;  // bit i: token i of the thread is allowed
    const uint8_t* mask = w.m >= 0 ? mask_of(w.m) : nullptr;
    p.path = -1;
    if (a.draft_tokens) p.path = path_token(row, w, tid);
    if (vec_row(row)) {
#pragma unroll
      for (int j = 0; j < kPer / 8; ++j) {
        const int v = token((j * kThreads + tid) * 8);
        if (v + 8 <= a.vocab) p.x[j] = *reinterpret_cast<const uint4*>(in + v);
        if (mask && v < a.vocab) p.ok &= ~(0xFFu << (8 * j)) | (uint32_t)mask[v / 8] << (8 * j);
      }
    } else {
      uint32_t* x2 = reinterpret_cast<uint32_t*>(p.x);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int v = token(j * kThreads + tid);
        const uint32_t e = v < a.vocab ? in[v] : 0;
        x2[j / 2] = j & 1 ? x2[j / 2] | e << 16 : e;
        if (mask && v < a.vocab && !(mask[v >> 3] >> (v & 7) & 1)) p.ok &= ~(1u << j);
      }
    }
    return p;
  };
  auto enlist = [&](int v, uint32_t before) {
    if (before == 0) list[atomicAdd(listed, 1)] = (uint16_t)v;
  };

  // Marks and list of request r's text and biases in the slice; starts and ends
  // with the CTA's threads together.
  auto mark_request = [&](int r) {
    __syncthreads();
    for (int i = tid; i < kSlice * (kWide ? 4 : 2) / 16; i += kThreads)
      reinterpret_cast<uint4*>(smem + SM::kMarks)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) *listed = 0;
    __syncthreads();
    if (a.history) {
      const int len = a.history_lens[r], pl = a.prompt_lens ? a.prompt_lens[r] : 0;
      const int len_c = (int)min((int64_t)max(len, 0), a.ld_history), pl_c = min(max(pl, 0), len_c);
      if ((len != len_c || pl != pl_c) && tid == 0) record_status(a.status, kStatusTableRange);
      const int32_t* h = a.history + r * a.ld_history;
      auto mark = [&](int i, int id) {
        const int v = place(id);
        if (v >= 0) enlist(v, i < pl_c ? marks.set(v, kMarkPrompt) : marks.add(v, kMarkWritten));
      };
      const int quads = (reinterpret_cast<uintptr_t>(h) & 15) ? 0 : len_c / 4;
      // Few tokens of a text lie in the slice: the thread finds which of its 16
      // do, and then marks those alone (their ids once more, from L1), instead of
      // taking part in its neighbours' marks 16 times.
      for (int i0 = tid; i0 < quads; i0 += 4 * kThreads) {
        uint32_t in_slice = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = i0 + k * kThreads;
          const int4 id = i < quads ? reinterpret_cast<const int4*>(h)[i] : make_int4(-1, -1, -1, -1);
          in_slice |= (uint32_t)((place(id.x) >= 0) | (place(id.y) >= 0) << 1 | (place(id.z) >= 0) << 2 |
                                 (place(id.w) >= 0) << 3) << (4 * k);
        }
        for (; in_slice; in_slice &= in_slice - 1) {
          const int e = __ffs(in_slice) - 1, i = 4 * (i0 + (e >> 2) * kThreads) + (e & 3);
          mark(i, h[i]);
        }
      }
      for (int i = 4 * quads + tid; i < len_c; i += kThreads) mark(i, h[i]);
    }
    if (a.bias_start) {
      int b0 = a.bias_start[r], b1 = a.bias_start[r + 1];
      if (b0 < 0 || b1 < b0 || b1 > a.n_biases) {
        if (tid == 0) record_status(a.status, kStatusTableRange);
        b0 = b1 = 0;  // (counting on from any b0 could overflow)
      }
      // Entries of tokens named once need no order.  How often a token is named
      // is counted in its place in the bias array.
      int* named = reinterpret_cast<int*>(bias);
      bool any = false;
      for (int i = b0 + tid; i < b1; i += kThreads) {
        const int v = place(a.bias_ids[i]);
        if (v >= 0) {
          named[v] = 0;
          any = true;
        }
      }
      if (__syncthreads_or(any)) {
        for (int i = b0 + tid; i < b1; i += kThreads) {
          const int v = place(a.bias_ids[i]);
          if (v >= 0) {
            atomicAdd(named + v, 1);
            enlist(v, marks.set(v, kMarkBias));
          }
        }
        __syncthreads();
        bool again = false;
        for (int i = b0 + tid; i < b1; i += kThreads) {
          const int v = place(a.bias_ids[i]);
          if (v >= 0) {
            if (named[v] == 1) bias[v] = a.bias_values[i];  // no other entry looks at it
            else again = true;
          }
        }
        if (__syncthreads_or(again)) {
          // Some token is named more than once: the list anew, in order, by one
          // warp, entries of the same token among its 32 added in order too.
          for (int i = b0 + tid; i < b1; i += kThreads) {
            const int v = place(a.bias_ids[i]);
            if (v >= 0) bias[v] = 0.f;
          }
          __syncthreads();
          if (tid < 32) {
            for (int base = b0; base < b1; base += 32) {
              const int i = base + tid;
              const int v = i < b1 ? place(a.bias_ids[i]) : -1;
              const bool here = v >= 0;
              const float y = here ? a.bias_values[i] : 0.f;
              const unsigned same = __match_any_sync(0xffffffffu, here ? v : -1 - tid);
              const bool lead = here && (same & ((1u << tid) - 1)) == 0;
              float s = lead ? bias[v] : 0.f;
              for (int j = 0; j < 32; ++j) {
                const float z = __shfl_sync(0xffffffffu, y, j);
                if (same >> j & 1) s += z;
              }
              if (lead) bias[v] = s;
              __syncwarp();
            }
          }
        }
      }
    }
    __syncthreads();
  };

  const bool marked = a.history || a.draft_tokens || a.bias_start;
  RowPart<kPer> next = fetch(row0);
  int made = -1, own = 0;  // the request whose marks are there; its listed tokens
  float rep = 1.f, freq = 0.f, pres = 0.f;
  for (int row = row0; row < row1; ++row) {
    const RowPart<kPer> p = next;
    const RowInfo w = info[row - row0];
    if (row + 1 < row1) next = fetch(row + 1);
    if (w.r < 0) continue;
    uint8_t* out = out_of(row);
    if (vec_row(row)) {
#pragma unroll
      for (int j = 0; j < kPer / 8; ++j) {
        const int v = token((j * kThreads + tid) * 8);
        if (v >= a.vocab) break;
        const uint32_t ok = p.ok >> (8 * j);
        if (v + 8 <= a.vocab) {
          const uint32_t e[4] = {allow2(p.x[j].x, ok), allow2(p.x[j].y, ok >> 2),
                                 allow2(p.x[j].z, ok >> 4), allow2(p.x[j].w, ok >> 6)};
          if (a.out_fp32) {
            uint4* o = reinterpret_cast<uint4*>(out) + v / 4;
            o[0] = make_uint4(e[0] << 16, e[0] & 0xFFFF0000u, e[1] << 16, e[1] & 0xFFFF0000u);
            o[1] = make_uint4(e[2] << 16, e[2] & 0xFFFF0000u, e[3] << 16, e[3] & 0xFFFF0000u);
          } else {
            reinterpret_cast<uint4*>(out)[v / 8] = make_uint4(e[0], e[1], e[2], e[3]);
          }
        } else {  // the row's last tokens
          for (int q = 0; v + q < a.vocab; ++q) {
            const uint32_t e = ok >> q & 1 ? in_of(row)[v + q] : 0xFF80u;
            if (a.out_fp32) reinterpret_cast<uint32_t*>(out)[v + q] = e << 16;
            else reinterpret_cast<uint16_t*>(out)[v + q] = (uint16_t)e;
          }
        }
      }
    } else {
      const uint32_t* x2 = reinterpret_cast<const uint32_t*>(p.x);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int v = token(j * kThreads + tid);
        if (v >= a.vocab) break;
        const uint32_t e = p.ok >> j & 1 ? (j & 1 ? x2[j / 2] >> 16 : x2[j / 2] & 0xFFFF) : 0xFF80u;
        if (a.out_fp32) reinterpret_cast<uint32_t*>(out)[v] = e << 16;
        else reinterpret_cast<uint16_t*>(out)[v] = (uint16_t)e;
      }
    }

    if (marked) {
      if (w.r != made) {
        if (a.repetition) rep = a.repetition[w.r];
        if (a.frequency) freq = a.frequency[w.r];
        if (a.presence) pres = a.presence[w.r];
        mark_request(w.r);
        made = w.r;
        own = *listed;
        __syncthreads();  // own was read
      }
      int far = -1;  // (paths have up to 256 tokens: two a thread where a CTA has 128)
      if (a.draft_tokens) {
        if (kThreads < kMaxTreeTokens) far = path_token(row, w, tid + kThreads);
        if (p.path >= 0) enlist(p.path, marks.add(p.path, kMarkWritten));
        if (far >= 0) enlist(far, marks.add(far, kMarkWritten));
      }
      __syncthreads();  // the stream is through, the list complete
      const int many = *listed;
      const uint16_t* in = in_of(row);
      const uint8_t* mask = w.m >= 0 ? mask_of(w.m) : nullptr;
      for (int i = tid; i < many; i += kThreads) {
        const int at = list[i], v = token(at);
        const uint32_t mk = marks.get(at), times = mk / kMarkWritten;
        float x = bf16_to_f(in[v]);  // (in place: as it was where it is allowed)
        if (times || (mk & kMarkPrompt)) x = x > 0.f ? x / rep : x * rep;
        if (times) x = x - freq * (float)times - pres;
        if (mk & kMarkBias) x += bias[at];
        if (w.m == -2 || (mask && !(mask[v >> 3] >> (v & 7) & 1))) x = -INFINITY;
        if (a.out_fp32) reinterpret_cast<float*>(out)[v] = x;
        else reinterpret_cast<uint16_t*>(out)[v] = f_to_bf16(x);
      }
      if (a.draft_tokens && row + 1 < row1) {
        __syncthreads();
        if (p.path >= 0) marks.add(p.path, 0u - kMarkWritten);
        if (far >= 0) marks.add(far, 0u - kMarkWritten);
        if (tid == 0) *listed = own;
        __syncthreads();
      }
    }
  }
}

template <int kThreads, int kPer, bool kWide>
static cudaError_t launch_logits(const LogitsArgs& a, int num_sms, cudaStream_t st) {
  using SM = LogitsSmem<kThreads, kPer, kWide>;
  const int smem = SM::bytes(a.bias_start != nullptr);
  if (smem > 48 * 1024) {
    // the largest size, whatever this call's: another thread's call may be about to launch
    cudaError_t e = cudaFuncSetAttribute(process_logits_kernel<kThreads, kPer, kWide>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         SM::bytes(true));
    if (e != cudaSuccess) return e;
  }
  // As many rows a CTA as leave four CTAs an SM, but with marks no more than a
  // request's, and if possible a whole fraction of them: rows of another request
  // have to wait for marks of their own (64 requests of one row and 1500 tokens:
  // 27 us with one row a CTA, 33 with three; 8 trees of 16 and 1500 tokens: 35
  // with four, 41 with six).  A request's rows are taken to be S / n_reqs: requests
  // without rows make that too few, and marks are made again for every row (the
  // trees above among 512 requests: 111 us instead of 46).
  const int slices = (a.vocab + SM::kSlice - 1) / SM::kSlice;
  const int64_t parts = (int64_t)a.S * slices;
  int rows = (int)std::max<int64_t>(1, std::min<int64_t>(kLogRows, parts / (4 * num_sms)));
  if (a.history || a.draft_tokens || a.bias_start) {
    const int own = std::max(1, a.S / a.n_reqs);
    rows = std::min(rows, own);
    for (int d = rows; 2 * d > rows; --d)
      if (own % d == 0) {
        rows = d;
        break;
      }
  }
  const int64_t ctas = (int64_t)((a.S + rows - 1) / rows) * slices;
  return launch_k(process_logits_kernel<kThreads, kPer, kWide>, dim3((unsigned)ctas), dim3(kThreads),
                  smem, st, a, slices, make_fastdiv((uint32_t)slices), rows);
}

cudaError_t launch_process_logits(const LogitsArgs& a, int num_sms, cudaStream_t st) {
  const bool wide = a.history && a.ld_history + kMaxTreeTokens > kNarrowText;
  if ((int64_t)a.S * ((a.vocab + 4095) / 4096) < num_sms)
    return wide ? launch_logits<128, 16, true>(a, num_sms, st)
                : launch_logits<128, 16, false>(a, num_sms, st);
  if (!a.history || a.ld_history < 2048) return launch_logits<256, 16, false>(a, num_sms, st);
  return wide ? launch_logits<256, 32, true>(a, num_sms, st)
              : launch_logits<256, 32, false>(a, num_sms, st);
}

}  // namespace tpk
