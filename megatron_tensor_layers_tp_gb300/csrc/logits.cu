// Penalties, biases and grammar masks on logits.
//
// x = logit; seen tokens: x > 0 ? x / repetition : x * repetition;
// x -= frequency * count; x -= presence * [count > 0]; x += bias; tokens not
// allowed: -infinity.  Counts come from the request's text and the drafted
// tokens on the row's path.
//
// Memory-bound: 2 bytes in, 2 or 4 out and a mask bit a token.  A row's
// vocabulary is cut into slices, one CTA each, 16 tokens a thread.  A thread
// first puts its logits and mask bits in flight; meanwhile the CTA reads the
// request's text and marks what it touches of the slice in shared memory
// (integer atomics: their order does not matter): 16 bits a token, or 32 where
// a text is long enough to overflow them.  Almost all marks are zero, so the
// rules cost one 16-byte shared load for eight tokens.  The biases sit in a
// slice-sized array that is neither cleared nor read except where a mark says
// so.
//
// Slices of 8192 tokens (512 threads, four CTAs an SM) keep the repeated
// reading of the text small; with too few rows to fill the GPU that way,
// slices of 2048 (128 threads): one row of 128256 logits @@ us instead of @@.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "paged.h"
#include "ptx.cuh"

namespace tpk {

constexpr int kLogPer = 16;  // tokens of a thread

// Marks of a token: bit 0 = in the prompt, bit 1 = has a bias, the rest = times
// written by the model.
constexpr uint32_t kMarkPrompt = 1, kMarkBias = 2, kMarkWritten = 4;
// the longest text (and path) whose counts fit 16-bit marks
constexpr int64_t kNarrowText = (1 << 14) - 1;

template <bool kWide>
struct Marks {
  uint32_t* w;
  __device__ __forceinline__ void add(int v, uint32_t x) {
    if constexpr (kWide) atomicAdd(w + v, x);
    else atomicAdd(w + (v >> 1), x << (16 * (v & 1)));
  }
  __device__ __forceinline__ void set(int v, uint32_t x) {
    if constexpr (kWide) atomicOr(w + v, x);
    else atomicOr(w + (v >> 1), x << (16 * (v & 1)));
  }
  __device__ __forceinline__ uint32_t get(int v) const {
    if constexpr (kWide) return w[v];
    else return (w[v >> 1] >> (16 * (v & 1))) & 0xFFFF;
  }
  // any mark among tokens v .. v + 7 (v a multiple of 8)
  __device__ __forceinline__ bool any8(int v) const {
    const uint4* p = reinterpret_cast<const uint4*>(w + (kWide ? v : v >> 1));
    uint4 a = p[0];
    if constexpr (kWide) {
      const uint4 b = p[1];
      a.x |= b.x; a.y |= b.y; a.z |= b.z; a.w |= b.w;
    }
    return (a.x | a.y | a.z | a.w) != 0;
  }
};

// One request's numbers for the rules on a single logit.
struct Rules {
  float rep, freq, pres;
};
__device__ __forceinline__ float apply_rules(float x, uint32_t mark, const float* bias,
                                             const Rules& r) {
  const uint32_t n = mark / kMarkWritten;
  if (n || (mark & kMarkPrompt)) x = x > 0.f ? x / r.rep : x * r.rep;
  if (n) x = x - r.freq * (float)n - r.pres;
  if (mark & kMarkBias) x += *bias;
  return x;
}

template <int kThreads, bool kWide>
__global__ void __launch_bounds__(kThreads) process_logits_kernel(const LogitsArgs a, int slices) {
  constexpr int kSlice = kThreads * kLogPer;
  extern __shared__ __align__(16) uint32_t sm[];
  Marks<kWide> marks{sm};
  float* bias = reinterpret_cast<float*>(sm + (kWide ? kSlice : kSlice / 2));  // with a.bias_start
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x / slices, slice = blockIdx.x - row * slices;
  const int v0 = slice * kSlice, n = min(kSlice, a.vocab - v0);
  const int tid = threadIdx.x;
  const uint16_t* in = a.logits + row * a.ld + v0;
  uint8_t* out = static_cast<uint8_t*>(a.out) + (row * a.ld_out + v0) * (a.out_fp32 ? 4 : 2);

  // The thread's tokens: two runs of 8 where the rows allow 16-byte accesses,
  // else 16 single ones a CTA's width apart.
  const bool vec = ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  uint4 x[2];
  uint32_t ok = 0xFFFFFFFFu;  // bit i: token i of the thread is allowed
  const int m = a.allowed ? (a.allowed_row ? a.allowed_row[row] : row) : -1;
  const uint8_t* mask = m >= 0 && m < a.n_allowed
                            ? reinterpret_cast<const uint8_t*>(a.allowed + m * a.ld_allowed) + v0 / 8
                            : nullptr;
  const bool bad_mask = a.allowed && (m < -1 || m >= a.n_allowed);
  if (bad_mask) ok = 0;
  if (vec) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = (j * kThreads + tid) * 8;
      if (i + 8 <= n) {
        x[j] = *reinterpret_cast<const uint4*>(in + i);
      } else {
        uint16_t e[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) e[q] = i + q < n ? in[i + q] : 0;
        x[j] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
      }
      if (mask && i < n) ok &= ~(0xFFu << (8 * j)) | (uint32_t)mask[i / 8] << (8 * j);
    }
  } else {
    uint16_t e[kLogPer];
#pragma unroll
    for (int j = 0; j < kLogPer; ++j) {
      const int i = j * kThreads + tid;
      e[j] = i < n ? in[i] : 0;
      if (mask && i < n && !(mask[i >> 3] >> (i & 7) & 1)) ok &= ~(1u << j);
    }
    x[0] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
    x[1] = make_uint4(e[8] | e[9] << 16, e[10] | e[11] << 16, e[12] | e[13] << 16, e[14] | e[15] << 16);
  }

  const int r = a.row_req ? a.row_req[row] : row;
  if (r < 0 || r >= a.n_reqs) {
    if (r != -1 && tid == 0) record_status(a.status, kStatusTableRange);
    return;
  }
  if (bad_mask && tid == 0) record_status(a.status, kStatusTableRange);
  const Rules ru = {a.repetition ? a.repetition[r] : 1.f, a.frequency ? a.frequency[r] : 0.f,
                    a.presence ? a.presence[r] : 0.f};
  const bool marked = a.history || a.draft_tokens || a.bias_start;
  if (marked) {
    for (int i = tid; i < (kWide ? kSlice : kSlice / 2) / 4; i += kThreads)
      reinterpret_cast<uint4*>(sm)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  if (a.history) {
    const int len = a.history_lens[r], pl = a.prompt_lens ? a.prompt_lens[r] : 0;
    const int len_c = (int)min((int64_t)max(len, 0), a.ld_history), pl_c = min(max(pl, 0), len_c);
    if ((len != len_c || pl != pl_c) && tid == 0) record_status(a.status, kStatusTableRange);
    const int32_t* h = a.history + r * a.ld_history;
#pragma unroll 4
    for (int i = tid; i < len_c; i += kThreads) {
      const uint32_t v = (uint32_t)h[i] - (uint32_t)v0;  // (a foreign id becomes a large one)
      if (v < (uint32_t)n) {
        if (i < pl_c) marks.set(v, kMarkPrompt);
        else marks.add(v, kMarkWritten);
      }
    }
  }
  if (a.draft_tokens) {
    const int q0 = a.q_start[r];
    const int64_t T = (int64_t)a.q_start[r + 1] - q0;
    if (q0 < 0 || T < 0 || q0 + T > a.S) {
      if (tid == 0) record_status(a.status, kStatusTableRange);
    } else {
      for (int t = tid; t < min((int)T, 64 * a.tree_words); t += kThreads)
        if ((a.tree_mask[(int64_t)row * a.tree_words + (t >> 6)] >> (t & 63)) & 1) {
          const uint32_t v = (uint32_t)a.draft_tokens[q0 + t] - (uint32_t)v0;
          if (v < (uint32_t)n) marks.add(v, kMarkWritten);
        }
    }
  }
  if (a.bias_start) {
    const int b0 = a.bias_start[r];
    int b1 = a.bias_start[r + 1];
    if (b0 < 0 || b1 < b0 || b1 > a.n_biases) {
      if (tid == 0) record_status(a.status, kStatusTableRange);
      b1 = b0;
    }
    // Entries of tokens named once need no order.  How often a token is named
    // is counted in its place in the bias array.
    int* named = reinterpret_cast<int*>(bias);
    bool any = false;
    for (int i = b0 + tid; i < b1; i += kThreads) {
      const uint32_t v = (uint32_t)a.bias_ids[i] - (uint32_t)v0;
      if (v < (uint32_t)n) {
        named[v] = 0;
        any = true;
      }
    }
    if (__syncthreads_or(any)) {
      for (int i = b0 + tid; i < b1; i += kThreads) {
        const uint32_t v = (uint32_t)a.bias_ids[i] - (uint32_t)v0;
        if (v < (uint32_t)n) {
          atomicAdd(named + v, 1);
          marks.set(v, kMarkBias);
        }
      }
      __syncthreads();
      bool again = false;
      for (int i = b0 + tid; i < b1; i += kThreads) {
        const uint32_t v = (uint32_t)a.bias_ids[i] - (uint32_t)v0;
        if (v < (uint32_t)n) {
          if (named[v] == 1) bias[v] = a.bias_values[i];  // no other entry looks at it
          else again = true;
        }
      }
      if (__syncthreads_or(again)) {
        // Some token is named more than once: the list anew, in order, by one
        // warp, entries of the same token among its 32 added in order too.
        for (int i = b0 + tid; i < b1; i += kThreads) {
          const uint32_t v = (uint32_t)a.bias_ids[i] - (uint32_t)v0;
          if (v < (uint32_t)n) bias[v] = 0.f;
        }
        __syncthreads();
        if (tid < 32) {
          for (int base = b0; base < b1; base += 32) {
            const int i = base + tid;
            const uint32_t v = i < b1 ? (uint32_t)a.bias_ids[i] - (uint32_t)v0 : 0xFFFFFFFFu;
            const bool here = v < (uint32_t)n;
            const float y = here ? a.bias_values[i] : 0.f;
            const unsigned same = __match_any_sync(0xffffffffu, here ? (int)v : -1 - tid);
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
  if (marked) __syncthreads();

  if (vec) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = (j * kThreads + tid) * 8;
      if (i >= n) break;
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      float f[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        f[q] = __uint_as_float(q & 1 ? w[q >> 1] & 0xFFFF0000u : w[q >> 1] << 16);
      if (marked && marks.any8(i)) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t mk = marks.get(i + q);
          if (mk) f[q] = apply_rules(f[q], mk, bias + i + q, ru);
        }
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = ok >> (8 * j + q) & 1 ? f[q] : -INFINITY;
      if (i + 8 <= n) {
        if (a.out_fp32) {
          float4* o = reinterpret_cast<float4*>(out) + i / 4;
          o[0] = make_float4(f[0], f[1], f[2], f[3]);
          o[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
          reinterpret_cast<uint4*>(out)[i / 8] =
              make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                         pack_bf16x2(f[6], f[7]));
        }
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (i + q < n) {
            if (a.out_fp32) reinterpret_cast<float*>(out)[i + q] = f[q];
            else reinterpret_cast<uint16_t*>(out)[i + q] = f_to_bf16(f[q]);
          }
      }
    }
  } else {
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
    for (int j = 0; j < kLogPer; ++j) {
      const int i = j * kThreads + tid;
      if (i >= n) break;
      float f = __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
      const uint32_t mk = marked ? marks.get(i) : 0;
      if (mk) f = apply_rules(f, mk, bias + i, ru);
      if (!(ok >> j & 1)) f = -INFINITY;
      if (a.out_fp32) reinterpret_cast<float*>(out)[i] = f;
      else reinterpret_cast<uint16_t*>(out)[i] = f_to_bf16(f);
    }
  }
}

template <int kThreads, bool kWide>
static cudaError_t launch_logits(const LogitsArgs& a, cudaStream_t st) {
  constexpr int kSlice = kThreads * kLogPer;
  const int smem = kSlice * (kWide ? 4 : 2) + (a.bias_start ? kSlice * 4 : 0);
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(process_logits_kernel<kThreads, kWide>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  const int slices = (a.vocab + kSlice - 1) / kSlice;
  return launch_k(process_logits_kernel<kThreads, kWide>, dim3((unsigned)((int64_t)a.S * slices)),
                  dim3(kThreads), smem, st, a, slices);
}

cudaError_t launch_process_logits(const LogitsArgs& a, int num_sms, cudaStream_t st) {
  const bool wide = a.history && a.ld_history + kMaxTreeTokens > kNarrowText;
  if ((int64_t)a.S * ((a.vocab + 8191) / 8192) >= num_sms)
    return wide ? launch_logits<512, true>(a, st) : launch_logits<512, false>(a, st);
  return wide ? launch_logits<128, true>(a, st) : launch_logits<128, false>(a, st);
}

}  // namespace tpk
