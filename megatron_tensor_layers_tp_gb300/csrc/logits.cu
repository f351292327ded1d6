// Penalties, biases and grammar masks on logits.
//
// x = logit; seen tokens: x > 0 ? x / repetition : x * repetition;
// x -= frequency * count; x -= presence * [count > 0]; x += bias; tokens not
// allowed: -infinity.  Counts come from the request's text and the drafted
// tokens on the row's path.
//
// A row's vocabulary is cut into slices of 8192 tokens, one CTA each.  The
// CTA counts its slice's tokens in shared memory (integer atomics: the order
// does not matter), adds up the biases there, then streams the logits once:
// memory-bound, 2 bytes in and 2 or 4 out a token.  The history is read once
// a slice, from L2 after the first.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "paged.h"
#include "ptx.cuh"

namespace tpk {

constexpr int kLogThreads = 512;
constexpr int kLogSlice = 8192;

// One request's numbers for the rules on a single logit.
struct Rules {
  float rep, freq, pres;
};

// cnt: bit 0 = seen in the prompt, the rest = times written by the model
__device__ __forceinline__ float apply_rules(float x, uint32_t cnt, float bias, const Rules& r) {
  if (cnt) {
    x = x > 0.f ? x / r.rep : x * r.rep;
    const uint32_t n = cnt >> 1;
    if (n) x = x - r.freq * (float)n - r.pres;
  }
  return x + bias;
}

__global__ void __launch_bounds__(kLogThreads) process_logits_kernel(const LogitsArgs a, int slices) {
  extern __shared__ uint32_t sm[];
  uint32_t* cnt = sm;                                            // [kLogSlice]
  float* bias = reinterpret_cast<float*>(sm + kLogSlice);        // [kLogSlice]
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x / slices, slice = blockIdx.x - row * slices;
  const int v0 = slice * kLogSlice, n = min(kLogSlice, a.vocab - v0);
  const int tid = threadIdx.x;
  const int r = a.row_req ? a.row_req[row] : row;
  if (r < 0 || r >= a.n_reqs) {
    if (r != -1 && tid == 0) record_status(a.status, kStatusTableRange);
    return;
  }
  for (int i = tid; i < kLogSlice; i += kLogThreads) {
    cnt[i] = 0;
    bias[i] = 0.f;
  }
  __syncthreads();
  if (a.history) {
    const int len = a.history_lens[r], pl = a.prompt_lens ? a.prompt_lens[r] : 0;
    const int len_c = (int)min((int64_t)max(len, 0), a.ld_history), pl_c = min(max(pl, 0), len_c);
    if ((len != len_c || pl != pl_c) && tid == 0) record_status(a.status, kStatusTableRange);
    const int32_t* h = a.history + r * a.ld_history;
    for (int i = tid; i < len_c; i += kLogThreads) {
      const int64_t v = (int64_t)h[i] - v0;
      if (v < 0 || v >= n) continue;
      if (i < pl_c) atomicOr(&cnt[v], 1u);
      else atomicAdd(&cnt[v], 2u);
    }
  }
  if (a.draft_tokens) {
    const int q0 = a.q_start[r];
    const int64_t T = (int64_t)a.q_start[r + 1] - q0;
    if (q0 < 0 || T < 0 || q0 + T > a.S) {
      if (tid == 0) record_status(a.status, kStatusTableRange);
    } else {
      for (int t = tid; t < min((int)T, 64 * a.tree_words); t += kLogThreads)
        if ((a.tree_mask[(int64_t)row * a.tree_words + (t >> 6)] >> (t & 63)) & 1) {
          const int64_t v = (int64_t)a.draft_tokens[q0 + t] - v0;
          if (v >= 0 && v < n) atomicAdd(&cnt[v], 2u);
        }
    }
  }
  if (a.bias_start && tid < 32) {
    // one warp, 32 entries at a time in list order; entries of the same token
    // are added in that order too
    const int b0 = a.bias_start[r], b1 = a.bias_start[r + 1];
    if (b0 < 0 || b1 < b0 || b1 > a.n_biases) {
      if (tid == 0) record_status(a.status, kStatusTableRange);
    } else {
      for (int base = b0; base < b1; base += 32) {
        const int i = base + tid;
        const int64_t v = i < b1 ? (int64_t)a.bias_ids[i] - v0 : -1;
        const bool in = v >= 0 && v < n;
        const float x = in ? a.bias_values[i] : 0.f;
        const unsigned same = __match_any_sync(0xffffffffu, in ? (int)v : -1 - tid);
        const bool lead = in && (same & ((1u << tid) - 1)) == 0;
        float s = lead ? bias[v] : 0.f;
        for (int j = 0; j < 32; ++j) {
          const float y = __shfl_sync(0xffffffffu, x, j);
          if (same >> j & 1) s += y;
        }
        if (lead) bias[v] = s;
        __syncwarp();
      }
    }
  }
  __syncthreads();
  const Rules ru = {a.repetition ? a.repetition[r] : 1.f, a.frequency ? a.frequency[r] : 0.f,
                    a.presence ? a.presence[r] : 0.f};
  const uint32_t* ok = nullptr;
  bool none = false;
  if (a.allowed) {
    const int m = a.allowed_row ? a.allowed_row[row] : row;
    if (m >= 0 && m < a.n_allowed) ok = a.allowed + m * a.ld_allowed + v0 / 32;
    else if (m != -1) {
      none = true;
      if (tid == 0) record_status(a.status, kStatusTableRange);
    }
  }
  const uint16_t* in = a.logits + row * a.ld + v0;
  for (int i = tid; i < n; i += kLogThreads) {
    float x = apply_rules(bf16_to_f(in[i]), cnt[i], bias[i], ru);
    if (none || (ok && !(ok[i >> 5] >> (i & 31) & 1))) x = -INFINITY;
    if (a.out_fp32) static_cast<float*>(a.out)[row * a.ld_out + v0 + i] = x;
    else static_cast<uint16_t*>(a.out)[row * a.ld_out + v0 + i] = f_to_bf16(x);
  }
}

cudaError_t launch_process_logits(const LogitsArgs& a, cudaStream_t st) {
  const int smem = kLogSlice * 8;
  cudaError_t e = cudaFuncSetAttribute(process_logits_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int slices = (a.vocab + kLogSlice - 1) / kLogSlice;
  return launch_k(process_logits_kernel, dim3((unsigned)((int64_t)a.S * slices)), dim3(kLogThreads),
                  smem, st, a, slices);
}

}  // namespace tpk
