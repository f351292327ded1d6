// Attention of a step's new tokens over the paged KV cache.
//
// Row (token i of sequence b, Q head h) sees the old tokens 0..old-1 and the
// new tokens t of its sequence whose bit is set in its tree mask (chains:
// t <= i).  o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m) with s_j = q.k_j /
// sqrt(d) and the running maximum m, in one pass over the keys.
//
// One warp per row: the lanes share the head's elements, a key's score is a
// warp sum.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "paged.h"
#include "ptx.cuh"

namespace tpk {

// Sequence b's first row, new tokens and old length; an inconsistent one has
// no tokens (and sets the status).
struct SeqInfo {
  int q0, T, old;
};
__device__ __forceinline__ SeqInfo seq_info(const TreeAttnArgs& a, int b) {
  SeqInfo s;
  s.q0 = a.q_start[b];
  const int q1 = a.q_start[b + 1];
  s.old = a.old_lens[b];
  s.T = q1 - s.q0;
  if (s.q0 < 0 || q1 < s.q0 || q1 > a.n_tokens || s.T > a.max_new || s.old < 0 ||
      (int64_t)s.old + s.T > a.cap) {
    record_status(a.status, kStatusTableRange);
    s.T = 0;
  }
  return s;
}

template <int D>
__global__ void __launch_bounds__(256) tree_attn_kernel(const TreeAttnArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int E = D / 32;  // elements of a lane
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int row = (int)(w / a.n_heads), h = (int)(w % a.n_heads);
  if (row >= a.n_tokens) return;
  int b = -1;
  SeqInfo s = {0, 0, 0};
  for (int i = 0; i < a.n_seqs && b < 0; ++i) {
    s = seq_info(a, i);
    if (row >= s.q0 && row < s.q0 + s.T) b = i;
  }
  if (b < 0) return;
  const int i = row - s.q0, g = h / a.group, copy = g / a.kv_r, local = g % a.kv_r;
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = bf16_to_f(a.q[row * a.ld_q + h * D + lane * E + e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < s.old + s.T; ++j) {
    const int t = j - s.old;
    if (t >= 0) {
      const bool sees = a.tree_mask
                            ? (a.tree_mask[(int64_t)row * a.tree_words + (t >> 6)] >> (t & 63)) & 1
                            : t <= i;
      if (!sees) continue;
    }
    const int pg = (int)fast_div((uint32_t)j, a.div_page);
    const int page = a.table[(int64_t)b * a.ld_table + pg];
    const bool ok = page >= 0 && page < a.n_pages;
    if (!ok) record_status(a.status, kStatusTableRange);
    const int64_t at =
        ((((int64_t)copy * a.n_pages + (ok ? page : 0)) * a.kv_r + local) * a.page_size + j -
         pg * a.page_size) * D + lane * E;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x += ok ? q[e] * bf16_to_f(a.k[at + e]) : 0.f;
#pragma unroll
    for (int f = 16; f; f >>= 1) x += __shfl_xor_sync(0xffffffffu, x, f);
    x *= a.scale_log2;
    const float mn = fmaxf(m, x);
    const float al = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(x - mn);
    m = mn;
    l = l * al + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * al + (ok ? p * bf16_to_f(a.v[at + e]) : 0.f);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) a.o[row * a.ld_o + h * D + lane * E + e] = f_to_bf16(o[e] * inv);
}

cudaError_t launch_tree_attn(const TreeAttnArgs& a, cudaStream_t st) {
  const int64_t warps = (int64_t)a.n_tokens * a.n_heads;
  const dim3 grid((unsigned)((warps + 7) / 8));
  return a.head_dim == 128 ? launch_k(tree_attn_kernel<128>, grid, dim3(256), 0, st, a)
                           : launch_k(tree_attn_kernel<64>, grid, dim3(256), 0, st, a);
}

}  // namespace tpk
