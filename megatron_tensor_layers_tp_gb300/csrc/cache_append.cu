// RoPE on q and k and the new K/V rows into their cache slots, after the
// column-parallel qkv projection.
//
// Pair (j, j + d/2) of a head turns by position * theta^(-2j/d); cos and sin
// come from the model's table (fp32, from double).  Each element is read once
// and written once: memory-bound.  One CTA per token; a thread owns one
// 8-element chunk of a head's first half and the chunk d/2 further on (16-byte
// loads and stores, both members of eight pairs in one thread), keeps the
// eight rotation factors of its chunk in registers and walks over the heads,
// two at a time.  V heads are the same two chunks, copied.  The rows' loads do
// not depend on the token's position and slot and are issued first; the CTA has
// as many threads, up to 256 or 128, as deal the heads out evenly.
//
// While the rows fit the GPU at once, 256 threads take a row fastest (8 rows of
// 32 + 16 heads of 128: 1.9 us, 2.3 with 128); beyond that smaller CTAs, more of
// them on an SM and out of step with one another, keep the memory busier: 8191
// rows of 40 + 8 heads of 128 (200 MB): 33.4 us, 6.0 TB/s, with 128 threads, 38.1
// with 256 (64: the same); of 32 + 16 heads of 64: 18.9 and 25.8.  Measured
// before: 60 us with a CTA walking over tokens, the next row's loads ahead of
// this one's stores; 40-74 us with fewer registers and more threads an SM.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.h"
#include "ptx.cuh"

namespace tpk {


__device__ __forceinline__ void rotate8(uint4& lo, uint4& hi, const float2 (&cs)[8]) {
  uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a0 = __uint_as_float(a[i] << 16), a1 = __uint_as_float(a[i] & 0xFFFF0000u);
    const float b0 = __uint_as_float(b[i] << 16), b1 = __uint_as_float(b[i] & 0xFFFF0000u);
    const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
    a[i] = pack_bf16x2(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
    b[i] = pack_bf16x2(b0 * c0.x + a0 * c0.y, b1 * c1.x + a1 * c1.y);
  }
  lo = make_uint4(a[0], a[1], a[2], a[3]);
  hi = make_uint4(b[0], b[1], b[2], b[3]);
}

template <int kThreads>  // at most
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const CacheAppendArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int token = blockIdx.x, d = a.head_dim, half = d / 2;
  const int chunks = d / 16;
  const int c = threadIdx.x % chunks, h0 = threadIdx.x / chunks, hstep = blockDim.x / chunks;
  const int hq = a.q ? a.n_heads : 0, heads = hq + 2 * a.n_kv;
  const uint16_t* row = a.qkv + (int64_t)token * a.n_r + 8 * c;
  // head h of the list: the Q heads, then the K heads, then the V heads
  auto source = [&](int h) {
    if (h < hq) {
      const int r = (int)fast_div((uint32_t)h, a.div_q);
      return row + r * a.rank_stride + (h - r * a.q_per_rank) * d;
    }
    const bool is_v = h - hq >= a.n_kv;
    const int g = is_v ? h - hq - a.n_kv : h - hq;
    const int copy = (int)fast_div((uint32_t)g, a.div_kv), local = g - copy * a.kv_r;
    return row + (int64_t)copy * a.kv_replicas * a.rank_stride +
           (a.q_per_rank + (is_v ? a.kv_r : 0) + local) * d;
  };
  uint4 lo[2], hi[2];
  auto fetch = [&](int h) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int hh = h + y * hstep;
      if (hh < heads) {
        const uint16_t* src = source(hh);
        lo[y] = *reinterpret_cast<const uint4*>(src);
        hi[y] = *reinterpret_cast<const uint4*>(src + half);
      }
    }
  };
  fetch(h0);

  const int pos = a.positions[token];
  int slot = a.slots[token];
  const bool pos_ok = pos >= 0 && pos < a.max_positions;
  const bool slot_ok = slot >= -1 && slot < a.n_pages * a.page_size;
  if ((!pos_ok || !slot_ok) && threadIdx.x == 0) record_status(a.status, kStatusTableRange);
  if (!pos_ok || !slot_ok) slot = -1;
  float2 cs[8];
  const float4* rp = reinterpret_cast<const float4*>(a.rope + (int64_t)(pos_ok ? pos : 0) * half + 8 * c);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = rp[i];
    cs[2 * i] = make_float2(f.x, f.y);
    cs[2 * i + 1] = make_float2(f.z, f.w);
  }
  const int page = slot < 0 ? 0 : (int)fast_div((uint32_t)slot, a.div_page);
  const int off = slot - page * a.page_size;

  for (int h = h0; h < heads; h += 2 * hstep) {
    if (h != h0) fetch(h);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int hh = h + y * hstep;
      if (hh >= heads) break;
      uint16_t* dst;
      if (hh < hq) {
        if (pos_ok) rotate8(lo[y], hi[y], cs);
        else lo[y] = hi[y] = make_uint4(0, 0, 0, 0);
        dst = a.q + token * a.ld_q + hh * d + 8 * c;
      } else {
        if (slot < 0) break;
        const bool is_v = hh - hq >= a.n_kv;
        const int g = is_v ? hh - hq - a.n_kv : hh - hq;
        const int copy = (int)fast_div((uint32_t)g, a.div_kv), local = g - copy * a.kv_r;
        if (!is_v) rotate8(lo[y], hi[y], cs);
        dst = (is_v ? a.v : a.k) +
              ((((int64_t)copy * a.n_pages + page) * a.kv_r + local) * a.page_size + off) * d + 8 * c;
      }
      *reinterpret_cast<uint4*>(dst) = lo[y];
      *reinterpret_cast<uint4*>(dst + half) = hi[y];
    }
  }
}

template <int kThreads>
static cudaError_t launch_append(const CacheAppendArgs& a, cudaStream_t st) {
  const int chunks = a.head_dim / 16, heads = (a.q ? a.n_heads : 0) + 2 * a.n_kv;
  const int turns = (heads * chunks + kThreads - 1) / kThreads;
  const int lanes = (heads + turns - 1) / turns;  // heads at a time
  return launch_k(cache_append_kernel<kThreads>, dim3(a.M), dim3(lanes * chunks), 0, st, a);
}

cudaError_t launch_cache_append(const CacheAppendArgs& a, int num_sms, cudaStream_t st) {
  return a.M > 4 * num_sms ? launch_append<128>(a, st) : launch_append<256>(a, st);
}

}  // namespace tpk
