// Attention of a step's new tokens over the paged KV cache, on the tensor
// cores (tcgen05).
//
// Row (token i of sequence b, Q head h) sees the old tokens 0..old-1 and the
// new tokens t of its sequence whose bit is set in its tree mask (chains:
// t <= i).  o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m) with s_j = q.k_j /
// sqrt(d) and the running maximum m, in one pass over the keys.
//
// Every Q head of a KV head and every new token of a sequence share its keys:
// they are the rows of query tiles (row = token * group + head, whole tokens,
// up to 128 rows), so K and V are read once for up to 128 / group tokens.  With
// one tile per sequence and KV head the cache's bytes bound the kernel: a
// 64-key tile of K and V (32 KB at d = 128) takes an SM 0.73 us at its share of
// the memory rate, its two products 0.14 us and its exponentials 0.2 us.  With
// many tiles (chunks) the round trip of a tile does: scores -> probabilities ->
// P V -> the buffer's next scores, 0.4-0.5 us a tile over all buffers.  Short
// calls are bound by what a part of an item costs besides its tiles (4-5 us:
// the first copies, the groups' meeting, the pieces) and by the join (1.5-3 us).
//
// Measured: one token behind 700 old ones, 32 heads of 128 over 8 KV heads:
// 14 us; 16 trees of 8-32 tokens behind 150-2048, 40 heads over 8 (80 MB): 36 us;
// 64 trees of 2-8 tokens behind 1500-4096, 32 heads over 8 (740 MB): 120 us,
// 6.1 TB/s; 6 chunks of 100-256 tokens behind up to 8000, 32 heads of 64 over 4
// (64 GFLOP in whole tiles): 93 us, 690 TFLOP/s.
//
// Work is the flat sequence of (sequence, KV head, query tile, key tile), an
// item's fixed work counted as kItemCost tiles more, split evenly over one CTA
// per SM.  A CTA finds its range from the lengths on the GPU, so a captured
// launch follows them.  An item cut between CTAs leaves unnormalised fp32
// pieces, and the last CTA to finish one (a ticket, no waiting) joins them in
// key order: deterministic.  Where all others are there before it begins to write
// its own, it keeps that in registers (the chunks 93 us instead of 96), by the same
// operations in the same order.  The pieces lie [4 elements][row], so that lane =
// row reads and writes whole lines with every load in flight (a second kernel
// for the join cost 3-5 us a call; the join with rows of pieces and loads one
// after another, 50; joined rows straight into o instead of through shared
// memory, 3).
//
// Roles of the 20 warps:
//   warps 0-3  : K and V tiles by TMA into rings, through the page table, each
//                every other tile of a group: boxes end where pages end, a box
//                costs its warp about 130 cycles to issue (32 boxes a tile at
//                8-key pages) and a tile some 1500 in waits and look-ups;
//   warps 4, 5 : one thread each issues S = Q K^T of a softmax group into tensor
//                memory;
//   warps 6, 7 : one thread each issues O += P V of a group, with P read from
//                tensor memory and V as it lies in the page (the head's elements
//                contiguous).  Issuing costs about 65 cycles a product, 80 a
//                commit and 100-150 a wait: one thread for all products set the
//                pace (1850-2000 cycles a tile, nothing else busy), and so did
//                one for both groups' S (1300; the chunks above 134 us instead of 109);
//   warp 8     : the CTA's parts of items, announced to the other warps two
//                ahead, and the next item's query tile while this one's softmax
//                ends.  (Every role finding the parts by itself spilled
//                registers into the issuing loops: twice the time.);
//   warps 12-15, 16-19: two softmax groups.  They take alternate key tiles, each
//                with its own running maximum, sum and O, so that neither
//                waits for the other's maxima; the two states meet at the
//                item's end.  A thread owns a row and holds a tile's 64 scores
//                in registers.
// Each group has two S buffers, three where tensor memory holds them (heads of
// 64): the products of its next tiles run while it works on this one.  (Two
// instead of three: 113 us for 8000-key chunks, not 110.  Measured before each
// group's scores had an issuing thread of their own, when the chunks took 134:
// one buffer and 128-key tiles 172; two warpgroups a group, each with half of a
// tile's keys, 159.)
// P overwrites S in place, rounded to bf16: the product with V takes both of its
// operands in one 16-bit type, and V is bf16.  That moves o by at most 2^-8 of
// sum p |v|; measured, the error against 64 bits is 0.0023 of the output's norm
// instead of 0.0017 with the output's own rounding alone.  The sums take p
// before its rounding, in fp32.  O is rescaled only when a
// row's maximum rose by more than 2^8 since its last rescaling: the sums are
// relative to the older maximum until then, which is exact algebra and keeps
// every p below 2^8.
//
// What rows do not see must not reach them: masked scores become -inf by a
// select, and in tiles that hold new tokens (or the end) the softmax group
// clears V rows behind the end, and takes infinities and NaN out of the new
// tokens' V (0 * inf would spread them to rows that do not see the token); the
// rows that do see such an element get it added at the end (nonfinite_v).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "paged.h"
#include "ptx.cuh"

namespace tpk {

constexpr int kTreeThreads = 640;
constexpr int kTreeSoftmax = 256;        // threads of the two softmax groups, the last ones
constexpr int kTreeFirst = kTreeThreads - kTreeSoftmax;
// registers of a thread after the hand-over: together no more than the launch
// brought (checked by the host, since a take-over beyond it would never end)
constexpr int kTreeRegsOther = 64, kTreeRegsSoftmax = 144;
constexpr float kRescaleLog2 = 8.f;
// An item's fixed work in key tiles.  With 8, 12, 16, 24: the chunks above 95.8,
// 93.6, 93.4, 95.1 us, with heads of 128 (24-key pages) 144.6, 145.1, 146.3, 148.5;
// 64 long sequences 119.7, 120.5, 122.0, 125.1; one token behind 700 14.5, 14.2,
// 13.6, 13.3; 32 single tokens behind 1000 38.3, 36.9, 36.2, 35.6.
constexpr int kItemCost = 12;
constexpr int kMaxGrid = 1024;
// Up to so many rows of an item its pieces are joined in finer cuts (16, 32, 48, 64
// rows of one sequence behind 4000 tokens: 16.6, 17.4, 21.7, 21.9 us so, 17.7,
// 19.1, 20.4, 20.6 in wider ones; of 16 sequences behind 1100: 25.9, 26.3, 27.5,
// 27.6 and 26.8, 26.9, 27.2, 26.9; heads of 128).
constexpr int kFewRows = 32;

// One CTA's part of an item: key tiles [k0, k1) of nt of (sequence b, KV head
// g, query tile qi), the sequence's first row, new tokens and old length; of an
// item cut between CTAs, the first and last CTA that have a part, and where in
// its two piece slots the first has it.  k1 = 0: no more parts.
struct Seg {
  int b, g, qi, k0, k1, nt, q0, T, old, first, last, slot;
};

template <int D>
struct TreeSmem {
  static constexpr int kTile = kTreeKeys * D * 2;    // a K or V tile
  static constexpr int kDepth = D == 128 ? 2 : 5;     // tiles of each of the four rings
  // S buffers of a group: as many as tensor memory's 512 columns hold beside O
  static constexpr int kBufs = (512 / 2 - D) / kTreeKeys < 3 ? (512 / 2 - D) / kTreeKeys : 3;
  static_assert(kBufs <= kDepth, "a tile's scores imply that the fill before its V was consumed");
  static constexpr int kOut = kTreeRows * D * 2;      // after the query tile: rows of o on their way out
  static constexpr int kRing = 2 * kOut;
  static constexpr int kMeet = kRing + 4 * kDepth * kTile;  // (m, l) of the two groups
  static constexpr int kBars = kMeet + 2 * kTreeRows * 8;
  static constexpr int kTotal = kBars + 1024 + 1024;  // + alignment of the base
  static_assert(kTotal <= 227 * 1024, "shared memory of one CTA");
};
// after the ring
struct TreeCtl {
  uint64_t full[20], empty[20];
  uint64_t s_full[6], p_ready[6], pv_done[6], q_full, q_free, drain;  // [group][S buffer]
  uint64_t seg_full[4], seg_free[4];
  Seg seg[4];
  long long warp_sum[kTreeThreads / 32];
  long long total, u0, x0, x1;
  int b0;
  int poison[2];
  int last;
  uint32_t tmem;
};
static_assert(sizeof(TreeCtl) <= 1024, "control block");

// Sequence b's first row, new tokens, old length and tiles; an inconsistent
// one has no tokens (and sets the status).
struct SeqInfo {
  int q0, T, old, qt, nt;
};
__device__ __forceinline__ SeqInfo seq_info(const TreeAttnArgs& a, int b) {
  SeqInfo s;
  s.q0 = a.q_start[b];
  const int q1 = a.q_start[b + 1];
  s.old = a.old_lens[b];
  const int64_t T = (int64_t)q1 - s.q0;
  s.T = (int)T;
  if (s.q0 < 0 || T < 0 || q1 > a.n_tokens || T > a.max_new || s.old < 0 ||
      s.old + T > a.cap) {
    record_status(a.status, kStatusTableRange);
    s.T = 0;
  }
  s.qt = (s.T + a.tile_toks - 1) / a.tile_toks;
  s.nt = s.T ? (s.old + s.T + kTreeKeys - 1) / kTreeKeys : 0;
  return s;
}
// The flat positions of a sequence: every item's tiles after its fixed cost.
__device__ __forceinline__ int64_t positions(const TreeAttnArgs& a, const SeqInfo& s) {
  return (int64_t)a.n_kv * s.qt * (s.nt + kItemCost);
}

// range_begin without a 64-bit division where 32 bits hold the product.
__device__ __forceinline__ int64_t range_at(int c, int64_t T, int G) {
  if (T <= 0xFFFFFFFFll / kMaxGrid) return (uint32_t)c * (uint32_t)T / (uint32_t)G;
  return range_begin(c, T, G);
}

// A CTA's parts in order.  A part that lies within the item's fixed cost has
// no tiles and is passed over: the parts with tiles are those of consecutive
// CTAs.
struct SegIter {
  const TreeAttnArgs& a;
  int64_t x, x1, u;  // flat position, its end, position inside sequence b
  int b;
  SeqInfo s;
  __device__ __forceinline__ SegIter(const TreeAttnArgs& a_, int64_t x_, int64_t x1_, int64_t u_,
                                     int b_)
      : a(a_), x(x_), x1(x1_), u(u_), b(b_) {
    if (x < x1) s = seq_info(a, b);
  }
  __device__ __forceinline__ Seg next(int64_t W, int G) {
    while (x < x1) {
      while (u >= positions(a, s)) {  // at most to the last sequence: x < x1 <= W
        u -= positions(a, s);
        ++b;
        s = seq_info(a, b);
      }
      const int cost = s.nt + kItemCost;
      const int64_t item = u <= INT32_MAX ? (int64_t)((uint32_t)u / (uint32_t)cost) : u / cost;
      const int at = (int)(u - item * cost);
      const int64_t left = x1 - x;
      const int end = (int)(left < cost - at ? at + left : cost);
      const int64_t begin = x - at;
      x += end - at;
      u += end - at;
      if (end <= kItemCost) continue;
      Seg sg;
      sg.b = b;
      sg.g = (uint32_t)item / (uint32_t)s.qt;
      sg.qi = (int)item - sg.g * s.qt;
      sg.k0 = max(at - kItemCost, 0);
      sg.k1 = end - kItemCost;
      sg.nt = s.nt;
      sg.q0 = s.q0;
      sg.T = s.T;
      sg.old = s.old;
      if (sg.k1 - sg.k0 < s.nt) {
        sg.first = owner_of(begin + kItemCost, W, G);
        sg.last = owner_of(begin + cost - 1, W, G);
        sg.slot = range_at(sg.first, W, G) < begin ? 1 : 0;  // after the end of another item
      }
      return sg;
    }
    Seg none;
    none.k1 = 0;
    return none;
  }
};

// 32 bits: which of the keys key0 .. key0 + 31 row `row` (token i of its
// sequence) sees.
__device__ __forceinline__ uint32_t sees32(const TreeAttnArgs& a, const Seg& s, int i, int key0) {
  const int base = key0 - s.old;  // drafted token of bit 0
  if (base <= -32) return 0xFFFFFFFFu;
  uint32_t m = 0xFFFFFFFFu;
  int n = s.T - base;  // bits that exist
  if (a.tree_mask) {
    const uint32_t* w =
        reinterpret_cast<const uint32_t*>(a.tree_mask + (int64_t)(s.q0 + i) * a.tree_words);
    const int words = 2 * a.tree_words;
    if (base < 0) {
      m = (w[0] << -base) | ((1u << -base) - 1);
    } else {
      const int wi = base >> 5, sh = base & 31;
      const uint32_t lo = wi < words ? w[wi] : 0, hi = wi + 1 < words ? w[wi + 1] : 0;
      m = __funnelshift_r(lo, hi, sh);
    }
  } else {
    n = min(n, i + 1 - base);
  }
  return n >= 32 ? m : (n <= 0 ? 0 : m & ((1u << n) - 1));
}

// The page a key lies in; outside the cache: -1 (with the status).
__device__ __forceinline__ int page_of(const TreeAttnArgs& a, int b, int pg) {
  const int p = a.table[(int64_t)b * a.ld_table + pg];
  if (p >= 0 && p < a.n_pages) return p;
  record_status(a.status, kStatusTableRange);
  return -1;
}

// Infinities and NaN among the V elements e0 .. e0 + 31 of the new tokens that
// row i sees in the part's keys: what they add to the row's o.
__device__ __noinline__ void nonfinite_v(const TreeAttnArgs& a, const Seg& s, int i, int e0,
                                         float (&o)[32]) {
  for (int e = 0; e < 32; ++e) o[e] = 0.f;
  const int g = s.g, end = min(s.k1 * kTreeKeys, s.old + s.T);
  for (int j = max(s.k0 * kTreeKeys, s.old); j < end; ++j) {
    if (!(sees32(a, s, i, j) & 1)) continue;
    const int pg = (int)fast_div((uint32_t)j, a.div_page), page = page_of(a, s.b, pg);
    if (page < 0) continue;
    const uint16_t* v =
        a.v + ((((int64_t)(g / a.kv_r) * a.n_pages + page) * a.kv_r + g % a.kv_r) * a.page_size + j -
               pg * a.page_size) * a.head_dim + e0;
    for (int e = 0; e < 32; ++e)
      if ((v[e] & 0x7F80) == 0x7F80) o[e] += bf16_to_f(v[e]);
  }
}

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, d;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 d, x, y, z;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, d;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 d, x, y;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return d;
}

__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(__cvta_generic_to_global(p)) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Bits 15 and 31: whether the bf16 in that half is an infinity or NaN (an
// exponent of ones and one more carries into the sign's place).
__device__ __forceinline__ uint32_t nonfinite2(uint32_t x) {
  return (x & 0x7F807F80u) + 0x00800080u;
}
__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t x) {
  if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
  if ((x & 0x7F800000u) == 0x7F800000u) x &= 0x0000FFFFu;
  return x;
}

// Joins the pieces of an item, in key order, into the rows of o in shared
// memory.  Eight warps share the blocks of 32 rows: lane = row, and a warp takes
// kPer groups of 4 elements at a time, with the loads of kBatch pieces in flight.
// (Not inlined: the softmax loops stay together in the instruction cache.)
template <int D, int kPer, int kBatch>
__device__ __noinline__ void join_pieces(const TreeAttnArgs& a, const Seg& s, int rows, int w, int lane,
                                         uint8_t* sOut) {
  const int blocks = (rows + 31) >> 5;
  constexpr int kTurns = D / 4 / kPer;  // turns of a block
  for (int t = w; t < blocks * kTurns; t += 8) {
    const int r = (t % blocks) * 32 + lane, g0 = t / blocks * kPer;
    const bool on = r < rows;
    float M = -INFINITY, L = 0.f;
    float4 o[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = s.first; p0 <= s.last; p0 += kBatch) {
      float2 ml[kBatch];
      float4 y[kBatch][kPer];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int64_t at = (int64_t)(p0 + b) * 2 + (p0 + b == s.first ? s.slot : 0);
        const bool here = on && p0 + b <= s.last;
        const float4* src = reinterpret_cast<const float4*>(a.partials + at * kTreeRows * D) + r;
        ml[b] = here ? __ldcg(&a.ml[at * kTreeRows + r]) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int q = 0; q < kPer; ++q)
          y[b][q] = here ? __ldcg(src + (g0 + q) * kTreeRows) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float Mn = M;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) Mn = fmaxf(Mn, ml[b].x);
      const float u = M == -INFINITY ? 0.f : ex2_approx(M - Mn);
      M = Mn;
      L = __fmul_rn(L, u);
#pragma unroll
      for (int q = 0; q < kPer; ++q)
        o[q] = make_float4(__fmul_rn(o[q].x, u), __fmul_rn(o[q].y, u), __fmul_rn(o[q].z, u),
                           __fmul_rn(o[q].w, u));
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float v = ml[b].x == -INFINITY ? 0.f : ex2_approx(ml[b].x - Mn);
        L = __fmaf_rn(ml[b].y, v, L);
#pragma unroll
        for (int q = 0; q < kPer; ++q)
          o[q] = make_float4(__fmaf_rn(y[b][q].x, v, o[q].x), __fmaf_rn(y[b][q].y, v, o[q].y),
                             __fmaf_rn(y[b][q].z, v, o[q].z), __fmaf_rn(y[b][q].w, v, o[q].w));
      }
    }
    const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
    if (on) {
      uint2* dst = reinterpret_cast<uint2*>(sOut + r * D * 2);
#pragma unroll
      for (int q = 0; q < kPer; ++q)  // the 16-byte chunks of a row are swizzled by row
        dst[((((g0 + q) >> 1) ^ (r & 7)) << 1) + ((g0 + q) & 1)] =
            make_uint2(pack_p(o[q].x * inv, o[q].y * inv), pack_p(o[q].z * inv, o[q].w * inv));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kTreeThreads, 1)
tree_attn_kernel(const __grid_constant__ TreeAttnArgs a) {
  using SM = TreeSmem<D>;
  // Rings: K and V of each softmax group, (2 * group + (V: 1)) * R on.  Each has
  // one consumer, so that whoever waits for a fill has itself consumed the one
  // before it in that place: a parity then tells the two apart.
  constexpr int R = SM::kDepth;
  constexpr int NB = SM::kBufs, kColO = 2 * NB * kTreeKeys;  // tensor memory: S buffers, then O
  constexpr int HB = kTreeKeys * 128, HQ = kTreeRows * 128;  // bytes of 64 elements of a K/V, Q tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;
  uint8_t* sOut = smem + SM::kOut;
  uint8_t* ring = smem + SM::kRing;
  float2* meet = reinterpret_cast<float2*>(smem + SM::kMeet);
  TreeCtl& ctl = *reinterpret_cast<TreeCtl*>(smem + SM::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4 * R; ++i) { mbar_init(&ctl.full[i], 1); mbar_init(&ctl.empty[i], 1); }
    for (int i = 0; i < 2 * SM::kBufs; ++i) {
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.p_ready[i], 4);
      mbar_init(&ctl.pv_done[i], 1);
    }
    ctl.poison[0] = ctl.poison[1] = 0;
    for (int i = 0; i < 4; ++i) {
      mbar_init(&ctl.seg_full[i], 1);
      mbar_init(&ctl.seg_free[i], kTreeLoaders + 4 + kTreeSoftmax / 32);
    }
    mbar_init(&ctl.q_full, 1);
    mbar_init(&ctl.q_free, 2);
    mbar_init(&ctl.drain, 4);
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&a.tmQ);
    tma_prefetch_desc(&a.tmK);
    tma_prefetch_desc(&a.tmV);
  }
  if (warp == 4) { tmem_alloc(&ctl.tmem, 512); tmem_relinquish(); }
  pdl_wait();

  // This CTA's range: thread t sums the tiles of a run of sequences; the
  // thread whose run holds the range's begin looks it up.
  // No more CTAs take part than there are positions, so that an item's pieces
  // lie with consecutive CTAs.
  int G = gridDim.x;
  const int c = blockIdx.x;
  {
    const int per = (a.n_seqs + kTreeThreads - 1) / kTreeThreads;
    const int lo = min(a.n_seqs, (int)threadIdx.x * per), hi = min(a.n_seqs, lo + per);
    long long sum = 0;
    for (int b = lo; b < hi; ++b) {
      const SeqInfo s = seq_info(a, b);
      sum += positions(a, s);
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) ctl.warp_sum[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kTreeThreads / 32; ++w) {
      const long long y = ctl.warp_sum[w];
      if (w < warp) before += y;
      total += y;
    }
    long long at = before + incl - sum;
    if (total < G) G = (int)total;
    const long long x0 = c < G ? range_at(c, total, G) : total;
    if (x0 >= at && x0 < at + sum) {
      int b = lo;
      while (true) {
        const SeqInfo s = seq_info(a, b);
        const long long n = positions(a, s);
        if (x0 < at + n) break;
        at += n;
        ++b;
      }
      ctl.b0 = b;
      ctl.u0 = x0 - at;
    }
    if (threadIdx.x == 0) {
      ctl.total = total;
      ctl.x0 = x0;
      ctl.x1 = c < G ? range_at(c + 1, total, G) : total;
    }
    __syncthreads();
  }
  const uint32_t tmem = ctl.tmem;
  const int64_t W = ctl.total;
  const int64_t x0 = ctl.x0, x1 = ctl.x1;

  // A wait that runs out is remembered and nothing waits after it: every role
  // then runs to its end without touching the copies or products.
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = mbar_wait(bar, parity, a.status);
  };
  auto wait2 = [&](uint64_t* bar0, uint32_t parity0, uint64_t* bar1, uint32_t parity1) {
    if (!ok) return;
    const uint32_t got = mbar_try_wait2(bar0, parity0, bar1, parity1);
    if (!(got & 1)) ok = mbar_wait(bar0, parity0, a.status);
    if (!(got & 2)) wait(bar1, parity1);
  };
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    wait(bar, parity);
    __syncwarp();
  };

  // the next announced part; k1 = 0 when there is none (or the wait ran out)
  auto fetch = [&](uint32_t seg) -> Seg {
    wait(&ctl.seg_full[seg & 3], (seg >> 2) & 1);
    Seg sg = ctl.seg[seg & 3];
    if (!ok) sg.k1 = 0;
    return sg;
  };
  auto done_with = [&](uint32_t seg) { mbar_arrive(&ctl.seg_free[seg & 3]); };

  // The softmax warpgroups take over registers that the others do not need.
  if (warp < kTreeFirst / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTreeRegsOther));
    if (warp < kTreeLoaders) {
      // ------------------------------------------------------------ K and V
      const uint64_t pol = policy_evict_first();
      const int rows = a.box_rows, boxes = kTreeKeys / rows;
      // lane -> (box, 64-element half)
      const int box = D == 128 ? lane >> 1 : lane, half = D == 128 ? lane & 1 : 0;
      const int grp = warp & 1, turn = warp >> 1;  // every other tile of a group is the warp's
      uint32_t gj = 0;              // the group's tiles before this part
      uint32_t mine[2] = {0, 0};    // this warp's last fills + 1 (K, V)
      for (uint32_t seg = 0;; ++seg) {
        const Seg sg = fetch(seg);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok || sg.k1 == 0) break;
        const int copy = sg.g / a.kv_r, local = sg.g - copy * a.kv_r;
        const int len = sg.old + sg.T, n = sg.k1 - sg.k0;
        const int32_t* row = a.table + (int64_t)sg.b * a.ld_table;
        const int last = (int)fast_div((uint32_t)min(len, sg.k1 * kTreeKeys) - 1, a.div_page);
        // A tile's page numbers, one a box, loaded two of the warp's tiles
        // ahead.
        auto load = [&](int i) {
          const int pg = (int)fast_div((uint32_t)((sg.k0 + i) * kTreeKeys + box * rows), a.div_page);
          return i < n && box < boxes && pg <= last ? row[pg] : 0;
        };
        const int i0 = grp + 2 * ((turn - gj) & 1);
        int page = load(i0), next = load(i0 + 4);
        for (int i = i0; ok && i < n; i += 4) {
          const int after = load(i + 8);
          const int kt = sg.k0 + i;
          const int here = min(boxes, (len - kt * kTreeKeys + rows - 1) / rows);
          const int key = kt * kTreeKeys + box * rows;
          const int off = key - (int)fast_div((uint32_t)key, a.div_page) * a.page_size;
          int z = (copy * a.n_pages + page) * a.kv_r + local;
          if (box < here && (page < 0 || page >= a.n_pages)) {
            record_status(a.status, kStatusTableRange);
            z = a.slices;  // outside the tensor map: zeros
          }
          const uint32_t j = gj + (i >> 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t st = (2 * grp + kv) * R + j % R;
            if (lane == 0) wait(&ctl.empty[st], (j / R & 1) ^ 1);  // one lane polls
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (ok) {
              mine[kv] = j + 1;
              if (lane == 0) mbar_arrive_expect_tx(&ctl.full[st], here * rows * D * 2);
              __syncwarp();
              if (box < here) {
                uint8_t* dst = ring + st * SM::kTile + half * HB + box * rows * 128;
                const CUtensorMap* tm = kv ? &a.tmV : &a.tmK;
                if (a.kv_once) tma_load_3d(dst, tm, &ctl.full[st], half * 64, off, z, pol);
                else tma_load_3d_plain(dst, tm, &ctl.full[st], half * 64, off, z);
              }
            }
          }
          page = next;
          next = after;
        }
        gj += (n - grp + 1) >> 1;
        __syncwarp();
        if (lane == 0) done_with(seg);
      }
      // Never leave with copies still landing in shared memory.  (A fill that
      // another, perhaps another warp's, follows in its place landed before
      // that.)
      if (lane == 0) {
        for (uint32_t back = 0; back < R; back += 2)
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t j = mine[kv] - 1 - back;
            if (mine[kv] > back && (!ok || j + R >= gj))
              mbar_wait(&ctl.full[(2 * grp + kv) * R + j % R], j / R & 1, a.status);
          }
      }
      __syncwarp();
    } else if (warp >= 4 && warp < 8) {
      // ------------------------------------------------------------ products
      if (lane == 0) {
        uint32_t kb = 0, kp = 0;  // the next tile's S buffer (of the group's), and parity
        uint32_t st = 0, ph = 0;  // the next tile's place in its ring, and parity
        const int grp = warp & 1;
        if (warp < 6) {
          constexpr uint32_t idS = idesc_bf16_f32(kTreeRows, kTreeKeys);
          const uint64_t dq = smem_desc_sw128(sQ);
          const uint64_t dk0 = smem_desc_sw128(ring + 2 * grp * R * SM::kTile);
          uint64_t *full = ctl.full + 2 * grp * R, *empty = ctl.empty + 2 * grp * R;
          for (uint32_t seg = 0;; ++seg) {
            const Seg sg = fetch(seg);
            const int n = sg.k1 ? sg.k1 - sg.k0 : 0;
            if (n == 0) break;
            done_with(seg);
            wait(&ctl.q_full, seg & 1);
            for (int i = grp; i < n; i += 2) {
              const int k = grp * NB + kb;
              // P of the buffer's last tile was read, K is there
              wait2(&ctl.pv_done[k], kp ^ 1, &full[st], ph);
              if (!ok) break;
              tc_fence_after();
              const uint64_t dk = dk0 + st * (SM::kTile >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                tc_mma_f16(tmem + k * kTreeKeys, dq + (kk >> 2) * (HQ >> 4) + (kk & 3) * 2,
                           dk + (kk >> 2) * (HB >> 4) + (kk & 3) * 2, idS, kk > 0);
              tc_commit(&ctl.s_full[k]);
              tc_commit(&empty[st]);
              if (++st == R) { st = 0; ph ^= 1; }
              if (++kb == NB) { kb = 0; kp ^= 1; }
            }
            if (ok) tc_commit(&ctl.q_free);
          }
        } else {
          constexpr uint32_t idO = idesc_bf16_f32_bmn(kTreeRows, D);
          const uint32_t dO = tmem + kColO + grp * D;
          const uint64_t dv0 = smem_desc_mn_sw128(ring + (2 * grp + 1) * R * SM::kTile, HB);
          uint64_t *full = ctl.full + (2 * grp + 1) * R, *empty = ctl.empty + (2 * grp + 1) * R;
          for (uint32_t seg = 0;; ++seg) {
            const Seg sg = fetch(seg);
            const int n = sg.k1 ? sg.k1 - sg.k0 : 0;
            if (n == 0) break;
            done_with(seg);
            for (int i = grp; i < n; i += 2) {
              const int k = grp * NB + kb;
              wait2(&ctl.p_ready[k], kp, &full[st], ph);
              if (!ok) break;
              tc_fence_after();
              const uint64_t dv = dv0 + st * (SM::kTile >> 4);
#pragma unroll
              for (int kk = 0; kk < kTreeKeys / 16; ++kk)
                tc_mma_f16_ta(dO, tmem + k * kTreeKeys + 8 * kk, dv + 128 * kk, idO, i >= 2 || kk > 0);
              tc_commit(&ctl.pv_done[k]);
              tc_commit(&empty[st]);
              if (++st == R) { st = 0; ph ^= 1; }
              if (++kb == NB) { kb = 0; kp ^= 1; }
            }
          }
        }
        tc_commit(&ctl.drain);
        mbar_wait(&ctl.drain, 0, a.status);
      }
      __syncwarp();
    } else if (warp == 8) {
      // ------------------------------------------------------------ parts, queries
      SegIter it(a, x0, x1, ctl.u0, ctl.b0);
      uint32_t told = 0;
      bool more = true;
      auto announce = [&]() {
        const Seg sg = it.next(W, G);
        wait(&ctl.seg_free[told & 3], ((told >> 2) & 1) ^ 1);
        __syncwarp();
        if (lane == 0) {
          ctl.seg[told & 3] = sg;
          mbar_arrive(&ctl.seg_full[told & 3]);
        }
        __syncwarp();
        ++told;
        more = sg.k1 > 0;
      };
      announce();
      if (more) announce();
      // A query tile is a box of the group's heads and its tokens.  (Rows
      // behind the item's hold other tokens or zeros; nothing reads their o.)
      uint32_t asked = 0;
      for (uint32_t seg = 0;; ++seg) {
        const Seg sg = ctl.seg[seg & 3];
        if (sg.k1 == 0) break;
        if (lane == 0) {
          wait(&ctl.q_free, (seg & 1) ^ 1);
          if (ok) {
            ++asked;
            mbar_arrive_expect_tx(&ctl.q_full, a.tile_rows * D * 2);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d_plain(sQ + h * HQ, &a.tmQ, &ctl.q_full, h * 64, sg.g * a.group,
                                sg.q0 + sg.qi * a.tile_toks);
          }
        }
        __syncwarp();
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (more) announce();
      }
      if (lane == 0 && asked) mbar_wait(&ctl.q_full, (asked - 1) & 1, a.status);  // landed
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTreeRegsSoftmax));
    // ------------------------------------------------------------ softmax
    const int grp = (warp - kTreeFirst / 32) >> 2, quad = warp & 3;
    const int tid = threadIdx.x - kTreeFirst;       // 0..255 over both groups
    const int r = quad * 32 + lane;          // the thread's row of the tile
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + lanes, tO = tmem + lanes + kColO + grp * D;
    uint32_t gj = 0;   // the group's tiles before this part
    uint32_t kb = 0, kp = 0;  // the next tile's S buffer (of the group's), and parity
    // waits for the products with P of the group's last tile
    auto wait_pv = [&]() {
      warp_wait(&ctl.pv_done[grp * NB + (kb ? kb - 1 : NB - 1)], kb ? kp : kp ^ 1);
    };
    for (uint32_t seg = 0;; ++seg) {
      const Seg s = fetch(seg);
      // all of them go on, or none: they meet at named barriers below
      if (bar_sync_or(1, kTreeSoftmax, s.k1 == 0)) break;
      const int row0 = s.qi * a.tile_rows, rows = min(a.tile_rows, s.T * a.group - row0);
      const bool warp_live = quad * 32 < rows;
      const int tok = (int)fast_div((uint32_t)(row0 + min(r, rows - 1)), a.div_group);
      const int n = s.k1 - s.k0, len = s.old + s.T;
      // The running maximum (in units of log2) and sum.  Rows behind the item's hold
      // other queries, or anything: a maximum that no score exceeds keeps them out of
      // the vote on rescaling.  (NaN there took one token behind 20000 from 25 to 29 us.)
      float m = r < rows ? -INFINITY : INFINITY, l = 0.f;
      uint32_t vis[2];
      // tile i: scores from tensor memory, P back into it
      auto tile = [&](auto tail_tag, int i) {
        constexpr bool kTail = decltype(tail_tag)::value;
        const uint32_t t = tS + (grp * NB + kb) * kTreeKeys;
        // Two halves of 32 keys: one's scores arrive while the other's are worked on.
        float x[2][32];
        auto mask = [&](int h) {
          if constexpr (kTail) {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[h][e] = (vis[h] >> e & 1) ? x[h][e] : -INFINITY;
          }
        };
        float2 sums[2];
        auto probabilities = [&](int h, float sub) {
          uint32_t y[16];
          const float2 scale = make_float2(a.scale_log2, a.scale_log2), minus = make_float2(-sub, -sub);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 z = fma2(make_float2(x[h][2 * e], x[h][2 * e + 1]), scale, minus);
            const float2 p = make_float2(ex2_approx(z.x), ex2_approx(z.y));
            sums[e & 1] = add2(sums[e & 1], p);
            y[e] = pack_p(p.x, p.y);
          }
          tmem_st16(t + 16 * h, y);
        };
        // The probabilities relative to the maximum so far, before the tile's
        // own maximum is known: most tiles do not raise it by 2^8, and neither
        // chain then waits for the other.
        sums[0] = sums[1] = make_float2(0.f, 0.f);
        tmem_ld32(t, x[0]);
        tmem_ld32(t + 32, x[1]);
        tmem_ld_wait32(x[0]);
        mask(0);
        probabilities(0, m);
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 16; ++e)
          tops[e & 3] = fmaxf(tops[e & 3], fmaxf(x[0][2 * e], x[0][2 * e + 1]));
        tmem_ld_wait32(x[1]);
        mask(1);
        probabilities(1, m);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          tops[e & 3] = fmaxf(tops[e & 3], fmaxf(x[1][2 * e], x[1][2 * e + 1]));
        const float top =
            fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * a.scale_log2;
        const bool rise = top > m + kRescaleLog2 || m == -INFINITY;
        if (__any_sync(0xffffffffu, rise)) {
          const float mn = rise ? top : m;
          if (i >= 2) {
            const float al = rise && top > m ? ex2_approx(m - mn) : 1.f;  // m = -inf: 0
            wait_pv();
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              float o[16];
              uint32_t z[16];
              tmem_ld16(tO + 16 * q, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) z[e] = __float_as_uint(o[e] * al);
              tmem_st16(tO + 16 * q, z);
            }
            l *= al;
          }
          m = mn;
          // masked scores: exp2(-inf - sub) = 0
          const float sub = m == -INFINITY ? 0.f : m;
          sums[0] = sums[1] = make_float2(0.f, 0.f);
          probabilities(0, sub);
          probabilities(1, sub);
        }
        l += (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
        tmem_st_wait();
      };
      for (int i = grp; i < n; i += 2) {
        const int key0 = (s.k0 + i) * kTreeKeys, k = grp * NB + kb;
        const bool tail = key0 + kTreeKeys > s.old;
        // (Scores first: with them, the fill before this one in V's place was
        // consumed.)
        warp_wait(&ctl.s_full[k], kp);
        tc_fence_after();
        if (tail) {
          // V of keys behind the end and non-finite V of new tokens: two
          // threads a key, each half of its elements
          const uint32_t j = gj + (i >> 1), st = (2 * grp + 1) * R + j % R;
          warp_wait(&ctl.full[st], j / R & 1);
          const int kr = r & 63, key = key0 + kr;
          uint8_t* v = ring + st * SM::kTile + kr * 128;
          auto chunk = [&](int ch) {  // of the thread's D / 16
            const int c8 = (r >> 6) * (D / 16) + ch;
            return reinterpret_cast<uint4*>(v + (c8 >> 3) * HB + (((c8 ^ kr) & 7) << 4));
          };
          if (key >= len) {
#pragma unroll
            for (int ch = 0; ch < D / 16; ++ch) *chunk(ch) = make_uint4(0, 0, 0, 0);
          } else if (key >= s.old) {
            uint32_t found = 0;
#pragma unroll
            for (int ch = 0; ch < D / 16; ++ch) {
              const uint4 w = *chunk(ch);
              found |= nonfinite2(w.x) | nonfinite2(w.y) | nonfinite2(w.z) | nonfinite2(w.w);
            }
            if (found & 0x80008000u) {
              ctl.poison[seg & 1] = 1;
              for (int ch = 0; ch < D / 16; ++ch) {
                uint4* p = chunk(ch);
                *p = make_uint4(drop_nonfinite(p->x), drop_nonfinite(p->y), drop_nonfinite(p->z),
                                drop_nonfinite(p->w));
              }
            }
          }
          vis[0] = sees32(a, s, tok, key0);
          vis[1] = sees32(a, s, tok, key0 + 32);
          fence_proxy_async_smem();
        }
        if (warp_live) {
          if (tail) tile(std::true_type(), i);
          else tile(std::false_type(), i);
        }
        if (++kb == NB) { kb = 0; kp ^= 1; }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.p_ready[k]);
      }

      // Of a cut item, whether every other piece is there already: this one then
      // need not be written.
      const bool whole = s.k0 == 0 && s.k1 == s.nt;
      int* ticket = a.tickets + ((int64_t)s.b * a.n_kv + s.g) * a.q_tiles_max + s.qi;
      if (tid == 0) {
        ctl.last = 0;
        if (!whole && rows > kFewRows && ld_acquire(ticket) == s.last - s.first) {
          *ticket = 0;
          ctl.last = 1;
        }
      }
      // The two groups' states meet, and each takes one half of the head's
      // elements of both O.
      if (n > grp) wait_pv();
      meet[grp * kTreeRows + r] = make_float2(m, l);
      bar_sync(1, kTreeSoftmax);
      tc_fence_after();
      const bool joins = ctl.last != 0;
      const bool live = r < rows;
      if (warp_live) {
        const float2 ml0 = meet[r], ml1 = n > 1 ? meet[kTreeRows + r] : make_float2(-INFINITY, 0.f);
        const float M = fmaxf(ml0.x, ml1.x);
        float w0 = ml0.x == -INFINITY ? 0.f : ex2_approx(ml0.x - M);
        float w1 = ml1.x == -INFINITY ? 0.f : ex2_approx(ml1.x - M);
        const float L = ml0.y * w0 + ml1.y * w1;
        const int64_t piece = (int64_t)c * 2 + (!whole && c == s.first ? s.slot : 0);
        if (!whole && !joins && live && grp == 0) a.ml[piece * kTreeRows + r] = make_float2(M, L);
        if (whole) {
          const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
          w0 *= inv;
          w1 *= inv;
        }
        const uint32_t keep0 = w0 != 0.f ? ~0u : 0u, keep1 = w1 != 0.f ? ~0u : 0u;
        const bool poison = ctl.poison[seg & 1] != 0;
#pragma unroll 1
        for (int q = 0; q < D / 64; ++q) {  // 32 elements a turn
          const int e0 = grp * (D / 2) + 32 * q;
          float o0[32], o1[32];
          tmem_ld32(tmem + lanes + kColO + e0, o0);
          tmem_ld32(tmem + lanes + kColO + D + e0, o1);
          tmem_ld_wait32(o0);
          tmem_ld_wait32(o1);
          // a state without keys may stand next to anything in tensor memory
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o0[e] = fmaf(__uint_as_float(__float_as_uint(o0[e]) & keep0), w0,
                         __uint_as_float(__float_as_uint(o1[e]) & keep1) * w1);
          if (poison && live) {
            float add[32];  // (its own array: o0 stays in registers)
            nonfinite_v(a, ctl.seg[seg & 3], tok, e0, add);
#pragma unroll
            for (int e = 0; e < 32; ++e) o0[e] += add[e];
          }
          if (joins) {
            // the other pieces and this one, in the order and with the operations
            // of join_pieces
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
              float Mr = -INFINITY, Lr = 0.f, acc[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[e] = 0.f;
              for (int p0 = s.first; p0 <= s.last; p0 += 2) {
                float2 pml[2];
                float4 y[2][4];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  const int64_t at = (int64_t)(p0 + b) * 2 + (p0 + b == s.first ? s.slot : 0);
                  const bool here = live && p0 + b <= s.last && p0 + b != c;
                  const float4* src = reinterpret_cast<const float4*>(a.partials + at * kTreeRows * D) +
                                      ((e0 + h) >> 2) * kTreeRows + r;
                  pml[b] = here ? __ldcg(&a.ml[at * kTreeRows + r]) : make_float2(-INFINITY, 0.f);
#pragma unroll
                  for (int q = 0; q < 4; ++q)
                    y[b][q] = here ? __ldcg(src + q * kTreeRows) : make_float4(0.f, 0.f, 0.f, 0.f);
                  if (p0 + b == c) {
                    pml[b] = make_float2(M, L);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                      y[b][q] = make_float4(o0[h + 4 * q], o0[h + 4 * q + 1], o0[h + 4 * q + 2],
                                            o0[h + 4 * q + 3]);
                  }
                }
                const float Mn = fmaxf(fmaxf(Mr, pml[0].x), pml[1].x);
                const float u = Mr == -INFINITY ? 0.f : ex2_approx(Mr - Mn);
                Mr = Mn;
                Lr = __fmul_rn(Lr, u);
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[e] = __fmul_rn(acc[e], u);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  const float v = pml[b].x == -INFINITY ? 0.f : ex2_approx(pml[b].x - Mn);
                  Lr = __fmaf_rn(pml[b].y, v, Lr);
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    acc[4 * q] = __fmaf_rn(y[b][q].x, v, acc[4 * q]);
                    acc[4 * q + 1] = __fmaf_rn(y[b][q].y, v, acc[4 * q + 1]);
                    acc[4 * q + 2] = __fmaf_rn(y[b][q].z, v, acc[4 * q + 2]);
                    acc[4 * q + 3] = __fmaf_rn(y[b][q].w, v, acc[4 * q + 3]);
                  }
                }
              }
              const float inv = Lr > 0.f || Lr != Lr ? 1.f / Lr : 0.f;
#pragma unroll
              for (int e = 0; e < 16; ++e) o0[h + e] = acc[e] * inv;
            }
          }
          if (whole || joins) {
            // through shared memory: rows of o leave as whole lines
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(sOut + r * D * 2 + ((((e0 + e) >> 3) ^ (r & 7)) << 4)) =
                  make_uint4(pack_p(o0[e], o0[e + 1]), pack_p(o0[e + 2], o0[e + 3]),
                             pack_p(o0[e + 4], o0[e + 5]), pack_p(o0[e + 6], o0[e + 7]));
          } else {
            // [4 elements][row]: a warp's stores are contiguous
            float4* dst = reinterpret_cast<float4*>(a.partials + piece * kTreeRows * D) +
                          (e0 >> 2) * kTreeRows + r;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e * kTreeRows] = make_float4(o0[4 * e], o0[4 * e + 1], o0[4 * e + 2], o0[4 * e + 3]);
          }
        }
      }
      tc_fence_before();
      if (tid == 0) ctl.poison[(seg + 1) & 1] = 0;
      bar_sync(1, kTreeSoftmax);  // O was read; the rows are in shared memory, or the pieces written
      bool finish = whole || joins;
      if (!finish) {
        if (tid == 0) {
          fence_acq_rel_gpu();
          const bool last = atomicAdd(ticket, 1) == s.last - s.first;
          if (last) *ticket = 0;
          fence_acq_rel_gpu();
          ctl.last = last;
        }
        bar_sync(1, kTreeSoftmax);
        finish = ctl.last != 0;
        if (finish) {
          // Few rows, as single tokens have, are cut finer, so that every warp has
          // some, and mostly lie in more pieces.
          if (rows <= kFewRows) join_pieces<D, 4, 4>(a, ctl.seg[seg & 3], rows, tid >> 5, lane, sOut);
          else join_pieces<D, 8, 2>(a, ctl.seg[seg & 3], rows, tid >> 5, lane, sOut);
          bar_sync(1, kTreeSoftmax);
        }
      }
      if (finish) {
        const int ch = tid % (D / 8);
        for (int rr = tid / (D / 8); rr < rows; rr += kTreeSoftmax / (D / 8)) {
          const int i = (int)fast_div((uint32_t)(row0 + rr), a.div_group);
          const int h = row0 + rr - i * a.group;
          *reinterpret_cast<uint4*>(a.o + (s.q0 + i) * a.ld_o + (s.g * a.group + h) * D + ch * 8) =
              *reinterpret_cast<const uint4*>(sOut + rr * D * 2 + ((ch ^ (rr & 7)) << 4));
        }
      }
      gj += (n - grp + 1) >> 1;
      __syncwarp();
      if (lane == 0) done_with(seg);
    }
  }
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
static cudaError_t launch_tree(const TreeAttnArgs& a, cudaStream_t st) {
  static const cudaError_t regs = [] {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, tree_attn_kernel<D>);
    if (e != cudaSuccess) return e;
    return fa.numRegs * kTreeThreads <
                   (kTreeThreads - kTreeSoftmax) * kTreeRegsOther + kTreeSoftmax * kTreeRegsSoftmax
               ? cudaErrorLaunchOutOfResources
               : cudaSuccess;
  }();
  if (regs != cudaSuccess) return regs;
  // every call: the attribute is the current device's
  cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       TreeSmem<D>::kTotal);
  if (e != cudaSuccess) return e;
  return launch_k(tree_attn_kernel<D>, dim3(a.grid), dim3(kTreeThreads), TreeSmem<D>::kTotal, st, a);
}

cudaError_t launch_tree_attn(const TreeAttnArgs& a, cudaStream_t st) {
  return a.head_dim == 128 ? launch_tree<128>(a, st) : launch_tree<64>(a, st);
}

}  // namespace tpk
