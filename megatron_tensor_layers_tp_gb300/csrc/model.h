// The model object behind the C ABI and the helpers that every entry point
// uses: status codes, counted and timed launches, tensor maps.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <utility>
#include <vector>

#include "internal.h"
#include "tp.h"

namespace tpk {
// Output-feature tile widths of the prefill orientation, widest first.
constexpr int kPrefillBNs[] = {256, 224, 192, 160, 128};
constexpr int kNumPrefillBN = 5;
constexpr int kPrefillBN = kPrefillBNs[0];

struct ShardedLinear {
  uint16_t* data = nullptr;  // [t][rows][cols]
  uint16_t* bias = nullptr;  // optional: [ranks][rows] (column-parallel) or [rows] (row-parallel)
  int rows = 0, cols = 0;    // per rank
  int ranks = 0;             // t, or attn_tp for the attention block
  CUtensorMap tm_a;          // box (64, 128, 1): weight on the MMA M side (decode)
  CUtensorMap tm_b[kNumPrefillBN];  // box (64, kPrefillBNs[i], 1): weight on the MMA N side (prefill)
  CUtensorMap tm_h[kNumPrefillBN];  // box (64, kPrefillBNs[i] / 2, 1): one CTA's half (CTA pairs)
};

struct LayerShards {
  ShardedLinear qkv, gate_up, o, down;
  // qkv and gate_up with the preceding RMSNorm's weight folded into their
  // columns (W[n][k] * w[k]): the decoder layer's GEMMs read these, and the
  // raw hidden state; tp_column_linear keeps the plain shards
  ShardedLinear qkv_folded, gate_up_folded;
  uint16_t* attn_norm = nullptr;
  uint16_t* mlp_norm = nullptr;
};
}  // namespace tpk

struct tp_model {
  tp_config_t cfg;
  int device = 0;
  int num_sms = 0;
  bool host_coherent = false;  // the GPU reaches host memory coherently (NVLink-C2C)
  std::vector<tpk::LayerShards> layers;
  uint16_t* embed = nullptr;  // [Vp][H] = t shards of [Vp/t][H]
  tpk::ShardedLinear lm;
  uint16_t* final_norm = nullptr;
  uint16_t* ones = nullptr;  // [H] bf16 1.0: the norm weight once it is folded
  float2* rope = nullptr;
  int* status = nullptr;
  std::vector<std::pair<void*, size_t>> allocs;  // device buffers and their sizes
  mutable tp_stats_t stats;
  // per-launch timing (tp_profile)
  bool profiling = false;
  struct Rec { const char* name; cudaEvent_t a, b; };
  mutable std::vector<Rec> recs;
  mutable std::vector<cudaEvent_t> pool;
  mutable size_t pool_used = 0;
};

namespace tpk {

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int cdiv(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline tp_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return TP_OK;
  if (e == cudaErrorMemoryAllocation) return TP_ERR_OOM;
  return TP_ERR_CUDA;
}

#define TP_CHECK_CUDA(expr)                         \
  do {                                              \
    cudaError_t _e = (expr);                        \
    if (_e != cudaSuccess) return cuda_status(_e);  \
  } while (0)

constexpr size_t kMaxProfiled = 16384;

// Every kernel launch of the library goes through here: counted, and timed
// with two events on the launch stream while profiling is enabled.
template <class F>
cudaError_t launch(const tp_model* m, const char* name, cudaStream_t st, F&& f) {
  m->stats.kernel_launches++;
  if (!m->profiling || m->recs.size() >= kMaxProfiled) return f();
  while (m->pool.size() < m->pool_used + 2) {
    cudaEvent_t ev;
    cudaError_t e = cudaEventCreate(&ev);
    if (e != cudaSuccess) return e;
    m->pool.push_back(ev);
  }
  cudaEvent_t a = m->pool[m->pool_used++], b = m->pool[m->pool_used++];
  cudaError_t e = cudaEventRecord(a, st);
  if (e != cudaSuccess) return e;
  e = f();
  if (e != cudaSuccess) return e;
  m->recs.push_back({name, a, b});
  return cudaEventRecord(b, st);
}

// 3-D bf16 tensor map (inner K, rows, slices) with a (64, box_rows, box_slices)
// box and 128-byte swizzle; reads outside the extents return zeros.
// When the slices sit closer together than the rows (rank shards side by side
// in one [rows, t*K] buffer), the dimensions are ordered (K, slice, rows) so
// the strides increase; *slice_mid reports which order was used.
bool make_tmap(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t slices,
               uint64_t row_stride_bytes, uint64_t slice_stride_bytes, uint32_t box_rows,
               int* slice_mid = nullptr, uint32_t box_slices = 1);

}  // namespace tpk
