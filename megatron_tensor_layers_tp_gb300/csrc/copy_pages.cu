// Pages of the cache copied in every layer at once.
//
// Memory-bound: bytes in, bytes out.  A run is one head's tokens of a page,
// contiguous; a warp takes a run at a time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "paged.h"
#include "ptx.cuh"

namespace tpk {

constexpr int kCpThreads = 256, kCpWarps = kCpThreads / 32;

__global__ void __launch_bounds__(kCpThreads) copy_pages_kernel(const __grid_constant__ CopyPagesArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int said = *a.n_moves, n = min(max(said, 0), a.max_moves);
  if (said != n && blockIdx.x == 0 && threadIdx.x == 0) record_status(a.status, kStatusTableRange);
  const int heads = a.copies * a.kv_r, pools = 2 * a.layers;
  const int64_t runs = (int64_t)n * pools * heads;
  for (int64_t run = (int64_t)blockIdx.x * kCpWarps + (threadIdx.x >> 5); run < runs;
       run += (int64_t)gridDim.x * kCpWarps) {
    const int move = (int)(run / (pools * heads)), rest = (int)(run - (int64_t)move * pools * heads);
    const int pool = (int)fast_div((uint32_t)rest, a.div_heads), head = rest - pool * heads;
    const int copy = (int)fast_div((uint32_t)head, a.div_kv), local = head - copy * a.kv_r;
    const int from = a.moves[3 * move], to = a.moves[3 * move + 1], tokens = a.moves[3 * move + 2];
    if ((uint32_t)from >= (uint32_t)a.n_pages || (uint32_t)to >= (uint32_t)a.n_pages || tokens < 0 ||
        tokens > a.page_size) {
      if (rest == 0 && lane == 0) record_status(a.status, kStatusTableRange);
      continue;
    }
    if (from == to) continue;
    const int64_t page = (int64_t)a.page_size * a.row;  // words of a head's page
    uint4* base = a.pools[pool];
    const uint4* in = base + (((int64_t)copy * a.n_pages + from) * a.kv_r + local) * page;
    uint4* out = base + (((int64_t)copy * a.n_pages + to) * a.kv_r + local) * page;
    const int words = tokens * a.row;
    for (int i = lane; i < words; i += 256) {
      uint4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (i + 32 * k < words) x[k] = in[i + 32 * k];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (i + 32 * k < words) out[i + 32 * k] = x[k];
    }
  }
}

cudaError_t launch_copy_pages(const CopyPagesArgs& a, int num_sms, cudaStream_t st) {
  const int64_t runs = (int64_t)a.max_moves * 2 * a.layers * a.copies * a.kv_r;
  const int grid = (int)std::min<int64_t>((runs + kCpWarps - 1) / kCpWarps, 8 * num_sms);
  return launch_k(copy_pages_kernel, dim3(grid), dim3(kCpThreads), 0, st, a);
}

}  // namespace tpk
