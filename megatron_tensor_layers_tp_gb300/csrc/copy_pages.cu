// Pages of the cache copied in every layer at once.
//
// Memory-bound: bytes in, bytes out.  A run is one head's tokens of a page, contiguous;
// a warp takes 4 KB of one at a time, eight 16-byte words a lane in flight.  The
// number of moves is on the GPU: a fixed grid of CTAs, 16 an SM, strides over them (150
// pages of 16 tokens, half full, in 32 layers of 8 heads of 128: 47.3 us, 6.7 TB/s; 8 an
// SM 48.5, 4 an SM 50.7; pieces of 2 KB 51, of 8 KB 53.5).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "paged.h"
#include "ptx.cuh"

namespace tpk {

constexpr int kCpThreads = 256, kCpWarps = kCpThreads / 32;
constexpr int kCpWords = 256;  // 16-byte words of a piece

__global__ void __launch_bounds__(kCpThreads) copy_pages_kernel(const __grid_constant__ CopyPagesArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int said = *a.n_moves, n = min(max(said, 0), a.max_moves);
  if (said != n && blockIdx.x == 0 && threadIdx.x == 0) record_status(a.status, kStatusTableRange);
  const int64_t pieces = (int64_t)n * a.move_pieces;
  for (int64_t piece = (int64_t)blockIdx.x * kCpWarps + (threadIdx.x >> 5); piece < pieces;
       piece += (int64_t)gridDim.x * kCpWarps) {
    const int move = pieces <= INT32_MAX ? (int)fast_div((uint32_t)piece, a.div_move) : (int)(piece / a.move_pieces);
    const uint32_t rest = (uint32_t)(piece - (int64_t)move * a.move_pieces);
    const uint32_t run = fast_div(rest, a.div_run), pool = fast_div(run, a.div_heads);
    const int first = (int)(rest - run * a.run_pieces) * kCpWords, head = (int)(run - pool * (a.copies * a.kv_r));
    const int copy = (int)fast_div((uint32_t)head, a.div_kv), local = head - copy * a.kv_r;
    const int from = a.moves[3 * move], to = a.moves[3 * move + 1], tokens = a.moves[3 * move + 2];
    if ((uint32_t)from >= (uint32_t)a.n_pages || (uint32_t)to >= (uint32_t)a.n_pages || tokens < 0 ||
        tokens > a.page_size) {
      if (rest == 0 && lane == 0) record_status(a.status, kStatusTableRange);
      continue;
    }
    const int left = tokens * a.row - first;  // words of the run from here on
    if (from == to || left <= 0) continue;
    const int64_t page = (int64_t)a.page_size * a.row;  // words of a head's page
    uint4* base = a.pools[pool] + first + lane;
    const uint4* in = base + (((int64_t)copy * a.n_pages + from) * a.kv_r + local) * page;
    uint4* out = base + (((int64_t)copy * a.n_pages + to) * a.kv_r + local) * page;
    uint4 x[kCpWords / 32];
#pragma unroll
    for (int k = 0; k < kCpWords / 32; ++k)
      if (lane + 32 * k < left) x[k] = in[32 * k];
#pragma unroll
    for (int k = 0; k < kCpWords / 32; ++k)
      if (lane + 32 * k < left) out[32 * k] = x[k];
  }
}

cudaError_t launch_copy_pages(CopyPagesArgs a, int num_sms, cudaStream_t st) {
  a.run_pieces = (a.page_size * a.row + kCpWords - 1) / kCpWords;
  a.move_pieces = 2 * a.layers * a.copies * a.kv_r * a.run_pieces;
  a.div_move = make_fastdiv((uint32_t)a.move_pieces);
  a.div_run = make_fastdiv((uint32_t)a.run_pieces);
  const int64_t pieces = (int64_t)a.max_moves * a.move_pieces;
  const int grid = (int)std::min<int64_t>((pieces + kCpWarps - 1) / kCpWarps, 16 * num_sms);
  return launch_k(copy_pages_kernel, dim3(grid), dim3(kCpThreads), 0, st, a);
}

}  // namespace tpk
