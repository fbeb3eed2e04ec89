// group_rows.cu -- the plan of a grouped product: row numbers sorted by
// group id, stable, with the groups' offsets (a counting sort).
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

// One CTA: histogram, exclusive scan, then the rows chunk by chunk, the warps
// of a chunk in turn, so that rows of one group keep their order.
__global__ void __launch_bounds__(1024) group_rows_kernel(int n, int G, const int32_t* __restrict__ ids,
                                                          int32_t* __restrict__ offsets, int32_t* __restrict__ rows) {
  __shared__ int base[kMaxGroups + 1];
  __shared__ int wtot[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int g = tid; g <= G; g += 1024) base[g] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += 1024) {
    const int id = ids[i];
    atomicAdd(&base[id >= 0 && id < G ? id : G], 1);
  }
  __syncthreads();
  // exclusive scan over the groups (G <= 1024, one per thread), then the rows of no group
  const int c = tid < G ? base[tid] : 0;
  int s = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += v;
  }
  if (lane == 31) wtot[warp] = s;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; w++) before += wtot[w];
  __syncthreads();
  if (tid < G) {
    base[tid] = before + s - c;
    offsets[tid] = before + s - c;
    if (tid == G - 1) {
      base[G] = before + s;
      offsets[G] = before + s;
    }
  }
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += 1024) {
    const int i = i0 + tid;
    const int id = i < n ? ids[i] : -1;
    const int key = i < n ? (id >= 0 && id < G ? id : G) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, key);
    const int rank = __popc(same & ((1u << lane) - 1u));
    for (int w = 0; w < 32; w++) {
      if (w == warp && key >= 0) {
        rows[base[key] + rank] = i;
        __syncwarp(__activemask());
        if (rank == 0) base[key] += __popc(same);
      }
      __syncthreads();
    }
  }
}

}  // namespace

cudaError_t launch_group_rows(int n, int n_groups, const int32_t* ids, int32_t* offsets, int32_t* rows, uint32_t*,
                              cudaStream_t s) {
  group_rows_kernel<<<1, 1024, 0, s>>>(n, n_groups, ids, offsets, rows);
  return cudaGetLastError();
}

}  // namespace moe
