// group_rows.cu -- the plan of a grouped product: row numbers sorted by group
// id, stable, with the groups' offsets.
//
// A counting sort in one launch.  Every warp owns a stretch of the ids and
// counts them by group in a table of its own, the warps' and CTAs' counts are
// summed in order, and every warp walks its stretch again and places its rows
// (32 ids at a time: lanes with equal ids find each other by ballots and rank
// themselves).  So the order is that of the rows.
//
// The work is a few bytes a row; what bounds it is the chain of dependent
// steps.  Up to 1024 rows one CTA does all (4.5 us against 5.2 of a cluster,
// 128 groups), above that a cluster of eight, whose counts meet in distributed
// shared memory (2048 rows 5.4 against 5.7 us, 16384 6.6 against 22, 65536
// 9.2).
#include "sort.cuh"

namespace moe {

namespace {

__global__ void __launch_bounds__(1024) group_rows_kernel(int n, int G, int bits, int stretch, const int32_t* ids, int32_t* offsets,
                                                          int32_t* rows) {
  extern __shared__ uint8_t raw[];
  pdl_trigger();
  sort_rows(n, G, bits, stretch, ids, offsets, rows, raw, [] { pdl_wait(); });
}

}  // namespace

cudaError_t launch_group_rows(int n, int n_groups, const int32_t* ids, int32_t* offsets, int32_t* rows,
                              cudaStream_t s) {
  const int ctas = n <= 1024 ? 1 : kSortCtas, stretch = sort_stretch(n, ctas), bits = sort_bits(n_groups);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(1024);
  cfg.dynamicSmemBytes = sort_bytes(n, n_groups, stretch);
  if (cfg.dynamicSmemBytes > 48 * 1024) {
    // the most of any call, so that calls of other threads never lower it
    const int most = (int)sort_bytes(kMaxRows, kMaxGroups, sort_stretch(kMaxRows, kSortCtas));
    cudaError_t e = cudaFuncSetAttribute(group_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
  }
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, group_rows_kernel, n, n_groups, bits, stretch, ids, offsets, rows);
}

}  // namespace moe
