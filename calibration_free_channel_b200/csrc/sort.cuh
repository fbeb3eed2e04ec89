// sort.cuh -- the counting sort of group_rows.cu, shared with the block's
// routing of few tokens (block.cu), which runs it on ids it has just chosen.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace moe {

constexpr int kSortWarps = 32;
constexpr int kSortCtas = 8;
constexpr int kBatch = 8;  // ids a lane loads at a time

struct SortSide {
  int total[kMaxGroups + 1];  // this CTA's rows of each group, then the first position of each
  int scan[kSortWarps];
};

// Called by 1024 threads of one CTA, or of each of the cluster's; raw: dynamic
// shared memory of sort_bytes.  `ready` is called once what precedes it has
// been set up: the ids may be read afterwards.
template <typename F>
__device__ __forceinline__ void sort_rows(int n, int G, int bits, int stretch, const int32_t* ids, int32_t* offsets,
                                          int32_t* rows, uint8_t* raw, F ready) {
  SortSide& s = *reinterpret_cast<SortSide*>(raw);
  int* table = reinterpret_cast<int*>(raw + sizeof(SortSide));  // [warps][G + 1]
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, keys = G + 1;
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int i0 = min((rank * kSortWarps + warp) * stretch, n), i1 = min(i0 + stretch, n);
  // warps that own a stretch: their tables are summed
  const int left = n - rank * kSortWarps * stretch;
  const int active = left <= 0 ? 0 : min((left + stretch - 1) / stretch, kSortWarps);
  int* mine = table + warp * keys;
  for (int i = tid; i < active * keys; i += 1024) table[i] = 0;
  ready();
  __syncthreads();
  auto walk = [&](auto f) {
    for (int b = i0; b < i1; b += 32 * kBatch) {
      int key[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; j++) {
        const int i = b + 32 * j + lane;
        const int id = i < i1 ? ids[i] : 0;
        key[j] = i < i1 ? (id >= 0 && id < G ? id : G) : -1;
      }
#pragma unroll
      for (int j = 0; j < kBatch; j++) {
        if (b + 32 * j >= i1) break;
        // lanes with the same key, a ballot for each bit of it (match.any takes
        // a step for each distinct key: 1900 cycles instead of 150 for 32 of them)
        unsigned same = __ballot_sync(0xffffffffu, key[j] >= 0);
        for (int bit = 0; bit < bits; bit++) {
          const bool on = (key[j] >> bit) & 1;
          const unsigned m = __ballot_sync(0xffffffffu, on);
          same &= on ? m : ~m;
        }
        const int before = __popc(same & ((1u << lane) - 1u));
        f(key[j], b + 32 * j + lane, before, __popc(same));
        __syncwarp();
      }
    }
  };
  // counts need no order: one shared add each (by ballots, as in the
  // second walk, 65536 rows took 13.2 us instead of 9.2)
  for (int b = i0; b < i1; b += 32 * kBatch) {
    int id[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; j++) {
      const int i = b + 32 * j + lane;
      id[j] = i < i1 ? ids[i] : 0;
    }
#pragma unroll
    for (int j = 0; j < kBatch; j++)
      if (b + 32 * j + lane < i1) atomicAdd(&mine[id[j] >= 0 && id[j] < G ? id[j] : G], 1);
  }
  __syncthreads();
  // per group: the warps' counts to exclusive prefixes, and the CTA's total
  for (int k = tid; k < keys; k += 1024) {
    int run = 0;
    for (int w0 = 0; w0 < active; w0 += 8) {
      int c[8];
#pragma unroll
      for (int w = 0; w < 8; w++) c[w] = w0 + w < active ? table[(w0 + w) * keys + k] : 0;
#pragma unroll
      for (int w = 0; w < 8; w++) {
        if (w0 + w < active) table[(w0 + w) * keys + k] = run;
        run += c[w];
      }
    }
    s.total[k] = run;
  }
  if (ctas > 1)
    cluster.sync();
  else
    __syncthreads();
  // per group: rows in the CTAs before, and in all; then the groups' prefix
  // (thread k has group k, the last thread the rows of no group as well)
  int below = 0, all = 0, none_below = 0;
  auto sums = [&](int k, int& lo, int& sum) {
    if (ctas == 1) {
      sum = s.total[k];
      return;
    }
    int c[kSortCtas];
#pragma unroll
    for (int i = 0; i < kSortCtas; i++) c[i] = *cluster.map_shared_rank(&s.total[k], i);
#pragma unroll
    for (int i = 0; i < kSortCtas; i++) {
      if (i < rank) lo += c[i];
      sum += c[i];
    }
  };
  if (tid < G) sums(tid, below, all);
  if (tid == 1023) {
    int none = 0;
    sums(G, none_below, none);
  }
  int inc = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s.scan[warp] = inc;
  if (ctas > 1)
    cluster.sync();  // the totals have been read everywhere
  else
    __syncthreads();
  int warps = s.scan[lane];  // every warp scans the warps' sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, warps, o);
    if (lane >= o) warps += v;
  }
  const int sum = __shfl_sync(0xffffffffu, warps, 31);
  const int run = (warp ? __shfl_sync(0xffffffffu, warps, warp - 1) : 0) + inc - all;
  if (tid < G) {
    s.total[tid] = run + below;
    if (rank == 0) offsets[tid] = run;
  }
  if (tid == 1023) {
    s.total[G] = sum + none_below;
    if (rank == 0) offsets[G] = sum;
  }
  __syncthreads();
  walk([&](int key, int i, int before, int count) {
    const int at = key >= 0 ? mine[key] : 0;
    __syncwarp();
    if (key >= 0) {
      rows[s.total[key] + at + before] = i;
      if (before == 0) mine[key] = at + count;
    }
  });
}

// ids per warp, and bits of a key, of n ids in G groups on `ctas` CTAs.
inline int sort_stretch(int n, int ctas) { return ((n + ctas * kSortWarps - 1) / (ctas * kSortWarps) + 31) / 32 * 32; }
inline int sort_bits(int n_groups) {
  int bits = 1;
  while (n_groups >> bits) bits++;
  return bits;
}
inline size_t sort_bytes(int n, int n_groups, int stretch) {
  const int warps = n < kSortWarps * stretch ? (n + stretch - 1) / stretch : kSortWarps;
  return sizeof(SortSide) + sizeof(int) * (size_t)warps * (n_groups + 1);
}

}  // namespace moe
