// grouped.cu -- products over ragged groups of rows (expert products of
// prompts, per-request adapters) on the tensor cores.
//
// D[channel, row] = sum_k W_g[channel, k] x[row, k]: the weights are the A
// operand (128 channels, the lanes of the accumulator), the rows of a group
// the B operand (its columns).  The groups are ragged, and a column count may
// be any multiple of 16, so a tile pads a group by 15 rows at most; with the
// rows as lanes it would pad by up to 127.  For SwiGLU the 32 lanes of each
// warp hold 16 gate and the 16 up channels they belong with, so that a value
// and its gate meet in one shuffle.
//
// One CTA per SM walks the tiles (group, rows, channels).  Warp 0 fills a
// ring of shared-memory stages by bulk tensor copies (weights in boxes, rows
// in boxes or gathered four at a time through the plan's row list), one
// thread of warp 1 issues the products, warps 4 .. 7 read the accumulator
// back, transform and store; two accumulators let that overlap the next
// tile's products.
#include <cudaTypedefs.h>

#include "kernels.h"
#include "tensor.cuh"

namespace moe {

bool tensor_map(CUtensorMap* m, const void* base, uint64_t x, uint64_t y, uint64_t z, uint64_t row_bytes,
                uint64_t mat_bytes, uint32_t box_x, uint32_t box_y) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return (PFN_cuTensorMapEncodeTiled_v12000) nullptr;
    }
    return (PFN_cuTensorMapEncodeTiled_v12000)f;
  }();
  if (!encode) return false;
  const cuuint64_t dims[3] = {x, y, z}, strides[2] = {row_bytes, mat_bytes};
  const cuuint32_t box[3] = {box_x, box_y, 1}, step[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, z ? 3 : 2, const_cast<void*>(base), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr int kGThreads = 256;
constexpr int kLanes = 128;                // channels per tile (gate and up together)
constexpr int kBlockK = 64;                // K per stage: one 128-byte swizzled row
constexpr int kMaxCols = 256;              // rows per tile
constexpr int kABytes = kLanes * kBlockK * 2;
constexpr int kMaxStages = 8;
constexpr int kBoxRows = 32;               // rows per box of an ungathered x
constexpr int kSmemBudget = 227 * 1024 - 1024;  // 1024: the ring's alignment

struct Maps {
  CUtensorMap x, w, w_up;
};

struct TileArgs {
  int G, P, n_x, n_y, N, K, ldy;
  int cols;      // rows per tile at most (multiple of 32)
  int stages, stage_bytes;
  int layout, gather, x_div, y_fp32;
  const int32_t* x_rows;
  const int32_t* offsets;
  const int32_t* y_rows;
  void* y;
  uint32_t* err;
};

// Shared memory behind the ring.
struct Side {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int stop, tiles;
  int scan[kGThreads / 32];
  int y_row[kMaxCols];
  int first[kMaxGroups];       // first sorted position of each group
  int rows[kMaxGroups];        // rows of each group
  int before[kMaxGroups + 1];  // row tiles of the groups before
};

// Checks the plan and lays its groups out as row tiles; every thread of the CTA.
__device__ void lay_tiles(const TileArgs& a, Side& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kPer = kMaxGroups / kGThreads;
  int n[kPer], t[kPer], sum = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int g = tid * kPer + i;
    n[i] = t[i] = 0;
    if (g < a.G) {
      const int p0 = a.offsets[g], p1 = a.offsets[g + 1];
      bad |= p0 < 0 || p1 < p0 || p1 > a.P;
      n[i] = p1 - p0;
      t[i] = bad ? 0 : (n[i] + a.cols - 1) / a.cols;
      s.first[g] = p0;
      s.rows[g] = n[i];
    }
    sum += t[i];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s.scan[warp] = inc;
  bad = __syncthreads_or(bad);
  int run = inc - sum;
  for (int w = 0; w < warp; w++) run += s.scan[w];
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int g = tid * kPer + i;
    if (g < a.G) s.before[g] = run;
    run += t[i];
    if (g == a.G - 1) {
      s.before[a.G] = run;
      s.tiles = bad ? 0 : run;  // offsets that do not ascend within the rows: nothing is computed
      if (bad) atomicOr(a.err, kErrBadPlan);
    }
  }
  __syncthreads();
}

struct Tile {
  int g, p0, n, c0;  // group, first sorted position, rows, channel tile
};
// Unit u of the walk: the channel tiles of a row tile follow one another (they
// share its rows), the row tiles of a group too (they share its weights).
__device__ __forceinline__ Tile tile_of(const TileArgs& a, const Side& s, int u, int n_ct) {
  const int q = u / n_ct;
  int lo = 0, hi = a.G - 1;  // the last group with before[g] <= q
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (s.before[m] <= q)
      lo = m;
    else
      hi = m - 1;
  }
  // a group's row tiles are as even as steps of 16 allow
  const int rows = s.rows[lo], nt = (rows + a.cols - 1) / a.cols;
  const int size = ((rows + nt - 1) / nt + 15) & ~15, at = (q - s.before[lo]) * size;
  Tile t;
  t.g = lo;
  t.p0 = s.first[lo] + at;
  t.n = min(size, rows - at);
  t.c0 = u - q * n_ct;
  return t;
}

template <bool kSwiglu>
__global__ void __launch_bounds__(kGThreads, 1) tiles_kernel(const __grid_constant__ Maps maps, const TileArgs a) {
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  Side& s = *reinterpret_cast<Side*>(ring + (size_t)a.stages * a.stage_bytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kChan = kSwiglu ? kLanes / 2 : kLanes;  // output channels per tile
  if (tid == 0) {
    for (int i = 0; i < a.stages; i++) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], 4);
    }
    mbar_init(&s.drain, 1);
    s.stop = 0;
    fence_mbar_init();
    tma_prefetch(&maps.x);
    tma_prefetch(&maps.w);
    if (kSwiglu) tma_prefetch(&maps.w_up);
  }
  if (warp == 2) tmem_alloc(&s.tmem, 512);
  pdl_trigger();
  pdl_wait();
  tc_fence_before();
  lay_tiles(a, s);
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  const int n_ct = (a.N + kChan - 1) / kChan, units = s.tiles * n_ct, nkb = (a.K + kBlockK - 1) / kBlockK;
  volatile int* stop = &s.stop;

  if (warp == 0) {
    // ---------------------------------------------------------- copies
    int it = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const Tile t = tile_of(a, s, u, n_ct);
      const int quads = (t.n + 15) / 16 * 4, boxes = (t.n + kBoxRows - 1) / kBoxRows;
      const uint32_t bytes = kABytes + (a.gather ? quads * 4 : boxes * kBoxRows) * 128;
      int r[2][4];
      if (a.gather) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            // rows past the tile's end repeat its last one (their columns are not stored)
            const int j = min((lane + 32 * h) * 4 + i, t.n - 1);
            int row = a.x_rows[t.p0 + j];
            row = row < 0 ? -1 : row / a.x_div;
            if (row < 0 || row >= a.n_x) {
              atomicOr(a.err, kErrBadPlan);
              row = 0;
            }
            r[h][i] = row;
          }
      }
      for (int kb = 0; kb < nkb; kb++, it++) {
        const int st = it % a.stages;
        ok = wait_or_stop(&s.empty[st], ((it / a.stages) & 1) ^ 1, stop, a.err);
        if (__any_sync(0xffffffffu, !ok)) {
          ok = false;
          break;
        }
        uint8_t* A = ring + (size_t)st * a.stage_bytes;
        uint8_t* B = A + kABytes;
        const int k0 = kb * kBlockK;
        if (lane == 0) {
          mbar_expect_tx(&s.full[st], bytes);
          if (kSwiglu) {
#pragma unroll
            for (int q = 0; q < 4; q++) {
              tma_3d(A + q * 4096, &maps.w, k0, t.c0 * kChan + q * 16, t.g, &s.full[st]);
              tma_3d(A + q * 4096 + 2048, &maps.w_up, k0, t.c0 * kChan + q * 16, t.g, &s.full[st]);
            }
          } else if (a.layout) {
            tma_3d(A, &maps.w, t.c0 * kChan, k0, t.g, &s.full[st]);
            tma_3d(A + kABytes / 2, &maps.w, t.c0 * kChan + 64, k0, t.g, &s.full[st]);
          } else {
            tma_3d(A, &maps.w, k0, t.c0 * kChan, t.g, &s.full[st]);
          }
          if (!a.gather)
            for (int b = 0; b < boxes; b++)
              tma_2d(B + b * kBoxRows * 128, &maps.x, k0, t.p0 + b * kBoxRows, &s.full[st]);
        }
        __syncwarp();
        if (a.gather) {
#pragma unroll
          for (int h = 0; h < 2; h++)
            if (lane + 32 * h < quads) tma_gather4(B + (lane + 32 * h) * 512, &maps.x, k0, r[h], &s.full[st]);
        }
        __syncwarp();
      }
    }
    // after a timeout: the copies in flight must land before the CTA ends
    if (!ok && lane == 0)
      for (int i = it > a.stages ? it - a.stages : 0; i < it; i++)
        mbar_wait_bounded(&s.full[i % a.stages], (i / a.stages) & 1, a.err);
  } else if (warp == 1 && lane == 0) {
    // -------------------------------------------------------- products
    int it = 0, ti = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x, ti++) {
      const Tile t = tile_of(a, s, u, n_ct);
      const uint32_t d = tmem + (ti & 1) * kMaxCols;
      const uint32_t idesc = mma_desc(kLanes, (t.n + 15) & ~15, !kSwiglu && a.layout);
      ok = wait_or_stop(&s.acc_empty[ti & 1], ((ti >> 1) & 1) ^ 1, stop, a.err);
      if (!ok) break;
      tc_fence_after();
      for (int kb = 0; kb < nkb; kb++, it++) {
        const int st = it % a.stages;
        ok = wait_or_stop(&s.full[st], (it / a.stages) & 1, stop, a.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t A = smem_u32(ring + (size_t)st * a.stage_bytes);
        const uint64_t bd = tile_desc(A + kABytes, 16);
        const int steps = min(kBlockK, a.K - kb * kBlockK + 15) / 16;  // past K the stage holds zeros
        if (!kSwiglu && a.layout) {
          const uint64_t ad = tile_desc(A, kABytes / 2);
          for (int k = 0; k < steps; k++) mma_bf16(d, ad + k * (2048 >> 4), bd + k * 2, idesc, kb + k > 0);
        } else {
          const uint64_t ad = tile_desc(A, 16);
          for (int k = 0; k < steps; k++) mma_bf16(d, ad + k * 2, bd + k * 2, idesc, kb + k > 0);
        }
        mma_commit(&s.empty[st]);
      }
      if (ok) mma_commit(&s.acc_full[ti & 1]);
    }
    if (!ok) {  // after a timeout: the products in flight must end before the CTA does
      mma_commit(&s.drain);
      mbar_wait_bounded(&s.drain, 0, a.err);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------- read back, store
    const int q4 = warp - 4, et = tid - 128;
    int ti = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, ti++) {
      const Tile t = tile_of(a, s, u, n_ct);
      for (int j = et; j < t.n; j += 128) {
        int q = a.y_rows ? a.y_rows[t.p0 + j] : t.p0 + j;
        if (q < 0 || q >= a.n_y) {
          atomicOr(a.err, kErrBadPlan);
          q = -1;
        }
        if (a.gather) {  // a row that is not there has no result
          const int row = a.x_rows[t.p0 + j];
          if (row < 0 || row / a.x_div >= a.n_x) q = -1;
        }
        s.y_row[j] = q;
      }
      const bool ok = wait_or_stop(&s.acc_full[ti & 1], (ti >> 1) & 1, stop, a.err);
      if (bar_any(1, 128, !ok)) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q4 * 32) << 16) + (ti & 1) * kMaxCols;
      for (int j0 = 0; j0 < t.n; j0 += 32) {
        float v[32];
        tmem_ld32(acc + j0, v);
        if (kSwiglu) {
          // lanes 0..15 hold the gates, 16..31 the ups of channels c: the lower
          // half finishes the even column of a pair, the upper half the odd one
          const int c = t.c0 * kChan + q4 * 16 + (lane & 15);
          const bool up = lane >= 16;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float o = __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j + 1], 16);
            const float g = up ? o : v[j], w = up ? v[j + 1] : o;
            const int jj = j0 + j + (up ? 1 : 0);
            if (jj < t.n && c < a.N) {
              const int q = s.y_row[jj];
              if (q >= 0)
                static_cast<uint16_t*>(a.y)[(size_t)q * a.ldy + c] = f2bf16(__fdividef(g, 1.0f + __expf(-g)) * w);
            }
          }
        } else if (a.y_fp32) {
          const int c = t.c0 * kChan + q4 * 32 + lane;
#pragma unroll
          for (int j = 0; j < 32; j++)
            if (j0 + j < t.n && c < a.N) {
              const int q = s.y_row[j0 + j];
              if (q >= 0) static_cast<float*>(a.y)[(size_t)q * a.ldy + c] = v[j];
            }
        } else {
          // two channels to a word: the even lane of a pair takes the even column
          const int c = t.c0 * kChan + q4 * 32 + (lane & ~1);
          const bool odd = lane & 1;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float o = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
            const uint32_t w = odd ? f2bf16(o) | ((uint32_t)f2bf16(v[j + 1]) << 16)
                                   : f2bf16(v[j]) | ((uint32_t)f2bf16(o) << 16);
            const int jj = j0 + j + (odd ? 1 : 0);
            if (jj < t.n && c < a.N) {
              const int q = s.y_row[jj];
              if (q >= 0) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.y) + (size_t)q * a.ldy + c) = w;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.acc_empty[ti & 1]);
      bar_any(1, 128, false);  // y_row is rewritten for the next tile
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) tmem_free(tmem, 512);
}

// One CTA per (token position, 256 channels).
__global__ void __launch_bounds__(256) adapter_kernel(AdapterArgs a) {
  extern __shared__ float sh[];
  float* xs = sh;        // [K]
  float* z = sh + a.K;   // [r]
  const int p = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = a.rows[p];
  if (t < 0 || t >= a.T) {
    if (tid == 0) atomicOr(a.err, kErrBadPlan);
    return;
  }
  int lo = 0, hi = a.A;  // the first group that ends behind p
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (a.offsets[m + 1] > p) hi = m; else lo = m + 1;
  }
  const int g = lo;
  for (int k = tid; k < a.K; k += 256) xs[k] = bf16f(a.x[(size_t)t * a.K + k]);
  __syncthreads();
  for (int j = warp; j < a.r; j += 8) {
    float s = 0.0f;
    if (g < a.A) {
      for (int k = lane; k < a.K; k += 32) s = fmaf(xs[k], bf16f(a.a[((size_t)g * a.r + j) * a.K + k]), s);
      s = warp_sum(s) * (a.scale ? a.scale[g] : 1.0f);
    }
    if (lane == 0) z[j] = s;
  }
  __syncthreads();
  const int n = blockIdx.y * 256 + tid;
  if (n >= a.N) return;
  float s = 0.0f;
  if (a.w)
    for (int k = 0; k < a.K; k++) s = fmaf(xs[k], bf16f(a.w[(size_t)n * a.K + k]), s);
  if (g < a.A)
    for (int j = 0; j < a.r; j++) s = fmaf(z[j], bf16f(a.b[((size_t)g * a.N + n) * a.r + j]), s);
  if (a.base) s += bf16f(a.base[(size_t)t * a.N + n]);
  a.y[(size_t)t * a.N + n] = f2bf16(s);
}

int sm_count() {
  static thread_local int dev_of = -1, count = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev != dev_of) {
    if (cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    dev_of = dev;
  }
  return count;
}

template <bool kSwiglu>
cudaError_t run_tiles(const Maps& m, TileArgs t, cudaStream_t s) {
  t.stage_bytes = kABytes + t.cols * 128;
  t.stages = (kSmemBudget - (int)sizeof(Side)) / t.stage_bytes;
  if (t.stages > kMaxStages) t.stages = kMaxStages;
  const size_t smem = 1024 + (size_t)t.stages * t.stage_bytes + sizeof(Side);
  cudaError_t e = cudaFuncSetAttribute(tiles_kernel<kSwiglu>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int chan = kSwiglu ? kLanes / 2 : kLanes, n_ct = (t.N + chan - 1) / chan;
  const long most = ((long)(t.P + t.cols - 1) / t.cols + (t.G < t.P ? t.G : t.P)) * n_ct;  // units at most
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(most < sms ? most : sms));
  cfg.blockDim = dim3(kGThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tiles_kernel<kSwiglu>, m, t);
}

}  // namespace

cudaError_t launch_grouped(const GroupedArgs& a, cudaStream_t s) {
  TileArgs t = {};
  t.G = a.G;
  t.P = a.P;
  t.n_x = a.n_x;
  t.n_y = a.n_y;
  t.N = a.N;
  t.K = a.K;
  t.ldy = a.ldy;
  t.layout = a.layout;
  t.gather = a.x_rows != nullptr;
  t.x_div = a.x_div;
  t.y_fp32 = a.y_fp32;
  t.x_rows = a.x_rows;
  t.offsets = a.offsets;
  t.y_rows = a.y_rows;
  t.y = a.y;
  t.err = a.err;
  t.cols = a.P < kMaxCols ? (a.P + 31) / 32 * 32 : kMaxCols;
  Maps m;
  const uint64_t N = a.N, K = a.K;
  bool ok = tensor_map(&m.x, a.x, K, a.n_x, 0, 2ull * a.ldx, 0, kBlockK, t.gather ? 1 : kBoxRows);
  if (a.w_up) {
    ok = ok && tensor_map(&m.w, a.w, K, N, a.G, 2 * K, 2 * N * K, kBlockK, 16) &&
         tensor_map(&m.w_up, a.w_up, K, N, a.G, 2 * K, 2 * N * K, kBlockK, 16);
  } else {
    ok = ok && (a.layout ? tensor_map(&m.w, a.w, N, K, a.G, 2 * N, 2 * N * K, 64, kBlockK)
                         : tensor_map(&m.w, a.w, K, N, a.G, 2 * K, 2 * N * K, kBlockK, kLanes));
    m.w_up = m.w;
  }
  if (!ok) return cudaErrorInvalidValue;
  return a.w_up ? run_tiles<true>(m, t, s) : run_tiles<false>(m, t, s);
}

cudaError_t launch_adapter(const AdapterArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(float) * (a.K + a.r);
  cudaError_t e = cudaFuncSetAttribute(adapter_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  adapter_kernel<<<dim3(a.T, (a.N + 255) / 256), 256, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
