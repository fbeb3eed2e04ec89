// grouped.cu -- products over ragged groups of rows (expert products of
// prompts, per-request adapters) on the tensor cores.
//
// D[channel, row] = sum_k W_g[channel, k] x[row, k]: the weights are the A
// operand (channels are the lanes of the accumulator), the rows of a group
// the B operand (its columns).  The groups are ragged, and a column count may
// be any multiple of 32, so a tile pads a group by 31 rows at most; with the
// rows as lanes it would pad by up to 255.
//
// A pair of CTAs works on 256 channels by up to 256 rows: each CTA holds the
// operands of its own 128 channels and of half of the rows, which halves what
// a CTA has to fetch for the rows (32 KB instead of 48 KB for 128 x 256 x 64
// multiply-adds).  The pairs walk the tiles (group, rows, channels).  In each CTA
// warp 0 fetches boxes by bulk tensor copies into a ring of stages; warps
// 8 .. 11 fetch the rows where they are gathered through the plan's row list
// (16-byte copies; gathering bulk copies move four rows in about 80 cycles,
// a third of the rate that the products need); one thread of the pair's first CTA issues the
// products; warps 4 .. 7 read the accumulator back, transform and store.  Two
// accumulators let that overlap the next tile's products.
//
// For SwiGLU a CTA's 128 lanes are 64 gate and the same 64 up channels; the
// warps of a gate and an up quarter swap half of their columns through shared
// memory.
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

constexpr int kGThreads = 384;
constexpr int kLanes = 128;                // channels per CTA (gate and up together)
constexpr int kBlockK = 64;                // K per stage: one 128-byte swizzled row
constexpr int kMaxCols = 256;              // rows per tile
constexpr int kABytes = kLanes * kBlockK * 2;
constexpr int kMaxStages = 8;
constexpr int kRowBoxes = 4;               // boxes of 128, 64, 32 and 16 rows
constexpr int kSmemBudget = 227 * 1024 - 1024;  // 1024: the ring's alignment

struct Maps {
  CUtensorMap x[kRowBoxes], w, w_up;
};

struct TileArgs {
  int G, P, n_x, n_y, N, K, ldx, ldy;
  int cols;      // rows per tile at most (multiple of 32)
  int stages, stage_bytes;
  int layout, gather, x_div, y_fp32;
  const uint16_t* x;
  const int32_t* x_rows;
  const int32_t* offsets;
  const int32_t* y_rows;
  void* y;
  uint32_t* err;
};

// Shared memory behind the ring.
struct Side {
  uint64_t full[kMaxStages], landed[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int stop, tiles;
  int scan[kGThreads / 32];
  alignas(16) int y_row[kMaxCols];  // result row of each column, -1: none; even columns, then odd ones
  float swap[2][2][2][16][32];      // [quarter][turn][from the up side][column][lane]
  int first[kMaxGroups];            // first sorted position of each group
  int rows[kMaxGroups];             // rows of each group
  int before[kMaxGroups + 1];       // row tiles of the groups before
};

// A role's place in the ring: the stage, and how often it has gone round.
struct Turn {
  int st = 0, round = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++st == stages) {
      st = 0;
      round ^= 1;
    }
  }
};

// Checks the plan and lays its groups out as row tiles; every thread of the CTA.
__device__ void lay_tiles(const TileArgs& a, Side& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kPer = (kMaxGroups + kGThreads - 1) / kGThreads;
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
  // a group's row tiles are as even as steps of 32 allow
  const int rows = s.rows[lo], nt = (rows + a.cols - 1) / a.cols;
  const int size = ((rows + nt - 1) / nt + 31) & ~31, at = (q - s.before[lo]) * size;
  Tile t;
  t.g = lo;
  t.p0 = s.first[lo] + at;
  t.n = min(size, rows - at);
  t.c0 = u - q * n_ct;
  return t;
}

// The rows of x at sorted positions, gathered: thread i of 128 copies the
// 16-byte piece i % 8 of rows i / 8 + 16 m of this CTA's half of the tile.  A
// stage's copies arrive on landed[stage] as they complete; warp 3 passes that
// on to the issuing CTA, so that the copying threads never wait for their copies.
__device__ void gather_rows(const TileArgs& a, Side& s, uint8_t* ring, int units, int n_ct, int nkb, int rank) {
  const int t = threadIdx.x - 256, piece = t & 7, r0 = t >> 3;
  volatile int* stop = &s.stop;
  Turn it;
  bool ok = true;
  for (int u = blockIdx.x >> 1; u < units && ok; u += gridDim.x >> 1) {
    const Tile tl = tile_of(a, s, u, n_ct);
    const int half = ((tl.n + 31) & ~31) >> 1;
    const uint16_t* src[8];
#pragma unroll
    for (int m = 0; m < 8; m++) {
      // rows past the tile's end repeat its last one (their columns are not stored)
      int row = 0;
      if (r0 + 16 * m < half) {
        row = a.x_rows[tl.p0 + min(rank * half + r0 + 16 * m, tl.n - 1)];
        row = row < 0 ? -1 : row / a.x_div;
        if (row < 0 || row >= a.n_x) {
          atomicOr(a.err, kErrBadPlan);
          row = 0;
        }
      }
      src[m] = a.x + (size_t)row * a.ldx + piece * 8;
    }
    for (int kb = 0; kb < nkb; kb++, it.next(a.stages)) {
      const int st = it.st;
      ok = wait_or_stop(&s.empty[st], it.round ^ 1, stop, a.err);
      if (__any_sync(0xffffffffu, !ok)) {
        ok = false;
        break;
      }
      const uint32_t dst = smem_u32(ring + (size_t)st * a.stage_bytes + kABytes) + r0 * 128 + ((piece ^ (r0 & 7)) << 4);
      const bool in = kb * kBlockK + piece * 8 < a.K;
#pragma unroll
      for (int m = 0; m < 8; m++)
        if (r0 + 16 * m < half) cp_async16(dst + m * 2048, in ? src[m] + kb * kBlockK : a.x, in);
      cp_async_arrive(&s.landed[st]);
    }
  }
  cp_async_wait_all();
}

// Passes each stage of gathered rows on: complete here, made visible to the
// tensor cores, announced to the issuing CTA.
__device__ void announce_rows(const TileArgs& a, Side& s, int units, int nkb) {
  const uint32_t full = peer_u32(s.full, 0);
  Turn it;
  for (int u = blockIdx.x >> 1; u < units; u += gridDim.x >> 1)
    for (int kb = 0; kb < nkb; kb++, it.next(a.stages)) {
      if (!wait_or_stop(&s.landed[it.st], it.round, &s.stop, a.err)) return;
      fence_proxy_async();
      mbar_arrive_at(full + it.st * 8);
    }
}

template <bool kSwiglu>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGThreads, 1)
    tiles_kernel(const __grid_constant__ Maps maps, const TileArgs a) {
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  Side& s = *reinterpret_cast<Side*>(ring + (size_t)a.stages * a.stage_bytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x & 1;
  constexpr int kChan = kSwiglu ? kLanes / 2 : kLanes;  // output channels per CTA
  if (tid == 0) {
    for (int i = 0; i < a.stages; i++) {
      mbar_init(&s.full[i], a.gather ? 3 : 1);  // the boxes' announcement, and the gathered rows' of each CTA
      mbar_init(&s.landed[i], 128);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], 8);  // four warps of each CTA
    }
    mbar_init(&s.drain, 1);
    s.stop = 0;
    fence_mbar_init();
    for (int i = 0; i < kRowBoxes; i++) tma_prefetch(&maps.x[i]);
    tma_prefetch(&maps.w);
    if (kSwiglu) tma_prefetch(&maps.w_up);
  }
  if (warp == 2) tmem_alloc(&s.tmem, 512);
  pdl_trigger();
  pdl_wait();
  tc_fence_before();
  lay_tiles(a, s);
  cluster_arrive();
  cluster_wait();  // the pair's barriers are ready
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  const int n_ct = (a.N + 2 * kChan - 1) / (2 * kChan), units = s.tiles * n_ct, nkb = (a.K + kBlockK - 1) / kBlockK;
  const int u0 = blockIdx.x >> 1, du = gridDim.x >> 1;
  volatile int* stop = &s.stop;

  if ((warp == 0 || (warp == 2 && !a.gather)) && lane == 0) {
    // ----------------------- boxes: the weights (warp 0), the rows (warp 2)
    const bool rows = warp == 2;
    Turn it;
    int filled = 0;
    bool ok = true;
    const uint32_t full = peer_u32(s.full, 0);
    for (int u = u0; u < units && ok; u += du) {
      const Tile t = tile_of(a, s, u, n_ct);
      const int half = ((t.n + 31) & ~31) >> 1, c0 = (t.c0 * 2 + rank) * kChan, p = t.p0 + rank * half;
      const uint32_t bytes = 2 * (kABytes + (a.gather ? 0 : half * 128));  // of both CTAs
      for (int k0 = 0; k0 < a.K; k0 += kBlockK, it.next(a.stages), filled++) {
        ok = wait_or_stop(&s.empty[it.st], it.round ^ 1, stop, a.err);
        if (!ok) break;
        uint8_t* A = ring + (size_t)it.st * a.stage_bytes;
        const uint32_t bar = full + it.st * 8;
        if (rows) {
          uint8_t* B = A + kABytes;
          if (half == 128) {
            tma_2d(B, &maps.x[0], k0, p, bar);
          } else {
            int at = 0;
#pragma unroll
            for (int b = 1; b < kRowBoxes; b++) {
              const int h = 128 >> b;
              if (half & h) {
                tma_2d(B + at * 128, &maps.x[b], k0, p + at, bar);
                at += h;
              }
            }
          }
          continue;
        }
        if (rank == 0) mbar_expect_tx(&s.full[it.st], bytes);
        if (kSwiglu) {
          tma_3d(A, &maps.w, k0, c0, t.g, bar);
          tma_3d(A + kABytes / 2, &maps.w_up, k0, c0, t.g, bar);
        } else if (a.layout) {
          tma_3d(A, &maps.w, c0, k0, t.g, bar);
          tma_3d(A + kABytes / 2, &maps.w, c0 + 64, k0, t.g, bar);
        } else {
          tma_3d(A, &maps.w, k0, c0, t.g, bar);
        }
      }
    }
    // after a timeout: the copies in flight must land before the pair ends
    if (!ok && rank == 0)
      for (int i = filled > a.stages ? filled - a.stages : 0; i < filled; i++)
        mbar_wait_bounded(&s.full[i % a.stages], (i / a.stages) & 1, a.err);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // -------------------------------------------------------- products
    Turn it;
    int ti = 0;
    bool ok = true;
    for (int u = u0; u < units && ok; u += du, ti++) {
      const Tile t = tile_of(a, s, u, n_ct);
      const uint32_t d = tmem + (ti & 1) * kMaxCols;
      const uint32_t idesc = mma_desc(2 * kLanes, (t.n + 31) & ~31, !kSwiglu && a.layout);
      ok = wait_or_stop(&s.acc_empty[ti & 1], ((ti >> 1) & 1) ^ 1, stop, a.err);
      if (!ok) break;
      tc_fence_after();
      for (int kb = 0; kb < nkb; kb++, it.next(a.stages)) {
        const int st = it.st;
        ok = wait_or_stop(&s.full[st], it.round, stop, a.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t A = smem_u32(ring + (size_t)st * a.stage_bytes);
        const uint64_t bd = tile_desc(A + kABytes, 16);
        const int steps = (min(kBlockK, a.K - kb * kBlockK) + 15) / 16;  // past K the stage holds zeros
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
    if (!ok) {  // after a timeout: the products in flight must end before the pair does
      mma_commit(&s.drain);
      mbar_wait_bounded(&s.drain, 0, a.err);
    }
  } else if (warp == 3 && lane == 0) {
    if (a.gather) announce_rows(a, s, units, nkb);
  } else if (warp >= 8) {
    if (a.gather) gather_rows(a, s, ring, units, n_ct, nkb, rank);
  } else if (warp >= 4) {
    // ------------------------------------------------- read back, store
    const int q4 = warp - 4, et = tid - 128;
    const bool odd = lane & 1;
    int ti = 0, turn = 0;
    for (int u = u0; u < units; u += du, ti++) {
      const Tile t = tile_of(a, s, u, n_ct);
      for (int j = et; j < ((t.n + 31) & ~31); j += 128) {
        int q = -1;
        if (j < t.n) {
          q = a.y_rows ? a.y_rows[t.p0 + j] : t.p0 + j;
          if (q < 0 || q >= a.n_y) {
            atomicOr(a.err, kErrBadPlan);
            q = -1;
          }
          if (a.gather) {  // a row that is not there has no result
            const int row = a.x_rows[t.p0 + j];
            if (row < 0 || row / a.x_div >= a.n_x) q = -1;
          }
        }
        s.y_row[(j & 1) * (kMaxCols / 2) + (j >> 1)] = q;
      }
      const bool ok = wait_or_stop(&s.acc_full[ti & 1], (ti >> 1) & 1, stop, a.err);
      if (bar_any(1, 128, !ok)) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q4 * 32) << 16) + (ti & 1) * kMaxCols;
      for (int j0 = 0; j0 < t.n; j0 += 32) {
        float v[32];
        tmem_ld32(acc + j0, v);
        if (kSwiglu) {
          // the gate side finishes the even columns, the up side the odd ones
          const bool up = q4 >= 2;
          float(&out)[16][32] = s.swap[q4 & 1][turn][up ? 1 : 0];
          float(&in)[16][32] = s.swap[q4 & 1][turn][up ? 0 : 1];
          turn ^= 1;
#pragma unroll
          for (int i = 0; i < 16; i++) out[i][lane] = up ? v[2 * i] : v[2 * i + 1];
          bar_any(2 + (q4 & 1), 64, false);
          float r[16];
#pragma unroll
          for (int i = 0; i < 16; i++) {
            const float o = in[i][lane], g = up ? o : v[2 * i], w = up ? v[2 * i + 1] : o;
            r[i] = __fdividef(g, 1.0f + __expf(-g)) * w;
          }
          const int* q_of = s.y_row + (up ? kMaxCols / 2 : 0) + (j0 >> 1);
          const int cw = (t.c0 * 2 + rank) * kChan + (q4 & 1) * 32;
          uint16_t* y = static_cast<uint16_t*>(a.y);
          if (a.ldy & 1) {  // rows that start on odd words
            const int c = cw + lane;
#pragma unroll
            for (int i = 0; i < 16; i++) {
              const int q = q_of[i];
              if (q >= 0 && c < a.N) y[(size_t)q * a.ldy + c] = f2bf16(r[i]);
            }
          } else {
            const int c = cw + (lane & ~1);
            if (c < a.N) y += c;
            const bool in_n = c < a.N;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float o = __shfl_xor_sync(0xffffffffu, odd ? r[i] : r[i + 1], 1);
              const uint32_t w = odd ? bf16x2(o, r[i + 1]) : bf16x2(r[i], o);
              const int q = q_of[i + (odd ? 1 : 0)];
              if (q >= 0 && in_n) *reinterpret_cast<uint32_t*>(y + (size_t)q * a.ldy) = w;
            }
          }
        } else if (a.y_fp32) {
          const int c = (t.c0 * 2 + rank) * kChan + q4 * 32 + lane;
          const bool in_n = c < a.N;
          float* y = static_cast<float*>(a.y) + c;
#pragma unroll
          for (int j = 0; j < 32; j++) {
            const int q = s.y_row[(j & 1) * (kMaxCols / 2) + ((j0 + j) >> 1)];
            if (q >= 0 && in_n) y[(size_t)q * a.ldy] = v[j];
          }
        } else {
          // two channels to a word: the even lane of a pair takes the even column
          const int c = (t.c0 * 2 + rank) * kChan + q4 * 32 + (lane & ~1);
          const bool in_n = c < a.N;
          uint16_t* y = static_cast<uint16_t*>(a.y) + c;
          const int4* q_of = reinterpret_cast<const int4*>(s.y_row + (odd ? kMaxCols / 2 : 0) + (j0 >> 1));
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int4 q = q_of[i];
            const int qs[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
              const int j = 8 * i + 2 * k;
              const float o = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
              const uint32_t w = odd ? bf16x2(o, v[j + 1]) : bf16x2(v[j], o);
              if (qs[k] >= 0 && in_n) *reinterpret_cast<uint32_t*>(y + (size_t)qs[k] * a.ldy) = w;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(peer_u32(&s.acc_empty[ti & 1], 0));
      bar_any(1, 128, false);  // y_row is rewritten for the next tile
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();  // neither CTA leaves while the other may still signal it
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
  t.stage_bytes = kABytes + t.cols / 2 * 128;
  t.stages = (kSmemBudget - (int)sizeof(Side)) / t.stage_bytes;
  if (t.stages > kMaxStages) t.stages = kMaxStages;
  const size_t smem = 1024 + (size_t)t.stages * t.stage_bytes + sizeof(Side);
  cudaError_t e = cudaFuncSetAttribute(tiles_kernel<kSwiglu>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int chan = kSwiglu ? kLanes : 2 * kLanes, n_ct = (t.N + chan - 1) / chan;
  const long most = ((long)(t.P + t.cols - 1) / t.cols + (t.G < t.P ? t.G : t.P)) * n_ct;  // units at most
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * (most < sms / 2 ? most : sms / 2)));
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
  t.x = a.x;
  t.ldx = a.ldx;
  Maps m;
  const uint64_t N = a.N, K = a.K;
  bool ok = true;
  for (int b = 0; b < kRowBoxes; b++)
    ok = ok && tensor_map(&m.x[b], a.x, K, a.n_x, 0, 2ull * a.ldx, 0, kBlockK, 128 >> b);
  if (a.w_up) {
    ok = ok && tensor_map(&m.w, a.w, K, N, a.G, 2 * K, 2 * N * K, kBlockK, kLanes / 2) &&
         tensor_map(&m.w_up, a.w_up, K, N, a.G, 2 * K, 2 * N * K, kBlockK, kLanes / 2);
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
