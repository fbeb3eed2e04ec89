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
// a third of the rate that the products need); warp 1 of the pair's first CTA issues the
// products; warps 4 .. 7 read the accumulator back, transform and store.  Two
// accumulators let that overlap the next tile's products.
//
// For SwiGLU a CTA's 128 lanes are 64 gate and the same 64 up channels; the
// warps of a gate and an up quarter swap half of their columns through shared
// memory.
//
// Adapters: the tiles run over all tokens, sorted by adapter, and the shared
// projection's sum over K goes on over the adapters that the tile meets, as
// further stages: A is B_g, B the rows of z = scale x A_g^T (adapter.cu), the
// accumulator's columns those of the adapter, widened to multiples of 32 with
// zero rows.  So the low-rank term costs its own bytes and products only.
// For many values of z it comes from these tiles (kLowRank: W_g = A_g, and a
// group's range of positions widened as z's is).
//
// A call with few tiles splits their sums over K: each part is written in
// fp32, and the CTA that arrives last adds them in order and finishes the tile.
//
// What bounds it: few rows a group, the weights' bytes (128 experts of 768 x
// 2048, gate and up, 4 rows each: 134 us, 6.0 TB/s); many, the stages' way
// through a ring that holds 192 KB a CTA (512 rows each: 340 us, 1214 TFLOP/s,
// where a batched library product of the same shape, without the SwiGLU, takes
// 314; 388 us gathered), and in a row of calls the power limit (about 1.0 GHz at 990 W).  Copies of
// the weights into L2 ahead of the ring made every size slower, since they
// cost the copy engine as much as the copies themselves; so did tiles sorted by
// size, for few rows by more than the better balance gave for many.
#include <cudaTypedefs.h>

#include "kernels.h"
#include "tensor.cuh"

namespace moe {

bool tensor_map(CUtensorMap* m, const void* base, uint64_t x, uint64_t y, uint64_t z, uint64_t row_bytes,
                uint64_t mat_bytes, uint32_t box_x, uint32_t box_y, uint32_t box_z) {
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
  const cuuint32_t box[3] = {box_x, box_y, box_z}, step[3] = {1, 1, 1};
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
constexpr int kMaxPairs = 74;              // CTA pairs of a launch
constexpr int kMaxSplit = 8;               // parts of a tile's sum
// Where z comes from: adapter.cu takes 16 rows at a time and reads A_g again
// for each, so its time goes with T r K and it leaves the tiles that follow
// less shared memory; z's tiles cost the same at any rank, and a wave of their
// own.  Whole calls, adapter.cu against tiles: rank 64, K = N = 2048, 8
// adapters, 2048 tokens 35.4 against 46.1 us, 3000 49.2 against 47.2, 8000 110
// against 91; rank 16 4100 tokens 45.9 against 60.2, 8000 81.7 against 91.9;
// rank 128 2048 tokens 41.3 against 46.3.  K = 4096 beside 4096 channels, rank
// 16, 2500 tokens 116 against 103, 4100 146 against 160, 8000 240 against 231.
bool few_values(long T, int r, int K) {
  return T <= 2048 || (T * r <= 2048 * 64 && K <= 2048);
}
// Stages of K that a part has at least (one token, 2048 x 2048: 12.8 us at 8,
// 13.2 at 4, 17.8 without parts; K = 512: 10.3 without, 11.1 with two).
constexpr int kMinPart = 8;
constexpr int kRowBoxes = 4;               // boxes of 128, 64, 32 and 16 rows
constexpr int kSmemBudget = 227 * 1024 - 1024;  // 1024: the ring's alignment

enum Mode { kPlain, kSwiglu, kAdapter, kLowRank };

struct Maps {
  CUtensorMap x[kRowBoxes], w, w_up;
  CUtensorMap x_rest[kRowBoxes];  // x in two terms
  CUtensorMap z[kRowBoxes], z2, b;  // adapters (z2: 16 rows of both halves)
};

struct TileArgs {
  int G, P, n_x, n_y, N, K, ldx, ldy;
  int cols;      // rows per tile at most (multiple of 32)
  int b_rows;    // rows a stage has room for, per CTA
  int stages, stage_bytes;
  int layout, gather, x_div, y_fp32;
  int max_split;
  int late_trigger;       // the next launch starts once everything before this one is complete
  int two_terms;          // x is the sum of x and x_rest (in boxes)
  const uint16_t* x;
  const int32_t* x_rows;
  const int32_t* offsets;
  const int32_t* y_rows;
  void* y;
  uint16_t* y_rest;       // kSwiglu: what the rounding of y leaves, or null
  uint32_t* err;
  uint32_t* count;        // [kMaxPairs][2] arrivals of a split tile's parts
  float* part;            // [kMaxPairs][2][cols / 4][128][4] the parts (four columns of a lane together)
  // adapters (G of them; the tiles run over all P rows)
  int r, has_w;
  const uint16_t* base;
  const uint16_t* w;      // as Maps has them
  const uint16_t* z;
  const uint16_t* b;
  const float* scale;     // kLowRank
  size_t z_half;          // elements of one of z's halves
};

// Shared memory behind the ring.
struct Side {
  uint64_t full[kMaxStages], landed[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int stop, tiles, last;
  unsigned long long scan[kGThreads / 32];
  alignas(16) int y_row[kMaxCols];  // result row of each column, -1: none; even columns, then odd ones
  int first[kMaxGroups];            // first sorted position of each group
  int rows[kMaxGroups];             // rows of each group
  int before[kMaxGroups];           // row tiles of the groups before (adapters: rows of z before)
  int z_before[kMaxGroups];         // kLowRank: rows of z before
  float swap[2][2][2][16][32];      // kSwiglu: [quarter][turn][from the up side][column][lane]
};

// What a mode's launch has of it (swap is last).
template <int kMode>
constexpr int side_bytes() {
  return (int)sizeof(Side) - (kMode == kSwiglu ? 0 : (int)sizeof(float) * 2 * 2 * 2 * 16 * 32);
}

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
template <int kMode>
__device__ void lay_tiles(const TileArgs& a, Side& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kPer = (kMaxGroups + kGThreads - 1) / kGThreads;
  constexpr bool kZ = kMode == kAdapter || kMode == kLowRank;  // z's rows are counted too
  int t[kPer], z[kPer];
  unsigned long long sum = 0;  // row tiles, and rows of z in the high half
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int g = tid * kPer + i;
    t[i] = z[i] = 0;
    if (g < a.G) {
      const int p0 = a.offsets ? __ldcg(a.offsets + g) : 0, p1 = a.offsets ? __ldcg(a.offsets + g + 1) : a.P;
      const bool fine = p0 >= 0 && p1 >= p0 && p1 <= a.P;
      bad |= !fine;
      if (fine && kZ) z[i] = padded_rows(p0, p1);
      const int rows = !fine ? 0 : kMode == kLowRank ? z[i] : p1 - p0;
      s.first[g] = kMode == kLowRank ? p0 & ~31 : p0;
      s.rows[g] = rows;
      t[i] = (rows + a.cols - 1) / a.cols;
    }
    sum += (unsigned)t[i] | (unsigned long long)z[i] << 32;
  }
  unsigned long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s.scan[warp] = inc;
  bad = __syncthreads_or(bad);
  unsigned long long run = inc - sum;
  for (int w = 0; w < warp; w++) run += s.scan[w];
  int tiles = (int)run, zr = (int)(run >> 32);
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int g = tid * kPer + i;
    if (g < a.G) {
      s.before[g] = kMode == kAdapter ? zr : tiles;
      if (kMode == kLowRank) s.z_before[g] = zr;
    }
    tiles += t[i];
    zr += z[i];
    if (g == a.G - 1) {
      if (kMode == kAdapter) tiles = (a.P + a.cols - 1) / a.cols;  // over all rows
      s.tiles = bad ? 0 : tiles;  // offsets that do not ascend within the rows: nothing is computed
      if (bad) atomicOr(a.err, kErrBadPlan);
    }
  }
  __syncthreads();
}

// The walk: units of work, each a tile and one of the parts of its sum.
struct Walk {
  int n_ct, split, units, nkb;  // channel tiles, parts per tile, units, stages of K
};
template <int kMode>
__device__ __forceinline__ Walk walk_of(const TileArgs& a, const Side& s) {
  constexpr int kChan = kMode == kSwiglu ? kLanes / 2 : kLanes;
  Walk w;
  w.n_ct = (a.N + 2 * kChan - 1) / (2 * kChan);
  w.nkb = kMode == kAdapter && !a.has_w ? 0 : (a.K + kBlockK - 1) / kBlockK;
  const int tiles = s.tiles * w.n_ct, pairs = gridDim.x >> 1;
  w.split = 1;
  if (tiles > 0 && 2 * tiles <= pairs) {
    w.split = min(a.max_split, pairs / tiles);
    if (w.nkb) w.split = min(w.split, max(1, w.nkb / kMinPart));
  }
  w.units = tiles * w.split;
  return w;
}

struct Tile {
  int g, p0, n, c0;     // group, first sorted position, rows, channel tile
  int index, part;      // of the tile, of its part
  int k0, k1;           // stages of K
};
// Unit u: the parts of a tile follow one another, the channel tiles of a row
// tile too (they share its rows), the row tiles of a group too (they share its
// weights).
template <int kMode>
__device__ __forceinline__ Tile tile_of(const TileArgs& a, const Side& s, const Walk& w, int u) {
  Tile t;
  t.index = w.split == 1 ? u : u / w.split;
  t.part = u - t.index * w.split;
  t.k0 = w.nkb * t.part / w.split;
  t.k1 = w.nkb * (t.part + 1) / w.split;
  const int q = t.index / w.n_ct;
  t.c0 = t.index - q * w.n_ct;
  int lo = 0, rows = a.P, before = 0, first = 0;
  if (kMode != kAdapter) {
    int hi = a.G - 1;  // the last group with before[g] <= q
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (s.before[m] <= q)
        lo = m;
      else
        hi = m - 1;
    }
    rows = s.rows[lo];
    before = s.before[lo];
    first = s.first[lo];
  }
  // a group's row tiles are as even as steps of 32 allow
  const int nt = (rows + a.cols - 1) / a.cols;
  const int size = ((rows + nt - 1) / nt + 31) & ~31, at = (q - before) * size;
  t.g = lo;
  t.p0 = first + at;
  t.n = min(size, rows - at);
  return t;
}

// The stages that follow those of K: f(g, c, w, kb, h, nh) for adapter g with
// columns [c, c + w) of the tile, block kb of its rank, and nh of z's two
// halves from h (both where they fit into a stage).  Without a projection the
// first is a stage of zeros (g = G) that sets the whole accumulator.  A split
// tile's parts share its adapters.  f returns whether to go on.
template <typename F>
__device__ __forceinline__ bool adapter_steps(const TileArgs& a, const Side& s, const Walk& w, const Tile& t, F f) {
  const int n = (t.n + 31) & ~31;
  if (!a.has_w && !f(a.G, 0, n, 0, 0, 1)) return false;
  // the first adapter that ends behind position p, and the first that begins at or behind it
  int lo = 0, hi = a.G;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (s.first[m] + s.rows[m] > t.p0)
      hi = m;
    else
      lo = m + 1;
  }
  int end = a.G;
  for (int low = lo; low < end;) {
    const int m = (low + end) >> 1;
    if (s.first[m] >= t.p0 + t.n)
      end = m;
    else
      low = m + 1;
  }
  if (w.split > 1) {
    const int all = end - lo;
    end = lo + all * (t.part + 1) / w.split;
    lo += all * t.part / w.split;
  }
  for (int g = lo; g < end; g++) {
    const int first = s.first[g], rows = s.rows[g];
    if (rows == 0) continue;
    const int c = max((first & ~31) - t.p0, 0);
    const int cols = min(((first + rows + 31) & ~31) - t.p0, n) - c;
    const int nh = cols <= a.b_rows ? 2 : 1;
    for (int kb = 0; kb * kBlockK < a.r; kb++)
      for (int h = 0; h < 2; h += nh)
        if (!f(g, c, cols, kb, h, nh)) return false;
  }
  return true;
}

// Channel c of sorted position p from the definition, without the tensor cores
// (and without base), for values that came out as NaN.  32 columns that several
// adapters meet in get the products of each, for the positions that it does not
// own with rows of zeros: nothing, unless its B_g is not finite there, and NaN
// then.  And an infinity of B_g times the two terms of z may be infinities of
// both signs; here the terms are added first.  Few values ever need it, and it
// is slow: 64 values of K at a time, each lane on rows of its own (one such
// adapter of 32, 64 tokens, 2048 x 2048: 2 ms a call instead of 25 us).
__device__ __forceinline__ float own_sum(const TileArgs& a, const Side& s, int p, int c) {
  int g = 0, hi = a.G;  // the first adapter that ends behind p
  while (g < hi) {
    const int m = (g + hi) >> 1;
    if (s.first[m] + s.rows[m] > p)
      hi = m;
    else
      g = m + 1;
  }
  auto add8 = [](uint4 x, uint4 rest, uint4 w, float& sum) {
    const uint32_t xv[4] = {x.x, x.y, x.z, x.w}, rv[4] = {rest.x, rest.y, rest.z, rest.w}, wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      sum = fmaf(bf16lo(xv[i]) + bf16lo(rv[i]), bf16lo(wv[i]), sum);
      sum = fmaf(bf16hi(xv[i]) + bf16hi(rv[i]), bf16hi(wv[i]), sum);
    }
  };
  float sum = 0.0f;
  if (g < a.G && s.first[g] <= p) {
    pdl_wait();  // z
    const uint16_t* z = a.z + (size_t)(s.before[g] + p - (s.first[g] & ~31)) * a.r;
    const uint16_t* b = a.b + ((size_t)g * a.N + c) * a.r;
    for (int j = 0; j < a.r; j += 8) {
      add8(__ldcg(reinterpret_cast<const uint4*>(z + j)), __ldcg(reinterpret_cast<const uint4*>(z + a.z_half + j)),
           __ldcg(reinterpret_cast<const uint4*>(b + j)), sum);
    }
  }
  if (a.has_w) {
    const int t = __ldcg(a.x_rows + p);
    if (t < 0 || t >= a.n_x) return sum;  // recorded where its row was fetched
    const uint16_t *x = a.x + (size_t)t * a.ldx, *w = a.w + (size_t)c * a.K;
    for (int k0 = 0; k0 < a.K && sum == sum; k0 += 64)
#pragma unroll
      for (int k = k0; k < k0 + 64; k += 8)
        if (k < a.K)
          add8(__ldcg(reinterpret_cast<const uint4*>(x + k)), make_uint4(0u, 0u, 0u, 0u),
               __ldcg(reinterpret_cast<const uint4*>(w + k)), sum);
  }
  return sum;
}

// The rows of x at sorted positions, gathered: thread i of 128 copies the
// 16-byte piece i % 8 of rows i / 8 + 16 m of this CTA's half of the tile.  A
// stage's copies arrive on landed[stage] as they complete; warp 3 passes that
// on to the issuing CTA, so that the copying threads never wait for their copies.
template <int kMode>
__device__ void gather_rows(const TileArgs& a, Side& s, uint8_t* ring, const Walk& w, int rank) {
  const int t = threadIdx.x - 256, piece = t & 7, r0 = t >> 3;
  volatile int* stop = &s.stop;
  Turn it;
  bool ok = true;
  for (int u = blockIdx.x >> 1; u < w.units && ok; u += gridDim.x >> 1) {
    const Tile tl = tile_of<kMode>(a, s, w, u);
    const int half = ((tl.n + 31) & ~31) >> 1;
    const uint16_t* src[8];
#pragma unroll
    for (int m = 0; m < 8; m++) {
      // rows past the tile's end repeat its last one (their columns are not
      // stored, or as zeros)
      int row = 0;
      if (r0 + 16 * m < half) {
        row = __ldcg(a.x_rows + min(tl.p0 + min(rank * half + r0 + 16 * m, tl.n - 1), a.P - 1));
        row = row < 0 ? -1 : row / a.x_div;
        if (row < 0 || row >= a.n_x) {
          atomicOr(a.err, kErrBadPlan);
          row = 0;
        }
      }
      src[m] = a.x + (size_t)row * a.ldx + piece * 8;
    }
    auto stage_free = [&] {
      ok = wait_or_stop(&s.empty[it.st], it.round ^ 1, stop, a.err);
      ok = !__any_sync(0xffffffffu, !ok);
      return ok;
    };
    for (int kb = tl.k0; kb < tl.k1; kb++, it.next(a.stages)) {
      if (!stage_free()) break;
      const uint32_t dst =
          smem_u32(ring + (size_t)it.st * a.stage_bytes + kABytes) + r0 * 128 + ((piece ^ (r0 & 7)) << 4);
      const bool in = kb * kBlockK + piece * 8 < a.K;
#pragma unroll
      for (int m = 0; m < 8; m++)
        cp_async16_if(dst + m * 2048, src[m] + (in ? kb * kBlockK : 0), in, r0 + 16 * m < half);
      cp_async_arrive(&s.landed[it.st]);
    }
    if (kMode == kAdapter && ok)  // nothing to copy, but the stage is announced like any other
      adapter_steps(a, s, w, tl, [&](int, int, int, int, int, int) {
        if (!stage_free()) return false;
        cp_async_arrive(&s.landed[it.st]);
        it.next(a.stages);
        return true;
      });
  }
  cp_async_wait_all();
}

// Passes each stage of gathered rows on: complete here, made visible to the
// tensor cores, announced to the issuing CTA.
template <int kMode>
__device__ void announce_rows(const TileArgs& a, Side& s, const Walk& w) {
  const uint32_t full = peer_u32(s.full, 0);
  Turn it;
  auto pass_on = [&] {
    if (!wait_or_stop(&s.landed[it.st], it.round, &s.stop, a.err)) return false;
    fence_proxy_async();
    mbar_arrive_at(full + it.st * 8);
    it.next(a.stages);
    return true;
  };
  for (int u = blockIdx.x >> 1; u < w.units; u += gridDim.x >> 1) {
    const Tile t = tile_of<kMode>(a, s, w, u);
    for (int kb = t.k0; kb < t.k1; kb++)
      if (!pass_on()) return;
    if (kMode == kAdapter &&
        !adapter_steps(a, s, w, t, [&](int, int, int, int, int, int) { return pass_on(); }))
      return;
  }
}

// The sum of the parts, in their order, of 32 columns (the first n of them):
// kCols columns at a time with all of their loads in flight.
template <int kParts, int kCols>
__device__ __forceinline__ void add_parts(const float* p, size_t stride, int parts, int n, float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; j += kCols) {
    float4 x[kParts][kCols / 4];
#pragma unroll
    for (int i = 0; i < kParts; i++)
#pragma unroll
      for (int k = 0; k < kCols / 4; k++)
        x[i][k] = i < parts && j + 4 * k < n
                      ? __ldcg(reinterpret_cast<const float4*>(p + i * stride + (j + 4 * k) * kLanes))
                      : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kCols / 4; k++) {
      float4 s = x[0][k];
#pragma unroll
      for (int i = 1; i < kParts; i++) {
        s.x += x[i][k].x;
        s.y += x[i][k].y;
        s.z += x[i][k].z;
        s.w += x[i][k].w;
      }
      v[j + 4 * k] = s.x;
      v[j + 4 * k + 1] = s.y;
      v[j + 4 * k + 2] = s.z;
      v[j + 4 * k + 3] = s.w;
    }
  }
}

// silu(g) m.  With h = exp(-|g| / 2) it is g m / (1 + h^2) for g >= 0 and
// g h m h / (1 + h^2) below: the divisor stays in [1, 2], and no factor leaves
// the range of fp32 before the result does (exp(-g) overflows from g = -88.7
// on, and a quick division by more than 2^126 gives zero).
__device__ __forceinline__ float silu_times(float g, float m) {
  const float h = expf(-0.5f * fabsf(g));
  const float q = __fdividef(g < 0.0f ? g * h : g, fmaf(h, h, 1.0f)) * m;
  return g < 0.0f ? q * h : q;
}

template <int kMode>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGThreads, 1)
    tiles_kernel(const __grid_constant__ Maps maps, const TileArgs a) {
  extern __shared__ uint8_t raw[];
  uint8_t* ring = raw + (-smem_u32(raw) & 1023u);  // (an index: the compiler still sees shared memory)
  Side& s = *reinterpret_cast<Side*>(ring + (size_t)a.stages * a.stage_bytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x & 1;
  constexpr int kChan = kMode == kSwiglu ? kLanes / 2 : kLanes;  // output channels per CTA
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
    if (kMode == kAdapter || !a.gather)
      for (int i = 0; i < kRowBoxes; i++) tma_prefetch(kMode == kAdapter ? &maps.z[i] : &maps.x[i]);
    tma_prefetch(&maps.w);
    if (kMode == kSwiglu) tma_prefetch(&maps.w_up);
    if (kMode == kAdapter) tma_prefetch(&maps.b);
  }
  if (warp == 2) tmem_alloc(&s.tmem, 512);
  // Adapters: the launch before this one, of z, lets it start only once
  // everything earlier has completed, so only z is waited for.  (The plan, x
  // and base are read through L2, not through an L1 that was filled earlier.)
  if (kMode != kAdapter) {
    if (!a.late_trigger) pdl_trigger();
    pdl_wait();
    if (a.late_trigger) pdl_trigger();
  }
  tc_fence_before();
  lay_tiles<kMode>(a, s);
  cluster_arrive();
  cluster_wait();  // the pair's barriers are ready
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  const Walk w = walk_of<kMode>(a, s);
  const int u0 = blockIdx.x >> 1, du = gridDim.x >> 1;
  volatile int* stop = &s.stop;
  // x in two terms: the pair's first CTA holds the rows of the one, the second
  // those of the other, and the accumulator has columns for both
  const bool two = kMode == kPlain && a.two_terms;

  if (warp == 0 || (warp == 2 && !a.gather)) {
    // ----------------------- boxes: the weights (warp 0), the rows (warp 2).
    // Whoever waits on the ring waits for every stage in turn: a role that left
    // stages out could fall two rounds behind, which a phase's parity hides.
    const bool rows = warp == 2;
    bool z_ready = false;
    Turn it;
    int filled = 0;
    bool ok = true;
    const uint32_t full = peer_u32(s.full, 0);
    // `half` rows from row p of a matrix, in boxes of 128, 64, 32 and 16
    auto fetch_rows = [&](uint8_t* B, const CUtensorMap* m, int half, auto copy) {
      if (half == 128) {
        copy(B, &m[0], 0);
        return;
      }
      int at = 0;
#pragma unroll
      for (int b = 1; b < kRowBoxes; b++)
        if (half & (128 >> b)) {
          copy(B + at * 128, &m[b], at);
          at += 128 >> b;
        }
    };
    for (int u = u0; u < w.units && ok; u += du) {
      const Tile t = tile_of<kMode>(a, s, w, u);
      const int cols = (t.n + 31) & ~31, c0 = (t.c0 * 2 + rank) * kChan;
      const int half = two ? cols : cols >> 1, p = two ? t.p0 : t.p0 + rank * half;  // this CTA's rows
      const uint32_t bytes = 2 * (kABytes + (a.gather ? 0 : half * 128));  // of both CTAs
      for (int kb = t.k0; kb < t.k1; kb++, it.next(a.stages), filled++) {
        const int k0 = kb * kBlockK;
        ok = warp_wait(&s.empty[it.st], it.round ^ 1, stop, a.err);
        if (!ok) break;
        uint8_t* A = ring + (size_t)it.st * a.stage_bytes;
        const uint32_t bar = full + it.st * 8;
        if (rows) {
          fetch_rows(A + kABytes, two && rank ? maps.x_rest : maps.x, half,
                     [&](uint8_t* to, const CUtensorMap* m, int at) { tma_2d(to, m, k0, p + at, bar); });
          continue;
        }
        if (rank == 0) mbar_expect(&s.full[it.st], bytes);
        if (kMode == kSwiglu) {
          tma_3d(A, &maps.w, k0, c0, t.g, bar);
          tma_3d(A + kABytes / 2, &maps.w_up, k0, c0, t.g, bar);
        } else if (kMode == kPlain && a.layout) {
          tma_3d(A, &maps.w, c0, k0, t.g, bar);
          tma_3d(A + kABytes / 2, &maps.w, c0 + 64, k0, t.g, bar);
        } else {
          tma_3d(A, &maps.w, k0, c0, t.g, bar);
        }
      }
      if (kMode == kAdapter && ok)
        ok = adapter_steps(a, s, w, t, [&](int g, int c, int cols, int kb, int h, int nh) {
          if (!warp_wait(&s.empty[it.st], it.round ^ 1, stop, a.err)) return false;
          uint8_t* A = ring + (size_t)it.st * a.stage_bytes;
          const uint32_t bar = full + it.st * 8;
          if (rank == 0) mbar_expect(&s.full[it.st], 2 * (kABytes + nh * (cols >> 1) * 128));
          tma_3d(A, &maps.b, kb * kBlockK, c0, g, bar);  // adapter G: outside, zeros
          if (!z_ready) pdl_wait();
          z_ready = true;
          // rows of z: those of the column range, this CTA's half of them
          const int hc = cols >> 1;
          const int zr = g < a.G ? s.before[g] + t.p0 + c - (s.first[g] & ~31) + rank * hc : 0;
          if (nh == 2 && hc == 16)
            tma_3d(A + kABytes, &maps.z2, kb * kBlockK, zr, 0, bar);
          else
            for (int i = 0; i < nh; i++)
              fetch_rows(A + kABytes + i * hc * 128, maps.z, hc, [&](uint8_t* to, const CUtensorMap* m, int at) {
              tma_3d(to, m, kb * kBlockK, zr + at, g < a.G ? h + i : 2, bar);  // 2: outside, zeros
            });
          it.next(a.stages);
          filled++;
          return true;
        });
    }
    // after a timeout: the copies in flight must land before the pair ends
    if (!ok && rank == 0 && lane == 0)
      for (int i = filled > a.stages ? filled - a.stages : 0; i < filled; i++)
        mbar_wait_bounded(&s.full[i % a.stages], (i / a.stages) & 1, a.err);
  } else if (warp == 1 && rank == 0) {
    // -------------------------------------------------------- products
    Turn it;
    int ti = 0;
    bool ok = true;
    // descriptors of the first stage; a stage, and a step of K, further
    const bool mn_a = kMode == kPlain && a.layout;
    const uint64_t a_desc = tile_desc(smem_u32(ring), mn_a ? kABytes / 2 : 16);
    const uint64_t b_desc = tile_desc(smem_u32(ring) + kABytes, 16);
    const int stage16 = a.stage_bytes >> 4;
    const uint64_t a_step = mn_a ? 2048 >> 4 : 2;
    for (int u = u0; u < w.units && ok; u += du, ti++) {
      const Tile t = tile_of<kMode>(a, s, w, u);
      const uint32_t d = tmem + (ti & 1) * kMaxCols;
      const uint32_t idesc = mma_desc(2 * kLanes, ((t.n + 31) & ~31) << (two ? 1 : 0), mn_a);
      ok = warp_wait(&s.acc_empty[ti & 1], ((ti >> 1) & 1) ^ 1, stop, a.err);
      if (!ok) break;
      tc_fence_after();
      for (int kb = t.k0; kb < t.k1; kb++, it.next(a.stages)) {
        ok = warp_wait(&s.full[it.st], it.round, stop, a.err);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ad = a_desc + (uint64_t)(it.st * stage16), bd = b_desc + (uint64_t)(it.st * stage16);
        const int left = a.K - kb * kBlockK;
        if (left >= kBlockK) {
#pragma unroll
          for (int k = 0; k < kBlockK / 16; k++) mma_bf16(d, ad + k * a_step, bd + k * 2, idesc, kb > t.k0 || k > 0);
        } else {  // past K the stage holds zeros
          for (int k = 0; k * 16 < left; k++) mma_bf16(d, ad + k * a_step, bd + k * 2, idesc, kb > t.k0 || k > 0);
        }
        mma_commit(&s.empty[it.st]);
      }
      if (kMode == kAdapter && ok)
        ok = adapter_steps(a, s, w, t, [&](int g, int c, int cols, int kb, int h, int nh) {
          if (!warp_wait(&s.full[it.st], it.round, stop, a.err)) return false;
          tc_fence_after();
          const uint32_t A = smem_u32(ring + (size_t)it.st * a.stage_bytes);
          const uint64_t ad = tile_desc(A, 16);
          const uint32_t id = mma_desc(2 * kLanes, cols, false);
          const int steps = g < a.G ? (min(kBlockK, a.r - kb * kBlockK) + 15) / 16 : 1;
          for (int i = 0; i < nh; i++) {
            const uint64_t bd = tile_desc(A + kABytes + i * (cols >> 1) * 128, 16);
            for (int k = 0; k < steps; k++) mma_bf16(d + c, ad + k * 2, bd + k * 2, id, g < a.G);
          }
          mma_commit(&s.empty[it.st]);
          it.next(a.stages);
          return true;
        });
      if (ok) mma_commit(&s.acc_full[ti & 1]);
    }
    if (!ok) {  // after a timeout: the products in flight must end before the pair does
      mma_commit(&s.drain);
      if (lane == 0) mbar_wait_bounded(&s.drain, 0, a.err);
    }
  } else if (warp == 3 && lane == 0) {
    if (a.gather) announce_rows<kMode>(a, s, w);
  } else if (warp >= 8) {
    if (a.gather) gather_rows<kMode>(a, s, ring, w, rank);
  } else if (warp >= 4) {
    // ------------------------------------------------- read back, store
    const int q4 = warp - 4, et = tid - 128;
    const bool odd = lane & 1;
    int ti = 0, turn = 0;
    for (int u = u0; u < w.units; u += du, ti++) {
      const Tile t = tile_of<kMode>(a, s, w, u);
      for (int j = et; j < ((t.n + 31) & ~31); j += 128) {
        int q = -1;
        if (kMode == kLowRank) {
          // row q of z, or of zeros (-2 - q) where the adapter does not own the position
          const int p = t.p0 + j;
          if (j < t.n) {
            q = s.z_before[t.g] + p - s.first[t.g];
            const bool own = p >= __ldcg(a.offsets + t.g) && p < __ldcg(a.offsets + t.g + 1);
            const int row = own ? __ldcg(a.x_rows + p) : -1;
            if (row < 0 || row >= a.n_x) q = -2 - q;
          }
        } else if (j < t.n) {
          q = a.y_rows ? __ldcg(a.y_rows + t.p0 + j) : t.p0 + j;
          if (q < 0 || q >= a.n_y) {
            atomicOr(a.err, kErrBadPlan);
            q = -1;
          }
          if (a.gather) {  // a row that is not there has no result
            const int row = __ldcg(a.x_rows + t.p0 + j);
            if (row < 0 || row / a.x_div >= a.n_x) q = -1;
          }
        }
        s.y_row[(j & 1) * (kMaxCols / 2) + (j >> 1)] = q;
      }
      const bool ok = wait_or_stop(&s.acc_full[ti & 1], (ti >> 1) & 1, stop, a.err);
      if (bar_any(1, 128, !ok)) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q4 * 32) << 16) + (ti & 1) * kMaxCols;
      auto load_columns = [&](int j0, float (&v)[32]) {
        tmem_ld32(acc + j0, v);
        if (two) {
          float rest[32];
          tmem_ld32(acc + ((t.n + 31) & ~31) + j0, rest);
#pragma unroll
          for (int j = 0; j < 32; j++)  // (an infinite weight: the first term has its sign, the second may have the other)
            v[j] = isfinite(v[j]) ? v[j] + rest[j] : v[j];
        }
      };
      bool finish = true;
      const size_t part_size = (size_t)2 * a.cols * kLanes;
      float* part0 = a.part + (size_t)t.index * w.split * part_size + (size_t)rank * a.cols * kLanes + (q4 * 32 + lane) * 4;
      if (w.split > 1) {
        float* mine = part0 + t.part * part_size;
        for (int j0 = 0; j0 < t.n; j0 += 32) {
          float v[32];
          load_columns(j0, v);
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            __stcg(reinterpret_cast<float4*>(mine + (j0 + j) * kLanes), make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]));
        }
        __threadfence();
        bar_any(1, 128, false);
        if (et == 0) {
          uint32_t* count = a.count + t.index * 2 + rank;
          const bool last = atomicAdd(count, 1u) == (uint32_t)w.split - 1;
          if (last) *count = 0u;  // as it was found
          __threadfence();
          s.last = last;
        }
        bar_any(1, 128, false);
        finish = s.last != 0;
      }
      for (int j0 = 0; j0 < t.n && finish; j0 += 32) {
        float v[32];
        if (w.split > 1) {
          if (w.split <= 4)
            add_parts<4, 16>(part0 + j0 * kLanes, part_size, w.split, t.n - j0, v);
          else
            add_parts<kMaxSplit, 8>(part0 + j0 * kLanes, part_size, w.split, t.n - j0, v);
        } else {
          load_columns(j0, v);
        }
        if (kMode == kAdapter) {
          float some[4] = {};  // NaN if a value is (or if infinities meet)
#pragma unroll
          for (int j = 0; j < 32; j++) some[j & 3] += v[j];
          const float sum = (some[0] + some[1]) + (some[2] + some[3]);
          if (__any_sync(0xffffffffu, sum != sum)) {
            const int c = (t.c0 * 2 + rank) * kChan + q4 * 32 + lane;
#pragma unroll 1
            for (int i = 0; i < 32 && j0 + i < t.n; i++) {
              float old = 0.0f;
#pragma unroll
              for (int j = 0; j < 32; j++) old = j == i ? v[j] : old;
              if (c < a.N && old != old) {
                const float now = own_sum(a, s, t.p0 + j0 + i, c);
#pragma unroll
                for (int j = 0; j < 32; j++) v[j] = j == i ? now : v[j];
              }
              __syncwarp();
            }
          }
        }
        if (kMode == kSwiglu) {
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
            const float o = in[i][lane], g = up ? o : v[2 * i], m = up ? v[2 * i + 1] : o;
            r[i] = silu_times(g, m);
          }
          const int* q_of = s.y_row + (up ? kMaxCols / 2 : 0) + (j0 >> 1);
          const int cw = (t.c0 * 2 + rank) * kChan + (q4 & 1) * 32;
          uint16_t* y = static_cast<uint16_t*>(a.y);
          if (a.ldy & 1) {  // rows that start on odd words
            const int c = cw + lane;
#pragma unroll
            for (int i = 0; i < 16; i++) {
              const int q = q_of[i];
              st16_if(y + (size_t)q * a.ldy + c, f2bf16(r[i]), q >= 0 && c < a.N);
            }
          } else {
            const int c = cw + (lane & ~1);
            const bool in_n = c < a.N;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float o = __shfl_xor_sync(0xffffffffu, odd ? r[i] : r[i + 1], 1);
              const float lo = odd ? o : r[i], hi = odd ? r[i + 1] : o;
              const int q = q_of[i + (odd ? 1 : 0)];
              uint32_t p2 = bf16x2(lo, hi);
              if (a.y_rest) {
                uint32_t rest;
                bf16_terms(lo, hi, p2, rest);
                st32_if(a.y_rest + (size_t)q * a.ldy + c, rest, q >= 0 && in_n);
              }
              st32_if(y + (size_t)q * a.ldy + c, p2, q >= 0 && in_n);
            }
          }
        } else if (kMode == kPlain && a.y_fp32) {
          const int c = (t.c0 * 2 + rank) * kChan + q4 * 32 + lane;
          const bool in_n = c < a.N;
          float* y = static_cast<float*>(a.y) + c;
#pragma unroll
          for (int j = 0; j < 32; j++) {
            const int q = s.y_row[(j & 1) * (kMaxCols / 2) + ((j0 + j) >> 1)];
            st32_if(y + (size_t)q * a.ldy, __float_as_uint(v[j]), q >= 0 && in_n);
          }
        } else if (kMode == kLowRank) {
          // the value and what its rounding leaves, two channels to a word
          const int c = q4 * 32 + (lane & ~1);
          const bool in_n = rank == 0 && c < a.N;
          const float scale = a.scale ? a.scale[t.g] : 1.0f;
          uint16_t* z = static_cast<uint16_t*>(a.y) + c;
#pragma unroll
          for (int i = 0; i < 16; i++) {
            const float o = __shfl_xor_sync(0xffffffffu, odd ? v[2 * i] : v[2 * i + 1], 1);
            int q = s.y_row[(odd ? kMaxCols / 2 : 0) + (j0 >> 1) + i];
            const bool own = q >= 0, some = q != -1;
            if (!own) q = -2 - q;
            const float lo = own ? (odd ? o : v[2 * i]) * scale : 0.0f, hi = own ? (odd ? v[2 * i + 1] : o) * scale : 0.0f;
            uint32_t top, rest;
            bf16_terms(lo, hi, top, rest);
            st32_if(z + (size_t)q * a.N, top, some && in_n);
            st32_if(z + a.z_half + (size_t)q * a.N, rest, some && in_n);
          }
        } else {
          // two channels to a word: the even lane of a pair takes the even column
          const int c = (t.c0 * 2 + rank) * kChan + q4 * 32 + (lane & ~1);
          const bool in_n = c < a.N;
          uint16_t* y = static_cast<uint16_t*>(a.y) + c;
          int qs[16];
          const int4* q_of = reinterpret_cast<const int4*>(s.y_row + (odd ? kMaxCols / 2 : 0) + (j0 >> 1));
#pragma unroll
          for (int i = 0; i < 4; i++) *reinterpret_cast<int4*>(qs + 4 * i) = q_of[i];
          uint32_t bw[16];
          if (kMode == kAdapter && a.base) {
#pragma unroll
            for (int i = 0; i < 16; i++)
              bw[i] = ld32_if(a.base + (size_t)qs[i] * a.ldy + c, qs[i] >= 0 && in_n);
          }
#pragma unroll
          for (int i = 0; i < 16; i++) {
            const float o = __shfl_xor_sync(0xffffffffu, odd ? v[2 * i] : v[2 * i + 1], 1);
            float lo = odd ? o : v[2 * i], hi = odd ? v[2 * i + 1] : o;
            if (kMode == kAdapter && a.base) {
              lo += bf16lo(bw[i]);
              hi += bf16hi(bw[i]);
            }
            st32_if(y + (size_t)qs[i] * a.ldy, bf16x2(lo, hi), qs[i] >= 0 && in_n);
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
  if (kMode == kAdapter) pdl_wait();  // whoever waits for this launch waits for the one before it too
}

// What a device answered once: its SM count, and which kernels have been
// given their shared memory on it.
struct DeviceState {
  int dev = -1, sms = 0;
  bool allowed[4] = {};
};
cudaError_t device_state(DeviceState** out) {
  static thread_local DeviceState state;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev != state.dev) {
    state = DeviceState();
    e = cudaDeviceGetAttribute(&state.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    state.dev = dev;
  }
  *out = &state;
  return state.sms < 2 ? cudaErrorInvalidDevice : cudaSuccess;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Rows per tile at most for n rows: all of them up to 256.
int most_cols(int n) { return n < kMaxCols ? (n + 31) / 32 * 32 : kMaxCols; }

template <int kMode>
cudaError_t run_tiles(const Maps& m, TileArgs t, cudaStream_t s) {
  // (32 at least: an adapter's narrowest columns with both halves of z)
  t.b_rows = t.two_terms ? t.cols : t.cols / 2 < 32 ? 32 : t.cols / 2;
  t.stage_bytes = kABytes + t.b_rows * 128;
  // Beside the launch of z in adapter.cu, whose CTAs take up to 73 KB, a pair
  // finds room only if it takes the rest at most; it starts 5 us later otherwise.
  const int budget = kMode == kAdapter && few_values(t.P, t.r, t.K) ? kSmemBudget - 74 * 1024 : kSmemBudget;
  t.stages = (budget - side_bytes<kMode>()) / t.stage_bytes;
  if (t.stages > kMaxStages) t.stages = kMaxStages;
  t.max_split = kMode == kLowRank ? 1 : kMaxSplit;
  const size_t smem = 1024 + (size_t)t.stages * t.stage_bytes + side_bytes<kMode>();
  DeviceState* dev = nullptr;
  cudaError_t e = device_state(&dev);
  if (e == cudaSuccess && !dev->allowed[kMode]) {
    e = cudaFuncSetAttribute(tiles_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget + 1024);
    dev->allowed[kMode] = e == cudaSuccess;
  }
  if (e != cudaSuccess) return e;
  const int pairs = dev->sms / 2 < kMaxPairs ? dev->sms / 2 : kMaxPairs;
  const int chan = kMode == kSwiglu ? kLanes : 2 * kLanes;
  const long n_ct = (t.N + chan - 1) / chan;
  // units at most: the tiles, each in as many parts as there may be
  long most = (long)(t.P + t.cols - 1) / t.cols;
  if (kMode != kAdapter) most += 2 * (t.G < t.P ? t.G : t.P);
  most *= n_ct * kMaxSplit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * (most < pairs ? most : pairs)));
  cfg.blockDim = dim3(kGThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tiles_kernel<kMode>, m, t);
}

// Rows per tile: the most, halved while a call's tiles would leave more than
// half of the CTA pairs without one (the weights are then read once per row
// tile, from L2).
int choose_cols(int n, int groups, int N, int chan) {
  int cols = most_cols(n);
  const long n_ct = (N + chan - 1) / chan;
  while (cols > 32) {
    const long row_tiles = (n + cols - 1) / cols;
    if ((row_tiles > groups ? row_tiles : groups) * n_ct * 2 > kMaxPairs) break;
    cols = (cols / 2 + 31) / 32 * 32;
  }
  return cols;
}

// Rows per tile of z: as few as leave each CTA pair one tile at most (an
// adapter's widened range adds up to one and a half).
int low_rank_cols(int T, int A) {
  const int left = kMaxPairs - 3 * (A < kMaxPairs / 6 ? A : kMaxPairs / 6) / 2;
  const int cols = ((T + left - 1) / left + 31) / 32 * 32;
  return cols < kMaxCols ? cols : kMaxCols;
}

bool row_maps(CUtensorMap* m, const void* base, uint64_t x, uint64_t y, uint64_t z, uint64_t row_bytes,
              uint64_t mat_bytes) {
  for (int b = 0; b < kRowBoxes; b++)
    if (!tensor_map(&m[b], base, x, y, z, row_bytes, mat_bytes, kBlockK, 128 >> b)) return false;
  return true;
}

}  // namespace

size_t split_bytes(int n_rows) {
  return align256(sizeof(uint32_t) * 2 * kMaxPairs) + sizeof(float) * 2 * kMaxPairs * kLanes * (size_t)most_cols(n_rows);
}

cudaError_t launch_grouped(const GroupedArgs& a, cudaStream_t s) {
  TileArgs t = {};
  t.G = a.G;
  t.P = a.P;
  t.n_x = a.n_x;
  t.n_y = a.n_y;
  t.N = a.N;
  t.K = a.K;
  t.ldx = a.ldx;
  t.ldy = a.ldy;
  t.layout = a.layout;
  t.gather = a.x_rows != nullptr;
  t.x_div = a.x_div;
  t.y_fp32 = a.y_fp32;
  t.late_trigger = a.late_trigger;
  t.x = a.x;
  t.x_rows = a.x_rows;
  t.offsets = a.offsets;
  t.y_rows = a.y_rows;
  t.y = a.y;
  t.err = a.err;
  t.count = static_cast<uint32_t*>(a.split);
  t.part = reinterpret_cast<float*>(static_cast<char*>(a.split) + align256(sizeof(uint32_t) * 2 * kMaxPairs));
  t.cols = choose_cols(a.P, a.G < a.P ? a.G : a.P, a.N, a.w_up ? kLanes : 2 * kLanes);
  t.two_terms = a.x_rest != nullptr;
  if (t.two_terms && t.cols > kMaxCols / 2) t.cols = kMaxCols / 2;  // both terms fit into a stage
  t.y_rest = a.y_rest;
  Maps m;  // (what a mode does not use stays unset)
  const uint64_t N = a.N, K = a.K;
  bool ok = t.gather || row_maps(m.x, a.x, K, a.n_x, 0, 2ull * a.ldx, 0);
  if (t.two_terms) ok = ok && row_maps(m.x_rest, a.x_rest, K, a.n_x, 0, 2ull * a.ldx, 0);
  if (a.w_up)
    ok = ok && tensor_map(&m.w, a.w, K, N, a.G, 2 * K, 2 * N * K, kBlockK, kLanes / 2) &&
         tensor_map(&m.w_up, a.w_up, K, N, a.G, 2 * K, 2 * N * K, kBlockK, kLanes / 2);
  else
    ok = ok && (a.layout ? tensor_map(&m.w, a.w, N, K, a.G, 2 * N, 2 * N * K, 64, kBlockK)
                         : tensor_map(&m.w, a.w, K, N, a.G, 2 * K, 2 * N * K, kBlockK, kLanes));
  if (!ok) return cudaErrorInvalidValue;
  return a.w_up ? run_tiles<kSwiglu>(m, t, s) : run_tiles<kPlain>(m, t, s);
}

cudaError_t launch_adapter(const AdapterArgs& a, cudaStream_t s) {
  const uint64_t N = a.N, K = a.K, r = a.r, zr = adapter_z_rows(a.T, a.A);
  // z on the tensor cores
  const bool many = !few_values(a.T, a.r, a.K);
  TileArgs z = {};
  Maps mz;
  if (many) {
    z.G = a.A;
    z.P = z.n_x = a.T;
    z.N = a.r;
    z.K = z.ldx = a.K;
    z.gather = 1;
    z.x_div = 1;
    z.x = a.x;
    z.x_rows = a.rows;
    z.offsets = a.offsets;
    z.y = a.z;
    z.err = a.err;
    z.scale = a.scale;
    z.z_half = zr * a.r;
    z.late_trigger = 1;
    z.cols = low_rank_cols(a.T, a.A);
    if (!tensor_map(&mz.w, a.a, K, r, a.A, 2 * K, 2 * K * r, kBlockK, kLanes)) return cudaErrorInvalidValue;
  }
  TileArgs t = {};
  t.G = a.A;
  t.P = t.n_x = t.n_y = a.T;
  t.N = t.ldy = a.N;
  t.K = t.ldx = a.K;
  t.gather = 1;
  t.x_div = 1;
  t.x = a.x;
  t.x_rows = t.y_rows = a.rows;
  t.offsets = a.offsets;
  t.y = a.y;
  t.err = a.err;
  t.count = static_cast<uint32_t*>(a.split);
  t.part = reinterpret_cast<float*>(static_cast<char*>(a.split) + align256(sizeof(uint32_t) * 2 * kMaxPairs));
  t.r = a.r;
  t.w = a.w;
  t.z = a.z;
  t.b = a.b;
  t.z_half = zr * a.r;
  t.has_w = a.w != nullptr;
  t.base = a.base;
  t.cols = choose_cols(a.T, 1, a.N, 2 * kLanes);
  Maps m;
  const bool ok = row_maps(m.z, a.z, r, zr, 2, 2 * r, 2 * r * zr) &&
                  tensor_map(&m.z2, a.z, r, zr, 2, 2 * r, 2 * r * zr, kBlockK, 16, 2) &&
                  tensor_map(&m.b, a.b, r, N, a.A, 2 * r, 2 * r * N, kBlockK, kLanes) &&
                  (!a.w || tensor_map(&m.w, a.w, K, N, 1, 2 * K, 2 * N * K, kBlockK, kLanes));
  if (!ok) return cudaErrorInvalidValue;
  if (!a.w) m.w = m.b;
  // (the maps are ready, so that the second launch follows the first at once)
  const cudaError_t e = many ? run_tiles<kLowRank>(mz, z, s) : launch_adapter_down(a, s);
  return e == cudaSuccess ? run_tiles<kAdapter>(m, t, s) : e;
}

}  // namespace moe
