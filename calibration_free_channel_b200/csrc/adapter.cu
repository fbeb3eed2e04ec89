// adapter.cu -- z = scale_g x A_g^T, the first half of the low-rank adapters
// (grouped.cu multiplies it by B_g beside the shared projection).
//
// z has r <= 128 columns: 2 T r K multiply-adds against T K + r K inputs, so
// it is bound by reading x and the adapters once, not by products.  One CTA
// takes 16 sorted positions of one adapter; its 16 warps split K (above rank 64 also the columns), each loading
// 16-byte pieces of the rows of x and of A_g straight into the operands of
// mma.sync (which values of K an operand slot holds is free, as long as x and
// A_g agree: a thread's 8 consecutive values serve two products).
//
// 64 tokens of 32 adapters, rank 32, K = 2048: 6 us, four of them waiting for
// loads that each touch eight rows.
//
// (Loads here and in block.cu are plain ones: a launch that starts before its
// predecessor's end may not read what that wrote through the read-only path.)
//
// z is held as two bf16 terms, the rounded value and what the rounding left,
// 16 significant bits together: rounding it to one would add as much error as
// the rounding of the result.  Rows of z that a 32-row step of the tiles
// reaches but the adapter does not own are zero.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kRowsZ = 16;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// kNT: tiles of 8 columns of z that a warp computes; kHalves: 2 where the
// columns are split over two sets of warps (r > 64).
template <int kNT, int kHalves>
__global__ void __launch_bounds__(512) z_kernel(AdapterArgs a, size_t z_rows) {
  constexpr int kKWarps = 16 / kHalves, kCols = 8 * kNT * kHalves;
  extern __shared__ float red[];  // [kKWarps][kRowsZ][kCols]
  __shared__ int first[kMaxGroups], before[kMaxGroups + 1], scan[16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();  // what starts now finds everything earlier complete
  // the adapters' rows of z: the prefix of the padded row counts
  constexpr int kPer = kMaxGroups / 512;
  int n[kPer], sum = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int g = tid * kPer + i;
    n[i] = 0;
    if (g < a.A) {
      const int p0 = a.offsets[g], p1 = a.offsets[g + 1];
      const bool fine = p0 >= 0 && p1 >= p0 && p1 <= a.T;
      bad |= !fine;
      first[g] = p0;
      if (fine) n[i] = padded_rows(p0, p1);
    }
    sum += n[i];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scan[warp] = inc;
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(a.err, kErrBadPlan);
    return;
  }
  int run = inc - sum;
  for (int w = 0; w < warp; w++) run += scan[w];
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const int g = tid * kPer + i;
    if (g < a.A) before[g] = run;
    run += n[i];
    if (g == a.A - 1) before[a.A] = run;
  }
  __syncthreads();

  const int units = before[a.A] / kRowsZ, r = a.r, gr = lane >> 2, t4 = lane & 3;
  const int kw = warp % kKWarps, j0 = warp / kKWarps * 8 * kNT;  // this warp's share of K, its first column
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    int lo = 0, hi = a.A - 1;  // the last adapter with before[g] <= row
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (before[m] <= u * kRowsZ)
        lo = m;
      else
        hi = m - 1;
    }
    const int g = lo, p0 = first[g], p1 = a.offsets[g + 1];
    const int q0 = (p0 & ~31) + u * kRowsZ - before[g];  // first position, may lie before p0 or behind p1
    float acc[kNT][4];
#pragma unroll
    for (int i = 0; i < kNT; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) acc[i][j] = 0.0f;
    if (q0 + kRowsZ > p0 && q0 < p1) {
      const uint16_t* xr[2];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int p = q0 + gr + 8 * h;
        xr[h] = nullptr;
        if (p >= p0 && p < p1) {
          const int t = a.rows[p];
          if (t >= 0 && t < a.T)
            xr[h] = a.x + (size_t)t * a.K;
          else
            atomicOr(a.err, kErrBadPlan);
        }
      }
      const uint16_t* A = a.a + (size_t)g * r * a.K;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll(16 / kNT < 8 ? 16 / kNT : 8)
      for (int k0 = kw * 32; k0 < a.K; k0 += 32 * kKWarps) {
        const int k = k0 + t4 * 8;
        const bool in = k < a.K;
        uint4 x0 = in && xr[0] ? *reinterpret_cast<const uint4*>(xr[0] + k) : zero;
        uint4 x1 = in && xr[1] ? *reinterpret_cast<const uint4*>(xr[1] + k) : zero;
        uint4 b[kNT];
#pragma unroll
        for (int i = 0; i < kNT; i++) {
          const int j = j0 + i * 8 + gr;
          b[i] = in && j < r ? *reinterpret_cast<const uint4*>(A + (size_t)j * a.K + k) : zero;
        }
#pragma unroll
        for (int i = 0; i < kNT; i++) {
          mma16816(acc[i], x0.x, x1.x, x0.y, x1.y, b[i].x, b[i].y);
          mma16816(acc[i], x0.z, x1.z, x0.w, x1.w, b[i].z, b[i].w);
        }
      }
    }
    // sum over the warps (their shares of K), in order
    float* mine = red + kw * kRowsZ * kCols + j0;
#pragma unroll
    for (int i = 0; i < kNT; i++) {
      const int j = i * 8 + 2 * t4;
      *reinterpret_cast<float2*>(mine + gr * kCols + j) = make_float2(acc[i][0], acc[i][1]);
      *reinterpret_cast<float2*>(mine + (gr + 8) * kCols + j) = make_float2(acc[i][2], acc[i][3]);
    }
    __syncthreads();
    const float scale = a.scale ? a.scale[g] : 1.0f;
    for (int i = tid; i < kRowsZ * r; i += 512) {
      const int row = i / r, j = i - row * r;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kKWarps; w++) v += red[(w * kRowsZ + row) * kCols + j];
      const int p = q0 + row;  // (a row that is not the adapter's: zeros times its weights may be NaN)
      v = p >= p0 && p < p1 ? v * scale : 0.0f;
      const size_t at = ((size_t)u * kRowsZ + row) * r + j;
      uint32_t top, rest;
      bf16_terms(v, 0.0f, top, rest);
      a.z[at] = (uint16_t)top;
      a.z[z_rows * r + at] = (uint16_t)rest;
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_adapter_down(const AdapterArgs& a, cudaStream_t s) {
  const size_t zr = adapter_z_rows(a.T, a.A);
  const long units = (long)(zr / kRowsZ);  // at most
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units < 592 ? units : 592));  // twice what the SMs hold
  cfg.blockDim = dim3(512);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto kernel, int floats) {
    cfg.dynamicSmemBytes = sizeof(float) * kRowsZ * floats;
    if (cfg.dynamicSmemBytes > 32 * 1024) {
      cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes);
      if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kernel, a, zr);
  };
  if (a.r <= 16) return go(z_kernel<2, 1>, 16 * 16);
  if (a.r <= 32) return go(z_kernel<4, 1>, 16 * 32);
  if (a.r <= 64) return go(z_kernel<8, 1>, 16 * 64);
  return go(z_kernel<8, 2>, 8 * 128);
}

}  // namespace moe
