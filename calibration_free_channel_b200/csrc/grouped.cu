// grouped.cu -- products over ragged groups of rows (expert products of
// prompts, per-request adapters).
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kTile = 64, kStep = 16;

// The sorted positions [p0, p1) of group g, clamped to [0, P]; a plan that
// breaks the rules is recorded and the group left out.
__device__ __forceinline__ bool group_range(const int32_t* offsets, int g, int P, uint32_t* err, int& p0, int& p1) {
  p0 = offsets[g];
  p1 = offsets[g + 1];
  if (p0 < 0 || p1 < p0 || p1 > P) {
    atomicOr(err, kErrBadPlan);
    p0 = p1 = 0;
    return false;
  }
  return true;
}

// 64 rows x 64 channels per CTA, blockIdx.y = group, the group's row tiles in
// turn; fp32 sums over the whole of K.
__global__ void __launch_bounds__(256) grouped_kernel(GroupedArgs a) {
  __shared__ float xs[kStep][kTile + 4], ws[kStep][kTile + 4], us[kStep][kTile + 4];
  __shared__ int xr[kTile];
  const int g = blockIdx.y, n0 = blockIdx.x * kTile, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const bool swiglu = a.w_up != nullptr;
  int g0, g1;
  if (!group_range(a.offsets, g, a.P, a.err, g0, g1)) return;
  for (int p0 = g0; p0 < g1; p0 += kTile) {
    __syncthreads();
    if (tid < kTile) {
      const int p = p0 + tid;
      int r = -1;
      if (p < g1) {
        r = a.x_rows ? a.x_rows[p] : p;
        if (a.x_rows && r >= 0) r /= a.x_div;
        if (r < 0 || r >= a.n_x) {
          atomicOr(a.err, kErrBadPlan);
          r = -1;
        }
      }
      xr[tid] = r;
    }
    __syncthreads();
    float acc[4][4] = {}, acu[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kStep) {
      for (int i = tid; i < kTile * kStep; i += 256) {
        const int m = i / kStep, k = i % kStep;
        xs[k][m] = xr[m] >= 0 && k0 + k < a.K ? bf16f(a.x[(size_t)xr[m] * a.K + k0 + k]) : 0.0f;
        const int n = a.layout ? i % kTile : i / kStep, kw = a.layout ? i / kTile : i % kStep;
        const bool in = n0 + n < a.N && k0 + kw < a.K;
        const size_t at = a.layout ? ((size_t)g * a.K + k0 + kw) * a.N + n0 + n : ((size_t)g * a.N + n0 + n) * a.K + k0 + kw;
        ws[kw][n] = in ? bf16f(a.w[at]) : 0.0f;
        if (swiglu) us[kw][n] = in ? bf16f(a.w_up[at]) : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kStep; k++)
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int j = 0; j < 4; j++) {
            acc[i][j] = fmaf(xs[k][ty * 4 + i], ws[k][tx * 4 + j], acc[i][j]);
            if (swiglu) acu[i][j] = fmaf(xs[k][ty * 4 + i], us[k][tx * 4 + j], acu[i][j]);
          }
      __syncthreads();
    }
    for (int i = 0; i < 4; i++) {
      const int p = p0 + ty * 4 + i;
      if (p >= g1 || xr[ty * 4 + i] < 0) continue;
      const int q = a.y_rows ? a.y_rows[p] : p;
      if (q < 0 || q >= a.n_y) {
        atomicOr(a.err, kErrBadPlan);
        continue;
      }
      for (int j = 0; j < 4; j++) {
        const int n = n0 + tx * 4 + j;
        if (n >= a.N) continue;
        const float v = swiglu ? acc[i][j] / (1.0f + __expf(-acc[i][j])) * acu[i][j] : acc[i][j];
        if (a.y_fp32)
          static_cast<float*>(a.y)[(size_t)q * a.N + n] = v;
        else
          static_cast<uint16_t*>(a.y)[(size_t)q * a.N + n] = f2bf16(v);
      }
    }
  }
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

}  // namespace

cudaError_t launch_grouped(const GroupedArgs& a, cudaStream_t s) {
  grouped_kernel<<<dim3((a.N + kTile - 1) / kTile, a.G), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_adapter(const AdapterArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(float) * (a.K + a.r);
  cudaError_t e = cudaFuncSetAttribute(adapter_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  adapter_kernel<<<dim3(a.T, (a.N + 255) / 256), 256, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
