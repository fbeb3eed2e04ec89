// block.cu -- the all-channel MoE block over any number of tokens: routing,
// grouping of the (token, slot) pairs by expert, the two grouped products and
// the weighted sum of a token's pairs.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

// Router logits: exact bf16 products, fp64 sums.  One warp per (token, 4 experts).
__global__ void __launch_bounds__(256) logits_kernel(BlockArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x, e0 = (blockIdx.y * 8 + warp) * 4;
  double s[4] = {};
  for (int k = lane; k < a.d; k += 32) {
    const double x = bf16f(a.x[(size_t)t * a.d + k]);
#pragma unroll
    for (int j = 0; j < 4; j++)
      if (e0 + j < a.E) s[j] = fma(x, (double)bf16f(a.w_router[(size_t)(e0 + j) * a.d + k]), s[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const double v = warp_sum(s[j]);
    if (lane == 0 && e0 + j < a.E)
      a.logits[(size_t)t * a.E + e0 + j] = v + (a.bias ? (double)a.bias[e0 + j] : 0.0);
  }
}

// Top-e of each token (ties to the lower id) and the softmax weights over the
// chosen logits; one warp per token.
__global__ void __launch_bounds__(256) choose_kernel(BlockArgs a) {
  const int lane = threadIdx.x & 31, t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= a.B) return;
  const double* L = a.logits + (size_t)t * a.E;
  uint32_t taken = 0;
  double l0 = 0.0, mine = 0.0;
  int my_id = 0;
  for (int s = 0; s < a.top_e; s++) {
    double bv = -INFINITY;
    int bi = 0x7fffffff;
    for (int m = 0; lane + 32 * m < a.E; m++) {
      if (taken & (1u << m)) continue;
      const double v = L[lane + 32 * m];
      if (bi == 0x7fffffff || v > bv) {
        bv = v;
        bi = lane + 32 * m;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(0xffffffffu, bv, o);
      const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
      if (oi != 0x7fffffff && (bi == 0x7fffffff || ov > bv || (ov == bv && oi < bi))) {
        bv = ov;
        bi = oi;
      }
    }
    if ((bi & 31) == lane) taken |= 1u << (bi >> 5);
    if (s == 0) l0 = bv;
    if (lane == s) {
      mine = bv;
      my_id = bi;
    }
  }
  const double ex = lane < a.top_e ? exp(mine - l0) : 0.0;
  const double den = warp_sum(ex);
  if (lane < a.top_e) {
    a.ids[(size_t)t * a.top_e + lane] = my_id;
    a.wts[(size_t)t * a.top_e + lane] = (float)(ex / den);
    if (a.ids_out) a.ids_out[(size_t)t * a.top_e + lane] = my_id;
  }
}

// y[t] = bf16(residual[t] + sum over the slots, in slot order, of w out).
__global__ void __launch_bounds__(256) combine_kernel(BlockArgs a) {
  const int t = blockIdx.x;
  for (int j = threadIdx.x * 4; j < a.d; j += 256 * 4) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < a.top_e; k++) {
      const float w = a.wts[(size_t)t * a.top_e + k];
      const float4 v = *reinterpret_cast<const float4*>(a.out + ((size_t)t * a.top_e + k) * a.d + j);
      s.x = fmaf(w, v.x, s.x);
      s.y = fmaf(w, v.y, s.y);
      s.z = fmaf(w, v.z, s.z);
      s.w = fmaf(w, v.w, s.w);
    }
    if (a.residual) {
      const uint2 r = *reinterpret_cast<const uint2*>(a.residual + (size_t)t * a.d + j);
      s.x += bf16lo(r.x);
      s.y += bf16hi(r.x);
      s.z += bf16lo(r.y);
      s.w += bf16hi(r.y);
    }
    uint2 o;
    o.x = f2bf16(s.x) | ((uint32_t)f2bf16(s.y) << 16);
    o.y = f2bf16(s.z) | ((uint32_t)f2bf16(s.w) << 16);
    *reinterpret_cast<uint2*>(a.y + (size_t)t * a.d + j) = o;
  }
}

// row stride of the SwiGLU values: bulk copies want 16-byte rows
int lda(int I) { return (I + 7) / 8 * 8; }

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

size_t block_layout(int B, int E, int top_e, int I, int d, void* base, BlockArgs* a) {
  const size_t P = (size_t)B * top_e;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align256(off + bytes);
    return o;
  };
  // the error word and the split sums' counters sit where they do for every
  // shape and every grouped entry point, so a workspace may be reused for another
  const size_t o_err = take(16), o_split = take(split_bytes((int)P)), o_log = take(sizeof(double) * B * E), o_ids = take(sizeof(int32_t) * P),
               o_w = take(sizeof(float) * P), o_off = take(sizeof(int32_t) * (E + 1)),
               o_rows = take(sizeof(int32_t) * P), o_a = take(sizeof(uint16_t) * P * lda(I)),
               o_out = take(sizeof(float) * P * d);
  if (base && a) {
    char* p = static_cast<char*>(base);
    a->err = reinterpret_cast<uint32_t*>(p + o_err);
    a->logits = reinterpret_cast<double*>(p + o_log);
    a->ids = reinterpret_cast<int32_t*>(p + o_ids);
    a->wts = reinterpret_cast<float*>(p + o_w);
    a->offsets = reinterpret_cast<int32_t*>(p + o_off);
    a->rows = reinterpret_cast<int32_t*>(p + o_rows);
    a->a = reinterpret_cast<uint16_t*>(p + o_a);
    a->out = reinterpret_cast<float*>(p + o_out);
    a->split = p + o_split;
  }
  return off;
}

cudaError_t launch_block(const BlockArgs& a, cudaStream_t s) {
  const int P = a.B * a.top_e;
  logits_kernel<<<dim3(a.B, (a.E + 31) / 32), 256, 0, s>>>(a);
  choose_kernel<<<(a.B + 7) / 8, 256, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_group_rows(P, a.E, a.ids, a.offsets, a.rows, a.err, s);
  if (e != cudaSuccess) return e;
  GroupedArgs g = {};
  g.G = a.E;
  g.P = P;
  g.n_x = a.B;
  g.n_y = P;
  g.N = a.I;
  g.K = a.d;
  g.x = a.x;
  g.x_rows = a.rows;
  g.x_div = a.top_e;
  g.offsets = a.offsets;
  g.w = a.w_gate;
  g.w_up = a.w_up;
  g.y = a.a;
  g.ldx = a.d;
  g.ldy = lda(a.I);
  g.err = a.err;
  g.split = a.split;
  e = launch_grouped(g, s);
  if (e != cudaSuccess) return e;
  GroupedArgs h = {};
  h.G = a.E;
  h.P = P;
  h.n_x = P;
  h.n_y = P;
  h.N = a.d;
  h.K = a.I;
  h.layout = 1;
  h.x = a.a;
  h.x_div = 1;
  h.offsets = a.offsets;
  h.w = a.w_down;
  h.y = a.out;
  h.ldx = lda(a.I);
  h.ldy = a.d;
  h.y_fp32 = 1;
  h.y_rows = a.rows;
  h.err = a.err;
  h.split = a.split;
  e = launch_grouped(h, s);
  if (e != cudaSuccess) return e;
  combine_kernel<<<a.B, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
