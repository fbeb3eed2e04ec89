// block.cu -- the all-channel MoE block over any number of tokens: routing,
// grouping of the (token, slot) pairs by expert, the two grouped products and
// the weighted sum of a token's pairs.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kExactTokens = 32;  // up to here every logit is summed in fp64

// Routing.  The rule is fp64: logits of exact products summed in 64 bits, the
// largest top_e, ties to the lower id, slot 0 the largest.  Up to kExactTokens
// tokens the logits are computed so (route.cu).  Above that, fp64 products of
// every token with every expert would cost more than the experts' products of
// the tokens; there the tensor cores compute logits with fp32 sums (exact
// products), which are off by at most
//   delta = d 2^-23 |x| |w_e|  (2-norms)
// (every partial sum is bounded by |x| |w_e|, and a step of 16 products rounds
// 17 terms).  Experts whose fp32 logits are more than 2 delta apart are in the
// right order; the others near or above the last chosen place are computed
// again in fp64, and the order of the candidates is decided by that.
__device__ __forceinline__ double dot64(const uint16_t* x, const uint16_t* w, int d, int lane) {
  double s = 0.0;
  for (int k = lane * 8; k < d; k += 256) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(x + k)), b = __ldg(reinterpret_cast<const uint4*>(w + k));
    const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {  // products of two bf16 are exact in fp32
      s += (double)(bf16lo(av[i]) * bf16lo(bv[i]));
      s += (double)(bf16hi(av[i]) * bf16hi(bv[i]));
    }
  }
  return warp_sum(s);
}

__device__ __forceinline__ float norm2(const uint16_t* x, int d, int lane) {
  float s = 0.0f;
  for (int k = lane * 8; k < d; k += 256) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(x + k));
    const uint32_t av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      s = fmaf(bf16lo(av[i]), bf16lo(av[i]), s);
      s = fmaf(bf16hi(av[i]), bf16hi(av[i]), s);
    }
  }
  return sqrtf(warp_sum(s)) * 1.001f;  // an upper bound: the fp32 sum is off by less
}

__global__ void __launch_bounds__(256) norms_kernel(BlockArgs a) {
  const int e = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  if (e >= a.E) return;
  const float n = norm2(a.w_router + (size_t)e * a.d, a.d, lane);
  if (lane == 0) a.w_norm[e] = n;
}

// The chosen experts of a token, one to a lane (rank -1: none), with their
// logits: ids by rank, softmax weights over the chosen.
__device__ __forceinline__ void put_choice(const BlockArgs& a, int t, int rank, int id, double v) {
  const bool in = rank >= 0 && rank < a.top_e;
  double m = in ? v : -INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
  const double ex = in ? (double)expf((float)(v - m)) : 0.0;
  const double den = warp_sum(ex);
  if (in) {
    const size_t at = (size_t)t * a.top_e + rank;
    a.ids[at] = id;
    a.wts[at] = (float)(ex / den);
    if (a.ids_out) a.ids_out[at] = id;
  }
}

// The largest `most` of E values (value(e), every lane may ask for any of its
// e = lane + 32 m), in order, ties to the lower id: lane s gets the s-th, as
// long as more(s, value) says so before it is taken.  Returns how many.
template <typename V, typename F, typename M>
__device__ __forceinline__ int take_largest(int E, int lane, int most, F value, M more, V& mine, int& my_id) {
  uint32_t taken = 0;
  int s = 0;
  for (; s < most; s++) {
    V bv = -INFINITY;
    int bi = 0x7fffffff;
    for (int m = 0; lane + 32 * m < E; m++) {
      if (taken & (1u << m)) continue;
      const V v = value(lane + 32 * m);
      if (bi == 0x7fffffff || v > bv) {
        bv = v;
        bi = lane + 32 * m;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const V ov = __shfl_xor_sync(0xffffffffu, bv, o);
      const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
      if (oi != 0x7fffffff && (bi == 0x7fffffff || ov > bv || (ov == bv && oi < bi))) {
        bv = ov;
        bi = oi;
      }
    }
    if (bi == 0x7fffffff || !more(s, bv)) break;
    if ((bi & 31) == lane) taken |= 1u << (bi >> 5);
    if (lane == s) {
      mine = bv;
      my_id = bi;
    }
  }
  return s;
}

// One warp per token.  kExact: the logits are fp64 already.
template <bool kExact>
__global__ void __launch_bounds__(256) choose_kernel(BlockArgs a) {
  const int lane = threadIdx.x & 31, t = blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_trigger();
  pdl_wait();
  if (t >= a.B) return;
  if (kExact) {
    const double* L = a.logits + (size_t)t * a.E;
    double v = 0.0;
    int id = 0;
    const int n = take_largest(
        a.E, lane, a.top_e, [&](int e) { return L[e]; }, [](int, double) { return true; }, v, id);
    put_choice(a, t, lane < n ? lane : -1, id, v);
    return;
  }
  const float* L = a.approx + (size_t)t * a.E;
  const uint16_t* x = a.x + (size_t)t * a.d;
  float w_max = 0.0f, l_max = 0.0f;
  for (int e = lane; e < a.E; e += 32) {
    w_max = fmaxf(w_max, a.w_norm[e]);
    l_max = fmaxf(l_max, fabsf(L[e]) + (a.bias ? fabsf(a.bias[e]) : 0.0f));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    w_max = fmaxf(w_max, __shfl_xor_sync(0xffffffffu, w_max, o));
    l_max = fmaxf(l_max, __shfl_xor_sync(0xffffffffu, l_max, o));
  }
  // the sum's error, and the bias's addition
  const float apart = 2.0f * ((float)a.d * 0x1p-23f * norm2(x, a.d, lane) * w_max + 0x1p-23f * l_max);
  float v = 0.0f, last = 0.0f;
  int id = 0;
  const int n = take_largest(
      a.E, lane, 32, [&](int e) { return L[e] + (a.bias ? a.bias[e] : 0.0f); },
      [&](int s, float b) {
        if (s < a.top_e) last = b;
        return s < a.top_e || last - b <= apart;
      },
      v, id);
  if (n == 32 && a.E > 32) {
    // too many near the border (equal rows, a token of zeros): all of them in fp64
    double all[32];
    for (int e = 0; e < a.E; e++) {
      const double s = dot64(x, a.w_router + (size_t)e * a.d, a.d, lane) + (a.bias ? (double)a.bias[e] : 0.0);
      if ((e & 31) == lane) all[e >> 5] = s;
    }
    double w = 0.0;
    const int k = take_largest(
        a.E, lane, a.top_e, [&](int e) { return all[e >> 5]; }, [](int, double) { return true; }, w, id);
    put_choice(a, t, lane < k ? lane : -1, id, w);
    return;
  }
  const float up = __shfl_up_sync(0xffffffffu, v, 1), down = __shfl_down_sync(0xffffffffu, v, 1);
  const bool near = lane < n && ((lane > 0 && !(up - v > apart)) || (lane + 1 < n && !(v - down > apart)));
  double exact = (double)v;
  for (unsigned todo = __ballot_sync(0xffffffffu, near); todo; todo &= todo - 1) {
    const int s = __ffs(todo) - 1, e = __shfl_sync(0xffffffffu, id, s);
    const double l = dot64(x, a.w_router + (size_t)e * a.d, a.d, lane) + (a.bias ? (double)a.bias[e] : 0.0);
    if (lane == s) exact = l;
  }
  int rank = 0;
  for (int s = 0; s < n; s++) {
    const double o = __shfl_sync(0xffffffffu, exact, s);
    const int oi = __shfl_sync(0xffffffffu, id, s);
    // (a NaN counts as the largest: whatever the order, the ranks stay distinct)
    const bool mine_nan = exact != exact, o_nan = o != o;
    if (o_nan || mine_nan ? (o_nan && (!mine_nan || oi < id)) : (o > exact || (o == exact && oi < id))) rank++;
  }
  put_choice(a, t, lane < n ? rank : -1, id, exact);
}

// y[t] = bf16(residual[t] + sum over the slots, in slot order, of w out).
__global__ void __launch_bounds__(256) combine_kernel(BlockArgs a) {
  const int t = blockIdx.x;
  pdl_trigger();
  pdl_wait();
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
  const size_t o_err = take(16), o_split = take(split_bytes((int)P)), o_log = take(B <= kExactTokens ? sizeof(double) * B * E : 0),
               o_apx = take(B <= kExactTokens ? 0 : sizeof(float) * B * E), o_wn = take(sizeof(float) * E), o_ids = take(sizeof(int32_t) * P),
               o_w = take(sizeof(float) * P), o_off = take(sizeof(int32_t) * (E + 1)),
               o_rows = take(sizeof(int32_t) * P), o_a = take(sizeof(uint16_t) * P * lda(I)),
               o_out = take(sizeof(float) * P * d);
  if (base && a) {
    char* p = static_cast<char*>(base);
    a->err = reinterpret_cast<uint32_t*>(p + o_err);
    a->logits = reinterpret_cast<double*>(p + o_log);
    a->approx = reinterpret_cast<float*>(p + o_apx);
    a->w_norm = reinterpret_cast<float*>(p + o_wn);
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
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto launch = [&](auto kernel, int grid) {
    cfg.gridDim = dim3(grid);
    return cudaLaunchKernelEx(&cfg, kernel, a);
  };
  cudaError_t e;
  if (a.B <= kExactTokens) {
    RouteArgs r = {};
    r.B = a.B;
    r.E = a.E;
    r.d = a.d;
    r.x = a.x;
    r.w_router = a.w_router;
    r.bias = a.bias;
    r.ws.logits = a.logits;
    e = launch_logits(r, s);
    if (e == cudaSuccess) e = launch(choose_kernel<true>, (a.B + 7) / 8);
  } else {
    e = launch(norms_kernel, (a.E + 7) / 8);
    if (e != cudaSuccess) return e;
    GroupedArgs l = {};
    l.G = 1;
    l.P = l.n_x = l.n_y = a.B;
    l.N = l.ldy = a.E;
    l.K = l.ldx = a.d;
    l.x = a.x;
    l.x_div = 1;
    l.w = a.w_router;
    l.y = a.approx;
    l.y_fp32 = 1;
    l.err = a.err;
    l.split = a.split;
    e = launch_grouped(l, s);
    if (e == cudaSuccess) e = launch(choose_kernel<false>, (a.B + 7) / 8);
  }
  if (e != cudaSuccess) return e;
  e = launch_group_rows(P, a.E, a.ids, a.offsets, a.rows, s);
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
  return launch(combine_kernel, a.B);
}

}  // namespace moe
