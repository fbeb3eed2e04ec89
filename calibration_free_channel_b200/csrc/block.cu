// block.cu -- the all-channel MoE block over any number of tokens: routing,
// grouping of the (token, slot) pairs by expert, the two grouped products and
// the weighted sum of a token's pairs.
#include "common.cuh"
#include "kernels.h"
#include "sort.cuh"

namespace moe {

namespace {

// Up to here every logit is summed in fp64 (whole Qwen-sized block: 32 tokens
// 210 us against 229 by the tensor cores' logits, 64 248 against 253, 128 258
// against 256).
constexpr int kExactTokens = 64;

// Routing.  The rule is fp64: logits of exact products summed in 64 bits, the
// largest top_e, ties to the lower id, slot 0 the largest.  Up to kExactTokens
// tokens the logits are computed so (route.cu).  Above that, fp64 products of
// every token with every expert would cost more than the experts' products of
// the tokens; there the tensor cores compute logits with fp32 sums (exact
// products), which are off by at most
//   delta = d 2^-23 |x| |w_e|  (2-norms)
// and a sixteenth more (every partial sum is bounded by |x| |w_e|, and a step
// of 16 products cuts 17 terms), and by 2^-125 for each product that may be
// too small for a normal number.  Experts whose fp32 logits are more than 2 delta apart are in the
// right order; the others near or above the last chosen place are computed
// again in fp64, and the order of the candidates is decided by that.  Where a
// sum may leave the range of fp32, all of a token's are.
__device__ __forceinline__ void dot64x2(const uint16_t* x, const uint16_t* w0, const uint16_t* w1, int d, int lane,
                                        double& s0, double& s1) {
  s0 = s1 = 0.0;
#pragma unroll 4
  for (int k = lane * 8; k < d; k += 256) {
    const uint4 a = *reinterpret_cast<const uint4*>(x + k), b = *reinterpret_cast<const uint4*>(w0 + k),
                c = *reinterpret_cast<const uint4*>(w1 + k);
    const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w}, cv[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {  // products of two bf16 are exact in fp64 (in fp32 the smallest and largest are not)
      const double lo = bf16lo(av[i]), hi = bf16hi(av[i]);
      s0 = fma(lo, (double)bf16lo(bv[i]), s0);
      s0 = fma(hi, (double)bf16hi(bv[i]), s0);
      s1 = fma(lo, (double)bf16lo(cv[i]), s1);
      s1 = fma(hi, (double)bf16hi(cv[i]), s1);
    }
  }
  s0 = warp_sum(s0);
  s1 = warp_sum(s1);
}

// A logit that is not a number ranks last (the token's weights are NaN then).
template <typename V>
__device__ __forceinline__ V ranked(V v) {
  return v == v ? v : (V)-INFINITY;
}

// An upper bound of the 2-norm: fp32 sums are off by less than a thousandth
// unless squares leave the range, and are summed in fp64 then.
__device__ __forceinline__ float norm2(const uint16_t* x, int d, int lane) {
  float s = 0.0f;
#pragma unroll 4
  for (int k = lane * 8; k < d; k += 256) {
    const uint4 a = *reinterpret_cast<const uint4*>(x + k);
    const uint32_t av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      s = fmaf(bf16lo(av[i]), bf16lo(av[i]), s);
      s = fmaf(bf16hi(av[i]), bf16hi(av[i]), s);
    }
  }
  s = warp_sum(s);
  if (s > 0x1p-60f && s < 0x1p120f) return sqrtf(s) * 1.001f;
  double t = 0.0;
  for (int k = lane; k < d; k += 32) {
    const double v = bf16f(x[k]);
    t = fma(v, v, t);
  }
  return __double2float_ru(sqrt(warp_sum(t)) * 1.001);
}

__global__ void __launch_bounds__(256) norms_kernel(BlockArgs a) {
  // beside the logits' launch, which lets this one start when everything
  // earlier is complete
  const int e = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  pdl_trigger();
  if (e < a.E) {
    const float n = norm2(a.w_router + (size_t)e * a.d, a.d, lane);
    if (lane == 0) a.w_norm[e] = n;
  }
  pdl_wait();  // whoever waits for this launch waits for the logits too
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

// Takes the largest of the values that the lanes hold (expert lane + 32 m in
// v[m]), ties to the lower id; `taken` marks this lane's that are gone.
template <int kM, typename V>
__device__ __forceinline__ void largest(const V (&v)[kM], int E, int lane, uint32_t& taken, V& best, int& id) {
  best = -INFINITY;
  id = 0x7fffffff;
#pragma unroll
  for (int m = 0; m < kM; m++)
    if (lane + 32 * m < E && !(taken >> m & 1) && (id == 0x7fffffff || v[m] > best)) {
      best = v[m];
      id = lane + 32 * m;
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const V ov = __shfl_xor_sync(0xffffffffu, best, o);
    const int oi = __shfl_xor_sync(0xffffffffu, id, o);
    if (oi != 0x7fffffff && (id == 0x7fffffff || ov > best || (ov == best && oi < id))) {
      best = ov;
      id = oi;
    }
  }
  if ((id & 31) == lane && id != 0x7fffffff) taken |= 1u << (id >> 5);
}

// The choice by fp64 logits, one warp; E <= 32 kM.
template <int kM>
__device__ __forceinline__ void choose_exact(const BlockArgs& a, int t, int lane) {
  uint32_t taken = 0;
  int id = 0;
  double v[kM], mine = 0.0;
#pragma unroll
  for (int m = 0; m < kM; m++) v[m] = lane + 32 * m < a.E ? ranked(a.logits[(size_t)t * a.E + lane + 32 * m]) : 0.0;
  for (int s = 0; s < a.top_e; s++) {
    double best;
    int e;
    largest(v, a.E, lane, taken, best, e);
    if (lane == s) {
      mine = best;
      id = e;
    }
  }
  put_choice(a, t, lane < a.top_e ? lane : -1, id, mine);
}

// Few tokens and experts: the choice and the plan of its pairs in one CTA,
// one launch less (of about 4 us each) in the chain of a small block.
__global__ void __launch_bounds__(1024) choose_and_group_kernel(BlockArgs a, int bits, int stretch) {
  extern __shared__ uint8_t raw[];
  pdl_trigger();
  sort_rows(a.B * a.top_e, a.E, bits, stretch, a.ids, a.offsets, a.rows, raw, [&] {
    pdl_wait();
    for (int t = threadIdx.x >> 5; t < a.B; t += 32) choose_exact<4>(a, t, threadIdx.x & 31);
    __syncthreads();  // (the ids, written through global memory by this CTA)
  });
}

// The logits of two experts for token x, in fp64.
__device__ __forceinline__ void exact_logits(const BlockArgs& a, const uint16_t* x, int e0, int e1, int lane,
                                             double& l0, double& l1) {
  dot64x2(x, a.w_router + (size_t)e0 * a.d, a.w_router + (size_t)e1 * a.d, a.d, lane, l0, l1);
  l0 = ranked(l0 + (a.bias ? (double)a.bias[e0] : 0.0));
  l1 = ranked(l1 + (a.bias ? (double)a.bias[e1] : 0.0));
}

// One warp per token, E <= 32 kM.  kExact: the logits are fp64 already.
template <int kM, bool kExact>
__global__ void __launch_bounds__(256) choose_kernel(BlockArgs a) {
  const int lane = threadIdx.x & 31, t = blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_trigger();
  pdl_wait();
  if (t >= a.B) return;
  uint32_t taken = 0;
  int id = 0;
  if (kExact) {
    choose_exact<kM>(a, t, lane);
    return;
  }
  const uint16_t* x = a.x + (size_t)t * a.d;
  float v[kM], w_max = 0.0f, l_max = 0.0f;
#pragma unroll
  for (int m = 0; m < kM; m++) {
    const int e = lane + 32 * m;
    v[m] = 0.0f;
    if (e < a.E) {
      const float l = a.approx[(size_t)t * a.E + e], b = a.bias ? a.bias[e] : 0.0f;
      v[m] = ranked(l + b);
      w_max = fmaxf(w_max, a.w_norm[e]);
      // (a bias of -infinity takes an expert out, in any precision: with it here
      // every logit would be summed in fp64, 8192 tokens 1534 instead of 851 us)
      if (v[m] > -INFINITY) l_max = fmaxf(l_max, fabsf(l) + fabsf(b));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    w_max = fmaxf(w_max, __shfl_xor_sync(0xffffffffu, w_max, o));
    l_max = fmaxf(l_max, __shfl_xor_sync(0xffffffffu, l_max, o));
  }
  // the sum's error, and the bias's addition
  const float most = norm2(x, a.d, lane) * w_max;
  const float apart = 2.0f * (1.0625f * (float)a.d * (0x1p-23f * most + 0x1p-125f) + 0x1p-23f * l_max);
  const bool in_range = most < 0x1p126f && l_max < 0x1p126f;
  // the chosen by these logits, in order, one to a lane, and behind them
  // those within reach of the last
  float mine = 0.0f, last = 0.0f;
  int n = 0;
  for (; in_range && n < 32 && n < a.E; n++) {
    float best;
    int e;
    largest(v, a.E, lane, taken, best, e);
    if (n >= a.top_e && !(last - best <= apart)) break;
    if (n < a.top_e) last = best;
    if (lane == n) {
      mine = best;
      id = e;
    }
  }
  if (!in_range || (n == 32 && a.E > 32)) {
    // out of range, or too many within reach (equal rows, a token of zeros): all of them in fp64
    double all[kM], got = 0.0;
#pragma unroll
    for (int m = 0; m < kM; m++) {
      all[m] = 0.0;
      for (int l = 0; l < 32 && l + 32 * m < a.E; l += 2) {
        double s0, s1;
        exact_logits(a, x, l + 32 * m, min(l + 1 + 32 * m, a.E - 1), lane, s0, s1);
        if (l == lane) all[m] = s0;
        if (l + 1 == lane) all[m] = s1;
      }
    }
    taken = 0;
    for (int s = 0; s < a.top_e; s++) {
      double best;
      int e;
      largest(all, a.E, lane, taken, best, e);
      if (lane == s) {
        got = best;
        id = e;
      }
    }
    put_choice(a, t, lane < a.top_e ? lane : -1, id, got);
    return;
  }
  const float up = __shfl_up_sync(0xffffffffu, mine, 1), down = __shfl_down_sync(0xffffffffu, mine, 1);
  const bool near = lane < n && ((lane > 0 && !(up - mine > apart)) || (lane + 1 < n && !(mine - down > apart)));
  double exact = (double)mine;
  for (unsigned todo = __ballot_sync(0xffffffffu, near); todo;) {  // two at a time
    const int s0 = __ffs(todo) - 1;
    todo &= todo - 1;
    const int s1 = todo ? __ffs(todo) - 1 : s0;
    todo &= todo - 1;
    double l0, l1;
    exact_logits(a, x, __shfl_sync(0xffffffffu, id, s0), __shfl_sync(0xffffffffu, id, s1), lane, l0, l1);
    if (lane == s0) exact = l0;
    if (lane == s1) exact = l1;
  }
  int rank = 0;
  for (int s = 0; s < n; s++) {
    const double o = __shfl_sync(0xffffffffu, exact, s);
    const int oi = __shfl_sync(0xffffffffu, id, s);
    if (o > exact || (o == exact && oi < id)) rank++;
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

// The SwiGLU values go to the second product as bf16, which adds as much error
// to the result as its own rounding does.  While an expert has 64 tokens or
// fewer on average they are held in two bf16 terms, 16 significant bits: the
// second product is bound by its weights there, and the second term's rows and
// products cost 2 % of the whole (1024 tokens, 128 experts, top-8: 301 against
// 295 us).  Above that they cost more: 9 % at 2048 tokens, 18 % at 8192 (1000
// against 846 us), in the end half of the products again; one term it is there,
// as wide as every input and output of the block, and the result's error
// against 64 bits 0.0023 of it instead of 0.0017.
bool two_terms(int B, int E, int top_e) { return (long)B * top_e <= 64L * E; }

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
               o_rest = take(two_terms(B, E, top_e) ? sizeof(uint16_t) * P * lda(I) : 0),
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
    a->a_rest = two_terms(B, E, top_e) ? reinterpret_cast<uint16_t*>(p + o_rest) : nullptr;
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
  const int by8 = (a.B + 7) / 8;
  bool grouped = false;
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
    if (e == cudaSuccess && a.E <= 128) {
      const int stretch = sort_stretch(P, 1);
      cudaLaunchConfig_t one = cfg;
      one.gridDim = dim3(1);
      one.blockDim = dim3(1024);
      one.dynamicSmemBytes = sort_bytes(P, a.E, stretch);  // (32 warps' tables of 129 counts at most)
      e = cudaLaunchKernelEx(&one, choose_and_group_kernel, a, sort_bits(a.E), stretch);
      grouped = true;
    } else if (e == cudaSuccess) {
      e = launch(choose_kernel<32, true>, by8);
    }
  } else {
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
    l.late_trigger = 1;
    e = launch_grouped(l, s);
    if (e == cudaSuccess) e = launch(norms_kernel, (a.E + 7) / 8);
    if (e == cudaSuccess)
      e = a.E <= 128 ? launch(choose_kernel<4, false>, by8) : launch(choose_kernel<32, false>, by8);
  }
  if (e == cudaSuccess && !grouped) e = launch_group_rows(P, a.E, a.ids, a.offsets, a.rows, s);
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
  g.y_rest = a.a_rest;
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
  h.x_rest = a.a_rest;
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
