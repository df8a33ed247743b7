// The gradient of a router's weights with respect to its logits, the picks being
// fixed (moe_route_grad).  With g the gradient of the weights w and m = sum g w / sum w
// over the picks (renormalised weights; else 0):
//   sigmoid  w (1 - s) (g - m) at the picks,   softmax, renormalised  w (g - m) at the picks,
//   softmax  sum over e's picks of g w - s[e] sum g w  at every expert e, at picks as
//            (1 - s[e]) (e's g w) - s[e] (the others' g w).
// Dividing by sum w, not by the scale, makes m the weights' own mean: a part common to
// all g cancels to the last bit however w was rounded.
//
// One wavefront per token: lane i holds pick i, and expert 4 (lane + 64 j) + i is
// element i of a lane's vector j; elements are stored one by one, as rows start anywhere.
//
// 4096 tokens of 256 experts 4.7 us, 777 of 300, every expert's gradient, 4.9: a launch
// alone is 1.9, the rest a token's loads, reductions and stores, not measured apart.
#include "chunk_dev.h"

namespace moe {

namespace {

struct RouteGradArgs {
  const void* logits;
  const int32_t* ids;
  const float *w, *gw;
  void* out;
  int T, E, k;
  bool lbf, obf, sigmoid, renorm;
};

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

__device__ __forceinline__ double readlane_f64(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __builtin_bit_cast(double, hi << 32 | lo);
}

// V: vectors of four experts a lane.  DENSE: every expert has a gradient.
template <int V, bool DENSE>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs a) {
  const int lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (t >= a.T) return;
  const size_t row = (size_t)t * a.E;
  f32x4 d[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * (lane + 64 * j) + i;
      d[j][i] = DENSE ? (e < a.E ? load1(a.logits, a.lbf, row + e) : -INFINITY) : 0.f;
    }
  }
  // the picks, one a lane
  int id = -1;
  float w = 0.f, g = 0.f;
  if (lane < a.k) {
    id = a.ids[(size_t)t * a.k + lane];
    w = a.w[(size_t)t * a.k + lane];
    g = a.gw[(size_t)t * a.k + lane];
  }
  const bool live = (uint32_t)id < (uint32_t)a.E && w != 0.f;
  if (!live) {
    w = g = 0.f;
    id = -1;
  }
  const float x = live && (DENSE || a.sigmoid) ? load1(a.logits, a.lbf, row + id) : -INFINITY;
  const double gw = (double)g * w, all = wave_sum_f64(gw);
  float mine;
  if constexpr (DENSE) {
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, d[j][i]);  // a NaN is no maximum
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    auto power = [&](float v) { return v > kLowestLogit ? (v == top ? 1.f : expf(v - top)) : 0.f; };  // 0 for NaN
    int tops = 0;
    float below = 0.f;  // sum of the powers but those of the largest logit, which are 1
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[j][i] = power(d[j][i]);
        const bool is_top = d[j][i] == 1.f;
        tops += __popcll(__ballot(is_top));
        below += is_top ? 0.f : d[j][i];
      }
    below = wave_sum(below);
    const double sum = (double)((float)tops + below), inv = sum > 0.0 ? 1.0 / sum : 0.0;
    // At a pick g w - s sum g w as g w (1 - s) - s (the other experts' g w), with 1 - s from the
    // other powers: of a confident router's leader, s near 1, the two terms' difference
    // would keep few of their digits, or none (777 tokens of 300 experts 4.9 us, 4.75 with it).
    double own = 0.0, other = 0.0;
    bool first = live;  // of the picks of its expert
    for (int i = 0; i < a.k; ++i) {
      const bool same = __builtin_amdgcn_readlane(id, i) == id;
      const double v = readlane_f64(gw, i);
      own += same ? v : 0.0;
      other += same ? 0.0 : v;
      first = first && !(same && i < lane);
    }
    const float s = power(x), away = s == 1.f ? (float)(tops - 1) + below : (float)tops + (below - s);
    mine = (float)(sum > 0.0 ? (own * away - s * other) * inv : own);
    if (!first) id = -1;
    const float f = -(float)(all * inv);
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] *= f;
  } else {
    double mean = 0.0;
    if (a.renorm) {
      const double total = wave_sum_f64((double)w);
      mean = total != 0.0 ? all / total : 0.0;
    }
    mine = w * (a.sigmoid && live ? gate_sigmoid(-x) : 1.f) * (float)(g - mean);
  }
  for (int i = 0; i < a.k; ++i) {
    const int e = __builtin_amdgcn_readlane(id, i);
    const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), i));
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int n = 0; n < 4; ++n)
        if (e == 4 * (lane + 64 * j) + n) d[j][n] = DENSE ? v : d[j][n] + v;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = 4 * (lane + 64 * j);
    if (a.obf) {
      uint16_t* o = (uint16_t*)a.out + row + e;
#pragma unroll
      for (int n = 0; n < 4; ++n)
        if (e + n < a.E) o[n] = bf16_of(d[j][n]);
    } else {
      float* o = (float*)a.out + row + e;
#pragma unroll
      for (int n = 0; n < 4; ++n)
        if (e + n < a.E) o[n] = d[j][n];
    }
  }
}

template <int V>
void run(const RouteGradArgs& a, hipStream_t s) {
  const dim3 grid((a.T + 3) / 4), block(256);
  if (a.sigmoid || a.renorm)
    launch(MOE_PROF_ROUTE, route_grad_kernel<V, false>, grid, block, 0, s, a);
  else
    launch(MOE_PROF_ROUTE, route_grad_kernel<V, true>, grid, block, 0, s, a);
}

}  // namespace

moe_status launch_route_grad(const moe_router* R, const void* logits, moe_dtype lt, int T, const int32_t* ids,
                             const float* w, const float* gw, void* glogits, moe_dtype gt, hipStream_t s) {
  const RouteGradArgs a{logits, ids, w,  gw, glogits, T, R->E, R->k, lt == MOE_BF16, gt == MOE_BF16,
                        R->scoring == MOE_SCORE_SIGMOID, R->renorm != 0};
  if (R->E <= 256)
    run<1>(a, s);
  else if (R->E <= 512)
    run<2>(a, s);
  else
    run<4>(a, s);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
