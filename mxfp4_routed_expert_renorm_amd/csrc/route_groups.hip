// Expert choice by softmax or sigmoid scores, a balance bias and groups of
// experts (moe_route_groups).  Scores are compared in double precision: a
// score is an exponential, and two choices that differ by less than fp32's
// rounding of it would otherwise change places.
//
// One wavefront per token, its choices in LDS.
#include "common.h"

namespace moe {

namespace {

constexpr int kMaxE = 1024;
constexpr float kLowest = -0x1.fep127f;  // bf16's lowest value: a logit there or below masks its expert

// the better of (v, i) and another lane's: the larger value, then the lower index
__device__ __forceinline__ void wave_best(double& v, int& i) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const double ov = __shfl_xor(v, off, 64);
    const int oi = __shfl_xor(i, off, 64);
    if (ov > v || (ov == v && oi < i)) v = ov, i = oi;
  }
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

__global__ __launch_bounds__(64) void route_groups_kernel(moe_router R, const void* __restrict__ logits, bool lbf16,
                                                          const float* __restrict__ bias, int32_t* __restrict__ ids,
                                                          float* __restrict__ w) {
  __shared__ double score[kMaxE], choice[kMaxE];
  __shared__ double gval[64];
  const int lane = threadIdx.x, E = R.E, gs = E / R.groups;
  const size_t at = (size_t)blockIdx.x * E;
  const double inf = __longlong_as_double(0x7ff0000000000000ll);
  double top = -inf, sum = 0.0;
  for (int e = lane; e < E; e += 64) {
    float l = lbf16 ? __uint_as_float((uint32_t)((const uint16_t*)logits)[at + e] << 16)
                    : ((const float*)logits)[at + e];
    const double x = l > kLowest ? (double)l : -inf;  // NaN fails the comparison
    score[e] = x;
    top = x > top ? x : top;
  }
  if (R.scoring == MOE_SCORE_SOFTMAX) {
    int unused = 0;
    wave_best(top, unused);
    for (int e = lane; e < E; e += 64) {
      const double x = score[e];
      sum += x == -inf ? 0.0 : x == top ? 1.0 : exp(x - top);
    }
    sum = wave_sum_f64(sum);
  }
  for (int e = lane; e < E; e += 64) {
    const double x = score[e];
    double s = 0.0, c = -inf;
    if (x != -inf) {
      s = R.scoring == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-x)) : (x == top ? 1.0 : exp(x - top)) / sum;
      c = bias ? s + (double)bias[e] : s;
      if (!(c == c)) c = -inf;
    }
    score[e] = c == -inf ? 0.0 : s;
    choice[e] = c;
  }
  __syncthreads();
  unsigned long long in = ~0ull;  // groups that stay
  if (R.topk_groups < R.groups) {
    if (lane < R.groups) {
      double a = -inf, b = -inf;
      for (int j = 0; j < gs; ++j) {
        const double c = choice[lane * gs + j];
        if (c > a) {
          b = a;
          a = c;
        } else if (c > b) {
          b = c;
        }
      }
      gval[lane] = R.group_score == MOE_GROUP_TOP2 && b > -inf ? a + b : a;
    }
    __syncthreads();
    int rank = 64;
    if (lane < R.groups) {
      const double v = gval[lane];
      rank = 0;
      for (int g = 0; g < R.groups; ++g) rank += gval[g] > v || (gval[g] == v && g < lane);
    }
    in = __ballot(rank < R.topk_groups);
  }
  // a pick leaves by joining `taken`, its lane's bit set per expert round
  uint32_t taken = 0;
  double mine_s = -1.0;
  int mine_e = 0x7fffffff;
  for (int r = 0; r < R.k; ++r) {
    double best = -inf;
    int be = 0x7fffffff;
    for (int j = 0; lane + 64 * j < E; ++j) {
      const int e = lane + 64 * j;
      if (((taken >> j) & 1) || !((in >> (e / gs)) & 1)) continue;
      const double c = choice[e];
      if (be == 0x7fffffff || c > best) best = c, be = e;
    }
    wave_best(best, be);  // lanes without a candidate: -inf at an index no expert has
    if ((be & 63) == lane) taken |= 1u << (be >> 6);
    if (lane == r) mine_e = be, mine_s = score[be];
  }
  // falling score, ties to the lower expert: each pick's place by counting
  double total = 0.0;
  int place = 0;
  for (int r = 0; r < R.k; ++r) {
    const double s = __shfl(mine_s, r, 64);
    const int e = __shfl(mine_e, r, 64);
    total += s;
    place += s > mine_s || (s == mine_s && e < mine_e);
  }
  if (lane < R.k) {
    double v = mine_s;
    if (R.renorm) v = total > 0.0 ? v / total : 0.0;
    ids[(size_t)blockIdx.x * R.k + place] = mine_e;
    w[(size_t)blockIdx.x * R.k + place] = (float)(v * (double)R.scale);
  }
}

}  // namespace

moe_status launch_route_groups(const moe_router* R, const void* logits, moe_dtype lt, const float* bias, int T,
                               int32_t* ids, float* w, hipStream_t s) {
  launch(MOE_PROF_ROUTE, route_groups_kernel, dim3(T), dim3(64), 0, s, *R, logits, lt == MOE_BF16, bias, ids, w);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
