// Expert choice by softmax or sigmoid scores, a balance bias and groups of
// experts (moe_route_groups).  Scores are compared in double precision: a
// score is an exponential, and two choices that differ by less than fp32's
// rounding of it would otherwise change places.
//
// One wavefront per token, expert lane + 64 j in register j of a lane.  The k
// best choices are found without sorting: their images (order-preserving
// integers) are compared with a threshold that is halved in until exactly k are
// not below it.  A step is one comparison and one count of a lane mask per
// register, whatever k is.
//
// An exponential in double precision costs some 70 instructions, and with one
// for every expert a launch of 4096 tokens is bound by them.  So the choices are
// first formed in fp32, whose error is bounded, to find which experts can be
// among the k best at all: those within the bound of the k-th.  They are mostly
// k, and only they, one a lane, get scores in double precision.  Where fp32
// cannot tell the groups apart, or leaves more than 64 experts, the wavefront
// takes every score in double precision instead (as where the bias or an
// infinity would break the bound, and for softmax with a bias, whose denominator
// counts in the comparison).  A softmax that is not renormalised needs its
// denominator, a double exponential an expert, for the weights alone: 777 tokens of
// 300 experts 8.8 us, renormalised 8.0.
//
// Instructions and their latency bound it, not bytes: 4096 tokens of 256 experts
// (sigmoid, bias, 8 of 256 out of 4 of 8 groups) 10.1 us, 587 vector and 658
// scalar instructions a wavefront, four wavefronts a SIMD, whose vector instructions
// fill 9,400 of its 16,800 cycles: the rest are waits in a chain of threshold steps,
// each a count that decides the next.  Without groups 7.8 us; with every score in double
// 10.9 us, with k rounds of a maximum over 64-bit values 36 us.  One token: 5.4 us.
#include "chunk_dev.h"
#include "route_dev.h"

namespace moe {

namespace {

constexpr int kWaves = 4;  // tokens a workgroup
constexpr uint32_t kMasked = 0x000fffffu;  // high word of -inf's image
// fp32 choices, with |bias| <= kMaxBias, are off by less than 8e-7: the score by
// 2.1e-7 (s (1 - s) of the exponential's relative error, |x| 2^-23 and two steps,
// and the reciprocal's step), the sum with the bias by half a step of 9.  Two of
// them are told apart beyond twice that; sums of two, rounded once more, beyond
// 5.4e-6.
constexpr float kMaxBias = 8.0f, kApart = 2e-6f, kGroupsApart = 8e-6f;
constexpr float kLowest = -0x1.fep127f;  // bf16's lowest value: a logit there or below masks its expert

__device__ __forceinline__ double make_f64(uint32_t lo, uint32_t hi) {
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ uint32_t lo32(double v) { return (uint32_t)__double_as_longlong(v); }
__device__ __forceinline__ uint32_t hi32(double v) { return (uint32_t)((uint64_t)__double_as_longlong(v) >> 32); }

__device__ __forceinline__ double readlane_f64(double v, int lane) {
  return make_f64(__builtin_amdgcn_readlane(lo32(v), lane), __builtin_amdgcn_readlane(hi32(v), lane));
}

// sum over the wavefront, in every lane (the moves of wave_ext_u32)
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  return make_f64(__builtin_amdgcn_update_dpp(0, (int)lo32(v), CTRL, 0xF, 0xF, false),
                  __builtin_amdgcn_update_dpp(0, (int)hi32(v), CTRL, 0xF, 0xF, false));
}

__device__ __forceinline__ double wave_sum_f64(double v) {
  v += dpp_f64<dpp::kQuadXor1>(v);
  v += dpp_f64<dpp::kQuadXor2>(v);
  v += dpp_f64<dpp::kRowHalfMirror>(v);
  v += dpp_f64<dpp::kRowMirror>(v);
  const auto a = __builtin_amdgcn_permlane16_swap(lo32(v), lo32(v), false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(hi32(v), hi32(v), false, false);
  v = make_f64(a[0], b[0]) + make_f64(a[1], b[1]);
  const auto c = __builtin_amdgcn_permlane32_swap(lo32(v), lo32(v), false, false);
  const auto d = __builtin_amdgcn_permlane32_swap(hi32(v), hi32(v), false, false);
  return make_f64(c[0], d[0]) + make_f64(c[1], d[1]);
}

// how many of the wavefront's keys are at or above t
template <int EPL>
__device__ __forceinline__ int count_from(const uint32_t (&key)[EPL], uint32_t t) {
  int n = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) n += __popcll(__ballot(key[j] >= t));
  return n;
}

// The threshold at or above which `need` keys lie, or, where a tie makes that
// impossible, the tied value: the largest threshold with at least `need`.
// Keys of 0 are no candidates; there are `need` others at least.  Keys up to
// `far` lie apart from the others and are looked at only if those do not suffice.
template <int EPL>
__device__ __forceinline__ uint32_t threshold(const uint32_t (&key)[EPL], int need, uint32_t far = 0) {
  if (far && count_from(key, far + 1u) < need) far = 0;
  uint32_t most = 0, least = 0xffffffffu;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    most = key[j] > most ? key[j] : most;
    least = min(least, key[j] - far - 1u);  // 0 .. far wrap to the top
  }
  uint32_t lo = __builtin_amdgcn_readfirstlane(wave_ext_u32<false>(least)) + far + 1u;
  uint32_t hi = __builtin_amdgcn_readfirstlane(wave_ext_u32<true>(most));
  if (count_from(key, hi) >= need) return hi;
  while (hi - lo > 1u) {  // at least `need` from lo on, fewer from hi on
    const uint32_t mid = lo + (hi - lo) / 2;
    const int n = count_from(key, mid);
    if (n == need) return mid;
    if (n > need)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float readlane_any(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double readlane_any(double v, int lane) { return readlane_f64(v, lane); }

// The groups that stay, a bit each, from the choices (-inf: masked).  last: the
// value of the last that stays; apart: how far it is above the best that does not;
// near: whether a group's value is within kApart of it without being equal.
template <class F, int EPL>
__device__ __forceinline__ uint64_t best_groups(const moe_router& R, const F (&c)[EPL], F* lds, F* last, F* apart,
                                                bool* near) {
  const int lane = threadIdx.x & 63, gs = R.E / R.groups;
  const F inf = (F)INFINITY;
  int per = 64;  // lanes a group: a power of two
  while (per * R.groups > 64) per >>= 1;
#pragma unroll
  for (int j = 0; j < EPL; ++j) lds[lane + 64 * j] = c[j];
  wave_turn();
  const int g = lane / per;
  F first = -inf, second = -inf;  // the two best of this lane's part of its group
  if (g < R.groups) {
    for (int i = lane % per; i < gs; i += per) {
      const F v = lds[g * gs + i];
      second = fmax(second, fmin(first, v));
      first = fmax(first, v);
    }
  }
  for (int off = 1; off < per; off *= 2) {
    const F f = __shfl_xor(first, off, 64), n = __shfl_xor(second, off, 64);
    second = fmax(fmax(second, n), fmin(first, f));
    first = fmax(first, f);
  }
  const F value = R.group_score == MOE_GROUP_TOP2 && second > -inf ? first + second : first;
  int rank = 0;
  for (int i = 0; i < R.groups; ++i) {
    const F v = readlane_any(value, i * per);
    rank += v > value || (v == value && i < g);
  }
  const bool leads = g < R.groups && lane % per == 0;
  const uint64_t kept = __ballot(leads && rank < R.topk_groups);
  *last = readlane_any(value, __ffsll((unsigned long long)__ballot(leads && rank == R.topk_groups - 1)) - 1);
  *apart = *last - readlane_any(value, __ffsll((unsigned long long)__ballot(leads && rank == R.topk_groups)) - 1);
  *near = __ballot(leads && value != *last && fabs(value - *last) <= (F)kApart) != 0;
  if (per == 1) return kept;
  uint64_t stay = 0;
  for (int i = 0; i < R.groups; ++i) stay |= ((kept >> (i * per)) & 1) << i;
  return stay;
}

__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// Lane i < n of the picks' lanes holds one: expert e, score s (ascending e over
// the lanes).  Writes them in order of falling score, ties to the lower expert.
__device__ __forceinline__ void write_picks(const moe_router& R, uint64_t picks, int e, double s, double over,
                                            int32_t* __restrict__ ids, float* __restrict__ w) {
  const int lane = threadIdx.x & 63;
  double total = 0.0;
  int place = 0;
  for (uint64_t m = picks; m; m &= m - 1) {
    const int i = __ffsll((unsigned long long)m) - 1;
    const double v = readlane_f64(s, i);
    total += v;
    place += v > s || (v == s && i < lane);
  }
  if ((picks >> lane) & 1) {
    const double by = R.renorm ? total : over;
    ids[place] = e;
    w[place] = (float)((by > 0.0 ? s / by : 0.0) * (double)R.scale);
  }
}

// a softmax's exponential in double precision; a masked expert's is 0 (NaN too)
__device__ __forceinline__ double soft_exp(float l, float top) {
  return !(l > kLowest) ? 0.0 : l == top ? 1.0 : exp((double)l - (double)top);
}

template <int EPL>
__global__ __launch_bounds__(64 * kWaves) void route_groups_kernel(moe_router R, int T, uint32_t inv_gs,
                                                                   const void* __restrict__ logits, bool lbf16,
                                                                   const float* __restrict__ bias,
                                                                   int32_t* __restrict__ ids, float* __restrict__ w) {
  __shared__ double choice[kWaves][EPL * 64];
  __shared__ double pick_s[kWaves][64];
  __shared__ int pick_e[kWaves][64];
  __shared__ float pick_l[kWaves][64], pick_b[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.x * kWaves + wave, E = R.E;
  if (t >= T) return;  // the whole wavefront: nothing below is shared between wavefronts
  const double inf = __longlong_as_double(0x7ff0000000000000ll);
  const size_t at = (size_t)t * E;
  float l[EPL], b[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = min(lane + 64 * j, E - 1);
    l[j] = lbf16 ? __uint_as_float((uint32_t)((const uint16_t*)logits)[at + e] << 16) : ((const float*)logits)[at + e];
    b[j] = bias ? bias[e] : 0.f;
  }

  const bool sigmoid_scores = R.scoring == MOE_SCORE_SIGMOID;
  float top = 0.f;  // softmax: the largest logit
  if (!sigmoid_scores) {
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) best = max(best, sel_key(l[j]));
    top = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(key_value(wave_ext_u32<true>(best)))));
  }
  int32_t* my_ids = ids + (size_t)t * R.k;
  float* my_w = w + (size_t)t * R.k;

  if (sigmoid_scores || (!bias && top > kLowest && top < INFINITY)) {
    float c[EPL];
    bool wide = false;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const bool live = l[j] > kLowest;
      if (sigmoid_scores) {
        c[j] = sigmoid(l[j]) + b[j];
        wide |= live && fabsf(b[j]) > kMaxBias;
        c[j] = live && c[j] == c[j] ? c[j] : -INFINITY;
      } else {
        c[j] = live ? __expf(l[j] - top) : -INFINITY;
      }
    }
    bool sure = __ballot(wide) == 0;
    uint64_t stay = ~0ull;
    if (sure && R.topk_groups < R.groups) {
      float last, apart;
      bool near;
      if (!sigmoid_scores && R.group_score == MOE_GROUP_MAX) {
        // by the logits themselves, down to where scores underflow.  Ties of logits are ties of the
        // scores, but scores also tie where logits differ by less than a double exponential shows.
        float v[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) v[j] = l[j] > kLowest ? l[j] : -INFINITY;
        stay = best_groups<float, EPL>(R, v, (float*)choice[wave], &last, &apart, &near);
        sure = last > top - 700.f && (apart == 0.f ? !near : apart > kApart);
      } else {
        stay = best_groups<float, EPL>(R, c, (float*)choice[wave], &last, &apart, &near);
        sure = apart > kGroupsApart;
      }
    }
    if (sure) {
      uint32_t key[EPL];
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int e = lane + 64 * j;
        key[j] = e < E && ((stay >> (((uint32_t)e * inv_gs) >> 22)) & 1) ? sel_key(c[j]) : 0u;
      }
      constexpr uint32_t kNone = 0x007fffffu;  // -inf's image
      const uint32_t cut = threshold(key, R.k, kNone);
      const uint32_t from = cut > kNone ? sel_key(key_value(cut) - kApart) : 0u;
      const int n = cut > kNone ? count_from(key, from) : 65;
      if (n <= 64) {  // one candidate a lane, in order of id
        int at = 0;
        wave_turn();
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const uint64_t in = __ballot(key[j] >= from);
          if ((in >> lane) & 1) {
            const int p = at + lanes_below(in);
            pick_e[wave][p] = lane + 64 * j;
            pick_l[wave][p] = l[j];
            pick_b[wave][p] = b[j];
          }
          at += __popcll(in);
        }
        wave_turn();
        const int e = pick_e[wave][lane];
        const double x = (double)pick_l[wave][lane];
        const double z = exp(sigmoid_scores ? -x : x - (double)top);
        const double s = sigmoid_scores ? 1.0 / (1.0 + z) : z;
        uint64_t picks = n == 64 ? ~0ull : (1ull << n) - 1;
        if (n > R.k) {
          const double ch = sigmoid_scores ? s + (double)pick_b[wave][lane] : s;
          int before = 0;
          for (int i = 0; i < n; ++i) {
            const double v = readlane_f64(ch, i);
            before += v > ch || (v == ch && i < lane);
          }
          picks = __ballot(lane < n && before < R.k);
        }
        double over = 1.0;
        if (!sigmoid_scores && !R.renorm) {  // the weights' denominator: every expert's exponential
          over = 0.0;
#pragma unroll
          for (int j = 0; j < EPL; ++j) over += lane + 64 * j < E ? soft_exp(l[j], top) : 0.0;
          over = wave_sum_f64(over);
        }
        write_picks(R, picks, e, s, over, my_ids, my_w);
        return;
      }
    }
  }

  // every score in double precision; a masked expert's are 0 and -inf
  double s[EPL], c[EPL];
  if (sigmoid_scores) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) s[j] = l[j] > kLowest ? 1.0 / (1.0 + exp(-(double)l[j])) : 0.0;  // NaN: 0
  } else {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      s[j] = soft_exp(l[j], top);
      sum += lane + 64 * j < E ? s[j] : 0.0;
    }
    sum = wave_sum_f64(sum);
#pragma unroll
    for (int j = 0; j < EPL; ++j) s[j] = sum > 0.0 ? s[j] / sum : 0.0;
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    c[j] = s[j] + (double)b[j];
    const bool live = l[j] > kLowest && c[j] > -inf;
    c[j] = live ? c[j] + 0.0 : -inf;  // -0 becomes 0
    s[j] = live ? s[j] : 0.0;
  }
  uint64_t stay = ~0ull;  // groups
  if (R.topk_groups < R.groups) {
    double last, apart;
    bool near;
    wave_turn();
    stay = best_groups<double, EPL>(R, c, choice[wave], &last, &apart, &near);
  }

  // images: 0 for what is no candidate
  uint32_t hi[EPL], lo[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 64 * j;
    const uint64_t u = (uint64_t)__double_as_longlong(c[j]);
    const uint64_t image = (u >> 63) ? ~u : u | 0x8000000000000000ull;
    const bool in = e < E && ((stay >> (((uint32_t)e * inv_gs) >> 22)) & 1);
    hi[j] = in ? (uint32_t)(image >> 32) : 0u;
    lo[j] = (uint32_t)image;
  }
  const uint32_t cut = threshold(hi, R.k, kMasked);
  uint64_t take[EPL];  // lanes whose register j is picked
  int n = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    take[j] = __ballot(hi[j] >= cut);
    n += __popcll(take[j]);
  }
  if (n > R.k) {  // a tie on the high words at the cut
    n = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      take[j] = __ballot(hi[j] > cut);
      n += __popcll(take[j]);
    }
    // low words as keys: halved so that no candidate's is 0, the lowest bit apart
    uint32_t key[EPL];
    int left = R.k - n;
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = hi[j] == cut ? (lo[j] >> 1) + 1u : 0u;
    const uint32_t cut1 = threshold(key, left);
    uint32_t bit[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const uint64_t above = __ballot(key[j] > cut1);
      take[j] |= above;
      left -= __popcll(above);
      bit[j] = key[j] == cut1 ? (lo[j] & 1u) + 1u : 0u;
    }
    const uint32_t cut2 = threshold(bit, left);
    int taken = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const uint64_t above = __ballot(bit[j] > cut2);
      take[j] |= above;
      taken += __popcll(above);
    }
    left -= taken;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {  // equal choices: the lower ids
      const uint64_t same = __ballot(bit[j] == cut2);
      const int before = lanes_below(same);
      take[j] |= __ballot(bit[j] == cut2 && before < left);
      left -= min(left, (int)__popcll(same));
    }
  }

  // picks to the lanes in order of id
  int from = 0;
  wave_turn();
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    if ((take[j] >> lane) & 1) {
      const int p = from + lanes_below(take[j]);
      pick_s[wave][p] = s[j];
      pick_e[wave][p] = lane + 64 * j;
    }
    from += __popcll(take[j]);
  }
  wave_turn();
  write_picks(R, R.k == 64 ? ~0ull : (1ull << R.k) - 1, pick_e[wave][lane], pick_s[wave][lane], 1.0, my_ids, my_w);
}

}  // namespace

moe_status launch_route_groups(const moe_router* R, const void* logits, moe_dtype lt, const float* bias, int T,
                               int32_t* ids, float* w, hipStream_t s) {
  const int epl = (R->E + 63) / 64, gs = R->E / R->groups;
  const uint32_t inv = ((1u << 22) + gs - 1) / gs;  // e / gs = e inv >> 22 for e < 1024
  const dim3 grid((T + kWaves - 1) / kWaves), block(64 * kWaves);
  const bool h = lt == MOE_BF16;
  // registers a lane: every count up to 8, where 128 to 512 experts lie, then 12 and 16
  auto* kernel = epl <= 1   ? route_groups_kernel<1>
                 : epl == 2 ? route_groups_kernel<2>
                 : epl == 3 ? route_groups_kernel<3>
                 : epl == 4 ? route_groups_kernel<4>
                 : epl == 5 ? route_groups_kernel<5>
                 : epl == 6 ? route_groups_kernel<6>
                 : epl <= 8 ? route_groups_kernel<8>
                 : epl <= 12 ? route_groups_kernel<12>
                             : route_groups_kernel<16>;
  launch(MOE_PROF_ROUTE, kernel, grid, block, 0, s, *R, T, inv, logits, h, bias, ids, w);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
