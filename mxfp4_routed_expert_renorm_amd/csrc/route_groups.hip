// Expert choice by softmax or sigmoid scores, a balance bias and groups of
// experts (moe_route_groups).  Scores are compared in double precision: a
// score is an exponential, and two choices that differ by less than fp32's
// rounding of it would otherwise change places.
//
// One wavefront per token, expert lane + 64 j in register j of a lane.  The k
// best choices are found without sorting: their 64-bit images (order-preserving
// integers) are compared with a threshold that is halved in until exactly k are
// not below it, first on the images' high words, and only where those tie on
// the low words and then on the expert ids.  A step is one comparison and one
// count of a lane mask per register, whatever k is.  What is picked goes
// through LDS in order of expert id and finds its place by counting.
#include "route_dev.h"

namespace moe {

namespace {

constexpr int kMaxE = 1024;
constexpr int kWaves = 4;  // tokens a workgroup
constexpr uint32_t kMasked = 0x000fffffu;  // high word of -inf's image
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

template <int EPL>
__global__ __launch_bounds__(64 * kWaves) void route_groups_kernel(moe_router R, int T, uint32_t inv_gs,
                                                                   const void* __restrict__ logits, bool lbf16,
                                                                   const float* __restrict__ bias,
                                                                   int32_t* __restrict__ ids, float* __restrict__ w) {
  __shared__ double choice[kWaves][EPL * 64];
  __shared__ double pick_s[kWaves][64];
  __shared__ int pick_e[kWaves][64];
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

  // scores and choices; a masked expert's are 0 and -inf
  double s[EPL], c[EPL];
  if (R.scoring == MOE_SCORE_SIGMOID) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) s[j] = l[j] > kLowest ? 1.0 / (1.0 + exp(-(double)l[j])) : 0.0;  // NaN: 0
  } else {
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) best = max(best, sel_key(l[j]));
    const float top = key_value(wave_ext_u32<true>(best));
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      s[j] = !(l[j] > kLowest) ? 0.0 : l[j] == top ? 1.0 : exp((double)l[j] - (double)top);
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
    const int gs = E / R.groups;
    int per = 64;  // lanes a group: a power of two
    while (per * R.groups > 64) per >>= 1;
#pragma unroll
    for (int j = 0; j < EPL; ++j) choice[wave][lane + 64 * j] = c[j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const int g = lane / per;
    double first = -inf, second = -inf;  // the two best of this lane's part of its group
    if (g < R.groups) {
      for (int i = lane % per; i < gs; i += per) {
        const double v = choice[wave][g * gs + i];
        second = fmax(second, fmin(first, v));
        first = fmax(first, v);
      }
    }
    for (int off = 1; off < per; off *= 2) {
      const double f = __shfl_xor(first, off, 64), n = __shfl_xor(second, off, 64);
      second = fmax(fmax(second, n), fmin(first, f));
      first = fmax(first, f);
    }
    const double value = R.group_score == MOE_GROUP_TOP2 && second > -inf ? first + second : first;
    int rank = 0;
    for (int i = 0; i < R.groups; ++i) {
      const double v = readlane_f64(value, i * per);
      rank += v > value || (v == value && i < g);
    }
    const uint64_t kept = __ballot(g < R.groups && rank < R.topk_groups && lane % per == 0);
    if (per == 1) {
      stay = kept;
    } else {
      stay = 0;
      for (int i = 0; i < R.groups; ++i) stay |= ((kept >> (i * per)) & 1) << i;
    }
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
      const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
      take[j] |= __ballot(bit[j] == cut2 && before < left);
      left -= min(left, (int)__popcll(same));
    }
  }

  // picks in order of id, then each to its place: falling score, ties to the lower id
  int from = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    if ((take[j] >> lane) & 1) {
      const int p = from + __builtin_amdgcn_mbcnt_hi((uint32_t)(take[j] >> 32),
                                                     __builtin_amdgcn_mbcnt_lo((uint32_t)take[j], 0));
      pick_s[wave][p] = s[j];
      pick_e[wave][p] = lane + 64 * j;
    }
    from += __popcll(take[j]);
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  const double mine = pick_s[wave][lane];
  const int e = pick_e[wave][lane];
  double total = 0.0;
  int place = 0;
  for (int i = 0; i < R.k; ++i) {
    const double v = readlane_f64(mine, i);
    total += v;
    place += v > mine || (v == mine && i < lane);
  }
  if (lane < R.k) {
    double v = mine;
    if (R.renorm) v = total > 0.0 ? v / total : 0.0;
    ids[(size_t)t * R.k + place] = e;
    w[(size_t)t * R.k + place] = (float)(v * (double)R.scale);
  }
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
