// Tokens' rows into the experts' order and back, with the gradients
// (moe_permute, moe_unpermute, moe_unpermute_grad).
//
// All three move rows and are bound by memory.
#include "chunk_dev.h"

#include <type_traits>

namespace moe {

namespace {

// ------------------------------------------------------------ into the order

struct PermuteArgs {
  const void* x;
  const int32_t* ids;
  void* xs;
  int32_t *offsets, *perm, *rows;
  int T, k, H, E;
};

// eight elements as they are: a NaN keeps its payload
template <bool BF16>
struct Chunk {
  std::conditional_t<BF16, uint4, f32x8> v;
  __device__ __forceinline__ void load(const void* x, size_t at, int n) {
    if constexpr (BF16)
      v = ld8h_to((const uint16_t*)x + at, n);
    else
      v = ld8f_to((const float*)x + at, n);
  }
  __device__ __forceinline__ void store(void* xs, size_t at, int n) const {
    if constexpr (BF16) {
      uint16_t* o = (uint16_t*)xs + at;
      if (n >= 8) {
        stream8h(o, v);
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 7; ++e)
          if (e < n) o[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
      }
    } else {
      store8<false, true>(xs, at, n, v);
    }
  }
};

// exclusive sum over the threads of a workgroup of WAVES wavefronts; and the total
template <int WAVES>
__device__ __forceinline__ int group_scan(int v, int* part, int& total) {
  const int wave = threadIdx.x >> 6, up_to = wave_scan(v);
  if ((threadIdx.x & 63) == 63) part[wave] = up_to;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    before += w < wave ? part[w] : 0;
    total += part[w];
  }
  return before + up_to - v;
}

// Few pairs, one launch: a workgroup finds its token's places by itself, pair p of expert
// e standing behind the pairs q with (ids[q], q) < (e, p), and writes the token's row there.
// Workgroup 0 counts the experts' pairs.  An id outside [0, E) is above all as unsigned.
template <bool BF16>
__global__ __launch_bounds__(256) void permute_few_kernel(PermuteArgs a) {
  const int P = a.T * a.k, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (blockIdx.x == 0) {
    if (blockIdx.y) return;
    __shared__ int hist[1024], part[4];
    for (int e = threadIdx.x; e < 1024; e += 256) hist[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < P; i += 256) {
      const uint32_t e = (uint32_t)a.ids[i];
      if (e < (uint32_t)a.E) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    int v[4], sum = 0, total;
#pragma unroll
    for (int j = 0; j < 4; ++j) sum += v[j] = hist[threadIdx.x * 4 + j];
    int at = group_scan<4>(sum, part, total);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = threadIdx.x * 4 + j;
      if (e < a.E) a.offsets[e] = at;
      at += v[j];
    }
    if (threadIdx.x == 0) a.offsets[a.E] = total;
    return;
  }
  __shared__ int32_t part[4][8], to[64];
  const int t = blockIdx.x - 1;
  int at = (blockIdx.y * 256 + threadIdx.x) * 8;
  Chunk<BF16> v;
  if (a.xs && at < a.H) v.load(a.x, (size_t)t * a.H + at, a.H - at);
  for (int r0 = 0; r0 < a.k; r0 += 8) {
    const int first = t * a.k + r0;
    uint32_t e[8];
    int n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[i] = (uint32_t)a.ids[min(first + i, P - 1)];
      n[i] = 0;
    }
    for (int q0 = wave * 64; q0 < P; q0 += 1024) {
      uint32_t id[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int q = q0 + 256 * j + lane;
        id[j] = (uint32_t)a.ids[min(q, P - 1)];
        if (q >= P) id[j] = ~0u;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int from = q0 + 256 * j;
        if (from + 64 <= first || from >= first + 8) {
          const uint32_t below = from < first;
#pragma unroll
          for (int i = 0; i < 8; ++i) n[i] += __popcll(__ballot(id[j] < e[i] + below));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) n[i] += __popcll(__ballot(id[j] < e[i] + (from + lane < first + i)));
        }
      }
    }
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) part[wave][i] = n[i];
    }
    __syncthreads();
    if (threadIdx.x < 8 && r0 + threadIdx.x < a.k) {
      const int i = threadIdx.x, p = first + i;
      const int at = part[0][i] + part[1][i] + part[2][i] + part[3][i];
      const bool live = (uint32_t)a.ids[p] < (uint32_t)a.E;
      to[r0 + i] = live ? at : -1;
      if (blockIdx.y == 0) {
        a.rows[p] = live ? at : -1;
        if (live) a.perm[at] = p;
      }
    }
    __syncthreads();
  }
  if (!a.xs) return;
  while (at < a.H) {
    for (int r = 0; r < a.k; ++r)
      if (to[r] >= 0) v.store(a.xs, (size_t)to[r] * a.H + at, a.H - at);
    at += gridDim.y * 2048;
    if (at < a.H) v.load(a.x, (size_t)t * a.H + at, a.H - at);
  }
}

// Many pairs, two launches.  The first counts each chunk's pairs of each expert; in the
// second a chunk's workgroup sums the chunks before its own, ranks its pairs in order
// and copies its tokens' rows.
__global__ __launch_bounds__(256) void permute_count_kernel(const int32_t* __restrict__ ids, int P, int E, int n,
                                                            int32_t* __restrict__ counts) {
  __shared__ int hist[1024];
  for (int e = threadIdx.x; e < E; e += 256) hist[e] = 0;
  __syncthreads();
  const int lo = blockIdx.x * n, hi = min(P, lo + n);
  for (int i = lo + threadIdx.x; i < hi; i += 256) {
    const uint32_t e = (uint32_t)ids[i];
    if (e < (uint32_t)E) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256) counts[(size_t)blockIdx.x * E + e] = hist[e];
}

constexpr int kRankWaves = 8;

template <bool BF16>
__global__ __launch_bounds__(1024) void permute_place_kernel(PermuteArgs a, int tokens, int bits,
                                                             const int32_t* __restrict__ counts) {
  extern __shared__ int lds[];
  int* next = lds;                      // [kRankWaves][E]: where a wavefront's next pair of an expert goes
  int* to = lds + kRankWaves * a.E;     // [tokens * k]
  __shared__ int before[1024], all[1024], part[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int P = a.T * a.k, n = tokens * a.k, lo = blockIdx.x * n, here = min(n, P - lo);
  before[tid] = all[tid] = 0;
  for (int i = tid; i < kRankWaves * a.E; i += 1024) next[i] = 0;
  __syncthreads();
  {
    // 2^bits >= E columns side by side
    const int e = tid & ((1 << bits) - 1), step = 1024 >> bits;
    int sum = 0, mine = 0;
    if (e < a.E) {
#pragma unroll 8
      for (int c = tid >> bits; c < (int)gridDim.x; c += step) {
        const int v = counts[(size_t)c * a.E + e];
        sum += v;
        mine += c < (int)blockIdx.x ? v : 0;
      }
      atomicAdd(&all[e], sum);
      atomicAdd(&before[e], mine);
    }
  }
  // a wavefront's pairs: whole batches of 64, in order
  const int each = (here + kRankWaves * 64 - 1) / (kRankWaves * 64) * 64;
  const int from = min(wave * each, here), end = wave < kRankWaves ? min(from + each, here) : from;
  for (int i = from + lane; i < end; i += 64) {
    const uint32_t e = (uint32_t)a.ids[lo + i];
    if (e < (uint32_t)a.E) atomicAdd(&next[wave * a.E + e], 1);
  }
  __syncthreads();
  int total;
  int run = group_scan<16>(all[tid], part, total);
  if (blockIdx.x == 0) {
    if (tid < a.E) a.offsets[tid] = run;
    if (tid == 0) a.offsets[a.E] = total;
  }
  if (tid < a.E) {
    run += before[tid];
#pragma unroll
    for (int w = 0; w < kRankWaves; ++w) {
      const int v = next[w * a.E + tid];
      next[w * a.E + tid] = run;
      run += v;
    }
  }
  __syncthreads();
  for (int i0 = from; i0 < end; i0 += 64) {
    const int i = i0 + lane;
    const uint32_t e = i < end ? (uint32_t)a.ids[lo + i] : ~0u;
    const bool live = e < (uint32_t)a.E;
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    const int below = __popcll(same & (((uint64_t)1 << lane) - 1));
    int at = -1;
    if (live) {
      volatile int* slot = next + wave * a.E + e;
      at = *slot + below;
      if ((same >> lane) == 1) *slot = at + 1;  // the last of the expert's pairs
      a.perm[at] = lo + i;
    }
    __builtin_amdgcn_wave_barrier();
    if (i < end) {
      to[i] = at;
      a.rows[lo + i] = at;
    }
  }
  if (!a.xs) return;
  __syncthreads();
  // units of 512 elements of a token
  const int segs = (a.H + 511) / 512, units = here / a.k * segs, first = blockIdx.x * tokens;
  constexpr int kAhead = 4;
  for (int u0 = wave; u0 < units; u0 += 16 * kAhead) {
    Chunk<BF16> v[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int u = u0 + 16 * j, t = u / segs, at = ((u - t * segs) * 64 + lane) * 8;
      if (u < units && at < a.H) v[j].load(a.x, (size_t)(first + t) * a.H + at, a.H - at);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int u = u0 + 16 * j, t = u / segs, at = ((u - t * segs) * 64 + lane) * 8;
      if (u < units && at < a.H)
        for (int r = 0; r < a.k; ++r) {
          const int row = to[t * a.k + r];
          if (row >= 0) v[j].store(a.xs, (size_t)row * a.H + at, a.H - at);
        }
    }
  }
}

// ------------------------------------------------------------ back

struct UnpermuteArgs {
  const void *ys, *base;
  void* out;
  const int32_t* rows;
  const float* w;
  int T, k, H, M, segs;  // segs: wavefronts a row
};

// A wavefront takes 64 chunks of eight elements of one token; the ranks' chunks are
// requested eight at a time.
template <bool YBF16, bool OBF16>
__global__ __launch_bounds__(256) void unpermute_kernel(UnpermuteArgs a) {
  const int wave = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane(wave / a.segs), seg = wave - t * a.segs;
  const int e = (seg * 64 + lane) * 8, n = a.H - e;
  if (t >= a.T || n <= 0) return;
  f32x8 acc = f32x8(0.f);
  for (int r0 = 0; r0 < a.k && a.M > 0; r0 += 8) {
    f32x8 v[8];
    float w[8];
    bool live[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = min(r0 + i, a.k - 1);
      const int row = a.rows[(size_t)t * a.k + r];
      live[i] = r0 + i < a.k && (uint32_t)row < (uint32_t)a.M;
      w[i] = a.w ? a.w[(size_t)t * a.k + r] : 1.0f;
      v[i] = load8<YBF16>(a.ys, (size_t)(live[i] ? row : 0) * a.H + e, n);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (live[i]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = fmaf(w[i], v[i][j], acc[j]);
      }
  }
  const size_t at = (size_t)t * a.H + e;
  if (a.base) acc += load8<OBF16>(a.base, at, n);
  store8<OBF16>(a.out, at, n, acc);
}

// ------------------------------------------------------------ the way back's gradient

struct GradArgs {
  const void *gout, *ys;
  void* gys;
  const int32_t* rows;
  const float* w;
  float* gw;
  int T, k, H, M, per_row;  // per_row: threads a token, 64, 128 or 256
};

// A token's threads go over its row once for every eight ranks: a chunk of gout meets
// the ranks' chunks of ys (their products are summed) and leaves as theirs of gys.
template <bool GBF16, bool YBF16>
__global__ __launch_bounds__(256) void unpermute_grad_kernel(GradArgs a) {
  __shared__ float red[4][8];
  const int in_row = threadIdx.x & (a.per_row - 1), wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int token = blockIdx.x * (256 / a.per_row) + threadIdx.x / a.per_row;
  const bool here = token < a.T;
  const int t = __builtin_amdgcn_readfirstlane(min(token, a.T - 1));
  for (int r0 = 0; r0 < a.k; r0 += 8) {
    int row[8];
    float w[8], dot[8];
    bool live[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = min(r0 + i, a.k - 1);
      row[i] = a.rows[(size_t)t * a.k + r];
      live[i] = here && r0 + i < a.k && (uint32_t)row[i] < (uint32_t)a.M;
      w[i] = a.w ? a.w[(size_t)t * a.k + r] : 1.0f;
      dot[i] = 0.f;
    }
    for (int e = in_row * 8; e < a.H; e += a.per_row * 8) {
      const int n = a.H - e;
      const f32x8 g = load8<GBF16>(a.gout, (size_t)t * a.H + e, n);
      f32x8 y[8];
      if (a.gw && a.M > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = load8<YBF16>(a.ys, (size_t)(live[i] ? row[i] : 0) * a.H + e, n);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (live[i]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) dot[i] = fmaf(g[j], y[i][j], dot[i]);
          }
      }
      if (a.gys) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (live[i]) store8<YBF16>(a.gys, (size_t)row[i] * a.H + e, n, g * w[i]);
      }
    }
    if (!a.gw) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) dot[i] = wave_sum(dot[i]);
    if (a.per_row > 64) {
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) red[wave][i] = dot[i];
      }
      __syncthreads();
    }
    if (here && in_row < 8 && r0 + in_row < a.k) {
      float s = 0.f;
      if (a.per_row > 64) {
        for (int v = 0; v < a.per_row / 64; ++v) s += red[wave + v][in_row];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) s = in_row == i ? dot[i] : s;
      }
      a.gw[(size_t)t * a.k + r0 + in_row] = s;
    }
    if (a.per_row > 64) __syncthreads();
  }
}

}  // namespace

// Every workgroup of the few-pair form reads all ids.
constexpr int kFewPairs = 4096;
constexpr int kChunks = 256;

static int chunk_tokens(int T) { return (T + kChunks - 1) / kChunks; }

size_t permute_scratch_bytes(int T, int k, int E) {
  if (T * k <= kFewPairs) return 0;
  const int tokens = chunk_tokens(T);
  return (size_t)((T + tokens - 1) / tokens) * E * sizeof(int32_t);
}

moe_status launch_permute(const void* x, moe_dtype xt, int T, int k, int H, int E, const int32_t* ids, void* xs,
                          int32_t* offsets, int32_t* perm, int32_t* rows, int32_t* scratch, hipStream_t s) {
  const PermuteArgs a{x, ids, xs, offsets, perm, rows, T, k, H, E};
  const bool bf16 = xt == MOE_BF16;
  if (T * k <= kFewPairs) {
    const int segs = xs ? min((H + 2047) / 2048, max(1, 1024 / max(T, 1))) : 1;
    launch(MOE_PROF_PERMUTE, bf16 ? permute_few_kernel<true> : permute_few_kernel<false>, dim3(T + 1, segs), dim3(256), 0,
           s, a);
  } else {
    const int tokens = chunk_tokens(T), chunks = (T + tokens - 1) / tokens;
    int bits = 0;
    while ((1 << bits) < E) ++bits;
    launch(MOE_PROF_PERMUTE, permute_count_kernel, dim3(chunks), dim3(256), 0, s, ids, T * k, E, tokens * k, scratch);
    MOE_LAUNCH_CHECK();
    const size_t lds = (size_t)(kRankWaves * E + tokens * k) * sizeof(int);
    launch(MOE_PROF_PERMUTE, bf16 ? permute_place_kernel<true> : permute_place_kernel<false>, dim3(chunks), dim3(1024), lds,
           s, a, tokens, bits, (const int32_t*)scratch);
  }
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

moe_status launch_unpermute(const void* ys, moe_dtype yt, int M, const int32_t* rows, const float* w, const void* base,
                            int T, int k, int H, void* out, moe_dtype ot, hipStream_t s) {
  UnpermuteArgs a{ys, base, out, rows, w, T, k, H, M, (H + 511) / 512};
  const bool yb = yt == MOE_BF16, ob = ot == MOE_BF16;
  auto f = yb ? (ob ? unpermute_kernel<true, true> : unpermute_kernel<true, false>)
              : (ob ? unpermute_kernel<false, true> : unpermute_kernel<false, false>);
  launch(MOE_PROF_PERMUTE, f, dim3((unsigned)(((size_t)T * a.segs + 3) / 4)), dim3(256), 0, s, a);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

moe_status launch_unpermute_grad(const void* gout, moe_dtype gt, const void* ys, moe_dtype yt, int M,
                                 const int32_t* rows, const float* w, int T, int k, int H, void* gys, float* gw,
                                 hipStream_t s) {
  GradArgs a{gout, ys, gys, rows, w, gw, T, k, H, M, H <= 512 ? 64 : H <= 1024 ? 128 : 256};
  const bool gb = gt == MOE_BF16, yb = yt == MOE_BF16;
  auto f = gb ? (yb ? unpermute_grad_kernel<true, true> : unpermute_grad_kernel<true, false>)
              : (yb ? unpermute_grad_kernel<false, true> : unpermute_grad_kernel<false, false>);
  const int tokens = 256 / a.per_row;
  launch(MOE_PROF_PERMUTE, f, dim3((T + tokens - 1) / tokens), dim3(256), 0, s, a);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
