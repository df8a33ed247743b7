// Tokens' rows into the experts' order and back, with the gradients
// (moe_permute, moe_unpermute, moe_unpermute_grad).
//
// All three move rows and are bound by memory.
#include "chunk_dev.h"

#include <type_traits>

namespace moe {

namespace {

// A row's last chunk of eight elements that is not whole lies eight from the row's end, and
// the first `skip` of them are the chunk's before it: partial loads, each a branch and short
// loads that are waited for, took 5 of 12 us of a combine of 777 rows of 2047.  Rows of
// fewer than eight elements have them all the same.
struct Place {
  int at, skip, n;
  __device__ __forceinline__ Place(int e, int H, int size = 8)
      : at(max(min(e, H - size), 0)), skip(e - at), n(min(H, size)) {}
};

// what a chunk has beyond the chunk before it
template <bool BF16>
__device__ __forceinline__ void store_rest(void* p, size_t row, Place c, f32x8 v) {
  if (c.skip == 0) {
    store8<BF16, true>(p, row + c.at, c.n, v);
  } else {
#pragma unroll
    for (int j = 1; j < 8; ++j)
      if (j >= c.skip) store8<BF16>(p, row + c.at + j, 1, f32x8(v[j]));
  }
}

// ------------------------------------------------------------ into the order

struct PermuteArgs {
  const void* x;
  const int32_t* ids;
  void* xs;
  int32_t *offsets, *perm, *rows;
  int T, k, H, E;
};

typedef uint32_t u32x4_word __attribute__((ext_vector_type(4), aligned(4)));

// 16 bytes of a row as they are: a NaN keeps its payload
template <bool BF16>
struct Chunk {
  static constexpr int kSize = BF16 ? 8 : 4;
  uint4 v;
  __device__ __forceinline__ void load(const void* x, size_t row, int e, int H) {
    const Place c(e, H, kSize);
    if constexpr (BF16) {
      v = ld8h_to((const uint16_t*)x + row + c.at, c.n);
    } else {
      const uint32_t* p = (const uint32_t*)x + row + c.at;
      if (c.n == 4)
        v = ld4w(p);
      else
        v = make_uint4(p[0], c.n > 1 ? p[1] : 0, c.n > 2 ? p[2] : 0, 0);
    }
  }
  __device__ __forceinline__ void store(void* xs, size_t row, int e, int H) const {
    const Place c(e, H, kSize);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (BF16) {
      uint16_t* o = (uint16_t*)xs + row + c.at;
      if (c.n == 8) {
        stream8h(o, v);
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (j < c.n) o[j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
      }
    } else {
      uint32_t* o = (uint32_t*)xs + row + c.at;
      if (c.n == 4) {
        __builtin_nontemporal_store(u32x4_word{v.x, v.y, v.z, v.w}, (u32x4_word*)o);
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (j < c.n) o[j] = w[j];
      }
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

// Few pairs, one launch: a workgroup finds its token's places by itself, pair p of expert e
// standing behind the pairs q with (ids[q], q) < (e, p), and writes the token's row there.
// Workgroup 0 counts the experts' pairs.  An id outside [0, E) is above all as unsigned.
// 64 tokens x 8 of 4096 bf16: 4.2 us, of which the launch is 1.9.
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
  int e0 = (blockIdx.y * 256 + threadIdx.x) * Chunk<BF16>::kSize;
  Chunk<BF16> v;
  if (a.xs && e0 < a.H) v.load(a.x, (size_t)t * a.H, e0, a.H);
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
  while (e0 < a.H) {
    for (int r = 0; r < a.k; ++r)
      if (to[r] >= 0) v.store(a.xs, (size_t)to[r] * a.H, e0, a.H);
    e0 += gridDim.y * 256 * Chunk<BF16>::kSize;
    if (e0 < a.H) v.load(a.x, (size_t)t * a.H, e0, a.H);
  }
}

// Many pairs, two launches.  The first counts each chunk's pairs of each expert; in the
// second a chunk's workgroup sums the chunks before its own, ranks its pairs in order
// and copies its tokens' rows, each read once and written k times.  4096 tokens x 8 of 4096
// bf16: 63 us, 4.8 TB/s (a large copy: 5.1).  Streaming stores 63 us, cached ones 72; rows of
// 4095 81 us, and 89 where a wavefront's chunks are 16 wavefronts' apart.
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
  // A wavefront takes kAhead chunks a lane, one behind the other, of a token: what a row that
  // starts inside a cache line leaves of a line is written next.
  constexpr int kAhead = 4, kUnit = 64 * Chunk<BF16>::kSize;
  const int segs = (a.H + kAhead * kUnit - 1) / (kAhead * kUnit), units = here / a.k * segs;
  for (int u = wave; u < units; u += 16) {
    const int t = u / segs, e0 = (u - t * segs) * kAhead * kUnit + lane * Chunk<BF16>::kSize;
    const size_t from = (size_t)(blockIdx.x * tokens + t) * a.H;
    Chunk<BF16> v[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (e0 + j * kUnit < a.H) v[j].load(a.x, from, e0 + j * kUnit, a.H);
    for (int r = 0; r < a.k; ++r) {
      const int row = to[t * a.k + r];
      if (row < 0) continue;
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (e0 + j * kUnit < a.H) v[j].store(a.xs, (size_t)row * a.H, e0 + j * kUnit, a.H);
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
// requested eight at a time.  Bound by memory: 4096 tokens x 8 of 4096 bf16 57 us, 5.3 TB/s;
// 777 x 6 of 2047 onto an fp32 base 7.1 us, 4.2 TB/s.
template <bool YBF16, bool OBF16>
__global__ __launch_bounds__(256) void unpermute_kernel(UnpermuteArgs a) {
  const int wave = (blockIdx.y * gridDim.x + blockIdx.x) * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane(wave / a.segs), seg = wave - t * a.segs;
  const int e = (seg * 64 + lane) * 8;
  if (t >= a.T || e >= a.H) return;
  const Place c(e, a.H);
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
      v[i] = load8<YBF16>(a.ys, (size_t)(live[i] ? row : 0) * a.H + c.at, c.n);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (live[i]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = fmaf(w[i], v[i][j], acc[j]);
      }
  }
  const size_t at = (size_t)t * a.H;
  if (a.base) acc += load8<OBF16>(a.base, at + c.at, c.n);
  store_rest<OBF16>(a.out, at, c, acc);
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
// the ranks' chunks of ys (their products are summed) and leaves as theirs of gys.  Bound
// by memory: 4096 tokens x 8 of 4096 bf16 116 us, 4.9 TB/s; 509 x 6 of 2047 fp32 12.7 us,
// 3.9 TB/s.
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
      const Place c(e, a.H);
      const f32x8 g = load8<GBF16>(a.gout, (size_t)t * a.H + c.at, c.n);
      f32x8 y[8];
      if (a.gw && a.M > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = load8<YBF16>(a.ys, (size_t)(live[i] ? row[i] : 0) * a.H + c.at, c.n);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (live[i]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) dot[i] += j >= c.skip ? g[j] * y[i][j] : 0.0f;
          }
      }
      if (a.gys) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (live[i]) store_rest<YBF16>(a.gys, (size_t)row[i] * a.H, c, g * w[i]);
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

// Every workgroup of the few-pair form reads all ids.  Both forms, k = 8, rows of 512 and of
// 4096 bf16, us: 4096 pairs 6.9 against 10.0 and 10.9 against 14.6, 8192 pairs 14.0 against
// 11.6 and 21.8 against 22.5, 16384 pairs 38.9 against 12.6 and 45.6 against 37.0.
constexpr int kFewPairs = 6144;
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
    const int wide = bf16 ? 2048 : 1024, segs = xs ? min((H + wide - 1) / wide, max(1, 1024 / max(T, 1))) : 1;
    auto f = bf16 ? permute_few_kernel<true> : permute_few_kernel<false>;
    launch(MOE_PROF_PERMUTE, f, dim3(T + 1, segs), dim3(256), 0, s, a);
  } else {
    const int tokens = chunk_tokens(T), chunks = (T + tokens - 1) / tokens;
    int bits = 0;
    while ((1 << bits) < E) ++bits;
    launch(MOE_PROF_PERMUTE, permute_count_kernel, dim3(chunks), dim3(256), 0, s, ids, T * k, E, tokens * k, scratch);
    MOE_LAUNCH_CHECK();
    const size_t lds = (size_t)(kRankWaves * E + tokens * k) * sizeof(int);
    auto f = bf16 ? permute_place_kernel<true> : permute_place_kernel<false>;
    launch(MOE_PROF_PERMUTE, f, dim3(chunks), dim3(1024), lds, s, a, tokens, bits, (const int32_t*)scratch);
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
  // a dimension of a launch has fewer than 2^32 threads, and the largest sizes need 2^33
  constexpr int kAcross = 1 << 22;
  const int groups = (int)(((size_t)T * a.segs + 3) / 4);
  launch(MOE_PROF_PERMUTE, f, dim3(min(groups, kAcross), (groups + kAcross - 1) / kAcross), dim3(256), 0, s, a);
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
