// Tokens' rows into the experts' order and back, with the gradients
// (moe_permute, moe_unpermute, moe_unpermute_grad).
//
// All three move rows and are bound by memory.
#include "chunk_dev.h"

namespace moe {

size_t group_wide_scratch_ints(int n, int nkeys);
moe_status launch_group_wide(const int32_t* keys, int n, int nkeys, int32_t* counts, int32_t* offsets,
                             int32_t* perm, int32_t* scratch, hipStream_t s);

namespace {

// ------------------------------------------------------------ into the order

// rows: the inverse of perm, -1 for pairs without an expert
__global__ __launch_bounds__(256) void invert_kernel(const int32_t* __restrict__ ids, int P, int E,
                                                     const int32_t* __restrict__ offsets,
                                                     const int32_t* __restrict__ perm, int32_t* __restrict__ rows) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= P) return;
  if ((uint32_t)ids[i] >= (uint32_t)E) rows[i] = -1;
  if (i < offsets[E]) rows[perm[i]] = i;
}

// eight elements as they are: a NaN keeps its payload
template <bool BF16>
__device__ __forceinline__ void copy8(const void* x, size_t from, void* xs, size_t to, int n) {
  if constexpr (BF16) {
    const uint16_t* i = (const uint16_t*)x + from;
    uint16_t* o = (uint16_t*)xs + to;
    if (n >= 8) {
      st8h(o, ld8h(i));
    } else {
      for (int e = 0; e < n; ++e) o[e] = i[e];
    }
  } else {
    store8<false>(xs, to, n, ld8f_to((const float*)x + from, n));
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void copy_rows_kernel(const void* __restrict__ x, int k, int H, int E,
                                                        const int32_t* __restrict__ offsets,
                                                        const int32_t* __restrict__ perm, void* __restrict__ xs) {
  const int i = blockIdx.x;
  if (i >= offsets[E]) return;
  const size_t from = (size_t)(perm[i] / k) * H, to = (size_t)i * H;
  for (int e = threadIdx.x * 8; e < H; e += 256 * 8) copy8<BF16>(x, from + e, xs, to + e, H - e);
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

size_t permute_scratch_bytes(int T, int k, int E) {
  return (E + group_wide_scratch_ints(T * k, E)) * sizeof(int32_t);
}

moe_status launch_permute(const void* x, moe_dtype xt, int T, int k, int H, int E, const int32_t* ids, void* xs,
                          int32_t* offsets, int32_t* perm, int32_t* rows, int32_t* scratch, hipStream_t s) {
  const int P = T * k;
  const moe_status st = launch_group_wide(ids, P, E, scratch, offsets, perm, scratch + E, s);
  if (st != MOE_OK || P == 0) return st;
  launch(MOE_PROF_PERMUTE, invert_kernel, dim3((P + 255) / 256), dim3(256), 0, s, ids, P, E, (const int32_t*)offsets,
         (const int32_t*)perm, rows);
  if (xs) {
    auto f = xt == MOE_BF16 ? copy_rows_kernel<true> : copy_rows_kernel<false>;
    launch(MOE_PROF_PERMUTE, f, dim3(P), dim3(256), 0, s, x, k, H, E, (const int32_t*)offsets, (const int32_t*)perm, xs);
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
