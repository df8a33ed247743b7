// Low-rank adapters of many requests beside a shared projection
// (moe_lora_add): out[t] = base[t] + scale * B (A x[t]) with the adapter of
// the token's request.
//
// Two forms, chosen by the number of tokens:
//   - token_kernel: one token a workgroup on the vector units, so a decode
//     batch whose tokens all have adapters of their own reads each adapter
//     once;
//   - tile_kernel: 16 tokens a workgroup on the matrix units, one pass per
//     distinct adapter of the 16.
// Both compute A x whole in every workgroup that needs it (from the caches
// after the first) and split the outputs over workgroups, so the call is one
// launch and needs no workspace.
#include "chunk_dev.h"

namespace moe {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kMaxRank = 128;

__device__ __forceinline__ int rank_of(const moe_lora& L, int id) {
  return L.ranks ? max(0, min(L.ranks[id], L.r)) : L.r;
}

// ------------------------------------------------------------ a token a workgroup

constexpr int kTokThreads = 512, kTokWaves = kTokThreads / 64;

template <bool XBF16, bool YBF16>
__global__ __launch_bounds__(kTokThreads) void token_kernel(moe_lora L, const void* __restrict__ x,
                                                            const int32_t* __restrict__ ids, const void* base,
                                                            void* out, int per) {
  __shared__ __align__(16) float v[kMaxRank];
  const int t = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int id = ids[t];
  const bool has = id >= 0 && id < L.num;
  const int rank = has ? rank_of(L, id) : 0;
  const uint16_t* A = (const uint16_t*)L.a + (has ? (size_t)id * L.r * L.K : 0);
  const uint16_t* B = (const uint16_t*)L.b + (has ? (size_t)id * L.N * L.r : 0);
  const float scale = has && L.scale ? L.scale[id] : 1.0f;
  const int K = L.K, n0 = blockIdx.y * per, n1 = min(L.N, n0 + per);
  if (threadIdx.x < kMaxRank) v[threadIdx.x] = 0.0f;
  __syncthreads();
  constexpr int R = 2;  // rows of A a wavefront multiplies at once
  const int kfull = K & ~511;
  for (int j = wave * R; j < rank; j += kTokWaves * R) {
    float acc[R] = {};
    const uint16_t* row[R];
#pragma unroll
    for (int i = 0; i < R; ++i) row[i] = A + (size_t)min(j + i, rank - 1) * K;
    const size_t at = (size_t)t * K;
#pragma unroll 4
    for (int k = lane * 8; k < kfull; k += 512) {
      const f32x8 xv = load8<XBF16>(x, at + k, 8);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const f32x8 av = widen(ld8h(row[i] + k));
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i] = fmaf(xv[e], av[e], acc[i]);
      }
    }
    const int k = kfull + lane * 8;
    if (k < K) {
      const f32x8 xv = load8<XBF16>(x, at + k, K - k);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const f32x8 av = widen(ld8h_to(row[i] + k, K - k));
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i] = fmaf(xv[e], av[e], acc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float s = wave_sum(acc[i]);
      if (lane == 0 && j + i < rank) v[j + i] = s * scale;
    }
  }
  __syncthreads();
  for (int n = n0 + threadIdx.x; n < n1; n += kTokThreads) {
    const size_t at = (size_t)t * L.N + n;
    float acc = 0.f;
    for (int j = 0; j < rank; j += 8) {
      const f32x8 bv = widen(ld8h_to(B + (size_t)n * L.r + j, rank - j));
#pragma unroll
      for (int e = 0; e < 8; ++e) acc = fmaf(v[j + e], bv[e], acc);
    }
    if (base) acc += YBF16 ? bf(((const uint16_t*)base)[at]) : ((const float*)base)[at];
    if (YBF16)
      ((uint16_t*)out)[at] = f32_to_bf16(acc);
    else
      ((float*)out)[at] = acc;
  }
}

// ----------------------------------------------------------- 16 tokens a workgroup
//
// v_mfma_f32_16x16x32_bf16: lane l supplies row (first operand) or column
// (second) l % 16 at K positions 8 (l / 16) .. + 7, and receives column l % 16,
// rows 4 (l / 16) .. + 3.  v_mfma_f32_16x16x4_f32: one K position, l / 16.
// A contraction may take its positions in any order as long as both operands
// take the same, so a lane reads 16 consecutive elements of its row at a time.
//
// A x: first operand the rows of A (16 of them a "task": one adapter, 16 of its
// ranks), second the tokens; the wavefronts split K and their parts meet in
// LDS.  The sum of a token's own adapter is split into bf16 parts whose sum is
// the fp32 value (two parts, off by at most 2^-16 of it, for bf16 outputs;
// three, exact, for fp32), so the second product runs on bf16 operands too.
//
// B v: first operand 16 outputs, second the tokens.  Output row m of product q
// stands for output 16 (m / 4) + 4 q + m % 4 of a block of 64, so that four
// products leave 16 consecutive outputs of a token in each lane.  The parts
// and ranks of v are one list of chunks of eight, four to a product.  Every
// adapter of the tile has its own sum and a token takes its own adapter's, so
// one adapter's NaN cannot reach another's tokens.

constexpr int kTileThreads = 512, kTileWaves = kTileThreads / 64;
constexpr int kPass = 4;                 // tasks per pass over x
constexpr int kUnroll = 2;               // blocks of K in flight
constexpr int kVStride = kMaxRank + 8;   // bf16 elements of a token's row of v parts

// fp32 -> bf16 by truncation: what is left over is exact
__device__ __forceinline__ uint16_t take_bf16(float& f) {
  const uint32_t u = __float_as_uint(f) & 0xffff0000u;
  const float rest = f - __uint_as_float(u);
  f = rest == rest ? rest : 0.0f;  // an infinity leaves nothing over
  return (uint16_t)(u >> 16);
}

// A lane's 16 consecutive outputs of its token, n of them (<= 0: none) inside N.
template <bool YBF16>
struct Out {
  uint4 h[2];
  f32x8 f[2];

  __device__ __forceinline__ void load(const void* base, size_t at, int n) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (YBF16)
        h[i] = base ? ld8h_to((const uint16_t*)base + at + 8 * i, n - 8 * i) : make_uint4(0, 0, 0, 0);
      else
        f[i] = base ? ld8f_to((const float*)base + at + 8 * i, n - 8 * i) : f32x8(0.f);
    }
  }

  __device__ __forceinline__ void store(void* out, size_t at, int n, const v4f (&d)[4]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f32x8 w;
      if constexpr (YBF16)
        w = widen(h[i]);
      else
        w = f[i];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] += d[2 * i + (e >> 2)][e & 3];
      store8<YBF16>(out, at + 8 * i, n - 8 * i, w);
    }
  }
};

// B v of one adapter for the 64 outputs at nb.  FULL: all of them inside N, the
// rank a multiple of eight.
template <int NS, bool FULL>
__device__ __forceinline__ void expand(const uint16_t* __restrict__ B, const uint16_t (&vs)[NS][16][kVStride], int nb,
                                       int N, int r, int rank, v4f (&d)[4]) {
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int c8 = (rank + 7) / 8, chunks = NS * c8;
  for (int m = 0; m < chunks; m += 4) {
    const int c = m + g, cc = min(c, chunks - 1), pt = (cc >= c8) + (cc >= 2 * c8), j = (cc - pt * c8) * 8;
    uint4 vv = *(const uint4*)&vs[pt][col][j], bv[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = nb + (col >> 2) * 16 + q * 4 + (col & 3);
      bv[q] = FULL ? ld8h(B + (size_t)n * r + j) : ld8h_to(B + (size_t)min(n, N - 1) * r + j, rank - j);
      if (c >= chunks) bv[q] = make_uint4(0, 0, 0, 0);
    }
    if (c >= chunks) vv = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      d[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, bv[q]), __builtin_bit_cast(v8bf, vv),
                                                     d[q], 0, 0, 0);
  }
}

// One block of 64 K positions of NP tasks: this lane's 16 elements at k.  FULL:
// the block lies inside K.
template <bool XBF16, int NP, bool FULL>
__device__ __forceinline__ void shrink_block(const void* __restrict__ xrow, const uint16_t* const (&arow)[kPass], int k,
                                             int K, v4f (&acc)[kPass]) {
  if (XBF16) {
    const uint16_t* xp = (const uint16_t*)xrow + k;
    uint4 xv[2], av[NP][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) xv[h] = FULL ? ld8h(xp + 8 * h) : ld8h_to(xp + 8 * h, K - k - 8 * h);
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        av[p][h] = FULL ? ld8h(arow[p] + k + 8 * h) : ld8h_to(arow[p] + k + 8 * h, K - k - 8 * h);
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        acc[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, av[p][h]),
                                                         __builtin_bit_cast(v8bf, xv[h]), acc[p], 0, 0, 0);
  } else {
    const float* xp = (const float*)xrow + k;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x8 xv = FULL ? ld8f(xp + 8 * h) : ld8f_to(xp + 8 * h, K - k - 8 * h);
      f32x8 av[NP];
#pragma unroll
      for (int p = 0; p < NP; ++p)
        av[p] = widen(FULL ? ld8h(arow[p] + k + 8 * h) : ld8h_to(arow[p] + k + 8 * h, K - k - 8 * h));
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[p] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[p][e], xv[e], acc[p], 0, 0, 0);
    }
  }
}

template <bool XBF16, int NP>
__device__ __forceinline__ void shrink(const void* __restrict__ xrow, const uint16_t* const (&arow)[kPass], int wave,
                                       int g, int K, v4f (&acc)[kPass]) {
  const int full = K / 64;  // whole blocks; block b goes to wavefront b % kTileWaves
  int b = wave;
  for (; b + (kUnroll - 1) * kTileWaves < full; b += kUnroll * kTileWaves) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      shrink_block<XBF16, NP, true>(xrow, arow, (b + u * kTileWaves) * 64 + g * 16, K, acc);
  }
  for (; b < full; b += kTileWaves) shrink_block<XBF16, NP, true>(xrow, arow, b * 64 + g * 16, K, acc);
  if (b == full && b * 64 < K) shrink_block<XBF16, NP, false>(xrow, arow, b * 64 + g * 16, K, acc);
}

template <bool XBF16, bool YBF16>
__global__ __launch_bounds__(kTileThreads) void tile_kernel(moe_lora L, const void* __restrict__ x, int T,
                                                            const int32_t* __restrict__ ids, const void* base,
                                                            void* out, int per) {
  constexpr int NS = YBF16 ? 2 : 3;
  __shared__ __align__(16) float part[kTileWaves][kPass][16][16];  // [wave][task][token][rank]
  __shared__ __align__(16) uint16_t vs[NS][16][kVStride];
  __shared__ int tok_slot[16], ad_id[16], ad_rank[16], n_ad, n_task;
  __shared__ uint8_t task_slot[128], task_tile[128];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.x * 16, K = L.K, N = L.N, r = L.r;

  if (wave == 0) {
    const int id = lane < 16 && t0 + lane < T ? ids[t0 + lane] : -1;
    const bool has = lane < 16 && id >= 0 && id < L.num;
    int lead = lane;
    for (int i = 15; i >= 0; --i)
      if (__shfl(id, i, 64) == id) lead = i;
    const uint64_t leads = __ballot(has && lead == lane);
    const uint64_t before = (1ull << lane) - 1;
    const int rank = has ? rank_of(L, id) : 0;
    int at = 0;  // tasks of the adapters before this one
    const int tiles = (rank + 15) / 16;
    for (int i = 0; i < 16; ++i) {
      const int ti = __shfl(tiles, i, 64);
      if (((leads >> i) & 1) && i < lane) at += ti;
    }
    if (lane < 16) tok_slot[lane] = has ? __popcll(leads & ((1ull << lead) - 1)) : -1;
    if ((leads >> lane) & 1) {
      const int slot = __popcll(leads & before);
      ad_id[slot] = id;
      ad_rank[slot] = rank;
      for (int i = 0; i < tiles; ++i) task_slot[at + i] = (uint8_t)slot, task_tile[at + i] = (uint8_t)i;
    }
    int total = 0;
    for (int i = 0; i < 16; ++i) {
      const int ti = __shfl(tiles, i, 64);
      if ((leads >> i) & 1) total += ti;
    }
    if (lane == 0) n_ad = __popcll(leads), n_task = total;
  }
  __syncthreads();
  const int ntask = n_task, nad = n_ad;

  // A x, kPass tasks at a time
  const char* xrow = (const char*)x + (size_t)min(t0 + col, T - 1) * K * (XBF16 ? 2 : 4);
  for (int p0 = 0; p0 < ntask; p0 += kPass) {
    v4f acc[kPass] = {};
    const uint16_t* arow[kPass];
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int q = min(p0 + p, ntask - 1), slot = task_slot[q];
      arow[p] = (const uint16_t*)L.a + ((size_t)ad_id[slot] * r + min(task_tile[q] * 16 + col, ad_rank[slot] - 1)) * K;
    }
    const int np = min(kPass, ntask - p0);
    if (np == 1)
      shrink<XBF16, 1>(xrow, arow, wave, g, K, acc);
    else if (np == 2)
      shrink<XBF16, 2>(xrow, arow, wave, g, K, acc);
    else
      shrink<XBF16, kPass>(xrow, arow, wave, g, K, acc);
#pragma unroll
    for (int p = 0; p < kPass; ++p) *(v4f*)&part[wave][p][col][g * 4] = acc[p];
    __syncthreads();
    for (int i = threadIdx.x; i < np * 256; i += kTileThreads) {
      const int p = i >> 8, tok = (i >> 4) & 15, rk = i & 15, q = p0 + p, slot = task_slot[q];
      if (tok_slot[tok] == slot) {
        float s = 0.f;
#pragma unroll
        for (int wv = 0; wv < kTileWaves; ++wv) s += part[wv][p][tok][rk];
        const int j = task_tile[q] * 16 + rk;
        if (L.scale) s *= L.scale[ad_id[slot]];
        if (j >= ad_rank[slot]) s = 0.f;
#pragma unroll
        for (int n = 0; n < NS; ++n) vs[n][tok][j] = take_bf16(s);
      }
    }
    __syncthreads();
  }

  // B v and the base, a block of 64 outputs a wavefront at a time
  const int n0 = blockIdx.y * per, n1 = min(N, n0 + per), myslot = tok_slot[col], t = t0 + col;
  bool whole = r % 8 == 0;  // no adapter of the tile ends inside a chunk of eight ranks
  for (int s = 0; s < nad; ++s) whole = whole && ad_rank[s] % 8 == 0;
  for (int nb = n0 + wave * 64; nb < n1; nb += kTileWaves * 64) {
    const bool inside = nb + 64 <= N;
    const size_t at = (size_t)min(t, T - 1) * N + nb + g * 16;
    Out<YBF16> y;
    y.load(base, at, inside ? 16 : N - nb - g * 16);
    v4f acc[4] = {};
    for (int s = 0; s < nad; ++s) {
      v4f d[4] = {};
      const uint16_t* B = (const uint16_t*)L.b + (size_t)ad_id[s] * N * r;
      if (inside && whole)
        expand<NS, true>(B, vs, nb, N, r, ad_rank[s], d);
      else
        expand<NS, false>(B, vs, nb, N, r, ad_rank[s], d);
      if (s == myslot) {
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = d[q];
      }
    }
    if (t < T) y.store(out, at, inside ? 16 : N - nb - g * 16, acc);
  }
}

template <bool XBF16, bool YBF16>
void run(const moe_lora* L, const void* x, int T, const int32_t* ids, const void* base, void* out, hipStream_t s) {
  constexpr int kTokens = 128, kGroups = 256;
  if (T <= kTokens) {
    const int split = max(1, min(kGroups / T, (L->N + 127) / 128));
    const int per = ((L->N + split - 1) / split + 63) / 64 * 64;
    launch(MOE_PROF_LORA, token_kernel<XBF16, YBF16>, dim3(T, (L->N + per - 1) / per), dim3(kTokThreads), 0, s, *L, x,
           ids, base, out, per);
  } else {
    const int tiles = (T + 15) / 16;
    const int split = max(1, min((kGroups + tiles - 1) / tiles, (L->N + 64 * kTileWaves - 1) / (64 * kTileWaves)));
    const int per = ((L->N + split - 1) / split + 63) / 64 * 64;
    launch(MOE_PROF_LORA, tile_kernel<XBF16, YBF16>, dim3(tiles, (L->N + per - 1) / per), dim3(kTileThreads), 0, s, *L,
           x, T, ids, base, out, per);
  }
}

}  // namespace

moe_status launch_lora(const moe_lora* L, const void* x, moe_dtype xt, int T, const int32_t* ids, const void* base,
                       void* out, moe_dtype yt, hipStream_t s) {
  if (xt == MOE_BF16 && yt == MOE_BF16)
    run<true, true>(L, x, T, ids, base, out, s);
  else if (xt == MOE_BF16)
    run<true, false>(L, x, T, ids, base, out, s);
  else if (yt == MOE_BF16)
    run<false, true>(L, x, T, ids, base, out, s);
  else
    run<false, false>(L, x, T, ids, base, out, s);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
