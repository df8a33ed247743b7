// Low-rank adapters of many requests beside a shared projection
// (moe_lora_add): out[t] = base[t] + scale * B (A x[t]) with the adapter of
// the token's request.
//
// Two forms, chosen by the host from the sizes (token_form):
//   - token_kernel: one token a workgroup on the vector units, so a decode
//     batch whose tokens all have adapters of their own reads each adapter
//     once;
//   - tile_kernel: 16 tokens a workgroup on the matrix units, a product for
//     every distinct adapter of the 16.
// Both compute A x whole in every workgroup that needs it (from the caches
// after the first) and split the outputs over workgroups, so the call is one
// launch and needs no workspace.
#include <type_traits>

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
//
// A x: a wavefront takes R rows of A at a time, a lane eight K positions of each
// at a stride of 512, S such steps in flight.  B v: LANES lanes share a row of B,
// each with its eight ranks of v in registers, so that a wavefront's loads are
// contiguous.  The first rows of B and the base do not depend on A x and are
// requested before it: what is left is a chain of the id, the adapter's rank where
// the bank has ranks, A and the reductions.  That chain bounds small calls (K = N =
// 4096, rank 16, one token: 4.3 us, of which 1.9 are a launch; A comes in two bursts
// of 2048 positions, the second requested after the first).  At rank 64, 64 tokens
// of 64 adapters take 17.1 us for 67 MB, 3.9 TB/s: a token's four workgroups draw all
// of its A each, 0.66 MB a workgroup with x and B, and wait for a group of rows whole
// before they request the next.  With ranks 8 to 64 mixed, half the bytes, the tokens
// of rank 64 set the pace: 17.0 us.

constexpr int kTokThreads = 512, kTokWaves = kTokThreads / 64;
constexpr int kTokOut = 1024;  // outputs gathered in LDS before they are written

// the elements [from, to) of a chunk of eight bf16 values, the others zero
__device__ __forceinline__ uint4 keep8h(uint4 h, int from, int to) {
  auto word = [&](uint32_t u, int i) {
    return (i >= from && i < to ? u & 0xffffu : 0u) | (i + 1 >= from && i + 1 < to ? u & 0xffff0000u : 0u);
  };
  return make_uint4(word(h.x, 0), word(h.y, 2), word(h.z, 4), word(h.w, 6));
}

// eight products of a chunk of x with a chunk of a row of A, onto acc
template <bool XBF16>
struct XChunk;

template <>
struct XChunk<true> {
  uint4 h;
  __device__ __forceinline__ void load(const void* x, size_t at, int n) { h = ld8h_to((const uint16_t*)x + at, n); }
  __device__ __forceinline__ void drop(int n) { h = keep8h(h, n, 8); }
  __device__ __forceinline__ float dot(uint4 a, float acc) const {
    return dot2_bf16(h.w, a.w, dot2_bf16(h.z, a.z, dot2_bf16(h.y, a.y, dot2_bf16(h.x, a.x, acc))));
  }
};

template <>
struct XChunk<false> {
  f32x8 f;
  __device__ __forceinline__ void load(const void* x, size_t at, int n) { f = ld8f_to((const float*)x + at, n); }
  __device__ __forceinline__ void drop(int n) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e >= n ? f[e] : 0.f;
  }
  __device__ __forceinline__ float dot(uint4 a, float acc) const {
    const f32x8 w = widen(a);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc = fmaf(f[e], w[e], acc);
    return acc;
  }
};

// R rows of A from row j on with x's row at `at`: their sums, in every lane
template <bool XBF16, int R, int S>
__device__ __forceinline__ void token_rows(const void* __restrict__ x, size_t at, const uint16_t* __restrict__ A, int j,
                                           int rank, int K, float (&acc)[R]) {
  const int lane = threadIdx.x & 63;
  const uint16_t* row[R];
#pragma unroll
  for (int i = 0; i < R; ++i) acc[i] = 0.f, row[i] = A + (size_t)min(j + i, rank - 1) * K;
  int k = lane * 8;
  if (K >= 8) {
    for (int k0 = 0; k0 < K; k0 += 512 * S) {
      XChunk<XBF16> xv[S];
      uint4 av[S][R];
#pragma unroll
      for (int u = 0; u < S; ++u) {
        const int step = k0 + 512 * u;
        if (step >= K) break;
        const int from = min(step + k, K - 8);  // a chunk over the end is read from K - 8 on
        xv[u].load(x, at + from, 8);
#pragma unroll
        for (int i = 0; i < R; ++i) av[u][i] = ld8h(row[i] + from);
      }
#pragma unroll
      for (int u = 0; u < S; ++u) {
        const int step = k0 + 512 * u;
        if (step >= K) break;
        if (step + 512 > K) xv[u].drop(max(0, step + k - (K - 8)));  // what it has in common with others
#pragma unroll
        for (int i = 0; i < R; ++i) acc[i] = xv[u].dot(av[u][i], acc[i]);
      }
    }
  } else if (k < K) {
    XChunk<XBF16> xv;
    xv.load(x, at + k, K - k);
#pragma unroll
    for (int i = 0; i < R; ++i) acc[i] = xv.dot(ld8h_to(row[i] + k, K - k), acc[i]);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) acc[i] = wave_sum(acc[i]);
}

template <bool XBF16, bool YBF16, int LANES, int R, int S>
__device__ __forceinline__ void token_body(const moe_lora& L, const void* __restrict__ x, int t, int rank, float scale,
                                           const uint16_t* __restrict__ A, const uint16_t* __restrict__ B,
                                           const void* base, void* out, int n0, int n1, float* v, float* o) {
  constexpr int kRows = 64 / LANES, kStep = kTokWaves * kRows;   // rows of B a wavefront, a workgroup loads at once
  constexpr int U = kStep * 8 <= kTokOut ? 8 : kTokOut / kStep;  // such loads in flight
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = L.r, part = (lane % LANES) * 8;
  const size_t yt = (size_t)t * L.N, end = (size_t)L.N * r;  // end of B
  auto load_rows = [&](uint4(&bv)[U], int at) {  // rows at .. of this workgroup's outputs, past the last one again;
                                                 // a chunk may run into the next row
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t from = (size_t)min(at + wave * kRows + lane / LANES + kStep * u, n1 - 1) * r + min(part, (r - 1) / 8 * 8);
      bv[u] = from + 8 <= end ? ld8h(B + from) : ld8h_part(B + from, (int)(end - from));
    }
  };
  auto load_y = [&](float(&y)[2], int n) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = n + threadIdx.x + i * kTokThreads;
      y[i] = base && e < n1 ? load1(base, YBF16, yt + e) : 0.f;
    }
  };
  uint4 bv[U];
  float y[2];
  load_rows(bv, n0);
  load_y(y, n0);
  for (int j = wave * R; j < rank; j += kTokWaves * R) {
    float acc[R];
    token_rows<XBF16, R, S>(x, (size_t)t * L.K, A, j, rank, L.K, acc);
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (lane == 0 && j + i < rank) v[j + i] = acc[i] * scale;
  }
  __syncthreads();
  f32x8 mine;
#pragma unroll
  for (int e = 0; e < 8; ++e) mine[e] = part + e < rank ? v[part + e] : 0.f;
  for (int n = n0; n < n1; n += kTokOut) {
    const int m = min(kTokOut, n1 - n);
    for (int at = 0; at < m; at += kStep * U) {
      if (n + at != n0) load_rows(bv, n + at);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const f32x8 w = widen(rank - part >= 8 ? bv[u] : keep8h(bv[u], 0, rank - part));
        float acc = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc = fmaf(mine[e], w[e], acc);
#pragma unroll
        for (int off = 1; off < LANES; off *= 2) acc += __shfl_xor(acc, off, 64);
        const int at_u = at + wave * kRows + lane / LANES + kStep * u;
        if (lane % LANES == 0 && at_u < m) o[at_u] = acc;
      }
    }
    __syncthreads();
    if (n != n0) load_y(y, n);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = threadIdx.x + i * kTokThreads;
      if (e < m) {
        if constexpr (YBF16)
          ((uint16_t*)out)[yt + n + e] = bf16_of(y[i] + o[e]);
        else
          ((float*)out)[yt + n + e] = y[i] + o[e];
      }
    }
    __syncthreads();
  }
}

// WIDE: banks of ranks over 16, whose forms take so many registers that a compute
// unit holds one workgroup instead of two: without the split, 400 tokens of
// K = N = 1024, rank 4, take 5.3 us instead of 3.9.
template <bool XBF16, bool YBF16, bool WIDE>
__global__ __launch_bounds__(kTokThreads, WIDE ? 2 : 4) void token_kernel(moe_lora L, const void* __restrict__ x,
                                                                          const int32_t* __restrict__ ids,
                                                                          const void* base, void* out, int per) {
  __shared__ __align__(16) float v[kMaxRank];
  __shared__ __align__(16) float o[kTokOut];
  constexpr int S = XBF16 ? 8 : 4;
  const int t = blockIdx.x, id = ids[t];
  const bool has = id >= 0 && id < L.num;
  const int rank = has ? rank_of(L, id) : 0;
  const float scale = has && L.scale ? L.scale[id] : 1.0f;
  const uint16_t* A = (const uint16_t*)L.a + (has ? (size_t)id * L.r * L.K : 0);
  const uint16_t* B = (const uint16_t*)L.b + (has ? (size_t)id * L.N * L.r : 0);
  const int n0 = blockIdx.y * per, n1 = min(L.N, n0 + per);
  if (rank == 0) {
    if (out == base) return;
    for (int e = n0 + threadIdx.x; e < n1; e += kTokThreads) {
      const size_t to = (size_t)t * L.N + e;
      if constexpr (YBF16)
        ((uint16_t*)out)[to] = base ? ((const uint16_t*)base)[to] : 0;
      else
        ((float*)out)[to] = base ? ((const float*)base)[to] : 0.f;
    }
  } else if (rank <= 8) {
    token_body<XBF16, YBF16, 1, 1, 8>(L, x, t, rank, scale, A, B, base, out, n0, n1, v, o);
  } else if (rank <= 16) {
    token_body<XBF16, YBF16, 2, 2, 4>(L, x, t, rank, scale, A, B, base, out, n0, n1, v, o);
  } else if constexpr (WIDE) {
    if (rank <= 32)
      token_body<XBF16, YBF16, 4, 4, 4>(L, x, t, rank, scale, A, B, base, out, n0, n1, v, o);
    else if (rank <= 64)
      token_body<XBF16, YBF16, 8, 4, S>(L, x, t, rank, scale, A, B, base, out, n0, n1, v, o);
    else
      token_body<XBF16, YBF16, 16, 4, S>(L, x, t, rank, scale, A, B, base, out, n0, n1, v, o);
  }
}

// ----------------------------------------------------------- 16 tokens a workgroup
//
// v_mfma_f32_16x16x32_bf16: lane l supplies row (first operand) or column
// (second) l % 16 at K positions 8 (l / 16) .. + 7, and receives column l % 16,
// rows 4 (l / 16) .. + 3.  fp32 values enter it as three bf16 parts whose sum they
// are exactly.
// Read straight from memory that layout touches a row a lane, sixteen bytes of
// it, which the cache serves a lane at a time; so every wavefront loads whole
// lines, eight or more lanes a row, and turns them in a part of LDS that is its
// own (no barrier; 16-byte pieces XOR-swizzled so that the eight lanes served
// together fall on different banks).
//
// A x: first operand the rows of A (16 of them a "task": one adapter, 16 of its
// ranks), second the tokens; the wavefronts split K in slabs of 64 and their
// parts meet in LDS.  The sum of a token's own adapter is split as fp32 inputs are,
// so the second product runs on bf16 operands and loses nothing of it, for bf16
// outputs too: two parts cut below 2^-15 of it, always towards 0, and a base that
// cancels the sum's upper bits leaves little else.
//
// B v: first operand the tokens' parts, second 16 outputs.  Column m of product q
// stands for output 4 m + q of a block of 64, so that four products leave four
// consecutive outputs of four tokens in each lane, a line of each token in 16.  B
// comes in slabs of 32 ranks.  Each adapter's product goes to its own tokens only,
// so one adapter's NaN cannot reach another's tokens.
//
// Large calls are bound by memory: 4096 tokens, K = N = 4096, rank 32, bf16, one
// request: 23.1 us, 4.4 TB/s over x, base, out and the adapter (5.2 is a copy's
// rate).  A tile at the border of two requests takes longer than the others, and
// at 4096 tokens every compute unit has one tile: twelve requests 30.0 us.

constexpr int kTileWaves = 8, kTileThreads = 64 * kTileWaves;
constexpr int kMaxPass = 8;             // most tasks per pass over x
constexpr int kVStride = kMaxRank + 8;  // bf16 elements of a token's row of v parts
constexpr int kParts = 3;               // bf16 parts of an fp32 value

// fp32 -> bf16 by truncation: what is left over is exact
__device__ __forceinline__ uint16_t take_bf16(float& f) {
  const uint32_t u = __float_as_uint(f) & 0xffff0000u;
  const float rest = f - __uint_as_float(u);
  f = fabsf(f) == INFINITY ? 0.0f : rest;  // an infinity leaves nothing over; a NaN, which may truncate to one, itself
  return (uint16_t)(u >> 16);
}

// four consecutive outputs of a token, n of them (<= 0: none) inside N
template <bool YBF16>
struct Four {
  uint32_t u[YBF16 ? 2 : 4];

  __device__ __forceinline__ void load(const void* base, size_t at, int n) {
    if constexpr (YBF16) {
      u[0] = u[1] = 0;
      if (!base) return;
      const uint16_t* p = (const uint16_t*)base + at;
      if (n >= 4) {
        const Packed4h v = *(const Packed4h*)p;
        u[0] = v.x, u[1] = v.y;
      } else {
        u[0] = ld2h_part(p, n), u[1] = ld2h_part(p + 2, n - 2);
      }
    } else {
      u[0] = u[1] = u[2] = u[3] = 0;
      if (!base) return;
      const float* p = (const float*)base + at;
      if (n >= 4) {
        const Packed4f v = *(const Packed4f*)p;
        u[0] = __float_as_uint(v.x), u[1] = __float_as_uint(v.y), u[2] = __float_as_uint(v.z), u[3] = __float_as_uint(v.w);
      } else {
        u[0] = __float_as_uint(ld1f_if(p, n > 0)), u[1] = __float_as_uint(ld1f_if(p + 1, n > 1));
        u[2] = __float_as_uint(ld1f_if(p + 2, n > 2));
      }
    }
  }

  __device__ __forceinline__ void load_all(const void* base, size_t at) {
    if constexpr (YBF16) {
      const Packed4h v = *(const Packed4h*)((const uint16_t*)base + at);
      u[0] = v.x, u[1] = v.y;
    } else {
      const Packed4f v = *(const Packed4f*)((const float*)base + at);
      u[0] = __float_as_uint(v.x), u[1] = __float_as_uint(v.y), u[2] = __float_as_uint(v.z), u[3] = __float_as_uint(v.w);
    }
  }

  // d and what was loaded, in one rounding; `keep`: the bits that were loaded
  __device__ __forceinline__ void add(v4f d, bool keep) {
    if constexpr (YBF16) {
      d += v4f{bf16_lo(u[0]), bf16_hi(u[0]), bf16_lo(u[1]), bf16_hi(u[1])};
      u[0] = keep ? u[0] : pack2(d[0], d[1]);
      u[1] = keep ? u[1] : pack2(d[2], d[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = keep ? u[i] : __float_as_uint(d[i] + __uint_as_float(u[i]));
    }
  }

  __device__ __forceinline__ void store_all(void* out, size_t at) const {
    if constexpr (YBF16)
      stream4h((uint16_t*)out + at, make_uint2(u[0], u[1]));
    else
      stream4f((float*)out + at, f32x4{__uint_as_float(u[0]), __uint_as_float(u[1]), __uint_as_float(u[2]),
                                       __uint_as_float(u[3])});
  }

  __device__ __forceinline__ void store(void* out, size_t at, int n) const {
    if constexpr (YBF16) {
      uint16_t* p = (uint16_t*)out + at;
      if (n >= 4) {
        *(Packed4h*)p = Packed4h{u[0], u[1]};
      } else {
        if (n > 0) p[0] = (uint16_t)u[0];
        if (n > 1) p[1] = (uint16_t)(u[0] >> 16);
        if (n > 2) p[2] = (uint16_t)u[1];
      }
    } else {
      uint32_t* p = (uint32_t*)out + at;
      if (n >= 4) {
        *(Packed4f*)p = Packed4f{__uint_as_float(u[0]), __uint_as_float(u[1]), __uint_as_float(u[2]), __uint_as_float(u[3])};
      } else {
        if (n > 0) p[0] = u[0];
        if (n > 1) p[1] = u[1];
        if (n > 2) p[2] = u[2];
      }
    }
  }
};

// a wavefront's slab of 64 K positions of the 16 tokens, a 16-byte piece a lane
// and load.  FULL: the slab lies inside K.
template <bool XBF16>
struct XSlab {
  static constexpr int kX = XBF16 ? 2 : 4;                                  // pieces a lane
  static constexpr int kXParts = XBF16 ? 1 : kParts, kBytes = kXParts * 16 * 128;  // bf16 parts of an element in LDS
  uint4 x[kX];

  template <bool FULL>
  __device__ __forceinline__ void load(const void* const (&xrow)[kX], int k0, int K) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kX; ++i) {
      if constexpr (XBF16) {
        const int k8 = k0 + (lane & 7) * 8;
        x[i] = FULL ? ld8h((const uint16_t*)xrow[i] + k8) : ld8h_to((const uint16_t*)xrow[i] + k8, K - k8);
      } else {
        const int k4 = k0 + (lane & 15) * 4;
        const float* f = (const float*)xrow[i] + k4;
        if (FULL || K - k4 >= 4) {
          const Packed4f v = *(const Packed4f*)f;
          x[i] = make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w));
        } else {
          x[i] = make_uint4(__float_as_uint(ld1f_if(f, k4 < K)), __float_as_uint(ld1f_if(f + 1, k4 + 1 < K)),
                            __float_as_uint(ld1f_if(f + 2, k4 + 2 < K)), 0u);
        }
      }
    }
  }

  __device__ __forceinline__ void put(char* lds) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kX; ++i) {
      if constexpr (XBF16) {
        const int row = i * 8 + (lane >> 3);
        *(uint4*)(lds + row * 128 + ((lane & 7) ^ (row & 7)) * 16) = x[i];
      } else {  // four elements, each in three parts
        const int row = i * 4 + (lane >> 4), c = lane & 15;
        char* to = lds + row * 128 + ((c >> 1) ^ (row & 7)) * 16 + (c & 1) * 8;
        float f[4] = {__uint_as_float(x[i].x), __uint_as_float(x[i].y), __uint_as_float(x[i].z), __uint_as_float(x[i].w)};
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
          const uint32_t h0 = take_bf16(f[0]), h1 = take_bf16(f[1]), h2 = take_bf16(f[2]), h3 = take_bf16(f[3]);
          *(uint2*)(to + p * 2048) = make_uint2(h0 | (h1 << 16), h2 | (h3 << 16));
        }
      }
    }
  }
};

// where a lane's two rows of each of a pass's tasks are: the adapter's A, bytes from there
struct ARows {
  const char* base[kMaxPass];
  uint32_t off[kMaxPass][2];
};

// the same positions of NP tasks of 16 ranks
template <int NP>
struct ASlab {
  uint4 a[NP][2];

  template <bool FULL>
  __device__ __forceinline__ void load(const ARows& rows, int k0, int K) {
    const int k8 = k0 + (threadIdx.x & 7) * 8;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint16_t* at = (const uint16_t*)(rows.base[p] + (rows.off[p][i] + (uint32_t)k8 * 2));
        a[p][i] = FULL ? ld8h(at) : ld8h_to(at, K - k8);
      }
  }

  __device__ __forceinline__ void put(char* lds) const {
    const int lane = threadIdx.x & 63, c8 = lane & 7;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = i * 8 + (lane >> 3);
        *(uint4*)(lds + p * 2048 + row * 128 + (c8 ^ (row & 7)) * 16) = a[p][i];
      }
  }
};

template <bool XBF16, int NP>
__device__ __forceinline__ void slab_product(const XSlab<XBF16>& x, const ASlab<NP>& a, char* lds, v4f (&acc)[kMaxPass]) {
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  wave_turn();  // the last slab has been read
  x.put(lds);
  a.put(lds + XSlab<XBF16>::kBytes);
  wave_turn();
  const char* xl = lds + col * 128;
  const char* al = lds + XSlab<XBF16>::kBytes + col * 128;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = ((h * 4 + g) ^ (col & 7)) * 16;
    v8bf xv[XSlab<XBF16>::kXParts];
#pragma unroll
    for (int i = 0; i < XSlab<XBF16>::kXParts; ++i) xv[i] = *(const v8bf*)(xl + i * 2048 + at);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const v8bf av = *(const v8bf*)(al + p * 2048 + at);
#pragma unroll
      for (int i = 0; i < XSlab<XBF16>::kXParts; ++i)
        acc[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, xv[i], acc[p], 0, 0, 0);
    }
  }
}

// A x over this wavefront's slabs of K (slab b belongs to wavefront
// b % kTileWaves), kAhead of them in flight.  The next loads are always issued,
// past the last slab again for the last: with a known number of them in flight
// the compiler waits for the slab it needs and no more.
template <bool XBF16>
struct Shrink {
  static constexpr int kAhead = XBF16 ? 3 : 1;
  XSlab<XBF16> x[kAhead + 1];
  const void* xrow[XSlab<XBF16>::kX];
  int first, full, last, K;  // this wavefront's first slab, the whole slabs, its last whole one

  __device__ __forceinline__ int slab(int i) const { return min(first + i * kTileWaves, last); }

  // x does not depend on the adapters: its first slabs are requested before they are known
  __device__ __forceinline__ void begin() {
    if (first < full) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) x[i].template load<true>(xrow, slab(i) * 64, K);
    }
  }

  // after begin()
  template <int NP>
  __device__ __forceinline__ void run(const ARows& arow, char* lds, v4f (&acc)[kMaxPass]) {
    if (first < full) {
      // A comes from the L2: the more tasks a slab has, the fewer slabs ahead
      constexpr int D = kAhead + 1, DA = NP <= 2 ? D : NP <= 4 ? 2 : 1;
      ASlab<NP> a[DA];
#pragma unroll
      for (int i = 0; i < DA - 1; ++i) a[i].template load<true>(arow, slab(i) * 64, K);
      for (int i = 0; first + i * kTileWaves < full; i += D) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
          a[(u + DA - 1) % DA].template load<true>(arow, slab(i + u + DA - 1) * 64, K);
          x[(u + D - 1) % D].template load<true>(xrow, slab(i + u + D - 1) * 64, K);
          if (first + (i + u) * kTileWaves < full) slab_product<XBF16, NP>(x[u], a[u % DA], lds, acc);
        }
      }
    }
    if (full % kTileWaves == first && full * 64 < K) {
      XSlab<XBF16> xe;
      ASlab<NP> ae;
      xe.template load<false>(xrow, full * 64, K);
      ae.template load<false>(arow, full * 64, K);
      slab_product<XBF16, NP>(xe, ae, lds, acc);
    }
  }
};

// A step of the second product: one adapter's ranks 8 j0 .. + 31
struct Step {
  const uint16_t* B;
  int slot, rank, j0;
};

// a step from LDS, in scalar registers
__device__ __forceinline__ Step fetch(const Step* list, int i) {
  const uint64_t b = (uint64_t)list[i].B;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b), hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  return Step{(const uint16_t*)(((uint64_t)hi << 32) | lo), (int)__builtin_amdgcn_readfirstlane(list[i].slot),
              (int)__builtin_amdgcn_readfirstlane(list[i].rank), (int)__builtin_amdgcn_readfirstlane(list[i].j0)};
}

// 64 rows of B (outputs nb ..) of a step, a 16-byte piece a lane and load; ranks
// behind the adapter's are zero
struct Pieces {
  uint4 p[4];

  // loads without a branch, whole pieces: what lies behind a row's end is masked by put(), but has to be there
  __device__ __forceinline__ void load(const Step& s, int nb, int r) {
    const int lane = threadIdx.x & 63, j = min(s.j0 + (lane & 3), (r - 1) / 8) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = ld8h(s.B + (size_t)(nb + i * 16 + (lane >> 2)) * r + j);
  }

  __device__ __forceinline__ void load_part(const Step& s, int nb, int N, int r) {
    const int lane = threadIdx.x & 63, j = (s.j0 + (lane & 3)) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = ld8h_to(s.B + (size_t)min(nb + i * 16 + (lane >> 2), N - 1) * r + j, s.rank - j);
  }

  // to LDS: row n of the 64 lies at 16 (n % 4) + n / 4
  __device__ __forceinline__ void put(const Step& s, char* lds) const {
    const int lane = threadIdx.x & 63, c = lane & 3, left = s.rank - (s.j0 + c) * 8;
    const uint32_t m0 = left >= 2 ? ~0u : left == 1 ? 0xffffu : 0u, m1 = left >= 4 ? ~0u : left == 3 ? 0xffffu : 0u,
                   m2 = left >= 6 ? ~0u : left == 5 ? 0xffffu : 0u, m3 = left >= 8 ? ~0u : left == 7 ? 0xffffu : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = i * 16 + (lane >> 2), m = n >> 2;
      *(uint4*)(lds + ((n & 3) * 16 + m) * 64 + (c ^ ((m >> 1) & 3)) * 16) =
          make_uint4(p[i].x & m0, p[i].y & m1, p[i].z & m2, p[i].w & m3);
    }
  }
};

// the products of a step's pieces with the parts of v
__device__ __forceinline__ void multiply(const Step& s, const uint16_t (&vs)[kParts][16][kVStride], const char* lds,
                                         v4f (&d)[4]) {
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  v8bf bv[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) bv[q] = *(const v8bf*)(lds + (q * 16 + col) * 64 + (g ^ ((col >> 1) & 3)) * 16);
#pragma unroll
  for (int m = 0; m < kParts; ++m) {
    const v8bf vv = *(const v8bf*)&vs[m][col][(s.j0 + g) * 8];
#pragma unroll
    for (int q = 0; q < 4; ++q) d[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vv, bv[q], d[q], 0, 0, 0);
  }
}

// a step's result to its own tokens: acc takes d where the token's slot is the step's
__device__ __forceinline__ void take(const Step& s, const int (&slot)[4], const v4f (&d)[4], v4f (&acc)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q][i] = slot[i] == s.slot ? d[q][i] : acc[q][i];
}

template <bool YBF16>
__device__ __forceinline__ void load_base(Four<YBF16> (&y)[4], const void* base, const size_t (&row)[4], int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i].load_all(base, row[i] + n);
}

// tokens without an adapter (slot -1) keep the base's bits
template <bool YBF16>
__device__ __forceinline__ void store_sum(Four<YBF16> (&y)[4], const int (&slot)[4], void* out,
                                          const size_t (&row)[4], int n, const v4f (&acc)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i].add(v4f{acc[0][i], acc[1][i], acc[2][i], acc[3][i]}, slot[i] < 0);
    y[i].store_all(out, row[i] + n);
  }
}

// The second product over whole blocks of 64 outputs, every kTileWaves-th from nb
// to n1.  G steps a block (ONCE), their settings in scalar registers throughout;
// or any number of steps, G at a time.  All loads and stores of a block are
// unconditional, so the pieces of the next G steps (fetched as soon as the last
// have gone to LDS) and the next block's base stay in flight meanwhile.
// `ready` is called once the first loads are under way: v is there after it.
// BASED: there is a base.
template <bool YBF16, bool BASED, int G, bool ONCE, class Ready>
__device__ __forceinline__ void blocks(Ready&& ready, const moe_lora& L, const Step* list, int steps,
                                       const int (&slot)[4], const size_t (&row)[4],
                                       const uint16_t (&vs)[kParts][16][kVStride], int nb, int n1, const void* base,
                                       void* out, char* lds) {
  const int n = (threadIdx.x & 15) * 4, r = L.r;
  Four<YBF16> y[4] = {}, y_next[4] = {};
  Pieces p[G];
  Step s[G];
#pragma unroll
  for (int g = 0; g < G; ++g) s[g] = fetch(list, ONCE ? g : min(g, steps - 1));
  if (nb < n1) {
    if constexpr (BASED) load_base(y, base, row, nb + n);
#pragma unroll
    for (int g = 0; g < G; ++g) p[g].load(s[g], nb, r);
  }
  ready();
  for (; nb < n1; nb += kTileWaves * 64) {
    const int nb2 = nb + kTileWaves * 64 < n1 ? nb + kTileWaves * 64 : nb;
    v4f acc[4] = {}, d[4] = {};
    if constexpr (BASED) load_base(y_next, base, row, nb2 + n);
    for (int u = 0; u < (ONCE ? G : steps); u += G) {
      const bool end = ONCE || u + G >= steps;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if constexpr (!ONCE) s[g] = fetch(list, min(u + g, steps - 1));
        wave_turn();  // the last pieces have been read
        p[g].put(s[g], lds);
        wave_turn();
        p[g].load(ONCE ? s[g] : fetch(list, end ? min(g, steps - 1) : min(u + G + g, steps - 1)), end ? nb2 : nb, r);
        if (ONCE || u + g < steps) {  // no memory but LDS in here
          if (s[g].j0 == 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q) d[q] = v4f{0.f, 0.f, 0.f, 0.f};
          }
          multiply(s[g], vs, lds, d);
          take(s[g], slot, d, acc);
        }
      }
    }
    store_sum(y, slot, out, row, nb + n, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = y_next[i];
  }
}

template <bool XBF16, bool YBF16>
__global__ __launch_bounds__(kTileThreads) void tile_kernel(moe_lora L, const void* __restrict__ x, int T,
                                                            const int32_t* __restrict__ ids, const void* base,
                                                            void* out, int per, int split, int work) {
  // tasks per pass over x, and a wavefront's LDS for them: x 2 or 6 KB, A 2 KB a task (later a slab of B)
  constexpr int kPass = XBF16 ? 8 : 4, kStage = XSlab<XBF16>::kBytes + kPass * 2048;
  __shared__ __align__(16) char stage[kTileWaves][kStage];
  __shared__ __align__(16) uint16_t vs[kParts][16][kVStride];
  __shared__ int tok_slot[16], ad_id[16], ad_rank[16], n_task, n_step;
  __shared__ float ad_scale[16];
  __shared__ uint8_t task_slot[128], task_tile[128];
  __shared__ Step step[64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
  // workgroups go to the 8 XCDs in turn: each XCD takes a run of tiles, whose
  // adapters are few and stay in its L2
  const int each = gridDim.x / 8, w = (blockIdx.x % 8) * each + blockIdx.x / 8;
  if (w >= work) return;
  const int t0 = w / split * 16, n0 = w % split * per, K = L.K, N = L.N, r = L.r;
  char* lds = stage[wave];

  Shrink<XBF16> ax;
  ax.first = wave, ax.full = K / 64, ax.K = K;
  ax.last = wave < ax.full ? ax.full - 1 - (ax.full - 1 - wave) % kTileWaves : 0;
#pragma unroll
  for (int i = 0; i < XSlab<XBF16>::kX; ++i) {
    const size_t row = (size_t)min(t0 + (XBF16 ? i * 8 + (lane >> 3) : i * 4 + (lane >> 4)), T - 1) * K;
    ax.xrow[i] = XBF16 ? (const void*)((const uint16_t*)x + row) : (const void*)((const float*)x + row);
  }
  // the tile's distinct adapters and their tasks; loads return in order, so the
  // first wavefront asks for these before it asks for x
  int id = -1, rank = 0;
  float scale = 1.0f;
  bool has = false;
  if (wave == 0) {
    if (lane < 16) id = ids[min(t0 + lane, T - 1)];  // past the end: the last token again
    has = lane < 16 && id >= 0 && id < L.num;
    if (has) rank = rank_of(L, id);
    has = rank > 0;  // an adapter of no rank is none
    if (has && L.scale) scale = L.scale[id];
  }
  ax.begin();
  if (wave == 0) {
    int lead = lane;  // the first of the tokens with this id
#pragma unroll
    for (int i = 15; i >= 0; --i)
      if (__builtin_amdgcn_readlane(id, i) == id) lead = i;
    const uint64_t leads = __ballot(has && lead == lane);
    const int tiles = (rank + 15) / 16, slabs = (rank + 31) / 32;
    int at = 0, total = 0, step_at = 0, steps = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int ti = ((leads >> i) & 1) ? __builtin_amdgcn_readlane(tiles, i) : 0;
      const int si = ((leads >> i) & 1) ? __builtin_amdgcn_readlane(slabs, i) : 0;
      at += i < lane ? ti : 0;
      step_at += i < lane ? si : 0;
      total += ti;
      steps += si;
    }
    if (lane < 16) tok_slot[lane] = has ? __popcll(leads & ((1ull << lead) - 1)) : -1;
    if ((leads >> lane) & 1) {
      const int slot = __popcll(leads & ((1ull << lane) - 1));
      ad_id[slot] = id;
      ad_rank[slot] = rank;
      ad_scale[slot] = scale;
      for (int i = 0; i < tiles; ++i) task_slot[at + i] = (uint8_t)slot, task_tile[at + i] = (uint8_t)i;
      const uint16_t* B = (const uint16_t*)L.b + (size_t)id * N * r;
      for (int i = 0; i < slabs; ++i) step[step_at + i] = Step{B, slot, rank, i * 4};
    }
    if (lane == 0) n_task = total, n_step = steps;
  }
  for (int i = threadIdx.x; i < (int)sizeof(vs) / 4; i += kTileThreads) ((uint32_t*)vs)[i] = 0;
  __syncthreads();
  const int ntask = __builtin_amdgcn_readfirstlane(n_task), steps = __builtin_amdgcn_readfirstlane(n_step);

  // A x, kPass tasks at a time
  auto join = [&](int p0, int np) {  // the wavefronts' sums of a pass, split and put to the tokens
    __syncthreads();
    for (int i = threadIdx.x; i < np * 256; i += kTileThreads) {
      const int p = i >> 8, tok = (i >> 4) & 15, rk = i & 15, q = p0 + p, slot = task_slot[q];
      if (tok_slot[tok] == slot) {
        float s = 0.f;
#pragma unroll
        for (int wv = 0; wv < kTileWaves; ++wv) s += ((const float*)stage[wv])[i];
        const int j = task_tile[q] * 16 + rk;
        s *= ad_scale[slot];
        if (j >= ad_rank[slot]) s = 0.f;
#pragma unroll
        for (int n = 0; n < kParts; ++n) vs[n][tok][j] = take_bf16(s);
      }
    }
    __syncthreads();
  };
  for (int p0 = 0; p0 < ntask; p0 += kPass) {
    v4f acc[kMaxPass] = {};
    const int np = min(kPass, ntask - p0);
    ARows arow;
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int q = min(p0 + p, ntask - 1), slot = __builtin_amdgcn_readfirstlane(task_slot[q]);
      arow.base[p] = (const char*)L.a + (size_t)__builtin_amdgcn_readfirstlane(ad_id[slot]) * r * K * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        arow.off[p][i] = (uint32_t)min(task_tile[q] * 16 + i * 8 + (lane >> 3), ad_rank[slot] - 1) * (uint32_t)K * 2u;
    }
    if (p0 > 0) ax.begin();
    if (np == 1)
      ax.template run<1>(arow, lds, acc);
    else if (np == 2)
      ax.template run<2>(arow, lds, acc);
    else if (np <= 4 || kPass == 4)
      ax.template run<4>(arow, lds, acc);
    else if constexpr (kPass == 8)
      ax.template run<8>(arow, lds, acc);
    wave_turn();
#pragma unroll
    for (int p = 0; p < kPass; ++p) *(v4f*)(lds + ((p * 16 + col) * 16 + g * 4) * 4) = acc[p];
    if (p0 + kPass < ntask) join(p0, np);
  }

  // B v and the base, a block of 64 outputs a wavefront at a time; a lane has
  // four outputs of the four tokens 4 g .. + 3.  Rows past the last token repeat
  // it, its stores too.
  int slot[4];
  size_t row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    slot[i] = tok_slot[g * 4 + i];
    row[i] = (size_t)min(t0 + g * 4 + i, T - 1) * N;
  }
  const int n1 = min(N, n0 + per);
  int nb = n0 + wave * 64;
  auto last = [&] {
    if (ntask > 0) join((ntask - 1) / kPass * kPass, (ntask - 1) % kPass + 1);
  };
  if (steps > 0) {
    // whole blocks (per is a multiple of 64); where r is not a multiple of eight the
    // last pieces run into the next seven rows, which have to be inside B
    const int whole = r % 8 == 0 ? n1 / 64 * 64 : max(0, min(n1, N - 7)) / 64 * 64;
    auto run = [&](auto g, auto once) {
      constexpr int G = decltype(g)::value;
      constexpr bool ONCE = decltype(once)::value;
      if (base)
        blocks<YBF16, true, G, ONCE>(last, L, step, steps, slot, row, vs, nb, whole, base, out, lds);
      else
        blocks<YBF16, false, G, ONCE>(last, L, step, steps, slot, row, vs, nb, whole, base, out, lds);
    };
    using yes = std::true_type;
    if (steps == 1)
      run(std::integral_constant<int, 1>(), yes());
    else if (steps == 2)
      run(std::integral_constant<int, 2>(), yes());
    else if (steps == 3)
      run(std::integral_constant<int, 3>(), yes());
    else if (steps == 4)
      run(std::integral_constant<int, 4>(), yes());
    else
      run(std::integral_constant<int, 4>(), std::false_type());
    if (nb < whole) nb += (whole - nb + kTileWaves * 64 - 1) / (kTileWaves * 64) * (kTileWaves * 64);
  } else {
    last();
  }
  for (; nb < n1; nb += kTileWaves * 64) {
    Four<YBF16> y[4];
    v4f acc[4] = {}, d[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i].load(base, row[i] + nb + col * 4, N - nb - col * 4);
    for (int u = 0; u < steps; ++u) {
      const Step s = fetch(step, u);
      Pieces p;
      p.load_part(s, nb, N, r);
      wave_turn();
      p.put(s, lds);
      wave_turn();
      if (s.j0 == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) d[q] = v4f{0.f, 0.f, 0.f, 0.f};
      }
      multiply(s, vs, lds, d);
      take(s, slot, d, acc);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i].add(v4f{acc[0][i], acc[1][i], acc[2][i], acc[3][i]}, slot[i] < 0);
      y[i].store(out, row[i] + nb + col * 4, N - nb - col * 4);
    }
  }
}

// Which form.  The token form reads A and B once a token and keeps a compute unit
// (two tokens on one up to rank 16) for a chain of reads; the tile form once a
// tile and distinct adapter, but takes 8 us for a tile at least.  Both measured
// over 150 drawn calls (K, N 64..4096, r 1..64, up to 64 requests): this rule is
// 1.0% off the better of the two on the mean (62% at most, where both take under 15
// us), the token form alone 23%, the tile form alone 101%.  E.g. K = N = 4096, r = 16,
// bf16, twelve requests: 128 tokens 8.6 against 14.9 us, 1024 tokens 24.9 against 15.6.
bool token_form(const moe_lora* L, int T) {
  const double products = (double)T * L->r * ((double)L->K + L->N);
  return T <= 128 || (products <= 24e6 && (T <= 512 || (L->r <= 16 && T <= 1536)));
}

template <bool XBF16, bool YBF16>
void run(const moe_lora* L, const void* x, int T, const int32_t* ids, const void* base, void* out, hipStream_t s) {
  constexpr int kGroups = 256;  // one workgroup a compute unit
  if (token_form(L, T)) {
    const int split = max(1, min(kGroups / T, (L->N + 127) / 128));
    const int per = ((L->N + split - 1) / split + 63) / 64 * 64;
    auto* kernel = L->r > 16 ? token_kernel<XBF16, YBF16, true> : token_kernel<XBF16, YBF16, false>;
    launch(MOE_PROF_LORA, kernel, dim3(T, (L->N + per - 1) / per), dim3(kTokThreads), 0, s, *L, x, ids, base, out, per);
  } else {
    const int tiles = (T + 15) / 16;
    const int split = max(1, min(kGroups / tiles, (L->N + 63) / 64));  // no second round for a few workgroups
    const int per = ((L->N + split - 1) / split + 63) / 64 * 64;
    const int parts = (L->N + per - 1) / per, work = tiles * parts;
    launch(MOE_PROF_LORA, tile_kernel<XBF16, YBF16>, dim3((work + 7) / 8 * 8), dim3(kTileThreads), 0, s, *L, x, T, ids,
           base, out, per, parts, work);
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
