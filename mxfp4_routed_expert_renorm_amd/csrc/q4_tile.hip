// Products with 4-bit weights for many rows: tiles of up to 128 rows on MFMA.
#include "q4_dev.h"

namespace moe {

namespace {

using namespace q4;

typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kFold = 0;  // E2M1 codes with E8M0 scales: the scale goes into the convert, exactly

// v_mfma_f32_32x32x16_bf16: lane l supplies row (x) or column (codes) l % 32 at inputs
// 8 (l / 32) on, and gets rows 8 (i / 4) + 4 (l / 32) + i % 4 of column l % 32.
__device__ __forceinline__ v16f mfma(v8bf a, v8bf b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// GR: inputs whose products are summed before they are scaled (kFold: all).
// A workgroup takes TM * 32 rows and 4 * NT * 32 rows of the matrix; a wavefront NT * 32
// of them (SWIGLU: 32 gate rows and the 32 up rows that go with them).
template <bool XF32, bool FP4, int GR, int NT, int TM>
struct TileKernel {
  static constexpr int BK = XF32 ? 64 : 128;       // inputs a stage: 256 bytes of a row of x
  static constexpr int kPieces = TM * 2;           // 16-byte pieces of x a thread stages
  static constexpr int kW = BK / 64;               // 16-byte pieces of codes a lane and column
  static constexpr int kS = BK / 32;               // scales a lane and column
  static constexpr int kPer = XF32 ? 4 : 8;        // elements of x a piece

  struct Stage {
    u32x4_t x[kPieces];
    u32x4_t w[NT][kW];
    float s[NT][kS], z[NT][kS];
  };

  template <int NL>
  __device__ static __forceinline__ void body(const Q4Args& a, const Tile& tile, u32x4_t* lds) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 31, h = lane >> 5;
    const uint8_t* codes = a.codes + tile.e * a.code_stride;
    const uint8_t* scales = (const uint8_t*)a.scales + tile.e * a.scale_stride;
    const uint8_t* zeros = a.zeros ? a.zeros + tile.e * a.zero_stride : nullptr;
    int n[NT];  // this lane's rows of the matrix, and the outputs they stand for
    int out[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      out[i] = a.swiglu ? blockIdx.x * 128 + wave * 32 + c : (blockIdx.x * 4 + wave) * NT * 32 + 32 * i + c;
      n[i] = min(out[i], a.N - 1) + (a.swiglu ? i * a.N : 0);
    }
    v16f acc[NL][NT];
#pragma unroll
    for (int m = 0; m < NL; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[m][i][r] = 0.f;

    auto load = [&](Stage& s, int k0) {
#pragma unroll
      for (int j = 0; j < 2 * NL; ++j) {
        const int p = tid + 256 * j, row = min(p >> 4, tile.rows - 1), k = k0 + (p & 15) * kPer;
        const size_t at = (size_t)(tile.row + row) * a.K + min(k, a.K - kPer);
        if constexpr (XF32) {
          const Packed4f v = *(const Packed4f*)((const float*)a.x + at);
          s.x[j] = u32x4_t{__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w)};
        } else {
          const uint4 v = ld8h((const uint16_t*)a.x + at);
          s.x[j] = u32x4_t{v.x, v.y, v.z, v.w};
        }
        if (k >= a.K) s.x[j] = u32x4_t{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int u = 0; u < kW; ++u)
          s.w[i][u] = *(const u32x4_t*)(codes + (size_t)n[i] * (a.K / 2) +
                                        min(k0 / 2 + 32 * u + 16 * h, a.K / 2 - 16));
#pragma unroll
        for (int u = 0; u < kS; ++u) {
          if (GR > 32 && u % (GR / 32)) continue;
          const size_t at = (size_t)n[i] * a.groups + min(k0 + 32 * u, a.K - 32) / a.group;
          s.s[i][u] = load_scale(scales, a.st, at);
          s.z[i][u] = FP4 ? 0.f : zeros ? (float)zeros[at] : 8.f;
        }
      }
    };
    auto store = [&](const Stage& s, int buf) {
#pragma unroll
      for (int j = 0; j < 2 * NL; ++j) {
        const int p = tid + 256 * j, row = p >> 4, ch = p & 15;
        lds[buf * TM * 512 + row * 16 + (ch ^ (row & 15))] = s.x[j];
      }
    };
    auto rows_of_x = [&](int buf, int m, int step) {  // 16 inputs of 32 rows
      const int row = 32 * m + c;
      const u32x4_t* at = lds + buf * TM * 512 + row * 16;
      XPart<XF32> x;
      if constexpr (XF32) {
        const u32x4_t u = at[(4 * step + 2 * h) ^ (row & 15)], v = at[(4 * step + 2 * h + 1) ^ (row & 15)];
        x.split(f32x8{__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w),
                      __uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)});
      } else {
        x.p[0] = as_bf(at[(2 * step + h) ^ (row & 15)]);
      }
      return x;
    };
    auto codes_of = [&](const Stage& s, int i, int u, uint32_t (&d)[4]) {  // d[j]: this half's dword of step j
      d[0] = s.w[i][u].x, d[1] = s.w[i][u].y, d[2] = s.w[i][u].z, d[3] = s.w[i][u].w;
      const auto p = __builtin_amdgcn_permlane32_swap(d[0], d[1], false, false);
      const auto q = __builtin_amdgcn_permlane32_swap(d[2], d[3], false, false);
      d[0] = p[0], d[1] = q[0], d[2] = p[1], d[3] = q[1];
    };

    Stage cur, next;
    load(cur, 0);
    store(cur, 0);
    const int stages = (a.K + BK - 1) / BK;
    for (int st = 0; st < stages; ++st) {
      __syncthreads();
      const int buf = st & 1;
      load(next, min(st + 1, stages - 1) * BK);
#pragma unroll
      for (int u = 0; u < kW; ++u) {
        uint32_t d[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) codes_of(cur, i, u, d[i]);
        if constexpr (GR == kFold) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v8bf w[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) w[i] = fp4_to_bf16_scaled(d[i][j], cur.s[i][2 * u + j / 2]);
#pragma unroll
            for (int m = 0; m < NL; ++m) {
              const XPart<XF32> x = rows_of_x(buf, m, 4 * u + j);
#pragma unroll
              for (int p = XPart<XF32>::kParts - 1; p >= 0; --p)
#pragma unroll
                for (int i = 0; i < NT; ++i) acc[m][i] = mfma(x.p[p], w[i], acc[m][i]);
            }
          }
        } else {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            v8bf w[NT][2];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int j = 0; j < 2; ++j) w[i][j] = codes_to_bf16<FP4>(d[i][2 * g + j], cur.z[i][2 * u + g]);
#pragma unroll
            for (int m = 0; m < NL; ++m) {
              v16f part[NT];
#pragma unroll
              for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) part[i][r] = 0.f;
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const XPart<XF32> x = rows_of_x(buf, m, 4 * u + 2 * g + j);
#pragma unroll
                for (int p = XPart<XF32>::kParts - 1; p >= 0; --p)
#pragma unroll
                  for (int i = 0; i < NT; ++i) part[i] = mfma(x.p[p], w[i][j], part[i]);
              }
#pragma unroll
              for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[m][i][r] = fmaf(cur.s[i][2 * u + g], part[i][r], acc[m][i][r]);
            }
          }
        }
      }
      store(next, buf ^ 1);
      cur = next;
    }
#pragma unroll
    for (int m = 0; m < NL; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (NT == 2 && i == 1 && a.swiglu) continue;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int row = 32 * m + 8 * (r / 4) + 4 * h + r % 4;
          float v = acc[m][i][r];
          if (NT == 2 && a.swiglu) v *= gate_sigmoid(v) * acc[m][NT - 1][r];
          if (row < tile.rows && out[i] < a.N) {
            const size_t to = (size_t)(tile.row + row) * a.N + out[i];
            if (a.ybf)
              ((uint16_t*)a.y)[to] = bf16_of(v);
            else
              ((float*)a.y)[to] = v;
          }
        }
      }
  }
};

template <bool XF32, bool FP4, int GR, int NT, int TM>
__global__ __launch_bounds__(256) void q4_tile_kernel(Q4Args a) {
  extern __shared__ u32x4_t lds[];
  Tile tile;
  if (!find_tile(a, blockIdx.z * kTilesY + blockIdx.y, 32 * TM, tile)) return;
  typedef TileKernel<XF32, FP4, GR, NT, TM> Kernel;
  const int live = (tile.rows + 31) / 32;
  if (TM > 3 && live == 4)
    Kernel::template body<TM < 4 ? TM : 4>(a, tile, lds);
  else if (TM > 2 && live == 3)
    Kernel::template body<TM < 3 ? TM : 3>(a, tile, lds);
  else if (live == 2)
    Kernel::template body<2>(a, tile, lds);
  else
    Kernel::template body<1>(a, tile, lds);
}

template <bool XF32, bool FP4, int GR, int NT, int TM>
void run(const Q4Args& a, hipStream_t s) {
  const int size = 32 * TM, cols = a.swiglu ? 128 : 128 * NT;
  const int tiles = a.offsets ? a.T / size + min(a.num, a.T) : (a.T + size - 1) / size;
  const dim3 grid((a.N + cols - 1) / cols, min(tiles, kTilesY), (tiles + kTilesY - 1) / kTilesY);
  launch(MOE_PROF_Q4, q4_tile_kernel<XF32, FP4, GR, NT, TM>, grid, dim3(256), (size_t)2 * TM * 512 * 16, s, a);
}

template <bool XF32, bool FP4>
void run_types(const Q4Args& a, hipStream_t s) {
  if constexpr (FP4) {
    if (a.st == MOE_SCALE_E8M0) {
      run<XF32, FP4, kFold, 2, 4>(a, s);
      return;
    }
  }
  run<XF32, FP4, 32, 2, 2>(a, s);
}

}  // namespace

moe_status launch_q4_tile(const Q4Args& a, bool xf32, bool fp4, hipStream_t s) {
  if (xf32)
    fp4 ? run_types<true, true>(a, s) : run_types<true, false>(a, s);
  else
    fp4 ? run_types<false, true>(a, s) : run_types<false, false>(a, s);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
