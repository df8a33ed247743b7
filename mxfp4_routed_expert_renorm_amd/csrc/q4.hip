// Products with matrices of 4-bit codes and a scale per group of inputs
// (moe_q4_linear, moe_q4_grouped), on bf16 MFMA.
//
// Codes become bf16 exactly (integers up to 15 off a zero point, E2M1 values); bf16 x
// is taken as it is and fp32 x as three bf16 parts that hold all its bits, so every
// product is exact.  A group's products are summed by the matrix units in fp32, then
// scaled and added to the row's sum.
#include "q4_dev.h"

namespace moe {

namespace {

using namespace q4;

constexpr int kWaves = 8;

// 16 outputs (SWIGLU: and the 16 above them) for up to 16 TT rows of x.  The wavefronts
// take blocks of 128 inputs in turn; their sums meet in LDS.  MFMA 16x16x32: lane l
// supplies row (x) or column (codes) l % 16 at inputs 8 (l / 16) on, and gets rows
// 4 (l / 16) + i of column l % 16.
template <bool XF32, bool FP4, int TT, bool GLU>
__global__ __launch_bounds__(64 * kWaves) void q4_rows_kernel(Q4Args a) {
  constexpr int NT = GLU ? 2 : 1;
  __shared__ float red[kWaves][NT * TT * 256];
  Tile tile;
  if (!find_tile<false>(a, blockIdx.z * kTilesY + blockIdx.y, 16 * TT, tile)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const int n = min((int)blockIdx.x * 16 + c, a.N - 1);
  const uint8_t* codes = a.codes + tile.e * a.code_stride;
  const uint8_t* scales = (const uint8_t*)a.scales + tile.e * a.scale_stride;
  const uint8_t* zeros = a.zeros ? a.zeros + tile.e * a.zero_stride : nullptr;
  size_t xrow[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) xrow[i] = (size_t)(tile.row + min(16 * i + c, tile.rows - 1)) * a.K;
  v4f acc[NT][TT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[i][t] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave * 128; k0 < a.K; k0 += kWaves * 128) {
    uint32_t d[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint4 v = ld_stream16(codes + (size_t)(n + i * a.N) * (a.K / 2) + min(k0 / 2 + 16 * q, a.K / 2 - 16));
      d[i][0] = v.x, d[i][1] = v.y, d[i][2] = v.z, d[i][3] = v.w;
      transpose4(d[i]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + 32 * j;
      if (k >= a.K) break;
      const int g = group_of(a, k / 32);
      v8bf w[NT];
      float s[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const size_t at = (size_t)(n + i * a.N) * a.groups + g;
        s[i] = scale_of(raw_scale(scales, a.st, at), a.st);
        w[i] = codes_to_bf16<FP4>(d[i][j], FP4 ? 0.f : zeros ? (float)zeros[at] : 8.f);
      }
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        XPart<XF32> x;
        x.load(a.x, xrow[t] + k + 8 * q);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          v4f part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int p = XPart<XF32>::kParts - 1; p >= 0; --p)
            part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.p[p], w[i], part, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][t][r] = fmaf(s[i], part[r], acc[i][t][r]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) *(v4f*)&red[wave][((i * TT + t) * 64 + lane) * 4] = acc[i][t];
  __syncthreads();
  for (int o = threadIdx.x; o < TT * 256; o += 64 * kWaves) {
    const int t = o >> 8, r = (o >> 4) & 15, col = o & 15;  // row r and column col of row tile t
    const int at = (t * 64 + (r >> 2) * 16 + col) * 4 + (r & 3);
    float v[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int u = 0; u < kWaves; ++u) v[i] += red[u][i * TT * 256 + at];
    }
    if (GLU) v[0] *= gate_sigmoid(v[0]) * v[NT - 1];
    const int out = blockIdx.x * 16 + col, row = 16 * t + r;
    if (out < a.N && row < tile.rows) {
      const size_t to = (size_t)(tile.row + row) * a.N + out;
      if (a.ybf)
        ((uint16_t*)a.y)[to] = bf16_of(v[0]);
      else
        ((float*)a.y)[to] = v[0];
    }
  }
}

template <bool XF32, bool FP4, int TT>
void run_rows(const Q4Args& a, hipStream_t s) {
  const int size = 16 * TT;
  // a matrix's last tile may be short: at most one such a matrix that has rows
  const int tiles = a.offsets ? a.T / size + min(a.num, a.T) : (a.T + size - 1) / size;
  const dim3 grid((a.N + 15) / 16, min(tiles, kTilesY), (tiles + kTilesY - 1) / kTilesY), block(64 * kWaves);
  if (a.swiglu)
    launch(MOE_PROF_Q4, q4_rows_kernel<XF32, FP4, TT, true>, grid, block, 0, s, a);
  else
    launch(MOE_PROF_Q4, q4_rows_kernel<XF32, FP4, TT, false>, grid, block, 0, s, a);
}

template <bool XF32, bool FP4>
void run_q4(const Q4Args& a, hipStream_t s) {
  if (a.T > 64 && (uintptr_t)a.x % 16 == 0) {
    launch_q4_tile(a, XF32, FP4, s);
    return;
  }
  run_rows<XF32, FP4, 1>(a, s);
}

}  // namespace

moe_status launch_q4(const moe_q4* q, const void* x, moe_dtype xt, int T, const int32_t* offsets, void* y, moe_dtype yt,
                     hipStream_t s) {
  const Q4Args a{x, q->codes, q->zeros, q->scales, y, offsets, T, q->K, q->N, q->num, q->group, q->K / q->group, q->st,
                 q->act == MOE_Q4_SWIGLU, yt == MOE_BF16, q->code_stride, q->scale_stride, q->zero_stride,
                 q->group == 32 ? 0u : (uint32_t)(((uint64_t)1 << 32) / (q->group / 32)) + 1, q->group == 32};
  const bool xf = xt == MOE_F32, fp4 = q->code == MOE_Q4_FP4;
  if (xf)
    fp4 ? run_q4<true, true>(a, s) : run_q4<true, false>(a, s);
  else
    fp4 ? run_q4<false, true>(a, s) : run_q4<false, false>(a, s);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
