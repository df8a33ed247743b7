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

// How a block of 128 inputs meets its scales.
enum {
  kFold = 0,   // E2M1 codes, E8M0 scales of 32: in the convert, which is exact
  kBlock = 1,  // the block lies in one group: its sum is scaled
  kChunk = 2   // each 32 inputs' sum is scaled
};

// 16 outputs for up to 16 rows of x.  The wavefronts share the blocks of 128 inputs, the
// codes of some of them requested at once, and their sums meet in LDS; of a SWIGLU matrix
// half of them take the gate's rows, half the rows that go with them.  MFMA 16x16x32: lane l
// supplies row (x) or column (codes) l % 16 at eight inputs that l / 16 tells, and gets rows
// 4 (l / 16) + i of column l % 16.
//
// Sixteen lanes that load from sixteen rows take sixteen cycles of the cache, from one row
// two, and at 16 bytes of codes a lane that bounds the kernel before the memory does.  So
// codes and x come row by row and go through LDS to the lanes that take them, and the lanes
// of a row load the scales of different blocks and exchange them.
//
// Measured, integer codes, groups of 128: one row by 4096 x 4096 5.8 us (1.9 the launch; the
// 8.8 MB take 1.7), by 8192 x 4096 8.5; 64 rows of 64 experts, SWIGLU of 2048, 63 to 68 us, 2.7
// TB/s, where the conversion (37 us of it), LDS and the memory (36) take about as long.
// Tried and slower or no faster: x straight to the lanes for up to four rows (70 us), twice
// the codes requested at once (68), two or four groups of outputs a workgroup (70, 72).
template <bool XF32, bool FP4, int MODE, int W>
struct Rows {
  static constexpr int U = (!FP4 && MODE == kChunk) || W == 16 ? 2 : 4;  // blocks a turn, as many as registers allow
  static constexpr int kPieces = 4 * U;                   // of 16 bytes of codes a row and turn
  // Zero points: sum q x - z sum x with the sum of x from a matrix of ones, which costs the
  // matrix units one instruction, or, where that would be three, off the codes, which costs
  // the others ten a dword.
  static constexpr bool kOnes = !FP4 && !XF32;
  // Whether an instruction takes 32 inputs in a row, and not eight of each chunk.
  static constexpr bool kInRow = MODE == kChunk || XF32;
  static constexpr int xs = XF32 ? 4 : 2;
  static constexpr int kUnits = XF32 ? 2 : 1, kSteps = 4 / kUnits;  // 256 bytes of x's rows, and instructions on them
  static constexpr int kScales = MODE == kChunk ? 4 : 1;           // words of scales a lane and turn

  struct __attribute__((packed, aligned(1))) Word {
    uint32_t v;
  };
  // A wavefront's own: 16 rows of a turn of codes, or a unit of x.  Row r's piece of 16
  // bytes p lies at p ^ r % 16.
  struct Smem {
    union {
      float red[W][256];
      u32x4_t x[W][256];
    };
  };

  static __device__ __forceinline__ void run(const Q4Args& a, const Tile& tile, Smem& sm) {
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = a.swiglu ? W / 2 : W, up = wave >= waves ? a.N : 0;  // that share a row, and its place
    const int blocks = (a.K + 127) / 128, per = (blocks + waves - 1) / waves;
    const int first = (up ? wave - waves : wave) * per, end = min(first + per, blocks);  // of this wavefront
    const int units = min(end * kUnits, (a.K * xs + 255) / 256);  // of x: each holds some of a row
    const uint8_t* codes = a.codes + tile.e * a.code_stride;
    const uint8_t* x0 = (const uint8_t*)a.x + (size_t)tile.row * a.K * xs;
    // Scales lie at any alignment of theirs, but each within an aligned word: that word is
    // loaded, and the bytes are picked when it is used.
    const int st = MODE == kFold ? (int)MOE_SCALE_E8M0 : a.st;
    const int shift = st == MOE_F32 ? 2 : st == MOE_BF16 ? 1 : 0;
    const uint8_t* scales = (const uint8_t*)a.scales + tile.e * a.scale_stride;
    const uint8_t* zeros = a.zeros ? a.zeros + tile.e * a.zero_stride : scales;
    const uint32_t sfrom = (uint32_t)((uintptr_t)scales & 3), zfrom = (uint32_t)((uintptr_t)zeros & 3);
    scales -= sfrom, zeros -= zfrom;

    const int n0 = blockIdx.x * 16, mine_n = min(n0 + c, a.N - 1) + up;  // the lane's row of the matrix
    const uint32_t srow = (uint32_t)mine_n * (uint32_t)a.groups;
    uint32_t xat[4];  // piece l % 16 of rows 4 j + l / 16
#pragma unroll
    for (int j = 0; j < 4; ++j) xat[j] = (uint32_t)min(4 * j + q, tile.rows - 1) * (uint32_t)(a.K * xs) + 16 * c;
    v4f acc = {0.f, 0.f, 0.f, 0.f};

    // Past a row's end, or x's last row, other pieces come in their place: they are
    // multiplied by zero or not at all.
    u32x4_t xv[4], got[4];
    auto load_x = [&](int unit) {
      const uint8_t* xp = x0 + unit * 256;
      const int left = a.K * xs - unit * 256;  // bytes of a row
      const int back = left < 256 ? max(0, 16 * c - (left - 16)) : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (4 * j >= tile.rows) break;
        const uint4 h = ld8h((const uint16_t*)(xp + (xat[j] - (uint32_t)back)));
        xv[j] = u32x4_t{h.x, h.y, h.z, h.w};
      }
    };
    // x's rows of a unit through LDS to the lanes that multiply them, the next unit requested
    // in between
    auto turn_x = [&](int next) {
      u32x4_t* mine = sm.x[wave];
#pragma unroll
      for (int j = 0; j < 4; ++j) mine[(4 * j + q) * 16 + (c ^ (4 * j + q))] = xv[j];
      if (next < units) load_x(next);
      wave_turn();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = XF32 ? 8 * (j / 2) + 2 * q + j % 2 : kInRow ? 4 * j + q : 4 * q + j;
        got[j] = mine[c * 16 + (at ^ c)];
      }
      wave_turn();
    };
    // A turn's codes: w[u], block u's chunk l / 16 of row l % 16, or (kInRow) that dword of
    // each of its chunks.
    u32x4_t w[U];
    auto load_codes = [&](int b0) {
      int row = n0 + lane / kPieces;
      asm volatile("" : "+v"(row));  // places are formed anew, not kept
      const int piece = min(lane % kPieces, min(4 * (end - b0), a.K / 32 - 4 * b0) - 1);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const uint32_t at = (uint32_t)(min(row + 64 / kPieces * j, a.N - 1) + up) * (uint32_t)(a.K / 2) + 16 * piece;
        w[j] = __builtin_nontemporal_load((const u32x4_t*)(codes + b0 * 64 + at));
      }
    };
    auto turn_codes = [&] {
      u32x4_t* mine = sm.x[wave];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int r = 64 / kPieces * j + lane / kPieces;
        mine[r * 16 + ((lane % kPieces) ^ r)] = w[j];
      }
      wave_turn();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (kInRow) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[u][j] = ((const uint32_t*)&mine[c * 16 + ((4 * u + j) ^ c)])[q];
        } else {
          w[u] = mine[c * 16 + ((4 * u + q) ^ c)];
        }
      }
      wave_turn();
    };
    // Scales and zero points of a turn: those of its block l / 16.
    const bool vec = MODE == kChunk && a.group == 32 && a.K % 128 == 0;
    const int last = a.K / 32 - 1;
    uint32_t ws[kScales], wz[kScales];
    auto place = [&](int b0, int j) {  // of chunk j, or of the block
      return srow + (uint32_t)group_of(a, min(4 * (b0 + q) + j, last));
    };
    auto load_scales = [&](int b0) {
      if constexpr (MODE == kFold) {  // four bytes
        ws[0] = ((const Word*)(scales + (sfrom + srow + min(4 * (b0 + q), a.groups - 4))))->v;
      } else if (vec) {
        const uint32_t at = srow + 4 * min(b0 + q, blocks - 1);
        const uint8_t* p = scales + (sfrom + (at << shift));
        if (st == MOE_F32) {
          const Packed4f f = *(const Packed4f*)p;
          ws[0] = __float_as_uint(f.x), ws[kScales / 4] = __float_as_uint(f.y);
          ws[kScales / 2] = __float_as_uint(f.z), ws[kScales - 1] = __float_as_uint(f.w);
        } else if (st == MOE_BF16) {
          const Packed4h f = *(const Packed4h*)p;
          ws[0] = f.x, ws[kScales / 4] = f.y;
        } else {
          ws[0] = ((const Word*)p)->v;
        }
        if constexpr (!FP4) wz[0] = ((const Word*)(zeros + (zfrom + (a.zeros ? at : at << shift))))->v;
      } else {
#pragma unroll
        for (int j = 0; j < kScales; ++j) {
          const uint32_t at = place(b0, j);
          ws[j] = *(const uint32_t*)(scales + ((sfrom + (at << shift)) & ~3u));
          if constexpr (!FP4) wz[j] = *(const uint32_t*)(zeros + ((zfrom + (a.zeros ? at : at << shift)) & ~3u));
        }
      }
    };
    float s[kScales], z[kScales];  // as values; kFold: four bytes still
    auto take_scales = [&](int b0) {
#pragma unroll
      for (int j = 0; j < kScales; ++j) {
        if constexpr (MODE == kFold) {
          const int skip = 4 * (b0 + q) - min(4 * (b0 + q), a.groups - 4);  // in a row's last block
          s[j] = __uint_as_float(ws[0] >> (8 * min(skip, 3)));
        } else if (vec) {
          const uint32_t v = st == MOE_F32    ? ws[j]
                             : st == MOE_BF16 ? ws[j / 2] >> (16 * (j % 2))
                                              : (ws[0] >> (8 * j)) & 255;
          s[j] = scale_of(v, st);
          if constexpr (!FP4) z[j] = a.zeros ? (float)((wz[0] >> (8 * j)) & 255) : 8.f;
        } else {
          const uint32_t at = place(b0, j), v = ws[j] >> (8 * ((sfrom + (at << shift)) & 3));
          s[j] = scale_of(st == MOE_SCALE_E8M0 ? v & 255 : v, st);
          if constexpr (!FP4) z[j] = a.zeros ? (float)((wz[j] >> (8 * ((zfrom + at) & 3))) & 255) : 8.f;
        }
      }
    };
    auto of_block = [&](float v, int u) {  // lane row u's value in every row
      return __int_as_float(__builtin_amdgcn_ds_bpermute((16 * u + c) * 4, __float_as_int(v)));
    };
    // block u of the turn; chunks: of its four, in the row's last block fewer
    auto multiply = [&](int u, int block) {
      const int chunks = a.K / 32 - 4 * block;
      float sj = 0.f, zj = 0.f;
      uint32_t bytes = 0;
      v4f part, ones;
      auto start = [&](int j) {
        ones = part = v4f{0.f, 0.f, 0.f, 0.f};
        sj = of_block(s[j], u);
        if constexpr (!FP4) zj = of_block(z[j], u);
      };
      auto add = [&] {
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = fmaf(sj, kOnes ? fmaf(-zj, ones[r], part[r]) : part[r], acc[r]);
      };
      if constexpr (MODE == kBlock) start(0);
      if constexpr (MODE == kFold) {
        bytes = __float_as_uint(of_block(s[0], u));
        if (!kInRow) bytes >>= 8 * q;
      }
#pragma unroll
      for (int half = 0; half < kUnits; ++half) {
        if (half && 2 * half >= chunks) break;
        turn_x(block * kUnits + half + 1);
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
          const int j = half * kSteps + step;
          if (kInRow && j >= chunks) break;
          if constexpr (MODE == kChunk) start(j);
          v8bf v;
          if constexpr (MODE == kFold) {
            // the convert takes the exponent field as the E8M0 byte
            const float f = __uint_as_float((kInRow ? bytes >> (8 * j) : bytes) << 23);
            v = fp4_to_bf16_scaled(!kInRow && chunks < 4 && q >= chunks ? 0u : w[u][j], f);
          } else if constexpr (kOnes) {
            v = int4_to_bf16(w[u][j]);
          } else {
            v = codes_to_bf16<FP4>(w[u][j], zj);
          }
          XPart<XF32> x;
          if constexpr (XF32) {
            const u32x4_t lo = got[2 * step], hi = got[2 * step + 1];
            x.split(f32x8{__uint_as_float(lo.x), __uint_as_float(lo.y), __uint_as_float(lo.z), __uint_as_float(lo.w),
                          __uint_as_float(hi.x), __uint_as_float(hi.y), __uint_as_float(hi.z), __uint_as_float(hi.w)});
          } else {
            x.p[0] = as_bf(got[j]);
            if (!kInRow && chunks < 4) x.p[0] = q >= chunks ? as_bf(u32x4_t{0, 0, 0, 0}) : x.p[0];
          }
#pragma unroll
          for (int p = XPart<XF32>::kParts - 1; p >= 0; --p) {
            v4f& to = MODE == kFold ? acc : part;
            to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.p[p], v, to, 0, 0, 0);
            if constexpr (kOnes) {
              constexpr uint32_t one = 0x3f803f80u;
              ones = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.p[p], as_bf(u32x4_t{one, one, one, one}), ones, 0, 0, 0);
            }
          }
          if constexpr (MODE == kChunk) add();
        }
      }
      if constexpr (MODE == kBlock) add();
    };

    for (int b0 = first; b0 < end; b0 += U) {
      load_codes(b0);
      load_scales(b0);
      if (b0 == first) load_x(first * kUnits);
      turn_codes();
      take_scales(b0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u && b0 + u >= end) break;
        multiply(u, b0 + u);
      }
    }
    __syncthreads();  // the sums take the place of x
    *(v4f*)&sm.red[wave][lane * 4] = acc;
    __syncthreads();
    for (int o = threadIdx.x; o < tile.rows * 16; o += 64 * W) {
      const int row = o >> 4, col = o & 15, at = ((row >> 2) * 16 + col) * 4 + (row & 3), out = n0 + col;
      float v = 0.f, other = 0.f;
#pragma unroll
      for (int u = 0; u < W / 2; ++u) v += sm.red[u][at], other += sm.red[W / 2 + u][at];
      v = a.swiglu ? v * (gate_sigmoid(v) * other) : v + other;
      if (out < a.N) {
        const size_t to = (size_t)(tile.row + row) * a.N + out;
        if (a.ybf)
          ((uint16_t*)a.y)[to] = bf16_of(v);
        else
          ((float*)a.y)[to] = v;
      }
    }
  }
};

template <bool XF32, bool FP4, int MODE, int W>
__global__ __launch_bounds__(64 * W, 4) void q4_rows_kernel(Q4Args a) {
  // all arguments at once, not one after the other as they are needed
  asm volatile("" ::"s"(a.x), "s"(a.codes), "s"(a.scales), "s"(a.zeros), "s"(a.y), "s"(a.offsets), "s"(a.T), "s"(a.K),
               "s"(a.N), "s"(a.st), "s"(a.groups), "s"(a.magic), "s"(a.unit));
  typedef Rows<XF32, FP4, MODE, W> Kernel;
  __shared__ typename Kernel::Smem sm;
  Tile tile;
  if (!find_tile<false>(a, blockIdx.z * kTilesY + blockIdx.y, 16, tile)) return;
  Kernel::run(a, tile, sm);
}

template <bool XF32, bool FP4, int MODE>
void run_rows(const Q4Args& a, hipStream_t s) {
  const int tiles = tile_groups(a, 16), cols = (a.N + 15) / 16;
  const dim3 grid(cols, min(tiles, kTilesY), (tiles + kTilesY - 1) / kTilesY);
  // Twice the wavefronts where a compute unit has one workgroup only: a wavefront's blocks are
  // a chain of waits.  One token, 4096 inputs, 2048 outputs 5.1 us against 5.4, 4096 5.8
  // against 6.1; 8192 9.9 against 8.6, 64 rows of 64 experts 86 against 63.
  if ((long)cols * tiles <= 256)
    launch(MOE_PROF_Q4, q4_rows_kernel<XF32, FP4, MODE, 16>, grid, dim3(1024), 0, s, a);
  else
    launch(MOE_PROF_Q4, q4_rows_kernel<XF32, FP4, MODE, 8>, grid, dim3(512), 0, s, a);
}

// Whether tiles of 128 rows are worth it.  The few-row form's workgroups take 16 rows of 16
// matrix rows and run 512 at a time, the tiles' 128 of 128 (SWIGLU 256) and run 256 at a
// time, each turn as long as thousands of the small ones.  Both measured, 4096 inputs and
// 4096 outputs, us a turn of tiles (up to 1024 rows) and rows of the small form in that
// time: MXFP4 33 and 180, other E2M1 36 and 200, integer codes 53 and 265, groups under 128
// 72 to 104 and 340 to 370, fp32 x 115 to 192 and 340 to 450.  SWIGLU, integer codes, 2048
// outputs of 64 experts, the small form and tiles: 512 rows 192 and 266, 1024 rows 276 and
// 278, 2048 rows 442 and 331.
template <bool XF32, bool FP4>
bool use_tiles(const Q4Args& a) {
  if ((uintptr_t)a.x % 16) return false;  // the tiles' direct loads to LDS
  const int live = std::min(a.num, a.T);
  const long small = (a.offsets ? a.T / 16 + live / 2 : (a.T + 15) / 16) * (long)((a.N + 15) / 16) * (a.swiglu ? 2 : 1);
  const long large = (a.offsets ? a.T / 128 + live : (a.T + 127) / 128) * (long)((a.N + 127) / 128);
  const bool plain = !XF32 && (a.group % 128 == 0 || (FP4 && a.st == MOE_SCALE_E8M0 && a.group == 32));
  return small > (plain ? (FP4 ? 3000 : 4000) : 6000) * ((large + 255) / 256);
}

template <bool XF32, bool FP4>
moe_status run_q4(const Q4Args& a, hipStream_t s) {
  if (use_tiles<XF32, FP4>(a)) return launch_q4_tile(a, XF32, FP4, s);
  if (FP4 && a.st == MOE_SCALE_E8M0 && a.group == 32 && a.K >= 128)
    run_rows<XF32, FP4, FP4 ? kFold : kChunk>(a, s);
  else if (a.group % 128 == 0)
    run_rows<XF32, FP4, kBlock>(a, s);
  else
    run_rows<XF32, FP4, kChunk>(a, s);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

moe_status launch_q4(const moe_q4* q, const void* x, moe_dtype xt, int T, const int32_t* offsets, void* y, moe_dtype yt,
                     hipStream_t s) {
  const Q4Args a{x, q->codes, q->zeros, q->scales, y, offsets, T, q->K, q->N, q->num, q->group, q->K / q->group, q->st,
                 q->act == MOE_Q4_SWIGLU, yt == MOE_BF16, q->code_stride, q->scale_stride, q->zero_stride,
                 q->group == 32 ? 0u : (uint32_t)(((uint64_t)1 << 32) / (q->group / 32)) + 1, q->group == 32};
  const bool xf = xt == MOE_F32, fp4 = q->code == MOE_Q4_FP4;
  if (xf) return fp4 ? run_q4<true, true>(a, s) : run_q4<true, false>(a, s);
  return fp4 ? run_q4<false, true>(a, s) : run_q4<false, false>(a, s);
}

}  // namespace moe
