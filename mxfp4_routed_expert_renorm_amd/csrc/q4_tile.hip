// Products with 4-bit weights for many rows: tiles of 128 rows on MFMA.
//
// A workgroup of eight wavefronts takes 128 rows of x and 128 or 256 rows of the matrix;
// a wavefront two blocks of 32 rows of x and one or two of the matrix.  Stages of 256
// bytes of x's rows and the codes and scales that go with them come by direct loads into a
// ring in LDS, ahead of the one that is multiplied.  Nothing in the loop is loaded to
// registers: the compiler cannot count such loads among direct ones and waits for all.
// Codes are converted where they are used: twice for the two halves of the rows, which
// costs less than bf16 through LDS.
//
// Measured, 4096 rows of 32 experts, SWIGLU of 2048, 4096 inputs: MXFP4 205 to 211 us, 650 to
// 670 TFLOP/s (some 90 row tiles, a third of them short; 16384 rows 574 us, 958 TFLOP/s; a large
// bf16 product 1170 to 1410); integer codes in groups of 128 315 us, of 32 501, fp32 x 549.  Bound by
// the conversion of the codes, which leaves the matrix units waiting, then by the short tiles.
#include "q4_dev.h"

namespace moe {

namespace {

using namespace q4;

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(1))) void* gptr_t;
typedef __attribute__((address_space(3))) void* lptr_t;

// When the products of a stage's inputs are scaled.
enum {
  kFold = 0,   // E2M1 codes, E8M0 scales a chunk of 32: in the convert, which is exact
  kFold2 = 1,  // the same where a stage's scales may lie in two words
  kChunk = 2,  // the sum of each 32 inputs
  kStage = 3   // the sum of the stage, which lies in one group
};

constexpr int kRows = 128;

// v_mfma_f32_32x32x16_bf16: lane l supplies row (x) or column (codes) l % 32 at inputs
// 8 (l / 32) on, and gets rows 8 (i / 4) + 4 (l / 32) + i % 4 of column l % 32.
__device__ __forceinline__ v16f mfma(v8bf a, v8bf b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

template <bool XF32, bool FP4, int MODE, int NT>
struct TileKernel {
  static constexpr int BK = XF32 ? 64 : 128;        // inputs a stage
  static constexpr int kCols = 128 * NT;            // rows of the matrix
  static constexpr int kXSlots = kRows * 16;        // 16-byte slots of a stage
  static constexpr int kPer = BK / 32;              // slots of codes a row
  static constexpr int kWSlots = kCols * kPer;
  static constexpr int kWLoads = (kWSlots / 64 + 7) / 8;  // loads a wavefront
  static constexpr bool kFolded = MODE == kFold || MODE == kFold2;
  // words of scales and of zero points that a row's stage takes
  static constexpr int kSWords = MODE == kFold2 ? 2 : MODE == kChunk ? kPer : 1;
  static constexpr int kWords = kSWords + (FP4 ? 0 : kSWords);
  static constexpr int kLoads = 4 + kWLoads + kWords;
  static constexpr int kRing = MODE == kChunk ? 2 : 3;  // stages; LDS holds no third with words a chunk
  struct Smem {
    u32x4_t x[kRing][kXSlots];
    u32x4_t w[kRing][kWSlots];
    uint32_t s[kRing][8][kWords][64];  // a wavefront's own, a row of the matrix a lane
  };
  // The matrix row of this workgroup's row r (of either half of a SWIGLU matrix).
  static __device__ __forceinline__ int out_of(const Q4Args& a, int r) {
    return a.swiglu ? blockIdx.x * 128 + (r >> 6) * 32 + (r & 31) : blockIdx.x * kCols + r;
  }
  static __device__ __forceinline__ int row_of(const Q4Args& a, int r) {
    return min(out_of(a, r), a.N - 1) + (a.swiglu && (r & 32) ? a.N : 0);
  }

  static __device__ __forceinline__ void run(const Q4Args& a, const Tile& tile, Smem& sm) {
    const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave & 1, wn = wave >> 1;
    constexpr int xs = XF32 ? 4 : 2;
    const uint8_t* codes = a.codes + tile.e * a.code_stride;
    const uint8_t* scales = (const uint8_t*)a.scales + tile.e * a.scale_stride;
    const uint8_t* zeros = a.zeros ? a.zeros + tile.e * a.zero_stride : nullptr;
    const uint8_t* x0 = (const uint8_t*)a.x + (size_t)tile.row * a.K * xs;
    const int st = kFolded ? (int)MOE_SCALE_E8M0 : a.st;
    const int size = st == MOE_F32 ? 4 : st == MOE_BF16 ? 2 : 1;  // of a scale
    const int whole = a.K / BK, stages = (a.K + BK - 1) / BK;

    // Slot 16 r + p holds piece p ^ (r % 16) of x's row r, slot 4 r + p (2 r + p) piece
    // p ^ (r / 4 % 4) (p) of the matrix's: the rows that an instruction reads lie on
    // distinct banks.
    uint32_t xat[4], wat[kWLoads];  // this lane's pieces of stage 0
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 4 * j + (lane >> 4);  // of the wavefront's 16
      xat[j] = (uint32_t)min(16 * wave + r, tile.rows - 1) * (a.K * xs) + 16 * ((lane & 15) ^ r);
    }
#pragma unroll
    for (int j = 0; j < kWLoads; ++j) {
      const int slot = ((wave * kWLoads + j) * 64 + lane) % kWSlots, r = slot / kPer;
      wat[j] = (uint32_t)row_of(a, r) * (uint32_t)(a.K / 2) + 16 * (kPer == 4 ? (slot & 3) ^ ((r >> 2) & 3) : slot & 1);
    }
    auto issue = [&](int stage, int buf) {
      const uint8_t *xp = x0 + stage * 256, *wp = codes + stage * (BK / 2);
      uint32_t xo[4], wo[kWLoads];
#pragma unroll
      for (int j = 0; j < 4; ++j) xo[j] = xat[j];
#pragma unroll
      for (int j = 0; j < kWLoads; ++j) wo[j] = wat[j];
      if (stage >= whole) {  // pieces past the rows' ends: others of the row in their place, which nothing reads
        const int over = min(stage, stages - 1) * 256, xpieces = a.K * xs - over, wpieces = xpieces / xs / 2;
        xp = x0 + over, wp = codes + over / xs / 2;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = 16 * ((lane & 15) ^ (4 * j + (lane >> 4)));
          xo[j] -= at - min(at, xpieces - 16);
        }
#pragma unroll
        for (int j = 0; j < kWLoads; ++j) {
          const int slot = ((wave * kWLoads + j) * 64 + lane) % kWSlots, r = slot / kPer;
          const int at = 16 * (kPer == 4 ? (slot & 3) ^ ((r >> 2) & 3) : slot & 1);
          wo[j] -= at - min(at, wpieces - 16);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        __builtin_amdgcn_global_load_lds((gptr_t)(xp + xo[j]), (lptr_t)(&sm.x[buf][(wave * 4 + j) * 64]), 16, 0, 0);
#pragma unroll
      for (int j = 0; j < kWLoads; ++j)
        __builtin_amdgcn_global_load_lds((gptr_t)(wp + wo[j]),
                                         (lptr_t)(&sm.w[buf][(wave * kWLoads + j) * 64 % kWSlots]), 16, 0, 0);
    };
    // Scales lie at any alignment of theirs, but each within an aligned word: that word is
    // loaded, and the bytes are picked when it is used.
    const uint32_t sfrom = (uint32_t)((uintptr_t)scales & 3), zfrom = (uint32_t)((uintptr_t)zeros & 3);
    const uint8_t *swords = scales - sfrom, *zwords = zeros ? zeros - zfrom : swords;
    const int last = a.K / 32 - 1;
    const uint32_t srow = (uint32_t)row_of(a, wn * 32 * NT + (NT == 2 ? lane : c)) * (uint32_t)a.groups;
    uint32_t crow[NT];  // of the rows whose codes the lane converts
#pragma unroll
    for (int i = 0; i < NT; ++i) crow[i] = (uint32_t)row_of(a, wn * 32 * NT + 32 * i + c) * (uint32_t)a.groups;
    auto issue_scales = [&](int stage, int buf) {
      const int c0 = min(stage, stages - 1) * kPer;
      auto one = [&](const uint8_t* base, uint32_t at, int word) {
        __builtin_amdgcn_global_load_lds((gptr_t)(base + (at & ~3u)), (lptr_t)(&sm.s[buf][wave][word][0]), 4, 0, 0);
      };
#pragma unroll
      for (int u = 0; u < kSWords; ++u) {
        if constexpr (kFolded) {
          const uint32_t end = (uint32_t)((a.swiglu ? 2 * a.N : a.N) * a.groups - 1);  // the matrix's last scale
          one(swords, sfrom + (u ? min(srow + c0 + 4 * u, end) : srow + c0), u);
        } else {
          const uint32_t at = srow + group_of(a, min(c0 + u, last));
          one(swords, sfrom + at * size, u);
          if constexpr (!FP4) one(zwords, zfrom + (zeros ? at : 0), kSWords + u);
        }
      }
    };
    // the scale and the zero point of block i's row for chunk u (of the stage in buf)
    auto scale_at = [&](int stage, int buf, int i, int u) {
      const uint32_t at = sfrom + (crow[i] + group_of(a, min(stage * kPer + u, last))) * size;
      const uint32_t v = sm.s[buf][wave][u][32 * i + c] >> (8 * (at & 3));
      return st == MOE_F32 ? __uint_as_float(v) : st == MOE_BF16 ? __uint_as_float(v << 16) : e8m0_to_f32(v & 255);
    };
    auto zero_at = [&](int stage, int buf, int i, int u) {
      if (FP4 || !zeros) return FP4 ? 0.f : 8.f;
      const uint32_t at = zfrom + crow[i] + group_of(a, min(stage * kPer + u, last));
      return (float)((sm.s[buf][wave][kSWords + u][32 * i + c] >> (8 * (at & 3))) & 255);
    };
    // all of a stage's bytes of block i's row, for folding
    auto bytes_at = [&](int stage, int buf, int i) {
      const uint32_t at = (sfrom + crow[i] + stage * kPer) & 3, lo = sm.s[buf][wave][0][32 * i + c];
      if constexpr (MODE == kFold2)
        return __builtin_amdgcn_alignbyte(sm.s[buf][wave][kSWords - 1][32 * i + c], lo, at);
      else
        return lo >> (8 * at);
    };
    // Places in a stage's slots: of x, its row of block wm (the other block's 64 rows on)
    // and instruction; of the matrix, its row of block 0 and half of the stage.
    uint32_t xslot[BK / 16][XF32 ? 2 : 1], wslot[BK / 64];
#pragma unroll
    for (int u = 0; u < BK / 64; ++u) {
      const int r = wn * 32 * NT + c;
      wslot[u] = r * kPer + (kPer == 4 ? (2 * u + h) ^ ((r >> 2) & 3) : h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 32 * wm + c, sw = r & 15;
        if constexpr (XF32) {
          const int at = 8 * h + 2 * j;
          xslot[j][0] = r * 16 + (at ^ sw);
          xslot[j][1] = r * 16 + ((at + 1) ^ sw);
        } else {
          xslot[4 * u + j][0] = r * 16 + ((8 * u + 4 * h + j) ^ sw);
        }
      }
    }

    const int live = (tile.rows + 31) / 32;
    const int blocks = wm < live ? (wm + 2 < live ? 2 : 1) : 0;  // of this wavefront: wm and wm + 2
    v16f acc[2][NT];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[m][i][r] = 0.f;

    // What half u of a stage reads from LDS: the blocks' codes, and of block wm + 2 m of x
    // the inputs of instruction j.
    struct Half {
      u32x4_t q[NT], x[4][2][XF32 ? 2 : 1];
    };
    auto read_half = [&](auto nm, Half& f, int buf, int u) {
#pragma unroll
      for (int i = 0; i < NT; ++i) f.q[i] = sm.w[buf][wslot[u] + i * 32 * kPer];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int m = 0; m < decltype(nm)::value; ++m)
#pragma unroll
          for (int p = 0; p < (XF32 ? 2 : 1); ++p) f.x[j][m][p] = sm.x[buf][m * 64 * 16 + xslot[4 * u + j][p]];
    };
    auto x_of = [](const u32x4_t(&v)[XF32 ? 2 : 1]) {
      XPart<XF32> x;
      const u32x4_t lo = v[0];
      if constexpr (XF32) {
        const u32x4_t hi = v[1];
        x.split(f32x8{__uint_as_float(lo.x), __uint_as_float(lo.y), __uint_as_float(lo.z), __uint_as_float(lo.w),
                      __uint_as_float(hi.x), __uint_as_float(hi.y), __uint_as_float(hi.z), __uint_as_float(hi.w)});
      } else {
        x.p[0] = as_bf(lo);
      }
      return x;
    };

    // chunks: of 32 inputs, that the stage holds (four and more if it is whole)
    auto multiply = [&](auto nm, auto whole, int stage, int buf, int chunks) {
      constexpr int NM = decltype(nm)::value;
      constexpr bool kWhole = decltype(whole)::value;
      uint32_t bytes[NT];
      if constexpr (kFolded) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          bytes[i] = bytes_at(stage, buf, i);
          // The bytes past the row's end are another row's, or nobody's: as 255, 254 or 253 they
          // would make weights that x of 0 does not take away.
          if (!kWhole) bytes[i] &= (1u << (8 * chunks)) - 1;
          bytes[i] >>= 8 * h;
        }
      }
      v16f part[NM][NT];  // of the stage
      if constexpr (MODE == kStage) {
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) part[m][i][r] = 0.f;
      }
      // Everything is requested before the first product, or it would wait for its LDS read
      // each time.
      Half f[BK / 64];
#pragma unroll
      for (int u = 0; u < BK / 64; ++u) read_half(nm, f[u], buf, u);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < BK / 64; ++u) {
        if (!kWhole && 2 * u >= chunks) break;
        float s[NT], z[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if constexpr (kFolded)  // the convert takes the exponent field as the E8M0 byte
            s[i] = __uint_as_float((bytes[i] >> (16 * u) << 23) & 0x7f800000u);
          else
            z[i] = zero_at(stage, buf, i, 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v8bf w[NT];
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            if constexpr (kFolded)
              w[i] = fp4_to_bf16_scaled(f[u].q[i][j], s[i]);
            else
              w[i] = codes_to_bf16<FP4>(f[u].q[i][j], z[i]);
          }
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            XPart<XF32> x = x_of(f[u].x[j][m]);
            if (!kWhole && 2 * u + 1 >= chunks && h) {
#pragma unroll
              for (int p = 0; p < XPart<XF32>::kParts; ++p) x.p[p] = as_bf(u32x4_t{0, 0, 0, 0});
            }
#pragma unroll
            for (int p = XPart<XF32>::kParts - 1; p >= 0; --p)
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                if constexpr (kFolded)
                  acc[m][i] = mfma(x.p[p], w[i], acc[m][i]);
                else
                  part[m][i] = mfma(x.p[p], w[i], part[m][i]);
              }
          }
        }
      }
      if constexpr (MODE == kStage) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float s = scale_at(stage, buf, i, 0);
#pragma unroll
          for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[m][i][r] = fmaf(s, part[m][i][r], acc[m][i][r]);
        }
      }
    };

    // The same a chunk at a time, each scaled by itself.  Chunks that the compiler mixes need
    // more registers than there are: a loop.
    auto multiply_chunks = [&](auto nm, int stage, int buf, int chunks) {
#pragma unroll 1
      for (int g = 0; g < chunks; ++g) {
        u32x4_t xv[2][2][XF32 ? 2 : 1];
        uint32_t d[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {  // this half's codes of the chunk's two instructions: 16 j + 8 h on
          const int r = wn * 32 * NT + 32 * i + c;
          const uint32_t* q = (const uint32_t*)&sm.w[buf][r * kPer + (kPer == 4 ? g ^ ((r >> 2) & 3) : g)];
          d[i][0] = q[h], d[i][1] = q[2 + h];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int m = 0; m < decltype(nm)::value; ++m)
#pragma unroll
            for (int p = 0; p < (XF32 ? 2 : 1); ++p) {
              const int r = 32 * (wm + 2 * m) + c, at = XF32 ? 8 * g + 4 * j + 2 * h + p : 4 * g + 2 * j + h;
              xv[j][m][p] = sm.x[buf][r * 16 + (at ^ (r & 15))];
            }
        float s[NT];
        v8bf w[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          s[i] = scale_at(stage, buf, i, g);
          const float z = zero_at(stage, buf, i, g);
#pragma unroll
          for (int j = 0; j < 2; ++j) w[i][j] = codes_to_bf16<FP4>(d[i][j], z);
        }
#pragma unroll
        for (int m = 0; m < decltype(nm)::value; ++m) {
          v16f sum[NT];
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) sum[i][r] = 0.f;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const XPart<XF32> x = x_of(xv[j][m]);
#pragma unroll
            for (int p = XPart<XF32>::kParts - 1; p >= 0; --p)
#pragma unroll
              for (int i = 0; i < NT; ++i) sum[i] = mfma(x.p[p], w[i][j], sum[i]);
          }
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[m][i][r] = fmaf(s[i], sum[i][r], acc[m][i][r]);
        }
      }
    };
    auto issue_all = [&](int stage, int buf) {
      issue_scales(stage, buf);
      issue(stage, buf);
    };
#pragma unroll
    for (int p = 0; p < kRing - 1; ++p) issue_all(p, p);
    auto go = [&](auto nm) {
      int buf = 0;
      auto stage = [&](auto all, int s) {
        // This wavefront's loads of stage s are done when no more than those of the later
        // ones are under way; the barrier says so of everyone's, and that everyone is
        // done with stage s - 1, whose slots the next one to load takes.  A bare barrier: a
        // fenced one would wait for every load.
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLoads * (kRing - 2)) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        issue_all(s + kRing - 1, buf == 0 ? kRing - 1 : buf - 1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (decltype(nm)::value > 0) {
          if constexpr (MODE == kChunk)
            multiply_chunks(nm, s, buf, min(a.K / 32 - s * kPer, kPer));
          else
            multiply(nm, all, s, buf, a.K / 32 - s * kPer);
        }
        buf = buf == kRing - 1 ? 0 : buf + 1;
      };
      // Rows end inside a stage in two forms: kChunk counts its chunks, and kFold2 takes the last
      // stage by itself.  Built for kStage too, which has none, that stage made registers spill.
      for (int s = 0; s < (MODE == kFold2 ? whole : stages); ++s) stage(std::true_type{}, s);
      if constexpr (MODE == kFold2) {
        if (whole < stages) stage(std::false_type{}, whole);
      }
    };
    if (blocks == 2)
      go(std::integral_constant<int, 2>{});
    else if (blocks == 1)
      go(std::integral_constant<int, 1>{});
    else
      go(std::integral_constant<int, 0>{});
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing writes to LDS after the workgroup's end

#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (i == 1 && a.swiglu) continue;
        const int out = out_of(a, wn * 32 * NT + 32 * i + c);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int row = 32 * (wm + 2 * m) + 8 * (r / 4) + 4 * h + r % 4;
          float v = acc[m][i][r];
          if (NT == 2 && a.swiglu) v *= gate_sigmoid(v) * acc[m][NT - 1][r];
          if (row < tile.rows && out < a.N) {
            const size_t to = (size_t)(tile.row + row) * a.N + out;
            if (a.ybf)
              ((uint16_t*)a.y)[to] = bf16_of(v);
            else
              ((float*)a.y)[to] = v;
          }
        }
      }
  }
};

template <bool XF32, bool FP4, int MODE, int NT>
__global__ __launch_bounds__(512) void q4_tile_kernel(Q4Args a) {
  typedef TileKernel<XF32, FP4, MODE, NT> Kernel;
  __shared__ typename Kernel::Smem sm;
  Tile tile;
  if (!find_tile<true>(a, blockIdx.z * kTilesY + blockIdx.y, kRows, tile)) return;
  Kernel::run(a, tile, sm);
}

template <bool XF32, bool FP4, int MODE, int NT>
void run(const Q4Args& a, hipStream_t s) {
  const int cols = a.swiglu ? 128 : 128 * NT;
  const int tiles = tile_groups(a, kRows);
  const dim3 grid((a.N + cols - 1) / cols, min(tiles, kTilesY), (tiles + kTilesY - 1) / kTilesY);
  launch(MOE_PROF_Q4, q4_tile_kernel<XF32, FP4, MODE, NT>, grid, dim3(512), 0, s, a);
}

template <bool XF32, bool FP4, int MODE>
void run_shape(const Q4Args& a, hipStream_t s) {
  // A workgroup of 256 matrix rows takes 1.65 times one of 128 (4096 inputs, integer codes 89
  // and 53 us, MXFP4 50 and 33), so that the smaller one wins where it fills turns of the
  // chip that the larger would not: 1024 rows by 4096 MXFP4 37 us against 53; 2048 rows of
  // integer codes are one turn of the larger, 95 us, or two of the smaller.  SWIGLU has 32 gate
  // and 32 up rows in a wavefront and takes the larger.
  const long tiles = tile_groups(a, kRows), w1 = tiles * ((a.N + 127) / 128), w2 = tiles * ((a.N + 255) / 256);
  if (a.swiglu || 1.65 * ((w2 + 255) / 256) < (double)((w1 + 255) / 256))
    run<XF32, FP4, MODE, 2>(a, s);
  else
    run<XF32, FP4, MODE, 1>(a, s);
}

template <bool XF32, bool FP4>
void run_types(const Q4Args& a, hipStream_t s) {
  if constexpr (FP4) {
    if (a.st == MOE_SCALE_E8M0 && a.group == 32) {
      // a stage's scales, two or four, lie in one word, or (four that start anywhere) in two
      const int at = (int)(((uintptr_t)a.scales | (a.num > 1 ? a.scale_stride : 0) | (uintptr_t)a.groups) & 3);
      if (at == 0 || (XF32 && at == 2)) {
        run_shape<XF32, FP4, kFold>(a, s);
        return;
      }
      if constexpr (!XF32) {
        run_shape<XF32, FP4, kFold2>(a, s);
        return;
      }
    }
  }
  if (a.group % (XF32 ? 64 : 128) == 0)
    run_shape<XF32, FP4, kStage>(a, s);
  else
    run_shape<XF32, FP4, kChunk>(a, s);
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
