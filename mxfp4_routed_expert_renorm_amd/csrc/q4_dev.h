// What the kernels of the products with 4-bit weights share: their arguments, the
// codes' and inputs' ways to bf16, and the search for a row tile's matrix.
#pragma once

#include <algorithm>
#include <type_traits>

#include "chunk_dev.h"

namespace moe {

namespace q4 {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kTilesY = 32768;  // row tiles along a grid's second dimension

struct Q4Args {
  const void* x;
  const uint8_t *codes, *zeros;
  const void* scales;
  void* y;
  const int32_t* offsets;  // NULL: one matrix
  int T, K, N, num, group, groups, st;
  bool swiglu, ybf;
  size_t code_stride, scale_stride, zero_stride;
  uint32_t magic;  // 2^32 / (group / 32), rounded up, less 2^32 where that is its size
  int unit;        // 1: groups of 32, else 0
};

__device__ __forceinline__ v8bf as_bf(u32x4_t v) { return __builtin_bit_cast(v8bf, v); }

// A lane's eight codes of one dword as bf16, in order.
template <bool FP4>
__device__ __forceinline__ v8bf codes_to_bf16(uint32_t d, float zero) {
  if constexpr (FP4) {
    return as_bf(u32x4_t{fp4x2_to_bf16x2<0>(d), fp4x2_to_bf16x2<1>(d), fp4x2_to_bf16x2<2>(d), fp4x2_to_bf16x2<3>(d)});
  } else {
    // A byte 0..15 read as FP8 E4M3 is that many times 2^-9 (subnormals, then the first
    // binade): one convert gives two integers.
    const uint32_t even = d & 0x0f0f0f0fu, odd = (d >> 4) & 0x0f0f0f0fu;
    const v2f e0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(even, 512.f, false);
    const v2f o0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(odd, 512.f, false);
    const v2f e1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(even, 512.f, true);
    const v2f o1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(odd, 512.f, true);
    return as_bf(u32x4_t{pack2(e0[0] - zero, o0[0] - zero), pack2(e0[1] - zero, o0[1] - zero),
                         pack2(e1[0] - zero, o1[0] - zero), pack2(e1[1] - zero, o1[1] - zero)});
  }
}

// Integer codes 0..15 as they are: the same convert straight to bf16
__device__ __forceinline__ v8bf int4_to_bf16(uint32_t d) {
  const uint32_t even = d & 0x0f0f0f0fu, odd = (d >> 4) & 0x0f0f0f0fu;
  const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400), hi = __builtin_amdgcn_perm(odd, even, 0x07030602);
  auto two = [](uint32_t v, auto word) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.f, decltype(word)::value));
  };
  return as_bf(u32x4_t{two(lo, std::false_type{}), two(lo, std::true_type{}), two(hi, std::false_type{}),
                       two(hi, std::true_type{})});
}

// E2M1 codes with their block's power of two: exact
__device__ __forceinline__ v8bf fp4_to_bf16_scaled(uint32_t d, float scale) {
  return as_bf(u32x4_t{fp4x2_to_bf16x2_scaled<0>(d, scale), fp4x2_to_bf16x2_scaled<1>(d, scale),
                       fp4x2_to_bf16x2_scaled<2>(d, scale), fp4x2_to_bf16x2_scaled<3>(d, scale)});
}

// Eight consecutive elements of x as one or three bf16 parts.  fp32 by truncation:
// each part takes eight bits and what is left over is exact.
template <bool XF32>
struct XPart {
  static constexpr int kParts = XF32 ? 3 : 1;
  v8bf p[kParts];
  __device__ __forceinline__ void split(f32x8 f) {
    if constexpr (XF32) {
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        u32x4_t r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo = __float_as_uint(f[2 * i]), hi = __float_as_uint(f[2 * i + 1]);
          r[i] = __builtin_amdgcn_perm(hi, lo, 0x07060302);
          f[2 * i] -= __uint_as_float(lo & 0xffff0000u);
          f[2 * i + 1] -= __uint_as_float(hi & 0xffff0000u);
        }
        p[part] = as_bf(r);
      }
    }
  }
};

__device__ __forceinline__ float scale_of(uint32_t raw, int st) {
  return st == MOE_F32 ? __uint_as_float(raw) : st == MOE_BF16 ? __uint_as_float(raw << 16) : e8m0_to_f32(raw);
}

// The group of the inputs from 32 c on.
__device__ __forceinline__ int group_of(const Q4Args& a, int c) {
  return (int)__umulhi((uint32_t)c, a.magic) + c * a.unit;
}

// The matrix and the rows of the row tile that a workgroup takes, of `size` rows each but
// for a matrix's last.  False: there is none.
struct Tile {
  int e, row, rows;
};

// Row tiles of a launch: a matrix's last may be short, one at most for each that has rows.
inline int tile_groups(const Q4Args& a, int size) {
  return a.offsets ? a.T / size + std::min(a.num, a.T) : (a.T + size - 1) / size;
}

// LARGE: tiles of more than half the size come first, so that the chip does not end on
// them alone.
template <bool LARGE>
__device__ __forceinline__ bool find_tile(const Q4Args& a, int tile, int size, Tile& o) {
  if (!a.offsets) {
    o = {0, tile * size, min(size, a.T - tile * size)};
    return o.rows > 0;
  }
  const int lane = threadIdx.x & 63;
  int before = 0;  // tiles so far
#pragma unroll
  for (int pass = 0; pass < (LARGE ? 2 : 1); ++pass) {
    for (int e0 = 0; e0 < a.num; e0 += 64) {
      const int e = e0 + lane, from = a.offsets[min(e, a.num)], to = a.offsets[min(e + 1, a.num)];
      const int lo = min(max(from, 0), a.T), hi = min(max(to, lo), a.T);  // past the last: no rows
      const int all = (hi - lo + size - 1) / size, first = LARGE ? (hi - lo + size / 2 - 1) / size : all;
      const int mine = pass ? all - first : first, incl = wave_scan(mine), start = before + incl - mine;
      const uint64_t hit = __ballot(tile >= start && tile < start + mine);
      if (hit) {
        const int l = __ffsll((unsigned long long)hit) - 1;
        const int in = tile - __builtin_amdgcn_readlane(start, l) + (pass ? __builtin_amdgcn_readlane(first, l) : 0);
        const int row = __builtin_amdgcn_readlane(lo, l) + in * size;
        o = {e0 + l, row, min(size, __builtin_amdgcn_readlane(hi, l) - row)};
        return true;
      }
      before = __builtin_amdgcn_readlane(before + incl, 63);
    }
  }
  return false;
}

}  // namespace q4

moe_status launch_q4_tile(const q4::Q4Args& a, bool xf32, bool fp4, hipStream_t s);

}  // namespace moe
