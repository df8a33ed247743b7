// Chunks of eight consecutive bf16 or fp32 elements at any element-aligned
// address: one or two 16-byte accesses where all eight are there (the hardware
// takes global accesses at any alignment), single elements at the end of a row.
// Shared by the norms, the adapters and the routing by groups.
#pragma once

#include "common.h"

namespace moe {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

struct __attribute__((packed, aligned(2))) Packed8h {
  uint32_t x, y, z, w;
};
struct __attribute__((packed, aligned(2))) Packed4h {
  uint32_t x, y;
};
struct __attribute__((packed, aligned(4))) Packed4f {
  float x, y, z, w;
};

__device__ __forceinline__ uint4 ld8h(const uint16_t* p) {
  const Packed8h v = *(const Packed8h*)p;
  return make_uint4(v.x, v.y, v.z, v.w);
}

__device__ __forceinline__ void st8h(uint16_t* p, uint4 v) { *(Packed8h*)p = Packed8h{v.x, v.y, v.z, v.w}; }

// the first n of eight bf16 elements, the others zero
__device__ __forceinline__ uint32_t ld2h_part(const uint16_t* p, int n) {
  const uint32_t lo = n > 0 ? p[0] : 0, hi = n > 1 ? p[1] : 0;
  return lo | (hi << 16);
}

__device__ __forceinline__ uint4 ld8h_part(const uint16_t* p, int n) {
  return make_uint4(ld2h_part(p, n), ld2h_part(p + 2, n - 2), ld2h_part(p + 4, n - 4), ld2h_part(p + 6, n - 6));
}

__device__ __forceinline__ uint4 ld8h_to(const uint16_t* p, int n) { return n >= 8 ? ld8h(p) : ld8h_part(p, n); }

__device__ __forceinline__ f32x8 ld8f(const float* p) {
  const Packed4f a = *(const Packed4f*)p, b = *(const Packed4f*)(p + 4);
  return f32x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

__device__ __forceinline__ uint4 ld4w(const uint32_t* p) {
  const Packed4f v = *(const Packed4f*)p;
  return make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w));
}

__device__ __forceinline__ float ld1f_if(const float* p, bool there) { return there ? *p : 0.0f; }

__device__ __forceinline__ f32x8 ld8f_to(const float* p, int n) {
  if (n >= 8) return ld8f(p);
  return f32x8{ld1f_if(p, n > 0),     ld1f_if(p + 1, n > 1), ld1f_if(p + 2, n > 2), ld1f_if(p + 3, n > 3),
               ld1f_if(p + 4, n > 4), ld1f_if(p + 5, n > 5), ld1f_if(p + 6, n > 6), 0.0f};
}

__device__ __forceinline__ f32x8 widen(uint4 h) {
  return f32x8{bf16_lo(h.x), bf16_hi(h.x), bf16_lo(h.y), bf16_hi(h.y),
               bf16_lo(h.z), bf16_hi(h.z), bf16_lo(h.w), bf16_hi(h.w)};
}

// sum of the lanes up to this one
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, dpp::kRowBcast15, 0xa, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, dpp::kRowBcast31, 0xc, 0xf, false);
  return v;
}

// fp32 -> bf16, to nearest even, NaN stays NaN: one instruction for two.  With
// the rounding in integer steps the norms, though bound by memory, took 13.3
// instead of 12.2 us and 28.9 instead of 27.4 (4096 x 4096).
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

__device__ __forceinline__ uint16_t bf16_of(float f) { return (uint16_t)pack2(f, 0.0f); }

// Stores of results that this kernel does not read again: they leave the L2 as
// they come instead of at the kernel's end, when all dirty lines are written back.
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void stream4h(uint16_t* p, uint2 v) {
  __builtin_nontemporal_store(u32x2_any{v.x, v.y}, (u32x2_any*)p);
}

__device__ __forceinline__ void stream8h(uint16_t* p, uint4 v) {
  __builtin_nontemporal_store(u32x4_any{v.x, v.y, v.z, v.w}, (u32x4_any*)p);
}

__device__ __forceinline__ void stream4f(float* p, f32x4 v) {
  __builtin_nontemporal_store(f32x4_any{v[0], v[1], v[2], v[3]}, (f32x4_any*)p);
}

template <bool BF16>
__device__ __forceinline__ f32x8 load8(const void* p, size_t at, int n) {
  if constexpr (BF16)
    return widen(ld8h_to((const uint16_t*)p + at, n));
  else
    return ld8f_to((const float*)p + at, n);
}

template <bool BF16, bool STREAM = false>
__device__ __forceinline__ void store8(void* p, size_t at, int n, f32x8 v) {
  if constexpr (BF16) {
    uint16_t* o = (uint16_t*)p + at;
    if (n >= 8) {
      const uint4 h = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
      if constexpr (STREAM)
        stream8h(o, h);
      else
        st8h(o, h);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) o[e] = bf16_of(v[e]);
    }
  } else {
    float* o = (float*)p + at;
    if (n >= 8) {
      if constexpr (STREAM) {
        stream4f(o, f32x4{v[0], v[1], v[2], v[3]});
        stream4f(o + 4, f32x4{v[4], v[5], v[6], v[7]});
      } else {
        *(Packed4f*)o = Packed4f{v[0], v[1], v[2], v[3]};
        *(Packed4f*)(o + 4) = Packed4f{v[4], v[5], v[6], v[7]};
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) o[e] = v[e];
    }
  }
}

// A chunk whose type is known at run time only (the same for the whole launch):
// as it was loaded, and widened.
__device__ __forceinline__ f32x8 load8_raw(const void* p, bool bf16, size_t at, int n) {
  if (!bf16) return ld8f_to((const float*)p + at, n);
  const uint4 h = ld8h_to((const uint16_t*)p + at, n);
  return f32x8{__uint_as_float(h.x), __uint_as_float(h.y), __uint_as_float(h.z), __uint_as_float(h.w), 0, 0, 0, 0};
}

__device__ __forceinline__ f32x8 widen_raw(f32x8 v, bool bf16) {
  if (!bf16) return v;
  return widen(make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
}

__device__ __forceinline__ float load1(const void* p, bool bf16, size_t at) {
  return bf16 ? bf(((const uint16_t*)p)[at]) : ((const float*)p)[at];
}

constexpr float kLowestLogit = -0x1.fep127f;  // bf16's lowest value: a logit there or below masks its expert

// 1 / (1 + e^-g): the hardware's exponential of 2 and reciprocal, each within a
// step of fp32, the argument's rounding growing with |g|
__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// 1 / (1 + e^-g) within 8 roundings (2^-24) of its value wherever g lies, 0 where that is
// below 2^-126.  e^-g is 2^t, t = -g log2(e); what rounding took from t comes back as a
// factor 1 + rest ln(2), or the error would grow with |g|, to some |g| roundings.  From
// 2^128 on the power is infinite and takes no factor: infinity times a rest of 0, or with
// one below 0 added to itself, is NaN.  The hardware's power of 2 and reciprocal are each
// within a step.  moe_norm_out, 4096 x 4096 bf16, a gate per element 32.0 -> 32.8 us; with
// the library's expf 33.4.
__device__ __forceinline__ float gate_sigmoid(float g) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eRest = 1.925963e-8f, kLn2 = 0.6931472f;  // log2(e) in two parts
  const float t = -kLog2e * g, p = __builtin_amdgcn_exp2f(t);
  const float rest = fmaf(-kLog2eRest, g, fmaf(-kLog2e, g, -t));
  const float e = fabsf(t) < 128.0f ? fmaf(p, rest * kLn2, p) : p;  // beyond, 1 + e is 1 or infinite, or g is NaN
  return __builtin_amdgcn_rcpf(1.0f + e);
}

// what a wavefront's lanes wrote to its LDS may now be read by its other lanes
__device__ __forceinline__ void wave_turn() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace moe
