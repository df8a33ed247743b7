// Low-rank adapters of many requests beside a shared projection
// (moe_lora_add): out[t] = base[t] + scale * B (A x[t]) with the adapter of
// the token's request.
//
// One workgroup per token: A x into LDS, one wavefront per row of A, then a
// thread per output.
#include "common.h"

namespace moe {

namespace {

constexpr int kMaxRank = 128;

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

template <bool XBF16, bool YBF16>
__global__ __launch_bounds__(256) void lora_kernel(moe_lora L, const void* __restrict__ x,
                                                   const int32_t* __restrict__ ids, const void* base, void* out) {
  __shared__ float v[kMaxRank];
  const int t = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int id = ids[t];
  const bool has = id >= 0 && id < L.num;
  const int rank = has ? (L.ranks ? max(0, min(L.ranks[id], L.r)) : L.r) : 0;
  const uint16_t* A = (const uint16_t*)L.a + (has ? (size_t)id * L.r * L.K : 0);
  const uint16_t* B = (const uint16_t*)L.b + (has ? (size_t)id * L.N * L.r : 0);
  for (int j = wave; j < rank; j += 4) {
    float acc = 0.f;
    for (int i = lane; i < L.K; i += 64) {
      const size_t at = (size_t)t * L.K + i;
      acc = fmaf(XBF16 ? bf(((const uint16_t*)x)[at]) : ((const float*)x)[at], bf(A[(size_t)j * L.K + i]), acc);
    }
    acc = wave_sum(acc);
    if (lane == 0) v[j] = L.scale ? acc * L.scale[id] : acc;
  }
  __syncthreads();
  for (int n = threadIdx.x; n < L.N; n += 256) {
    const size_t at = (size_t)t * L.N + n;
    float acc = 0.f;
    for (int j = 0; j < rank; ++j) acc = fmaf(v[j], bf(B[(size_t)n * L.r + j]), acc);
    if (base) acc += YBF16 ? bf(((const uint16_t*)base)[at]) : ((const float*)base)[at];
    if (YBF16)
      ((uint16_t*)out)[at] = f32_to_bf16(acc);
    else
      ((float*)out)[at] = acc;
  }
}

}  // namespace

moe_status launch_lora(const moe_lora* L, const void* x, moe_dtype xt, int T, const int32_t* ids, const void* base,
                       void* out, moe_dtype yt, hipStream_t s) {
  const dim3 grid(T), block(256);
  const bool xb = xt == MOE_BF16, yb = yt == MOE_BF16;
  if (xb && yb)
    launch(MOE_PROF_LORA, lora_kernel<true, true>, grid, block, 0, s, *L, x, ids, base, out);
  else if (xb)
    launch(MOE_PROF_LORA, lora_kernel<true, false>, grid, block, 0, s, *L, x, ids, base, out);
  else if (yb)
    launch(MOE_PROF_LORA, lora_kernel<false, true>, grid, block, 0, s, *L, x, ids, base, out);
  else
    launch(MOE_PROF_LORA, lora_kernel<false, false>, grid, block, 0, s, *L, x, ids, base, out);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
