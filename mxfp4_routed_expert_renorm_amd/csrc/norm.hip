// RMS norms around a block: before it (moe_norm_in), and after it with the
// gate, the residual scale and the next block's norm in one pass
// (moe_norm_out).
//
//   r = residual + alpha * act(gate) * RMS(y; w_post),  next = RMS(r; w_pre)
//
// One workgroup owns one row, which it keeps in LDS as fp32 between the two
// sums, so every input is read once and out may overwrite an input.
#include "common.h"

namespace moe {

namespace {

__device__ __forceinline__ float ld(const void* p, bool bf16, size_t i) {
  return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}

__device__ __forceinline__ void st(void* p, bool bf16, size_t i, float v) {
  if (bf16)
    ((uint16_t*)p)[i] = f32_to_bf16(v);
  else
    ((float*)p)[i] = v;
}

struct NormArgs {
  const void *y, *residual, *gate, *post_w, *pre_w;
  void *out, *next_out;
  float eps, offset, alpha, next_eps, next_offset;
  int H, gate_kind;
  bool post, sigmoid, ybf, rbf, gbf, wbf, nwbf, nbf;
};

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0] + red[1] + red[2] + red[3];
  __syncthreads();
  return v;
}

__global__ __launch_bounds__(256) void norm_kernel(NormArgs a) {
  extern __shared__ float row[];
  __shared__ float red[4];
  const size_t at = (size_t)blockIdx.x * a.H;
  float ss = 0.f;
  for (int i = threadIdx.x; i < a.H; i += 256) {
    const float v = ld(a.y, a.ybf, at + i);
    row[i] = v;
    ss = fmaf(v, v, ss);
  }
  if (a.out) {
    const float rs = a.post ? 1.0f / sqrtf(block_sum(ss, red) / (float)a.H + a.eps) : 1.0f;
    ss = 0.f;
    for (int i = threadIdx.x; i < a.H; i += 256) {
      float z = row[i] * rs;
      if (a.post && a.post_w) z *= a.offset + ld(a.post_w, a.wbf, i);
      if (a.gate_kind != MOE_GATE_NONE) {
        float g = ld(a.gate, a.gbf,
                     a.gate_kind == MOE_GATE_CHANNEL ? (size_t)i
                     : a.gate_kind == MOE_GATE_TOKEN ? (size_t)blockIdx.x
                                                     : at + i);
        if (a.sigmoid) g = 1.0f / (1.0f + expf(-g));
        z *= g;
      }
      const float r = fmaf(a.alpha, z, ld(a.residual, a.rbf, at + i));
      row[i] = r;
      ss = fmaf(r, r, ss);
    }
    for (int i = threadIdx.x; i < a.H; i += 256) st(a.out, a.rbf, at + i, row[i]);
  }
  if (!a.next_out) return;
  const float rs = 1.0f / sqrtf(block_sum(ss, red) / (float)a.H + a.next_eps);
  for (int i = threadIdx.x; i < a.H; i += 256) {
    const float w = a.pre_w ? a.next_offset + ld(a.pre_w, a.nwbf, i) : 1.0f;
    st(a.next_out, a.nbf, at + i, row[i] * rs * w);
  }
}

moe_status run(const NormArgs& a, int T, hipStream_t s) {
  launch(MOE_PROF_NORM, norm_kernel, dim3(T), dim3(256), (size_t)a.H * 4, s, a);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

moe_status launch_norm_in(const moe_norm* n, const void* x, moe_dtype xt, int T, void* out, moe_dtype ot,
                          hipStream_t s) {
  NormArgs a{};
  a.y = x;
  a.ybf = xt == MOE_BF16;
  a.H = n->H;
  a.pre_w = n->pre_w;
  a.nwbf = n->wt == MOE_BF16;
  a.next_eps = n->eps;
  a.next_offset = n->weight_offset;
  a.next_out = out;
  a.nbf = ot == MOE_BF16;
  return run(a, T, s);
}

moe_status launch_norm_out(const moe_norm* n, const void* y, moe_dtype yt, const void* residual, const void* gate,
                           moe_dtype gt, int T, void* out, moe_dtype rt, const moe_norm* next, void* next_out,
                           moe_dtype nt, hipStream_t s) {
  NormArgs a{};
  a.y = y;
  a.ybf = yt == MOE_BF16;
  a.residual = residual;
  a.out = out;
  a.rbf = rt == MOE_BF16;
  a.H = n->H;
  a.eps = n->eps;
  a.offset = n->weight_offset;
  a.alpha = n->alpha;
  a.post = n->post_norm != 0;
  a.post_w = n->post_w;
  a.wbf = n->wt == MOE_BF16;
  a.gate = gate;
  a.gbf = gt == MOE_BF16;
  a.gate_kind = n->gate;
  a.sigmoid = n->gate_act == MOE_GATE_SIGMOID;
  if (next) {
    a.pre_w = next->pre_w;
    a.nwbf = next->wt == MOE_BF16;
    a.next_eps = next->eps;
    a.next_offset = next->weight_offset;
    a.next_out = next_out;
    a.nbf = nt == MOE_BF16;
  }
  return run(a, T, s);
}

}  // namespace moe
