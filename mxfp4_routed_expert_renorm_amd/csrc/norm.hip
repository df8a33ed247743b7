// RMS norms around a block: before it (moe_norm_in), and after it with the
// gate, the residual scale and the next block's norm in one pass
// (moe_norm_out).
//
//   r = residual + alpha * act(gate) * RMS(y; w_post),  next = RMS(r; w_pre)
//
// A row belongs to a group of 64 to 1024 threads of one workgroup and stays in
// their registers from its only read to its writes, so out may overwrite an
// input.  A thread holds V chunks of eight consecutive elements; everything a
// row needs (weights and gate too) is requested before the first sum is formed.
// Sums and everything between are fp32; each output is rounded once.
//
// Bound by memory: 4096 x 4096 bf16, norm_in 12.1 us (67 MB, 5.5 TB/s; a copy of
// as many bytes, which stays in the Infinity Cache from call to call, takes 10.6),
// norm_out with a channel gate and the next norm 24.3 us (134 MB, 5.5 TB/s; a copy
// 26.7).  Large results are stored streaming: with ordinary stores the lines
// left dirty in the L2s are written back at the kernel's end, 13.3 and 28.2 us.
// Rows of odd width pay for stores that share lines: 509 x 2047 6.3 us, 509 x 2048
// 4.5.  One row: 2.2 and 3.1 us, of which 1.9 are a launch.
#include "chunk_dev.h"

namespace moe {

namespace {

struct NormArgs {
  const void *y, *residual, *gate, *post_w, *pre_w;
  void *out, *next_out;
  float eps, offset, alpha, next_eps, next_offset, inv_h;
  int T, H, gate_kind, per_row;  // per_row: threads a row, a power of two >= 64
  bool post, sigmoid, gbf, wbf, nwbf;
};

// The sum over a row's threads, in all of them.  red: one float a wavefront.
__device__ __forceinline__ float row_sum(float v, int per_row, float* red) {
  v = wave_sum(v);
  if (per_row == 64) return v;
  const int wave = threadIdx.x >> 6, waves = per_row >> 6, first = wave & ~(waves - 1);
  if ((threadIdx.x & 63) == 0) red[wave] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < waves; ++i) v += red[first + i];
  return v;
}

// 1 / (1 + e^-g) within 8 roundings (2^-24) of its value wherever g lies.  e^-g is
// 2^t, t = -g log2(e); what rounding took from t comes back as a factor 1 + rest ln(2),
// or the error would grow with |g|, to some |g| roundings.  The hardware's power of 2
// and reciprocal are each within a step.  4096 x 4096 bf16, a gate per element 32.0 ->
// 32.8 us; with the library's expf 33.4.
__device__ __forceinline__ float gate_sigmoid(float g) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eRest = 1.925963e-8f, kLn2 = 0.6931472f;  // log2(e) in two parts
  const float t = -kLog2e * g, p = __builtin_amdgcn_exp2f(t);
  const float rest = fmaf(-kLog2eRest, g, fmaf(-kLog2e, g, -t));
  const float e = fabsf(t) < 150.0f ? fmaf(p, rest * kLn2, p) : p;  // beyond, 0 or infinity (and NaN) as they are
  return __builtin_amdgcn_rcpf(1.0f + e);
}

template <bool XBF16, bool OBF16, int V>
__global__ __launch_bounds__(1024) void norm_in_kernel(NormArgs a) {
  __shared__ float red[16];
  const int in_row = threadIdx.x & (a.per_row - 1);
  const int row = blockIdx.x * (blockDim.x / a.per_row) + threadIdx.x / a.per_row;
  const bool live = row < a.T;
  const size_t at = (size_t)min(row, a.T - 1) * a.H;
  f32x8 x[V], w[V];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = (i * a.per_row + in_row) * 8;
    x[i] = load8<XBF16>(a.y, at + e, a.H - e);
    w[i] = a.pre_w ? load8_raw(a.pre_w, a.nwbf, e, a.H - e) : f32x8(0.f);
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[i][j], x[i][j], ss);
  const float rs = rsqrtf(fmaf(row_sum(ss, a.per_row, red), a.inv_h, a.next_eps));
  if (!live) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = (i * a.per_row + in_row) * 8;
    f32x8 o = x[i] * rs;
    if (a.pre_w) o *= a.next_offset + widen_raw(w[i], a.nwbf);
    store8<OBF16, V == 2>(a.next_out, at + e, a.H - e, o);
  }
}

// LOOP: as many workgroups as the chip holds at a time go over the rows, with the
// weights and a channel gate in registers throughout (read again for every row,
// from the caches, they are nearly as many bytes as the row's own).  4096 rows of
// 4096 24.3 instead of 27.5 us, 1200 rows 8.6 instead of 10.8, 1500 of 5120 13.7
// instead of 18.1; the same for norm_in gained 4% at 4096 rows and lost 18% at 1200,
// so its rows stay one a group of threads.
template <bool YBF16, bool RBF16, bool NBF16, int V, bool LOOP>
__global__ __launch_bounds__(1024) void norm_out_kernel(NormArgs a) {
  __shared__ float red[LOOP ? 2 : 1][2][16];
  const int in_row = threadIdx.x & (a.per_row - 1), rows = blockDim.x / a.per_row;
  const bool elementwise = a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL;
  int row0 = blockIdx.x * rows, turn = 0;
  f32x8 y[V], r[V], w[V], g[V], nw[V];
  auto load_weights = [&](int i) {
    const int e = (i * a.per_row + in_row) * 8, n = a.H - e;
    w[i] = a.post && a.post_w ? load8_raw(a.post_w, a.wbf, e, n) : f32x8(0.f);
    nw[i] = a.next_out && a.pre_w ? load8_raw(a.pre_w, a.nwbf, e, n) : f32x8(0.f);
  };
  if constexpr (LOOP) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = (i * a.per_row + in_row) * 8;
      g[i] = a.gate_kind == MOE_GATE_CHANNEL ? load8_raw(a.gate, a.gbf, e, a.H - e) : f32x8(0.f);
      load_weights(i);
    }
  }
  do {
    const int row = row0 + threadIdx.x / a.per_row;
    const bool live = row < a.T;
    const size_t at = (size_t)min(row, a.T - 1) * a.H;
    float tok = 1.f;
    if (a.gate_kind == MOE_GATE_TOKEN) tok = load1(a.gate, a.gbf, min(row, a.T - 1));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = (i * a.per_row + in_row) * 8, n = a.H - e;
      y[i] = load8<YBF16>(a.y, at + e, n);
      r[i] = load8<RBF16>(a.residual, at + e, n);
      if constexpr (LOOP) {
        if (a.gate_kind == MOE_GATE_FULL) g[i] = load8_raw(a.gate, a.gbf, at + e, n);
      } else {
        g[i] = elementwise ? load8_raw(a.gate, a.gbf, a.gate_kind == MOE_GATE_FULL ? at + e : e, n) : f32x8(0.f);
        load_weights(i);
      }
    }
    float c = a.alpha;
    if (a.post) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(y[i][j], y[i][j], ss);
      const float rs = rsqrtf(fmaf(row_sum(ss, a.per_row, red[turn][0]), a.inv_h, a.eps));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        y[i] *= rs;
        if (a.post_w) y[i] *= a.offset + widen_raw(w[i], a.wbf);
      }
    }
    if (a.gate_kind == MOE_GATE_TOKEN) c *= a.sigmoid ? gate_sigmoid(tok) : tok;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (elementwise) {
        f32x8 f = widen_raw(g[i], a.gbf);
        if (a.sigmoid) {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = gate_sigmoid(f[j]);
        }
        y[i] *= f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[i][j] = fmaf(c, y[i][j], r[i][j]);
        ss = fmaf(r[i][j], r[i][j], ss);
      }
    }
    if (live) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = (i * a.per_row + in_row) * 8;
        store8<RBF16, V == 2>(a.out, at + e, a.H - e, r[i]);
      }
    }
    if (a.next_out) {
      const float rs = rsqrtf(fmaf(row_sum(ss, a.per_row, red[turn][1]), a.inv_h, a.next_eps));
      if (!live) break;  // only in the last turn
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = (i * a.per_row + in_row) * 8;
        r[i] *= rs;
        if (a.pre_w) r[i] *= a.next_offset + widen_raw(nw[i], a.nwbf);
        store8<NBF16, V == 2>(a.next_out, at + e, a.H - e, r[i]);
      }
    }
    if (LOOP) turn ^= 1;
  } while (LOOP && (row0 += gridDim.x * rows) < a.T);
}

struct Shape {
  dim3 grid, block;
  int v;
  bool loop;
};

constexpr int kCUs = 256;

// One chunk a thread up to 2^20 elements, where a row's latency counts, two (and
// streaming stores) above, where bandwidth does.  H = 4096, with one and two:
// norm_in 1 row 2.2 and 2.4 us, 256 rows 2.7 and 2.8, 512 rows 3.15 and 3.05, 1024
// rows 4.7 and 3.7, 4096 rows 14.1 and 12.0; norm_out 1 row 3.1 and 4.0, 256 rows 3.9
// and 4.7, 512 rows 5.2 and 5.0, 1024 rows 9.3 and 8.1, 4096 rows 31.4 and 24.4.  The
// same from H = 520 to 8192: at 2^22 elements two gain 22 to 42% (norm_in) and 7 to 23%.
// Rows of at most 64 chunks have no second one for their 64 threads: 16384 x 256
// norm_in 6.8 and 8.1, norm_out 11.9 and 15.5; 8192 x 512 4.75 and 4.95, 9.3 and 9.6.
// From 2^23 elements on the rows' loop, which comes with two, outweighs that for
// norm_out where most of the 64 have one: 32768 x 512 31.1 and 24.6, 43691 x 384 36.0
// and 32.2, but 52429 x 320 39.1 and 38.8, 65536 x 256 41.7 and 46.2.
Shape shape(NormArgs& a, bool may_loop) {
  const int chunks = (a.H + 7) / 8;
  const size_t n = (size_t)a.T * a.H;
  const bool two = chunks > 1024 || (chunks > 64 ? n > (size_t)1 << 20 : may_loop && chunks > 40 && n > (size_t)1 << 23);
  const int v = two ? 2 : 1;
  int per = 64;
  while (per * v < chunks) per *= 2;
  const int block = max(per, 256), rows = block / per;
  a.per_row = per;
  a.inv_h = 1.0f / (float)a.H;
  const int blocks = (a.T + rows - 1) / rows, resident = kCUs * 1024 / block;
  const bool loop = may_loop && v == 2 && blocks > resident;
  return {dim3(loop ? resident : blocks), dim3(block), v, loop};
}

template <bool XB, bool OB>
void run_in(NormArgs& a, hipStream_t s) {
  const Shape h = shape(a, false);
  if (h.v == 1)
    launch(MOE_PROF_NORM, norm_in_kernel<XB, OB, 1>, h.grid, h.block, 0, s, a);
  else
    launch(MOE_PROF_NORM, norm_in_kernel<XB, OB, 2>, h.grid, h.block, 0, s, a);
}

template <bool YB, bool RB, bool NB>
void run_out(NormArgs& a, hipStream_t s) {
  const Shape h = shape(a, true);
  if (h.v == 1)
    launch(MOE_PROF_NORM, norm_out_kernel<YB, RB, NB, 1, false>, h.grid, h.block, 0, s, a);
  else if (!h.loop)
    launch(MOE_PROF_NORM, norm_out_kernel<YB, RB, NB, 2, false>, h.grid, h.block, 0, s, a);
  else
    launch(MOE_PROF_NORM, norm_out_kernel<YB, RB, NB, 2, true>, h.grid, h.block, 0, s, a);
}

}  // namespace

moe_status launch_norm_in(const moe_norm* n, const void* x, moe_dtype xt, int T, void* out, moe_dtype ot,
                          hipStream_t s) {
  NormArgs a{};
  a.y = x;
  a.T = T;
  a.H = n->H;
  a.pre_w = n->pre_w;
  a.nwbf = n->wt == MOE_BF16;
  a.next_eps = n->eps;
  a.next_offset = n->weight_offset;
  a.next_out = out;
  const bool xb = xt == MOE_BF16, ob = ot == MOE_BF16;
  if (xb)
    ob ? run_in<true, true>(a, s) : run_in<true, false>(a, s);
  else
    ob ? run_in<false, true>(a, s) : run_in<false, false>(a, s);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

moe_status launch_norm_out(const moe_norm* n, const void* y, moe_dtype yt, const void* residual, const void* gate,
                           moe_dtype gt, int T, void* out, moe_dtype rt, const moe_norm* next, void* next_out,
                           moe_dtype nt, hipStream_t s) {
  NormArgs a{};
  a.y = y;
  a.residual = residual;
  a.out = out;
  a.T = T;
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
  }
  const bool yb = yt == MOE_BF16, rb = rt == MOE_BF16, nb = next && nt == MOE_BF16;
  if (yb) {
    if (rb)
      nb ? run_out<true, true, true>(a, s) : run_out<true, true, false>(a, s);
    else
      nb ? run_out<true, false, true>(a, s) : run_out<true, false, false>(a, s);
  } else {
    if (rb)
      nb ? run_out<false, true, true>(a, s) : run_out<false, true, false>(a, s);
    else
      nb ? run_out<false, false, true>(a, s) : run_out<false, false, false>(a, s);
  }
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
