// C entry points of the MoE library: validate every argument, then enqueue.
//
// Validation happens before any launch and fails with a targeted message
// rather than producing wrong math, the behaviour "Running DeepSeek-V4-Flash
// across four free GPUs" (§Step 2, Check it divides; §Step 7, the slot-count
// floor) asks of a serving runtime.
#include <algorithm>
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "common.h"

namespace moe {

static thread_local std::string g_last_error;

void set_error(const char* fmt, ...) {
  char buf[1024];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
}

moe_status fail(moe_status st, const char* fmt, ...) {
  char buf[1024];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

moe_status launch_route(const float* logits, int T, int E, int k, int32_t* ids, float* w, hipStream_t s);
moe_status launch_router_logits(const void* x, moe_dtype xt, const float* wr, int T, int E, int H, float* logits,
                                hipStream_t s);
moe_status launch_dequant(const uint8_t* record, int H, int I, int prec, int matrix, float* out, hipStream_t s);
moe_status launch_stream_read(const void* buf, size_t bytes, uint32_t* sink, hipStream_t s);
bool decode_shape_ok(int H, int I);
size_t prefill_workspace_bytes(int H, int I, int T, int k, int has_shared);
moe_status launch_quant_mxfp8(const void* x, long rows, int K, uint8_t* codes, uint8_t* scales, hipStream_t s);
size_t group_wide_scratch_ints(int n, int nkeys);
moe_status launch_group_wide(const int32_t* keys, int n, int nkeys, int32_t* counts, int32_t* offsets,
                             int32_t* perm, int32_t* scratch, hipStream_t s);
moe_status launch_prefill(const moe_layer* Lr, int E, const void* x, int T, int k, const int32_t* ids, const float* w,
                          void* out, void* workspace, hipStream_t s);
bool b1_path_ok(int H, int I, int K1, bool xbf16, bool obf16);
bool b1_route_ok(int E, int num_slots);
bool b1s_path_ok(int H, int I, int K1, bool xbf16, bool obf16, bool has_prec);
bool b1s_route_ok(int E, int num_slots);
moe_status launch_b1s(const moe_layer* L, const float* logits, int E, const void* x, int k, int32_t* slot_ids,
                      float* w, uint16_t* h, void* out, hipStream_t s);
moe_status launch_b1(const moe_layer* L, const float* logits, int E, const void* x, int k, int32_t* slot_ids,
                     const int8_t* prec, float* w, uint16_t* h, void* out, hipStream_t s);
size_t decode_plan_ints(int P);
bool decode_mfma_ok(int H, int I);
size_t decode_mfma_plan_ints(int P);
size_t fused_sync_bytes();
bool fused_path_ok(const moe_layer* L, int K1, bool xbf16, bool obf16, bool has_prec);
moe_status launch_fused_b1(const moe_layer* L, const float* logits, int E, const void* x, int k, int32_t* slot_ids,
                           float* w, uint16_t* h, void* out, uint32_t* sync, hipStream_t s);
bool fused_s_path_ok(const moe_layer* L, int K1, bool xbf16, bool obf16, bool has_prec);
moe_status launch_fused_b1s(const moe_layer* L, const float* logits, int E, const void* x, int k, int32_t* slot_ids,
                            float* w, uint16_t* h, void* out, uint32_t* sync, hipStream_t s);
moe_status launch_decode_mfma(const moe_layer* Lr, const void* x, int T, int k, const int32_t* slot_ids, const float* w,
                              void* out, uint16_t* h, float* y, int32_t* plan, hipStream_t s);

moe_status launch_route_groups(const moe_router* R, const void* logits, moe_dtype lt, const float* bias, int T,
                               int32_t* ids, float* w, hipStream_t s);
moe_status launch_norm_in(const moe_norm* n, const void* x, moe_dtype xt, int T, void* out, moe_dtype ot,
                          hipStream_t s);
moe_status launch_norm_out(const moe_norm* n, const void* y, moe_dtype yt, const void* residual, const void* gate,
                           moe_dtype gt, int T, void* out, moe_dtype rt, const moe_norm* next, void* next_out,
                           moe_dtype nt, hipStream_t s);
moe_status launch_lora(const moe_lora* L, const void* x, moe_dtype xt, int T, const int32_t* ids, const void* base,
                       void* out, moe_dtype yt, hipStream_t s);

size_t permute_scratch_bytes(int T, int k, int E);
moe_status launch_permute(const void* x, moe_dtype xt, int T, int k, int H, int E, const int32_t* ids, void* xs,
                          int32_t* offsets, int32_t* perm, int32_t* rows, int32_t* scratch, hipStream_t s);
moe_status launch_unpermute(const void* ys, moe_dtype yt, int M, const int32_t* rows, const float* w, const void* base,
                            int T, int k, int H, void* out, moe_dtype ot, hipStream_t s);
moe_status launch_unpermute_grad(const void* gout, moe_dtype gt, const void* ys, moe_dtype yt, int M,
                                 const int32_t* rows, const float* w, int T, int k, int H, void* gys, float* gw,
                                 hipStream_t s);
moe_status launch_route_grad(const moe_router* R, const void* logits, moe_dtype lt, int T, const int32_t* ids,
                             const float* w, const float* gw, void* glogits, moe_dtype gt, hipStream_t s);
moe_status launch_q4(const moe_q4* q, const void* x, moe_dtype xt, int T, const int32_t* offsets, void* y, moe_dtype yt,
                     hipStream_t s);

static bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

static size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace moe

using namespace moe;

#define REQUIRE(cond, st, ...)          \
  do {                                  \
    if (!(cond)) return fail(st, __VA_ARGS__); \
  } while (0)

extern "C" {

const char* moe_last_error(void) { return g_last_error.c_str(); }

const char* moe_version(void) { return "moe-mi355x 0.1 (gfx950)"; }

size_t moe_fp4_expert_bytes(int H, int I) {
  if (H <= 0 || I <= 0) return 0;
  return record_layout(H, I, 4).bytes;
}

size_t moe_int2_expert_bytes(int H, int I) {
  if (H <= 0 || I <= 0) return 0;
  return record_layout(H, I, 2).bytes;
}

moe_status moe_router_logits(const void* x, moe_dtype xt, const float* w_router, int T, int E, int H, float* logits,
                             moe_stream_t stream) {
  REQUIRE(T >= 0 && E >= 1 && H >= 1, MOE_ESHAPE, "moe_router_logits: bad sizes T=%d E=%d H=%d", T, E, H);
  REQUIRE(xt == MOE_F32 || xt == MOE_BF16, MOE_EINVAL, "moe_router_logits: bad dtype %d", (int)xt);
  REQUIRE(T == 0 || (x && w_router && logits), MOE_EINVAL, "moe_router_logits: NULL pointer");
  return launch_router_logits(x, xt, w_router, T, E, H, logits, (hipStream_t)stream);
}

moe_status moe_route(const float* logits, int T, int E, int k, int32_t* ids, float* w, moe_stream_t stream) {
  REQUIRE(T >= 0, MOE_ESHAPE, "moe_route: T=%d < 0", T);
  REQUIRE(E >= 1 && E <= 1024, MOE_ESHAPE, "moe_route: E=%d outside 1..1024", E);
  REQUIRE(k >= 1 && k <= E && k <= 64, MOE_EINVAL, "moe_route: k=%d must satisfy 1 <= k <= min(E=%d, 64)", k, E);
  REQUIRE(T == 0 || (logits && ids && w), MOE_EINVAL, "moe_route: NULL pointer");
  return launch_route(logits, T, E, k, ids, w, (hipStream_t)stream);
}

moe_status moe_group(const int32_t* keys, int n, int nkeys, int32_t* counts, int32_t* offsets, int32_t* perm,
                     moe_stream_t stream) {
  REQUIRE(n >= 0 && n <= (1 << 20), MOE_ESHAPE, "moe_group: n=%d outside 0..2^20", n);
  REQUIRE(nkeys >= 1 && nkeys <= 4096, MOE_ESHAPE, "moe_group: nkeys=%d outside 1..4096", nkeys);
  REQUIRE(counts && offsets && (n == 0 || (keys && perm)), MOE_EINVAL, "moe_group: NULL pointer");
  return launch_group(keys, n, nkeys, counts, offsets, perm, (hipStream_t)stream);
}

size_t moe_group_scratch_bytes(int n, int nkeys) {
  if (n < 0 || n > (1 << 20) || nkeys < 1 || nkeys > 4096) return 0;
  return group_wide_scratch_ints(n, nkeys) * sizeof(int32_t);
}

moe_status moe_group_wide(const int32_t* keys, int n, int nkeys, int32_t* counts, int32_t* offsets, int32_t* perm,
                          void* scratch, moe_stream_t stream) {
  REQUIRE(n >= 0 && n <= (1 << 20), MOE_ESHAPE, "moe_group_wide: n=%d outside 0..2^20", n);
  REQUIRE(nkeys >= 1 && nkeys <= 4096, MOE_ESHAPE, "moe_group_wide: nkeys=%d outside 1..4096", nkeys);
  REQUIRE(counts && offsets && (n == 0 || (keys && perm)), MOE_EINVAL, "moe_group_wide: NULL pointer");
  REQUIRE(group_wide_scratch_ints(n, nkeys) == 0 || (scratch && aligned(scratch, 4)), MOE_EINVAL,
          "moe_group_wide: scratch is NULL or not 4-byte aligned (%zu bytes needed)",
          group_wide_scratch_ints(n, nkeys) * sizeof(int32_t));
  return launch_group_wide(keys, n, nkeys, counts, offsets, perm, (int32_t*)scratch, (hipStream_t)stream);
}

size_t moe_expert_workspace_sync_offset(int H, int I, int T, int k, int has_shared) {
  if (H <= 0 || I <= 0 || T < 0 || k <= 0) return 0;
  const size_t P = (size_t)T * (size_t)(k + (has_shared ? 1 : 0));
  return align256(P * I * 4) + align256(P * H * 4) +
         align256(std::max(decode_plan_ints((int)P), decode_mfma_plan_ints((int)P)) * 4);
}

size_t moe_expert_workspace_bytes(int H, int I, int T, int k, int has_shared) {
  if (H <= 0 || I <= 0 || T < 0 || k <= 0) return 0;
  return moe_expert_workspace_sync_offset(H, I, T, k, has_shared) + align256(fused_sync_bytes());
}

static moe_status check_layer(const moe_layer* L, const char* who) {
  REQUIRE(L, MOE_EINVAL, "%s: layer is NULL", who);
  REQUIRE(decode_shape_ok(L->H, L->I), MOE_ESHAPE,
          "%s: H=%d I=%d unsupported (need multiples of 32 with H/32, I/32 a power of two in 4..64 or 128/256)", who,
          L->H, L->I);
  const size_t fb = record_layout(L->H, L->I, 4).bytes, ib = record_layout(L->H, L->I, 2).bytes;
  REQUIRE(L->fp4_base || L->num_slots == 0, MOE_EINVAL, "%s: fp4_base is NULL with num_slots=%d", who, L->num_slots);
  REQUIRE(L->num_slots >= 0 && L->num_int2 >= 0, MOE_EINVAL, "%s: negative slot counts", who);
  REQUIRE(L->num_slots == 0 || (L->fp4_stride >= fb && L->fp4_stride % 16 == 0), MOE_EINVAL,
          "%s: fp4_stride=%zu must be >= %zu and a multiple of 16", who, L->fp4_stride, fb);
  REQUIRE(!L->int2_base || L->num_int2 == 0 || (L->int2_stride >= ib && L->int2_stride % 16 == 0), MOE_EINVAL,
          "%s: int2_stride=%zu must be >= %zu and a multiple of 16", who, L->int2_stride, ib);
  REQUIRE(aligned(L->fp4_base, 16) && aligned(L->int2_base, 16) && aligned(L->shared, 16), MOE_EINVAL,
          "%s: expert records must be 16-byte aligned", who);
  return MOE_OK;
}

}  // extern "C"

namespace moe {

// The expert MLP of moe_expert_forward.  sync: the words the single launch
// keeps between calls; NULL puts them at the end of the workspace (the public
// entry point's layout), and then the workspace must cover them too.
moe_status expert_forward_impl(const moe_layer* layer, const void* x, moe_dtype xt, int T, int k,
                               const int32_t* slot_ids, const int8_t* prec, const float* w, void* out, moe_dtype ot,
                               void* workspace, size_t workspace_bytes, uint32_t* sync, hipStream_t s) {
  moe_status st = check_layer(layer, "moe_expert_forward");
  if (st != MOE_OK) return st;
  REQUIRE(T >= 0 && T <= 65536, MOE_ESHAPE, "moe_expert_forward: T=%d outside 0..65536", T);
  REQUIRE(k >= 1 && k <= 64, MOE_EINVAL, "moe_expert_forward: k=%d outside 1..64", k);
  REQUIRE(xt == MOE_F32 || xt == MOE_BF16, MOE_EINVAL, "moe_expert_forward: bad activation dtype %d", (int)xt);
  REQUIRE(w || ot == MOE_F32, MOE_EINVAL, "moe_expert_forward: per-rank outputs (w == NULL) are fp32");
  REQUIRE(ot == MOE_F32 || ot == MOE_BF16, MOE_EINVAL, "moe_expert_forward: bad output dtype %d", (int)ot);
  if (T == 0) return MOE_OK;
  REQUIRE(x && slot_ids && out && workspace, MOE_EINVAL, "moe_expert_forward: NULL pointer");
  REQUIRE(aligned(x, 16) && aligned(out, 16) && aligned(workspace, 256), MOE_EINVAL,
          "moe_expert_forward: x/out must be 16-byte and workspace 256-byte aligned");
  const int has_shared = layer->shared ? 1 : 0;
  const size_t need = sync ? moe_expert_workspace_sync_offset(layer->H, layer->I, T, k, has_shared)
                           : moe_expert_workspace_bytes(layer->H, layer->I, T, k, has_shared);
  REQUIRE(workspace_bytes >= need, MOE_ENOMEM, "moe_expert_forward: workspace %zu bytes < %zu needed",
          workspace_bytes, need);
  const int nkeys = layer->num_slots + (layer->int2_base ? layer->num_int2 : 0) + 1;
  REQUIRE(T == 1 || nkeys <= 4096, MOE_ESHAPE,
          "moe_expert_forward: batched grouping supports at most 4095 slots + 2-bit entries (got %d)", nkeys - 1);
  const int K1 = k + has_shared;
  const size_t P = (size_t)T * K1;
  char* ws = (char*)workspace;
  float* h = (float*)ws;
  float* y = (float*)(ws + align256(P * layer->I * 4));
  int32_t* plan = (int32_t*)(ws + align256(P * layer->I * 4) + align256(P * layer->H * 4));
  float* yout = w ? y : (float*)out;
  if (!sync) sync = (uint32_t*)(ws + moe_expert_workspace_sync_offset(layer->H, layer->I, T, k, has_shared));
  if (T == 1 && w && fused_path_ok(layer, K1, xt == MOE_BF16, ot == MOE_BF16, prec != nullptr))
    return launch_fused_b1(layer, nullptr, 0, x, k, const_cast<int32_t*>(slot_ids), const_cast<float*>(w),
                           (uint16_t*)h, out, sync, s);
  if (T == 1 && w && b1_path_ok(layer->H, layer->I, K1, xt == MOE_BF16, ot == MOE_BF16))  // reads slot_ids and w only
    return launch_b1(layer, nullptr, 0, x, k, const_cast<int32_t*>(slot_ids), prec, const_cast<float*>(w),
                     (uint16_t*)h, out, s);
  if (T == 1 && w && fused_s_path_ok(layer, K1, xt == MOE_BF16, ot == MOE_BF16, prec != nullptr))
    return launch_fused_b1s(layer, nullptr, 0, x, k, const_cast<int32_t*>(slot_ids), const_cast<float*>(w),
                            (uint16_t*)h, out, sync, s);
  if (T == 1 && w && b1s_path_ok(layer->H, layer->I, K1, xt == MOE_BF16, ot == MOE_BF16, prec != nullptr))
    return launch_b1s(layer, nullptr, 0, x, k, const_cast<int32_t*>(slot_ids), const_cast<float*>(w), (uint16_t*)h,
                      out, s);
  // batches of bf16 tokens, all FP4, weighted output: bf16 MFMA on weights dequantised in registers
  if (T >= 2 && w && !prec && xt == MOE_BF16 && ot == MOE_BF16 && decode_mfma_ok(layer->H, layer->I) &&
      P * (size_t)layer->I * 2 < ((size_t)1 << 31) && (size_t)T * layer->H * 2 < ((size_t)1 << 31))
    return launch_decode_mfma(layer, x, T, k, slot_ids, w, out, (uint16_t*)h, y, plan, s);
  st = launch_expert_decode(layer, x, xt, T, k, slot_ids, prec, h, yout, plan, s);
  if (st != MOE_OK) return st;
  if (w) return launch_combine(y, w, prec, T, k, layer->H, has_shared, out, ot, s);
  return MOE_OK;
}

// moe_layer_decode with the same sync convention as expert_forward_impl.
moe_status layer_decode_impl(const moe_layer* layer, const float* logits, int E, const void* x, moe_dtype xt, int k,
                             int32_t* ids, float* w, void* out, moe_dtype ot, void* workspace, size_t workspace_bytes,
                             uint32_t* sync, hipStream_t s) {
  moe_status st = check_layer(layer, "moe_layer_decode");
  if (st != MOE_OK) return st;
  REQUIRE(E >= 1 && E <= 1024, MOE_ESHAPE, "moe_layer_decode: E=%d outside 1..1024", E);
  REQUIRE(k >= 1 && k <= E && k <= 64, MOE_EINVAL, "moe_layer_decode: k=%d must satisfy 1 <= k <= min(E=%d, 64)", k,
          E);
  REQUIRE(layer->num_slots >= E, MOE_ECACHE_SMALL,
          "moe_layer_decode: the layer must hold every expert (num_slots=%d < E=%d); use the slot cache instead",
          layer->num_slots, E);
  REQUIRE(xt == MOE_F32 || xt == MOE_BF16, MOE_EINVAL, "moe_layer_decode: bad activation dtype %d", (int)xt);
  REQUIRE(ot == MOE_F32 || ot == MOE_BF16, MOE_EINVAL, "moe_layer_decode: bad output dtype %d", (int)ot);
  REQUIRE(logits && x && ids && w && out && workspace, MOE_EINVAL, "moe_layer_decode: NULL pointer");
  REQUIRE(aligned(x, 16) && aligned(out, 16) && aligned(workspace, 256), MOE_EINVAL,
          "moe_layer_decode: x/out must be 16-byte and workspace 256-byte aligned");
  const int has_shared = layer->shared ? 1 : 0;
  const size_t need = sync ? moe_expert_workspace_sync_offset(layer->H, layer->I, 1, k, has_shared)
                           : moe_expert_workspace_bytes(layer->H, layer->I, 1, k, has_shared);
  REQUIRE(workspace_bytes >= need, MOE_ENOMEM, "moe_layer_decode: workspace %zu bytes < %zu needed", workspace_bytes,
          need);
  if (!sync)
    sync = (uint32_t*)((char*)workspace + moe_expert_workspace_sync_offset(layer->H, layer->I, 1, k, has_shared));
  if (fused_path_ok(layer, k + has_shared, xt == MOE_BF16, ot == MOE_BF16, false) &&
      b1_route_ok(E, layer->num_slots))
    return launch_fused_b1(layer, logits, E, x, k, ids, w, (uint16_t*)workspace, out, sync, s);
  if (b1_path_ok(layer->H, layer->I, k + has_shared, xt == MOE_BF16, ot == MOE_BF16) && b1_route_ok(E, layer->num_slots))
    return launch_b1(layer, logits, E, x, k, ids, nullptr, w, (uint16_t*)workspace, out, s);
  if (fused_s_path_ok(layer, k + has_shared, xt == MOE_BF16, ot == MOE_BF16, false) &&
      b1s_route_ok(E, layer->num_slots))
    return launch_fused_b1s(layer, logits, E, x, k, ids, w, (uint16_t*)workspace, out, sync, s);
  if (b1s_path_ok(layer->H, layer->I, k + has_shared, xt == MOE_BF16, ot == MOE_BF16, false) &&
      b1s_route_ok(E, layer->num_slots))
    return launch_b1s(layer, logits, E, x, k, ids, w, (uint16_t*)workspace, out, s);
  st = launch_route(logits, 1, E, k, ids, w, s);
  if (st != MOE_OK) return st;
  return expert_forward_impl(layer, x, xt, 1, k, ids, nullptr, w, out, ot, workspace, workspace_bytes, sync, s);
}

}  // namespace moe

extern "C" {

moe_status moe_expert_forward(const moe_layer* layer, const void* x, moe_dtype xt, int T, int k,
                              const int32_t* slot_ids, const int8_t* prec, const float* w, void* out, moe_dtype ot,
                              void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  return expert_forward_impl(layer, x, xt, T, k, slot_ids, prec, w, out, ot, workspace, workspace_bytes, nullptr,
                             (hipStream_t)stream);
}

moe_status moe_layer_decode(const moe_layer* layer, const float* logits, int E, const void* x, moe_dtype xt, int k,
                            int32_t* ids, float* w, void* out, moe_dtype ot, void* workspace, size_t workspace_bytes,
                            moe_stream_t stream) {
  return layer_decode_impl(layer, logits, E, x, xt, k, ids, w, out, ot, workspace, workspace_bytes, nullptr,
                           (hipStream_t)stream);
}

moe_status moe_combine(const float* y, const float* w, const int8_t* prec, int T, int k, int H, int has_shared,
                       void* out, moe_dtype ot, moe_stream_t stream) {
  REQUIRE(T >= 0 && k >= 1 && H >= 4 && H % 4 == 0, MOE_ESHAPE, "moe_combine: bad sizes T=%d k=%d H=%d", T, k, H);
  REQUIRE(ot == MOE_F32 || ot == MOE_BF16, MOE_EINVAL, "moe_combine: bad output dtype %d", (int)ot);
  if (T == 0) return MOE_OK;
  REQUIRE(y && w && out, MOE_EINVAL, "moe_combine: NULL pointer");
  REQUIRE(aligned(y, 16) && aligned(out, 8), MOE_EINVAL, "moe_combine: y must be 16-byte, out 8-byte aligned");
  return launch_combine(y, w, prec, T, k, H, has_shared ? 1 : 0, out, ot, (hipStream_t)stream);
}

moe_status moe_quant_mxfp8(const void* x, int rows, int K, uint8_t* codes, uint8_t* scales, moe_stream_t stream) {
  REQUIRE(rows >= 0 && K >= 32 && K % 32 == 0, MOE_ESHAPE, "moe_quant_mxfp8: rows=%d K=%d (K a multiple of 32)", rows,
          K);
  if (rows == 0) return MOE_OK;
  REQUIRE(x && codes && scales, MOE_EINVAL, "moe_quant_mxfp8: NULL pointer");
  REQUIRE(aligned(x, 16) && aligned(codes, 16), MOE_EINVAL, "moe_quant_mxfp8: x and codes must be 16-byte aligned");
  return launch_quant_mxfp8(x, rows, K, codes, scales, (hipStream_t)stream);
}

size_t moe_prefill_workspace_bytes(int H, int I, int T, int k, int has_shared) {
  if (H <= 0 || I <= 0 || T < 0 || k <= 0) return 0;
  return prefill_workspace_bytes(H, I, T, k, has_shared);
}

moe_status moe_prefill_forward(const moe_layer* layer, const void* x, int T, int k, const int32_t* ids, const float* w,
                               void* out, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  REQUIRE(layer, MOE_EINVAL, "moe_prefill_forward: layer is NULL");
  const int H = layer->H, I = layer->I, E = layer->num_slots;
  REQUIRE(H >= 256 && I >= 128 && H % 256 == 0 && I % 128 == 0, MOE_ESHAPE,
          "moe_prefill_forward: H=%d must be a multiple of 256 and I=%d a multiple of 128", H, I);
  REQUIRE(E >= 1 && E <= 4095, MOE_ESHAPE, "moe_prefill_forward: num_slots (experts) = %d outside 1..4095", E);
  REQUIRE(k >= 1 && k <= E && k <= 64, MOE_EINVAL, "moe_prefill_forward: k=%d (E=%d)", k, E);
  const int K1 = k + (layer->shared ? 1 : 0);
  REQUIRE(T >= 0 && (long)T * K1 <= (1L << 20), MOE_ESHAPE, "moe_prefill_forward: T=%d too large", T);
  REQUIRE((long)T * K1 * I < (1L << 31) && (long)T * H < (1L << 31), MOE_ESHAPE,
          "moe_prefill_forward: T=%d: activations beyond 2 GiB per matrix", T);
  if (T == 0) return MOE_OK;
  REQUIRE(layer->fp4_base && x && ids && w && out && workspace, MOE_EINVAL, "moe_prefill_forward: NULL pointer");
  const size_t fb = record_layout(H, I, 4).bytes;
  REQUIRE(layer->fp4_stride >= fb && layer->fp4_stride % 16 == 0, MOE_EINVAL,
          "moe_prefill_forward: fp4_stride=%zu must be >= %zu and a multiple of 16", layer->fp4_stride, fb);
  REQUIRE(aligned(layer->fp4_base, 16) && aligned(layer->shared, 16) && aligned(x, 16) && aligned(out, 16) &&
              aligned(workspace, 256),
          MOE_EINVAL, "moe_prefill_forward: records, x, out 16-byte and workspace 256-byte aligned");
  const size_t need = prefill_workspace_bytes(H, I, T, k, layer->shared ? 1 : 0);
  REQUIRE(workspace_bytes >= need, MOE_ENOMEM, "moe_prefill_forward: workspace %zu bytes < %zu needed",
          workspace_bytes, need);
  return launch_prefill(layer, E, x, T, k, ids, w, out, workspace, (hipStream_t)stream);
}

moe_status moe_debug_dequant(const uint8_t* record, int H, int I, int prec, int matrix, float* out,
                             moe_stream_t stream) {
  REQUIRE(H > 0 && I > 0 && H % 32 == 0 && I % 32 == 0, MOE_ESHAPE, "moe_debug_dequant: H=%d I=%d", H, I);
  REQUIRE(prec >= 0 && prec <= 2, MOE_EINVAL, "moe_debug_dequant: mode=%d (0 FP4, 1 2-bit, 2 FP4 scaled convert)",
          prec);
  REQUIRE(matrix >= 0 && matrix <= 2, MOE_EINVAL, "moe_debug_dequant: matrix=%d", matrix);
  REQUIRE(record && out, MOE_EINVAL, "moe_debug_dequant: NULL pointer");
  REQUIRE(aligned(record, 4), MOE_EINVAL, "moe_debug_dequant: record must be 4-byte aligned");
  return launch_dequant(record, H, I, prec, matrix, out, (hipStream_t)stream);
}

moe_status moe_debug_stream_read(const void* buf, size_t bytes, uint32_t* sink, moe_stream_t stream) {
  REQUIRE(buf && sink, MOE_EINVAL, "moe_debug_stream_read: NULL pointer");
  REQUIRE(aligned(buf, 16) && bytes % 16 == 0, MOE_EINVAL,
          "moe_debug_stream_read: buf must be 16-byte aligned and bytes a multiple of 16");
  if (bytes == 0) return MOE_OK;
  return launch_stream_read(buf, bytes, sink, (hipStream_t)stream);
}

}  // extern "C"

// ------------------------------------------------------------ around the experts

namespace {

constexpr int kMaxTokens = 1 << 20;  // rows of the calls below: a grid of 1024-thread workgroups stays below 2^32 threads

bool is_dtype(moe_dtype t) { return t == MOE_F32 || t == MOE_BF16; }
size_t dsize(moe_dtype t) { return t == MOE_BF16 ? 2 : 4; }

// A buffer of a call.  Workgroups write their rows while others still read theirs,
// so an output may share memory with another buffer only row for row: the same one.
struct Buffer {
  const void* p;
  size_t bytes;
};

bool overlap(Buffer a, Buffer b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return a.p && b.p && x < y + b.bytes && y < x + a.bytes;
}
bool overlap_part(Buffer a, Buffer b) { return a.p != b.p && overlap(a, b); }

moe_status check_norm(const moe_norm* n, const char* who) {
  REQUIRE(n, MOE_EINVAL, "%s: norm is NULL", who);
  REQUIRE(n->H >= 1 && n->H <= 16384, MOE_ESHAPE, "%s: H=%d outside 1..16384", who, n->H);
  REQUIRE(n->eps >= 0.0f && std::isfinite(n->eps), MOE_EINVAL, "%s: eps=%g must be finite and >= 0", who, (double)n->eps);
  REQUIRE(std::isfinite(n->weight_offset) && std::isfinite(n->alpha), MOE_EINVAL,
          "%s: weight_offset and alpha must be finite", who);
  REQUIRE(is_dtype(n->wt), MOE_EINVAL, "%s: bad weight dtype %d", who, (int)n->wt);
  REQUIRE(aligned(n->pre_w, dsize(n->wt)) && aligned(n->post_w, dsize(n->wt)), MOE_EINVAL,
          "%s: norm weights must be aligned to their element", who);
  REQUIRE(n->post_norm == 0 || n->post_norm == 1, MOE_EINVAL, "%s: post_norm=%d", who, n->post_norm);
  REQUIRE(n->gate >= MOE_GATE_NONE && n->gate <= MOE_GATE_FULL, MOE_EINVAL, "%s: gate=%d", who, n->gate);
  REQUIRE(n->gate_act == MOE_GATE_LINEAR || n->gate_act == MOE_GATE_SIGMOID, MOE_EINVAL, "%s: gate_act=%d", who,
          n->gate_act);
  return MOE_OK;
}

moe_status check_router(const moe_router* R, const char* who) {
  REQUIRE(R, MOE_EINVAL, "%s: router is NULL", who);
  REQUIRE(R->E >= 1 && R->E <= 1024, MOE_ESHAPE, "%s: E=%d outside 1..1024", who, R->E);
  REQUIRE(R->k >= 1 && R->k <= R->E && R->k <= 64, MOE_EINVAL,
          "%s: k=%d must satisfy 1 <= k <= min(E=%d, 64)", who, R->k, R->E);
  REQUIRE(R->scoring == MOE_SCORE_SOFTMAX || R->scoring == MOE_SCORE_SIGMOID, MOE_EINVAL,
          "%s: scoring=%d", who, R->scoring);
  REQUIRE(R->groups >= 1 && R->groups <= 64 && R->E % R->groups == 0, MOE_EINVAL,
          "%s: groups=%d must be 1..64 and divide E=%d", who, R->groups, R->E);
  REQUIRE(R->topk_groups >= 1 && R->topk_groups <= R->groups, MOE_EINVAL,
          "%s: topk_groups=%d outside 1..groups=%d", who, R->topk_groups, R->groups);
  REQUIRE(R->topk_groups * (R->E / R->groups) >= R->k, MOE_EINVAL,
          "%s: topk_groups=%d groups of %d experts hold fewer than k=%d", who, R->topk_groups,
          R->E / R->groups, R->k);
  REQUIRE(R->group_score == MOE_GROUP_MAX || R->group_score == MOE_GROUP_TOP2, MOE_EINVAL,
          "%s: group_score=%d", who, R->group_score);
  REQUIRE(R->renorm == 0 || R->renorm == 1, MOE_EINVAL, "%s: renorm=%d", who, R->renorm);
  REQUIRE(std::isfinite(R->scale), MOE_EINVAL, "%s: scale must be finite", who);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_route_groups(const moe_router* R, const void* logits, moe_dtype lt, const float* bias, int T,
                            int32_t* ids, float* w, moe_stream_t stream) {
  const moe_status st = check_router(R, "moe_route_groups");
  if (st != MOE_OK) return st;
  REQUIRE(is_dtype(lt), MOE_EINVAL, "moe_route_groups: bad dtype %d", (int)lt);
  REQUIRE(T >= 0 && T <= kMaxTokens, MOE_ESHAPE, "moe_route_groups: T=%d outside 0..2^20", T);
  if (T == 0) return MOE_OK;
  REQUIRE(logits && ids && w, MOE_EINVAL, "moe_route_groups: NULL pointer");
  REQUIRE(aligned(logits, dsize(lt)) && aligned(bias, 4) && aligned(ids, 4) && aligned(w, 4), MOE_EINVAL,
          "moe_route_groups: pointers must be aligned to their element");
  const Buffer in{logits, (size_t)T * R->E * dsize(lt)}, b{bias, (size_t)R->E * 4};
  const Buffer oi{ids, (size_t)T * R->k * 4}, ow{w, (size_t)T * R->k * 4};
  REQUIRE(!overlap(oi, ow) && !overlap(oi, in) && !overlap(ow, in) && !overlap(oi, b) && !overlap(ow, b), MOE_EINVAL,
          "moe_route_groups: ids and w may overlap neither each other nor an input");
  return launch_route_groups(R, logits, lt, bias, T, ids, w, (hipStream_t)stream);
}

moe_status moe_norm_in(const moe_norm* norm, const void* x, moe_dtype xt, int T, void* out, moe_dtype ot,
                       moe_stream_t stream) {
  const moe_status st = check_norm(norm, "moe_norm_in");
  if (st != MOE_OK) return st;
  REQUIRE(is_dtype(xt) && is_dtype(ot), MOE_EINVAL, "moe_norm_in: bad dtype %d or %d", (int)xt, (int)ot);
  REQUIRE(T >= 0 && T <= kMaxTokens, MOE_ESHAPE, "moe_norm_in: T=%d outside 0..2^20", T);
  if (T == 0) return MOE_OK;
  REQUIRE(x && out, MOE_EINVAL, "moe_norm_in: NULL pointer");
  REQUIRE(aligned(x, dsize(xt)) && aligned(out, dsize(ot)), MOE_EINVAL,
          "moe_norm_in: pointers must be aligned to their element");
  REQUIRE(x != out || xt == ot, MOE_EINVAL, "moe_norm_in: out may be x only where their types are equal");
  const size_t n = (size_t)T * norm->H;
  const Buffer o{out, n * dsize(ot)};
  REQUIRE(!overlap_part(o, {x, n * dsize(xt)}) && !overlap(o, {norm->pre_w, norm->H * dsize(norm->wt)}), MOE_EINVAL,
          "moe_norm_in: out may be x, but overlap no input otherwise");
  return launch_norm_in(norm, x, xt, T, out, ot, (hipStream_t)stream);
}

moe_status moe_norm_out(const moe_norm* norm, const void* y, moe_dtype yt, const void* residual, const void* gate,
                        moe_dtype gt, int T, void* out, moe_dtype rt, const moe_norm* next, void* next_out,
                        moe_dtype nt, moe_stream_t stream) {
  moe_status st = check_norm(norm, "moe_norm_out");
  if (st != MOE_OK) return st;
  if (next && (st = check_norm(next, "moe_norm_out (next)")) != MOE_OK) return st;
  REQUIRE(!next == !next_out, MOE_EINVAL, "moe_norm_out: next and next_out must both be given or both be NULL");
  REQUIRE(!next || next->H == norm->H, MOE_ESHAPE, "moe_norm_out: next norm has H=%d, not %d", next ? next->H : 0,
          norm->H);
  REQUIRE(is_dtype(yt) && is_dtype(rt) && (!next || is_dtype(nt)) && (norm->gate == MOE_GATE_NONE || is_dtype(gt)),
          MOE_EINVAL, "moe_norm_out: bad dtype (y %d, residual %d, gate %d, next %d)", (int)yt, (int)rt, (int)gt,
          (int)nt);
  REQUIRE(T >= 0 && T <= kMaxTokens, MOE_ESHAPE, "moe_norm_out: T=%d outside 0..2^20", T);
  if (T == 0) return MOE_OK;
  REQUIRE(y && residual && out, MOE_EINVAL, "moe_norm_out: NULL pointer");
  REQUIRE((norm->gate == MOE_GATE_NONE) == !gate, MOE_EINVAL, "moe_norm_out: gate=%d needs %s gate pointer",
          norm->gate, norm->gate == MOE_GATE_NONE ? "no" : "a");
  REQUIRE(aligned(y, dsize(yt)) && aligned(residual, dsize(rt)) && aligned(out, dsize(rt)) &&
              (!gate || aligned(gate, dsize(gt))) && (!next || aligned(next_out, dsize(nt))),
          MOE_EINVAL, "moe_norm_out: pointers must be aligned to their element");
  REQUIRE(out != next_out, MOE_EINVAL, "moe_norm_out: out and next_out are the same buffer");
  REQUIRE((out != y || yt == rt) && (!next || ((next_out != y || yt == nt) && (next_out != residual || rt == nt))),
          MOE_EINVAL, "moe_norm_out: an output may be an input's buffer only where their types are equal");
  REQUIRE(!gate || (gate != out && gate != next_out), MOE_EINVAL, "moe_norm_out: gate may not be an output's buffer");
  const size_t n = (size_t)T * norm->H;
  const size_t gates = norm->gate == MOE_GATE_CHANNEL ? norm->H : norm->gate == MOE_GATE_TOKEN ? T : n;
  const Buffer outs[2] = {{out, n * dsize(rt)}, {next_out, n * dsize(nt)}};
  for (const Buffer& o : outs)
    REQUIRE(!overlap_part(o, {y, n * dsize(yt)}) && !overlap_part(o, {residual, n * dsize(rt)}) &&
                !overlap(o, {gate, gates * dsize(gt)}) && !overlap(o, {norm->post_w, norm->H * dsize(norm->wt)}) &&
                (!next || !overlap(o, {next->pre_w, norm->H * dsize(next->wt)})),
            MOE_EINVAL, "moe_norm_out: an output may be y's or residual's buffer, but overlap no input otherwise");
  REQUIRE(!overlap(outs[0], outs[1]), MOE_EINVAL, "moe_norm_out: out and next_out overlap");
  return launch_norm_out(norm, y, yt, residual, gate, gt, T, out, rt, next, next_out, nt, (hipStream_t)stream);
}

moe_status moe_lora_add(const moe_lora* L, const void* x, moe_dtype xt, int T, const int32_t* adapter_ids,
                        const void* base, void* out, moe_dtype yt, moe_stream_t stream) {
  REQUIRE(L, MOE_EINVAL, "moe_lora_add: lora is NULL");
  REQUIRE(L->K >= 1 && L->K <= 65536 && L->N >= 1 && L->N <= 65536, MOE_ESHAPE,
          "moe_lora_add: K=%d N=%d outside 1..65536", L->K, L->N);
  REQUIRE(L->r >= 1 && L->r <= 128, MOE_ESHAPE, "moe_lora_add: r=%d outside 1..128", L->r);
  REQUIRE(L->num >= 0 && L->num <= 65536, MOE_ESHAPE, "moe_lora_add: num=%d outside 0..65536", L->num);
  REQUIRE(L->num == 0 || (L->a && L->b), MOE_EINVAL, "moe_lora_add: the bank is NULL with num=%d", L->num);
  REQUIRE(aligned(L->a, 2) && aligned(L->b, 2) && aligned(L->scale, 4) && aligned(L->ranks, 4), MOE_EINVAL,
          "moe_lora_add: the bank must be aligned to its elements");
  REQUIRE(is_dtype(xt) && is_dtype(yt), MOE_EINVAL, "moe_lora_add: bad dtype %d or %d", (int)xt, (int)yt);
  REQUIRE(T >= 0 && T <= kMaxTokens, MOE_ESHAPE, "moe_lora_add: T=%d outside 0..2^20", T);
  if (T == 0) return MOE_OK;
  REQUIRE(x && adapter_ids && out, MOE_EINVAL, "moe_lora_add: NULL pointer");
  REQUIRE(aligned(x, dsize(xt)) && aligned(adapter_ids, 4) && aligned(base, dsize(yt)) && aligned(out, dsize(yt)),
          MOE_EINVAL, "moe_lora_add: pointers must be aligned to their element");
  REQUIRE(x != out, MOE_EINVAL, "moe_lora_add: out may not be x");
  const size_t N = (size_t)L->N, K = (size_t)L->K, r = (size_t)L->r, num = (size_t)L->num;
  const Buffer o{out, T * N * dsize(yt)};
  REQUIRE(!overlap_part(o, {base, T * N * dsize(yt)}) && !overlap(o, {x, T * K * dsize(xt)}) &&
              !overlap(o, {adapter_ids, (size_t)T * 4}) && !overlap(o, {L->a, num * r * K * 2}) &&
              !overlap(o, {L->b, num * N * r * 2}) && !overlap(o, {L->scale, num * 4}) && !overlap(o, {L->ranks, num * 4}),
          MOE_EINVAL, "moe_lora_add: out may be base, but overlap no input otherwise");
  return launch_lora(L, x, xt, T, adapter_ids, base, out, yt, (hipStream_t)stream);
}

}  // extern "C"

// ------------------------------------------------------------ to the experts and back

namespace {

constexpr int kMaxPairs = 1 << 20;  // pairs of a sort, as moe_group's keys, and sorted rows
constexpr int kMaxWidth = 65536;

// the sizes of moe_unpermute and its gradient
moe_status check_rows(int T, int k, int H, int M, const char* who) {
  REQUIRE(T >= 0 && T <= kMaxTokens, MOE_ESHAPE, "%s: T=%d outside 0..2^20", who, T);
  REQUIRE(k >= 1 && k <= 64, MOE_EINVAL, "%s: k=%d outside 1..64", who, k);
  REQUIRE(H >= 1 && H <= kMaxWidth, MOE_ESHAPE, "%s: H=%d outside 1..65536", who, H);
  REQUIRE(M >= 0 && M <= kMaxPairs, MOE_ESHAPE, "%s: M=%d outside 0..2^20", who, M);
  return MOE_OK;
}

bool pairs_ok(int T, int k, int E) {
  return T >= 0 && k >= 1 && k <= 64 && (long)T * k <= kMaxPairs && E >= 1 && E <= 1024;
}

moe_status check_q4(const moe_q4* q, const char* who) {
  REQUIRE(q, MOE_EINVAL, "%s: q4 is NULL", who);
  REQUIRE(q->K >= 32 && q->K <= kMaxWidth && q->K % 32 == 0 && q->N >= 1 && q->N <= kMaxWidth, MOE_ESHAPE,
          "%s: K=%d must be a multiple of 32 up to 65536 and N=%d lie in 1..65536", who, q->K, q->N);
  REQUIRE(q->num >= 1 && q->num <= 1024, MOE_ESHAPE, "%s: num=%d outside 1..1024", who, q->num);
  REQUIRE(q->group >= 32 && q->group % 32 == 0 && q->K % q->group == 0, MOE_ESHAPE,
          "%s: group=%d must be a multiple of 32 that divides K=%d", who, q->group, q->K);
  REQUIRE(q->code == MOE_Q4_INT4 || q->code == MOE_Q4_FP4, MOE_EINVAL, "%s: code=%d", who, q->code);
  REQUIRE(q->act == MOE_Q4_LINEAR || q->act == MOE_Q4_SWIGLU, MOE_EINVAL, "%s: act=%d", who, q->act);
  REQUIRE(is_dtype(q->st) || q->st == MOE_SCALE_E8M0, MOE_EINVAL, "%s: bad scale type %d", who, (int)q->st);
  REQUIRE(q->codes && q->scales, MOE_EINVAL, "%s: codes or scales are NULL", who);
  REQUIRE(!q->zeros || q->code == MOE_Q4_INT4, MOE_EINVAL, "%s: zero points belong to integer codes", who);
  const size_t ss = q->st == MOE_SCALE_E8M0 ? 1 : dsize(q->st);
  REQUIRE(aligned(q->codes, 16) && aligned(q->scales, ss), MOE_EINVAL,
          "%s: codes must be 16-byte aligned, scales aligned to their element", who);
  const size_t R = (size_t)q->N * (q->act == MOE_Q4_SWIGLU ? 2 : 1), n = R * (q->K / q->group);
  REQUIRE(q->num == 1 || (q->code_stride >= R * (q->K / 2) && q->code_stride % 16 == 0), MOE_EINVAL,
          "%s: code_stride=%zu must be >= %zu and a multiple of 16", who, q->code_stride, R * (q->K / 2));
  REQUIRE(q->num == 1 || (q->scale_stride >= n * ss && q->scale_stride % ss == 0), MOE_EINVAL,
          "%s: scale_stride=%zu must be >= %zu and a multiple of the scales' element", who, q->scale_stride, n * ss);
  REQUIRE(q->num == 1 || !q->zeros || q->zero_stride >= n, MOE_EINVAL, "%s: zero_stride=%zu must be >= %zu", who,
          q->zero_stride, n);
  return MOE_OK;
}

// the buffers of a product of T rows; offsets NULL: one matrix
moe_status check_q4_call(const moe_q4* q, const void* x, moe_dtype xt, int T, const int32_t* offsets, const void* y,
                         moe_dtype yt, const char* who) {
  REQUIRE(x && y, MOE_EINVAL, "%s: NULL pointer", who);
  REQUIRE(aligned(x, dsize(xt)) && aligned(y, dsize(yt)) && aligned(offsets, 4), MOE_EINVAL,
          "%s: pointers must be aligned to their element", who);
  const size_t R = (size_t)q->N * (q->act == MOE_Q4_SWIGLU ? 2 : 1), n = R * (q->K / q->group), last = q->num - 1;
  const size_t ss = q->st == MOE_SCALE_E8M0 ? 1 : dsize(q->st);
  const Buffer o{y, (size_t)T * q->N * dsize(yt)};
  REQUIRE(!overlap(o, {x, (size_t)T * q->K * dsize(xt)}) && !overlap(o, {offsets, (q->num + 1) * (size_t)4}) &&
              !overlap(o, {q->codes, last * q->code_stride + R * (q->K / 2)}) &&
              !overlap(o, {q->scales, last * q->scale_stride + n * ss}) &&
              !overlap(o, {q->zeros, last * q->zero_stride + n}),
          MOE_EINVAL, "%s: y may overlap no input", who);
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_permute_scratch_bytes(int T, int k, int E) { return pairs_ok(T, k, E) ? permute_scratch_bytes(T, k, E) : 0; }

moe_status moe_permute(const void* x, moe_dtype xt, int T, int k, int H, int E, const int32_t* ids, void* xs,
                       int32_t* offsets, int32_t* perm, int32_t* rows, void* scratch, size_t scratch_bytes,
                       moe_stream_t stream) {
  REQUIRE(k >= 1 && k <= 64, MOE_EINVAL, "moe_permute: k=%d outside 1..64", k);
  REQUIRE(T >= 0 && (long)T * k <= kMaxPairs, MOE_ESHAPE, "moe_permute: T=%d, k=%d: T*k outside 0..2^20", T, k);
  REQUIRE(E >= 1 && E <= 1024, MOE_ESHAPE, "moe_permute: E=%d outside 1..1024", E);
  REQUIRE(!x == !xs, MOE_EINVAL, "moe_permute: x and xs must both be given or both be NULL");
  REQUIRE(!x || (H >= 1 && H <= kMaxWidth), MOE_ESHAPE, "moe_permute: H=%d outside 1..65536", H);
  REQUIRE(!x || is_dtype(xt), MOE_EINVAL, "moe_permute: bad dtype %d", (int)xt);
  REQUIRE(offsets && (T == 0 || (ids && perm && rows)), MOE_EINVAL, "moe_permute: NULL pointer");
  const size_t P = (size_t)T * k, need = permute_scratch_bytes(T, k, E);
  REQUIRE((!x || (aligned(x, dsize(xt)) && aligned(xs, dsize(xt)))) && aligned(ids, 4) && aligned(offsets, 4) &&
              aligned(perm, 4) && aligned(rows, 4) && aligned(scratch, 4),
          MOE_EINVAL, "moe_permute: pointers must be aligned to their element");
  REQUIRE(need == 0 || (scratch && scratch_bytes >= need), MOE_ENOMEM, "moe_permute: scratch %zu bytes < %zu needed",
          scratch ? scratch_bytes : (size_t)0, need);
  const Buffer in[2] = {{x, x ? (size_t)T * H * dsize(xt) : 0}, {ids, P * 4}};
  const Buffer outs[5] = {{xs, x ? P * H * dsize(xt) : 0}, {offsets, (E + 1) * (size_t)4}, {perm, P * 4}, {rows, P * 4},
                          {need ? scratch : nullptr, need}};
  for (int i = 0; i < 5; ++i) {
    for (const Buffer& b : in)
      REQUIRE(!overlap(outs[i], b), MOE_EINVAL, "moe_permute: an output or the scratch overlaps an input");
    for (int j = 0; j < i; ++j)
      REQUIRE(!overlap(outs[i], outs[j]), MOE_EINVAL, "moe_permute: outputs and scratch may not overlap each other");
  }
  return launch_permute(x, xt, T, k, H, E, ids, xs, offsets, perm, rows, (int32_t*)scratch, (hipStream_t)stream);
}

moe_status moe_unpermute(const void* ys, moe_dtype yt, int M, const int32_t* rows, const float* w, const void* base,
                         int T, int k, int H, void* out, moe_dtype ot, moe_stream_t stream) {
  const moe_status st = check_rows(T, k, H, M, "moe_unpermute");
  if (st != MOE_OK) return st;
  REQUIRE(is_dtype(yt) && is_dtype(ot), MOE_EINVAL, "moe_unpermute: bad dtype %d or %d", (int)yt, (int)ot);
  if (T == 0) return MOE_OK;
  REQUIRE((ys || M == 0) && rows && out, MOE_EINVAL, "moe_unpermute: NULL pointer");
  REQUIRE(aligned(ys, dsize(yt)) && aligned(rows, 4) && aligned(w, 4) && aligned(base, dsize(ot)) &&
              aligned(out, dsize(ot)),
          MOE_EINVAL, "moe_unpermute: pointers must be aligned to their element");
  const size_t n = (size_t)T * H, P = (size_t)T * k;
  const Buffer o{out, n * dsize(ot)};
  REQUIRE(!overlap_part(o, {base, n * dsize(ot)}) && !overlap(o, {ys, (size_t)M * H * dsize(yt)}) &&
              !overlap(o, {rows, P * 4}) && !overlap(o, {w, P * 4}),
          MOE_EINVAL, "moe_unpermute: out may be base, but overlap no input otherwise");
  return launch_unpermute(ys, yt, M, rows, w, base, T, k, H, out, ot, (hipStream_t)stream);
}

moe_status moe_unpermute_grad(const void* gout, moe_dtype gt, const void* ys, moe_dtype yt, int M, const int32_t* rows,
                              const float* w, int T, int k, int H, void* gys, float* gw, moe_stream_t stream) {
  const moe_status st = check_rows(T, k, H, M, "moe_unpermute_grad");
  if (st != MOE_OK) return st;
  REQUIRE(is_dtype(gt) && is_dtype(yt), MOE_EINVAL, "moe_unpermute_grad: bad dtype %d or %d", (int)gt, (int)yt);
  if (T == 0 || (!gw && (!gys || M == 0))) return MOE_OK;
  REQUIRE(gout && rows && (!gw || ys || M == 0), MOE_EINVAL, "moe_unpermute_grad: NULL pointer");
  REQUIRE(aligned(gout, dsize(gt)) && aligned(ys, dsize(yt)) && aligned(rows, 4) && aligned(w, 4) &&
              aligned(gys, dsize(yt)) && aligned(gw, 4),
          MOE_EINVAL, "moe_unpermute_grad: pointers must be aligned to their element");
  const size_t P = (size_t)T * k, m = (size_t)M * H * dsize(yt);
  const Buffer g{gout, (size_t)T * H * dsize(gt)}, r{rows, P * 4}, wb{w, P * 4}, y{ys, m}, oy{gys, m}, ow{gw, P * 4};
  REQUIRE(!overlap_part(oy, y) && !overlap(oy, g) && !overlap(oy, r) && !overlap(oy, wb) && !overlap(ow, y) &&
              !overlap(ow, g) && !overlap(ow, r) && !overlap(ow, wb) && !overlap(oy, ow),
          MOE_EINVAL, "moe_unpermute_grad: gys may be ys, but no output may overlap an input or the other otherwise");
  return launch_unpermute_grad(gout, gt, ys, yt, M, rows, w, T, k, H, gys, gw, (hipStream_t)stream);
}

moe_status moe_route_grad(const moe_router* R, const void* logits, moe_dtype lt, int T, const int32_t* ids,
                          const float* w, const float* gw, void* glogits, moe_dtype gt, moe_stream_t stream) {
  const moe_status st = check_router(R, "moe_route_grad");
  if (st != MOE_OK) return st;
  REQUIRE(is_dtype(lt) && is_dtype(gt), MOE_EINVAL, "moe_route_grad: bad dtype %d or %d", (int)lt, (int)gt);
  REQUIRE(T >= 0 && T <= kMaxTokens, MOE_ESHAPE, "moe_route_grad: T=%d outside 0..2^20", T);
  if (T == 0) return MOE_OK;
  REQUIRE(logits && ids && w && gw && glogits, MOE_EINVAL, "moe_route_grad: NULL pointer");
  REQUIRE(aligned(logits, dsize(lt)) && aligned(ids, 4) && aligned(w, 4) && aligned(gw, 4) && aligned(glogits, dsize(gt)),
          MOE_EINVAL, "moe_route_grad: pointers must be aligned to their element");
  const size_t n = (size_t)T * R->E, P = (size_t)T * R->k * 4;
  const Buffer o{glogits, n * dsize(gt)};
  REQUIRE(!overlap(o, {logits, n * dsize(lt)}) && !overlap(o, {ids, P}) && !overlap(o, {w, P}) && !overlap(o, {gw, P}),
          MOE_EINVAL, "moe_route_grad: glogits may overlap no input");
  return launch_route_grad(R, logits, lt, T, ids, w, gw, glogits, gt, (hipStream_t)stream);
}

moe_status moe_q4_linear(const moe_q4* q, const void* x, moe_dtype xt, int T, void* y, moe_dtype yt,
                         moe_stream_t stream) {
  moe_status st = check_q4(q, "moe_q4_linear");
  if (st != MOE_OK) return st;
  REQUIRE(is_dtype(xt) && is_dtype(yt), MOE_EINVAL, "moe_q4_linear: bad dtype %d or %d", (int)xt, (int)yt);
  REQUIRE(T >= 0 && T <= kMaxTokens, MOE_ESHAPE, "moe_q4_linear: T=%d outside 0..2^20", T);
  if (T == 0) return MOE_OK;
  if ((st = check_q4_call(q, x, xt, T, nullptr, y, yt, "moe_q4_linear")) != MOE_OK) return st;
  return launch_q4(q, x, xt, T, nullptr, y, yt, (hipStream_t)stream);
}

moe_status moe_q4_grouped(const moe_q4* q, const void* x, moe_dtype xt, int P, const int32_t* offsets, void* y,
                          moe_dtype yt, moe_stream_t stream) {
  moe_status st = check_q4(q, "moe_q4_grouped");
  if (st != MOE_OK) return st;
  REQUIRE(is_dtype(xt) && is_dtype(yt), MOE_EINVAL, "moe_q4_grouped: bad dtype %d or %d", (int)xt, (int)yt);
  REQUIRE(P >= 0 && P <= kMaxPairs, MOE_ESHAPE, "moe_q4_grouped: P=%d outside 0..2^20", P);
  if (P == 0) return MOE_OK;
  REQUIRE(offsets, MOE_EINVAL, "moe_q4_grouped: NULL pointer");
  if ((st = check_q4_call(q, x, xt, P, offsets, y, yt, "moe_q4_grouped")) != MOE_OK) return st;
  return launch_q4(q, x, xt, P, offsets, y, yt, (hipStream_t)stream);
}

}  // extern "C"
