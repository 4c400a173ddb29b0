// C-ABI entry points of libmoe.so: argument checks, workspace layout, launch
// order.  Every check runs before the first launch, so a rejected call writes
// nothing.  No entry point allocates, frees, synchronises or keeps state.
#include <math.h>

#include <initializer_list>
#include <mutex>

#include "moe_common.h"

namespace {

using moe::ActParams;

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool dtype_ok(int d) { return d == MOE_F32 || d == MOE_BF16; }
inline size_t dsize(int d) { return d == MOE_BF16 ? 2 : 4; }
// moe_combine sees no expert count: the size check takes the largest one
constexpr int32_t kCombineAnyExperts = moe::kMaxExperts;

// Sizes shared by all entry points.  An expert-parallel share may hold fewer
// experts than a token selects (k_le_e = false for its expert count).
moe_status_t check_sizes(int64_t n, int32_t e, int32_t k, bool k_le_e = true) {
  if (n < 0 || e < 1 || e > moe::kMaxExperts || k < 1 || k > moe::kMaxTopk || (k_le_e && k > e))
    return MOE_ERR_SHAPE;
  if (n > (int64_t)0x7fffffff / k) return MOE_ERR_SHAPE;
  return MOE_OK;
}

moe_status_t check_ffn_sizes(int32_t hidden, int32_t inter) {
  if (hidden < 8 || inter < 8 || hidden % 8 || inter % 8) return MOE_ERR_SHAPE;
  if (hidden > (1 << 24) || inter > (1 << 24)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

size_t experts_ws_bytes(int64_t n, int32_t k, int32_t hidden, int32_t inter, int dt) {
  const size_t m = (size_t)n * k;
  size_t b = align256(m * inter * dsize(dt));  // activation rows a[M, inter]
  if (k > 1) b += align256(m * hidden * dsize(dt));  // weighted expert outputs y[M, hidden]
  return b;
}

moe_status_t check_routing_struct(const moe_routing_t *r, bool for_route, int64_t n) {
  if (!r) return MOE_ERR_NULL;
  if (!dtype_ok(r->w_dtype)) return MOE_ERR_DTYPE;
  if (n == 0) return MOE_OK;
  const void *need_exp[] = {r->offsets, r->col_sorted, r->row_sorted, r->gate_scal};
  for (const void *p : need_exp) {
    if (!p) return MOE_ERR_NULL;
    if (!aligned16(p)) return MOE_ERR_ALIGN;
  }
  if (for_route) {
    const void *need_rt[] = {r->topk_idx, r->topk_w, r->bitmatrix, r->col_sum};
    for (const void *p : need_rt) {
      if (!p) return MOE_ERR_NULL;
      if (!aligned16(p)) return MOE_ERR_ALIGN;
    }
  }
  return MOE_OK;
}

moe_status_t act_params(moe_act_t act, moe_w13_layout_t layout, const moe_act_params_t *p,
                        ActParams *out) {
  if (act != MOE_ACT_SILU && act != MOE_ACT_SWIGLU_OAI && act != MOE_ACT_RELU2)
    return MOE_ERR_UNSUPPORTED;
  if (layout != MOE_W13_PACKED && layout != MOE_W13_INTERLEAVED) return MOE_ERR_UNSUPPORTED;
  if (act == MOE_ACT_RELU2 && layout != MOE_W13_PACKED) return MOE_ERR_UNSUPPORTED;
  const uint32_t set = p ? p->set : 0u;
  if (set & ~(MOE_PARAM_ALPHA | MOE_PARAM_BETA | MOE_PARAM_LIMIT)) return MOE_ERR_UNSUPPORTED;
  // unset fields keep the plain-SwiGLU defaults; SiLU reads only the limit
  out->alpha = 1.f;
  out->beta = 0.f;
  out->limit = INFINITY;
  if (act == MOE_ACT_RELU2) return MOE_OK;
  if (set & MOE_PARAM_LIMIT) {
    if (!(p->limit >= 0.f)) return MOE_ERR_SHAPE;  // also rejects NaN
    out->limit = p->limit;
  }
  if (act == MOE_ACT_SWIGLU_OAI) {
    if (set & MOE_PARAM_ALPHA) out->alpha = p->alpha;
    if (set & MOE_PARAM_BETA) out->beta = p->beta;
    if (!isfinite(out->alpha) || !isfinite(out->beta)) return MOE_ERR_SHAPE;
  }
  return MOE_OK;
}

// Checks shared by the expert entry points: sizes, dtype, activation, routing.
moe_status_t check_expert_args(moe_dtype_t dtype, int64_t n, int32_t hidden, int32_t e,
                               int32_t inter, int32_t k, moe_act_t act, moe_w13_layout_t layout,
                               const moe_act_params_t *params, const moe_routing_t *routing,
                               ActParams *prm, bool share = false) {
  moe_status_t st = check_sizes(n, e, k, !share);
  if (st != MOE_OK) return st;
  if ((st = check_ffn_sizes(hidden, inter)) != MOE_OK) return st;
  if (!dtype_ok(dtype)) return MOE_ERR_DTYPE;
  // the GEMMs address one expert's w13 / w2 block, x and the activation rows
  // with 32-bit byte offsets
  const int64_t lim = 0x7fffffff, es = (int64_t)dsize(dtype);
  if ((int64_t)2 * inter * hidden * es > lim || n * hidden * es > lim ||
      n * k * (int64_t)inter * es > lim || n * k * (int64_t)hidden * es > lim)
    return MOE_ERR_SHAPE;
  if ((st = act_params(act, layout, params, prm)) != MOE_OK) return st;
  return check_routing_struct(routing, false, n);
}

moe_status_t check_ptrs(std::initializer_list<const void *> ptrs) {
  for (const void *p : ptrs) {
    if (!p) return MOE_ERR_NULL;
    if (!aligned16(p)) return MOE_ERR_ALIGN;
  }
  return MOE_OK;
}

// Threads of a launch, in whole workgroups of up to 1024.
constexpr int64_t kMostThreads = 0xffffffffLL - 1023;

// Sizes and types of the calls that move rows between token and sorted order.
moe_status_t check_rows(moe_dtype_t dtype, int64_t n, int32_t hidden, int32_t k,
                        const moe_routing_t *routing, bool weights) {
  moe_status_t st = check_sizes(n, kCombineAnyExperts, k, false);
  if (st != MOE_OK) return st;
  if (check_ffn_sizes(hidden, 8) != MOE_OK) return MOE_ERR_SHAPE;
  if (!dtype_ok(dtype)) return MOE_ERR_DTYPE;
  // one thread per 16-byte chunk of a token row, and a grid's threads are counted in 32 bits
  if (n * hidden * (int64_t)dsize(dtype) / 16 > kMostThreads) return MOE_ERR_SHAPE;
  if (!routing) return MOE_ERR_NULL;
  return weights && !dtype_ok(routing->w_dtype) ? MOE_ERR_DTYPE : MOE_OK;
}

// Operands of the block norm, either direction: which of them a call has
// follows from y, w_post, w_pre and the gate.
moe_status_t check_block_norm(const void *x, const void *y, moe_dtype_t dtype, int64_t n,
                              int32_t hidden, const moe_block_norm_t *norm) {
  if (n < 0 || n > 0x7fffffffLL || hidden < 8 || hidden % 8 || hidden > moe::kMaxNormHidden)
    return MOE_ERR_SHAPE;
  if (!dtype_ok(dtype)) return MOE_ERR_DTYPE;
  if (!norm) return MOE_ERR_NULL;
  if (!(norm->eps > 0.f) || !isfinite(norm->eps) || !isfinite(norm->residual_scale))
    return MOE_ERR_SHAPE;
  if (norm->gate_kind != MOE_GATE_NONE && norm->gate_kind != MOE_GATE_TOKEN &&
      norm->gate_kind != MOE_GATE_CHANNEL)
    return MOE_ERR_UNSUPPORTED;
  // a norm or a gate of the block's output needs that output; a call without
  // it must have the norm ahead of a block to do
  if (n > 0 && !y && (norm->w_post || norm->gate_kind != MOE_GATE_NONE || !norm->w_pre))
    return MOE_ERR_NULL;
  if (n > 0 && !x) return MOE_ERR_NULL;
  if (norm->gate_kind != MOE_GATE_NONE && n > 0 && !norm->gate) return MOE_ERR_NULL;
  for (const void *p : {x, y, norm->w_post, norm->w_pre, norm->gate})
    if (!aligned16(p)) return MOE_ERR_ALIGN;
  return MOE_OK;
}

moe::BlockNormArgs block_norm_args(const void *x, const void *y, int64_t n, int32_t hidden,
                                   const moe_block_norm_t *norm) {
  moe::BlockNormArgs g{};
  g.x = x;
  g.y = y;
  g.w_post = norm->w_post;
  g.w_pre = norm->w_pre;
  g.gate = norm->gate;
  g.gate_kind = norm->gate_kind;
  g.n_tokens = n;
  g.hidden = hidden;
  g.residual_scale = norm->residual_scale;
  g.eps = norm->eps;
  return g;
}

moe_status_t check_ws(const void *ws, size_t have, size_t need) {
  if (need == 0) return MOE_OK;
  if (!ws) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_ALIGN;
  return have < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

size_t y_bytes(int64_t n, int32_t k, int32_t hidden, int dt) {
  return k > 1 ? align256((size_t)n * k * hidden * dsize(dt)) : 0;
}

moe_status_t check_experts(const void *x, moe_dtype_t dtype, int64_t n, int32_t hidden,
                           const void *w13, const void *w2, int32_t e, int32_t inter, int32_t k,
                           moe_act_t act, moe_w13_layout_t layout, const moe_act_params_t *params,
                           const moe_routing_t *routing, void *out, void *ws, size_t ws_bytes,
                           ActParams *prm, bool share = false) {
  moe_status_t st = check_expert_args(dtype, n, hidden, e, inter, k, act, layout, params,
                                      routing, prm, share);
  if (st != MOE_OK || n == 0) return st;
  if ((st = check_ptrs({x, w13, w2, out})) != MOE_OK) return st;
  return check_ws(ws, ws_bytes, experts_ws_bytes(n, k, hidden, inter, dtype));
}

moe_status_t check_route(const void *logits, moe_dtype_t dt, int64_t n, int32_t e, int32_t k,
                         const moe_routing_t *out, void *ws, size_t ws_bytes) {
  moe_status_t st = check_sizes(n, e, k);
  if (st != MOE_OK) return st;
  if (!dtype_ok(dt)) return MOE_ERR_DTYPE;
  if ((st = check_routing_struct(out, true, n)) != MOE_OK) return st;
  if (out->w_dtype != dt) return MOE_ERR_DTYPE;  // the weights inherit the gating dtype
  if (n == 0) return MOE_OK;
  if (!logits) return MOE_ERR_NULL;
  if (!aligned16(logits)) return MOE_ERR_ALIGN;
  if (!ws) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_ALIGN;
  if (ws_bytes < moe::route_scratch_bytes(n, e, k)) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

// Router GEMM operands: x [n, hidden], w_gate [e, hidden], logits_out [n, e].
moe_status_t check_gate(const void *x, const void *w_gate, moe_dtype_t dt, int64_t n,
                        int32_t hidden, int32_t e, void *logits_out) {
  if (!dtype_ok(dt)) return MOE_ERR_DTYPE;
  if (hidden < 8 || hidden % 8 || hidden > (1 << 24) || e < 1 || e > moe::kMaxExperts || n < 0)
    return MOE_ERR_SHAPE;
  const int64_t lim = 0x7fffffff, es = (int64_t)dsize(dt);
  if (n * hidden * es > lim || n * e * es > lim || (int64_t)e * hidden * es > lim)
    return MOE_ERR_SHAPE;
  if (n == 0) return MOE_OK;
  return check_ptrs({x, w_gate, logits_out});
}

// The expert-parallel share [lo, lo + nl) must lie inside [0, e).
moe_status_t check_share(int32_t e, int32_t lo, int32_t nl) {
  if (lo < 0 || nl < 1 || lo > e - nl) return MOE_ERR_SHAPE;
  return MOE_OK;
}

hipError_t run_w13(const void *x, moe_dtype_t dtype, int64_t n, int32_t hidden, const void *w13,
                   int32_t e, int32_t inter, int32_t k, moe_act_t act, moe_w13_layout_t layout,
                   const ActParams &prm, const moe_routing_t *r, void *a, hipStream_t s,
                   const void *w13_scale = nullptr) {
  return moe::launch_gemm1(x, w13, a, r->offsets, r->col_sorted, dtype, n, k, e, hidden, inter,
                           act, layout, prm, s, false,
                           reinterpret_cast<const uint8_t *>(w13_scale));
}

hipError_t run_w2(const void *a, moe_dtype_t dtype, int64_t n, int32_t hidden, const void *w2,
                  int32_t e, int32_t inter, int32_t k, const moe_routing_t *r, void *out, void *y,
                  hipStream_t s, bool share = false, bool unit_gate = false,
                  const void *w2_scale = nullptr) {
  const bool direct = k == 1;  // one row per token: GEMM2 writes the output rows itself
  if (!direct && moe::gemm2_combine_fits(dtype, n, k, e, hidden, inter, w2_scale != nullptr))
    return moe::launch_gemm2_combine(a, w2, out, r->offsets, r->row_sorted,
                                     unit_gate ? nullptr : r->gate_scal, (moe_dtype_t)r->w_dtype,
                                     n, k, e, hidden, inter, s,
                                     reinterpret_cast<const uint8_t *>(w2_scale));
  hipError_t err = moe::launch_gemm2(a, w2, direct ? out : y, r->offsets, r->col_sorted,
                                     unit_gate ? nullptr : r->gate_scal,
                                     (moe_dtype_t)r->w_dtype, dtype, n, k, e, hidden, inter,
                                     direct, s, reinterpret_cast<const uint8_t *>(w2_scale));
  if (err != hipSuccess) return err;
  // an expert share leaves the rows of tokens routed elsewhere to be zeroed
  if (direct) return share ? moe::launch_zero_unrouted(r->row_sorted, out, dtype, n, hidden, s)
                           : err;
  return moe::launch_combine(y, r->row_sorted, out, dtype, n, k, hidden, s);
}

moe_status_t run_experts(const void *x, moe_dtype_t dtype, int64_t n, int32_t hidden,
                         const void *w13, const void *w2, int32_t e, int32_t inter, int32_t k,
                         moe_act_t act, moe_w13_layout_t layout, const ActParams &prm,
                         const moe_routing_t *r, void *out, void *ws, hipStream_t s,
                         bool share = false, const void *w13_scale = nullptr,
                         const void *w2_scale = nullptr) {
  // workspace: activation rows a[M, inter], then (topk > 1) weighted rows y[M, hidden]
  char *base = reinterpret_cast<char *>(ws);
  void *a = base;
  void *y = base + align256((size_t)n * k * inter * dsize(dtype));
  if (run_w13(x, dtype, n, hidden, w13, e, inter, k, act, layout, prm, r, a, s, w13_scale) !=
      hipSuccess)
    return MOE_ERR_HIP;
  if (run_w2(a, dtype, n, hidden, w2, e, inter, k, r, out, y, s, share, false, w2_scale) !=
      hipSuccess)
    return MOE_ERR_HIP;
  return MOE_OK;
}

// Scratch of moe_forward_noalloc, for callers that cannot allocate device
// memory: a file-scope device array of MOE_NOALLOC_SCRATCH_BYTES.  Every GPU
// the library runs on holds its own copy, at its own address, until the
// process ends.  In host code the array's name is only a stand-in, never a
// device address: kernels receive the address hipGetSymbolAddress returns for
// the device, resolved once per device with that device current.
constexpr int kMaxDevices = 64;
struct ScratchSlot {
  std::once_flag once;
  void *ptr = nullptr;
  hipError_t err = hipSuccess;
};
ScratchSlot g_scratch[kMaxDevices];

}  // namespace

static __device__ __align__(256) char scratch[MOE_NOALLOC_SCRATCH_BYTES];

namespace {

// Device address of `scratch` on the device that runs stream s (the current
// device for the null stream).  The first call on a device makes that device
// current for the lookup and restores the caller's device.
hipError_t noalloc_scratch(hipStream_t s, void **out) {
  int cur = 0;
  hipError_t e = hipGetDevice(&cur);
  if (e != hipSuccess) return e;
  int dev = cur;
  if (s != nullptr) {
    hipDevice_t d = 0;
    if ((e = hipStreamGetDevice(s, &d)) != hipSuccess) return e;
    dev = (int)d;
  }
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  ScratchSlot &slot = g_scratch[dev];
  std::call_once(slot.once, [&] {
    if (dev != cur && (slot.err = hipSetDevice(dev)) != hipSuccess) return;
    slot.err = hipGetSymbolAddress(&slot.ptr, HIP_SYMBOL(scratch));
    if (dev != cur) {
      const hipError_t back = hipSetDevice(cur);
      if (slot.err == hipSuccess) slot.err = back;
    }
  });
  if (slot.err != hipSuccess) return slot.err;
  *out = slot.ptr;
  return hipSuccess;
}

}  // namespace

extern "C" {

size_t moe_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t topk, int32_t hidden,
                           int32_t inter, moe_dtype_t dtype) {
  if (check_sizes(n_tokens, n_experts, topk) != MOE_OK || !dtype_ok(dtype)) return 0;
  if (inter != 0 && check_ffn_sizes(hidden, inter) != MOE_OK) return 0;
  if (inter == 0 && hidden != 0 && check_ffn_sizes(hidden, 8) != MOE_OK) return 0;
  // routing scratch, plus the router GEMM's when hidden is given; the expert
  // intermediates reuse the same bytes once the routing has run
  const size_t route = moe::route_scratch_bytes(n_tokens, n_experts, topk) +
                       (hidden ? moe::gate_scratch_bytes(n_tokens, n_experts, hidden, dtype) : 0);
  size_t ffn = 0;
  if (inter != 0) ffn = experts_ws_bytes(n_tokens, topk, hidden, inter, dtype);
  const size_t b = route > ffn ? route : ffn;
  return b ? b : 256;
}

moe_status_t moe_route(const void *logits, moe_dtype_t logits_dtype, int64_t n_tokens,
                       int32_t n_experts, int32_t topk, const moe_routing_t *out,
                       void *workspace, size_t ws_bytes, void *stream) {
  moe_status_t st =
      check_route(logits, logits_dtype, n_tokens, n_experts, topk, out, workspace, ws_bytes);
  if (st != MOE_OK || n_tokens == 0) return st;
  if (moe::launch_route(logits, logits_dtype, n_tokens, n_experts, topk, 0, n_experts, out,
                        workspace, (hipStream_t)stream) != hipSuccess)
    return MOE_ERR_HIP;
  return MOE_OK;
}

moe_status_t moe_experts(const void *x, moe_dtype_t dtype, int64_t n_tokens, int32_t hidden,
                         const void *w13, const void *w2, int32_t n_experts, int32_t inter,
                         int32_t topk, moe_act_t act, moe_w13_layout_t layout,
                         const moe_act_params_t *params, const moe_routing_t *routing, void *out,
                         void *workspace, size_t ws_bytes, void *stream) {
  ActParams prm;
  moe_status_t st = check_experts(x, dtype, n_tokens, hidden, w13, w2, n_experts, inter, topk,
                                  act, layout, params, routing, out, workspace, ws_bytes, &prm);
  if (st != MOE_OK || n_tokens == 0) return st;
  return run_experts(x, dtype, n_tokens, hidden, w13, w2, n_experts, inter, topk, act, layout,
                     prm, routing, out, workspace, (hipStream_t)stream);
}

moe_status_t moe_experts_w13(const void *x, moe_dtype_t dtype, int64_t n_tokens, int32_t hidden,
                             const void *w13, int32_t n_experts, int32_t inter, int32_t topk,
                             moe_act_t act, moe_w13_layout_t layout,
                             const moe_act_params_t *params, const moe_routing_t *routing,
                             void *act_out, void *stream) {
  ActParams prm;
  moe_status_t st = check_expert_args(dtype, n_tokens, hidden, n_experts, inter, topk, act,
                                      layout, params, routing, &prm);
  if (st != MOE_OK || n_tokens == 0) return st;
  if ((st = check_ptrs({x, w13, act_out})) != MOE_OK) return st;
  return run_w13(x, dtype, n_tokens, hidden, w13, n_experts, inter, topk, act, layout, prm,
                 routing, act_out, (hipStream_t)stream) == hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

moe_status_t moe_experts_w2(const void *act_in, moe_dtype_t dtype, int64_t n_tokens,
                            int32_t hidden, const void *w2, int32_t n_experts, int32_t inter,
                            int32_t topk, const moe_routing_t *routing, void *out,
                            void *workspace, size_t ws_bytes, void *stream) {
  ActParams prm;
  moe_status_t st = check_expert_args(dtype, n_tokens, hidden, n_experts, inter, topk,
                                      MOE_ACT_SILU, MOE_W13_PACKED, nullptr, routing, &prm);
  if (st != MOE_OK || n_tokens == 0) return st;
  if ((st = check_ptrs({act_in, w2, out})) != MOE_OK) return st;
  if ((st = check_ws(workspace, ws_bytes, y_bytes(n_tokens, topk, hidden, dtype))) != MOE_OK)
    return st;
  return run_w2(act_in, dtype, n_tokens, hidden, w2, n_experts, inter, topk, routing, out,
                workspace, (hipStream_t)stream) == hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

moe_status_t moe_experts_w2_rows(const void *act_in, moe_dtype_t dtype, int64_t n_tokens,
                                 int32_t hidden, const void *w2, int32_t n_experts, int32_t inter,
                                 int32_t topk, const moe_routing_t *routing, void *y_sorted,
                                 void *stream) {
  ActParams prm;
  moe_status_t st = check_expert_args(dtype, n_tokens, hidden, n_experts, inter, topk,
                                      MOE_ACT_SILU, MOE_W13_PACKED, nullptr, routing, &prm, true);
  if (st != MOE_OK || n_tokens == 0) return st;
  if ((st = check_ptrs({act_in, w2, y_sorted})) != MOE_OK) return st;
  return moe::launch_gemm2(act_in, w2, y_sorted, routing->offsets, routing->col_sorted,
                           routing->gate_scal, (moe_dtype_t)routing->w_dtype, dtype, n_tokens,
                           topk, n_experts, hidden, inter, false, (hipStream_t)stream) ==
                 hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

moe_status_t moe_combine(const void *y_sorted, moe_dtype_t dtype, int64_t n_tokens,
                         int32_t hidden, int32_t topk, const moe_routing_t *routing, void *out,
                         void *stream) {
  moe_status_t st = check_sizes(n_tokens, kCombineAnyExperts, topk, false);
  if (st != MOE_OK) return st;
  if (check_ffn_sizes(hidden, 8) != MOE_OK) return MOE_ERR_SHAPE;
  if (!dtype_ok(dtype)) return MOE_ERR_DTYPE;
  // one thread per 16-byte chunk of out: the grid must stay below 2^31 workgroups of 256
  if (n_tokens * hidden * (int64_t)dsize(dtype) / 16 > 0x7fffffffLL * 256) return MOE_ERR_SHAPE;
  if (!routing) return MOE_ERR_NULL;
  if (n_tokens == 0) return MOE_OK;
  if ((st = check_ptrs({y_sorted, routing->row_sorted, out})) != MOE_OK) return st;
  return moe::launch_combine(y_sorted, routing->row_sorted, out, dtype, n_tokens, topk, hidden,
                             (hipStream_t)stream) == hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

moe_status_t moe_dispatch(const void *x, moe_dtype_t dtype, int64_t n_tokens, int32_t hidden,
                          int32_t topk, const moe_routing_t *routing, void *x_sorted,
                          void *stream) {
  moe_status_t st = check_rows(dtype, n_tokens, hidden, topk, routing, false);
  if (st != MOE_OK || n_tokens == 0) return st;
  if ((st = check_ptrs({x, routing->row_sorted, x_sorted})) != MOE_OK) return st;
  return moe::launch_dispatch(x, routing->row_sorted, x_sorted, dtype, n_tokens, topk, hidden,
                              (hipStream_t)stream) == hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

moe_status_t moe_combine_weighted(const void *y_sorted, moe_dtype_t dtype, int64_t n_tokens,
                                  int32_t hidden, int32_t topk, const moe_routing_t *routing,
                                  void *out, void *stream) {
  moe_status_t st = check_rows(dtype, n_tokens, hidden, topk, routing, true);
  if (st != MOE_OK || n_tokens == 0) return st;
  if ((st = check_ptrs({y_sorted, routing->row_sorted, routing->topk_w, out})) != MOE_OK)
    return st;
  return moe::launch_combine_weighted(y_sorted, routing->row_sorted, routing->topk_w,
                                      (moe_dtype_t)routing->w_dtype, out, dtype, n_tokens, topk,
                                      hidden, (hipStream_t)stream) == hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

moe_status_t moe_combine_weighted_backward(const void *d_out, const void *y_sorted,
                                           moe_dtype_t dtype, int64_t n_tokens, int32_t hidden,
                                           int32_t topk, const moe_routing_t *routing,
                                           void *d_y_sorted, float *d_topk_w, void *stream) {
  moe_status_t st = check_rows(dtype, n_tokens, hidden, topk, routing, true);
  if (st != MOE_OK || n_tokens == 0) return st;
  if (n_tokens * 256 > kMostThreads) return MOE_ERR_SHAPE;  // up to four waves a token
  if ((st = check_ptrs({d_out, y_sorted, routing->row_sorted, routing->topk_w, d_y_sorted,
                        d_topk_w})) != MOE_OK)
    return st;
  return moe::launch_combine_weighted_backward(
             d_out, y_sorted, routing->row_sorted, routing->topk_w, (moe_dtype_t)routing->w_dtype,
             d_y_sorted, d_topk_w, dtype, n_tokens, topk, hidden,
             (hipStream_t)stream) == hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

moe_status_t moe_route_backward(const float *d_topk_w, int64_t n_tokens, int32_t n_experts,
                                int32_t topk, const moe_routing_t *routing, void *d_logits,
                                void *stream) {
  moe_status_t st = check_sizes(n_tokens, n_experts, topk);
  if (st != MOE_OK) return st;
  if (n_tokens * n_experts > kMostThreads) return MOE_ERR_SHAPE;
  if (!routing) return MOE_ERR_NULL;
  if (!dtype_ok(routing->w_dtype)) return MOE_ERR_DTYPE;
  if (n_tokens == 0) return MOE_OK;
  if ((st = check_ptrs({d_topk_w, routing->topk_idx, routing->topk_w, d_logits})) != MOE_OK)
    return st;
  return moe::launch_route_backward(d_topk_w, routing->topk_idx, routing->topk_w, d_logits,
                                    (moe_dtype_t)routing->w_dtype, n_tokens, n_experts, topk,
                                    (hipStream_t)stream) == hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

moe_status_t moe_forward(const void *x, const void *logits, moe_dtype_t dtype, int64_t n_tokens,
                         int32_t hidden, const void *w13, const void *w2, int32_t n_experts,
                         int32_t inter, int32_t topk, moe_act_t act, moe_w13_layout_t layout,
                         const moe_act_params_t *params, const moe_routing_t *routing_out,
                         void *out, void *workspace, size_t ws_bytes, void *stream) {
  ActParams prm;
  moe_status_t st = check_route(logits, dtype, n_tokens, n_experts, topk, routing_out, workspace,
                                ws_bytes);
  if (st != MOE_OK) return st;
  st = check_experts(x, dtype, n_tokens, hidden, w13, w2, n_experts, inter, topk, act, layout,
                     params, routing_out, out, workspace, ws_bytes, &prm);
  if (st != MOE_OK || n_tokens == 0) return st;
  hipStream_t s = (hipStream_t)stream;
  // the routing scratch is dead once the routing kernels ran (stream order), so
  // the expert intermediates reuse the same workspace bytes
  if (moe::launch_route(logits, dtype, n_tokens, n_experts, topk, 0, n_experts, routing_out,
                        workspace, s) != hipSuccess)
    return MOE_ERR_HIP;
  return run_experts(x, dtype, n_tokens, hidden, w13, w2, n_experts, inter, topk, act, layout,
                     prm, routing_out, out, workspace, s);
}

moe_status_t moe_forward_noalloc(const void *x, const void *logits, moe_dtype_t dtype,
                                 int64_t n_tokens, int32_t hidden, const void *w13,
                                 const void *w2, int32_t n_experts, int32_t inter, int32_t topk,
                                 moe_act_t act, moe_w13_layout_t layout,
                                 const moe_act_params_t *params, const moe_routing_t *routing_out,
                                 void *out, void *stream) {
  // the sizes must fit the static scratch; checked before anything else
  const size_t need = moe_workspace_bytes(n_tokens, n_experts, topk, hidden, inter, dtype);
  if (need == 0) return check_sizes(n_tokens, n_experts, topk) != MOE_OK ? MOE_ERR_SHAPE
                        : !dtype_ok(dtype)                            ? MOE_ERR_DTYPE
                                                                      : MOE_ERR_SHAPE;
  if (need > (size_t)MOE_NOALLOC_SCRATCH_BYTES) return MOE_ERR_SCRATCH;
  // every check of moe_forward, with a stand-in for the workspace (never
  // dereferenced by the checks) of the scratch's size
  void *const ws_stand_in = reinterpret_cast<void *>((uintptr_t)256);
  ActParams prm;
  moe_status_t st = check_route(logits, dtype, n_tokens, n_experts, topk, routing_out,
                                ws_stand_in, MOE_NOALLOC_SCRATCH_BYTES);
  if (st != MOE_OK) return st;
  st = check_experts(x, dtype, n_tokens, hidden, w13, w2, n_experts, inter, topk, act, layout,
                     params, routing_out, out, ws_stand_in, MOE_NOALLOC_SCRATCH_BYTES, &prm);
  if (st != MOE_OK || n_tokens == 0) return st;
  hipStream_t s = (hipStream_t)stream;
  void *ws = nullptr;
  if (noalloc_scratch(s, &ws) != hipSuccess) return MOE_ERR_HIP;
  // the same launches as moe_forward, into this GPU's copy of the scratch
  if (moe::launch_route(logits, dtype, n_tokens, n_experts, topk, 0, n_experts, routing_out, ws,
                        s) != hipSuccess)
    return MOE_ERR_HIP;
  return run_experts(x, dtype, n_tokens, hidden, w13, w2, n_experts, inter, topk, act, layout,
                     prm, routing_out, out, ws, s);
}

moe_status_t moe_route_ep(const void *logits, moe_dtype_t logits_dtype, int64_t n_tokens,
                          int32_t n_experts, int32_t topk, int32_t local_offset, int32_t n_local,
                          const moe_routing_t *out, void *workspace, size_t ws_bytes,
                          void *stream) {
  moe_status_t st = check_share(n_experts, local_offset, n_local);
  if (st != MOE_OK) return st;
  st = check_route(logits, logits_dtype, n_tokens, n_experts, topk, out, workspace, ws_bytes);
  if (st != MOE_OK || n_tokens == 0) return st;
  if (moe::launch_route(logits, logits_dtype, n_tokens, n_experts, topk, local_offset, n_local,
                        out, workspace, (hipStream_t)stream) != hipSuccess)
    return MOE_ERR_HIP;
  return MOE_OK;
}

moe_status_t moe_experts_ep(const void *x, moe_dtype_t dtype, int64_t n_tokens, int32_t hidden,
                            const void *w13, const void *w2, int32_t n_local, int32_t inter,
                            int32_t topk, moe_act_t act, moe_w13_layout_t layout,
                            const moe_act_params_t *params, const moe_routing_t *routing,
                            void *out, void *workspace, size_t ws_bytes, void *stream) {
  ActParams prm;
  moe_status_t st = check_experts(x, dtype, n_tokens, hidden, w13, w2, n_local, inter, topk, act,
                                  layout, params, routing, out, workspace, ws_bytes, &prm, true);
  if (st != MOE_OK || n_tokens == 0) return st;
  return run_experts(x, dtype, n_tokens, hidden, w13, w2, n_local, inter, topk, act, layout, prm,
                     routing, out, workspace, (hipStream_t)stream, true);
}

moe_status_t moe_forward_ep(const void *x, const void *logits, moe_dtype_t dtype,
                            int64_t n_tokens, int32_t hidden, const void *w13, const void *w2,
                            int32_t n_experts, int32_t local_offset, int32_t n_local,
                            int32_t inter, int32_t topk, moe_act_t act, moe_w13_layout_t layout,
                            const moe_act_params_t *params, const moe_routing_t *routing_out,
                            void *out, void *workspace, size_t ws_bytes, void *stream) {
  ActParams prm;
  moe_status_t st = check_share(n_experts, local_offset, n_local);
  if (st != MOE_OK) return st;
  st = check_route(logits, dtype, n_tokens, n_experts, topk, routing_out, workspace, ws_bytes);
  if (st != MOE_OK) return st;
  st = check_experts(x, dtype, n_tokens, hidden, w13, w2, n_local, inter, topk, act, layout,
                     params, routing_out, out, workspace, ws_bytes, &prm, true);
  if (st != MOE_OK || n_tokens == 0) return st;
  hipStream_t s = (hipStream_t)stream;
  if (moe::launch_route(logits, dtype, n_tokens, n_experts, topk, local_offset, n_local,
                        routing_out, workspace, s) != hipSuccess)
    return MOE_ERR_HIP;
  return run_experts(x, dtype, n_tokens, hidden, w13, w2, n_local, inter, topk, act, layout, prm,
                     routing_out, out, workspace, s, true);
}

moe_status_t moe_gate_route(const void *x, const void *w_gate, moe_dtype_t dtype,
                            int64_t n_tokens, int32_t hidden, int32_t n_experts, int32_t topk,
                            void *logits_out, const moe_routing_t *out, void *workspace,
                            size_t ws_bytes, void *stream) {
  moe_status_t st = check_gate(x, w_gate, dtype, n_tokens, hidden, n_experts, logits_out);
  if (st != MOE_OK) return st;
  st = check_route(logits_out, dtype, n_tokens, n_experts, topk, out, workspace, ws_bytes);
  if (st != MOE_OK || n_tokens == 0) return st;
  if (ws_bytes < moe::route_scratch_bytes(n_tokens, n_experts, topk) +
                     moe::gate_scratch_bytes(n_tokens, n_experts, hidden, dtype))
    return MOE_ERR_WORKSPACE;
  if (moe::launch_route(logits_out, dtype, n_tokens, n_experts, topk, 0, n_experts, out,
                        workspace, (hipStream_t)stream, x, w_gate, hidden) != hipSuccess)
    return MOE_ERR_HIP;
  return MOE_OK;
}

moe_status_t moe_gate_forward(const void *x, const void *w_gate, moe_dtype_t dtype,
                              int64_t n_tokens, int32_t hidden, const void *w13, const void *w2,
                              int32_t n_experts, int32_t inter, int32_t topk, moe_act_t act,
                              moe_w13_layout_t layout, const moe_act_params_t *params,
                              void *logits_out, const moe_routing_t *routing_out, void *out,
                              void *workspace, size_t ws_bytes, void *stream) {
  ActParams prm;
  moe_status_t st = check_gate(x, w_gate, dtype, n_tokens, hidden, n_experts, logits_out);
  if (st != MOE_OK) return st;
  st = check_route(logits_out, dtype, n_tokens, n_experts, topk, routing_out, workspace,
                   ws_bytes);
  if (st != MOE_OK) return st;
  st = check_experts(x, dtype, n_tokens, hidden, w13, w2, n_experts, inter, topk, act, layout,
                     params, routing_out, out, workspace, ws_bytes, &prm);
  if (st != MOE_OK || n_tokens == 0) return st;
  if (ws_bytes < moe::route_scratch_bytes(n_tokens, n_experts, topk) +
                     moe::gate_scratch_bytes(n_tokens, n_experts, hidden, dtype))
    return MOE_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  if (moe::launch_route(logits_out, dtype, n_tokens, n_experts, topk, 0, n_experts, routing_out,
                        workspace, s, x, w_gate, hidden) != hipSuccess)
    return MOE_ERR_HIP;
  return run_experts(x, dtype, n_tokens, hidden, w13, w2, n_experts, inter, topk, act, layout,
                     prm, routing_out, out, workspace, s);
}

moe_status_t moe_experts_weighted_input(const void *x, moe_dtype_t dtype, int64_t n_tokens,
                                        int32_t hidden, const void *w13, const void *w2,
                                        int32_t n_experts, int32_t inter, int32_t topk,
                                        moe_act_t act, moe_w13_layout_t layout,
                                        const moe_act_params_t *params,
                                        const moe_routing_t *routing, void *out, void *workspace,
                                        size_t ws_bytes, void *stream) {
  ActParams prm;
  moe_status_t st = check_expert_args(dtype, n_tokens, hidden, n_experts, inter, topk, act,
                                      layout, params, routing, &prm);
  if (st != MOE_OK || n_tokens == 0) return st;
  if ((st = check_ptrs({x, w13, w2, out})) != MOE_OK) return st;
  const size_t base = experts_ws_bytes(n_tokens, topk, hidden, inter, dtype);
  const size_t xs_bytes = align256((size_t)n_tokens * topk * hidden * dsize(dtype));
  if ((st = check_ws(workspace, ws_bytes, base + xs_bytes)) != MOE_OK) return st;
  // workspace: a[M, inter], (topk > 1) y[M, hidden], then the scaled rows xs[M, hidden]
  hipStream_t s = (hipStream_t)stream;
  char *ws = reinterpret_cast<char *>(workspace);
  void *a = ws;
  void *y = ws + align256((size_t)n_tokens * topk * inter * dsize(dtype));
  void *xs = ws + base;
  if (moe::launch_scale_gather(x, routing->col_sorted, routing->gate_scal,
                               (moe_dtype_t)routing->w_dtype, routing->offsets, n_experts, dtype,
                               n_tokens, topk, hidden, xs, s) != hipSuccess ||
      moe::launch_gemm1(xs, w13, a, routing->offsets, routing->col_sorted, dtype, n_tokens, topk,
                        n_experts, hidden, inter, act, layout, prm, s, true) != hipSuccess ||
      run_w2(a, dtype, n_tokens, hidden, w2, n_experts, inter, topk, routing, out, y, s, false,
             true) != hipSuccess)
    return MOE_ERR_HIP;
  return MOE_OK;
}

moe_status_t moe_quantize_mxfp4(const void *w, moe_dtype_t dtype, int32_t n_experts,
                                int32_t rows, int32_t k, void *q, void *scales, void *stream) {
  if (!dtype_ok(dtype)) return MOE_ERR_DTYPE;
  if (n_experts < 1 || rows < 1 || k < 32 || k % 32 || k > (1 << 24)) return MOE_ERR_SHAPE;
  if ((int64_t)n_experts * rows * k * (int64_t)dsize(dtype) > 0x7fffffffLL * 8)
    return MOE_ERR_SHAPE;
  moe_status_t st = check_ptrs({w, q});
  if (st != MOE_OK) return st;
  if (!scales) return MOE_ERR_NULL;
  return moe::launch_quantize_mxfp4(w, dtype, n_experts, rows, k, q, scales,
                                    (hipStream_t)stream) == hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

namespace {
// MXFP4 weights: bf16 layer, K of both GEMMs (hidden, inter) a multiple of 32,
// codes and scales present and 16-byte aligned.
moe_status_t check_mxfp4(moe_dtype_t dtype, int32_t hidden, int32_t inter, const void *w13_s,
                         const void *w2_s) {
  if (dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (hidden % 32 || inter % 32) return MOE_ERR_SHAPE;
  return check_ptrs({w13_s, w2_s});
}
}  // namespace

moe_status_t moe_experts_mxfp4(const void *x, moe_dtype_t dtype, int64_t n_tokens,
                               int32_t hidden, const void *w13_q, const void *w13_s,
                               const void *w2_q, const void *w2_s, int32_t n_experts,
                               int32_t inter, int32_t topk, moe_act_t act,
                               moe_w13_layout_t layout, const moe_act_params_t *params,
                               const moe_routing_t *routing, void *out, void *workspace,
                               size_t ws_bytes, void *stream) {
  ActParams prm;
  moe_status_t st = check_experts(x, dtype, n_tokens, hidden, w13_q, w2_q, n_experts, inter,
                                  topk, act, layout, params, routing, out, workspace, ws_bytes,
                                  &prm);
  if (st != MOE_OK) return st;
  if ((st = check_mxfp4(dtype, hidden, inter, w13_s, w2_s)) != MOE_OK || n_tokens == 0)
    return st;
  return run_experts(x, dtype, n_tokens, hidden, w13_q, w2_q, n_experts, inter, topk, act, layout,
                     prm, routing, out, workspace, (hipStream_t)stream, false, w13_s, w2_s);
}

moe_status_t moe_forward_mxfp4(const void *x, const void *logits, moe_dtype_t dtype,
                               int64_t n_tokens, int32_t hidden, const void *w13_q,
                               const void *w13_s, const void *w2_q, const void *w2_s,
                               int32_t n_experts, int32_t inter, int32_t topk, moe_act_t act,
                               moe_w13_layout_t layout, const moe_act_params_t *params,
                               const moe_routing_t *routing_out, void *out, void *workspace,
                               size_t ws_bytes, void *stream) {
  ActParams prm;
  moe_status_t st = check_route(logits, dtype, n_tokens, n_experts, topk, routing_out, workspace,
                                ws_bytes);
  if (st != MOE_OK) return st;
  st = check_experts(x, dtype, n_tokens, hidden, w13_q, w2_q, n_experts, inter, topk, act,
                     layout, params, routing_out, out, workspace, ws_bytes, &prm);
  if (st != MOE_OK) return st;
  if ((st = check_mxfp4(dtype, hidden, inter, w13_s, w2_s)) != MOE_OK || n_tokens == 0)
    return st;
  hipStream_t s = (hipStream_t)stream;
  if (moe::launch_route(logits, dtype, n_tokens, n_experts, topk, 0, n_experts, routing_out,
                        workspace, s) != hipSuccess)
    return MOE_ERR_HIP;
  return run_experts(x, dtype, n_tokens, hidden, w13_q, w2_q, n_experts, inter, topk, act, layout,
                     prm, routing_out, out, workspace, s, false, w13_s, w2_s);
}

namespace {
bool group_ok(int32_t g) { return g == 32 || g == 64 || g == 128; }

// Scratch of the 4-bit experts: activation rows a[M, 2, inter] (two bf16 parts
// of every value), then (topk > 1) the weighted expert rows y[M, hidden] in fp32.
size_t int4_act_bytes(int64_t n, int32_t k, int32_t inter) {
  return align256((size_t)n * k * inter * 4);
}
size_t int4_ws_bytes(int64_t n, int32_t k, int32_t hidden, int32_t inter) {
  return int4_act_bytes(n, k, inter) + (k > 1 ? align256((size_t)n * k * hidden * 4) : 0);
}

moe_status_t check_int4_weights(const moe_int4_weights_t *w) {
  if (!w || !w->q || !w->scales) return MOE_ERR_NULL;
  if (!aligned16(w->q) || !aligned16(w->scales) || !aligned16(w->zeros)) return MOE_ERR_ALIGN;
  return MOE_OK;
}

moe_status_t check_int4(const void *x, int64_t n, int32_t hidden, const moe_int4_weights_t *w13,
                        const moe_int4_weights_t *w2, int32_t e, int32_t inter, int32_t k,
                        int32_t group, moe_act_t act, moe_w13_layout_t layout,
                        const moe_act_params_t *params, const moe_routing_t *routing, void *out,
                        void *ws, size_t ws_bytes, ActParams *prm) {
  moe_status_t st = check_expert_args(MOE_BF16, n, hidden, e, inter, k, act, layout, params,
                                      routing, prm);
  if (st != MOE_OK) return st;
  if (!group_ok(group) || hidden % group || inter % group) return MOE_ERR_SHAPE;
  if (n == 0) return MOE_OK;
  if ((st = check_int4_weights(w13)) != MOE_OK || (st = check_int4_weights(w2)) != MOE_OK)
    return st;
  if ((st = check_ptrs({x, out})) != MOE_OK) return st;
  return check_ws(ws, ws_bytes, int4_ws_bytes(n, k, hidden, inter));
}

moe_status_t run_int4(const void *x, int64_t n, int32_t hidden, const moe_int4_weights_t *w13,
                      const moe_int4_weights_t *w2, int32_t e, int32_t inter, int32_t k,
                      int32_t group, moe_act_t act, moe_w13_layout_t layout, const ActParams &prm,
                      const moe_routing_t *routing, void *out, void *ws, hipStream_t s) {
  char *base = reinterpret_cast<char *>(ws);
  return moe::launch_experts_int4({w13->q, w13->scales, w13->zeros}, {w2->q, w2->scales, w2->zeros},
                                  x, routing, out, base, base + int4_act_bytes(n, k, inter), n, k,
                                  e, hidden, inter, group, act, layout, prm, s) == hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

moe_status_t check_int4_array(int32_t e, int32_t rows, int32_t k, int32_t group) {
  if (e < 1 || rows < 1 || k < 1 || k > (1 << 24) || !group_ok(group) || k % group)
    return MOE_ERR_SHAPE;
  // one thread per eight weights at most
  if ((int64_t)e * rows > kMostThreads / (k / 8)) return MOE_ERR_SHAPE;
  return MOE_OK;
}
}  // namespace

size_t moe_int4_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t topk, int32_t hidden,
                                int32_t inter) {
  if (check_sizes(n_tokens, n_experts, topk) != MOE_OK ||
      check_ffn_sizes(hidden, inter) != MOE_OK)
    return 0;
  // the expert scratch reuses the routing's once the routing has run
  const size_t route = moe::route_scratch_bytes(n_tokens, n_experts, topk);
  const size_t ffn = int4_ws_bytes(n_tokens, topk, hidden, inter);
  const size_t b = route > ffn ? route : ffn;
  return b ? b : 256;
}

moe_status_t moe_quantize_int4(const void *w, moe_dtype_t dtype, int32_t n_experts, int32_t rows,
                               int32_t k, int32_t group, void *q, void *scales, void *zeros,
                               void *stream) {
  if (!dtype_ok(dtype)) return MOE_ERR_DTYPE;
  moe_status_t st = check_int4_array(n_experts, rows, k, group);
  if (st != MOE_OK) return st;
  if ((st = check_ptrs({w, q, scales})) != MOE_OK) return st;
  if (!aligned16(zeros)) return MOE_ERR_ALIGN;
  return moe::launch_quantize_int4(w, dtype, n_experts, rows, k, group, {q, scales, zeros},
                                   (hipStream_t)stream) == hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

moe_status_t moe_dequantize_int4(const moe_int4_weights_t *w, int32_t n_experts, int32_t rows,
                                 int32_t k, int32_t group, void *out, void *stream) {
  moe_status_t st = check_int4_array(n_experts, rows, k, group);
  if (st != MOE_OK) return st;
  if ((st = check_int4_weights(w)) != MOE_OK) return st;
  if ((st = check_ptrs({out})) != MOE_OK) return st;
  return moe::launch_dequantize_int4({w->q, w->scales, w->zeros}, n_experts, rows, k, group, out,
                                     (hipStream_t)stream) == hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

moe_status_t moe_experts_int4(const void *x, int64_t n_tokens, int32_t hidden,
                              const moe_int4_weights_t *w13, const moe_int4_weights_t *w2,
                              int32_t n_experts, int32_t inter, int32_t topk, int32_t group,
                              moe_act_t act, moe_w13_layout_t layout,
                              const moe_act_params_t *params, const moe_routing_t *routing,
                              void *out, void *workspace, size_t ws_bytes, void *stream) {
  ActParams prm;
  moe_status_t st = check_int4(x, n_tokens, hidden, w13, w2, n_experts, inter, topk, group, act,
                               layout, params, routing, out, workspace, ws_bytes, &prm);
  if (st != MOE_OK || n_tokens == 0) return st;
  return run_int4(x, n_tokens, hidden, w13, w2, n_experts, inter, topk, group, act, layout, prm,
                  routing, out, workspace, (hipStream_t)stream);
}

moe_status_t moe_forward_int4(const void *x, const void *logits, int64_t n_tokens, int32_t hidden,
                              const moe_int4_weights_t *w13, const moe_int4_weights_t *w2,
                              int32_t n_experts, int32_t inter, int32_t topk, int32_t group,
                              moe_act_t act, moe_w13_layout_t layout,
                              const moe_act_params_t *params, const moe_routing_t *routing_out,
                              void *out, void *workspace, size_t ws_bytes, void *stream) {
  ActParams prm;
  moe_status_t st = check_route(logits, MOE_BF16, n_tokens, n_experts, topk, routing_out,
                                workspace, ws_bytes);
  if (st != MOE_OK) return st;
  st = check_int4(x, n_tokens, hidden, w13, w2, n_experts, inter, topk, group, act, layout,
                  params, routing_out, out, workspace, ws_bytes, &prm);
  if (st != MOE_OK || n_tokens == 0) return st;
  hipStream_t s = (hipStream_t)stream;
  if (moe::launch_route(logits, MOE_BF16, n_tokens, n_experts, topk, 0, n_experts, routing_out,
                        workspace, s) != hipSuccess)
    return MOE_ERR_HIP;
  return run_int4(x, n_tokens, hidden, w13, w2, n_experts, inter, topk, group, act, layout, prm,
                  routing_out, out, workspace, s);
}

size_t moe_block_norm_workspace_bytes(int64_t n_tokens, int32_t hidden, moe_dtype_t dtype) {
  if (n_tokens < 0 || n_tokens > 0x7fffffffLL || hidden < 8 || hidden % 8 ||
      hidden > moe::kMaxNormHidden || !dtype_ok(dtype))
    return 0;
  const size_t b = align256(moe::block_norm_scratch_bytes(n_tokens, hidden, dtype));
  return b ? b : 256;
}

moe_status_t moe_block_norm(const void *x, const void *y, moe_dtype_t dtype, int64_t n_tokens,
                            int32_t hidden, const moe_block_norm_t *norm, void *x_out,
                            void *n_out, float *rstd_post, float *rstd_pre, void *stream) {
  moe_status_t st = check_block_norm(x, y, dtype, n_tokens, hidden, norm);
  if (st != MOE_OK || n_tokens == 0) return st;
  if ((y && !x_out) || (norm->w_pre && !n_out)) return MOE_ERR_NULL;
  for (const void *p : {(const void *)x_out, (const void *)n_out, (const void *)rstd_post,
                        (const void *)rstd_pre})
    if (!aligned16(p)) return MOE_ERR_ALIGN;
  moe::BlockNormArgs g = block_norm_args(x, y, n_tokens, hidden, norm);
  g.x_out = x_out;
  g.n_out = n_out;
  g.rstd_post = rstd_post;
  g.rstd_pre = rstd_pre;
  return moe::launch_block_norm(g, dtype, (hipStream_t)stream) == hipSuccess ? MOE_OK
                                                                             : MOE_ERR_HIP;
}

moe_status_t moe_block_norm_backward(const void *d_x_out, const void *d_n_out, const void *x,
                                     const void *y, moe_dtype_t dtype, int64_t n_tokens,
                                     int32_t hidden, const moe_block_norm_t *norm,
                                     const float *rstd_post, const float *rstd_pre, void *d_x,
                                     void *d_y, float *d_w_post, float *d_w_pre, float *d_gate,
                                     void *workspace, size_t ws_bytes, void *stream) {
  moe_status_t st = check_block_norm(x, y, dtype, n_tokens, hidden, norm);
  if (st != MOE_OK) return st;
  const bool token_gate = norm->gate_kind == MOE_GATE_TOKEN;
  if (n_tokens > 0) {
    // something flows back, and everything it flows through is there
    if ((!d_x_out && !norm->w_pre) || !d_x || (y && !d_y)) return MOE_ERR_NULL;
    if (norm->w_pre && (!d_n_out || !rstd_pre)) return MOE_ERR_NULL;
    if (norm->w_post && !rstd_post) return MOE_ERR_NULL;
    if (token_gate && !d_gate) return MOE_ERR_NULL;
  }
  if ((norm->w_pre && !d_w_pre) || (norm->w_post && !d_w_post) ||
      (norm->gate_kind == MOE_GATE_CHANNEL && !d_gate))
    return MOE_ERR_NULL;
  for (const void *p : {d_x_out, d_n_out, (const void *)rstd_post, (const void *)rstd_pre,
                        (const void *)d_x, (const void *)d_y, (const void *)d_w_post,
                        (const void *)d_w_pre, (const void *)d_gate})
    if (!aligned16(p)) return MOE_ERR_ALIGN;
  if ((st = check_ws(workspace, ws_bytes,
                     moe::block_norm_scratch_bytes(n_tokens, hidden, dtype))) != MOE_OK)
    return st;
  moe::BlockNormArgs g = block_norm_args(x, y, n_tokens, hidden, norm);
  g.d_x_out = d_x_out;
  g.d_n_out = d_n_out;
  g.rstd_post = const_cast<float *>(rstd_post);
  g.rstd_pre = const_cast<float *>(rstd_pre);
  g.d_x = d_x;
  g.d_y = d_y;
  g.d_gate = token_gate ? d_gate : nullptr;
  g.partial = reinterpret_cast<float *>(workspace);
  const moe::ColumnSums sums{norm->w_pre ? d_w_pre : nullptr, norm->w_post ? d_w_post : nullptr,
                             norm->gate_kind == MOE_GATE_CHANNEL ? d_gate : nullptr};
  return moe::launch_block_norm_backward(g, sums, dtype, (hipStream_t)stream) == hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

moe_status_t moe_block_forward(const void *x, const void *w_gate, moe_dtype_t dtype,
                               int64_t n_tokens, int32_t hidden, const void *w13, const void *w2,
                               int32_t n_experts, int32_t inter, int32_t topk, moe_act_t act,
                               moe_w13_layout_t layout, const moe_act_params_t *params,
                               const moe_block_norm_t *norm, void *logits_out,
                               const moe_routing_t *routing_out, void *x_out, void *workspace,
                               size_t ws_bytes, void *stream) {
  // workspace: what moe_gate_forward takes, then the block's normed rows, which
  // the block's output replaces (the rows are dead once GEMM1 has run)
  const size_t inner = align256(
      moe_workspace_bytes(n_tokens, n_experts, topk, hidden, inter, dtype));
  if (inner == 0) return !dtype_ok(dtype) ? MOE_ERR_DTYPE : MOE_ERR_SHAPE;
  moe_status_t st = check_block_norm(x, x, dtype, n_tokens, hidden, norm);
  if (st != MOE_OK) return st;
  ActParams prm;
  if (n_tokens > 0) {
    if (!norm->w_pre || !x_out) return MOE_ERR_NULL;
    if (!aligned16(x_out)) return MOE_ERR_ALIGN;
    if ((st = check_ws(workspace, ws_bytes,
                       inner + align256((size_t)n_tokens * hidden * dsize(dtype)))) != MOE_OK)
      return st;
  }
  char *rows = reinterpret_cast<char *>(workspace) + inner;
  if ((st = check_gate(rows, w_gate, dtype, n_tokens, hidden, n_experts, logits_out)) != MOE_OK)
    return st;
  st = check_route(logits_out, dtype, n_tokens, n_experts, topk, routing_out, workspace, inner);
  if (st != MOE_OK) return st;
  st = check_experts(rows, dtype, n_tokens, hidden, w13, w2, n_experts, inter, topk, act, layout,
                     params, routing_out, rows, workspace, inner, &prm);
  if (st != MOE_OK || n_tokens == 0) return st;
  hipStream_t s = (hipStream_t)stream;
  moe::BlockNormArgs pre{};
  pre.x = x;
  pre.w_pre = norm->w_pre;
  pre.n_out = rows;
  pre.n_tokens = n_tokens;
  pre.hidden = hidden;
  pre.residual_scale = 1.f;
  pre.eps = norm->eps;
  if (moe::launch_block_norm(pre, dtype, s) != hipSuccess ||
      moe::launch_route(logits_out, dtype, n_tokens, n_experts, topk, 0, n_experts, routing_out,
                        workspace, s, rows, w_gate, hidden) != hipSuccess)
    return MOE_ERR_HIP;
  st = run_experts(rows, dtype, n_tokens, hidden, w13, w2, n_experts, inter, topk, act, layout, prm,
                   routing_out, rows, workspace, s);
  if (st != MOE_OK) return st;
  moe::BlockNormArgs post = block_norm_args(x, rows, n_tokens, hidden, norm);
  post.w_pre = nullptr;
  post.x_out = x_out;
  return moe::launch_block_norm(post, dtype, s) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

const char *moe_status_str(moe_status_t status) {
  switch (status) {
    case MOE_OK: return "ok";
    case MOE_ERR_NULL: return "required pointer is NULL";
    case MOE_ERR_SHAPE: return "size out of range or inconsistent";
    case MOE_ERR_DTYPE: return "unknown or mismatched dtype";
    case MOE_ERR_UNSUPPORTED: return "unsupported activation/layout combination";
    case MOE_ERR_ALIGN: return "pointer not 16-byte aligned";
    case MOE_ERR_WORKSPACE: return "workspace missing or too small";
    case MOE_ERR_HIP: return "HIP launch failed";
    case MOE_ERR_SCRATCH:
      return "sizes need more than the library's static scratch (MOE_NOALLOC_SCRATCH_BYTES)";
  }
  return "unknown status";
}

}  // extern "C"
