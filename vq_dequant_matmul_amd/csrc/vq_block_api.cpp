// vq_block_api.cpp -- C ABI of the operators around the routed experts: 4-bit
// products, the router and its selection, the norms at a block's ends.
// Argument checks follow vq_api.cpp: host-visible values only, a message
// naming the field.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/vq.h"
#include "vq_host.hpp"
#include "vq_internal.hpp"

using vq::aligned;
using vq::fail;
using vq::hip_fail;
using vq::ok;

namespace {

vq_status check_float_dtype(vq_dtype dt, const char *name)
{
    if (dt != VQ_F32 && dt != VQ_BF16)
        return fail(VQ_ERR_INVALID_ARGUMENT, "%s = %d: must be VQ_F32 or VQ_BF16", name, (int)dt);
    return VQ_OK;
}

// ---- 4-bit products ------------------------------------------------------------

vq_status check_q4(const vq_q4_tensor *t, const char *name)
{
    if (!t)
        return fail(VQ_ERR_INVALID_ARGUMENT, "%s: descriptor is NULL", name);
    if (t->rows < 1)
        return fail(VQ_ERR_INVALID_ARGUMENT, "%s.rows = %d: must be >= 1", name, t->rows);
    if (t->group != 32 && t->group != 64 && t->group != 128)
        return fail(VQ_ERR_UNSUPPORTED, "%s.group = %d: supported group sizes are 32, 64 and 128",
                    name, t->group);
    if (t->cols < t->group || t->cols % t->group != 0)
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "%s.cols = %d: must be a positive multiple of group = %d", name, t->cols,
                    t->group);
    if (t->scale_dtype != VQ_F16 && t->scale_dtype != VQ_BF16)
        return fail(VQ_ERR_INVALID_ARGUMENT, "%s.scale_dtype = %d: must be VQ_F16 or VQ_BF16",
                    name, (int)t->scale_dtype);
    if (!t->codes || !t->scales)
        return fail(VQ_ERR_INVALID_ARGUMENT, "%s: codes and scales must be non-NULL", name);
    if (!aligned(t->codes, 16) || !aligned(t->scales, 16) || !aligned(t->biases, 16))
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "%s: codes, scales and biases must be 16-byte aligned", name);
    if (t->rows > vq::kMaxQ4Rows || t->cols > vq::kMaxQ4Cols ||
        (int64_t)t->rows * t->cols > ((int64_t)1 << 40))
        return fail(VQ_ERR_UNSUPPORTED,
                    "%s is %dx%d: tensor too large (at most %d rows, %d cols and 2^40 weights)",
                    name, t->rows, t->cols, vq::kMaxQ4Rows, vq::kMaxQ4Cols);
    return VQ_OK;
}

vq::Q4Dev to_dev(const vq_q4_tensor &t)
{
    return {t.codes, t.scales, t.biases, t.rows, t.cols, t.group, t.scale_dtype == VQ_BF16};
}

vq_status check_dense(int32_t n_tokens, const void *x, vq_dtype x_dtype, const void *y,
                      const char *y_name)
{
    vq_status st = check_float_dtype(x_dtype, "x_dtype");
    if (st != VQ_OK)
        return st;
    if (n_tokens < 0 || n_tokens > vq::kDenseMaxTokens)
        return fail(VQ_ERR_INVALID_ARGUMENT, "n_tokens = %d: must be in [0, %d]", n_tokens,
                    vq::kDenseMaxTokens);
    if (n_tokens == 0)
        return VQ_OK;
    if (!x || !aligned(x, 16))
        return fail(VQ_ERR_INVALID_ARGUMENT, "x: must be a non-NULL, 16-byte aligned device pointer");
    if (!y || !aligned(y, 4))
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "%s: must be a non-NULL, 4-byte aligned device pointer", y_name);
    return VQ_OK;
}

// ---- selection -------------------------------------------------------------------

vq_status check_route(const vq_route_config *c, int32_t n_tokens, vq_dtype logits_dtype)
{
    if (!c)
        return fail(VQ_ERR_INVALID_ARGUMENT, "cfg is NULL");
    if (c->n_experts < 1)
        return fail(VQ_ERR_INVALID_ARGUMENT, "cfg.n_experts = %d: must be >= 1", c->n_experts);
    if (c->n_experts > vq::kMaxSelectExperts)
        return fail(VQ_ERR_UNSUPPORTED, "cfg.n_experts = %d: at most %d are supported",
                    c->n_experts, vq::kMaxSelectExperts);
    if (c->top_k < 1 || c->top_k > c->n_experts)
        return fail(VQ_ERR_INVALID_ARGUMENT, "cfg.top_k = %d: must be in [1, n_experts = %d]",
                    c->top_k, c->n_experts);
    if (c->top_k > vq::kMaxRouteTopK)
        return fail(VQ_ERR_UNSUPPORTED, "cfg.top_k = %d: at most %d are supported", c->top_k,
                    vq::kMaxRouteTopK);
    if (c->score != VQ_SCORE_SOFTMAX && c->score != VQ_SCORE_SIGMOID)
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "cfg.score = %d: must be VQ_SCORE_SOFTMAX or VQ_SCORE_SIGMOID", c->score);
    if (!std::isfinite(c->scale))
        return fail(VQ_ERR_INVALID_ARGUMENT, "cfg.scale: must be finite");
    if (n_tokens < 0)
        return fail(VQ_ERR_INVALID_ARGUMENT, "n_tokens = %d: must be >= 0", n_tokens);
    return check_float_dtype(logits_dtype, "logits_dtype");
}

size_t dtype_size(vq_dtype dt) { return dt == VQ_F32 ? 4 : 2; }

// ---- norms -----------------------------------------------------------------------

vq_status check_stream(const void *p, int64_t stride, int32_t hidden, const char *name)
{
    if (!p)
        return VQ_OK;
    if (!aligned(p, 16))
        return fail(VQ_ERR_INVALID_ARGUMENT, "%s: must be 16-byte aligned", name);
    if (stride < hidden || stride % 8 != 0)
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "%s_stride = %lld: must be a multiple of 8, at least hidden = %d", name,
                    (long long)stride, hidden);
    return VQ_OK;
}

vq_status check_norm(const vq_block_norm_args *a)
{
    if (!a)
        return fail(VQ_ERR_INVALID_ARGUMENT, "args is NULL");
    if (a->n_tokens < 0)
        return fail(VQ_ERR_INVALID_ARGUMENT, "n_tokens = %d: must be >= 0", a->n_tokens);
    if (a->n_tokens > vq::kMaxNormTokens)
        return fail(VQ_ERR_UNSUPPORTED, "n_tokens = %d: at most %d are supported", a->n_tokens,
                    vq::kMaxNormTokens);
    if (a->hidden < 8 || a->hidden % 8 != 0)
        return fail(VQ_ERR_INVALID_ARGUMENT, "hidden = %d: must be a positive multiple of 8",
                    a->hidden);
    if (a->hidden > vq::kMaxNormHidden)
        return fail(VQ_ERR_UNSUPPORTED, "hidden = %d: at most %d is supported", a->hidden,
                    vq::kMaxNormHidden);
    vq_status st;
    if ((st = check_float_dtype(a->h_dtype, "h_dtype")) != VQ_OK ||
        (st = check_float_dtype(a->y_dtype, "y_dtype")) != VQ_OK ||
        (st = check_float_dtype(a->x_dtype, "x_dtype")) != VQ_OK ||
        (st = check_float_dtype(a->weight_dtype, "weight_dtype")) != VQ_OK)
        return st;
    if (a->gate_kind != VQ_GATE_NONE && a->gate_kind != VQ_GATE_TOKEN &&
        a->gate_kind != VQ_GATE_CHANNEL)
        return fail(VQ_ERR_INVALID_ARGUMENT, "gate_kind = %d: must be one of VQ_GATE_*",
                    a->gate_kind);
    // without tokens the arrays with a row or value per token may be NULL; a gate
    // per channel may not: its gradient reads it all the same
    const bool token_gate = a->gate_kind == VQ_GATE_TOKEN;
    if ((a->gate_kind != VQ_GATE_NONE) != (a->gate != nullptr) &&
        !(token_gate && a->n_tokens == 0))
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "gate: must be given with VQ_GATE_TOKEN and VQ_GATE_CHANNEL, and only then");
    if (!a->y && (a->post_weight || a->gate) && a->n_tokens > 0)
        return fail(VQ_ERR_INVALID_ARGUMENT, "post_weight and gate need y");
    if (!(a->eps > 0.0f) || !std::isfinite(a->eps))
        return fail(VQ_ERR_INVALID_ARGUMENT, "eps = %g: must be positive and finite",
                    (double)a->eps);
    if (!std::isfinite(a->weight_offset) || !std::isfinite(a->skip_scale) ||
        !std::isfinite(a->block_scale))
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "weight_offset, skip_scale and block_scale must be finite");
    if (!aligned(a->post_weight, 16) || !aligned(a->pre_weight, 16) || !aligned(a->gate, 16))
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "post_weight, pre_weight and gate must be 16-byte aligned");
    if ((st = check_stream(a->h, a->h_stride, a->hidden, "h")) != VQ_OK ||
        (st = check_stream(a->y, a->y_stride, a->hidden, "y")) != VQ_OK ||
        (st = check_stream(a->h_out, a->h_out_stride, a->hidden, "h_out")) != VQ_OK ||
        (st = check_stream(a->x, a->x_stride, a->hidden, "x")) != VQ_OK)
        return st;
    return VQ_OK;
}

}  // namespace

VQ_EXPORT vq_status vq_q4_gemv(const vq_q4_tensor *W, int32_t n_tokens, const void *x,
                               vq_dtype x_dtype, float *y, int32_t accumulate, void *stream)
{
    vq_status st = check_q4(W, "W");
    if (st != VQ_OK || (st = check_dense(n_tokens, x, x_dtype, y, "y")) != VQ_OK)
        return st;
    if (n_tokens == 0)
        return ok();
    vq::Q4Launch L = {};
    L.t[0] = L.t[1] = to_dev(*W);
    L.nproj = 1;
    L.x = x;
    L.x_f32 = x_dtype == VQ_F32;
    L.n = n_tokens;
    L.y = y;
    L.accumulate = accumulate != 0;
    const hipError_t e = vq::launch_q4(L, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "vq_q4_gemv");
}

VQ_EXPORT vq_status vq_q4_gate_up(const vq_q4_tensor *gate, const vq_q4_tensor *up,
                                  int32_t n_tokens, const void *x, vq_dtype x_dtype, float *h,
                                  void *stream)
{
    vq_status st = check_q4(gate, "gate");
    if (st != VQ_OK || (st = check_q4(up, "up")) != VQ_OK)
        return st;
    if (up->rows != gate->rows || up->cols != gate->cols)
        return fail(VQ_ERR_INVALID_ARGUMENT, "up is %dx%d but gate is %dx%d", up->rows, up->cols,
                    gate->rows, gate->cols);
    if (up->group != gate->group || up->scale_dtype != gate->scale_dtype ||
        (up->biases == nullptr) != (gate->biases == nullptr))
        return fail(VQ_ERR_UNSUPPORTED,
                    "gate and up must share group, scale_dtype and whether they have biases "
                    "(they run in one fused kernel)");
    if ((st = check_dense(n_tokens, x, x_dtype, h, "h")) != VQ_OK)
        return st;
    if (n_tokens == 0)
        return ok();
    vq::Q4Launch L = {};
    L.t[0] = to_dev(*gate);
    L.t[1] = to_dev(*up);
    L.nproj = 2;
    L.x = x;
    L.x_f32 = x_dtype == VQ_F32;
    L.n = n_tokens;
    L.y = h;
    const hipError_t e = vq::launch_q4(L, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "vq_q4_gate_up");
}

VQ_EXPORT vq_status vq_router_logits(int32_t n_experts, int32_t hidden, const uint16_t *w,
                                     int32_t n_tokens, const void *x, vq_dtype x_dtype,
                                     float *logits, void *stream)
{
    if (n_experts < 1)
        return fail(VQ_ERR_INVALID_ARGUMENT, "n_experts = %d: must be >= 1", n_experts);
    if (hidden < 64 || hidden % 64 != 0)
        return fail(VQ_ERR_INVALID_ARGUMENT, "hidden = %d: must be a positive multiple of 64",
                    hidden);
    if (n_experts > vq::kMaxRouterRows || hidden > vq::kMaxQ4Cols)
        return fail(VQ_ERR_UNSUPPORTED,
                    "n_experts = %d, hidden = %d: router too large (at most %d by %d)", n_experts,
                    hidden, vq::kMaxRouterRows, vq::kMaxQ4Cols);
    if (!w || !aligned(w, 16))
        return fail(VQ_ERR_INVALID_ARGUMENT, "w: must be a non-NULL, 16-byte aligned device pointer");
    vq_status st = check_dense(n_tokens, x, x_dtype, logits, "logits");
    if (st != VQ_OK)
        return st;
    if (n_tokens == 0)
        return ok();
    const vq::LogitsLaunch L = {w, n_experts, hidden, x, x_dtype == VQ_F32, n_tokens, logits};
    const hipError_t e = vq::launch_router_logits(L, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "vq_router_logits");
}

VQ_EXPORT size_t vq_moe_route_workspace_size(const vq_route_config *cfg, int32_t n_tokens)
{
    if (check_route(cfg, n_tokens, VQ_F32) != VQ_OK)
        return 0;
    return vq::route_workspace_bytes(cfg->n_experts, n_tokens);
}

VQ_EXPORT vq_status vq_moe_route(const vq_route_config *cfg, int32_t n_tokens,
                                 const void *logits, vq_dtype logits_dtype, const float *bias,
                                 const uint8_t *mask, int32_t *topk_ids, float *topk_weights,
                                 int32_t *counts, float *loss, void *workspace,
                                 size_t workspace_bytes, void *stream)
{
    vq_status st = check_route(cfg, n_tokens, logits_dtype);
    if (st != VQ_OK)
        return st;
    if ((counts == nullptr) != (loss == nullptr))
        return fail(VQ_ERR_INVALID_ARGUMENT, "counts and loss must both be given or both be NULL");
    if (n_tokens == 0 && !counts)
        return ok();
    if (n_tokens > 0) {
        if (!logits || !aligned(logits, dtype_size(logits_dtype)))
            return fail(VQ_ERR_INVALID_ARGUMENT,
                        "logits: must be a non-NULL device pointer, aligned to its type");
        if (!topk_ids || !topk_weights || !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
            return fail(VQ_ERR_INVALID_ARGUMENT,
                        "topk_ids and topk_weights must be non-NULL, 4-byte aligned");
    }
    if (!aligned(bias, 4) || !aligned(counts, 4) || !aligned(loss, 4))
        return fail(VQ_ERR_INVALID_ARGUMENT, "bias, counts and loss must be 4-byte aligned");
    if (counts) {
        const size_t need = vq::route_workspace_bytes(cfg->n_experts, n_tokens);
        if (!workspace || workspace_bytes < need || !aligned(workspace, 256))
            return fail(VQ_ERR_WORKSPACE,
                        "workspace: need %zu bytes, 256-byte aligned (got %zu bytes at %p)", need,
                        workspace_bytes, workspace);
    }
    const vq::RouteLaunch L = {cfg->n_experts, cfg->top_k, cfg->score == VQ_SCORE_SIGMOID,
                               cfg->renormalize != 0, cfg->scale, n_tokens, logits,
                               logits_dtype == VQ_BF16, bias, mask, topk_ids, topk_weights, counts,
                               loss, workspace};
    const hipError_t e = vq::launch_route(L, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "vq_moe_route");
}

VQ_EXPORT vq_status vq_moe_route_grad(const vq_route_config *cfg, int32_t n_tokens,
                                      const void *logits, vq_dtype logits_dtype,
                                      const uint8_t *mask, const int32_t *topk_ids,
                                      const float *d_weights, const int32_t *counts,
                                      const float *d_loss, void *d_logits, void *stream)
{
    vq_status st = check_route(cfg, n_tokens, logits_dtype);
    if (st != VQ_OK)
        return st;
    if ((counts == nullptr) != (d_loss == nullptr))
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "counts and d_loss must both be given or both be NULL");
    if (n_tokens == 0)
        return ok();
    const size_t a = dtype_size(logits_dtype);
    if (!logits || !d_logits || !aligned(logits, a) || !aligned(d_logits, a))
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "logits and d_logits must be non-NULL device pointers, aligned to their type");
    if (d_weights && (!topk_ids || !aligned(topk_ids, 4) || !aligned(d_weights, 4)))
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "topk_ids must be given with d_weights, both 4-byte aligned");
    if (!aligned(counts, 4) || !aligned(d_loss, 4))
        return fail(VQ_ERR_INVALID_ARGUMENT, "counts and d_loss must be 4-byte aligned");
    const vq::RouteGradLaunch L = {cfg->n_experts, cfg->top_k, cfg->score == VQ_SCORE_SIGMOID,
                                   cfg->renormalize != 0, cfg->scale, n_tokens, logits,
                                   logits_dtype == VQ_BF16, mask, topk_ids, d_weights, counts,
                                   d_loss, d_logits};
    const hipError_t e = vq::launch_route_grad(L, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "vq_moe_route_grad");
}

VQ_EXPORT vq_status vq_block_norm(const vq_block_norm_args *a, void *stream)
{
    vq_status st = check_norm(a);
    if (st != VQ_OK)
        return st;
    if (a->n_tokens == 0)
        return ok();
    if (!a->h)
        return fail(VQ_ERR_INVALID_ARGUMENT, "h must be non-NULL");
    if (!a->h_out && !a->x)
        return fail(VQ_ERR_INVALID_ARGUMENT, "h_out or x must be non-NULL");
    const hipError_t e = vq::launch_block_norm(*a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "vq_block_norm");
}

VQ_EXPORT size_t vq_block_norm_grad_workspace_size(const vq_block_norm_args *a)
{
    if (check_norm(a) != VQ_OK)
        return 0;
    return vq::block_norm_grad_workspace_bytes(*a);
}

VQ_EXPORT vq_status vq_block_norm_grad(const vq_block_norm_args *a, const void *d_h_out,
                                       const void *d_x, void *d_h, void *d_y,
                                       float *d_post_weight, float *d_pre_weight, float *d_gate,
                                       void *workspace, size_t workspace_bytes, void *stream)
{
    vq_status st = check_norm(a);
    if (st != VQ_OK)
        return st;
    if ((d_y || d_post_weight || d_gate) && !a->y && a->n_tokens > 0)
        return fail(VQ_ERR_INVALID_ARGUMENT, "d_y, d_post_weight and d_gate need y");
    if (d_post_weight && !a->post_weight)
        return fail(VQ_ERR_INVALID_ARGUMENT, "d_post_weight needs post_weight");
    if (d_pre_weight && !a->pre_weight)
        return fail(VQ_ERR_INVALID_ARGUMENT, "d_pre_weight needs pre_weight");
    if (d_gate && a->gate_kind == VQ_GATE_NONE)
        return fail(VQ_ERR_INVALID_ARGUMENT, "d_gate needs a gate");
    if (!aligned(d_post_weight, 16) || !aligned(d_pre_weight, 16) || !aligned(d_gate, 16))
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "d_post_weight, d_pre_weight and d_gate must be 16-byte aligned");
    if (a->n_tokens > 0) {
        if (!d_h_out && !d_x)
            return fail(VQ_ERR_INVALID_ARGUMENT, "d_h_out or d_x must be non-NULL");
        if ((d_x || d_pre_weight) && !a->h_out)
            return fail(VQ_ERR_INVALID_ARGUMENT, "h_out must be non-NULL: d_x and d_pre_weight need it");
        if ((st = check_stream(d_h_out, a->h_out_stride, a->hidden, "d_h_out (h_out)")) != VQ_OK ||
            (st = check_stream(d_x, a->x_stride, a->hidden, "d_x (x)")) != VQ_OK ||
            (st = check_stream(d_h, a->h_stride, a->hidden, "d_h (h)")) != VQ_OK ||
            (st = check_stream(d_y, a->y_stride, a->hidden, "d_y (y)")) != VQ_OK)
            return st;
    }
    const size_t need = vq::block_norm_grad_workspace_bytes(*a);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return fail(VQ_ERR_WORKSPACE,
                    "workspace: need %zu bytes, 256-byte aligned (got %zu bytes at %p)", need,
                    workspace_bytes, workspace);
    const vq::NormGradLaunch L = {*a, d_h_out, d_x, d_h, d_y, d_post_weight, d_pre_weight, d_gate,
                                  static_cast<float *>(workspace)};
    const hipError_t e = vq::launch_block_norm_grad(L, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "vq_block_norm_grad");
}

// ---- one MoE block ------------------------------------------------------------------

namespace {

// The workspace: the block's input x, what the router says, the block's
// output y, the shared expert's h, and the routed FFN's own workspace.
struct BlockWs {
    size_t x, logits, ids, weights, y, shared, ffn, total;
};

size_t round_up(size_t v) { return (v + 255) / 256 * 256; }

vq_status check_block(const vq_moe_block_args *B, int32_t n_tokens, BlockWs *ws)
{
    if (!B)
        return fail(VQ_ERR_INVALID_ARGUMENT, "B is NULL");
    if (n_tokens < 0 || n_tokens > vq::kDenseMaxTokens)
        return fail(VQ_ERR_INVALID_ARGUMENT, "n_tokens = %d: must be in [0, %d]", n_tokens,
                    vq::kDenseMaxTokens);
    // (the FFN's own checks, all of them: nothing runs, and h stays as it is,
    // where a later step would refuse the sizes)
    vq_status st = vq::check_moe_ffn(B->gate, B->up, B->down, n_tokens, B->route.top_k);
    if (st != VQ_OK || (st = check_route(&B->route, n_tokens, VQ_F32)) != VQ_OK ||
        (st = check_float_dtype(B->x_dtype, "x_dtype")) != VQ_OK)
        return st;
    const int hidden = B->gate->cols;
    if (hidden > vq::kMaxNormHidden)
        return fail(VQ_ERR_UNSUPPORTED, "gate.cols = %d: the norms take at most %d", hidden,
                    vq::kMaxNormHidden);
    if (B->route.n_experts != B->gate->n_experts)
        return fail(VQ_ERR_INVALID_ARGUMENT, "route.n_experts = %d but gate has %d experts",
                    B->route.n_experts, B->gate->n_experts);
    if (!B->router || !aligned(B->router, 16))
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "router: must be a non-NULL, 16-byte aligned device pointer");
    if (!aligned(B->route_bias, 4))
        return fail(VQ_ERR_INVALID_ARGUMENT, "route_bias: must be 4-byte aligned");
    if (!B->pre_weight)
        return fail(VQ_ERR_INVALID_ARGUMENT, "pre_weight must be non-NULL");
    const bool shared = B->shared_gate || B->shared_up || B->shared_down;
    if (shared) {
        if ((st = check_q4(B->shared_gate, "shared_gate")) != VQ_OK ||
            (st = check_q4(B->shared_up, "shared_up")) != VQ_OK ||
            (st = check_q4(B->shared_down, "shared_down")) != VQ_OK)
            return st;
        if (B->shared_gate->cols != hidden || B->shared_down->rows != hidden ||
            B->shared_down->cols != B->shared_gate->rows)
            return fail(VQ_ERR_INVALID_ARGUMENT,
                        "shared expert: gate is %dx%d and down %dx%d for hidden size %d",
                        B->shared_gate->rows, B->shared_gate->cols, B->shared_down->rows,
                        B->shared_down->cols, hidden);
    }
    const size_t n = n_tokens, k = B->route.top_k;
    ws->x = 0;
    ws->logits = ws->x + round_up(n * hidden * dtype_size(B->x_dtype));
    ws->ids = ws->logits + round_up(n * B->route.n_experts * 4);
    ws->weights = ws->ids + round_up(n * k * 4);
    ws->y = ws->weights + round_up(n * k * 4);
    ws->shared = ws->y + round_up(n * hidden * 4);
    ws->ffn = ws->shared + (shared ? round_up(n * B->shared_gate->rows * 4) : 0);
    const size_t ffn =
        n_tokens == 0 ? 0
                      : vq_moe_ffn_workspace_size(B->gate, B->up, B->down, n_tokens, B->route.top_k);
    ws->total = ws->ffn + round_up(ffn);
    return VQ_OK;
}

vq_block_norm_args block_norm_args(const vq_moe_block_args &B, int32_t n_tokens, float *h)
{
    vq_block_norm_args a = {};
    a.n_tokens = n_tokens;
    a.hidden = B.gate->cols;
    a.h_dtype = a.y_dtype = VQ_F32;
    a.x_dtype = B.x_dtype;
    a.weight_dtype = B.weight_dtype;
    a.h_stride = a.y_stride = a.h_out_stride = a.x_stride = a.hidden;
    a.h = h;
    a.eps = B.eps;
    a.weight_offset = B.weight_offset;
    a.skip_scale = a.block_scale = 1.0f;
    return a;
}

}  // namespace

VQ_EXPORT size_t vq_moe_block_workspace_size(const vq_moe_block_args *B, int32_t n_tokens)
{
    BlockWs ws;
    return check_block(B, n_tokens, &ws) == VQ_OK ? ws.total : 0;
}

VQ_EXPORT vq_status vq_moe_block(const vq_moe_block_args *B, int32_t n_tokens, float *h,
                                 const float *attn, const void *attn_weight,
                                 const void *next_weight, void *x_next, void *workspace,
                                 size_t workspace_bytes, void *stream)
{
    BlockWs ws;
    vq_status st = check_block(B, n_tokens, &ws);
    if (st != VQ_OK)
        return st;
    if (attn_weight && !attn)
        return fail(VQ_ERR_INVALID_ARGUMENT, "attn_weight needs attn");
    if ((next_weight == nullptr) != (x_next == nullptr) && n_tokens > 0)
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "next_weight and x_next must both be given or both be NULL");
    if (n_tokens == 0)
        return ok();
    if (!h)
        return fail(VQ_ERR_INVALID_ARGUMENT, "h must be non-NULL");
    if (!workspace || workspace_bytes < ws.total || !aligned(workspace, 256))
        return fail(VQ_ERR_WORKSPACE,
                    "workspace: need %zu bytes, 256-byte aligned (got %zu bytes at %p)", ws.total,
                    workspace_bytes, workspace);
    char *base = static_cast<char *>(workspace);
    void *x = base + ws.x;
    float *logits = reinterpret_cast<float *>(base + ws.logits);
    int32_t *ids = reinterpret_cast<int32_t *>(base + ws.ids);
    float *weights = reinterpret_cast<float *>(base + ws.weights);
    float *y = reinterpret_cast<float *>(base + ws.y);
    float *sh = reinterpret_cast<float *>(base + ws.shared);

    // both norms' arguments are checked before anything runs
    vq_block_norm_args in = block_norm_args(*B, n_tokens, h);
    in.y = attn;
    in.post_weight = attn_weight;
    in.pre_weight = B->pre_weight;
    in.h_out = attn ? h : nullptr;
    in.x = x;
    if (attn) {
        in.skip_scale = B->skip_scale;
        in.block_scale = B->block_scale;
    }
    vq_block_norm_args out = block_norm_args(*B, n_tokens, h);
    out.y = y;
    out.post_weight = B->post_weight;
    out.gate = B->channel_gate;
    out.gate_kind = B->channel_gate ? VQ_GATE_CHANNEL : VQ_GATE_NONE;
    out.pre_weight = next_weight;
    out.h_out = h;
    out.x = x_next;
    out.skip_scale = B->skip_scale;
    out.block_scale = B->block_scale;
    if ((st = check_norm(&in)) != VQ_OK || (st = check_norm(&out)) != VQ_OK)
        return st;
    if (B->shared_gate &&
        (B->shared_up->rows != B->shared_gate->rows || B->shared_up->cols != B->shared_gate->cols ||
         B->shared_up->group != B->shared_gate->group ||
         B->shared_up->scale_dtype != B->shared_gate->scale_dtype ||
         (B->shared_up->biases == nullptr) != (B->shared_gate->biases == nullptr)))
        return fail(VQ_ERR_INVALID_ARGUMENT,
                    "shared_up must share shape, group, scale_dtype and biases with shared_gate");

    const int hidden = B->gate->cols;
    if ((st = vq_block_norm(&in, stream)) != VQ_OK ||
        (st = vq_router_logits(B->route.n_experts, hidden, B->router, n_tokens, x, B->x_dtype,
                               logits, stream)) != VQ_OK ||
        (st = vq_moe_route(&B->route, n_tokens, logits, VQ_F32, B->route_bias, nullptr, ids,
                           weights, nullptr, nullptr, nullptr, 0, stream)) != VQ_OK ||
        (st = vq_moe_ffn(B->gate, B->up, B->down, n_tokens, B->route.top_k, x, B->x_dtype, ids,
                         weights, y, base + ws.ffn, ws.total - ws.ffn, stream)) != VQ_OK)
        return st;
    if (B->shared_gate &&
        ((st = vq_q4_gate_up(B->shared_gate, B->shared_up, n_tokens, x, B->x_dtype, sh, stream)) !=
             VQ_OK ||
         (st = vq_q4_gemv(B->shared_down, n_tokens, sh, VQ_F32, y, 1, stream)) != VQ_OK))
        return st;
    return vq_block_norm(&out, stream);
}
