// experts_api.hip -- C entry points of the expert operations (include/ep.h):
// argument checks, then the launches.  Nothing here allocates or waits.
#include <cmath>

#include "route.h"

using namespace ep;

namespace {

struct Traced {
    explicit Traced(const char *name) { api_trace_push(name); }
    ~Traced() { api_trace_pop(); }
};

bool al(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int done(hipError_t e) { return e == hipSuccess ? EP_OK : api_hip_error(e); }

int check_rows_dims(int32_t tokens, int32_t hidden)
{
    if (tokens < 0 || tokens > kMaxTokens || hidden <= 0 || hidden > kMaxHidden)
        return EP_ERR_INVALID;
    return hidden % 8 != 0 ? EP_ERR_ALIGN : EP_OK;
}

int check_expert_dims(const ep_dims *d, int32_t inter, int32_t unit)
{
    if (d == nullptr)
        return EP_ERR_INVALID;
    int rc = check_rows_dims(d->num_tokens, d->hidden);
    if (rc != EP_OK)
        return rc;
    if (d->num_topk < 1 || d->num_topk > kMaxTopk || d->num_ranks < 1 || d->num_ranks > kMaxRanks ||
        d->num_experts < 1 || d->num_experts > kMaxExperts || d->num_experts % d->num_ranks != 0)
        return EP_ERR_INVALID;
    if (inter <= 0 || inter > kMaxHidden)
        return EP_ERR_INVALID;
    return inter % unit != 0 || d->hidden % unit != 0 ? EP_ERR_ALIGN : EP_OK;
}

// Every launch of a call stays within one grid (checked before the first one).
bool grids_fit(int64_t rows, int64_t groups, int64_t hidden, int64_t inter, bool grads)
{
    const int64_t cols = (hidden > inter ? hidden : inter) / 128 + 1;
    if (tiles_at_most(rows, groups, cols) > kMaxTileBlocks)
        return false;
    return !grads || groups * (2 * inter / 256 + 1) * (hidden / 256 + 1) <= kMaxTileBlocks;
}

int check_groups(const ep_dims *d, const ep_expert_groups *g)
{
    if (g == nullptr || g->num_rows < 0 || g->pair_cap < 0)
        return EP_ERR_INVALID;
    if (g->num_rows > INT32_MAX || g->num_rows * d->num_topk > INT32_MAX || g->pair_cap > INT32_MAX)
        return EP_ERR_INVALID;
    if (g->expert_offsets == nullptr || (g->num_rows > 0 && g->row_pair == nullptr) ||
        (g->pair_cap > 0 && (g->pair_row == nullptr || g->pair_slot == nullptr)))
        return EP_ERR_INVALID;
    if (!al(g->expert_offsets, 4) || !al(g->pair_row, 4) || !al(g->pair_slot, 4) || !al(g->row_pair, 4))
        return EP_ERR_ALIGN;
    return EP_OK;
}

ExpertFfn ffn_of(const ep_dims *d, int32_t inter, const ep_expert_groups *g, const float *weights)
{
    ExpertFfn f{};
    f.experts = d->num_experts;
    f.hidden = d->hidden;
    f.inter = inter;
    f.topk = d->num_topk;
    f.rows = g->num_rows;
    f.pairs = g->pair_cap;
    f.offsets = g->expert_offsets;
    f.pair_row = g->pair_row;
    f.pair_slot = g->pair_slot;
    f.row_pair = g->row_pair;
    f.weights = weights;
    return f;
}

// The dims' experts, ranks and choices under a router.
int check_router(const ep_dims *d, const ep_router *r)
{
    if (d == nullptr || r == nullptr)
        return EP_ERR_INVALID;
    if (d->num_tokens < 0 || d->num_tokens > kMaxTokens || d->num_topk < 1 || d->num_topk > kMaxTopk ||
        d->num_ranks < 1 || d->num_ranks > kMaxRanks || d->num_experts < 1 || d->num_experts > kMaxExperts ||
        d->num_experts % d->num_ranks != 0)
        return EP_ERR_INVALID;
    if (r->score != EP_SCORE_SOFTMAX && r->score != EP_SCORE_SIGMOID)
        return EP_ERR_INVALID;
    if (r->num_groups < 1 || r->num_groups > kMaxRouteGroups || d->num_experts % r->num_groups != 0 ||
        r->topk_groups < 1 || r->topk_groups > r->num_groups || !std::isfinite(r->scale))
        return EP_ERR_INVALID;
    return EP_OK;
}

RouteRule rule_of(const ep_dims *d, const ep_router *r, const float *bias, const int32_t *rank_mask)
{
    RouteRule q{};
    q.experts = d->num_experts;
    q.topk = d->num_topk;
    q.groups = r->num_groups;
    q.topk_groups = r->topk_groups;
    q.epr = d->num_experts / d->num_ranks;
    q.size = q.experts / q.groups;
    q.lanes = 64;
    while (q.lanes * q.groups > 64)
        q.lanes /= 2;
    q.per_size = 1.0f / float(q.size);
    q.soft = r->score == EP_SCORE_SOFTMAX;
    q.normalize = r->normalize != 0;
    q.scale = r->scale;
    q.bias = bias;
    q.rank_mask = rank_mask;
    return q;
}

int check_adapters(const ep_adapter_dims *d)
{
    if (d == nullptr || d->num_tokens < 0 || d->num_tokens > kMaxTokens || d->in_features <= 0 ||
        d->in_features > kMaxHidden || d->out_features <= 0 || d->out_features > kMaxHidden || d->rank <= 0 ||
        d->rank > kMaxRank || d->num_adapters < 1 || d->num_adapters > kMaxAdapters)
        return EP_ERR_INVALID;
    return d->in_features % 8 != 0 || d->out_features % 8 != 0 || d->rank % 8 != 0 ? EP_ERR_ALIGN : EP_OK;
}

AdapterShape adapters_of(const ep_adapter_dims *d, const int64_t *ids, const float *scales)
{
    return {d->num_tokens, d->in_features, d->out_features, d->rank, d->num_adapters, ids, scales};
}

}  // namespace

extern "C" {

size_t ep_adapter_workspace(const ep_adapter_dims *dims, int32_t backward)
{
    if (check_adapters(dims) != EP_OK)
        return 0;
    return adapter_workspace(adapters_of(dims, nullptr, nullptr), backward != 0);
}

int ep_adapter_product(const ep_adapter_dims *dims, const void *x, const int64_t *adapter_ids, const void *down,
                       const void *up, const float *scales, const void *base, void *out, void *hidden, void *workspace,
                       size_t workspace_bytes, ep_stream_t stream)
{
    Traced trace("ep_adapter_product");
    const int rc = check_adapters(dims);
    if (rc != EP_OK)
        return rc;
    const size_t need = ep_adapter_workspace(dims, 0);
    if (down == nullptr || up == nullptr || scales == nullptr ||
        (dims->num_tokens > 0 && (x == nullptr || adapter_ids == nullptr || out == nullptr || (workspace == nullptr && need > 0))))
        return EP_ERR_INVALID;
    if (!al(x, 16) || !al(down, 16) || !al(up, 16) || !al(base, 16) || !al(out, 16) || !al(hidden, 16) ||
        !al(workspace, 256) || !al(adapter_ids, 8) || !al(scales, 4))
        return EP_ERR_ALIGN;
    if (workspace_bytes < need)
        return EP_ERR_CAPACITY;
    if (dims->num_tokens == 0)
        return EP_OK;
    return done(launch_adapter(adapters_of(dims, adapter_ids, scales), x, down, up, base, out, hidden, workspace,
                               static_cast<hipStream_t>(stream)));
}

int ep_adapter_product_backward(const ep_adapter_dims *dims, const void *dy, const void *x, const int64_t *adapter_ids,
                                const void *down, const void *up, const float *scales, const void *hidden,
                                const void *dx_base, void *dx, void *ddown, void *dup, void *workspace,
                                size_t workspace_bytes, ep_stream_t stream)
{
    Traced trace("ep_adapter_product_backward");
    const int rc = check_adapters(dims);
    if (rc != EP_OK)
        return rc;
    if (down == nullptr || up == nullptr || scales == nullptr || ddown == nullptr || dup == nullptr ||
        workspace == nullptr ||
        (dims->num_tokens > 0 && (dy == nullptr || x == nullptr || adapter_ids == nullptr || hidden == nullptr ||
                                  dx == nullptr)))
        return EP_ERR_INVALID;
    if (!al(dy, 16) || !al(x, 16) || !al(down, 16) || !al(up, 16) || !al(hidden, 16) || !al(dx_base, 16) || !al(dx, 16) ||
        !al(ddown, 16) || !al(dup, 16) || !al(workspace, 256) || !al(adapter_ids, 8) || !al(scales, 4))
        return EP_ERR_ALIGN;
    // the gradients' blocks are one launch, counted in 32 bits
    const int64_t runs = (int64_t(dims->in_features) + 63) / 64 + (int64_t(dims->out_features) + 63) / 64;
    if (dims->num_adapters * runs > kMaxGradBlocks)
        return EP_ERR_INVALID;
    if (workspace_bytes < ep_adapter_workspace(dims, 1))
        return EP_ERR_CAPACITY;
    return done(launch_adapter_backward(adapters_of(dims, adapter_ids, scales), dy, x, down, up, hidden, dx_base, dx,
                                        ddown, dup, workspace, static_cast<hipStream_t>(stream)));
}

size_t ep_route_workspace(const ep_dims *dims)
{
    if (dims == nullptr || dims->num_tokens < 0 || dims->num_tokens > kMaxTokens || dims->num_experts < 1 ||
        dims->num_experts > kMaxExperts)
        return 0;
    return size_t(route_parts(dims->num_tokens, dims->num_experts)) * dims->num_experts * sizeof(float);
}

int ep_route(const ep_dims *dims, const ep_router *router, const void *logits, int32_t logits_bf16, const float *bias,
             const int32_t *rank_mask, int64_t *topk_idx, float *topk_weights, float *score_sums, void *workspace,
             size_t workspace_bytes, ep_stream_t stream)
{
    Traced trace("ep_route");
    const int rc = check_router(dims, router);
    if (rc != EP_OK)
        return rc;
    const bool any = dims->num_tokens > 0;
    if (any && (logits == nullptr || topk_idx == nullptr || topk_weights == nullptr))
        return EP_ERR_INVALID;
    if (!al(logits, logits_bf16 != 0 ? 2 : 4) || !al(bias, 4) || !al(rank_mask, 4) || !al(topk_idx, 8) ||
        !al(topk_weights, 4) || !al(score_sums, 4) || !al(workspace, 4))
        return EP_ERR_ALIGN;
    if (score_sums != nullptr) {
        if (any && workspace == nullptr)
            return EP_ERR_INVALID;
        if (workspace_bytes < ep_route_workspace(dims))
            return EP_ERR_CAPACITY;
    }
    return done(launch_route(rule_of(dims, router, bias, rank_mask), dims->num_tokens, logits, logits_bf16 != 0, topk_idx,
                             topk_weights, score_sums, static_cast<float *>(workspace),
                             static_cast<hipStream_t>(stream)));
}

size_t ep_ll_moe_workspace(const ep_dims *dims, int32_t inter)
{
    if (check_expert_dims(dims, inter, 8) != EP_OK || dims->num_tokens > kMoeTokens || dims->num_experts > kMoeExperts)
        return 0;
    return moe_workspace(dims->num_tokens, dims->num_experts, dims->num_topk, inter);
}

int ep_ll_moe(const ep_dims *dims, int32_t inter, const ep_router *router, const void *x, const void *w_router,
              int32_t w_router_fp32, const float *bias, const int32_t *rank_mask, const void *w13,
              const float *w13_scale, const void *w2, const float *w2_scale, const void *residual, int64_t *topk_idx,
              float *topk_weights, void *y, void *workspace, size_t workspace_bytes, ep_stream_t stream)
{
    Traced trace("ep_ll_moe");
    if ((w13_scale != nullptr) != (w2_scale != nullptr))
        return EP_ERR_INVALID;
    int rc = check_expert_dims(dims, inter, w13_scale != nullptr ? 128 : 8);
    if (rc == EP_OK)
        rc = check_router(dims, router);
    if (rc != EP_OK)
        return rc;
    if (dims->num_tokens > kMoeTokens || dims->num_experts > kMoeExperts)
        return EP_ERR_TOO_LARGE;
    if (w_router == nullptr || w13 == nullptr || w2 == nullptr ||
        (dims->num_tokens > 0 && (x == nullptr || topk_idx == nullptr || topk_weights == nullptr || y == nullptr ||
                                  workspace == nullptr)))
        return EP_ERR_INVALID;
    if (!al(x, 16) || !al(w_router, 16) || !al(w13, 16) || !al(w2, 16) || !al(residual, 16) || !al(y, 16) ||
        !al(workspace, 256) || !al(bias, 4) || !al(rank_mask, 4) || !al(w13_scale, 4) || !al(w2_scale, 4) ||
        !al(topk_idx, 8) || !al(topk_weights, 4))
        return EP_ERR_ALIGN;
    if (workspace_bytes < ep_ll_moe_workspace(dims, inter))
        return EP_ERR_CAPACITY;
    if (dims->num_tokens == 0)
        return EP_OK;
    MoeCall c{};
    c.T = dims->num_tokens;
    c.H = dims->hidden;
    c.I = inter;
    c.x = x;
    c.w_router = w_router;
    c.router_f32 = w_router_fp32 != 0;
    c.w13 = w13;
    c.w13_scale = w13_scale;
    c.w2 = w2;
    c.w2_scale = w2_scale;
    c.residual = residual;
    c.topk_idx = topk_idx;
    c.topk_weights = topk_weights;
    c.y = y;
    c.workspace = workspace;
    return done(launch_moe(rule_of(dims, router, bias, rank_mask), c, static_cast<hipStream_t>(stream)));
}

int ep_route_backward(const ep_dims *dims, const ep_router *router, const float *dtopk_weights, const void *logits,
                      int32_t logits_bf16, const int64_t *topk_idx, const float *dscore_sums, void *dlogits,
                      ep_stream_t stream)
{
    Traced trace("ep_route_backward");
    const int rc = check_router(dims, router);
    if (rc != EP_OK)
        return rc;
    if (dims->num_tokens > 0 &&
        (dtopk_weights == nullptr || logits == nullptr || topk_idx == nullptr || dlogits == nullptr))
        return EP_ERR_INVALID;
    const size_t size = logits_bf16 != 0 ? 2 : 4;
    if (!al(dtopk_weights, 4) || !al(logits, size) || !al(topk_idx, 8) || !al(dscore_sums, 4) || !al(dlogits, size))
        return EP_ERR_ALIGN;
    return done(launch_route_backward(rule_of(dims, router, nullptr, nullptr), dims->num_tokens, dtopk_weights, logits,
                                      logits_bf16 != 0, topk_idx, dscore_sums, dlogits,
                                      static_cast<hipStream_t>(stream)));
}


int ep_rms_norm(int32_t num_tokens, int32_t hidden, float eps, const void *x, const void *residual,
                const void *weight, void *residual_out, void *out, void *out_q, float *out_scale,
                float *rstd, ep_stream_t stream)
{
    Traced trace("ep_rms_norm");
    int rc = check_rows_dims(num_tokens, hidden);
    if (rc != EP_OK)
        return rc;
    if (!(eps >= 0.0f) || !std::isfinite(eps))
        return EP_ERR_INVALID;
    if ((residual_out != nullptr && residual == nullptr) || (out == nullptr && out_q == nullptr) ||
        (out_q != nullptr) != (out_scale != nullptr))
        return EP_ERR_INVALID;
    if (num_tokens > 0 && (x == nullptr || weight == nullptr))
        return EP_ERR_INVALID;
    if (out_q != nullptr && hidden % 128 != 0)
        return EP_ERR_ALIGN;
    if (!al(x, 16) || !al(residual, 16) || !al(weight, 16) || !al(residual_out, 16) || !al(out, 16) ||
        !al(out_q, 8) || !al(out_scale, 4) || !al(rstd, 4))
        return EP_ERR_ALIGN;
    return done(launch_rms_norm(num_tokens, hidden, eps, x, residual, weight, residual_out, out, out_q,
                                out_scale, rstd, static_cast<hipStream_t>(stream)));
}

size_t ep_rms_norm_backward_workspace(int32_t num_tokens, int32_t hidden)
{
    if (check_rows_dims(num_tokens, hidden) != EP_OK)
        return 0;
    return size_t(rms_norm_parts(num_tokens)) * hidden * sizeof(float);
}

int ep_rms_norm_backward(int32_t num_tokens, int32_t hidden, const void *dout, const void *h,
                         const void *weight, const float *rstd, const void *dresidual, void *dx,
                         float *dweight, void *workspace, size_t workspace_bytes, ep_stream_t stream)
{
    Traced trace("ep_rms_norm_backward");
    int rc = check_rows_dims(num_tokens, hidden);
    if (rc != EP_OK)
        return rc;
    if (dweight == nullptr ||
        (num_tokens > 0 && (dout == nullptr || h == nullptr || weight == nullptr || rstd == nullptr ||
                            dx == nullptr || workspace == nullptr)))
        return EP_ERR_INVALID;
    if (!al(dout, 16) || !al(h, 16) || !al(weight, 16) || !al(dresidual, 16) || !al(dx, 16) ||
        !al(workspace, 16) || !al(rstd, 4) || !al(dweight, 4))
        return EP_ERR_ALIGN;
    if (workspace_bytes < ep_rms_norm_backward_workspace(num_tokens, hidden))
        return EP_ERR_CAPACITY;
    return done(launch_rms_norm_backward(num_tokens, hidden, dout, h, weight, rstd, dresidual, dx,
                                         dweight, static_cast<float *>(workspace),
                                         static_cast<hipStream_t>(stream)));
}

int ep_fp8_product(int32_t m, int32_t n, int32_t k, const void *a_q, const float *a_scale,
                   const void *w_q, const float *w_scale, void *out, ep_stream_t stream)
{
    Traced trace("ep_fp8_product");
    if (m < 0 || m > kMaxTokens || n <= 0 || n > kMaxHidden || k <= 0 || k > kMaxHidden)
        return EP_ERR_INVALID;
    if (k % 128 != 0 || n % 8 != 0)
        return EP_ERR_ALIGN;
    if (m > 0 && (a_q == nullptr || a_scale == nullptr || w_q == nullptr || w_scale == nullptr ||
                  out == nullptr))
        return EP_ERR_INVALID;
    if (!al(a_q, 16) || !al(w_q, 16) || !al(out, 16) || !al(a_scale, 4) || !al(w_scale, 4))
        return EP_ERR_ALIGN;
    if (!grids_fit(m, 1, n, 128, false))
        return EP_ERR_INVALID;
    if (m == 0)
        return EP_OK;
    return done(launch_fp8_product(m, n, k, a_q, a_scale, w_q, w_scale, out,
                                   static_cast<hipStream_t>(stream)));
}

int ep_ll_expert_ffn(const ep_dims *dims, int32_t num_slots, int32_t inter, const void *packed_x,
                     const int32_t *packed_count, const void *w13, const void *w2, void *act, void *out,
                     ep_stream_t stream)
{
    Traced trace("ep_ll_expert_ffn");
    int rc = check_expert_dims(dims, inter, 8);
    if (rc != EP_OK)
        return rc;
    if (num_slots < 1 || num_slots > kMaxLLSlots)
        return EP_ERR_INVALID;
    if (dims->num_tokens > num_slots)
        return EP_ERR_CAPACITY;
    if (packed_x == nullptr || packed_count == nullptr || w13 == nullptr || w2 == nullptr ||
        act == nullptr || out == nullptr)
        return EP_ERR_INVALID;
    if (!al(packed_x, 16) || !al(w13, 16) || !al(w2, 16) || !al(act, 16) || !al(out, 16) ||
        !al(packed_count, 4))
        return EP_ERR_ALIGN;
    const int64_t pairs = int64_t(dims->num_tokens) * dims->num_topk;
    if (!grids_fit(pairs, dims->num_experts, dims->hidden, inter, false))
        return EP_ERR_INVALID;
    if (pairs == 0)
        return EP_OK;
    return done(launch_ll_expert_ffn(dims->num_experts, dims->num_ranks, num_slots, dims->hidden, inter,
                                     pairs, packed_count, packed_x, w13, w2, act, out,
                                     static_cast<hipStream_t>(stream)));
}

int ep_ll_expert_ffn_fp8(const ep_dims *dims, int32_t num_slots, int32_t inter, const void *packed_q,
                         const float *packed_scale, const int32_t *packed_count, const void *w13_q,
                         const float *w13_scale, const void *w2_q, const float *w2_scale, void *act_q,
                         float *act_scale, void *out, ep_stream_t stream)
{
    Traced trace("ep_ll_expert_ffn_fp8");
    int rc = check_expert_dims(dims, inter, 128);
    if (rc != EP_OK)
        return rc;
    if (num_slots < 1 || num_slots > kMaxLLSlots)
        return EP_ERR_INVALID;
    if (dims->num_tokens > num_slots)
        return EP_ERR_CAPACITY;
    if (packed_q == nullptr || packed_scale == nullptr || packed_count == nullptr || w13_q == nullptr ||
        w13_scale == nullptr || w2_q == nullptr || w2_scale == nullptr || act_q == nullptr ||
        act_scale == nullptr || out == nullptr)
        return EP_ERR_INVALID;
    if (!al(packed_q, 16) || !al(w13_q, 16) || !al(w2_q, 16) || !al(act_q, 16) || !al(out, 16) ||
        !al(packed_scale, 4) || !al(packed_count, 4) || !al(w13_scale, 4) || !al(w2_scale, 4) ||
        !al(act_scale, 4))
        return EP_ERR_ALIGN;
    const int64_t pairs = int64_t(dims->num_tokens) * dims->num_topk;
    if (!grids_fit(pairs, dims->num_experts, dims->hidden, inter, false))
        return EP_ERR_INVALID;
    if (pairs == 0)
        return EP_OK;
    return done(launch_ll_expert_ffn_fp8(dims->num_experts, dims->num_ranks, num_slots, dims->hidden,
                                         inter, pairs, packed_count, packed_q, packed_scale, w13_q,
                                         w13_scale, w2_q, w2_scale, act_q, act_scale, out,
                                         static_cast<hipStream_t>(stream)));
}

int ep_expert_rows(const ep_dims *dims, const int32_t *rank_prefix, const int64_t *recv_topk_idx,
                   int64_t num_rows, int64_t pair_cap, int32_t *counts, int32_t *expert_offsets,
                   int32_t *pair_row, int32_t *pair_slot, int32_t *row_pair, ep_stream_t stream)
{
    Traced trace("ep_expert_rows");
    int rc = check_expert_dims(dims, 8, 8);
    if (rc != EP_OK)
        return rc;
    if (rank_prefix == nullptr || counts == nullptr || (num_rows > 0 && recv_topk_idx == nullptr))
        return EP_ERR_INVALID;
    const ep_expert_groups g{num_rows, pair_cap, expert_offsets, pair_row, pair_slot, row_pair};
    rc = check_groups(dims, &g);
    if (rc != EP_OK)
        return rc;
    if (!al(rank_prefix, 4) || !al(recv_topk_idx, 8) || !al(counts, 4))
        return EP_ERR_ALIGN;
    const int64_t rows = num_rows < dims->num_tokens ? num_rows : dims->num_tokens;
    if (pair_cap < rows * dims->num_topk)
        return EP_ERR_CAPACITY;
    return done(launch_expert_rows(dims->num_experts, dims->num_experts / dims->num_ranks,
                                   dims->num_topk, num_rows, rank_prefix, recv_topk_idx, pair_cap, counts,
                                   expert_offsets, pair_row, pair_slot, row_pair,
                                   static_cast<hipStream_t>(stream)));
}

int ep_expert_ffn(const ep_dims *dims, int32_t inter, const ep_expert_groups *groups, const void *x,
                  const float *topk_weights, const void *w13, const void *w2, void *act, float *gate_up,
                  float *terms, void *y, ep_stream_t stream)
{
    Traced trace("ep_expert_ffn");
    int rc = check_expert_dims(dims, inter, 8);
    if (rc == EP_OK)
        rc = check_groups(dims, groups);
    if (rc != EP_OK)
        return rc;
    if (w13 == nullptr || w2 == nullptr ||
        (groups->num_rows > 0 && (x == nullptr || topk_weights == nullptr || y == nullptr)) ||
        (groups->pair_cap > 0 && (act == nullptr || terms == nullptr)))
        return EP_ERR_INVALID;
    if (!al(x, 16) || !al(w13, 16) || !al(w2, 16) || !al(act, 16) || !al(gate_up, 16) || !al(terms, 16) ||
        !al(y, 16) || !al(topk_weights, 4))
        return EP_ERR_ALIGN;
    if (!grids_fit(groups->pair_cap, dims->num_experts, dims->hidden, inter, false))
        return EP_ERR_INVALID;
    return done(launch_expert_ffn(ffn_of(dims, inter, groups, topk_weights), x, w13, w2, act, gate_up,
                                  terms, y, static_cast<hipStream_t>(stream)));
}

int ep_expert_ffn_backward(const ep_dims *dims, int32_t inter, const ep_expert_groups *groups,
                           const void *dy, const void *x, const float *topk_weights, const void *w13,
                           const void *w2, const float *gate_up, void *dgate_up, void *act, float *terms,
                           float *parts, void *dx, float *dtopk_weights, void *dw13, void *dw2,
                           ep_stream_t stream)
{
    Traced trace("ep_expert_ffn_backward");
    int rc = check_expert_dims(dims, inter, 8);
    if (rc == EP_OK)
        rc = check_groups(dims, groups);
    if (rc != EP_OK)
        return rc;
    if (w13 == nullptr || w2 == nullptr || dw13 == nullptr || dw2 == nullptr ||
        (groups->num_rows > 0 && (dy == nullptr || x == nullptr || topk_weights == nullptr ||
                                  dx == nullptr || dtopk_weights == nullptr)) ||
        (groups->pair_cap > 0 && (gate_up == nullptr || dgate_up == nullptr || act == nullptr ||
                                  terms == nullptr || parts == nullptr)))
        return EP_ERR_INVALID;
    if (!al(dy, 16) || !al(x, 16) || !al(w13, 16) || !al(w2, 16) || !al(gate_up, 16) ||
        !al(dgate_up, 16) || !al(act, 16) || !al(terms, 16) || !al(dx, 16) || !al(dw13, 16) ||
        !al(dw2, 16) || !al(parts, 4) || !al(topk_weights, 4) || !al(dtopk_weights, 4))
        return EP_ERR_ALIGN;
    if (!grids_fit(groups->pair_cap, dims->num_experts, dims->hidden, inter, true))
        return EP_ERR_INVALID;
    return done(launch_expert_ffn_backward(ffn_of(dims, inter, groups, topk_weights), dy, x, w13, w2,
                                           gate_up, dgate_up, act, parts, terms, dx, dtopk_weights, dw13,
                                           dw2, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
