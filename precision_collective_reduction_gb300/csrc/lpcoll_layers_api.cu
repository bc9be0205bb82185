// lpcoll_layers_api.cu -- entry points of the operators around the collectives
// of a layer: argument checks on the host, then the kernels' launchers. The
// semantics of each call are documented in include/lpcoll.h.
#include <math.h>

#include "lpcoll_checks.h"
#include "lpcoll_layers.cuh"

namespace lpc {

namespace {

constexpr size_t kMaxIndex = 0x7FFFFFFF;  // rows and slots are counted in int32

// A pointer to `count` elements; none are needed for an empty array.
int check_array(const void *p, size_t count) { return count == 0 ? LPCOLL_OK : check_ptr(p); }

// As check_array for an array that may be left out.
int check_optional(const void *p) { return p == nullptr || !misaligned(p) ? LPCOLL_OK : LPCOLL_ERR_ALIGN; }

// Sizes of the calls that move rows (dispatch, combine and its gradient).
int check_rows(size_t ntokens, int topk, size_t nrows, size_t hidden, int dtype)
{
    if (bad_dtype(dtype) || topk < 1 || topk > LPCOLL_MAX_TOPK)
        return LPCOLL_ERR_ARG;
    if (ntokens > kMaxIndex / static_cast<size_t>(topk) || nrows > kMaxIndex)
        return LPCOLL_ERR_ARG;
    // the grids: CTAs of 256 lanes along every token's row
    constexpr size_t kMaxCtas = static_cast<size_t>(1) << 30;
    const size_t per_token = hidden / 256 + 1;
    if (ntokens != 0 && per_token > kMaxCtas / ntokens)
        return LPCOLL_ERR_ARG;
    return LPCOLL_OK;
}

int check_norm(int gate_kind, float eps, size_t ntokens, size_t hidden, int dtype)
{
    if (bad_dtype(dtype) || gate_kind < LPCOLL_GATE_NONE || gate_kind > LPCOLL_GATE_FULL)
        return LPCOLL_ERR_ARG;
    if (!(eps > 0.0f) || isinf(eps) || ntokens > kMaxIndex)
        return LPCOLL_ERR_ARG;
    return hidden > LPCOLL_MAX_HIDDEN ? LPCOLL_ERR_UNSUPPORTED : LPCOLL_OK;
}

size_t gate_elems(int gate_kind, size_t ntokens, size_t hidden)
{
    switch (gate_kind) {
    case LPCOLL_GATE_CHANNEL: return hidden;
    case LPCOLL_GATE_TOKEN: return ntokens;
    case LPCOLL_GATE_FULL: return ntokens * hidden;
    default: return 0;
    }
}

size_t norm_workspace(size_t ntokens, size_t hidden, int dtype)
{
    return static_cast<size_t>(2) * norm_backward_parts(ntokens, hidden, dtype) * hidden *
           sizeof(float);
}

int check_route(int dtype, size_t ntokens, int nexperts, int topk)
{
    if (bad_dtype(dtype) || nexperts < 1 || nexperts > LPCOLL_MAX_EXPERTS || topk < 1 ||
        topk > LPCOLL_MAX_TOPK || topk > nexperts)
        return LPCOLL_ERR_ARG;
    return ntokens > kMaxIndex / static_cast<size_t>(topk) ? LPCOLL_ERR_ARG : LPCOLL_OK;
}

}  // namespace

}  // namespace lpc

using namespace lpc;

extern "C" {

int expert_route(const void *logits, lpcoll_dtype dtype, size_t ntokens, int nexperts, int topk,
                 int renormalize, int32_t *ids, float *weights, void *stream)
{
    int st = check_route(dtype, ntokens, nexperts, topk);
    if (st != LPCOLL_OK || ntokens == 0)
        return st;
    st = first_error({check_ptr(logits), check_ptr(ids), check_ptr(weights)});
    if (st != LPCOLL_OK)
        return st;
    const size_t slots = ntokens * topk;
    debug_begin();
    debug_range(logits, ntokens * nexperts * elem_bytes(dtype), false);
    debug_range(ids, slots * sizeof(int32_t), true);
    debug_range(weights, slots * sizeof(float), true);
    RouteArgs a = {};
    a.logits = logits;
    a.ids = ids;
    a.weights = weights;
    a.tokens = ntokens;
    a.experts = nexperts;
    a.topk = topk;
    a.renormalize = renormalize;
    a.dtype = dtype;
    return finish(launch_route(a, static_cast<cudaStream_t>(stream)));
}

int expert_route_backward(const void *logits, lpcoll_dtype dtype, size_t ntokens, int nexperts,
                          int topk, int renormalize, const int32_t *ids, const float *weights,
                          const float *dweights, void *dlogits, void *stream)
{
    int st = check_route(dtype, ntokens, nexperts, topk);
    if (st != LPCOLL_OK || ntokens == 0)
        return st;
    st = first_error({renormalize ? LPCOLL_OK : check_ptr(logits), check_ptr(ids),
                      check_ptr(weights), check_ptr(dweights), check_ptr(dlogits)});
    if (st != LPCOLL_OK)
        return st;
    const size_t slots = ntokens * topk, all = ntokens * nexperts * elem_bytes(dtype);
    debug_begin();
    if (!renormalize)
        debug_range(logits, all, false);
    debug_range(ids, slots * sizeof(int32_t), false);
    debug_range(weights, slots * sizeof(float), false);
    debug_range(dweights, slots * sizeof(float), false);
    debug_range(dlogits, all, true);
    RouteArgs a = {};
    a.logits = logits;
    a.ids = const_cast<int32_t *>(ids);
    a.weights = const_cast<float *>(weights);
    a.dweights = dweights;
    a.dlogits = dlogits;
    a.tokens = ntokens;
    a.experts = nexperts;
    a.topk = topk;
    a.renormalize = renormalize;
    a.dtype = dtype;
    return finish(launch_route_backward(a, static_cast<cudaStream_t>(stream)));
}

size_t expert_sort_workspace_bytes(size_t nslots, int nexperts)
{
    if (nexperts < 1 || nexperts > LPCOLL_MAX_EXPERTS || nslots > kMaxIndex)
        return 0;
    const int chunks = sort_chunks(nslots);
    return chunks > 1 ? static_cast<size_t>(chunks) * nexperts * sizeof(int32_t) : 0;
}

int expert_sort(const int32_t *ids, size_t nslots, int nexperts, size_t capacity,
                int32_t *slot_row, int32_t *row_slot, int32_t *offsets, int32_t *counts,
                void *workspace, size_t workspace_bytes, void *stream)
{
    if (nexperts < 1 || nexperts > LPCOLL_MAX_EXPERTS || nslots > kMaxIndex ||
        capacity > kMaxIndex / static_cast<size_t>(nexperts))
        return LPCOLL_ERR_ARG;
    const size_t need = expert_sort_workspace_bytes(nslots, nexperts);
    if (workspace_bytes < need)
        return LPCOLL_ERR_ARG;
    const size_t rows = capacity > 0 ? capacity * nexperts : nslots;
    const int st = first_error({check_array(ids, nslots), check_array(slot_row, nslots),
                                check_array(row_slot, rows), check_ptr(offsets),
                                check_ptr(counts), check_array(workspace, need)});
    if (st != LPCOLL_OK)
        return st;
    debug_begin();
    debug_range(ids, nslots * sizeof(int32_t), false);
    debug_range(slot_row, nslots * sizeof(int32_t), true);
    debug_range(row_slot, rows * sizeof(int32_t), true);
    debug_range(offsets, (static_cast<size_t>(nexperts) + 1) * sizeof(int32_t), true);
    debug_range(counts, static_cast<size_t>(nexperts) * sizeof(int32_t), true);
    debug_range(workspace, need, true);
    SortArgs a = {};
    a.ids = ids;
    a.slot_row = slot_row;
    a.row_slot = row_slot;
    a.offsets = offsets;
    a.counts = counts;
    a.chunk_counts = static_cast<int32_t *>(workspace);
    a.slots = static_cast<int>(nslots);
    a.experts = nexperts;
    a.capacity = static_cast<int>(capacity);
    a.rows = static_cast<int>(rows);
    return finish(launch_sort(a, static_cast<cudaStream_t>(stream)));
}

int expert_dispatch(const void *x, size_t ntokens, int topk, size_t nrows, size_t hidden,
                    lpcoll_dtype dtype, int block, const int32_t *slot_row,
                    const int32_t *row_slot, void *out, uint8_t *codes, float *scales,
                    void *stream)
{
    int st = check_rows(ntokens, topk, nrows, hidden, dtype);
    if (st != LPCOLL_OK)
        return st;
    if (block != 0 && block != LPCOLL_BLOCK)
        return LPCOLL_ERR_UNSUPPORTED;
    if (nrows == 0 || hidden == 0)
        return LPCOLL_OK;
    const bool lp = block != 0;
    st = first_error({check_array(x, ntokens), check_array(slot_row, ntokens),
                      check_ptr(row_slot), lp ? LPCOLL_OK : check_ptr(out),
                      lp ? check_ptr(codes) : LPCOLL_OK, lp ? check_ptr(scales) : LPCOLL_OK});
    if (st != LPCOLL_OK)
        return st;
    debug_begin();
    debug_range(x, ntokens * hidden * elem_bytes(dtype), false);
    debug_range(slot_row, ntokens * topk * sizeof(int32_t), false);
    debug_range(row_slot, nrows * sizeof(int32_t), false);
    if (lp) {
        debug_range(codes, nrows * hidden, true);
        debug_range(scales, nrows * blocks_of(hidden, block) * sizeof(float), true);
    } else {
        debug_range(out, nrows * hidden * elem_bytes(dtype), true);
    }
    RowsArgs a = {};
    a.x = x;
    a.out = out;
    a.codes = codes;
    a.scales = scales;
    a.slot_row = slot_row;
    a.row_slot = row_slot;
    a.tokens = ntokens;
    a.nrows = nrows;
    a.hidden = hidden;
    a.topk = topk;
    a.dtype = dtype;
    return finish(launch_dispatch(a, lp, static_cast<cudaStream_t>(stream)));
}

int expert_combine(const void *rows, const uint8_t *codes, const float *scales, size_t ntokens,
                   int topk, size_t nrows, size_t hidden, lpcoll_dtype dtype, int block,
                   const int32_t *slot_row, const float *weights, void *out, void *stream)
{
    int st = check_rows(ntokens, topk, nrows, hidden, dtype);
    if (st != LPCOLL_OK)
        return st;
    if (block != 0 && block != LPCOLL_BLOCK)
        return LPCOLL_ERR_UNSUPPORTED;
    if (ntokens == 0 || hidden == 0)
        return LPCOLL_OK;
    const bool lp = block != 0;
    st = first_error({lp ? LPCOLL_OK : check_array(rows, nrows),
                      lp ? check_array(codes, nrows) : LPCOLL_OK,
                      lp ? check_array(scales, nrows) : LPCOLL_OK, check_ptr(slot_row),
                      check_optional(weights), check_ptr(out)});
    if (st != LPCOLL_OK)
        return st;
    debug_begin();
    if (lp) {
        debug_range(codes, nrows * hidden, false);
        debug_range(scales, nrows * blocks_of(hidden, block) * sizeof(float), false);
    } else {
        debug_range(rows, nrows * hidden * elem_bytes(dtype), false);
    }
    debug_range(slot_row, ntokens * topk * sizeof(int32_t), false);
    debug_range(weights, ntokens * topk * sizeof(float), false);
    debug_range(out, ntokens * hidden * elem_bytes(dtype), true);
    RowsArgs a = {};
    a.rows = rows;
    a.codes = const_cast<uint8_t *>(codes);
    a.scales = const_cast<float *>(scales);
    a.weights = weights;
    a.out = out;
    a.slot_row = slot_row;
    a.tokens = ntokens;
    a.nrows = nrows;
    a.hidden = hidden;
    a.topk = topk;
    a.dtype = dtype;
    return finish(launch_combine(a, lp, static_cast<cudaStream_t>(stream)));
}

int expert_combine_backward(const void *dout, const void *rows, size_t ntokens, int topk,
                            size_t nrows, size_t hidden, lpcoll_dtype dtype,
                            const int32_t *slot_row, const int32_t *row_slot,
                            const float *weights, void *drows, float *dweights, void *stream)
{
    int st = check_rows(ntokens, topk, nrows, hidden, dtype);
    if (st != LPCOLL_OK)
        return st;
    const size_t slots = ntokens * topk, all = nrows * hidden;
    if (all == 0 && (slots == 0 || dweights == nullptr))
        return LPCOLL_OK;
    st = first_error({check_array(dout, ntokens * hidden),
                      dweights != nullptr ? check_array(rows, all) : LPCOLL_OK,
                      check_array(slot_row, slots), check_array(row_slot, nrows),
                      check_optional(weights), check_array(drows, all),
                      check_optional(dweights)});
    if (st != LPCOLL_OK)
        return st;
    debug_begin();
    debug_range(dout, ntokens * hidden * elem_bytes(dtype), false);
    if (dweights != nullptr)
        debug_range(rows, all * elem_bytes(dtype), false);
    debug_range(slot_row, slots * sizeof(int32_t), false);
    debug_range(row_slot, nrows * sizeof(int32_t), false);
    debug_range(weights, slots * sizeof(float), false);
    debug_range(drows, all * elem_bytes(dtype), true);
    debug_range(dweights, slots * sizeof(float), true);
    RowsArgs a = {};
    a.x = dout;
    a.rows = rows;
    a.weights = weights;
    a.out = drows;
    a.dweights = dweights;
    a.slot_row = slot_row;
    a.row_slot = row_slot;
    a.tokens = ntokens;
    a.nrows = nrows;
    a.hidden = hidden;
    a.topk = topk;
    a.dtype = dtype;
    return finish(launch_combine_backward(a, static_cast<cudaStream_t>(stream)));
}

int residual_norm(const void *const *h, int nranks, const void *x, const void *gate,
                  int gate_kind, const void *w_post, const void *w_pre, float res_scale,
                  float branch_scale, float eps, size_t ntokens, size_t hidden,
                  lpcoll_dtype dtype, void *x_out, void *n_out, void *h_sum, void *stream)
{
    int st = check_norm(gate_kind, eps, ntokens, hidden, dtype);
    if (st == LPCOLL_OK && (nranks < 1 || nranks > LPCOLL_MAX_RANKS))
        st = LPCOLL_ERR_ARG;
    if (st != LPCOLL_OK || ntokens == 0 || hidden == 0)
        return st;
    st = first_error({check_rank_array(h, nranks), check_ptr(x),
                      gate_kind != LPCOLL_GATE_NONE ? check_ptr(gate) : LPCOLL_OK,
                      check_optional(w_post), check_optional(w_pre), check_ptr(x_out),
                      w_pre != nullptr ? check_ptr(n_out) : LPCOLL_OK, check_optional(h_sum)});
    if (st != LPCOLL_OK)
        return st;
    const size_t es = elem_bytes(dtype), all = ntokens * hidden * es;
    NormArgs a = {};
    debug_begin();
    for (int r = 0; r < nranks; ++r) {
        a.h[r] = h[r];
        debug_range(h[r], all, false);
    }
    debug_range(x, all, false);
    debug_range(gate, gate_elems(gate_kind, ntokens, hidden) * es, false);
    debug_range(w_post, hidden * es, false);
    debug_range(w_pre, hidden * es, false);
    debug_range(x_out, all, true);
    debug_range(w_pre != nullptr ? n_out : nullptr, all, true);
    debug_range(h_sum, all, true);
    a.nranks = nranks;
    a.x = x;
    a.gate = gate;
    a.w_post = w_post;
    a.w_pre = w_pre;
    a.x_out = x_out;
    a.n_out = n_out;
    a.h_sum = h_sum;
    a.gate_kind = gate_kind;
    a.res_scale = res_scale;
    a.branch_scale = branch_scale;
    a.eps = eps;
    a.tokens = ntokens;
    a.hidden = static_cast<int>(hidden);
    a.dtype = dtype;
    return finish(launch_residual_norm(a, static_cast<cudaStream_t>(stream)));
}

size_t residual_norm_backward_workspace_bytes(size_t ntokens, size_t hidden, lpcoll_dtype dtype)
{
    if (check_norm(LPCOLL_GATE_NONE, 1.0f, ntokens, hidden, dtype) != LPCOLL_OK)
        return 0;
    return norm_workspace(ntokens, hidden, dtype);
}

int residual_norm_backward(const void *dx_out, const void *dn_out, const void *h,
                           const void *x_out, const void *gate, int gate_kind,
                           const void *w_post, const void *w_pre, float res_scale,
                           float branch_scale, float eps, size_t ntokens, size_t hidden,
                           lpcoll_dtype dtype, void *dx, void *dh, void *dgate, float *dw_post,
                           float *dw_pre, void *workspace, size_t workspace_bytes, void *stream)
{
    int st = check_norm(gate_kind, eps, ntokens, hidden, dtype);
    if (st != LPCOLL_OK)
        return st;
    if (w_post == nullptr)
        dw_post = nullptr;
    if (w_pre == nullptr)
        dw_pre = nullptr;
    if (gate_kind == LPCOLL_GATE_NONE)
        dgate = nullptr;
    if (hidden == 0) {
        // rows of no elements: only a token's gate has a gradient, a sum over nothing
        if (gate_kind != LPCOLL_GATE_TOKEN || dgate == nullptr || ntokens == 0)
            return LPCOLL_OK;
        st = check_ptr(dgate);
        return st != LPCOLL_OK ? st
                               : finish(cudaMemsetAsync(dgate, 0, ntokens * sizeof(float),
                                                        static_cast<cudaStream_t>(stream)));
    }
    const size_t need = norm_workspace(ntokens, hidden, dtype);
    if (workspace_bytes < need)
        return LPCOLL_ERR_ARG;
    const size_t count = ntokens;
    st = first_error({dx_out != nullptr || w_pre != nullptr ? check_optional(dx_out)
                                                            : check_array(dx_out, count),
                      w_pre != nullptr ? check_array(dn_out, count) : LPCOLL_OK,
                      check_array(h, count), check_array(x_out, count),
                      check_array(gate, gate_elems(gate_kind, ntokens, hidden)),
                      check_optional(w_post), check_optional(w_pre), check_array(dx, count),
                      check_array(dh, count), check_optional(dgate), check_optional(dw_post),
                      check_optional(dw_pre), check_array(workspace, need)});
    if (st != LPCOLL_OK)
        return st;
    const size_t es = elem_bytes(dtype), all = ntokens * hidden * es;
    const size_t ngate = gate_elems(gate_kind, ntokens, hidden);
    debug_begin();
    debug_range(dx_out, all, false);
    debug_range(w_pre != nullptr ? dn_out : nullptr, all, false);
    debug_range(h, all, false);
    debug_range(x_out, all, false);
    debug_range(gate, ngate * es, false);
    debug_range(w_post, hidden * es, false);
    debug_range(w_pre, hidden * es, false);
    debug_range(dx, all, true);
    debug_range(dh, all, true);
    debug_range(dgate, ngate * (gate_kind == LPCOLL_GATE_FULL ? es : sizeof(float)), true);
    debug_range(dw_post, hidden * sizeof(float), true);
    debug_range(dw_pre, hidden * sizeof(float), true);
    debug_range(workspace, need, true);
    NormArgs a = {};
    a.h[0] = h;
    a.nranks = 1;
    a.x = x_out;
    a.gate = gate;
    a.w_post = w_post;
    a.w_pre = w_pre;
    a.dx_out = dx_out;
    a.dn_out = dn_out;
    a.dx = dx;
    a.dh = dh;
    a.dgate = dgate;
    a.dw_post = dw_post;
    a.dw_pre = dw_pre;
    a.partial = static_cast<float *>(workspace);
    a.gate_kind = gate_kind;
    a.res_scale = res_scale;
    a.branch_scale = branch_scale;
    a.eps = eps;
    a.tokens = ntokens;
    a.hidden = static_cast<int>(hidden);
    a.dtype = dtype;
    return finish(launch_residual_norm_backward(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
