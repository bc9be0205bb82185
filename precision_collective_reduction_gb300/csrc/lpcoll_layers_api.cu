// lpcoll_layers_api.cu -- entry points of the operators around the collectives
// of a layer: argument checks on the host, then the kernels' launchers. The
// semantics of each call are documented in include/lpcoll.h.
#include <math.h>

#include "lpcoll_checks.h"
#include "lpcoll_layers.cuh"

namespace lpc {

namespace {

constexpr size_t kMaxIndex = 0x7FFFFFFF;  // rows and slots are counted in int32
// columns of calls that LPCOLL_MAX_HIDDEN does not limit: counted in int32 too
constexpr size_t kMaxHidden = static_cast<size_t>(1) << 30;

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

// Workspace of a layer norm's gradients.
size_t layer_norm_workspace(size_t ntokens, size_t hidden, int dtype, bool dropout)
{
    return static_cast<size_t>(2) * layer_norm_parts(ntokens, hidden, dtype, dropout) * hidden *
           sizeof(float);
}

// Sizes of residual_dropout without a norm: CTAs along every token's row.
int check_dropout(float p, size_t ntokens, size_t hidden, int dtype)
{
    if (bad_dtype(dtype) || !(p >= 0.0f && p < 1.0f) || hidden > kMaxHidden)
        return LPCOLL_ERR_ARG;
    return check_rows(ntokens, 1, 0, hidden, dtype);
}

// The random words that are kept, and what a kept value is multiplied by.
DropArgs drop_args(const uint64_t *rng, float p, size_t first_row)
{
    DropArgs d;
    d.rng = reinterpret_cast<const unsigned long long *>(rng);
    d.first_row = first_row;
    d.least = static_cast<uint32_t>(static_cast<double>(p) * 4294967296.0);
    d.scale = static_cast<float>(1.0 / (1.0 - static_cast<double>(p)));
    return d;
}

int check_embed(size_t ntokens, size_t vocab, size_t hidden, int dtype, int index)
{
    if ((index != LPCOLL_I32 && index != LPCOLL_I64) || hidden > kMaxHidden)
        return LPCOLL_ERR_ARG;
    return check_rows(ntokens, 1, vocab, hidden, dtype);
}

size_t index_bytes(int index) { return index == LPCOLL_I64 ? 8 : 4; }

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

int layer_norm(const void *x, const void *w, const void *b, float eps, size_t ntokens,
               size_t hidden, lpcoll_dtype dtype, void *out, void *stream)
{
    int st = check_norm(LPCOLL_GATE_NONE, eps, ntokens, hidden, dtype);
    if (st != LPCOLL_OK || ntokens == 0 || hidden == 0)
        return st;
    st = first_error({check_ptr(x), check_optional(w), check_optional(b), check_ptr(out)});
    if (st != LPCOLL_OK)
        return st;
    const size_t es = elem_bytes(dtype), all = ntokens * hidden * es;
    debug_begin();
    debug_range(x, all, false);
    debug_range(w, hidden * es, false);
    debug_range(b, hidden * es, false);
    debug_range(out, all, true);
    LayerNormArgs a = {};
    a.x = x;
    a.w = w;
    a.b = b;
    a.n_out = out;
    a.eps = eps;
    a.tokens = ntokens;
    a.hidden = static_cast<int>(hidden);
    a.dtype = dtype;
    return finish(launch_layer_norm(a, static_cast<cudaStream_t>(stream)));
}

size_t layer_norm_backward_workspace_bytes(size_t ntokens, size_t hidden, lpcoll_dtype dtype)
{
    if (check_norm(LPCOLL_GATE_NONE, 1.0f, ntokens, hidden, dtype) != LPCOLL_OK)
        return 0;
    return layer_norm_workspace(ntokens, hidden, dtype, false);
}

int layer_norm_backward(const void *dout, const void *x, const void *w, float eps,
                        size_t ntokens, size_t hidden, lpcoll_dtype dtype, void *dx, float *dw,
                        float *db, void *workspace, size_t workspace_bytes, void *stream)
{
    int st = check_norm(LPCOLL_GATE_NONE, eps, ntokens, hidden, dtype);
    if (st != LPCOLL_OK)
        return st;
    const bool sums = dw != nullptr || db != nullptr;
    const size_t need = sums ? layer_norm_workspace(ntokens, hidden, dtype, false) : 0;
    if (workspace_bytes < need)
        return LPCOLL_ERR_ARG;
    if (hidden == 0 || (!sums && (dx == nullptr || ntokens == 0)))
        return LPCOLL_OK;
    st = first_error({check_array(dout, ntokens), check_array(x, ntokens), check_optional(w),
                      check_optional(dx), check_optional(dw), check_optional(db),
                      check_array(workspace, need)});
    if (st != LPCOLL_OK)
        return st;
    const size_t es = elem_bytes(dtype), all = ntokens * hidden * es;
    debug_begin();
    debug_range(dout, all, false);
    debug_range(x, all, false);
    debug_range(w, hidden * es, false);
    debug_range(dx, all, true);
    debug_range(dw, hidden * sizeof(float), true);
    debug_range(db, hidden * sizeof(float), true);
    debug_range(workspace, need, true);
    LayerNormArgs a = {};
    a.x = x;
    a.w = w;
    a.dn_out = dout;
    a.dx = dx;
    a.dw = dw;
    a.db = db;
    a.partial = static_cast<float *>(workspace);
    a.eps = eps;
    a.tokens = ntokens;
    a.hidden = static_cast<int>(hidden);
    a.dtype = dtype;
    return finish(launch_layer_norm_backward(a, static_cast<cudaStream_t>(stream)));
}

int residual_dropout(const void *const *h, int nranks, const void *x, const uint64_t *rng,
                     float p, size_t first_row, const void *w, const void *b, float eps,
                     size_t ntokens, size_t hidden, lpcoll_dtype dtype, void *x_out, void *n_out,
                     void *stream)
{
    int st = check_dropout(p, ntokens, hidden, dtype);
    const bool norm = n_out != nullptr;
    if (st == LPCOLL_OK && norm)
        st = check_norm(LPCOLL_GATE_NONE, eps, ntokens, hidden, dtype);
    if (st == LPCOLL_OK && (nranks < 1 || nranks > LPCOLL_MAX_RANKS))
        st = LPCOLL_ERR_ARG;
    if (st != LPCOLL_OK || ntokens == 0 || hidden == 0)
        return st;
    LayerNormArgs a = {};
    a.drop = drop_args(rng, p, first_row);
    st = first_error({check_rank_array(h, nranks), check_optional(x),
                      a.drop.least != 0 ? check_ptr(rng) : LPCOLL_OK,
                      norm ? check_optional(w) : LPCOLL_OK, norm ? check_optional(b) : LPCOLL_OK,
                      check_ptr(x_out), check_optional(n_out)});
    if (st != LPCOLL_OK)
        return st;
    const size_t es = elem_bytes(dtype), all = ntokens * hidden * es;
    debug_begin();
    for (int r = 0; r < nranks; ++r) {
        a.h[r] = h[r];
        debug_range(h[r], all, false);
    }
    debug_range(x, all, false);
    debug_range(a.drop.least != 0 ? rng : nullptr, 2 * sizeof(uint64_t), false);
    debug_range(norm ? w : nullptr, hidden * es, false);
    debug_range(norm ? b : nullptr, hidden * es, false);
    debug_range(x_out, all, true);
    debug_range(n_out, all, true);
    a.nranks = nranks;
    a.x = x;
    a.w = w;
    a.b = b;
    a.x_out = x_out;
    a.n_out = n_out;
    a.eps = eps;
    a.tokens = ntokens;
    a.hidden = static_cast<int>(hidden);
    a.dtype = dtype;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return finish(norm ? launch_dropout_norm(a, s) : launch_dropout(a, s));
}

size_t residual_dropout_backward_workspace_bytes(size_t ntokens, size_t hidden,
                                                 lpcoll_dtype dtype)
{
    if (check_norm(LPCOLL_GATE_NONE, 1.0f, ntokens, hidden, dtype) != LPCOLL_OK)
        return 0;
    return layer_norm_workspace(ntokens, hidden, dtype, true);
}

int residual_dropout_backward(const void *dx_out, const void *dn_out, const void *x_out,
                              const uint64_t *rng, float p, size_t first_row, const void *w,
                              float eps, size_t ntokens, size_t hidden, lpcoll_dtype dtype,
                              void *dx, void *dh, float *dw, float *db, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    int st = check_dropout(p, ntokens, hidden, dtype);
    const bool sums = dw != nullptr || db != nullptr;
    const bool norm = dn_out != nullptr;
    if (st == LPCOLL_OK && (norm || sums))
        st = check_norm(LPCOLL_GATE_NONE, eps, ntokens, hidden, dtype);
    if (st != LPCOLL_OK)
        return st;
    const size_t need = norm && sums ? layer_norm_workspace(ntokens, hidden, dtype, true) : 0;
    if (workspace_bytes < need)
        return LPCOLL_ERR_ARG;
    const bool rows = ntokens != 0 && (dx != nullptr || dh != nullptr);
    if (hidden == 0 || (!sums && !rows))
        return LPCOLL_OK;
    LayerNormArgs a = {};
    a.drop = drop_args(rng, p, first_row);
    if (dh == nullptr)  // the generator is not read
        a.drop.least = 0;
    const bool drop = a.drop.least != 0;
    st = first_error({norm || !rows ? check_optional(dx_out) : check_ptr(dx_out),
                      check_optional(dn_out), norm ? check_array(x_out, ntokens) : LPCOLL_OK,
                      drop && ntokens != 0 ? check_ptr(rng) : LPCOLL_OK,
                      norm ? check_optional(w) : LPCOLL_OK, check_optional(dx),
                      check_optional(dh), check_optional(dw), check_optional(db),
                      check_array(workspace, need)});
    if (st != LPCOLL_OK)
        return st;
    const size_t es = elem_bytes(dtype), all = ntokens * hidden * es;
    debug_begin();
    debug_range(dx_out, all, false);
    debug_range(dn_out, all, false);
    debug_range(norm ? x_out : nullptr, all, false);
    debug_range(drop ? rng : nullptr, 2 * sizeof(uint64_t), false);
    debug_range(norm ? w : nullptr, hidden * es, false);
    debug_range(dx, all, true);
    debug_range(dh, all, true);
    debug_range(dw, hidden * sizeof(float), true);
    debug_range(db, hidden * sizeof(float), true);
    debug_range(workspace, need, true);
    a.tokens = ntokens;
    a.hidden = static_cast<int>(hidden);
    a.dtype = dtype;
    a.dx = dx;
    a.dw = dw;
    a.db = db;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (norm) {
        a.x = x_out;
        a.w = w;
        a.dx_out = dx_out;
        a.dn_out = dn_out;
        a.dh = dh;
        a.partial = static_cast<float *>(workspace);
        a.eps = eps;
        return finish(launch_dropout_norm_backward(a, s));
    }
    // without the norm's part, dh is dx_out through the same mask
    a.h[0] = dx_out;
    a.nranks = 1;
    a.x_out = dh;
    cudaError_t e = rows ? launch_dropout(a, s) : cudaSuccess;
    if (e == cudaSuccess && sums)
        e = launch_layer_norm_sums(a, 0, s);
    return finish(e);
}

size_t expert_balance_workspace_bytes(size_t ntokens, int nexperts)
{
    if (check_route(LPCOLL_F32, ntokens, nexperts, 1) != LPCOLL_OK)
        return 0;
    return balance_workspace(ntokens, nexperts);
}

int expert_balance(const void *logits, lpcoll_dtype dtype, size_t ntokens, int nexperts,
                   const int32_t *ids, int topk, const uint8_t *valid, float coef, float *loss,
                   int32_t *counts, float *prob_sums, void *workspace, size_t workspace_bytes,
                   void *stream)
{
    int st = check_route(dtype, ntokens, nexperts, topk);
    if (st != LPCOLL_OK)
        return st;
    const size_t need = balance_workspace(ntokens, nexperts);
    if (workspace_bytes < need)
        return LPCOLL_ERR_ARG;
    st = first_error({check_array(logits, ntokens), check_array(ids, ntokens),
                      check_optional(valid), check_ptr(loss), check_ptr(counts),
                      check_ptr(prob_sums), check_array(workspace, need)});
    if (st != LPCOLL_OK)
        return st;
    debug_begin();
    debug_range(logits, ntokens * nexperts * elem_bytes(dtype), false);
    debug_range(ids, ntokens * topk * sizeof(int32_t), false);
    debug_range(valid, ntokens, false);
    debug_range(loss, sizeof(float), true);
    debug_range(counts, (static_cast<size_t>(nexperts) + 1) * sizeof(int32_t), true);
    debug_range(prob_sums, nexperts * sizeof(float), true);
    debug_range(workspace, need, true);
    BalanceArgs a = {};
    a.logits = logits;
    a.ids = ids;
    a.valid = valid;
    a.loss = loss;
    a.counts = counts;
    a.prob_sums = prob_sums;
    a.rows = static_cast<float *>(workspace);
    a.coef = coef;
    a.tokens = ntokens;
    a.experts = nexperts;
    a.topk = topk;
    a.dtype = dtype;
    return finish(launch_balance(a, static_cast<cudaStream_t>(stream)));
}

int expert_balance_backward(const void *logits, lpcoll_dtype dtype, size_t ntokens, int nexperts,
                            const uint8_t *valid, const int32_t *counts, float coef,
                            const float *dloss, int accumulate, void *dlogits, void *stream)
{
    int st = check_route(dtype, ntokens, nexperts, 1);
    if (st != LPCOLL_OK || ntokens == 0)
        return st;
    st = first_error({check_ptr(logits), check_optional(valid), check_ptr(counts),
                      check_ptr(dloss), check_ptr(dlogits)});
    if (st != LPCOLL_OK)
        return st;
    const size_t all = ntokens * nexperts * elem_bytes(dtype);
    debug_begin();
    debug_range(logits, all, false);
    debug_range(valid, ntokens, false);
    debug_range(counts, (static_cast<size_t>(nexperts) + 1) * sizeof(int32_t), false);
    debug_range(dloss, sizeof(float), false);
    debug_range(dlogits, all, true);
    BalanceArgs a = {};
    a.logits = logits;
    a.valid = valid;
    a.counts = const_cast<int32_t *>(counts);
    a.dloss = dloss;
    a.dlogits = dlogits;
    a.coef = coef;
    a.tokens = ntokens;
    a.experts = nexperts;
    a.topk = 1;
    a.dtype = dtype;
    a.accumulate = accumulate;
    return finish(launch_balance_backward(a, static_cast<cudaStream_t>(stream)));
}

int token_embed(const void *table, size_t vocab, const void *ids, lpcoll_index index,
                int64_t first_id, size_t ntokens, size_t hidden, lpcoll_dtype dtype, float scale,
                void *out, void *stream)
{
    int st = check_embed(ntokens, vocab, hidden, dtype, index);
    if (st != LPCOLL_OK || ntokens == 0 || hidden == 0)
        return st;
    st = first_error({check_array(table, vocab), check_ptr(ids), check_ptr(out)});
    if (st != LPCOLL_OK)
        return st;
    const size_t row = hidden * elem_bytes(dtype);
    debug_begin();
    debug_range(table, vocab * row, false);
    debug_range(ids, ntokens * index_bytes(index), false);
    debug_range(out, ntokens * row, true);
    EmbedArgs a = {};
    a.table = table;
    a.out = out;
    a.ids = ids;
    a.ids64 = index == LPCOLL_I64;
    a.first_id = first_id;
    a.scale = scale;
    a.tokens = ntokens;
    a.vocab = vocab;
    a.hidden = hidden;
    a.dtype = dtype;
    return finish(launch_embed(a, static_cast<cudaStream_t>(stream)));
}

size_t token_embed_backward_workspace_bytes(size_t ntokens, size_t vocab, size_t hidden)
{
    if (check_embed(ntokens, vocab, hidden, LPCOLL_F32, LPCOLL_I32) != LPCOLL_OK)
        return 0;
    return embed_workspace(ntokens, vocab, hidden);
}

int token_embed_backward(const void *dout, const void *ids, lpcoll_index index, int64_t first_id,
                         size_t ntokens, size_t vocab, size_t hidden, lpcoll_dtype dtype,
                         float scale, int accumulate, float *dtable, void *workspace,
                         size_t workspace_bytes, void *stream)
{
    int st = check_embed(ntokens, vocab, hidden, dtype, index);
    if (st != LPCOLL_OK)
        return st;
    const size_t need = embed_workspace(ntokens, vocab, hidden);
    if (workspace_bytes < need)
        return LPCOLL_ERR_ARG;
    if (vocab == 0 || hidden == 0 || (ntokens == 0 && accumulate))
        return LPCOLL_OK;
    st = first_error({check_array(dout, ntokens), check_array(ids, ntokens), check_ptr(dtable),
                      check_array(workspace, need)});
    if (st != LPCOLL_OK)
        return st;
    debug_begin();
    debug_range(dout, ntokens * hidden * elem_bytes(dtype), false);
    debug_range(ids, ntokens * index_bytes(index), false);
    debug_range(dtable, vocab * hidden * sizeof(float), true);
    debug_range(workspace, need, true);
    EmbedArgs a = {};
    a.dout = dout;
    a.dtable = dtable;
    a.ids = ids;
    a.ids64 = index == LPCOLL_I64;
    a.first_id = first_id;
    a.scale = scale;
    a.tokens = ntokens;
    a.vocab = vocab;
    a.hidden = hidden;
    a.dtype = dtype;
    a.accumulate = accumulate;
    a.workspace = workspace;
    return finish(launch_embed_backward(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
