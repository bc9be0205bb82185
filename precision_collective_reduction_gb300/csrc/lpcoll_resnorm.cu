// lpcoll_resnorm.cu -- the end of a transformer block in one pass: the sum of
// the ranks' partial products, the norm after the block, gate, residual and
// the norm before the next block (residual_norm), and the gradients
// (residual_norm_backward).
//
//   h  = sum_r h_r                                    (rank order)
//   u  = h r1 w_post,   r1 = 1 / sqrt(mean h^2 + eps)   (or u = h)
//   x' = alpha x + beta g u
//   n  = x' r2 w_pre,   r2 = 1 / sqrt(mean x'^2 + eps)
//
// Every input is read and every output written once; all arithmetic and sums
// are FP32, rounded once at each output. HBM traffic bounds both directions
// once there are enough tokens.
//
// A row belongs to a "team" of whole warps: a part of a CTA for short rows, a
// CTA, or the CTAs of a cluster, which add up their sums through distributed
// shared memory. A thread of a team always holds the same columns, so what
// the weights and gates of a channel give stays in its registers, and a team
// goes through its rows one after the other while its next rows are on their
// way into shared memory (cp.async): each thread copies and reads its own
// columns only, so no barrier guards them. Where shared memory holds one row of a
// team (8 ranks of 4096 or 8192 BF16 columns, the FP32 gradient of 8192), a forward
// team sends for its next row once this one's columns are read, before the sums
// meet, and a gradient's team at the row's end. Rows of that many bytes keep DRAM
// busy all the same: 8192 x 8192 of 8 ranks 238 us, 4096 x 8192 FP32 gradient 132 us
// (bytes at the copy rate: 238 and 119).
//
// Measured on one GB300, BF16: 16384 x 8192 forward 161 us (6.7 TB/s, DRAM), the
// gradient of 8192 x 8192 124 us (6.5 TB/s; a team's phases between barriers), 32
// x 8192 of 8 ranks 5.7 us (latency).
#include "lpcoll_rows.cuh"

namespace lpc {

namespace {

// Forms of both kernels. kPlain is for calls without clusters in which every
// thread has all its columns, both norms are there, one rank's h, no full gate
// and, in the gradient, dx_out: without the conditions around every access the compiler
// interleaves a thread's accesses (gradient of 8192 x 8192 BF16 143 -> 134 us). Calls
// without it pay: 16384 x 8192 BF16 with the second norm alone 216 us, with both 161.
// kWide is for the forward pass of rows of more than 8192 columns, in a CTA of
// 1024 threads with 16 columns each at 64 registers a thread, the weights from
// L1 each time (8192 x 12288 BF16: 167 us, 241 with a cluster of two CTAs and the
// weights in registers; the gradient of 4096 rows, which keeps its sums too, 268
// against 174; 180 now, the price of the unaligned cluster barriers).

// Streams of a row: x, a full gate if there is one, then the ranks' h.
template <int DT, int W, int kElems, int kMode>
__global__ void __launch_bounds__(kMode == kWide ? kWideThreads : kThreadsOne<kElems>, 1)
residual_norm_kernel(const __grid_constant__ NormArgs a, const Deal deal, int streams)
{
    wait_prior_grid();
    extern __shared__ uint4 ring_smem[];
    __shared__ float red[2][kMaxWarps][8];
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int NV = kElems / kN;
    const Member<DT, W, kElems, kMode, false> me(deal, a, streams, reinterpret_cast<char *>(ring_smem));
    const bool post = kMode == kPlain || a.w_post != nullptr;
    const bool pre = kMode == kPlain || a.w_pre != nullptr;
    const bool full = kMode != kPlain && a.gate_kind == LPCOLL_GATE_FULL;
    const int h0 = full ? 2 : 1, nranks = kMode == kPlain ? 1 : a.nranks;
    void *const h_sum = kMode == kPlain ? nullptr : a.h_sum;
    const float per_hidden = __fdiv_rn(1.0f, static_cast<float>(a.hidden));
    const auto fetch = [&](size_t t, int stage) {
        if (t < a.tokens) {
            for (int r = 0; r < nranks; ++r)
                me.copy(stage, h0 + r, a.h[r], t);
            me.copy(stage, 0, a.x, t);
            if (full)
                me.copy(stage, 1, a.gate, t);
        }
        copy_commit();
    };
    for (int s = 0; s < deal.stages; ++s)
        fetch(me.t0 + s * me.step, s);

    Vec<kN> wq[NV];  // beta w_post, times a channel's gate
    typename Pack<DT, W>::Raw wp[NV];
    const bool channel = a.gate_kind == LPCOLL_GATE_CHANNEL;
    if constexpr (kMode != kWide)
        me.weights(a, post, channel, pre, a.branch_scale, wq, wp);
    const auto scale = [&](int c) {
        if constexpr (kMode == kWide)
            return me.scale(a, post, channel, a.branch_scale, c);
        else
            return wq[c];
    };
    const auto w_pre = [&](int c) {
        if constexpr (kMode == kWide)
            return load_vec_of<DT, W>(a.w_pre, me.col(c));
        else
            return unpack<DT, W>(wp[c]);
    };

    // The ranks' sum for the row in `stage`, left in FP32 in the place of the
    // first ranks' values, and this thread's part of the sum of its squares.
    const auto sum_ranks = [&](size_t t, int stage) {
        Acc<kN> sq = {};
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            Vec<kN> h = me.read(t, stage, h0, c);
            if (nranks > 1) {
#pragma unroll 4
                for (int r = 1; r < nranks; ++r)
                    h = add(h, me.read(t, stage, h0 + r, c));
                me.keep(t, stage, h0, c, h);
            }
            add_products(sq, h, h);
        }
        return fold(sq);
    };

    // Each turn ends row t and takes the next row's sum of squares of h with
    // its own of x', so that there is one barrier per row.
    int stage = 0, turn = 0;
    float r1 = 1.0f;
    me.ready(deal.stages - 1);
    const bool summed = post || nranks > 1;
    if (summed) {
        float s[1] = {me.t0 < a.tokens ? sum_ranks(me.t0, 0) : 0.0f};
        if (post) {
            team_sums(s, red[1], deal, me.first_warp);
            r1 = inv_rms(s[0], per_hidden, a.eps);
        }
    }
    for (size_t t = me.t0; t < a.tokens; t += me.step, turn ^= 1) {
        const float gate_t = a.gate_kind == LPCOLL_GATE_TOKEN ? load_one<DT>(a.gate, t) : 1.0f;
        const float f = r1 * gate_t;
        Vec<kN> v[NV];
        Acc<kN> sq = {};
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            v[c] = nranks > 1 ? me.kept(t, stage, h0, c) : me.read(t, stage, h0, c);
            if (h_sum != nullptr)
                store_vec_of<DT, W>(h_sum, me.elem(t, c), v[c]);
            Vec<kN> u = mul(mul(f, scale(c)), v[c]);
            if (full)
                u = mul(u, me.read(t, stage, 1, c));
            v[c] = fma(a.res_scale, me.read(t, stage, 0, c), u);
            add_products(sq, v[c], v[c]);
            store_vec_of<DT, W>(a.x_out, me.elem(t, c), v[c]);
        }
        fetch(t + deal.stages * me.step, stage);
        stage = stage + 1 == deal.stages ? 0 : stage + 1;
        me.ready(deal.stages - 1);
        float s[2] = {fold(sq), summed && t + me.step < a.tokens ? sum_ranks(t + me.step, stage) : 0.0f};
        if (post || pre)
            team_sums(s, red[turn], deal, me.first_warp);
        r1 = post ? inv_rms(s[1], per_hidden, a.eps) : 1.0f;
        if (pre) {
            const float r2 = inv_rms(s[0], per_hidden, a.eps);
#pragma unroll
            for (int c = 0; c < NV; ++c)
                if (me.has(c))
                    store_vec_of<DT, W>(a.n_out, me.elem(t, c),
                                        mul(mul(r2, w_pre(c)), v[c]));
        }
    }
    if (kMode != kPlain && deal.cluster > 1)
        cluster_barrier();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------------------
// Gradients. With q = dn w_pre and c2 = r2^2 mean(q x'), the gradient of x' is
// D = dx' + r2 (q - x' c2). The gradient through the first norm needs the sum
// of beta g w_post D h, which is linear in D; so with P = g w_post h (g without
// a token's own gate) the six sums h^2, x'^2, q x', P dx', P q, P x' of one
// pass over the row give every factor of the second:
//   sum(P D) = sum(P dx') + r2 (sum(P q) - c2 sum(P x')).
// A thread keeps the sums over tokens of its columns in registers, S = sum
// beta r1 h D (times a gate that differs by token) and dw_pre = sum dn x' r2,
// and the CTA leaves them in the workspace, [2][CTAs][hidden]; a second launch
// adds those up in order: dw_post = g S, and dgate = w_post S for a gate per
// channel.
// ---------------------------------------------------------------------------

// Row streams of a stage.
enum Stream { kH = 0, kDx = 1, kX = 2, kDn = 3, kGate = 4 };

template <int DT, int W, int kElems, int kMode>
__global__ void __launch_bounds__(kThreadsOne<kElems>, 1)
residual_norm_backward_kernel(const __grid_constant__ NormArgs a, const Deal deal, int streams)
{
    wait_prior_grid();
    extern __shared__ uint4 ring_smem[];
    __shared__ float red[2][kMaxWarps][8];
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int NV = kElems / kN;
    const Member<DT, W, kElems, kMode, kMode == kPlain> me(deal, a, streams, reinterpret_cast<char *>(ring_smem));
    const bool post = kMode == kPlain || a.w_post != nullptr;
    const bool pre = kMode == kPlain || a.w_pre != nullptr;
    const bool given = kMode == kPlain || a.dx_out != nullptr;
    const bool full = kMode != kPlain && a.gate_kind == LPCOLL_GATE_FULL;
    const int H = a.hidden;
    const float per_hidden = __fdiv_rn(1.0f, static_cast<float>(H));
    const auto fetch = [&](size_t t, int stage) {
        if (t < a.tokens) {
            me.copy(stage, kH, a.h[0], t);
            if (given)
                me.copy(stage, kDx, a.dx_out, t);
            if (pre) {
                me.copy(stage, kX, a.x, t);
                me.copy(stage, kDn, a.dn_out, t);
            }
            if (full)
                me.copy(stage, kGate, a.gate, t);
        }
        copy_commit();
    };
    for (int s = 0; s < deal.stages; ++s)
        fetch(me.t0 + s * me.step, s);

    Vec<kN> wq[NV];                    // w_post times a channel's gate
    typename Pack<DT, W>::Raw wp[NV];  // w_pre
    Vec<kN> S[NV], s_pre[NV];
    me.weights(a, post, a.gate_kind == LPCOLL_GATE_CHANNEL, pre, 1.0f, wq, wp);
#pragma unroll
    for (int c = 0; c < NV; ++c)
        S[c] = s_pre[c] = splat<kN>(0.0f);

    // a token's gate, read a row ahead
    const auto gate_of = [&](size_t t) {
        return a.gate_kind == LPCOLL_GATE_TOKEN && t < a.tokens ? load_one<DT>(a.gate, t) : 1.0f;
    };

    // a thread's part of the six sums of the row in `stage`
    const auto row_sums = [&](size_t t, int stage, float (&s)[6]) {
        Acc<kN> v[6] = {};
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            const Vec<kN> h = me.read(t, stage, kH, c);
            Vec<kN> p = mul(wq[c], h);
            add_products(v[0], h, h);
            if (full)
                p = mul(p, me.read(t, stage, kGate, c));
            if (given)
                add_products(v[3], p, me.read(t, stage, kDx, c));
            if (pre) {
                const Vec<kN> x = me.read(t, stage, kX, c);
                const Vec<kN> q = mul(me.read(t, stage, kDn, c), unpack<DT, W>(wp[c]));
                add_products(v[1], x, x);
                add_products(v[2], q, x);
                add_products(v[4], p, q);
                add_products(v[5], p, x);
            }
        }
#pragma unroll
        for (int i = 0; i < 6; ++i)
            s[i] = fold(v[i]);
    };

    int stage = 0, turn = 0;
    float gate_next = gate_of(me.t0);
    for (size_t t = me.t0; t < a.tokens; t += me.step, turn ^= 1) {
        const float gate_t = gate_next;
        gate_next = gate_of(t + me.step);
        me.ready(deal.stages - 1);
        float s[6];
        row_sums(t, stage, s);
        team_sums(s, red[turn], deal, me.first_warp);
        const float r1 = post ? inv_rms(s[0], per_hidden, a.eps) : 1.0f;
        const float r2 = pre ? inv_rms(s[1], per_hidden, a.eps) : 0.0f;
        const float c2 = pre ? r2 * r2 * s[2] * per_hidden : 0.0f;
        const float pd = fmaf(r2, fmaf(-c2, s[5], s[4]), s[3]);
        const float bt = a.branch_scale * gate_t;
        // dh = f1 wq g D - f2 h;  S += f1 g h D
        const float f1 = r1 * bt;
        const float f2 = post ? r1 * (r1 * r1 * bt * pd * per_hidden) : 0.0f;
        if (a.gate_kind == LPCOLL_GATE_TOKEN && a.dgate != nullptr && me.col0 == 0)
            store_f32(static_cast<float *>(a.dgate) + t, a.branch_scale * r1 * pd);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (!me.has(c))
                continue;
            Vec<kN> d = splat<kN>(0.0f);
            if (given)
                d = me.read(t, stage, kDx, c);
            if (pre) {
                const Vec<kN> x = me.read(t, stage, kX, c), dn = me.read(t, stage, kDn, c);
                const Vec<kN> q = mul(dn, unpack<DT, W>(wp[c]));
                s_pre[c] = fma(mul(r2, dn), x, s_pre[c]);
                d = fma(r2, fma(-c2, x, q), d);
            }
            const Vec<kN> dx = mul(a.res_scale, d);
            const Vec<kN> h = me.read(t, stage, kH, c);
            if (full) {
                if (a.dgate != nullptr)
                    store_vec_of<DT, W>(a.dgate, me.elem(t, c),
                                        mul(mul(mul(f1, wq[c]), h), d));
                d = mul(d, me.read(t, stage, kGate, c));
            }
            const Vec<kN> e = mul(f1, d);
            S[c] = fma(h, e, S[c]);
            store_vec_of<DT, W>(a.dx, me.elem(t, c), dx);
            store_vec_of<DT, W>(a.dh, me.elem(t, c), fma(wq[c], e, mul(-f2, h)));
        }
        fetch(t + deal.stages * me.step, stage);
        stage = stage + 1 == deal.stages ? 0 : stage + 1;
    }
    copy_wait(0);
    if (kMode != kPlain && deal.cluster > 1)
        cluster_barrier();  // no CTA leaves while another reads its sums

    if (a.partial != nullptr)
        leave_sums<DT, W>(me, deal, s_pre, S, a.partial, reinterpret_cast<float *>(ring_smem));
}

// Column sums of the workspace: a CTA adds 32 columns of one of the two sums.
// 32 threads per column take every 32nd CTA's part, all in flight at once (kPer
// of them, for as many CTAs per SM), and a warp adds up a column's 32.
constexpr int kPer = (kSms + 31) / 32;

template <int DT, int kPerSm>
__global__ void __launch_bounds__(1024)
norm_column_sums_kernel(const __grid_constant__ NormArgs a, int parts, int column_ctas)
{
    wait_prior_grid();
    __shared__ float red[32][33];
    const int which = blockIdx.x / column_ctas;
    const bool channel = a.gate_kind == LPCOLL_GATE_CHANNEL;
    float *const dgate = channel ? static_cast<float *>(a.dgate) : nullptr;
    if (which == 0 ? a.dw_pre == nullptr : a.dw_post == nullptr && dgate == nullptr)
        return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = (blockIdx.x % column_ctas) * 32;
    const float *p = a.partial + static_cast<size_t>(which) * parts * a.hidden + first + lane;
    constexpr int kParts = kPer * kPerSm;
    float v[kParts];
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const int q = i * 32 + warp;
        v[i] = q < parts && first + lane < a.hidden
                   ? load_f32(p + static_cast<size_t>(q) * a.hidden)
                   : 0.0f;
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kParts; ++i)
        sum += v[i];
    red[warp][lane] = sum;
    __syncthreads();
    sum = warp_sum(red[lane][warp]);
    const int col = first + warp;
    if (lane != 0 || col >= a.hidden)
        return;
    if (which == 0 || parts == 0) {  // no tokens: zeros, whatever the weights hold
        if (which == 0)
            store_f32(a.dw_pre + col, sum);
        else if (a.dw_post != nullptr)
            store_f32(a.dw_post + col, 0.0f);
        if (which == 1 && dgate != nullptr)
            store_f32(dgate + col, 0.0f);
        return;
    }
    if (a.dw_post != nullptr)
        store_f32(a.dw_post + col, channel ? sum * load_one<DT>(a.gate, col) : sum);
    if (dgate != nullptr)
        store_f32(dgate + col, a.w_post != nullptr ? sum * load_one<DT>(a.w_post, col) : sum);
}

// A row is one CTA's, or, where there are few tokens or the row does not fit
// one, a cluster's. 16 columns a thread halve what a row costs besides its
// columns (sums, addresses), 8 columns give twice the warps. 8192 columns in
// BF16: the gradients of 8192 tokens take 134 us with 16 and 177 with 8, the
// forward pass of 16384 tokens 183 and 160 (8192 tokens of 8 ranks at 4096 columns
// 121 and 125). 8 are also faster where latency counts (32 tokens: 5.6 against 6.1 us)
// and for the shortest rows (128 columns: 7.2 against 9.0 us).
Plan make_plan(size_t tokens, int hidden, int dtype, int streams, bool gradient)
{
    const int width = row_width(hidden, dtype);
    const int kn = width / static_cast<int>(dtype_bytes(dtype));
    constexpr int kRow = 8192;  // columns of the largest CTA but kWide's
    Plan p;
    p.wide = !gradient && tokens > kSms && hidden > kRow && width == 16 &&
             static_cast<size_t>(hidden) * width / kn * streams <= kSmemOne;
    int cluster = hidden > kRow && !p.wide ? 2 : 1;
    // few tokens: a row over up to 8 CTAs, while there are SMs left and a CTA
    // keeps two warps
    while (cluster < kMaxCluster && tokens * cluster * 2 <= kSms && hidden >= 512 * cluster * 2)
        cluster *= 2;
    // many ranks: until a row of all streams fits the shared memory
    while (!p.wide && cluster < kMaxCluster &&
           (static_cast<size_t>(hidden) * width / kn / cluster + 2048) * streams > kSmemOne)
        cluster *= 2;
    const bool light =
        !gradient && streams <= 2 && hidden <= kRow && dtype == LPCOLL_BF16;
    p.elems = !p.wide && (hidden <= 256 || tokens <= kSms || light) ? 8 : 16;
    const int room = p.wide ? kWideThreads : (p.elems == 8 ? kThreadsOne<8> : kThreadsOne<16>);
    return deal_rows(p, cluster, tokens, hidden, dtype, streams, gradient, Room{room});
}

Plan backward_plan(size_t tokens, int hidden, int dtype, int gate_kind)
{
    const int streams = gate_kind == LPCOLL_GATE_FULL ? 5 : 4;
    return make_plan(tokens, hidden, dtype, streams, true);
}

template <int DT, int W>
cudaError_t backward_dt(const NormArgs &a, const Plan &p, cudaStream_t st)
{
    const bool full = a.gate_kind == LPCOLL_GATE_FULL;
    const int streams = full ? 5 : 4;
    if constexpr (W == 16) {
        if (p.even && p.deal.cluster == 1 && !full && a.w_post != nullptr && a.w_pre != nullptr &&
            a.dx_out != nullptr)
            return launch_plan(p.elems == 8 ? residual_norm_backward_kernel<DT, W, 8, kPlain>
                                            : residual_norm_backward_kernel<DT, W, 16, kPlain>,
                               a, p, streams, st);
    }
    return launch_plan(p.elems == 8 ? residual_norm_backward_kernel<DT, W, 8, kGeneral>
                                    : residual_norm_backward_kernel<DT, W, 16, kGeneral>,
                       a, p, streams, st);
}

template <int DT, int W>
cudaError_t forward_dt(const NormArgs &a, cudaStream_t st)
{
    const bool full = a.gate_kind == LPCOLL_GATE_FULL;
    const int streams = a.nranks + 1 + (full ? 1 : 0);
    const Plan p = make_plan(a.tokens, a.hidden, a.dtype, streams, false);
    if constexpr (W == 16) {
        if (p.wide)
            return launch_plan(residual_norm_kernel<DT, W, 16, kWide>, a, p, streams, st);
        if (p.even && p.deal.cluster == 1 && !full && a.w_post != nullptr && a.w_pre != nullptr &&
            a.nranks == 1 && a.h_sum == nullptr)
            return launch_plan(p.elems == 8 ? residual_norm_kernel<DT, W, 8, kPlain>
                                            : residual_norm_kernel<DT, W, 16, kPlain>,
                               a, p, streams, st);
    }
    return launch_plan(p.elems == 8 ? residual_norm_kernel<DT, W, 8, kGeneral>
                                    : residual_norm_kernel<DT, W, 16, kGeneral>,
                       a, p, streams, st);
}

template <int DT> cudaError_t column_sums(const NormArgs &a, int parts, cudaStream_t st)
{
    static_assert(kMaxCtas == 3, "one kernel per number of CTAs per SM");
    const int ctas = (a.hidden + 31) / 32;
    const auto kernel = parts <= kSms ? norm_column_sums_kernel<DT, 1>
                                      : (parts <= 2 * kSms ? norm_column_sums_kernel<DT, 2>
                                                           : norm_column_sums_kernel<DT, 3>);
    return launch_kernel_block(kernel, static_cast<size_t>(2) * ctas, 1024, 0, st, a, parts, ctas);
}

}  // namespace

int norm_backward_parts(size_t tokens, size_t hidden, int dtype)
{
    if (hidden == 0 || tokens == 0)
        return 0;
    // the same workspace for every kind of gate
    const int h = static_cast<int>(hidden);
    const int some = backward_plan(tokens, h, dtype, LPCOLL_GATE_NONE).ctas;
    const int full = backward_plan(tokens, h, dtype, LPCOLL_GATE_FULL).ctas;
    return some > full ? some : full;
}

cudaError_t launch_residual_norm(const NormArgs &a, cudaStream_t st)
{
    return LPC_BY_ROW(forward_dt, a.dtype, static_cast<size_t>(a.hidden), a, st);
}

cudaError_t launch_residual_norm_backward(const NormArgs &args, cudaStream_t st)
{
    NormArgs a = args;
    const bool sums = a.dw_pre != nullptr || a.dw_post != nullptr ||
                      (a.gate_kind == LPCOLL_GATE_CHANNEL && a.dgate != nullptr);
    if (!sums)
        a.partial = nullptr;
    int parts = 0;
    if (a.tokens > 0) {
        const Plan p = backward_plan(a.tokens, a.hidden, a.dtype, a.gate_kind);
        parts = p.ctas;
        const cudaError_t e =
            LPC_BY_ROW(backward_dt, a.dtype, static_cast<size_t>(a.hidden), a, p, st);
        if (e != cudaSuccess)
            return e;
    }
    if (!sums)
        return cudaSuccess;
    return a.dtype == LPCOLL_F32 ? column_sums<LPCOLL_F32>(a, parts, st)
                                 : column_sums<LPCOLL_BF16>(a, parts, st);
}

}  // namespace lpc
