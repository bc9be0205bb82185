// lpcoll_layers.cuh -- what the kernels around the collectives share (router,
// sort by expert, dispatch, combine, residual norm): element access at a
// row's own alignment, sums over a warp and a CTA, and the launchers.
//
// Rows of these operators are `hidden` elements long and follow one another
// without padding, so a row starts on a 16-byte boundary only if its length
// in bytes is a multiple of 16. Each kernel exists for accesses of W = 16, 8
// and 4 bytes, and of 2 bytes (BF16 rows of odd length).
#pragma once

#include "lpcoll_device.cuh"

namespace lpc {

// One access of a lane: W bytes.
template <int DT, int W> struct Pack;
template <int DT> struct Pack<DT, 16> {
    using Raw = uint4;
    static constexpr int kN = Fmt<DT>::kVec;
};
template <int DT> struct Pack<DT, 8> {
    using Raw = uint2;
    static constexpr int kN = Fmt<DT>::kVec / 2;
};
template <int DT> struct Pack<DT, 4> {
    using Raw = uint32_t;
    static constexpr int kN = Fmt<DT>::kVec / 4;
};
template <> struct Pack<LPCOLL_BF16, 2> {
    using Raw = uint16_t;
    static constexpr int kN = 1;
};
// The narrowest access: one element.
template <int DT> constexpr int kOne = 16 / Fmt<DT>::kVec;

inline size_t dtype_bytes(int dtype) { return dtype == LPCOLL_F32 ? 4 : 2; }

// Access width that every row of `hidden` elements allows.
inline int row_width(size_t hidden, int dtype)
{
    const size_t bytes = hidden * dtype_bytes(dtype);
    return bytes % 16 == 0 ? 16 : (bytes % 8 == 0 ? 8 : (bytes % 4 == 0 ? 4 : 2));
}

// fn<dtype, width>(...) for a call's dtype and row length.
#define LPC_BY_WIDTH(fn, DT, width, ...)                                                     \
    ((width) == 16 ? fn<DT, 16>(__VA_ARGS__)                                                 \
                   : ((width) == 8 ? fn<DT, 8>(__VA_ARGS__) : fn<DT, 4>(__VA_ARGS__)))
#define LPC_BY_ROW(fn, dtype, hidden, ...)                                                   \
    ((dtype) == LPCOLL_F32                                                                   \
         ? LPC_BY_WIDTH(fn, LPCOLL_F32, row_width(hidden, dtype), __VA_ARGS__)               \
         : (row_width(hidden, dtype) == 2                                                    \
                ? fn<LPCOLL_BF16, 2>(__VA_ARGS__)                                            \
                : LPC_BY_WIDTH(fn, LPCOLL_BF16, row_width(hidden, dtype), __VA_ARGS__)))

template <int DT, int W>
__device__ __forceinline__ typename Pack<DT, W>::Raw load_pack(const void *base, size_t e0)
{
    using Raw = typename Pack<DT, W>::Raw;
    constexpr int kEs = sizeof(Raw) / Pack<DT, W>::kN;
    const Raw *p = reinterpret_cast<const Raw *>(static_cast<const char *>(base) + e0 * kEs);
    return LPC_READ_OK(p, sizeof(Raw)) ? *p : Raw{};
}

template <int DT, int W>
__device__ __forceinline__ void store_pack(void *base, size_t e0, typename Pack<DT, W>::Raw v)
{
    using Raw = typename Pack<DT, W>::Raw;
    constexpr int kEs = sizeof(Raw) / Pack<DT, W>::kN;
    Raw *p = reinterpret_cast<Raw *>(static_cast<char *>(base) + e0 * kEs);
    if (LPC_WRITE_OK(p, sizeof(Raw)))
        *p = v;
}

template <int DT, int W>
__device__ __forceinline__ void widen_pack(typename Pack<DT, W>::Raw v,
                                           float (&x)[Pack<DT, W>::kN])
{
    if constexpr (W == 16) {
        widen<DT>(v, x);
    } else if constexpr (W == 8) {
        const uint32_t w[2] = {v.x, v.y};
        if constexpr (DT == LPCOLL_F32) {
            x[0] = __uint_as_float(w[0]);
            x[1] = __uint_as_float(w[1]);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                x[2 * j] = __uint_as_float(w[j] << 16);
                x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        }
    } else if constexpr (DT == LPCOLL_F32) {
        x[0] = __uint_as_float(v);
    } else {
        x[0] = __uint_as_float(static_cast<uint32_t>(v) << 16);
        if constexpr (W == 4)
            x[1] = __uint_as_float(v & 0xFFFF0000u);
    }
}

template <int DT, int W>
__device__ __forceinline__ typename Pack<DT, W>::Raw
narrow_pack(const float (&x)[Pack<DT, W>::kN])
{
    if constexpr (W == 16) {
        return narrow<DT>(x);
    } else if constexpr (W == 8) {
        if constexpr (DT == LPCOLL_F32) {
            return make_uint2(__float_as_uint(x[0]), __float_as_uint(x[1]));
        } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(x[2], x[3]);
            return make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                              *reinterpret_cast<const uint32_t *>(&hi));
        }
    } else if constexpr (DT == LPCOLL_F32) {
        return __float_as_uint(x[0]);
    } else if constexpr (W == 4) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[0], x[1]);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        return __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
    }
}

__device__ __forceinline__ int32_t load_i32(const int32_t *p)
{
    return LPC_READ_OK(p, sizeof(int32_t)) ? *p : 0;
}

__device__ __forceinline__ void store_i32(int32_t *p, int32_t v)
{
    if (LPC_WRITE_OK(p, sizeof(int32_t)))
        *p = v;
}

__device__ __forceinline__ float load_f32(const float *p)
{
    return LPC_READ_OK(p, sizeof(float)) ? *p : 0.0f;
}

__device__ __forceinline__ void store_f32(float *p, float v)
{
    if (LPC_WRITE_OK(p, sizeof(float)))
        *p = v;
}

// Two FP32 products, sums, or products and sums, in one instruction; each half rounds
// as the scalar operation does.
__device__ __forceinline__ float2 mul_pair(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

__device__ __forceinline__ float2 add_pair(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

__device__ __forceinline__ float2 fma_pair(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// Sum over the lanes of a warp, the same bits in every lane and run.
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
    return v;
}

// Launches as launch_kernel does, with CTAs of any size; `cluster` CTAs form a
// thread-block cluster (1: none). Internal linkage for the same reason.
template <typename... Params, typename... Args>
static cudaError_t launch_kernel_cluster(void (*kernel)(Params...), size_t grid, int threads,
                                         int cluster, size_t smem, cudaStream_t stream,
                                         Args... args)
{
#ifdef LPCOLL_DEBUG_BOUNDS
    const cudaError_t de = cudaMemcpyToSymbolAsync(g_debug_ranges, &debug_pending(),
                                                   sizeof(DebugRanges), 0,
                                                   cudaMemcpyHostToDevice, stream);
    if (de != cudaSuccess)
        return de;
#endif
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename... Params, typename... Args>
static cudaError_t launch_kernel_block(void (*kernel)(Params...), size_t grid, int threads,
                                       size_t smem, cudaStream_t stream, Args... args)
{
    return launch_kernel_cluster(kernel, grid, threads, 1, smem, stream, args...);
}

// -- launchers (one translation unit each; called by lpcoll_layers_api.cu) --

struct RouteArgs {
    const void *logits;
    int32_t *ids;
    float *weights;
    const float *dweights;  // backward
    void *dlogits;          // backward
    size_t tokens;
    int experts, topk, renormalize, dtype;
};
cudaError_t launch_route(const RouteArgs &a, cudaStream_t st);
cudaError_t launch_route_backward(const RouteArgs &a, cudaStream_t st);

struct SortArgs {
    const int32_t *ids;
    int32_t *slot_row, *row_slot, *offsets, *counts;
    int32_t *chunk_counts;  // workspace: [experts][chunks]
    int slots, experts, capacity, rows;
    int chunks, chunk_len;
};
// Chunks (CTAs) that a sort of `slots` slots runs in; 1 needs no workspace.
int sort_chunks(size_t slots);
cudaError_t launch_sort(SortArgs a, cudaStream_t st);

struct RowsArgs {
    const void *x;       // tokens' side: [tokens, hidden] (dispatch: read, backward: dout)
    void *out;           // the other side, written
    const void *rows;    // experts' side, read (combine and its backward)
    uint8_t *codes;      // experts' side as FP8 payloads
    float *scales;
    const float *weights;
    float *dweights;
    const int32_t *slot_row, *row_slot;
    size_t tokens, nrows, hidden;
    int topk, dtype;
};
cudaError_t launch_dispatch(const RowsArgs &a, bool lp, cudaStream_t st);
cudaError_t launch_combine(const RowsArgs &a, bool lp, cudaStream_t st);
cudaError_t launch_combine_backward(const RowsArgs &a, cudaStream_t st);

struct NormArgs {
    const void *h[LPCOLL_MAX_RANKS];
    int nranks;
    const void *x, *gate, *w_post, *w_pre;
    void *x_out, *n_out, *h_sum;
    // backward: x holds x_out, h[0] the block's output
    const void *dx_out, *dn_out;
    void *dx, *dh, *dgate;
    float *dw_post, *dw_pre;
    float *partial;  // workspace of the sums over tokens
    int gate_kind;
    float res_scale, branch_scale, eps;
    size_t tokens;
    int hidden, dtype;
};
// Partial sums over tokens that a backward call keeps (CTAs of its row kernel).
int norm_backward_parts(size_t tokens, size_t hidden, int dtype);
cudaError_t launch_residual_norm(const NormArgs &a, cudaStream_t st);
cudaError_t launch_residual_norm_backward(const NormArgs &a, cudaStream_t st);

// Dropout's random numbers (lpcoll_philox.cuh).
struct DropArgs {
    const unsigned long long *rng;  // seed, offset (device memory)
    unsigned long long first_row;
    uint32_t least;  // smallest word that is kept; 0: all are, and rng is not read
    float scale;     // 1 / (1 - p)
};

struct LayerNormArgs {
    const void *h[LPCOLL_MAX_RANKS];  // partial products; none for layer_norm
    int nranks;
    const void *x;  // layer_norm: its input; else the residual or NULL; gradients: x'
    const void *w, *b;
    void *x_out, *n_out;
    const void *dx_out, *dn_out;  // gradients
    void *dx, *dh;
    float *dw, *db;
    float *partial;  // workspace of the sums over tokens
    DropArgs drop;
    float eps;
    size_t tokens;
    int hidden, dtype;
};

// Rows of sums that a gradient leaves in its workspace, and their sums.
int layer_norm_parts(size_t tokens, size_t hidden, int dtype, bool dropout);
cudaError_t launch_layer_norm_sums(const LayerNormArgs &a, int parts, cudaStream_t st);
cudaError_t launch_layer_norm(const LayerNormArgs &a, cudaStream_t st);
cudaError_t launch_layer_norm_backward(const LayerNormArgs &a, cudaStream_t st);
// residual_dropout with its norm, and without.
cudaError_t launch_dropout_norm(const LayerNormArgs &a, cudaStream_t st);
cudaError_t launch_dropout_norm_backward(const LayerNormArgs &a, cudaStream_t st);
cudaError_t launch_dropout(const LayerNormArgs &a, cudaStream_t st);

struct BalanceArgs {
    const void *logits;
    const int32_t *ids;
    const uint8_t *valid;  // NULL: every token is
    float *loss, *prob_sums;
    int32_t *counts;
    float *rows;           // workspace: sums and counts of each CTA
    const float *dloss;    // backward
    void *dlogits;         // backward
    float coef;
    size_t tokens;
    int experts, topk, dtype, accumulate;
};
// Rows that a call's launch of CTAs leaves (1: all in one cluster), and their bytes.
int balance_rows(size_t tokens);
size_t balance_workspace(size_t tokens, int experts);
cudaError_t launch_balance(const BalanceArgs &a, cudaStream_t st);
cudaError_t launch_balance_backward(const BalanceArgs &a, cudaStream_t st);

struct EmbedArgs {
    const void *table;     // forward
    void *out;             // forward
    const void *dout;      // backward
    float *dtable;         // backward
    const void *ids;
    int ids64;             // ids are int64_t, not int32_t
    long long first_id;
    float scale;
    size_t tokens, vocab, hidden;
    int dtype, accumulate;
    void *workspace;       // backward
};
size_t embed_workspace(size_t tokens, size_t vocab, size_t hidden);
cudaError_t launch_embed(const EmbedArgs &a, cudaStream_t st);
cudaError_t launch_embed_backward(const EmbedArgs &a, cudaStream_t st);

}  // namespace lpc
