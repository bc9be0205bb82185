// lpcoll_embed.cu -- the rows of a vocabulary shard (token_embed) and their
// gradient (token_embed_backward):
//
//   out_t = scale table[id_t - first_id], zeros for ids of other shards
//   dtable_v = scale sum over t with id_t = first_id + v of dout_t   (FP32)
//
// Both move rows, and HBM traffic bounds them. The gradient sorts the tokens by
// row of the table (stable, so that a row's terms come in the order of their
// tokens), then goes through the sorted tokens in tiles: a run of equal rows that
// lies in one tile is added up in registers and written once; runs over several
// tiles leave one partial row per tile in the workspace, which a last launch adds
// in order. So frequent tokens are shared out over many CTAs without atomics on
// floating-point values, and the same call gives the same bits. Rows of the table
// without a token are cleared by other CTAs of the sort's and the sums' launches, which
// keep DRAM busy while those wait for memory.
//
// Measured on one GB300 (bytes at the copy rate in brackets): the rows of 16384 tokens of
// 8192 BF16 from one of four shards 49 us (46), from a whole table 70 (63: 201 MB are read
// for 157 MB of distinct rows, which do not all stay in L2 beside the outputs); in one
// piece of 16 bytes a lane and CTAs of 4 KB 76. The gradient of 16384 tokens into 32000 x 8192: 226 us
// (194), of them the sort 14-20, which clears 144 MB meanwhile, the sums 195, the last launch
// 6; with a sort of four launches, the clearing behind the sums and 4 rows in flight a lane
// 295. 777 tokens into 4001 x 1025 FP32: 13 us (2.5), the latencies of three launches.
#include "lpcoll_layers.cuh"

namespace lpc {

namespace {

constexpr int kSms = 152;
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kLanes = 256;

// How a row is cut: `lanes` lanes of each of `segs` CTAs go through it in pieces of 16
// bytes (of the table or of dout), `pieces` of them, `ahead` at a time; short rows
// share a CTA, `rows` of them.
struct RowCut {
    unsigned segs, pieces;
    int lanes, rows;
};

RowCut cut(size_t hidden, int dtype, int ahead, int most)
{
    const size_t per_piece = 16 / dtype_bytes(dtype);
    const size_t pieces = (hidden + per_piece - 1) / per_piece;
    const size_t lanes = (pieces + ahead - 1) / ahead;
    RowCut r;
    r.pieces = static_cast<unsigned>(pieces);
    r.segs = static_cast<unsigned>((lanes + most - 1) / most);
    r.lanes = static_cast<int>((lanes + r.segs - 1) / r.segs);
    r.rows = r.segs > 1 ? 1 : most / r.lanes;
    return r;
}

// The row and the first piece of a thread.
struct Place {
    size_t row;
    unsigned piece;
    bool idle;  // a lane behind the CTA's rows
};
__device__ __forceinline__ Place place_of(const RowCut &c, size_t cta)
{
    Place p = {cta, threadIdx.x, threadIdx.x >= static_cast<unsigned>(c.lanes * c.rows)};
    if (c.segs > 1) {
        p.row = cta / c.segs;
        p.piece += static_cast<unsigned>(cta % c.segs) * c.lanes;
    } else if (c.rows > 1) {
        const unsigned which = threadIdx.x / c.lanes;
        p.row = cta * c.rows + which;
        p.piece -= which * c.lanes;
    }
    return p;
}

// Row of the shard of token t, or -1.
__device__ __forceinline__ long long row_of(const EmbedArgs &a, size_t t)
{
    long long id;
    if (a.ids64) {
        const long long *p = static_cast<const long long *>(a.ids) + t;
        id = LPC_READ_OK(p, 8) ? *p : -1;
    } else {
        id = load_i32(static_cast<const int32_t *>(a.ids) + t);
    }
    // in unsigned numbers, so that no id overflows
    const unsigned long long row =
        static_cast<unsigned long long>(id) - static_cast<unsigned long long>(a.first_id);
    return id >= a.first_id && row < a.vocab ? static_cast<long long>(row) : -1;
}

constexpr int kPieces = 4;  // that a lane of the forward pass has in flight

template <int DT, int W>
__global__ void __launch_bounds__(kLanes)
embed_kernel(const __grid_constant__ EmbedArgs a, const RowCut c)
{
    wait_prior_grid();
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int kCols = Fmt<DT>::kVec;
    constexpr int kPacks = kCols / kN;
    const Place p = place_of(c, blockIdx.x);
    if (p.idle || p.row >= a.tokens)
        return;
    const long long row = row_of(a, p.row);
    const unsigned step = c.segs * c.lanes;
    const size_t to = p.row * a.hidden, from = static_cast<size_t>(row >= 0 ? row : 0) * a.hidden;
    const bool plain = a.scale == 1.0f;
    typename Pack<DT, W>::Raw raw[kPieces][kPacks];
    const auto has = [&](int u, int i) {
        const unsigned piece = p.piece + u * step;
        return W == 16 ? piece < c.pieces : piece * kCols + i * kN < a.hidden;
    };
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
#pragma unroll
        for (int i = 0; i < kPacks; ++i) {
            raw[u][i] = {};
            if (row >= 0 && has(u, i))
                raw[u][i] = load_pack<DT, W>(a.table, from + (p.piece + u * step) * kCols + i * kN);
        }
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
#pragma unroll
        for (int i = 0; i < kPacks; ++i) {
            if (!has(u, i))
                continue;
            if (row >= 0 && !plain) {  // other rows are +0, whatever the scale
                float x[kN];
                widen_pack<DT, W>(raw[u][i], x);
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    x[j] = x[j] * a.scale;
                raw[u][i] = narrow_pack<DT, W>(x);
            }
            store_pack<DT, W>(a.out, to + (p.piece + u * step) * kCols + i * kN, raw[u][i]);
        }
}

// ---------------------------------------------------------------------------
// Tokens sorted by row: a radix sort of (row, token), digits of up to kDigitBits
// bits, each pass a stable counting sort. Here, for more than kClusterTokens, the
// tokens are cut into chunks, one CTA each: a first launch counts the digits of every
// chunk, and a CTA of the second adds up the counts of the chunks before its own.
// Tokens without a row have the key `vocab` and come last.
// ---------------------------------------------------------------------------

constexpr int kDigitBits = 9;  // 10^6 tokens into 128000 rows: 262 us, with 8 (a pass more) 287
constexpr int kDigits = 1 << kDigitBits;
constexpr int kMaxChunks = 128;  // 300000 tokens of 512 BF16: 166 us, with 64 176, with 256 185

struct SortPlan {
    int passes, bits;  // bits of a digit
};

SortPlan sort_plan(size_t vocab)
{
    int key_bits = 1;
    while (key_bits < 32 && (vocab >> key_bits) != 0)
        ++key_bits;
    SortPlan p;
    p.passes = (key_bits + kDigitBits - 1) / kDigitBits;
    p.bits = (key_bits + p.passes - 1) / p.passes;
    return p;
}

// Tokens of a chunk, and chunks.
size_t chunk_len(size_t tokens)
{
    const size_t even = (tokens + kMaxChunks - 1) / kMaxChunks;
    return (even + kThreads - 1) / kThreads * kThreads;
}
size_t chunks_of(size_t tokens) { return (tokens + chunk_len(tokens) - 1) / chunk_len(tokens); }

struct RadixArgs {
    const int32_t *keys, *order;  // of the pass before; NULL in the first
    int32_t *keys_out, *order_out;
    int32_t *counts;   // [chunks][digits]
    uint32_t *used;    // bit v: row v has a token
    int tokens, shift, bits, chunks, chunk_len, words;
};

__device__ __forceinline__ int key_of(const EmbedArgs &e, const RadixArgs &a, int i)
{
    if (a.keys != nullptr)
        return load_i32(a.keys + i);
    const long long row = row_of(e, static_cast<size_t>(i));
    return static_cast<int>(row >= 0 ? row : static_cast<long long>(e.vocab));
}

__global__ void __launch_bounds__(kThreads)
radix_count_kernel(const __grid_constant__ EmbedArgs e, const RadixArgs a)
{
    wait_prior_grid();
    __shared__ int hist[kDigits];
    const int digits = 1 << a.bits;
    for (int d = threadIdx.x; d < digits; d += kThreads)
        hist[d] = 0;
    __syncthreads();
    if (a.keys == nullptr) {  // the first pass's placing launch sets the bits
        const int stride = static_cast<int>(gridDim.x) * kThreads;
        for (int w = static_cast<int>(blockIdx.x) * kThreads + static_cast<int>(threadIdx.x);
             w < a.words; w += stride)
            store_i32(reinterpret_cast<int32_t *>(a.used) + w, 0);
    }
    const long long lo = static_cast<long long>(blockIdx.x) * a.chunk_len;
    const long long end = min(lo + a.chunk_len, static_cast<long long>(a.tokens));
    for (long long i = lo + threadIdx.x; i < end; i += kThreads)
        atomicAdd(&hist[key_of(e, a, static_cast<int>(i)) >> a.shift & (digits - 1)], 1);
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kThreads)
        store_i32(a.counts + static_cast<size_t>(blockIdx.x) * digits + d, hist[d]);
}

__global__ void __launch_bounds__(kThreads)
radix_place_kernel(const __grid_constant__ EmbedArgs e, const RadixArgs a)
{
    wait_prior_grid();
    // next[w][d]: place of warp w's next token of digit d
    __shared__ int next[kWarpsPerCta][kDigits];
    __shared__ int before[kDigits];  // tokens of a digit in the chunks before
    __shared__ int total[kDigits];
    __shared__ int warp_total[kWarpsPerCta];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int digits = 1 << a.bits;
    for (int d = tid; d < digits; d += kThreads)
#pragma unroll
        for (int w = 0; w < kWarpsPerCta; ++w)
            next[w][d] = 0;
    __syncthreads();

    const long long lo = static_cast<long long>(blockIdx.x) * a.chunk_len;
    const long long end = min(lo + a.chunk_len, static_cast<long long>(a.tokens));
    const int part = (a.chunk_len / kWarpsPerCta + 31) & ~31;
    const long long w_lo = lo + static_cast<long long>(warp) * part;
    const long long w_end = min(w_lo + part, end);
    for (long long i = w_lo + lane; i < w_end; i += 32)
        atomicAdd(&next[warp][key_of(e, a, static_cast<int>(i)) >> a.shift & (digits - 1)], 1);
    // a thread per digit, several chunks' counts in flight
    for (int d = tid; d < digits; d += kThreads) {
        int sum = 0, prior = 0;
#pragma unroll 16
        for (int c = 0; c < a.chunks; ++c) {
            const int v = load_i32(a.counts + static_cast<size_t>(c) * digits + d);
            sum += v;
            prior += c < static_cast<int>(blockIdx.x) ? v : 0;
        }
        total[d] = sum;
        before[d] = prior;
    }
    __syncthreads();
    // places of the warps' tokens, from the digit's first of this chunk on
    for (int d = tid; d < digits; d += kThreads) {
        int run = 0;
#pragma unroll
        for (int w = 0; w < kWarpsPerCta; ++w) {
            const int v = next[w][d];
            next[w][d] = run;
            run += v;
        }
    }
    __syncthreads();
    // exclusive sum over the digits, kPer consecutive ones per thread
    constexpr int kPer = kDigits / kThreads;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        sum += tid * kPer + i < digits ? total[tid * kPer + i] : 0;
    int scan = sum;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int v = __shfl_up_sync(kAll, scan, m);
        scan += lane >= m ? v : 0;
    }
    if (lane == 31)
        warp_total[warp] = scan;
    __syncthreads();
    int first = scan - sum;
#pragma unroll
    for (int w = 0; w < kWarpsPerCta; ++w)
        first += w < warp ? warp_total[w] : 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int d = tid * kPer + i;
        if (d < digits) {
            before[d] += first;
            first += total[d];
        }
    }
    __syncthreads();

    for (long long s0 = w_lo; s0 < w_end; s0 += 32) {
        const int i = static_cast<int>(s0) + lane;
        const bool there = s0 + lane < w_end;
        const int key = there ? key_of(e, a, i) : -1;
        const int d = there ? key >> a.shift & (digits - 1) : -1;
        const unsigned same = __match_any_sync(kAll, d);
        if (there) {
            const int at = before[d] + next[warp][d] + __popc(same & ((1u << lane) - 1u));
            store_i32(a.keys_out + at, key);
            store_i32(a.order_out + at, a.order != nullptr ? load_i32(a.order + i) : i);
            if (a.keys == nullptr && key < static_cast<int>(e.vocab) &&
                LPC_WRITE_OK(a.used + (key >> 5), 4))
                atomicOr(a.used + (key >> 5), 1u << (key & 31));
        }
        __syncwarp();
        if (there && lane == __ffs(same) - 1)
            next[warp][d] += __popc(same);
        __syncwarp();
    }
}

// Columns of a lane in FP32, kCols of them in the layout of dout's accesses.
template <int DT, int W> struct LaneCols {
    static constexpr int kN = Pack<DT, W>::kN;
    static constexpr int kCols = Fmt<DT>::kVec;
    static constexpr int kPacks = kCols / kN;
    static constexpr int WF = W * 4 / (16 / kCols) > 16 ? 16 : W * 4 / (16 / kCols);  // bytes of an FP32 access
    size_t col, hidden;
    __device__ __forceinline__ bool has(int i) const { return W == 16 || col + i * kN < hidden; }
    __device__ __forceinline__ void load(const void *base, size_t row,
                                         typename Pack<DT, W>::Raw (&raw)[kPacks]) const
    {
#pragma unroll
        for (int i = 0; i < kPacks; ++i) {
            raw[i] = {};
            if (has(i))
                raw[i] = load_pack<DT, W>(base, row * hidden + col + i * kN);
        }
    }
    __device__ __forceinline__ void add(const typename Pack<DT, W>::Raw (&raw)[kPacks],
                                        float (&acc)[kCols]) const
    {
#pragma unroll
        for (int i = 0; i < kPacks; ++i) {
            float x[kN];
            widen_pack<DT, W>(raw[i], x);
#pragma unroll
            for (int j = 0; j < kN; ++j)
                acc[i * kN + j] += x[j];
        }
    }
    // FP32 rows, in accesses of WF bytes (their rows' alignment).
    __device__ __forceinline__ void load_f(const float *base, size_t row, float (&v)[kCols]) const
    {
        constexpr int kF = WF / 4;
#pragma unroll
        for (int i = 0; i < kCols / kF; ++i) {
            float x[kF] = {};
            if (W == 16 || col + i * kF < hidden)
                widen_pack<LPCOLL_F32, WF>(
                    load_pack<LPCOLL_F32, WF>(base, row * hidden + col + i * kF), x);
#pragma unroll
            for (int j = 0; j < kF; ++j)
                v[i * kF + j] = x[j];
        }
    }
    __device__ __forceinline__ void store_f(float *base, size_t row, const float (&v)[kCols]) const
    {
        constexpr int kF = WF / 4;
#pragma unroll
        for (int i = 0; i < kCols / kF; ++i) {
            if (W != 16 && col + i * kF >= hidden)
                continue;
            float x[kF];
#pragma unroll
            for (int j = 0; j < kF; ++j)
                x[j] = v[i * kF + j];
            store_pack<LPCOLL_F32, WF>(base, row * hidden + col + i * kF,
                                       narrow_pack<LPCOLL_F32, WF>(x));
        }
    }
    // The finished sum of a row of the table.
    __device__ __forceinline__ void finish(const EmbedArgs &a, size_t row,
                                           const float (&acc)[kCols]) const
    {
        float v[kCols];
        if (a.accumulate)
            load_f(a.dtable, row, v);
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            const float s = acc[j] * a.scale;
            v[j] = a.accumulate ? v[j] + s : s;
        }
        store_f(a.dtable, row, v);
    }
};

// Zeros into the `rows` rows from v0 on whose bit in `used` is not set: a warp a row
// where there are enough of them, else a CTA.
template <int DT, int W>
__device__ __forceinline__ void clear_rows(const EmbedArgs &a, size_t v0, int rows,
                                           const uint32_t *used)
{
    constexpr int WF = LaneCols<DT, W>::WF;
    constexpr int kF = WF / 4;
    const float zero[kF] = {};
    const int warps = blockDim.x >> 5;
    const bool narrow = rows >= warps;
    const int lane = narrow ? threadIdx.x & 31 : threadIdx.x, lanes = narrow ? 32 : blockDim.x;
    for (int i = narrow ? threadIdx.x >> 5 : 0; i < rows; i += narrow ? warps : 1) {
        if (v0 + i >= a.vocab || (used[i >> 5] >> (i & 31) & 1u) != 0)
            continue;
        float *const row = a.dtable + (v0 + i) * a.hidden;
#pragma unroll 4
        for (size_t col = static_cast<size_t>(lane) * kF; col < a.hidden;
             col += static_cast<size_t>(lanes) * kF)
            store_pack<LPCOLL_F32, WF>(row, col, narrow_pack<LPCOLL_F32, WF>(zero));
    }
}

// ---------------------------------------------------------------------------
// The same sort in one launch, for up to kClusterTokens: a cluster of up to kSortCtas
// CTAs holds all keys and tokens in its shared memory, each CTA the places [rank n,
// rank n + n) of the order, and a pass writes them to their next places, in whatever
// CTA those are. A cluster barrier tells that all counts of a pass are there, another
// that all of its writes are. A CTA takes 2048 tokens before there is another.
// ---------------------------------------------------------------------------

constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
// As many as the shared memory of 8 CTAs holds. Against the launches through memory: 8192
// tokens into 32000 x 2048 BF16 64 us and 68, 16384 into 128000 x 1024 108 and 118, 32768
// into 32000 x 4096 155 and 160, 65536 into 32000 x 1024 90 and 87.
constexpr int kClusterTokens = 65536;

__device__ __forceinline__ unsigned sort_rank()
{
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void sort_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n\t"
                 "barrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t remote(const void *p, unsigned rank)
{
    const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    uint32_t far;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(local), "r"(rank));
    return far;
}

// Clears some rows of the table that no token has; the CTA looks for them in all ids.
template <int DT, int W>
__device__ __forceinline__ void clear_unused(const EmbedArgs &e, size_t v0, int rows, int *smem)
{
    uint32_t *const used = reinterpret_cast<uint32_t *>(smem);
    for (int w = threadIdx.x; w * 32 < rows; w += kSortThreads)
        used[w] = 0;
    __syncthreads();
#pragma unroll 8
    for (size_t t = threadIdx.x; t < e.tokens; t += kSortThreads) {
        const long long row = row_of(e, t) - static_cast<long long>(v0);
        if (row >= 0 && row < rows)
            atomicOr(&used[row >> 5], 1u << (row & 31));
    }
    __syncthreads();
    clear_rows<DT, W>(e, v0, rows, used);
}

// The first cluster sorts. Meanwhile the CTAs of the others clear `clear` rows of the
// table each.
template <int DT, int W>
__global__ void __launch_bounds__(kSortThreads)
cluster_sort_kernel(const __grid_constant__ EmbedArgs e, const RadixArgs a, int passes, int log_n,
                    int ctas, int clear)
{
    wait_prior_grid();
    extern __shared__ int sort_smem[];
    if (blockIdx.x >= static_cast<unsigned>(ctas)) {
        clear_unused<DT, W>(e, static_cast<size_t>(blockIdx.x - ctas) * clear, clear, sort_smem);
        return;
    }
    __shared__ int warp_total[kSortWarps];
    const int n = 1 << log_n, digits = 1 << a.bits;
    // [2][n] keys, [2][n] tokens, [warps][digits] places, [digits] counts, [digits] firsts
    int *const keys = sort_smem, *const order = keys + 2 * n;
    int *const next = order + 2 * n, *const count = next + kSortWarps * digits;
    int *const first = count + digits;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = sort_rank();
    const int lo = static_cast<int>(rank) * n;
    const int mine = max(0, min(n, a.tokens - lo));
    const int part = n / kSortWarps;  // a multiple of 32
    const int w_lo = warp * part, w_end = min(w_lo + part, mine);
    for (int w = static_cast<int>(rank) * kSortThreads + tid; w < a.words; w += ctas * kSortThreads)
        store_i32(reinterpret_cast<int32_t *>(a.used) + w, 0);
    for (int i = tid; i < mine; i += kSortThreads) {
        keys[i] = key_of(e, a, lo + i);
        order[i] = lo + i;
    }
    int from = 0;
    for (int pass = 0, shift = 0; pass < passes; ++pass, shift += a.bits, from ^= 1) {
        const int *const key_in = keys + from * n, *const order_in = order + from * n;
        for (int d = tid; d < kSortWarps * digits; d += kSortThreads)
            next[d] = 0;
        __syncthreads();
        for (int i = w_lo + lane; i < w_end; i += 32)
            atomicAdd(&next[warp * digits + (key_in[i] >> shift & (digits - 1))], 1);
        __syncthreads();
        int sum = 0;
        if (tid < digits) {
            int v[kSortWarps];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w)
                v[w] = next[w * digits + tid];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                next[w * digits + tid] = sum;
                sum += v[w];
            }
            count[tid] = sum;
        }
        sort_barrier();
        int total = 0, prior = 0;
        if (tid < digits) {
            int v[kSortCtas];
#pragma unroll
            for (int c = 0; c < kSortCtas; ++c) {
                v[c] = 0;
                if (c < ctas)
                    asm volatile("ld.shared::cluster.s32 %0, [%1];"
                                 : "=r"(v[c])
                                 : "r"(remote(count + tid, c))
                                 : "memory");
            }
#pragma unroll
            for (int c = 0; c < kSortCtas; ++c) {
                total += v[c];
                prior += c < static_cast<int>(rank) ? v[c] : 0;
            }
        }
        // exclusive sum of the totals over the digits
        int scan = total;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int v = __shfl_up_sync(kAll, scan, m);
            scan += lane >= m ? v : 0;
        }
        if (lane == 31)
            warp_total[warp] = scan;
        __syncthreads();
        if (tid < digits) {
            int before = scan - total + prior;
            for (int w = 0; w < warp; ++w)
                before += warp_total[w];
            first[tid] = before;
        }
        __syncthreads();
        for (int s0 = w_lo; s0 < w_end; s0 += 32) {
            const int i = s0 + lane;
            const bool there = i < w_end;
            const int key = there ? key_in[i] : -1;
            const int d = there ? key >> shift & (digits - 1) : -1;
            const unsigned same = __match_any_sync(kAll, d);
            if (there) {
                const int at = first[d] + next[warp * digits + d] +
                               __popc(same & ((1u << lane) - 1u));
                const int place = (from ^ 1) * n + (at & (n - 1));
                const unsigned owner = static_cast<unsigned>(at) >> log_n;
                asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(remote(keys + place, owner)),
                             "r"(key)
                             : "memory");
                asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(remote(order + place, owner)),
                             "r"(order_in[i])
                             : "memory");
            }
            __syncwarp();
            if (there && lane == __ffs(same) - 1)
                next[warp * digits + d] += __popc(same);
            __syncwarp();
        }
        sort_barrier();
    }
    for (int i = tid; i < mine; i += kSortThreads) {
        const int key = keys[from * n + i];
        store_i32(a.keys_out + lo + i, key);
        store_i32(a.order_out + lo + i, order[from * n + i]);
        // the bits were cleared before the last barrier; one for each run of the CTA
        if (key < static_cast<int>(e.vocab) && (i == 0 || keys[from * n + i - 1] != key) &&
            LPC_WRITE_OK(a.used + (key >> 5), 4))
            atomicOr(a.used + (key >> 5), 1u << (key & 31));
    }
}

// ---------------------------------------------------------------------------
// Sums of the sorted tokens' rows.
// ---------------------------------------------------------------------------

constexpr int kAhead = 8;        // rows that a lane loads before it adds them
constexpr int kMaxTile = 1024;   // sorted tokens of a CTA

struct SumArgs {
    const int32_t *keys, *order;
    const uint32_t *used;
    float *head, *tail;  // [tiles][hidden]: runs that came from the tile before, that go on
    int tokens, tile, tiles;
    size_t sum_ctas;     // the others clear
    unsigned every;      // every so many CTAs one that sums, as long as there are any
    int clear;           // rows of the table that one of the others clears
    size_t cleared;      // rows that the sort's launch has cleared
};

__device__ __forceinline__ int key_at(const SumArgs &s, long long i)
{
    return i >= 0 && i < s.tokens ? load_i32(s.keys + i) : -1;
}

// Rows of the table that a CTA clears: some 64 KB of them, a power of 2 up to 32. (200
// tokens into 8000 x 1024 6.9 us, with 16 KB 10.7, with 256 KB 8.4; 8192 into 32000 x 2048
// 64, 70 and 67.)
int rows_to_clear(size_t hidden)
{
    int rows = 1;
    while (rows < 32 && rows * hidden * sizeof(float) < 64 * 1024)
        rows *= 2;
    return rows;
}

template <int DT, int W>
__global__ void __launch_bounds__(kLanes)
embed_sums_kernel(const __grid_constant__ EmbedArgs a, const SumArgs s, const RowCut c)
{
    wait_prior_grid();
    using Cols = LaneCols<DT, W>;
    constexpr int kCols = Cols::kCols;
    // the CTAs that sum wait for memory, the others keep it busy meanwhile
    const size_t sums_before = min(s.sum_ctas, (blockIdx.x + static_cast<size_t>(s.every) - 1) / s.every);
    if (blockIdx.x % s.every != 0 || sums_before == s.sum_ctas) {
        const size_t v0 = s.cleared + (blockIdx.x - sums_before) * s.clear;
        const uint32_t bits =
            (s.used != nullptr && LPC_READ_OK(s.used + v0 / 32, 4) ? s.used[v0 / 32] : 0u) >>
            (v0 % 32);
        clear_rows<DT, W>(a, v0, s.clear, &bits);
        return;
    }
    // the keys of the CTA's tiles with one on either side, and the tokens
    extern __shared__ int keys_smem[];
    const size_t cta = sums_before;
    const long long cta_tile = static_cast<long long>(cta / c.segs) * c.rows;
    const int span = s.tile * c.rows;
    int *const keys = keys_smem, *const order = keys_smem + span + 2;
    const long long cta_lo = cta_tile * s.tile;
    for (int i = threadIdx.x; i < span + 2; i += blockDim.x) {
        keys[i] = key_at(s, cta_lo + i - 1);
        if (i < span && cta_lo + i < s.tokens)
            order[i] = load_i32(s.order + cta_lo + i);
    }
    __syncthreads();
    const Place p = place_of(c, cta);
    const Cols cols{static_cast<size_t>(p.piece) * kCols, a.hidden};
    const long long tile = static_cast<long long>(p.row);
    if (p.idle || tile >= s.tiles || cols.col >= a.hidden)
        return;
    const long long lo = tile * s.tile;
    const int first = static_cast<int>(lo - cta_lo);  // keys[first + 1] is the tile's first
    const int n = static_cast<int>(min(static_cast<long long>(s.tile), s.tokens - lo));
    const int vocab = static_cast<int>(a.vocab);
    float acc[kCols] = {};
    bool started = keys[first] != keys[first + 1];  // the run begins in this tile
    for (int i0 = 0; i0 < n && keys[first + 1 + i0] != vocab; i0 += kAhead) {
        typename Pack<DT, W>::Raw raw[kAhead][Cols::kPacks];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i0 + j < n && keys[first + 1 + i0 + j] != vocab)
                cols.load(a.dout, static_cast<size_t>(order[first + i0 + j]), raw[j]);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int at = first + 1 + i0 + j;
            if (i0 + j >= n || keys[at] == vocab)
                break;
            cols.add(raw[j], acc);
            const bool ends = keys[at + 1] != keys[at];
            if (ends || i0 + j + 1 == n) {
                if (started && ends)
                    cols.finish(a, static_cast<size_t>(keys[at]), acc);
                else
                    cols.store_f(started ? s.tail : s.head, static_cast<size_t>(tile), acc);
                started = true;
#pragma unroll
                for (int q = 0; q < kCols; ++q)
                    acc[q] = 0.0f;
            }
        }
    }
}

// The runs that begin in a tile and go on in the next ones.
template <int DT, int W>
__global__ void __launch_bounds__(kLanes)
embed_join_kernel(const __grid_constant__ EmbedArgs a, const SumArgs s, const RowCut c)
{
    wait_prior_grid();
    using Cols = LaneCols<DT, W>;
    constexpr int kCols = Cols::kCols;
    const Place p = place_of(c, blockIdx.x);
    const long long tile = static_cast<long long>(p.row);
    const Cols cols{static_cast<size_t>(p.piece) * kCols, a.hidden};
    if (p.idle || tile >= s.tiles || cols.col >= a.hidden)
        return;
    const long long lo = tile * s.tile, next = lo + s.tile;
    const int run = key_at(s, next - 1), after = key_at(s, next);
    const int start = key_at(s, lo), before = key_at(s, lo - 1);
    if (next >= s.tokens || after != run || run == static_cast<int>(a.vocab) ||
        (start == run && before == run))
        return;  // ends with the tile, or began before it
    // the next tiles' partial rows together with their first keys, some at a time, up to
    // the first key that is not the run's (what stands in that tile's row is not used)
    float acc[kCols];
    cols.load_f(s.tail, static_cast<size_t>(tile), acc);
    bool more = true;
    for (long long i = tile + 1; more && i < s.tiles; i += kAhead) {
        float v[kAhead][kCols];
        int key[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            key[j] = key_at(s, (i + j) * s.tile);
            if (i + j < s.tiles)
                cols.load_f(s.head, static_cast<size_t>(i + j), v[j]);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            more = more && key[j] == run;
            if (more)
#pragma unroll
                for (int q = 0; q < kCols; ++q)
                    acc[q] += v[j][q];
        }
    }
    cols.finish(a, static_cast<size_t>(run), acc);
}

// ---------------------------------------------------------------------------
// Few tokens: one launch, without a sort. A CTA for each token (and kLanes pieces of
// its row) looks through all ids: if an earlier token has the same row it has nothing to
// do, else it adds up the rows of the tokens that have. (Long lists in four parts, by as
// many groups of lanes, were slower: 512 tokens of 1024 FP32 with 64 tokens a row 8.4 us
// where one list takes 6.6, all of one row of 4096 BF16 42.1 and 41.1.) Two CTAs an SM
// leave the registers for all of a lane's rows in flight: 100 tokens into 8000 x 1024 BF16
// 6.3 us, 7.1 with the compiler's own choice, though 512 into 8000 x 8192, which are mostly
// clearing, 49.7 and 45.7.
// ---------------------------------------------------------------------------

// Against the sort and its launches: 200 tokens into 8000 x 1024 BF16 6.9 us and 12.4, 512
// 9.5 and 13.2, 900 13.8 and 14.1; into 8000 x 8192 512 50 and 48, 900 69 and 51.
constexpr int kFewTokens = 512;

template <int DT, int W>
__global__ void __launch_bounds__(kLanes, 2)
embed_few_kernel(const __grid_constant__ EmbedArgs a, unsigned segs, int clear)
{
    wait_prior_grid();
    using Cols = LaneCols<DT, W>;
    constexpr int kCols = Cols::kCols;
    __shared__ uint32_t same[kFewTokens / 32];  // bit t: token t has this CTA's row
    __shared__ int list[kFewTokens];
    const int T = static_cast<int>(a.tokens), tid = threadIdx.x, lane = tid & 31;
    const size_t sum_ctas = a.tokens * segs;
    if (blockIdx.x >= sum_ctas) {
        const size_t v0 = (blockIdx.x - sum_ctas) * clear;
        uint32_t bits = 0;
        for (int t = tid; t < T; t += kLanes) {
            const long long row = row_of(a, t) - static_cast<long long>(v0);
            if (row >= 0 && row < clear)
                bits |= 1u << row;
        }
        if (tid == 0)
            same[0] = 0;
        __syncthreads();
        if (bits != 0)
            atomicOr(&same[0], bits);
        __syncthreads();
        clear_rows<DT, W>(a, v0, clear, same);
        return;
    }
    const int mine = static_cast<int>(blockIdx.x / segs);
    const long long row = row_of(a, mine);
    if (row < 0)
        return;
    bool earlier = false;
    for (int w = tid >> 5; w * 32 < T; w += kLanes / 32) {
        const int t = w * 32 + lane;
        const bool hit = t < T && row_of(a, t) == row;
        earlier = earlier || (hit && t < mine);
        const uint32_t bits = __ballot_sync(kAll, hit);
        if (lane == 0)
            same[w] = bits;
    }
    if (__syncthreads_or(earlier))
        return;
    int n = 0;
    for (int w = 0; w * 32 < T; ++w)
        n += __popc(same[w]);
    for (int i = tid; i < n; i += kLanes) {
        int left = i, w = 0;
        while (left >= __popc(same[w]))
            left -= __popc(same[w++]);
        list[i] = w * 32 + static_cast<int>(__fns(same[w], 0, left + 1));
    }
    __syncthreads();
    const Cols cols{(static_cast<size_t>(blockIdx.x % segs) * kLanes + tid) * kCols, a.hidden};
    if (cols.col >= a.hidden)
        return;
    float acc[kCols] = {};
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        typename Pack<DT, W>::Raw raw[kAhead][Cols::kPacks];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i0 + j < n)
                cols.load(a.dout, static_cast<size_t>(list[i0 + j]), raw[j]);
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i0 + j < n)
                cols.add(raw[j], acc);
    }
    cols.finish(a, static_cast<size_t>(row), acc);
}

// Sorted tokens of a tile: few, so that small batches fill the GPU, and more where
// there are many tokens, so that the partial rows stay few. 900 tokens into 8000 x 1024
// BF16 14.1 us, with 16 15.6, with 32 19.7, though 8192 into 4000 x 2048, twice a row,
// 35, 30 and 28; 16384 into 128000 x 1024 108 with 32, 105 with 16, 114 with 64, 32768 into
// 32000 x 4096 155, 166 and 156.
int tile_len(size_t tokens)
{
    if (tokens <= 8192)
        return 8;
    size_t len = (tokens / 4096 + 31) / 32 * 32;
    len = len > 32 ? len : 32;
    return static_cast<int>(len < kMaxTile ? len : kMaxTile);
}

size_t aligned(size_t bytes) { return (bytes + 255) / 256 * 256; }

// The workspace: keys and order, twice and with the digits' counts where the sort goes
// through memory, the used rows' bits, and the partial rows.
struct Scratch {
    size_t keys, counts, used, partial;  // bytes of one
    size_t words, tiles;
    int copies;  // of keys and order
    size_t all() const { return 2 * copies * keys + counts + used + 2 * partial; }
};

Scratch scratch(size_t tokens, size_t vocab, size_t hidden)
{
    Scratch s;
    s.words = (vocab + 31) / 32;
    s.tiles = (tokens + tile_len(tokens) - 1) / tile_len(tokens);
    s.keys = aligned(tokens * sizeof(int32_t));
    s.copies = tokens > kClusterTokens ? 2 : 1;
    s.counts = tokens > kClusterTokens ? aligned(kDigits * chunks_of(tokens) * sizeof(int32_t)) : 0;
    s.used = aligned(s.words * sizeof(uint32_t));
    s.partial = aligned(s.tiles * hidden * sizeof(float));
    return s;
}

template <int DT, int W> cudaError_t embed_dt(const EmbedArgs &a, cudaStream_t st)
{
    RowCut c = cut(a.hidden, a.dtype, kPieces, kLanes);
    if (a.tokens * c.segs < static_cast<size_t>(kSms) * 4 * c.rows)  // few: a piece a lane
        c = cut(a.hidden, a.dtype, 1, kLanes);
    const size_t ctas = (a.tokens + c.rows - 1) / c.rows * c.segs;
    return launch_kernel_block(embed_kernel<DT, W>, ctas, c.lanes * c.rows, 0, st, a, c);
}

template <int DT, int W> cudaError_t few_dt(const EmbedArgs &a, cudaStream_t st)
{
    const int clear = rows_to_clear(a.hidden);
    const size_t clear_ctas = a.accumulate ? 0 : (a.vocab + clear - 1) / clear;
    const size_t seg = static_cast<size_t>(kLanes) * Fmt<DT>::kVec;
    const unsigned segs = static_cast<unsigned>((a.hidden + seg - 1) / seg);
    return launch_kernel_block(embed_few_kernel<DT, W>, a.tokens * segs + clear_ctas, kLanes, 0, st,
                               a, segs, clear);
}

// The sort in one launch, and with it the first `cleared` rows of the table cleared
// where they have no token: as much as the sort takes time for, on the SMs that it
// leaves free.
template <int DT, int W>
cudaError_t cluster_sort_dt(const EmbedArgs &a, const RadixArgs &r, int passes, size_t &cleared,
                            cudaStream_t st)
{
    const size_t free = kSms - kSortCtas;
    constexpr int kMostRows = 512;
    int log_n = 11, sorting = 1;
    while (sorting < kSortCtas && (sorting << log_n) < r.tokens)
        sorting *= 2;
    while ((sorting << log_n) < r.tokens)
        ++log_n;
    const size_t smem =
        ((static_cast<size_t>(4) << log_n) + (kSortWarps + 2) * (1u << r.bits)) * sizeof(int);
    // some 6 us and 0.7 ns a token, at 45 GB/s an SM (2000 tokens into 8000 x 1024 BF16
    // 17.8 us, with half of it 20.1; 16384 into 128000 x 1024 108, with twice as much 114)
    const size_t bytes = 256 * 1024 + 32 * a.tokens;
    int rows = kMostRows;
    while (rows > 1 && rows * a.hidden * sizeof(float) > bytes)
        rows /= 2;
    const size_t need = a.accumulate ? 0 : (a.vocab + rows - 1) / rows;
    // whole clusters
    const size_t ctas = (need < free ? need : free) / kSortCtas * kSortCtas;
    cleared = ctas * rows;
    // always the same value: calls of several threads must not undo each other's
    const cudaError_t e = cudaFuncSetAttribute(
        cluster_sort_kernel<DT, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e != cudaSuccess)
        return e;
    return launch_kernel_cluster(cluster_sort_kernel<DT, W>, sorting + ctas, kSortThreads, sorting,
                                 smem, st, a, r, passes, log_n, sorting, rows);
}

template <int DT, int W>
cudaError_t sums_dt(const EmbedArgs &a, SumArgs s, cudaStream_t st)
{
    RowCut c = cut(a.hidden, a.dtype, 1, kLanes);
    while (c.rows > 1 && c.rows * s.tile > kMaxTile)
        c.rows /= 2;
    s.sum_ctas = (static_cast<size_t>(s.tiles) + c.rows - 1) / c.rows * c.segs;
    s.clear = rows_to_clear(a.hidden);
    const size_t clear = a.accumulate || s.cleared >= a.vocab
                             ? 0
                             : (a.vocab - s.cleared + s.clear - 1) / s.clear;
    if (s.sum_ctas + clear == 0)
        return cudaSuccess;
    s.every = s.sum_ctas == 0 ? 1 : static_cast<unsigned>((s.sum_ctas + clear) / s.sum_ctas);
    const size_t smem = (2 * static_cast<size_t>(s.tile) * c.rows + 2) * sizeof(int);
    const cudaError_t e = launch_kernel_block(embed_sums_kernel<DT, W>, s.sum_ctas + clear,
                                              kLanes, smem, st, a, s, c);
    if (e != cudaSuccess || s.tiles <= 1)
        return e;
    return launch_kernel_block(embed_join_kernel<DT, W>, s.sum_ctas, kLanes, 0, st, a, s, c);
}

}  // namespace

size_t embed_workspace(size_t tokens, size_t vocab, size_t hidden)
{
    return tokens <= kFewTokens ? 0 : scratch(tokens, vocab, hidden).all();
}

cudaError_t launch_embed(const EmbedArgs &a, cudaStream_t st)
{
    return LPC_BY_ROW(embed_dt, a.dtype, a.hidden, a, st);
}

cudaError_t launch_embed_backward(const EmbedArgs &a, cudaStream_t st)
{
    SumArgs s = {};
    if (a.tokens > 0 && a.tokens <= kFewTokens)
        return LPC_BY_ROW(few_dt, a.dtype, a.hidden, a, st);
    if (a.tokens > 0) {
        const Scratch w = scratch(a.tokens, a.vocab, a.hidden);
        const SortPlan p = sort_plan(a.vocab);
        char *at = static_cast<char *>(a.workspace);
        int32_t *keys[2] = {}, *order[2] = {};
        for (int i = 0; i < w.copies; ++i) {
            keys[i] = reinterpret_cast<int32_t *>(at);
            order[i] = reinterpret_cast<int32_t *>(at + w.keys);
            at += 2 * w.keys;
        }
        RadixArgs r = {};
        r.counts = reinterpret_cast<int32_t *>(at);
        r.used = reinterpret_cast<uint32_t *>(at + w.counts);
        at += w.counts + w.used;
        s.head = reinterpret_cast<float *>(at);
        s.tail = reinterpret_cast<float *>(at + w.partial);
        r.tokens = static_cast<int>(a.tokens);
        r.words = static_cast<int>(w.words);
        r.bits = p.bits;
        r.chunks = static_cast<int>(chunks_of(a.tokens));
        r.chunk_len = static_cast<int>(chunk_len(a.tokens));
        if (a.tokens <= kClusterTokens) {
            r.keys_out = keys[0];
            r.order_out = order[0];
            const cudaError_t e =
                LPC_BY_ROW(cluster_sort_dt, a.dtype, a.hidden, a, r, p.passes, s.cleared, st);
            if (e != cudaSuccess)
                return e;
            r.keys = r.keys_out;
            r.order = r.order_out;
        }
        for (int i = 0; i < p.passes && a.tokens > kClusterTokens; ++i) {
            r.shift = i * p.bits;
            r.keys_out = keys[i & 1];
            r.order_out = order[i & 1];
            cudaError_t e = launch_kernel_block(radix_count_kernel, r.chunks, kThreads, 0, st, a, r);
            if (e == cudaSuccess)
                e = launch_kernel_block(radix_place_kernel, r.chunks, kThreads, 0, st, a, r);
            if (e != cudaSuccess)
                return e;
            r.keys = r.keys_out;
            r.order = r.order_out;
        }
        s.keys = r.keys;
        s.order = r.order;
        s.used = r.used;
        s.tokens = static_cast<int>(a.tokens);
        s.tile = tile_len(a.tokens);
        s.tiles = static_cast<int>(w.tiles);
    }
    return LPC_BY_ROW(sums_dt, a.dtype, a.hidden, a, s, st);
}

}  // namespace lpc
