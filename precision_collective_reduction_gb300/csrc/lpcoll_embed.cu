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
// in order. So frequent tokens are shared out over many CTAs without atomics, and
// the same call gives the same bits. Rows of the table without a token are
// cleared by CTAs of the same launch.
#include "lpcoll_layers.cuh"

namespace lpc {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kLanes = 256;

// How a row is cut: `segs` CTAs of `lanes` lanes with 16 bytes (of the table or of
// dout) each; short rows share a CTA, `rows` of them.
struct RowCut {
    unsigned segs;
    int lanes, rows;
};

RowCut cut(size_t hidden, int dtype)
{
    const size_t per_lane = 16 / dtype_bytes(dtype);
    const size_t lanes = (hidden + per_lane - 1) / per_lane;
    RowCut r;
    r.segs = static_cast<unsigned>((lanes + kLanes - 1) / kLanes);
    r.lanes = static_cast<int>((lanes + r.segs - 1) / r.segs);
    r.rows = r.segs > 1 ? 1 : kLanes / r.lanes;
    return r;
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

template <int DT, int W>
__global__ void __launch_bounds__(kLanes)
embed_kernel(const __grid_constant__ EmbedArgs a, const RowCut c)
{
    wait_prior_grid();
    constexpr int kN = Pack<DT, W>::kN;
    constexpr int kCols = Fmt<DT>::kVec;
    constexpr int kPacks = kCols / kN;
    const int which = static_cast<int>(threadIdx.x) / c.lanes;
    const size_t t = static_cast<size_t>(blockIdx.x / c.segs) * c.rows + which;
    const size_t col = (static_cast<size_t>(blockIdx.x % c.segs) * c.lanes +
                        (static_cast<int>(threadIdx.x) - which * c.lanes)) * kCols;
    if (t >= a.tokens || col >= a.hidden)
        return;
    const long long row = row_of(a, t);
    typename Pack<DT, W>::Raw raw[kPacks];
#pragma unroll
    for (int i = 0; i < kPacks; ++i) {
        raw[i] = {};
        if (row >= 0 && (W == 16 || col + i * kN < a.hidden))
            raw[i] = load_pack<DT, W>(a.table, static_cast<size_t>(row) * a.hidden + col + i * kN);
    }
#pragma unroll
    for (int i = 0; i < kPacks; ++i) {
        if (W != 16 && col + i * kN >= a.hidden)
            continue;
        float x[kN];
        widen_pack<DT, W>(raw[i], x);
        if (row >= 0)  // other rows are +0, whatever the scale
#pragma unroll
            for (int j = 0; j < kN; ++j)
                x[j] = x[j] * a.scale;
        store_pack<DT, W>(a.out, t * a.hidden + col + i * kN, narrow_pack<DT, W>(x));
    }
}

// ---------------------------------------------------------------------------
// Tokens sorted by row: a radix sort of (row, token), digits of up to kDigitBits
// bits, each pass a stable counting sort. The tokens are cut into chunks, one CTA
// each; with more than one, a first launch counts the digits of every chunk, and a
// CTA of the second adds up the counts of the chunks before its own. Tokens
// without a row have the key `vocab` and come last.
// ---------------------------------------------------------------------------

constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kMaxChunks = 128;
constexpr int kOneChunk = 2048;  // tokens that one CTA sorts in one launch a pass
constexpr int kMinChunk = 512;

struct SortPlan {
    int passes, bits;  // bits of a digit
    int chunks, chunk_len;
};

SortPlan sort_plan(size_t tokens, size_t vocab)
{
    int key_bits = 1;
    while (key_bits < 32 && (vocab >> key_bits) != 0)
        ++key_bits;
    SortPlan p;
    p.passes = (key_bits + kDigitBits - 1) / kDigitBits;
    p.bits = (key_bits + p.passes - 1) / p.passes;
    size_t len = kOneChunk;
    if (tokens > kOneChunk) {
        const size_t even = (tokens + kMaxChunks - 1) / kMaxChunks;
        len = (even + kThreads - 1) / kThreads * kThreads;
        len = len > kMinChunk ? len : kMinChunk;
    }
    p.chunk_len = static_cast<int>(len);
    p.chunks = tokens == 0 ? 1 : static_cast<int>((tokens + len - 1) / len);
    return p;
}

struct RadixArgs {
    const int32_t *keys, *order;  // of the pass before; NULL in the first
    int32_t *keys_out, *order_out;
    int32_t *counts;   // [digits][chunks]
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
        store_i32(a.counts + static_cast<size_t>(d) * a.chunks + blockIdx.x, hist[d]);
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
    if (a.keys == nullptr && a.chunks == 1)
        for (int w = tid; w < a.words; w += kThreads)
            store_i32(reinterpret_cast<int32_t *>(a.used) + w, 0);
    __syncthreads();

    const long long lo = static_cast<long long>(blockIdx.x) * a.chunk_len;
    const long long end = min(lo + a.chunk_len, static_cast<long long>(a.tokens));
    const int part = (a.chunk_len / kWarpsPerCta + 31) & ~31;
    const long long w_lo = lo + static_cast<long long>(warp) * part;
    const long long w_end = min(w_lo + part, end);
    for (long long i = w_lo + lane; i < w_end; i += 32)
        atomicAdd(&next[warp][key_of(e, a, static_cast<int>(i)) >> a.shift & (digits - 1)], 1);
    if (a.chunks > 1) {
        // a warp per digit, a lane per chunk
        constexpr int kSteps = kMaxChunks / 32;
        for (int d = warp; d < digits; d += kWarpsPerCta) {
            int sum = 0, prior = 0;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int c = i * 32 + lane;
                const int v = c < a.chunks
                                  ? load_i32(a.counts + static_cast<size_t>(d) * a.chunks + c)
                                  : 0;
                sum += v;
                prior += c < static_cast<int>(blockIdx.x) ? v : 0;
            }
            sum = __reduce_add_sync(kAll, sum);
            prior = __reduce_add_sync(kAll, prior);
            if (lane == 0) {
                total[d] = sum;
                before[d] = prior;
            }
        }
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
        if (a.chunks == 1) {
            total[d] = run;
            before[d] = 0;
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

// ---------------------------------------------------------------------------
// Sums of the sorted tokens' rows.
// ---------------------------------------------------------------------------

constexpr int kAhead = 4;        // rows that a lane loads before it adds them
constexpr int kClearRows = 8;    // rows of the table that a CTA clears

struct SumArgs {
    const int32_t *keys, *order;
    const uint32_t *used;
    float *head, *tail;  // [tiles][hidden]: runs that came from the tile before, that go on
    int tokens, tile, tiles;
    size_t sum_ctas;     // the CTAs behind these clear
};

__device__ __forceinline__ int key_at(const SumArgs &s, long long i)
{
    return i >= 0 && i < s.tokens ? load_i32(s.keys + i) : -1;
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

template <int DT, int W>
__global__ void __launch_bounds__(kLanes)
embed_sums_kernel(const __grid_constant__ EmbedArgs a, const SumArgs s, const RowCut c)
{
    wait_prior_grid();
    using Cols = LaneCols<DT, W>;
    constexpr int kCols = Cols::kCols;
    const int which = static_cast<int>(threadIdx.x) / c.lanes;
    const int lane = static_cast<int>(threadIdx.x) - which * c.lanes;
    if (blockIdx.x >= s.sum_ctas) {  // clears rows without a token
        const size_t v0 = (blockIdx.x - s.sum_ctas) * kClearRows;
        const uint32_t bits =
            s.used != nullptr && LPC_READ_OK(s.used + v0 / 32, 4) ? s.used[v0 / 32] : 0u;
        const float zero[kCols] = {};
        for (int i = which; i < kClearRows; i += c.rows) {
            if (v0 + i >= a.vocab || (bits >> ((v0 + i) % 32) & 1u) != 0)
                continue;
            for (unsigned seg = 0; seg < c.segs; ++seg) {
                const Cols cols{(static_cast<size_t>(seg) * c.lanes + lane) * kCols, a.hidden};
                if (cols.col < a.hidden)
                    cols.store_f(a.dtable, v0 + i, zero);
            }
        }
        return;
    }
    const long long tile = static_cast<long long>(blockIdx.x / c.segs) * c.rows + which;
    const Cols cols{(static_cast<size_t>(blockIdx.x % c.segs) * c.lanes + lane) * kCols, a.hidden};
    if (tile >= s.tiles || cols.col >= a.hidden)
        return;
    const long long lo = tile * s.tile;
    const long long end = min(lo + s.tile, static_cast<long long>(s.tokens));
    const int vocab = static_cast<int>(a.vocab);
    float acc[kCols] = {};
    int run = key_at(s, lo);
    bool started = key_at(s, lo - 1) != run;  // the run begins in this tile
    for (long long i0 = lo; i0 < end && run != vocab; i0 += kAhead) {
        int key[kAhead + 1];
        typename Pack<DT, W>::Raw raw[kAhead][Cols::kPacks];
#pragma unroll
        for (int j = 0; j <= kAhead; ++j)
            key[j] = key_at(s, i0 + j);
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i0 + j < end && key[j] != vocab)
                cols.load(a.dout, static_cast<size_t>(load_i32(s.order + i0 + j)), raw[j]);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (i0 + j >= end || key[j] == vocab)
                break;
            cols.add(raw[j], acc);
            const bool ends = key[j + 1] != key[j];
            if (ends || i0 + j + 1 == end) {
                if (started && ends)
                    cols.finish(a, static_cast<size_t>(key[j]), acc);
                else
                    cols.store_f(started ? s.tail : s.head, static_cast<size_t>(tile), acc);
                started = true;
#pragma unroll
                for (int q = 0; q < kCols; ++q)
                    acc[q] = 0.0f;
            }
            run = key[j + 1];
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
    const int which = static_cast<int>(threadIdx.x) / c.lanes;
    const int lane = static_cast<int>(threadIdx.x) - which * c.lanes;
    const long long tile = static_cast<long long>(blockIdx.x / c.segs) * c.rows + which;
    const Cols cols{(static_cast<size_t>(blockIdx.x % c.segs) * c.lanes + lane) * kCols, a.hidden};
    if (tile >= s.tiles || cols.col >= a.hidden)
        return;
    const long long lo = tile * s.tile, next = lo + s.tile;
    const int run = key_at(s, next - 1);
    if (next >= s.tokens || run == static_cast<int>(a.vocab) || key_at(s, next) != run)
        return;  // ends with the tile
    if (key_at(s, lo) == run && key_at(s, lo - 1) == run)
        return;  // began before it
    // the last tile of the run: its first key is the run's, the next tile's is not
    long long at = tile + 1, above = s.tiles;  // key of tile `at` is the run's, of `above` not
    while (above - at > 1) {
        const long long mid = (at + above) / 2;
        if (key_at(s, mid * s.tile) == run)
            at = mid;
        else
            above = mid;
    }
    float acc[kCols];
    cols.load_f(s.tail, static_cast<size_t>(tile), acc);
    for (long long i = tile + 1; i <= at; i += kAhead) {
        float v[kAhead][kCols];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i + j <= at)
                cols.load_f(s.head, static_cast<size_t>(i + j), v[j]);
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i + j <= at)
#pragma unroll
                for (int q = 0; q < kCols; ++q)
                    acc[q] += v[j][q];
    }
    cols.finish(a, static_cast<size_t>(run), acc);
}

// Sorted tokens of a tile: few, so that small batches fill the GPU, and more where
// there are many tokens, so that the partial rows stay few.
int tile_len(size_t tokens)
{
    if (tokens <= 4096)
        return 8;
    const size_t len = (tokens / 4096 + 31) / 32 * 32;
    return static_cast<int>(len > 32 ? len : 32);
}

size_t aligned(size_t bytes) { return (bytes + 255) / 256 * 256; }

// The workspace: keys and order twice, the digits' counts, the used rows' bits, and
// the partial rows.
struct Scratch {
    size_t keys, counts, used, partial;  // bytes of one
    size_t words, tiles;
    size_t all() const { return 4 * keys + counts + used + 2 * partial; }
};

Scratch scratch(size_t tokens, size_t vocab, size_t hidden)
{
    Scratch s;
    s.words = (vocab + 31) / 32;
    s.tiles = (tokens + tile_len(tokens) - 1) / tile_len(tokens);
    s.keys = aligned(tokens * sizeof(int32_t));
    s.counts = aligned(static_cast<size_t>(kDigits) * sort_plan(tokens, vocab).chunks *
                       sizeof(int32_t));
    s.used = aligned(s.words * sizeof(uint32_t));
    s.partial = aligned(s.tiles * hidden * sizeof(float));
    return s;
}

template <int DT, int W> cudaError_t embed_dt(const EmbedArgs &a, cudaStream_t st)
{
    const RowCut c = cut(a.hidden, a.dtype);
    const size_t ctas = (a.tokens + c.rows - 1) / c.rows * c.segs;
    return launch_kernel_block(embed_kernel<DT, W>, ctas, c.lanes * c.rows, 0, st, a, c);
}

template <int DT, int W>
cudaError_t sums_dt(const EmbedArgs &a, SumArgs s, cudaStream_t st)
{
    const RowCut c = cut(a.hidden, a.dtype);
    s.sum_ctas = (static_cast<size_t>(s.tiles) + c.rows - 1) / c.rows * c.segs;
    const size_t clear = a.accumulate ? 0 : (a.vocab + kClearRows - 1) / kClearRows;
    if (s.sum_ctas + clear == 0)
        return cudaSuccess;
    const cudaError_t e = launch_kernel_block(embed_sums_kernel<DT, W>, s.sum_ctas + clear,
                                              c.lanes * c.rows, 0, st, a, s, c);
    if (e != cudaSuccess || s.tiles <= 1)
        return e;
    return launch_kernel_block(embed_join_kernel<DT, W>, s.sum_ctas, c.lanes * c.rows, 0, st, a, s,
                               c);
}

}  // namespace

size_t embed_workspace(size_t tokens, size_t vocab, size_t hidden)
{
    return tokens == 0 ? 0 : scratch(tokens, vocab, hidden).all();
}

cudaError_t launch_embed(const EmbedArgs &a, cudaStream_t st)
{
    return LPC_BY_ROW(embed_dt, a.dtype, a.hidden, a, st);
}

cudaError_t launch_embed_backward(const EmbedArgs &a, cudaStream_t st)
{
    SumArgs s = {};
    if (a.tokens > 0) {
        const Scratch w = scratch(a.tokens, a.vocab, a.hidden);
        const SortPlan p = sort_plan(a.tokens, a.vocab);
        char *at = static_cast<char *>(a.workspace);
        int32_t *keys[2], *order[2];
        for (int i = 0; i < 2; ++i) {
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
        r.chunks = p.chunks;
        r.chunk_len = p.chunk_len;
        for (int i = 0; i < p.passes; ++i) {
            r.shift = i * p.bits;
            r.keys_out = keys[i & 1];
            r.order_out = order[i & 1];
            if (p.chunks > 1) {
                const cudaError_t e =
                    launch_kernel_block(radix_count_kernel, p.chunks, kThreads, 0, st, a, r);
                if (e != cudaSuccess)
                    return e;
            }
            const cudaError_t e =
                launch_kernel_block(radix_place_kernel, p.chunks, kThreads, 0, st, a, r);
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
