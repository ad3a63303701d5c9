// embed.hip -- the embedding of tokens and its gradient (gfx950).
//
//   y_t = scale table[id_t]         dtable[v] = scale sum over t with id_t = v of dy_t
//
// Bound by HBM: forward each row read and written, backward dy read once and
// dtable written once. The gradient's sums are taken in a fixed order, so results
// are the same every time: the tokens are sorted by their ids (a stable radix
// sort, 9 bits a pass, of numbers only), each row's tokens then follow one
// another, and a wave adds up a row's, in their order, in registers to the one
// write of it, zeros where there are none. A row with more tokens than a slice of
// the sorted order is long gets the sum of each slice first and then theirs, by
// quarters, so a token that makes up all of a text costs no more than many that
// do not.
//
// Measured (bf16, 16384 tokens of 2048, a tenth of them padding, the r-th most
// frequent of 50001 rows about 1/r as often as the first): forward 17 us, sort and
// starts 29, the frequent rows' slices 11 and rows 45 to
// 48 (5.2 to 5.6 TB/s).
#include <cmath>

#include "embed_internal.h"
#include "seq_host.h"
#include "seq_tokens.h"

namespace gconv {
namespace {

constexpr int kBits = 9, kBins = 1 << kBits;
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct Embed {
    const void *table, *ids, *dy;
    void *y, *dtable;
    int64_t tokens, rows;     // of all sequences; of the table
    int64_t per_seq, dy_seq, dy_tok;
    int dim, wide;
    float scale;
    // sorting
    uint32_t *key[2], *at[2]; // [tokens]: ids (rows for one outside the table) and tokens, in two orders
    uint32_t* counts;         // [blocks][kBins]
    uint32_t* start;          // [rows + 1]: first place of each row's tokens
    int blocks, chunk;        // of the sort: tokens of a block, a multiple of kThreads
    int shift;
    // sums
    float* part;              // [slices][2][dim]: of the row that runs into a slice, and of the one that runs out
    int slice;                // tokens
    int64_t slices;           // none where no row can have more tokens than one
    int64_t stretches;        // of columns
    int flat;                 // dy's rows follow one another at its tokens' stride
    // sums for rows that have tokens alone (embed_internal.h)
    const float* weight;      // [tokens]
    void* runs;               // a row's sum, at its tokens' first place
    int64_t row0, row1;       // rows that are asked for
};

__device__ __forceinline__ uint32_t key_of(const Embed& a, int64_t t)
{
    const int64_t id = a.wide ? ((const int64_t*)a.ids)[t] : (int64_t)((const int32_t*)a.ids)[t];
    return id >= 0 && id < a.rows ? (uint32_t)id : (uint32_t)a.rows;
}

// A thread: a piece of V columns (the last of a row begins further left where it
// would end past it) of R tokens, whose rows are under way together.
template <typename T, int V, int R>
__global__ __launch_bounds__(kThreads) void embed_fwd(Embed a, int px)
{
    const int per = kThreads / px, tx = threadIdx.x % px, ty = threadIdx.x / px;
    const int64_t t0 = (int64_t)blockIdx.x * per * R + ty;
    uint32_t id[R];
#pragma unroll
    for (int i = 0; i < R; ++i) id[i] = t0 + i * per < a.tokens ? key_of(a, t0 + i * per) : (uint32_t)a.rows;
    for (int first = tx * V; first < a.dim; first += px * V) {
        const int col = min(first, a.dim - V);
        Packed<T, V> p[R];
#pragma unroll
        for (int i = 0; i < R; ++i) p[i] = *(const Packed<T, V>*)((const T*)a.table + (int64_t)(id[i] < a.rows ? id[i] : 0) * a.dim + col);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (t0 + i * per >= a.tokens) break;
            Packed<T, V> o;
#pragma unroll
            for (int e = 0; e < V; ++e) o.e[e] = id[i] < a.rows ? (T)(a.scale * (float)p[i].e[e]) : (T)0.f;
            *(Packed<T, V>*)((T*)a.y + (t0 + i * per) * a.dim + col) = o;
        }
    }
}

// ---- sorting ----------------------------------------------------------------------

template <bool FIRST>
__device__ __forceinline__ uint32_t sort_key(const Embed& a, int from, int64_t i)
{
    return FIRST ? key_of(a, i) : a.key[from][i];
}

// How many of a block's keys have each digit.
template <bool FIRST>
__global__ __launch_bounds__(kThreads) void embed_count(Embed a, int from)
{
    __shared__ uint32_t bins[kBins];
    for (int i = threadIdx.x; i < kBins; i += kThreads) bins[i] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.tokens);
    for (int64_t t = t0 + threadIdx.x; t < t1; t += kThreads) atomicAdd(&bins[sort_key<FIRST>(a, from, t) >> a.shift & (kBins - 1)], 1u);
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads) a.counts[(int64_t)blockIdx.x * kBins + i] = bins[i];
}

// Sum of v over the threads before this one.
__device__ __forceinline__ uint32_t exclusive_sum(uint32_t v, uint32_t* red)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t s = v;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const uint32_t o = __shfl_up(s, k);
        if (lane >= k) s += o;
    }
    if (lane == 63) red[wave] = s;
    __syncthreads();
    uint32_t before = 0;
    for (int k = 0; k < wave; ++k) before += red[k];
    __syncthreads();
    return before + s - v;
}

// Puts a block's keys in their places: those of smaller digits, of earlier
// blocks, of earlier waves, and of the wave's earlier keys come before each. A
// wave takes 64 keys that follow one another at a time; lanes with the same digit
// find one another by a vote on each of its bits.
template <bool FIRST>
__global__ __launch_bounds__(kThreads) void embed_place(Embed a, int from, int to)
{
    static_assert(kBins == 2 * kThreads, "two digits a thread");
    __shared__ uint32_t next[kWaves][kBins], red[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // this thread's digits: all of them before this block, and in all
    uint32_t mine[2] = {0, 0}, all[2] = {0, 0};
#pragma unroll 8
    for (int k = 0; k < a.blocks; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t c = a.counts[(int64_t)k * kBins + threadIdx.x * 2 + i];
            all[i] += c;
            if (k < (int)blockIdx.x) mine[i] += c;
        }
    const uint32_t before = exclusive_sum(all[0] + all[1], red);
    for (int i = threadIdx.x; i < kWaves * kBins; i += kThreads) next[0][i] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * a.chunk, own = t0 + (int64_t)wave * (a.chunk / kWaves);
    const int64_t end = min(own + a.chunk / kWaves, a.tokens);
    for (int64_t t = own + lane; t < end; t += 64) atomicAdd(&next[wave][sort_key<FIRST>(a, from, t) >> a.shift & (kBins - 1)], 1u);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t at = before + (i ? all[0] : 0) + mine[i];
        for (int k = 0; k < kWaves; ++k) {
            const uint32_t c = next[k][threadIdx.x * 2 + i];
            next[k][threadIdx.x * 2 + i] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t t = own; t < end; t += 64) {
        const bool have = t + lane < end;
        const uint32_t key = have ? sort_key<FIRST>(a, from, t + lane) : 0, digit = key >> a.shift & (kBins - 1);
        uint64_t same = __ballot(have);
#pragma unroll
        for (int b = 0; b < kBits; ++b) {
            const uint64_t set = __ballot(digit >> b & 1);
            same &= digit >> b & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        const uint32_t place = have ? next[wave][digit] + rank : 0;
        __builtin_amdgcn_wave_barrier();
        if (have && rank == 0) next[wave][digit] += __popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (have) {
            a.key[to][place] = key;
            a.at[to][place] = FIRST ? (uint32_t)(t + lane) : a.at[from][t + lane];
        }
    }
}

// start[v] = the first place whose key is v or more.
__global__ __launch_bounds__(kThreads) void embed_starts(Embed a, int from)
{
    const int64_t v = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (v > a.rows) return;
    int64_t lo = 0, hi = a.tokens;
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (a.key[from][mid] < v) lo = mid + 1;
        else hi = mid;
    }
    a.start[v] = (uint32_t)lo;
}

// ---- sums -------------------------------------------------------------------------

// A lane's pieces of a row: V columns each, W of them, 64 lanes' side by side. No
// branches: a piece that would end past the row begins further left (or is the
// row's last once more), so that the rows of many tokens load side by side; what
// two lanes hold twice is the same and they write the same.
template <int V, int W>
struct Sum {
    float v[W][V] = {};
    template <typename U>
    __device__ __forceinline__ void add(const U* row, const int (&col)[W], float weight = 1.f)
    {
        Packed<U, V> p[W];
#pragma unroll
        for (int k = 0; k < W; ++k) p[k] = *(const Packed<U, V>*)(row + col[k]);
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) v[k][e] = fmaf(weight, (float)p[k].e[e], v[k][e]);
    }
    // first: the column of the lane's first piece, before any was moved; STREAM: past the caches
    template <bool STREAM = false, typename U>
    __device__ __forceinline__ void store(U* row, const int (&col)[W], int first, int dim, float scale) const
    {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            if (first + k * 64 * V >= dim) break;
            Packed<U, V> o;
#pragma unroll
            for (int e = 0; e < V; ++e) o.e[e] = (U)(v[k][e] * scale);
            if constexpr (STREAM) {
                typedef uint32_t words __attribute__((ext_vector_type(4), aligned(2)));
                __builtin_nontemporal_store(__builtin_bit_cast(words, o), (words*)(row + col[k]));
            } else {
                *(Packed<U, V>*)(row + col[k]) = o;
            }
        }
    }
};

template <int V, int W>
__device__ __forceinline__ void columns(int first, int dim, int (&col)[W])
{
#pragma unroll
    for (int k = 0; k < W; ++k) col[k] = min(first + k * 64 * V, dim - V);
}

// dy's row of a token.
template <typename T>
__device__ __forceinline__ const T* dy_row(const Embed& a, uint32_t t)
{
    if (a.flat) return (const T*)a.dy + t * a.dy_tok;
    const uint32_t n = t / (uint32_t)a.per_seq;
    return (const T*)a.dy + n * a.dy_seq + (int64_t)(t - n * (uint32_t)a.per_seq) * a.dy_tok;
}

// Adds dy of the tokens at places [p0, p1), whose numbers the lanes read 64 at a
// time, eight tokens' rows under way at once.
template <typename T, int V, int W, bool RUNS>
__device__ __forceinline__ void add_tokens(const Embed& a, const uint32_t* at, uint32_t p0, uint32_t p1, const int (&col)[W], Sum<V, W>& sum)
{
    const int lane = threadIdx.x & 63;
    for (uint32_t p = p0; p < p1; p += 64) {
        const uint32_t mine = at[min(p + lane, p1 - 1)];
        const int weight = RUNS ? __builtin_bit_cast(int, a.weight[mine]) : 0;
        auto weight_of = [&](int i) { return RUNS ? __builtin_bit_cast(float, __builtin_amdgcn_readlane(weight, i)) : 1.f; };
        const int n = (int)min(p1 - p, 64u);
        constexpr int U = 8;
        int i = 0;
        for (; i + U <= n; i += U) {
            Packed<T, V> r[U][W];
#pragma unroll
            for (int q = 0; q < U; ++q) {
                const T* row = dy_row<T>(a, __builtin_amdgcn_readlane(mine, i + q));
#pragma unroll
                for (int k = 0; k < W; ++k) r[q][k] = *(const Packed<T, V>*)(row + col[k]);
            }
#pragma unroll
            for (int q = 0; q < U; ++q)
#pragma unroll
                for (int k = 0; k < W; ++k)
#pragma unroll
                    for (int e = 0; e < V; ++e) sum.v[k][e] = fmaf(weight_of(i + q), (float)r[q][k].e[e], sum.v[k][e]);
        }
        for (; i < n; ++i) sum.add(dy_row<T>(a, __builtin_amdgcn_readlane(mine, i)), col, weight_of(i));
    }
}

// The slices' sums of rows with more tokens than a slice has: such a row runs
// into a slice, out of it, or both. A wave a slice and stretch of columns.
template <typename T, int V, int W, bool RUNS>
__global__ __launch_bounds__(kThreads) void embed_slices(Embed a, int from)
{
    constexpr int kCols = 64 * W * V;
    const int lane = threadIdx.x & 63;
    const int64_t id = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), s = id / a.stretches;
    if (s >= a.slices) return;
    const int c0 = (int)(id - s * a.stretches) * kCols + lane * V;
    int col[W];
    columns<V, W>(c0, a.dim, col);
    const uint32_t p0 = (uint32_t)(s * a.slice), p1 = (uint32_t)min(s * a.slice + a.slice, a.tokens);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const uint32_t k = a.key[from][which ? p1 - 1 : p0];
        if (k >= a.row1 || (RUNS && k < a.row0)) continue;
        const uint32_t b = a.start[k], e = a.start[k + 1];
        if (e - b <= (uint32_t)a.slice || (which == 0 ? b > p0 : b <= p0)) continue;
        Sum<V, W> sum;
        add_tokens<T, V, W, RUNS>(a, a.at[from], max(b, p0), min(e, p1), col, sum);
        sum.store(a.part + (s * 2 + which) * a.dim, col, c0, a.dim, 1.f);
    }
}

// Rows of dtable, a wave a row: rows that follow one another in turn, the next
// one's tokens looked up while one is written. The first workgroups take the rows
// with more tokens than a slice has, each a stretch of that of the slice in which
// it begins, from the slices' sums: a quarter of them a wave, then the quarters.
template <typename T, int V, int W, bool RUNS, bool STREAM>
__global__ __launch_bounds__(kThreads) void embed_rows(Embed a, int from)
{
    constexpr int kCols = 64 * W * V;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    auto to = [&](int64_t r, uint32_t b) { return RUNS ? (T*)a.runs + (int64_t)b * a.dim : (T*)a.dtable + r * a.dim; };
    if (blockIdx.x < a.slices * a.stretches) {
        __shared__ float red[kWaves][W][V][64];
        const int64_t s0 = blockIdx.x / a.stretches;
        const int c0 = (int)(blockIdx.x - s0 * a.stretches) * kCols;
        const uint32_t p0 = (uint32_t)(s0 * a.slice), p1 = (uint32_t)min(s0 * a.slice + a.slice, a.tokens);
        const uint32_t k = a.key[from][p1 - 1];
        if (k >= a.row1 || (RUNS && k < a.row0)) return;
        const uint32_t b = a.start[k], e = a.start[k + 1];
        if (e - b <= (uint32_t)a.slice || b < p0) return;
        const int64_t s1 = (e - 1) / a.slice + 1, per = (s1 - s0 + kWaves - 1) / kWaves;
        Sum<V, W> sum;
        int col[W];
        columns<V, W>(c0 + lane * V, a.dim, col);
        const int64_t from_s = s0 + wave * per, to_s = min(from_s + per, s1);
#pragma unroll 4
        for (int64_t s = from_s; s < to_s; ++s) sum.add(a.part + (s * 2 + (b > s * a.slice ? 1 : 0)) * a.dim, col);
#pragma unroll
        for (int q = 0; q < W; ++q)
#pragma unroll
            for (int i = 0; i < V; ++i) red[wave][q][i][lane] = sum.v[q][i];
        __syncthreads();
        if (wave != 0) return;
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
#pragma unroll
            for (int q = 0; q < W; ++q)
#pragma unroll
                for (int i = 0; i < V; ++i) sum.v[q][i] += red[w][q][i][lane];
        sum.store(to(k, b), col, c0 + lane * V, a.dim, a.scale);
        return;
    }
    const int64_t before = a.slices * a.stretches, waves = (gridDim.x - before) * kWaves, first = (blockIdx.x - before) * kWaves + wave;
    const int64_t per = (a.row1 - a.row0 + waves - 1) / waves, r0 = a.row0 + first * per, r1 = min(r0 + per, a.row1);
    if (r0 >= r1) return;
    uint32_t b = a.start[r0], e = a.start[r0 + 1];
    for (int64_t r = r0; r < r1; ++r) {
        const uint32_t next = r + 1 < r1 ? a.start[r + 2] : 0;
        if (e - b <= (uint32_t)a.slice && (!RUNS || e > b)) {
            for (int c0 = 0; c0 < a.dim; c0 += kCols) {
                Sum<V, W> sum;
                int col[W];
                columns<V, W>(c0 + lane * V, a.dim, col);
                add_tokens<T, V, W, RUNS>(a, a.at[from], b, e, col, sum);
                sum.template store<STREAM>(to(r, b), col, c0 + lane * V, a.dim, a.scale);
            }
        }
        b = e;
        e = next;
    }
}

// ---- host ------------------------------------------------------------------------

constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int64_t kMaxDim = (int64_t)1 << 24;

int check_desc(const gconv_embed_desc* d)
{
    if (!d) return fail(GCONV_ERR_NULL, "descriptor is NULL");
    if (d->dtype != GCONV_F32 && d->dtype != GCONV_BF16) return fail(GCONV_ERR_ARG, "unknown dtype %lld", (long long)d->dtype);
    if (d->index != GCONV_I32 && d->index != GCONV_I64) return fail(GCONV_ERR_ARG, "unknown index type %lld", (long long)d->index);
    if (d->sequences < 0 || d->tokens < 0 || d->rows < 1 || d->dim < 1)
        return fail(GCONV_ERR_SHAPE, "need sequences, tokens >= 0 and rows, dim >= 1 (got %lld, %lld, %lld, %lld)", (long long)d->sequences,
                    (long long)d->tokens, (long long)d->rows, (long long)d->dim);
    if (d->rows >= (int64_t)1 << 31) return fail(GCONV_ERR_UNSUPPORTED, "rows=%lld not below 2^31", (long long)d->rows);
    if (d->dim > kMaxDim) return fail(GCONV_ERR_UNSUPPORTED, "dim=%lld above %lld", (long long)d->dim, (long long)kMaxDim);
    if (d->sequences > kMaxTokens || d->tokens > kMaxTokens || (d->tokens > 0 && d->sequences > kMaxTokens / d->tokens))
        return fail(GCONV_ERR_UNSUPPORTED, "too many ids");
    if (!std::isfinite((float)d->scale)) return fail(GCONV_ERR_ARG, "scale must be finite as float32");
    return GCONV_OK;
}

// Columns of a lane's piece (16 bytes, or one where a row has not as many) and
// pieces of a lane.
void pieces(bool bf16, int64_t dim, int* v, int* w)
{
    const int most = bf16 ? 8 : 4;
    *v = dim >= most ? most : 1;
    *w = dim <= 64 * *v ? 1 : 2;
}

struct Layout {
    size_t key[2], at[2], counts, start, part, bytes;
};

void plan(const gconv_embed_desc* d, Embed* a, Layout* l)
{
    a->tokens = d->sequences * d->tokens;
    a->per_seq = std::max<int64_t>(d->tokens, 1);
    a->rows = a->row1 = d->rows;
    a->dim = (int)d->dim;
    a->wide = d->index == GCONV_I64;
    a->scale = (float)d->scale;
    a->dy_seq = d->dy_stride[0];
    a->dy_tok = d->dy_stride[1];
    a->flat = d->sequences == 1 || d->dy_stride[0] == d->tokens * d->dy_stride[1];
    // at most 256 blocks, each of which reads all of their counts
    int64_t chunk = 512;
    while (a->tokens > chunk * 256) chunk *= 2;
    a->chunk = (int)chunk;
    a->blocks = (int)((a->tokens + chunk - 1) / chunk);
    // four waves add up a long row's slices, beside the other rows: a slice a sixteenth as long as the slices of a token
    // that makes up the text are many (16384 tokens, half of them one: slices of 32 10.5 + 44.6 us, of 64 15.1 + 48.2)
    int64_t slice = 32;
    while (slice * slice * 16 < a->tokens && slice < 4096) slice *= 2;
    a->slice = (int)slice;
    a->slices = a->tokens > slice ? (a->tokens + slice - 1) / slice : 0;
    int v, w;
    pieces(d->dtype == GCONV_BF16, d->dim, &v, &w);
    a->stretches = (a->dim + 64 * v * w - 1) / (64 * v * w);
    Cut cut;
    for (int i = 0; i < 2; ++i) l->key[i] = cut.take(a->tokens * 4);
    for (int i = 0; i < 2; ++i) l->at[i] = cut.take(a->tokens * 4);
    l->counts = cut.take((int64_t)a->blocks * kBins * 4);
    l->start = cut.take((a->rows + 1) * 4);
    l->part = cut.take(a->slices * 2 * a->dim * 4);
    l->bytes = cut.bytes;
}

int width(int64_t dim, int64_t v)
{
    int px = 1;
    while (px < kThreads && px * v < dim) px *= 2;
    return px;
}

// The sort; which of the two orders holds its result.
int sort(Embed a, hipStream_t st)
{
    int bits = 1;
    while ((a.rows >> bits) > 0) ++bits;
    const unsigned blocks = (unsigned)a.blocks;
    int from = 0;
    for (int done = 0, pass = 0; done < bits && blocks > 0; done += kBits, ++pass) {
        a.shift = done;
        const int to = pass & 1;
        if (pass == 0) {
            embed_count<true><<<blocks, kThreads, 0, st>>>(a, 0);
            embed_place<true><<<blocks, kThreads, 0, st>>>(a, 0, to);
        } else {
            embed_count<false><<<blocks, kThreads, 0, st>>>(a, from);
            embed_place<false><<<blocks, kThreads, 0, st>>>(a, from, to);
        }
        from = to;
    }
    embed_starts<<<(unsigned)((a.rows + kThreads) / kThreads), kThreads, 0, st>>>(a, from);
    return from;
}

template <typename T, bool RUNS>
void sums(const Embed& a, int from, hipStream_t st)
{
    const unsigned slices = (unsigned)((a.slices * a.stretches + kWaves - 1) / kWaves);
    const unsigned rows = (unsigned)(a.slices * a.stretches + std::min<int64_t>((a.row1 - a.row0 + kWaves - 1) / kWaves, 4096));
    auto go = [&](auto v, auto w) {
        constexpr int V = decltype(v)::value, W = decltype(w)::value;
        if (slices) embed_slices<T, V, W, RUNS><<<slices, kThreads, 0, st>>>(a, from);
        if constexpr (!RUNS && V > 1) {
            // A table that would push most else out of the 256 MB cache behind the L2s, and not stay there itself, is stored past
            // it (with an update that reads it after: of 205 MB 199 us past it, 205 through it; of 131 MB 146 and 136).
            if (a.rows * a.dim * (int64_t)sizeof(T) >= (int64_t)160 << 20) {
                embed_rows<T, V, W, RUNS, true><<<rows, kThreads, 0, st>>>(a, from);
                return;
            }
        }
        embed_rows<T, V, W, RUNS, false><<<rows, kThreads, 0, st>>>(a, from);
    };
    int v, w;
    pieces(sizeof(T) == 2, a.dim, &v, &w);
    constexpr std::integral_constant<int, 16 / sizeof(T)> most;
    if (v == 1) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
    else if (w == 1) go(most, std::integral_constant<int, 1>{});
    else go(most, std::integral_constant<int, 2>{});
}

int check_launch(const Embed& a)
{
    if (a.slices * a.stretches + 4096 > max_blocks(kThreads))
        return fail(GCONV_ERR_UNSUPPORTED, "too many ids");
    return GCONV_OK;
}

void place(const Layout& l, void* workspace, Embed* a)
{
    char* w = (char*)workspace;
    for (int i = 0; i < 2; ++i) {
        a->key[i] = (uint32_t*)(w + l.key[i]);
        a->at[i] = (uint32_t*)(w + l.at[i]);
    }
    a->counts = (uint32_t*)(w + l.counts);
    a->start = (uint32_t*)(w + l.start);
    a->part = (float*)(w + l.part);
}

gconv_embed_desc desc_of(const EmbedRuns& r)
{
    gconv_embed_desc d{};
    d.dtype = GCONV_BF16;
    d.index = r.wide ? GCONV_I64 : GCONV_I32;
    d.sequences = 1;
    d.tokens = r.tokens;
    d.rows = r.rows;
    d.dim = r.dim;
    d.dy_stride[1] = r.pitch;
    d.scale = 1.0;
    return d;
}

}  // namespace

size_t embed_runs_workspace(const EmbedRuns& r)
{
    const gconv_embed_desc d = desc_of(r);
    Embed a{};
    Layout l{};
    plan(&d, &a, &l);
    return l.bytes;
}

void embed_runs_sort(EmbedRuns* r, hipStream_t st)
{
    const gconv_embed_desc d = desc_of(*r);
    Embed a{};
    Layout l{};
    plan(&d, &a, &l);
    place(l, r->workspace, &a);
    a.ids = r->ids;
    r->order = sort(a, st);
    r->start = a.start;
}

void embed_runs_sum(const EmbedRuns& r, int64_t row0, int64_t row1, hipStream_t st)
{
    const gconv_embed_desc d = desc_of(r);
    Embed a{};
    Layout l{};
    plan(&d, &a, &l);
    place(l, r.workspace, &a);
    a.dy = r.src;
    a.weight = r.weight;
    a.runs = r.sums;
    a.row0 = row0;
    a.row1 = row1;
    sums<__bf16, true>(a, r.order, st);
}

}  // namespace gconv

using namespace gconv;

extern "C" {

int gconv_embed_workspace_size(const gconv_embed_desc* d, size_t* bytes)
{
    const int st = check_desc(d);
    if (st != GCONV_OK) return st;
    if (!bytes) return fail(GCONV_ERR_NULL, "bytes pointer is NULL");
    Embed a{};
    Layout l{};
    plan(d, &a, &l);
    *bytes = l.bytes;
    return GCONV_OK;
}

int gconv_embed_fwd(const gconv_embed_desc* d, const void* table, const void* ids, void* y, void* stream)
{
    int st = check_desc(d);
    if (st != GCONV_OK) return st;
    const int64_t tokens = d->sequences * d->tokens, es = d->dtype == GCONV_BF16 ? 2 : 4, is = d->index == GCONV_I64 ? 8 : 4;
    if (!table || (tokens > 0 && (!ids || !y))) return fail(GCONV_ERR_NULL, "table, ids and y must be non-NULL");
    const Span in[] = {{table, d->rows * d->dim * es}, {ids, tokens * is}};
    const Span out[] = {{y, tokens * d->dim * es}};
    st = check_overlap(in, out);
    if (st != GCONV_OK) return st;
    Embed a{};
    Layout l{};
    plan(d, &a, &l);
    a.table = table;
    a.ids = ids;
    a.y = y;
    int v, w;
    pieces(d->dtype == GCONV_BF16, d->dim, &v, &w);
    const int px = width(d->dim, v), per = kThreads / px;
    // four tokens a thread where that leaves every CU several workgroups (16384 tokens of 2048: 25.1 us by one, 23.4 by four)
    const int r = v > 1 && tokens / per >= 4 * 2048 ? 4 : 1;
    const int64_t blocks = (tokens + per * r - 1) / (per * r);
    if (blocks > max_blocks(kThreads)) return fail(GCONV_ERR_UNSUPPORTED, "too many ids");
    (void)hipGetLastError();
    if (blocks > 0) {
        auto go = [&](auto t, auto most) {
            using T = decltype(t);
            constexpr int V = decltype(most)::value;
            hipStream_t st = (hipStream_t)stream;
            if (v == 1) embed_fwd<T, 1, 1><<<(unsigned)blocks, kThreads, 0, st>>>(a, px);
            else if (r == 1) embed_fwd<T, V, 1><<<(unsigned)blocks, kThreads, 0, st>>>(a, px);
            else embed_fwd<T, V, 4><<<(unsigned)blocks, kThreads, 0, st>>>(a, px);
        };
        if (d->dtype == GCONV_BF16) go((__bf16)0.f, std::integral_constant<int, 8>{});
        else go(0.f, std::integral_constant<int, 4>{});
    }
    return finish();
}

int gconv_embed_bwd(const gconv_embed_desc* d, const void* dy, const void* ids, void* dtable, void* workspace, size_t workspace_bytes,
                    void* stream)
{
    int st = check_desc(d);
    if (st != GCONV_OK) return st;
    const int64_t tokens = d->sequences * d->tokens, es = d->dtype == GCONV_BF16 ? 2 : 4, is = d->index == GCONV_I64 ? 8 : 4;
    if (!dtable || (tokens > 0 && (!ids || !dy))) return fail(GCONV_ERR_NULL, "dy, ids and dtable must be non-NULL");
    const Span in[] = {strided_span(dy, es, d->sequences, d->dy_stride[0], d->tokens, d->dy_stride[1], 1, 0, d->dim), {ids, tokens * is}};
    const Span out[] = {{dtable, d->rows * d->dim * es}};
    st = check_overlap(in, out);
    if (st != GCONV_OK) return st;
    Embed a{};
    Layout l{};
    plan(d, &a, &l);
    st = check_workspace(workspace, workspace_bytes, l.bytes);
    if (st != GCONV_OK) return st;
    st = check_launch(a);
    if (st != GCONV_OK) return st;
    place(l, workspace, &a);
    a.dy = dy;
    a.ids = ids;
    a.dtable = dtable;
    (void)hipGetLastError();
    hipStream_t hs = (hipStream_t)stream;
    const int order = sort(a, hs);
    if (d->dtype == GCONV_BF16) sums<__bf16, false>(a, order, hs);
    else sums<float, false>(a, order, hs);
    return finish();
}

}  // extern "C"
