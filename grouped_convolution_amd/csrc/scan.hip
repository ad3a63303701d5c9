// scan.hip -- the selective state space scan: a recurrence whose decay and
// inputs depend on the token (gfx950).
//
//   dt_t = softplus(raw_t + dt_bias)           (or raw_t + dt_bias)
//   h_t  = exp(dt_t a) h_{t-1} + dt_t u_t b_t  for each channel and state
//   y_t  = (c_t . h_t + skip u_t) silu(gate_t)
//
// and backward, with dy' = dy silu(gate) and the adjoint state g:
//
//   g_t = c_t dy'_t + exp(dt_{t+1} a) g_{t+1}      m_t = exp(dt_t a) h_{t-1} g_t
//   dc_t = sum over channels of dy'_t h_t           db_t = sum over channels of dt_t u_t g_t
//   da = sum_t dt_t m_t         s_t = sum over states of b_t g_t
//   du_t = dt_t s_t + skip dy'_t         ddt_t = u_t s_t + sum over states of a m_t
//
// The decays differ for every (token, channel, state), so there is no product of
// matrices in it: what bounds it is the vector pipes, one exponential (a quarter
// of the rate) and four operations for each of them forward.
//
// A workgroup takes 64 channels, a lane each, and NW waves, each with two or four
// of the states in registers: b_t and c_t are then the same for a whole wave. They
// come from LDS, one read for all lanes (backward, where registers are short, from
// scalar memory as operands). What depends on (token, channel) alone (softplus,
// gate, sums over the waves) is done once for a tile of tokens by all threads and
// passed through LDS.
//
// Long sequences are cut into chunks: a first kernel runs each chunk from a zero
// state, a second carries the states over the chunks, and the last starts each
// chunk from its true state. The decay over a chunk is exp(a sum dt), so a chunk
// passes on one number a channel for it. Backward, the same first kernel also
// makes what the chunk adds to the adjoint before it, sum_t (decay from the
// chunk's start to t) c_t dy'_t, running forward, and leaves the state before every
// eighth token: the last kernel walks back over the chunk in tiles of eight, each
// run forward from there first.
//
// Tokens carry marks (first or last of a sequence, or of none), made beforehand
// with b and c in float32, four states side by side.
//
// Measured (bf16, 16 states, under the profiler): forward of 4 x 2048 tokens of
// 4096 channels 275 us; of one sequence of 32768 tokens of 2048 channels, in chunks,
// 256 + 346 (508 in all without the profiler), the vector pipes 91% busy; backward
// of 4 x 2048 of 4096 850, 601 of them in the last kernel (84% busy); without the
// profiler 750, and both ways 993. A token of 256 sequences of 4096: 34 us, 4.2 TB/s
// of states.
#include "device_util.h"
#include "seq_host.h"
#include "seq_tokens.h"

namespace gconv {
namespace {

constexpr int kLanes = 64;   // channels of a workgroup
constexpr int kSpw = 4;      // states that lie together in memory
constexpr int kTile = 16;    // tokens passed through LDS at once
constexpr int kBack = 8;     // the same, of the backward pass
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

enum { FIRST = 1, LAST = 2 };  // marks of a token; the sequence's number is above them, a token of none is -1

struct Scan {
    const void *u, *dt, *b, *c, *gate, *dy;
    const float *a, *skip, *dt_bias, *init, *dfinal;
    void *y, *du, *ddt, *dgate;
    float *final_, *dinit;
    Sequences seq;
    int64_t u_s[2], dt_s[2], gate_s[2], dy_s[2], b_s[3], c_s[3];
    float* bc;          // [groups][NW][places][8]: four of b, four of c
    int32_t* mark;      // [places]
    float* ends;        // [chunks][blocks][NW][4][64]: states; later those before each chunk
    float* adds;        // the same of the adjoint; later that after each chunk
    float* sums;        // [chunks][blocks][64]: sum of dt
    int32_t* breaks;    // [chunks]: whether a sequence begins in it
    float* hist;        // backward, [places / kBack][blocks][NW][4][64]: states before every kBack tokens, from 0 before the chunk
    float* hist_sum;    // [places / kBack][blocks][64]: sum of dt since the chunk's start; not a number where a sequence has begun since
    float* part_a;      // [chunks][blocks][NW][4][64]: of da
    float* part_d;      // [chunks][2][dim]: of dskip and ddt_bias
    float* part_bc;     // [blocks of a group][groups][NW][places][8]: of db and dc
    int64_t rows;       // tokens of all sequences
    int64_t pad, places;  // of a stretch and of all: its tokens up to a whole tile, those past its end like tokens of none
    int64_t per, chunks;  // chunks of a stretch (a sequence, or all packed tokens), of all
    int chunk;          // tokens
    int dim, states, groups;
    int gdim, gblocks;  // channels of a group, workgroups along them
    int blocks;         // groups * gblocks
    int softplus;
};

// What a workgroup works at.
struct Where {
    int g, gb, block;      // group, workgroup along its channels, workgroup along all
    int c0, left;          // first channel, channels
    int64_t chunk, outer;
    int64_t t0;            // first token, in its stretch
    int n;                 // tokens
    int64_t row0;          // first token, of all
    int64_t place0;        // its place in the workspace
};

__device__ __forceinline__ Where where(const Scan& a)
{
    Where w;
    w.block = (int)(blockIdx.x % (unsigned)a.blocks);
    w.chunk = blockIdx.x / (unsigned)a.blocks;
    w.g = w.block / a.gblocks;
    w.gb = w.block - w.g * a.gblocks;
    w.c0 = w.g * a.gdim + w.gb * kLanes;
    w.left = min(kLanes, a.gdim - w.gb * kLanes);
    w.outer = w.chunk / a.per;
    w.t0 = (w.chunk - w.outer * a.per) * a.chunk;
    w.n = (int)min((int64_t)a.chunk, a.seq.tokens - w.t0);
    w.row0 = w.outer * a.seq.tokens + w.t0;
    w.place0 = w.outer * a.pad + w.t0;
    return w;
}

// softplus(x) = max(x, 0) + log(1 + w), w = exp(-|x|): the logarithm of 1 + w as
// it was rounded, and what the rounding left of w (at most 2^-24, where w is near
// 1 and half as much would be right; exact where w is small), so no less exact
// relative to it than w is: off by some |x| half steps, from the rounding of the
// exponential's argument.
__device__ __forceinline__ float softplus_of(float x)
{
    const float w = __builtin_amdgcn_exp2f(fabsf(x) * -kLog2e), v = 1.f + w;
    return fmaxf(x, 0.f) + fmaf(__builtin_amdgcn_logf(v), kLn2, w - (v - 1.f));
}

// V elements of a row as they were loaded. As whole words, not elements: where the
// ways to load them meet, elements would be taken apart, which waits for the load.
template <typename T, int V>
struct Bits {
    static constexpr int N = (V * (int)sizeof(T) + 3) / 4;
    struct __attribute__((packed, aligned(sizeof(T)))) Words {
        uint32_t w[N];
    };
    uint32_t w[N];
    __device__ __forceinline__ float get(int e) const
    {
        if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, w[e]);
        const uint32_t v = w[e / 2];
        return __builtin_bit_cast(float, e & 1 ? v & 0xffff0000u : v << 16);
    }
    // from `row`; unless all of it is there (the same for a workgroup), `have` elements, the others 0
    __device__ __forceinline__ void load(const T* row, bool whole, int have)
    {
        if constexpr (V * sizeof(T) < 4) {
            w[0] = 0;
            if (have > 0) w[0] = *(const uint16_t*)row;
        } else if (whole) {
            const Words v = *(const Words*)row;
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = v.w[i];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = 0;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < have) {
                    if constexpr (sizeof(T) == 4) w[e] = *(const uint32_t*)(row + e);
                    else w[e / 2] |= (uint32_t) * (const uint16_t*)(row + e) << (e & 1 ? 16 : 0);
                }
        }
    }
};

// ---- marks, b and c -------------------------------------------------------------

// A thread: the marks of a token and four states of one group.
template <typename T>
__global__ __launch_bounds__(256) void scan_prep(Scan a, int nw)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t k = id / a.places, place = id - k * a.places;
    const int g = (int)k / nw, w = (int)k - g * nw;
    if (g >= a.groups) return;
    const int64_t outer = place / a.pad, t = place - outer * a.pad;
    int n = (int)outer, mark = 0;
    if (t >= a.seq.tokens) {
        n = -1;
    } else if (!a.seq.cu) {
        mark = (t == 0 ? FIRST : 0) | (t == a.seq.tokens - 1 ? LAST : 0);
    } else {
        n = a.seq.find(t);
        if (n < 0 || n >= a.seq.count) n = -1;
        else mark = (t == a.seq.bound(n) ? FIRST : 0) | (t == a.seq.bound(n + 1) - 1 ? LAST : 0);
    }
    if (k == 0) a.mark[place] = n < 0 ? -1 : n * 4 + mark;
    f4 b = {0, 0, 0, 0}, c = {0, 0, 0, 0};
    if (n >= 0) {
        const T* pb = (const T*)a.b + outer * a.b_s[0] + t * a.b_s[1] + g * a.b_s[2];
        const T* pc = (const T*)a.c + outer * a.c_s[0] + t * a.c_s[1] + g * a.c_s[2];
#pragma unroll
        for (int s = 0; s < kSpw; ++s) {
            if (w * kSpw + s >= a.states) break;
            b[s] = (float)pb[w * kSpw + s];
            c[s] = (float)pc[w * kSpw + s];
        }
    }
    f4* o = (f4*)(a.bc + id * 8);
    o[0] = b;
    o[1] = c;
}

// Sequences without tokens: the state after them is the one before, and the
// gradients likewise.
__global__ __launch_bounds__(256) void scan_empty(Sequences seq, const float* from, float* to, int64_t size)
{
    for (int64_t n = blockIdx.x; n < seq.count; n += gridDim.x) {
        if (seq.cu ? seq.bound((int)n + 1) > seq.bound((int)n) : seq.tokens > 0) continue;
        for (int64_t i = blockIdx.y * 256 + threadIdx.x; i < size; i += gridDim.y * 256) to[n * size + i] = from ? from[n * size + i] : 0.f;
    }
}

// ---- parts that the kernels share -------------------------------------------------

// Rates up to this one, whose product with log2(e) leaves float32's range or comes near its end, count as -infinity.
constexpr float kNoMemory = -2e38f;

// a, with kNoMemory in place of what counts as -infinity: it leaves as little of a state (of steps above 1e-36), but a
// step of 0 (of a token of no sequence, say) leaves all of it, where 0 times infinity is not a number.
__device__ __forceinline__ float rate_of(float a) { return a < kNoMemory ? kNoMemory : a; }

// a as a factor of the step's gradient: 0 for what counts as -infinity, whose decay is 0 or 1 and has none (kNoMemory in
// its place would take the gradient of a step of 0, where the decay is 1, out of float32's range, and softplus's slope
// of 0 with it).
__device__ __forceinline__ float rate_factor(float a) { return a <= kNoMemory ? 0.f : a; }

// Read-only while the kernel runs, at an address that is the same for a wave: scalar loads.
typedef const __attribute__((address_space(4))) float* scalar_floats;

// Asks for TOKENS tokens' b and c of a wave, a line of the scalar cache each 64
// bytes, well before they are used: from memory they take longer than a few
// tokens' work. settle() is where they have to be there.
template <int TOKENS>
struct Ahead {
    float line[TOKENS / 2];
    __device__ __forceinline__ void ask(scalar_floats p)
    {
#pragma unroll
        for (int i = 0; i < TOKENS / 2; ++i) line[i] = p[i * 16];
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void settle() const
    {
#pragma unroll
        for (int i = 0; i < TOKENS / 2; ++i) asm volatile("" ::"s"(line[i]));
    }
};

// The kernel's arguments, read again: what only tokens with marks ask for does not
// stay in scalar registers, of which the rest of the kernel has need.
__device__ __forceinline__ const __attribute__((address_space(4))) Scan* again()
{
    auto p = (const __attribute__((address_space(4))) Scan*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return p;
}

// The states of lane's channel that its wave holds.
template <int SPW>
struct Mine {
    typedef float fs __attribute__((ext_vector_type(SPW)));
    int lane, wave;
    int ch;         // channel, clamped to one that exists
    bool live;
    int at;         // element of [dim][states]
    int have;       // states that exist, of SPW
    __device__ __forceinline__ static Mine of(const Scan& a, const Where& w)
    {
        Mine m;
        m.lane = threadIdx.x & 63;
        m.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        m.live = m.lane < w.left;
        m.ch = w.c0 + (m.live ? m.lane : 0);
        m.at = m.ch * a.states + m.wave * SPW;
        m.have = m.live ? max(0, min(SPW, a.states - m.wave * SPW)) : 0;
        return m;
    }
    // p[n][dim][states] of sequence n, or 0: no branches, a state that does not
    // exist is read (and written) past the resource's end
    __device__ __forceinline__ uint32_t offset(int s) const { return s < have ? (uint32_t)(at + s) * 4 : kOOB; }
    __device__ __forceinline__ fs get(int dim, int states, const float* p, int64_t n) const
    {
        const int64_t size = (int64_t)dim * states;
        const __amdgpu_buffer_rsrc_t r = make_rsrc(p + (p ? n * size : 0), p ? (uint32_t)size * 4 : 0);
        fs v;
#pragma unroll
        for (int s = 0; s < SPW; ++s) v[s] = load_f32(r, offset(s));
        return v;
    }
    __device__ __forceinline__ fs rates(const Scan& a) const
    {
        fs v = get(a.dim, a.states, a.a, 0);
#pragma unroll
        for (int s = 0; s < SPW; ++s) v[s] = rate_of(v[s]);
        return v;
    }
    __device__ __forceinline__ void put(int dim, int states, float* p, int64_t n, fs v) const
    {
        const int64_t size = (int64_t)dim * states;
        const __amdgpu_buffer_rsrc_t r = make_rsrc(p + (p ? n * size : 0), p ? (uint32_t)size * 4 : 0);
#pragma unroll
        for (int s = 0; s < SPW; ++s) store_f32(r, offset(s), v[s]);
    }
    // element of [groups][fours][places][8] where its states are, before the place
    __device__ __forceinline__ int64_t four(const Scan& a, int g, int fours) const { return (int64_t)(g * fours + wave * SPW / 4) * a.places; }
    // ... and within the eight
    __device__ __forceinline__ int within() const { return wave * SPW % 4; }
    // index into `ends` and its like, of state s
    __device__ __forceinline__ int64_t slot(const Scan& a, int64_t chunk, int block, int nw, int s) const
    {
        return ((((chunk * a.blocks + block) * nw + wave) * SPW + s) * kLanes) + lane;
    }
};

// A workgroup's pieces of a tile of tokens, V channels each: as many as make one a
// thread, so that all waves share what is done for (token, channel) alone.
template <int NW, int TILE>
struct Pieces {
    static constexpr int V = TILE / NW < 1 ? 1 : TILE / NW > 4 ? 4 : TILE / NW;
    static constexpr int kRow = kLanes / V, kThreads = NW * 64, kPer = TILE * kRow / kThreads;
    static_assert(TILE * kRow % kThreads == 0, "whole rounds");
    typedef float fv __attribute__((ext_vector_type(V)));
    static __device__ __forceinline__ int of(int i) { return i * kThreads + (int)threadIdx.x; }
};

template <typename T, int V>
__device__ __forceinline__ void load_at(Bits<T, V>& to, const void* p, const int64_t* stride, const Where& w, int64_t t, int col)
{
    const T* row = (const T*)p + w.outer * stride[0] + t * stride[1] + w.c0;
    to.load(row + col, w.left == kLanes, w.left - col);
}

template <typename T, int V>
__device__ __forceinline__ void store_at(const Where& w, T* row, int col, const float (&v)[V])
{
    if (w.left != kLanes) {
        store_piece<T, V>(row, col, w.left, v);
        return;
    }
    Packed<T, V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) o.e[e] = (T)v[e];
    *(Packed<T, V>*)(row + col) = o;
}

// dt and dt u of a piece; 0 for a token of no sequence.
template <typename T, int V, typename F>
__device__ __forceinline__ void step_sizes(const Scan& a, const F& bias, const Bits<T, V>& raw, const Bits<T, V>& u, bool real, F* dt, F* dtu)
{
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float v = raw.get(e) + bias[e];
        if (a.softplus) v = softplus_of(v);
        (*dt)[e] = real ? v : 0.f;
        (*dtu)[e] = real ? v * u.get(e) : 0.f;
    }
}

template <typename F, int V>
__device__ __forceinline__ F of_channels(const float* p, const Where& w, int col)
{
    F v = {};
    if (p) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (col + e < w.left) v[e] = p[w.c0 + col + e];
    }
    return v;
}

// (arguments so large that the exponential leaves float32's range give 0 or 1)
__device__ __forceinline__ float sigm(float z) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -kLog2e)); }
__device__ __forceinline__ float silu_of(float z) { return z * sigm(z); }

// dy' of a piece; 0 for a token of no sequence.
template <typename F, typename T, int V>
__device__ __forceinline__ F gated(const Scan& a, const Bits<T, V>& dy, const Bits<T, V>& gate, bool real)
{
    F v;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        v[e] = dy.get(e);
        if (a.gate) v[e] *= silu_of(gate.get(e));
        v[e] = real ? v[e] : 0.f;
    }
    return v;
}

// ---- forward ----------------------------------------------------------------------

// OUT: the outputs, from the state before each chunk; else each chunk's own
// contribution to the state after it (and, ADJ, to the adjoint before it).
template <typename T, int NW, int SPW, bool OUT, bool ADJ>
__global__ __launch_bounds__(NW * 64) void scan_run(Scan a)
{
    using Q = Pieces<NW, kTile>;
    constexpr int V = Q::V;
    typedef typename Q::fv fv;
    constexpr int kW = ADJ ? 3 : 2;
    __shared__ float sd[2][kTile][kW][kLanes];            // dt, dt u (, dy')
    __shared__ f4 sbc[2][NW * SPW / 4][kTile][2];          // b and c of the tile
    __shared__ float yp[OUT ? 2 : 1][OUT ? NW : 1][OUT ? kTile : 1][kLanes];
    const Where w = where(a);
    const Mine<SPW> m = Mine<SPW>::of(a, w);
    typedef typename Mine<SPW>::fs fs;
    const int col = threadIdx.x % Q::kRow * V;
    const fv bias = of_channels<fv, V>(a.dt_bias, w, col), skip = of_channels<fv, V>(a.skip, w, col);

    const fs a2 = m.rates(a) * kLog2e;
    // What the chunk adds to the adjoint before it is `r` as it is when a sequence begins: no later token can reach that
    // adjoint, and one that is not finite would, as 0 times it. (Kept aside rather than not computed further: loops for
    // chunks in which none has begun and others cost 1 to 2% of the whole backward pass, this nothing.)
    fs h = {}, p = {}, r = {}, reached = {};
    p += 1.f;
    float total = 0.f;
    int broken = 0;
    if (OUT && a.per > 1) {
#pragma unroll
        for (int s = 0; s < SPW; ++s) h[s] = a.ends[m.slot(a, w.chunk, w.block, NW, s)];
    }
    struct Raw {
        Bits<T, V> u, dt, z, dy;
        int mark;
    } raw[Q::kPer];
    Bits<T, V> cur_u[Q::kPer], cur_z[Q::kPer], old_u[Q::kPer], old_z[Q::kPer];  // of this tile and the one before
    int cur_mark[Q::kPer], old_mark[Q::kPer];
    // marks of a tile, a token a lane: asked for a tile ahead, as loads come back in order
    auto mark_of = [&](int tile) { return a.mark[w.place0 + tile * kTile + (m.lane & (kTile - 1))]; };
    int mk = mark_of(0), mk_next = -1;
    constexpr int kFours = NW * SPW / 4;
    f4 raw_bc;
    const bool brings = (int)threadIdx.x < kFours * kTile * 2;  // 16 bytes of b or c a tile
    const float* bc = a.bc + (((int64_t)w.g * kFours + threadIdx.x / (kTile * 2)) * a.places + w.place0) * 8 + threadIdx.x % (kTile * 2) * 4;
    auto fetch = [&](int tile) {
        if (brings) raw_bc = *(const f4*)(bc + tile * kTile * 8);
#pragma unroll
        for (int i = 0; i < Q::kPer; ++i) {
            const int q = Q::of(i), in = q / Q::kRow, tok = min(tile * kTile + in, w.n - 1);
            raw[i].mark = a.mark[w.place0 + tile * kTile + in];
            load_at<T, V>(raw[i].u, a.u, a.u_s, w, w.t0 + tok, col);
            load_at<T, V>(raw[i].dt, a.dt, a.dt_s, w, w.t0 + tok, col);
            if ((OUT || ADJ) && a.gate) load_at<T, V>(raw[i].z, a.gate, a.gate_s, w, w.t0 + tok, col);
            if (ADJ) load_at<T, V>(raw[i].dy, a.dy, a.dy_s, w, w.t0 + tok, col);
        }
    };
    auto stage = [&](int tile) {  // of what was fetched
        if (brings) (&sbc[tile & 1][0][0][0])[threadIdx.x] = raw_bc;
#pragma unroll
        for (int i = 0; i < Q::kPer; ++i) {
            const bool real = raw[i].mark >= 0;
            fv dt, dtu;
            step_sizes<T, V>(a, bias, raw[i].dt, raw[i].u, real, &dt, &dtu);
            float(*row)[kLanes] = sd[tile & 1][Q::of(i) / Q::kRow];
            *(fv*)&row[0][col] = dt;
            *(fv*)&row[1][col] = dtu;
            if constexpr (ADJ) *(fv*)&row[kW - 1][col] = gated<fv, T, V>(a, raw[i].dy, raw[i].z, real);
            if (OUT) {
                old_u[i] = cur_u[i];
                old_z[i] = cur_z[i];
                old_mark[i] = cur_mark[i];
                cur_u[i] = raw[i].u;
                cur_z[i] = raw[i].z;
                cur_mark[i] = raw[i].mark;
            }
        }
    };
    const int tiles = (w.n + kTile - 1) / kTile;
    fetch(0);
    stage(0);
    __syncthreads();
    // One barrier a tile: while the waves run over a tile, its outputs go to one
    // buffer, those of the tile before are read from the other, and the next
    // tile's inputs are put beside this one's.
    for (int tile = 0; tile < tiles + (OUT ? 1 : 0); ++tile) {
        if (tile + 1 < tiles) {
            mk_next = mark_of(tile + 1);
            fetch(tile + 1);
        }
        if (tile < tiles) {
            const uint32_t firsts = (uint32_t)__ballot(mk >= 0 && (mk & FIRST)) & ((1u << kTile) - 1);
            const uint32_t lasts = (uint32_t)__ballot(mk >= 0 && (mk & LAST)) & ((1u << kTile) - 1);
            auto token = [&](int i, auto marked) {
                if (ADJ && i % kBack == 0) {
                    const int64_t at = ((w.place0 + tile * kTile + i) / kBack * a.blocks + w.block);
#pragma unroll
                    for (int s = 0; s < SPW; ++s) a.hist[((at * NW + m.wave) * SPW + s) * kLanes + m.lane] = h[s];
                    if (m.wave == 0) a.hist_sum[at * kLanes + m.lane] = broken ? __builtin_nanf("") : total;
                }
                if (decltype(marked)::value && (firsts >> i & 1)) {
                    h = m.get(again()->dim, again()->states, again()->init, __builtin_amdgcn_readlane(mk, i) >> 2);
                    if (ADJ && !broken) reached = r;
                    broken = 1;
                }
                const float dt = sd[tile & 1][i][0][m.lane], dtu = sd[tile & 1][i][1][m.lane];
                const float* o = (const float*)&sbc[tile & 1][m.wave * SPW / 4][i][0] + m.within();
                const fs ob = *(const fs*)o, oc = *(const fs*)(o + 4);
                float y = 0.f, dy = 0.f;
                if (ADJ) dy = sd[tile & 1][i][kW - 1][m.lane];
                if (!OUT) total += dt;
#pragma unroll
                for (int s = 0; s < SPW; ++s) {
                    const float e = __builtin_amdgcn_exp2f(dt * a2[s]);
                    h[s] = fmaf(e, h[s], dtu * ob[s]);
                    if (OUT) y = fmaf(oc[s], h[s], y);
                    if (ADJ) {
                        p[s] *= e;
                        r[s] = fmaf(p[s], oc[s] * dy, r[s]);
                    }
                }
                if (OUT) yp[tile & 1][OUT ? m.wave : 0][OUT ? i : 0][m.lane] = y;
                if (decltype(marked)::value && (lasts >> i & 1)) {
                    const int n = __builtin_amdgcn_readlane(mk, i) >> 2;
                    if (OUT && again()->final_) m.put(again()->dim, again()->states, again()->final_, n, h);
                    if (ADJ && again()->dfinal) r += p * m.get(again()->dim, again()->states, again()->dfinal, n);
                    h = fs{};
                }
            };
            // (without marks the tokens are one stretch of code, whose loads are all under way early)
            if ((firsts | lasts) == 0) {
#pragma unroll
                for (int i = 0; i < kTile; ++i) token(i, std::false_type{});
            } else {
#pragma unroll 1
                for (int i = 0; i < kTile; ++i) token(i, std::true_type{});
            }
        }
        if (OUT && tile > 0) {
            const bool last = tile == tiles;  // nothing has been staged since
#pragma unroll
            for (int i = 0; i < Q::kPer; ++i) {
                const int in = Q::of(i) / Q::kRow, tok = (tile - 1) * kTile + in;
                if (tok >= w.n) continue;
                const Bits<T, V> u = last ? cur_u[i] : old_u[i];
                fv v = {};
#pragma unroll
                for (int k = 0; k < NW; ++k) v += *(const fv*)&yp[OUT ? (tile - 1) & 1 : 0][OUT ? k : 0][OUT ? in : 0][col];
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] = fmaf(skip[e], u.get(e), v[e]);
                if (a.gate) {
                    const Bits<T, V> z = last ? cur_z[i] : old_z[i];
#pragma unroll
                    for (int e = 0; e < V; ++e) v[e] *= silu_of(z.get(e));
                }
                const bool real = (last ? cur_mark[i] : old_mark[i]) >= 0;
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = real ? v[e] : 0.f;
                store_at<T, V>(w, (T*)a.y + (w.row0 + tok) * a.dim + w.c0, col, o);
            }
        }
        if (tile + 1 < tiles) {
            stage(tile + 1);
        }
        mk = mk_next;
        __syncthreads();
    }
    if (!OUT) {
#pragma unroll
        for (int s = 0; s < SPW; ++s) {
            a.ends[m.slot(a, w.chunk, w.block, NW, s)] = h[s];
            if (ADJ) a.adds[m.slot(a, w.chunk, w.block, NW, s)] = broken ? reached[s] : r[s];
        }
        if (m.wave == 0) a.sums[(w.chunk * a.blocks + w.block) * kLanes + m.lane] = total;
        if (w.block == 0 && threadIdx.x == 0) a.breaks[w.chunk] = broken;
    }
}

// Carries states over the chunks of a stretch: what `ends` holds becomes the
// state before each chunk, and (backward) what `adds` holds the adjoint after it.
// A thread: one state of one channel. Where a sequence begins in a chunk, nothing
// from before it comes through.
__global__ __launch_bounds__(256) void scan_carry(Scan a, int nw, int64_t outers)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, size = (int64_t)a.blocks * nw * kSpw * kLanes;
    const int64_t outer = id / size, at = id - outer * size;
    if (outer >= outers) return;
    const int lane = (int)(at % kLanes), state = (int)(at / kLanes % (nw * kSpw)), block = (int)(at / kLanes / (nw * kSpw));
    const int g = block / a.gblocks, in = (block - g * a.gblocks) * kLanes + lane;
    const bool have = in < a.gdim && state < a.states;
    const float a2 = have ? rate_of(a.a[(int64_t)(g * a.gdim + in) * a.states + state]) * kLog2e : 0.f;
    const int64_t c0 = outer * a.per;
    const float* sums = a.sums + block * kLanes + lane;
    const bool back = blockIdx.y != 0;
    float* v = (back ? a.adds : a.ends) + at;
    constexpr int U = 8;
    float h = 0.f;
    for (int64_t c = 0; c < a.per; c += U) {
        float e[U], s[U];
        int b[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t k = min(c + i, a.per - 1), n = c0 + (back ? a.per - 1 - k : k);
            e[i] = v[n * size];
            s[i] = sums[n * a.blocks * kLanes];
            b[i] = a.breaks[n];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (c + i >= a.per) break;
            const int64_t k = c + i, n = c0 + (back ? a.per - 1 - k : k);
            v[n * size] = h;
            h = b[i] ? e[i] : fmaf(__builtin_amdgcn_exp2f(s[i] * a2), h, e[i]);
        }
    }
}

// ---- backward ---------------------------------------------------------------------

// Sums over lanes, in which registers that hold different sums meet: after each
// step half as many registers hold them, each sum in half as many lanes. 64 sums
// over 64 lanes take some 2 operations each, where each alone would take 6.
template <int CTRL>
__device__ __forceinline__ float moved(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Lanes 0 to 31 get a's sum over lanes l and l + 32, the others b's.
__device__ __forceinline__ float meet32(float a, float b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t x = r[0], y = r[1];  // (a bit_cast of an element itself takes the first one's bits)
    return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}

// Of each 32 lanes the first 16 get a's sum over lanes l and l + 16, the others b's.
__device__ __forceinline__ float meet16(float a, float b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t x = r[0], y = r[1];  // (a bit_cast of an element itself takes the first one's bits)
    return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}

// Of each 16 (then 8) lanes the first half get a's sum over lanes l and 15 - l (7 - l), the others b's.
__device__ __forceinline__ float meet8(float a, float b, int lane)
{
    const float x = a + moved<0x140>(a), y = b + moved<0x140>(b);
    return lane & 8 ? y : x;
}

__device__ __forceinline__ float meet4(float a, float b, int lane)
{
    const float x = a + moved<0x141>(a), y = b + moved<0x141>(b);
    return lane & 4 ? y : x;
}

// The sum over four lanes, in each of them.
__device__ __forceinline__ float quad_sum(float v)
{
    v += moved<0xb1>(v);
    return v + moved<0x4e>(v);
}

// One token's four states' values over 64 channels, in sixteens: row r of 16 lanes
// has state 0, 2, 1, 3.
__device__ __forceinline__ float join_states(const float (&v)[4]) { return meet16(meet32(v[0], v[1]), meet32(v[2], v[3])); }
// ... two states': the halves of the wave have one each.
__device__ __forceinline__ float join_states(const float (&v)[2]) { return meet32(v[0], v[1]); }

// Four tokens of those: lane l has token (l >> 3 & 1) + 2 (l >> 2 & 1).
__device__ __forceinline__ float join_tokens(const float* v, int lane)
{
    return quad_sum(meet4(meet8(v[0], v[1], lane), meet8(v[2], v[3], lane), lane));
}

// Eight tokens of two states: lane l has token (l >> 4 & 1) + 2 (l >> 3 & 1) + 4 (l >> 2 & 1).
__device__ __forceinline__ float join_pairs(const float* v, int lane)
{
    const float x = meet8(meet16(v[0], v[1]), meet16(v[2], v[3]), lane), y = meet8(meet16(v[4], v[5]), meet16(v[6], v[7]), lane);
    return quad_sum(meet4(x, y, lane));
}

// A chunk's gradients, tile by tile from the last: forward over its tokens, with
// their states and decays in registers, and back over them.
//
// (The sums over channels, dc and db, by products with a matrix of ones held the
// waves up: a float32 product takes the matrix pipe 32 cycles for 64 values.)
template <typename T, int NW, int SPW>
__global__ __launch_bounds__(NW * 64, SPW == 2 ? 4 : 1) void scan_back(Scan a)
{
    constexpr int kThreads = NW * 64;
    // A thread's pieces of a tile: V channels of a token.
    constexpr int V = NW <= 2 ? 4 : NW == 4 ? 2 : 1, kRow = kLanes / V, kPieces = kBack * kRow;
    constexpr int kPer = (kPieces + kThreads - 1) / kThreads;
    __shared__ float sd[kBack][3][kLanes];            // dt, dt u, dy'
    __shared__ float part[3][NW][kBack][kLanes];      // of s, the sum of a m, and y
    typedef float fv __attribute__((ext_vector_type(V)));
    typedef typename Mine<SPW>::fs fs;
    const Where w = where(a);
    const Mine<SPW> m = Mine<SPW>::of(a, w);
    const int col = (threadIdx.x % kRow) * V;          // channel of the workgroup's
    const int in0 = threadIdx.x / kRow;                // token of the tile, of the thread's first piece
    const bool works = (int)threadIdx.x < kPieces, whole = w.left == kLanes;
    fv bias, skip, s_skip, s_bias;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const bool in = col + e < w.left;
        bias[e] = in && a.dt_bias ? a.dt_bias[w.c0 + col + e] : 0.f;
        skip[e] = in && a.skip ? a.skip[w.c0 + col + e] : 0.f;
        s_skip[e] = s_bias[e] = 0.f;
    }
    const fs rate = m.get(a.dim, a.states, a.a, 0);
    fs av, a2;
#pragma unroll
    for (int s = 0; s < SPW; ++s) {
        av[s] = rate_factor(rate[s]);
        a2[s] = rate_of(rate[s]) * kLog2e;
    }
    fs before0 = {}, g = {}, da = {};  // the state before the chunk; the adjoint after it
    if (a.per > 1) {
#pragma unroll
        for (int s = 0; s < SPW; ++s) {
            before0[s] = a.ends[m.slot(a, w.chunk, w.block, NW, s)];
            g[s] = a.adds[m.slot(a, w.chunk, w.block, NW, s)];
        }
    }
    struct Raw {
        Bits<T, V> u, dt, z, dy;
        int mark;
    };
    Raw raw[kPer], next[kPer];
    // Rows of the thread's first piece; the workgroup's are as far on for every tile.
    auto first = [&](const void* p, const int64_t* stride) {
        return (const T*)p + w.outer * stride[0] + (w.t0 + in0) * stride[1] + w.c0 + col;
    };
    const T *pu = first(a.u, a.u_s), *pdt = first(a.dt, a.dt_s), *pz = a.gate ? first(a.gate, a.gate_s) : nullptr, *pdy = first(a.dy, a.dy_s);
    auto load = [&](Bits<T, V>& to, const T* p, int64_t step, int tok) { to.load(p + (tok - in0) * step, whole, w.left - col); };
    auto fetch = [&](Raw (&to)[kPer], int tile) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int in = in0 + i * (kThreads / kRow), tok = tile * kBack + in;
            to[i].mark = -1;
            if (!works || tok >= w.n) continue;
            const auto* k = again();
            to[i].mark = k->mark[w.place0 + tok];
            load(to[i].u, pu, k->u_s[1], tok);
            load(to[i].dt, pdt, k->dt_s[1], tok);
            if (k->gate) load(to[i].z, pz, k->gate_s[1], tok);
            load(to[i].dy, pdy, k->dy_s[1], tok);
        }
    };
    auto stage = [&]() {
        if (!works) return;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const bool real = raw[i].mark >= 0;
            float(*row)[kLanes] = sd[in0 + i * (kThreads / kRow)];
            fv dt, dtu, dy;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float v = raw[i].dt.get(e) + bias[e];
                if (a.softplus) v = softplus_of(v);
                dt[e] = real ? v : 0.f;
                dtu[e] = real ? v * raw[i].u.get(e) : 0.f;
                float y = raw[i].dy.get(e);
                if (a.gate) y *= silu_of(raw[i].z.get(e));
                dy[e] = real ? y : 0.f;
            }
            *(fv*)&row[0][col] = dt;
            *(fv*)&row[1][col] = dtu;
            *(fv*)&row[2][col] = dy;
        }
    };
    const int tiles = (w.n + kBack - 1) / kBack;
    const scalar_floats bc = (scalar_floats)(a.bc + (m.four(a, w.g, NW * SPW / 4) + w.place0) * 8 + m.within());
    float* out_bc = a.part_bc + (m.four(a, w.gb * a.groups + w.g, NW * SPW / 4) + w.place0) * 8 + m.within();

    // lane's place in a tile's [8 tokens][db, dc][4 states]
    const int out_at = SPW == 4 ? ((m.lane >> 3 & 1) + 2 * (m.lane >> 2 & 1) + (m.lane & 2 ? 4 : 0)) * 8 + (m.lane & 1) * 4 + (m.lane >> 5) +
                                      2 * (m.lane >> 4 & 1)
                                : ((m.lane >> 4 & 1) + 2 * (m.lane >> 3 & 1) + 4 * (m.lane >> 2 & 1)) * 8 + (m.lane & 1) * 4 + (m.lane >> 5);
    // marks of a tile, a token a lane: asked for a tile ahead, as loads come back in order
    auto mark_of = [&](int tile) { return a.mark[w.place0 + tile * kBack + (m.lane & (kBack - 1))]; };
    int mk = mark_of(tiles - 1), mk_next = -1;
    uint32_t firsts = 0, lasts = 0;
    auto marks = [&]() {
        firsts = (uint32_t)__ballot(mk >= 0 && (mk & FIRST)) & ((1u << kBack) - 1);
        lasts = (uint32_t)__ballot(mk >= 0 && (mk & LAST)) & ((1u << kBack) - 1);
    };
    // The state before a tile: its chunk's own part, and what is left of the state before the chunk.
    fs own, own_next;
    float since, since_next;
    auto history = [&](int tile, fs& v, float& sum) {
        const int64_t at = (w.place0 / kBack + tile) * a.blocks + w.block;
#pragma unroll
        for (int s = 0; s < SPW; ++s) v[s] = a.hist[((at * NW + m.wave) * SPW + s) * kLanes + m.lane];
        sum = a.hist_sum[at * kLanes + m.lane];
    };
    Ahead<kBack> ahead;
    fetch(raw, tiles - 1);
    history(tiles - 1, own, since);
    ahead.ask(bc + (tiles - 1) * kBack * 8);
    ahead.settle();
    for (int tile = tiles - 1; tile >= 0; --tile) {
        stage();
        __syncthreads();
        marks();
        if (tile > 0) {
            mk_next = mark_of(tile - 1);
            fetch(next, tile - 1);
            history(tile - 1, own_next, since_next);
            ahead.ask(bc + (tile - 1) * kBack * 8);
        }
        fs h = own;
        if (since == since) {  // (no sequence has begun since the chunk's start)
#pragma unroll
            for (int s = 0; s < SPW; ++s) h[s] = fmaf(__builtin_amdgcn_exp2f(since * a2[s]), before0[s], own[s]);
        }
        float sum_c[kBack], sum_b[kBack];
        auto tokens = [&](auto marked) {
            fs before[kBack], e[kBack];
#pragma unroll
            for (int i = 0; i < kBack; ++i) {
                if (decltype(marked)::value && (firsts >> i & 1)) h = m.get(again()->dim, again()->states, again()->init, __builtin_amdgcn_readlane(mk, i) >> 2);
                const float dt = sd[i][0][m.lane], dtu = sd[i][1][m.lane], dy = sd[i][2][m.lane];
                const scalar_floats o = bc + (tile * kBack + i) * 8;
                before[i] = h;
                float y = 0.f, v[SPW];
#pragma unroll
                for (int s = 0; s < SPW; ++s) {
                    e[i][s] = __builtin_amdgcn_exp2f(dt * a2[s]);
                    h[s] = fmaf(e[i][s], h[s], dtu * o[s]);
                    y = fmaf(o[4 + s], h[s], y);
                    v[s] = dy * h[s];
                }
                sum_c[i] = join_states(v);
                part[2][m.wave][i][m.lane] = y;
                if (decltype(marked)::value && (lasts >> i & 1)) h = fs{};
            }
#pragma unroll
            for (int i = kBack - 1; i >= 0; --i) {
                if (decltype(marked)::value && (lasts >> i & 1)) g = m.get(again()->dim, again()->states, again()->dfinal, __builtin_amdgcn_readlane(mk, i) >> 2);
                const float dt = sd[i][0][m.lane], dtu = sd[i][1][m.lane], dy = sd[i][2][m.lane];
                const scalar_floats o = bc + (tile * kBack + i) * 8;
                float fed = 0.f, moved = 0.f, v[SPW];
#pragma unroll
                for (int s = 0; s < SPW; ++s) {
                    g[s] = fmaf(o[4 + s], dy, g[s]);
                    v[s] = g[s] * dtu;
                    fed = fmaf(g[s], o[s], fed);
                    g[s] *= e[i][s];
                    const float q = g[s] * before[i][s];
                    da[s] = fmaf(q, dt, da[s]);
                    moved = fmaf(q, av[s], moved);
                }
                sum_b[i] = join_states(v);
                part[0][m.wave][i][m.lane] = fed;
                part[1][m.wave][i][m.lane] = moved;
                if (decltype(marked)::value && (firsts >> i & 1)) {
                    if (again()->dinit) m.put(again()->dim, again()->states, again()->dinit, __builtin_amdgcn_readlane(mk, i) >> 2, g);
                    g = fs{};
                }
            }
        };
        if ((firsts | lasts) == 0) tokens(std::false_type{});
        else tokens(std::true_type{});
        // of four lanes with the same sums each writes another: db and dc, of four states those of tokens 0 to 3 and of 4 to 7
        static_assert(kBack == 8, "two groups of four tokens");
        if constexpr (SPW == 4) {
            const float b0 = join_tokens(sum_b, m.lane), c0 = join_tokens(sum_c, m.lane), b1 = join_tokens(sum_b + 4, m.lane),
                        c1 = join_tokens(sum_c + 4, m.lane);
            out_bc[tile * kBack * 8 + out_at] = m.lane & 2 ? (m.lane & 1 ? c1 : b1) : (m.lane & 1 ? c0 : b0);
        } else {
            const float b0 = join_pairs(sum_b, m.lane), c0 = join_pairs(sum_c, m.lane);
            if ((m.lane & 2) == 0) out_bc[tile * kBack * 8 + out_at] = m.lane & 1 ? c0 : b0;
        }
        __syncthreads();
        if (works) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int in = in0 + i * (kThreads / kRow), tok = tile * kBack + in;
                if (tok >= w.n) continue;
                const bool real = raw[i].mark >= 0;
                const fv dt = *(const fv*)&sd[in][0][col], dy = *(const fv*)&sd[in][2][col];
                fv fed = *(const fv*)&part[0][0][in][col], moved = *(const fv*)&part[1][0][in][col], y = {};
#pragma unroll
                for (int k = 1; k < NW; ++k) {
                    fed += *(const fv*)&part[0][k][in][col];
                    moved += *(const fv*)&part[1][k][in][col];
                }
                const auto* k = again();
                const int64_t row = (w.row0 + tok) * k->dim + w.c0;
                float du[V], dd[V], dz[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float u = raw[i].u.get(e);
                    du[e] = real ? fmaf(dt[e], fed[e], skip[e] * dy[e]) : 0.f;
                    float v = fmaf(u, fed[e], moved[e]);
                    if (a.softplus) v *= sigm(raw[i].dt.get(e) + bias[e]);
                    dd[e] = real ? v : 0.f;
                    s_bias[e] += dd[e];
                    s_skip[e] = real ? fmaf(dy[e], u, s_skip[e]) : s_skip[e];
                }
                auto store = [&](void* p, const float (&v)[V]) {
                    T* q = (T*)p + row;
                    if (!whole) {
                        store_piece<T, V>(q, col, w.left, v);
                        return;
                    }
                    Packed<T, V> o;
#pragma unroll
                    for (int e = 0; e < V; ++e) o.e[e] = (T)v[e];
                    *(Packed<T, V>*)(q + col) = o;
                };
                store(k->du, du);
                store(k->ddt, dd);
                if (k->gate) {
#pragma unroll
                    for (int k = 0; k < NW; ++k) y += *(const fv*)&part[2][k][in][col];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float z = raw[i].z.get(e), sg = sigm(z);
                        const float v = raw[i].dy.get(e) * fmaf(skip[e], raw[i].u.get(e), y[e]) * (sg * fmaf(z, 1.f - sg, 1.f));
                        dz[e] = real ? v : 0.f;
                    }
                    store(k->dgate, dz);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) raw[i] = next[i];
        if (tile > 0) ahead.settle();
        own = own_next;
        since = since_next;
        mk = mk_next;
        __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < SPW; ++s) a.part_a[m.slot(a, w.chunk, w.block, NW, s)] = da[s];
    // the channels' sums over the threads that had them, in order
    constexpr int kRows = (kPieces < kThreads ? kPieces : kThreads) / kRow;
    static_assert(kRows <= kBack && 3 * NW >= 2, "room for the sums");
    if (works) {
        *(fv*)&part[0][0][in0][col] = s_skip;
        *(fv*)&part[1][0][in0][col] = s_bias;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * kLanes; i += NW * 64) {
        const int which = i / kLanes, ch = i % kLanes;
        float v = 0.f;
        for (int k = 0; k < kRows; ++k) v += part[which][0][k][ch];
        if (ch < w.left) a.part_d[(w.chunk * 2 + which) * a.dim + w.c0 + ch] = v;
    }
}

// Sums over chunks: of da (blockIdx.y 0, a column for each state of each
// workgroup's lanes), dskip and ddt_bias. 64 columns a workgroup, 16 slices of
// the chunks, then the slices.
__global__ __launch_bounds__(1024) void scan_fold(Scan a, int nw, float* da, float* dskip, float* dbias)
{
    __shared__ float red[16][65];
    const int c = threadIdx.x & 63, slice = threadIdx.x >> 6, which = blockIdx.y;
    const int64_t size = (int64_t)a.blocks * nw * kSpw * kLanes, col = (int64_t)blockIdx.x * 64 + c;
    float* out = which == 0 ? da : which == 1 ? dskip : dbias;
    const int64_t columns = which == 0 ? size : a.dim, pitch = which == 0 ? size : 2 * (int64_t)a.dim;
    if (!out || (int64_t)blockIdx.x * 64 >= columns) return;
    const float* p = which == 0 ? a.part_a + col : a.part_d + (int64_t)(which - 1) * a.dim + col;
    float s = 0.f;
    if (col < columns) {
        int64_t i = slice;
        for (; i + 48 < a.chunks; i += 64) {
            const float v0 = p[i * pitch], v1 = p[(i + 16) * pitch], v2 = p[(i + 32) * pitch], v3 = p[(i + 48) * pitch];
            s += v0; s += v1; s += v2; s += v3;
        }
        for (; i < a.chunks; i += 16) s += p[i * pitch];
    }
    red[slice][c] = s;
    __syncthreads();
    if (slice != 0 || col >= columns) return;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) v += red[k][c];
    if (which) {
        out[col] = v;
        return;
    }
    const int state = (int)(col / kLanes % (nw * kSpw)), block = (int)(col / kLanes / (nw * kSpw));
    const int g = block / a.gblocks, in = (block - g * a.gblocks) * kLanes + c;
    if (in < a.gdim && state < a.states) out[(int64_t)(g * a.gdim + in) * a.states + state] = v;
}

// db and dc: the sums over a group's workgroups. A thread: four states of a token
// and group, of both.
template <typename T>
__global__ __launch_bounds__(256) void scan_fold_bc(Scan a, int nw, T* db, T* dc)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, size = a.places * a.groups * nw;
    const int64_t k = id / a.places, place = id - k * a.places, outer = place / a.pad, t = place - outer * a.pad;
    if (id >= size || t >= a.seq.tokens) return;
    const int w = (int)k % nw;
    f4 b = {0, 0, 0, 0}, c = b;
    const float* p = a.part_bc + id * 8;
    constexpr int U = 4;
    for (int i0 = 0; i0 < a.gblocks; i0 += U) {
        f4 vb[U], vc[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const f4* q = (const f4*)(p + (int64_t)min(i0 + i, a.gblocks - 1) * size * 8);
            vb[i] = q[0];
            vc[i] = q[1];
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i0 + i < a.gblocks) {
                b += vb[i];
                c += vc[i];
            }
    }
    const int64_t at = ((outer * a.seq.tokens + t) * a.groups + k / nw) * a.states + w * kSpw;
    const bool real = a.mark[place] >= 0;
#pragma unroll
    for (int s = 0; s < kSpw; ++s)
        if (w * kSpw + s < a.states) {
            db[at + s] = (T)(real ? b[s] : 0.f);
            dc[at + s] = (T)(real ? c[s] : 0.f);
        }
}

// ---- one token --------------------------------------------------------------------

struct Step {
    const void *u, *dt, *b, *c, *gate;
    const float *a, *skip, *dt_bias;
    float* state;
    const int32_t* slots;
    void* y;
    int64_t u_s, dt_s, gate_s, b_s[2], c_s[2];
    int64_t batch, num_slots;
    int dim, states, gdim, softplus;
    int per;       // lanes of a channel: a power of two, four states each
    int along;     // sequences a workgroup takes, one after another
};

// A thread: four states of a channel, for a few sequences. Bound by the states'
// traffic.
template <typename T>
__global__ __launch_bounds__(256) void scan_step(Step a)
{
    const int lane = threadIdx.x % a.per;
    const int blocks = (int)(((int64_t)a.dim * a.per + 255) / 256);
    const int64_t first = (int64_t)(blockIdx.x / (unsigned)blocks) * a.along;
    const int64_t id = (int64_t)(blockIdx.x % (unsigned)blocks) * 256 + threadIdx.x;
    const int ch = (int)(id / a.per), s0 = lane * kSpw, g = min(ch, a.dim - 1) / a.gdim;
    const bool live = ch < a.dim;
    const int64_t at = (int64_t)ch * a.states + s0;
    const int have = live ? min(kSpw, a.states - s0) : 0;
    const bool whole = a.states % 4 == 0;  // (then have is 4 or not above 0)
    f4 a2 = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < kSpw; ++s)
        if (s < have) a2[s] = rate_of(a.a[at + s]) * kLog2e;
    const float skip = live && a.skip ? a.skip[ch] : 0.f, bias = live && a.dt_bias ? a.dt_bias[ch] : 0.f;
    for (int64_t i = first; i < min(first + a.along, a.batch); ++i) {
        const int64_t slot = a.slots ? a.slots[i] : i;
        const bool known = slot >= 0 && slot < a.num_slots;
        T* y = (T*)a.y + i * a.dim;
        if (!known) {
            if (live && lane == 0) y[ch] = (T)0.f;
            continue;
        }
        float sum = 0.f, u = 0.f, z = 0.f;
        if (have > 0) {
            u = (float)((const T*)a.u)[i * a.u_s + ch];
            float dt = (float)((const T*)a.dt)[i * a.dt_s + ch] + bias;
            if (a.gate) z = (float)((const T*)a.gate)[i * a.gate_s + ch];
            float* h = a.state + slot * a.dim * a.states + at;
            Bits<float, 4> old;
            Bits<T, 4> b, c;
            old.load(h, whole, have);
            b.load((const T*)a.b + i * a.b_s[0] + g * a.b_s[1] + s0, whole, have);
            c.load((const T*)a.c + i * a.c_s[0] + g * a.c_s[1] + s0, whole, have);
            if (a.softplus) dt = softplus_of(dt);
            float now[4];
#pragma unroll
            for (int s = 0; s < kSpw; ++s) {
                now[s] = fmaf(__builtin_amdgcn_exp2f(dt * a2[s]), old.get(s), dt * u * b.get(s));
                sum = s < have ? fmaf(c.get(s), now[s], sum) : sum;
            }
            if (whole) *(Packed<float, 4>*)h = Packed<float, 4>{{now[0], now[1], now[2], now[3]}};
            else store_piece<float, 4>(h, 0, have, now);
        }
        for (int k = a.per / 2; k > 0; k >>= 1) sum += __shfl_xor(sum, k);
        if (live && lane == 0) {
            float v = fmaf(skip, u, sum);
            if (a.gate) v *= silu_of(z);
            y[ch] = (T)v;
        }
    }
}

// ---- host ------------------------------------------------------------------------

constexpr int kMaxStates = 64;
constexpr int64_t kCus = 256;
constexpr int64_t kMaxDim = (int64_t)1 << 20;  // (times 64 states of 4 bytes: a sequence's states stay below 2^31 bytes)
constexpr int64_t kMaxRows = (int64_t)1 << 31;

int check_desc(const gconv_scan_desc* d)
{
    if (!d) return fail(GCONV_ERR_NULL, "descriptor is NULL");
    if (d->dtype != GCONV_F32 && d->dtype != GCONV_BF16) return fail(GCONV_ERR_ARG, "unknown dtype %lld", (long long)d->dtype);
    if (d->sequences < 0 || d->tokens < 0 || d->dim < 1 || d->states < 1 || d->groups < 1)
        return fail(GCONV_ERR_SHAPE, "need sequences, tokens >= 0 and dim, states, groups >= 1 (got %lld, %lld, %lld, %lld, %lld)",
                    (long long)d->sequences, (long long)d->tokens, (long long)d->dim, (long long)d->states, (long long)d->groups);
    if (d->dim % d->groups) return fail(GCONV_ERR_GROUPS, "dim=%lld not divisible by groups=%lld", (long long)d->dim, (long long)d->groups);
    if (d->packed && d->tokens > 0 && d->sequences == 0) return fail(GCONV_ERR_SHAPE, "tokens of no sequence");
    if (d->states > kMaxStates) return fail(GCONV_ERR_UNSUPPORTED, "states=%lld above %d", (long long)d->states, kMaxStates);
    if (d->dim > kMaxDim) return fail(GCONV_ERR_UNSUPPORTED, "dim=%lld above %lld", (long long)d->dim, (long long)kMaxDim);
    if (d->sequences > ((int64_t)1 << 28) || d->tokens > ((int64_t)1 << 30) ||
        (!d->packed && d->tokens > 0 && d->sequences > kMaxRows / d->tokens))
        return fail(GCONV_ERR_UNSUPPORTED, "too many rows");
    return GCONV_OK;
}

int waves_of(int64_t states)
{
    int nw = 1;
    while (nw * kSpw < states) nw *= 2;
    return nw;
}

int64_t outer_of(const gconv_scan_desc* d) { return d->packed ? 1 : d->sequences; }
int64_t rows_of(const gconv_scan_desc* d) { return outer_of(d) * d->tokens; }

struct Layout {
    int nw;
    size_t bc, mark, ends, adds, sums, breaks, hist, hist_sum, part_a, part_d, part_bc, bytes;
};

// Workgroups of the forward pass. A sequence is cut, and then run over twice, only
// where there is less than one workgroup a CU; then into as many chunks as make
// three, as many as run at once (32768 tokens of 2048 channels: 513 us in chunks
// for 768 workgroups, 640 for 512; 4 x 2048 of 4096, 256 workgroups uncut: 265,
// and 280 in three chunks).
constexpr int64_t kForwardBlocks = 768;
// ... and the backward pass, whose longer chunks carry fewer states from one to
// the next but need as many workgroups: 128 tokens, else 64 (4 x 2048 of 4096: 1141
// and 1175 us; 3 x 613 of 300: the last kernel 47 and 27), or 32 where there is less
// than one a CU (3 x 613 of 300, 180 of 64: 21; 2048 of 1024, 512 of 64: 86 in all
// by 64 and 95 by 32).
constexpr int64_t kBackBlocks = 1024;

void plan(const gconv_scan_desc* d, bool back, Scan* a, Layout* l)
{
    l->nw = waves_of(d->states);
    a->rows = rows_of(d);
    a->dim = (int)d->dim;
    a->states = (int)d->states;
    a->groups = (int)d->groups;
    a->gdim = a->dim / a->groups;
    a->gblocks = (a->gdim + kLanes - 1) / kLanes;
    a->blocks = a->groups * a->gblocks;
    a->softplus = d->softplus != 0;
    a->seq.tokens = d->tokens;
    a->seq.count = (int)d->sequences;
    int64_t chunk;
    if (back) {
        auto blocks = [&](int64_t of) { return outer_of(d) * a->blocks * ((d->tokens + of - 1) / of); };
        chunk = blocks(128) >= kBackBlocks ? 128 : blocks(64) >= kCus ? 64 : 32;
    } else {
        const int64_t have = std::max<int64_t>(1, outer_of(d) * a->blocks);
        const int64_t per = have >= kCus ? 1 : (kForwardBlocks + have - 1) / have;
        chunk = std::max<int64_t>(4 * kTile, ((d->tokens + per - 1) / per + kTile - 1) / kTile * kTile);
        chunk = std::min<int64_t>(chunk, (int64_t)1 << 30);
    }
    a->chunk = (int)chunk;
    a->per = std::max<int64_t>(1, (d->tokens + chunk - 1) / chunk);
    a->chunks = d->tokens > 0 ? outer_of(d) * a->per : 0;
    a->pad = (d->tokens + kTile - 1) / kTile * kTile;
    a->places = outer_of(d) * a->pad;
    const int64_t states = a->chunks * a->blocks * l->nw * kSpw * kLanes * 4;
    Cut cut;
    l->bc = cut.take(a->places * a->groups * l->nw * 8 * 4);
    l->mark = cut.take(a->places * 4);
    const bool cuts = a->per > 1;
    l->ends = cut.take(cuts || back ? states : 0);
    l->sums = cut.take(cuts || back ? a->chunks * a->blocks * kLanes * 4 : 0);
    l->breaks = cut.take(cuts || back ? a->chunks * 4 : 0);
    l->adds = cut.take(back ? states : 0);
    l->hist = cut.take(back ? a->places / kBack * a->blocks * l->nw * kSpw * kLanes * 4 : 0);
    l->hist_sum = cut.take(back ? a->places / kBack * a->blocks * kLanes * 4 : 0);
    l->part_a = cut.take(back ? states : 0);
    l->part_d = cut.take(back ? a->chunks * 2 * a->dim * 4 : 0);
    l->part_bc = cut.take(back ? a->places * a->groups * l->nw * 8 * 4 * a->gblocks : 0);
    l->bytes = cut.bytes;
}

// Whether the forward pass gives a wave two states: twice the waves where there
// is no more than a workgroup a CU (4 x 2048 of 4096: 278 us, by four states 292;
// by one, with 16 waves, 311).
bool narrow_forward(const Scan& a) { return a.chunks * a.blocks <= kCus; }

void place(const Layout& l, void* workspace, Scan* a)
{
    char* w = (char*)workspace;
    a->bc = (float*)(w + l.bc);
    a->mark = (int32_t*)(w + l.mark);
    a->ends = (float*)(w + l.ends);
    a->sums = (float*)(w + l.sums);
    a->breaks = (int32_t*)(w + l.breaks);
    a->adds = (float*)(w + l.adds);
    a->hist = (float*)(w + l.hist);
    a->hist_sum = (float*)(w + l.hist_sum);
    a->part_a = (float*)(w + l.part_a);
    a->part_d = (float*)(w + l.part_d);
    a->part_bc = (float*)(w + l.part_bc);
}

// Whether every launch of a call stays below what a launch takes, before any is made.
int check_blocks(const Scan& a, int nw, bool back)
{
    // (the backward pass's last kernel has twice the waves, up to 16, and its sums of da a workgroup of 1024 threads for
    // every 64 states of the workgroups' lanes)
    const int waves = back ? std::min(2 * nw, 16) : nw;
    if (a.chunks > max_blocks(waves * 64) / a.blocks || a.places > max_blocks(256) / (a.groups * nw) * 256 ||
        a.chunks / a.per * a.blocks * nw >= max_blocks(256))
        return fail(GCONV_ERR_UNSUPPORTED, "too many rows");
    if (back && (int64_t)a.blocks * nw * kSpw > max_blocks(1024)) return fail(GCONV_ERR_UNSUPPORTED, "too many groups and states");
    return GCONV_OK;
}

void strides(const gconv_scan_desc* d, Scan* a)
{
    auto two = [&](const int64_t* s, int64_t* o) {
        o[0] = d->packed ? 0 : s[0];
        o[1] = s[1];
    };
    two(d->u_stride, a->u_s);
    two(d->dt_stride, a->dt_s);
    two(d->gate_stride, a->gate_s);
    two(d->dy_stride, a->dy_s);
    two(d->b_stride, a->b_s);
    two(d->c_stride, a->c_s);
    a->b_s[2] = d->b_stride[2];
    a->c_s[2] = d->c_stride[2];
}

// f(waves, states of a wave) for `fours` times four states.
template <typename F>
void by_fours(int fours, F f)
{
    constexpr std::integral_constant<int, 4> four;
    switch (fours) {
        case 1: f(std::integral_constant<int, 1>{}, four); break;
        case 2: f(std::integral_constant<int, 2>{}, four); break;
        case 4: f(std::integral_constant<int, 4>{}, four); break;
        case 8: f(std::integral_constant<int, 8>{}, four); break;
        default: f(std::integral_constant<int, 16>{}, four); break;
    }
}

// ... with two states a wave, where a workgroup's waves then are no more than 16.
template <typename F>
void by_twos(int fours, F f)
{
    constexpr std::integral_constant<int, 2> two;
    switch (fours) {
        case 1: f(std::integral_constant<int, 2>{}, two); break;
        case 2: f(std::integral_constant<int, 4>{}, two); break;
        case 4: f(std::integral_constant<int, 8>{}, two); break;
        case 8: f(std::integral_constant<int, 16>{}, two); break;
        default: f(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{}); break;
    }
}

template <typename F>
void by_type(int64_t dtype, F f)
{
    if (dtype == GCONV_BF16) f((__bf16)0.f);
    else f(0.f);
}

unsigned blocks_of(int64_t threads, int per) { return (unsigned)((threads + per - 1) / per); }

}  // namespace
}  // namespace gconv

using namespace gconv;

extern "C" {

int gconv_scan_workspace_size(const gconv_scan_desc* d, int op, size_t* bytes)
{
    const int st = check_desc(d);
    if (st != GCONV_OK) return st;
    if (op != GCONV_SCAN_FWD && op != GCONV_SCAN_BWD) return fail(GCONV_ERR_ARG, "unknown op %d", op);
    if (!bytes) return fail(GCONV_ERR_NULL, "bytes pointer is NULL");
    Scan a{};
    Layout l{};
    plan(d, op == GCONV_SCAN_BWD, &a, &l);
    *bytes = l.bytes;
    return GCONV_OK;
}

int gconv_scan_fwd(const gconv_scan_desc* d, const void* u, const void* dt, const float* a_, const void* b, const void* c, const float* skip,
                   const void* gate, const float* dt_bias, const int32_t* cu_seqlens, const float* initial_state, void* y,
                   float* final_state, void* workspace, size_t workspace_bytes, void* stream)
{
    int st = check_desc(d);
    if (st != GCONV_OK) return st;
    const int64_t rows = rows_of(d), es = d->dtype == GCONV_BF16 ? 2 : 4, held = d->sequences * d->dim * d->states * 4;
    if (!a_ || (rows > 0 && (!u || !dt || !b || !c || !y))) return fail(GCONV_ERR_NULL, "u, dt, a, b, c and y must be non-NULL");
    if ((d->packed != 0) != (cu_seqlens != nullptr)) return fail(GCONV_ERR_NULL, "cu_seqlens must be given with packed sequences, and only then");
    const int64_t o = outer_of(d);
    const Span in[] = {strided_span(u, es, o, d->u_stride[0], d->tokens, d->u_stride[1], 1, 0, d->dim),
                       strided_span(dt, es, o, d->dt_stride[0], d->tokens, d->dt_stride[1], 1, 0, d->dim),
                       strided_span(gate, es, o, d->gate_stride[0], d->tokens, d->gate_stride[1], 1, 0, d->dim),
                       strided_span(b, es, o, d->b_stride[0], d->tokens, d->b_stride[1], d->groups, d->b_stride[2], d->states),
                       strided_span(c, es, o, d->c_stride[0], d->tokens, d->c_stride[1], d->groups, d->c_stride[2], d->states),
                       {a_, d->dim * d->states * 4}, {skip, d->dim * 4}, {dt_bias, d->dim * 4}, {cu_seqlens, (d->sequences + 1) * 4},
                       {initial_state, held}};
    const Span out[] = {{y, rows * d->dim * es}, {final_state, held}};
    st = check_overlap(in, out);
    if (st != GCONV_OK) return st;
    Scan a{};
    Layout l{};
    plan(d, false, &a, &l);
    st = check_blocks(a, l.nw, false);
    if (st != GCONV_OK) return st;
    st = check_workspace(workspace, workspace_bytes, l.bytes);
    if (st != GCONV_OK) return st;
    place(l, workspace, &a);
    strides(d, &a);
    a.u = u;
    a.dt = dt;
    a.a = a_;
    a.b = b;
    a.c = c;
    a.skip = skip;
    a.gate = gate;
    a.dt_bias = dt_bias;
    a.init = initial_state;
    a.y = y;
    a.final_ = final_state;
    a.seq.cu = cu_seqlens;
    hipStream_t hs = (hipStream_t)stream;
    (void)hipGetLastError();
    if (final_state && d->sequences > 0 && (d->packed || d->tokens == 0))
        scan_empty<<<dim3((unsigned)std::min<int64_t>(d->sequences, 1 << 16), (unsigned)std::min<int64_t>(64, (d->dim * d->states + 255) / 256)), 256, 0, hs>>>(a.seq, initial_state, final_state, d->dim * d->states);
    if (rows == 0) return finish();
    by_type(d->dtype, [&](auto t) {
        using T = decltype(t);
        scan_prep<T><<<blocks_of(a.places * a.groups * l.nw, 256), 256, 0, hs>>>(a, l.nw);
        const unsigned blocks = (unsigned)(a.chunks * a.blocks);
        auto run = [&](auto n, auto m) {
            constexpr int NW = decltype(n)::value, SPW = decltype(m)::value;
            if (a.per > 1) {
                scan_run<T, NW, SPW, false, false><<<blocks, NW * 64, 0, hs>>>(a);
                scan_carry<<<blocks_of(a.chunks / a.per * a.blocks * l.nw * kSpw * kLanes, 256), 256, 0, hs>>>(a, l.nw, a.chunks / a.per);
            }
            scan_run<T, NW, SPW, true, false><<<blocks, NW * 64, 0, hs>>>(a);
        };
        if (narrow_forward(a)) by_twos(l.nw, run);
        else by_fours(l.nw, run);
    });
    return finish();
}

int gconv_scan_bwd(const gconv_scan_desc* d, const void* dy, const void* u, const void* dt, const float* a_, const void* b, const void* c,
                   const float* skip, const void* gate, const float* dt_bias, const int32_t* cu_seqlens, const float* initial_state,
                   const float* d_final_state, void* du, void* ddt, float* da, void* db, void* dc, float* dskip, void* dgate,
                   float* ddt_bias, float* d_initial_state, void* workspace, size_t workspace_bytes, void* stream)
{
    int st = check_desc(d);
    if (st != GCONV_OK) return st;
    const int64_t rows = rows_of(d), es = d->dtype == GCONV_BF16 ? 2 : 4, held = d->sequences * d->dim * d->states * 4;
    if (!a_ || !da || (rows > 0 && (!dy || !u || !dt || !b || !c || !du || !ddt || !db || !dc)))
        return fail(GCONV_ERR_NULL, "dy, u, dt, a, b, c and their gradients must be non-NULL");
    if ((skip != nullptr) != (dskip != nullptr)) return fail(GCONV_ERR_NULL, "skip and dskip go together");
    if ((dt_bias != nullptr) != (ddt_bias != nullptr)) return fail(GCONV_ERR_NULL, "dt_bias and ddt_bias go together");
    if ((gate != nullptr) != (dgate != nullptr) && rows > 0) return fail(GCONV_ERR_NULL, "gate and dgate go together");
    if ((d->packed != 0) != (cu_seqlens != nullptr)) return fail(GCONV_ERR_NULL, "cu_seqlens must be given with packed sequences, and only then");
    const int64_t o = outer_of(d), wide = rows * d->dim * es, narrow = rows * d->groups * d->states * es;
    const Span in[] = {strided_span(u, es, o, d->u_stride[0], d->tokens, d->u_stride[1], 1, 0, d->dim),
                       strided_span(dt, es, o, d->dt_stride[0], d->tokens, d->dt_stride[1], 1, 0, d->dim),
                       strided_span(gate, es, o, d->gate_stride[0], d->tokens, d->gate_stride[1], 1, 0, d->dim),
                       strided_span(dy, es, o, d->dy_stride[0], d->tokens, d->dy_stride[1], 1, 0, d->dim),
                       strided_span(b, es, o, d->b_stride[0], d->tokens, d->b_stride[1], d->groups, d->b_stride[2], d->states),
                       strided_span(c, es, o, d->c_stride[0], d->tokens, d->c_stride[1], d->groups, d->c_stride[2], d->states),
                       {a_, d->dim * d->states * 4}, {skip, d->dim * 4}, {dt_bias, d->dim * 4}, {cu_seqlens, (d->sequences + 1) * 4},
                       {initial_state, held}, {d_final_state, held}};
    const Span out[] = {{du, wide}, {ddt, wide}, {dgate, wide}, {db, narrow}, {dc, narrow}, {da, d->dim * d->states * 4},
                        {dskip, d->dim * 4}, {ddt_bias, d->dim * 4}, {d_initial_state, held}};
    st = check_overlap(in, out);
    if (st != GCONV_OK) return st;
    Scan a{};
    Layout l{};
    plan(d, true, &a, &l);
    st = check_blocks(a, l.nw, true);
    if (st != GCONV_OK) return st;
    st = check_workspace(workspace, workspace_bytes, l.bytes);
    if (st != GCONV_OK) return st;
    place(l, workspace, &a);
    strides(d, &a);
    a.u = u;
    a.dt = dt;
    a.a = a_;
    a.b = b;
    a.c = c;
    a.skip = skip;
    a.gate = gate;
    a.dy = dy;
    a.dt_bias = dt_bias;
    a.init = initial_state;
    a.dfinal = d_final_state;
    a.du = du;
    a.ddt = ddt;
    a.dgate = dgate;
    a.dinit = d_initial_state;
    a.seq.cu = cu_seqlens;
    hipStream_t hs = (hipStream_t)stream;
    (void)hipGetLastError();
    if (d_initial_state && d->sequences > 0 && (d->packed || d->tokens == 0))
        scan_empty<<<dim3((unsigned)std::min<int64_t>(d->sequences, 1 << 16), (unsigned)std::min<int64_t>(64, (d->dim * d->states + 255) / 256)), 256, 0, hs>>>(a.seq, d_final_state, d_initial_state, d->dim * d->states);
    by_type(d->dtype, [&](auto t) {
        using T = decltype(t);
        if (rows > 0) {
            scan_prep<T><<<blocks_of(a.places * a.groups * l.nw, 256), 256, 0, hs>>>(a, l.nw);
            const unsigned blocks = (unsigned)(a.chunks * a.blocks);
            by_fours(l.nw, [&](auto n, auto m) {
                constexpr int NW = decltype(n)::value, SPW = decltype(m)::value;
                scan_run<T, NW, SPW, false, true><<<blocks, NW * 64, 0, hs>>>(a);
            });
            if (a.per > 1)
                scan_carry<<<dim3(blocks_of(a.chunks / a.per * a.blocks * l.nw * kSpw * kLanes, 256), 2), 256, 0, hs>>>(a, l.nw, a.chunks / a.per);
            by_twos(l.nw, [&](auto n, auto m) {
                constexpr int NW = decltype(n)::value, SPW = decltype(m)::value;
                scan_back<T, NW, SPW><<<blocks, NW * 64, 0, hs>>>(a);
            });
            scan_fold_bc<T><<<blocks_of(a.places * a.groups * l.nw, 256), 256, 0, hs>>>(a, l.nw, (T*)db, (T*)dc);
        }
    });
    const int64_t columns = std::max<int64_t>((int64_t)a.blocks * l.nw * kSpw * kLanes, d->dim);
    scan_fold<<<dim3(blocks_of(columns, 64), 3), 1024, 0, hs>>>(a, l.nw, da, dskip, ddt_bias);
    return finish();
}

int gconv_scan_step(const gconv_scan_desc* d, const void* u, const void* dt, const float* a_, const void* b, const void* c,
                    const float* skip, const void* gate, const float* dt_bias, float* state, const int32_t* slots, int64_t num_slots,
                    void* y, void* stream)
{
    int st = check_desc(d);
    if (st != GCONV_OK) return st;
    if (d->packed || d->tokens) return fail(GCONV_ERR_ARG, "a step takes one token of each sequence: packed and tokens must be 0");
    if (num_slots < 0) return fail(GCONV_ERR_SHAPE, "num_slots must be >= 0");
    const int64_t es = d->dtype == GCONV_BF16 ? 2 : 4, n = d->sequences;
    if (!a_ || (n > 0 && (!u || !dt || !b || !c || !y || (num_slots > 0 && !state))))
        return fail(GCONV_ERR_NULL, "u, dt, a, b, c, state and y must be non-NULL");
    if (!slots && num_slots < n) return fail(GCONV_ERR_SHAPE, "%lld sequences, %lld states", (long long)n, (long long)num_slots);
    if (num_slots > kMaxRows) return fail(GCONV_ERR_UNSUPPORTED, "too many states");
    const Span in[] = {strided_span(u, es, n, d->u_stride[0], 1, 0, 1, 0, d->dim), strided_span(dt, es, n, d->dt_stride[0], 1, 0, 1, 0, d->dim),
                       strided_span(gate, es, n, d->gate_stride[0], 1, 0, 1, 0, d->dim),
                       strided_span(b, es, n, d->b_stride[0], 1, 0, d->groups, d->b_stride[2], d->states),
                       strided_span(c, es, n, d->c_stride[0], 1, 0, d->groups, d->c_stride[2], d->states),
                       {a_, d->dim * d->states * 4}, {skip, d->dim * 4}, {dt_bias, d->dim * 4}, {slots, n * 4}};
    const Span out[] = {{state, num_slots * d->dim * d->states * 4}, {y, n * d->dim * es}};
    st = check_overlap(in, out);
    if (st != GCONV_OK) return st;
    (void)hipGetLastError();
    if (n == 0) return finish();
    Step a{};
    a.u = u;
    a.dt = dt;
    a.b = b;
    a.c = c;
    a.gate = gate;
    a.a = a_;
    a.skip = skip;
    a.dt_bias = dt_bias;
    a.state = state;
    a.slots = slots;
    a.y = y;
    a.u_s = d->u_stride[0];
    a.dt_s = d->dt_stride[0];
    a.gate_s = d->gate_stride[0];
    a.b_s[0] = d->b_stride[0];
    a.b_s[1] = d->b_stride[2];
    a.c_s[0] = d->c_stride[0];
    a.c_s[1] = d->c_stride[2];
    a.batch = n;
    a.num_slots = num_slots;
    a.dim = (int)d->dim;
    a.states = (int)d->states;
    a.gdim = a.dim / (int)d->groups;
    a.softplus = d->softplus != 0;
    a.per = waves_of(d->states);
    const int64_t blocks = (d->dim * a.per + 255) / 256;
    a.along = (int)std::max<int64_t>(1, std::min<int64_t>(8, n * blocks / 2048));
    const int64_t all = (n + a.along - 1) / a.along;
    if (all > max_blocks(256) / blocks) return fail(GCONV_ERR_UNSUPPORTED, "too many rows");
    by_type(d->dtype, [&](auto t) { scan_step<decltype(t)><<<(unsigned)(all * blocks), 256, 0, (hipStream_t)stream>>>(a); });
    return finish();
}

}  // extern "C"
