// linattn.hip -- linear attention with a decay for each head (gfx950).
//
//   S_t = lambda S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t
//
// A sequence is cut into segments, a segment into chunks of 64 tokens. Within
// a chunk the recurrence is two matrix products and a mask,
//
//   O = (Q K^T o D) V + diag(lambda^(i+1)) Q S,   D_ij = lambda^(i-j) for j <= i,
//   S' = lambda^64 S + (diag(lambda^(63-j)) K)^T V,
//
// all on the matrix cores. Three kernels:
//   segment_sums   what each segment adds to the state (float32 accuracy)
//   scan_states    the state before each segment, and the final state
//   chunk_outputs  walks the chunks of a segment with its state in registers
// so the tokens are read once (k and v twice) and states pass through memory
// once a segment only. The host picks the segment length so that segments x
// heads give about two workgroups a CU. All three are bound by memory: 32768
// tokens x 16 heads take 66 us for 268 MB, 14 for 67 and 129 for 537 (4.1, 4.9
// and 4.2 TB/s; a large copy reaches 5.2).
//
// The gradients are the same recurrence with the roles of the tensors changed,
// forwards for dq and backwards in time for dk and dv:
//   dq_i = scale S_i do_i                     (queries do, keys v, values k)
//   R_j  = lambda R_{j+1} + scale q_j do_j^T, R_{L-1} = dS_final + scale q do^T
//   dk_j = R_j v_j, dv_j = R_j^T k_j,  dS_init = lambda R_0.
#include <algorithm>

#include "gconv.h"
#include "gconv_internal.h"
#include "device_util.h"
#include "seq_util.h"

namespace gconv {
namespace {

constexpr int kChunk = 64;
constexpr int kThreads = 256;

// One of q, k, v in the role it plays in a pass.
struct Operand {
    const void* p;
    int64_t seq, tok, head;  // strides in elements
    int hdiv;                // q heads that share one of its heads
    int dim;
    int vec;                 // rows start on 16 bytes and hold whole 16-byte pieces
    const char* end;         // of the tensor's last row; NULL where that is not known
};

struct Pass {
    Operand q, k, v;         // queries; keys and values, whose products are the state
    const float* log_decay;
    const int32_t* cu;       // NULL: sequences of `tokens` each
    int64_t tokens;
    int sequences, heads, dk, dv;  // dk, dv: of the state's rows and columns (keys, values)
    int seg;                 // tokens of a segment
    int slots, slots_per_seq;
    int reverse;             // tokens are taken from the last to the first
    int e0;                  // exponent of the initial state at the first token
    int final_more;          // one more decay on the way to the final state (and a non-empty sequence)
    float pscale, iscale, vscale;  // on products within a chunk, on the state's answer, on what enters the state
    float* states;           // [slots][heads][DV][DK], or transposed (state_t)
    int state_t;
    const float* init;       // [sequences][heads][rows][cols]
    float* fin;
    void* out;
    int64_t out_seq, out_tok, out_head;
    int out_f32;             // float32 output whatever T
};

__device__ __forceinline__ float dpow(float g, int n) { return n == 0 ? 1.f : expf(g * (float)n); }

struct Place {
    int n;          // sequence
    int64_t start;  // its first token in packed tensors
    int len;
    int s;          // segment of it
};

// Segment slot -> sequence and segment. Packed: sequence n's segments have the
// slots cu[n] / seg + n and up, which never meet those of n + 1.
__device__ __forceinline__ int64_t cu_at(const Pass& a, int n)
{
    const int64_t v = a.cu[n];
    return v < 0 ? 0 : v > a.tokens ? a.tokens : v;
}

__device__ __forceinline__ Place seq_place(const Pass& a, int n)
{
    Place p{n, 0, (int)a.tokens, 0};
    if (a.cu) {
        p.start = cu_at(a, n);
        const int64_t end = cu_at(a, n + 1);
        p.len = end > p.start ? (int)(end - p.start) : 0;
    }
    return p;
}

__device__ __forceinline__ int first_slot(const Pass& a, int n)
{
    return a.cu ? (int)(cu_at(a, n) / a.seg) + n : n * a.slots_per_seq;
}

__device__ __forceinline__ Place slot_place(const Pass& a, int slot)
{
    int n;
    if (a.cu) {
        int lo = 0, hi = a.sequences - 1;  // the last sequence whose first slot is not past this one
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first_slot(a, mid) <= slot) lo = mid; else hi = mid - 1;
        }
        n = lo;
    } else {
        n = slot / a.slots_per_seq;
    }
    Place p = seq_place(a, n);
    p.s = slot - first_slot(a, n);
    return p;
}

// Zeros a head's output in the rows of packed tensors that no sequence holds,
// those before the first and after the last. The segment slots of the first
// and the last sequence reach as far as them: a slot's workgroup takes the rows
// where its segment would lie.
template <typename T>
__device__ __forceinline__ void clear_rows(const Pass& a, const Place& p, int h, int slot)
{
    auto clear = [&](int64_t from, int64_t to) {
        for (int64_t i = threadIdx.x; i < (to - from) * a.dv; i += kThreads) {
            const int64_t at = (from + i / a.dv) * a.out_tok + (int64_t)h * a.out_head + i % a.dv;
            if (a.out_f32) ((float*)a.out)[at] = 0.f;
            else ((T*)a.out)[at] = (T)0.f;
        }
    };
    if (p.n == 0 && p.s <= 0) clear((int64_t)slot * a.seg, min((int64_t)(slot + 1) * a.seg, cu_at(a, 0)));
    if (p.n == a.sequences - 1 && p.s >= 0) {
        const int64_t at = p.start + (int64_t)p.s * a.seg;
        clear(max(at, p.start + p.len), min(at + a.seg, a.tokens));
    }
}

// Token `t` (in the order of the pass) of an operand's head.
template <typename T>
__device__ __forceinline__ const T* row_of(const Operand& o, const Pass& a, const Place& p, int h, int64_t t)
{
    const int64_t tok = p.start + (a.reverse ? p.len - 1 - t : t);
    return (const T*)o.p + (a.cu ? 0 : (int64_t)p.n * o.seq) + tok * o.tok + (int64_t)(h / o.hdiv) * o.head;
}

// Reads of an operand's rows, 16 bytes a lane, for tokens t0 .. t0 + n - 1 of a
// head. All loads of a chunk are in flight at once, so none may have a branch
// with a wait in it (one by one they took 8 us a chunk). VEC: every row holds
// whole aligned 16-byte pieces, and buffer loads give 0 outside. Otherwise a
// piece is read where it starts, whatever its alignment and although it may
// reach past its row, and `mask` clears what is not the row's when the value
// is used; only a chunk at the tensor's very end reads element by element.
template <typename T, bool VEC>
struct Reader {
    static constexpr int E = 16 / (int)sizeof(T);
    const T* low;    // the chunk's row at the lowest address
    int64_t tok;
    int n, dim, reverse;
    bool edge;
    __amdgpu_buffer_rsrc_t rsrc;

    __device__ __forceinline__ Reader(const Operand& o, const Pass& a, const Place& p, int h, int t0, int n_)
        : tok(o.tok), n(n_), dim(o.dim), reverse(a.reverse)
    {
        low = row_of<T>(o, a, p, h, a.reverse ? t0 + n - 1 : t0);
        if constexpr (VEC) {
            rsrc = make_rsrc(low, (uint32_t)(((n - 1) * tok + dim) * (int64_t)sizeof(T)));
        } else {
            edge = !o.end || (const char*)(low + (n - 1) * tok + (dim + E - 1) / E * E) > o.end;
        }
    }
    __device__ __forceinline__ u4 load(int row, int col) const
    {
        const bool live = row < n && col < dim;
        const int r = reverse ? n - 1 - row : row;
        if constexpr (VEC) {
            return __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(
                                              rsrc, live ? (uint32_t)(r * (int)tok + col) * (uint32_t)sizeof(T) : kOOB, 0, 0));
        } else {
            struct __attribute__((packed, aligned(sizeof(T)))) Loose { u4 v; };
            return ((const Loose*)(low + (live ? r * tok + col : 0)))->v;
        }
    }
    __device__ __forceinline__ u4 load_edge(int row, int col) const
    {
        if (row >= n) return u4{0, 0, 0, 0};
        return load16<T>(low + (reverse ? n - 1 - row : row) * tok, col, dim);
    }
    static __device__ __forceinline__ u4 mask(u4 v, int row, int col, int n, int dim)
    {
        if constexpr (!VEC) {
            const int keep = row < n ? dim - col : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2) v[i] = keep >= 2 * i + 2 ? v[i] : keep == 2 * i + 1 ? v[i] & 0xffffu : 0u;
                else v[i] = keep > i ? v[i] : 0u;
            }
        }
        return v;
    }
};

// A chunk of 64 rows x D of an operand: global memory -> registers -> LDS.
template <typename T, int D, bool VEC>
struct Stage {
    static constexpr int E = 16 / (int)sizeof(T);
    static constexpr int kVpr = D * (int)sizeof(T) / 16;            // 16-byte pieces of a row
    static constexpr int kN = kChunk * kVpr / kThreads;             // pieces of a thread
    // bf16: 32 bytes past a multiple of 256 (or 160), so that the 8 rows x 32
    // bytes of a transposing read and the 16 rows of a fragment's lanes lie in
    // different banks; fp32: 16 bytes past it, for the 4 rows x 64 bytes of its
    // column reads
    static constexpr int kPitch = D + (sizeof(T) == 2 ? 16 : 4);
    u4 r[kN];
    int rows, dim;

    __device__ __forceinline__ void load(const Operand& o, const Pass& a, const Place& p, int h, int t0, int n, int tid)
    {
        const Reader<T, VEC> in(o, a, p, h, t0, n);
        rows = n;
        dim = o.dim;
        if (!VEC && in.edge) {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int idx = tid + i * kThreads;
                r[i] = in.load_edge(idx / kVpr, idx % kVpr * E);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int idx = tid + i * kThreads;
            r[i] = in.load(idx / kVpr, idx % kVpr * E);
        }
    }

    template <int P = kPitch>
    __device__ __forceinline__ void store(T* tile, int tid)
    {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int idx = tid + i * kThreads, row = idx / kVpr, c = idx % kVpr;
            r[i] = Reader<T, VEC>::mask(r[i], row, c * E, rows, dim);
            *(u4*)(tile + row * P + c * E) = r[i];
        }
    }

    __device__ __forceinline__ bool nonfinite() const
    {
        bool b = false;
#pragma unroll
        for (int i = 0; i < kN; ++i) b |= any_nonfinite<T>(r[i]);
        return b;
    }
};

// The weight of each of a fragment's rows (its tokens), in frag_rows order.
template <typename T>
__device__ __forceinline__ void row_weights(const float* w, int row0, int lane, float* out)
{
    const int g = lane >> 4;
    *(f4*)out = *(const f4*)(w + row0 + 4 * g);
    if constexpr (sizeof(T) == 2) *(f4*)(out + 4) = *(const f4*)(w + row0 + 16 + 4 * g);
}

// w x v as fragments that add up to it: one fp32 fragment, or NT bf16 parts of
// 8 bits each, cut off one after another (three hold all 24 bits of the
// float32 product). An infinity or a NaN is the first part's alone.
template <typename T, int NT>
__device__ __forceinline__ void weighted(u4 v, const float* w, u4* out)
{
    if constexpr (sizeof(T) == 4) {
        f4 x = __builtin_bit_cast(f4, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] *= w[i];
        out[0] = __builtin_bit_cast(u4, x);
    } else {
        float x[8], z = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = __builtin_bit_cast(float, i & 1 ? v[i >> 1] & 0xffff0000u : v[i >> 1] << 16) * w[i];
            z = fmaf(x[i], 0.f, z);  // a NaN where one is not finite
        }
        if (__any(z != 0.f)) {
#pragma unroll
            for (int i = 0; i < 8; ++i)  // a NaN whose bits are all in the low half stays one
                if (x[i] != x[i]) x[i] = __builtin_bit_cast(float, 0x7fc00000u);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a = __builtin_bit_cast(uint32_t, x[2 * i]), b = __builtin_bit_cast(uint32_t, x[2 * i + 1]);
                    out[t][i] = a >> 16 | b & 0xffff0000u;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float top = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x[i]) & 0xffff0000u);
                    x[i] = finite_bits<float>(x[i]) ? x[i] - top : 0.f;
                }
            }
            return;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                out[t][i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, x[2 * i + 1]), __builtin_bit_cast(uint32_t, x[2 * i]), 0x07060302u);
            if (t + 1 < NT) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] -= __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x[i]) & 0xffff0000u);
            }
        }
    }
}

// ---- what each segment adds to the state -------------------------------------
//
// L = vscale sum_j lambda^(n-1-j) k_j v_j^T over the segment's n tokens, one
// workgroup a (segment, head). The weighted values are split into three bf16
// parts, so the states keep float32 accuracy: they come back to the caller.
template <typename T, int DK, int DV, bool VEC>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) void segment_sums(Pass a)
{
    using SK = Stage<T, DK, VEC>;
    using SV = Stage<T, DV, VEC>;
    constexpr int NT = sizeof(T) == 2 ? 3 : 1;
    constexpr int RT = DK / 16, CT = DV / 64;
    __shared__ __align__(16) T Ks[kChunk * SK::kPitch];
    __shared__ __align__(16) T Vs[kChunk * SV::kPitch];
    __shared__ __align__(16) float wt[kChunk];

    const int b = xcd_remap(blockIdx.x, gridDim.x);
    const int h = b % a.heads, slot = b / a.heads;
    const Place p = slot_place(a, slot);
    const int t0 = p.s * a.seg;
    if (p.s < 0 || t0 >= p.len) return;
    const int n = min(a.seg, p.len - t0);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const float g = a.log_decay[h];

    f4 S[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) S[r][c] = f4{0, 0, 0, 0};

    SK sk;
    SV sv;
    // From the last chunk to the first: chunk_outputs starts with the first, and
    // what was read last is still in the cache behind the L2s.
    const int first = (n - 1) / kChunk * kChunk;
    sk.load(a.k, a, p, h, t0 + first, n - first, tid);
    sv.load(a.v, a, p, h, t0 + first, n - first, tid);
    for (int c0 = first; c0 >= 0; c0 -= kChunk) {
        __syncthreads();
        sk.store(Ks, tid);
        sv.store(Vs, tid);
        if (tid < kChunk) wt[tid] = c0 + tid < n ? dpow(g, n - 1 - c0 - tid) : 0.f;
        __syncthreads();
        if (c0 > 0) {
            sk.load(a.k, a, p, h, t0 + c0 - kChunk, kChunk, tid);
            sv.load(a.v, a, p, h, t0 + c0 - kChunk, kChunk, tid);
        }
#pragma unroll
        for (int ks = 0; ks < kChunk; ks += Frag<T>::kStep) {
            float w[8];
            row_weights<T>(wt, ks, lane, w);
            u4 fv[CT][NT];
#pragma unroll
            for (int c = 0; c < CT; ++c)
                weighted<T, NT>(frag_rows(Vs, SV::kPitch, ks, (wave * CT + c) * 16, lane), w, fv[c]);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const u4 fk = frag_rows(Ks, SK::kPitch, ks, r * 16, lane);
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int t = NT - 1; t >= 0; --t) S[r][c] = mma<T>(fk, fv[c][t], S[r][c]);
            }
        }
    }
    float* out = a.states + ((int64_t)slot * a.heads + h) * (DK * DV);
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int col = (wave * CT + c) * 16 + (lane & 15);
#pragma unroll
        for (int r = 0; r < RT; ++r) *(f4*)(out + col * DK + r * 16 + 4 * (lane >> 4)) = S[r][c] * a.vscale;
    }
}

// ---- the state before each segment -------------------------------------------
//
// Replaces each segment's sum by the state before it and writes the final
// state. One thread four rows of a column; a segment is one step of the scan.
// Bound by memory: the 33 MB of states of 512 segments take 13 us, 5.1 TB/s.
// (More loads in flight than U, clamped at the end, took 30 us.)
constexpr int scan_parts(int DK, int DV) { return DK * DV / 4 / kThreads; }  // workgroups of a state

template <int DK, int DV>
__global__ __launch_bounds__(kThreads) void scan_states(Pass a)
{
    constexpr int kParts = scan_parts(DK, DV);
    const int part = blockIdx.x % kParts, nh = blockIdx.x / kParts;
    const int h = nh % a.heads, n = nh / a.heads;
    // 16 columns x 16 quads of rows a workgroup pass: 64-byte pieces on both sides
    const int cols = DV / 16;
    const int col = (part % cols) * 16 + (threadIdx.x & 15);
    const int row = ((part / cols) * 16 + (threadIdx.x >> 4)) * 4;
    const Place p = seq_place(a, n);
    const int count = (p.len + a.seg - 1) / a.seg;
    const float g = a.log_decay[h];
    f4 s = {0, 0, 0, 0};
    const int64_t at = ((int64_t)n * a.heads + h) * a.dk * a.dv;
    if (a.init && col < a.dv) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row + i < a.dk) s[i] = a.init[at + (int64_t)(row + i) * a.dv + col];
    }
    if (count > 0) {
        float* base = a.states + ((int64_t)first_slot(a, n) * a.heads + h) * (DK * DV) + col * DK + row;
        const int64_t step = (int64_t)a.heads * (DK * DV);
        const float full = dpow(g, a.seg);
        constexpr int U = 4;  // loads in flight
        for (int i = 0; i < count; i += U) {
            f4 l[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u < count) l[u] = *(const f4*)(base + (i + u) * step);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i + u >= count) break;
                *(f4*)(base + (i + u) * step) = s;
                const int len = min(a.seg, p.len - (i + u) * a.seg);
                const int e = len - (i + u == 0 ? 1 - a.e0 : 0);
                const float d = e == a.seg ? full : dpow(g, e);
                s = s * d + l[u];
            }
        }
        if (a.final_more) s *= dpow(g, 1);
    }
    if (a.fin && col < a.dv) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row + i < a.dk) a.fin[at + (int64_t)(row + i) * a.dv + col] = s[i];
    }
}

// ---- the outputs of a segment, chunk by chunk ----------------------------------
//
// One workgroup of four waves a (segment, head). Each wave owns a quarter of
// the state's columns, in registers, and answers all 64 queries for them:
//   P^T = K Q^T        16 queries a wave; weighted, masked, and exchanged
//                      through LDS
//   O^T = S^T Q^T, scaled by lambda^(i+1) (one factor a lane), + V^T P^T
//   S   = lambda^64 S + K^T (w V)
// The accumulators of S, packed, are the fragments of its product as they lie,
// and a wave reads no values but its own columns', for the output and the
// state both. (With the queries dealt to the waves instead, each of them read
// all of S and V: 142 us for 32768 tokens x 16 heads.)
// In bf16 the products' operands P and S are rounded to bf16, as q, k and v
// are: each rounding is at most 2^-8 of a term, the size of the output's own.
// The accumulators, the state and the weights stay in float32; w V goes in as
// two bf16 parts of 8 bits, so that the state does not gather roundings from
// chunk to chunk (one part: the output 2.7e-3 off in the 2-norm where two give
// 2.4e-3 and its own rounding is 1.7e-3). The caller's final state does not
// come from here but from segment_sums.
template <typename T, int DK, int DV, bool VEC>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) void chunk_outputs(Pass a)
{
    using SK = Stage<T, DK, VEC>;
    using SV = Stage<T, DV, VEC>;
    constexpr int KST = Frag<T>::kStep;
    constexpr int RT = DK / 16, CT = DV / 64, QS = DK / KST;
    constexpr int QT = kChunk / 16;  // tiles of 16 queries
    constexpr int TPK = KST / 16;    // 16-token tiles of one reduction step
    constexpr int NT = sizeof(T) == 2 ? 2 : 1;
    // 16 bytes past a multiple of 128: 16 rows x 16 bytes in different banks
    constexpr int QP = DK + 16 / (int)sizeof(T), PP = kChunk + 16 / (int)sizeof(T);
    __shared__ __align__(16) T Ks[kChunk * SK::kPitch];
    __shared__ __align__(16) T Vs[kChunk * SV::kPitch];
    __shared__ __align__(16) T Qs[kChunk * QP];
    __shared__ __align__(16) T Ps[kChunk * PP];
    __shared__ __align__(16) float wt[kChunk];
    __shared__ float pw[kChunk + 1];
    __shared__ int nonfin[2];

    const int b = xcd_remap(blockIdx.x, gridDim.x);
    const int h = b % a.heads, slot = b / a.heads;
    const Place p = slot_place(a, slot);
    const int t0 = p.s * a.seg;
    if (a.cu) clear_rows<T>(a, p, h, slot);
    if (p.s < 0 || t0 >= p.len) return;
    const int n = min(a.seg, p.len - t0);
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const float ld = a.log_decay[h];
    auto out_at = [&](int t) {  // the output row of token t of the segment
        const int64_t tok = p.start + (a.reverse ? p.len - 1 - (t0 + t) : t0 + t);
        return (a.cu ? 0 : (int64_t)p.n * a.out_seq) + tok * a.out_tok + (int64_t)h * a.out_head;
    };
    SK sk, sq;
    SV sv;
    auto load = [&](int c0) {
        const int m = min(kChunk, n - c0);
        sk.load(a.k, a, p, h, t0 + c0, m, tid);
        sv.load(a.v, a, p, h, t0 + c0, m, tid);
        sq.load(a.q, a, p, h, t0 + c0, m, tid);
    };
    load(0);

    // The state before the segment, in the layout the update produces.
    f4 S[RT][CT];
    const float* st = a.states + ((int64_t)slot * a.heads + h) * (DK * DV);
    if (!a.state_t) {
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int r = 0; r < RT; ++r) S[r][c] = *(const f4*)(st + ((wave * CT + c) * 16 + li) * DK + r * 16 + 4 * g);
    } else {
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[r][c][i] = st[(r * 16 + 4 * g + i) * DV + (wave * CT + c) * 16 + li];
    }
    if (tid <= kChunk) pw[tid] = dpow(ld, tid);
    if (tid < kChunk) wt[tid] = a.vscale * dpow(ld, kChunk - 1 - tid);
    if (tid < 2) nonfin[tid] = 0;
    // Weights of an accumulator tile of P^T (rows: keys 4g + r, column: query li):
    // on the diagonal, and for keys 16 tokens earlier; each 16 more is one factor.
    float wdiag[4], woff[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        wdiag[r] = a.pscale * dpow(ld, max(li - 4 * g - r, 0));
        woff[r] = a.pscale * dpow(ld, 16 + li - 4 * g - r);
    }
    const float p16 = dpow(ld, 16), p32 = dpow(ld, 32);

    for (int c0 = 0; c0 < n; c0 += kChunk) {
        const int m = min(kChunk, n - c0);
        const int par = (c0 / kChunk) & 1;
        __syncthreads();  // the last chunk's tiles have been read (and nonfin is set up)
        sk.store(Ks, tid);
        sv.store(Vs, tid);
        sq.template store<QP>(Qs, tid);
        if (sv.nonfinite()) nonfin[par] = 1;
        __syncthreads();
        const bool more = c0 + kChunk < n;
        if (more) load(c0 + kChunk);
        const bool odd = nonfin[par] != 0;
        if (tid == 0) nonfin[par ^ 1] = 0;

        // the products of the wave's queries with the chunk's keys up to them
        {
            u4 fq[QS];
#pragma unroll
            for (int s = 0; s < QS; ++s) fq[s] = frag_cols<T>(Qs, QP, wave * 16, s * KST, lane);
#pragma unroll
            for (int jt = 0; jt < QT; ++jt) {
                if (jt >= (wave / TPK + 1) * TPK) break;  // the reduction steps that the query's products take
                f4 P = {0, 0, 0, 0};
                if (jt <= wave) {
#pragma unroll
                    for (int s = 0; s < QS; ++s) P = mma<T>(frag_cols<T>(Ks, SK::kPitch, jt * 16, s * KST, lane), fq[s], P);
                    if (jt == wave) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) P[r] = li >= 4 * g + r ? P[r] * wdiag[r] : 0.f;
                    } else {
                        const int far = wave - jt - 1;
                        const float f = far == 0 ? 1.f : far == 1 ? p16 : p32;
#pragma unroll
                        for (int r = 0; r < 4; ++r) P[r] *= woff[r] * f;
                    }
                }
                T* to = Ps + (wave * 16 + li) * PP + jt * 16 + 4 * g;
                if constexpr (sizeof(T) == 2) *(u2*)to = pack4(P);
                else *(f4*)to = P;
            }
        }

        // the state's answers
        const bool lead = p.s == 0 && c0 == 0;
        f4 O[QT][CT];
        {
            u4 fs[QS][CT];
#pragma unroll
            for (int s = 0; s < QS; ++s)
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    if constexpr (sizeof(T) == 2) {
                        const u2 lo = pack4(S[2 * s][c]), hi = pack4(S[2 * s + 1][c]);
                        fs[s][c] = u4{lo[0], lo[1], hi[0], hi[1]};
                    } else {
                        fs[s][c] = __builtin_bit_cast(u4, S[s][c]);
                    }
                }
#pragma unroll
            for (int t = 0; t < QT; ++t) {
#pragma unroll
                for (int c = 0; c < CT; ++c) O[t][c] = f4{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < QS; ++s) {
                    const u4 fq = frag_split<T>(Qs, QP, t * 16, s * KST, lane);
#pragma unroll
                    for (int c = 0; c < CT; ++c) O[t][c] = mma<T>(fs[s][c], fq, O[t][c]);
                }
                const float rd = a.iscale * pw[t * 16 + li + (lead ? a.e0 : 1)];
#pragma unroll
                for (int c = 0; c < CT; ++c) O[t][c] *= rd;
            }
        }
        __syncthreads();  // P is there

        // the chunk's own tokens, up to each query
        u4 fv[kChunk / KST][CT];
#pragma unroll
        for (int ks = 0; ks < kChunk / KST; ++ks)
#pragma unroll
            for (int c = 0; c < CT; ++c) fv[ks][c] = frag_rows(Vs, SV::kPitch, ks * KST, (wave * CT + c) * 16, lane);
#pragma unroll
        for (int ks = 0; ks < kChunk / KST; ++ks)
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                // masked weights are 0, and 0 x infinity is a NaN: such values are
                // kept out of the product and added by themselves below
                u4 v = fv[ks][c];
                if (odd) v = drop_nonfinite<T>(v);
#pragma unroll
                for (int t = ks * TPK; t < QT; ++t)
                    O[t][c] = mma<T>(v, frag_split<T>(Ps, PP, t * 16, ks * KST, lane), O[t][c]);
            }
        if (odd) {
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                const int qi = t * 16 + li;
                const T* qrow = Qs + qi * QP;
#pragma unroll 1
                for (int j = 0; j <= qi; ++j) {
                    const T* krow = Ks + j * SK::kPitch;
                    float dot = 0.f;
#pragma unroll 1
                    for (int d = 0; d < a.k.dim; ++d) dot += (float)qrow[d] * (float)krow[d];
                    dot *= a.pscale * pw[qi - j];
#pragma unroll
                    for (int c = 0; c < CT; ++c)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const T v = Vs[j * SV::kPitch + (wave * CT + c) * 16 + 4 * g + r];
                            if (!finite_bits<T>(v)) O[t][c][r] += dot * (float)v;
                        }
                }
            }
        }

        const bool quads = (a.dv & 3) == 0;  // dense rows: quads of outputs are aligned
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int qi = t * 16 + li;
            if (qi >= m) continue;
            const int64_t at = out_at(c0 + qi);
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int col = (wave * CT + c) * 16 + 4 * g;
                if (a.out_f32 || sizeof(T) == 4) {
                    float* o = (float*)a.out + at + col;
                    if (quads) {
                        if (col < a.dv) *(f4*)o = O[t][c];
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (col + r < a.dv) o[r] = O[t][c][r];
                    }
                } else {
                    T* o = (T*)a.out + at + col;
                    if (quads) {
                        if (col < a.dv) *(u2*)o = pack4(O[t][c]);
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (col + r < a.dv) o[r] = (T)O[t][c][r];
                    }
                }
            }
        }

        // the state after the chunk (not needed after the segment's last)
        if (more) {
            const float d = pw[kChunk - (lead ? 1 - a.e0 : 0)];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < CT; ++c) S[r][c] *= d;
#pragma unroll
            for (int ks = 0; ks < kChunk / KST; ++ks) {
                float w[8];
                row_weights<T>(wt, ks * KST, lane, w);
                u4 fw[CT][NT];
#pragma unroll
                for (int c = 0; c < CT; ++c) weighted<T, NT>(fv[ks][c], w, fw[c]);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const u4 fk = frag_rows(Ks, SK::kPitch, ks * KST, r * 16, lane);
#pragma unroll
                    for (int c = 0; c < CT; ++c)
#pragma unroll
                        for (int t = NT - 1; t >= 0; --t) S[r][c] = mma<T>(fk, fw[c][t], S[r][c]);
                }
            }
        }
    }
}

// ---- gradients of shared heads ---------------------------------------------------
//
// out[row][kh][d] = sum over the rep heads that share kh, in order, of the
// float32 gradients part[row][kh rep + i][d]; four elements a thread where d
// is a multiple of four. Bound by reading the parts, which mostly still are in
// the cache behind the L2s: so it follows the kernel that makes them at once.
template <typename T, int W>
__global__ __launch_bounds__(kThreads) void sum_heads(const float* part, T* out, int64_t count, int rep, int d)
{
    typedef float vec __attribute__((ext_vector_type(W)));
    const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * W;
    if (i >= count) return;
    const int64_t row = i / d;
    const float* q = part + row * rep * d + i % d;
    vec s = *(const vec*)q;
#pragma unroll 4
    for (int r = 1; r < rep; ++r) s += *(const vec*)(q + (int64_t)r * d);
    struct __attribute__((aligned(sizeof(T)))) Out { T e[W]; } o;
#pragma unroll
    for (int k = 0; k < W; ++k) o.e[k] = (T)s[k];
    *(Out*)(out + i) = o;
}

int sum_heads_width(int64_t d) { return d % 4 == 0 ? 4 : 1; }

int64_t sum_heads_blocks(int64_t count, int64_t d) { return (count / sum_heads_width(d) + kThreads - 1) / kThreads; }

template <typename T>
void launch_sum_heads(const float* part, void* out, int64_t count, int rep, int d, hipStream_t st)
{
    const unsigned grid = (unsigned)sum_heads_blocks(count, d);
    if (grid == 0) return;
    if (sum_heads_width(d) == 4) sum_heads<T, 4><<<grid, kThreads, 0, st>>>(part, (T*)out, count, rep, d);
    else sum_heads<T, 1><<<grid, kThreads, 0, st>>>(part, (T*)out, count, rep, d);
}

// ---- one token --------------------------------------------------------------------
//
// A workgroup updates CW columns of one head's state: each thread reads its
// pieces of the state, adds k v^T, writes them back and keeps q_row x S; the
// rows' partial answers meet in LDS. With float32 inputs all of a thread's loads
// are in flight at once and the state's traffic, 8 dk dv bytes a head, bounds it
// (256 tokens of 16 heads: 88 us for 541 MB, 6.1 TB/s). bf16 inputs are converted
// as they are loaded, which waits for each row's before the next row's: the same
// states take 120 us, 4.5 TB/s. One token of 16 heads takes its latency, 5.5 us.
struct Step {
    Operand q, k, v;
    const float* log_decay;
    float* state;
    const int32_t* slots;
    int64_t num_slots;
    void* out;
    int heads, dk, dv, vec;
    float scale;
};

template <typename T, int CW>
__global__ __launch_bounds__(kThreads) void step_kernel(Step a)
{
    constexpr int LC = CW / 4;             // lanes across a row's columns
    constexpr int RG = kThreads / LC;      // rows of one pass
    constexpr int NP = 128 / RG;           // passes over up to 128 rows
    __shared__ f4 red[RG][LC];
    const int tiles = (a.dv + CW - 1) / CW;
    const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles;
    const int h = bh % a.heads, b = bh / a.heads;
    const int tid = threadIdx.x, lc = tid % LC, rg = tid / LC;
    const int col = tile * CW + lc * 4;
    const int64_t slot = a.slots ? (int64_t)a.slots[b] : b;
    T* out = (T*)a.out + ((int64_t)b * a.heads + h) * a.dv;
    if (slot < 0 || slot >= a.num_slots) {
        for (int c = tid; c < CW; c += kThreads)
            if (tile * CW + c < a.dv) out[tile * CW + c] = (T)0.f;
        return;
    }
    float* S = a.state + (slot * a.heads + h) * a.dk * a.dv;
    const T* q = (const T*)a.q.p + b * a.q.seq + (int64_t)h * a.q.head;
    const T* k = (const T*)a.k.p + b * a.k.seq + (int64_t)(h / a.k.hdiv) * a.k.head;
    const T* v = (const T*)a.v.p + b * a.v.seq + (int64_t)(h / a.v.hdiv) * a.v.head;

    f4 s[NP], vv = {0, 0, 0, 0};
    float kk[NP], qq[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int row = rg + i * RG;
        s[i] = f4{0, 0, 0, 0};
        kk[i] = qq[i] = 0.f;
        if (row < a.dk) {
            const float* r = S + (int64_t)row * a.dv + col;
            if (a.vec) {
                if (col < a.dv) s[i] = *(const f4*)r;
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (col + c < a.dv) s[i][c] = r[c];
            }
            kk[i] = (float)k[row];
            qq[i] = (float)q[row];
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (col + c < a.dv) vv[c] = (float)v[col + c];
    const float lam = expf(a.log_decay[h]);
    f4 o = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int row = rg + i * RG;
        if (row < a.dk) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[i][c] = fmaf(lam, s[i][c], kk[i] * vv[c]);
                o[c] = fmaf(qq[i], s[i][c], o[c]);
            }
            float* r = S + (int64_t)row * a.dv + col;
            if (a.vec) {
                if (col < a.dv) *(f4*)r = s[i];
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (col + c < a.dv) r[c] = s[i][c];
            }
        }
    }
    red[rg][lc] = o;
    __syncthreads();
    if (tid < CW) {
        float t = 0.f;
        const float* f = (const float*)&red[0][0];
#pragma unroll
        for (int r = 0; r < RG; ++r) t += f[r * CW + tid];
        if (tile * CW + tid < a.dv) out[tile * CW + tid] = (T)(t * a.scale);
    }
}

// ---- host -----------------------------------------------------------------------

constexpr int64_t kMaxTokens = (int64_t)1 << 30;

int check_desc(const gconv_linattn_desc* d, bool step)
{
    if (!d) return fail(GCONV_ERR_NULL, "descriptor is NULL");
    if (d->dtype != GCONV_F32 && d->dtype != GCONV_BF16) return fail(GCONV_ERR_ARG, "unknown dtype %lld", (long long)d->dtype);
    if (d->sequences < 0 || d->tokens < 0 || d->heads < 1 || d->kv_heads < 1)
        return fail(GCONV_ERR_SHAPE, "need sequences, tokens >= 0 and heads, kv_heads >= 1 (got %lld, %lld, %lld, %lld)",
                    (long long)d->sequences, (long long)d->tokens, (long long)d->heads, (long long)d->kv_heads);
    if (d->heads % d->kv_heads != 0)
        return fail(GCONV_ERR_GROUPS, "heads=%lld not divisible by kv_heads=%lld", (long long)d->heads, (long long)d->kv_heads);
    if (d->dk < 1 || d->dv < 1) return fail(GCONV_ERR_SHAPE, "need dk, dv >= 1 (got %lld, %lld)", (long long)d->dk, (long long)d->dv);
    if (d->dk > 128 || d->dv > 128)
        return fail(GCONV_ERR_UNSUPPORTED, "head sizes above 128 (dk=%lld, dv=%lld)", (long long)d->dk, (long long)d->dv);
    if (d->heads > 65536 || d->sequences > kMaxTokens || d->tokens > kMaxTokens || d->sequences * d->heads > kMaxTokens ||
        (!step && d->sequences > 0 && d->tokens > kMaxTokens / (d->packed ? 1 : d->sequences)))
        return fail(GCONV_ERR_UNSUPPORTED, "more than 2^30 tokens, or sequences x heads, or more than 65536 heads");
    if (step && (d->packed || d->tokens)) return fail(GCONV_ERR_ARG, "a single-token step has packed == 0 and tokens == 0");
    return GCONV_OK;
}

struct Plan {
    int seg, slots, slots_per_seq, DK, DV;
    int64_t state_elems;   // of one set of segment states
    int64_t rows;          // tokens in all
};

int pad64(int64_t d) { return d <= 64 ? 64 : 128; }

// Segments x heads come to about 512 workgroups, two for each of the 256 CUs
// (both fit: 64 KB of LDS each), and a segment is whole chunks. Each of packed
// sequences ends in a part of one, so as many fewer are planned, down to half
// (7264 tokens in 12 sequences: 110 us, 120 with segments for 512 workgroups
// before the parts).
int make_plan(const gconv_linattn_desc* d, int op, Plan* p)
{
    p->rows = d->packed ? d->tokens : d->sequences * d->tokens;
    const int64_t per_head = std::max<int64_t>(1, 512 / d->heads);
    const int64_t whole = d->packed ? std::max((per_head + 1) / 2, per_head - d->sequences) : per_head;
    const int64_t seg = (p->rows + whole - 1) / whole;
    p->seg = (int)std::max<int64_t>(kChunk, (seg + kChunk - 1) / kChunk * kChunk);
    p->slots_per_seq = (int)((d->tokens + p->seg - 1) / p->seg);
    const int64_t slots = d->packed ? d->tokens / p->seg + d->sequences : d->sequences * p->slots_per_seq;
    p->DK = pad64(d->dk);
    p->DV = pad64(d->dv);
    if (slots * d->heads > max_blocks(kThreads) || d->sequences * d->heads * scan_parts(p->DK, p->DV) > max_blocks(kThreads))
        return fail(GCONV_ERR_UNSUPPORTED, "too many sequences x heads");
    if (op == GCONV_LINATTN_BWD && d->heads != d->kv_heads &&
        (sum_heads_blocks(p->rows * d->kv_heads * d->dk, d->dk) > max_blocks(kThreads) ||
         sum_heads_blocks(p->rows * d->kv_heads * d->dv, d->dv) > max_blocks(kThreads)))
        return fail(GCONV_ERR_UNSUPPORTED, "too many tokens x kv_heads");
    p->slots = (int)slots;
    p->state_elems = slots * d->heads * p->DK * p->DV;
    return GCONV_OK;
}

// The end of a strided tensor whose strides are not negative, else NULL.
const char* end_of(const gconv_linattn_desc* d, const void* p, const int64_t* s, int64_t heads, int64_t dim, int64_t es)
{
    if (s[1] < 0 || s[2] < 0 || (!d->packed && s[0] < 0) || d->tokens < 1 || d->sequences < 1) return nullptr;
    int64_t last = (d->tokens - 1) * s[1] + (heads - 1) * s[2] + dim;
    if (!d->packed) last += (d->sequences - 1) * s[0];
    return (const char*)p + last * es;
}

Operand operand(const gconv_linattn_desc* d, const void* p, const int64_t* stride, int64_t heads, int hdiv, int64_t dim, int64_t es)
{
    Operand o{p, stride[0], stride[1], stride[2], hdiv, (int)dim, 0, end_of(d, p, stride, heads, dim, es)};
    // (a chunk's 64 rows span less than 2^31 bytes)
    o.vec = stride[1] >= 0 && stride[1] < ((int64_t)1 << 22) && ((uintptr_t)p & 15) == 0 && stride[0] * es % 16 == 0 && stride[1] * es % 16 == 0 && stride[2] * es % 16 == 0 &&
            dim * es % 16 == 0;
    return o;
}

template <typename T, int DK, int DV>
void launch_states(const Pass& a, hipStream_t st)
{
    const unsigned grid = a.slots * a.heads;
    if (grid > 0) {
        if (a.k.vec && a.v.vec) segment_sums<T, DK, DV, true><<<grid, kThreads, 0, st>>>(a);
        else segment_sums<T, DK, DV, false><<<grid, kThreads, 0, st>>>(a);
    }
    if (a.sequences > 0)
        scan_states<DK, DV><<<(unsigned)(a.sequences * a.heads * scan_parts(DK, DV)), kThreads, 0, st>>>(a);
}

template <typename T>
void states(const Pass& a, int DK, int DV, hipStream_t st)
{
    if (DK == 64 && DV == 64) launch_states<T, 64, 64>(a, st);
    else if (DK == 64) launch_states<T, 64, 128>(a, st);
    else if (DV == 64) launch_states<T, 128, 64>(a, st);
    else launch_states<T, 128, 128>(a, st);
}

template <typename T, int DK, int DV>
void launch_outputs(const Pass& a, hipStream_t st)
{
    const unsigned grid = a.slots * a.heads;
    if (grid == 0) return;
    if (a.q.vec && a.k.vec && a.v.vec) chunk_outputs<T, DK, DV, true><<<grid, kThreads, 0, st>>>(a);
    else chunk_outputs<T, DK, DV, false><<<grid, kThreads, 0, st>>>(a);
}

template <typename T>
void outputs(const Pass& a, int DK, int DV, hipStream_t st)
{
    if (DK == 64 && DV == 64) launch_outputs<T, 64, 64>(a, st);
    else if (DK == 64) launch_outputs<T, 64, 128>(a, st);
    else if (DV == 64) launch_outputs<T, 128, 64>(a, st);
    else launch_outputs<T, 128, 128>(a, st);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

size_t workspace_bytes(const gconv_linattn_desc* d, const Plan& p, int op)
{
    const size_t one = up256((size_t)p.state_elems * 4);
    if (op == GCONV_LINATTN_FWD) return one;
    // float32 gradients of each q head where heads share k and v
    const size_t part = d->heads != d->kv_heads ? up256((size_t)p.rows * d->heads * d->dk * 4) + up256((size_t)p.rows * d->heads * d->dv * 4) : 0;
    return one + part;
}

struct Range {
    const void* p;
    int64_t bytes;
};

bool meets(const Range& a, const Range& b)
{
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    return (const char*)a.p < (const char*)b.p + b.bytes && (const char*)b.p < (const char*)a.p + a.bytes;
}

// Bytes from the first to past the last element of a strided tensor whose
// strides are not negative (others are taken as one element).
Range span(const void* p, const gconv_linattn_desc* d, const int64_t* s, int64_t heads, int64_t dim, bool step)
{
    const int64_t es = d->dtype == GCONV_BF16 ? 2 : 4;
    if (d->sequences == 0 || (!step && d->tokens == 0)) return Range{p, 0};
    int64_t last = (heads - 1) * std::max<int64_t>(s[2], 0) + dim;
    if (!step) last += (d->tokens - 1) * std::max<int64_t>(s[1], 0);
    if (!d->packed) last += (d->sequences - 1) * std::max<int64_t>(s[0], 0);
    return Range{p, last * es};
}

template <typename T>
int run_fwd(const Plan& p, const Pass& a, hipStream_t st)
{
    states<T>(a, p.DK, p.DV, st);
    outputs<T>(a, p.DK, p.DV, st);
    return finish();
}

// Dense [.., heads, d] output.
void dense_out(Pass* a, void* out, int64_t heads, int64_t d)
{
    a->out = out;
    a->out_head = d;
    a->out_tok = heads * d;
    a->out_seq = a->tokens * a->out_tok;
}

// `a`: the forward pass's operands; `dout`: the gradient of o; `part`: float32
// gradients of each q head, where heads share k and v.
template <typename T>
int run_bwd(const gconv_linattn_desc* d, const Plan& p, const Pass& a, const Operand& dout, const float* d_final,
            void* dq, void* dk, void* dv, float* d_init, float* part, hipStream_t st)
{
    const int rep = (int)(d->heads / d->kv_heads);
    // the states before each segment, forwards in time, and dq
    states<T>(a, p.DK, p.DV, st);
    Pass b = a;
    b.q = dout;
    b.k = a.v;
    b.v = a.k;
    b.dk = a.dv;
    b.dv = a.dk;
    b.state_t = 1;
    dense_out(&b, dq, d->heads, d->dk);
    outputs<T>(b, p.DV, p.DK, st);

    // the states of the gradient, backwards in time (in the place of the others)
    Pass r = a;
    r.k = a.q;
    r.v = dout;
    r.reverse = 1;
    r.e0 = 0;
    r.vscale = a.pscale;
    r.iscale = 1.f;
    r.init = d_final;
    r.fin = d_init;
    r.final_more = 1;
    states<T>(r, p.DK, p.DV, st);
    r.out_f32 = part != nullptr;
    float* part_dv = part ? part + up256((size_t)p.rows * d->heads * d->dk * 4) / 4 : nullptr;
    Pass v = r;
    v.q = a.k;
    dense_out(&v, part ? part_dv : dv, d->heads, d->dv);
    outputs<T>(v, p.DK, p.DV, st);
    if (part) launch_sum_heads<T>(part_dv, dv, p.rows * d->kv_heads * d->dv, rep, (int)d->dv, st);
    Pass k = r;
    k.q = a.v;
    k.k = dout;
    k.v = a.q;
    k.dk = a.dv;
    k.dv = a.dk;
    k.state_t = 1;
    dense_out(&k, part ? part : dk, d->heads, d->dk);
    outputs<T>(k, p.DV, p.DK, st);
    if (part) launch_sum_heads<T>(part, dk, p.rows * d->kv_heads * d->dk, rep, (int)d->dk, st);
    return finish();
}

}  // namespace
}  // namespace gconv

using namespace gconv;

extern "C" {

int gconv_linattn_workspace_size(const gconv_linattn_desc* d, int op, size_t* bytes)
{
    int st = check_desc(d, false);
    if (st != GCONV_OK) return st;
    if (!bytes) return fail(GCONV_ERR_NULL, "bytes pointer is NULL");
    if (op != GCONV_LINATTN_FWD && op != GCONV_LINATTN_BWD) return fail(GCONV_ERR_ARG, "bad op %d", op);
    Plan p;
    st = make_plan(d, op, &p);
    if (st != GCONV_OK) return st;
    *bytes = workspace_bytes(d, p, op);
    return GCONV_OK;
}

namespace {

// Checks that the forward and the backward pass share, and their common Pass.
int common(const gconv_linattn_desc* d, int op, const void* q, const void* k, const void* v, const float* log_decay,
           const int32_t* cu, void* ws, size_t ws_bytes, Plan* p, Pass* a)
{
    int st = check_desc(d, false);
    if (st != GCONV_OK) return st;
    st = make_plan(d, op, p);
    if (st != GCONV_OK) return st;
    const bool some = p->rows > 0 && d->sequences > 0;
    if (p->rows > 0 && d->sequences == 0) return fail(GCONV_ERR_SHAPE, "tokens without a sequence");
    if (!log_decay || (some && (!q || !k || !v))) return fail(GCONV_ERR_NULL, "q, k, v and log_decay must be non-NULL");
    if ((d->packed != 0) != (cu != nullptr))
        return fail(GCONV_ERR_NULL, "cu_seqlens must be given with packed sequences, and only then");
    const size_t need = workspace_bytes(d, *p, op);
    if (ws_bytes < need || (need > 0 && !ws)) return fail(GCONV_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", ws_bytes, need);
    if (need > 0 && ((uintptr_t)ws & 15) != 0) return fail(GCONV_ERR_WORKSPACE, "workspace pointer %p is not 16-byte aligned", ws);
    const int64_t es = d->dtype == GCONV_BF16 ? 2 : 4;
    const int rep = (int)(d->heads / d->kv_heads);
    *a = Pass{};
    a->q = operand(d, q, d->q_stride, d->heads, 1, d->dk, es);
    a->k = operand(d, k, d->k_stride, d->kv_heads, rep, d->dk, es);
    a->v = operand(d, v, d->v_stride, d->kv_heads, rep, d->dv, es);
    a->log_decay = log_decay;
    a->cu = cu;
    a->tokens = d->tokens;
    a->sequences = (int)d->sequences;
    a->heads = (int)d->heads;
    a->dk = (int)d->dk;
    a->dv = (int)d->dv;
    a->seg = p->seg;
    a->slots = p->slots;
    a->slots_per_seq = p->slots_per_seq;
    a->e0 = 1;
    a->pscale = a->iscale = (float)d->scale;
    a->vscale = 1.f;
    a->states = (float*)ws;
    return GCONV_OK;
}

}  // namespace

int gconv_linattn_fwd(const gconv_linattn_desc* d, const void* q, const void* k, const void* v, const float* log_decay,
                      const int32_t* cu_seqlens, const float* initial_state, void* o, float* final_state,
                      void* workspace, size_t workspace_bytes_, void* stream)
{
    Plan p;
    Pass a;
    int st = common(d, GCONV_LINATTN_FWD, q, k, v, log_decay, cu_seqlens, workspace, workspace_bytes_, &p, &a);
    if (st != GCONV_OK) return st;
    if (p.rows > 0 && !o) return fail(GCONV_ERR_NULL, "o must be non-NULL");
    const int64_t es = d->dtype == GCONV_BF16 ? 2 : 4;
    const int64_t sb = d->sequences * d->heads * d->dk * d->dv * 4;
    const Range in[] = {span(q, d, d->q_stride, d->heads, d->dk, false), span(k, d, d->k_stride, d->kv_heads, d->dk, false),
                        span(v, d, d->v_stride, d->kv_heads, d->dv, false), {log_decay, d->heads * 4}, {initial_state, sb},
                        {cu_seqlens, (d->sequences + 1) * 4}};
    const Range out[] = {{o, p.rows * d->heads * d->dv * es}, {final_state, sb}};
    for (const Range& w : out)
        for (const Range& r : in)
            if (meets(w, r)) return fail(GCONV_ERR_ARG, "o or final_state overlaps an input");
    if (meets(out[0], out[1])) return fail(GCONV_ERR_ARG, "o overlaps final_state");
    a.init = initial_state;
    a.fin = final_state;
    dense_out(&a, o, d->heads, d->dv);
    hipStream_t hs = (hipStream_t)stream;
    (void)hipGetLastError();
    return d->dtype == GCONV_BF16 ? run_fwd<__bf16>(p, a, hs) : run_fwd<float>(p, a, hs);
}

int gconv_linattn_bwd(const gconv_linattn_desc* d, const void* dout, const void* q, const void* k, const void* v,
                      const float* log_decay, const int32_t* cu_seqlens, const float* initial_state,
                      const float* d_final_state, void* dq, void* dk, void* dv, float* d_initial_state,
                      void* workspace, size_t workspace_bytes_, void* stream)
{
    Plan p;
    Pass a;
    int st = common(d, GCONV_LINATTN_BWD, q, k, v, log_decay, cu_seqlens, workspace, workspace_bytes_, &p, &a);
    if (st != GCONV_OK) return st;
    if (p.rows > 0 && (!dout || !dq || !dk || !dv)) return fail(GCONV_ERR_NULL, "dout, dq, dk and dv must be non-NULL");
    const int64_t es = d->dtype == GCONV_BF16 ? 2 : 4;
    const int64_t sb = d->sequences * d->heads * d->dk * d->dv * 4;
    const Range in[] = {span(q, d, d->q_stride, d->heads, d->dk, false), span(k, d, d->k_stride, d->kv_heads, d->dk, false),
                        span(v, d, d->v_stride, d->kv_heads, d->dv, false), span(dout, d, d->do_stride, d->heads, d->dv, false),
                        {log_decay, d->heads * 4}, {initial_state, sb}, {d_final_state, sb},
                        {cu_seqlens, (d->sequences + 1) * 4}};
    const Range out[] = {{dq, p.rows * d->heads * d->dk * es}, {dk, p.rows * d->kv_heads * d->dk * es},
                         {dv, p.rows * d->kv_heads * d->dv * es}, {d_initial_state, sb}};
    for (const Range& w : out)
        for (const Range& r : in)
            if (meets(w, r)) return fail(GCONV_ERR_ARG, "a gradient overlaps an input");
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (meets(out[i], out[j])) return fail(GCONV_ERR_ARG, "two gradients overlap");
    a.init = initial_state;
    const Operand od = operand(d, dout, d->do_stride, d->heads, 1, d->dv, es);
    float* part = nullptr;
    if (d->heads != d->kv_heads) part = (float*)((char*)workspace + up256((size_t)p.state_elems * 4));
    hipStream_t hs = (hipStream_t)stream;
    (void)hipGetLastError();
    if (d->dtype == GCONV_BF16) return run_bwd<__bf16>(d, p, a, od, d_final_state, dq, dk, dv, d_initial_state, part, hs);
    return run_bwd<float>(d, p, a, od, d_final_state, dq, dk, dv, d_initial_state, part, hs);
}

int gconv_linattn_step(const gconv_linattn_desc* d, const void* q, const void* k, const void* v, const float* log_decay,
                       float* state, const int32_t* slots, int64_t num_slots, void* o, void* stream)
{
    const int st = check_desc(d, true);
    if (st != GCONV_OK) return st;
    if (num_slots < 0) return fail(GCONV_ERR_SHAPE, "num_slots=%lld must be >= 0", (long long)num_slots);
    if (!slots && num_slots < d->sequences)
        return fail(GCONV_ERR_SHAPE, "%lld sequences without slots need as many states (got %lld)", (long long)d->sequences,
                    (long long)num_slots);
    if (d->sequences > 0 && (!q || !k || !v || !log_decay || !o || (num_slots > 0 && !state)))
        return fail(GCONV_ERR_NULL, "q, k, v, log_decay, state and o must be non-NULL");
    const int64_t es = d->dtype == GCONV_BF16 ? 2 : 4;
    const Range in[] = {span(q, d, d->q_stride, d->heads, d->dk, true), span(k, d, d->k_stride, d->kv_heads, d->dk, true),
                        span(v, d, d->v_stride, d->kv_heads, d->dv, true), {log_decay, d->heads * 4},
                        {slots, d->sequences * 4}};
    const Range out[] = {{o, d->sequences * d->heads * d->dv * es}, {state, num_slots * d->heads * d->dk * d->dv * 4}};
    for (const Range& w : out)
        for (const Range& r : in)
            if (meets(w, r)) return fail(GCONV_ERR_ARG, "o or state overlaps an input");
    if (meets(out[0], out[1])) return fail(GCONV_ERR_ARG, "o overlaps state");
    const int64_t bh = d->sequences * d->heads;
    if (bh > max_blocks(kThreads)) return fail(GCONV_ERR_UNSUPPORTED, "too many sequences x heads");
    hipStream_t hs = (hipStream_t)stream;
    (void)hipGetLastError();
    if (d->sequences == 0) return finish();
    Step a{};
    const int rep = (int)(d->heads / d->kv_heads);
    a.q = operand(d, q, d->q_stride, d->heads, 1, d->dk, es);
    a.k = operand(d, k, d->k_stride, d->kv_heads, rep, d->dk, es);
    a.v = operand(d, v, d->v_stride, d->kv_heads, rep, d->dv, es);
    a.log_decay = log_decay;
    a.state = state;
    a.slots = slots;
    a.num_slots = num_slots;
    a.out = o;
    a.heads = (int)d->heads;
    a.dk = (int)d->dk;
    a.dv = (int)d->dv;
    a.scale = (float)d->scale;
    a.vec = ((uintptr_t)state & 15) == 0 && d->dv % 4 == 0;
    // Few heads in all: 32 columns a workgroup, four times as many of them.
    const int cw = bh < 512 ? 32 : 128;
    const unsigned grid = (unsigned)(bh * ((d->dv + cw - 1) / cw));
    if (d->dtype == GCONV_BF16) {
        if (cw == 32) step_kernel<__bf16, 32><<<grid, kThreads, 0, hs>>>(a);
        else step_kernel<__bf16, 128><<<grid, kThreads, 0, hs>>>(a);
    } else {
        if (cw == 32) step_kernel<float, 32><<<grid, kThreads, 0, hs>>>(a);
        else step_kernel<float, 128><<<grid, kThreads, 0, hs>>>(a);
    }
    return finish();
}

}  // extern "C"
