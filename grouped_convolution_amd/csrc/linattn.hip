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
// heads give about two workgroups a CU.
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

// Token `t` (in the order of the pass) of an operand's head.
template <typename T>
__device__ __forceinline__ const T* row_of(const Operand& o, const Pass& a, const Place& p, int h, int64_t t)
{
    const int64_t tok = p.start + (a.reverse ? p.len - 1 - t : t);
    return (const T*)o.p + (a.cu ? 0 : (int64_t)p.n * o.seq) + tok * o.tok + (int64_t)(h / o.hdiv) * o.head;
}

// A chunk of 64 rows x D of an operand: global memory -> registers -> LDS.
template <typename T, int D>
struct Stage {
    static constexpr int kVpr = D * (int)sizeof(T) / 16;            // 16-byte pieces of a row
    static constexpr int kN = kChunk * kVpr / kThreads;             // pieces of a thread
    static constexpr int kPitch = D + 16 / (int)sizeof(T);
    u4 r[kN];

    __device__ __forceinline__ void load(const Operand& o, const Pass& a, const Place& p, int h, int t0, int n, int tid)
    {
        const T* base = row_of<T>(o, a, p, h, t0);
        const int64_t step = a.reverse ? -o.tok : o.tok;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int idx = tid + i * kThreads, row = idx / kVpr, c = idx % kVpr;
            r[i] = u4{0, 0, 0, 0};
            if (row < n) r[i] = load16<T>(base + row * step, c * (16 / (int)sizeof(T)), o.dim, o.vec);
        }
    }

    __device__ __forceinline__ void store(T* tile, int tid) const
    {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int idx = tid + i * kThreads, row = idx / kVpr, c = idx % kVpr;
            *(u4*)(tile + row * kPitch + c * (16 / (int)sizeof(T))) = r[i];
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
// 8 bits each (three hold the float32 product, its error below 2^-24).
template <typename T, int NT>
__device__ __forceinline__ void weighted(u4 v, const float* w, u4* out)
{
    if constexpr (sizeof(T) == 4) {
        f4 x = __builtin_bit_cast(f4, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] *= w[i];
        out[0] = __builtin_bit_cast(u4, x);
    } else {
        const bf8 b = __builtin_bit_cast(bf8, v);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)b[i] * w[i];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            bf8 part;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                part[i] = (__bf16)x[i];
                // what the part leaves; nothing where it took an infinity or a NaN
                if (t + 1 < NT) x[i] = finite_bits<float>(x[i]) && finite_bits<__bf16>(part[i]) ? x[i] - (float)part[i] : 0.f;
            }
            out[t] = __builtin_bit_cast(u4, part);
        }
    }
}

// ---- what each segment adds to the state -------------------------------------
//
// L = vscale sum_j lambda^(n-1-j) k_j v_j^T over the segment's n tokens, one
// workgroup a (segment, head). The weighted values are split into three bf16
// parts, so the states keep float32 accuracy: they come back to the caller.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(kThreads) void segment_sums(Pass a)
{
    using SK = Stage<T, DK>;
    using SV = Stage<T, DV>;
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
    const float l64 = dpow(g, kChunk);

    f4 S[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) S[r][c] = f4{0, 0, 0, 0};

    SK sk;
    SV sv;
    sk.load(a.k, a, p, h, t0, min(kChunk, n), tid);
    sv.load(a.v, a, p, h, t0, min(kChunk, n), tid);
    for (int c0 = 0; c0 < n; c0 += kChunk) {
        const int m = min(kChunk, n - c0);
        __syncthreads();
        sk.store(Ks, tid);
        sv.store(Vs, tid);
        if (tid < kChunk) wt[tid] = tid < m ? dpow(g, m - 1 - tid) : 0.f;
        __syncthreads();
        if (c0 + kChunk < n) {
            const int m2 = min(kChunk, n - c0 - kChunk);
            sk.load(a.k, a, p, h, t0 + c0 + kChunk, m2, tid);
            sv.load(a.v, a, p, h, t0 + c0 + kChunk, m2, tid);
        }
        const float decay = m == kChunk ? l64 : dpow(g, m);
        if (c0 > 0) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < CT; ++c) S[r][c] *= decay;
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
template <int DK, int DV>
__global__ __launch_bounds__(kThreads) void scan_states(Pass a)
{
    constexpr int kParts = DK * DV / 4 / kThreads;
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
// One workgroup of four waves a (segment, head). Each wave answers 16 queries
// of the chunk and owns a quarter of the state's columns:
//   P^T = K Q^T        accumulator tiles, weighted and masked, packed into the
//                      fragments of the next product as they lie
//   O^T = S^T Q^T, scaled by lambda^(i+1) (one factor a lane), + V^T P^T
//   S   = lambda^64 S + K^T (w V)
// In bf16 the products' operands P, S and w V are rounded to bf16, as q, k and
// v are: each rounding is at most 2^-8 of a term, the size of the output's own.
// The accumulators, the state and the weights stay in float32, and the
// caller's final state does not come from here but from segment_sums.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) void chunk_outputs(Pass a)
{
    using SK = Stage<T, DK>;
    using SV = Stage<T, DV>;
    constexpr int E = Frag<T>::kElems, KST = Frag<T>::kStep;
    constexpr int RT = DK / 16, CT = DV / 64, OT = DV / 16, QS = DK / KST;
    constexpr int TPK = KST / 16;  // 16-token tiles of one reduction step
    constexpr int SP = SK::kPitch;
    __shared__ __align__(16) T Ks[kChunk * SK::kPitch];
    __shared__ __align__(16) T Vs[kChunk * SV::kPitch];
    __shared__ __align__(16) T St[DV * SP];
    __shared__ __align__(16) float wt[kChunk];
    __shared__ float pw[kChunk + 1];
    __shared__ int nonfin[2];

    const int b = xcd_remap(blockIdx.x, gridDim.x);
    const int h = b % a.heads, slot = b / a.heads;
    const Place p = slot_place(a, slot);
    const int t0 = p.s * a.seg;
    if (p.s < 0 || t0 >= p.len) return;
    const int n = min(a.seg, p.len - t0);
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const float ld = a.log_decay[h];

    SK sk;
    SV sv;
    sk.load(a.k, a, p, h, t0, min(kChunk, n), tid);
    sv.load(a.v, a, p, h, t0, min(kChunk, n), tid);

    // The state before the segment, in the layout the update produces.
    f4 S[RT][CT];
    const float* st = a.states + ((int64_t)slot * a.heads + h) * (DK * DV);
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int col = (wave * CT + c) * 16 + li;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int row = r * 16 + 4 * g;
            if (!a.state_t) {
                S[r][c] = *(const f4*)(st + col * DK + row);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) S[r][c][i] = st[(row + i) * DV + col];
            }
        }
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
        if (sv.nonfinite()) nonfin[par] = 1;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            T* col = St + ((wave * CT + c) * 16 + li) * SP + 4 * g;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if constexpr (sizeof(T) == 2) *(u2*)(col + r * 16) = pack4(S[r][c]);
                else *(f4*)(col + r * 16) = S[r][c];
            }
        }
        const int qi = wave * 16 + li;  // this lane's query in the chunk
        const bool live = qi < m;
        const T* qrow = row_of<T>(a.q, a, p, h, live ? t0 + c0 + qi : t0);
        u4 fq[QS];
#pragma unroll
        for (int s = 0; s < QS; ++s) {
            fq[s] = u4{0, 0, 0, 0};
            if (live) fq[s] = load16<T>(qrow, s * KST + g * E, a.q.dim, a.q.vec);
        }
        __syncthreads();
        const bool more = c0 + kChunk < n;
        if (more) {
            const int m2 = min(kChunk, n - c0 - kChunk);
            sk.load(a.k, a, p, h, t0 + c0 + kChunk, m2, tid);
            sv.load(a.v, a, p, h, t0 + c0 + kChunk, m2, tid);
        }
        const bool odd = nonfin[par] != 0;
        if (tid == 0) nonfin[par ^ 1] = 0;

        // the state's answer
        const bool lead = p.s == 0 && c0 == 0;
        f4 O[OT];
#pragma unroll
        for (int t = 0; t < OT; ++t) {
            O[t] = f4{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < QS; ++s) O[t] = mma<T>(frag_cols<T>(St, SP, t * 16, s * KST, lane), fq[s], O[t]);
        }
        const float rd = a.iscale * pw[qi + (lead ? a.e0 : 1)];
#pragma unroll
        for (int t = 0; t < OT; ++t) O[t] *= rd;

        // the chunk's own tokens, up to the query
#pragma unroll
        for (int ks = 0; ks < kChunk / KST; ++ks) {
            if (ks * TPK > wave) break;
            f4 P[TPK];
#pragma unroll
            for (int u = 0; u < TPK; ++u) {
                const int jt = ks * TPK + u;
                P[u] = f4{0, 0, 0, 0};
                if (jt > wave) continue;
#pragma unroll
                for (int s = 0; s < QS; ++s) P[u] = mma<T>(frag_cols<T>(Ks, SK::kPitch, jt * 16, s * KST, lane), fq[s], P[u]);
                if (jt == wave) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) P[u][r] = li >= 4 * g + r ? P[u][r] * wdiag[r] : 0.f;
                } else {
                    const int far = wave - jt - 1;
                    const float f = far == 0 ? 1.f : far == 1 ? p16 : p32;
#pragma unroll
                    for (int r = 0; r < 4; ++r) P[u][r] *= woff[r] * f;
                }
            }
            u4 fp;
            if constexpr (sizeof(T) == 2) {
                const u2 lo = pack4(P[0]), hi = pack4(P[1]);
                fp = u4{lo[0], lo[1], hi[0], hi[1]};
            } else {
                fp = __builtin_bit_cast(u4, P[0]);
            }
#pragma unroll
            for (int t = 0; t < OT; ++t) {
                u4 fv = frag_rows(Vs, SV::kPitch, ks * KST, t * 16, lane);
                // masked weights are 0, and 0 x infinity is a NaN: such values are
                // kept out of the product and added by themselves below
                if (odd) fv = drop_nonfinite<T>(fv);
                O[t] = mma<T>(fv, fp, O[t]);
            }
        }
        if (odd && live) {
#pragma unroll 1
            for (int j = 0; j <= qi; ++j) {
                const T* krow = Ks + j * SK::kPitch;
                float dot = 0.f;
#pragma unroll 1
                for (int d = 0; d < a.k.dim; ++d) dot += (float)qrow[d] * (float)krow[d];
                dot *= a.pscale * pw[qi - j];
#pragma unroll
                for (int t = 0; t < OT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const T v = Vs[j * SV::kPitch + t * 16 + 4 * g + r];
                        if (!finite_bits<T>(v)) O[t][r] += dot * (float)v;
                    }
            }
        }

        if (live) {
            const int64_t tok = p.start + (a.reverse ? p.len - 1 - (t0 + c0 + qi) : t0 + c0 + qi);
            const int64_t at = (a.cu ? 0 : (int64_t)p.n * a.out_seq) + tok * a.out_tok + (int64_t)h * a.out_head;
            const bool quads = (a.dv & 3) == 0;  // dense rows: quads of outputs are aligned
#pragma unroll
            for (int t = 0; t < OT; ++t) {
                const int col = t * 16 + 4 * g;
                if (a.out_f32 || sizeof(T) == 4) {
                    float* o = (float*)a.out + at + col;
                    if (quads) {
                        if (col < a.dv) *(f4*)o = O[t];
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (col + r < a.dv) o[r] = O[t][r];
                    }
                } else {
                    T* o = (T*)a.out + at + col;
                    if (quads) {
                        if (col < a.dv) *(u2*)o = pack4(O[t]);
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (col + r < a.dv) o[r] = (T)O[t][r];
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
            for (int ks = 0; ks < kChunk; ks += KST) {
                float w[8];
                row_weights<T>(wt, ks, lane, w);
                u4 fv[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    weighted<T, 1>(frag_rows(Vs, SV::kPitch, ks, (wave * CT + c) * 16, lane), w, &fv[c]);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const u4 fk = frag_rows(Ks, SK::kPitch, ks, r * 16, lane);
#pragma unroll
                    for (int c = 0; c < CT; ++c) S[r][c] = mma<T>(fk, fv[c], S[r][c]);
                }
            }
        }
    }
}

// ---- gradients of shared heads ---------------------------------------------------
//
// out[row][kh][d] = sum over the rep heads that share kh, in order, of the
// float32 gradients part[row][kh rep + i][d].
template <typename T>
__global__ __launch_bounds__(kThreads) void sum_heads(const float* part, T* out, int64_t count, int rep, int d)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= count) return;
    const int64_t row = i / d;
    const float* q = part + row * rep * d + i % d;
    float s = q[0];
    for (int r = 1; r < rep; ++r) s += q[(int64_t)r * d];
    out[i] = (T)s;
}

// ---- one token --------------------------------------------------------------------
//
// A workgroup updates CW columns of one head's state: each thread reads its
// pieces of the state (all in flight at once), adds k v^T, writes them back
// and keeps q_row x S; the rows' partial answers meet in LDS. Bound by the
// state's traffic, 8 dk dv bytes a head.
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
// (both fit: 70 KB of LDS each), and a segment is whole chunks.
int make_plan(const gconv_linattn_desc* d, Plan* p)
{
    p->rows = d->packed ? d->tokens : d->sequences * d->tokens;
    const int64_t per_head = std::max<int64_t>(1, 512 / d->heads);
    const int64_t seg = (p->rows + per_head - 1) / per_head;
    p->seg = (int)std::max<int64_t>(kChunk, (seg + kChunk - 1) / kChunk * kChunk);
    p->slots_per_seq = (int)((d->tokens + p->seg - 1) / p->seg);
    const int64_t slots = d->packed ? d->tokens / p->seg + d->sequences : d->sequences * p->slots_per_seq;
    if (slots * d->heads > kMaxTokens) return fail(GCONV_ERR_UNSUPPORTED, "too many sequences x heads");
    p->slots = (int)slots;
    p->DK = pad64(d->dk);
    p->DV = pad64(d->dv);
    p->state_elems = slots * d->heads * p->DK * p->DV;
    return GCONV_OK;
}

Operand operand(const void* p, const int64_t* stride, int hdiv, int64_t dim, int64_t es)
{
    Operand o{p, stride[0], stride[1], stride[2], hdiv, (int)dim, 0};
    o.vec = ((uintptr_t)p & 15) == 0 && stride[0] * es % 16 == 0 && stride[1] * es % 16 == 0 && stride[2] * es % 16 == 0 &&
            dim * es % 16 == 0;
    return o;
}

template <typename T, int DK, int DV>
void launch_states(const Pass& a, hipStream_t st)
{
    if (a.slots > 0) segment_sums<T, DK, DV><<<a.slots * a.heads, kThreads, 0, st>>>(a);
    if (a.sequences > 0)
        scan_states<DK, DV><<<a.sequences * a.heads * (DK * DV / 4 / kThreads), kThreads, 0, st>>>(a);
}

template <typename T>
void states(const Pass& a, int DK, int DV, hipStream_t st)
{
    if (DK == 64 && DV == 64) launch_states<T, 64, 64>(a, st);
    else if (DK == 64) launch_states<T, 64, 128>(a, st);
    else if (DV == 64) launch_states<T, 128, 64>(a, st);
    else launch_states<T, 128, 128>(a, st);
}

template <typename T>
void outputs(const Pass& a, int DK, int DV, hipStream_t st)
{
    const int grid = a.slots * a.heads;
    if (grid == 0) return;
    if (DK == 64 && DV == 64) chunk_outputs<T, 64, 64><<<grid, kThreads, 0, st>>>(a);
    else if (DK == 64) chunk_outputs<T, 64, 128><<<grid, kThreads, 0, st>>>(a);
    else if (DV == 64) chunk_outputs<T, 128, 64><<<grid, kThreads, 0, st>>>(a);
    else chunk_outputs<T, 128, 128><<<grid, kThreads, 0, st>>>(a);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

size_t workspace_bytes(const gconv_linattn_desc* d, const Plan& p, int op)
{
    const size_t one = up256((size_t)p.state_elems * 4);
    if (op == GCONV_LINATTN_FWD) return one;
    // float32 gradients of each q head where heads share k and v
    const size_t part = d->heads != d->kv_heads ? up256((size_t)p.rows * d->heads * (d->dk + d->dv) * 4) : 0;
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
    float* part_dv = part ? part + p.rows * d->heads * d->dk : nullptr;
    Pass v = r;
    v.q = a.k;
    dense_out(&v, part ? part_dv : dv, d->heads, d->dv);
    outputs<T>(v, p.DK, p.DV, st);
    Pass k = r;
    k.q = a.v;
    k.k = dout;
    k.v = a.q;
    k.dk = a.dv;
    k.dv = a.dk;
    k.state_t = 1;
    dense_out(&k, part ? part : dk, d->heads, d->dk);
    outputs<T>(k, p.DV, p.DK, st);
    if (part && p.rows > 0) {
        const int64_t nk = p.rows * d->kv_heads * d->dk, nv = p.rows * d->kv_heads * d->dv;
        sum_heads<T><<<(unsigned)((nk + kThreads - 1) / kThreads), kThreads, 0, st>>>(part, (T*)dk, nk, rep, (int)d->dk);
        sum_heads<T><<<(unsigned)((nv + kThreads - 1) / kThreads), kThreads, 0, st>>>(part_dv, (T*)dv, nv, rep, (int)d->dv);
    }
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
    st = make_plan(d, &p);
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
    st = make_plan(d, p);
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
    a->q = operand(q, d->q_stride, 1, d->dk, es);
    a->k = operand(k, d->k_stride, rep, d->dk, es);
    a->v = operand(v, d->v_stride, rep, d->dv, es);
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
    const Operand od = operand(dout, d->do_stride, 1, d->dv, es);
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
    hipStream_t hs = (hipStream_t)stream;
    (void)hipGetLastError();
    if (d->sequences == 0) return finish();
    Step a{};
    const int rep = (int)(d->heads / d->kv_heads);
    a.q = operand(q, d->q_stride, 1, d->dk, es);
    a.k = operand(k, d->k_stride, rep, d->dk, es);
    a.v = operand(v, d->v_stride, rep, d->dv, es);
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
    const int64_t bh = d->sequences * d->heads;
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
