// normgate.hip -- the norms before and after a block, its gate and its residual
// scale, fused (gfx950).
//
//   y = x + scale * act(gate) * (b * rb * w_post),   rb = (mean b^2 + eps)^-1/2
//   h = y * ry * w_pre,                              ry = (mean y^2 + eps)^-1/2
//
// A row is held in registers from its one read to its one write: TPR threads a
// row (4 to 1024: 962626 rows of 32 took 783 us, forward and backward, by 16
// threads each, 200 by 4 and 164 without branches), eight elements (VPT 16-byte
// pieces) a thread, so both norms and every product cost no second pass.
// Workgroups walk over rows with the weights in registers. What bounds it is HBM:
// (b, gate, x in; y, h out) forward, at the copy rate (16384 rows of 4096: 125
// us, 5.3 TB/s), and the same with their gradients backward, where the sums over
// rows and up to five tensors' values leave few waves a SIMD (262144 rows of 128:
// 70 us, 4.8 TB/s; 16384 of 4096: 281 us, 3.9 TB/s). Above 4096 columns 1024
// threads leave 128 registers each and 16 to 129 values spill (4000 of 8000: 235
// us, in which 1.0 GB pass for the 0.5 that are needed). Tried and dropped:
// loading the next row ahead (forward 127 -> 147 us: fewer waves), reading past
// odd rows' ends and masking (76 -> 102 us).
//
// Backward, with e = dh w_pre and yn = y ry:
//   dy' = dy + ry (e - yn mean(e yn))                          dx = dy'
//   db  = rb (f - bn mean(f bn)),  f = dy' scale a w_post, bn = b rb
//   dgate = dy' scale n a'(gate),  n = bn w_post
// and the sums over rows dw_post = S dy' scale a bn, dscale = S dy' a n,
// dw_pre = S dh yn: float32 sums in registers for a workgroup's rows, then over
// the workgroups in order, so results are the same every time.
#include <algorithm>

#include "gconv.h"
#include "gconv_internal.h"
#include "seq_util.h"

namespace gconv {
namespace {

constexpr int kPerThread = 8;  // elements of a row a thread holds

struct Rows {
    const void* p;      // NULL: absent
    int64_t seq, tok;   // strides in elements
};

struct Norm {
    Rows x, b, gate, dy, dh;
    const void *w_post, *scale, *w_pre;
    void *y, *h, *dx, *db, *dgate;   // dense [sequences][tokens][dim] (dgate: [sequences][dim] where a gate is a sequence's)
    float* part;        // [blocks][3][dim] sums over rows; then [blocks][dim] of a sequence's gate
    float* gate_part;   // NULL: a workgroup sees whole sequences and writes dgate itself
    int64_t tokens, rows;
    int groups;         // of rows that one workgroup never mixes: sequences (with a gate each), or 1
    int splits;         // workgroups of a group, or 1 with `groups` spread over the grid
    int64_t group_rows;
    int dim, act, gate_seq;
    int flat;           // rows follow one another at their token strides: the sequence is not asked for
    float eps, inv_dim;
};

// 16 bytes at any element boundary; past the row's end element by element.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Loose {
    u4 v;
};

template <typename T>
__device__ __forceinline__ u4 load_loose(const T* row, int col, int dim)
{
    constexpr int E = 16 / sizeof(T);
    if (col + E <= dim) return ((const Loose<T>*)(row + col))->v;
    T e[E];
#pragma unroll
    for (int i = 0; i < E; ++i) e[i] = col + i < dim ? row[col + i] : (T)0.f;
    return __builtin_bit_cast(u4, e);
}

// Pieces of ones.
template <typename T>
__device__ __forceinline__ u4 ones()
{
    constexpr uint32_t one = sizeof(T) == 2 ? 0x3f803f80u : 0x3f800000u;
    return u4{one, one, one, one};
}

template <typename T>
struct Vals {
    static constexpr int E = 16 / sizeof(T);
    float v[E];
    __device__ __forceinline__ Vals() {}
    __device__ __forceinline__ explicit Vals(u4 raw)
    {
        struct Pack { T e[E]; } p = __builtin_bit_cast(Pack, raw);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = (float)p.e[i];
    }
    __device__ __forceinline__ void store(T* row, int col, int dim) const
    {
        struct Pack { T e[E]; } p;
#pragma unroll
        for (int i = 0; i < E; ++i) p.e[i] = (T)v[i];
        if (col + E <= dim) {
            ((Loose<T>*)(row + col))->v = __builtin_bit_cast(u4, p);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (col + i < dim) row[col + i] = p.e[i];
        }
    }
};

__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// act(z).
__device__ __forceinline__ float act_of(float z, int act)
{
    return act == GCONV_ACT_NONE ? z : act == GCONV_ACT_SIGMOID ? sigmoid(z) : z * sigmoid(z);
}

// Sum over the TPR threads of a row, the same in all of them. `red`: one float
// a wave; every call of a kernel alternates between two of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red, int wave)
{
    constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
    for (int m = W / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[wave] = v;
        __syncthreads();
        float s = 0.f;
        const int first = wave & ~(TPR / 64 - 1);
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) s += red[first + i];
        v = s;
    }
    return v;
}

template <typename T>
__device__ __forceinline__ const T* row_ptr(const Rows& r, int64_t n, int64_t t)
{
    return (const T*)r.p + n * r.seq + t * r.tok;
}

// Row r's sequence and its token in that. (A 64-bit division costs more than
// the rest of a short row.)
__device__ __forceinline__ void place_of(const Norm& a, int64_t r, int64_t* n, int64_t* t)
{
    *n = 0;
    *t = r;
    if (a.flat) return;
    *n = a.rows <= 0x7fffffff ? (int64_t)((uint32_t)r / (uint32_t)a.tokens) : r / a.tokens;
    *t = r - *n * a.tokens;
}

template <typename T, int TPR>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_fwd(Norm a)
{
    constexpr int E = 16 / sizeof(T), VPT = kPerThread / E, NT = TPR > 256 ? TPR : 256, RPB = NT / TPR;
    __shared__ float red[2][NT / 64];
    const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR, wave = threadIdx.x >> 6;
    u4 wp[VPT], sc[VPT], wq[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int col = (i * TPR + lane) * E;
        wp[i] = load_loose((const T*)a.w_post, col, a.dim);
        if (a.scale) sc[i] = load_loose((const T*)a.scale, col, a.dim);
        if (a.w_pre) wq[i] = load_loose((const T*)a.w_pre, col, a.dim);
    }
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB) {
        const bool live = r0 + sub < a.rows;
        const int64_t r = live ? r0 + sub : r0;
        int64_t n, t;
        place_of(a, r, &n, &t);
        u4 rb_[VPT], rg[VPT], rx[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (i * TPR + lane) * E;
            rb_[i] = load_loose(row_ptr<T>(a.b, n, t), col, a.dim);
            if (a.gate.p) rg[i] = load_loose(row_ptr<T>(a.gate, n, t), col, a.dim);
            if (a.x.p) rx[i] = load_loose(row_ptr<T>(a.x, n, t), col, a.dim);
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const Vals<T> b(rb_[i]);
#pragma unroll
            for (int e = 0; e < E; ++e) ss = fmaf(b.v[e], b.v[e], ss);
        }
        const float rb = rsqrtf(row_sum<TPR>(ss, red[0], wave) * a.inv_dim + a.eps);
        Vals<T> y[VPT];
        float sy = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (i * TPR + lane) * E;
            const Vals<T> b(rb_[i]), wpv(wp[i]);
            Vals<T> g, x, scv;
            if (a.scale) scv = Vals<T>(sc[i]);
            if (a.gate.p) g = Vals<T>(rg[i]);
            if (a.x.p) x = Vals<T>(rx[i]);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float v = b.v[e] * rb * wpv.v[e];
                if (a.gate.p) v *= act_of(g.v[e], a.act);
                if (a.scale) v *= scv.v[e];
                if (a.x.p) v += x.v[e];
                // columns past the row hold 0 x act(0): 0 but for a gate of NaN bits, which load as 0
                y[i].v[e] = v;
                sy = fmaf(v, v, sy);
            }
            if (live) y[i].store((T*)a.y + r * a.dim, col, a.dim);
        }
        if (a.h) {
            const float ry = rsqrtf(row_sum<TPR>(sy, red[1], wave) * a.inv_dim + a.eps);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const Vals<T> wqv(wq[i]);
#pragma unroll
                for (int e = 0; e < E; ++e) y[i].v[e] *= ry * wqv.v[e];
                if (live) y[i].store((T*)a.h + r * a.dim, (i * TPR + lane) * E, a.dim);
            }
        } else if (TPR > 64) {
            __syncthreads();  // red[0] is written again by the next row
        }
    }
}

// Keeps the weights in registers as they were loaded: converted outside the
// loop over rows they would take up twice as many. Where 1024 threads leave 128
// registers each (4000 rows of 8000, forward and backward: 346 us for 409;
// shorter rows lose some 2%).
constexpr int kTight = 1024;
template <int N>
__device__ __forceinline__ void keep_raw(u4 (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(v[i]));
}

// One workgroup: the rows split, split + splits, ... of a group, or (splits ==
// 1) whole groups, a stretch of them.
template <typename T, int TPR, bool PRE, bool GSEQ>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_bwd(Norm a)
{
    constexpr int E = 16 / sizeof(T), VPT = kPerThread / E, NT = TPR > 256 ? TPR : 256, RPB = NT / TPR;
    __shared__ float red[2][NT / 64];
    __shared__ float col_red[RPB > 1 ? NT * E : 1];
    const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR, wave = threadIdx.x >> 6;
    u4 wp[VPT], sc[VPT], wq[VPT];
    float s_post[VPT][E], s_scale[VPT][E], s_pre[VPT][E], s_gate[VPT][E];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int col = (i * TPR + lane) * E;
        wp[i] = load_loose((const T*)a.w_post, col, a.dim);
        sc[i] = a.scale ? load_loose((const T*)a.scale, col, a.dim) : ones<T>();
        if (PRE) wq[i] = load_loose((const T*)a.w_pre, col, a.dim);
#pragma unroll
        for (int e = 0; e < E; ++e) s_post[i][e] = s_scale[i][e] = s_pre[i][e] = s_gate[i][e] = 0.f;
    }
    // Adds a thread's column sums over the workgroup's row slots, in order, and
    // hands the total of each column to `put`.
    auto columns = [&](const float (&s)[VPT][E], auto put) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (i * TPR + lane) * E;
            if constexpr (RPB > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < E; ++e) col_red[threadIdx.x * E + e] = s[i][e];
                __syncthreads();
                if (sub == 0) {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        float v = 0.f;
                        for (int q = 0; q < RPB; ++q) v += col_red[(q * TPR + lane) * E + e];
                        if (col + e < a.dim) put(col + e, v);
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (col + e < a.dim) put(col + e, s[i][e]);
            }
        }
    };

    int g0, g1, split;
    if (a.splits > 1) {
        g0 = blockIdx.x / a.splits;
        g1 = g0 + 1;
        split = blockIdx.x % a.splits;
    } else {
        g0 = (int)((int64_t)blockIdx.x * a.groups / gridDim.x);
        g1 = (int)((int64_t)(blockIdx.x + 1) * a.groups / gridDim.x);
        split = 0;
    }
    for (int g = g0; g < g1; ++g) {
        for (int64_t q0 = (int64_t)split * RPB; q0 < a.group_rows; q0 += (int64_t)a.splits * RPB) {
            const bool live = q0 + sub < a.group_rows;
            const int64_t r = (int64_t)g * a.group_rows + (live ? q0 + sub : q0);
            int64_t n = g, t = r - (int64_t)g * a.group_rows;
            if (!GSEQ) place_of(a, r, &n, &t);
            // What is absent counts as what leaves the formulas as they are (a gate
            // of ones, x = 0), and a row past the last has no gradient, so nothing
            // below has a branch for it.
            u4 rb_[VPT], rg[VPT], rx[VPT], rdy[VPT], rdh[VPT];
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int col = (i * TPR + lane) * E;
                rb_[i] = load_loose(row_ptr<T>(a.b, n, t), col, a.dim);
                rg[i] = a.gate.p ? load_loose(row_ptr<T>(a.gate, n, t), col, a.dim) : ones<T>();
                rdy[i] = load_loose(row_ptr<T>(a.dy, n, t), col, a.dim);
                if constexpr (PRE) {
                    rx[i] = a.x.p ? load_loose(row_ptr<T>(a.x, n, t), col, a.dim) : u4{0, 0, 0, 0};
                    rdh[i] = load_loose(row_ptr<T>(a.dh, n, t), col, a.dim);
                }
            }
            if constexpr (TPR >= kTight) {
                keep_raw(wp);
                keep_raw(sc);
                if (PRE) keep_raw(wq);
            }
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const Vals<T> b(rb_[i]);
#pragma unroll
                for (int e = 0; e < E; ++e) ss = fmaf(b.v[e], b.v[e], ss);
            }
            const float rb = rsqrtf(row_sum<TPR>(ss, red[0], wave) * a.inv_dim + a.eps);
            // the gate's sigmoid, 1 where the activation has none: act(z) is it times z (or 1)
            float sg[VPT][E];
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) sg[i][e] = 1.f;
            if (a.act != GCONV_ACT_NONE) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const Vals<T> z(rg[i]);
#pragma unroll
                    for (int e = 0; e < E; ++e) sg[i][e] = sigmoid(z.v[e]);
                }
            }
            const bool plain = a.act == GCONV_ACT_SIGMOID;
            float ry = 0.f, m1 = 0.f;
            Vals<T> y[VPT];
            if constexpr (PRE) {
                float sy = 0.f, se = 0.f;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    if (!live) rdy[i] = rdh[i] = u4{0, 0, 0, 0};
                    const Vals<T> b(rb_[i]), dh(rdh[i]), wpv(wp[i]), wqv(wq[i]), z(rg[i]), x(rx[i]), scv(sc[i]);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float av = sg[i][e] * (plain ? 1.f : z.v[e]);
                        y[i].v[e] = fmaf(b.v[e] * rb * wpv.v[e] * av, scv.v[e], x.v[e]);
                        sy = fmaf(y[i].v[e], y[i].v[e], sy);
                        se = fmaf(dh.v[e] * wqv.v[e], y[i].v[e], se);
                    }
                }
                ry = rsqrtf(row_sum<TPR>(sy, red[1], wave) * a.inv_dim + a.eps);
                m1 = row_sum<TPR>(se, red[0], wave) * a.inv_dim * ry;
            }
            // dy' and what follows from it; f (for db) is kept for the last reduction
            Vals<T> f[VPT];
            float sf = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int col = (i * TPR + lane) * E;
                if (!PRE && !live) rdy[i] = u4{0, 0, 0, 0};
                const Vals<T> b(rb_[i]), wpv(wp[i]), z(rg[i]), scv(sc[i]);
                Vals<T> dyv(rdy[i]), dz, dh, wqv;
                if constexpr (PRE) {
                    dh = Vals<T>(rdh[i]);
                    wqv = Vals<T>(wq[i]);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float zz = plain ? 1.f : z.v[e], sig = sg[i][e], av = sig * zz;
                    const float da = a.act == GCONV_ACT_NONE ? 1.f : fmaf(zz, sig * (1.f - sig), plain ? 0.f : sig);
                    const float bn = b.v[e] * rb, nn = bn * wpv.v[e];
                    float d = dyv.v[e];
                    if constexpr (PRE) {
                        const float yn = y[i].v[e] * ry;
                        d += ry * (dh.v[e] * wqv.v[e] - yn * m1);
                        s_pre[i][e] = fmaf(dh.v[e], yn, s_pre[i][e]);
                    }
                    dyv.v[e] = d;
                    const float du = d * scv.v[e];
                    s_post[i][e] = fmaf(du * av, bn, s_post[i][e]);
                    s_scale[i][e] = fmaf(d * av, nn, s_scale[i][e]);
                    dz.v[e] = du * nn * da;
                    if (GSEQ) s_gate[i][e] += dz.v[e];
                    f[i].v[e] = du * av * wpv.v[e];
                    sf = fmaf(f[i].v[e], bn, sf);
                }
                if (live) {
                    if (a.dx) dyv.store((T*)a.dx + r * a.dim, col, a.dim);
                    if (!GSEQ && a.dgate) dz.store((T*)a.dgate + r * a.dim, col, a.dim);
                }
            }
            const float m2 = row_sum<TPR>(sf, red[1], wave) * a.inv_dim;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const Vals<T> b(rb_[i]);
#pragma unroll
                for (int e = 0; e < E; ++e) f[i].v[e] = rb * (f[i].v[e] - b.v[e] * rb * m2);
                if (live) f[i].store((T*)a.db + r * a.dim, (i * TPR + lane) * E, a.dim);
            }
        }
        if constexpr (GSEQ) {
            if (a.gate_part) {
                float* p = a.gate_part + (int64_t)blockIdx.x * a.dim;
                columns(s_gate, [&](int col, float v) { p[col] = v; });
            } else {
                T* p = (T*)a.dgate + (int64_t)g * a.dim;
                columns(s_gate, [&](int col, float v) { p[col] = (T)v; });
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) s_gate[i][e] = 0.f;
        }
    }
    float* p = a.part + (int64_t)blockIdx.x * 3 * a.dim;
    columns(s_post, [&](int col, float v) { p[col] = v; });
    if (a.scale) columns(s_scale, [&](int col, float v) { p[a.dim + col] = v; });
    if constexpr (PRE) columns(s_pre, [&](int col, float v) { p[2 * a.dim + col] = v; });
}

// out[which][col] = sum over `count` partial rows, in an order fixed by the
// shape: 64 columns a workgroup, 16 slices of the rows, then the slices. The
// first layer of the grid folds the weights' gradients, the others those of
// the sequences' gates.
template <typename T>
struct Fold {
    const float* part;
    int64_t stride, group_stride;  // between partial rows, between a group's first rows
    int count, dim;
    T* out[3];
};

template <typename T>
__global__ __launch_bounds__(1024) void fold_rows(Fold<T> weights, Fold<T> gates)
{
    __shared__ float red[16][65];
    const int c = threadIdx.x & 63, slice = threadIdx.x >> 6;
    const int col = blockIdx.x * 64 + c, which = blockIdx.y;
    const Fold<T>& a = blockIdx.z == 0 ? weights : gates;
    const int group = blockIdx.z == 0 ? 0 : blockIdx.z - 1;
    T* out = which == 0 ? a.out[0] : which == 1 ? a.out[1] : a.out[2];
    if (!out) return;
    const float* p = a.part + group * a.group_stride + (int64_t)which * a.dim + col;
    float s = 0.f;
    if (col < a.dim) {
        int i = slice;
        for (; i + 48 < a.count; i += 64) {
            const float v0 = p[i * a.stride], v1 = p[(i + 16) * a.stride], v2 = p[(i + 32) * a.stride], v3 = p[(i + 48) * a.stride];
            s += v0; s += v1; s += v2; s += v3;
        }
        for (; i < a.count; i += 16) s += p[i * a.stride];
    }
    red[slice][c] = s;
    __syncthreads();
    if (slice == 0 && col < a.dim) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) v += red[k][c];
        out[(int64_t)group * a.dim + col] = (T)v;
    }
}

// ---- host ------------------------------------------------------------------------

constexpr int64_t kMaxDim = 1024 * kPerThread;
constexpr int64_t kMaxRows = (int64_t)1 << 40;

int check_desc(const gconv_normgate_desc* d)
{
    if (!d) return fail(GCONV_ERR_NULL, "descriptor is NULL");
    if (d->dtype != GCONV_F32 && d->dtype != GCONV_BF16) return fail(GCONV_ERR_ARG, "unknown dtype %lld", (long long)d->dtype);
    if (d->gate < GCONV_GATE_NONE || d->gate > GCONV_GATE_SEQUENCE) return fail(GCONV_ERR_ARG, "unknown gate %lld", (long long)d->gate);
    if (d->act < GCONV_ACT_NONE || d->act > GCONV_ACT_SILU) return fail(GCONV_ERR_ARG, "unknown activation %lld", (long long)d->act);
    if (d->sequences < 0 || d->tokens < 0 || d->dim < 1)
        return fail(GCONV_ERR_SHAPE, "need sequences, tokens >= 0 and dim >= 1 (got %lld, %lld, %lld)", (long long)d->sequences,
                    (long long)d->tokens, (long long)d->dim);
    if (d->dim > kMaxDim) return fail(GCONV_ERR_UNSUPPORTED, "dim=%lld above %lld", (long long)d->dim, (long long)kMaxDim);
    if (d->sequences > ((int64_t)1 << 30) || d->tokens > ((int64_t)1 << 30) ||
        (d->tokens > 0 && d->sequences > kMaxRows / d->tokens))
        return fail(GCONV_ERR_UNSUPPORTED, "too many rows");
    if (!(d->eps >= 0)) return fail(GCONV_ERR_ARG, "eps must be >= 0");
    return GCONV_OK;
}

// Threads a row: the power of two that holds it at eight elements each.
int row_threads(const gconv_normgate_desc* d)
{
    int tpr = 4;
    while (tpr * kPerThread < d->dim) tpr *= 2;
    return tpr;
}

struct Grid {
    int blocks, groups, splits;
    int64_t group_rows;
    size_t part, gate_part;  // bytes
};

Grid bwd_grid(const gconv_normgate_desc* d)
{
    const int tpr = row_threads(d);
    const int rpb = tpr < 256 ? 256 / tpr : 1;
    const int64_t want = tpr == 1024 ? 256 : 512;  // workgroups: about what fits at once
    Grid g{};
    const bool seq = d->gate == GCONV_GATE_SEQUENCE;
    g.groups = seq ? (int)d->sequences : 1;
    g.group_rows = seq ? d->tokens : d->sequences * d->tokens;
    if (g.groups >= want) {
        g.splits = 1;
        g.blocks = (int)want;
    } else {
        g.splits = (int)std::max<int64_t>(1, std::min(want / std::max(g.groups, 1), (g.group_rows + rpb - 1) / rpb));
        g.blocks = g.groups * g.splits;
    }
    g.part = ((size_t)g.blocks * 3 * d->dim * 4 + 255) / 256 * 256;
    g.gate_part = seq && g.splits > 1 ? (size_t)g.blocks * d->dim * 4 : 0;
    return g;
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

Range span(const void* p, const gconv_normgate_desc* d, const int64_t* s, bool seq)
{
    if (d->sequences == 0 || d->tokens == 0) return Range{p, 0};
    const int64_t last = (d->sequences - 1) * std::max<int64_t>(s[0], 0) + (seq ? 0 : (d->tokens - 1) * std::max<int64_t>(s[1], 0)) + d->dim;
    return Range{p, last * (d->dtype == GCONV_BF16 ? 2 : 4)};
}

template <typename T, int TPR>
void launch_row(const Norm& a, bool bwd, int blocks, hipStream_t st)
{
    constexpr int NT = TPR > 256 ? TPR : 256;
    if (!bwd) norm_fwd<T, TPR><<<blocks, NT, 0, st>>>(a);
    else if (a.w_pre && a.gate_seq) norm_bwd<T, TPR, true, true><<<blocks, NT, 0, st>>>(a);
    else if (a.w_pre) norm_bwd<T, TPR, true, false><<<blocks, NT, 0, st>>>(a);
    else if (a.gate_seq) norm_bwd<T, TPR, false, true><<<blocks, NT, 0, st>>>(a);
    else norm_bwd<T, TPR, false, false><<<blocks, NT, 0, st>>>(a);
}

template <typename T>
void launch(const Norm& a, int tpr, bool bwd, int blocks, hipStream_t st)
{
    switch (tpr) {
        case 4: launch_row<T, 4>(a, bwd, blocks, st); break;
        case 8: launch_row<T, 8>(a, bwd, blocks, st); break;
        case 16: launch_row<T, 16>(a, bwd, blocks, st); break;
        case 32: launch_row<T, 32>(a, bwd, blocks, st); break;
        case 64: launch_row<T, 64>(a, bwd, blocks, st); break;
        case 128: launch_row<T, 128>(a, bwd, blocks, st); break;
        case 256: launch_row<T, 256>(a, bwd, blocks, st); break;
        case 512: launch_row<T, 512>(a, bwd, blocks, st); break;
        default: launch_row<T, 1024>(a, bwd, blocks, st); break;
    }
}

template <typename T>
void run_bwd(const gconv_normgate_desc* d, const Norm& a, const Grid& g, void* dw_post, void* dscale, void* dw_pre, hipStream_t st)
{
    const int tpr = row_threads(d);
    if (g.blocks > 0) launch<T>(a, tpr, true, g.blocks, st);
    Fold<T> f{a.part, (int64_t)3 * d->dim, 0, g.blocks, (int)d->dim, {(T*)dw_post, (T*)dscale, (T*)dw_pre}};
    const unsigned cols = (unsigned)((d->dim + 63) / 64);
    Fold<T> s{};
    if (a.gate_part)
        s = Fold<T>{a.gate_part, d->dim, (int64_t)g.splits * d->dim, g.splits, (int)d->dim, {(T*)a.dgate, nullptr, nullptr}};
    fold_rows<T><<<dim3(cols, 3, a.gate_part ? 1 + (unsigned)g.groups : 1), 1024, 0, st>>>(f, s);
}

bool follow(const gconv_normgate_desc* d, const Rows& r)
{
    return !r.p || d->sequences == 1 || r.seq == d->tokens * r.tok;
}

void fill(const gconv_normgate_desc* d, Norm* a)
{
    a->flat = follow(d, a->x) && follow(d, a->b) && follow(d, a->gate) && follow(d, a->dy) && follow(d, a->dh);
    a->tokens = std::max<int64_t>(d->tokens, 1);
    a->rows = d->sequences * d->tokens;
    a->dim = (int)d->dim;
    a->act = d->gate == GCONV_GATE_NONE ? GCONV_ACT_NONE : (int)d->act;
    a->gate_seq = d->gate == GCONV_GATE_SEQUENCE;
    a->eps = (float)d->eps;
    a->inv_dim = 1.f / (float)d->dim;
}

}  // namespace
}  // namespace gconv

using namespace gconv;

extern "C" {

int gconv_normgate_workspace_size(const gconv_normgate_desc* d, size_t* bytes)
{
    const int st = check_desc(d);
    if (st != GCONV_OK) return st;
    if (!bytes) return fail(GCONV_ERR_NULL, "bytes pointer is NULL");
    const Grid g = bwd_grid(d);
    *bytes = g.part + g.gate_part;
    return GCONV_OK;
}

int gconv_normgate_fwd(const gconv_normgate_desc* d, const void* x, const void* b, const void* gate, const void* w_post,
                       const void* scale, const void* w_pre, void* y, void* h, void* stream)
{
    const int st = check_desc(d);
    if (st != GCONV_OK) return st;
    const int64_t rows = d->sequences * d->tokens, es = d->dtype == GCONV_BF16 ? 2 : 4;
    if (!w_post || (rows > 0 && (!b || !y))) return fail(GCONV_ERR_NULL, "b, w_post and y must be non-NULL");
    if ((d->gate != GCONV_GATE_NONE) != (gate != nullptr) && rows > 0)
        return fail(GCONV_ERR_NULL, "gate must be given unless there is none");
    if ((w_pre != nullptr) != (h != nullptr) && rows > 0) return fail(GCONV_ERR_NULL, "w_pre and h go together");
    const Range in[] = {span(x, d, d->x_stride, false), span(b, d, d->b_stride, false),
                        span(gate, d, d->gate_stride, d->gate == GCONV_GATE_SEQUENCE), {w_post, d->dim * es},
                        {scale, d->dim * es}, {w_pre, d->dim * es}};
    const Range out[] = {{y, rows * d->dim * es}, {h, rows * d->dim * es}};
    for (const Range& w : out)
        for (const Range& r : in)
            if (meets(w, r)) return fail(GCONV_ERR_ARG, "y or h overlaps an input");
    if (meets(out[0], out[1])) return fail(GCONV_ERR_ARG, "y overlaps h");
    hipStream_t hs = (hipStream_t)stream;
    (void)hipGetLastError();
    if (rows == 0) return finish();
    Norm a{};
    a.x = Rows{x, d->x_stride[0], d->x_stride[1]};
    a.b = Rows{b, d->b_stride[0], d->b_stride[1]};
    a.gate = Rows{gate, d->gate_stride[0], d->gate == GCONV_GATE_SEQUENCE ? 0 : d->gate_stride[1]};
    fill(d, &a);
    a.w_post = w_post;
    a.scale = scale;
    a.w_pre = w_pre;
    a.y = y;
    a.h = h;
    const int tpr = row_threads(d);
    const int64_t rpb = tpr < 256 ? 256 / tpr : 1;
    const int blocks = (int)std::min<int64_t>((rows + rpb - 1) / rpb, 2048);
    if (d->dtype == GCONV_BF16) launch<__bf16>(a, tpr, false, blocks, hs);
    else launch<float>(a, tpr, false, blocks, hs);
    return finish();
}

int gconv_normgate_bwd(const gconv_normgate_desc* d, const void* dy, const void* dh, const void* x, const void* b, const void* gate,
                       const void* w_post, const void* scale, const void* w_pre, void* dx, void* db, void* dgate, void* dw_post,
                       void* dscale, void* dw_pre, void* workspace, size_t workspace_bytes, void* stream)
{
    const int st = check_desc(d);
    if (st != GCONV_OK) return st;
    const int64_t rows = d->sequences * d->tokens, es = d->dtype == GCONV_BF16 ? 2 : 4;
    const bool some = rows > 0;
    if (!w_post || !dw_post || (some && (!dy || !b || !db))) return fail(GCONV_ERR_NULL, "dy, b, w_post, db and dw_post must be non-NULL");
    if ((d->gate != GCONV_GATE_NONE) != (gate != nullptr) && some) return fail(GCONV_ERR_NULL, "gate must be given unless there is none");
    if ((gate != nullptr) != (dgate != nullptr) && some) return fail(GCONV_ERR_NULL, "gate and dgate go together");
    // (a sequence without tokens has a gate whose gradient, 0, is written)
    if (d->gate == GCONV_GATE_SEQUENCE && d->sequences > 0 && !dgate)
        return fail(GCONV_ERR_NULL, "dgate must be non-NULL for a gate for each sequence");
    if ((scale != nullptr) != (dscale != nullptr)) return fail(GCONV_ERR_NULL, "scale and dscale go together");
    if ((w_pre != nullptr) != (dw_pre != nullptr) || ((w_pre != nullptr) != (dh != nullptr) && some))
        return fail(GCONV_ERR_NULL, "w_pre, dh and dw_pre go together");
    if (dx && !x && some) return fail(GCONV_ERR_NULL, "dx without x");
    const Grid g = bwd_grid(d);
    const size_t need = g.part + g.gate_part;
    if (workspace_bytes < need || (need > 0 && !workspace))
        return fail(GCONV_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace_bytes, need);
    if (need > 0 && ((uintptr_t)workspace & 15) != 0)
        return fail(GCONV_ERR_WORKSPACE, "workspace pointer %p is not 16-byte aligned", workspace);
    const bool gs = d->gate == GCONV_GATE_SEQUENCE;
    const Range in[] = {span(x, d, d->x_stride, false), span(b, d, d->b_stride, false), span(gate, d, d->gate_stride, gs),
                        span(dy, d, d->dy_stride, false), span(dh, d, d->dh_stride, false), {w_post, d->dim * es},
                        {scale, d->dim * es}, {w_pre, d->dim * es}};
    const Range out[] = {{dx, rows * d->dim * es}, {db, rows * d->dim * es}, {dgate, (gs ? d->sequences : rows) * d->dim * es},
                         {dw_post, d->dim * es}, {dscale, d->dim * es}, {dw_pre, d->dim * es}};
    for (const Range& w : out)
        for (const Range& r : in)
            if (meets(w, r)) return fail(GCONV_ERR_ARG, "a gradient overlaps an input");
    for (int i = 0; i < 6; ++i)
        for (int j = 0; j < i; ++j)
            if (meets(out[i], out[j])) return fail(GCONV_ERR_ARG, "two gradients overlap");
    hipStream_t hs = (hipStream_t)stream;
    (void)hipGetLastError();
    Norm a{};
    a.x = Rows{x, d->x_stride[0], d->x_stride[1]};
    a.b = Rows{b, d->b_stride[0], d->b_stride[1]};
    a.gate = Rows{gate, d->gate_stride[0], d->gate == GCONV_GATE_SEQUENCE ? 0 : d->gate_stride[1]};
    a.dy = Rows{dy, d->dy_stride[0], d->dy_stride[1]};
    a.dh = Rows{dh, d->dh_stride[0], d->dh_stride[1]};
    fill(d, &a);
    a.w_post = w_post;
    a.scale = scale;
    a.w_pre = w_pre;
    a.dx = dx;
    a.db = db;
    a.dgate = dgate;
    a.part = (float*)workspace;
    a.gate_part = g.gate_part ? (float*)((char*)workspace + g.part) : nullptr;
    a.groups = g.groups;
    a.splits = g.splits;
    a.group_rows = g.group_rows;
    // (without rows the sums are 0: the kernels write them, from groups of no rows)
    if (d->dtype == GCONV_BF16) run_bwd<__bf16>(d, a, g, dw_post, dscale, dw_pre, hs);
    else run_bwd<float>(d, a, g, dw_post, dscale, dw_pre, hs);
    return finish();
}

}  // extern "C"
