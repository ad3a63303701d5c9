// xent.hip -- softmax cross entropy of tokens against a vocabulary, and its
// gradients, without keeping the logits (gfx950).
//
//   z = scale h w^T     lse_i = log sum_v exp(z_iv)     loss_i = lse_i - z_i,target
//   dz_iv = scale ((dloss_i + dlse_i) exp(z_iv - lse_i) - dloss_i [v = target_i])
//   dh = dz w           dw = dz^T h
//
// Four matrix products of one kernel, with what is special in their epilogues:
//
//   LSE  z of a tile, of which each row leaves its largest value and the sum of
//        exponentials below it; a second kernel joins the tiles of a row
//   DZ   z of a tile again, and dz from it, in bfloat16, for a piece of the
//        vocabulary at a time, so that what is held does not grow with it
//   DH   dz times the piece's rows of w, added up over the pieces in float32
//   DW   dz transposed times h: the piece's rows of dw, whole
//
// Computing z twice costs a quarter of the whole; keeping it would take as many
// bytes as all of dz. Bound by the matrix pipes.
//
// The products take bfloat16. float32 operands are made into three bfloat16 parts
// (8 bits and a sign each, so that together they are the float32), and the six
// products of parts that count are added up in float32: what is left out is
// 2^-23 of a product at most, two of float32's own roundings. A float32 operand
// that is infinite gives NaN.
//
// dz is rounded to bfloat16 (or three parts) as the second products' operand. Of
// bfloat16's, the target's entry, which outweighs a row's others, would be most of
// the error in dh and dw (2.4e-3 of their norm, with the outputs' own 1.7e-3): what
// its rounding leaves is kept in float32 for each token, and dh gets that times
// the target's row of w, dw that times h, summed over the tokens of a target (in
// float32; the sums wait in bfloat16, whose 2^-9 of them are 2^-18 of the entry).
// What is left of dz's rounding is 2.3e-5 of the norm of dh and dw, whose own
// rounding is 1.66e-3.
//
// Tokens that do not count (a target outside the vocabulary) have rows of zeros
// in place of their h, so nothing in them reaches dw.
//
// Measured: 8192 bfloat16 tokens of 2048 against 65536 entries, under the profiler
// LSE 1.85 ms (1.19 PFLOP/s), DZ 2.16, DH 1.66 and DW 1.75 (1.26), with the sort and
// the targets' sums 7.54 in all; without it 7.2 to 7.6, by the card. A large library
// product of random bfloat16 reaches 1.21 PFLOP/s.
#include <cmath>
#include <limits>

#include "device_util.h"
#include "embed_internal.h"
#include "lds_copy.h"
#include "seq_host.h"
#include "seq_tokens.h"

namespace gconv {
namespace {

constexpr int kStepK = 64;  // reduction length of a stage
constexpr float kLog2e = 1.44269504088896340736f;

enum Op { LSE = 0, DZ = 1, DH = 2, DW = 3 };

// A matrix of bfloat16 parts.
struct Operand {
    const __bf16* p;
    int64_t pitch, plane;  // elements between rows, between parts
};

struct Gemm {
    Operand q, p;        // whose rows (columns, for one that is transposed) are the output's rows and columns
    int rows, cols;      // of the output
    int64_t depth;       // length of the reduction
    int parts;           // of the operands: 1 or 3
    int tq, tp, splits;
    // LSE, DZ
    const void* targets;
    int wide;            // targets of 64 bits
    int col0;            // vocabulary entry of column 0
    float scale;
    float2* part;        // LSE: [tp][rows]
    float* picked;       // LSE: the target's z
    const float *lse, *dloss, *dlse;
    __bf16* dz;          // [parts][rows][dz_pitch]
    int64_t dz_pitch, dz_plane;
    int stream;          // dz is stored past the caches
    int vocab;
    float* left;         // DZ: [rows], what rounding left of the target's dz; DH reads it (NULL: 0)
    // DH, DW
    Operand w;           // DH: of the whole vocabulary
    const uint32_t* start;  // DW: where the sums of what is left begin for each column of dz, ...
    const __bf16* fix;      // ... [tokens][cols] (NULL: none)
    float* sums;         // [splits][rows][cols]
    void* out;           // [rows][cols]: NULL while the sums go on
    int add, vec;        // sums hold something; out takes this many elements at once
};

__device__ __forceinline__ int64_t target_of(const Gemm& a, int row)
{
    return a.wide ? ((const int64_t*)a.targets)[row] : (int64_t)((const int32_t*)a.targets)[row];
}

// How far right of column col0 a target lies, -1 if not at all.
__device__ __forceinline__ int wanted(int64_t target, int col0)
{
    const int64_t d = target - col0;
    return d >= 0 && d < 0x7fffffff ? (int)d : -1;
}

// Parts of float32 operands whose products are taken, the small ones first.
// (past the last, which the loads of stages that are not there ask for, the last)
__device__ __forceinline__ int part_q(int parts, int seg) { return parts == 1 ? 0 : 0x201100 >> (20 - 4 * min(seg, 5)) & 3; }
__device__ __forceinline__ int part_p(int parts, int seg) { return parts == 1 ? 0 : 0x021010 >> (20 - 4 * min(seg, 5)) & 3; }

// Stages are loaded from a base that moves on with them, at offsets that stay:
// no operand is too large for 32 bits, and a stage past the last has a size of 0.

// An operand whose reduction runs along its rows: [R][64] elements, the 16-byte
// pieces of row r at piece ^ (r & 7), so that lanes served together read
// different banks.
template <int R, int NW, int FRAGS>
struct AlongRows {
    static constexpr int kLoads = R / 8 / NW;
    static constexpr int kBytes = R * 128;
    static_assert(R % (8 * NW) == 0, "whole loads a wave");
    const __bf16* base;
    uint32_t off[kLoads];
    uint32_t at[2];
    __device__ __forceinline__ void init(const Operand& o, int row0, int rows, int64_t, int wave, int lane, int frag0)
    {
        base = o.p + (int64_t)row0 * o.pitch;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = (i * NW + wave) * 8 + (lane >> 3);
            off[i] = row0 + r < rows ? (uint32_t)(r * o.pitch + ((lane & 7) ^ (r & 7)) * 8) * 2 : kOOB;
        }
        const int li = lane & 15, g = lane >> 4;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) at[ks] = (frag0 + li) * 128 + (((ks * 4 + g) ^ (li & 7)) * 16);
    }
    __device__ __forceinline__ u4 stage(const Operand& o, int part, int64_t k0, bool there) const
    {
        return resource(base + part * o.plane + k0, there ? kOOB : 0);
    }
    __device__ __forceinline__ void load(u4 rs, uint32_t tile, int i, int wave) const { copy_lds(rs, tile + (i * NW + wave) * 1024, off[i]); }
    __device__ __forceinline__ u4 frag(const char* tile, int t, int ks) const { return *(const u4*)(tile + at[ks] + t * (16 * 128)); }
};

// An operand whose reduction runs across its rows: [64][C] elements, read with
// transposing loads (16 lanes: 4 rows x 16 columns). The 32-byte pieces of a row
// are swizzled so that the eight rows of 32 lanes lie in different banks. Rows
// past the reduction's end lie past the resource's.
template <int C, int NW, int FRAGS>
struct AcrossRows {
    static constexpr int kPieces = C / 8;
    static constexpr int kLoads = kStepK * kPieces / 64 / NW;
    static constexpr int kBytes = kStepK * C * 2;
    static_assert(kStepK * kPieces % (64 * NW) == 0, "whole loads a wave");
    const __bf16* base;
    int64_t left;  // bytes from the base to the last row's end
    uint32_t off[kLoads];
    uint32_t at[FRAGS];
    static __device__ __forceinline__ int swz(int row)
    {
        return C % 128 == 0 ? (row & 3) | ((row >> 1) & 4) : ((row >> 1) & 1) | ((row >> 2) & 2);
    }
    __device__ __forceinline__ void init(const Operand& o, int col0, int, int64_t depth, int wave, int lane, int frag0)
    {
        base = o.p + col0;
        left = (depth * o.pitch - col0) * 2;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = (i * NW + wave) * 64 + lane, row = q / kPieces, p = q % kPieces;
            const int64_t from = (row * o.pitch + ((p ^ (swz(row) << 1)) * 8)) * 2;
            off[i] = (uint32_t)min(from, (int64_t)kOOB);  // (rows that exist lie below it)
        }
        const int li = lane & 15, g = lane >> 4;
        const int row = 8 * g + (li >> 2);  // rows + 4 and + 32 have the same swizzle
#pragma unroll
        for (int t = 0; t < FRAGS; ++t) at[t] = row * (C * 2) + ((((frag0 >> 4) + t) ^ swz(row)) * 32) + (li & 3) * 8;
    }
    __device__ __forceinline__ u4 stage(const Operand& o, int part, int64_t k0, bool there) const
    {
        const int64_t bytes = left - k0 * o.pitch * 2;
        return resource(base + part * o.plane + k0 * o.pitch, there ? (uint32_t)min(bytes, (int64_t)kOOB) : 0);
    }
    __device__ __forceinline__ void load(u4 rs, uint32_t tile, int i, int wave) const { copy_lds(rs, tile + (i * NW + wave) * 1024, off[i]); }
    __device__ __forceinline__ u4 frag(const char* tile, int t, int ks) const
    {
        const char* p = tile + at[t] + ks * (32 * C * 2);
        const u2 lo = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p));
        const u2 hi = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + 4 * C * 2)));
        return u4{lo[0], lo[1], hi[0], hi[1]};
    }
};

// v in bfloat16; past its largest value cut off in place of rounded up to infinity.
__device__ __forceinline__ __bf16 part_of(float v)
{
    const __bf16 o = (__bf16)v;
    return finite_bits(o) || !finite_bits(v) ? o : __builtin_bit_cast(__bf16, (uint16_t)(__builtin_bit_cast(uint32_t, v) >> 16));
}

// v in three bfloat16 parts, whose sum it is but for what lies below the last.
__device__ __forceinline__ void split3(float v, __bf16 (&o)[3])
{
    o[0] = part_of(v);
    const float r = v - (float)o[0];
    o[1] = (__bf16)r;
    o[2] = (__bf16)(r - (float)o[1]);
}

// A tile of bfloat16 by way of LDS, so that it is stored in whole lines: a lane of
// the accumulators holds 8 bytes of each of 16 rows. put() takes the four columns
// from `col` of row `row` of the tile, the 8-byte pieces of a row at piece ^ (row &
// 15), so that 16 rows' lie in different banks; store() writes the tile.
template <int BQ, int BP, int THREADS>
struct TileOut {
    static __device__ __forceinline__ void put(char* lds, int row, int col, u2 v)
    {
        *(u2*)(lds + row * (BP * 2) + ((col / 4) ^ (row & 15)) * 8) = v;
    }
    // STREAM: past the caches
    template <bool STREAM = false>
    static __device__ __forceinline__ void store(const char* lds, __bf16* out, int64_t pitch, int rows, int cols)
    {
#pragma unroll 4
        for (int i = threadIdx.x; i < BQ * (BP / 8); i += THREADS) {
            const int row = i / (BP / 8), col = i % (BP / 8) * 8, x = row & 15;
            if (row >= rows || col >= cols) continue;
            const u4 v = *(const u4*)(lds + row * (BP * 2) + ((col / 4) ^ (x & ~1)) * 8);
            const u4 o = x & 1 ? u4{v[2], v[3], v[0], v[1]} : v;
            if constexpr (STREAM) __builtin_nontemporal_store(o, (u4*)(out + row * pitch + col));
            else *(u4*)(out + row * pitch + col) = o;
        }
    }
};

// One BQ x BP tile of an output (of one of its splits). The matrix instruction's
// rows run along the output's columns, so a lane holds four consecutive elements
// of an output row: those of row li, columns 4 g to 4 g + 3 of each 16 x 16.
// Eight waves, two a SIMD, so that one multiplies while the other waits, over a
// ring of 64-long stages.
template <typename T, int BQ, int BP, int WQ, int WP, int OP>
__global__ __launch_bounds__(64 * WQ * WP, 1) void xent_gemm(Gemm a)
{
    constexpr int NW = WQ * WP;
    constexpr int FQ = BQ / WQ / 16, FP = BP / WP / 16;
    using SQ = std::conditional_t<OP == DW, AcrossRows<BQ, NW, FQ>, AlongRows<BQ, NW, FQ>>;
    using SP = std::conditional_t<OP == LSE || OP == DZ, AlongRows<BP, NW, FP>, AcrossRows<BP, NW, FP>>;
    constexpr int kBuf = SQ::kBytes + SP::kBytes;
    constexpr int kLoads = SQ::kLoads + SP::kLoads;
    constexpr int kRing = std::min(3, 160 * 1024 / kBuf);
    __shared__ __align__(1024) char lds[kRing * kBuf];

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wq = wave % WQ, wp = wave / WQ;
    const int per = a.tq * a.tp;
    const int b = xcd_remap(blockIdx.x, gridDim.x);
    const int split = b / per, L = b - split * per;
    // strips of 8 tiles of rows: the blocks that run together on an XCD share their panels
    const int strip = L / (8 * a.tp), first = strip * 8, high = min(a.tq - first, 8), in = L - strip * 8 * a.tp;
    const int tq = first + in % high, tp = in / high;
    const int i0 = tq * BQ, j0 = tp * BP;

    SQ sq;
    SP sp;
    sq.init(a.q, i0, a.rows, a.depth, wave, lane, wq * (BQ / WQ));
    sp.init(a.p, j0, a.cols, a.depth, wave, lane, wp * (BP / WP));
    const int along = (int)((a.depth + kStepK - 1) / kStepK), all = along * (a.parts == 1 ? 1 : 6);
    const int s0 = (int)((int64_t)all * split / a.splits), s1 = (int)((int64_t)all * (split + 1) / a.splits);

    f4 acc[FQ][FP];
#pragma unroll
    for (int i = 0; i < FQ; ++i)
#pragma unroll
        for (int j = 0; j < FP; ++j) acc[i][j] = f4{0, 0, 0, 0};

    const uint32_t lds_at = (uint32_t)(uintptr_t)(lds_char*)lds;
    int seg = s0 / along, at = s0 - seg * along, next_stage = s0;
    u4 rq, rp;
    auto aim = [&]() {  // at the next stage to load
        const bool there = next_stage < s1;
        rq = sq.stage(a.q, part_q(a.parts, seg), (int64_t)at * kStepK, there);
        rp = sp.stage(a.p, part_p(a.parts, seg), (int64_t)at * kStepK, there);
        ++next_stage;
        if (++at == along) {
            at = 0;
            ++seg;
        }
    };
    auto issue = [&](int n, uint32_t buf) {  // load n of that stage
        if (n < SQ::kLoads) sq.load(rq, lds_at + buf, n, wave);
        else sp.load(rp, lds_at + buf + SQ::kBytes, n - SQ::kLoads, wave);
    };
    u4 fq[2][FQ], fp[2][FP];
    auto read = [&](int ks, int n, uint32_t buf) {  // fragment n of half ks of a stage
        if (n < FP) fp[ks][n] = sp.frag(lds + buf + SQ::kBytes, n, ks);
        else fq[ks][n - FP] = sq.frag(lds + buf, n - FP, ks);
    };
    // Half a stage: its products, and spread among them the reads of the next
    // half's fragments and (second halves) the loads of a stage.
    constexpr int kMmas = FQ * FP;
    auto half = [&](int ks, uint32_t from, uint32_t into) {
        int rd = 0, ld = 0;
#pragma unroll
        for (int n = 0; n < kMmas; ++n) {
            while (rd < FQ + FP && n * (FQ + FP) * 3 >= rd * kMmas * 2) read(ks ^ 1, rd++, from);
            while (ks == 1 && ld < kLoads && n * kLoads >= ld * kMmas) issue(ld++, into);
            const int i = n / FP, j = n % FP;
            acc[i][j] = mma<__bf16>(fp[ks][j], fq[ks][i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        while (rd < FQ + FP) read(ks ^ 1, rd++, from);
        while (ks == 1 && ld < kLoads) issue(ld++, into);
    };
#pragma unroll
    for (int st = 0; st < kRing; ++st) {
        aim();
#pragma unroll
        for (int n = 0; n < kLoads; ++n) issue(n, st * kBuf);
    }
    wait_loads<(kRing - 1) * kLoads>();
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int n = 0; n < FQ + FP; ++n) read(0, n, 0);
    __builtin_amdgcn_sched_barrier(0);
    // In the middle of a stage the next one has landed and this one has been read
    // by all waves, so the stage kRing on is loaded into its place.
    uint32_t cur = 0;
    for (int st = s0; st < s1; ++st) {
        const uint32_t next = cur + kBuf == kRing * kBuf ? 0 : cur + kBuf;
        aim();
        half(0, cur, 0);
        wait_loads<(kRing - 2) * kLoads>();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        half(1, next, cur);
        cur = next;
    }
    wait_loads<0>();  // no load may land after the workgroup's end, or in what the epilogue puts there
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");

    const int row0 = i0 + wq * (BQ / WQ) + li, col0 = j0 + wp * (BP / WP) + 4 * g;
    if constexpr (OP == LSE) {
        __builtin_amdgcn_s_barrier();
        float2* red = (float2*)lds;  // [WP][BQ]
#pragma unroll
        for (int i = 0; i < FQ; ++i) {
            const int row = row0 + i * 16;
            const int want = wanted(row < a.rows ? target_of(a, row) : -1, col0);
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < FP; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float z = acc[i][j][r] * a.scale;
                    acc[i][j][r] = col0 + j * 16 + r < a.cols ? z : -INFINITY;
                    top = fmaxf(top, acc[i][j][r]);
                    if (want == j * 16 + r) a.picked[row] = z;
                }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            // (values that are all -infinity have a sum of 0, those that hold +infinity one of infinity; the latter's is taken
            // below the largest float, so that in a join it is not multiplied by an exponential that has become 0)
            const float below = top == INFINITY ? std::numeric_limits<float>::max() : top == -INFINITY ? 0.f : top;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < FP; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) sum += __builtin_amdgcn_exp2f((acc[i][j][r] - below) * kLog2e);
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (g == 0) red[wp * BQ + wq * (BQ / WQ) + i * 16 + li] = float2{below, sum};
        }
        __syncthreads();
        for (int r = tid; r < BQ; r += 64 * NW) {
            if (i0 + r >= a.rows) break;
            float2 v = red[r];
#pragma unroll
            for (int k = 1; k < WP; ++k) {
                const float2 o = red[k * BQ + r];
                if (o.y == 0.f) continue;  // nothing but -infinity
                if (v.y == 0.f) {
                    v = o;
                    continue;
                }
                const float m = fmaxf(v.x, o.x);
                v.y = v.y * __builtin_amdgcn_exp2f((v.x - m) * kLog2e) + o.y * __builtin_amdgcn_exp2f((o.x - m) * kLog2e);
                v.x = m;
            }
            a.part[(int64_t)tp * a.rows + i0 + r] = v;
        }
    } else if constexpr (OP == DZ) {
        using Out = TileOut<BQ, BP, 64 * NW>;
        constexpr int kParts = sizeof(T) == 2 ? 1 : 3;
#pragma unroll
        for (int i = 0; i < FQ; ++i) {
            const int row = row0 + i * 16;
            const bool there = row < a.rows;
            const int64_t target = there ? target_of(a, row) : -1;
            const bool counts = target >= 0 && target < a.vocab;
            const float dl = counts ? a.dloss[row] * a.scale : 0.f;
            const float all_of = counts ? (a.dlse ? fmaf(a.dlse[row], a.scale, dl) : dl) : 0.f;
            const float low = there ? a.lse[row] * kLog2e : 0.f, up = a.scale * kLog2e;
            const int want = wanted(target - a.col0, col0);
#pragma unroll
            for (int j = 0; j < FP; ++j) {
                const int col = col0 + j * 16;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float v = all_of * __builtin_amdgcn_exp2f(fmaf(acc[i][j][r], up, -low));
                    if (want == j * 16 + r) {
                        v -= dl;
                        if (kParts == 1 && counts) a.left[row] = v - (float)(__bf16)v;
                    }
                    if (!counts || col + r >= a.cols) v = 0.f;
                    acc[i][j][r] = v;
                }
            }
        }
        // (a part of float32's is left in the accumulators for the next)
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < FQ; ++i)
#pragma unroll
                for (int j = 0; j < FP; ++j) {
                    bf4 e;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float v = acc[i][j][r];
                        e[r] = kParts == 1 ? (__bf16)v : part_of(v);
                        if (kParts > 1) acc[i][j][r] = v - (float)e[r];
                    }
                    Out::put(lds, row0 - i0 + i * 16, col0 - j0 + j * 16, __builtin_bit_cast(u2, e));
                }
            __syncthreads();
            __bf16* o = a.dz + k * a.dz_plane + (int64_t)i0 * a.dz_pitch + j0;
            const int cols = (int)min(a.dz_pitch - j0, (int64_t)BP);
            if (a.stream) Out::template store<true>(lds, o, a.dz_pitch, a.rows - i0, cols);
            else Out::store(lds, o, a.dz_pitch, a.rows - i0, cols);
        }
    } else {
        float* sums = a.sums ? a.sums + (int64_t)split * a.rows * a.cols : nullptr;
        if (sizeof(T) == 2 && split == 0 && (a.left || a.fix)) {
#pragma unroll
            for (int i = 0; i < FQ; ++i) {
                const int row = row0 + i * 16;
                if (row >= a.rows) continue;
                const __bf16* from;
                float weight = 1.f;
                if constexpr (OP == DH) {
                    const int64_t target = target_of(a, row);
                    if (target < 0 || target >= a.vocab) continue;
                    from = a.w.p + target * a.w.pitch;
                    weight = a.left[row];
                    if (weight == 0.f) continue;  // (nor times an infinite w)
                } else {
                    if (a.start[row] == a.start[row + 1]) continue;
                    from = a.fix + (int64_t)a.start[row] * a.cols;
                }
#pragma unroll
                for (int j = 0; j < FP; ++j) {
                    const int col = col0 + j * 16;
                    if (col >= a.cols) continue;
                    const Packed<__bf16, 4> v = load_piece<__bf16, 4>(from, col, a.cols);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(weight, (float)v.e[r], acc[i][j][r]);
                }
            }
        }
        if (sizeof(T) == 2 && a.vec == 8 && a.out && !a.add) {
            using Out = TileOut<BQ, BP, 64 * NW>;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < FQ; ++i)
#pragma unroll
                for (int j = 0; j < FP; ++j) Out::put(lds, row0 - i0 + i * 16, col0 - j0 + j * 16, pack4(acc[i][j]));
            __syncthreads();
            Out::store(lds, (__bf16*)a.out + (int64_t)i0 * a.cols + j0, a.cols, a.rows - i0, min(a.cols - j0, BP));
            return;
        }
#pragma unroll
        for (int i = 0; i < FQ; ++i) {
            const int row = row0 + i * 16;
            if (row >= a.rows) continue;
            const int64_t at_row = (int64_t)row * a.cols;
#pragma unroll
            for (int j = 0; j < FP; ++j) {
                const int col = col0 + j * 16;
                if (col >= a.cols) continue;
                f4 v = acc[i][j];
                const bool whole = a.vec > 1 && col + 4 <= a.cols;
                if (a.add) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (col + r < a.cols) v[r] += sums[at_row + col + r];
                }
                if (a.out) {
                    T* o = (T*)a.out + at_row + col;
                    if (whole) {
                        if constexpr (sizeof(T) == 2) *(u2*)o = pack4(v);
                        else *(f4*)o = v;
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (col + r < a.cols) o[r] = (T)v[r];
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (col + r < a.cols) sums[at_row + col + r] = v[r];
                }
            }
        }
    }
}

// lse and loss of 64 rows: 16 slices of the tiles' parts, then the slices.
__global__ __launch_bounds__(1024) void xent_join(const float2* part, int tiles, int rows, const float* picked, const void* targets, int wide,
                                                  int64_t vocab, float* loss, float* lse)
{
    __shared__ float2 red[16][64];
    const int c = threadIdx.x & 63, slice = threadIdx.x >> 6;
    const int64_t row = (int64_t)blockIdx.x * 64 + c;
    float2 v = {0.f, 0.f};
    auto join = [&](float2 o) {
        if (o.y == 0.f) return;
        if (v.y == 0.f) {
            v = o;
            return;
        }
        const float m = fmaxf(v.x, o.x);
        v.y = v.y * __builtin_amdgcn_exp2f((v.x - m) * kLog2e) + o.y * __builtin_amdgcn_exp2f((o.x - m) * kLog2e);
        v.x = m;
    };
    if (row < rows) {
        int i = slice;
        for (; i + 48 < tiles; i += 64) {
            const float2 o0 = part[(int64_t)i * rows + row], o1 = part[(int64_t)(i + 16) * rows + row];
            const float2 o2 = part[(int64_t)(i + 32) * rows + row], o3 = part[(int64_t)(i + 48) * rows + row];
            join(o0); join(o1); join(o2); join(o3);
        }
        for (; i < tiles; i += 16) join(part[(int64_t)i * rows + row]);
    }
    red[slice][c] = v;
    __syncthreads();
    if (slice || row >= rows) return;
    for (int k = 1; k < 16; ++k) join(red[k][c]);
    // (a row of -infinity has the sum 0, whose logarithm that is)
    const float l = v.x + logf(v.y);
    lse[row] = l;
    const int64_t t = wide ? ((const int64_t*)targets)[row] : (int64_t)((const int32_t*)targets)[row];
    loss[row] = t >= 0 && t < vocab ? l - picked[row] : 0.f;
}

// out = the sum of the splits' sums.
template <typename T>
__global__ __launch_bounds__(256) void xent_fold(const float* sums, int splits, int64_t count, T* out)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= count) return;
    float v = 0.f;
    int k = 0;
    for (; k + 4 <= splits; k += 4) {
        const float v0 = sums[k * count + i], v1 = sums[(k + 1) * count + i], v2 = sums[(k + 2) * count + i], v3 = sums[(k + 3) * count + i];
        v += v0; v += v1; v += v2; v += v3;
    }
    for (; k < splits; ++k) v += sums[k * count + i];
    out[i] = (T)v;
}

// Rows as the products take them: bfloat16 parts, padded with zeros to whole
// stages; rows of tokens that do not count (targets given) are 0.
template <typename T>
__global__ __launch_bounds__(256) void xent_pack(const T* src, int64_t seq, int64_t tok, int64_t tokens, int64_t rows, int dim, int pitch,
                                                 const void* targets, int wide, int64_t vocab, __bf16* dst)
{
    const int pieces = pitch / 8;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, row = id / pieces;
    if (row >= rows) return;
    const int col = (int)(id - row * pieces) * 8;
    bool counts = true;
    if (targets) {
        const int64_t t = wide ? ((const int64_t*)targets)[row] : (int64_t)((const int32_t*)targets)[row];
        counts = t >= 0 && t < vocab;
    }
    const int64_t n = row / tokens;
    Packed<T, 8> v = load_piece<T, 8>(src + n * seq + (row - n * tokens) * tok, col, dim);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (!counts) v.e[e] = (T)0.f;
    bf8 o[3];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (sizeof(T) == 2) {
            o[0][e] = v.e[e];
        } else {
            __bf16 s[3];
            split3(v.e[e], s);
#pragma unroll
            for (int k = 0; k < 3; ++k) o[k][e] = s[k];
        }
    }
#pragma unroll
    for (int k = 0; k < (sizeof(T) == 2 ? 1 : 3); ++k) *(bf8*)(dst + k * rows * pitch + row * pitch + col) = o[k];
}

// ---- host ------------------------------------------------------------------------

constexpr int64_t kMaxDim = (int64_t)1 << 20;
constexpr int64_t kMaxVocab = (int64_t)1 << 30;
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kHeld = (int64_t)1 << 29;  // bytes of dz at once, about

int check_desc(const gconv_xent_desc* d)
{
    if (!d) return fail(GCONV_ERR_NULL, "descriptor is NULL");
    if (d->dtype != GCONV_F32 && d->dtype != GCONV_BF16) return fail(GCONV_ERR_ARG, "unknown dtype %lld", (long long)d->dtype);
    if (d->index != GCONV_I32 && d->index != GCONV_I64) return fail(GCONV_ERR_ARG, "unknown index type %lld", (long long)d->index);
    if (d->sequences < 0 || d->tokens < 0 || d->vocab < 1 || d->dim < 1)
        return fail(GCONV_ERR_SHAPE, "need sequences, tokens >= 0 and vocab, dim >= 1 (got %lld, %lld, %lld, %lld)", (long long)d->sequences,
                    (long long)d->tokens, (long long)d->vocab, (long long)d->dim);
    if (d->dim > kMaxDim) return fail(GCONV_ERR_UNSUPPORTED, "dim=%lld above %lld", (long long)d->dim, (long long)kMaxDim);
    if (d->vocab > kMaxVocab) return fail(GCONV_ERR_UNSUPPORTED, "vocab=%lld above %lld", (long long)d->vocab, (long long)kMaxVocab);
    if (d->sequences > kMaxRows || d->tokens > kMaxRows || (d->tokens > 0 && d->sequences > kMaxRows / d->tokens))
        return fail(GCONV_ERR_UNSUPPORTED, "too many tokens");
    if (!std::isfinite((float)d->scale)) return fail(GCONV_ERR_ARG, "scale must be finite as float32");
    return GCONV_OK;
}

struct Tile {
    int kind, q, p;
};
constexpr Tile kTiles[] = {{0, 256, 256}, {1, 128, 128}, {2, 64, 256}, {3, 128, 256}, {4, 128, 192}};

// Parts of a reduction that a product with few tiles is cut into: as many as
// there are CUs without work, each at least 8 stages long.
int splits_of(const Tile& t, int64_t rows, int64_t cols, int64_t stages)
{
    const int64_t count = std::max<int64_t>(1, (rows + t.q - 1) / t.q) * ((cols + t.p - 1) / t.p);
    return (int)std::max<int64_t>(1, std::min<int64_t>(256 / count, stages / 8));
}

// The tile that takes least: whole rounds of 256 workgroups, each a tile's area
// over the rate it reaches (8192 tokens x 65536 entries of 2048: LSE 1814, 2665,
// 3154, 2142 and 2285 us; DH and DW 1700, 2620, 2760, 2000 and 2270) for each
// stage, 65536 of which take 1.8 us; and the splits' sums, which are written and
// read at 4 TB/s. stages: 0 for LSE and DZ, which have no splits.
Tile tile_of(int64_t rows, int64_t cols, int64_t stages)
{
    const double rate[] = {1.0, 0.68, 0.57, 0.85, stages ? 0.72 : 0.82};
    int best = 0;
    double least = 0;
    for (int i = 0; i < 5; ++i) {
        const Tile& t = kTiles[i];
        const int64_t count = ((rows + t.q - 1) / t.q) * ((cols + t.p - 1) / t.p);
        const int splits = stages ? splits_of(t, rows, cols, stages) : 1;
        double cost = (double)((count * splits + 255) / 256) * t.q * t.p / rate[i];
        if (stages) cost *= (double)stages / splits;
        if (splits > 1) cost += (double)splits * rows * cols * (65536 / 1.8 * 8 / 4e6);
        if (i == 0 || cost < least) {
            least = cost;
            best = i;
        }
    }
    return kTiles[best];
}

struct Plan {
    int64_t rows, pitch;       // tokens; padded dim
    int parts, segs;
    bool pack_h, pack_w;
    Tile lse, dz, dh, dw;
    int64_t lse_tiles;
    int64_t piece, pieces;     // vocabulary entries of a piece
    int dh_splits, dw_splits;
    size_t h, w, part, picked, dzs, dh_sums, dw_sums, left, runs, fix, bytes;
};

// Whether the products read w itself.
bool as_it_is(const gconv_xent_desc* d) { return d->dtype == GCONV_BF16 && d->dim % kStepK == 0; }

EmbedRuns runs_of(const gconv_xent_desc* d, const void* targets)
{
    EmbedRuns r{};
    r.ids = targets;
    r.wide = d->index == GCONV_I64;
    r.tokens = d->sequences * d->tokens;
    r.rows = d->vocab;
    r.dim = d->dim;
    return r;
}

// (whether h can be read itself is not known before its address is: the
// workspace always has room for it)
void make_plan(const gconv_xent_desc* d, bool back, Plan* p)
{
    p->rows = d->sequences * d->tokens;
    p->pitch = (d->dim + kStepK - 1) / kStepK * kStepK;
    p->parts = d->dtype == GCONV_BF16 ? 1 : 3;
    p->segs = p->parts == 1 ? 1 : 6;
    Cut cut;
    p->h = cut.take(p->rows * p->pitch * p->parts * 2);
    p->w = cut.take(as_it_is(d) ? 0 : d->vocab * p->pitch * p->parts * 2);
    if (!back) {
        p->lse = tile_of(p->rows, d->vocab, 0);
        p->lse_tiles = (d->vocab + p->lse.p - 1) / p->lse.p;
        p->part = cut.take(p->lse_tiles * p->rows * 8);
        p->picked = cut.take(p->rows * 4);
    } else {
        const int64_t most = kHeld / (std::max<int64_t>(p->rows, 1) * p->parts * 2) / 256 * 256;
        const int64_t all = (d->vocab + 255) / 256 * 256;
        p->piece = std::min(all, std::max<int64_t>(2048, most));
        p->pieces = (d->vocab + p->piece - 1) / p->piece;
        p->piece = ((d->vocab + p->pieces - 1) / p->pieces + 255) / 256 * 256;  // even ones
        p->pieces = (d->vocab + p->piece - 1) / p->piece;
        const int64_t cols = std::min(p->piece, d->vocab);
        const int64_t dh_stages = (cols + kStepK - 1) / kStepK * p->segs, dw_stages = (p->rows + kStepK - 1) / kStepK * p->segs;
        p->dz = tile_of(p->rows, cols, 0);
        p->dh = tile_of(p->rows, d->dim, dh_stages);
        p->dw = tile_of(cols, d->dim, dw_stages);
        p->dh_splits = splits_of(p->dh, p->rows, d->dim, dh_stages);
        p->dw_splits = splits_of(p->dw, cols, d->dim, dw_stages);
        p->dzs = cut.take(p->rows * p->piece * p->parts * 2);
        p->dh_sums = cut.take(p->dh_splits > 1 || p->pieces > 1 ? p->rows * d->dim * 4 * p->dh_splits : 0);
        p->dw_sums = cut.take(p->dw_splits > 1 ? cols * d->dim * 4 * p->dw_splits : 0);
        if (p->parts == 1) {
            p->left = cut.take(p->rows * 4);
            p->runs = cut.take((int64_t)embed_runs_workspace(runs_of(d, nullptr)));
            p->fix = cut.take(p->rows * d->dim * 2);
        }
    }
    p->bytes = cut.bytes;
}

int64_t tiles_of(const Tile& t, int64_t rows, int64_t cols) { return ((rows + t.q - 1) / t.q) * ((cols + t.p - 1) / t.p); }

// Whether every launch of a call stays below what a launch takes, before any is made. (The sums by target have a
// workgroup for some 32 tokens or more and 1024 columns: fewer than the sums' folding has.)
int check_launches(const gconv_xent_desc* d, const Plan& p, bool back)
{
    const int64_t cols = std::min(p.piece, d->vocab), most = max_blocks(512);
    bool fits = std::max(p.rows, d->vocab) <= max_blocks(256) / (p.pitch / 8) * 256;  // packing
    if (!back) {
        fits = fits && tiles_of(p.lse, p.rows, d->vocab) <= most && p.rows / 64 < max_blocks(1024);
    } else {
        fits = fits && tiles_of(p.dz, p.rows, cols) <= most && tiles_of(p.dh, p.rows, d->dim) * p.dh_splits <= most &&
               tiles_of(p.dw, cols, d->dim) * p.dw_splits <= most && (d->dim / 256 + 1) * p.rows <= max_blocks(256) &&
               (d->dim / 256 + 1) * cols <= max_blocks(256);
    }
    return fits ? GCONV_OK : fail(GCONV_ERR_UNSUPPORTED, "too many tokens, entries or elements for a launch");
}

template <typename T, int OP>
void launch(Gemm a, const Tile& t, hipStream_t st)
{
    a.tq = (a.rows + t.q - 1) / t.q;
    a.tp = (a.cols + t.p - 1) / t.p;
    const unsigned n = (unsigned)((int64_t)a.tq * a.tp * a.splits);
    if (t.kind == 0) xent_gemm<T, 256, 256, 2, 4, OP><<<n, 512, 0, st>>>(a);
    else if (t.kind == 1) xent_gemm<T, 128, 128, 2, 4, OP><<<n, 512, 0, st>>>(a);
    else if (t.kind == 2) xent_gemm<T, 64, 256, 1, 8, OP><<<n, 512, 0, st>>>(a);
    else if (t.kind == 3) xent_gemm<T, 128, 256, 2, 4, OP><<<n, 512, 0, st>>>(a);
    else xent_gemm<T, 128, 192, 2, 4, OP><<<n, 512, 0, st>>>(a);
}

template <typename T>
void pack(const void* src, int64_t seq, int64_t tok, int64_t tokens, int64_t rows, int64_t dim, int64_t pitch, const void* targets, int wide,
          int64_t vocab, __bf16* dst, hipStream_t st)
{
    const int64_t blocks = (rows * (pitch / 8) + 255) / 256;
    xent_pack<T><<<(unsigned)blocks, 256, 0, st>>>((const T*)src, seq, tok, std::max<int64_t>(tokens, 1), rows, (int)dim, (int)pitch, targets,
                                                   wide, vocab, dst);
}

template <typename T>
int forward(const gconv_xent_desc* d, const Plan& p, const void* h, const void* w, const void* targets, float* loss, float* lse, char* ws,
            hipStream_t st)
{
    const bool flat = d->sequences == 1 || d->tokens == 1 || d->h_stride[0] == d->tokens * d->h_stride[1];
    const int64_t step = d->tokens == 1 && d->sequences > 1 ? d->h_stride[0] : d->h_stride[1];
    Gemm a{};
    a.q = Operand{(const __bf16*)h, step, 0};
    a.p = Operand{(const __bf16*)w, d->dim, 0};
    // h is read itself where it is bfloat16 rows of whole stages at 16-byte boundaries, one after another
    if (!as_it_is(d) || !flat || step % 8 || step < d->dim || step > kMaxDim || ((uintptr_t)h & 15)) {
        a.q = Operand{(const __bf16*)(ws + p.h), p.pitch, p.rows * p.pitch};
        pack<T>(h, d->h_stride[0], d->h_stride[1], d->tokens, p.rows, d->dim, p.pitch, nullptr, 0, 0, (__bf16*)(ws + p.h), st);
    }
    if (!as_it_is(d)) {
        a.p = Operand{(const __bf16*)(ws + p.w), p.pitch, d->vocab * p.pitch};
        pack<T>(w, 0, d->dim, d->vocab, d->vocab, d->dim, p.pitch, nullptr, 0, 0, (__bf16*)(ws + p.w), st);
    }
    a.rows = (int)p.rows;
    a.cols = a.vocab = (int)d->vocab;
    a.depth = p.pitch;
    a.parts = p.parts;
    a.splits = 1;
    a.targets = targets;
    a.wide = d->index == GCONV_I64;
    a.scale = (float)d->scale;
    a.part = (float2*)(ws + p.part);
    a.picked = (float*)(ws + p.picked);
    launch<T, LSE>(a, p.lse, st);
    xent_join<<<(unsigned)((p.rows + 63) / 64), 1024, 0, st>>>(a.part, (int)p.lse_tiles, (int)p.rows, a.picked, targets, a.wide, d->vocab, loss, lse);
    return finish();
}

template <typename T>
int backward(const gconv_xent_desc* d, const Plan& p, const float* dloss, const float* dlse, const float* lse, const void* h, const void* w,
             const void* targets, void* dh, void* dw, char* ws, hipStream_t st)
{
    const int wide = d->index == GCONV_I64;
    const Operand hp{(const __bf16*)(ws + p.h), p.pitch, p.rows * p.pitch};
    Operand wp{(const __bf16*)w, d->dim, 0};
    pack<T>(h, d->h_stride[0], d->h_stride[1], d->tokens, p.rows, d->dim, p.pitch, targets, wide, d->vocab, (__bf16*)(ws + p.h), st);
    if (!as_it_is(d)) {
        wp = Operand{(const __bf16*)(ws + p.w), p.pitch, d->vocab * p.pitch};
        pack<T>(w, 0, d->dim, d->vocab, d->vocab, d->dim, p.pitch, nullptr, 0, 0, (__bf16*)(ws + p.w), st);
    }
    EmbedRuns runs = runs_of(d, targets);
    float* left = sizeof(T) == 2 ? (float*)(ws + p.left) : nullptr;
    if (left) {
        runs.workspace = ws + p.runs;
        runs.src = hp.p;
        runs.pitch = hp.pitch;
        runs.weight = left;
        runs.sums = ws + p.fix;
        embed_runs_sort(&runs, st);
    }
    const Operand dz{(const __bf16*)(ws + p.dzs), p.piece, p.rows * p.piece};
    const int vec = d->dim % 8 == 0 ? 8 : d->dim % 4 == 0 ? 4 : 1;
    for (int64_t i = 0; i < p.pieces; ++i) {
        const int64_t v0 = i * p.piece, cols = std::min(p.piece, d->vocab - v0);
        const Operand rows{wp.p + v0 * wp.pitch, wp.pitch, wp.plane};
        Gemm a{};
        a.q = hp;
        a.p = rows;
        a.rows = (int)p.rows;
        a.cols = (int)cols;
        a.vocab = (int)d->vocab;
        a.col0 = (int)v0;
        a.depth = p.pitch;
        a.parts = p.parts;
        a.splits = 1;
        a.targets = targets;
        a.wide = wide;
        a.scale = (float)d->scale;
        a.lse = lse;
        a.dloss = dloss;
        a.dlse = dlse;
        a.dz = (__bf16*)(ws + p.dzs);
        a.dz_pitch = dz.pitch;
        a.dz_plane = dz.plane;
        a.left = left;
        // where dz would not stay in the 256 MB cache behind the L2s, past it: the operands stay (537 MB: 2 x 1088 and
        // 2 x 843 us for DZ and DH, 2 x 1108 and 2 x 866 through it)
        a.stream = p.rows * p.piece * p.parts * 2 >= (int64_t)160 << 20;
        launch<T, DZ>(a, p.dz, st);
        Gemm b{};
        b.q = dz;
        b.p = rows;
        b.rows = (int)p.rows;
        b.cols = (int)d->dim;
        b.depth = cols;
        b.parts = p.parts;
        b.splits = p.dh_splits;
        b.sums = p.dh_splits > 1 || p.pieces > 1 ? (float*)(ws + p.dh_sums) : nullptr;
        b.add = i > 0;
        b.out = p.dh_splits == 1 && i + 1 == p.pieces ? dh : nullptr;
        b.vec = ((uintptr_t)dh & 15) == 0 ? vec : 1;
        // (with the last piece every token has what is left of its target's)
        b.left = i + 1 == p.pieces ? left : nullptr;
        b.w = wp;
        b.targets = targets;
        b.wide = wide;
        b.vocab = (int)d->vocab;
        launch<T, DH>(b, p.dh, st);
        Gemm c{};
        c.q = dz;
        c.p = hp;
        c.rows = (int)cols;
        c.cols = (int)d->dim;
        c.depth = p.rows;
        c.parts = p.parts;
        c.splits = p.dw_splits;
        T* to = (T*)dw + v0 * d->dim;
        c.sums = p.dw_splits > 1 ? (float*)(ws + p.dw_sums) : nullptr;
        c.out = p.dw_splits > 1 ? nullptr : to;
        c.vec = ((uintptr_t)to & 15) == 0 ? vec : 1;
        if (left) {
            embed_runs_sum(runs, v0, v0 + cols, st);
            c.start = runs.start + v0;
            c.fix = (const __bf16*)runs.sums;
        }
        launch<T, DW>(c, p.dw, st);
        if (p.dw_splits > 1) {
            const int64_t count = cols * d->dim;
            xent_fold<T><<<(unsigned)((count + 255) / 256), 256, 0, st>>>(c.sums, p.dw_splits, count, to);
        }
    }
    if (p.dh_splits > 1) {
        const int64_t count = p.rows * d->dim;
        xent_fold<T><<<(unsigned)((count + 255) / 256), 256, 0, st>>>((float*)(ws + p.dh_sums), p.dh_splits, count, (T*)dh);
    }
    return finish();
}

template <typename T>
__global__ __launch_bounds__(256) void xent_zero(T* p, int64_t count)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < count) p[i] = (T)0.f;
}

}  // namespace
}  // namespace gconv

using namespace gconv;

extern "C" {

int gconv_xent_workspace_size(const gconv_xent_desc* d, int op, size_t* bytes)
{
    const int st = check_desc(d);
    if (st != GCONV_OK) return st;
    if (op != GCONV_XENT_FWD && op != GCONV_XENT_BWD) return fail(GCONV_ERR_ARG, "unknown op %d", op);
    if (!bytes) return fail(GCONV_ERR_NULL, "bytes pointer is NULL");
    Plan p{};
    make_plan(d, op == GCONV_XENT_BWD, &p);
    *bytes = p.bytes;
    return GCONV_OK;
}

int gconv_xent_fwd(const gconv_xent_desc* d, const void* h, const void* w, const void* targets, float* loss, float* lse, void* workspace,
                   size_t workspace_bytes, void* stream)
{
    int st = check_desc(d);
    if (st != GCONV_OK) return st;
    const int64_t rows = d->sequences * d->tokens, es = d->dtype == GCONV_BF16 ? 2 : 4, is = d->index == GCONV_I64 ? 8 : 4;
    if (!w || (rows > 0 && (!h || !targets || !loss || !lse))) return fail(GCONV_ERR_NULL, "h, w, targets, loss and lse must be non-NULL");
    if (as_it_is(d) && ((uintptr_t)w & 15) != 0) return fail(GCONV_ERR_ARG, "w %p is not 16-byte aligned", w);
    const Span in[] = {strided_span(h, es, d->sequences, d->h_stride[0], d->tokens, d->h_stride[1], 1, 0, d->dim), {w, d->vocab * d->dim * es},
                       {targets, rows * is}};
    const Span out[] = {{loss, rows * 4}, {lse, rows * 4}};
    st = check_overlap(in, out);
    if (st != GCONV_OK) return st;
    Plan p{};
    make_plan(d, false, &p);
    st = check_launches(d, p, false);
    if (st != GCONV_OK) return st;
    st = check_workspace(workspace, workspace_bytes, p.bytes);
    if (st != GCONV_OK) return st;
    (void)hipGetLastError();
    if (rows == 0) return finish();
    if (d->dtype == GCONV_BF16) return forward<__bf16>(d, p, h, w, targets, loss, lse, (char*)workspace, (hipStream_t)stream);
    return forward<float>(d, p, h, w, targets, loss, lse, (char*)workspace, (hipStream_t)stream);
}

int gconv_xent_bwd(const gconv_xent_desc* d, const float* dloss, const float* dlse, const void* h, const void* w, const void* targets,
                   const float* lse, void* dh, void* dw, void* workspace, size_t workspace_bytes, void* stream)
{
    int st = check_desc(d);
    if (st != GCONV_OK) return st;
    const int64_t rows = d->sequences * d->tokens, es = d->dtype == GCONV_BF16 ? 2 : 4, is = d->index == GCONV_I64 ? 8 : 4;
    if (!w || !dw || (rows > 0 && (!h || !targets || !dloss || !lse || !dh)))
        return fail(GCONV_ERR_NULL, "dloss, h, w, targets, lse, dh and dw must be non-NULL");
    if (as_it_is(d) && ((uintptr_t)w & 15) != 0) return fail(GCONV_ERR_ARG, "w %p is not 16-byte aligned", w);
    const Span in[] = {strided_span(h, es, d->sequences, d->h_stride[0], d->tokens, d->h_stride[1], 1, 0, d->dim), {w, d->vocab * d->dim * es},
                       {targets, rows * is}, {dloss, rows * 4}, {dlse, rows * 4}, {lse, rows * 4}};
    const Span out[] = {{dh, rows * d->dim * es}, {dw, d->vocab * d->dim * es}};
    st = check_overlap(in, out);
    if (st != GCONV_OK) return st;
    Plan p{};
    make_plan(d, true, &p);
    st = check_launches(d, p, true);
    if (st != GCONV_OK) return st;
    st = check_workspace(workspace, workspace_bytes, p.bytes);
    if (st != GCONV_OK) return st;
    hipStream_t hs = (hipStream_t)stream;
    (void)hipGetLastError();
    if (rows == 0) {
        const int64_t count = d->vocab * d->dim;
        if ((count + 255) / 256 > max_blocks(256)) return fail(GCONV_ERR_UNSUPPORTED, "too many elements for a launch");
        if (d->dtype == GCONV_BF16) xent_zero<<<(unsigned)((count + 255) / 256), 256, 0, hs>>>((__bf16*)dw, count);
        else xent_zero<<<(unsigned)((count + 255) / 256), 256, 0, hs>>>((float*)dw, count);
        return finish();
    }
    if (d->dtype == GCONV_BF16) return backward<__bf16>(d, p, dloss, dlse, lse, h, w, targets, dh, dw, (char*)workspace, hs);
    return backward<float>(d, p, dloss, dlse, lse, h, w, targets, dh, dw, (char*)workspace, hs);
}

}  // extern "C"
