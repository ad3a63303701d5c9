// ortho.hip -- the orthogonalised update of a weight gradient (gfx950).
//
// Each group's gradient U, as an m x n matrix (m <= n; a tall one is taken
// transposed), is scaled to norm 1 and sent through `steps` rounds of
//
//   A = X X^T      B = b A + c A^2      X' = a X + B X
//
// (Newton-Schulz: the polynomial a s + b s^3 + c s^5 of every singular value,
// which brings them all near 1). All three are matrix products of one kernel:
//
//   GRAM    A[i][j]  = sum_k X[i][k] X[j][k]   tiles with i <= j, mirrored
//   SQUARE  B[i][j]  = b A[i][j] + c sum_k A[i][k] A[j][k]   likewise
//   UPDATE  X'[i][j] = a X[i][j] + sum_k B[i][k] X[k][j]
//
// Bound by the matrix pipes and the power they draw: 5 rounds of 4096 x 9216
// are 2.7 TFLOP with the symmetric halves left out and take 2.55 ms, 1.04
// PFLOP/s; the loops over stages run at 1.22 (a large fp16 library product
// reaches 1.39 here), and zeros in place of data, which draw less power, take a
// sixth less. What is left outside the loops is the update's epilogue, 28 us of
// each of its three rounds, in which all of the chip reads and writes X.
//
// X, A and B are kept in fp16, times 2^12, and the products in float32.
// Rounding them is what the matrix pipes ask for; fp16 has 11 bits where bf16
// has 8 and its short range is no matter: the entries of X, A and B are at
// most 1.3, 1.5 and 2.9 (the singular values stay below 1.21), and 2^12 puts
// everything above 2^-26 into fp16's normal range. After five rounds a random
// gradient of full rank is 1.5e-3 off the 64-bit result (in the 2-norm, before
// the bf16 output's own 1.7e-3) and one of low rank 2.8e-3, where bf16 operands
// would leave 1e-2 and 2e-2; a constant gradient, whose entries are all rounded
// the same way, is up to 1.5e-2 off. What fp16 leaves of X is kept
// too and joins the term a X: directions that hold next to nothing of the
// gradient grow by a in every round, 485 times in five, and rounding noise
// there would grow with them (a rank-one gradient came back 15% off).
#include <algorithm>

#include "gconv.h"
#include "ortho_internal.h"

namespace gconv {
namespace {

constexpr int kStepK = 64;        // reduction length of a stage

enum Op { GRAM = 0, SQUARE = 1, UPDATE = 2 };

struct Ortho {
    const h16* x;    // [groups][m][np]
    h16* rest;       // 2^11 times what x leaves of X; UPDATE replaces it in place
    const h16* s;    // SQUARE: A, UPDATE: B, [groups][m][mp]
    h16* out;        // A, B or X'
    void* last;      // UPDATE: the bf16 result, NULL before the last step
    int64_t xs, ss;  // elements of a group's X, of its A
    int64_t us;      // of its gradient
    int m, n, np, mp;  // np, mp: row pitches, multiples of 64 (zeros past n, m)
    int tq, tp;      // tiles along the rows and columns of the output
    int tall;        // the result is stored transposed, [n][m]
    int read_rest, write_rest;
};

// Stage of an operand whose reduction runs along its rows in memory: [R][64]
// elements, the 16-byte pieces of row r at piece ^ (r & 7), so the 8 lanes
// that are served together read 8 different sets of banks.
template <int R, int NW>
struct AlongRows {
    static constexpr int kLoads = R / 8 / NW;
    static constexpr int kBytes = R * 128;
    static_assert(R % (8 * NW) == 0, "whole loads a wave");
    uint32_t off[kLoads];  // byte offsets of this lane's pieces; rows past the last read 0
    uint32_t at[2];        // of this lane's first fragment of either half
    __device__ __forceinline__ void init(int row0, int rows, int pitch, int wave, int lane, int frag0)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = (i * NW + wave) * 8 + (lane >> 3);
            off[i] = row0 + r < rows ? (uint32_t)(((row0 + r) * (int64_t)pitch + (((lane & 7) ^ (r & 7)) * 8)) * 2) : kOOB;
        }
        const int li = lane & 15, g = lane >> 4;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) at[ks] = (frag0 + li) * 128 + (((ks * 4 + g) ^ (li & 7)) * 16);
    }
    __device__ __forceinline__ void load(u4 rs, uint32_t tile, int i, int wave)
    {
        copy_lds(rs, tile + (i * NW + wave) * 1024, off[i]);
        off[i] += kStepK * 2;
    }
    __device__ __forceinline__ u4 frag(const char* tile, int t, int ks) const
    {
        return *(const u4*)(tile + at[ks] + t * (16 * 128));
    }
};

// Stage of an operand whose reduction runs across its rows: [64][C] elements,
// read with transposing loads (16 lanes: 4 rows x 16 columns). The 32-byte
// pieces of a row are swizzled so that the eight rows of 32 lanes lie in
// different banks.
template <int C, int NW, int FRAGS>
struct AcrossRows {
    static constexpr int kPieces = C / 8;
    static constexpr int kLoads = kStepK * kPieces / 64 / NW;
    static constexpr int kBytes = kStepK * C * 2;
    static_assert(kStepK * kPieces % (64 * NW) == 0, "whole loads a wave");
    uint32_t off[kLoads];
    uint32_t step;
    uint32_t at[FRAGS];
    static __device__ __forceinline__ int swz(int row)
    {
        return C % 128 == 0 ? (row & 3) | ((row >> 1) & 4) : ((row >> 1) & 1) | ((row >> 2) & 2);
    }
    // rows past the last lie past the resource's end, below 2^32
    __device__ __forceinline__ void init(int col0, int, int pitch, int wave, int lane, int frag0)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = (i * NW + wave) * 64 + lane, row = q / kPieces, p = q % kPieces;
            off[i] = (uint32_t)(((int64_t)row * pitch + col0 + ((p ^ (swz(row) << 1)) * 8)) * 2);
        }
        step = (uint32_t)kStepK * (uint32_t)pitch * 2;  // 2^31 at the longest side
        const int li = lane & 15, g = lane >> 4;
        const int row = 8 * g + (li >> 2);  // rows + 4 and + 32 have the same swizzle
#pragma unroll
        for (int t = 0; t < FRAGS; ++t)
            at[t] = row * (C * 2) + ((((frag0 >> 4) + t) ^ swz(row)) * 32) + (li & 3) * 8;
    }
    __device__ __forceinline__ void load(u4 rs, uint32_t tile, int i, int wave)
    {
        copy_lds(rs, tile + (i * NW + wave) * 1024, off[i]);
        off[i] += step;
    }
    __device__ __forceinline__ u4 frag(const char* tile, int t, int ks) const
    {
        const char* p = tile + at[t] + ks * (32 * C * 2);
        const u2 lo = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p));
        const u2 hi = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + 4 * C * 2)));
        return u4{lo[0], lo[1], hi[0], hi[1]};
    }
};

// Tile L of the triangle q <= p: columns of tiles, top to bottom.
__device__ __forceinline__ void triangle(int L, int* q, int* p)
{
    int j = (int)((sqrtf(8.f * (float)L + 1.f) - 1.f) * 0.5f);
    while (j * (j + 1) / 2 > L) --j;
    while ((j + 1) * (j + 2) / 2 <= L) ++j;
    *p = j;
    *q = L - j * (j + 1) / 2;
}

// One BQ x BP tile of an output. The matrix instruction's rows run along the
// output's columns, so a lane holds four consecutive elements of an output row.
// Eight waves, two a SIMD, so that one multiplies while the other waits (with
// four larger ones: Gram matrix 185 us for 151), over a ring of 64-long stages.
template <int BQ, int BP, int WQ, int WP, int OP>
__global__ __launch_bounds__(64 * WQ * WP, 1) void ortho_gemm(Ortho a)
{
    constexpr int NW = WQ * WP;
    constexpr int FQ = BQ / WQ / 16, FP = BP / WP / 16;
    using SQ = AlongRows<BQ, NW>;
    using SP = std::conditional_t<OP == UPDATE, AcrossRows<BP, NW, FP>, AlongRows<BP, NW>>;
    constexpr int kBuf = SQ::kBytes + SP::kBytes;
    constexpr int kLoads = SQ::kLoads + SP::kLoads;
    // Stages that the LDS of a CU holds, 3 at most, and 4 of the smallest tile,
    // whose stages are too short for a load to arrive in two of them (300 x 5000
    // 157 us for 176, 1024 x 2304 167 for 180; 8 groups of 512 x 512, which put
    // several workgroups on a CU, 123 for 118; 6 stages 171, 172, 151).
    constexpr int kRing = std::min(BQ == 64 ? 4 : 3, 160 * 1024 / kBuf);
    __shared__ __align__(1024) char lds[kRing * kBuf];

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wq = wave % WQ, wp = wave / WQ;
    const int per = OP == UPDATE ? a.tq * a.tp : a.tp * (a.tp + 1) / 2;
    const int b = xcd_remap(blockIdx.x, gridDim.x);
    const int grp = b / per, L = b - grp * per;
    int tq, tp;
    if (OP == UPDATE) {
        // strips of 8 tiles of rows: the blocks that run together on an XCD share their panels
        const int strip = L / (8 * a.tp), first = strip * 8, h = min(a.tq - first, 8), in = L - strip * 8 * a.tp;
        tq = first + in % h;
        tp = in / h;
    } else {
        triangle(L, &tq, &tp);
    }
    const int i0 = tq * BQ, j0 = tp * BP;
    const h16* x = a.x + grp * a.xs;
    const h16* s = a.s + grp * a.ss;
    const int kt_end = (OP == GRAM ? a.np : a.mp) / kStepK;
    const uint32_t xbytes = (uint32_t)a.m * a.np * 2, sbytes = (uint32_t)a.m * a.mp * 2;
    const u4 rq = OP == GRAM ? resource(x, xbytes) : resource(s, sbytes);
    const u4 rp = OP == SQUARE ? resource(s, sbytes) : resource(x, xbytes);
    SQ sq;
    SP sp;
    sq.init(i0, a.m, OP == GRAM ? a.np : a.mp, wave, lane, wq * (BQ / WQ));
    sp.init(j0, a.m, OP == SQUARE ? a.mp : a.np, wave, lane, wp * (BP / WP));

    f4 acc[FQ][FP];
#pragma unroll
    for (int i = 0; i < FQ; ++i)
#pragma unroll
        for (int j = 0; j < FP; ++j) acc[i][j] = f4{0, 0, 0, 0};

    const uint32_t lds_at = (uint32_t)(uintptr_t)(lds_char*)lds;
    auto issue = [&](int n, uint32_t buf) {  // load n of a stage
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
            if (rd < FQ + FP && n * (FQ + FP) * 3 >= rd * kMmas * 2) read(ks ^ 1, rd++, from);
            if (ks == 1 && ld < kLoads && n * kLoads >= ld * kMmas) issue(ld++, into);
            const int i = n / FP, j = n % FP;
            acc[i][j] = mma16(fp[ks][j], fq[ks][i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
#pragma unroll
    for (int st = 0; st < kRing; ++st)
#pragma unroll
        for (int n = 0; n < kLoads; ++n) issue(n, st * kBuf);
    wait_loads<(kRing - 1) * kLoads>();
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int n = 0; n < FQ + FP; ++n) read(0, n, 0);
    __builtin_amdgcn_sched_barrier(0);
    // In the middle of a stage the next one has landed and this one has been
    // read by all waves, so the stage kRing on is loaded into its place. Loads
    // past the last stage are made and lead nowhere.
    uint32_t cur = 0;
    for (int kt = 0; kt < kt_end; ++kt) {
        const uint32_t next = cur + kBuf == kRing * kBuf ? 0 : cur + kBuf;
        half(0, cur, 0);
        wait_loads<(kRing - 2) * kLoads>();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        half(1, next, cur);
        cur = next;
    }
    wait_loads<0>();  // no load may land after the workgroup's end

    // Buffer accesses with offsets past the end where an element is not there:
    // no branches, so a row of fragments is loaded while the last is stored.
    auto offset = [&](int row, int col, int rows, int pitch) {
        return row < rows && col < pitch ? (uint32_t)((row * (int64_t)pitch + col) * 2) : kOOB;
    };
    const int row0 = i0 + wq * (BQ / WQ) + li, col0 = j0 + wp * (BP / WP) + 4 * g;
    if constexpr (OP == UPDATE) {
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(x, xbytes), rr = make_rsrc(a.rest + grp * a.xs, xbytes);
        const __amdgpu_buffer_rsrc_t ro = make_rsrc(a.out + grp * a.xs, xbytes);
        const __amdgpu_buffer_rsrc_t rl = make_rsrc((__bf16*)a.last + grp * a.us, a.last ? (uint32_t)a.us * 2 : 0);
        h4 old[2][FP], old_rest[2][FP];
        auto fetch = [&](int i) {
#pragma unroll
            for (int j = 0; j < FP; ++j) {
                const uint32_t o = offset(row0 + i * 16, col0 + j * 16, a.m, a.np);
                old[i & 1][j] = __builtin_bit_cast(h4, __builtin_amdgcn_raw_buffer_load_b64(rx, o, 0, 0));
                if (a.read_rest) old_rest[i & 1][j] = __builtin_bit_cast(h4, __builtin_amdgcn_raw_buffer_load_b64(rr, o, 0, 0));
            }
        };
        fetch(0);
#pragma unroll
        for (int i = 0; i < FQ; ++i) {
            if (i + 1 < FQ) fetch(i + 1);
            const int row = row0 + i * 16;
#pragma unroll
            for (int j = 0; j < FP; ++j) {
                const int col = col0 + j * 16;
                f4 v = acc[i][j] * (1.f / kScale);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float o = (float)old[i & 1][j][r];
                    if (a.read_rest) o = fmaf((float)old_rest[i & 1][j][r], 1.f / kRest, o);
                    v[r] = fmaf(kA, o, v[r]);
                }
                if (!a.last) {
                    const uint32_t o = offset(row, col, a.m, a.np);
                    h4 left;
                    const h4 w = split4(v, &left);
                    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, w), ro, o, 0, 0);
                    if (a.write_rest) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, left), rr, o, 0, 0);
                    continue;
                }
                v *= 1.f / kScale;
                if (!a.tall && (a.n & 3) == 0) {
                    __builtin_amdgcn_raw_buffer_store_b64(pack4(v), rl, offset(row, col, a.m, a.n), 0, 0);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t o = a.tall ? offset(col + r, row, a.n, a.m) : offset(row, col + r, a.m, a.n);
                        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v[r]), rl, o, 0, 0);
                    }
                }
            }
        }
    } else {
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(s, sbytes), ro = make_rsrc(a.out + grp * a.ss, sbytes);
        h4 old[2][FP];
        auto fetch = [&](int i) {
#pragma unroll
            for (int j = 0; j < FP; ++j)
                old[i & 1][j] = __builtin_bit_cast(h4, __builtin_amdgcn_raw_buffer_load_b64(
                                                           rs, offset(row0 + i * 16, col0 + j * 16, a.m, a.mp), 0, 0));
        };
        if (OP == SQUARE) fetch(0);
#pragma unroll
        for (int i = 0; i < FQ; ++i) {
            if (OP == SQUARE && i + 1 < FQ) fetch(i + 1);
            const int row = row0 + i * 16;
#pragma unroll
            for (int j = 0; j < FP; ++j) {
                const int col = col0 + j * 16;
                f4 v = acc[i][j] * (1.f / kScale);
                if constexpr (OP == SQUARE) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] = fmaf(kC, v[r], kB * (float)old[i & 1][j][r]);
                }
                const h4 w = half4(v);
                __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, w), ro, offset(row, col, a.m, a.mp), 0, 0);
                if (tq != tp) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const h16 e = w[r];
                        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, e), ro, offset(col + r, row, a.m, a.mp), 0, 0);
                    }
                }
            }
        }
    }
}

// ---- scaling ---------------------------------------------------------------------
//
// The sum of squares of each group, in 64 bits so that no gradient is too
// large or too small, by blocks; then X = 2^12 U / (norm + eps) in fp16, rows
// padded with zeros to the pitch, transposed where U is tall.

constexpr int kNormThreads = 256;

struct Prep {
    const void* u;
    double* part;    // [groups][blocks]
    h16 *x, *rest;
    int64_t us, xs;
    int blocks, rows, cols;  // of U
    int np, tall;
    int vec, vec_rows;  // groups hold whole 16-byte pieces; rows whole fours, aligned
    double eps;
};

template <typename T>
__global__ __launch_bounds__(kNormThreads) void ortho_norm(Prep a)
{
    constexpr int E = 16 / sizeof(T);
    __shared__ double red[kNormThreads / 64];
    const int blk = blockIdx.x % a.blocks, grp = blockIdx.x / a.blocks;
    const T* u = (const T*)a.u + grp * a.us;
    double s = 0;
    if (a.vec) {
        for (int64_t i = ((int64_t)blk * kNormThreads + threadIdx.x) * E; i < a.us; i += (int64_t)a.blocks * kNormThreads * E) {
            struct Pack { T e[E]; } p = __builtin_bit_cast(Pack, *(const u4*)(u + i));
#pragma unroll
            for (int e = 0; e < E; ++e) s = fma((double)(float)p.e[e], (double)(float)p.e[e], s);
        }
    } else {
        for (int64_t i = (int64_t)blk * kNormThreads + threadIdx.x; i < a.us; i += (int64_t)a.blocks * kNormThreads)
            s = fma((double)(float)u[i], (double)(float)u[i], s);
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kNormThreads / 64; ++w) s += red[w];
        a.part[blockIdx.x] = s;
    }
}

// 64 x 64 of X a block.
template <typename T>
__global__ __launch_bounds__(256) void ortho_scale(Prep a)
{
    __shared__ float tile[64][65];
    __shared__ double factor;
    const int tr = a.tall ? (a.cols + 63) / 64 : (a.rows + 63) / 64, tc = a.np / 64;
    const int grp = blockIdx.x / (tr * tc), t = blockIdx.x % (tr * tc);
    const int r0 = t / tc * 64, c0 = t % tc * 64;
    if (threadIdx.x < 64) {
        double s = 0;
        for (int i = threadIdx.x; i < a.blocks; i += 64) s += a.part[(int64_t)grp * a.blocks + i];
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m);
        if (threadIdx.x == 0) factor = (double)kScale / (sqrt(s) + a.eps);
    }
    __syncthreads();
    const double f = factor;
    const T* u = (const T*)a.u + grp * a.us;
    const int q = threadIdx.x & 15, r = threadIdx.x >> 4;
    const int m = a.tall ? a.cols : a.rows;
    f4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        // a.tall: U's rows are X's columns
        const int ur = (a.tall ? c0 : r0) + r + k * 16, uc = (a.tall ? r0 : c0) + q * 4;
        v[k] = f4{0, 0, 0, 0};
        if (ur < a.rows) {
            const T* p = u + (int64_t)ur * a.cols + uc;
            if (a.vec_rows && uc < a.cols) {
                struct __attribute__((aligned(4 * sizeof(T)))) Four { T e[4]; } w = *(const Four*)p;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[k][e] = (float)((double)(float)w.e[e] * f);
            } else {
                // zeros past the row's end even where the factor is not finite
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (uc + e < a.cols) v[k][e] = (float)((double)(float)p[e] * f);
            }
        }
    }
    if (a.tall) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) tile[q * 4 + e][r + k * 16] = v[k][e];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[k][e] = tile[r + k * 16][q * 4 + e];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int row = r0 + r + k * 16;
        if (row >= m) continue;
        const int64_t at = grp * a.xs + (int64_t)row * a.np + c0 + q * 4;
        h4 left;
        *(h4*)(a.x + at) = split4(v[k], &left);
        *(h4*)(a.rest + at) = left;
    }
}

// ---- host ------------------------------------------------------------------------

int check_desc(const gconv_ortho_desc* d)
{
    if (!d) return fail(GCONV_ERR_NULL, "descriptor is NULL");
    if (d->dtype != GCONV_F32 && d->dtype != GCONV_BF16) return fail(GCONV_ERR_ARG, "unknown dtype %lld", (long long)d->dtype);
    if (d->filters < 1 || d->inner < 1 || d->groups < 1)
        return fail(GCONV_ERR_SHAPE, "need filters, inner, groups >= 1 (got %lld, %lld, %lld)", (long long)d->filters,
                    (long long)d->inner, (long long)d->groups);
    if (d->filters % d->groups != 0)
        return fail(GCONV_ERR_GROUPS, "filters=%lld not divisible by groups=%lld", (long long)d->filters, (long long)d->groups);
    if (d->steps < 1 || d->steps > 1000) return fail(GCONV_ERR_ARG, "steps=%lld must be 1..1000", (long long)d->steps);
    if (!(d->eps >= 0)) return fail(GCONV_ERR_ARG, "eps must be >= 0");
    return GCONV_OK;
}

struct Plan {
    int64_t m, n, mp, np, us, xs, ss, groups;
    int tall, blocks;
    int small;         // workgroups a group of the small kernels; 0: the general ones
    size_t x0, x1, rest, A, B, norm, gram, bytes;  // offsets in the workspace
};

int make_plan(const gconv_ortho_desc* d, Plan* p)
{
    const int64_t rows = d->filters / d->groups;
    constexpr int64_t kMost = (int64_t)1 << 29;     // elements of a matrix: byte offsets stay below 2^31
    constexpr int64_t kLongest = (int64_t)1 << 24;  // 64 rows past the last: below 2^32
    if (d->inner > kLongest || rows > kLongest) return fail(GCONV_ERR_UNSUPPORTED, "a group's matrix has a side above 2^24");
    p->groups = d->groups;
    p->tall = rows > d->inner;
    p->m = std::min(rows, d->inner);
    p->n = std::max(rows, d->inner);
    p->mp = (p->m + 63) / 64 * 64;
    p->np = (p->n + 63) / 64 * 64;
    p->us = rows * d->inner;
    p->xs = p->m * p->np;
    p->ss = p->m * p->mp;
    if (p->xs > kMost) return fail(GCONV_ERR_UNSUPPORTED, "a group's matrix has more than 2^29 elements");
    if (d->groups > ((int64_t)1 << 40) / p->xs || d->groups > (1 << 20))
        return fail(GCONV_ERR_UNSUPPORTED, "too many groups");
    // about 2048 workgroups in all, 16 elements or more a thread
    const int64_t want = std::max<int64_t>(1, 2048 / d->groups);
    p->blocks = (int)std::min<int64_t>(want, (p->us + kNormThreads * 16 - 1) / (kNormThreads * 16));
    p->small = ortho_small_blocks(p->m, p->np);
    // (no launch of the general kernels has more threads than one with a workgroup for each 64 x 64 of X)
    if (p->small > 0 ? d->groups * p->small > max_blocks(kSmallThreads)
                     : d->groups * (p->mp / 64) * (p->np / 64) > max_blocks(256))
        return fail(GCONV_ERR_UNSUPPORTED, "too many groups");
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += (n + 1023) / 1024 * 1024;
        return o;
    };
    const size_t g = (size_t)d->groups;
    p->rest = take(g * p->xs * 2);
    if (p->small != 1) {
        p->x0 = take(g * p->xs * 2);
        p->norm = take(g * p->blocks * 8);
    }
    if (p->small == 0) {
        p->x1 = take(g * p->xs * 2);
        p->A = take(g * p->ss * 2);
        p->B = take(g * p->ss * 2);
        take(1024);  // loads past a matrix's last stage read up to here
    } else {
        p->gram = take(g * ortho_small_gram_bytes(p->m, p->small));
    }
    p->bytes = at;
    return GCONV_OK;
}

template <int BQ, int BP, int WQ, int WP, int OP>
void launch(Ortho a, int64_t groups, hipStream_t st)
{
    a.tq = (a.m + BQ - 1) / BQ;
    a.tp = ((OP == UPDATE ? a.n : a.m) + BP - 1) / BP;
    const int64_t per = OP == UPDATE ? (int64_t)a.tq * a.tp : (int64_t)a.tp * (a.tp + 1) / 2;
    ortho_gemm<BQ, BP, WQ, WP, OP><<<(unsigned)(per * groups), 64 * WQ * WP, 0, st>>>(a);
}

// The tile whose whole rounds of 256 workgroups take least: its area over a
// rate, of which one set serves all three products, as it only has to put the
// tiles in order. It does: with one product's tile forced, at 16 sizes from 512
// x 512 to 4096 x 9216 and of 1 to 32 groups, no tile was quicker than the
// rule's by more than the noise of 2%. What others cost, us of a whole update:
//   4096 x 9216 (2585)  update 256x192; 256 +196, 192 +229, 128 +254
//                       Gram matrix 192; 256 +180, 128 +341; square 192; 256 +76
//   2048 x 8192 (745)   update 256; 192 +68, 128 +126; Gram 128; 192 +167, 64 +171
//   1500 x 6000 (469)   update 192; 256 +58, 128 +87; Gram 64; 128 +6, 192 +123
//   1024 x 2304 (169)   update 128; 64 +10, 192 +55; Gram 64; 128 +37, 192 +97
//   8 of 512 x 512 (122), 2 of 128 x 1200 (83): all 64; 128 +3 to +20
template <int OP>
void product(const Ortho& a, int64_t groups, hipStream_t st)
{
    struct Tile { int q, p; double rate; };
    constexpr Tile tiles[] = {{256, 256, 1.0}, {256, 192, 0.8}, {192, 192, 0.75}, {128, 128, 0.68}, {64, 64, 0.4}};
    int best = 0;
    double least = 0;
    for (int i = 0; i < 5; ++i) {
        const Tile& t = tiles[i];
        if (OP != UPDATE && t.q != t.p) continue;
        const int64_t tq = (a.m + t.q - 1) / t.q, tp = ((OP == UPDATE ? a.n : a.m) + t.p - 1) / t.p;
        const int64_t count = groups * (OP == UPDATE ? tq * tp : tp * (tp + 1) / 2);
        const double cost = (double)((count + 255) / 256) * t.q * t.p / t.rate;
        if (i == 0 || cost < least) {
            least = cost;
            best = i;
        }
    }
    switch (best) {
        case 0: return launch<256, 256, 2, 4, OP>(a, groups, st);
        case 1:
            if constexpr (OP == UPDATE) return launch<256, 192, 4, 2, OP>(a, groups, st);
            return;
        case 2: return launch<192, 192, 2, 4, OP>(a, groups, st);
        case 3: return launch<128, 128, 2, 4, OP>(a, groups, st);
        default: return launch<64, 64, 2, 2, OP>(a, groups, st);
    }
}

Prep prep(const OrthoArgs& a)
{
    const int64_t es = a.bf16 ? 2 : 4;
    Prep r{};
    r.u = a.u;
    r.part = a.norm_part;
    r.x = a.x;
    r.rest = a.rest;
    r.us = a.us;
    r.xs = a.xs;
    r.blocks = a.norm_blocks;
    r.rows = a.rows;
    r.cols = a.cols;
    r.np = a.np;
    r.tall = a.tall;
    r.vec = ((uintptr_t)a.u & 15) == 0 && a.us * es % 16 == 0;
    r.vec_rows = (uintptr_t)a.u % (4 * es) == 0 && a.cols % 4 == 0;
    r.eps = a.eps;
    return r;
}

}  // namespace

void ortho_launch_norm(const OrthoArgs& a, hipStream_t st)
{
    const Prep r = prep(a);
    const unsigned grid = (unsigned)(a.norm_blocks * a.groups);
    if (a.bf16) ortho_norm<__bf16><<<grid, kNormThreads, 0, st>>>(r);
    else ortho_norm<float><<<grid, kNormThreads, 0, st>>>(r);
}

}  // namespace gconv

using namespace gconv;

extern "C" {

int gconv_orthogonalize_workspace_size(const gconv_ortho_desc* d, size_t* bytes)
{
    int st = check_desc(d);
    if (st != GCONV_OK) return st;
    if (!bytes) return fail(GCONV_ERR_NULL, "bytes pointer is NULL");
    Plan p{};
    st = make_plan(d, &p);
    if (st != GCONV_OK) return st;
    *bytes = p.bytes;
    return GCONV_OK;
}

int gconv_orthogonalize(const gconv_ortho_desc* d, const void* u, void* out, void* workspace, size_t workspace_bytes, void* stream)
{
    int st = check_desc(d);
    if (st != GCONV_OK) return st;
    Plan p{};
    st = make_plan(d, &p);
    if (st != GCONV_OK) return st;
    if (!u || !out) return fail(GCONV_ERR_NULL, "u and out must be non-NULL");
    if (!workspace || workspace_bytes < p.bytes)
        return fail(GCONV_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace_bytes, p.bytes);
    if (((uintptr_t)workspace & 15) != 0) return fail(GCONV_ERR_WORKSPACE, "workspace pointer %p is not 16-byte aligned", workspace);
    if (((uintptr_t)out & 7) != 0) return fail(GCONV_ERR_ARG, "out %p is not 8-byte aligned", out);
    const int64_t es = d->dtype == GCONV_BF16 ? 2 : 4, count = p.us * p.groups;
    const char *ub = (const char*)u, *ob = (const char*)out;
    if (ub < ob + count * 2 && ob < ub + count * es) return fail(GCONV_ERR_ARG, "out overlaps u");
    hipStream_t hs = (hipStream_t)stream;
    (void)hipGetLastError();
    char* w = (char*)workspace;

    OrthoArgs o{};
    o.u = u;
    o.bf16 = d->dtype == GCONV_BF16;
    o.out = out;
    o.x = (h16*)(w + p.x0);
    o.rest = (h16*)(w + p.rest);
    o.norm_part = (double*)(w + p.norm);
    o.gram_part = (float*)(w + p.gram);
    o.groups = p.groups;
    o.steps = d->steps;
    o.us = p.us;
    o.xs = p.xs;
    o.rows = (int)(d->filters / d->groups);
    o.cols = (int)d->inner;
    o.m = (int)p.m;
    o.n = (int)p.n;
    o.np = (int)p.np;
    o.tall = p.tall;
    o.norm_blocks = p.blocks;
    o.eps = d->eps;
    if (p.small > 0) {
        ortho_small(o, p.small, hs);
        return finish();
    }

    ortho_launch_norm(o, hs);
    const unsigned ns = (unsigned)((p.m + 63) / 64 * (p.np / 64) * p.groups);
    if (o.bf16) ortho_scale<__bf16><<<ns, 256, 0, hs>>>(prep(o));
    else ortho_scale<float><<<ns, 256, 0, hs>>>(prep(o));

    Ortho a{};
    a.rest = (h16*)(w + p.rest);
    a.xs = p.xs;
    a.ss = p.ss;
    a.us = p.us;
    a.m = (int)p.m;
    a.n = (int)p.n;
    a.mp = (int)p.mp;
    a.np = (int)p.np;
    a.tall = p.tall;
    h16 *x = (h16*)(w + p.x0), *y = (h16*)(w + p.x1), *A = (h16*)(w + p.A), *B = (h16*)(w + p.B);
    for (int64_t i = 0; i < d->steps; ++i) {
        a.x = x;
        a.s = A;
        a.out = A;
        product<GRAM>(a, p.groups, hs);
        a.out = B;
        product<SQUARE>(a, p.groups, hs);
        a.s = B;
        a.out = y;
        a.last = i + 1 == d->steps ? out : nullptr;
        a.read_rest = d->steps - i > kRestSteps;
        a.write_rest = d->steps - i - 1 > kRestSteps;
        product<UPDATE>(a, p.groups, hs);
        std::swap(x, y);
    }
    return finish();
}

}  // extern "C"
