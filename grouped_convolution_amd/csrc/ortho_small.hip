// ortho_small.hip -- the orthogonalised update of matrices of at most 96 rows,
// or 128 rows of at most 256 columns (gfx950): few products, so what counts is
// the number of launches and the waits between them.
//
// A workgroup of eight waves keeps a block of X's columns in LDS with the
// m x m matrices beside it. A short X is one workgroup's and one launch does
// everything. Of a longer one the columns are dealt to blocks, and one launch
// does a round of all of them:
//
//   A = sum of the blocks' Gram matrices (of the last launch), A^2 and B, by
//   every block for itself; X' = a X + B X and its Gram matrix, of the block.
//
// So a round is one launch, and the blocks meet only in the float32 partial
// Gram matrices, which all of them add in the same order. What bounds it is
// the chain of short steps with a barrier after each: of 128 x 128, one
// product with its split takes 4 us where its matrix instructions need 1.3.
// (20 x 30: 12 us, the general kernels 63; 64 x 64: 19 for 63; 32 groups of
// 64 x 640: 57 for 81; 64 x 10000: 87 for 222.)
//
// A and B are split into two fp16 parts each (22 bits): with so few products
// the second part is nearly free, and small matrices average less rounding
// away (20 x 30: 2.1e-3 off where one part gives 2.7e-3; 100 x 100: 1.9e-3
// for 2.2e-3, the bf16 output's own rounding being 1.7e-3).
#include <algorithm>

#include "ortho_internal.h"

namespace gconv {
namespace {

constexpr int kThreads = kSmallThreads;

enum Mode { WHOLE = 0, START = 1, ROUND = 2 };

// By rows up to 32, 64, 96, 128. kWholeCols: columns up to which one workgroup
// takes a whole matrix; past them several are quicker (32 x 2000: 34 us for
// 69; 64 x 500: 45 both ways; 96 x 640: 67 for 90; 128 x 256: 70, and so the
// general kernels). kBlockCols: the most columns of one of several.
// kMoreBlocks: blocks of kShortCols columns up to which more blocks are
// quicker than longer ones, for all that each adds up all blocks' sums.
constexpr int kWholeCols[4] = {704, 512, 448, 256};
constexpr int kBlockCols[3] = {1024, 512, 320};
constexpr int kMoreBlocks[3] = {64, 24, 12};
constexpr int kShortCols = 128;

struct Small {
    OrthoArgs o;
    int blocks, cols;  // of a group; of a block, a multiple of 64
    int step;          // ROUND: its number
};

// The threads' share of the 16-byte pieces of X is moved so that the 8 rows
// a fragment's lanes read together, and the 4 + 4 rows of a transposing
// read, lie in different banks.
__device__ __forceinline__ int x_swz(int row) { return (row & 7) ^ ((row >> 1) & 4); }

// A barrier for LDS alone: a wave's stores to memory, which only itself reads
// again, need not have arrived.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
}

template <int FT, typename T, int MODE>
__global__ __launch_bounds__(kThreads, 1) void ortho_small_kernel(Small a)
{
    constexpr int MP = 32 * FT;               // rows, padded with zeros
    constexpr int XP = (MODE == WHOLE ? kWholeCols[FT - 1] : kBlockCols[FT - 1 < 2 ? FT - 1 : 2]) * 2;
    constexpr int MPITCH = MP * 2 + 16;       // of A's and B's parts
    constexpr int PART = MP * MPITCH;
    __shared__ __align__(16) char X[MP * XP];
    __shared__ __align__(16) char R[2 * PART];  // A or B: high and low parts; or float32 tiles on their way
    __shared__ double red[kThreads / 64];

    const OrthoArgs& o = a.o;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int team = wave >> 2, br = wave >> 1 & 1, bc = wave & 1;  // half of the reduction; quarter of the m x m matrix
    const int grp = blockIdx.x / a.blocks, blk = blockIdx.x % a.blocks;
    const int col0 = blk * a.cols, cols = min(a.cols, o.np - col0);
    const int64_t xbase = grp * o.xs + col0;
    const T* u = (const T*)o.u + grp * o.us;
    auto x_at = [&](int row, int piece) { return X + row * XP + ((piece ^ x_swz(row)) * 16); };

    // ---- X's block into LDS
    if constexpr (MODE == ROUND) {
        // 16 bytes a lane, straight to LDS; rows past the last read 0
        const u4 rs = resource(o.x + grp * o.xs, (uint32_t)o.m * o.np * 2);
        const uint32_t at = (uint32_t)(uintptr_t)(lds_char*)X;
        for (int i = wave; i < MP * XP / 1024; i += kThreads / 64) {
            const int q = i * 64 + lane, row = q / (XP / 16), c = (q % (XP / 16)) ^ x_swz(row);
            copy_lds(rs, at + i * 1024, row < o.m && c * 8 < cols ? (uint32_t)((row * o.np + col0 + c * 8) * 2) : kOOB);
        }
    } else {
        constexpr int E = 16 / sizeof(T);
        double s = 0;
        if constexpr (MODE == WHOLE) {
            constexpr int U = 8;  // loads in flight
            if (((uintptr_t)u & 15) == 0) {
                const int64_t whole = o.us / E;
                for (int64_t i = tid; i < whole; i += U * kThreads) {
                    u4 raw[U];
#pragma unroll
                    for (int k = 0; k < U; ++k) raw[k] = i + k * kThreads < whole ? ((const u4*)u)[i + k * kThreads] : u4{0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        struct Pack { T e[E]; } p = __builtin_bit_cast(Pack, raw[k]);
#pragma unroll
                        for (int e = 0; e < E; ++e) s = fma((double)(float)p.e[e], (double)(float)p.e[e], s);
                    }
                }
                const int64_t i = whole * E + tid;
                if (i < o.us) s = fma((double)(float)u[i], (double)(float)u[i], s);
            } else {
                for (int64_t i = tid; i < o.us; i += U * kThreads) {
                    float v[U];
#pragma unroll
                    for (int k = 0; k < U; ++k) v[k] = i + k * kThreads < o.us ? (float)u[i + k * kThreads] : 0.f;
#pragma unroll
                    for (int k = 0; k < U; ++k) s = fma((double)v[k], (double)v[k], s);
                }
            }
        } else {
            for (int i = tid; i < o.norm_blocks; i += kThreads) s += o.norm_part[(int64_t)grp * o.norm_blocks + i];
        }
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m);
        if (lane == 0) red[wave] = s;
        __syncthreads();
        s = red[0];
#pragma unroll
        for (int w = 1; w < kThreads / 64; ++w) s += red[w];
        const double f = (double)kScale / (sqrt(s) + o.eps);
        const int per = cols / 8, pieces = MP * per;
        const bool vec = !o.tall && ((uintptr_t)u & 15) == 0 && o.cols % E == 0;
        constexpr int U = 4;  // pieces in flight
        for (int i0 = tid; i0 < pieces; i0 += U * kThreads) {
            float v[U][8];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                // neighbouring threads along U's rows
                const int i = i0 + k * kThreads, row = o.tall ? i % MP : i / per, c = o.tall ? i / MP : i % per;
                const int col = col0 + c * 8;
                const bool live = i < pieces && row < o.m;
                if (vec) {
#pragma unroll
                    for (int e = 0; e < 8; e += E) {
                        struct __attribute__((aligned(16))) Pack { T e[E]; } p = {};
                        if (live && col + e < o.n) p = *(const Pack*)(u + (int64_t)row * o.cols + col + e);
#pragma unroll
                        for (int q = 0; q < E; ++q) v[k][e + q] = (float)p.e[q];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[k][e] = 0.f;
                        if (live && col + e < o.n)
                            v[k][e] = (float)u[o.tall ? (int64_t)(col + e) * o.cols + row : (int64_t)row * o.cols + col + e];
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int i = i0 + k * kThreads, row = o.tall ? i % MP : i / per, c = o.tall ? i / MP : i % per;
                if (i >= pieces) break;
                struct Piece { h4 h[2]; } hi, lo;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f4 w;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        // zeros outside the matrix even where the factor is not finite
                        const bool in = row < o.m && col0 + c * 8 + e * 4 + r < o.n;
                        w[r] = in ? (float)((double)v[k][e * 4 + r] * f) : 0.f;
                    }
                    hi.h[e] = split4(w, &lo.h[e]);
                }
                *(u4*)x_at(row, c) = __builtin_bit_cast(u4, hi);
                if (row < o.m) {
                    const int64_t at = xbase + (int64_t)row * o.np + c * 8;
                    if (o.steps > kRestSteps) *(u4*)(o.rest + at) = __builtin_bit_cast(u4, lo);
                    if (MODE == START) *(u4*)(o.x + at) = __builtin_bit_cast(u4, hi);
                }
            }
        }
        __syncthreads();
    }

    // A wave's quarter of an m x m matrix, FT x FT tiles. With an even FT the
    // teams number the rows of tiles apart, so that the first OWN of either
    // are the ones it keeps when the two halves of a sum are exchanged; else
    // the first team keeps all.
    typedef f4 Quarter[FT][FT];
    constexpr int OWN = FT % 2 == 0 ? FT / 2 : FT;
    const bool owner = FT % 2 == 0 || team == 0;
    auto tile_row = [&](int i) { return br * FT + (i + (FT % 2 == 0 ? team * OWN : 0)) % FT; };
    auto tile_col = [&](int j) { return bc * FT + j; };
    auto zero = [&](Quarter& q) {
#pragma unroll
        for (int i = 0; i < FT; ++i)
#pragma unroll
            for (int j = 0; j < FT; ++j) q[i][j] = f4{0, 0, 0, 0};
    };
    // Tiles as they lie in registers: [row][column][lane].
    auto tile_at = [&](char* base, int i, int j) { return (f4*)base + (tile_row(i) * (2 * FT) + tile_col(j)) * 64 + lane; };
    // Each team's tiles get the other's sums.
    auto combine = [&](Quarter& q) {
        if (FT % 2 == 0 || team == 1) {
#pragma unroll
            for (int i = FT % 2 == 0 ? OWN : 0; i < FT; ++i)
#pragma unroll
                for (int j = 0; j < FT; ++j) *tile_at(R, i, j) = q[i][j];
        }
        lds_barrier();
        if (owner) {
#pragma unroll
            for (int i = 0; i < OWN; ++i)
#pragma unroll
                for (int j = 0; j < FT; ++j) q[i][j] += *tile_at(R, i, j);
        }
        lds_barrier();
    };
    // The matrix into R, in two fp16 parts.
    auto put = [&](const Quarter& q) {
        if (owner) {
#pragma unroll
            for (int i = 0; i < OWN; ++i)
#pragma unroll
                for (int j = 0; j < FT; ++j) {
                    char* p = R + (tile_row(i) * 16 + li) * MPITCH + (tile_col(j) * 16 + 4 * g) * 2;
                    const h4 hi = half4(q[i][j]);
                    f4 left;
#pragma unroll
                    for (int r = 0; r < 4; ++r) left[r] = q[i][j][r] - (float)hi[r];
                    *(h4*)p = hi;
                    *(h4*)(p + PART) = half4(left);
                }
        }
        lds_barrier();
    };
    auto m_frag = [&](int part, int tile, int ks) {
        return *(const u4*)(R + part * PART + (tile * 16 + li) * MPITCH + ks * 64 + g * 16);
    };

    // X X^T of the block: each team half of the columns.
    auto gram = [&](Quarter& q) {
        zero(q);
        const int half = cols / 64;
        for (int ks = team * half; ks < (team + 1) * half; ++ks) {
            u4 fq[FT], fp[FT];
#pragma unroll
            for (int i = 0; i < FT; ++i) {
                fq[i] = *(const u4*)x_at(tile_row(i) * 16 + li, ks * 4 + g);
                fp[i] = *(const u4*)x_at(tile_col(i) * 16 + li, ks * 4 + g);
            }
#pragma unroll
            for (int i = 0; i < FT; ++i)
#pragma unroll
                for (int j = 0; j < FT; ++j) q[i][j] = mma16(fp[j], fq[i], q[i][j]);
        }
        combine(q);
    };
    // B = b A + c A^2 into R, from A (its tiles with their owners).
    auto polynomial = [&](const Quarter& A) {
        put(A);
        Quarter q;
        zero(q);
#pragma unroll 1
        for (int ks = team; ks < FT; ks += 2) {
            u4 ph[FT], pl[FT];
#pragma unroll
            for (int j = 0; j < FT; ++j) {
                ph[j] = m_frag(0, tile_col(j), ks);
                pl[j] = m_frag(1, tile_col(j), ks);
            }
#pragma unroll
            for (int i = 0; i < FT; ++i) {
                const u4 qh = m_frag(0, tile_row(i), ks), ql = m_frag(1, tile_row(i), ks);
#pragma unroll
                for (int j = 0; j < FT; ++j) q[i][j] = mma16(ph[j], qh, q[i][j]);
#pragma unroll
                for (int j = 0; j < FT; ++j) q[i][j] = mma16(ph[j], ql, q[i][j]);
#pragma unroll
                for (int j = 0; j < FT; ++j) q[i][j] = mma16(pl[j], qh, q[i][j]);
            }
        }
        lds_barrier();  // A has been read
        combine(q);
#pragma unroll
        for (int i = 0; i < OWN; ++i)
#pragma unroll
            for (int j = 0; j < FT; ++j) q[i][j] = q[i][j] * (kC / kScale) + A[i][j] * kB;
        put(q);
    };
    // Of a group: past the end where a row or column is not there, so none of
    // these accesses needs a branch.
    const uint32_t xbytes = (uint32_t)o.m * o.np * 2;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(o.x + grp * o.xs, xbytes), rr = make_rsrc(o.rest + grp * o.xs, xbytes);
    const __amdgpu_buffer_rsrc_t ro = make_rsrc((__bf16*)o.out + grp * o.us, (uint32_t)o.us * 2);
    const int tiles = cols / 16;
    auto rest_at = [&](int t0, int it, int t) {
        const int row = it * 16 + li, jt = t0 + t * 8;
        return row < o.m && jt < tiles ? (uint32_t)((row * o.np + col0 + jt * 16 + 4 * g) * 2) : kOOB;
    };
    u2 rest[2 * FT][2];
    auto fetch_rest = [&](int step, int t0) {
#pragma unroll
        for (int it = 0; it < 2 * FT; ++it)
#pragma unroll
            for (int t = 0; t < 2; ++t) rest[it][t] = u2{0, 0};
        if (o.steps - step > kRestSteps) {
#pragma unroll
            for (int it = 0; it < 2 * FT; ++it)
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    rest[it][t] = __builtin_bit_cast(u2, __builtin_amdgcn_raw_buffer_load_b64(rr, rest_at(t0, it, t), 0, 0));
        }
    };
    // X' = a X + B X, tiles of 16 columns by turns, two of a wave's at a time.
    auto update = [&](int step) {
        const bool last = step + 1 == o.steps;
        const bool write_rest = o.steps - step - 1 > kRestSteps;
        for (int t0 = wave; t0 < tiles; t0 += 16) {
            const bool two = t0 + 8 < tiles;
            auto at = [&](int it, int t) { return rest_at(t0, it, t); };
            if (t0 != wave || MODE != ROUND) fetch_rest(step, t0);
            u4 fp[2][FT];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int jt = t == 1 && two ? t0 + 8 : t0;
#pragma unroll
                for (int ks = 0; ks < FT; ++ks) {
                    const int row = ks * 32 + 8 * g + (li >> 2), piece = 2 * jt + (li >> 1 & 1);
                    const char *p0 = x_at(row, piece) + (li & 1) * 8, *p1 = x_at(row + 4, piece) + (li & 1) * 8;
                    const u2 lo = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p0));
                    const u2 hi = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p1));
                    fp[t][ks] = u4{lo[0], lo[1], hi[0], hi[1]};
                }
            }
#pragma unroll
            for (int it = 0; it < 2 * FT; ++it) {
                const int row = it * 16 + li;
                f4 v[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
                for (int ks = 0; ks < FT; ++ks) {
                    const u4 qh = m_frag(0, it, ks), ql = m_frag(1, it, ks);
#pragma unroll
                    for (int t = 0; t < 2; ++t) v[t] = mma16(fp[t][ks], qh, v[t]);
#pragma unroll
                    for (int t = 0; t < 2; ++t) v[t] = mma16(fp[t][ks], ql, v[t]);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t == 1 && !two) break;
                    h4* xp = (h4*)(x_at(row, 2 * (t0 + t * 8) + (g >> 1)) + (g & 1) * 8);
                    const h4 old = *xp, more = __builtin_bit_cast(h4, rest[it][t]);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        v[t][r] = fmaf(kA, fmaf((float)more[r], 1.f / kRest, (float)old[r]), v[t][r] * (1.f / kScale));
                    if (!last) {
                        h4 left;
                        const h4 hi = split4(v[t], &left);
                        *xp = hi;
                        if (write_rest) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, left), rr, at(it, t), 0, 0);
                        if (MODE == ROUND) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, hi), rx, at(it, t), 0, 0);
                        continue;
                    }
                    v[t] *= 1.f / kScale;
                    const int col = col0 + (t0 + t * 8) * 16 + 4 * g;
                    if (!o.tall && (o.n & 3) == 0) {
                        const uint32_t to = row < o.m && col < o.n ? (uint32_t)((row * o.n + col) * 2) : kOOB;
                        __builtin_amdgcn_raw_buffer_store_b64(pack4(v[t]), ro, to, 0, 0);
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint32_t to = row < o.m && col + r < o.n
                                                    ? (uint32_t)((o.tall ? (col + r) * o.m + row : row * o.n + col + r) * 2) : kOOB;
                            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v[t][r]), ro, to, 0, 0);
                        }
                    }
                }
            }
        }
    };

    constexpr int64_t kTiles = (int64_t)MP * MP;  // floats of a partial Gram matrix
    Quarter A;
    if constexpr (MODE == WHOLE) {
        for (int step = 0; step < o.steps; ++step) {
            gram(A);
#pragma unroll
            for (int i = 0; i < FT; ++i)
#pragma unroll
                for (int j = 0; j < FT; ++j) A[i][j] *= 1.f / kScale;
            polynomial(A);
            update(step);
            lds_barrier();
        }
        return;
    }
    // partial Gram matrices: of launch k in buffer k & 1
    float* parts = o.gram_part + (o.groups * ((MODE == START ? 0 : a.step + 1) & 1) + grp) * a.blocks * kTiles;
    if constexpr (MODE == ROUND) {
        const float* from = o.gram_part + (o.groups * (a.step & 1) + grp) * a.blocks * kTiles;
        zero(A);
        constexpr int U = FT == 1 ? 8 : FT == 2 ? 4 : 2;  // blocks' tiles in flight
#pragma unroll U
        for (int b = team; b < a.blocks; b += 2)  // one team the even blocks, one the odd
#pragma unroll
            for (int i = 0; i < FT; ++i)
#pragma unroll
                for (int j = 0; j < FT; ++j) A[i][j] += *tile_at((char*)(from + b * kTiles), i, j);
        wait_loads<0>();  // X's block is in LDS; combine's barriers tell the other waves
        combine(A);
        fetch_rest(a.step, wave);
#pragma unroll
        for (int i = 0; i < FT; ++i)
#pragma unroll
            for (int j = 0; j < FT; ++j) A[i][j] *= 1.f / kScale;
        polynomial(A);
        update(a.step);
        if (a.step + 1 == o.steps) return;
        lds_barrier();
    }
    gram(A);
    if (owner) {
#pragma unroll
        for (int i = 0; i < OWN; ++i)
#pragma unroll
            for (int j = 0; j < FT; ++j) *tile_at((char*)(parts + blk * kTiles), i, j) = A[i][j];
    }
}

template <int FT, typename T>
void run(const Small& s, hipStream_t st)
{
    const unsigned grid = (unsigned)(s.o.groups * s.blocks);
    if (FT == 4 || s.blocks == 1) {
        ortho_small_kernel<FT, T, WHOLE><<<grid, kThreads, 0, st>>>(s);
        return;
    }
    if constexpr (FT < 4) {
        ortho_launch_norm(s.o, st);
        ortho_small_kernel<FT, T, START><<<grid, kThreads, 0, st>>>(s);
        Small r = s;
        for (r.step = 0; r.step < s.o.steps; ++r.step) ortho_small_kernel<FT, T, ROUND><<<grid, kThreads, 0, st>>>(r);
    }
}

template <typename T>
void run_rows(const Small& s, hipStream_t st)
{
    switch ((s.o.m + 31) / 32) {
        case 1: return run<1, T>(s, st);
        case 2: return run<2, T>(s, st);
        case 3: return run<3, T>(s, st);
        default: return run<4, T>(s, st);
    }
}

}  // namespace

int ortho_small_blocks(int64_t m, int64_t np)
{
    if (m > 128) return 0;
    const int ft = (int)(m + 31) / 32 - 1;
    if (np <= kWholeCols[ft]) return 1;
    // Above 96 rows the general kernels are quicker (2 groups of 128 x 1200: 84
    // us, 112 by several workgroups here; 128 x 10000: 206 and 226).
    if (m > 96) return 0;
    // Every block adds up all blocks' Gram matrices: past 64 of them (of up to
    // 36 KB) the general kernels take over.
    const int64_t least = (np + kBlockCols[ft] - 1) / kBlockCols[ft];
    if (least > 64) return 0;
    return (int)std::max<int64_t>(least, std::min<int64_t>(np / kShortCols, kMoreBlocks[ft]));
}

size_t ortho_small_gram_bytes(int64_t m, int blocks)
{
    const int64_t mp = (m + 31) / 32 * 32;
    return blocks > 1 ? (size_t)(2 * blocks * mp * mp * 4) : 0;
}

void ortho_small(const OrthoArgs& a, int blocks, hipStream_t st)
{
    Small s{a, blocks, 0, 0};
    s.cols = (a.np / 64 + blocks - 1) / blocks * 64;  // about the same for each
    s.blocks = (a.np + s.cols - 1) / s.cols;
    if (a.bf16) run_rows<__bf16>(s, st);
    else run_rows<float>(s, st);
}

}  // namespace gconv
