// ortho_internal.h -- what the kernels of the orthogonalised update share.
#pragma once

#include "device_util.h"
#include "gconv_internal.h"
#include "lds_copy.h"
#include "seq_util.h"

namespace gconv {

typedef _Float16 h16;
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScale = 4096.f;  // of X, A and B as they are stored
constexpr float kRest = 2048.f;    // of the rest of X, over X
// Rounds before the end that take X without its rest: noise of 2^-12 grows
// 12 times at most there, and without it the strong directions come out a
// little closer (128 x 1200: 2.3e-3 off for 2.4e-3; rank one 3.3e-3, and
// 1.4e-2 with one round more).
constexpr int kRestSteps = 2;

__device__ __forceinline__ f4 mma16(u4 a, u4 b, f4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

__device__ __forceinline__ h4 half4(f4 v)
{
    return h4{(h16)v[0], (h16)v[1], (h16)v[2], (h16)v[3]};
}

// v in fp16, and what that leaves, times kRest.
__device__ __forceinline__ h4 split4(f4 v, h4* rest)
{
    const h4 h = half4(v);
#pragma unroll
    for (int r = 0; r < 4; ++r) (*rest)[r] = (h16)((v[r] - (float)h[r]) * kRest);
    return h;
}

// A gradient, its matrices and where they are kept: [groups][m][np] of X (m the
// shorter side of a group's matrix) in fp16 and of what fp16 leaves of it.
struct OrthoArgs {
    const void* u;
    int bf16;            // u's type
    void* out;           // [groups][rows][cols] in bf16
    h16 *x, *rest;
    double* norm_part;   // [groups][norm_blocks]: sums of squares
    float* gram_part;    // of the small kernels: two buffers of [groups][blocks][mp][mp]
    int64_t groups, steps;
    int64_t us, xs;      // elements of a group's gradient, of its X
    int rows, cols;      // of a group's gradient
    int m, n, np;        // np: n up to a multiple of 64 (zeros)
    int tall;            // X is the transposed gradient
    int norm_blocks;
    double eps;
};

void ortho_launch_norm(const OrthoArgs& a, hipStream_t st);

// ---- at most 128 rows (ortho_small.hip) ------------------------------------------
constexpr int kSmallThreads = 512;
// Workgroups a group takes: 1 where its X fits one workgroup's LDS, 0 where
// the general kernels are the better choice.
int ortho_small_blocks(int64_t m, int64_t np);
size_t ortho_small_gram_bytes(int64_t m, int blocks);  // of both buffers, a group
void ortho_small(const OrthoArgs& a, int blocks, hipStream_t st);

}  // namespace gconv
