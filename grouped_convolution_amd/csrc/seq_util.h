// seq_util.h -- device helpers shared by the sequence-model kernels (linear
// attention, the gated norm, the orthogonalised update): element types, MFMA
// fragments of 16 bytes and their loads from LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gconv {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4 lds_s4;

// One lane's fragment of an MFMA operand is 16 bytes along the reduction in
// both element types: 8 bf16 of one 16x16x32 product, or 4 floats, each of
// them one step of four 16x16x4 products. Lane l holds row (or column) l % 16
// and the 16 bytes of group g = l / 16. The accumulator holds column l % 16,
// rows 4 g + 0..3.
template <typename T>
struct Frag;

template <>
struct Frag<__bf16> {
    static constexpr int kStep = 32;  // reduction length of one fragment pair
    static constexpr int kElems = 8;  // elements a lane holds
};

template <>
struct Frag<float> {
    static constexpr int kStep = 16;
    static constexpr int kElems = 4;
};

template <typename T>
__device__ __forceinline__ f4 mma(u4 a, u4 b, f4 c);

template <>
__device__ __forceinline__ f4 mma<__bf16>(u4 a, u4 b, f4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
}

template <>
__device__ __forceinline__ f4 mma<float>(u4 a, u4 b, f4 c)
{
    const f4 x = __builtin_bit_cast(f4, a), y = __builtin_bit_cast(f4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ u2 pack4(f4 v)
{
    bf4 h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = (__bf16)v[i];
    return __builtin_bit_cast(u2, h);
}

// Fragment whose reduction runs along the rows of an LDS tile [row][col]: the
// lane's column is col0 + l % 16, and its elements are rows
//   bf16:  row0 + 16 (e / 4) + 4 g + e % 4   (transposing reads of 4 x 16 blocks)
//   fp32:  row0 + 4 g + e
// which is also the order in which accumulators of 16-row tiles, packed, form
// a fragment: the two meet in one product without a shuffle.
__device__ __forceinline__ u4 frag_rows(const __bf16* tile, int pitch, int row0, int col0, int lane)
{
    const int g = lane >> 4, i = lane & 15;
    const __bf16* p = tile + (row0 + 4 * g + (i >> 2)) * pitch + col0 + (i & 3) * 4;
    const u2 lo = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p));
    const u2 hi = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + 16 * pitch)));
    return u4{lo[0], lo[1], hi[0], hi[1]};
}

__device__ __forceinline__ u4 frag_rows(const float* tile, int pitch, int row0, int col0, int lane)
{
    const float* p = tile + (row0 + 4 * (lane >> 4)) * pitch + col0 + (lane & 15);
    f4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = p[e * pitch];
    return __builtin_bit_cast(u4, v);
}

// Fragment whose reduction runs along a row of the tile (16 contiguous bytes).
template <typename T>
__device__ __forceinline__ u4 frag_cols(const T* tile, int pitch, int row0, int col0, int lane)
{
    return *(const u4*)(tile + (row0 + (lane & 15)) * pitch + col0 + (lane >> 4) * Frag<T>::kElems);
}

// The same with the reduction in the order of frag_rows.
template <typename T>
__device__ __forceinline__ u4 frag_split(const T* tile, int pitch, int row0, int col0, int lane)
{
    const T* p = tile + (row0 + (lane & 15)) * pitch + col0 + (lane >> 4) * 4;
    if constexpr (sizeof(T) == 4) return *(const u4*)p;
    const u2 lo = *(const u2*)p, hi = *(const u2*)(p + 16);
    return u4{lo[0], lo[1], hi[0], hi[1]};
}

// 16 bytes of a row that holds `dim` elements, from element `col`, read one by
// one; elements past the row read 0.
template <typename T>
__device__ __forceinline__ u4 load16(const T* row, int col, int dim)
{
    constexpr int E = 16 / sizeof(T);
    T e[E];
#pragma unroll
    for (int i = 0; i < E; ++i) e[i] = col + i < dim ? row[col + i] : (T)0.f;
    return __builtin_bit_cast(u4, e);
}

template <typename T>
__device__ __forceinline__ bool finite_bits(T v);
template <>
__device__ __forceinline__ bool finite_bits<float>(float v)
{
    return (__builtin_bit_cast(uint32_t, v) & 0x7f800000u) != 0x7f800000u;
}
template <>
__device__ __forceinline__ bool finite_bits<__bf16>(__bf16 v)
{
    return (__builtin_bit_cast(uint16_t, v) & 0x7f80u) != 0x7f80u;
}

// Whether 16 bytes hold an infinity or a NaN.
template <typename T>
__device__ __forceinline__ bool any_nonfinite(u4 v);
template <>
__device__ __forceinline__ bool any_nonfinite<float>(u4 v)
{
    bool b = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) b |= (v[i] & 0x7f800000u) == 0x7f800000u;
    return b;
}
template <>
__device__ __forceinline__ bool any_nonfinite<__bf16>(u4 v)
{
    bool b = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) b |= (v[i] & 0x7f80u) == 0x7f80u || (v[i] & 0x7f800000u) == 0x7f800000u;
    return b;
}

// The 16 bytes with every infinity and NaN replaced by 0.
template <typename T>
__device__ __forceinline__ u4 drop_nonfinite(u4 v)
{
    constexpr int E = 16 / sizeof(T);
    struct Pack { T e[E]; } p = __builtin_bit_cast(Pack, v);
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (!finite_bits<T>(p.e[i])) p.e[i] = (T)0.f;
    return __builtin_bit_cast(u4, p);
}

}  // namespace gconv
