// seq_tokens.h -- device helpers of the operators that walk over tokens: pieces
// of a row at any alignment, packed sequences, activations.
#pragma once

#include "seq_util.h"

namespace gconv {

// V elements at any element boundary.
template <typename T, int V>
struct __attribute__((packed, aligned(sizeof(T)))) Packed {
    T e[V];
};

// V elements of a row of `dim` from `col`; those past its end are 0.
template <typename T, int V>
__device__ __forceinline__ Packed<T, V> load_piece(const T* row, int col, int dim)
{
    if (col + V <= dim) return *(const Packed<T, V>*)(row + col);
    Packed<T, V> p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.e[i] = col + i < dim ? row[col + i] : (T)0.f;
    return p;
}

template <typename T, int V>
__device__ __forceinline__ void store_piece(T* row, int col, int dim, const float (&v)[V])
{
    Packed<T, V> p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.e[i] = (T)v[i];
    if (col + V <= dim) {
        *(Packed<T, V>*)(row + col) = p;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (col + i < dim) row[col + i] = p.e[i];
    }
}

__device__ __forceinline__ float sigmoid_of(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// The sequences of a call: `count` of `tokens` each (cu NULL), or those that
// cu[0..count] cut out of `tokens`. What cu says is held to 0..tokens, so no
// value of it leads outside a tensor.
struct Sequences {
    const int32_t* cu;
    int64_t tokens;
    int count;
    __device__ __forceinline__ int64_t bound(int n) const
    {
        const int64_t v = cu[n];
        return v < 0 ? 0 : v > tokens ? tokens : v;
    }
    // Packed: the last n with cu[n] <= t, -1 before all.
    __device__ __forceinline__ int find(int64_t t) const
    {
        int lo = -1, hi = count;
        while (lo < hi) {
            const int mid = lo + (hi - lo + 1) / 2;
            if (bound(mid) <= t) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
};

}  // namespace gconv
