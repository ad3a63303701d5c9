// embed_internal.h -- sums over tokens of the same id, for other operators: the
// embedding's gradient without the rows that have no tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gconv {

// Tokens with ids 0..rows-1 (others do not count), a bfloat16 row of `dim` each.
struct EmbedRuns {
    const void* ids;      // [tokens], of 64 bits if `wide`
    int wide;
    int64_t tokens, rows, dim;
    void* workspace;      // embed_runs_workspace() bytes, 256-byte aligned
    // by embed_runs_sort:
    int order;
    const uint32_t* start;  // [rows + 1]: how many tokens have smaller ids
    // for embed_runs_sum:
    const void* src;      // [tokens] rows
    int64_t pitch;        // elements between them
    const float* weight;  // [tokens]
    // [tokens][dim]: that of id v, of weight x row over its tokens, at start[v]; taken in float32 and rounded to bfloat16,
    // as what they make up for is itself a rounding to it of another number
    void* sums;
};

size_t embed_runs_workspace(const EmbedRuns& r);
void embed_runs_sort(EmbedRuns* r, hipStream_t st);
// For the ids row0..row1-1.
void embed_runs_sum(const EmbedRuns& r, int64_t row0, int64_t row1, hipStream_t st);

}  // namespace gconv
