// seq_host.h -- host-side checks that the sequence operators' entry points share.
#pragma once

#include <algorithm>

#include "gconv.h"
#include "gconv_internal.h"

namespace gconv {

// Bytes that a pointer leads to.
struct Span {
    const void* p;
    int64_t bytes;
};

inline bool spans_meet(const Span& a, const Span& b)
{
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    return (const char*)a.p < (const char*)b.p + b.bytes && (const char*)b.p < (const char*)a.p + a.bytes;
}

// GCONV_OK if no output meets an input or another output.
template <int I, int O>
inline int check_overlap(const Span (&in)[I], const Span (&out)[O])
{
    for (int i = 0; i < O; ++i) {
        for (const Span& r : in)
            if (spans_meet(out[i], r)) return fail(GCONV_ERR_ARG, "an output overlaps an input");
        for (int j = 0; j < i; ++j)
            if (spans_meet(out[i], out[j])) return fail(GCONV_ERR_ARG, "two outputs overlap");
    }
    return GCONV_OK;
}

inline int check_workspace(const void* workspace, size_t given, size_t need)
{
    if (given < need || (need > 0 && !workspace))
        return fail(GCONV_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", given, need);
    if (need > 0 && ((uintptr_t)workspace & 15) != 0)
        return fail(GCONV_ERR_WORKSPACE, "workspace pointer %p is not 16-byte aligned", workspace);
    return GCONV_OK;
}

// A strided tensor [sequences][tokens][groups][width] as far as its last element.
inline Span strided_span(const void* p, int64_t es, int64_t sequences, int64_t s0, int64_t tokens, int64_t s1, int64_t groups,
                         int64_t s2, int64_t width)
{
    if (sequences <= 0 || tokens <= 0 || groups <= 0) return Span{p, 0};
    const int64_t last = (sequences - 1) * std::max<int64_t>(s0, 0) + (tokens - 1) * std::max<int64_t>(s1, 0) +
                         (groups - 1) * std::max<int64_t>(s2, 0) + width;
    return Span{p, last * es};
}

// What a workspace is cut into: parts of whole 256 bytes.
struct Cut {
    size_t bytes = 0;
    size_t take(int64_t n)
    {
        const size_t at = bytes;
        bytes += ((size_t)n + 255) / 256 * 256;
        return at;
    }
};

}  // namespace gconv
