// views.h -- the checks that the entry points of the attention and cache operators
// make of their arguments on the host: strided views, buffers, what may overlap.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstddef>
#include <cstdint>
#include <numeric>

#include "attention.h"
#include "mdcn.h"

namespace mdcn {

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxStride = int64_t(1) << 22;      // elements between a tensor's tokens

inline bool valid_dtype(mdcn_dtype t) { return t == MDCN_F32 || t == MDCN_F16 || t == MDCN_BF16; }

inline size_t elem_size(mdcn_dtype t) { return t == MDCN_F32 ? 4 : 2; }

// A [tokens][heads][dim] view: which bytes it may touch.
struct View {
    Heads h;
    int64_t tokens, heads, dim;
    size_t elem;

    const char *lo() const { return static_cast<const char *>(h.data); }
    const char *hi() const
    {
        if (tokens == 0 || heads == 0)
            return lo();
        return lo() + size_t((tokens - 1) * h.token_stride + (heads - 1) * h.head_stride + dim) *
                          elem;
    }
};

// Rows must not overlap each other: both strides non-negative, and one row of
// values apart where there is more than one.
inline mdcn_status check_view(const View &v)
{
    if (v.tokens < 0 || v.heads < 0 || v.tokens > kMaxTokens || v.heads > (1 << 20))
        return MDCN_E_SHAPE;
    if (v.h.token_stride < 0 || v.h.head_stride < 0 || v.h.token_stride > kMaxStride ||
        v.h.head_stride > (int64_t(1) << 40))
        return MDCN_E_SHAPE;
    if (v.tokens > 0 && v.heads > 0 && !v.h.data)
        return MDCN_E_NULL;
    return reinterpret_cast<uintptr_t>(v.h.data) % v.elem == 0 ? MDCN_OK : MDCN_E_SHAPE;
}

// An output's rows may not share values.
inline bool distinct_rows(const View &v)
{
    const int64_t t = v.h.token_stride, h = v.h.head_stride;
    if (v.tokens == 0 || v.heads == 0)
        return true;
    if (v.tokens <= 1)
        return v.heads <= 1 || h >= v.dim;
    if (v.heads <= 1)
        return t >= v.dim;
    return t >= h ? h >= v.dim && t >= (v.heads - 1) * h + v.dim
                  : t >= v.dim && h >= (v.tokens - 1) * t + v.dim;
}

// (an empty range overlaps nothing, wherever it lies)
inline bool overlap(const char *a0, const char *a1, const char *b0, const char *b1)
{
    return a0 < a1 && b0 < b1 && a0 < b1 && b0 < a1;
}

inline bool overlap(const View &a, const View &b) { return overlap(a.lo(), a.hi(), b.lo(), b.hi()); }

inline bool overlap(const View &a, const void *p, size_t bytes)
{
    const char *c = static_cast<const char *>(p);
    return overlap(a.lo(), a.hi(), c, c + bytes);
}

// Views that interleave in one allocation may overlap as address ranges without
// sharing a value.  Queries, keys and values in the rows of one projection: with one
// token stride, their rows are compared within a token.
inline bool apart_in_tokens(const View &a, const View &b)
{
    const int64_t t = a.h.token_stride * int64_t(a.elem);
    if (a.h.token_stride != b.h.token_stride || a.elem != b.elem || t == 0 || a.tokens <= 1)
        return false;
    const int64_t wa = ((a.heads - 1) * a.h.head_stride + a.dim) * int64_t(a.elem);
    const int64_t wb = ((b.heads - 1) * b.h.head_stride + b.dim) * int64_t(b.elem);
    int64_t off = int64_t(reinterpret_cast<uintptr_t>(b.lo()) -
                          reinterpret_cast<uintptr_t>(a.lo())) % t;
    if (off < 0)
        off += t;
    return wa <= off && off + wb <= t;
}

// Queries, keys and values of one head side by side: all rows of a view begin at one
// address modulo any divisor of the strides that are stepped over.
inline bool apart_in_heads(const View &a, const View &b)
{
    int64_t g = 0;
    for (const View *v : {&a, &b}) {
        g = std::gcd(g, v->tokens > 1 ? v->h.token_stride : 0);
        g = std::gcd(g, v->heads > 1 ? v->h.head_stride : 0);
    }
    g *= int64_t(a.elem);
    if (g == 0 || a.elem != b.elem)
        return false;
    int64_t off = int64_t(reinterpret_cast<uintptr_t>(b.lo()) -
                          reinterpret_cast<uintptr_t>(a.lo())) % g;
    if (off < 0)
        off += g;
    return a.dim * int64_t(a.elem) <= off && off + b.dim * int64_t(b.elem) <= g;
}

inline bool share_values(const View &a, const View &b)
{
    return overlap(a, b) && !apart_in_tokens(a, b) && !apart_in_heads(a, b);
}

inline bool same_view(const View &a, const View &b)
{
    return a.h.data == b.h.data && a.h.token_stride == b.h.token_stride &&
           a.h.head_stride == b.h.head_stride && a.tokens == b.tokens && a.heads == b.heads;
}

// A buffer without strides, and whether the call writes it.
struct Block {
    const void *p;
    size_t n;
    bool written;
};

// Whether a written one shares bytes with any other.
template <int N> bool blocks_overlap(const Block (&blocks)[N])
{
    for (const Block &x : blocks)
        for (const Block &y : blocks) {
            const char *a = static_cast<const char *>(x.p), *b = static_cast<const char *>(y.p);
            if (&x != &y && x.written && a && b && overlap(a, a + x.n, b, b + y.n))
                return true;
        }
    return false;
}

inline mdcn_status launched(hipError_t e) { return e == hipSuccess ? MDCN_OK : MDCN_E_LAUNCH; }

inline void *align_up(void *p)
{
    return reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(p) + 255) / 256 * 256);
}

// 16-byte rows: the kernels read and write 16 bytes at a time.  A token's row
// ends before the next one starts: a tile's copy tells rows past the end of a
// sequence by their offset.
inline mdcn_status check_attend_view(View &v)
{
    const mdcn_status st = check_view(v);
    if (st != MDCN_OK)
        return st;
    if (v.tokens <= 1)
        v.h.token_stride = (v.dim + 7) / 8 * 8;      // never stepped over
    if (v.h.token_stride < v.dim)
        return MDCN_E_SHAPE;
    const int64_t n = int64_t(16 / v.elem);
    if (v.h.token_stride % n || v.h.head_stride % n ||
        reinterpret_cast<uintptr_t>(v.h.data) % 16)
        return MDCN_E_SHAPE;
    return MDCN_OK;
}

}  // namespace mdcn
