// attention_api.cpp -- the extern "C" entry points of the attention operators
// (include/mdcn.h): validation on the host, launches on the caller's stream.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdio>
#include <new>
#include <numeric>

#include "attention.h"
#include "entry.h"
#include "mdcn.h"

struct mdcn_rotary {
    int32_t dim, pairs, axes, adjacent;
    mdcn::RotaryTable table;
};

struct mdcn_attention {
    int32_t q_heads, k_heads, dim, causal;
    float scale;
};

namespace {

using mdcn::AttendArgs;
using mdcn::Heads;
using mdcn::RotaryArgs;
using mdcn::RotaryKind;

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxStride = int64_t(1) << 22;      // elements between a tensor's tokens

bool valid_dtype(mdcn_dtype t) { return t == MDCN_F32 || t == MDCN_F16 || t == MDCN_BF16; }

size_t elem_size(mdcn_dtype t) { return t == MDCN_F32 ? 4 : 2; }

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
mdcn_status check_view(const View &v)
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
bool distinct_rows(const View &v)
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
bool overlap(const char *a0, const char *a1, const char *b0, const char *b1)
{
    return a0 < a1 && b0 < b1 && a0 < b1 && b0 < a1;
}

bool overlap(const View &a, const View &b) { return overlap(a.lo(), a.hi(), b.lo(), b.hi()); }

bool overlap(const View &a, const void *p, size_t bytes)
{
    const char *c = static_cast<const char *>(p);
    return overlap(a.lo(), a.hi(), c, c + bytes);
}

// Views that interleave in one allocation may overlap as address ranges without
// sharing a value.  Queries, keys and values in the rows of one projection: with one
// token stride, their rows are compared within a token.
bool apart_in_tokens(const View &a, const View &b)
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
bool apart_in_heads(const View &a, const View &b)
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

bool share_values(const View &a, const View &b)
{
    return overlap(a, b) && !apart_in_tokens(a, b) && !apart_in_heads(a, b);
}

bool same_view(const View &a, const View &b)
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

mdcn_status launched(hipError_t e) { return e == hipSuccess ? MDCN_OK : MDCN_E_LAUNCH; }

void *align_up(void *p)
{
    return reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(p) + 255) / 256 * 256);
}

// dims[0..3]: tokens, q_heads, k_heads, axis stride of the positions.
mdcn_status rotary_args(const mdcn_rotary *op, mdcn_dtype dtype, const int64_t *dims,
                        const int32_t *positions, RotaryArgs *a)
{
    if (!op || !dims)
        return MDCN_E_NULL;
    if (!valid_dtype(dtype))
        return MDCN_E_DTYPE;
    if (dims[0] < 0 || dims[0] > kMaxTokens || dims[1] < 0 || dims[2] < 0 ||
        dims[1] > (1 << 20) || dims[2] > (1 << 20) || dims[1] + dims[2] < 1)
        return MDCN_E_SHAPE;
    if (dims[3] < 0 || (op->axes > 1 && dims[3] < dims[0]))
        return MDCN_E_SHAPE;
    if (dims[0] > 0 && !positions)
        return MDCN_E_NULL;
    a->tokens = dims[0];
    a->q_heads = int32_t(dims[1]);
    a->k_heads = int32_t(dims[2]);
    a->axis_stride = dims[3];
    a->positions = positions;
    a->dim = op->dim;
    a->pairs = op->pairs;
    a->adjacent = op->adjacent;
    a->table = op->table;
    return MDCN_OK;
}

View rotary_view(const RotaryArgs &a, mdcn_dtype dtype, const void *data, bool keys,
                 const int64_t *strides)
{
    return View{Heads{data, strides[0], strides[1]}, a.tokens, keys ? a.k_heads : a.q_heads, a.dim,
                elem_size(dtype)};
}

// Inputs first, then outputs; an output may be exactly its input's view
// (every value is read before it is written, by the same lane).
mdcn_status check_rotary_views(const View *in, int n_in, const View *out, int n_out,
                               const RotaryArgs &a, int axes)
{
    const size_t pos_bytes = size_t((axes - 1) * a.axis_stride + a.tokens) * 4;
    for (int i = 0; i < n_in; ++i) {
        const mdcn_status st = check_view(in[i]);
        if (st != MDCN_OK)
            return st;
    }
    for (int o = 0; o < n_out; ++o) {
        const mdcn_status st = check_view(out[o]);
        if (st != MDCN_OK)
            return st;
        if (!distinct_rows(out[o]))
            return MDCN_E_ALIAS;
        for (int i = 0; i < n_in; ++i)
            if (share_values(in[i], out[o]) && !(n_in == n_out && i == o && same_view(in[i], out[o])))
                return MDCN_E_ALIAS;
        for (int p = 0; p < o; ++p)
            if (share_values(out[p], out[o]))
                return MDCN_E_ALIAS;
        if (a.tokens > 0 && overlap(out[o], a.positions, pos_bytes))
            return MDCN_E_ALIAS;
    }
    return MDCN_OK;
}

mdcn_status attend_dims(const mdcn_attention *op, mdcn_dtype dtype, const int64_t *dims,
                        AttendArgs *a)
{
    if (!op || !dims)
        return MDCN_E_NULL;
    if (!valid_dtype(dtype))
        return MDCN_E_DTYPE;
    if (dims[0] < 0 || dims[0] > (1 << 24) || dims[1] < 0 || dims[1] > kMaxTokens || dims[2] < 0 ||
        dims[2] > kMaxTokens)
        return MDCN_E_SHAPE;
    a->batch = int32_t(dims[0]);
    a->q_tokens = int32_t(dims[1]);
    a->k_tokens = int32_t(dims[2]);
    a->q_heads = op->q_heads;
    a->k_heads = op->k_heads;
    a->dim = op->dim;
    a->causal = op->causal;
    a->scale = op->scale;
    return MDCN_OK;
}

// 16-byte rows: the kernels read and write 16 bytes at a time.  A token's row
// ends before the next one starts: a tile's copy tells rows past the end of a
// sequence by their offset.
mdcn_status check_attend_view(View &v)
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

size_t up_256(size_t n) { return (n + 255) / 256 * 256; }

// The backward's row statistics, and the maxima that only fp16 has, up to the next 256 bytes.
size_t stats_bytes(const AttendArgs &a)
{
    return up_256(size_t(a.q_heads) * a.q_tokens * sizeof(float2));
}

size_t tops_bytes(mdcn_dtype dtype, const AttendArgs &a)
{
    return dtype == MDCN_F16
               ? stats_bytes(a) + up_256(size_t(a.k_heads) * a.k_tokens * sizeof(float))
               : 0;
}

}  // namespace

extern "C" {

mdcn_status mdcn_rotary_create(int32_t dim, int32_t axes, const int32_t *pairs, double base,
                               int32_t adjacent, int32_t round_robin, int32_t per_axis,
                               mdcn_rotary **out)
{
    if (!out || !pairs)
        return MDCN_E_NULL;
    *out = nullptr;
    if (dim <= 0 || dim % 2 || dim > mdcn::kMaxRotaryDim || axes < 1 ||
        axes > mdcn::kMaxRotaryAxes || !(base > 0.0) || !std::isfinite(base))
        return MDCN_E_ATTR;
    int32_t total = 0;
    for (int32_t i = 0; i < axes; ++i) {
        if (pairs[i] < 0 || pairs[i] > dim / 2)
            return MDCN_E_ATTR;
        total += pairs[i];
    }
    if (total < 1 || total > dim / 2)
        return MDCN_E_ATTR;
    mdcn_rotary *r = new (std::nothrow) mdcn_rotary();
    if (!r)
        return MDCN_E_INTERNAL;
    r->dim = dim;
    r->pairs = total;
    r->axes = axes;
    r->adjacent = adjacent != 0;
    // dealt in turn: pair j of every axis that has one, then pair j + 1
    int32_t n = 0;
    auto put = [&](int32_t axis, int32_t j) {
        constexpr long double kPi = 3.14159265358979323846264338327950288L;
        const long double e = per_axis ? static_cast<long double>(j) / pairs[axis]
                                       : static_cast<long double>(n) / total;
        const long double turns = std::pow(static_cast<long double>(base), -e) / (2 * kPi);
        const long double rounded = std::rint(std::ldexp(turns - std::floor(turns), 64));
        r->table.axis[n] = uint8_t(axis);
        r->table.turns[n] = rounded < std::ldexp(1.0L, 64) ? uint64_t(rounded) : 0;
        ++n;
    };
    if (round_robin) {
        for (int32_t j = 0; n < total; ++j)
            for (int32_t a = 0; a < axes; ++a)
                if (j < pairs[a])
                    put(a, j);
    } else {
        for (int32_t a = 0; a < axes; ++a)
            for (int32_t j = 0; j < pairs[a]; ++j)
                put(a, j);
    }
    *out = r;
    return MDCN_OK;
}

void mdcn_rotary_destroy(mdcn_rotary *op) { delete op; }

mdcn_status mdcn_rotate(const mdcn_rotary *op, mdcn_dtype dtype, const int64_t dims[12],
                        const void *q, const void *k, const int32_t *positions, int32_t inverse,
                        void *q_out, void *k_out, void *stream)
{
    try {
        RotaryArgs a = {};
        mdcn_status st = rotary_args(op, dtype, dims, positions, &a);
        if (st != MDCN_OK)
            return st;
        const View in[] = {rotary_view(a, dtype, q, false, dims + 4),
                           rotary_view(a, dtype, k, true, dims + 6)};
        const View out[] = {rotary_view(a, dtype, q_out, false, dims + 8),
                            rotary_view(a, dtype, k_out, true, dims + 10)};
        st = check_rotary_views(in, 2, out, 2, a, op->axes);
        if (st != MDCN_OK)
            return st;
        if (a.tokens == 0)
            return MDCN_OK;
        if ((st = mdcn::check_device()) != MDCN_OK)
            return st;
        a.inverse = inverse != 0;
        a.q = in[0].h;
        a.k = in[1].h;
        a.oq = out[0].h;
        a.ok = out[1].h;
        return launched(launch_rotary(RotaryKind::Rotate, dtype, a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MDCN_E_INTERNAL;
    }
}

mdcn_status mdcn_norm_rotate(const mdcn_rotary *op, mdcn_dtype dtype, const int64_t dims[12],
                             const void *q, const void *k, const int32_t *positions,
                             const void *q_gain, const void *k_gain, float eps, void *q_out,
                             void *k_out, void *stream)
{
    try {
        RotaryArgs a = {};
        mdcn_status st = rotary_args(op, dtype, dims, positions, &a);
        if (st != MDCN_OK)
            return st;
        if (!(eps >= 0.0f) || !std::isfinite(eps))
            return MDCN_E_ATTR;
        const View in[] = {rotary_view(a, dtype, q, false, dims + 4),
                           rotary_view(a, dtype, k, true, dims + 6)};
        const View out[] = {rotary_view(a, dtype, q_out, false, dims + 8),
                            rotary_view(a, dtype, k_out, true, dims + 10)};
        st = check_rotary_views(in, 2, out, 2, a, op->axes);
        if (st != MDCN_OK)
            return st;
        if ((a.q_heads && !q_gain) || (a.k_heads && !k_gain))
            return MDCN_E_NULL;
        const size_t gain_bytes = size_t(a.dim) * elem_size(dtype);
        for (const View &o : out)
            if ((q_gain && overlap(o, q_gain, gain_bytes)) ||
                (k_gain && overlap(o, k_gain, gain_bytes)))
                return MDCN_E_ALIAS;
        if (a.tokens == 0)
            return MDCN_OK;
        if ((st = mdcn::check_device()) != MDCN_OK)
            return st;
        a.q = in[0].h;
        a.k = in[1].h;
        a.oq = out[0].h;
        a.ok = out[1].h;
        a.q_gain = q_gain;
        a.k_gain = k_gain;
        a.eps = eps;
        return launched(
            launch_rotary(RotaryKind::NormRotate, dtype, a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MDCN_E_INTERNAL;
    }
}

mdcn_status mdcn_norm_rotate_backward_workspace_bytes(const mdcn_rotary *op, int64_t tokens,
                                                      size_t *bytes)
{
    if (!op || !bytes)
        return MDCN_E_NULL;
    if (tokens < 0 || tokens > kMaxTokens)
        return MDCN_E_SHAPE;
    *bytes = size_t(mdcn::rotary_backward_blocks(tokens)) * 2 * op->dim * sizeof(float) + 256;
    return MDCN_OK;
}

mdcn_status mdcn_norm_rotate_backward(const mdcn_rotary *op, mdcn_dtype dtype,
                                      const int64_t dims[16], const void *q, const void *k,
                                      const int32_t *positions, const void *q_gain,
                                      const void *k_gain, float eps, const void *grad_q_out,
                                      const void *grad_k_out, void *grad_q, void *grad_k,
                                      void *grad_q_gain, void *grad_k_gain, void *workspace,
                                      size_t workspace_bytes, void *stream_ptr)
{
    try {
        RotaryArgs a = {};
        mdcn_status st = rotary_args(op, dtype, dims, positions, &a);
        if (st != MDCN_OK)
            return st;
        if (!(eps >= 0.0f) || !std::isfinite(eps))
            return MDCN_E_ATTR;
        const View in[] = {rotary_view(a, dtype, q, false, dims + 4),
                           rotary_view(a, dtype, k, true, dims + 6),
                           rotary_view(a, dtype, grad_q_out, false, dims + 8),
                           rotary_view(a, dtype, grad_k_out, true, dims + 10)};
        const View out[] = {rotary_view(a, dtype, grad_q, false, dims + 12),
                            rotary_view(a, dtype, grad_k, true, dims + 14)};
        st = check_rotary_views(in, 4, out, 2, a, op->axes);
        if (st != MDCN_OK)
            return st;
        if ((a.q_heads && (!q_gain || !grad_q_gain)) || (a.k_heads && (!k_gain || !grad_k_gain)))
            return MDCN_E_NULL;
        size_t need = 0;
        st = mdcn_norm_rotate_backward_workspace_bytes(op, a.tokens, &need);
        if (st != MDCN_OK)
            return st;
        if (!workspace || workspace_bytes < need)
            return MDCN_E_WORKSPACE;
        const size_t gain_bytes = size_t(a.dim) * elem_size(dtype);
        const size_t pos_bytes =
            a.tokens ? size_t((op->axes - 1) * a.axis_stride + a.tokens) * 4 : 0;
        const Block small[] = {{workspace, workspace_bytes, true}, {grad_q_gain, gain_bytes, true},
                               {grad_k_gain, gain_bytes, true},    {q_gain, gain_bytes, false},
                               {k_gain, gain_bytes, false},        {positions, pos_bytes, false}};
        if (blocks_overlap(small))
            return MDCN_E_ALIAS;
        for (const Block &x : small) {
            if (!x.p)
                continue;
            for (const View &v : out)
                if (overlap(v, x.p, x.n))
                    return MDCN_E_ALIAS;
            for (const View &v : in)
                if (x.written && overlap(v, x.p, x.n))
                    return MDCN_E_ALIAS;
        }
        if ((st = mdcn::check_device()) != MDCN_OK)
            return st;
        a.inverse = 1;                       // the gradient is turned back
        a.q = in[0].h;
        a.k = in[1].h;
        a.gq = in[2].h;
        a.gk = in[3].h;
        a.oq = out[0].h;
        a.ok = out[1].h;
        a.q_gain = q_gain;
        a.k_gain = k_gain;
        a.eps = eps;
        a.partial = static_cast<float *>(align_up(workspace));
        const hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
        st = launched(launch_rotary(RotaryKind::NormRotateBackward, dtype, a, stream));
        return st != MDCN_OK
                   ? st
                   : launched(launch_gain_sum(dtype, a, grad_q_gain, grad_k_gain, stream));
    } catch (...) {
        return MDCN_E_INTERNAL;
    }
}

mdcn_status mdcn_attention_create(int32_t q_heads, int32_t k_heads, int32_t dim, int32_t causal,
                                  float scale, mdcn_attention **out)
{
    if (!out)
        return MDCN_E_NULL;
    *out = nullptr;
    if (q_heads < 1 || k_heads < 1 || q_heads > 65536 || q_heads % k_heads || dim < 8 || dim % 8 ||
        dim > mdcn::kMaxAttendDim || !(scale > 0.0f) || !std::isfinite(scale))
        return MDCN_E_ATTR;
    mdcn_attention *op = new (std::nothrow) mdcn_attention();
    if (!op)
        return MDCN_E_INTERNAL;
    op->q_heads = q_heads;
    op->k_heads = k_heads;
    op->dim = dim;
    op->causal = causal != 0;
    op->scale = scale;
    *out = op;
    return MDCN_OK;
}

void mdcn_attention_destroy(mdcn_attention *op) { delete op; }

mdcn_status mdcn_attend_workspace_bytes(const mdcn_attention *op, mdcn_dtype dtype,
                                        const int64_t dims[11], size_t *bytes)
{
    AttendArgs a = {};
    if (!bytes)
        return MDCN_E_NULL;
    const mdcn_status st = attend_dims(op, dtype, dims, &a);
    if (st != MDCN_OK)
        return st;
    *bytes = mdcn::attend_prefers_split(dtype, a) ? mdcn::attend_split_bytes(dtype, a.dim) + 256 : 0;
    return MDCN_OK;
}

mdcn_status mdcn_attend_filled(const mdcn_attention *op, mdcn_dtype dtype, const int64_t dims[11],
                               const void *q, const void *k, const void *v, const int32_t *cu_q,
                               const int32_t *cu_k, const int32_t *used_k, int32_t fill, void *out,
                               float *lse, void *workspace, size_t workspace_bytes,
                               void *stream_ptr)
{
    try {
        AttendArgs a = {};
        mdcn_status st = attend_dims(op, dtype, dims, &a);
        if (st != MDCN_OK)
            return st;
        const size_t e = elem_size(dtype);
        View in[] = {
            {{q, dims[3], dims[4]}, a.q_tokens, a.q_heads, a.dim, e},
            {{k, dims[5], dims[6]}, a.k_tokens, a.k_heads, a.dim, e},
            {{v, dims[7], dims[8]}, a.k_tokens, a.k_heads, a.dim, e},
        };
        View o = {{out, dims[9], dims[10]}, a.q_tokens, a.q_heads, a.dim, e};
        for (View &x : in)
            if ((st = check_attend_view(x)) != MDCN_OK)
                return st;
        if ((st = check_attend_view(o)) != MDCN_OK)
            return st;
        if (!cu_q || !cu_k || (a.q_tokens > 0 && !lse))
            return MDCN_E_NULL;
        size_t need = 0;
        if ((st = mdcn_attend_workspace_bytes(op, dtype, dims, &need)) != MDCN_OK)
            return st;
        const bool split = need > 0;
        if (split && (!workspace || workspace_bytes < need))
            return MDCN_E_WORKSPACE;
        const size_t lse_bytes = size_t(a.q_heads) * a.q_tokens * 4;
        const size_t cu_bytes = size_t(a.batch + 1) * 4;
        if (!distinct_rows(o) || overlap(o, lse, lse_bytes) || overlap(o, cu_q, cu_bytes) ||
            overlap(o, cu_k, cu_bytes) || (split && overlap(o, workspace, workspace_bytes)) ||
            (used_k && overlap(o, used_k, size_t(a.batch) * 4)))
            return MDCN_E_ALIAS;
        for (const View &x : in)
            if (share_values(x, o) || overlap(x, lse, lse_bytes) ||
                (split && overlap(x, workspace, workspace_bytes)))
                return MDCN_E_ALIAS;
        const Block small[] = {{lse, lse_bytes, true},
                               {split ? workspace : nullptr, workspace_bytes, true},
                               {cu_q, cu_bytes, false},
                               {cu_k, cu_bytes, false},
                               {used_k, size_t(a.batch) * 4, false}};
        if (blocks_overlap(small))
            return MDCN_E_ALIAS;
        a.fill = fill & (mdcn::kFillOut | mdcn::kFillLse);
        if (a.q_tokens == 0 || (a.batch == 0 && !a.fill))
            return MDCN_OK;
        if ((st = mdcn::check_device()) != MDCN_OK)
            return st;
        a.q = in[0].h;
        a.k = in[1].h;
        a.v = in[2].h;
        a.out = o.h;
        a.lse = lse;
        a.cu_q = cu_q;
        a.cu_k = cu_k;
        a.used_k = used_k;
        const hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
        if (!split)
            return launched(launch_attend(dtype, a, stream));
        a.workers = mdcn::attend_split_workers(dtype, a.dim);
        a.partial = static_cast<float *>(align_up(workspace));
        return launched(launch_attend_split(dtype, a, stream));
    } catch (...) {
        return MDCN_E_INTERNAL;
    }
}

mdcn_status mdcn_attend(const mdcn_attention *op, mdcn_dtype dtype, const int64_t dims[11],
                        const void *q, const void *k, const void *v, const int32_t *cu_q,
                        const int32_t *cu_k, const int32_t *used_k, void *out, float *lse,
                        void *workspace, size_t workspace_bytes, void *stream)
{
    return mdcn_attend_filled(op, dtype, dims, q, k, v, cu_q, cu_k, used_k, 0, out, lse, workspace,
                              workspace_bytes, stream);
}

mdcn_status mdcn_attend_backward_workspace_bytes(const mdcn_attention *op, mdcn_dtype dtype,
                                                 const int64_t dims[19], size_t *bytes)
{
    AttendArgs a = {};
    if (!bytes)
        return MDCN_E_NULL;
    const mdcn_status st = attend_dims(op, dtype, dims, &a);
    if (st != MDCN_OK)
        return st;
    const int splits = mdcn::attend_backward_splits(a);
    *bytes = stats_bytes(a) + tops_bytes(dtype, a) + 256;
    if (splits > 1)
        *bytes += size_t(splits) * 2 * a.k_tokens * a.k_heads * a.dim * sizeof(float);
    return MDCN_OK;
}

mdcn_status mdcn_attend_backward(const mdcn_attention *op, mdcn_dtype dtype,
                                 const int64_t dims[19], const void *q, const void *k,
                                 const void *v, const void *out, const float *lse,
                                 const void *grad_out, const int32_t *cu_q, const int32_t *cu_k,
                                 const int32_t *used_k, void *grad_q, void *grad_k, void *grad_v,
                                 void *workspace, size_t workspace_bytes, void *stream)
{
    try {
        AttendArgs a = {};
        mdcn_status st = attend_dims(op, dtype, dims, &a);
        if (st != MDCN_OK)
            return st;
        const size_t e = elem_size(dtype);
        auto view = [&](const void *p, int i, bool keys) {
            return View{{p, dims[3 + 2 * i], dims[4 + 2 * i]},
                        keys ? a.k_tokens : a.q_tokens,
                        keys ? a.k_heads : a.q_heads,
                        a.dim,
                        e};
        };
        View in[] = {view(q, 0, false), view(k, 1, true), view(v, 2, true),
                           view(out, 3, false), view(grad_out, 4, false)};
        View g[] = {view(grad_q, 5, false), view(grad_k, 6, true), view(grad_v, 7, true)};
        for (View &x : in)
            if ((st = check_attend_view(x)) != MDCN_OK)
                return st;
        for (View &x : g)
            if ((st = check_attend_view(x)) != MDCN_OK)
                return st;
        if (!cu_q || !cu_k || (a.q_tokens > 0 && !lse))
            return MDCN_E_NULL;
        size_t need = 0;
        if ((st = mdcn_attend_backward_workspace_bytes(op, dtype, dims, &need)) != MDCN_OK)
            return st;
        if (!workspace || workspace_bytes < need)
            return MDCN_E_WORKSPACE;
        const size_t lse_bytes = size_t(a.q_heads) * a.q_tokens * 4;
        const size_t cu_bytes = size_t(a.batch + 1) * 4;
        for (int i = 0; i < 3; ++i) {
            if (!distinct_rows(g[i]) || overlap(g[i], lse, lse_bytes) ||
                overlap(g[i], workspace, workspace_bytes) || overlap(g[i], cu_q, cu_bytes) ||
                overlap(g[i], cu_k, cu_bytes) ||
                (used_k && overlap(g[i], used_k, size_t(a.batch) * 4)))
                return MDCN_E_ALIAS;
            for (const View &x : in)
                if (share_values(x, g[i]))
                    return MDCN_E_ALIAS;
            for (int j = 0; j < i; ++j)
                if (share_values(g[i], g[j]))
                    return MDCN_E_ALIAS;
        }
        for (const View &x : in)
            if (overlap(x, workspace, workspace_bytes))
                return MDCN_E_ALIAS;
        const Block small[] = {{workspace, workspace_bytes, true},
                               {lse, lse_bytes, false},
                               {cu_q, cu_bytes, false},
                               {cu_k, cu_bytes, false},
                               {used_k, size_t(a.batch) * 4, false}};
        if (blocks_overlap(small))
            return MDCN_E_ALIAS;
        if (a.q_tokens == 0 && a.k_tokens == 0)
            return MDCN_OK;
        if ((st = mdcn::check_device()) != MDCN_OK)
            return st;
        a.q = in[0].h;
        a.k = in[1].h;
        a.v = in[2].h;
        a.out = in[3].h;
        a.go = in[4].h;
        a.dq = g[0].h;
        a.dk = g[1].h;
        a.dv = g[2].h;
        a.lse = const_cast<float *>(lse);
        a.stats = static_cast<float2 *>(align_up(workspace));
        char *const behind = reinterpret_cast<char *>(a.stats) + stats_bytes(a);
        a.row_tops = reinterpret_cast<float2 *>(behind);
        a.key_tops = reinterpret_cast<float *>(behind + stats_bytes(a));
        a.partial = reinterpret_cast<float *>(behind + tops_bytes(dtype, a));
        a.splits = mdcn::attend_backward_splits(a);
        a.cu_q = cu_q;
        a.cu_k = cu_k;
        a.used_k = used_k;
        return launched(launch_attend_backward(dtype, a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MDCN_E_INTERNAL;
    }
}

mdcn_status mdcn_describe_rotate(const mdcn_rotary *op, mdcn_dtype dtype, const int64_t dims[3],
                                 char *buf, size_t len)
{
    if (!op || !dims || !buf || len == 0)
        return MDCN_E_NULL;
    RotaryArgs a = {};
    const int64_t all[4] = {dims[0], dims[1], dims[2], dims[0]};
    const int32_t position = 0;                  // only looked at for being there
    const mdcn_status st = rotary_args(op, dtype, all, &position, &a);
    if (st != MDCN_OK)
        return st;
    if (a.tokens == 0) {
        std::snprintf(buf, len, "nothing to do");
        return MDCN_OK;
    }
    const mdcn::RotaryShape s = mdcn::rotary_shape(RotaryKind::Rotate, dtype, a);
    std::snprintf(buf, len, "width=%d lanes=%d rounds=%d waves_per_token=%d backward_blocks=%d",
                  s.width, s.lanes, s.rounds, s.waves, mdcn::rotary_backward_blocks(a.tokens));
    return MDCN_OK;
}

mdcn_status mdcn_describe_attend(const mdcn_attention *op, mdcn_dtype dtype, const int64_t dims[3],
                                 int32_t backward, char *buf, size_t len)
{
    if (!buf || len == 0)
        return MDCN_E_NULL;
    AttendArgs a = {};
    const mdcn_status st = attend_dims(op, dtype, dims, &a);
    if (st != MDCN_OK)
        return st;
    const int waves = mdcn::attend_key_waves(dtype, a), rows = waves == 1 ? 128 : 64;
    if (backward)
        std::snprintf(buf, len, "rows=%d key_waves=%d parts=%d", rows, waves,
                      mdcn::attend_backward_splits(a));
    else if (mdcn::attend_prefers_split(dtype, a))
        std::snprintf(buf, len, "split unit=%d workgroups=%d",
                      32 << mdcn::attend_split_unit_shift(a),
                      mdcn::attend_split_workers(dtype, a.dim));
    else
        std::snprintf(buf, len, "tile rows=%d key_waves=%d", rows, waves);
    return MDCN_OK;
}

}  // extern "C"
