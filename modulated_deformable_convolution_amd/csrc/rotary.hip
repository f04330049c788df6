// rotary.hip -- rotary positions with several axes on queries and keys, and
// the RMS norm of each head with the rotation in the same pass.
//
//   theta[t][i] = position[axis(i)][t] * frequency[i]
//   turn: (a, b) -> (a cos theta - b sin theta, a sin theta + b cos theta)
//   norm: n = x / sqrt(mean(x^2) + eps), y = turn(n * gain)
// backward, with g the output's gradient turned by -theta and h = g * gain:
//   dx = (h - n * mean(h * n)) / sqrt(mean(x^2) + eps),  dgain = sum g * n
// Pair i is channels (i, i + pairs), or (2i, 2i + 1) when adjacent; channels
// from 2 * pairs on are not turned.
//
// Angles: position * frequency in turns is taken in double and reduced to
// [-1/2, 1/2] there, so far positions (10^6 and more) lose nothing; sine and
// cosine of the rest in fp32.  They are computed once per token and lane and
// used for all heads of the token: at 40 heads the ~320 instructions of a lane's
// 8 pairs are a tenth of the work on the heads.
//
// A head is spread over G lanes (a power of two), each holding units of V
// values from the first channels of its pairs and the V second channels, so
// both partners of a pair are in one lane and every access is one V-wide
// vector; V is the widest of 8, 4, 2, 1 that divides the pairs, the unturned
// rest, and all strides and addresses.  Memory bound: one read and one write
// of each value (backward: two reads, one write).
#include "attention.h"
#include "device_common.h"

namespace mdcn {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

template <typename T, int V> struct alignas(V * sizeof(T)) Pack {
    T e[V];
};

template <typename T, int V>
__device__ __forceinline__ void load_pack(float (&o)[V], const T *p)
{
    const Pack<T, V> v = *reinterpret_cast<const Pack<T, V> *>(p);
#pragma unroll
    for (int j = 0; j < V; ++j)
        o[j] = to_f32(v.e[j]);
}

template <typename T, int V>
__device__ __forceinline__ void store_pack(T *p, const float (&o)[V])
{
    Pack<T, V> v;
#pragma unroll
    for (int j = 0; j < V; ++j)
        v.e[j] = from_f32<T>(o[j]);
    *reinterpret_cast<Pack<T, V> *>(p) = v;
}

// Unit u of a head: V pairs, as the channel offsets of its two vectors.  For
// adjacent pairs the two vectors are the halves of 2V consecutive channels.
template <int V>
__device__ __forceinline__ void unit_offsets(int u, int pairs, bool adjacent, int &lo, int &hi)
{
    const int turned = pairs / V;
    if (adjacent) {
        lo = u * 2 * V;
        hi = lo + V;
    } else if (u < turned) {
        lo = u * V;
        hi = lo + pairs;
    } else {
        lo = 2 * pairs + (u - turned) * 2 * V;
        hi = lo + V;
    }
}

// x[0..V) and x[V..2V) are a unit's two vectors.
template <int V>
__device__ __forceinline__ void turn_unit(float (&x)[2 * V], const float (&c)[V],
                                          const float (&s)[V], bool adjacent)
{
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (adjacent) {
            const float a = x[2 * j], b = x[2 * j + 1];
            x[2 * j] = a * c[j] - b * s[j];
            x[2 * j + 1] = a * s[j] + b * c[j];
        } else {
            const float a = x[j], b = x[j + V];
            x[j] = a * c[j] - b * s[j];
            x[j + V] = a * s[j] + b * c[j];
        }
    }
}

template <typename T, int V>
__device__ __forceinline__ void load_unit(float (&x)[2 * V], const T *p, int lo, int hi)
{
    float a[V];
    load_pack<T, V>(a, p + lo);
#pragma unroll
    for (int j = 0; j < V; ++j)
        x[j] = a[j];
    load_pack<T, V>(a, p + hi);
#pragma unroll
    for (int j = 0; j < V; ++j)
        x[V + j] = a[j];
}

template <typename T, int V>
__device__ __forceinline__ void store_unit(T *p, const float (&x)[2 * V], int lo, int hi)
{
    float a[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        a[j] = x[j];
    store_pack<T, V>(p + lo, a);
#pragma unroll
    for (int j = 0; j < V; ++j)
        a[j] = x[V + j];
    store_pack<T, V>(p + hi, a);
}

template <int U, int V>
__device__ __forceinline__ void angles(float (&c)[U][V], float (&s)[U][V], const RotaryArgs &a,
                                       int64_t t, int lane_in_head, int group)
{
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = (lane_in_head + u * group) * V + j;
            c[u][j] = 1.0f;
            s[u][j] = 0.0f;
            if (i < a.pairs) {
                const int p = a.positions[a.table.axis[i] * a.axis_stride + t];
                double turns = double(p) * a.table.turns[i];
                turns -= rint(turns);
                sincospif(float(2.0 * turns), &s[u][j], &c[u][j]);
                if (a.inverse)
                    s[u][j] = -s[u][j];
            }
        }
}

__device__ __forceinline__ float group_sum(float v, int group)
{
    for (int m = 1; m < group; m <<= 1)
        v += __shfl_xor(v, m, 64);
    return v;
}

// Forward (rotate, norm_rotate): one wave takes `per_wave` rounds of one
// token's heads, 64 / G heads a round.
template <typename T, int V, int U, bool NORM>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, int group, int units,
                                                          int per_wave, int waves_per_token)
{
    const int lane = threadIdx.x & 63;
    const int64_t w = int64_t(blockIdx.x) * kWaves + (threadIdx.x >> 6);
    const int64_t t = w / waves_per_token;
    if (t >= a.tokens)
        return;
    const int part = int(w - t * waves_per_token);
    const int li = lane & (group - 1);
    const int slots = 64 / group;
    const int rows = a.q_heads + a.k_heads;
    const bool adjacent = a.adjacent != 0;

    int lo[U], hi[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int unit = li + u * group;
        ok[u] = unit < units;
        unit_offsets<V>(ok[u] ? unit : 0, a.pairs, adjacent, lo[u], hi[u]);
    }
    float c[U][V], s[U][V];
    angles<U, V>(c, s, a, t, li, group);

    const float inv_dim = 1.0f / float(a.dim);
    const int r_end = min(rows, (part + 1) * per_wave * slots);
    for (int r0 = part * per_wave * slots; r0 < r_end; r0 += slots) {
        const int r = r0 + lane / group;
        const bool live = r < rows;
        const bool is_q = r < a.q_heads;
        const Heads &in = is_q ? a.q : a.k;
        const Heads &out = is_q ? a.oq : a.ok;
        const int h = live ? (is_q ? r : r - a.q_heads) : 0;
        const T *src = static_cast<const T *>(in.data) + t * in.token_stride + h * in.head_stride;
        float x[U][2 * V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < 2 * V; ++j)
                x[u][j] = 0.0f;
            if (live && ok[u])
                load_unit<T, V>(x[u], src, lo[u], hi[u]);
        }
        if (NORM) {
            float sum = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < 2 * V; ++j)
                    sum += x[u][j] * x[u][j];
            sum = group_sum(sum, group);
            const float inv = 1.0f / sqrtf(sum * inv_dim + a.eps);
            const T *gain = static_cast<const T *>(is_q ? a.q_gain : a.k_gain);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (live && ok[u]) {
                    float g[2 * V];
                    load_unit<T, V>(g, gain, lo[u], hi[u]);
#pragma unroll
                    for (int j = 0; j < 2 * V; ++j)
                        x[u][j] *= inv * g[j];
                }
        }
        T *dst = static_cast<T *>(const_cast<void *>(out.data)) + t * out.token_stride +
                 h * out.head_stride;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (live && ok[u]) {
                turn_unit<V>(x[u], c[u], s[u], adjacent);
                store_unit<T, V>(dst, x[u], lo[u], hi[u]);
            }
    }
}

// Backward of norm_rotate: a wave takes whole tokens, so that its sums of the
// gains' gradients stay in registers (fp32) until the end; they are joined
// over the block in LDS and written as one row of a.partial.  No atomics: the
// result does not depend on the order in which blocks run.
template <typename T, int V, int U>
__global__ __launch_bounds__(kThreads) void norm_rotate_backward_kernel(RotaryArgs a, int group,
                                                                        int units)
{
    __shared__ float sums[kWaves][2][kMaxRotaryDim];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & (group - 1);
    const int slots = 64 / group;
    const int rows = a.q_heads + a.k_heads;
    const bool adjacent = a.adjacent != 0;
    const float inv_dim = 1.0f / float(a.dim);

    int lo[U], hi[U];
    bool ok[U];
    float acc[2][U][2 * V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int unit = li + u * group;
        ok[u] = unit < units;
        unit_offsets<V>(ok[u] ? unit : 0, a.pairs, adjacent, lo[u], hi[u]);
#pragma unroll
        for (int j = 0; j < 2 * V; ++j)
            acc[0][u][j] = acc[1][u][j] = 0.0f;
    }

    for (int64_t t = int64_t(blockIdx.x) * kWaves + wave; t < a.tokens;
         t += int64_t(gridDim.x) * kWaves) {
        float c[U][V], s[U][V];
        angles<U, V>(c, s, a, t, li, group);
        for (int r0 = 0; r0 < rows; r0 += slots) {
            const int r = r0 + lane / group;
            const bool live = r < rows;
            const bool is_q = r < a.q_heads;
            const int h = live ? (is_q ? r : r - a.q_heads) : 0;
            const Heads &in = is_q ? a.q : a.k;
            const Heads &gr = is_q ? a.gq : a.gk;
            const Heads &out = is_q ? a.oq : a.ok;
            const T *src = static_cast<const T *>(in.data) + t * in.token_stride +
                           h * in.head_stride;
            const T *gsrc = static_cast<const T *>(gr.data) + t * gr.token_stride +
                            h * gr.head_stride;
            const T *gain = static_cast<const T *>(is_q ? a.q_gain : a.k_gain);
            float x[U][2 * V], g[U][2 * V], w[U][2 * V];
            float sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int j = 0; j < 2 * V; ++j)
                    x[u][j] = g[u][j] = w[u][j] = 0.0f;
                if (live && ok[u]) {
                    load_unit<T, V>(x[u], src, lo[u], hi[u]);
                    load_unit<T, V>(g[u], gsrc, lo[u], hi[u]);
                    load_unit<T, V>(w[u], gain, lo[u], hi[u]);
                }
                turn_unit<V>(g[u], c[u], s[u], adjacent);     // s is -sin here
#pragma unroll
                for (int j = 0; j < 2 * V; ++j) {
                    sum += x[u][j] * x[u][j];
                    dot += g[u][j] * w[u][j] * x[u][j];
                }
            }
            sum = group_sum(sum, group);
            dot = group_sum(dot, group);
            const float inv = 1.0f / sqrtf(sum * inv_dim + a.eps);
            const float corr = dot * inv * inv_dim;            // mean(h * n)
            T *dst = static_cast<T *>(const_cast<void *>(out.data)) + t * out.token_stride +
                     h * out.head_stride;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float d[2 * V];
#pragma unroll
                for (int j = 0; j < 2 * V; ++j) {
                    const float n = x[u][j] * inv;
                    d[j] = inv * (g[u][j] * w[u][j] - n * corr);
                    const float gn = live && ok[u] ? g[u][j] * n : 0.0f;
                    acc[0][u][j] += is_q ? gn : 0.0f;
                    acc[1][u][j] += is_q ? 0.0f : gn;
                }
                if (live && ok[u])
                    store_unit<T, V>(dst, d, lo[u], hi[u]);
            }
        }
    }

#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 2 * V; ++j) {
                float v = acc[k][u][j];
                for (int m = group; m < 64; m <<= 1)
                    v += __shfl_xor(v, m, 64);
                if (lane < group && ok[u])
                    sums[wave][k][j < V ? lo[u] + j : hi[u] + j - V] = v;
            }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.dim; i += kThreads) {
        const int k = i / a.dim, d = i % a.dim;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            v += sums[w][k][d];
        a.partial[int64_t(blockIdx.x) * 2 * a.dim + i] = v;
    }
}

// Column sums of partial[blocks][2 * dim]: 32 columns a block, 8 rows at a
// time (128-byte reads), joined in LDS.
template <typename T>
__global__ __launch_bounds__(256) void gain_sum_kernel(const float *partial, int blocks, int dim,
                                                       int k_heads, T *dq_gain, T *dk_gain)
{
    __shared__ float part[8][32];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x >> 5;
    float v = 0.0f;
    if (col < 2 * dim)
        for (int b = row; b < blocks; b += 8)
            v += partial[int64_t(b) * 2 * dim + col];
    part[row][threadIdx.x & 31] = v;
    __syncthreads();
    if (row == 0 && col < 2 * dim) {
        for (int r = 1; r < 8; ++r)
            v += part[r][threadIdx.x];
        if (col < dim)
            dq_gain[col] = from_f32<T>(v);
        else if (k_heads > 0)
            dk_gain[col - dim] = from_f32<T>(v);
    }
}

bool wide_enough(const Heads &h, int v, size_t elem)
{
    return !h.data || (h.token_stride % v == 0 && h.head_stride % v == 0 &&
                       reinterpret_cast<uintptr_t>(h.data) % (v * elem) == 0);
}

// The widest vector that every access of the call allows.
int vector_width(const RotaryArgs &a, RotaryKind kind, size_t elem)
{
    for (int v = int(16 / elem); v > 1; v /= 2) {
        const int rest = a.dim - 2 * a.pairs;
        bool ok = a.pairs % v == 0 && rest % (2 * v) == 0;
        for (const Heads *h : {&a.q, &a.k, &a.oq, &a.ok})
            ok = ok && wide_enough(*h, v, elem);
        if (kind == RotaryKind::NormRotateBackward)
            ok = ok && wide_enough(a.gq, v, elem) && wide_enough(a.gk, v, elem);
        if (kind != RotaryKind::Rotate)
            ok = ok && reinterpret_cast<uintptr_t>(a.q_gain) % (v * elem) == 0 &&
                 reinterpret_cast<uintptr_t>(a.k_gain) % (v * elem) == 0;
        if (ok)
            return v;
    }
    return 1;
}

template <typename T, int V, int U>
hipError_t launch_units(RotaryKind kind, const RotaryArgs &a, int group, int units, hipStream_t s)
{
    if (kind == RotaryKind::NormRotateBackward) {
        norm_rotate_backward_kernel<T, V, U>
            <<<rotary_backward_blocks(a.tokens), kThreads, 0, s>>>(a, group, units);
        return hipGetLastError();
    }
    const int slots = 64 / group;
    const int rounds = (a.q_heads + a.k_heads + slots - 1) / slots;
    // A few tokens (a decoding step) are spread over the chip by giving each
    // wave fewer of a token's heads; enough tokens to fill it take all of a
    // token's heads in one wave, which computes the angles once.
    const int64_t want = 4096;                     // waves that keep the chip busy
    int split = int((want + a.tokens - 1) / a.tokens);
    split = split < 1 ? 1 : split > rounds ? rounds : split;
    const int per_wave = (rounds + split - 1) / split;
    const int waves = (rounds + per_wave - 1) / per_wave;
    const int64_t blocks = (a.tokens * waves + kWaves - 1) / kWaves;
    if (blocks > INT32_MAX)
        return hipErrorInvalidValue;
    if (kind == RotaryKind::Rotate)
        rotary_kernel<T, V, U, false>
            <<<uint32_t(blocks), kThreads, 0, s>>>(a, group, units, per_wave, waves);
    else
        rotary_kernel<T, V, U, true>
            <<<uint32_t(blocks), kThreads, 0, s>>>(a, group, units, per_wave, waves);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t launch_width(RotaryKind kind, const RotaryArgs &a, hipStream_t s)
{
    const int units = a.dim / (2 * V);
    int group = 1;
    while (group < units && group < 64)
        group *= 2;
    if (units <= 64)
        return launch_units<T, V, 1>(kind, a, group, units, s);
    if constexpr (V == 1)                           // up to 128 units of single pairs
        return launch_units<T, V, 2>(kind, a, group, units, s);
    return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_type(RotaryKind kind, const RotaryArgs &a, hipStream_t s)
{
    switch (vector_width(a, kind, sizeof(T))) {
    case 8:
        if constexpr (sizeof(T) == 2)
            return launch_width<T, 8>(kind, a, s);
        return hipErrorInvalidValue;
    case 4:
        return launch_width<T, 4>(kind, a, s);
    case 2:
        return launch_width<T, 2>(kind, a, s);
    default:
        return launch_width<T, 1>(kind, a, s);
    }
}

}  // namespace

int rotary_backward_blocks(int64_t tokens)
{
    const int64_t need = (tokens + kWaves - 1) / kWaves;
    return int(need < 1024 ? (need > 0 ? need : 1) : 1024);
}

hipError_t launch_rotary(RotaryKind kind, mdcn_dtype dtype, const RotaryArgs &a, hipStream_t s)
{
    switch (dtype) {
    case MDCN_F32:
        return launch_type<float>(kind, a, s);
    case MDCN_F16:
        return launch_type<half_t>(kind, a, s);
    default:
        return launch_type<bf16_t>(kind, a, s);
    }
}

template <typename T>
static hipError_t gain_sum(const RotaryArgs &a, void *dq, void *dk, hipStream_t s)
{
    gain_sum_kernel<T><<<(2 * a.dim + 31) / 32, 256, 0, s>>>(
        a.partial, rotary_backward_blocks(a.tokens), a.dim, a.k_heads, static_cast<T *>(dq),
        static_cast<T *>(dk));
    return hipGetLastError();
}

hipError_t launch_gain_sum(mdcn_dtype dtype, const RotaryArgs &a, void *dq_gain, void *dk_gain,
                           hipStream_t s)
{
    switch (dtype) {
    case MDCN_F32:
        return gain_sum<float>(a, dq_gain, dk_gain, s);
    case MDCN_F16:
        return gain_sum<half_t>(a, dq_gain, dk_gain, s);
    default:
        return gain_sum<bf16_t>(a, dq_gain, dk_gain, s);
    }
}

}  // namespace mdcn
