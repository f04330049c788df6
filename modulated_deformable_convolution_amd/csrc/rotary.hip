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
// Angles: in units of 2^-64 turns, as 64-bit integers whose product with a position drops
// the whole turns by itself: off by 2^-34 turns at most at any int32 position (a
// rounded product of rounded doubles by 3e-7 rad at 2^31), of which the upper 32 bits
// are taken; sine and cosine in fp32.  A wave computes the
// pairs of a token once, one or two per lane, and shares them through LDS for all
// heads of the token.
//
// A head is spread over G lanes (a power of two), each holding units of V
// values from the first channels of its pairs and the V second channels, so
// both partners of a pair are in one lane and every access is one V-wide
// vector; V is the widest of 8, 4, 2, 1 that divides the pairs, the unturned
// rest, and all strides and addresses.  Bound by memory: one read and one write
// of each value (backward: two reads, one write), the next heads read while
// these are turned.  One MI355X: 51201 tokens of 20 heads of 128 in bf16 99 us
// (5.3 TB/s; a large copy reaches 4.8), fp32 198 us (5.3); norm and rotation of 16000
// tokens of 40 heads 68 us (4.8 TB/s), fp32 132 us (5.0); 8193 tokens of 20 heads of 96
// of which 36 pairs turn (V = 4, 12 of 16 lanes) forward 20 us (3.1 TB/s), backward
// 32 us (3.0 TB/s) and 4 us for the gains' sums.  With each lane's angles computed for itself
// and no rounds read ahead the first took 150 us.
#include "attention.h"
#include "device_common.h"

namespace mdcn {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxBackwardBlocks = 1024;

template <typename T, int V> struct alignas(V * sizeof(T) < 16 ? V * sizeof(T) : 16) Pack {
    T e[V];
};

// A unit as it lies in memory.
template <typename T, int V> struct Unit {
    Pack<T, V> lo, hi;

    __device__ __forceinline__ void load(const T *p, int lo_at, int hi_at)
    {
        lo = *reinterpret_cast<const Pack<T, V> *>(p + lo_at);
        hi = *reinterpret_cast<const Pack<T, V> *>(p + hi_at);
    }

    __device__ __forceinline__ void store(T *p, int lo_at, int hi_at) const
    {
        *reinterpret_cast<Pack<T, V> *>(p + lo_at) = lo;
        *reinterpret_cast<Pack<T, V> *>(p + hi_at) = hi;
    }

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int j = 0; j < V; ++j)
            lo.e[j] = hi.e[j] = T(0.0f);
    }

    __device__ __forceinline__ void get(float (&x)[2 * V]) const
    {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            x[j] = to_f32(lo.e[j]);
            x[V + j] = to_f32(hi.e[j]);
        }
    }

    __device__ __forceinline__ void set(const float (&x)[2 * V])
    {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            lo.e[j] = from_f32<T>(x[j]);
            hi.e[j] = from_f32<T>(x[V + j]);
        }
    }
};

// Unit u of a head: V pairs, as the channel offsets of its two vectors.  For
// adjacent pairs the two vectors are the halves of 2V consecutive channels.
template <int V, bool ADJ>
__device__ __forceinline__ void unit_offsets(int u, int pairs, int &lo, int &hi)
{
    const int turned = pairs / V;
    if (ADJ) {
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

// x[0..V) and x[V..2V) are a unit's two vectors.  V divides the pairs, so a unit is
// turned or left as it is as a whole: a turn by the angle 0 would multiply each
// channel by the other's 0, which is not nothing where that one is not finite.
template <int V, bool ADJ>
__device__ __forceinline__ void turn_unit(float (&x)[2 * V], const float (&c)[V],
                                          const float (&s)[V], bool turned)
{
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int lo = ADJ ? 2 * j : j, hi = ADJ ? 2 * j + 1 : j + V;
        const float a = x[lo], b = x[hi];
        x[lo] = turned ? a * c[j] - b * s[j] : a;
        x[hi] = turned ? a * s[j] + b * c[j] : b;
    }
}

// Sine and cosine of an angle in units of 2^-32 turns: quarter turns taken off, and the
// Taylor series on [-pi/4, pi/4] up to the terms below 2^-30.  The angle enters as a
// float and what that leaves, so that both are within 2^-24 of the exact values.
__device__ __forceinline__ void sine_cosine(int32_t angle, float &sine, float &cosine)
{
    const int n = int(uint32_t(angle) + (1u << 29)) >> 30;
    const double theta = double(int32_t(uint32_t(angle) - (uint32_t(n) << 30))) *
                         (6.283185307179586 / 4294967296.0);
    const float t = float(theta), rest = float(theta - double(t));
    const float z = t * t, z_rest = fmaf(t, t, -z) + 2.0f * t * rest;
    float p = fmaf(z, 1.0f / 362880, -1.0f / 5040);
    p = fmaf(z, p, 1.0f / 120);
    p = fmaf(z, p, -1.0f / 6);
    const float s = t + fmaf(t * z, p, rest);
    float q = fmaf(z, -1.0f / 3628800, 1.0f / 40320);
    q = fmaf(z, q, -1.0f / 720);
    q = fmaf(z, q, 1.0f / 24);
    const float c = 1.0f + (fmaf(z * z, q, -0.5f * z_rest) - 0.5f * z);
    const float a = n & 1 ? c : s, b = n & 1 ? s : c;
    sine = n & 2 ? -a : a;
    cosine = (n + 1) & 2 ? -b : b;
}

// Cosines and sines of one token's pairs, in LDS: each lane computes every
// 64th pair and all read what their units need, (1, 0) past the turned
// pairs.  A wave writes and reads its own table only.
struct Angles {
    alignas(16) float c[kMaxRotaryDim / 2], s[kMaxRotaryDim / 2];
};

template <int U, int V>
__device__ __forceinline__ void angles(float (&c)[U][V], float (&s)[U][V], Angles &table,
                                       const RotaryArgs &a, int64_t t, int lane, const int (&at)[U])
{
    __builtin_amdgcn_wave_barrier();                 // the last token's reads come first
    for (int i = lane; i < a.dim / 2; i += 64) {
        float cv = 1.0f, sv = 0.0f;
        if (i < a.pairs) {
            const int64_t p = a.positions[a.table.axis[i] * a.axis_stride + t];
            sine_cosine(int32_t(uint64_t(p) * a.table.turns[i] >> 32), sv, cv);
        }
        table.c[i] = cv;
        table.s[i] = a.inverse ? -sv : sv;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Pack<float, V> cv = *reinterpret_cast<const Pack<float, V> *>(table.c + at[u]);
        const Pack<float, V> sv = *reinterpret_cast<const Pack<float, V> *>(table.s + at[u]);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            c[u][j] = cv.e[j];
            s[u][j] = sv.e[j];
        }
    }
}

template <int CTRL> __device__ __forceinline__ float lane_add(float v)
{
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf,
                                                          true));
}

// Sum over the `group` lanes (a power of two, aligned) that share a head.  Up to
// 16 lanes without LDS: neighbours, pairs, then mirrored halves and rows.
__device__ __forceinline__ float group_sum(float v, int group)
{
    if (group > 1)
        v = lane_add<0xb1>(v);                       // quad: lane ^ 1
    if (group > 2)
        v = lane_add<0x4e>(v);                       // quad: lane ^ 2
    if (group > 4)
        v = lane_add<0x141>(v);                      // 7 - lane of each 8
    if (group > 8)
        v = lane_add<0x140>(v);                      // 15 - lane of each 16
    if (group > 16)
        v += __shfl_xor(v, 16, 64);
    if (group > 32)
        v += __shfl_xor(v, 32, 64);
    return v;
}

// Forward (rotate, norm_rotate): one wave takes `per_wave` rounds of one
// token's heads, 64 / G heads a round.
template <typename T, int V, int U, bool ADJ, bool ALL, bool NORM>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, int group, int units,
                                                          int per_wave, int waves_per_token)
{
    __shared__ Angles table[kWaves];
    const int lane = threadIdx.x & 63;
    const int64_t w = int64_t(blockIdx.x) * kWaves + (threadIdx.x >> 6);
    const int64_t t = w / waves_per_token;
    if (t >= a.tokens)
        return;
    const int part = int(w - t * waves_per_token);
    const int li = lane & (group - 1);
    const int slots = 64 / group;
    const int rows = a.q_heads + a.k_heads;

    int lo[U], hi[U], at[U];                         // at: the unit's first pair
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int unit = li + u * group;
        ok[u] = unit < units;
        at[u] = ok[u] ? unit * V : 0;
        unit_offsets<V, ADJ>(ok[u] ? unit : 0, a.pairs, lo[u], hi[u]);
    }

    // The heads of a round are read one round ahead, the first before the
    // angles are computed.
    auto fetch = [&](Unit<T, V>(&x)[U], int r) {
        const bool is_q = r < a.q_heads;
        const Heads &in = is_q ? a.q : a.k;
        const T *src = static_cast<const T *>(in.data) + t * in.token_stride +
                       (is_q ? r : r - a.q_heads) * in.head_stride;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u].clear();
            if (r < rows && ok[u])
                x[u].load(src, lo[u], hi[u]);
        }
    };
    const int r_begin = part * per_wave * slots + lane / group;
    const int r_end = min(rows, (part + 1) * per_wave * slots);
    Unit<T, V> next[U], gain_q[U], gain_k[U];
    fetch(next, r_begin);
    if (NORM) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            gain_q[u].clear();
            gain_k[u].clear();
            if (ok[u] && a.q_heads > 0)
                gain_q[u].load(static_cast<const T *>(a.q_gain), lo[u], hi[u]);
            if (ok[u] && a.k_heads > 0)
                gain_k[u].load(static_cast<const T *>(a.k_gain), lo[u], hi[u]);
        }
    }
    float c[U][V], s[U][V];
    angles<U, V>(c, s, table[threadIdx.x >> 6], a, t, lane, at);

    const float inv_dim = 1.0f / float(a.dim);
    // (the group sums need all lanes, also those whose row is past the end)
    for (int r = r_begin; r - lane / group < r_end; r += slots) {
        const bool live = r < rows;
        const bool is_q = r < a.q_heads;
        float x[U][2 * V];
#pragma unroll
        for (int u = 0; u < U; ++u)
            next[u].get(x[u]);
        if (r + slots - lane / group < r_end)
            fetch(next, r + slots);
        if (NORM) {
            float sum = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < 2 * V; ++j)
                    sum += x[u][j] * x[u][j];
            sum = group_sum(sum, group);
            const float inv = 1.0f / sqrtf(sum * inv_dim + a.eps);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Unit<T, V> w = is_q ? gain_q[u] : gain_k[u];
                float g[2 * V];
                w.get(g);
#pragma unroll
                for (int j = 0; j < 2 * V; ++j)
                    x[u][j] *= inv * g[j];
            }
        }
        const Heads &out = is_q ? a.oq : a.ok;
        T *dst = static_cast<T *>(const_cast<void *>(out.data)) + t * out.token_stride +
                 (is_q ? r : r - a.q_heads) * out.head_stride;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (live && ok[u]) {
                turn_unit<V, ADJ>(x[u], c[u], s[u], ALL || at[u] < a.pairs);
                Unit<T, V> y;
                y.set(x[u]);
                y.store(dst, lo[u], hi[u]);
            }
    }
}

// Backward of norm_rotate: a wave takes whole tokens, so that its sums of the
// gains' gradients stay in registers (fp32) until the end; they are joined
// over the block in LDS and written as one row of a.partial.  No atomics: the
// result does not depend on the order in which blocks run.
template <typename T, int V, int U, bool ADJ, bool ALL>
__global__ __launch_bounds__(kThreads) void norm_rotate_backward_kernel(RotaryArgs a, int group,
                                                                        int units)
{
    __shared__ Angles table[kWaves];
    __shared__ float sums[kWaves][2][kMaxRotaryDim];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & (group - 1);
    const int slots = 64 / group;
    const int rows = a.q_heads + a.k_heads;
    const float inv_dim = 1.0f / float(a.dim);

    int lo[U], hi[U], at[U];                         // at: the unit's first pair
    bool ok[U];
    float acc[2][U][2 * V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int unit = li + u * group;
        ok[u] = unit < units;
        at[u] = ok[u] ? unit * V : 0;
        unit_offsets<V, ADJ>(ok[u] ? unit : 0, a.pairs, lo[u], hi[u]);
#pragma unroll
        for (int j = 0; j < 2 * V; ++j)
            acc[0][u][j] = acc[1][u][j] = 0.0f;
    }

    Unit<T, V> gain_q[U], gain_k[U], next_x[U], next_g[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        gain_q[u].clear();
        gain_k[u].clear();
        if (ok[u] && a.q_heads > 0)
            gain_q[u].load(static_cast<const T *>(a.q_gain), lo[u], hi[u]);
        if (ok[u] && a.k_heads > 0)
            gain_k[u].load(static_cast<const T *>(a.k_gain), lo[u], hi[u]);
    }
    // one round ahead, over the ends of tokens
    auto fetch = [&](int64_t t, int r) {
        const bool is_q = r < a.q_heads;
        const int h = is_q ? r : r - a.q_heads;
        const Heads &in = is_q ? a.q : a.k;
        const Heads &gr = is_q ? a.gq : a.gk;
        const T *src = static_cast<const T *>(in.data) + t * in.token_stride + h * in.head_stride;
        const T *gsrc = static_cast<const T *>(gr.data) + t * gr.token_stride + h * gr.head_stride;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            next_x[u].clear();
            next_g[u].clear();
            if (t < a.tokens && r < rows && ok[u]) {
                next_x[u].load(src, lo[u], hi[u]);
                next_g[u].load(gsrc, lo[u], hi[u]);
            }
        }
    };
    const int64_t t_step = int64_t(gridDim.x) * kWaves;
    const int64_t t_first = int64_t(blockIdx.x) * kWaves + wave;
    fetch(t_first, lane / group);
    for (int64_t t = t_first; t < a.tokens; t += t_step) {
        float c[U][V], s[U][V];
        angles<U, V>(c, s, table[threadIdx.x >> 6], a, t, lane, at);
        for (int r0 = 0; r0 < rows; r0 += slots) {
            const int r = r0 + lane / group;
            const bool live = r < rows;
            const bool is_q = r < a.q_heads;
            float x[U][2 * V], g[U][2 * V], w[U][2 * V];
            float sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                next_x[u].get(x[u]);
                next_g[u].get(g[u]);
            }
            if (r0 + slots < rows)
                fetch(t, r + slots);
            else
                fetch(t + t_step, lane / group);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Unit<T, V> wu = is_q ? gain_q[u] : gain_k[u];
                wu.get(w[u]);
                turn_unit<V, ADJ>(g[u], c[u], s[u], ALL || at[u] < a.pairs);   // s: -sin
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
            const Heads &out = is_q ? a.oq : a.ok;
            T *dst = static_cast<T *>(const_cast<void *>(out.data)) + t * out.token_stride +
                     (is_q ? r : r - a.q_heads) * out.head_stride;
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
                if (live && ok[u]) {
                    Unit<T, V> y;
                    y.set(d);
                    y.store(dst, lo[u], hi[u]);
                }
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

// Column sums of partial[blocks][2 * dim]: 16 columns a workgroup, 64 rows at a
// time, joined in LDS; at most 16 independent reads a thread.
constexpr int kSumCols = 16, kSumRows = 64;

template <typename T>
__global__ __launch_bounds__(kSumCols * kSumRows) void gain_sum_kernel(const float *partial,
                                                                       int blocks, int dim,
                                                                       T *dq_gain, T *dk_gain)
{
    __shared__ float part[kSumRows][kSumCols + 1];
    const int x = threadIdx.x % kSumCols, row = threadIdx.x / kSumCols;
    const int col = blockIdx.x * kSumCols + x;
    float v[kMaxBackwardBlocks / kSumRows];
#pragma unroll
    for (int i = 0; i < kMaxBackwardBlocks / kSumRows; ++i) {
        const int b = row + i * kSumRows;
        v[i] = b < blocks && col < 2 * dim ? partial[int64_t(b) * 2 * dim + col] : 0.0f;
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxBackwardBlocks / kSumRows; ++i)
        sum += v[i];
    part[row][x] = sum;
    __syncthreads();
    for (int n = kSumRows / 2; n > 0; n /= 2) {
        if (row < n)
            part[row][x] += part[row + n][x];
        __syncthreads();
    }
    if (row == 0 && col < 2 * dim) {
        if (col < dim) {
            if (dq_gain)
                dq_gain[col] = from_f32<T>(part[0][x]);
        } else if (dk_gain) {
            dk_gain[col - dim] = from_f32<T>(part[0][x]);
        }
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

// Lanes of a head of `units` units.
int lanes_of(int units)
{
    int group = 1;
    while (group < units && group < 64)
        group *= 2;
    return group;
}

// Rounds of a wave and waves of a token.  A few tokens (a decoding step) are spread
// over the chip by giving each wave fewer of a token's heads; enough tokens to fill it
// take all of a token's heads in one wave, which computes the angles once.
void share_token(const RotaryArgs &a, int group, int &per_wave, int &waves)
{
    const int slots = 64 / group;
    const int rounds = (a.q_heads + a.k_heads + slots - 1) / slots;
    const int64_t want = 4096;                     // waves that keep the chip busy
    int split = int((want + a.tokens - 1) / a.tokens);
    split = split < 1 ? 1 : split > rounds ? rounds : split;
    per_wave = (rounds + split - 1) / split;
    waves = (rounds + per_wave - 1) / per_wave;
}

template <typename T, int V, int U, bool ADJ, bool ALL>
hipError_t launch_units(RotaryKind kind, const RotaryArgs &a, int group, int units, hipStream_t s)
{
    if (kind == RotaryKind::NormRotateBackward) {
        norm_rotate_backward_kernel<T, V, U, ADJ, ALL>
            <<<rotary_backward_blocks(a.tokens), kThreads, 0, s>>>(a, group, units);
        return hipGetLastError();
    }
    int per_wave, waves;
    share_token(a, group, per_wave, waves);
    const int64_t blocks = (a.tokens * waves + kWaves - 1) / kWaves;
    if (blocks > INT32_MAX)
        return hipErrorInvalidValue;
    if (kind == RotaryKind::Rotate)
        rotary_kernel<T, V, U, ADJ, ALL, false>
            <<<uint32_t(blocks), kThreads, 0, s>>>(a, group, units, per_wave, waves);
    else
        rotary_kernel<T, V, U, ADJ, ALL, true>
            <<<uint32_t(blocks), kThreads, 0, s>>>(a, group, units, per_wave, waves);
    return hipGetLastError();
}

// Heads whose channels are all turned need no choice between turned and left values (16000
// tokens of 40 heads of 128 with their norm: 68.0 us, with the choice 69.4).
template <typename T, int V, int U>
hipError_t launch_turns(RotaryKind kind, const RotaryArgs &a, int group, int units, hipStream_t s)
{
    if (2 * a.pairs == a.dim)
        return a.adjacent ? launch_units<T, V, U, true, true>(kind, a, group, units, s)
                          : launch_units<T, V, U, false, true>(kind, a, group, units, s);
    return a.adjacent ? launch_units<T, V, U, true, false>(kind, a, group, units, s)
                      : launch_units<T, V, U, false, false>(kind, a, group, units, s);
}

template <typename T, int V>
hipError_t launch_width(RotaryKind kind, const RotaryArgs &a, hipStream_t s)
{
    const int units = a.dim / (2 * V), group = lanes_of(units);
    if (units <= 64)
        return launch_turns<T, V, 1>(kind, a, group, units, s);
    if constexpr (V == 1)                           // up to 128 units of single pairs
        return launch_turns<T, V, 2>(kind, a, group, units, s);
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

RotaryShape rotary_shape(RotaryKind kind, mdcn_dtype dtype, const RotaryArgs &a)
{
    RotaryShape s;
    s.width = vector_width(a, kind, dtype == MDCN_F32 ? 4 : 2);
    s.lanes = lanes_of(a.dim / (2 * s.width));
    share_token(a, s.lanes, s.rounds, s.waves);
    return s;
}

int rotary_backward_blocks(int64_t tokens)
{
    const int64_t need = (tokens + kWaves - 1) / kWaves;
    return int(need < kMaxBackwardBlocks ? (need > 0 ? need : 1) : kMaxBackwardBlocks);
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
    gain_sum_kernel<T><<<(2 * a.dim + kSumCols - 1) / kSumCols, kSumCols * kSumRows, 0, s>>>(
        a.partial, rotary_backward_blocks(a.tokens), a.dim, static_cast<T *>(dq),
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
