// cache_attend.h -- pieces of the attention kernels on 4-bit caches (gfx950).
//
// out = softmax(scale q k^T) v with one pass over the used tokens.  Scores are computed as
// S^T = K Q^T on 16x16x32 MFMA tiles, 16 rows (queries times the heads that share a key head)
// a tile: lane 16 g + c then holds row c's scores of tokens 4 g .. 4 g + 3 of a strip, which,
// rounded, are the operand of O^T = V^T P^T without any exchange, as the order of an
// instruction's k index is free as long as both operands share it.  The strips are laid out
// so that a lane's fp4 words of keys and values are the other operands once converted.
//
// Keys, values and scales are exact in 16 bits; the conversion takes 2^e from a float's
// exponent bits and ignores the others, so an exponent byte needs one shift.
// Values of one byte are two channels of one token (one exponent); two converted tokens
// are regrouped by channel with two permutes.  fp32 queries and probabilities are
// split into three bf16 parts (products with fp4 values are exact in fp32): 2^-24, at a
// fifth of the time of fp32 MFMA.
#pragma once

#include "cache_common.h"

namespace mdcn {

// s_waitcnt lgkmcnt(0), nothing else
constexpr int kWaitLds = 0xc07f;

// Whole numbers that no kernel writes while this one runs, read through the scalar cache.
typedef const int32_t __attribute__((address_space(4))) *scalar_ints;

constexpr int kWaves = 4;                        // of a workgroup

__device__ __forceinline__ float4v mfma16(half8 a, half8 b, float4v c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float4v mfma16(bf16x8 a, bf16x8 b, float4v c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// The 16-bit operands that stand for a value of T: itself, or three bf16 parts.
template <typename T> struct Operand {
    typedef T type;
    typedef T vec __attribute__((ext_vector_type(8)));
    static constexpr int PARTS = 1;
};
template <> struct Operand<float> {
    typedef bf16_t type;
    typedef bf16x8 vec;
    static constexpr int PARTS = 3;
};

template <typename T> using Vec = typename Operand<T>::vec;

// v[0..7] as operands.  16-bit types: rounded to nearest even (queries are exact); fp32:
// each part is the rounded rest.
template <typename T> struct Parts {
    Vec<T> p[Operand<T>::PARTS];

    // Waits for the loads behind the values here: the compiler would at their first use,
    // in the loop, in every round, and for the copies of the tiles to come with them.
    __device__ __forceinline__ void settle()
    {
#pragma unroll
        for (int i = 0; i < Operand<T>::PARTS; ++i) {
            uint32_t w[4];
            __builtin_memcpy(w, &p[i], 16);
            asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]));
            __builtin_memcpy(&p[i], w, 16);
        }
    }

    __device__ __forceinline__ void set(const float (&v)[8])
    {
        typedef float f8 __attribute__((ext_vector_type(8)));
        f8 x = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
#pragma unroll
        for (int i = 0; i < Operand<T>::PARTS; ++i) {
            p[i] = __builtin_convertvector(x, Vec<T>);
            if (i + 1 < Operand<T>::PARTS)
                x -= __builtin_convertvector(p[i], f8);
        }
    }
};

template <typename T>
__device__ __forceinline__ float4v product(Vec<T> a, const Parts<T> &b, float4v c)
{
#pragma unroll
    for (int i = Operand<T>::PARTS - 1; i >= 0; --i)
        c = mfma16(a, b.p[i], c);
    return c;
}

// What a lane reads of a strip.
template <int N> struct Raw {
    Words<N> k, v, ve;
    uint32_t ke;

    __device__ __forceinline__ void load(const char *strip, int lane)
    {
        constexpr Strip S{N};
        k = *reinterpret_cast<const Words<N> *>(strip + lane * 4 * N);
        const char *e = strip + S.key_exps() + (lane & 15) * S.key_exp();
        if constexpr (N == 1)
            ke = *reinterpret_cast<const uint8_t *>(e);
        else if constexpr (N == 2)
            ke = *reinterpret_cast<const uint16_t *>(e);
        else
            ke = *reinterpret_cast<const uint32_t *>(e);
        v = *reinterpret_cast<const Words<N> *>(strip + S.values() + lane * 4 * N);
        ve = *reinterpret_cast<const Words<N> *>(strip + S.value_exps() + (lane >> 4) * 4 * N);
    }
};

// Byte i of w where a float has its exponent, other bits of no meaning around it.
__device__ __forceinline__ uint32_t exponent_at(uint32_t w, int i)
{
    return i < 3 ? w << (23 - 8 * i) : w >> 1;
}

template <typename T> __device__ __forceinline__ Vec<T> as_vec(const uint32_t (&w)[4])
{
    Vec<T> v;
    __builtin_memcpy(&v, w, 16);
    return v;
}

// Keys of block j of a strip: 8 channels of the lane's token.
template <typename T, int N>
__device__ __forceinline__ Vec<T> key_operand(const Raw<N> &r, int j)
{
    using E = typename Operand<T>::type;
    const uint32_t e = exponent_at(r.ke, j);
    const uint32_t w[4] = {fp4_pair<E, 0>(r.k.w[j], e), fp4_pair<E, 1>(r.k.w[j], e),
                           fp4_pair<E, 2>(r.k.w[j], e), fp4_pair<E, 3>(r.k.w[j], e)};
    return as_vec<T>(w);
}

// Values of block b of a strip: 4 tokens of the lane's two channels, half of an operand each.
template <typename T, int N>
__device__ __forceinline__ void value_halves(const Raw<N> &x, int b, uint32_t (&even)[2],
                                             uint32_t (&odd)[2])
{
    using E = typename Operand<T>::type;
    const uint32_t w = x.v.w[b], e = x.ve.w[b];
    const uint32_t t[4] = {fp4_pair<E, 0>(w, exponent_at(e, 0)), fp4_pair<E, 1>(w, exponent_at(e, 1)),
                           fp4_pair<E, 2>(w, exponent_at(e, 2)),
                           fp4_pair<E, 3>(w, exponent_at(e, 3))};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        even[i] = __builtin_amdgcn_perm(t[2 * i + 1], t[2 * i], 0x05040100u);
        odd[i] = __builtin_amdgcn_perm(t[2 * i + 1], t[2 * i], 0x07060302u);
    }
}

// Tokens of a strip that do not exist get exponents of finite values, whatever bytes there
// are; `left` of the lane's four tokens exist.
template <int N> __device__ __forceinline__ void settle_values(Raw<N> &x, int left)
{
    const uint32_t keep = left <= 0 ? 0u : left >= 4 ? ~0u : 0xffffffffu >> (32 - 8 * left);
#pragma unroll
    for (int b = 0; b < N; ++b)
        x.ve.w[b] = (x.ve.w[b] & keep) | (0x7f7f7f7fu & ~keep);
}

// The largest of the four lanes that hold one row.
__device__ __forceinline__ float max_groups(float v)
{
    uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    return max_halves(v);
}

__device__ __forceinline__ float sum_groups(float v)
{
    uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    u = __float_as_uint(v);
    const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// One row tile's maxima, sums (the lane's own tokens only) and M tiles of outputs.
template <int M> struct State {
    float4v o[M];
    float m, l;

    __device__ __forceinline__ void init()
    {
#pragma unroll
        for (int i = 0; i < M; ++i)
            o[i] = (float4v){};
        m = -INFINITY;
        l = 0.0f;
    }

    __device__ __forceinline__ void raise(float top, float c)
    {
        const float up = fmaxf(top, m);
        const float f = up == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m - up) * c);
#pragma unroll
        for (int i = 0; i < M; ++i)
            o[i] *= f;
        l *= f;
        m = up;
    }

    __device__ __forceinline__ void merge(const State &x, float c)
    {
        const float up = fmaxf(m, x.m);
        const float f = m == up ? 1.0f : __builtin_amdgcn_exp2f((m - up) * c);
        const float g = x.m == up ? 1.0f : __builtin_amdgcn_exp2f((x.m - up) * c);
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[i][j] = fmaf(x.o[i][j], g, o[i][j] * f);
        l = fmaf(x.l, g, l * f);
        m = up;
    }
};

// Scores of NS strips, -infinity where hidden, to probabilities, which are added up and
// rounded to operands of two strips each.
template <typename T, int M, int NS>
__device__ __forceinline__ void softmax(State<M> &st, const float4v (&sc)[NS],
                                        Parts<T> (&p)[NS / 2], float c, float margin)
{
    float top = -INFINITY;
#pragma unroll
    for (int s = 0; s < NS; ++s)
        top = fmaxf(top, fmaxf(fmaxf(sc[s][0], sc[s][1]), fmaxf(sc[s][2], sc[s][3])));
    top = max_groups(top);
    if (__ballot(top > st.m + margin))
        st.raise(top, c);
    const float off = st.m == -INFINITY ? 0.0f
                      : sizeof(T) == 4  ? st.m
                                        : fmaf(st.m, c, float(-kLift<T>));
#pragma unroll
    for (int i = 0; i < NS / 2; ++i) {
        float e8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = sc[2 * i + (e >> 2)][e & 3];
            e8[e] = __builtin_amdgcn_exp2f(sizeof(T) == 4 ? (v - off) * c : fmaf(v, c, -off));
        }
        st.l += ((e8[0] + e8[1]) + (e8[2] + e8[3])) + ((e8[4] + e8[5]) + (e8[6] + e8[7]));
        p[i].set(e8);
    }
}

// ---- the batch -------------------------------------------------------------

struct Piece {
    int q0, lq, lk;                              // first query, queries, tokens of the cache
};

__device__ __forceinline__ Piece piece_of(const CacheArgs &a, int b)
{
    Piece p;
    p.q0 = clamp_int(a.cu[b], 0, a.tokens);
    p.lq = clamp_int(a.cu[b + 1], p.q0, a.tokens) - p.q0;
    p.lk = a.pages ? clamp_int(a.used[b], 0, a.width << a.page_shift) : 0;
    return p;
}

// Row c of row tile `index` of a (sequence, key head), c = lane % 16.
struct Row16 {
    int row, token, head;
    bool live;

    __device__ __forceinline__ Row16(const CacheArgs &a, int q0, int lq, int kv_head, uint32_t index,
                                     int lane)
    {
        const uint32_t shared = uint32_t(a.q_heads / a.k_heads), packed = index * 16 + (lane & 15);
        row = int(packed / shared);
        live = row < lq;
        token = q0 + row;
        head = kv_head * int(shared) + int(packed % shared);
    }
};

// Channels 32 j + 8 (lane / 16) and on of the lane's row.
template <typename T>
__device__ __forceinline__ Parts<T> query_of(const CacheArgs &a, const Row16 &r, int j, int lane)
{
    const int ch = j * 32 + (lane >> 4) * 8;
    float v[8] = {};
    if (r.live && ch < a.dim) {
        struct alignas(16) {
            T e[8];
        } x;
        const char *p = row_ptr<T>(a.q, r.token, r.head) + ch * sizeof(T);
        __builtin_memcpy(&x, __builtin_assume_aligned(p, 16), sizeof(x));
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = to_f32(x.e[e]);
    }
    Parts<T> q;
    q.set(v);
    return q;
}

// The last token that a row sees.
__device__ __forceinline__ int last_of(const CacheArgs &a, const Piece &pc, const Row16 &r)
{
    return !r.live ? -1 : a.causal ? r.row + pc.lk - pc.lq : pc.lk - 1;
}

// The queries of a row tile, and the last token that each row sees.
template <typename T, int N> struct RowTile {
    Parts<T> q[N];
    int last;

    __device__ __forceinline__ void load(const CacheArgs &a, const Piece &pc, int kv_head,
                                         uint32_t index, int lane)
    {
        const Row16 r(a, pc.q0, pc.lq, kv_head, index, lane);
        last = last_of(a, pc, r);
#pragma unroll
        for (int j = 0; j < N; ++j)
            q[j] = query_of<T>(a, r, j, lane);
    }
};

// What row tiles first .. first + n - 1 see: all their rows the tokens up to `all`, none those
// past `any`.
struct Sight {
    int all, any;

    __device__ __forceinline__ Sight(const CacheArgs &a, const Piece &pc, uint32_t first, uint32_t n)
    {
        const uint32_t shared = uint32_t(a.q_heads / a.k_heads);
        const int low = int(first * 16 / shared), high = int(((first + n) * 16 - 1) / shared);
        all = a.causal ? low + pc.lk - pc.lq : pc.lk - 1;
        any = low >= pc.lq ? -1 : a.causal ? min(high, pc.lq - 1) + pc.lk - pc.lq : pc.lk - 1;
    }
};

// 8 channels of an output from two tiles of sums and the sum of weights.
template <typename T>
__device__ __forceinline__ void put_block(const CacheArgs &a, const Row16 &at, int b, float4v even,
                                          float4v odd, float sum, int lane)
{
    const int ch = b * 32 + (lane >> 4) * 8;
    if (ch >= a.dim)
        return;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    struct alignas(16) {
        T e[8];
    } v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float o = i & 1 ? odd[i >> 1] : even[i >> 1];
        v.e[i] = from_f32<T>(sum == 0.0f ? 0.0f : sizeof(T) == 4 ? o / sum : o * inv);
    }
    char *row = const_cast<char *>(row_ptr<T>(a.out, at.token, at.head));
    __builtin_memcpy(__builtin_assume_aligned(row + ch * sizeof(T), 16), &v, sizeof(v));
}

// Sums of fp32 and bf16 values may pass the type's range where their mean does not: the
// format goes to 6 * 2^125, the type to 1.3 times that, and weights to 2^8 each.  A power of two taken
// off them would cost the smallest values their bits (2^-121, of 2^-149), so rows whose
// sums of values are not finite, while those of weights are, are `lost`: the second kernel
// computes them again, as means (put_mean).  (fp16: 2^16 * 2^15 a token at most.)
//
// Outputs of blocks b0 .. b0 + M / 2 - 1 of a finished row tile, and its lse; whether a row is lost.
template <typename T, int M>
__device__ __forceinline__ bool finish(const CacheArgs &a, const State<M> &s, const Row16 &at, int b0,
                                       int lane, float &lse)
{
    const float sum = sum_groups(s.l);
    lse = sum == 0.0f ? -INFINITY : row_lse<T>(s.m, sum, a.scale);
    bool lost = false;
    if (at.live) {
        if constexpr (!__is_same(T, half_t)) {
            float all = 0.0f;                    // NaN if a sum is not finite
#pragma unroll
            for (int i = 0; i < M; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    all = fmaf(s.o[i][j], 0.0f, all);
            lost = all != all && sum < INFINITY;
        }
#pragma unroll
        for (int b = 0; b < M / 2; ++b)
            put_block<T>(a, at, b0 + b, s.o[2 * b], s.o[2 * b + 1], sum, lane);
        if (b0 == 0 && lane < 16)
            a.lse[int64_t(at.head) * a.tokens + at.token] = lse;
    }
    return __ballot(lost) != 0;
}

// What is not finite in block b of a row tile, while the row's lse is, once more from that lse:
// weights are at most a half, as are their sums, so no sum exceeds the largest value, and small
// values lose nothing.  Few registers and no LDS, one pair of strips at a time: for values that
// the format lets happen, not for speed (with every row lost the 48 caches of 1 to 16384 tokens take
// 1.6 ms instead of 0.09).
template <typename T, int N>
__device__ __forceinline__ void put_mean(const CacheArgs &a, const Piece &pc, int sequence, int kv_head,
                                         uint32_t tile, const Row16 &at, float lse, int b, int lane)
{
    constexpr Strip S{N};
    bool lost = false;
    if (const int ch = b * 32 + (lane >> 4) * 8; at.live && ch < a.dim && lse < INFINITY) {
        struct alignas(16) {
            T e[8];
        } x;
        const char *p = row_ptr<T>(a.out, at.token, at.head) + ch * sizeof(T);
        __builtin_memcpy(&x, __builtin_assume_aligned(p, 16), sizeof(x));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            lost |= !(fabsf(to_f32(x.e[i])) < INFINITY);
    }
    if (!__ballot(lost))
        return;
    const float c = a.scale * kLog2e, off = lse == -INFINITY ? 0.0f : fmaf(lse, kLog2e, 1.0f);
    const int last = last_of(a, pc, at), any = Sight(a, pc, tile, 1).any;
    const int strip_shift = a.page_shift - 4, held = (pc.lk + (1 << a.page_shift) - 1) >> a.page_shift;
    const int32_t *const pages = a.table + sequence * a.table_stride;
    const char *const heads = a.pool + int64_t(kv_head << strip_shift) * S.bytes();
    float4v even = {}, odd = {};
    float sum = 0.0f;
    for (int t = 0; t * 32 <= any; ++t) {
        asm volatile("" ::: "memory");           // queries are read again, not held
        float w[8];
        uint32_t ev[2][2], od[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int strip = 2 * t + i, tok = strip * 16 + (lane >> 4) * 4;
            const int page = pages[min(strip >> strip_shift, held - 1)];
            const bool gone = page < 0 || page >= a.pages;
            const char *const p = heads + int64_t(gone ? 0 : page) * a.page_stride +
                                  (strip & ((1 << strip_shift) - 1)) * S.bytes();
            Raw<1> x;                            // one block of keys, then of values
            float4v sc = {};
#pragma unroll 1
            for (int j = 0; j < N; ++j) {
                x.k.w[0] = *reinterpret_cast<const uint32_t *>(p + (lane * N + j) * 4);
                x.ke = uint8_t(p[S.key_exps() + (lane & 15) * S.key_exp() + j]);
                sc = product<T>(key_operand<T, 1>(x, 0), query_of<T>(a, at, j, lane), sc);
            }
            x.v.w[0] = *reinterpret_cast<const uint32_t *>(p + S.values() + (lane * N + b) * 4);
            x.ve.w[0] = *reinterpret_cast<const uint32_t *>(p + S.value_exps() +
                                                            ((lane >> 4) * N + b) * 4);
            settle_values(x, gone ? 0 : pc.lk - tok);
            value_halves<T, 1>(x, 0, ev[i], od[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[4 * i + e] =
                    gone || tok + e > last ? 0.0f : __builtin_amdgcn_exp2f(fmaf(sc[e], c, -off));
                sum += w[4 * i + e];
            }
        }
        Parts<T> weights;
        weights.set(w);
        Vec<T> ve, vo;
        __builtin_memcpy(&ve, ev, 16);
        __builtin_memcpy(&vo, od, 16);
        even = product<T>(ve, weights, even);
        odd = product<T>(vo, weights, odd);
    }
    sum = sum_groups(sum);
    if (lost)
        put_block<T>(a, at, b, even, odd, sum, lane);
}

// Fills rows of no sequence: the workgroups past `workers`.
template <typename T> __device__ __forceinline__ void fill_rows(const CacheArgs &a)
{
    const int part = int(blockIdx.x) - a.workers, parts = int(gridDim.x) - a.workers;
    if (a.fill & kFillOut)
        zero_outside<T>(a.out, a.cu, a.batch, a.tokens, a.q_heads, a.dim, part, parts);
    if (a.fill & kFillLse)
        outside_rows(a.cu, a.batch, a.tokens, a.q_heads, part, parts, [&](int token, int h) {
            a.lse[int64_t(h) * a.tokens + token] = -INFINITY;
        });
}

// `n` workgroups, enough units for all waves of each; workgroup i has units
// [units * i / n, units * (i + 1) / n).
struct Share {
    int units, n, each, rest;

    __device__ __forceinline__ Share(int units_, int workers) : units(units_)
    {
        n = min((units + kWaves - 1) / kWaves, workers);
        each = n > 0 ? units / n : 0;
        rest = units - each * n;
    }

    __device__ __forceinline__ int begin(int i) const { return i * each + i * rest / n; }

    // the workgroup that has unit u
    __device__ __forceinline__ int owner(int u) const
    {
        int i = min(int(float(u) * (float(n) / float(units))), n - 1);   // off by one at most
        while (i + 1 < n && begin(i + 1) <= u)
            ++i;
        while (i > 0 && begin(i) > u)
            --i;
        return i;
    }
};

// What the second kernel is to do: join the item that begins in a workgroup's range
// and does not end there, and compute again those that begin and end in it, if rows are lost.
struct Join {
    int q0, lq, lk, sequence, head, tile;
    int last;                                    // workgroup of its last part, -1: nothing
    int lost;

    __device__ __forceinline__ void init() { last = -1, lost = 0; }

    __device__ __forceinline__ void set(const Piece &p, int sequence_, int head_, int tile_, int last_)
    {
        q0 = p.q0, lq = p.lq, lk = p.lk;
        sequence = sequence_, head = head_, tile = tile_, last = last_;
    }

    __device__ __forceinline__ Piece piece() const { return Piece{q0, lq, lk}; }
};

// A part in the workspace: registers as they are, [row tile][2 n + m and l][lane].
template <int N> constexpr int part_floats() { return (8 * N + 2) * 64; }

template <int M>
__device__ __forceinline__ void put_state(float *p, const State<M> &s, int lane)
{
#pragma unroll
    for (int i = 0; i < M; ++i)
        reinterpret_cast<float4v *>(p)[i * 64 + lane] = s.o[i];
    p[M * 256 + lane] = s.m;
    p[M * 256 + 64 + lane] = s.l;
}

template <int M>
__device__ __forceinline__ void get_state(State<M> &s, const float *p, int lane)
{
#pragma unroll
    for (int i = 0; i < M; ++i)
        s.o[i] = reinterpret_cast<const float4v *>(p)[i * 64 + lane];
    s.m = p[M * 256 + lane];
    s.l = p[M * 256 + 64 + lane];
}

// The kernel for many rows: 16 * kWaves * R of one key head a workgroup.
constexpr int tile_row_tiles(bool f32) { return kWaves * (f32 ? 1 : 2); }
constexpr int kTileWorkers = 512;
hipError_t launch_cache_tile(mdcn_dtype dtype, const CacheArgs &a, hipStream_t s);

}  // namespace mdcn
