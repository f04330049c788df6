// cache_attend.hip -- attention against a key/value cache in 4 bits.
//
// out = softmax(scale q k^T) v with one pass over the used tokens, in tiles of 32 (two strips).
// Scores are computed as S^T = K Q^T on 16x16x32 MFMA tiles, 16 rows (queries times the heads
// that share a key head) a tile: a lane then holds one row's scores of 8 tokens, which,
// rounded, are the operand of O^T = V^T P^T without any exchange, as the order of an
// instruction's k index is free as long as both operands share it.  The strips are laid out
// so that a lane's fp4 words of keys and values are the other operands once
// converted: no LDS and no exchange between lanes but the row maximum's.
//
// Keys, values and scales are exact in 16 bits; the conversion takes 2^e from a float's
// exponent bits and ignores the others, so an exponent byte needs one shift.
// Values of one byte are two channels of one token (one exponent); two converted tokens
// are regrouped by channel with two permutes.  fp32 queries and probabilities are
// split into three bf16 parts (products with fp4 values are exact in fp32): 2^-24, at a
// sixth of the time of fp32 MFMA.
//
// The work, in units of 32 tokens of one (sequence, key head, row tile), is cut into equal
// contiguous ranges, one per workgroup, whatever the lengths: lengths are read on the
// GPU.  The four waves of a workgroup take a quarter of a range's tokens each and are joined
// in LDS; a (sequence, head, tile) that several workgroups share goes to the workspace
// in parts that a second kernel joins.
#include <algorithm>

#include "cache_common.h"

namespace mdcn {

namespace {

constexpr int kTile = 32;                        // tokens

// s_waitcnt lgkmcnt(0), nothing else
constexpr int kWaitLds = 0xc07f;

// Whole numbers that no kernel writes while this one runs, read through the scalar cache.
typedef const int32_t __attribute__((address_space(4))) *scalar_ints;

constexpr int kWaves = 4;

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

// What a lane reads of a strip, in LDS.
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

// Waves a SIMD that the registers leave room for: a row tile of 16-bit queries with its sums
// takes 48 of 128 of them, a second one or the three parts of fp32 as much again.
template <typename T, int N, int R> constexpr int row_waves()
{
    return R > 1 ? 2 : sizeof(T) == 4 ? 3 : 4;
}

// A wave's ring of staged tiles (two strips each), copied there asynchronously: as many as
// fit its share of the LDS, so that a compute unit has about 140 KB on their way.
// COPIES instructions copy a tile.
template <int N, int WAVES> struct Ring {
    static constexpr int TILE = 2 * Strip{N}.bytes();
    static constexpr int SHARE = 160 * 1024 / 4 / WAVES - 64;
    static constexpr int DEPTH = SHARE / TILE < 8 ? SHARE / TILE : 8;
    static constexpr int STEPS = (Strip{N}.bytes() + 1023) / 1024;
    static constexpr int COPIES = 2 * STEPS;

    // 16 bytes a lane; lanes past the strip's end are switched off (they would write LDS)
    static __device__ __forceinline__ void load(uint32_t lds, const char *strip, int lane)
    {
        const v4i r = row_resource(strip, Strip{N}.bytes());
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const uint32_t off = uint32_t(i * 1024 + lane * 16);
            if ((i + 1) * 1024 <= Strip{N}.bytes() || off < uint32_t(Strip{N}.bytes()))
                dma_row16(__builtin_amdgcn_readfirstlane(lds + i * 1024), r, off);
        }
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

// Values of block b of two strips: 8 tokens of the lane's two channels.
template <typename T, int N>
__device__ __forceinline__ void value_operands(const Raw<N> &x, const Raw<N> &y, int b,
                                               Vec<T> &even, Vec<T> &odd)
{
    using E = typename Operand<T>::type;
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const uint32_t w = s ? y.v.w[b] : x.v.w[b], e = s ? y.ve.w[b] : x.ve.w[b];
        const uint32_t t[4] = {
            fp4_pair<E, 0>(w, exponent_at(e, 0)), fp4_pair<E, 1>(w, exponent_at(e, 1)),
            fp4_pair<E, 2>(w, exponent_at(e, 2)), fp4_pair<E, 3>(w, exponent_at(e, 3))};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            lo[2 * s + i] = __builtin_amdgcn_perm(t[2 * i + 1], t[2 * i], 0x05040100u);
            hi[2 * s + i] = __builtin_amdgcn_perm(t[2 * i + 1], t[2 * i], 0x07060302u);
        }
    }
    even = as_vec<T>(lo);
    odd = as_vec<T>(hi);
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

// Outputs of blocks b0 .. b0 + M / 2 - 1 of a finished row, and its lse.
template <typename T, int M>
__device__ __forceinline__ void finish(const CacheArgs &a, const State<M> &s, int token, int head,
                                       int b0, int group, bool live)
{
    const float sum = sum_groups(s.l);
    if (!live)
        return;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    char *row = const_cast<char *>(row_ptr<T>(a.out, token, head));
#pragma unroll
    for (int b = 0; b < M / 2; ++b) {
        const int ch = (b0 + b) * 32 + group * 8;
        if (ch < a.dim) {
            struct alignas(16) {
                T e[8];
            } v;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float o = s.o[2 * b + (i & 1)][i >> 1];
                v.e[i] = from_f32<T>(sum == 0.0f ? 0.0f : sizeof(T) == 4 ? o / sum : o * inv);
            }
            __builtin_memcpy(__builtin_assume_aligned(row + ch * sizeof(T), 16), &v, sizeof(v));
        }
    }
    if (b0 == 0 && group == 0)
        a.lse[int64_t(head) * a.tokens + token] =
            sum == 0.0f ? -INFINITY : row_lse<T>(s.m, sum, a.scale);
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

// Units of an item, a (key head, row tile) of a sequence: one for each 32 << unit_shift tokens,
// after kItemCost for what an item costs whatever its length.
struct Units {
    int tiles, keys, all;
};

constexpr int kItemCost = 10;
// Tiles up to which one wave takes an item alone, without the others and their barriers.
constexpr int kAlone = 3;

template <int R> __device__ __forceinline__ Units units_of(const CacheArgs &a, const Piece &p)
{
    Units u;
    const uint32_t rows = uint32_t(p.lq) * uint32_t(a.q_heads / a.k_heads);
    u.tiles = int((rows + 16 * R - 1) / (16 * R));
    u.keys = ((p.lk + (kTile << a.unit_shift) - 1) >> (5 + a.unit_shift)) + kItemCost;
    u.all = u.tiles * a.k_heads * u.keys;
    return u;
}

template <int R> struct Chunk {
    Piece piece;
    int mine, upto;

    __device__ __forceinline__ void load(const CacheArgs &a, int b0, int lane)
    {
        piece = {};
        mine = 0;
        if (b0 + lane < a.batch) {
            piece = piece_of(a, b0 + lane);
            mine = units_of<R>(a, piece).all;
        }
        upto = wave_scan(mine);
    }
};

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

// What the second kernel is to join: the item that begins in a workgroup's range
// and does not end there.
struct Join {
    int q0, lq, head, tile;
    int last;                                    // workgroup of its last part, -1: nothing
    int pad[3];
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

// Joins the four waves' states into wave 0's.
template <int R, int M>
__device__ __forceinline__ void join_waves(State<M> (&s)[R], float *lds, float c, int wave, int lane)
{
    constexpr int FLOATS = (4 * M + 2) * 64;
#pragma unroll
    for (int half = 2; half >= 1; half /= 2) {
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                put_state(lds + ((wave - half) * R + r) * FLOATS, s[r], lane);
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                State<M> x;
                get_state(x, lds + (wave * R + r) * FLOATS, lane);
                s[r].merge(x, c);
            }
        }
        __syncthreads();
    }
}

template <typename T, int N, int R>
__global__ __launch_bounds__(256, (row_waves<T, N, R>())) void cache_attend_kernel(CacheArgs a)
{
    constexpr Strip S{N};
    using ring = Ring<N, row_waves<T, N, R>()>;
    constexpr int RING = ring::DEPTH * ring::TILE;
    constexpr int JOIN = 2 * R * part_floats<N>() * 4;
    __shared__ __align__(16) char smem[kWaves * RING > JOIN ? kWaves * RING : JOIN];
    float *const lds = reinterpret_cast<float *>(smem);

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const char *const own = smem + wave * RING;
    const uint32_t ring_lds = lds_address(own);
    const int col = lane & 15, grp = lane >> 4;
    const int shared = a.q_heads / a.k_heads;
    const float c = a.scale * kLog2e, margin = raise_margin(c);

    if (int(blockIdx.x) >= a.workers) {          // tokens of no sequence
        const int part = int(blockIdx.x) - a.workers, parts = int(gridDim.x) - a.workers;
        if (a.fill & kFillOut)
            zero_outside<T>(a.out, a.cu, a.batch, a.tokens, a.q_heads, a.dim, part, parts);
        if (a.fill & kFillLse)
            outside_rows(a.cu, a.batch, a.tokens, a.q_heads, part, parts, [&](int token, int h) {
                a.lse[int64_t(h) * a.tokens + token] = -INFINITY;
            });
        return;
    }

    Chunk<R> chunk;
    chunk.load(a, 0, lane);
    int units = __builtin_amdgcn_readlane(chunk.upto, 63);
    if (a.batch > 64) {
        int more = 0;
        for (int b = 64 + lane; b < a.batch; b += 64)
            more += units_of<R>(a, piece_of(a, b)).all;
        units += wave_sum(more);
    }
    const Share share(units, a.workers);
    Join *join = reinterpret_cast<Join *>(a.joins) + blockIdx.x;
    if (threadIdx.x == 0)
        join->last = -1;
    if (int(blockIdx.x) >= share.n)
        return;
    __syncthreads();                             // another wave may write it below
    const int u_begin = share.begin(int(blockIdx.x)), u_end = share.begin(int(blockIdx.x) + 1);
    const int strip_shift = a.page_shift - 4;

    int base = 0, turn = 0;
    for (int b0 = 0; b0 < a.batch && base < u_end; b0 += 64) {
        if (b0 > 0)
            chunk.load(a, b0, lane);
        const int s_end_l = base + chunk.upto, s_begin_l = s_end_l - chunk.mine;
        uint64_t mine = __ballot(chunk.mine > 0 && s_end_l > u_begin && s_begin_l < u_end);
        for (; mine; mine &= mine - 1) {
            const int i = __builtin_ctzll(mine);
            const int s_end = __builtin_amdgcn_readlane(s_end_l, i);
            const int s_begin = __builtin_amdgcn_readlane(s_begin_l, i);
            Piece pc;
            pc.q0 = __builtin_amdgcn_readlane(chunk.piece.q0, i);
            pc.lq = __builtin_amdgcn_readlane(chunk.piece.lq, i);
            pc.lk = __builtin_amdgcn_readlane(chunk.piece.lk, i);
            const Units un = units_of<R>(a, pc);
            const int shift = pc.lk - pc.lq;
            const int to = min(u_end, s_end);
            const auto row_pages = reinterpret_cast<scalar_ints>(
                reinterpret_cast<uintptr_t>(a.table + int64_t(b0 + i) * a.table_stride));
            const int held = (pc.lk + (1 << a.page_shift) - 1) >> a.page_shift;
            for (int u = max(u_begin, s_begin); u < to;) {
                // item: a (key head, row tile) of this sequence; keys [n0, n1) of it, in units
                const int item = (u - s_begin) / un.keys;
                const int i_begin = s_begin + item * un.keys;
                const int n0 = u - i_begin, n1 = min(to - i_begin, un.keys);
                u = i_begin + n1;
                const int kv_head = item / un.tiles, tile = item % un.tiles;
                if (kv_head >= a.k_heads)
                    return;                      // offsets that overlap beyond counting
                const int t0 = max(n0 - kItemCost, 0) << a.unit_shift;
                const int nt = (max(n1 - kItemCost, 0) << a.unit_shift) - t0;
                const bool alone = nt <= kAlone;
                if (alone && (turn++ & (kWaves - 1)) != wave)
                    continue;

                int last[R], token[R], head[R];
                bool live[R];
                Parts<T> q[R][N];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const uint32_t packed = (uint32_t(tile) * R + r) * 16 + col;
                    const int row = int(packed / uint32_t(shared));
                    live[r] = row < pc.lq;
                    token[r] = pc.q0 + row;
                    head[r] = kv_head * shared + int(packed % uint32_t(shared));
                    last[r] = a.causal ? row + shift : pc.lk - 1;
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const int ch = j * 32 + grp * 8;
                        float v[8] = {};
                        if (live[r] && ch < a.dim) {
                            struct alignas(16) {
                                T e[8];
                            } x;
                            __builtin_memcpy(&x,
                                             __builtin_assume_aligned(
                                                 row_ptr<T>(a.q, token[r], head[r]) +
                                                     ch * sizeof(T),
                                                 16),
                                             sizeof(x));
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                v[e] = to_f32(x.e[e]);
                        }
                        q[r][j].set(v);
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        q[r][j].settle();
                const int first_row = int(uint32_t(tile) * R * 16 / uint32_t(shared));
                const int last_row = min(int((uint32_t(tile) * R * 16 + R * 16 - 1) /
                                             uint32_t(shared)), pc.lq - 1);
                // all rows of the tile see the tokens up to `all_see`, none those past `any_sees`
                const int all_see = a.causal ? first_row + shift : pc.lk - 1;
                const int any_sees = a.causal ? last_row + shift : pc.lk - 1;

                const int visible = any_sees < 0 ? 0 : any_sees / kTile + 1;
                int w0 = t0, w1 = t0 + nt;
                if (!alone) {
                    w0 = t0 + nt / kWaves * wave + min(nt % kWaves, wave);
                    w1 = t0 + nt / kWaves * (wave + 1) + min(nt % kWaves, wave + 1);
                }
                w1 = min(w1, visible);

                State<2 * N> st[R];
#pragma unroll
                for (int r = 0; r < R; ++r)
                    st[r].init();

                // What strip s lies in: the page that the table names, or, if that is none, page 0.
                const char *const heads = a.pool + int64_t(kv_head << strip_shift) * S.bytes();
                auto page_of = [&](int s) { return row_pages[min(s >> strip_shift, held - 1)]; };
                auto stage = [&](uint32_t to, int s, int n) {
                    const uint32_t page = uint32_t(n) < uint32_t(a.pages) ? uint32_t(n) : 0u;
                    ring::load(to, heads + uint64_t(page) * uint32_t(a.page_stride) +
                                       (s & ((1 << strip_shift) - 1)) * S.bytes(), lane);
                    return page == uint32_t(n) ? 0 : 1;
                };
                int missing = 0;                 // two bits a tile of the ring, the oldest first
                int page0 = 0, page1 = 0;        // of the tile to be staged next
                auto next_pages = [&](int t) {
                    page0 = page_of(2 * t);
                    page1 = page_of(2 * t + 1);
                };
                auto stage_tile = [&](int t, int slot) {
                    const uint32_t to = ring_lds + uint32_t(slot) * ring::TILE;
                    const int m0 = stage(to, 2 * t, page0);
                    return m0 | stage(to + S.bytes(), 2 * t + 1, page1) << 1;
                };
                if (w0 < w1) {
                    next_pages(w0);
#pragma unroll
                    for (int i = 0; i < ring::DEPTH; ++i)
                        if (w0 + i < w1) {
                            missing |= stage_tile(w0 + i, i) << (2 * i);
                            next_pages(w0 + i + 1);
                        }
                }
                int slot = 0;
                for (int t = w0; t < w1; ++t) {
                    if (t + ring::DEPTH <= w1)
                        dma_wait<ring::COPIES *(ring::DEPTH - 1)>();
                    else
                        dma_wait<0>();
                    Raw<N> x[2];
                    x[0].load(own + slot * ring::TILE, lane);
                    x[1].load(own + slot * ring::TILE + S.bytes(), lane);
                    float4v sc[R][2] = {};
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            const Vec<T> k = key_operand<T, N>(x[s], j);
#pragma unroll
                            for (int r = 0; r < R; ++r)
                                sc[r][s] = product<T>(k, q[r][j], sc[r][s]);
                        }
                        __builtin_amdgcn_sched_barrier(0);      // 16 registers of keys, not 32
                    }
                    // the slot is filled again once it has been read; a wait that the compiler
                    // knows of, or it would wait for the page numbers too before it uses x
                    asm volatile("" ::: "memory");
                    __builtin_amdgcn_s_waitcnt(kWaitLds);
                    asm volatile("" ::: "memory");
                    const int gone = missing & 3;
                    missing >>= 2;
                    if (t + ring::DEPTH < w1) {
                        missing |= stage_tile(t + ring::DEPTH, slot) << (2 * (ring::DEPTH - 1));
                        next_pages(t + ring::DEPTH + 1);
                    }
                    slot = slot + 1 == ring::DEPTH ? 0 : slot + 1;

                    if (t * kTile + kTile - 1 > all_see || gone) {
                        asm volatile("");        // a branch, not selects in every round
                        const int tok = t * kTile + grp * 4;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            // tokens that do not exist: finite values, whatever bytes there are
                            const int left =
                                gone >> s & 1 ? 0 : clamp_int(pc.lk - (tok + 16 * s), 0, 4);
                            const uint32_t keep = left == 0 ? 0u : 0xffffffffu >> (32 - 8 * left);
#pragma unroll
                            for (int b = 0; b < N; ++b)
                                x[s].ve.w[b] = (x[s].ve.w[b] & keep) | (0x7f7f7f7fu & ~keep);
#pragma unroll
                            for (int r = 0; r < R; ++r)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (tok + 16 * s + e > last[r] || (gone >> s & 1))
                                        sc[r][s][e] = -INFINITY;
                        }
                    }
                    Parts<T> p[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float4v &s0 = sc[r][0], &s1 = sc[r][1];
                        const float top = max_groups(
                            fmaxf(fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s0[2], s0[3])),
                                  fmaxf(fmaxf(s1[0], s1[1]), fmaxf(s1[2], s1[3]))));
                        if (__ballot(top > st[r].m + margin))
                            st[r].raise(top, c);
                        const float off = st[r].m == -INFINITY
                                              ? 0.0f
                                              : sizeof(T) == 4
                                                    ? st[r].m
                                                    : fmaf(st[r].m, c, float(-kLift<T>));
                        float e8[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float v = sc[r][e >> 2][e & 3];
                            e8[e] = __builtin_amdgcn_exp2f(sizeof(T) == 4 ? (v - off) * c
                                                                          : fmaf(v, c, -off));
                        }
                        st[r].l += ((e8[0] + e8[1]) + (e8[2] + e8[3])) +
                                   ((e8[4] + e8[5]) + (e8[6] + e8[7]));
                        p[r].set(e8);
                    }
#pragma unroll
                    for (int b = 0; b < N; ++b) {
                        Vec<T> even, odd;
                        value_operands<T, N>(x[0], x[1], b, even, odd);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            st[r].o[2 * b] = product<T>(even, p[r], st[r].o[2 * b]);
                            st[r].o[2 * b + 1] = product<T>(odd, p[r], st[r].o[2 * b + 1]);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                if (!alone) {
                    __syncthreads();             // the rings become the waves' way to join
                    join_waves<R, 2 * N>(st, lds, c, wave, lane);
                }
                if (alone || wave == 0) {
                    if (n0 == 0 && n1 == un.keys) {
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            finish<T, 2 * N>(a, st[r], token[r], head[r], 0, grp, live[r]);
                    } else {
                        float *slot = a.partial + (int64_t(blockIdx.x) * 2 + (n0 == 0 ? 1 : 0)) *
                                                      (R * part_floats<N>());
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            put_state(slot + r * part_floats<N>(), st[r], lane);
                        if (n0 == 0 && lane == 0)
                            *join = Join{pc.q0, pc.lq, kv_head, tile,
                                         share.owner(i_begin + un.keys - 1), {}};
                    }
                }
            }
        }
        base += __builtin_amdgcn_readlane(chunk.upto, 63);
    }
}

// One workgroup per (workgroup of the first kernel, row tile and block of channels): joins
// the parts of the item that began there.  Its waves take every fourth part.
template <typename T, int N, int R>
__global__ __launch_bounds__(256) void cache_join_kernel(CacheArgs a)
{
    __shared__ __align__(16) float lds[2 * part_floats<1>()];
    const Join j = reinterpret_cast<const Join *>(a.joins)[blockIdx.x];
    if (j.last < 0)
        return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int r = int(blockIdx.y) / N, b = int(blockIdx.y) % N;
    const float c = a.scale * kLog2e;
    const int first = int(blockIdx.x), end = min(j.last, a.workers - 1);

    State<2> st[1];
    st[0].init();
    for (int i = first + wave; i <= end; i += kWaves) {
        const float *p = a.partial + ((int64_t(i) * 2 + (i == first ? 1 : 0)) * R + r) *
                                         part_floats<N>();
        State<2> x;
#pragma unroll
        for (int o = 0; o < 2; ++o)
            x.o[o] = reinterpret_cast<const float4v *>(p)[(2 * b + o) * 64 + lane];
        x.m = p[2 * N * 256 + lane];
        x.l = p[2 * N * 256 + 64 + lane];
        st[0].merge(x, c);
    }
    join_waves<1, 2>(st, lds, c, wave, lane);
    if (wave == 0) {
        const int shared = a.q_heads / a.k_heads;
        const uint32_t packed = (uint32_t(j.tile) * R + r) * 16 + (lane & 15);
        const int row = int(packed / uint32_t(shared));
        finish<T, 2>(a, st[0], j.q0 + row, j.head * shared + int(packed % uint32_t(shared)), b,
                     lane >> 4, row < j.lq);
    }
}

// Row tiles of a wave: as many as an average sequence has rows for, up to four.
int row_tiles(const CacheArgs &a)
{
    const double rows = a.batch ? double(a.tokens) / a.batch * (a.q_heads / a.k_heads) : 0;
    return rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
}

size_t part_bytes(const CacheArgs &a)
{
    return size_t(row_tiles(a)) * (8 * cache_blocks(a.dim) + 2) * 64 * sizeof(float);
}

template <typename T, int N, int R> hipError_t launch(const CacheArgs &a, hipStream_t s)
{
    const int64_t row_bytes = int64_t(a.tokens) * a.q_heads * a.dim * int64_t(sizeof(T));
    const int fills = a.fill ? fill_blocks(row_bytes) : 0;
    cache_attend_kernel<T, N, R><<<uint32_t(a.workers + fills), 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.workers == 0)
        return e;
    cache_join_kernel<T, N, R><<<dim3(uint32_t(a.workers), R * N), 256, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, int N> hipError_t launch_rows(const CacheArgs &a, hipStream_t s)
{
    switch (row_tiles(a)) {
    case 1:
        return launch<T, N, 1>(a, s);
    case 2:
        return launch<T, N, 2>(a, s);
    default:
        return launch<T, N, 4>(a, s);
    }
}

template <typename T> hipError_t launch_blocks(const CacheArgs &a, hipStream_t s)
{
    switch (cache_blocks(a.dim)) {
    case 1:
        return launch_rows<T, 1>(a, s);
    case 2:
        return launch_rows<T, 2>(a, s);
    case 3:
        return launch_rows<T, 3>(a, s);
    default:
        return launch_rows<T, 4>(a, s);
    }
}

}  // namespace

int cache_attend_workers(mdcn_dtype dtype, const CacheArgs &a)
{
    const int tiles = row_tiles(a);
    return 256 * (tiles > 1 ? 2 : dtype == MDCN_F32 ? 3 : 4);
}

size_t cache_attend_bytes(mdcn_dtype dtype, const CacheArgs &a)
{
    return size_t(cache_attend_workers(dtype, a)) * (2 * part_bytes(a) + sizeof(Join));
}

hipError_t launch_cache_attend(mdcn_dtype dtype, CacheArgs a, void *workspace, hipStream_t s)
{
    a.workers = a.batch ? cache_attend_workers(dtype, a) : 0;    // none: rows to fill only
    a.joins = static_cast<int4 *>(workspace);
    a.partial = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                          size_t(a.workers) * sizeof(Join));
    // units of a batch, at most (row tiles) x (key heads) x (units of all tokens)
    const double rows = double(a.tokens) * (a.q_heads / a.k_heads);
    const double tiles = rows / (16 * row_tiles(a)) + a.batch;
    const double keys = double(a.width) * (1 << a.page_shift) / kTile + kItemCost;
    a.unit_shift = 0;
    while (tiles * a.k_heads * (keys / (1 << a.unit_shift) + 1) > 1e9 && a.unit_shift < 20)
        ++a.unit_shift;
    switch (dtype) {
    case MDCN_F32:
        return launch_blocks<float>(a, s);
    case MDCN_F16:
        return launch_blocks<half_t>(a, s);
    default:
        return launch_blocks<bf16_t>(a, s);
    }
}

}  // namespace mdcn
