// attention_common.h -- pieces shared by the attention kernels (gfx950).
//
// Everything is built from two products on 32x32 MFMA tiles, with rows
// staged in LDS on one side and operands in registers on the other:
//   mm_rows: S[i][c] = sum_d tile[i][d] * frag[c][d]   (c = lane % 32)
//   mm_cols: acc[d][c] += sum_i tile[i][d] * p[i][c]
// An accumulator of a 32x32 tile holds column lane % 32 in every register and
// row 8*(r/4) + 4*(lane/32) + r%4 in register r.  So the result of mm_rows
// has one query (or key) per lane: a softmax row needs one exchange with lane
// ^ 32, and its registers, rounded, are the operand p of mm_cols without any
// exchange, because the order of an instruction's k index is free as long as
// both operands share it: half h of the wave takes rows 8*j + 4*h + (0..3).
// mm_cols needs the staged rows transposed: 16-bit types read them with the
// transposing LDS read (4 rows x 16 columns per 16 lanes), fp32 reads single
// values, which needs no transposition.
//
// LDS tiles: a row of DP values padded to a power of two of bytes (64..512);
// its 16-byte chunk c sits at c ^ swz(row), swz chosen so that both kinds of
// read (one chunk of 16 rows; four chunks of 4 rows) touch every bank once.
// Tiles are written by buffer loads straight to LDS; rows past the end
// and channels past dim are out of the buffer's range and arrive as zeros.
#pragma once

#include "attention.h"
#include "device_common.h"
#include "mfma_common.h"

namespace mdcn {

constexpr float kLog2e = 1.4426950408889634f;

typedef int v4i __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) short4v lds_short4;

// Layout of one staged tile row.
template <typename T, int DP> struct Row {
    static constexpr int BYTES = DP * int(sizeof(T));
    static constexpr int PITCH = BYTES <= 64 ? 64 : BYTES <= 128 ? 128 : BYTES <= 256 ? 256 : 512;
    static constexpr int CHUNKS = PITCH / 16;
    static constexpr int STEPS = BYTES / 32;     // mm_rows steps: two chunks each
    static constexpr int BLOCKS = DP / 32;       // mm_cols: 32-channel blocks
    // mm_cols steps: rows per Mma::step (16-bit: 16, fp32: 8)
    static constexpr int KROWS = sizeof(T) == 2 ? 16 : 8;

    static __device__ __forceinline__ int swz(int row)
    {
        if (CHUNKS == 4)
            return (row >> 2) & 3;
        if (CHUNKS == 8)
            return ((row >> 1) & 1) << 2 | ((row >> 2) & 3);
        if (sizeof(T) == 2)
            return (row & 3) << 2 | ((row >> 2) & 3);
        return ((row >> 2) & 1) << 3 | ((row >> 3) & 1) << 2 | (row & 3);
    }
};

// A row as mm_rows' register operand; the accumulators of mm_cols.
template <typename T, int DP> using Frag = uint4[Row<T, DP>::STEPS];
template <typename T, int DP> using Acc = float16v[Row<T, DP>::BLOCKS];

__device__ __forceinline__ uint32_t lds_address(const void *p)
{
    return uint32_t(reinterpret_cast<uintptr_t>((const lds_void *)p));
}

// 16 bytes per lane from rsrc + voff into LDS at lds + 16 * lane.  The
// compiler does not see the write; callers wait (dma_wait) and pass a barrier
// before any wave reads the data.
__device__ __forceinline__ void dma_row16(uint32_t lds, v4i rsrc, uint32_t voff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc)
                 : "memory");
}

// The same with 4 bytes per lane, to lds + 4 * lane.
__device__ __forceinline__ void dma_row4(uint32_t lds, v4i rsrc, uint32_t voff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc)
                 : "memory");
}

template <int N> __device__ __forceinline__ void dma_wait()
{
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

__device__ __forceinline__ v4i row_resource(const char *base, uint32_t bytes)
{
    const uint64_t v = reinterpret_cast<uint64_t>(base);
    v4i r;
    r.x = __builtin_amdgcn_readfirstlane(int(uint32_t(v)));
    r.y = __builtin_amdgcn_readfirstlane(int(uint32_t(v >> 32)) & 0xffff);
    r.z = __builtin_amdgcn_readfirstlane(int(bytes));
    r.w = 0x00020000;
    return r;
}

// Stages tiles of ROWS rows of two tensors (keys and values; queries and
// gradients) with WAVES waves: each wave's share of the copies, consecutive
// kilobytes of a tile.  The offsets of the first tensor's copies are kept;
// those of the second, whose tokens may lie at another stride, follow by one
// addition (rows past the end and channels past dim keep offsets out of range).
template <typename T, int DP, int ROWS, int WAVES> struct Stager {
    using R = Row<T, DP>;
    static constexpr int COPIES = ROWS * R::CHUNKS / 64 / WAVES;
    static constexpr int STEP = 64 / R::CHUNKS;      // rows of one copy
    static_assert(COPIES * 64 * WAVES == ROWS * R::CHUNKS, "copies fill the tile");
    uint32_t voff[COPIES];
    uint32_t shift0;                                 // of the second tensor's first row
    uint32_t stride[2], width;
    uint32_t slot;

    __device__ __forceinline__ void init(int64_t stride_a, int64_t stride_b, int dim, int wave,
                                         int lane)
    {
        stride[0] = uint32_t(stride_a) * uint32_t(sizeof(T));
        stride[1] = uint32_t(stride_b) * uint32_t(sizeof(T));
        width = uint32_t(dim) * uint32_t(sizeof(T));
        slot = uint32_t(wave * COPIES * 1024);
        const int row0 = wave * COPIES * STEP + lane / R::CHUNKS;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const int row = row0 + i * STEP;
            const uint32_t byte = uint32_t((lane % R::CHUNKS) ^ R::swz(row)) * 16;
            voff[i] = byte < width ? uint32_t(row) * stride[0] + byte : kOutside;
        }
        shift0 = uint32_t(row0) * (stride[1] - stride[0]);
    }

    // Rows [0, left) of the tile at `base` (ROWS at most) of tensor `which` to LDS at `lds`.
    template <int WHICH>
    __device__ __forceinline__ void load(uint32_t lds, const char *base, int left) const
    {
        const int n = left < ROWS ? left : ROWS;
        const v4i r = row_resource(base, n > 0 ? uint32_t(n - 1) * stride[WHICH] + width : 0);
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const uint32_t off =
                WHICH == 0 ? voff[i]
                           : voff[i] + shift0 + uint32_t(i * STEP) * (stride[1] - stride[0]);
            dma_row16(__builtin_amdgcn_readfirstlane(lds + slot + i * 1024), r, off);
        }
    }

    // Offset of channels past dim: out of range whatever shift is added.  A tile has at
    // most 256 rows of 2^23 bytes (fp32: 64 of 2^24), so a row's offset and the size of a
    // shift are at most 255 * 2^23 < 2^31: sums of this and a shift stay below 2^32 and
    // at least 2^23 above the second tensor's rows.
    static constexpr uint32_t kOutside = 0x80000000u;
};

// The register operand of mm_rows: row `src` (dim values, 16-byte aligned),
// zeros past dim or when src is null.
template <typename T, int DP>
__device__ __forceinline__ void load_frag(Frag<T, DP> &f, const T *src, int dim,
                                          int half)
{
#pragma unroll
    for (int k = 0; k < Row<T, DP>::STEPS; ++k) {
        const int d = (2 * k + half) * int(16 / sizeof(T));
        f[k] = make_uint4(0, 0, 0, 0);
        if (src && d < dim)
            f[k] = *reinterpret_cast<const uint4 *>(src + d);
    }
}

// Waits for the loads of `f` here.  Without it the compiler waits at the first
// use, inside the loop over the tiles, in every round -- and as it counts all
// loads in order, for the copies of the next tile too.
template <typename T, int DP> __device__ __forceinline__ void settle(Frag<T, DP> &f)
{
#pragma unroll
    for (int k = 0; k < Row<T, DP>::STEPS; ++k)
        asm volatile("" : "+v"(f[k].x), "+v"(f[k].y), "+v"(f[k].z), "+v"(f[k].w));
}

__device__ __forceinline__ void settle(float &v) { asm volatile("" : "+v"(v)); }

// Issued reads must not sink to their uses: the scheduler would keep two in
// flight, and every pair of MFMAs would wait for LDS.
__device__ __forceinline__ void reads_first() { __builtin_amdgcn_sched_barrier(0); }

// The staged operand of mm_rows: 32 rows at `tile`.
template <typename T, int DP>
__device__ __forceinline__ void load_rows(Frag<T, DP> &a, const char *tile, int lane)
{
    using R = Row<T, DP>;
    const int row = lane & 31, half = lane >> 5, sw = R::swz(row);
    const char *p = tile + row * R::PITCH;
#pragma unroll
    for (int k = 0; k < R::STEPS; ++k)
        a[k] = *reinterpret_cast<const uint4 *>(p + ((2 * k + half) ^ sw) * 16);
}

// Read k of load_rows alone.
template <typename T, int DP>
__device__ __forceinline__ uint4 row_frag(const char *tile, int k, int lane)
{
    using R = Row<T, DP>;
    const int row = lane & 31;
    return *reinterpret_cast<const uint4 *>(tile + row * R::PITCH +
                                            ((2 * k + (lane >> 5)) ^ R::swz(row)) * 16);
}

template <typename T, int DP>
__device__ __forceinline__ float16v mm_rows(const Frag<T, DP> &a, const Frag<T, DP> &f)
{
    float16v s = {};
#pragma unroll
    for (int k = 0; k < Row<T, DP>::STEPS; ++k)
        s = Mma<T>::step(a[k], f[k], s);
    return s;
}

template <typename T, int DP>
__device__ __forceinline__ float16v mm_rows(const char *tile, const Frag<T, DP> &f, int lane)
{
    Frag<T, DP> a;
    load_rows<T, DP>(a, tile, lane);
    return mm_rows<T, DP>(a, f);
}

// Registers r0.. of a 32x32 accumulator rounded to T (to nearest even) as the
// operand of mm_cols.  Probabilities and their gradients enter the second
// product in the inputs' type, as the matrix instructions need it; sums stay in fp32.
template <typename T>
__device__ __forceinline__ uint4 pack_p(const float16v &p, int r0)
{
    uint4 o;
    if constexpr (sizeof(T) == 4) {
        o = make_uint4(__float_as_uint(p[r0]), __float_as_uint(p[r0 + 1]),
                       __float_as_uint(p[r0 + 2]), __float_as_uint(p[r0 + 3]));
    } else {
        typedef float f2 __attribute__((ext_vector_type(2)));
        typedef T t2 __attribute__((ext_vector_type(2)));
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const t2 v = __builtin_convertvector((f2){p[r0 + 2 * i], p[r0 + 2 * i + 1]}, t2);
            __builtin_memcpy(&w[i], &v, 4);
        }
        o = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return o;
}

// Transposed operand of mm_cols step `step`, channel block `blk`.
template <typename T, int DP>
__device__ __forceinline__ uint4 col_frag(const char *tile, int step, int blk, int lane)
{
    using R = Row<T, DP>;
    const int half = lane >> 5;
    uint4 o;
    if constexpr (sizeof(T) == 2) {
        const int l = lane & 15;
        const int chunk = blk * 4 + ((lane >> 4) & 1) * 2 + ((l & 3) >> 1);
        uint2 w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = step * 16 + j * 8 + half * 4 + (l >> 2);
            const char *p = tile + row * R::PITCH + (chunk ^ R::swz(row)) * 16 + (l & 1) * 8;
            const short4v v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)p);
            __builtin_memcpy(&w[j], &v, 8);
        }
        o = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
    } else {
        const int d = blk * 32 + (lane & 31);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = step * 8 + half * 4 + j;
            w[j] = *reinterpret_cast<const uint32_t *>(
                tile + row * R::PITCH + ((d >> 2) ^ R::swz(row)) * 16 + (d & 3) * 4);
        }
        o = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return o;
}

// The staged operand of mm_cols: 32 rows at `tile`, every step and block.
template <typename T, int DP> struct Cols {
    using R = Row<T, DP>;
    static constexpr int STEPS = 32 / R::KROWS;
    uint4 f[STEPS][R::BLOCKS];

    __device__ __forceinline__ void load(const char *tile, int lane)
    {
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int d = 0; d < R::BLOCKS; ++d)
                f[s][d] = col_frag<T, DP>(tile, s, d, lane);
    }
};

template <typename T, int DP>
__device__ __forceinline__ void mm_cols(Acc<T, DP> &acc, const Cols<T, DP> &t, const float16v &p)
{
    using R = Row<T, DP>;
#pragma unroll
    for (int s = 0; s < Cols<T, DP>::STEPS; ++s) {
        const uint4 b = pack_p<T>(p, s * R::KROWS / 2);
#pragma unroll
        for (int d = 0; d < R::BLOCKS; ++d)
            acc[d] = Mma<T>::step(t.f[s][d], b, acc[d]);
    }
}

template <typename T, int DP>
__device__ __forceinline__ void mm_cols(Acc<T, DP> &acc, const char *tile, const float16v &p,
                                        int lane)
{
    using R = Row<T, DP>;
#pragma unroll
    for (int s = 0; s < 32 / R::KROWS; ++s) {
        const uint4 b = pack_p<T>(p, s * R::KROWS / 2);
#pragma unroll
        for (int d = 0; d < R::BLOCKS; ++d) {
            acc[d] = Mma<T>::step(col_frag<T, DP>(tile, s, d, lane), b, acc[d]);
        }
    }
}

// Row of register r of an accumulator.
__device__ __forceinline__ int acc_row(int r, int half) { return 8 * (r >> 2) + 4 * half + (r & 3); }

// The value of lane ^ 32.
__device__ __forceinline__ float swap_halves(float v)
{
    const uint32_t u = __float_as_uint(v);
    const auto w = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __uint_as_float((threadIdx.x & 32) ? w[0] : w[1]);
}

// The larger of the two halves' values.
__device__ __forceinline__ float max_halves(float v)
{
    const uint32_t u = __float_as_uint(v);
    const auto w = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
}

// acc[d][c] * factor to row `dst` of lane c (null: nothing is stored).
template <typename T, int DP>
__device__ __forceinline__ void store_cols(T *dst, const Acc<T, DP> &acc,
                                           float factor, int dim, int half)
{
    if (!dst)
        return;
#pragma unroll
    for (int b = 0; b < Row<T, DP>::BLOCKS; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int d = b * 32 + 8 * g + 4 * half;
            if (d < dim) {
                struct alignas(4 * sizeof(T)) {
                    T e[4];
                } v;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v.e[j] = from_f32<T>(acc[b][4 * g + j] * factor);
                __builtin_memcpy(__builtin_assume_aligned(dst + d, 4 * sizeof(T)), &v, sizeof(v));
            }
        }
}

// Keys of a wave's part of a tile of K or V: four parts of 64 rows of 256 bytes, with
// two stages of both, would not fit the LDS.
template <typename T, int DP, int KW> constexpr int tile_keys()
{
    return sizeof(T) == 2 && (KW < 4 || Row<T, DP>::PITCH <= 128) ? 64 : 32;
}

// Waves a SIMD that a tile kernel's registers are to leave room for: two workgroups
// of four waves, unless the LDS of one (two stages of K and V) leaves no room
// or 256 registers do not hold a wave's sums and operands.
template <typename T, int DP, int KW> constexpr int waves_per_simd()
{
    constexpr int lds = 4 * tile_keys<T, DP, KW>() * KW * Row<T, DP>::PITCH;
    return lds > 80 * 1024 || (sizeof(T) == 4 && DP > 96) ? 1 : 2;
}

// ---- softmax ---------------------------------------------------------------

// The running maximum is raised only when a score exceeds it by more than
// this many powers of two: e^s stays below 2^8 relative to the maximum, which
// costs no accuracy in fp32 sums and saves most rescalings.
constexpr float kRaise = 8.0f;

// The same in raw scores.  Finite, so that the first score raises the maximum from -infinity
// however small the scale is.
__device__ __forceinline__ float raise_margin(float c) { return fminf(kRaise / c, 3.0e38f); }

// fp16: exponentials are 2^7 e^(scale (s - m)), up to 2^15, where they are rounded for the
// product with v, so that weights down to 2^-21 are normal numbers there: thousands of
// keys of little weight may outweigh one whose value is small.  The sums have the factor
// too, so only lse has to know of it.
template <typename T> inline constexpr int kLift = 0;
template <> inline constexpr int kLift<half_t> = 7;

// log(sum of exponentials) of a row
template <typename T> __device__ __forceinline__ float row_lse(float m, float l, float scale)
{
    return fmaf(m, scale, logf(kLift<T> ? l * (1.0f / (1 << kLift<T>)) : l));
}

// Softmax state of one query row (both halves of the wave hold the same
// maximum; the sums are those of the half's own keys).
template <typename T, int DP> struct Softmax {
    Acc<T, DP> o;
    float m, l;

    __device__ __forceinline__ void init()
    {
#pragma unroll
        for (int b = 0; b < Row<T, DP>::BLOCKS; ++b)
            o[b] = (float16v){};
        m = -INFINITY;
        l = 0.0f;
    }

    // The row's largest of NS blocks of 32 scores (raw, -infinity where masked).
    template <int NS> static __device__ __forceinline__ float top_of(const float16v (&s)[NS])
    {
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            top[i] = fmaxf(s[0][i], s[0][i + 4]);
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int r = n == 0 ? 8 : 0; r < 16; r += 8)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top[i] = fmaxf(fmaxf(top[i], s[n][r + i]), s[n][r + i + 4]);
        return max_halves(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
    }

    // Raises the maximum if `top` needs it; returns what exps takes off the scores.
    __device__ __forceinline__ float raise(float top, float c, float margin)
    {
        if (__ballot(top > m + margin)) {
            const float up = fmaxf(top, m);
            const float f = up == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m - up) * c);
#pragma unroll
            for (int b = 0; b < Row<T, DP>::BLOCKS; ++b)
                o[b] *= f;
            l *= f;
            m = up;
        }
        return m == -INFINITY ? 0.0f : sizeof(T) == 4 ? m : fmaf(m, c, float(-kLift<T>));
    }

    // Turns scores into e^(scale (s - m)) and adds them up.  16-bit types: one fma,
    // m c taken off, which leaves 2^-24 |m c| at s = m; fp32: the difference
    // first, so that a row of one key has p = 1 exactly.
    template <int NS> __device__ __forceinline__ void exps(float16v (&s)[NS], float c, float off)
    {
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[n][r] = __builtin_amdgcn_exp2f(sizeof(T) == 4 ? (s[n][r] - off) * c
                                                                : fmaf(s[n][r], c, -off));
                sum[r & 3] += s[n][r];
            }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }

    template <int NS> __device__ __forceinline__ void step(float16v (&s)[NS], float c, float margin)
    {
        exps<NS>(s, c, raise(top_of<NS>(s), c, margin));
    }
};

// What a row's accumulators are made of: sum over its keys of weight(s, v row) *
// the row of k or v, for the forward and for the gradient of the queries.
struct RowTerms {
    int last;                 // last visible key
    float m;                  // forward: maximum; backward: lse in powers of two
    float delta;              // backward only
    float c;
};

template <typename T, int DP>
__device__ __forceinline__ float half_dot(const uint4 *f, const T *row, int dim, int half)
{
    constexpr int E = 16 / sizeof(T);
    float s = 0.0f;
    for (int i = 0; i < Row<T, DP>::STEPS; ++i) {
        const int d = (2 * i + half) * E;
        if (d >= dim)
            break;
        Vec16<T> a;
        a.raw = f[i];
        const Vec16<T> b = load16(row + d);
        for (int e = 0; e < E; ++e)
            s = fmaf(to_f32(a.e[e]), to_f32(b.e[e]), s);
    }
    return s + swap_halves(s);
}

// Recomputes the accumulators of keys [begin, end), of every KT keys the first
// KB, one key at a time, each lane for its own row: hidden keys are never
// touched, whatever they hold.  `g` is null in the forward.
template <typename T, int DP, int KB, int KT>
__device__ __attribute__((noinline)) void recompute(float16v *o, const uint4 *q, const uint4 *g,
                                                    const char *k, const char *v, uint32_t k_stride,
                                                    uint32_t v_stride, int begin, int end,
                                                    const RowTerms *t, int dim, int half)
{
    using R = Row<T, DP>;
    for (int b = 0; b < R::BLOCKS; ++b)
        o[b] = (float16v){};
    for (int j = begin; j < end; ++j) {
        if (KB < KT && (j - begin) % KT >= KB)
            continue;
        const T *kr = reinterpret_cast<const T *>(k + uint64_t(j) * k_stride);
        const T *vr = reinterpret_cast<const T *>(v + uint64_t(j) * v_stride);
        const float s = half_dot<T, DP>(q, kr, dim, half);
        const float dp = g ? half_dot<T, DP>(g, vr, dim, half) : 0.0f;
        if (j > t->last)
            continue;
        float w = exp2f(fmaf(s, t->c, g ? -t->m : fmaf(-t->m, t->c, float(kLift<T>))));
        if (g)
            w *= dp - t->delta;
        const T *row = g ? kr : vr;
        for (int b = 0; b < R::BLOCKS; ++b)
            for (int r = 0; r < 16; ++r) {
                const int d = b * 32 + acc_row(r, half);
                if (d < dim)
                    o[b][r] = fmaf(w, to_f32(row[d]), o[b][r]);
            }
    }
}

// After the tiles [begin, end) that a causal mask cuts, while the accumulators
// hold nothing else: where they are not finite, recomputes them without the hidden keys.
template <typename T, int DP, int KB, int KT, bool BACKWARD>
__device__ __forceinline__ void repair_hidden(Acc<T, DP> &acc, const Frag<T, DP> &qf,
                                              const Frag<T, DP> &gf, const char *k, const char *v,
                                              uint32_t k_stride, uint32_t v_stride, int begin,
                                              int end, const RowTerms &terms, int dim, int half)
{
    using R = Row<T, DP>;
    float bad = 0.0f;
#pragma unroll
    for (int i = 0; i < R::BLOCKS; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            bad += acc[i][r] * 0.0f;
    if (__any(bad != 0.0f)) {
        Acc<T, DP> o;                                    // copies: only they are
        Frag<T, DP> f, g;                                // addressed in memory
        const RowTerms t = terms;
#pragma unroll
        for (int i = 0; i < R::STEPS; ++i) {
            f[i] = qf[i];
            if (BACKWARD)
                g[i] = gf[i];
        }
        recompute<T, DP, KB, KT>(o, f, BACKWARD ? g : nullptr, k, v, k_stride, v_stride, begin, end,
                                 &t, dim, half);
#pragma unroll
        for (int i = 0; i < R::BLOCKS; ++i) {
            acc[i] = o[i];
            asm volatile("" : "+v"(acc[i]));             // as settle
        }
    }
}

// ---- packed sequences ------------------------------------------------------

struct Span {
    int q0, lq, k0, lk;       // first query and key row, their numbers
    int k_all;                // keys of the sequence, used or not
};

__device__ __forceinline__ int clamp_int(int v, int lo, int hi)
{
    return v < lo ? lo : v > hi ? hi : v;
}

// Rows of sequence b.  Offsets are clamped to the tensors, so that no offsets
// whatever lead to an access outside them.
__device__ __forceinline__ Span span_of(const AttendArgs &a, int b)
{
    Span s;
    s.q0 = clamp_int(a.cu_q[b], 0, a.q_tokens);
    s.lq = clamp_int(a.cu_q[b + 1], s.q0, a.q_tokens) - s.q0;
    s.k0 = clamp_int(a.cu_k[b], 0, a.k_tokens);
    s.k_all = clamp_int(a.cu_k[b + 1], s.k0, a.k_tokens) - s.k0;
    s.lk = a.used_k ? clamp_int(a.used_k[b], 0, s.k_all) : s.k_all;
    return s;
}

// The span that lane l holds, for all lanes.
__device__ __forceinline__ Span span_in(const Span &mine, int l)
{
    Span s;
    s.q0 = __builtin_amdgcn_readlane(mine.q0, l);
    s.lq = __builtin_amdgcn_readlane(mine.lq, l);
    s.k0 = __builtin_amdgcn_readlane(mine.k0, l);
    s.lk = __builtin_amdgcn_readlane(mine.lk, l);
    s.k_all = __builtin_amdgcn_readlane(mine.k_all, l);
    return s;
}

template <int CTRL, int ROWS> __device__ __forceinline__ int lane_moved(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}

// Sums over lanes 0..lane of the wave: within rows of 16, then across them.
__device__ __forceinline__ int wave_scan(int v)
{
    v += lane_moved<0x111, 0xf>(v);
    v += lane_moved<0x112, 0xf>(v);
    v += lane_moved<0x114, 0xf>(v);
    v += lane_moved<0x118, 0xf>(v);
    v += lane_moved<0x142, 0xa>(v);                  // lane 15 to lanes 16.., 47 to 48..
    v += lane_moved<0x143, 0xc>(v);                  // lane 31 to lanes 32..
    return v;
}

__device__ __forceinline__ int wave_sum(int v)
{
    return __builtin_amdgcn_readlane(wave_scan(v), 63);
}

template <typename T>
__device__ __forceinline__ const char *row_ptr(const Heads &h, int64_t token, int head)
{
    return reinterpret_cast<const char *>(static_cast<const T *>(h.data) + token * h.token_stride +
                                          head * h.head_stride);
}

// Calls f(token, i), i in [0, each), for the tokens before the first sequence and after
// the last (offsets `cu`), neighbouring i in neighbouring threads of `parts` workgroups.
template <class F>
__device__ __forceinline__ void outside_rows(const int32_t *cu, int batch, int tokens, int each,
                                             int part, int parts, F &&f)
{
    const int begin = clamp_int(cu[0], 0, tokens);
    const int end = clamp_int(cu[batch], begin, tokens);
    const int64_t all = int64_t(begin + tokens - end) * each;
    for (int64_t e = int64_t(part) * blockDim.x + threadIdx.x; e < all;
         e += int64_t(parts) * blockDim.x) {
        const int r = int(e / each);
        f(r < begin ? r : end + r - begin, int(e % each));
    }
}

// Zeros in the rows of `h` outside every sequence.
template <typename T>
__device__ __forceinline__ void zero_outside(const Heads &h, const int32_t *cu, int batch, int tokens,
                                             int heads, int dim, int part, int parts)
{
    const int vecs = dim / int(16 / sizeof(T));
    outside_rows(cu, batch, tokens, heads * vecs, part, parts, [&](int token, int i) {
        char *row = const_cast<char *>(row_ptr<T>(h, token, i / vecs));
        *reinterpret_cast<uint4 *>(row + i % vecs * 16) = make_uint4(0, 0, 0, 0);
    });
}

// Workgroups that fill beyond those of the tiles, for rows of `bytes` bytes in all.  They
// are there in every call, as only the GPU knows the offsets, and cost next to nothing
// where nothing is outside.
inline int fill_blocks(int64_t bytes)
{
    const int64_t n = bytes >> 18;
    return n < 1 ? 1 : n > 64 ? 64 : int(n);
}

// The sequence and its tile that hold tile t of the batch, where count(span)
// is the number of a sequence's tiles; false past the last tile.  Every lane
// of the wave must call it.
//
// Each sequence's last tiles come first.  `by_size` (up to 64 sequences): those
// of all sequences in the order of their index, the highest first, which is the
// order of their work under a causal mask: the longest start first (dk and dv of
// sequences of 2048 to 1 tokens 100 -> 90 us).
template <class F>
__device__ __forceinline__ bool find_tile(const AttendArgs &a, int t, int lane, bool by_size,
                                          F &&count, Span &sp, int &tile)
{
    if (by_size && a.batch <= 64) {
        Span s = {};
        if (lane < a.batch)
            s = span_of(a, lane);
        const int n = count(s);
        if (t >= wave_sum(n))
            return false;
        // the level: tiles of index `level` and more number more than t
        int level = 0, past = 1;
        while (wave_sum(max(0, n - past)) > t)
            level = past, past *= 2;
        while (past - level > 1) {
            const int mid = (level + past) / 2;
            if (wave_sum(max(0, n - mid)) > t)
                level = mid;
            else
                past = mid;
        }
        const int rank = t - wave_sum(max(0, n - level - 1));
        const int upto = wave_scan(n > level ? 1 : 0);
        const int l = __builtin_ctzll(__ballot(upto == rank + 1 && n > level));
        sp = span_in(s, l);
        tile = level;
        return true;
    }
    int base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        Span s = {};
        if (b0 + lane < a.batch)
            s = span_of(a, b0 + lane);
        const int mine = count(s);
        const int upto = wave_scan(mine);
        const uint64_t past = __ballot(base + upto > t);
        if (past) {
            const int l = __builtin_ctzll(past);
            sp = span_in(s, l);
            tile = __builtin_amdgcn_readlane(base + upto, l) - 1 - t;
            return true;
        }
        base += __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

}  // namespace mdcn
