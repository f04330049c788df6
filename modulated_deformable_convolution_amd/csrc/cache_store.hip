// cache_store.hip -- keys and values rounded to 4 bits into the pages of a cache, and
// read back.
//
// A block of 32 channels x becomes s m 2^e with e the smallest exponent for which
// max|x| <= 7 * 2^e: nothing is off by more than half a step (7 lies half-way between 6, the
// largest magnitude, and where 8 would be).  e comes from the bits of the maximum: with
// max|x| = f * 2^k, 1 <= f < 2, e is k - 2 if f <= 1.75 and k - 1 otherwise, a carry out
// of the mantissa.  x * 2^-e is exact and the conversion rounds to nearest even, so the
// codes do not depend on the order of any operation.
//
// One lane takes 8 channels of one token's key and value (16 bytes in 16-bit types);
// the block's maximum comes from the 4 lanes beside it, the NaN flag from all lanes
// of the head.  Its 8 key codes are one dword of the strip, its 8 value codes four bytes.
// A few tokens are bound by the round trips to offsets, table and values (48 tokens of 8 heads
// of 128 in bf16 3.4 us), many by memory: 7144 tokens of 8 heads of 80 in fp32 14 us each way, at 3
// TB/s of what has to move.  A strip's 16 tokens are taken by several workgroups, on XCDs of
// their own, whose L2s write back and fetch parts of the same lines: for 5.9 MB of strips 13.5 MB are
// written and 27.5 MB read.  (Waves of four times as many rows took 15.5 us.)
#include "cache_common.h"

namespace mdcn {

namespace {

template <typename T> struct Eight {
    float v[8];

    __device__ __forceinline__ void load(const char *p)
    {
        struct alignas(16) {
            T e[8];
        } x;
        __builtin_memcpy(&x, __builtin_assume_aligned(p, 16), sizeof(x));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = to_f32(x.e[i]);
    }

    __device__ __forceinline__ void store(char *p) const
    {
        struct alignas(16) {
            T e[8];
        } x;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x.e[i] = from_f32<T>(v[i]);
        __builtin_memcpy(__builtin_assume_aligned(p, 16), &x, sizeof(x));
    }
};

// The values of the quad's other lanes: CTRL is a quad permutation.
template <int CTRL> __device__ __forceinline__ float quad(float v)
{
    return __uint_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, false));
}

// The exponent byte of a block and this lane's 8 codes, x[0] in the lowest bits.
template <typename T>
__device__ __forceinline__ uint32_t encode(const float (&x)[8], int &exponent)
{
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        top = fmaxf(top, fabsf(x[i]));
    top = fmaxf(top, quad<0xb1>(top));               // lanes 1 0 3 2
    top = fmaxf(top, quad<0x4e>(top));               // lanes 2 3 0 1
    const int e = int((__float_as_uint(top) + 0x1fffffu) >> 23) - 2;
    exponent = clamp_int(e, ExpRange<T>::lo, ExpRange<T>::hi);
    const float scale = __uint_as_float(uint32_t(exponent) << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
    return w;
}

// What one lane is to do: 8 channels (`part` 8 of the head) of one row (token, head).
template <int N> struct Task {
    static constexpr int LANES = 4 * N;              // of a row
    static constexpr int ROWS = 64 / LANES;          // of a wave
    int token, head, part;
    bool live;

    __device__ __forceinline__ Task(const CacheArgs &a, int lane)
    {
        const int r = lane / LANES;
        const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
        const int64_t row = (int64_t(blockIdx.x) * 4 + wave) * ROWS + r;
        live = r < ROWS && row < int64_t(a.tokens) * a.k_heads;
        token = live ? int(row / a.k_heads) : 0;
        head = live ? int(row - int64_t(token) * a.k_heads) : 0;
        part = lane - r * LANES;
    }

    // The token's place, found for the tokens of the wave one after the other.
    __device__ __forceinline__ Place find(const CacheArgs &a, int lane, bool &inside) const
    {
        const Finder f(a, lane);
        Place p = {nullptr, 0};
        inside = false;
        uint64_t todo = __ballot(live);
        while (todo) {
            const int t = __builtin_amdgcn_readlane(token, __builtin_ctzll(todo));
            int64_t at = 0;
            const int b = f.find(a, t, lane, at);
            if (b >= 0) {
                const Place q = place_of(a, b, at, Strip{N}.bytes());
                if (live && token == t) {
                    p = q;
                    inside = true;
                }
            }
            todo &= ~__ballot(token == t);
        }
        if (p.strip)
            p.strip += int64_t(head) * ((1 << a.page_shift) / kStripTokens) * Strip{N}.bytes();
        return p;
    }
};

template <typename T, int N> __global__ __launch_bounds__(256) void cache_store_kernel(CacheArgs a)
{
    constexpr Strip S{N};
    const int lane = threadIdx.x & 63;
    const Task<N> t(a, lane);
    const int ch = t.part * 8;
    Eight<T> k = {}, v = {};
    if (t.live && ch < a.dim) {                      // on their way while the place is found
        k.load(row_ptr<T>(a.k, t.token, t.head) + ch * sizeof(T));
        v.load(row_ptr<T>(a.v, t.token, t.head) + ch * sizeof(T));
    }
    bool inside;
    const Place p = t.find(a, lane, inside);
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        nan |= k.v[i] != k.v[i] || v.v[i] != v.v[i];
    const uint64_t bad = __ballot(nan);
    const int first = lane / Task<N>::LANES * Task<N>::LANES;
    const bool row_bad = bad >> first & (~0ull >> (64 - Task<N>::LANES));
    if (row_bad)
        k = v = {};
    int ke, ve;
    const uint32_t kw = encode<T>(k.v, ke), vw = encode<T>(v.v, ve);
    if (!p.strip)
        return;
    const int blk = t.part >> 2, g = t.part & 3;
    *reinterpret_cast<uint32_t *>(p.strip + ((g * 16 + p.token) * N + blk) * 4) = kw;
    char *vp = p.strip + S.values() + (((p.token >> 2) * 16 + g * 4) * N + blk) * 4 + (p.token & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        vp[i * N * 4] = char(vw >> (8 * i));
    if (g == 0) {
        p.strip[S.key_exps() + p.token * S.key_exp() + blk] = char(row_bad ? kNanExp : ke);
        p.strip[S.value_exps() + ((p.token >> 2) * N + blk) * 4 + (p.token & 3)] = char(ve);
    }
}

__device__ __forceinline__ void decode(float (&x)[8], uint32_t w, int exponent)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    const float scale = __uint_as_float(uint32_t(exponent) << 23);
    const f2 y[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3)};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = y[i / 2][i % 2];
}

template <typename T, int N> __global__ __launch_bounds__(256) void cache_load_kernel(CacheArgs a)
{
    constexpr Strip S{N};
    const int lane = threadIdx.x & 63;
    const Task<N> t(a, lane);
    bool inside;
    const Place p = t.find(a, lane, inside);
    const int ch = t.part * 8;
    if (!t.live || ch >= a.dim || !(inside || a.fill))
        return;
    const bool put_k = inside || (a.fill & 1), put_v = inside || (a.fill & 2);
    Eight<T> k = {}, v = {};
    if (p.strip) {
        const int blk = t.part >> 2, g = t.part & 3, i = p.token;
        const uint32_t kw =
            *reinterpret_cast<const uint32_t *>(p.strip + ((g * 16 + i) * N + blk) * 4);
        const char *vp = p.strip + S.values() + (((i >> 2) * 16 + g * 4) * N + blk) * 4 + (i & 3);
        uint32_t vw = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            vw |= uint32_t(uint8_t(vp[c * N * 4])) << (8 * c);
        const int ke = uint8_t(p.strip[S.key_exps() + i * S.key_exp() + blk]);
        const int ve = uint8_t(p.strip[S.value_exps() + ((i >> 2) * N + blk) * 4 + (i & 3)]);
        decode(k.v, kw, ke);
        decode(v.v, vw, ke == kNanExp ? kNanExp : ve);
    }
    if (put_k)
        k.store(const_cast<char *>(row_ptr<T>(a.k, t.token, t.head)) + ch * sizeof(T));
    if (put_v)
        v.store(const_cast<char *>(row_ptr<T>(a.v, t.token, t.head)) + ch * sizeof(T));
}

template <typename T, int N> hipError_t launch(const CacheArgs &a, bool load, hipStream_t s)
{
    const int64_t rows = int64_t(a.tokens) * a.k_heads;
    const int64_t blocks = (rows + 4 * Task<N>::ROWS - 1) / (4 * Task<N>::ROWS);
    if (blocks > INT32_MAX)
        return hipErrorInvalidValue;
    if (load)
        cache_load_kernel<T, N><<<uint32_t(blocks), 256, 0, s>>>(a);
    else
        cache_store_kernel<T, N><<<uint32_t(blocks), 256, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T> hipError_t launch_blocks(const CacheArgs &a, bool load, hipStream_t s)
{
    switch (cache_blocks(a.dim)) {
    case 1:
        return launch<T, 1>(a, load, s);
    case 2:
        return launch<T, 2>(a, load, s);
    case 3:
        return launch<T, 3>(a, load, s);
    default:
        return launch<T, 4>(a, load, s);
    }
}

hipError_t launch_any(mdcn_dtype dtype, const CacheArgs &a, bool load, hipStream_t s)
{
    switch (dtype) {
    case MDCN_F32:
        return launch_blocks<float>(a, load, s);
    case MDCN_F16:
        return launch_blocks<half_t>(a, load, s);
    default:
        return launch_blocks<bf16_t>(a, load, s);
    }
}

}  // namespace

hipError_t launch_cache_store(mdcn_dtype dtype, const CacheArgs &a, hipStream_t s)
{
    return launch_any(dtype, a, false, s);
}

hipError_t launch_cache_load(mdcn_dtype dtype, const CacheArgs &a, hipStream_t s)
{
    return launch_any(dtype, a, true, s);
}

}  // namespace mdcn
