// cache_common.h -- device pieces shared by the kernels on 4-bit caches (gfx950).
#pragma once

#include "attention_common.h"
#include "cache.h"

namespace mdcn {

// Four bytes times N at an address that need be a multiple of 4 only.
template <int N> struct Words {
    uint32_t w[N];
};

// Finds the sequences of a packed tensor's tokens.  The offsets and lengths of 64 sequences
// are held one a lane: in a batch of no more than that a token costs no load.
struct Finder {
    int begin, end, used;

    __device__ __forceinline__ Finder(const CacheArgs &a, int lane)
    {
        begin = INT32_MAX;
        end = used = 0;
        if (a.batch <= 64 && lane < a.batch) {
            begin = a.cu[lane];
            end = a.cu[lane + 1];
            used = a.used[lane];
        }
    }

    // The sequence that token t belongs to, or -1, and the token's place in it; every lane
    // of the wave must call it with the same t.
    __device__ __forceinline__ int find(const CacheArgs &a, int t, int lane, int64_t &at) const
    {
        if (a.batch <= 64) {
            const uint64_t below = __ballot(begin <= t);
            if (below == 0)
                return -1;
            // (offsets that do not grow leave gaps: the last sequence that begins before t)
            const int b = 63 - __builtin_clzll(below);
            const int last = __builtin_amdgcn_readlane(end, b);
            at = int64_t(__builtin_amdgcn_readlane(used, b)) - min(last, a.tokens) + t;
            return t < last ? b : -1;
        }
        int lo = 0, n = a.batch;
        while (n > 0) {                          // 64 offsets at a time, evenly spread
            const int step = (n + 63) / 64, i = lane * step;
            const int below = __popcll(__ballot(i < n && a.cu[lo + i] <= t));
            if (below == 0)
                return -1;
            lo += (below - 1) * step;
            n = step == 1 ? 0 : min(step, n - (below - 1) * step);
        }
        const int last = a.cu[lo + 1];
        at = int64_t(a.used[lo]) - min(last, a.tokens) + t;
        return t < last ? lo : -1;
    }
};

// Where a token lies: its strip's first byte, head 0, or null; and its place there.
struct Place {
    char *strip;
    int token;
};

__device__ __forceinline__ Place place_of(const CacheArgs &a, int b, int64_t at, int strip_bytes)
{
    Place p = {nullptr, 0};
    if (at < 0 || at >= int64_t(a.width) << a.page_shift)
        return p;
    const int page = a.table[b * a.table_stride + (at >> a.page_shift)];
    if (page < 0 || page >= a.pages)
        return p;
    const int in = int(at) & ((1 << a.page_shift) - 1);
    p.strip = a.pool + page * a.page_stride + (in >> 4) * strip_bytes;
    p.token = in & 15;
    return p;
}

// Two of four fp4 values of a dword as two values of a 16-bit type, exactly; `scale`
// is 2^e as its exponent bits, other bits are ignored (an exponent of 255 gives NaN).
template <typename T, int BYTE> __device__ __forceinline__ uint32_t fp4_pair(uint32_t w, uint32_t scale)
{
    uint32_t r;
    if constexpr (__is_same(T, half_t)) {
        const auto v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, __uint_as_float(scale), BYTE);
        __builtin_memcpy(&r, &v, 4);
    } else {
        const auto v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, __uint_as_float(scale), BYTE);
        __builtin_memcpy(&r, &v, 4);
    }
    return r;
}

}  // namespace mdcn
