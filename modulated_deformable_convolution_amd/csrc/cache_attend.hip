// cache_attend.hip -- attention against a key/value cache in 4 bits: few query rows of each
// sequence (decoding), and the choice between the kernels.
//
// Bound by reading the used strips once.  The work, in units of 32 tokens of one (sequence,
// key head, row tile), is cut into equal contiguous ranges, one per workgroup, whatever the
// lengths: lengths are read on the GPU.  The four waves of a workgroup take a quarter of a
// range's tokens each, copy their strips to LDS asynchronously and convert them in
// registers, and are joined in LDS; a (sequence, head, tile) that several workgroups share
// goes to the workspace in parts that a second kernel joins.
//
// One MI355X, 32 query and 8 key heads of 128, pages of 16: 48 caches of 1 to 16384 tokens in
// bf16 82 to 85 us (384 MB; 430 past the L2s with the parts, 5.2 TB/s; strips alone read in this order
// reach 5.9) and 6 to join, 91 a call.  Taking the conversions, the exponentials or both away leaves that time
// as it is, pages that stay in the L2s halve it: memory bounds it.  Older waves are served
// first and end after half of the time; shares to match, priorities or smaller shares gained
// nothing.  One cache of 4097 tokens in fp16: 8.4 us and 5, round trips to memory.
#include <algorithm>
#include <cmath>

#include "cache_attend.h"

namespace mdcn {

namespace {

constexpr int kTile = 32;                        // tokens

// Waves a SIMD that the registers leave room for: a row tile of 16-bit queries with its sums
// takes 48 of 128 of them, a second one or the three parts of fp32 as much again.  More
// workgroups than run together, of less work each, are slower: calls on the 48 caches above take 97
// and 95 us with 1536 and 2048, 91 with 1024; on 400 of 1 to 200 tokens 46 and 51, 38 with 1024.
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

// Units of an item, a (key head, row tile) of a sequence: one for each 32 << unit_shift tokens,
// after kItemCost for what an item costs whatever its length.
struct Units {
    int tiles, keys, all;
};

// Calls with 0 / 5 / 10 / 20, 32/8 heads of 128 in bf16: 48 caches of 1 to 16384 tokens 101, 93, 91 and
// 92 us, 48 of 512 23, 22, 23 and 24; where caches are alike 0 is as good or better: 16 of 4096
// tokens 29, 30, 30 and 32, 400 of 1 to 200 36, 37, 38 and 38.
constexpr int kItemCost = 10;
// Tiles up to which one wave takes an item alone, without the others and their barriers.
// Calls with 0 / 3 / 8: the 48 caches 91, 91 and 93 us, 16 of 4096 tokens 30 each, 400 of 1 to 200
// 40, 38 and 31: more suits short caches, and costs long ones their balance.
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
    const int grp = lane >> 4;
    const float c = a.scale * kLog2e, margin = raise_margin(c);

    if (int(blockIdx.x) >= a.workers) {
        fill_rows<T>(a);
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
        join->init();
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

                RowTile<T, N> rows[R];
#pragma unroll
                for (int r = 0; r < R; ++r)
                    rows[r].load(a, pc, kv_head, uint32_t(tile) * R + r, lane);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        rows[r].q[j].settle();
                const Sight sight(a, pc, uint32_t(tile) * R, R);
                const int visible = sight.any < 0 ? 0 : sight.any / kTile + 1;
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
                                sc[r][s] = product<T>(k, rows[r].q[j], sc[r][s]);
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

                    if (t * kTile + kTile - 1 > sight.all || gone) {
                        asm volatile("");        // a branch, not selects in every round
                        const int tok = t * kTile + grp * 4;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            settle_values(x[s], gone >> s & 1 ? 0 : pc.lk - (tok + 16 * s));
#pragma unroll
                            for (int r = 0; r < R; ++r)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (tok + 16 * s + e > rows[r].last || (gone >> s & 1))
                                        sc[r][s][e] = -INFINITY;
                        }
                    }
                    Parts<T> p[R][1];
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        softmax<T>(st[r], sc[r], p[r], c, margin);
#pragma unroll
                    for (int b = 0; b < N; ++b) {
                        uint32_t w[2][2][2];
                        value_halves<T, N>(x[0], b, w[0][0], w[1][0]);
                        value_halves<T, N>(x[1], b, w[0][1], w[1][1]);
                        Vec<T> even, odd;
                        __builtin_memcpy(&even, w[0], 16);
                        __builtin_memcpy(&odd, w[1], 16);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            st[r].o[2 * b] = product<T>(even, p[r][0], st[r].o[2 * b]);
                            st[r].o[2 * b + 1] = product<T>(odd, p[r][0], st[r].o[2 * b + 1]);
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
                        bool lost = false;
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            float lse;
                            lost |= finish<T, 2 * N>(
                                a, st[r],
                                Row16(a, pc.q0, pc.lq, kv_head, uint32_t(tile) * R + r, lane), 0, lane,
                                lse);
                        }
                        if (lost && lane == 0)
                            join->lost = 1;
                    } else {
                        float *slot = a.partial + (int64_t(blockIdx.x) * 2 + (n0 == 0 ? 1 : 0)) *
                                                      (R * part_floats<N>());
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            put_state(slot + r * part_floats<N>(), st[r], lane);
                        if (n0 == 0 && lane == 0)
                            join->set(pc, b0 + i, kv_head, tile, share.owner(i_begin + un.keys - 1));
                    }
                }
            }
        }
        base += __builtin_amdgcn_readlane(chunk.upto, 63);
    }
}

// Block b of row tile r of the items that workgroup `worker` of the first kernel had to itself once
// more, as means: its units are counted as there, one sequence after the other.
template <typename T, int N, int ROWS>
__device__ __forceinline__ void means_of(const CacheArgs &a, int worker, int r, int b, int wave, int lane)
{
    int units = 0;
    for (int i = lane; i < a.batch; i += 64)
        units += units_of<ROWS>(a, piece_of(a, i)).all;
    const Share share(wave_sum(units), a.workers);
    const int u_begin = share.begin(worker), u_end = share.begin(worker + 1);
    int base = 0, turn = 0;
    for (int sequence = 0; sequence < a.batch && base < u_end; ++sequence) {
        const Piece pc = piece_of(a, sequence);
        const Units un = units_of<ROWS>(a, pc);
        for (int i = max(u_begin - base + un.keys - 1, 0) / un.keys;
             i < un.tiles * a.k_heads && base + (i + 1) * un.keys <= u_end; ++i)
            if ((turn++ & (kWaves - 1)) == wave) {
                const uint32_t tile = uint32_t(i % un.tiles) * ROWS + r;
                const Row16 at(a, pc.q0, pc.lq, i / un.tiles, tile, lane);
                const float lse = at.live ? a.lse[int64_t(at.head) * a.tokens + at.token] : 0.0f;
                put_mean<T, N>(a, pc, sequence, i / un.tiles, tile, at, lse, b, lane);
            }
        base += un.all;
    }
}

// One workgroup per (workgroup of the first kernel, row tile and block of channels): joins
// the parts of the item of ROWS row tiles that began there.  Its waves take every fourth part.
template <typename T, int N, int ROWS>
__global__ __launch_bounds__(256) void cache_join_kernel(CacheArgs a)
{
    __shared__ __align__(16) float lds[2 * part_floats<1>()];
    const Join j = reinterpret_cast<const Join *>(a.joins)[blockIdx.x];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int r = int(blockIdx.y) / N, b = int(blockIdx.y) % N;
    if constexpr (!__is_same(T, half_t))
        if (j.lost)
            means_of<T, N, ROWS>(a, int(blockIdx.x), r, b, wave, lane);
    if (j.last < 0)
        return;
    const float c = a.scale * kLog2e;
    const int first = int(blockIdx.x), end = min(j.last, a.workers - 1);

    constexpr int AT_ONCE = 4;                   // parts whose loads are on their way together
    State<2> st[1];
    st[0].init();
    for (int i0 = first + wave; i0 <= end; i0 += kWaves * AT_ONCE) {
        State<2> x[AT_ONCE];
#pragma unroll
        for (int n = 0; n < AT_ONCE; ++n) {
            const int i = i0 + n * kWaves;
            x[n].init();
            if (i <= end) {
                const float *p = a.partial + ((int64_t(i) * 2 + (i == first ? 1 : 0)) * ROWS + r) *
                                                 part_floats<N>();
#pragma unroll
                for (int o = 0; o < 2; ++o)
                    x[n].o[o] = reinterpret_cast<const float4v *>(p)[(2 * b + o) * 64 + lane];
                x[n].m = p[2 * N * 256 + lane];
                x[n].l = p[2 * N * 256 + 64 + lane];
            }
        }
#pragma unroll
        for (int n = 0; n < AT_ONCE; ++n)
            st[0].merge(x[n], c);
    }
    join_waves<1, 2>(st, lds, c, wave, lane);
    if (wave == 0) {
        const uint32_t tile = uint32_t(j.tile) * ROWS + r;
        const Row16 at(a, j.q0, j.lq, j.head, tile, lane);
        float lse;
        if (finish<T, 2>(a, st[0], at, b, lane, lse))
            put_mean<T, N>(a, j.piece(), j.sequence, j.head, tile, at, lse, b, lane);
    }
}

// Row tiles of an item, by the rows of an average sequence: one (fp32: of up to 64 rows) or
// two in the split kernel, which reads keys and values again for each item, kWaves or twice
// as many in the tile kernel.  Calls in us, 16 sequences of 4096 tokens (fp32: 2048), 32 query
// and 8 key heads of 128, with one row tile / two (fp32 has one only) / the tile kernel:
//   rows   16          20          32          48          64          128
//   bf16   31 34 64    39 35 64    39 35 64    50 47 69    59 47 69    93 65 74
//   fp32   23    41    30    45    30    46    41    47    47    48    74    71
int row_tiles(mdcn_dtype dtype, const CacheArgs &a)
{
    const bool f32 = dtype == MDCN_F32;
    const double rows = a.batch ? double(a.tokens) / a.batch * (a.q_heads / a.k_heads) : 0;
    return rows <= (f32 ? 64 : 16) ? 1 : rows <= 128 && !f32 ? 2 : tile_row_tiles(f32);
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

template <typename T, int N> hipError_t launch_rows(const CacheArgs &a, int tiles, hipStream_t s)
{
    if constexpr (sizeof(T) == 2)
        if (tiles == 2)
            return launch<T, N, 2>(a, s);
    return launch<T, N, 1>(a, s);
}

template <typename T> hipError_t launch_blocks(const CacheArgs &a, int tiles, hipStream_t s)
{
    switch (cache_blocks(a.dim)) {
    case 1:
        return launch_rows<T, 1>(a, tiles, s);
    case 2:
        return launch_rows<T, 2>(a, tiles, s);
    case 3:
        return launch_rows<T, 3>(a, tiles, s);
    default:
        return launch_rows<T, 4>(a, tiles, s);
    }
}

}  // namespace

// Units of a batch with queries in `sequences` sequences, at most: (row tiles) x (key heads) x
// (units of all tokens).
static double most_units(const CacheArgs &a, int tiles, int shift, int sequences)
{
    const int tokens = (tiles > 2 ? 64 : kTile) << shift;
    const double rows = double(a.tokens) * (a.q_heads / a.k_heads);
    const double keys = double(a.width) * (1 << a.page_shift) / tokens;
    return (rows / (16 * tiles) + sequences) * a.k_heads * (keys + kItemCost + 1);
}

CacheShape cache_attend_shape(mdcn_dtype dtype, const CacheArgs &a)
{
    const int tiles = row_tiles(dtype, a);
    const int most = tiles > 2 ? kTileWorkers : 256 * (tiles == 2 ? 2 : dtype == MDCN_F32 ? 3 : 4);
    int shift = 0;
    while (most_units(a, tiles, shift, a.batch) > 1e9 && shift < 20)
        ++shift;
    // no more workgroups than a small batch has work for; none: rows to fill only
    const int workers =
        int(std::min<double>(most, std::ceil(most_units(a, tiles, shift, a.batch) / kWaves)));
    return CacheShape{16 * tiles, a.batch ? workers : 0, (tiles > 2 ? 64 : kTile) << shift};
}

// What an item costs does not shrink with longer units: enough items pass any count.
bool cache_attend_countable(mdcn_dtype dtype, const CacheArgs &a)
{
    const CacheShape c = cache_attend_shape(dtype, a);
    const int tiles = c.rows / 16;
    const int shift = __builtin_ctz(unsigned(c.unit / (tiles > 2 ? 64 : kTile)));
    return a.batch == 0 || most_units(a, tiles, shift, std::min(a.batch, a.tokens)) <= 2e9;
}

size_t cache_attend_bytes(mdcn_dtype dtype, const CacheArgs &a)
{
    const CacheShape c = cache_attend_shape(dtype, a);
    const size_t part = size_t(c.rows / 16) * (8 * cache_blocks(a.dim) + 2) * 64 * sizeof(float);
    return size_t(c.workers) * (2 * part + sizeof(Join));
}

hipError_t launch_cache_attend(mdcn_dtype dtype, CacheArgs a, void *workspace, hipStream_t s)
{
    const CacheShape shape = cache_attend_shape(dtype, a);
    const int tiles = shape.rows / 16;
    a.workers = shape.workers;
    a.unit_shift = __builtin_ctz(unsigned(shape.unit / (tiles > 2 ? 64 : kTile)));
    a.joins = static_cast<int4 *>(workspace);
    a.partial = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                          size_t(a.workers) * sizeof(Join));
    if (tiles > 2)
        return launch_cache_tile(dtype, a, s);
    switch (dtype) {
    case MDCN_F32:
        return launch_blocks<float>(a, tiles, s);
    case MDCN_F16:
        return launch_blocks<half_t>(a, tiles, s);
    default:
        return launch_blocks<bf16_t>(a, tiles, s);
    }
}

}  // namespace mdcn
