// cache_attend_tile.hip -- attention against a key/value cache in 4 bits: many query rows of
// each sequence (prompts behind what the cache holds).
//
// Bound by the matrix and vector units.  A workgroup takes 16 * 4 * R rows of one key head, R row
// tiles a wave, and walks over the tokens 64 at a time: each wave converts one of the four
// strips to operands in LDS, which all waves then use, while the next strips are on their
// way to registers; one barrier a round, two buffers.  The work, counted by what the rows of
// an item see under the causal mask, is cut into equal contiguous ranges, one per
// workgroup; an item that several share goes to the workspace in parts.
//
// One MI355X, 32 query and 8 key heads of 128 in bf16: a call on six pieces of 2048 to 1 queries behind
// 8192 to 1 tokens 302 us, 14 of them to join (a product of 8192^3 in that many operations 193); 45 us
// go with the conversions, 34 with the exponentials.  LDS reads of operands are at 85 % of
// the vector units' time: 32 rows a wave, as 64 leave one wave a SIMD (1085 us when each wave
// converted for itself).  With 768, 1024 and 2048 workgroups instead of 512 the
// call takes 349, 310 and 335 us, one on 4096 queries of one prompt 239, 212 and 249 instead of 195.
#include "cache_attend.h"

namespace mdcn {

namespace {

constexpr int kRound = 64;                       // tokens
// Units that an item costs beside its tokens': with 0 / 3 / 8 the call above takes 357, 302 and 310 us,
// 4096 queries of one prompt 250, 195 and 207, 8 pieces of 300 to 650 queries behind 400 to 750
// tokens 106, 104 and 113.
constexpr int kItemCost = 3;

// Units of the items of one (sequence, key head), item i being rows 16 kWaves R i and on:
// what they see grows evenly under a causal mask, so the units before an item are a
// quadratic of its index, counted from the first item that sees a token at all: with more queries
// than tokens the earlier ones are `blind`.  So there are never more units than the host
// allows for (most_units).  In 64-bit floating point: the inner sum is exact, so every workgroup
// comes to the same whole numbers, however the operations are fused, and they grow with the index.
template <int R> struct Ladder {
    static constexpr int ROWS = 16 * kWaves * R;
    double first, step, per;
    int tiles, blind;

    __device__ __forceinline__ Ladder(const CacheArgs &a, const Piece &pc)
    {
        const int shared = a.q_heads / a.k_heads;
        tiles = int((uint32_t(pc.lq) * uint32_t(shared) + ROWS - 1) / ROWS);
        blind = a.causal ? int(uint32_t(max(pc.lq - pc.lk, 0)) * uint32_t(shared) / ROWS) : 0;
        step = a.causal ? double(ROWS) : 0.0;
        first = double(a.causal ? max(pc.lk - pc.lq, 0) : pc.lk) * shared + step;
        per = 1.0 / (2.0 * shared * double(kRound << a.unit_shift));
    }

    __device__ __forceinline__ int before(int i) const
    {
        const int n = max(i - blind, 0);
        return kItemCost * i + int(double(n) * (2.0 * first + double(n - 1) * step) * per);
    }

    __device__ __forceinline__ int item_of(int unit) const
    {
        int lo = 0, hi = tiles;                  // before(lo) <= unit < before(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (before(mid) <= unit)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    }
};

template <int R> struct Chunk {
    Piece piece;
    int mine, upto;

    __device__ __forceinline__ void load(const CacheArgs &a, int b0, int lane)
    {
        piece = {};
        mine = 0;
        if (b0 + lane < a.batch) {
            piece = piece_of(a, b0 + lane);
            const Ladder<R> l(a, piece);
            mine = l.before(l.tiles) * a.k_heads;
        }
        upto = wave_scan(mine);
    }
};

// The operands of a round in LDS, 1 KB each, as the lanes use them.
template <int N> struct Operands {
    static constexpr int KEYS = 4 * N * 1024;
    static constexpr int BYTES = 2 * KEYS;

    static __device__ __forceinline__ char *key(char *p, int strip, int block, int lane)
    {
        return p + (strip * N + block) * 1024 + lane * 16;
    }
    static __device__ __forceinline__ char *value(char *p, int pair, int block, int odd, int lane)
    {
        return p + KEYS + ((pair * N + block) * 2 + odd) * 1024 + lane * 16;
    }
};

template <typename T> __device__ __forceinline__ Vec<T> operand_at(const char *p)
{
    return *reinterpret_cast<const Vec<T> *>(p);
}

template <typename T, int N, int R> __global__ __launch_bounds__(256, 2) void cache_tile_kernel(CacheArgs a)
{
    constexpr Strip S{N};
    using Ops = Operands<N>;
    __shared__ __align__(1024) char smem[2 * Ops::BYTES];
    __shared__ __align__(16) int gone_of[2][kWaves];             // strips without a page

    if (int(blockIdx.x) >= a.workers) {
        fill_rows<T>(a);
        return;
    }
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int grp = lane >> 4;
    const float c = a.scale * kLog2e, margin = raise_margin(c);
    const int strip_shift = a.page_shift - 4;

    Chunk<R> chunk;
    chunk.load(a, 0, lane);
    int units = __builtin_amdgcn_readlane(chunk.upto, 63);
    if (a.batch > 64) {
        int more = 0;
        for (int b = 64 + lane; b < a.batch; b += 64) {
            const Ladder<R> l(a, piece_of(a, b));
            more += l.before(l.tiles) * a.k_heads;
        }
        units += wave_sum(more);
    }
    const Share share(units, a.workers);
    Join *join = reinterpret_cast<Join *>(a.joins) + blockIdx.x;
    if (threadIdx.x == 0)
        join->init();
    if (int(blockIdx.x) >= share.n)
        return;
    const int u_begin = share.begin(int(blockIdx.x)), u_end = share.begin(int(blockIdx.x) + 1);

    int base = 0;
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
            const Ladder<R> ladder(a, pc);
            const int of_head = __builtin_amdgcn_readfirstlane(ladder.before(ladder.tiles));
            const int to = min(u_end, s_end);
            const auto row_pages = reinterpret_cast<scalar_ints>(
                reinterpret_cast<uintptr_t>(a.table + int64_t(b0 + i) * a.table_stride));
            const int held = (pc.lk + (1 << a.page_shift) - 1) >> a.page_shift;
            for (int u = max(u_begin, s_begin); u < to;) {
                // item: 16 kWaves R rows of a key head; units [n0, n1) of its `all`
                const int kv_head = (u - s_begin) / of_head;
                if (kv_head >= a.k_heads)
                    return;                      // offsets that overlap beyond counting
                const int h_begin = s_begin + kv_head * of_head;
                const int tile = __builtin_amdgcn_readfirstlane(ladder.item_of(u - h_begin));
                const int i_begin = h_begin + __builtin_amdgcn_readfirstlane(ladder.before(tile));
                const int all =
                    __builtin_amdgcn_readfirstlane(ladder.before(tile + 1)) + h_begin - i_begin;
                const int n0 = u - i_begin, n1 = min(to - i_begin, all);
                u = i_begin + n1;

                // the rounds that go with these units
                const Sight sight(a, pc, uint32_t(tile) * kWaves * R, kWaves * R);
                const int visible = sight.any < 0 ? 0 : sight.any / kRound + 1;
                auto round_of = [&](int n) {
                    if (n >= all)
                        return visible;
                    return n <= kItemCost ? 0
                                          : int(int64_t(n - kItemCost) * visible / (all - kItemCost));
                };
                const int t0 = round_of(n0), t1 = round_of(n1);

                const uint32_t first = (uint32_t(tile) * kWaves + wave) * R;
                const Sight own(a, pc, first, R);
                RowTile<T, N> rows[R];
                State<2 * N> st[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    rows[r].load(a, pc, kv_head, first + r, lane);
                    st[r].init();
                }

                const char *const heads = a.pool + int64_t(kv_head << strip_shift) * S.bytes();
                Raw<N> x;
                int gone = 0;
                auto page_of = [&](int t) {
                    return row_pages[min((4 * t + wave) >> strip_shift, held - 1)];
                };
                auto fetch = [&](int t, int n) {  // this wave's strip of round t, in page n
                    const uint32_t page = uint32_t(n) < uint32_t(a.pages) ? uint32_t(n) : 0u;
                    gone = page == uint32_t(n) ? 0 : 1;
                    x.load(heads + uint64_t(page) * uint32_t(a.page_stride) +
                               ((4 * t + wave) & ((1 << strip_shift) - 1)) * S.bytes(),
                           lane);
                };
                auto convert = [&](int t) {
                    char *const to_lds = smem + (t & 1) * Ops::BYTES;
                    const int tok = t * kRound + wave * 16;
                    if (gone || tok + 16 > pc.lk)
                        settle_values(x, gone ? 0 : pc.lk - tok - grp * 4);
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        *reinterpret_cast<Vec<T> *>(Ops::key(to_lds, wave, j, lane)) =
                            key_operand<T, N>(x, j);
#pragma unroll
                    for (int b = 0; b < N; ++b) {
                        uint32_t w[2][2];
                        value_halves<T, N>(x, b, w[0], w[1]);
#pragma unroll
                        for (int odd = 0; odd < 2; ++odd)
                            *reinterpret_cast<uint2 *>(
                                Ops::value(to_lds, wave >> 1, b, odd, lane) + (wave & 1) * 8) =
                                make_uint2(w[odd][0], w[odd][1]);
                    }
                    if (lane == 0)
                        gone_of[t & 1][wave] = gone;
                };
                auto compute = [&](int t) {
                    char *const from = smem + (t & 1) * Ops::BYTES;
                    float4v sc[R][4] = {};
#pragma unroll
                    for (int s = 0; s < 4; ++s)
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            const Vec<T> k = operand_at<T>(Ops::key(from, s, j, lane));
#pragma unroll
                            for (int r = 0; r < R; ++r)
                                sc[r][s] = product<T>(k, rows[r].q[j], sc[r][s]);
                        }
                    const int4 g = *reinterpret_cast<const int4 *>(gone_of[t & 1]);
                    const int any_gone = __builtin_amdgcn_readfirstlane(g.x | g.y | g.z | g.w);
                    if (t * kRound + kRound - 1 > own.all || any_gone) {
                        asm volatile("");        // a branch, not selects in every round
                        const int missing[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                        for (int s = 0; s < 4; ++s)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
#pragma unroll
                                for (int r = 0; r < R; ++r)
                                    if (t * kRound + s * 16 + grp * 4 + e > rows[r].last || missing[s])
                                        sc[r][s][e] = -INFINITY;
                    }
                    Parts<T> p[R][2];
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        softmax<T>(st[r], sc[r], p[r], c, margin);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int b = 0; b < N; ++b)
#pragma unroll
                            for (int odd = 0; odd < 2; ++odd) {
                                const Vec<T> v = operand_at<T>(Ops::value(from, i, b, odd, lane));
#pragma unroll
                                for (int r = 0; r < R; ++r)
                                    st[r].o[2 * b + odd] =
                                        product<T>(v, p[r][i], st[r].o[2 * b + odd]);
                            }
                };
                int page = 0;
                if (t0 < t1) {
                    fetch(t0, page_of(t0));
                    page = page_of(t0 + 1);
                    convert(t0);
                    if (t0 + 1 < t1)
                        fetch(t0 + 1, page);
                    page = page_of(t0 + 2);
                }
                __syncthreads();
                for (int t = t0; t < t1; ++t) {
                    if (t * kRound <= own.any)
                        compute(t);
                    if (t + 1 < t1)
                        convert(t + 1);
                    if (t + 2 < t1) {
                        fetch(t + 2, page);
                        page = page_of(t + 3);
                    }
                    __syncthreads();
                }

                if (n0 == 0 && n1 == all) {
                    bool lost = false;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float lse;
                        lost |= finish<T, 2 * N>(
                            a, st[r], Row16(a, pc.q0, pc.lq, kv_head, first + r, lane), 0, lane, lse);
                    }
                    if (lost && lane == 0)
                        join->lost = 1;
                } else {
                    float *slot = a.partial + ((int64_t(blockIdx.x) * 2 + (n0 == 0 ? 1 : 0)) * kWaves +
                                               wave) * (R * part_floats<N>());
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        put_state(slot + r * part_floats<N>(), st[r], lane);
                    if (n0 == 0 && threadIdx.x == 0)
                        join->set(pc, b0 + i, kv_head, tile, share.owner(i_begin + all - 1));
                }
            }
        }
        base += __builtin_amdgcn_readlane(chunk.upto, 63);
    }
}

// Row tile r of the items that workgroup `worker` of the first kernel had to itself once more, as
// means: its units are counted as there, one sequence after the other.
template <typename T, int N, int ROWS>
__device__ __forceinline__ void means_of(const CacheArgs &a, int worker, int r, int lane)
{
    using Steps = Ladder<ROWS / kWaves>;
    int units = 0;
    for (int i = lane; i < a.batch; i += 64) {
        const Steps l(a, piece_of(a, i));
        units += l.before(l.tiles) * a.k_heads;
    }
    const Share share(wave_sum(units), a.workers);
    const int u_begin = share.begin(worker), u_end = share.begin(worker + 1);
    int base = 0;
    for (int sequence = 0; sequence < a.batch && base < u_end; ++sequence) {
        const Piece pc = piece_of(a, sequence);
        const Steps l(a, pc);
        for (int head = 0; head < a.k_heads; ++head) {
            for (int i = 0; i < l.tiles && base + l.before(i + 1) <= u_end; ++i) {
                if (base + l.before(i) < u_begin)
                    continue;
                const uint32_t tile = uint32_t(i) * ROWS + r;
                const Row16 at(a, pc.q0, pc.lq, head, tile, lane);
                const float lse = at.live ? a.lse[int64_t(at.head) * a.tokens + at.token] : 0.0f;
                for (int b = 0; b < N; ++b)
                    put_mean<T, N>(a, pc, sequence, head, tile, at, lse, b, lane);
            }
            base += l.before(l.tiles);
        }
    }
}

// One wave per (workgroup of the first kernel, row tile): joins the parts of the item that
// began there, the next part's registers on their way.
template <typename T, int N, int ROWS>
__global__ __launch_bounds__(256) void cache_tile_join_kernel(CacheArgs a)
{
    const Join j = reinterpret_cast<const Join *>(a.joins)[blockIdx.x];
    const int lane = threadIdx.x & 63;
    const int r = int(blockIdx.y) * kWaves + __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    if constexpr (!__is_same(T, half_t))
        if (j.lost)
            means_of<T, N, ROWS>(a, int(blockIdx.x), r, lane);
    if (j.last < 0)
        return;
    const float c = a.scale * kLog2e;
    const int first = int(blockIdx.x), end = min(j.last, a.workers - 1);
    auto part = [&](int i) {
        return a.partial +
               ((int64_t(i) * 2 + (i == first ? 1 : 0)) * ROWS + r) * part_floats<N>();
    };
    State<2 * N> st, x;
    get_state(st, part(first), lane);
    if (first < end)
        get_state(x, part(first + 1), lane);
    for (int i = first + 1; i <= end; ++i) {
        State<2 * N> y;
        if (i < end)
            get_state(y, part(i + 1), lane);
        st.merge(x, c);
        x = y;
    }
    const uint32_t tile = uint32_t(j.tile) * ROWS + r;
    const Row16 at(a, j.q0, j.lq, j.head, tile, lane);
    float lse;
    if (finish<T, 2 * N>(a, st, at, 0, lane, lse))
        for (int b = 0; b < N; ++b)
            put_mean<T, N>(a, j.piece(), j.sequence, j.head, tile, at, lse, b, lane);
}

template <typename T, int N> hipError_t launch(const CacheArgs &a, hipStream_t s)
{
    constexpr int ROWS = tile_row_tiles(sizeof(T) == 4), R = ROWS / kWaves;
    const int64_t row_bytes = int64_t(a.tokens) * a.q_heads * a.dim * int64_t(sizeof(T));
    const int fills = a.fill ? fill_blocks(row_bytes) : 0;
    cache_tile_kernel<T, N, R><<<uint32_t(a.workers + fills), 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.workers == 0)
        return e;
    cache_tile_join_kernel<T, N, ROWS><<<dim3(uint32_t(a.workers), R), 256, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T> hipError_t launch_blocks(const CacheArgs &a, hipStream_t s)
{
    switch (cache_blocks(a.dim)) {
    case 1:
        return launch<T, 1>(a, s);
    case 2:
        return launch<T, 2>(a, s);
    case 3:
        return launch<T, 3>(a, s);
    default:
        return launch<T, 4>(a, s);
    }
}

}  // namespace

hipError_t launch_cache_tile(mdcn_dtype dtype, const CacheArgs &a, hipStream_t s)
{
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
