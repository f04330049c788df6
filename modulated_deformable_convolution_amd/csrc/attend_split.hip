// attend_split.hip -- attention with few query rows per sequence (decoding
// against a key/value cache), forward.
//
// The same mathematics as attend.hip, bound by reading the used keys and values
// once.  The rows of one key head -- its group's heads times the new tokens --
// are packed into tiles of 32, so keys and values are read once per 32 rows.
// The work, in units of 32 keys of one (sequence, key head, row tile), is cut
// into equal contiguous ranges, one per workgroup, whatever the lengths:
// lengths are read on the GPU.  In a workgroup each wave takes a
// contiguous part of the range's keys and copies them to its own two LDS
// stages, with no barrier in the loop (only the wave's own copies are waited
// for); the waves' results are joined in LDS.  A (sequence, head, tile) that lies
// in one range is finished there; otherwise its parts (sums, maxima and
// unscaled outputs in fp32) go to the workspace and a second kernel joins them.
//
// One MI355X, bf16, 32 query and 8 key heads of 128: 48 caches of 1 to 16384
// tokens 263 to 273 us (1.6 GB, 6.0 TB/s; a copy's reads and writes reach 4.8) and 8 us
// to join; one cache of 4097 tokens 11 us and 5 us, round trips to memory.
#include <algorithm>
#include <cmath>

#include "attention_common.h"

namespace mdcn {

namespace {

constexpr int kTileRows = 32;
constexpr int kUnit = 32;                       // keys of one unit

// fp32 rows of more than 64 values take two waves' stages for one
template <typename T, int DP> constexpr int split_waves()
{
    return Row<T, DP>::PITCH > 256 ? 2 : 4;
}

template <typename T, int DP> constexpr int split_lds()
{
    return split_waves<T, DP>() * 4 * kUnit * Row<T, DP>::PITCH;
}

// Units of a sequence: `keys` per (key head, row tile), at least one.  A unit is
// 32 << unit_shift keys, the shift chosen on the host so that the units of any batch of
// this size can be counted in 31 bits (0 for all but huge caches).
struct Units {
    int tiles, keys, all;
};

__device__ __forceinline__ Units units_of(const AttendArgs &a, const Span &s)
{
    Units u;
    u.tiles = int((uint32_t(s.lq) * uint32_t(a.q_heads / a.k_heads) + kTileRows - 1) / kTileRows);
    const int keys = kUnit << a.unit_shift;
    u.keys = s.lk > keys ? (s.lk + keys - 1) >> (5 + a.unit_shift) : 1;
    u.all = u.tiles * a.k_heads * u.keys;
    return u;
}

// The units of 64 sequences, one per lane: its own and those up to it.
struct Chunk {
    Span span;
    int mine, upto;

    __device__ __forceinline__ void load(const AttendArgs &a, int b0, int lane)
    {
        span = {};
        mine = 0;
        if (b0 + lane < a.batch) {
            span = span_of(a, b0 + lane);
            mine = units_of(a, span).all;
        }
        upto = wave_scan(mine);
    }
};

// All units of the batch; `first` is the chunk of its first 64 sequences.
__device__ __forceinline__ int total_units(const AttendArgs &a, const Chunk &first, int lane)
{
    int sum = __builtin_amdgcn_readlane(first.upto, 63);
    if (a.batch > 64) {
        int more = 0;
        for (int b = 64 + lane; b < a.batch; b += 64)
            more += units_of(a, span_of(a, b)).all;
        sum += wave_sum(more);
    }
    return sum;
}

// How the units are shared: `n` workgroups, enough units for all waves of each;
// workgroup i has units [units * i / n, units * (i + 1) / n), so that equal items
// are cut alike and none straddles two of them needlessly.
struct Share {
    int units, n, each, rest;

    __device__ __forceinline__ Share(int units_, int workers, int waves) : units(units_)
    {
        n = min((units + waves - 1) / waves, workers);
        each = n > 0 ? units / n : 0;
        rest = units - each * n;
    }

    // units * i / n without the long product (n * n fits)
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

template <typename T, int DP>
__global__ __launch_bounds__(256) void attend_split_kernel(AttendArgs a)
{
    using R = Row<T, DP>;
    constexpr int NW = split_waves<T, DP>();
    constexpr int TILE = kUnit * R::PITCH;
    constexpr int OP = 33;                       // pitch of a joined output column, floats
    static_assert(DP * OP * 4 <= 4 * TILE, "a wave's outputs fit its stages");
    constexpr int PART = DP + 2;
    __shared__ __align__(1024) char smem[NW * 4 * TILE];
    __shared__ float stat[NW][2][32];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int half = lane >> 5;
    const int col = lane & 31;
    const int group = a.q_heads / a.k_heads;
    const float c = a.scale * kLog2e, margin = raise_margin(c);

    Chunk chunk;
    chunk.load(a, 0, lane);
    const int units = total_units(a, chunk, lane);
    const Share share(units, a.workers, NW);
    if (int(blockIdx.x) >= share.n)
        return;
    const int u_begin = share.begin(int(blockIdx.x)), u_end = share.begin(int(blockIdx.x) + 1);

    Stager<T, DP, kUnit, 1> st;
    st.init(a.k.token_stride, a.v.token_stride, a.dim, 0, lane);
    char *own = smem + wave * 4 * TILE;
    const uint32_t lds = lds_address(own);

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
            const Span sp = span_in(chunk.span, i);
            const Units un = units_of(a, sp);
            const int shift = sp.lk - sp.lq;
            const int to = min(u_end, s_end);
            for (int u = max(u_begin, s_begin); u < to;) {
                // item: a (key head, row tile) of this sequence; keys [n0, n1) of it, in units
                const int item = (u - s_begin) / un.keys;
                const int i_begin = s_begin + item * un.keys;
                const int n0 = u - i_begin;
                const int n1 = min(to - i_begin, un.keys);
                u = i_begin + n1;
                const int kv_head = item / un.tiles;
                const int tile = item % un.tiles;
                if (kv_head >= a.k_heads)
                    return;                      // offsets that overlap beyond counting

                const uint32_t packed = uint32_t(tile) * kTileRows + col;
                const int row = int(packed / uint32_t(group));
                const int head = kv_head * group + int(packed % uint32_t(group));
                const bool live = row < sp.lq;
                const int last = a.causal ? row + shift : sp.lk - 1;
                const int tile_first =
                    a.causal ? int(uint32_t(tile) * kTileRows / uint32_t(group)) + shift : sp.lk - 1;
                const int tile_last =
                    a.causal ? min(int((uint32_t(tile) * kTileRows + 31) / uint32_t(group)),
                                   sp.lq - 1) + shift
                             : sp.lk - 1;

                const char *kbase = row_ptr<T>(a.k, sp.k0, kv_head);
                const char *vbase = row_ptr<T>(a.v, sp.k0, kv_head);
                Softmax<T, DP> sm;
                sm.init();
                bool check = a.causal != 0;

                // this wave's tiles of 32 keys, from the last one down (see attend.hip)
                const int t0 = n0 << a.unit_shift, nt = (n1 - n0) << a.unit_shift;
                const int visible = tile_last < 0 ? 0 : tile_last / kUnit + 1;
                const int w0 = t0 + nt / NW * wave + min(nt % NW, wave);
                const int w1 = min(t0 + nt / NW * (wave + 1) + min(nt % NW, wave + 1), visible);
                auto stage = [&](int t, int buf) {
                    const int left = sp.lk - t * kUnit;
                    st.template load<0>(lds + buf * 2 * TILE,
                                        kbase + uint64_t(t) * kUnit * st.stride[0], left);
                    st.template load<1>(lds + buf * 2 * TILE + TILE,
                                        vbase + uint64_t(t) * kUnit * st.stride[1], left);
                };
                Frag<T, DP> qf;
                load_frag<T, DP>(
                    qf,
                    live ? reinterpret_cast<const T *>(row_ptr<T>(a.q, sp.q0 + row, head)) : nullptr,
                    a.dim, half);
                if (w1 > w0)
                    stage(w1 - 1, 0);
                auto repair = [&](int begin) {
                    repair_hidden<T, DP, 1, 1, false>(
                        sm.o, qf, qf, kbase, vbase, st.stride[0], st.stride[1], begin * kUnit,
                        min(w1 * kUnit, sp.lk), RowTerms{last, sm.m, 0.0f, c}, a.dim, half);
                };
                for (int j = 0; j < w1 - w0; ++j) {
                    const int t = w1 - 1 - j;
                    // the stage filled next was read last round: those reads are over
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    if (t > w0) {
                        stage(t - 1, (j + 1) & 1);
                        dma_wait<2 * Stager<T, DP, kUnit, 1>::COPIES>();
                    } else {
                        dma_wait<0>();
                    }
                    const char *kt = own + (j & 1) * 2 * TILE;
                    const bool cut = t * kUnit + kUnit - 1 > tile_first;
                    if (check && !cut) {
                        repair(t + 1);
                        check = false;
                    }
                    float16v s[1];
                    s[0] = mm_rows<T, DP>(kt, qf, lane);
                    if (cut) {
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            s[0][r] = t * kUnit + acc_row(r, half) <= last ? s[0][r] : -INFINITY;
                    }
                    sm.step(s, c, margin);
                    mm_cols<T, DP>(sm.o, kt + TILE, s[0], lane);
                }
                if (check && w1 > w0)
                    repair(w0);

                // join the waves: each leaves its outputs in its own stages
                const float l = sm.l + swap_halves(sm.l);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                float *mine_o = reinterpret_cast<float *>(own);
#pragma unroll
                for (int d = 0; d < R::BLOCKS; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        mine_o[(d * 32 + acc_row(r, half)) * OP + col] = sm.o[d][r];
                if (half == 0) {
                    stat[wave][0][col] = sm.m;
                    stat[wave][1][col] = l;
                }
                __syncthreads();
                const bool whole = n0 == 0 && n1 == un.keys;
                const int64_t rows = int64_t(sp.lq) * group - int64_t(tile) * kTileRows;
                const int live_rows = rows < kTileRows ? int(rows) : kTileRows;
                float *slot = a.partial + (int64_t(blockIdx.x) * 2 + (n0 == 0 ? 1 : 0)) *
                                              (kTileRows * PART);
                for (int e = threadIdx.x; e < live_rows * DP; e += 64 * NW) {
                    const int r = e / DP, d = e % DP;
                    float m = stat[0][0][r];
#pragma unroll
                    for (int w = 1; w < NW; ++w)
                        m = fmaxf(m, stat[w][0][r]);
                    float sum = 0.0f, o = 0.0f;
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const float mw = stat[w][0][r];
                        const float f = mw == m ? 1.0f : exp2f((mw - m) * c);
                        sum = fmaf(stat[w][1][r], f, sum);
                        o = fmaf(reinterpret_cast<const float *>(smem + w * 4 * TILE)[d * OP + r],
                                 f, o);
                    }
                    if (whole) {
                        const uint32_t pr = uint32_t(tile) * kTileRows + r;
                        const int qr = int(pr / uint32_t(group));
                        const int qh = kv_head * group + int(pr % uint32_t(group));
                        if (d < a.dim)
                            reinterpret_cast<T *>(const_cast<char *>(
                                row_ptr<T>(a.out, sp.q0 + qr, qh)))[d] =
                                from_f32<T>(sum == 0.0f ? 0.0f : o / sum);
                        if (d == 0)
                            a.lse[int64_t(qh) * a.q_tokens + sp.q0 + qr] =
                                sum == 0.0f ? -INFINITY : row_lse<T>(m, sum, a.scale);
                    } else {
                        slot[r * PART + 2 + d] = o;
                        if (d == 0) {
                            slot[r * PART] = m;
                            slot[r * PART + 1] = sum;
                        }
                    }
                }
                __syncthreads();
            }
        }
        base += __builtin_amdgcn_readlane(chunk.upto, 63);
    }
}

// One workgroup per (query token, head): joins the parts that several
// workgroups left of its item, if there are several.  Each wave takes every
// fourth part, four at a time so that their reads overlap.
template <typename T, int DP>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a)
{
    constexpr int NW = split_waves<T, DP>();
    constexpr int PART = DP + 2;
    constexpr int AT_ONCE = 4;
    __shared__ float stat[4][2];
    __shared__ float outs[4][DP];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int token = int(blockIdx.x / a.q_heads), head = int(blockIdx.x % a.q_heads);
    const int group = a.q_heads / a.k_heads;
    const float c = a.scale * kLog2e;

    Chunk chunk;
    chunk.load(a, 0, lane);
    const int units = total_units(a, chunk, lane);
    const Share share(units, a.workers, NW);
    int base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        if (b0 > 0)
            chunk.load(a, b0, lane);
        const uint64_t here =
            __ballot(token >= chunk.span.q0 && token < chunk.span.q0 + chunk.span.lq);
        if (!here) {
            base += __builtin_amdgcn_readlane(chunk.upto, 63);
            continue;
        }
        const int l = __builtin_ctzll(here);
        const Span sp = span_in(chunk.span, l);
        const Units un = units_of(a, sp);
        const uint32_t packed = uint32_t(token - sp.q0) * group + head % group;
        const int tile = int(packed / kTileRows), r = int(packed % kTileRows);
        const int first = base + __builtin_amdgcn_readlane(chunk.upto, l) -
                          __builtin_amdgcn_readlane(chunk.mine, l) +
                          (head / group * un.tiles + tile) * un.keys;
        // (the bounds only matter to offsets that overlap beyond counting)
        const int i0 = max(share.owner(first), 0);
        const int i1 = min(share.owner(first + un.keys - 1), a.workers - 1);
        if (i0 >= i1)
            return;                              // finished where it was computed
        float m = -INFINITY, sum = 0.0f, o[2] = {0.0f, 0.0f};
        for (int i = i0 + wave; i <= i1; i += 4 * AT_ONCE) {
            float pm[AT_ONCE], ps[AT_ONCE], po[AT_ONCE][2];
#pragma unroll
            for (int n = 0; n < AT_ONCE; ++n) {
                const int j = i + 4 * n;
                const bool ok = j <= i1;
                const float *p = a.partial +
                                 (2 * (ok ? j : i0) + (!ok || j == i0 ? 1 : 0)) *
                                     int64_t(kTileRows * PART) + r * PART;
                pm[n] = ok ? p[0] : -INFINITY;
                ps[n] = ok ? p[1] : 0.0f;
                po[n][0] = ok && lane < DP ? p[2 + lane] : 0.0f;
                po[n][1] = ok && lane + 64 < DP ? p[66 + lane] : 0.0f;
            }
            float up = m;
#pragma unroll
            for (int n = 0; n < AT_ONCE; ++n)
                up = fmaxf(up, pm[n]);
            const float f = m == up ? 1.0f : exp2f((m - up) * c);
            sum *= f;
            o[0] *= f;
            o[1] *= f;
#pragma unroll
            for (int n = 0; n < AT_ONCE; ++n) {
                const float g = pm[n] == up ? 1.0f : exp2f((pm[n] - up) * c);
                sum = fmaf(ps[n], g, sum);
                o[0] = fmaf(po[n][0], g, o[0]);
                o[1] = fmaf(po[n][1], g, o[1]);
            }
            m = up;
        }
        if (lane == 0) {
            stat[wave][0] = m;
            stat[wave][1] = sum;
        }
        if (lane < DP)
            outs[wave][lane] = o[0];
        if (lane + 64 < DP)
            outs[wave][lane + 64] = o[1];
        __syncthreads();
        if (int(threadIdx.x) < a.dim) {
            float top = stat[0][0];
#pragma unroll
            for (int w = 1; w < 4; ++w)
                top = fmaxf(top, stat[w][0]);
            float total = 0.0f, out = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float f = stat[w][0] == top ? 1.0f : exp2f((stat[w][0] - top) * c);
                total = fmaf(stat[w][1], f, total);
                out = fmaf(outs[w][threadIdx.x], f, out);
            }
            reinterpret_cast<T *>(const_cast<char *>(row_ptr<T>(a.out, token, head)))[threadIdx.x] =
                from_f32<T>(total == 0.0f ? 0.0f : out / total);
            if (threadIdx.x == 0)
                a.lse[int64_t(head) * a.q_tokens + token] =
                    total == 0.0f ? -INFINITY : row_lse<T>(top, total, a.scale);
        }
        return;
    }
    // the token belongs to no sequence
    if ((a.fill & kFillOut) && int(threadIdx.x) < a.dim)
        reinterpret_cast<T *>(const_cast<char *>(row_ptr<T>(a.out, token, head)))[threadIdx.x] =
            T(0.0f);
    if ((a.fill & kFillLse) && threadIdx.x == 0)
        a.lse[int64_t(head) * a.q_tokens + token] = -INFINITY;
}

template <typename T, int DP>
hipError_t launch(AttendArgs a, hipStream_t s)
{
    attend_split_kernel<T, DP><<<uint32_t(a.workers), 64 * split_waves<T, DP>(), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int64_t rows = int64_t(a.q_tokens) * a.q_heads;
    if (rows > INT32_MAX)
        return hipErrorInvalidValue;
    attend_join_kernel<T, DP><<<uint32_t(rows), 256, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_dim(const AttendArgs &a, hipStream_t s)
{
    if (a.dim <= 32)
        return launch<T, 32>(a, s);
    if (a.dim <= 64)
        return launch<T, 64>(a, s);
    if (a.dim <= 96)
        return launch<T, 96>(a, s);
    return launch<T, 128>(a, s);
}

constexpr int kComputeUnits = 256;

int padded_dim(int dim) { return dim <= 32 ? 32 : dim <= 64 ? 64 : dim <= 96 ? 96 : 128; }

}  // namespace

int attend_split_workers(mdcn_dtype dtype, int dim)
{
    // as many workgroups as fit the chip's LDS together (128 KiB each at a
    // 256- or 512-byte row, less below)
    const int bytes = padded_dim(dim) * (dtype == MDCN_F32 ? 4 : 2);
    return kComputeUnits * (bytes > 128 ? 1 : bytes > 64 ? 2 : 4);
}

// The two kernels' times in us beyond a launch.  The tile kernel on 64 queries takes
// 0.83 for each 128 keys (16 bits, up to 64 channels; 0.62 if four waves share
// them), 1.75 (more channels; 1.35) or, fp32, 3.9 for 64, and runs 256 workgroups at a
// time; the split kernel 1.0, 1.5 or 3.9 for each 32 keys x 32 rows of a wave, 7 for its
// second launch, 3.5 to pass on full tiles of more than 64 channels, and 3.4 ns
// for each row that is joined.  Measured on both sides (split against tile, us, 10
// of the host in both): 32 query and 8 key heads of 128 in bf16, one sequence of 1024
// keys, 1 and 8 queries 18 / 18 and 23 / 18; 8192 keys, 1, 128 and 256 queries 18 / 77,
// 73 / 82 and 125 / 86; eight heads of 64 in f16, 1024 keys 17 / 12, eight sequences
// of 8192 keys, 64 and 128 queries 44 / 50 and 72 / 53; fp32 of 80, 1024 keys, 512
// queries 57 / 68, in eight sequences, 128 queries 105 / 72.
// Only averages are known here: the lengths are on the GPU.
bool attend_prefers_split(mdcn_dtype dtype, const AttendArgs &a)
{
    if (a.batch == 0 || a.q_tokens == 0)
        return false;
    const bool f32 = dtype == MDCN_F32, wide = a.dim > 64;
    const bool four = attend_key_waves(dtype, a) == 4;
    const double queries = double(a.q_tokens) / a.batch, keys = double(a.k_tokens) / a.batch;
    const double tile_rows = queries * (a.q_heads / a.k_heads) / kTileRows;
    const double round = f32 ? 3.9 : wide ? (four ? 1.35 : 1.75) : (four ? 0.62 : 0.83);
    const double blocks = double(a.batch) * a.q_heads * std::ceil(queries / 64);
    const double tile = round * (keys / (f32 ? 64 : 128) + 0.5) * std::ceil(blocks / 256);
    const double units = double(a.batch) * a.k_heads * std::ceil(tile_rows) * (keys / kUnit + 1);
    const double waves = attend_split_workers(dtype, a.dim) * (f32 && wide ? 2 : 4);
    const double split = (f32 ? 3.9 : wide ? 1.5 : 1.0) * std::max(1.0, units / waves) + 7 +
                         (wide ? 3.5 * std::min(1.0, tile_rows) : 0.0) +
                         0.0034 * a.q_tokens * a.q_heads;
    return split < tile;
}

size_t attend_split_bytes(mdcn_dtype dtype, int dim)
{
    return size_t(attend_split_workers(dtype, dim)) * 2 * kTileRows * (padded_dim(dim) + 2) *
           sizeof(float);
}

int attend_split_unit_shift(const AttendArgs &a)
{
    // Units of a batch: at most (row tiles) x (key heads) x (units of all keys).
    const double tiles = double(a.q_tokens) * (a.q_heads / a.k_heads) / kTileRows + a.batch;
    int shift = 0;
    while (tiles * a.k_heads * (double(a.k_tokens >> (5 + shift)) + 1) > 1e9 && shift < 16)
        ++shift;
    return shift;
}

hipError_t launch_attend_split(mdcn_dtype dtype, AttendArgs a, hipStream_t s)
{
    a.unit_shift = attend_split_unit_shift(a);
    switch (dtype) {
    case MDCN_F32:
        return launch_dim<float>(a, s);
    case MDCN_F16:
        return launch_dim<half_t>(a, s);
    default:
        return launch_dim<bf16_t>(a, s);
    }
}

}  // namespace mdcn
