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

// Units of sequence b: `keys` per (key head, row tile), at least one.
struct Units {
    int tiles, keys;
    int64_t all;
};

__device__ __forceinline__ Units units_of(const AttendArgs &a, const Span &s)
{
    Units u;
    u.tiles = int((int64_t(s.lq) * (a.q_heads / a.k_heads) + kTileRows - 1) / kTileRows);
    u.keys = s.lk > 0 ? (s.lk + kUnit - 1) / kUnit : 1;
    u.all = int64_t(u.tiles) * a.k_heads * u.keys;
    return u;
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int l)
{
    const int lo = __shfl(int(uint32_t(v)), l, 64), hi = __shfl(int(v >> 32), l, 64);
    return int64_t(uint64_t(uint32_t(hi)) << 32 | uint32_t(lo));
}

__device__ __forceinline__ int64_t scan64(int64_t v, int lane)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int64_t o = shfl64(v, lane - m);
        v += lane >= m ? o : 0;
    }
    return v;
}

__device__ __forceinline__ int64_t total_units(const AttendArgs &a, int lane)
{
    int64_t sum = 0;
    for (int b = lane; b < a.batch; b += 64)
        sum += units_of(a, span_of(a, b)).all;
    return shfl64(scan64(sum, lane), 63);
}

// Workgroups that share the units: enough units for all waves of each.
__device__ __forceinline__ int64_t sharers(int64_t units, int workers, int waves)
{
    const int64_t most = (units + waves - 1) / waves;
    return most < workers ? most : workers;
}

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
    const float c = a.scale * kLog2e;

    const int64_t units = total_units(a, lane);
    const int64_t share = sharers(units, a.workers, NW);
    if (int64_t(blockIdx.x) >= share)
        return;
    const int64_t u_end = units * (int64_t(blockIdx.x) + 1) / share;
    const int64_t u_begin = units * int64_t(blockIdx.x) / share;

    Stager<T, DP, kUnit, 1> ks, vs;
    ks.init(a.k.token_stride, a.dim, 0, lane);
    vs.init(a.v.token_stride, a.dim, 0, lane);
    char *own = smem + wave * 4 * TILE;
    const uint32_t lds = lds_address(own);

    int64_t base = 0;
    for (int b0 = 0; b0 < a.batch && base < u_end; b0 += 64) {
        const int64_t mine = b0 + lane < a.batch ? units_of(a, span_of(a, b0 + lane)).all : 0;
        const int64_t upto = scan64(mine, lane);
        for (int i = 0; i < 64 && b0 + i < a.batch; ++i) {
            const int64_t s_end = base + shfl64(upto, i);
            const int64_t s_begin = s_end - shfl64(mine, i);
            if (s_end <= u_begin || s_begin >= u_end)
                continue;
            const int b = b0 + i;
            const Span sp = span_of(a, b);
            const Units un = units_of(a, sp);
            const int shift = sp.lk - sp.lq;
            const int64_t from = u_begin > s_begin ? u_begin : s_begin;
            const int64_t to = u_end < s_end ? u_end : s_end;
            for (int64_t u = from; u < to;) {
                // item: a (key head, row tile) of this sequence; keys [n0, n1) of it, in units
                const int item = int((u - s_begin) / un.keys);
                const int64_t i_begin = s_begin + int64_t(item) * un.keys;
                const int n0 = int(u - i_begin);
                const int n1 = int((to < i_begin + un.keys ? to : i_begin + un.keys) - i_begin);
                u = i_begin + n1;
                const int kv_head = item / un.tiles;
                const int tile = item % un.tiles;

                const int64_t packed = int64_t(tile) * kTileRows + col;
                const int row = int(packed / group);
                const int head = kv_head * group + int(packed % group);
                const bool live = row < sp.lq;
                const int last = a.causal ? row + shift : sp.lk - 1;
                const int tile_first =
                    a.causal ? int(int64_t(tile) * kTileRows / group) + shift : sp.lk - 1;
                const int tile_last =
                    a.causal ? min(int((int64_t(tile) * kTileRows + 31) / group), sp.lq - 1) + shift
                             : sp.lk - 1;

                Frag<T, DP> qf;
                load_frag<T, DP>(
                    qf,
                    live ? reinterpret_cast<const T *>(row_ptr<T>(a.q, sp.q0 + row, head)) : nullptr,
                    a.dim, half);
                const char *kbase = row_ptr<T>(a.k, sp.k0, kv_head);
                const char *vbase = row_ptr<T>(a.v, sp.k0, kv_head);
                Softmax<T, DP> sm;
                sm.init();
                bool check = a.causal != 0;

                // this wave's units, from the last one down (see attend.hip)
                const int w0 = n0 + int(int64_t(n1 - n0) * wave / NW);
                const int visible = tile_last < 0 ? 0 : tile_last / kUnit + 1;
                const int w1 = min(n0 + int(int64_t(n1 - n0) * (wave + 1) / NW), visible);
                auto stage = [&](int t, int buf) {
                    const int left = sp.lk - t * kUnit;
                    ks.load(lds + buf * 2 * TILE, kbase + uint64_t(t) * kUnit * ks.stride, left);
                    vs.load(lds + buf * 2 * TILE + TILE, vbase + uint64_t(t) * kUnit * vs.stride,
                            left);
                };
                auto repair = [&](int begin) {
                    repair_hidden<T, DP>(sm.o, qf, kbase, vbase, ks.stride, vs.stride,
                                         begin * kUnit, min(w1 * kUnit, sp.lk), last, sm.m, c,
                                         a.dim, half);
                };
                if (w1 > w0)
                    stage(w1 - 1, 0);
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
                    sm.step(s, c);
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
                        const int64_t pr = int64_t(tile) * kTileRows + r;
                        const int qr = int(pr / group), qh = kv_head * group + int(pr % group);
                        if (d < a.dim)
                            reinterpret_cast<T *>(const_cast<char *>(
                                row_ptr<T>(a.out, sp.q0 + qr, qh)))[d] =
                                from_f32<T>(sum == 0.0f ? 0.0f : o / sum);
                        if (d == 0)
                            a.lse[int64_t(qh) * a.q_tokens + sp.q0 + qr] =
                                sum == 0.0f ? -INFINITY : fmaf(m, a.scale, logf(sum));
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
        base += shfl64(upto, 63);
    }
}

// One wave per (query token, head): joins the parts that several workgroups
// left of its item, if there are several.
template <typename T, int DP>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a)
{
    constexpr int NW = split_waves<T, DP>();
    constexpr int PART = DP + 2;
    const int lane = threadIdx.x & 63;
    const int64_t w = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (w >= int64_t(a.q_tokens) * a.q_heads)
        return;
    const int token = int(w / a.q_heads), head = int(w % a.q_heads);
    const int group = a.q_heads / a.k_heads;

    const int64_t units = total_units(a, lane);
    const int64_t share = sharers(units, a.workers, NW);
    int64_t base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        Span mine = {};
        int64_t n = 0;
        if (b0 + lane < a.batch) {
            mine = span_of(a, b0 + lane);
            n = units_of(a, mine).all;
        }
        const int64_t upto = scan64(n, lane);
        const uint64_t here = __ballot(token >= mine.q0 && token < mine.q0 + mine.lq);
        if (here) {
            const int l = __builtin_ctzll(here);
            const Span sp = span_of(a, b0 + l);
            const Units un = units_of(a, sp);
            const int64_t packed = int64_t(token - sp.q0) * group + head % group;
            const int tile = int(packed / kTileRows), r = int(packed % kTileRows);
            const int64_t first = base + shfl64(upto, l) - shfl64(n, l) +
                                  (int64_t(head / group) * un.tiles + tile) * un.keys;
            const int64_t i0 = ((first + 1) * share - 1) / units;
            const int64_t i1 = ((first + un.keys) * share - 1) / units;
            if (i0 == i1)
                return;
            const float c = a.scale * kLog2e;
            float m = -INFINITY, sum = 0.0f, o[2] = {0.0f, 0.0f};
            for (int64_t i = i0; i <= i1; ++i) {
                const float *p = a.partial + (2 * i + (i == i0 ? 1 : 0)) * (kTileRows * PART) +
                                 r * PART;
                const float pm = p[0], up = fmaxf(m, pm);
                const float f = m == up ? 1.0f : exp2f((m - up) * c);
                const float g = pm == up ? 1.0f : exp2f((pm - up) * c);
                sum = sum * f + p[1] * g;
                o[0] = o[0] * f + (lane < DP ? p[2 + lane] * g : 0.0f);
                if (DP > 64)
                    o[1] = o[1] * f + (lane + 64 < DP ? p[2 + 64 + lane] * g : 0.0f);
                m = up;
            }
            T *dst = reinterpret_cast<T *>(const_cast<char *>(row_ptr<T>(a.out, token, head)));
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (lane + 64 * k < a.dim)
                    dst[lane + 64 * k] = from_f32<T>(sum == 0.0f ? 0.0f : o[k] / sum);
            if (lane == 0)
                a.lse[int64_t(head) * a.q_tokens + token] =
                    sum == 0.0f ? -INFINITY : fmaf(m, a.scale, logf(sum));
            return;
        }
        base += shfl64(upto, 63);
    }
}

template <typename T, int DP>
hipError_t launch(AttendArgs a, hipStream_t s)
{
    attend_split_kernel<T, DP><<<uint32_t(a.workers), 64 * split_waves<T, DP>(), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int64_t waves = int64_t(a.q_tokens) * a.q_heads;
    if ((waves + 3) / 4 > INT32_MAX)
        return hipErrorInvalidValue;
    attend_join_kernel<T, DP><<<uint32_t((waves + 3) / 4), 256, 0, s>>>(a);
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

size_t attend_split_bytes(mdcn_dtype dtype, int dim)
{
    return size_t(attend_split_workers(dtype, dim)) * 2 * kTileRows * (padded_dim(dim) + 2) *
           sizeof(float);
}

hipError_t launch_attend_split(mdcn_dtype dtype, const AttendArgs &a, hipStream_t s)
{
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
