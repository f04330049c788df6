// attend.hip -- attention over packed sequences, forward:
//   s[i][j] = scale * q_i . k_j,  p = softmax over the visible keys,
//   out_i = sum_j p_ij v_j,  lse_i = log(sum_j exp(s_ij))
// Row i of a sequence of lq queries and lk keys sees every key, or (causal)
// the keys j <= i + lk - lq.  A row that sees none gets zeros and -infinity.
//
// A workgroup takes 128 queries of one head, 32 per wave; K and V are staged
// in LDS in tiles of 64 keys (fp32: 32), two stages, one barrier per tile:
// the copies of the next tile run while this one is used.  One pass with the
// running maximum and sum.  The last tile comes first: the tiles
// that a causal mask cuts are then done before the accumulators hold
// anything else, so that what hidden rows of V spoil (0 * infinity) can be
// recomputed from these tiles alone.
#include "attention_common.h"

namespace mdcn {

namespace {

constexpr int kWaves = 4;
constexpr int kRows = 32 * kWaves;

template <typename T> constexpr int tile_keys() { return sizeof(T) == 2 ? 64 : 32; }

template <typename T, int DP>
__global__ __launch_bounds__(64 * kWaves, 2) void attend_kernel(AttendArgs a)
{
    using R = Row<T, DP>;
    constexpr int KB = tile_keys<T>();
    constexpr int NS = KB / 32;
    constexpr int TILE = KB * R::PITCH;
    __shared__ __align__(1024) char smem[4 * TILE];          // K, V, K, V

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int half = lane >> 5;

    // Key heads vary fastest over workgroups: neighbours on one XCD (every
    // eighth workgroup) then read the same keys and values through its L2.
    const int kv_head = blockIdx.x % a.k_heads;
    const int group = a.q_heads / a.k_heads;
    const int head = kv_head * group + (blockIdx.x / a.k_heads) % group;
    int b, tile;
    if (!find_tile(a.batch, int(blockIdx.x / a.q_heads), lane,
                   [&](int i) { return (span_of(a, i).lq + kRows - 1) / kRows; }, b, tile))
        return;
    Span sp = span_of(a, b);
    tile = (sp.lq + kRows - 1) / kRows - 1 - tile;           // long rows first

    const int r0 = tile * kRows + wave * 32;                 // wave's first row
    const int row = r0 + (lane & 31);
    const int shift = sp.lk - sp.lq;
    const bool live = row < sp.lq;
    const int last = a.causal ? row + shift : sp.lk - 1;     // last visible key
    const int block_last =
        a.causal ? min(tile * kRows + kRows, sp.lq) - 1 + shift : sp.lk - 1;
    const int nt = block_last < 0 ? 0 : (block_last + KB) / KB;
    const int wave_last = a.causal ? min(r0 + 31, sp.lq - 1) + shift : sp.lk - 1;
    const int wave_first = a.causal ? r0 + shift : sp.lk - 1;

    Frag<T, DP> qf;
    load_frag<T, DP>(qf, live ? reinterpret_cast<const T *>(row_ptr<T>(a.q, sp.q0 + row, head))
                              : nullptr,
                     a.dim, half);
    const char *kbase = row_ptr<T>(a.k, sp.k0, kv_head);
    const char *vbase = row_ptr<T>(a.v, sp.k0, kv_head);
    Stager<T, DP, KB, kWaves> ks, vs;
    ks.init(a.k.token_stride, a.dim, wave, lane);
    vs.init(a.v.token_stride, a.dim, wave, lane);

    Softmax<T, DP> sm;
    sm.init();
    const float c = a.scale * kLog2e;
    const uint32_t lds = lds_address(smem);
    bool check = a.causal != 0;                              // hidden keys seen so far

    auto stage = [&](int t, int buf) {
        const int left = sp.lk - t * KB;
        ks.load(lds + buf * 2 * TILE, kbase + uint64_t(t * KB) * ks.stride, left);
        vs.load(lds + buf * 2 * TILE + TILE, vbase + uint64_t(t * KB) * vs.stride, left);
    };
    auto repair = [&](int begin) {
        repair_hidden<T, DP>(sm.o, qf, kbase, vbase, ks.stride, vs.stride, begin,
                             min(wave_last + 1, sp.lk), last, sm.m, c, a.dim, half);
    };

    if (nt > 0)
        stage(nt - 1, 0);
    for (int i = 0; i < nt; ++i) {
        const int t = nt - 1 - i;
        dma_wait<0>();
        lds_barrier();
        if (t > 0)
            stage(t - 1, (i + 1) & 1);
        if (t * KB > wave_last)
            continue;                                        // nothing visible to this wave
        const char *kt = smem + (i & 1) * 2 * TILE;
        const bool cut = t * KB + KB - 1 > wave_first;       // some key is hidden to some row
        if (check && !cut) {
            repair((t + 1) * KB);
            check = false;
        }
        float16v s[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n)
            s[n] = mm_rows<T, DP>(kt + n * 32 * R::PITCH, qf, lane);
        if (cut) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    s[n][r] = t * KB + n * 32 + acc_row(r, half) <= last ? s[n][r] : -INFINITY;
        }
        sm.step(s, c);
#pragma unroll
        for (int n = 0; n < NS; ++n)
            mm_cols<T, DP>(sm.o, kt + TILE + n * 32 * R::PITCH, s[n], lane);
    }
    if (check && nt > 0)
        repair(0);

    const float l = sm.l + swap_halves(sm.l);
    if (live) {
        store_cols<T, DP>(
            reinterpret_cast<T *>(const_cast<char *>(row_ptr<T>(a.out, sp.q0 + row, head))), sm.o,
            l == 0.0f ? 0.0f : 1.0f / l, a.dim, half);
        if (half == 0)
            a.lse[int64_t(head) * a.q_tokens + sp.q0 + row] =
                l == 0.0f ? -INFINITY : fmaf(sm.m, a.scale, logf(l));
    }
}

template <typename T, int DP>
hipError_t launch(const AttendArgs &a, hipStream_t s)
{
    const int64_t tiles = int64_t(a.q_tokens / kRows) + (a.batch < a.q_tokens ? a.batch : a.q_tokens);
    const int64_t blocks = tiles * a.q_heads;
    if (blocks > INT32_MAX)
        return hipErrorInvalidValue;
    if (blocks == 0)
        return hipSuccess;
    attend_kernel<T, DP><<<uint32_t(blocks), 64 * kWaves, 0, s>>>(a);
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

}  // namespace

hipError_t launch_attend(mdcn_dtype dtype, const AttendArgs &a, hipStream_t s)
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
