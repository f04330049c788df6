// attend.hip -- attention over packed sequences, forward:
//   s[i][j] = scale * q_i . k_j,  p = softmax over the visible keys,
//   out_i = sum_j p_ij v_j,  lse_i = log(sum_j exp(s_ij))
// Row i of a sequence of lq queries and lk keys sees every key, or (causal)
// the keys j <= i + lk - lq.  A row that sees none gets zeros and -infinity.
//
// A workgroup takes 32 * RW queries of one head, 32 per wave, with KW waves to
// each 32 that share the keys; K and V are staged in LDS, 64 keys a wave (fp32:
// 32), two stages, one barrier per tile: the copies of the next tile run
// while this one is used.  One pass with the running maximum and sum.  The
// last tile comes first: the tiles that a causal mask cuts are then done before
// the accumulators hold anything else, so that what hidden rows of V spoil
// (0 * infinity) can be recomputed from these tiles alone.
//
// Bound by the matrix cores and the vector units in turn (a wave's tile of 64
// keys at 128 channels: 32 MFMAs of 32 cycles, 32 exponentials and ~150 other
// vector instructions), two waves a SIMD, and by the card's power.  One MI355X,
// bf16, 32 query and 8 key heads of 128: sequences of 4096 to 1 tokens, causal,
// 223 to 227 us among other work (830 TFLOP/s of the visible pairs), 250 in a row;
// 4096 x 4096 full 283 us (970), 16384 x 4096 1035 (1063), with zeros in place of
// random values 226 and 851, as a large matrix product does (769 against 608).  Not kept,
// with no gain: the next tile's scores computed among this one's exponentials,
// instruction by instruction; wave priorities; eight waves of 256 queries (6% slower);
// heads dealt over the XCDs otherwise.
#include "attention_common.h"

namespace mdcn {

namespace {

template <typename T, int DP, int RW, int KW>
__global__ __launch_bounds__(64 * RW * KW, (waves_per_simd<T, DP, KW>())) void attend_kernel(
    AttendArgs a)
{
    using R = Row<T, DP>;
    constexpr int ROWS = 32 * RW;
    constexpr int KB = tile_keys<T, DP, KW>();   // keys of a wave's part of a tile
    constexpr int NS = KB / 32;
    constexpr int KT = KB * KW;                  // keys of a tile
    constexpr int PART = KB * R::PITCH;
    constexpr int TILE = KT * R::PITCH;
    // reads of a tile ahead of their uses (fp32 rows would take twice the registers)
    constexpr bool AHEAD = sizeof(T) == 2;
    __shared__ __align__(1024) char smem[4 * TILE];          // K, V, K, V

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int rg = wave % RW, kg = wave / RW;
    const int half = lane >> 5;

    if (int(blockIdx.x) >= a.fill_from) {
        const int part = int(blockIdx.x) - a.fill_from, parts = int(gridDim.x) - a.fill_from;
        if (a.fill & kFillOut)
            zero_outside<T>(a.out, a.cu_q, a.batch, a.q_tokens, a.q_heads, a.dim, part, parts);
        if (a.fill & kFillLse)
            outside_rows(a.cu_q, a.batch, a.q_tokens, a.q_heads, part, parts, [&](int t, int h) {
                a.lse[int64_t(h) * a.q_tokens + t] = -INFINITY;
            });
        return;
    }

    // Key heads vary fastest over workgroups: neighbours on one XCD (every
    // eighth workgroup) then read the same keys and values through its L2.
    const int kv_head = blockIdx.x % a.k_heads;
    const int group = a.q_heads / a.k_heads;
    const int head = kv_head * group + (blockIdx.x / a.k_heads) % group;
    Span sp;
    int tile;
    if (!find_tile(a, int(blockIdx.x / a.q_heads), lane, a.causal,
                   [](const Span &s) { return (s.lq + ROWS - 1) / ROWS; }, sp, tile))
        return;

    const int r0 = tile * ROWS + rg * 32;                    // wave's first row
    const int row = r0 + (lane & 31);
    const int shift = sp.lk - sp.lq;
    const bool live = row < sp.lq;
    const int last = a.causal ? row + shift : sp.lk - 1;     // last visible key
    const int block_last = a.causal ? min(tile * ROWS + ROWS, sp.lq) - 1 + shift : sp.lk - 1;
    const int nt = block_last < 0 ? 0 : block_last / KT + 1;
    const int wave_last = a.causal ? min(r0 + 31, sp.lq - 1) + shift : sp.lk - 1;
    const int wave_first = a.causal ? r0 + shift : sp.lk - 1;

    const char *kbase = row_ptr<T>(a.k, sp.k0, kv_head);
    const char *vbase = row_ptr<T>(a.v, sp.k0, kv_head);
    Stager<T, DP, KT, RW * KW> st;
    st.init(a.k.token_stride, a.v.token_stride, a.dim, wave, lane);
    const uint32_t lds = lds_address(smem);
    // round i handles tile nt - 1 - i, in stage i & 1
    auto stage = [&](int i) {
        const int t = nt - 1 - i;
        const uint32_t at = lds + (i & 1) * 2 * TILE;
        st.template load<0>(at, kbase + uint64_t(t * KT) * st.stride[0], sp.lk - t * KT);
        st.template load<1>(at + TILE, vbase + uint64_t(t * KT) * st.stride[1], sp.lk - t * KT);
    };
    if (nt > 0)
        stage(0);

    Frag<T, DP> qf;
    load_frag<T, DP>(qf, live ? reinterpret_cast<const T *>(row_ptr<T>(a.q, sp.q0 + row, head))
                              : nullptr,
                     a.dim, half);
    settle<T, DP>(qf);
    Softmax<T, DP> sm;
    sm.init();
    const float c = a.scale * kLog2e, margin = raise_margin(c);
    bool check = a.causal != 0;                              // hidden keys seen so far
    auto repair = [&](int i) {
        // this wave's keys of the rounds before i, one round at a time
        repair_hidden<T, DP, KB, KT, false>(
            sm.o, qf, qf, kbase, vbase, st.stride[0], st.stride[1], (nt - i) * KT + kg * KB,
            min(wave_last + 1, sp.lk), RowTerms{last, sm.m, 0.0f, c}, a.dim, half);
    };

    for (int i = 0; i < nt; ++i) {
        const int key0 = (nt - 1 - i) * KT + kg * KB;        // wave's first key of this round
        dma_wait<0>();
        lds_barrier();
        if (i + 1 < nt)
            stage(i + 1);
        if (key0 > wave_last)
            continue;                                        // hidden from every row
        const bool cut = key0 + KB - 1 > wave_first;         // some key is hidden to some row
        if (check && !cut) {
            repair(i);
            check = false;
        }
        const char *kt = smem + (i & 1) * 2 * TILE + kg * PART;
        const char *vt = kt + TILE;
        float16v s[NS];
        Cols<T, DP> vf;
        if constexpr (AHEAD) {
            Frag<T, DP> kf[NS];
#pragma unroll
            for (int n = 0; n < NS; ++n)
                load_rows<T, DP>(kf[n], kt + n * 32 * R::PITCH, lane);
            reads_first();
#pragma unroll
            for (int n = 0; n < NS; ++n)
                s[n] = mm_rows<T, DP>(kf[n], qf);
            vf.load(vt, lane);
            reads_first();
        } else {
#pragma unroll
            for (int n = 0; n < NS; ++n)
                s[n] = mm_rows<T, DP>(kt + n * 32 * R::PITCH, qf, lane);
        }
        if (cut) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    s[n][r] = key0 + n * 32 + acc_row(r, half) <= last ? s[n][r] : -INFINITY;
        }
        sm.step(s, c, margin);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            if constexpr (AHEAD) {
                Cols<T, DP> next;
                if (n + 1 < NS) {
                    next.load(vt + (n + 1) * 32 * R::PITCH, lane);
                    reads_first();
                }
                mm_cols<T, DP>(sm.o, vf, s[n]);
                if (n + 1 < NS)
                    vf = next;
            } else {
                mm_cols<T, DP>(sm.o, vt + n * 32 * R::PITCH, s[n], lane);
            }
        }
    }
    if (check && nt > 0)
        repair(nt);

    float l = sm.l + swap_halves(sm.l);
    if constexpr (KW > 1) {
        // join the waves that shared a row's keys: all but the first leave
        // their sums in LDS
        static_assert((KW - 1) * RW * (DP + 2) * 32 * 4 <= 4 * TILE, "the sums fit the stages");
        __syncthreads();
        float *sums = reinterpret_cast<float *>(smem);
        auto at = [&](int g) { return sums + ((g - 1) * RW + rg) * (DP + 2) * 32 + (lane & 31); };
        if (kg > 0) {
            float *p = at(kg);
#pragma unroll
            for (int d = 0; d < R::BLOCKS; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    p[(d * 32 + acc_row(r, half)) * 32] = sm.o[d][r];
            if (half == 0) {
                p[DP * 32] = sm.m;
                p[(DP + 1) * 32] = l;
            }
        }
        __syncthreads();
        if (kg > 0)
            return;
#pragma unroll 1
        for (int g = 1; g < KW; ++g) {
            const float *p = at(g);
            const float m = p[DP * 32], up = fmaxf(sm.m, m);
            const float f = sm.m == up ? 1.0f : exp2f((sm.m - up) * c);
            const float h = m == up ? 1.0f : exp2f((m - up) * c);
#pragma unroll
            for (int d = 0; d < R::BLOCKS; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    sm.o[d][r] = sm.o[d][r] * f + p[(d * 32 + acc_row(r, half)) * 32] * h;
            l = l * f + p[(DP + 1) * 32] * h;
            sm.m = up;
        }
    }
    if (live) {
        store_cols<T, DP>(
            reinterpret_cast<T *>(const_cast<char *>(row_ptr<T>(a.out, sp.q0 + row, head))), sm.o,
            l == 0.0f ? 0.0f : 1.0f / l, a.dim, half);
        if (half == 0)
            a.lse[int64_t(head) * a.q_tokens + sp.q0 + row] =
                l == 0.0f ? -INFINITY : row_lse<T>(sm.m, l, a.scale);
    }
}

template <typename T, int DP, int RW, int KW>
hipError_t launch_shape(AttendArgs a, hipStream_t s)
{
    constexpr int ROWS = 32 * RW;
    const int64_t tiles = int64_t(a.q_tokens / ROWS) + (a.batch < a.q_tokens ? a.batch : a.q_tokens);
    int64_t blocks = tiles * a.q_heads;
    a.fill_from = blocks < INT32_MAX ? int(blocks) : INT32_MAX;
    if (a.fill)
        blocks += fill_blocks(int64_t(a.q_tokens) * a.q_heads * a.dim * sizeof(T));
    if (blocks > INT32_MAX)
        return hipErrorInvalidValue;
    if (blocks == 0)
        return hipSuccess;
    attend_kernel<T, DP, RW, KW><<<uint32_t(blocks), 64 * RW * KW, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, int DP> hipError_t launch(const AttendArgs &a, hipStream_t s)
{
    const int waves = attend_key_waves(sizeof(T) == 4 ? MDCN_F32 : MDCN_F16, a);
    if constexpr (sizeof(T) == 2)
        if (waves == 4)
            return launch_shape<T, DP, 2, 4>(a, s);
    return waves == 2 ? launch_shape<T, DP, 2, 2>(a, s) : launch_shape<T, DP, 4, 1>(a, s);
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

int attend_key_waves(mdcn_dtype dtype, const AttendArgs &a)
{
    // Up to one workgroup of 128 queries a compute unit, workgroups of 64
    // queries, two waves to the keys of each 32, spread further and end sooner
    // (208 workgroups of eight f16 heads of 64: 20.8 us against 26.8; fp32, 48
    // workgroups: 26 against 40).  Beyond, they stage twice the keys a
    // query (528 workgroups of bf16 heads of 128: 75 us against 55).
    if ((int64_t(a.q_tokens) / 128 + 1) * a.q_heads > 256)
        return 1;
    // Of those, four waves to the keys fill a compute unit that has no second
    // workgroup to run (bf16, one sequence, eight heads of 128, 1500 tokens: 23.9 us
    // against 29.7, dq 28.9 against 33.2; 16 heads, 700 tokens, causal: 17.0 against 18.8)
    // if the keys are many (200 and fewer: 8.4 against 7.6) and the workgroups no
    // more than the compute units (448: 26.4 against 19.6).  In fp32 a single wave
    // keeps the matrix cores busy (32.2 against 33.0, dq 41.5 against 40.6).
    const int64_t batch = a.batch < a.q_tokens ? a.batch : a.q_tokens;
    const int64_t blocks = (int64_t(a.q_tokens) / 64 + batch) * a.q_heads;
    return dtype != MDCN_F32 && blocks <= 256 && a.k_tokens >= 512 * int64_t(a.batch) ? 4 : 2;
}

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
