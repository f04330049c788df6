// attend_backward.hip -- gradients of attention over packed sequences.
//
//   p_ij = exp(s_ij - lse_i),  delta_i = sum_d go_id out_id
//   dv_j = sum_i p_ij go_i
//   ds_ij = p_ij (go_i . v_j - delta_i),  dq_i = scale sum_j ds_ij k_j,
//   dk_j = scale sum_i ds_ij q_i       (i over the rows of all heads that share j's head)
// p is recomputed from lse, so nothing of size queries x keys is stored.
//
// Kernels: delta; dk and dv, a workgroup per 128 keys walking over the queries of
// its group's heads, or several that share them, whose sums in the workspace a
// fourth kernel adds up; dq, a workgroup per 128 queries walking over the keys.
// Scores and go.v are computed in both (7 products instead of 5), in exchange for
// which no gradient is accumulated through memory: no atomics, the same bits
// every run, one rounding of each gradient.
//
// One MI355X, bf16, 16 query and 4 key heads of 128, 4096 x 4096 full: dk and dv
// 320 us (860 TFLOP/s of its four products), dq 188 us (1100 of its three).
// Sequences of 2048 to 1 tokens, causal: 14 + 90 + 13 + 67 us, where the
// longest rows of tiles and the start of a workgroup (about 8 us) bound it: 592
// workgroups cannot be spread evenly.
#include "attention_common.h"

namespace mdcn {

namespace {

constexpr int kWaves = 4;
constexpr int kRows = 32 * kWaves;

constexpr int kFar = 1 << 30;                 // more than any number of rows

// fp16 holds 2^-24 to 2^16, and probabilities p and score gradients p (go.v - delta)
// are often outside: among 2^14 keys p is about 2^-14, and go has any size.  Both are
// scaled by powers of two before they are rounded, which changes nothing else: p to
// 2^15 p, the score gradients by what takes
//   |go.v - delta| <= dim max|go| max|v| + max|delta|
// to at most 2^15.  The maxima are those of the rows that a sum runs over (values that
// are not finite left out), taken in the first kernel 32 rows at a time.  Cost of it all
// (16 query and 4 key heads of 128, the training step above): 176 -> 179 us; 64 sequences of
// 200, eight heads of 64: 63 -> 68.
template <typename T> constexpr bool kScaled = false;
template <> constexpr bool kScaled<half_t> = true;
constexpr int kTop = 15;

// The exponent of the scale for score gradients of at most `bound`.
__device__ __forceinline__ int scale_exponent(float bound)
{
    return bound > 0.0f ? kTop - __builtin_amdgcn_frexp_expf(bound) : 0;
}

// The largest finite |x| of a row's half that the lane holds.
template <typename T, int DP> __device__ __forceinline__ float top_of_row(const Frag<T, DP> &f)
{
    uint32_t top = 0;
    auto take = [&](uint32_t w) {
        const uint32_t lo = w & 0x7fff, hi = w >> 16 & 0x7fff;
        top = max(top, max(lo < 0x7c00 ? lo : 0, hi < 0x7c00 ? hi : 0));
    };
#pragma unroll
    for (int k = 0; k < Row<T, DP>::STEPS; ++k) {
        take(f[k].x);
        take(f[k].y);
        take(f[k].z);
        take(f[k].w);
    }
    const uint16_t bits = uint16_t(top);
    half_t v;
    __builtin_memcpy(&v, &bits, 2);
    return float(v);
}

__device__ __forceinline__ float finite_or_0(float v) { return fabsf(v) < INFINITY ? fabsf(v) : 0.0f; }

__device__ __forceinline__ float wave_top(float v)
{
#pragma unroll
    for (int m = 32; m > 0; m >>= 1)
        v = fmaxf(v, __shfl_xor(v, m));
    return v;
}

// {lse in powers of two, delta} of every (token, head): the diagonal of go.out for
// 32 rows of a head a wave.  On the matrix cores not for their rate (the reads
// bound it), but to add in the order in which the other kernels add go.v: a row that
// sees one key has out = v, and its ds is then exactly zero, as it should be.
//
// out has been rounded, and its error is in every score gradient of its row: little
// among many keys, but of the size of all other roundings together in rows that see
// few (causal sequences of 8 rows, bf16: dq off by 0.0029 instead of 0.0024, of which
// the rounding of dq itself is 0.0016).  In 16 bits rows that see 2 to 32 keys
// take sum(p go.v) over these instead, one more product of 32 keys a wave.
template <typename T, int DP>
__global__ __launch_bounds__(256) void attend_delta_kernel(AttendArgs a)
{
    if (int(blockIdx.x) >= a.fill_from) {
        // gradients of tokens that belong to no sequence
        const int part = int(blockIdx.x) - a.fill_from, parts = int(gridDim.x) - a.fill_from;
        zero_outside<T>(a.dq, a.cu_q, a.batch, a.q_tokens, a.q_heads, a.dim, part, parts);
        zero_outside<T>(a.dk, a.cu_k, a.batch, a.k_tokens, a.k_heads, a.dim, part, parts);
        zero_outside<T>(a.dv, a.cu_k, a.batch, a.k_tokens, a.k_heads, a.dim, part, parts);
        return;
    }
    const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31;
    Span sp;
    int tile;
    if (kScaled<T> && int(blockIdx.x) >= a.tops_from) {
        const int w = int((blockIdx.x - a.tops_from) * 4 +
                          __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)));
        const int kv_head = w % a.k_heads;
        if (!find_tile(a, w / a.k_heads, lane, false,
                       [](const Span &s) { return (s.lk + 31) / 32; }, sp, tile))
            return;
        const int key = tile * 32 + col;
        Frag<T, DP> v;
        load_frag<T, DP>(
            v, key < sp.lk ? reinterpret_cast<const T *>(row_ptr<T>(a.v, sp.k0 + key, kv_head)) : nullptr,
            a.dim, half);
        const float top = wave_top(top_of_row<T, DP>(v));
        if (lane == 0)
            a.key_tops[int64_t(kv_head) * a.k_tokens + sp.k0 + tile * 32] = top;
        return;
    }
    const int w = int(blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)));
    const int head = w % a.q_heads;
    if (!find_tile(a, w / a.q_heads, lane, false, [](const Span &s) { return (s.lq + 31) / 32; },
                   sp, tile))
        return;
    const int row = tile * 32 + col;
    const int64_t token = sp.q0 + row;
    const bool live = row < sp.lq;
    const int last = a.causal ? row + sp.lk - sp.lq : sp.lk - 1;
    const int64_t at = head * int64_t(a.q_tokens) + token;
    const float lse = live ? a.lse[at] * kLog2e : 0.0f;
    Frag<T, DP> g, o;
    load_frag<T, DP>(g, live ? reinterpret_cast<const T *>(row_ptr<T>(a.go, token, head)) : nullptr,
                     a.dim, half);
    load_frag<T, DP>(o, live ? reinterpret_cast<const T *>(row_ptr<T>(a.out, token, head)) : nullptr,
                     a.dim, half);
    const float16v d = mm_rows<T, DP>(g, o);
    float delta = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r)
        delta = acc_row(r, half) == col ? d[r] : delta;
    const bool few = sizeof(T) == 2 && live && last > 0 && last < 32;
    if (sizeof(T) == 2 && __any(few)) {
        const int kv_head = head / (a.q_heads / a.k_heads);
        const bool held = col < sp.lk;
        Frag<T, DP> q, kv;
        load_frag<T, DP>(
            q, live ? reinterpret_cast<const T *>(row_ptr<T>(a.q, token, head)) : nullptr, a.dim,
            half);
        load_frag<T, DP>(
            kv, held ? reinterpret_cast<const T *>(row_ptr<T>(a.k, sp.k0 + col, kv_head)) : nullptr,
            a.dim, half);
        const float16v s = mm_rows<T, DP>(kv, q);
        load_frag<T, DP>(
            kv, held ? reinterpret_cast<const T *>(row_ptr<T>(a.v, sp.k0 + col, kv_head)) : nullptr,
            a.dim, half);
        const float16v dp = mm_rows<T, DP>(kv, g);
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float p = __builtin_amdgcn_exp2f(fmaf(s[r], a.scale * kLog2e, -lse));
            sum += acc_row(r, half) <= last ? p * dp[r] : 0.0f;
        }
        sum += __shfl_xor(sum, 32);
        delta = few ? sum : delta;
    }
    if (live && half == (col >> 2 & 1))
        a.stats[at] = make_float2(kScaled<T> ? lse - kTop : lse, delta);
    if constexpr (kScaled<T>) {
        // (the lane of the other half holds no delta of its row)
        const bool own = live && half == (col >> 2 & 1);
        const float top_g = wave_top(top_of_row<T, DP>(g));
        const float top_d = wave_top(own ? finite_or_0(delta) : 0.0f);
        if (lane == 0)
            a.row_tops[head * int64_t(a.q_tokens) + sp.q0 + tile * 32] = make_float2(top_g, top_d);
    }
}

template <typename T, int DP, int RW, int KW>
__global__ __launch_bounds__(64 * RW * KW, (waves_per_simd<T, DP, KW>())) void attend_dq_kernel(
    AttendArgs a)
{
    using R = Row<T, DP>;
    constexpr int ROWS = 32 * RW;
    constexpr int KB = tile_keys<T, DP, KW>();   // keys of a wave's part of a tile
    constexpr int KT = KB * KW;                  // keys of a tile
    constexpr int PART = KB * R::PITCH;
    constexpr int TILE = KT * R::PITCH;
    constexpr bool AHEAD = sizeof(T) == 2;       // as in attend.hip
    __shared__ __align__(1024) char smem[4 * TILE];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int rg = wave % RW, kg = wave / RW;
    const int half = lane >> 5;
    const int kv_head = blockIdx.x % a.k_heads;
    const int group = a.q_heads / a.k_heads;
    const int head = kv_head * group + (blockIdx.x / a.k_heads) % group;
    Span sp;
    int tile;
    if (!find_tile(a, int(blockIdx.x / a.q_heads), lane, a.causal,
                   [](const Span &s) { return (s.lq + ROWS - 1) / ROWS; }, sp, tile))
        return;
    const int r0 = tile * ROWS + rg * 32;
    const int row = r0 + (lane & 31);
    const int shift = sp.lk - sp.lq;
    const bool live = row < sp.lq;
    const int last = a.causal ? row + shift : sp.lk - 1;
    const int block_last = a.causal ? min(tile * ROWS + ROWS, sp.lq) - 1 + shift : sp.lk - 1;
    const int nt = block_last < 0 ? 0 : block_last / KT + 1;
    const int wave_last = a.causal ? min(r0 + 31, sp.lq - 1) + shift : sp.lk - 1;
    const int wave_first = a.causal ? r0 + shift : sp.lk - 1;

    const char *kbase = row_ptr<T>(a.k, sp.k0, kv_head);
    const char *vbase = row_ptr<T>(a.v, sp.k0, kv_head);
    Stager<T, DP, KT, RW * KW> st;
    st.init(a.k.token_stride, a.v.token_stride, a.dim, wave, lane);
    const uint32_t lds = lds_address(smem);
    // round i handles tile nt - 1 - i, in stage i & 1: the tiles that a causal
    // mask cuts come first (see repair_hidden)
    auto stage = [&](int i) {
        const int t = nt - 1 - i;
        const int left = sp.lk - t * KT;
        const uint32_t at = lds + (i & 1) * 2 * TILE;
        st.template load<0>(at, kbase + uint64_t(t * KT) * st.stride[0], left);
        st.template load<1>(at + TILE, vbase + uint64_t(t * KT) * st.stride[1], left);
    };
    if (nt > 0)
        stage(0);

    Frag<T, DP> qf, gf;
    const int64_t token = sp.q0 + row;
    load_frag<T, DP>(qf, live ? reinterpret_cast<const T *>(row_ptr<T>(a.q, token, head)) : nullptr,
                     a.dim, half);
    load_frag<T, DP>(gf, live ? reinterpret_cast<const T *>(row_ptr<T>(a.go, token, head)) : nullptr,
                     a.dim, half);
    float2 stat = make_float2(0.0f, 0.0f);
    if (live)
        stat = a.stats[int64_t(head) * a.q_tokens + token];
    settle<T, DP>(qf);
    settle<T, DP>(gf);
    settle(stat.x);
    settle(stat.y);
    const float c = a.scale * kLog2e;
    float factor = a.scale;
    if constexpr (kScaled<T>) {
        // a row's own scale, which goes into its exponent: e^(s - lse) 2^x
        float top = 0.0f;
        const int keys = min(block_last + 1, sp.lk);
        const float *tops = a.key_tops + int64_t(kv_head) * a.k_tokens + sp.k0;
        for (int j = lane * 32; j < keys; j += 64 * 32)
            top = fmaxf(top, tops[j]);
        top = wave_top(top);
        const int x = scale_exponent(float(a.dim) * top * max_halves(top_of_row<T, DP>(gf)) +
                                     finite_or_0(stat.y));
        stat.x += float(kTop - x);
        factor = ldexpf(a.scale, -x);
    }

    Acc<T, DP> dq;
#pragma unroll
    for (int i = 0; i < R::BLOCKS; ++i)
        dq[i] = (float16v){};
    bool check = a.causal != 0;                              // hidden keys seen so far
    auto repair = [&](int i) {
        repair_hidden<T, DP, KB, KT, true>(
            dq, qf, gf, kbase, vbase, st.stride[0], st.stride[1], (nt - i) * KT + kg * KB,
            min(wave_last + 1, sp.lk), RowTerms{last, stat.x, stat.y, c}, a.dim, half);
    };
    for (int i = 0; i < nt; ++i) {
        dma_wait<0>();
        lds_barrier();
        if (i + 1 < nt)
            stage(i + 1);
        const int key0 = (nt - 1 - i) * KT + kg * KB;
        if (key0 > wave_last)
            continue;
        const char *kt = smem + (i & 1) * 2 * TILE + kg * PART;
        const bool cut = key0 + KB - 1 > wave_first;
        if (check && !cut) {
            repair(i);
            check = false;
        }
#pragma unroll
        for (int n = 0; n < KB / 32; ++n) {
            const char *kn = kt + n * 32 * R::PITCH;
            float16v s, dp;
            Cols<T, DP> kc;
            if constexpr (AHEAD) {
                Frag<T, DP> f;
                load_rows<T, DP>(f, kn, lane);
                reads_first();
                s = mm_rows<T, DP>(f, qf);
                load_rows<T, DP>(f, kn + TILE, lane);
                reads_first();
                dp = mm_rows<T, DP>(f, gf);
                kc.load(kn, lane);
                reads_first();
            } else {
                s = mm_rows<T, DP>(kn, qf, lane);
                dp = mm_rows<T, DP>(kn + TILE, gf, lane);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r)
                s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -stat.x)) * (dp[r] - stat.y);
            if (cut) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    s[r] = key0 + n * 32 + acc_row(r, half) <= last ? s[r] : 0.0f;
            }
            if constexpr (AHEAD)
                mm_cols<T, DP>(dq, kc, s);
            else
                mm_cols<T, DP>(dq, kn, s, lane);
        }
    }
    if (check && nt > 0)
        repair(nt);
    if constexpr (KW > 1) {
        // the sums of the waves that shared a row's keys, through LDS
        static_assert((KW - 1) * RW * DP * 32 * 4 <= 4 * TILE, "the sums fit the stages");
        __syncthreads();
        float *sums = reinterpret_cast<float *>(smem);
        auto at = [&](int g) { return sums + ((g - 1) * RW + rg) * DP * 32 + (lane & 31); };
        if (kg > 0) {
            float *p = at(kg);
#pragma unroll
            for (int d = 0; d < R::BLOCKS; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    p[(d * 32 + acc_row(r, half)) * 32] = dq[d][r];
        }
        __syncthreads();
        if (kg > 0)
            return;
#pragma unroll 1
        for (int g = 1; g < KW; ++g) {
            const float *p = at(g);
#pragma unroll
            for (int d = 0; d < R::BLOCKS; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    dq[d][r] += p[(d * 32 + acc_row(r, half)) * 32];
        }
    }
    if (live)
        store_cols<T, DP>(reinterpret_cast<T *>(const_cast<char *>(row_ptr<T>(a.dq, token, head))),
                          dq, factor, a.dim, half);
}

// One round of a wave on 32 queries and its 32 keys, the instructions in the
// order in which they are to run: the products q.k and go.v of the next 32
// queries (rows at `q_next`, `g_next`), with the probabilities p and ds of
// these ones computed between them; then p and ds times these queries' go and
// q.  A wave has its SIMD to itself (it holds 2 x 32 x DP sums and its keys
// and values in registers), so nothing else hides the vector work or LDS: each
// MFMA comes with a read eight MFMAs ahead of its use and a share of the vector
// instructions, and the scheduler may not move them.  The causal mask is always
// applied: two more vector instructions a score fit under the MFMAs, and a
// branch around them would have the sums moved between registers every round.
template <typename T, int DP>
__device__ __forceinline__ void dkv_round(Acc<T, DP> &dk, Acc<T, DP> &dv, float16v &s, float16v &dp,
                                          const Frag<T, DP> &kf, const Frag<T, DP> &vf,
                                          const char *q_next, const char *g_next,
                                          const char *q_tile, const char *g_tile,
                                          const float *stats, float c, float ds_scale,
                                          int first_row, int lane)
{
    using R = Row<T, DP>;
    constexpr int RM = 2 * R::STEPS;                       // row products
    constexpr int CM = 2 * R::BLOCKS * (32 / R::KROWS);    // column products
    constexpr int AHEAD = 8 < RM ? 8 : 4;
    const int half = lane >> 5;
    uint4 w[AHEAD];
    auto read = [&](int k) -> uint4 {
        if (k < RM)
            return row_frag<T, DP>(k < R::STEPS ? q_next : g_next, k % R::STEPS, lane);
        const int j = k - RM, d = j % (2 * R::BLOCKS);
        return col_frag<T, DP>(d < R::BLOCKS ? g_tile : q_tile, j / (2 * R::BLOCKS),
                               d % R::BLOCKS, lane);
    };
    float4v st[8];                                         // {lse, delta} of two rows each
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        w[k] = read(k);
#pragma unroll
    for (int g = 0; g < 8; ++g)
        st[g] = *reinterpret_cast<const float4v *>(stats + 2 * acc_row(2 * g, half));
    __builtin_amdgcn_sched_barrier(0);
    float16v ns = {}, ndp = {};
#pragma unroll
    for (int k = 0; k < RM; ++k) {
        if (k < R::STEPS)
            ns = Mma<T>::step(w[k % AHEAD], kf[k], ns);
        else
            ndp = Mma<T>::step(w[k % AHEAD], vf[k - R::STEPS], ndp);
        w[k % AHEAD] = read(k + AHEAD);
#pragma unroll
        for (int r = 16 * k / RM; r < 16 * (k + 1) / RM; ++r) {
            // rows before first_row do not see the lane's key: p = 2^-infinity
            const float lse =
                acc_row(r, 0) >= first_row - 4 * half ? st[r / 2][2 * r % 4] : INFINITY;
            s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse));
            dp[r] = dp[r] - st[r / 2][2 * r % 4 + 1];
            dp[r] = s[r] * (kScaled<T> ? dp[r] * ds_scale : dp[r]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    uint4 pp, pd;
#pragma unroll
    for (int j = 0; j < CM; ++j) {
        const int step = j / (2 * R::BLOCKS), d = j % (2 * R::BLOCKS);
        if (d == 0) {
            pp = pack_p<T>(s, step * R::KROWS / 2);
            pd = pack_p<T>(dp, step * R::KROWS / 2);
        }
        if (d < R::BLOCKS)
            dv[d] = Mma<T>::step(w[(RM + j) % AHEAD], pp, dv[d]);
        else
            dk[d - R::BLOCKS] = Mma<T>::step(w[(RM + j) % AHEAD], pd, dk[d - R::BLOCKS]);
        if (j + AHEAD < CM)
            w[(RM + j) % AHEAD] = read(RM + j + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
    }
    s = ns;
    dp = ndp;
}

template <typename T, int DP>
__global__ __launch_bounds__(64 * kWaves) void attend_dkv_kernel(AttendArgs a)
{
    using R = Row<T, DP>;
    constexpr int TILE = 32 * R::PITCH;
    constexpr int STAGE = 2 * TILE + 256;                  // q, go, then {lse, delta}
    constexpr int STAGES = 4;
    __shared__ __align__(1024) char smem[STAGES * STAGE];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int half = lane >> 5;
    const int kv_head = blockIdx.x % a.k_heads;
    const int group = a.q_heads / a.k_heads;
    const int part = (blockIdx.x / a.k_heads) % a.splits;
    Span sp;
    int tile;
    if (!find_tile(a, int(blockIdx.x / a.k_heads / a.splits), lane, a.causal,
                   [](const Span &s) { return (s.k_all + kRows - 1) / kRows; }, sp, tile))
        return;
    tile = (sp.k_all + kRows - 1) / kRows - 1 - tile;       // the first keys are seen by most rows
    const int k0 = tile * kRows + wave * 32;               // wave's first key
    const int key = k0 + (lane & 31);
    const int shift = sp.lk - sp.lq;
    const bool live = key < sp.lk;
    // first query that sees any of the workgroup's keys
    const int q_first = a.causal ? max(0, tile * kRows - shift) : 0;
    const int t0 = q_first / 32;
    const int nt = tile * kRows < sp.lk ? max(0, (sp.lq + 31) / 32 - t0) : 0;
    // this workgroup's part of the (head, 32 queries) pairs
    const int i_begin = int(int64_t(nt) * group * part / a.splits);
    const int i_end = int(int64_t(nt) * group * (part + 1) / a.splits);

    // waves 0 and 1 stage the queries, 2 and 3 their gradients; the rounds are
    // staged in order, so the next one's addresses are kept and stepped
    const Heads &src = wave < 2 ? a.q : a.go;
    Stager<T, DP, 32, 2> st;
    st.init(src.token_stride, src.token_stride, a.dim, wave & 1, lane);
    const int rows_step = 32 * int(st.stride[0]);
    int s_head = kv_head * group, s_t = 0, s_stage = 0;
    const char *s_row = nullptr;
    const float2 *s_stat = nullptr;
    auto stage_at = [&](int head, int t) {
        s_head = head;
        s_t = t;
        s_row = row_ptr<T>(src, sp.q0, head) + int64_t(t) * rows_step;
        s_stat = a.stats + int64_t(head) * a.q_tokens + sp.q0 + t * 32;
    };
    if (i_end > i_begin)
        stage_at(kv_head * group + i_begin / nt, t0 + i_begin % nt);
    const uint32_t lds = lds_address(smem) + (wave < 2 ? 0 : TILE);
    auto stage = [&]() {
        const int left = sp.lq - s_t * 32;
        st.template load<0>(lds + s_stage, s_row, left);
        if (wave == 0)
            dma_row4(__builtin_amdgcn_readfirstlane(lds + s_stage + 2 * TILE),
                     row_resource(reinterpret_cast<const char *>(s_stat),
                                  uint32_t(left < 32 ? left : 32) * 8),
                     uint32_t(lane) * 4);
        s_stage = s_stage == (STAGES - 1) * STAGE ? 0 : s_stage + STAGE;
        if (s_t + 1 < t0 + nt) {
            ++s_t;
            s_row += rows_step;
            s_stat += 32;
        } else {
            stage_at(s_head + 1, t0);
        }
    };
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (i_begin + i < i_end)
            stage();

    Frag<T, DP> kf, vf;
    load_frag<T, DP>(
        kf, live ? reinterpret_cast<const T *>(row_ptr<T>(a.k, sp.k0 + key, kv_head)) : nullptr,
        a.dim, half);
    load_frag<T, DP>(
        vf, live ? reinterpret_cast<const T *>(row_ptr<T>(a.v, sp.k0 + key, kv_head)) : nullptr,
        a.dim, half);
    settle<T, DP>(kf);
    settle<T, DP>(vf);
    const float c = a.scale * kLog2e;
    float ds_scale = 1.0f, dk_factor = 1.0f, dv_factor = 1.0f;
    if constexpr (kScaled<T>) {
        // a key's own scale, beyond that of p
        float top_g = 0.0f, top_d = 0.0f;
        for (int i = i_begin + lane; i < i_end; i += 64) {
            const float2 t = a.row_tops[int64_t(kv_head * group + i / nt) * a.q_tokens + sp.q0 +
                                        (t0 + i % nt) * 32];
            top_g = fmaxf(top_g, t.x);
            top_d = fmaxf(top_d, t.y);
        }
        const int x = scale_exponent(float(a.dim) * wave_top(top_g) *
                                         max_halves(top_of_row<T, DP>(vf)) +
                                     wave_top(top_d));
        ds_scale = ldexpf(1.0f, x - kTop);
        dk_factor = ldexpf(1.0f, -x);
        dv_factor = ldexpf(1.0f, -kTop);
    }

    Acc<T, DP> dk, dv;
#pragma unroll
    for (int i = 0; i < R::BLOCKS; ++i)
        dk[i] = dv[i] = (float16v){};
    float16v s = {}, dp = {};
    if (i_end > i_begin) {
        dma_wait<0>();
        lds_barrier();
        s = mm_rows<T, DP>(smem, kf, lane);
        dp = mm_rows<T, DP>(smem + TILE, vf, lane);
    }
    int t = i_end > i_begin ? t0 + i_begin % nt : 0;
    int at = 0;
    for (int i = i_begin; i < i_end; ++i) {
        // the next 32 queries have landed; those after them may be on their way
        if (i + 2 < i_end)
            dma_wait<Stager<T, DP, 32, 2>::COPIES>();
        else
            dma_wait<0>();
        lds_barrier();
        if (i + 3 < i_end)
            stage();
        const char *q_tile = smem + at;
        at = at == (STAGES - 1) * STAGE ? 0 : at + STAGE;
        const char *q_next = smem + at;                      // past the end: not used
        const float *stats = reinterpret_cast<const float *>(q_tile + 2 * TILE);
        // sees(q, key): key <= q + shift
        dkv_round<T, DP>(dk, dv, s, dp, kf, vf, q_next, q_next + TILE, q_tile, q_tile + TILE, stats,
                         c, ds_scale, a.causal ? key - shift - t * 32 : -kFar, lane);
        t = t + 1 < t0 + nt ? t + 1 : t0;
    }
    if (key < sp.k_all) {
        // keys that are not used get zeros, whatever the sums hold
        if (!live) {
#pragma unroll
            for (int i = 0; i < R::BLOCKS; ++i)
                dk[i] = dv[i] = (float16v){};
        }
        if (a.splits > 1) {
            const int64_t rows = int64_t(a.k_tokens) * a.k_heads;
            float *sum = a.partial + (2 * part * rows + int64_t(kv_head) * a.k_tokens + sp.k0 +
                                      key) * a.dim;
            store_cols<float, DP>(sum, dk, dk_factor, a.dim, half);
            store_cols<float, DP>(sum + rows * a.dim, dv, dv_factor, a.dim, half);
            return;
        }
        T *dst = reinterpret_cast<T *>(const_cast<char *>(row_ptr<T>(a.dk, sp.k0 + key, kv_head)));
        store_cols<T, DP>(dst, dk, a.scale * dk_factor, a.dim, half);
        dst = reinterpret_cast<T *>(const_cast<char *>(row_ptr<T>(a.dv, sp.k0 + key, kv_head)));
        store_cols<T, DP>(dst, dv, dv_factor, a.dim, half);
    }
}

constexpr int kSumRows = 16;

// Adds the parts [part][dk, dv][key head][token][dim] of the keys of every
// sequence, 16 keys a workgroup.
template <typename T>
__global__ __launch_bounds__(256) void attend_dkv_sum_kernel(AttendArgs a)
{
    const int kv_head = blockIdx.x % a.k_heads;
    Span sp;
    int tile;
    if (!find_tile(a, int(blockIdx.x / a.k_heads), threadIdx.x & 63, false,
                   [](const Span &s) { return (s.k_all + kSumRows - 1) / kSumRows; }, sp, tile))
        return;
    const int vecs = a.dim / 4;
    const int rows = min(kSumRows, sp.k_all - tile * kSumRows);
    const int64_t all = int64_t(a.k_tokens) * a.k_heads * a.dim;
    for (int e = threadIdx.x; e < 2 * rows * vecs; e += 256) {
        const int which = e / (rows * vecs), rest = e % (rows * vecs);
        const int row = rest / vecs, d = rest % vecs * 4;
        const int64_t token = sp.k0 + tile * kSumRows + row;
        const float *src = a.partial + which * all +
                           (int64_t(kv_head) * a.k_tokens + token) * a.dim + d;
        float4v sum = *reinterpret_cast<const float4v *>(src);
        for (int n = 1; n < a.splits; ++n)
            sum += *reinterpret_cast<const float4v *>(src + 2 * n * all);
        const float f = which == 0 ? a.scale : 1.0f;
        T *dst = reinterpret_cast<T *>(const_cast<char *>(
                     row_ptr<T>(which == 0 ? a.dk : a.dv, token, kv_head))) + d;
        struct alignas(4 * sizeof(T)) {
            T e[4];
        } v;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v.e[j] = from_f32<T>(sum[j] * f);
        __builtin_memcpy(__builtin_assume_aligned(dst, 4 * sizeof(T)), &v, sizeof(v));
    }
}

// At least the tiles of `rows` rows of any `batch` sequences.
int64_t tiles_of(int64_t tokens, int64_t batch, int rows)
{
    return tokens / rows + (batch < tokens ? batch : tokens);
}

template <typename T, int DP, int RW, int KW>
hipError_t launch_shape(AttendArgs a, hipStream_t s)
{
    const int64_t d_blocks = (tiles_of(a.q_tokens, a.batch, 32) * a.q_heads + 3) / 4;
    const int64_t q_blocks = tiles_of(a.q_tokens, a.batch, 32 * RW) * a.q_heads;
    const int64_t k_tiles = tiles_of(a.k_tokens, a.batch, kRows) * a.k_heads;
    const int64_t k_blocks = k_tiles * a.splits;
    const int64_t sum_blocks = tiles_of(a.k_tokens, a.batch, kSumRows) * a.k_heads;
    if (sum_blocks > INT32_MAX || q_blocks > INT32_MAX || k_blocks > INT32_MAX)
        return hipErrorInvalidValue;
    a.tops_from = int(d_blocks);
    const int64_t v_blocks =
        kScaled<T> ? (tiles_of(a.k_tokens, a.batch, 32) * a.k_heads + 3) / 4 : 0;
    if (4 * (d_blocks + v_blocks) > INT32_MAX)
        return hipErrorInvalidValue;
    a.fill_from = int(d_blocks + v_blocks);
    const int fill = fill_blocks((int64_t(a.q_tokens) * a.q_heads + 2 * int64_t(a.k_tokens) * a.k_heads) *
                                 a.dim * sizeof(T));
    attend_delta_kernel<T, DP><<<uint32_t(a.fill_from + fill), 256, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && k_blocks > 0) {
        attend_dkv_kernel<T, DP><<<uint32_t(k_blocks), 64 * kWaves, 0, s>>>(a);
        e = hipGetLastError();
        if (e == hipSuccess && a.splits > 1) {
            attend_dkv_sum_kernel<T><<<uint32_t(sum_blocks), 256, 0, s>>>(a);
            e = hipGetLastError();
        }
    }
    if (e == hipSuccess && q_blocks > 0) {
        attend_dq_kernel<T, DP, RW, KW><<<uint32_t(q_blocks), 64 * RW * KW, 0, s>>>(a);
        e = hipGetLastError();
    }
    return e;
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

int attend_backward_splits(const AttendArgs &a)
{
    // Enough workgroups for nearly two on each of the 256 compute units (dk and dv of
    // the training step above: 296 workgroups 151 us, 444 109, 592 91; the last few
    // are not worth a third on some: fp32, 1000 queries, 504 workgroups 39 us,
    // 576 46).  At least 3/2 times 32 queries to each, as a part costs its sums'
    // way through memory (fp32, 400 and fewer queries, 64 tiles: twice 44.6 + 5.5 us,
    // 3/2 times 38.3 + 6.6, once 44.8 + 8.6).
    const int64_t tiles = tiles_of(a.k_tokens, a.batch, kRows) * a.k_heads;
    const int64_t queries = int64_t(a.q_heads / a.k_heads) * a.q_tokens /
                            (32 * int64_t(a.batch > 0 ? a.batch : 1));
    int64_t n = tiles > 0 ? (480 + tiles - 1) / tiles : 1;
    const int64_t most = (2 * queries + 2) / 3;
    n = n < most ? n : most;
    return int(n < 1 ? 1 : n > 8 ? 8 : n);
}

hipError_t launch_attend_backward(mdcn_dtype dtype, const AttendArgs &a, hipStream_t s)
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
