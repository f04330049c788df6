// attend_backward.hip -- gradients of attention over packed sequences.
//
//   p_ij = exp(s_ij - lse_i),  delta_i = sum_d go_id out_id
//   dv_j = sum_i p_ij go_i
//   ds_ij = p_ij (go_i . v_j - delta_i),  dq_i = scale sum_j ds_ij k_j,
//   dk_j = scale sum_i ds_ij q_i       (i over the rows of all heads that share j's head)
// p is recomputed from lse, so nothing of size queries x keys is stored.
//
// Kernels: delta; dk and dv, a workgroup per 128 keys walking over the
// queries of its group's heads, or several that share them, whose sums in the
// workspace a fourth kernel adds up; dq, a workgroup per 128 queries walking over the keys.  Scores and go.v are computed in both (7 products
// instead of 5), in exchange for which no gradient is accumulated through
// memory: no atomics, the same bits every run, one rounding of each gradient.
#include "attention_common.h"

namespace mdcn {

namespace {

constexpr int kWaves = 4;
constexpr int kRows = 32 * kWaves;

template <typename T> constexpr int tile_rows() { return sizeof(T) == 2 ? 64 : 32; }

// delta: 16 lanes per (token, head)
template <typename T>
__global__ __launch_bounds__(256) void attend_delta_kernel(AttendArgs a)
{
    constexpr int E = 16 / sizeof(T);
    const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) >> 4;
    if (i >= int64_t(a.q_tokens) * a.q_heads)
        return;
    const int64_t token = i / a.q_heads;
    const int head = int(i % a.q_heads);
    const T *o = reinterpret_cast<const T *>(row_ptr<T>(a.out, token, head));
    const T *g = reinterpret_cast<const T *>(row_ptr<T>(a.go, token, head));
    float sum = 0.0f;
    for (int d = (threadIdx.x & 15) * E; d < a.dim; d += 16 * E) {
        const Vec16<T> x = load16(o + d), y = load16(g + d);
#pragma unroll
        for (int e = 0; e < E; ++e)
            sum = fmaf(to_f32(x.e[e]), to_f32(y.e[e]), sum);
    }
#pragma unroll
    for (int m = 1; m < 16; m <<= 1)
        sum += __shfl_xor(sum, m, 64);
    if ((threadIdx.x & 15) == 0)
        a.delta[head * int64_t(a.q_tokens) + token] = sum;
}

template <typename T, int DP>
__global__ __launch_bounds__(64 * kWaves, 2) void attend_dq_kernel(AttendArgs a)
{
    using R = Row<T, DP>;
    constexpr int KB = tile_rows<T>();
    constexpr int TILE = KB * R::PITCH;
    __shared__ __align__(1024) char smem[4 * TILE];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int half = lane >> 5;
    const int kv_head = blockIdx.x % a.k_heads;
    const int group = a.q_heads / a.k_heads;
    const int head = kv_head * group + (blockIdx.x / a.k_heads) % group;
    int b, tile;
    if (!find_tile(a.batch, int(blockIdx.x / a.q_heads), lane,
                   [&](int i) { return (span_of(a, i).lq + kRows - 1) / kRows; }, b, tile))
        return;
    const Span sp = span_of(a, b);
    tile = (sp.lq + kRows - 1) / kRows - 1 - tile;
    const int r0 = tile * kRows + wave * 32;
    const int row = r0 + (lane & 31);
    const int shift = sp.lk - sp.lq;
    const bool live = row < sp.lq;
    const int last = a.causal ? row + shift : sp.lk - 1;
    const int block_last = a.causal ? min(tile * kRows + kRows, sp.lq) - 1 + shift : sp.lk - 1;
    const int nt = block_last < 0 ? 0 : (block_last + KB) / KB;
    const int wave_last = a.causal ? min(r0 + 31, sp.lq - 1) + shift : sp.lk - 1;
    const int wave_first = a.causal ? r0 + shift : sp.lk - 1;

    Frag<T, DP> qf, gf;
    const int64_t token = sp.q0 + row;
    load_frag<T, DP>(qf, live ? reinterpret_cast<const T *>(row_ptr<T>(a.q, token, head)) : nullptr,
                     a.dim, half);
    load_frag<T, DP>(gf, live ? reinterpret_cast<const T *>(row_ptr<T>(a.go, token, head)) : nullptr,
                     a.dim, half);
    const int64_t stat = int64_t(head) * a.q_tokens + token;
    float lse2 = live ? a.lse[stat] * kLog2e : 0.0f;
    float delta = live ? a.delta[stat] : 0.0f;
    settle<T, DP>(qf);
    settle<T, DP>(gf);
    settle(lse2);
    settle(delta);
    const char *kbase = row_ptr<T>(a.k, sp.k0, kv_head);
    const char *vbase = row_ptr<T>(a.v, sp.k0, kv_head);
    Stager<T, DP, KB, kWaves> st;
    st.init(a.k.token_stride, a.v.token_stride, a.dim, wave, lane);
    const uint32_t lds = lds_address(smem);
    const float c = a.scale * kLog2e;

    Acc<T, DP> dq;
#pragma unroll
    for (int i = 0; i < R::BLOCKS; ++i)
        dq[i] = (float16v){};
    auto stage = [&](int t, int buf) {
        const int left = sp.lk - t * KB;
        st.template load<0>(lds + buf * 2 * TILE, kbase + uint64_t(t * KB) * st.stride[0], left);
        st.template load<1>(lds + buf * 2 * TILE + TILE, vbase + uint64_t(t * KB) * st.stride[1],
                            left);
    };
    if (nt > 0)
        stage(0, 0);
    for (int t = 0; t < nt; ++t) {
        dma_wait<0>();
        lds_barrier();
        if (t + 1 < nt)
            stage(t + 1, (t + 1) & 1);
        if (t * KB > wave_last)
            continue;
        const char *kt = smem + (t & 1) * 2 * TILE;
        const bool cut = t * KB + KB - 1 > wave_first;
#pragma unroll
        for (int n = 0; n < KB / 32; ++n) {
            const char *kn = kt + n * 32 * R::PITCH;
            float16v s = mm_rows<T, DP>(kn, qf, lane);
            const float16v dp = mm_rows<T, DP>(kn + TILE, gf, lane);
#pragma unroll
            for (int r = 0; r < 16; ++r)
                s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2)) * (dp[r] - delta);
            if (cut) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    s[r] = t * KB + n * 32 + acc_row(r, half) <= last ? s[r] : 0.0f;
            }
            mm_cols<T, DP>(dq, kn, s, lane);
        }
    }
    if (live)
        store_cols<T, DP>(reinterpret_cast<T *>(const_cast<char *>(row_ptr<T>(a.dq, token, head))),
                          dq, a.scale, a.dim, half);
}

template <typename T, int DP>
__global__ __launch_bounds__(64 * kWaves) void attend_dkv_kernel(AttendArgs a)
{
    using R = Row<T, DP>;
    constexpr int QB = tile_rows<T>();
    constexpr int TILE = QB * R::PITCH;
    constexpr int STAGE = 2 * TILE + 512;                  // q, go, then lse and delta
    __shared__ __align__(1024) char smem[2 * STAGE];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int half = lane >> 5;
    const int kv_head = blockIdx.x % a.k_heads;
    const int group = a.q_heads / a.k_heads;
    const int part = (blockIdx.x / a.k_heads) % a.splits;
    int b, tile;
    if (!find_tile(a.batch, int(blockIdx.x / a.k_heads / a.splits), lane,
                   [&](int i) { return (span_of(a, i).k_all + kRows - 1) / kRows; }, b, tile))
        return;
    const Span sp = span_of(a, b);
    const int k0 = tile * kRows + wave * 32;               // wave's first key
    const int key = k0 + (lane & 31);
    const int shift = sp.lk - sp.lq;
    const bool live = key < sp.lk;
    // first query that sees any of the workgroup's keys
    const int q_first = a.causal ? max(0, tile * kRows - shift) : 0;
    const int t0 = q_first / QB;
    const int nt = tile * kRows < sp.lk ? max(0, (sp.lq + QB - 1) / QB - t0) : 0;

    Frag<T, DP> kf, vf;
    load_frag<T, DP>(
        kf, live ? reinterpret_cast<const T *>(row_ptr<T>(a.k, sp.k0 + key, kv_head)) : nullptr,
        a.dim, half);
    load_frag<T, DP>(
        vf, live ? reinterpret_cast<const T *>(row_ptr<T>(a.v, sp.k0 + key, kv_head)) : nullptr,
        a.dim, half);
    Stager<T, DP, QB, kWaves> st;
    st.init(a.q.token_stride, a.go.token_stride, a.dim, wave, lane);
    settle<T, DP>(kf);
    settle<T, DP>(vf);
    const uint32_t lds = lds_address(smem);
    const float c = a.scale * kLog2e;

    Acc<T, DP> dk, dv;
#pragma unroll
    for (int i = 0; i < R::BLOCKS; ++i)
        dk[i] = dv[i] = (float16v){};

    auto stage = [&](int i, int buf) {
        const int head = kv_head * group + i / nt, t = t0 + i % nt;
        const int left = sp.lq - t * QB;
        const uint32_t at = lds + buf * STAGE;
        st.template load<0>(at, row_ptr<T>(a.q, sp.q0, head) + uint64_t(t * QB) * st.stride[0],
                            left);
        st.template load<1>(at + TILE,
                            row_ptr<T>(a.go, sp.q0, head) + uint64_t(t * QB) * st.stride[1], left);
        if (wave < 2) {
            const float *src = (wave == 0 ? a.lse : a.delta) + int64_t(head) * a.q_tokens + sp.q0 +
                               t * QB;
            const v4i r = row_resource(reinterpret_cast<const char *>(src),
                                       uint32_t(left < QB ? left : QB) * 4);
            dma_row4(__builtin_amdgcn_readfirstlane(at + 2 * TILE + wave * 256), r,
                     uint32_t(lane) * 4);
        }
    };
    // this workgroup's part of the (head, tile) pairs
    const int i_begin = int(int64_t(nt) * group * part / a.splits);
    const int i_end = int(int64_t(nt) * group * (part + 1) / a.splits);
    if (i_end > i_begin)
        stage(i_begin, 0);
    for (int i = i_begin; i < i_end; ++i) {
        dma_wait<0>();
        lds_barrier();
        if (i + 1 < i_end)
            stage(i + 1, (i + 1 - i_begin) & 1);
        const int q_tile = (t0 + i % nt) * QB;
        const char *qt = smem + ((i - i_begin) & 1) * STAGE;
        const float *stat = reinterpret_cast<const float *>(qt + 2 * TILE);
#pragma unroll
        for (int n = 0; n < QB / 32; ++n) {
            const int q0 = q_tile + n * 32;
            // sees(q, key): key <= q + shift
            if (a.causal && q0 + 31 + shift < k0)
                continue;                                  // no row sees any of the wave's keys
            const char *qn = qt + n * 32 * R::PITCH;
            float16v s = mm_rows<T, DP>(qn, kf, lane);
            float16v dp = mm_rows<T, DP>(qn + TILE, vf, lane);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float4v ls = *reinterpret_cast<const float4v *>(stat + n * 32 + 8 * g + 4 * half);
                const float4v de =
                    *reinterpret_cast<const float4v *>(stat + 64 + n * 32 + 8 * g + 4 * half);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[4 * g + j] = __builtin_amdgcn_exp2f(fmaf(s[4 * g + j], c, -ls[j] * kLog2e));
                    dp[4 * g + j] = s[4 * g + j] * (dp[4 * g + j] - de[j]);
                }
            }
            if (a.causal && q0 + shift < k0 + 31) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const bool sees = key <= q0 + acc_row(r, half) + shift;
                    s[r] = sees ? s[r] : 0.0f;
                    dp[r] = sees ? dp[r] : 0.0f;
                }
            }
            mm_cols<T, DP>(dv, qn + TILE, s, lane);
            mm_cols<T, DP>(dk, qn, dp, lane);
        }
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
            store_cols<float, DP>(sum, dk, 1.0f, a.dim, half);
            store_cols<float, DP>(sum + rows * a.dim, dv, 1.0f, a.dim, half);
            return;
        }
        T *dst = reinterpret_cast<T *>(const_cast<char *>(row_ptr<T>(a.dk, sp.k0 + key, kv_head)));
        store_cols<T, DP>(dst, dk, a.scale, a.dim, half);
        dst = reinterpret_cast<T *>(const_cast<char *>(row_ptr<T>(a.dv, sp.k0 + key, kv_head)));
        store_cols<T, DP>(dst, dv, 1.0f, a.dim, half);
    }
}

constexpr int kSumRows = 16;

// Adds the parts [part][dk, dv][key head][token][dim] of the keys of every
// sequence, 16 keys a workgroup.
template <typename T>
__global__ __launch_bounds__(256) void attend_dkv_sum_kernel(AttendArgs a)
{
    const int kv_head = blockIdx.x % a.k_heads;
    int b, tile;
    if (!find_tile(a.batch, int(blockIdx.x / a.k_heads), threadIdx.x & 63,
                   [&](int i) { return (span_of(a, i).k_all + kSumRows - 1) / kSumRows; }, b, tile))
        return;
    const Span sp = span_of(a, b);
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

template <typename T, int DP>
hipError_t launch(const AttendArgs &a, hipStream_t s)
{
    const int64_t rows = int64_t(a.q_tokens) * a.q_heads;
    const int64_t q_blocks = tiles_of(a.q_tokens, a.batch, kRows) * a.q_heads;
    const int64_t k_tiles = tiles_of(a.k_tokens, a.batch, kRows) * a.k_heads;
    const int64_t k_blocks = k_tiles * a.splits;
    const int64_t sum_blocks = tiles_of(a.k_tokens, a.batch, kSumRows) * a.k_heads;
    if (sum_blocks > INT32_MAX || (rows + 15) / 16 > INT32_MAX || q_blocks > INT32_MAX || k_blocks > INT32_MAX)
        return hipErrorInvalidValue;
    if (rows > 0)
        attend_delta_kernel<T><<<uint32_t((rows + 15) / 16), 256, 0, s>>>(a);
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
        attend_dq_kernel<T, DP><<<uint32_t(q_blocks), 64 * kWaves, 0, s>>>(a);
        e = hipGetLastError();
    }
    return e;
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

int attend_backward_splits(mdcn_dtype dtype, const AttendArgs &a)
{
    // Enough workgroups for two on each of the 256 compute units, with at
    // least two tiles of queries to each (a part costs its sums' way through memory).
    const int64_t tiles = tiles_of(a.k_tokens, a.batch, kRows) * a.k_heads;
    const int64_t queries = int64_t(a.q_heads / a.k_heads) * a.q_tokens /
                            ((dtype == MDCN_F32 ? 32 : 64) * int64_t(a.batch > 0 ? a.batch : 1));
    int64_t n = tiles > 0 ? (512 + tiles - 1) / tiles : 1;
    n = n < queries / 2 ? n : queries / 2;
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
