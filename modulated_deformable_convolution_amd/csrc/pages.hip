// pages.hip -- pages of a cache shared, given, taken back, moved and copied.
//
// The bookkeeping reads tables and counts of a few bytes a page, so its time is that of
// the round trips to memory between its steps: where tables and pool are small one workgroup does
// all steps, otherwise each step is a launch over the chip.  The pages themselves are copied
// by a kernel of their own, bound by memory.  Free pages are taken and pages moved in ascending
// order, by counts and ranks of chunks of 1024 pages; the only atomics are on whole numbers,
// whose order does not matter.
#include <algorithm>

#include "cache_common.h"

namespace mdcn {

namespace {

constexpr int kChunk = 1024;                     // pages of a chunk, threads of a workgroup
constexpr int kWavesOfChunk = kChunk / 64;

// The threads that share a step: one workgroup, or the grid.
struct Team {
    int tid, n;                                  // of the team
    int group, groups;                           // workgroup, workgroups
};

__device__ __forceinline__ Team team()
{
    return Team{int(blockIdx.x * kChunk + threadIdx.x), int(gridDim.x * kChunk), int(blockIdx.x),
                int(gridDim.x)};
}

// What other threads counted with atomics, past this compute unit's cache.
__device__ __forceinline__ int32_t counted(const int32_t *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Sums of v over the workgroup's threads up to this one; `all` becomes the sum over all.
__device__ __forceinline__ int group_scan(int v, int *lds, int &all)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int upto = wave_scan(v);
    if (lane == 63)
        lds[wave] = upto;
    __syncthreads();
    int before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kWavesOfChunk; ++w) {
        before += w < wave ? lds[w] : 0;
        all += lds[w];
    }
    __syncthreads();
    return before + upto;
}

int chunks_of(int pages) { return (pages + kChunk - 1) / kChunk; }

size_t up_16(size_t n) { return (n + 15) / 16 * 16; }

// ---- copies ----------------------------------------------------------------

constexpr int kSegment = 16384;                  // most bytes of a workgroup's turn

__host__ __device__ __forceinline__ int segments_of(int page_bytes)
{
    return (page_bytes + kSegment - 1) / kSegment;
}

// Page src[i] to dst[i] in every layer, i < count (or *counter, if there is one); the
// segments of a page are alike.  Past the caches, a turn a workgroup: 601 pages of 34 KB in 12
// layers 92 us (5.5 TB/s read and written, part of it from the last-level cache: 4 GiB of such pages
// in any order 4.8), through the caches or with 4096 workgroups of several turns 102, both 106.
// A page is a workgroup's turn however small: 1 GiB in pages of 4352 bytes at 4.9 TB/s, of 2176 at 3.7, of
// 1088 at 2.3, of 544 at 1.3.
__global__ __launch_bounds__(256) void copy_pages_kernel(PoolView from, PoolView to,
                                                         const int32_t *src, const int32_t *dst,
                                                         int count, const int32_t *counter)
{
    typedef uint32_t v4u __attribute__((ext_vector_type(4)));
    if (counter)
        count = min(count, *counter);
    const int segments = segments_of(from.page_bytes);
    const int size = (from.page_bytes / 16 + segments - 1) / segments * 16;
    const int64_t turns = int64_t(count) * from.layers * segments;
    for (int64_t t = blockIdx.x; t < turns; t += gridDim.x) {
        const int64_t pair = t / segments;
        const int seg = int(t - pair * segments);
        const int layer = int(pair / count), i = int(pair - int64_t(layer) * count);
        const int s = src[i], d = dst[i];
        if (s < 0 || s >= from.pages || d < 0 || d >= to.pages)
            continue;
        const int64_t begin = int64_t(seg) * size;
        const char *p = from.data + layer * from.layer_stride + s * from.page_stride + begin;
        char *q = to.data + layer * to.layer_stride + d * to.page_stride + begin;
        const int bytes = int(min(int64_t(size), from.page_bytes - begin));
        v4u v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = (k * 256 + int(threadIdx.x)) * 16;
            if (at < bytes)
                v[k] = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(p + at));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = (k * 256 + int(threadIdx.x)) * 16;
            if (at < bytes)
                __builtin_nontemporal_store(v[k], reinterpret_cast<v4u *>(q + at));
        }
    }
}

hipError_t launch_copies(const PoolView &from, const PoolView &to, const int32_t *src,
                         const int32_t *dst, int count, const int32_t *counter, hipStream_t s)
{
    const int64_t turns = int64_t(count) * from.layers * segments_of(from.page_bytes);
    if (turns == 0)
        return hipSuccess;
    const int blocks = int(std::min<int64_t>(turns, 65536));
    copy_pages_kernel<<<blocks, 256, 0, s>>>(from, to, src, dst, count, counter);
    return hipGetLastError();
}

// ---- fork ------------------------------------------------------------------

struct ForkState {
    int32_t *first;        // [rows_in] the first row that goes on from this one
    int32_t *fresh;        // [rows_out] pages that rows before this one take
    int32_t *copies;       // [rows_out] copies that rows before this one make
    int32_t *src, *dst;    // [rows_out] the copies
    int32_t *chunk;        // [chunks] free pages of a chunk, then those before it
    int32_t *free;         // [pages] the free pages that are taken
    int32_t *totals;       // copies, pages taken
};

struct ForkRow {
    int parent;            // -1: none
    int used, held, wants; // tokens and pages of the parent, pages of the result (used and
                           // new tokens count in 32 bits: a row holds 2^30 tokens at most)
    int excess;            // pages that the table has no room for (never more than new ones)
    int new_tokens;
    bool own;              // the last page held is a copy
};

__device__ __forceinline__ ForkRow fork_row(const PagesArgs &a, int i)
{
    ForkRow r;
    const int p = a.parents ? a.parents[i] : i;
    r.parent = p >= 0 && p < a.rows_in ? p : -1;
    r.used = r.parent < 0 ? 0 : int(min(int64_t(max(a.used[r.parent], 0)),
                                        int64_t(a.width) * a.page));
    r.new_tokens = a.new_tokens ? max(a.new_tokens[i], 0) : 0;
    r.held = int((uint32_t(r.used) + a.page - 1) / uint32_t(a.page));
    const uint32_t all = (uint32_t(r.used) + uint32_t(r.new_tokens) + a.page - 1) / uint32_t(a.page);
    r.wants = int(min(all, uint32_t(a.width)));
    r.excess = int(all - uint32_t(r.wants));
    r.own = false;
    return r;
}

__device__ __forceinline__ bool is_page(const PagesArgs &a, int p)
{
    return p >= 0 && p < a.pool.pages;
}

// The row's last page is a copy: it is full in part, and another row keeps it.
__device__ __forceinline__ bool copies_last(const PagesArgs &a, const ForkState &f, const ForkRow &r,
                                            int i)
{
    return r.parent >= 0 && r.used % a.page != 0 && counted(f.first + r.parent) != i &&
           is_page(a, a.table[int64_t(r.parent) * a.width + r.held - 1]);
}

__device__ void fork_init(const PagesArgs &a, const ForkState &f, const Team &t)
{
    for (int p = t.tid; p < a.pool.pages; p += t.n)
        a.owners_out[p] = a.owners[p];
    for (int r = t.tid; r < a.rows_in; r += t.n)
        f.first[r] = INT32_MAX;
}

__device__ void fork_first(const PagesArgs &a, const ForkState &f, const Team &t)
{
    for (int i = t.tid; i < a.rows_out; i += t.n) {
        const ForkRow r = fork_row(a, i);
        a.used_out[i] = int(min(int64_t(r.used) + r.new_tokens, int64_t(a.width) * a.page));
        if (r.parent >= 0)
            atomicMin(f.first + r.parent, i);
    }
}

// Entries that rows share with their parents; the counts follow where an entry of the
// result differs from the table's in the same place.
__device__ void fork_share(const PagesArgs &a, const ForkState &f, const Team &t)
{
    const uint32_t entries = uint32_t(max(a.rows_in, a.rows_out)) * a.width;
    for (uint32_t e = t.tid; e < entries; e += t.n) {
        const int i = int(e / uint32_t(a.width)), j = int(e - uint32_t(i) * a.width);
        const int old = i < a.rows_in ? a.table[e] : -1;
        int now = -1;
        if (i < a.rows_out) {
            const ForkRow r = fork_row(a, i);
            if (j < r.held && !(j == r.held - 1 && copies_last(a, f, r, i)))
                now = a.table[int64_t(r.parent) * a.width + j];
            if (!is_page(a, now))
                now = -1;
            a.table_out[e] = now;
        }
        if (old != now) {
            if (is_page(a, old))
                atomicAdd(a.owners_out + old, -1);
            if (now >= 0)
                atomicAdd(a.owners_out + now, 1);
        }
    }
}

__device__ void fork_count(const PagesArgs &a, const ForkState &f, const Team &t, int *lds)
{
    for (int c = t.group; c < (a.pool.pages + kChunk - 1) / kChunk; c += t.groups) {
        const int p = c * kChunk + int(threadIdx.x);
        int all;
        group_scan(p < a.pool.pages && counted(a.owners_out + p) <= 0 ? 1 : 0, lds, all);
        if (threadIdx.x == 0)
            f.chunk[c] = all;
    }
}

// One workgroup: what comes before each row and each chunk.
__device__ void fork_scan(const PagesArgs &a, const ForkState &f, int *lds)
{
    __shared__ unsigned long long excess;        // of a few rows may pass 32 bits
    int fresh = 0, copies = 0, free = 0, all;
    if (threadIdx.x == 0)
        excess = 0;
    __syncthreads();
    for (int i0 = 0; i0 < a.rows_out; i0 += kChunk) {
        const int i = i0 + int(threadIdx.x);
        int n = 0, own = 0;
        if (i < a.rows_out) {
            const ForkRow r = fork_row(a, i);
            own = copies_last(a, f, r, i) ? 1 : 0;
            n = own + max(0, r.wants - r.held);
            if (r.excess)
                atomicAdd(&excess, (unsigned long long)r.excess);
        }
        const int upto = group_scan(n, lds, all);
        if (i < a.rows_out)
            f.fresh[i] = fresh + upto - n;
        fresh += all;
        const int made = group_scan(own, lds, all);
        if (i < a.rows_out)
            f.copies[i] = copies + made - own;
        copies += all;
    }
    const int chunks = (a.pool.pages + kChunk - 1) / kChunk;
    for (int c0 = 0; c0 < chunks; c0 += kChunk) {
        const int c = c0 + int(threadIdx.x);
        const int n = c < chunks ? counted(f.chunk + c) : 0;
        const int upto = group_scan(n, lds, all);
        if (c < chunks)
            f.chunk[c] = free + upto - n;
        free += all;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned long long missing = excess + max(0, fresh - free);
        a.missing[0] = missing < INT32_MAX ? int(missing) : INT32_MAX;
        f.totals[0] = missing ? 0 : copies;
        f.totals[1] = min(fresh, free);
    }
}

__device__ void fork_list(const PagesArgs &a, const ForkState &f, const Team &t, int *lds)
{
    const int take = counted(f.totals + 1);
    for (int c = t.group; c < (a.pool.pages + kChunk - 1) / kChunk; c += t.groups) {
        const int before = counted(f.chunk + c);
        if (before >= take)
            break;                               // so do all later chunks
        const int p = c * kChunk + int(threadIdx.x);
        const int is_free = p < a.pool.pages && counted(a.owners_out + p) <= 0 ? 1 : 0;
        int all;
        const int rank = before + group_scan(is_free, lds, all) - 1;
        if (is_free && rank < take)
            f.free[rank] = p;
    }
}

__device__ void fork_take(const PagesArgs &a, const ForkState &f, const Team &t)
{
    const int take = counted(f.totals + 1);
    const uint32_t entries = uint32_t(a.rows_out) * a.width;
    for (uint32_t e = t.tid; e < entries; e += t.n) {
        const int i = int(e / uint32_t(a.width)), j = int(e - uint32_t(i) * a.width);
        const ForkRow r = fork_row(a, i);
        if (j < r.held - 1 || j >= max(r.wants, r.held))
            continue;
        const bool own = copies_last(a, f, r, i);
        if (j == r.held - 1 && !own)
            continue;
        const int rank = counted(f.fresh + i) + (own ? 1 : 0) + j - r.held;
        const int p = rank < take ? counted(f.free + rank) : -1;
        if (p >= 0) {
            a.table_out[e] = p;
            a.owners_out[p] = 1;
        }
        if (j == r.held - 1) {
            const int at = counted(f.copies + i);
            f.src[at] = a.table[int64_t(r.parent) * a.width + j];
            f.dst[at] = p;
        }
    }
}

// Rows, pages and entries up to which one workgroup does all steps, with what they count in
// LDS.  Forking 32 rows of 33 pages takes 6 us that way and 17 as steps of their own kernels,
// 512 rows of 20 14 and 19, 1024 of 16 18 and 20; compacting 512 pages 4 and 9, 4096 7 and 11, 8192
// 11 and 12, 16000 23 and 12.  The entries' bound is generous: at 32768 the steps are the
// faster ones, 24 and 20 us forking 1000 rows of 32 pages, 31 and 22 forking 2048 of 16, 16 and 11
// compacting.
constexpr int kSmallRows = 2048, kSmallPages = 8192, kSmallEntries = 32768;

struct ForkLds {
    int counts[kSmallPages];
    uint16_t list[kSmallPages];                  // the free pages that are taken
    int first[kSmallRows];
    int4 rows[kSmallRows];                       // parent, held (own copy: bit 31), wants, fresh
    int copies[kSmallRows];                      // which of the copies a row's is
    int sums[kWavesOfChunk];
    unsigned long long excess;
};

__global__ __launch_bounds__(kChunk) void fork_kernel(PagesArgs a, ForkState f)
{
    __shared__ ForkLds l;
    const int tid = threadIdx.x;
    if (tid == 0)
        l.excess = 0;
    for (int p = tid; p < a.pool.pages; p += kChunk)
        l.counts[p] = a.owners[p];
    for (int r = tid; r < a.rows_in; r += kChunk)
        l.first[r] = INT32_MAX;
    __syncthreads();

    constexpr int EACH = kSmallRows / kChunk;    // rows of a thread: tid, tid + kChunk
    ForkRow rows[EACH];
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int i = tid + k * kChunk;
        if (i < a.rows_out) {
            rows[k] = fork_row(a, i);
            if (rows[k].parent >= 0)
                atomicMin(&l.first[rows[k].parent], i);
        }
    }
    __syncthreads();
    int fresh = 0, copies = 0, all;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int i = tid + k * kChunk;
        if (k * kChunk >= a.rows_out)
            break;
        int source = -1, n = 0;
        if (i < a.rows_out) {
            ForkRow &r = rows[k];
            if (r.parent >= 0 && r.used % a.page != 0 && l.first[r.parent] != i)
                source = a.table[r.parent * a.width + r.held - 1];
            r.own = is_page(a, source);
            n = (r.own ? 1 : 0) + max(0, r.wants - r.held);
            if (r.excess)
                atomicAdd(&l.excess, (unsigned long long)r.excess);
            a.used_out[i] = int(min(int64_t(r.used) + r.new_tokens, int64_t(a.width) * a.page));
        }
        const int upto = group_scan(n, l.sums, all);
        if (i < a.rows_out)
            l.rows[i] = make_int4(rows[k].parent, rows[k].held | (rows[k].own ? 1 << 31 : 0),
                                  rows[k].wants, fresh + upto - n);
        fresh += all;
        const int own = i < a.rows_out && rows[k].own ? 1 : 0;
        const int made = group_scan(own, l.sums, all);
        if (own) {
            f.src[copies + made - 1] = source;
            l.copies[i] = copies + made - 1;
        }
        copies += all;
    }
    __syncthreads();

    // shared entries, and what they change in the counts
    const int entries = max(a.rows_in, a.rows_out) * a.width;
    constexpr int AT_ONCE = 8;
    for (int e0 = tid; e0 < entries; e0 += AT_ONCE * kChunk) {
        int old[AT_ONCE], now[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int e = e0 + k * kChunk;
            old[k] = now[k] = -1;
            if (e < entries) {
                const int i = int(uint32_t(e) / uint32_t(a.width)), j = e - i * a.width;
                if (i < a.rows_in)
                    old[k] = a.table[e];
                if (i < a.rows_out) {
                    const int4 r = l.rows[i];
                    if (j < (r.y & INT32_MAX) - (r.y < 0 ? 1 : 0))
                        now[k] = a.table[r.x * a.width + j];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int e = e0 + k * kChunk;
            if (!is_page(a, now[k]))
                now[k] = -1;
            if (e < a.rows_out * a.width)
                a.table_out[e] = now[k];
            if (old[k] != now[k]) {
                if (is_page(a, old[k]))
                    atomicAdd(&l.counts[old[k]], -1);
                if (now[k] >= 0)
                    atomicAdd(&l.counts[now[k]], 1);
            }
        }
    }
    __syncthreads();

    // the lowest free pages: each thread looks at as many pages, one after the other
    const int each = (a.pool.pages + kChunk - 1) / kChunk;
    const int p0 = min(tid * each, a.pool.pages), p1 = min(p0 + each, a.pool.pages);
    int mine = 0;
    for (int p = p0; p < p1; ++p)
        mine += l.counts[p] <= 0 ? 1 : 0;
    int free;
    int rank = group_scan(mine, l.sums, free) - mine;
    const int take = min(fresh, free);
    for (int p = p0; p < p1 && rank < take; ++p)
        if (l.counts[p] <= 0) {
            l.list[rank++] = uint16_t(p);
            l.counts[p] = 1;
        }
    __syncthreads();
    for (int p = tid; p < a.pool.pages; p += kChunk)
        a.owners_out[p] = l.counts[p];
    constexpr int LANES = 16;                    // of a row: few have more pages to take
    for (int i = tid / LANES; i < a.rows_out; i += kChunk / LANES) {
        const int4 r = l.rows[i];
        const int held = r.y & INT32_MAX, own = r.y < 0 ? 1 : 0;
        for (int k = tid % LANES; k < own + max(0, r.z - held); k += LANES) {
            const int p = r.w + k < take ? l.list[r.w + k] : -1;
            a.table_out[i * a.width + held - own + k] = p;
            if (own && k == 0)
                f.dst[l.copies[i]] = p;
        }
    }
    if (tid == 0) {
        const unsigned long long missing = l.excess + max(0, fresh - free);
        a.missing[0] = missing < INT32_MAX ? int(missing) : INT32_MAX;
        f.totals[0] = missing ? 0 : copies;
    }
}

template <int STEP> __global__ __launch_bounds__(kChunk) void fork_step_kernel(PagesArgs a, ForkState f)
{
    __shared__ int lds[kWavesOfChunk];
    const Team t = team();
    if (STEP == 0)
        fork_init(a, f, t);
    if (STEP == 1)
        fork_first(a, f, t);
    if (STEP == 2)
        fork_share(a, f, t);
    if (STEP == 3)
        fork_count(a, f, t, lds);
    if (STEP == 4)
        fork_scan(a, f, lds);
    if (STEP == 5)
        fork_list(a, f, t, lds);
    if (STEP == 6)
        fork_take(a, f, t);
}

int step_blocks(int64_t n) { return int(std::clamp<int64_t>((n + kChunk - 1) / kChunk, 1, 512)); }

// ---- compact ---------------------------------------------------------------

struct CompactState {
    int32_t *chunk;        // [chunks] held pages of a chunk, then those before it
    int32_t *src, *dst;    // [pages / 2] the moves
    int32_t *totals;       // moves, held pages, held pages that stay
};

__device__ void compact_count(const PagesArgs &a, const CompactState &f, const Team &t, int *lds)
{
    for (int c = t.group; c < (a.pool.pages + kChunk - 1) / kChunk; c += t.groups) {
        const int p = c * kChunk + int(threadIdx.x);
        int all;
        group_scan(p < a.pool.pages && a.owners[p] > 0 ? 1 : 0, lds, all);
        if (threadIdx.x == 0)
            f.chunk[c] = all;
    }
}

// One workgroup: what comes before each chunk, and below the number of held pages.
__device__ void compact_scan(const PagesArgs &a, const CompactState &f, int *lds)
{
    const int chunks = (a.pool.pages + kChunk - 1) / kChunk;
    int held = 0, all;
    for (int c0 = 0; c0 < chunks; c0 += kChunk) {
        const int c = c0 + int(threadIdx.x);
        const int n = c < chunks ? counted(f.chunk + c) : 0;
        const int upto = group_scan(n, lds, all);
        if (c < chunks)
            f.chunk[c] = held + upto - n;
        held += all;
    }
    __syncthreads();
    int stay = held;                             // all of them, if there is no page but these
    if (held < a.pool.pages) {
        const int c = held / kChunk, p = c * kChunk + int(threadIdx.x);
        group_scan(p < held && a.owners[p] > 0 ? 1 : 0, lds, all);
        stay = counted(f.chunk + c) + all;
    }
    if (threadIdx.x == 0) {
        f.totals[0] = held - stay;
        f.totals[1] = held;
        f.totals[2] = stay;
    }
}

__device__ void compact_list(const PagesArgs &a, const CompactState &f, const Team &t, int *lds)
{
    const int held = counted(f.totals + 1), stay = counted(f.totals + 2);
    for (int c = t.group; c < (a.pool.pages + kChunk - 1) / kChunk; c += t.groups) {
        const int p = c * kChunk + int(threadIdx.x);
        const int n = p < a.pool.pages ? a.owners[p] : 0;
        int all;
        const int before = counted(f.chunk + c) + group_scan(n > 0 ? 1 : 0, lds, all) - (n > 0 ? 1 : 0);
        if (p >= a.pool.pages)
            continue;
        if (p < held) {
            if (n <= 0)
                f.dst[p - before] = p;
            else
                a.owners_out[p] = n;
            a.moved[p] = n > 0 ? p : -1;
        } else {
            a.owners_out[p] = 0;
            if (n > 0)
                f.src[before - stay] = p;
            else
                a.moved[p] = -1;
        }
    }
}

__device__ void compact_number(const PagesArgs &a, const CompactState &f, const Team &t)
{
    const int moves = counted(f.totals);
    for (int k = t.tid; k < moves; k += t.n) {
        const int s = counted(f.src + k), d = counted(f.dst + k);
        a.moved[s] = d;
        a.owners_out[d] = a.owners[s];
    }
}

__device__ void compact_table(const PagesArgs &a, const Team &t)
{
    const uint32_t entries = uint32_t(a.rows_in) * a.width;
    for (uint32_t e = t.tid; e < entries; e += t.n) {
        const int p = a.table[e];
        a.table_out[e] = is_page(a, p) ? counted(a.moved + p) : -1;
    }
}

struct CompactLds {
    int counts[kSmallPages];
    int moved[kSmallPages];
    int sums[kWavesOfChunk];
    int below;
};

__global__ __launch_bounds__(kChunk) void compact_kernel(PagesArgs a, CompactState f)
{
    __shared__ CompactLds l;
    const int tid = threadIdx.x;
    if (tid == 0)
        l.below = 0;
    for (int p = tid; p < a.pool.pages; p += kChunk)
        l.counts[p] = a.owners[p];
    __syncthreads();
    const int each = (a.pool.pages + kChunk - 1) / kChunk;
    const int p0 = min(tid * each, a.pool.pages), p1 = min(p0 + each, a.pool.pages);
    int mine = 0, held;
    for (int p = p0; p < p1; ++p)
        mine += l.counts[p] > 0 ? 1 : 0;
    const int before = group_scan(mine, l.sums, held) - mine;
    // held pages that stay, below the number of all
    mine = 0;
    for (int p = p0; p < min(p1, held); ++p)
        mine += l.counts[p] > 0 ? 1 : 0;
    if (mine)
        atomicAdd(&l.below, mine);
    __syncthreads();
    const int stay = l.below, moves = held - stay;
    int rank = before;
    for (int p = p0; p < p1; ++p) {
        const bool there = l.counts[p] > 0;
        l.moved[p] = there && p < held ? p : -1;
        if (p < held && !there)
            f.dst[p - rank] = p;
        if (p >= held && there)
            f.src[rank - stay] = p;
        rank += there ? 1 : 0;
    }
    __syncthreads();
    for (int k = tid; k < moves; k += kChunk) {
        const int s = f.src[k], d = f.dst[k];
        l.moved[s] = d;
        l.counts[d] = l.counts[s];
    }
    __syncthreads();
    for (int p = tid; p < a.pool.pages; p += kChunk) {
        a.moved[p] = l.moved[p];
        a.owners_out[p] = p < held ? l.counts[p] : 0;
    }
    for (int e = tid; e < a.rows_in * a.width; e += kChunk) {
        const int p = a.table[e];
        a.table_out[e] = is_page(a, p) ? l.moved[p] : -1;
    }
    if (tid == 0)
        f.totals[0] = moves;
}

template <int STEP>
__global__ __launch_bounds__(kChunk) void compact_step_kernel(PagesArgs a, CompactState f)
{
    __shared__ int lds[kWavesOfChunk];
    const Team t = team();
    if (STEP == 0)
        compact_count(a, f, t, lds);
    if (STEP == 1)
        compact_scan(a, f, lds);
    if (STEP == 2)
        compact_list(a, f, t, lds);
    if (STEP == 3)
        compact_number(a, f, t);
    if (STEP == 4)
        compact_table(a, t);
}

// Cuts a workspace into arrays.
struct Cutter {
    char *p;

    int32_t *take(size_t n)
    {
        int32_t *r = reinterpret_cast<int32_t *>(p);
        p += up_16(n * 4);
        return r;
    }
};

}  // namespace

size_t pages_fork_bytes(const PagesArgs &a)
{
    return up_16(size_t(a.rows_in) * 4) + 4 * up_16(size_t(a.rows_out) * 4) +
           up_16(size_t(chunks_of(a.pool.pages)) * 4) + up_16(size_t(a.pool.pages) * 4) + 16;
}

hipError_t launch_pages_fork(const PagesArgs &a, void *workspace, hipStream_t s)
{
    Cutter cut{static_cast<char *>(workspace)};
    ForkState f;
    f.first = cut.take(a.rows_in);
    f.fresh = cut.take(a.rows_out);
    f.copies = cut.take(a.rows_out);
    f.src = cut.take(a.rows_out);
    f.dst = cut.take(a.rows_out);
    f.chunk = cut.take(chunks_of(a.pool.pages));
    f.free = cut.take(a.pool.pages);
    f.totals = cut.take(2);
    const int64_t entries = int64_t(std::max(a.rows_in, a.rows_out)) * a.width;
    if (entries <= kSmallEntries && a.pool.pages <= kSmallPages &&
        std::max(a.rows_in, a.rows_out) <= kSmallRows) {
        fork_kernel<<<1, kChunk, 0, s>>>(a, f);
    } else {
        const int rows = step_blocks(std::max(a.rows_in, a.rows_out));
        const int cells = step_blocks(entries), pages = step_blocks(a.pool.pages);
        fork_step_kernel<0><<<std::max(rows, pages), kChunk, 0, s>>>(a, f);
        fork_step_kernel<1><<<rows, kChunk, 0, s>>>(a, f);
        fork_step_kernel<2><<<cells, kChunk, 0, s>>>(a, f);
        fork_step_kernel<3><<<pages, kChunk, 0, s>>>(a, f);
        fork_step_kernel<4><<<1, kChunk, 0, s>>>(a, f);
        fork_step_kernel<5><<<pages, kChunk, 0, s>>>(a, f);
        fork_step_kernel<6><<<cells, kChunk, 0, s>>>(a, f);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.pool.layers == 0 || !a.parents)
        return e;                                // without parents no row shares a page
    return launch_copies(a.pool, a.pool, f.src, f.dst, a.rows_out, f.totals, s);
}

size_t pages_compact_bytes(const PagesArgs &a)
{
    return up_16(size_t(chunks_of(a.pool.pages)) * 4) + 2 * up_16(size_t(a.pool.pages / 2 + 1) * 4) +
           16;
}

hipError_t launch_pages_compact(const PagesArgs &a, void *workspace, hipStream_t s)
{
    Cutter cut{static_cast<char *>(workspace)};
    CompactState f;
    f.chunk = cut.take(chunks_of(a.pool.pages));
    f.src = cut.take(a.pool.pages / 2 + 1);
    f.dst = cut.take(a.pool.pages / 2 + 1);
    f.totals = cut.take(3);
    const int64_t entries = int64_t(a.rows_in) * a.width;
    if (entries <= kSmallEntries && a.pool.pages <= kSmallPages) {
        compact_kernel<<<1, kChunk, 0, s>>>(a, f);
    } else {
        const int pages = step_blocks(a.pool.pages);
        compact_step_kernel<0><<<pages, kChunk, 0, s>>>(a, f);
        compact_step_kernel<1><<<1, kChunk, 0, s>>>(a, f);
        compact_step_kernel<2><<<pages, kChunk, 0, s>>>(a, f);
        compact_step_kernel<3><<<step_blocks(a.pool.pages / 2), kChunk, 0, s>>>(a, f);
        compact_step_kernel<4><<<step_blocks(entries), kChunk, 0, s>>>(a, f);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.pool.layers == 0)
        return e;
    return launch_copies(a.pool, a.pool, f.src, f.dst, a.pool.pages / 2, f.totals, s);
}

hipError_t launch_pages_copy(const PoolView &src, const PoolView &dst, const int32_t *src_pages,
                             const int32_t *dst_pages, int32_t count, hipStream_t s)
{
    return launch_copies(src, dst, src_pages, dst_pages, count, nullptr, s);
}

}  // namespace mdcn
