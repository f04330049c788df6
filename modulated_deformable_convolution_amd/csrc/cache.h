// cache.h -- arguments and launchers of the operators on key/value caches in 4
// bits and on the pages they lie in.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstddef>
#include <cstdint>

#include "attention.h"
#include "mdcn.h"

struct mdcn_cache {
    int32_t k_heads, dim, page;
};

namespace mdcn {

constexpr int kStripTokens = 16;
constexpr int kBlockChannels = 32;

constexpr int cache_blocks(int dim) { return (dim + kBlockChannels - 1) / kBlockChannels; }

// A strip: 16 tokens of one head with n blocks of channels (the layout is in mdcn.h).
// A lane of a wave finds what it needs of a matrix tile in one piece: lane 16 g + t the key
// channels 8 g .. 8 g + 7 of token t, lane 16 g + r the channels 2 r, 2 r + 1 of the
// tokens 4 g .. 4 g + 3, of all blocks, and the exponents that belong to them.
struct Strip {
    int blocks;
    constexpr int key_exp() const { return blocks == 3 ? 4 : blocks; }   // bytes of a token
    constexpr int values() const { return 256 * blocks; }
    constexpr int key_exps() const { return 512 * blocks; }
    constexpr int value_exps() const { return key_exps() + 16 * key_exp(); }
    constexpr int bytes() const { return value_exps() + 16 * blocks; }
};

// Exponents are held as e + 127 within the limits of the type that the values are to
// be exact in: the smallest magnitude, 2^(e - 1), and the largest, 6 * 2^e.
template <typename T> struct ExpRange {
    static constexpr int lo = 127 - 120, hi = 127 + 125;
};
template <> struct ExpRange<_Float16> {
    static constexpr int lo = 127 - 23, hi = 127 + 13;
};

constexpr int kNanExp = 255;

struct CacheArgs {
    char *pool;
    int64_t page_stride;       // bytes
    const int32_t *table, *used, *cu;
    int64_t table_stride;
    int32_t pages, width;
    int32_t batch, tokens;     // tokens of k and v, or queries
    int32_t k_heads, dim;
    int32_t page_shift;        // a page is 1 << page_shift tokens
    Heads k, v;                // store: inputs, load: outputs
    int32_t fill;              // load: 1 k, 2 v; attention: kFillOut, kFillLse
    // attention
    Heads q, out;
    float *lse;
    int32_t q_heads, causal;
    float scale;
    int32_t workers, unit_shift;
    float *partial;
    int4 *joins;
};

hipError_t launch_cache_store(mdcn_dtype dtype, const CacheArgs &a, hipStream_t s);
hipError_t launch_cache_load(mdcn_dtype dtype, const CacheArgs &a, hipStream_t s);

// How a batch of these sizes is attended to: rows of a workgroup (more than 32: the tile
// kernel), workgroups, tokens of a unit of their work; and the workspace.
struct CacheShape {
    int rows, workers, unit;
};
CacheShape cache_attend_shape(mdcn_dtype dtype, const CacheArgs &a);
// Whether the kernels can count the batch's work in 31 bits.
bool cache_attend_countable(mdcn_dtype dtype, const CacheArgs &a);
size_t cache_attend_bytes(mdcn_dtype dtype, const CacheArgs &a);
hipError_t launch_cache_attend(mdcn_dtype dtype, CacheArgs a, void *workspace, hipStream_t s);

// A pool [layers][pages]; strides in bytes.
struct PoolView {
    char *data;
    int64_t page_stride, layer_stride;
    int32_t layers, pages;
    int32_t page_bytes;
};

struct PagesArgs {
    PoolView pool;
    const int32_t *table, *used, *owners, *parents, *new_tokens;
    int32_t *table_out, *used_out, *owners_out, *moved, *missing;
    int32_t page, rows_in, rows_out, width;
};

size_t pages_fork_bytes(const PagesArgs &a);
hipError_t launch_pages_fork(const PagesArgs &a, void *workspace, hipStream_t s);
size_t pages_compact_bytes(const PagesArgs &a);
hipError_t launch_pages_compact(const PagesArgs &a, void *workspace, hipStream_t s);
hipError_t launch_pages_copy(const PoolView &src, const PoolView &dst, const int32_t *src_pages,
                             const int32_t *dst_pages, int32_t count, hipStream_t s);

}  // namespace mdcn
