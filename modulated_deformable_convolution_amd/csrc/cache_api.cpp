// cache_api.cpp -- the extern "C" entry points of the operators on 4-bit caches and on
// pages (include/mdcn.h): validation on the host, launches on the caller's stream.
#include <hip/hip_runtime_api.h>

#include <cstdio>
#include <new>

#include "cache.h"
#include "entry.h"
#include "mdcn.h"
#include "views.h"

namespace {

using namespace mdcn;

constexpr int64_t kMaxRowTokens = int64_t(1) << 30;      // of a row of a table
constexpr int64_t kMaxPageStride = int64_t(1) << 40;     // bytes
constexpr int64_t kMaxPoolBytes = int64_t(1) << 60;      // from a pool's first page to its last
constexpr int64_t kMaxCacheStride = (int64_t(1) << 32) - 16;
constexpr int64_t kMaxEntries = (int64_t(1) << 31) - 1;  // of a table, and pages of a pool

int64_t page_bytes_of(const mdcn_cache &op)
{
    return int64_t(Strip{cache_blocks(op.dim)}.bytes()) * op.k_heads * (op.page / kStripTokens);
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// dims[0..5]: batch, tokens, pages, page stride, width and row stride of the table.
mdcn_status cache_dims(const mdcn_cache *op, mdcn_dtype dtype, const int64_t *dims, CacheArgs *a)
{
    if (!op || !dims)
        return MDCN_E_NULL;
    if (!valid_dtype(dtype))
        return MDCN_E_DTYPE;
    if (dims[0] < 0 || dims[0] > (1 << 24) || dims[1] < 0 || dims[1] > kMaxTokens || dims[2] < 0 ||
        dims[2] > kMaxEntries || dims[3] < 0 || dims[3] > kMaxCacheStride || dims[3] % 16 ||
        (dims[2] > 1 && dims[3] < page_bytes_of(*op)))
        return MDCN_E_SHAPE;
    if (dims[4] < 0 || dims[4] > kMaxRowTokens / op->page || dims[5] < 0 ||
        (dims[0] > 1 && dims[5] < dims[4]) || dims[5] > kMaxEntries)
        return MDCN_E_SHAPE;
    a->batch = int32_t(dims[0]);
    a->tokens = int32_t(dims[1]);
    a->pages = int32_t(dims[2]);
    a->page_stride = dims[3];
    a->width = int32_t(dims[4]);
    a->table_stride = dims[5];
    a->k_heads = op->k_heads;
    a->dim = op->dim;
    a->page_shift = __builtin_ctz(unsigned(op->page));
    return MDCN_OK;
}

// The buffers of every call: pool, table, lengths, offsets.  `written` tells of the pool.
struct CacheBlocks {
    Block b[4];

    CacheBlocks(const CacheArgs &a, const mdcn_cache &op, bool written)
        : b{{a.pool, a.pages ? size_t(a.pages - 1) * a.page_stride + page_bytes_of(op) : 0, written},
            {a.table, a.batch ? (size_t(a.batch - 1) * a.table_stride + a.width) * 4 : 0, false},
            {a.used, size_t(a.batch) * 4, false},
            {a.cu, size_t(a.batch + 1) * 4, false}}
    {
    }
};

mdcn_status check_cache_pointers(const CacheArgs &a)
{
    if (!a.cu || (a.batch > 0 && !a.used) || (a.batch > 0 && a.width > 0 && !a.table) ||
        (a.pages > 0 && !a.pool))
        return MDCN_E_NULL;
    return aligned16(a.pool) ? MDCN_OK : MDCN_E_SHAPE;
}

// Store reads k and v and writes the pool, load the other way round.
mdcn_status move_tokens(const mdcn_cache *op, mdcn_dtype dtype, const int64_t *dims, void *pool,
                        const int32_t *table, const int32_t *used, const int32_t *cu, bool load,
                        int32_t fill, const void *k, const void *v, void *stream)
{
    CacheArgs a = {};
    mdcn_status st = cache_dims(op, dtype, dims, &a);
    if (st != MDCN_OK)
        return st;
    const size_t e = elem_size(dtype);
    View views[] = {{{k, dims[6], dims[7]}, a.tokens, a.k_heads, a.dim, e},
                    {{v, dims[8], dims[9]}, a.tokens, a.k_heads, a.dim, e}};
    for (View &x : views)
        if ((st = check_attend_view(x)) != MDCN_OK)
            return st;
    a.pool = static_cast<char *>(pool);
    a.table = table;
    a.used = used;
    a.cu = cu;
    if ((st = check_cache_pointers(a)) != MDCN_OK)
        return st;
    const CacheBlocks blocks(a, *op, !load);
    if (blocks_overlap(blocks.b))
        return MDCN_E_ALIAS;
    for (const View &x : views) {
        if (load && !distinct_rows(x))
            return MDCN_E_ALIAS;
        for (const Block &b : blocks.b)
            if ((load || b.written) && b.p && overlap(x, b.p, b.n))
                return MDCN_E_ALIAS;
    }
    if (load && share_values(views[0], views[1]))
        return MDCN_E_ALIAS;
    if (a.tokens == 0 || (a.batch == 0 && !(load && (fill & 3))))
        return MDCN_OK;
    if ((st = mdcn::check_device()) != MDCN_OK)
        return st;
    a.k = views[0].h;
    a.v = views[1].h;
    a.fill = fill & 3;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return launched(load ? launch_cache_load(dtype, a, s) : launch_cache_store(dtype, a, s));
}

mdcn_status attend_args(const mdcn_attention *att, const mdcn_cache *op, mdcn_dtype dtype,
                        const int64_t *dims, CacheArgs *a)
{
    if (!att)
        return MDCN_E_NULL;
    const mdcn_status st = cache_dims(op, dtype, dims, a);
    if (st != MDCN_OK)
        return st;
    if (att->k_heads != op->k_heads || att->dim != op->dim)
        return MDCN_E_ATTR;
    if (dims[1] > kMaxEntries / (att->q_heads / att->k_heads))   // rows of a key head
        return MDCN_E_SHAPE;
    a->q_heads = att->q_heads;
    a->causal = att->causal;
    a->scale = att->scale;
    return cache_attend_countable(dtype, *a) ? MDCN_OK : MDCN_E_SHAPE;
}

// ---- pages -----------------------------------------------------------------

// layers, pages, bytes of a page, page and layer stride
mdcn_status pool_view(int64_t layers, int64_t pages, int64_t bytes, int64_t page_stride,
                      int64_t layer_stride, const void *data, PoolView *p)
{
    if (layers < 0 || layers > (1 << 20) || pages < 0 || pages > kMaxEntries || bytes < 0 ||
        bytes > (int64_t(1) << 30) || page_stride < 0 || page_stride > kMaxPageStride ||
        page_stride > kMaxPoolBytes / (pages + 1) || layer_stride < 0 ||
        layer_stride > kMaxPoolBytes / (layers + 1) || bytes % 16 || page_stride % 16 ||
        layer_stride % 16)
        return MDCN_E_SHAPE;
    // rows of bytes that do not overlap, pages within layers or layers within pages
    if ((pages > 1 && page_stride < bytes) || (layers > 1 && layer_stride < bytes))
        return MDCN_E_SHAPE;
    if (layers > 1 && pages > 1 && layer_stride < (pages - 1) * page_stride + bytes &&
        page_stride < (layers - 1) * layer_stride + bytes)
        return MDCN_E_SHAPE;
    if (layers > 0 && pages > 0 && bytes > 0 && !data)
        return MDCN_E_NULL;
    if (!aligned16(data))
        return MDCN_E_SHAPE;
    p->data = static_cast<char *>(const_cast<void *>(data));
    p->layers = int32_t(layers);
    p->pages = int32_t(pages);
    p->page_bytes = int32_t(bytes);
    p->page_stride = page_stride;
    p->layer_stride = layer_stride;
    return MDCN_OK;
}

size_t pool_bytes(const PoolView &p)
{
    if (!p.layers || !p.pages || !p.page_bytes)
        return 0;
    return size_t(p.layers - 1) * p.layer_stride + size_t(p.pages - 1) * p.page_stride + p.page_bytes;
}

mdcn_status table_dims(int64_t rows_in, int64_t rows_out, int64_t width, int64_t page, PagesArgs *a)
{
    if (rows_in < 0 || rows_out < 0 || width < 0 || page < 1 || page > (1 << 20) ||
        rows_in > kMaxEntries || rows_out > kMaxEntries || width > kMaxRowTokens / page ||
        (width > 0 && (rows_in > kMaxEntries / width || rows_out > kMaxEntries / width)))
        return MDCN_E_SHAPE;
    a->rows_in = int32_t(rows_in);
    a->rows_out = int32_t(rows_out);
    a->width = int32_t(width);
    a->page = int32_t(page);
    return MDCN_OK;
}

mdcn_status fork_args(const int64_t *dims, const void *pool, PagesArgs *a)
{
    if (!dims)
        return MDCN_E_NULL;
    const mdcn_status st = pool_view(dims[0], dims[1], dims[2], dims[3], dims[4], pool, &a->pool);
    return st != MDCN_OK ? st : table_dims(dims[6], dims[7], dims[8], dims[5], a);
}

mdcn_status compact_args(const int64_t *dims, const void *pool, PagesArgs *a)
{
    if (!dims)
        return MDCN_E_NULL;
    const mdcn_status st = pool_view(dims[0], dims[1], dims[2], dims[3], dims[4], pool, &a->pool);
    return st != MDCN_OK ? st : table_dims(dims[5], dims[5], dims[6], 1, a);
}

// Any address will do where only sizes are asked for.
const void *const kSomewhere = reinterpret_cast<const void *>(uintptr_t(256));

}  // namespace

extern "C" {

mdcn_status mdcn_cache_create(int32_t k_heads, int32_t dim, int32_t page, mdcn_cache **out)
{
    if (!out)
        return MDCN_E_NULL;
    *out = nullptr;
    if (k_heads < 1 || k_heads > 65536 || dim < 8 || dim % 8 || dim > mdcn::kMaxAttendDim ||
        page < kStripTokens || page > 256 || (page & (page - 1)))
        return MDCN_E_ATTR;
    mdcn_cache *op = new (std::nothrow) mdcn_cache();
    if (!op)
        return MDCN_E_INTERNAL;
    op->k_heads = k_heads;
    op->dim = dim;
    op->page = page;
    *out = op;
    return MDCN_OK;
}

void mdcn_cache_destroy(mdcn_cache *op) { delete op; }

mdcn_status mdcn_cache_page_bytes(const mdcn_cache *op, int64_t *bytes)
{
    if (!op || !bytes)
        return MDCN_E_NULL;
    *bytes = page_bytes_of(*op);
    return MDCN_OK;
}

mdcn_status mdcn_cache_store(const mdcn_cache *op, mdcn_dtype dtype, const int64_t dims[10],
                             const void *k, const void *v, const int32_t *table,
                             const int32_t *used, const int32_t *cu, void *pool, void *stream)
{
    try {
        return move_tokens(op, dtype, dims, pool, table, used, cu, false, 0, k, v, stream);
    } catch (...) {
        return MDCN_E_INTERNAL;
    }
}

mdcn_status mdcn_cache_load(const mdcn_cache *op, mdcn_dtype dtype, const int64_t dims[10],
                            const void *pool, const int32_t *table, const int32_t *used,
                            const int32_t *cu, int32_t fill, void *k, void *v, void *stream)
{
    try {
        return move_tokens(op, dtype, dims, const_cast<void *>(pool), table, used, cu, true, fill, k,
                           v, stream);
    } catch (...) {
        return MDCN_E_INTERNAL;
    }
}

mdcn_status mdcn_cache_attend_workspace_bytes(const mdcn_attention *att, const mdcn_cache *op,
                                              mdcn_dtype dtype, const int64_t dims[10],
                                              size_t *bytes)
{
    CacheArgs a = {};
    if (!bytes)
        return MDCN_E_NULL;
    const mdcn_status st = attend_args(att, op, dtype, dims, &a);
    if (st != MDCN_OK)
        return st;
    *bytes = a.tokens && a.batch ? mdcn::cache_attend_bytes(dtype, a) + 256 : 0;
    return MDCN_OK;
}

mdcn_status mdcn_cache_attend(const mdcn_attention *att, const mdcn_cache *op, mdcn_dtype dtype,
                              const int64_t dims[10], const void *q, const void *pool,
                              const int32_t *table, const int32_t *used, const int32_t *cu_q,
                              int32_t fill, void *out, float *lse, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    try {
        CacheArgs a = {};
        mdcn_status st = attend_args(att, op, dtype, dims, &a);
        if (st != MDCN_OK)
            return st;
        const size_t e = elem_size(dtype);
        View in = {{q, dims[6], dims[7]}, a.tokens, a.q_heads, a.dim, e};
        View o = {{out, dims[8], dims[9]}, a.tokens, a.q_heads, a.dim, e};
        if ((st = check_attend_view(in)) != MDCN_OK || (st = check_attend_view(o)) != MDCN_OK)
            return st;
        a.pool = static_cast<char *>(const_cast<void *>(pool));
        a.table = table;
        a.used = used;
        a.cu = cu_q;
        if ((st = check_cache_pointers(a)) != MDCN_OK)
            return st;
        if (a.tokens > 0 && !lse)
            return MDCN_E_NULL;
        size_t need = 0;
        if ((st = mdcn_cache_attend_workspace_bytes(att, op, dtype, dims, &need)) != MDCN_OK)
            return st;
        if (need && (!workspace || workspace_bytes < need))
            return MDCN_E_WORKSPACE;
        const size_t lse_bytes = size_t(a.q_heads) * a.tokens * 4;
        const CacheBlocks c(a, *op, false);
        const Block all[] = {{lse, lse_bytes, true},
                             {need ? workspace : nullptr, workspace_bytes, true},
                             c.b[0], c.b[1], c.b[2], c.b[3]};
        if (blocks_overlap(all))
            return MDCN_E_ALIAS;
        if (!distinct_rows(o) || share_values(in, o))
            return MDCN_E_ALIAS;
        for (const Block &b : all)
            if (b.p && (overlap(o, b.p, b.n) || (b.written && overlap(in, b.p, b.n))))
                return MDCN_E_ALIAS;
        a.fill = fill & (mdcn::kFillOut | mdcn::kFillLse);
        if (a.tokens == 0 || (a.batch == 0 && !a.fill))
            return MDCN_OK;
        if ((st = mdcn::check_device()) != MDCN_OK)
            return st;
        a.q = in.h;
        a.out = o.h;
        a.lse = lse;
        return launched(launch_cache_attend(dtype, a, need ? align_up(workspace) : nullptr,
                                            static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MDCN_E_INTERNAL;
    }
}

mdcn_status mdcn_describe_cache_attend(const mdcn_attention *att, const mdcn_cache *op,
                                       mdcn_dtype dtype, const int64_t dims[10], char *buf,
                                       size_t len)
{
    if (!buf || len == 0)
        return MDCN_E_NULL;
    CacheArgs a = {};
    const mdcn_status st = attend_args(att, op, dtype, dims, &a);
    if (st != MDCN_OK)
        return st;
    const mdcn::CacheShape c = mdcn::cache_attend_shape(dtype, a);
    std::snprintf(buf, len, "%s rows=%d workgroups=%d unit=%d", c.rows > 32 ? "tile" : "split",
                  c.rows, c.workers, c.unit);
    return MDCN_OK;
}

mdcn_status mdcn_pages_fork_workspace_bytes(const int64_t dims[9], size_t *bytes)
{
    if (!bytes)
        return MDCN_E_NULL;
    PagesArgs a = {};
    const mdcn_status st = fork_args(dims, kSomewhere, &a);
    if (st == MDCN_OK)
        *bytes = mdcn::pages_fork_bytes(a) + 256;
    return st;
}

mdcn_status mdcn_pages_fork(const int64_t dims[9], void *pool, const int32_t *table,
                            const int32_t *used, const int32_t *owners, const int32_t *parents,
                            const int32_t *new_tokens, int32_t *table_out, int32_t *used_out,
                            int32_t *owners_out, int32_t *missing, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    try {
        PagesArgs a = {};
        mdcn_status st = fork_args(dims, pool, &a);
        if (st != MDCN_OK)
            return st;
        if (!parents && a.rows_in != a.rows_out)
            return MDCN_E_SHAPE;
        const size_t in = size_t(a.rows_in) * a.width * 4, out = size_t(a.rows_out) * a.width * 4;
        const size_t counts = size_t(a.pool.pages) * 4, rows = size_t(a.rows_out) * 4;
        if ((in && !table) || (a.rows_in && !used) || (counts && (!owners || !owners_out)) ||
            (out && !table_out) || (rows && !used_out) || !missing)
            return MDCN_E_NULL;
        size_t need = 0;
        if ((st = mdcn_pages_fork_workspace_bytes(dims, &need)) != MDCN_OK)
            return st;
        if (!workspace || workspace_bytes < need)
            return MDCN_E_WORKSPACE;
        const Block all[] = {{a.pool.data, pool_bytes(a.pool), true},
                             {table, in, false},
                             {used, size_t(a.rows_in) * 4, false},
                             {owners, counts, false},
                             {parents, parents ? rows : 0, false},
                             {new_tokens, new_tokens ? rows : 0, false},
                             {table_out, out, true},
                             {used_out, rows, true},
                             {owners_out, counts, true},
                             {missing, 4, true},
                             {workspace, workspace_bytes, true}};
        if (blocks_overlap(all))
            return MDCN_E_ALIAS;
        if ((st = mdcn::check_device()) != MDCN_OK)
            return st;
        a.table = table;
        a.used = used;
        a.owners = owners;
        a.parents = parents;
        a.new_tokens = new_tokens;
        a.table_out = table_out;
        a.used_out = used_out;
        a.owners_out = owners_out;
        a.missing = missing;
        return launched(launch_pages_fork(a, align_up(workspace), static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MDCN_E_INTERNAL;
    }
}

mdcn_status mdcn_pages_compact_workspace_bytes(const int64_t dims[7], size_t *bytes)
{
    if (!bytes)
        return MDCN_E_NULL;
    PagesArgs a = {};
    const mdcn_status st = compact_args(dims, kSomewhere, &a);
    if (st == MDCN_OK)
        *bytes = mdcn::pages_compact_bytes(a) + 256;
    return st;
}

mdcn_status mdcn_pages_compact(const int64_t dims[7], void *pool, const int32_t *table,
                               const int32_t *owners, int32_t *table_out, int32_t *owners_out,
                               int32_t *moved, void *workspace, size_t workspace_bytes, void *stream)
{
    try {
        PagesArgs a = {};
        mdcn_status st = compact_args(dims, pool, &a);
        if (st != MDCN_OK)
            return st;
        const size_t cells = size_t(a.rows_in) * a.width * 4, counts = size_t(a.pool.pages) * 4;
        if ((cells && (!table || !table_out)) || (counts && (!owners || !owners_out || !moved)))
            return MDCN_E_NULL;
        size_t need = 0;
        if ((st = mdcn_pages_compact_workspace_bytes(dims, &need)) != MDCN_OK)
            return st;
        if (!workspace || workspace_bytes < need)
            return MDCN_E_WORKSPACE;
        const Block all[] = {{a.pool.data, pool_bytes(a.pool), true},
                             {table, cells, false},
                             {owners, counts, false},
                             {table_out, cells, true},
                             {owners_out, counts, true},
                             {moved, counts, true},
                             {workspace, workspace_bytes, true}};
        if (blocks_overlap(all))
            return MDCN_E_ALIAS;
        if (a.pool.pages == 0 && cells == 0)
            return MDCN_OK;
        if ((st = mdcn::check_device()) != MDCN_OK)
            return st;
        a.table = table;
        a.owners = owners;
        a.table_out = table_out;
        a.owners_out = owners_out;
        a.moved = moved;
        return launched(
            launch_pages_compact(a, align_up(workspace), static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MDCN_E_INTERNAL;
    }
}

mdcn_status mdcn_pages_copy(const int64_t dims[9], const void *src_pool, void *dst_pool,
                            const int32_t *src, const int32_t *dst, void *stream)
{
    try {
        if (!dims)
            return MDCN_E_NULL;
        PoolView from, to;
        mdcn_status st = pool_view(dims[0], dims[3], dims[2], dims[4], dims[5], src_pool, &from);
        if (st == MDCN_OK)
            st = pool_view(dims[0], dims[6], dims[2], dims[7], dims[8], dst_pool, &to);
        if (st != MDCN_OK)
            return st;
        if (dims[1] < 0 || dims[1] > kMaxEntries)
            return MDCN_E_SHAPE;
        if (dims[1] > 0 && (!src || !dst))
            return MDCN_E_NULL;
        const size_t list = size_t(dims[1]) * 4;
        const bool one = from.data == to.data && from.page_stride == to.page_stride &&
                         (from.layers <= 1 || from.layer_stride == to.layer_stride);
        const Block all[] = {{one ? nullptr : from.data, pool_bytes(from), false},
                             {to.data, pool_bytes(to), true},
                             {src, list, false},
                             {dst, list, false}};
        if (blocks_overlap(all))
            return MDCN_E_ALIAS;
        if (dims[1] == 0 || pool_bytes(from) == 0 || pool_bytes(to) == 0)
            return MDCN_OK;
        if ((st = mdcn::check_device()) != MDCN_OK)
            return st;
        return launched(launch_pages_copy(from, to, src, dst, int32_t(dims[1]),
                                          static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MDCN_E_INTERNAL;
    }
}

}  // extern "C"
