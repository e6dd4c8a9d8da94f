// kvx_cache_host.cpp -- host logic of page upkeep, append and attention: validation and
// descriptor packing.  Runs without a GPU except for the pointer checks of level 2.
#include <cuda_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>
#include <utility>
#include <vector>

#include "kvx_cache.h"
#include "kvx_internal.h"

namespace kvx {
namespace {

kvx_status fail(kvx_status st, char *msg, size_t len, const char *fmt, ...)
{
    if (msg && len > 0) {
        va_list ap;
        va_start(ap, fmt);
        vsnprintf(msg, len, fmt, ap);
        va_end(ap);
    }
    return st;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int64_t pages_of(int64_t tokens, int64_t page_size)
{
    return (tokens + page_size - 1) / page_size;
}

// Positions of a request stay below this, so that sums of two of them fit in 32 bits.
constexpr int32_t kMaxTokens = 1 << 30;
// Rows of a step (new tokens x query heads): with the last block of the chunk kernel, of up to
// 256 rows, they are counted in 32 bits.
constexpr int64_t kMaxRows = INT32_MAX - 255;

// The pool's own checks are those of a transfer without chunks.
kvx_status validate_pool(const kvx_pool *pool, int level, bool have_gpu, char *msg, size_t len)
{
    return validate(pool, nullptr, 0, nullptr, 0, 0, pool ? pool->num_layers : 0, KVX_OP_STORE,
                    level, have_gpu, msg, len);
}

}  // namespace

kvx_status validate_upkeep(const kvx_pool *pool, const int32_t *refs, const kvx_fork *forks,
                           int n_forks, const kvx_table *tables, int n_tables, int level,
                           bool have_gpu, char *msg, size_t len)
{
    kvx_status st = validate_pool(pool, level, have_gpu, msg, len);
    if (st != KVX_OK)
        return st;
    if (pool->num_pages > KVX_MAX_UPKEEP_PAGES)
        return fail(KVX_ERR_CAPACITY, msg, len, "%d pages exceed KVX_MAX_UPKEEP_PAGES (%d)",
                    pool->num_pages, KVX_MAX_UPKEEP_PAGES);
    if (!refs || !aligned(refs, 4))
        return fail(KVX_ERR_INVALID_ARG, msg, len, "refs is NULL or not 4-byte aligned");
    if (n_forks < 0 || n_tables < 0 || (n_forks > 0 && !forks) || (n_tables > 0 && !tables))
        return fail(KVX_ERR_INVALID_ARG, msg, len, "bad fork/table arrays (%d, %d)", n_forks,
                    n_tables);
    for (int i = 0; i < n_forks; ++i) {
        const kvx_fork &f = forks[i];
        if (f.shared_tokens < 0 || f.child_tokens < f.shared_tokens)
            return fail(KVX_ERR_INVALID_ARG, msg, len, "fork %d: shared_tokens %d, child_tokens "
                        "%d", i, f.shared_tokens, f.child_tokens);
        if (pages_of(f.child_tokens, pool->page_size) > pool->num_pages)
            return fail(KVX_ERR_INVALID_ARG, msg, len, "fork %d: %d tokens need more than the "
                        "pool's %d pages", i, f.child_tokens, pool->num_pages);
        if ((f.shared_tokens > 0 && !f.parent) || (f.child_tokens > 0 && !f.child))
            return fail(KVX_ERR_INVALID_ARG, msg, len, "fork %d: parent or child is NULL", i);
        if (!aligned(f.parent, 4) || !aligned(f.child, 4))
            return fail(KVX_ERR_ALIGNMENT, msg, len, "fork %d: tables not 4-byte aligned", i);
        if (f.copy != 0 && f.copy != 1)
            return fail(KVX_ERR_INVALID_ARG, msg, len, "fork %d: copy %d", i, f.copy);
        if (f.copy && f.parent == f.child && f.child)
            return fail(KVX_ERR_INVALID_ARG, msg, len, "fork %d: copy with child == parent", i);
    }
    for (int i = 0; i < n_tables; ++i) {
        if (tables[i].n_pages < 0)
            return fail(KVX_ERR_INVALID_ARG, msg, len, "table %d: n_pages %d", i,
                        tables[i].n_pages);
        if (tables[i].n_pages > 0 && !tables[i].pages)
            return fail(KVX_ERR_INVALID_ARG, msg, len, "table %d: pages is NULL", i);
        if (!aligned(tables[i].pages, 4))
            return fail(KVX_ERR_ALIGNMENT, msg, len, "table %d: not 4-byte aligned", i);
    }
    if (level <= 1)
        return KVX_OK;

    // Level 2: what one entry writes, no other entry reads or writes.
    struct Range {
        uintptr_t lo, hi;
        int entry;
        bool write;
    };
    try {
        std::vector<Range> r;
        for (int i = 0; i < n_forks; ++i) {
            const kvx_fork &f = forks[i];
            const uintptr_t c = reinterpret_cast<uintptr_t>(f.child);
            const uintptr_t p = reinterpret_cast<uintptr_t>(f.parent);
            if (f.child_tokens > 0)
                r.push_back({c, c + 4 * pages_of(f.child_tokens, pool->page_size), i, true});
            if (f.shared_tokens > 0 && f.parent != f.child)
                r.push_back({p, p + 4 * pages_of(f.shared_tokens, pool->page_size), i, false});
        }
        for (int i = 0; i < n_tables; ++i)
            if (tables[i].n_pages > 0) {
                const uintptr_t p = reinterpret_cast<uintptr_t>(tables[i].pages);
                r.push_back({p, p + 4 * uintptr_t(tables[i].n_pages), n_forks + i, true});
            }
        std::sort(r.begin(), r.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
        // Sorted by start: a range meets an earlier one iff it starts below the furthest end
        // seen so far; two ranges that only read may share.
        uintptr_t end_any = 0, end_write = 0;
        int who_any = -1, who_write = -1;
        for (const Range &x : r) {
            const int other = x.lo < end_write ? who_write : x.write && x.lo < end_any ? who_any : -1;
            if (other >= 0)
                return fail(KVX_ERR_OVERLAP, msg, len, "the tables of entries %d and %d meet",
                            other, x.entry);
            if (x.hi > end_any) {
                end_any = x.hi;
                who_any = x.entry;
            }
            if (x.write && x.hi > end_write) {
                end_write = x.hi;
                who_write = x.entry;
            }
        }
    } catch (const std::bad_alloc &) {
        return fail(KVX_ERR_CAPACITY, msg, len, "out of host memory");
    }
    return KVX_OK;
}

kvx_status pack_forks(const kvx_pool *pool, const kvx_fork *forks, int n, ForkEntry *out,
                      char *msg, size_t len)
{
    int64_t pages = 0, fresh = 0, copied = 0;
    for (int i = 0; i <= n; ++i) {
        ForkEntry &e = out[i];
        e = ForkEntry();
        e.page_begin = int32_t(pages);
        e.fresh_begin = int32_t(fresh);
        e.copy_begin = int32_t(copied);
        if (i == n)
            break;
        const kvx_fork &f = forks[i];
        const int32_t held = int32_t(pages_of(f.shared_tokens, pool->page_size));
        e.parent = f.parent;
        e.child = f.child;
        e.shared = f.shared_tokens;
        e.total = int32_t(pages_of(f.child_tokens, pool->page_size));
        e.grow = f.parent == f.child;
        e.full = e.grow ? held : f.copy ? 0 : f.shared_tokens / pool->page_size;
        pages += e.total;
        fresh += e.total - e.full;
        copied += held - e.full;
        if (pages > INT32_MAX)
            return fail(KVX_ERR_CAPACITY, msg, len, "the batch covers more than 2^31 pages");
    }
    return KVX_OK;
}

kvx_status pack_tables(const kvx_table *tables, int n, TableEntry *out, char *msg, size_t len)
{
    int64_t pages = 0;
    for (int i = 0; i <= n; ++i) {
        out[i] = {i < n ? tables[i].pages : nullptr, i < n ? tables[i].n_pages : 0,
                  int32_t(pages)};
        if (i < n)
            pages += tables[i].n_pages;
        if (pages > INT32_MAX)
            return fail(KVX_ERR_CAPACITY, msg, len, "the tables hold more than 2^31 entries");
    }
    return KVX_OK;
}

kvx_status validate_beams(const kvx_pool *pool, const int32_t *refs, const kvx_beams *beams,
                          int n, int level, bool have_gpu, char *msg, size_t len)
{
    kvx_status st = validate_pool(pool, level, have_gpu, msg, len);
    if (st != KVX_OK)
        return st;
    if (!refs || !aligned(refs, 4))
        return fail(KVX_ERR_INVALID_ARG, msg, len, "refs is NULL or not 4-byte aligned");
    if (n < 0 || (n > 0 && !beams))
        return fail(KVX_ERR_INVALID_ARG, msg, len, "bad beam array (%d)", n);
    for (int i = 0; i < n; ++i) {
        const kvx_beams &b = beams[i];
        if (b.width < 1 || b.width > KVX_MAX_BEAMS || b.n_tokens < 0)
            return fail(KVX_ERR_INVALID_ARG, msg, len, "group %d: width %d, n_tokens %d", i,
                        b.width, b.n_tokens);
        const int64_t pages = pages_of(b.n_tokens, pool->page_size);
        if (pages > pool->num_pages)
            return fail(KVX_ERR_INVALID_ARG, msg, len, "group %d: %d tokens need more than the "
                        "pool's %d pages", i, b.n_tokens, pool->num_pages);
        if (!b.parents || (b.n_tokens > 0 && !b.tables))
            return fail(KVX_ERR_INVALID_ARG, msg, len, "group %d: tables or parents is NULL", i);
        if (!aligned(b.tables, 4) || !aligned(b.parents, 4))
            return fail(KVX_ERR_ALIGNMENT, msg, len, "group %d: tables or parents not 4-byte "
                        "aligned", i);
        if (b.width > 1 && b.table_stride < pages)
            return fail(KVX_ERR_INVALID_ARG, msg, len, "group %d: table_stride %lld below %lld "
                        "entries", i, (long long)b.table_stride, (long long)pages);
        // The last beam's table ends within the address space.
        if (b.table_stride > INT64_MAX / 4 / KVX_MAX_BEAMS)
            return fail(KVX_ERR_INVALID_ARG, msg, len, "group %d: table_stride %lld", i,
                        (long long)b.table_stride);
    }
    if (level <= 1)
        return KVX_OK;

    // Level 2: no two groups write one table.  Tables of one group are table_stride apart.
    try {
        std::vector<std::pair<uintptr_t, int>> at;
        for (int i = 0; i < n; ++i)
            if (beams[i].n_tokens > 0)
                for (int b = 0; b < beams[i].width; ++b)
                    at.push_back({reinterpret_cast<uintptr_t>(beams[i].tables +
                                                              b * beams[i].table_stride), i});
        std::sort(at.begin(), at.end());
        for (size_t k = 1; k < at.size(); ++k) {
            const int g = at[k - 1].second;
            if (at[k - 1].first + 4 * pages_of(beams[g].n_tokens, pool->page_size) > at[k].first)
                return fail(KVX_ERR_OVERLAP, msg, len, "groups %d and %d: tables overlap", g,
                            at[k].second);
        }
    } catch (const std::bad_alloc &) {
        return fail(KVX_ERR_CAPACITY, msg, len, "out of host memory");
    }
    return KVX_OK;
}

kvx_status pack_beams(const kvx_pool *pool, const kvx_beams *beams, int n, BeamEntry *out,
                      char *msg, size_t len)
{
    int64_t columns = 0, copies = 0;
    for (int i = 0; i <= n; ++i) {
        BeamEntry &e = out[i];
        e = BeamEntry();
        e.col_begin = int32_t(columns);
        e.copy_begin = int32_t(copies);
        if (i == n)
            break;
        const kvx_beams &b = beams[i];
        e.tables = b.tables;
        e.stride = b.table_stride;
        e.parents = b.parents;
        e.width = b.width;
        e.full = b.n_tokens / pool->page_size;
        e.tail = b.n_tokens % pool->page_size;
        // Whole blocks of columns, so that none holds columns of two groups.
        columns += (pages_of(b.n_tokens, pool->page_size) + kBeamColumns - 1) / kBeamColumns *
                   kBeamColumns;
        copies += e.tail ? e.width - 1 : 0;
        if (columns > INT32_MAX)
            return fail(KVX_ERR_CAPACITY, msg, len, "the tables hold more than 2^31 entries");
    }
    return KVX_OK;
}

kvx_status validate_rope(const kvx_rope *rope, int head_dim, char *msg, size_t len)
{
    if (!rope)
        return fail(KVX_ERR_INVALID_ARG, msg, len, "rope is NULL");
    if (rope->rotary_dim < 16 || rope->rotary_dim % 16 || rope->rotary_dim > head_dim)
        return fail(KVX_ERR_INVALID_ARG, msg, len, "rotary_dim %d: a multiple of 16 up to %d is "
                    "supported", rope->rotary_dim, head_dim);
    if ((rope->interleaved != 0 && rope->interleaved != 1) || !std::isfinite(rope->magnitude))
        return fail(KVX_ERR_INVALID_ARG, msg, len, "interleaved %d, magnitude %g",
                    rope->interleaved, double(rope->magnitude));
    if (!rope->freqs)
        return fail(KVX_ERR_INVALID_ARG, msg, len, "freqs is NULL");
    if (!aligned(rope->freqs, 4) || !aligned(rope->positions, 4))
        return fail(KVX_ERR_ALIGNMENT, msg, len, "freqs or positions not 4-byte aligned");
    return KVX_OK;
}

kvx_status validate_select(const kvx_select_cfg *cfg, char *msg, size_t len)
{
    if (!cfg)
        return fail(KVX_ERR_INVALID_ARG, msg, len, "cfg is NULL");
    if (cfg->n_groups < 1 || cfg->width < 1 || cfg->width > KVX_MAX_BEAMS || cfg->vocab < 1 ||
        cfg->vocab > KVX_MAX_VOCAB || cfg->picks < 1 || cfg->picks > KVX_MAX_PICKS)
        return fail(KVX_ERR_INVALID_ARG, msg, len, "n_groups %d, width %d, vocab %d, picks %d",
                    cfg->n_groups, cfg->width, cfg->vocab, cfg->picks);
    if (cfg->type != KVX_TYPE_HALF && cfg->type != KVX_TYPE_BFLOAT && cfg->type != KVX_TYPE_FLOAT)
        return fail(KVX_ERR_INVALID_ARG, msg, len, "type %d", cfg->type);
    if (int64_t(cfg->n_groups) * cfg->width > INT32_MAX)
        return fail(KVX_ERR_CAPACITY, msg, len, "more than 2^31 beams");
    return KVX_OK;
}

void pack_slabs(const kvx_pool *pool, char **out)
{
    for (int l = 0; l < pool->num_layers; ++l)
        for (int k = 0; k < pool->kv_factor; ++k)
            *out++ = static_cast<char *>((k ? pool->v_pages : pool->k_pages)[l]);
}

kvx_status validate_attn(const kvx_pool *pool, const kvx_request *reqs, int n_req,
                         const int32_t *n_new, const int32_t *prefix, const kvx_attn_cfg *cfg,
                         int level, bool have_gpu, char *msg, size_t len)
{
    kvx_status st = validate_pool(pool, level, have_gpu, msg, len);
    if (st != KVX_OK)
        return st;
    if (!cfg)
        return fail(KVX_ERR_INVALID_ARG, msg, len, "cfg is NULL");
    if (pool->kv_factor != 2)
        return fail(KVX_ERR_INVALID_ARG, msg, len, "attention needs K and V pools (kv_factor 2)");
    if (cfg->q_heads <= 0 || cfg->kv_heads <= 0 || cfg->q_heads % cfg->kv_heads != 0)
        return fail(KVX_ERR_INVALID_ARG, msg, len, "q_heads %d, kv_heads %d", cfg->q_heads,
                    cfg->kv_heads);
    if (cfg->head_dim != 64 && cfg->head_dim != 128)
        return fail(KVX_ERR_INVALID_ARG, msg, len, "head_dim %d: 64 and 128 are supported",
                    cfg->head_dim);
    if ((cfg->type != KVX_TYPE_HALF && cfg->type != KVX_TYPE_BFLOAT) ||
        (cfg->kv_type != cfg->type && cfg->kv_type != KVX_TYPE_FP_EIGHT &&
         cfg->kv_type != KVX_TYPE_FP_FOUR))
        return fail(KVX_ERR_INVALID_ARG, msg, len, "type %d, kv_type %d", cfg->type,
                    cfg->kv_type);
    if (pool->token_bytes != kvx_token_bytes(cfg->kv_heads, cfg->head_dim, cfg->kv_type))
        return fail(KVX_ERR_INVALID_ARG, msg, len, "token_bytes %lld is not %d heads x %d of "
                    "kv_type %d", (long long)pool->token_bytes, cfg->kv_heads, cfg->head_dim,
                    cfg->kv_type);
    if (cfg->window < 0 || !(cfg->softcap >= 0.0f) || !std::isfinite(cfg->softcap) ||
        !std::isfinite(cfg->scale))
        return fail(KVX_ERR_INVALID_ARG, msg, len, "window %d, softcap %g, scale %g", cfg->window,
                    double(cfg->softcap), double(cfg->scale));
    if (!aligned(cfg->slopes, 4))
        return fail(KVX_ERR_ALIGNMENT, msg, len, "slopes not 4-byte aligned");
    if (n_req < 0 || (n_req > 0 && (!reqs || !n_new)))
        return fail(KVX_ERR_INVALID_ARG, msg, len, "bad request arrays (%d)", n_req);
    int64_t rows = 0;
    for (int r = 0; r < n_req; ++r) {
        const int p = prefix ? prefix[r] : 0;
        if (reqs[r].n_tokens < 0 || n_new[r] < 0 || n_new[r] > reqs[r].n_tokens)
            return fail(KVX_ERR_INVALID_ARG, msg, len, "request %d: n_tokens %d, n_new %d", r,
                        reqs[r].n_tokens, n_new[r]);
        if (reqs[r].n_tokens > kMaxTokens)
            return fail(KVX_ERR_CAPACITY, msg, len, "request %d: n_tokens %d exceeds 2^30", r,
                        reqs[r].n_tokens);
        if (p < 0 || p > reqs[r].n_tokens)
            return fail(KVX_ERR_INVALID_ARG, msg, len, "request %d: prefix %d of %d tokens", r,
                        p, reqs[r].n_tokens);
        if (n_new[r] > 0 && !reqs[r].page_table)
            return fail(KVX_ERR_INVALID_ARG, msg, len, "request %d: page_table is NULL", r);
        if (!aligned(reqs[r].page_table, 4))
            return fail(KVX_ERR_ALIGNMENT, msg, len, "request %d: page_table not 4-byte aligned",
                        r);
        rows += n_new[r];
    }
    if (rows * cfg->q_heads > kMaxRows)
        return fail(KVX_ERR_CAPACITY, msg, len, "%lld new tokens x %d heads exceed 2^31 - 256 "
                    "rows", (long long)rows, cfg->q_heads);
    if (level <= 1)
        return KVX_OK;

    // Level 2: the page ids that some row sees, against the host copies.
    for (int r = 0; r < n_req; ++r) {
        const int32_t *pt = reqs[r].page_table_host;
        if (!pt || n_new[r] == 0)
            continue;
        const int n = reqs[r].n_tokens, p = prefix ? prefix[r] : 0;
        const int64_t lo = cfg->window ? std::max<int64_t>(0, int64_t(n) - n_new[r] -
                                                                  cfg->window + 1) : 0;
        for (int64_t j = 0; j < pages_of(n, pool->page_size); ++j) {
            const bool seen = (j + 1) * pool->page_size > lo || j * pool->page_size < p;
            if (seen && (pt[j] < 0 || pt[j] >= pool->num_pages))
                return fail(KVX_ERR_PAGE_OUT_OF_RANGE, msg, len,
                            "request %d: page_table[%lld] = %d outside [0, %d)", r, (long long)j,
                            pt[j], pool->num_pages);
        }
    }
    return KVX_OK;
}

}  // namespace kvx

extern "C" {

static bool gpu_present()
{
    int n = 0;
    if (cudaGetDeviceCount(&n) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return n > 0;
}

kvx_status kvx_upkeep_validate(const kvx_pool *pool, const int32_t *refs, const kvx_fork *forks,
                               int n_forks, const kvx_table *tables, int n_tables, int level,
                               char *msg, size_t msg_len)
{
    return kvx::validate_upkeep(pool, refs, forks, n_forks, tables, n_tables, level,
                                level >= 2 && gpu_present(), msg, msg_len);
}

kvx_status kvx_beams_validate(const kvx_pool *pool, const int32_t *refs, const kvx_beams *beams,
                              int n_groups, int level, char *msg, size_t msg_len)
{
    return kvx::validate_beams(pool, refs, beams, n_groups, level, level >= 2 && gpu_present(),
                               msg, msg_len);
}

int64_t kvx_token_bytes(int kv_heads, int head_dim, int kv_type)
{
    if (kv_heads <= 0 || head_dim <= 0)
        return 0;
    const int64_t row = int64_t(kv_heads) * head_dim;
    switch (kv_type) {
    case KVX_TYPE_HALF:
    case KVX_TYPE_BFLOAT:
        return 2 * row;
    case KVX_TYPE_FP_EIGHT:
        return row;
    case KVX_TYPE_FP_FOUR:
        return head_dim % 16 ? 0 : (row / 2 + row / 16 + 15) / 16 * 16;
    }
    return 0;
}

kvx_status kvx_attn_validate(const kvx_pool *pool, const kvx_request *reqs, int n_req,
                             const int32_t *n_new, const int32_t *prefix,
                             const kvx_attn_cfg *cfg, int level, char *msg, size_t msg_len)
{
    return kvx::validate_attn(pool, reqs, n_req, n_new, prefix, cfg, level,
                              level >= 2 && gpu_present(), msg, msg_len);
}

}  // extern "C"
