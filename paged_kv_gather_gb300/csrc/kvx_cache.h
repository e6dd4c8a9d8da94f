// kvx_cache.h -- descriptors and host logic of the operators that work on the page pools in
// place: page upkeep (kvx_pages.cu), token append and attention (kvx_attend.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/kvx.h"

namespace kvx {

// ---------------------------------------------------------------------------- page upkeep

// One fork.  Child pages [0, full) are the parent's, [full, total) are free pages; of the
// parent's pages that hold shared tokens, [full, ceil(shared / page_size)) are copied unless
// the entry grows in place.  The *_begin fields are running totals over the entries, and one
// entry past the last holds the batch's totals.
struct ForkEntry {
    const int32_t *parent;
    int32_t *child;
    int32_t full;
    int32_t total;
    int32_t shared;      // tokens
    int32_t grow;        // child == parent: the shared entries stay as they are
    int32_t page_begin;  // child pages
    int32_t fresh_begin; // pages taken from the free ones
    int32_t copy_begin;  // pages copied
    int32_t pad;
};
static_assert(sizeof(ForkEntry) == 48, "descriptor layout");

struct TableEntry {
    int32_t *pages;
    int32_t n_pages;
    int32_t page_begin;
};
static_assert(sizeof(TableEntry) == 16, "descriptor layout");

// Table columns that a CTA of the reordering rewrites.
const int kBeamColumns = 128;

// One group of beams.  The *_begin fields are running totals over the groups, and one entry
// past the last holds the batch's.
struct BeamEntry {
    int32_t *tables;
    int64_t stride;
    const int32_t *parents;
    int32_t width;
    int32_t full;        // pages
    int32_t tail;        // tokens in the page behind them
    int32_t col_begin;   // table columns, in whole CTAs
    int32_t copy_begin;  // last pages that may be copied
    int32_t pad;
};
static_assert(sizeof(BeamEntry) == 48, "descriptor layout");

kvx_status validate_beams(const kvx_pool *pool, const int32_t *refs, const kvx_beams *beams,
                          int n, int level, bool have_gpu, char *msg, size_t len);
kvx_status pack_beams(const kvx_pool *pool, const kvx_beams *beams, int n, BeamEntry *out,
                      char *msg, size_t len);

kvx_status validate_upkeep(const kvx_pool *pool, const int32_t *refs, const kvx_fork *forks,
                           int n_forks, const kvx_table *tables, int n_tables, int level,
                           bool have_gpu, char *msg, size_t len);

// Fill out[n + 1]; KVX_ERR_CAPACITY when a total passes 2^31 - 1.
kvx_status pack_forks(const kvx_pool *pool, const kvx_fork *forks, int n, ForkEntry *out,
                      char *msg, size_t len);
kvx_status pack_tables(const kvx_table *tables, int n, TableEntry *out, char *msg, size_t len);

// Pool pointers as the kernels index them: out[slab], slab = layer * kv_factor + kv.
void pack_slabs(const kvx_pool *pool, char **out);

// ---------------------------------------------------------------------------- attention

// One request of a step, as the kernels read it.
struct AttnReq {
    const int32_t *table;
    int32_t n_tokens;
    int32_t n_new;
    int32_t prefix;
    int32_t row_begin;   // first row of the request in q, out, lse, k and v
    int32_t pad[2];
};
static_assert(sizeof(AttnReq) == 32, "descriptor layout");

// A CTA's share of the units (request, block of rows, KV head) laid end to end: where it
// begins, how many tiles of keys it takes, and which CTAs it meets at its ends.
struct AttnStart {
    int32_t request;
    int32_t block;
    int32_t head;
    int32_t tile;     // within the unit
    int32_t first;    // CTA that began the unit, if tile > 0
    int32_t last;     // CTA that ends the unit this share stops inside of, if it does; else the
                      // share that the CTA takes next, 0: none
    int64_t tiles;
    AttnReq req;      // of `request`: one load instead of two in a row
};
static_assert(sizeof(AttnStart) == 64, "descriptor layout");

// Tiles of T keys that cover [0, prefix) and [low, end), in order: `first` tiles from key 0,
// then the rest `skip` tiles further on; no tile twice.
#ifdef __CUDACC__
__host__ __device__
#endif
inline void key_tiles(int prefix, int low, int end, int T, int *first, int *skip, int *tiles)
{
    const int f = (prefix + T - 1) / T, l = low / T;
    if (f < l) {
        *first = f;
        *skip = l - f;
        *tiles = f + (end + T - 1) / T - l;
    } else {
        *first = 0;
        *skip = 0;
        *tiles = ((end > prefix ? end : prefix) + T - 1) / T;
    }
}

kvx_status validate_attn(const kvx_pool *pool, const kvx_request *reqs, int n_req,
                         const int32_t *n_new, const int32_t *prefix, const kvx_attn_cfg *cfg,
                         int level, bool have_gpu, char *msg, size_t len);

kvx_status validate_rope(const kvx_rope *rope, int head_dim, char *msg, size_t len);
kvx_status validate_select(const kvx_select_cfg *cfg, char *msg, size_t len);

}  // namespace kvx
