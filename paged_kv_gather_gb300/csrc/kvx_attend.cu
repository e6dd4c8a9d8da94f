// kvx_attend.cu -- append and attention over the pages of a paged KV cache: plans, entry
// points and the append kernel.  The attention kernels are in kvx_attend_rows.cuh and
// kvx_attend_tiles.cuh, the checks in kvx_cache_host.cpp.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "kvx_attend.cuh"
#include "kvx_attend_rows.cuh"
#include "kvx_attend_tiles.cuh"
#include "kvx_attend_plan.h"

namespace {

// ------------------------------------------------------------------------------- append

struct Append {
    Step step;
    const char *src[2];      // K, V
    int64_t stride[2];       // bytes between tokens
    char *pool[2];
    int64_t token_bytes;     // of the cache
    float scale[2];
    int32_t units;           // 16-byte units of a cache token
};

// 16 bytes of the cache from the new token's elements.
template <int TYPE, int KV>
struct Unit {
    uint4 in[KV == TYPE ? 1 : 2];

    __device__ __forceinline__ void load(const char *src, int u)
    {
#pragma unroll
        for (int i = 0; i < (KV == TYPE ? 1 : 2); ++i)
            in[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + (KV == TYPE ? u : 2 * u + i));
    }
    __device__ __forceinline__ uint4 value(float scale) const
    {
        if (KV == TYPE)
            return in[0];
        typedef typename Elem<TYPE>::T T;
        const T *x = reinterpret_cast<const T *>(in);
        unsigned r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            unsigned two[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 f = make_float2(Elem<TYPE>::load(x[4 * i + 2 * k]) / scale,
                                             Elem<TYPE>::load(x[4 * i + 2 * k + 1]) / scale);
                two[k] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
            }
            r[i] = two[0] | two[1] << 16;
        }
        return make_uint4(r[0], r[1], r[2], r[3]);
    }
};

// A warp per (new token, K or V), four 16-byte units of the cache in flight per lane.  The
// copy is bound by memory (8.2k tokens of 8 heads, 67 MB: 12 us, 5.6 TB/s); where few tokens
// are new, by the latency of a launch, table and data (64 tokens: 2.4 us).
template <int TYPE, int KV>
__global__ void __launch_bounds__(256)
kvx_append_kernel(const Append a)
{
    const int lane = threadIdx.x & 31;
    const int64_t job = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int row = int(job >> 1), kv = int(job & 1);
    wait_for_earlier_work();
    if (row >= a.step.rows)
        return;
    const char *src = a.src[kv] + row * a.stride[kv];
    Unit<TYPE, KV> x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < a.units)
            x[i].load(src, lane + 32 * i);
    const AttnReq q = a.step.reqs[request_of_row(a.step.reqs, a.step.n_req, row, lane)];
    const int pos = q.n_tokens - q.n_new + row - q.row_begin, nth = a.step.page.div(pos);
    const int page = q.table[nth];
    if (unsigned(page) >= unsigned(a.step.num_pages)) {
        if (lane == 0)
            atomicOr(a.step.status, KVX_DEV_PAGE_OUT_OF_RANGE);
        return;
    }
    uint4 *dst = reinterpret_cast<uint4 *>(
        a.pool[kv] +
        (int64_t(page) * a.step.page_size + pos - nth * a.step.page_size) * a.token_bytes);
#pragma unroll 1
    for (int u0 = lane; u0 < a.units; u0 += 128) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (u0 + 32 * i < a.units)
                dst[u0 + 32 * i] = x[i].value(a.scale[kv]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (u0 + 128 + 32 * i < a.units)
                x[i].load(src, u0 + 128 + 32 * i);
    }
}

// ---------------------------------------------------------------------------------- host

template <int TYPE, int KV, int D>
Kernel kernel_of(int kind)
{
    if (kind == kRows)
        return {reinterpret_cast<const void *>(kvx_attend_rows_kernel<TYPE, KV, D, 1>),
                kRowThreads, row_ctas_per_sm<KV, D, 1>(), row_smem<KV, D, 1>(),
                row_slot_floats<D, 1>(), nullptr, 0, 0, 0, row_smem<KV, D, 1>()};
    if (kind == kMoreRows)
        return {reinterpret_cast<const void *>(kvx_attend_rows_kernel<TYPE, KV, D, 2>),
                kRowThreads, row_ctas_per_sm<KV, D, 2>(), row_smem<KV, D, 2>(),
                row_slot_floats<D, 2>(), nullptr, 0, 0, 0, row_smem<KV, D, 2>()};
    return {reinterpret_cast<const void *>(kvx_attend_tiles_kernel<TYPE, KV, D>),
            TileShape<KV, D>::kThreads, 1,
            size_t(TileShape<KV, D>::kBytes), TileShape<KV, D>::kSlotFloats,
            reinterpret_cast<const void *>(kvx_attend_join_kernel<TYPE, D>), kJoinThreads,
            kBlockRows / kJoinRows, 0, size_t(TileShape<KV, D>::kBytes)};
}

Kernel pick_kernel(const kvx_attn_plan *p, int kind)
{
    const kvx_attn_cfg &c = p->cfg;
    if (c.kv_type == KVX_TYPE_FP_FOUR)
        return kvx::four_kernel(c, p->token_bytes, kind, p->most_parts[kind]);
    const bool half = c.type == KVX_TYPE_HALF, eight = c.kv_type == KVX_TYPE_FP_EIGHT;
    const int H = KVX_TYPE_HALF, B = KVX_TYPE_BFLOAT, F = KVX_TYPE_FP_EIGHT;
    if (c.head_dim == 64)
        return half ? eight ? kernel_of<H, F, 64>(kind) : kernel_of<H, H, 64>(kind)
                    : eight ? kernel_of<B, F, 64>(kind) : kernel_of<B, B, 64>(kind);
    return half ? eight ? kernel_of<H, F, 128>(kind) : kernel_of<H, H, 128>(kind)
                : eight ? kernel_of<B, F, 128>(kind) : kernel_of<B, B, 128>(kind);
}

// Lay the units of one kind end to end and give every CTA its share (struct Work).  Shares
// are equal in tiles plus what a unit costs besides them.  Whether units are cut at all is
// decided by an estimate of the slowest CTA's time: cutting evens the shares out, but each
// part of a cut unit has to be written, and joined by one of its CTAs.  A few units per CTA of
// the kernel for chunks may also be dealt out instead, whole and in any order, which evens
// them out without parts (2k tokens of 32 heads: 51.1 -> 35.8 us).
struct Scheduler {
    const kvx_attn_plan *p;
    const AttnReq *reqs;
    int n_req, kind, group, heads, block_rows, tile_keys;  // heads: units of a block of rows
    int64_t unit_cost, part_cost, join_cost;               // beyond the tiles, in tiles

    Scheduler(const kvx_attn_plan *p_, int kind_, const AttnReq *reqs_, int n)
        : p(p_), reqs(reqs_), n_req(n), kind(kind_), group(p_->cfg.q_heads / p_->cfg.kv_heads),
          heads(p_->cfg.kv_heads), block_rows(kind_ == kTiles ? kBlockRows : kRowMax),
          tile_keys(kind_ == kTiles ? kTileKeys : kRowTile)
    {
        if (kind == kTiles) {
            const bool plain = p->cfg.softcap == 0.0f;
            unit_cost = plain ? kUnitTiles : kUnitTiles / 2;
            part_cost = plain ? kPartTiles : kPartTiles / 2;
            join_cost = plain ? kLaunchTiles : kLaunchTiles / 2;
        } else if (p->cfg.kv_type == KVX_TYPE_FP_FOUR) {
            kvx::four_units(p->cfg, p->token_bytes, &heads, &tile_keys);
            unit_cost = kFourUnitTiles;
            part_cost = kFourPartTiles;
            join_cost = kFourJoinTiles;
        } else {
            const int64_t tile_bytes = 2 * tile_keys * p->token_bytes / heads;
            unit_cost = std::max<int64_t>(1, kUnitBytes / tile_bytes);
            part_cost = std::max<int64_t>(1, kPartBytes / tile_bytes);
            join_cost = 0;
        }
    }
    int blocks(const AttnReq &r) const
    {
        return int((int64_t(r.n_new) * group + block_rows - 1) / block_rows);
    }
    int tiles_of(const AttnReq &r, int block) const
    {
        const int64_t row0 = int64_t(block) * block_rows;
        const int64_t row1 = std::min<int64_t>(row0 + block_rows, int64_t(r.n_new) * group) - 1;
        const int pmin = r.n_tokens - r.n_new + int(row0 / group);
        const int pmax = r.n_tokens - r.n_new + int(row1 / group);
        int first, skip, tiles;
        kvx::key_tiles(r.prefix, p->cfg.window ? std::max(0, pmin - p->cfg.window + 1) : 0,
                       pmax + 1, tile_keys, &first, &skip, &tiles);
        return tiles;
    }

    // Place the shares, cutting no unit closer than `least` tiles to its ends; into `out`, if
    // not NULL.  Returns the CTAs, and the slowest one's time in *slowest.
    int place(int64_t shares, int64_t total, int64_t least, kvx::AttnStart *out,
              int64_t *slowest) const
    {
        int64_t at = 0, line = 0;     // of the unit, in cost and in tiles
        int64_t share = 0;            // shares begun
        int64_t begun = 0, load = 0;  // line position where the last of them begins, its time
        int ctas = 0;
        bool carry = false;           // one begins with the next unit
        *slowest = 0;
        auto start = [&](int r, int b, int h, int64_t tile, int first) {
            if (ctas > 0 && out)
                out[ctas - 1].tiles = line + tile - begun;
            begun = line + tile;
            if (out)
                out[ctas] = {r, b, h, int32_t(tile), first, 0, 0, reqs[r]};
            ++ctas;
            *slowest = std::max(*slowest, load);
            load = 0;
        };
        for (int r = 0; r < n_req; ++r)
            for (int b = 0, n = blocks(reqs[r]); b < n; ++b) {
                const int64_t t = tiles_of(reqs[r], b);
                for (int h = 0; h < heads; ++h) {
                    // Shares whose boundary falls on this unit: at its start, inside, at its end.
                    auto boundary = [&] { return share * total / shares - at - unit_cost; };
                    int first = ctas - 1;
                    int64_t cut = 0;
                    bool begin = carry;
                    for (carry = false; share < shares && boundary() < std::min(least, t); ++share)
                        begin = true;
                    if (begin) {
                        first = ctas;
                        start(r, b, h, 0, first);
                    }
                    for (; share < shares && boundary() < t; ++share) {
                        if (t - boundary() < least) {
                            carry = true;
                        } else if (boundary() > cut) {
                            load += boundary() - cut + unit_cost + part_cost;
                            cut = boundary();
                            start(r, b, h, cut, first);
                        }
                    }
                    load += t - cut + unit_cost + (cut ? part_cost : 0);
                    if (out)
                        for (int c = first; c < ctas - 1; ++c)
                            out[c].last = ctas - 1;
                    at += t + unit_cost;
                    line += t;
                }
            }
        *slowest = std::max(*slowest, load);
        if (out)
            out[ctas - 1].tiles = line - begun;
        return ctas;
    }

    // Deal the units out, the longest first, each to the CTA that has the least so far; into
    // `out`, if not NULL.  Returns the shares, one per unit, and the slowest CTA's time.
    int deal(int ctas, kvx::AttnStart *out, int64_t *slowest) const
    {
        int n = 0, shares = 0;
        for (int r = 0; r < n_req; ++r)
            for (int b = 0, end = blocks(reqs[r]); b < end; ++b)
                p->blocks[n++] = {tiles_of(reqs[r], b), r, b};
        std::sort(p->blocks, p->blocks + n, [](const DealBlock &a, const DealBlock &b) {
            return a.tiles != b.tiles       ? a.tiles > b.tiles
                   : a.request != b.request ? a.request < b.request
                                            : a.block < b.block;
        });
        auto later = [](const DealCta &a, const DealCta &b) {
            return a.load != b.load ? a.load > b.load : a.cta > b.cta;
        };
        DealCta *heap = p->heap;  // the least at 0
        for (int c = 0; c < ctas; ++c)
            heap[c] = {0, c, -1};
        *slowest = 0;
        for (int i = 0; i < n; ++i)
            for (int h = 0; h < heads; ++h) {
                DealCta c = heap[0];
                const DealBlock &u = p->blocks[i];
                // The first one of CTA c is share c: equal loads go by number.
                if (out) {
                    out[shares] = {u.request, u.block, h, 0, 0, 0, u.tiles, reqs[u.request]};
                    if (c.at >= 0)
                        out[c.at].last = shares;
                }
                c.at = shares++;
                c.load += u.tiles + unit_cost;
                *slowest = std::max(*slowest, c.load);
                int at = 0;
                for (int next; (next = 2 * at + 1) < ctas; at = next) {
                    next += next + 1 < ctas && later(heap[next], heap[next + 1]);
                    if (!later(c, heap[next]))
                        break;
                    heap[at] = heap[next];
                }
                heap[at] = c;
            }
        return shares;
    }

    // Lay out the shares into `out`, if not NULL; returns the CTAs, the slowest one's time in
    // tiles and the shares (more than CTAs where units are dealt out).
    int run(kvx::AttnStart *out, int64_t *time, int *n_shares) const
    {
        int64_t tiles = 0, total = 0, units = 0;
        for (int r = 0; r < n_req; ++r)
            for (int b = 0, n = blocks(reqs[r]); b < n; ++b) {
                const int64_t t = tiles_of(reqs[r], b);
                tiles += t * heads;
                total += (t + unit_cost) * heads;
                units += heads;
            }
        *time = 0;
        *n_shares = 0;
        if (tiles == 0)
            return 0;
        const int64_t slots = int64_t(p->ctx->num_sms) * pick_kernel(p, kind).ctas_per_sm;
        // Over a 4-bit cache a single tile may be a share: a request of 1000 tokens 10.8 -> 8.7 us.
        const bool four = p->cfg.kv_type == KVX_TYPE_FP_FOUR && kind != kTiles;
        const int64_t least = four ? part_cost : 2 * part_cost, whole = INT32_MAX;
        const int64_t shares = std::min(slots, std::max<int64_t>(1, tiles / least));
        int64_t cut_time, whole_time;
        place(shares, total, least, nullptr, &cut_time);
        place(slots, total, whole, nullptr, &whole_time);
        cut_time += join_cost;
        if (kind == kTiles && units > slots && units <= p->most_dealt()) {
            *n_shares = deal(int(slots), out, time);
            if (*time < std::min(cut_time, whole_time))
                return int(slots);
        }
        return *n_shares = whole_time <= cut_time ? place(slots, total, whole, out, time)
                                                  : place(shares, total, least, out, time);
    }
};

kvx_status fill_plan(kvx_attn_plan *p, const kvx_request *reqs, int n_req, const int32_t *n_new,
                     const int32_t *prefix, cudaStream_t s)
{
    kvx_ctx *ctx = p->ctx;
    cudaError_t e = cudaEventSynchronize(p->copied);  // the image may still be being read
    if (e != cudaSuccess)
        return kvx::cuda_err(ctx, e, "waiting for the plan's last copy");
    const int group = p->cfg.q_heads / p->cfg.kv_heads;
    AttnReq *lists[kKinds + 1];
    for (int k = 0; k <= kKinds; ++k)
        lists[k] = reinterpret_cast<AttnReq *>(p->host + p->reqs_at(k));
    int counts[kKinds] = {};
    int64_t rows = 0;
    for (int r = 0; r < n_req; ++r) {
        const AttnReq x = {reqs[r].page_table, reqs[r].n_tokens, n_new[r], prefix ? prefix[r] : 0,
                           int32_t(rows), {0, 0}};
        lists[kKinds][r] = x;
        if (n_new[r] > 0) {
            const int64_t n = int64_t(n_new[r]) * group;
            const int k = n <= 8 ? kRows : n <= kRowMax ? kMoreRows : kTiles;
            lists[k][counts[k]++] = x;
        }
        rows += n_new[r];
    }
    p->n_req = n_req;
    p->rows = rows;
    // Few requests of few rows beside chunks go with the chunks, if that costs less than the
    // launch they would otherwise have.
    const int few = counts[kRows] + counts[kMoreRows];
    if (few > 0 && counts[kTiles] > 0) {
        AttnReq *all = lists[kTiles] + counts[kTiles];
        std::copy(lists[kRows], lists[kRows] + counts[kRows], all);
        std::copy(lists[kMoreRows], lists[kMoreRows] + counts[kMoreRows], all + counts[kRows]);
        int64_t alone, together;
        int n;
        Scheduler(p, kTiles, lists[kTiles], counts[kTiles]).run(nullptr, &alone, &n);
        Scheduler(p, kTiles, lists[kTiles], counts[kTiles] + few).run(nullptr, &together, &n);
        if (together <= alone + kLaunchTiles) {
            counts[kTiles] += few;
            counts[kRows] = counts[kMoreRows] = 0;
        }
    }
    int shares = 0;
    for (int k = 0; k < kKinds; ++k) {
        kvx::AttnStart *starts = reinterpret_cast<kvx::AttnStart *>(p->host + p->starts_at(k));
        int64_t time;
        p->ctas[k] = Scheduler(p, k, lists[k], counts[k]).run(starts, &time, &shares);
        int32_t *cuts = reinterpret_cast<int32_t *>(p->host + p->cuts_at(k));
        p->cuts[k] = p->most_parts[k] = 0;
        for (int c = 0; c + 1 < p->ctas[k]; ++c)
            if (starts[c + 1].tile > 0 && starts[c + 1].first == c) {
                cuts[p->cuts[k]++] = c;
                p->most_parts[k] = std::max(p->most_parts[k], starts[c].last - c + 1);
            }
        p->most_rows[k] = 0;
        for (int i = 0; i < counts[k]; ++i)
            p->most_rows[k] = std::max<int>(p->most_rows[k], lists[k][i].n_new * group);
    }
    if (n_req) {
        e = cudaMemcpyAsync(p->dev, p->host,
                            p->starts_at(kTiles) + shares * sizeof(kvx::AttnStart),
                            cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess)
            e = cudaEventRecord(p->copied, s);
    }
    return e == cudaSuccess ? KVX_OK : kvx::cuda_err(ctx, e, "plan copy");
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Describe each layer's K and V as a matrix [slots][heads x head_dim] for tensor copies of
// runs of keys: the largest power of two that divides the page size, up to a tile, so that a
// run never crosses pages.  Runs below eight keys, a cache of 8 or 4 bits (converted on the way)
// and slots past the copies' 32-bit coordinates stay with plain copies (box 0).
kvx_status make_maps(kvx_attn_plan *p)
{
    int box = 1;
    while (box < kTileKeys && p->page_size % (2 * box) == 0)
        box *= 2;
    const int64_t slots = int64_t(p->num_pages) * p->page_size;
    if (p->cfg.kv_type != p->cfg.type || box < 8 || slots > INT32_MAX)
        return KVX_OK;
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                     cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn)
        return kvx::set_err(p->ctx, KVX_ERR_CUDA, "cuTensorMapEncodeTiled not found");
    p->maps = new (std::nothrow) CUtensorMap[2 * size_t(p->num_layers)];
    if (!p->maps)
        return kvx::set_err(p->ctx, KVX_ERR_CAPACITY, "out of host memory");
    for (int i = 0; i < 2 * p->num_layers; ++i) {
        const cuuint64_t dims[2] = {cuuint64_t(p->cfg.kv_heads) * p->cfg.head_dim,
                                    cuuint64_t(slots)};
        const cuuint64_t stride[1] = {cuuint64_t(p->token_bytes)};
        const cuuint32_t shape[2] = {64, cuuint32_t(box)}, step[2] = {1, 1};
        const CUresult r = reinterpret_cast<EncodeTiled>(fn)(
            p->maps + i,
            p->cfg.kv_type == KVX_TYPE_HALF ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                            : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
            2, p->pools[i], dims, stride, shape, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS)
            return kvx::set_err(p->ctx, KVX_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", int(r));
    }
    p->box = box;
    return KVX_OK;
}

}  // namespace

extern "C" {

kvx_status kvx_attn_plan_create(kvx_ctx *ctx, const kvx_pool *pool, const kvx_request *reqs,
                                int n_req, const int32_t *n_new, const int32_t *prefix,
                                const kvx_attn_cfg *cfg, kvx_stream_t stream,
                                kvx_attn_plan **out)
{
    if (!ctx || !out)
        return KVX_ERR_INVALID_ARG;
    *out = nullptr;
    kvx_status st = kvx::validate_attn(pool, reqs, n_req, n_new, prefix, cfg, ctx->validation,
                                       true, ctx->err, sizeof ctx->err);
    if (st != KVX_OK)
        return st;
    kvx::DeviceGuard guard(ctx->device);
    if (!guard.ok)
        return kvx::set_err(ctx, KVX_ERR_CUDA, "cannot make device %d current", ctx->device);
    kvx_attn_plan *p = new (std::nothrow) kvx_attn_plan;
    if (!p)
        return kvx::set_err(ctx, KVX_ERR_CAPACITY, "out of host memory");
    p->ctx = ctx;
    p->cfg = *cfg;
    if (p->cfg.scale == 0.0f)
        p->cfg.scale = 1.0f / std::sqrt(float(cfg->head_dim));
    if (p->cfg.window > 1 << 30)  // longer than any request
        p->cfg.window = 0;
    p->page_size = pool->page_size;
    p->num_pages = pool->num_pages;
    p->num_layers = pool->num_layers;
    p->token_bytes = pool->token_bytes;
    p->capacity = n_req;
    p->pools = new (std::nothrow) char *[2 * size_t(pool->num_layers)];
    p->blocks = new (std::nothrow) DealBlock[size_t(p->most_dealt())];
    p->heap = new (std::nothrow) DealCta[size_t(ctx->num_sms)];
    if (!p->pools || !p->blocks || !p->heap) {
        kvx_attn_plan_destroy(p);
        return kvx::set_err(ctx, KVX_ERR_CAPACITY, "out of host memory");
    }
    kvx::pack_slabs(pool, p->pools);
    if ((st = make_maps(p)) != KVX_OK) {
        kvx_attn_plan_destroy(p);
        return st;
    }
    size_t partial = 0;
    cudaError_t e = cudaSuccess;
    for (int k = 0; k < kKinds && e == cudaSuccess; ++k) {
        const Kernel kn = pick_kernel(p, k);
        partial = std::max(partial, 2 * size_t(ctx->num_sms) * kn.ctas_per_sm * kn.slot_floats *
                                        sizeof(float));
        e = cudaFuncSetAttribute(kn.fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(kn.most_smem));
    }
    if (e == cudaSuccess)
        e = cudaHostAlloc(reinterpret_cast<void **>(&p->host), p->bytes(), cudaHostAllocDefault);
    if (e == cudaSuccess)
        e = cudaMalloc(reinterpret_cast<void **>(&p->dev), p->bytes());
    if (e == cudaSuccess)
        e = cudaMalloc(reinterpret_cast<void **>(&p->partial), partial);
    const size_t counters = size_t(p->most_ctas()) * sizeof(unsigned int);
    if (e == cudaSuccess)
        e = cudaMalloc(reinterpret_cast<void **>(&p->counters), counters);
    if (e == cudaSuccess)
        e = cudaMemsetAsync(p->counters, 0, counters, reinterpret_cast<cudaStream_t>(stream));
    if (e == cudaSuccess)
        e = cudaEventCreateWithFlags(&p->copied, cudaEventDisableTiming);
    if (e != cudaSuccess) {
        kvx_attn_plan_destroy(p);
        return kvx::cuda_err(ctx, e, "plan allocation");
    }
    st = fill_plan(p, reqs, n_req, n_new, prefix, reinterpret_cast<cudaStream_t>(stream));
    if (st == KVX_OK && (e = cudaEventSynchronize(p->copied)) != cudaSuccess)
        st = kvx::cuda_err(ctx, e, "plan copy");
    if (st != KVX_OK) {
        kvx_attn_plan_destroy(p);
        return st;
    }
    *out = p;
    return KVX_OK;
}

kvx_status kvx_attn_plan_update(kvx_attn_plan *p, const kvx_request *reqs, int n_req,
                                const int32_t *n_new, const int32_t *prefix,
                                kvx_stream_t stream)
{
    if (!p)
        return KVX_ERR_INVALID_ARG;
    kvx_ctx *ctx = p->ctx;
    // The pool was checked when the plan was made; its pointers live on in the plan.
    const kvx_pool pool = {p->num_layers, 2, p->page_size, p->num_pages, p->token_bytes,
                           reinterpret_cast<void *const *>(p->pools),
                           reinterpret_cast<void *const *>(p->pools)};
    kvx_status st = kvx::validate_attn(&pool, reqs, n_req, n_new, prefix, &p->cfg,
                                       ctx->validation, true, ctx->err, sizeof ctx->err);
    if (st != KVX_OK)
        return st;
    if (n_req > p->capacity)
        return kvx::set_err(ctx, KVX_ERR_CAPACITY, "%d requests, the plan holds %d", n_req,
                            p->capacity);
    kvx::DeviceGuard guard(ctx->device);
    if (!guard.ok)
        return kvx::set_err(ctx, KVX_ERR_CUDA, "cannot make device %d current", ctx->device);
    return fill_plan(p, reqs, n_req, n_new, prefix, reinterpret_cast<cudaStream_t>(stream));
}

void kvx_attn_plan_destroy(kvx_attn_plan *p)
{
    if (!p)
        return;
    {
        kvx::DeviceGuard guard(p->ctx->device);
        cudaDeviceSynchronize();
        if (p->copied)
            cudaEventDestroy(p->copied);
        for (void *d : {static_cast<void *>(p->dev), static_cast<void *>(p->counters),
                        static_cast<void *>(p->partial)})
            if (d)
                cudaFree(d);
        if (p->host)
            cudaFreeHost(p->host);
    }
    delete[] p->maps;
    delete[] p->pools;
    delete[] p->blocks;
    delete[] p->heap;
    delete p;
}

kvx_status kvx_append_tokens(const kvx_attn_plan *p, int layer, const void *k, const void *v,
                             int64_t k_stride, int64_t v_stride, float k_scale, float v_scale,
                             kvx_stream_t stream)
{
    if (!p)
        return KVX_ERR_INVALID_ARG;
    if (p->rows == 0)
        return KVX_OK;
    if (p->cfg.kv_type == KVX_TYPE_FP_FOUR)
        return kvx::append_rotated(p, layer, nullptr, nullptr, 0, nullptr, 0, k, v, k_stride,
                                   v_stride, k_scale, v_scale,
                                   reinterpret_cast<cudaStream_t>(stream));
    kvx_status st = io_check(p, layer, k, &k_stride, p->cfg.kv_heads, "k");
    if (st == KVX_OK)
        st = io_check(p, layer, v, &v_stride, p->cfg.kv_heads, "v");
    if (st == KVX_OK)
        st = scales_check(p, k_scale, v_scale);
    if (st != KVX_OK)
        return st;
    kvx::DeviceGuard guard(p->ctx->device);
    if (!guard.ok)
        return kvx::set_err(p->ctx, KVX_ERR_CUDA, "cannot make device %d current",
                            p->ctx->device);
    Append a = {step_of(p), {static_cast<const char *>(k), static_cast<const char *>(v)},
                {k_stride, v_stride}, {p->pools[2 * layer], p->pools[2 * layer + 1]},
                p->token_bytes, {k_scale, v_scale}, int32_t(p->token_bytes / 16)};
    const void *fn =
        p->cfg.type == KVX_TYPE_HALF
            ? p->cfg.kv_type == KVX_TYPE_HALF
                  ? reinterpret_cast<const void *>(kvx_append_kernel<KVX_TYPE_HALF, KVX_TYPE_HALF>)
                  : reinterpret_cast<const void *>(
                        kvx_append_kernel<KVX_TYPE_HALF, KVX_TYPE_FP_EIGHT>)
        : p->cfg.kv_type == KVX_TYPE_BFLOAT
            ? reinterpret_cast<const void *>(kvx_append_kernel<KVX_TYPE_BFLOAT, KVX_TYPE_BFLOAT>)
            : reinterpret_cast<const void *>(
                  kvx_append_kernel<KVX_TYPE_BFLOAT, KVX_TYPE_FP_EIGHT>);
    void *args[] = {&a};
    const cudaError_t e = launch_early(fn, dim3(unsigned((2 * p->rows + 7) / 8)), 256, 0,
                                       reinterpret_cast<cudaStream_t>(stream), args);
    return e == cudaSuccess ? KVX_OK : kvx::cuda_err(p->ctx, e, "append launch");
}

kvx_status kvx_attend(const kvx_attn_plan *p, int layer, const void *q, int64_t q_stride,
                      void *out, int64_t out_stride, float *lse, float k_scale, float v_scale,
                      kvx_stream_t stream)
{
    if (!p)
        return KVX_ERR_INVALID_ARG;
    if (p->rows == 0)
        return KVX_OK;
    kvx_status st = io_check(p, layer, q, &q_stride, p->cfg.q_heads, "q");
    if (st == KVX_OK)
        st = io_check(p, layer, out, &out_stride, p->cfg.q_heads, "out");
    if (st != KVX_OK)
        return st;
    if (reinterpret_cast<uintptr_t>(lse) & 3)
        return kvx::set_err(p->ctx, KVX_ERR_ALIGNMENT, "lse not 4-byte aligned");
    if (!std::isfinite(k_scale) || !std::isfinite(v_scale))
        return kvx::set_err(p->ctx, KVX_ERR_INVALID_ARG, "k_scale %g, v_scale %g",
                            double(k_scale), double(v_scale));
    kvx::DeviceGuard guard(p->ctx->device);
    if (!guard.ok)
        return kvx::set_err(p->ctx, KVX_ERR_CUDA, "cannot make device %d current",
                            p->ctx->device);
    const Attend a = {static_cast<const char *>(q), static_cast<char *>(out), lse, q_stride,
                      out_stride, p->pools[2 * layer], p->pools[2 * layer + 1], p->token_bytes,
                      p->cfg.slopes, p->ctx->status_dev, p->cfg.q_heads, p->cfg.kv_heads,
                      p->cfg.q_heads / p->cfg.kv_heads, p->cfg.window, p->page_size, p->num_pages,
                      Divisor::of(p->page_size), p->box, p->cfg.scale * k_scale, p->cfg.softcap, v_scale};
    for (int k = 0; k < kKinds; ++k) {
        if (p->ctas[k] == 0)
            continue;
        const Kernel kn = pick_kernel(p, k);
        const Work w = {reinterpret_cast<const AttnReq *>(p->dev + p->reqs_at(k)),
                        reinterpret_cast<const kvx::AttnStart *>(p->dev + p->starts_at(k)),
                        reinterpret_cast<const int32_t *>(p->dev + p->cuts_at(k)),
                        p->counters, p->partial};
        CUtensorMap none = {};
        CUtensorMap *maps[2] = {p->box ? p->maps + 2 * layer : &none,
                                p->box ? p->maps + 2 * layer + 1 : &none};
        // The kernels of few rows take the first two.
        void *args[] = {const_cast<Attend *>(&a), const_cast<Work *>(&w), maps[0], maps[1]};
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        cudaError_t e = launch_early(kn.fn, dim3(unsigned(p->ctas[k])), kn.threads, kn.smem, s,
                                     args);
        if (e == cudaSuccess && kn.join && p->cuts[k])
            e = launch_early(kn.join,
                             dim3(unsigned(p->cuts[k]),
                                  unsigned(kn.join_slices ? kn.join_slices
                                                          : kn.join_heads * p->most_rows[k])),
                             kn.join_threads, 0, s, args);
        if (e != cudaSuccess)
            return kvx::cuda_err(p->ctx, e, "attention launch");
    }
    return KVX_OK;
}

}  // extern "C"
