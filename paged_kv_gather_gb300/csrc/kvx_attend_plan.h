// kvx_attend_plan.h -- the plan behind kvx_attn_plan: a step's batch on the device, what every
// kernel that works on it takes from it, and how the attention kernels are named.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kvx_attend.cuh"
#include "kvx_cache.h"
#include "kvx_ctx.h"

// The attention kernels by the rows (new tokens x heads that share a KV head) of a request:
// up to 8, up to 16, more.
enum { kRows = 0, kMoreRows = 1, kTiles = 2, kKinds = 3 };

// What a unit costs beyond its tiles, and what each part of one costs that is cut, measured:
// in bytes of K and V read meanwhile for the kernels of few rows, in tiles for the other
// (half as many where a cap on the scores makes tiles take twice as long).
const int64_t kUnitBytes = 128 << 10, kPartBytes = 48 << 10;
const int64_t kUnitTiles = 4, kPartTiles = 2;

// A launch more, in tiles' time.
const int64_t kLaunchTiles = 3;

// The same of the kernel of few rows over a 4-bit cache, whose parts are joined by a launch of
// its own, in its tiles.
const int64_t kFourUnitTiles = 2, kFourPartTiles = 1, kFourJoinTiles = 2;

// Up to this many units per SM are dealt out one by one (Scheduler::deal); past it the shares
// of the line come out as even, and the descriptors long.
const int kDealtPerSm = 16;

// Scratch of the schedule.
struct DealBlock {
    int64_t tiles;
    int32_t request, block;
};
struct DealCta {
    int64_t load;
    int32_t cta, at;  // its number, its latest share
};

// Kernel of a kind, with its shared memory and the floats of a partial result.
struct Kernel {
    const void *fn;
    int threads, ctas_per_sm;
    size_t smem;
    int slot_floats;
    const void *join;  // of the parts of cut units, or NULL: the kernel joins them itself
    int join_threads;
    int join_slices;   // CTAs that share out a unit's rows, or 0 ...
    int join_heads;    // ... for one CTA per head of a unit and row of a request
    size_t most_smem;  // of any plan's launch of fn: what is asked for once and stays
};

struct kvx_attn_plan {
    kvx_ctx *ctx = nullptr;
    kvx_attn_cfg cfg = {};
    int32_t page_size = 0, num_pages = 0, num_layers = 0;
    int64_t token_bytes = 0;
    char **pools = nullptr;    // host: [2 * layer + kv]
    int capacity = 0;          // requests
    int n_req = 0;
    int64_t rows = 0;
    int ctas[kKinds] = {};     // of each kernel's launch
    int cuts[kKinds] = {};     // units that it cuts
    int most_parts[kKinds] = {};  // of one of them
    int most_rows[kKinds] = {};   // of a request: new tokens x heads that share a KV head
    // Descriptors: [AttnReq of each kind, of all][CTAs of each kind that begin a unit that is
    // cut][AttnStart of each kind, the last one's with room for units dealt out]; a pinned image,
    // and the device's copy.
    char *host = nullptr, *dev = nullptr;
    DealBlock *blocks = nullptr;       // [most_dealt()]
    DealCta *heap = nullptr;           // [num_sms]
    CUtensorMap *maps = nullptr;       // host: as pools, where the cache is copied by tensor copies
    int32_t box = 0;                   // keys per copy, 0: it is not
    unsigned int *counters = nullptr;  // [most_ctas()], zero between launches
    float *partial = nullptr;          // serves one kind's launch after the other
    cudaEvent_t copied = nullptr;      // the last update's copy

    int most_ctas() const { return 2 * ctx->num_sms; }  // of a launch
    int most_dealt() const { return kDealtPerSm * ctx->num_sms; }
    size_t reqs_at(int k) const  // k = kKinds: all requests, for append
    {
        return size_t(k) * capacity * sizeof(AttnReq);
    }
    size_t cuts_at(int k) const
    {
        return reqs_at(kKinds + 1) + size_t(k) * most_ctas() * sizeof(int32_t);
    }
    size_t starts_at(int k) const
    {
        return (cuts_at(kKinds) + 63) / 64 * 64 +
               size_t(k) * most_ctas() * sizeof(kvx::AttnStart);
    }
    size_t bytes() const
    {
        return starts_at(kTiles) +
               std::max(most_ctas(), most_dealt()) * sizeof(kvx::AttnStart);
    }
};

namespace {

struct Step {
    const AttnReq *reqs;
    unsigned int *status;
    int32_t n_req;
    int32_t rows;
    int32_t page_size;
    int32_t num_pages;
    Divisor page;
};

// Request of a row: the last r with row_begin <= row that has rows.  Requests without new
// tokens share their row_begin with the next one, and the last of equals is taken.
__device__ __forceinline__ int request_of_row(const AttnReq *reqs, int n, int row, int lane)
{
    int lo = 0, hi = n;  // row_begin[lo] <= row < row_begin[hi]
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int idx = lo + lane * step;
        const bool ok = idx < hi && __ldg(&reqs[idx].row_begin) <= row;
        const unsigned m = __ballot_sync(0xffffffffu, ok);
        lo += (31 - __clz(m)) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

inline Step step_of(const kvx_attn_plan *p)
{
    return {reinterpret_cast<const AttnReq *>(p->dev + p->reqs_at(kKinds)), p->ctx->status_dev,
            p->n_req, int32_t(p->rows), p->page_size, p->num_pages, Divisor::of(p->page_size)};
}

// A launch that may start while the kernel ahead of it on the stream drains; the kernels
// themselves wait for that one's completion before they touch memory.
inline cudaError_t launch_early(const void *fn, dim3 ctas, int threads, size_t smem,
                                cudaStream_t s, void **args)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = ctas;
    lc.blockDim = dim3(unsigned(threads));
    lc.dynamicSmemBytes = smem;
    lc.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelExC(&lc, fn, args);
}

// The checks of one tensor of a step: its layer, pointer, and stride, which is returned in bytes.
inline kvx_status io_check(const kvx_attn_plan *p, int layer, const void *x, int64_t *stride,
                           int64_t heads, const char *what)
{
    const int64_t packed = heads * p->cfg.head_dim;
    if (layer < 0 || layer >= p->num_layers)
        return kvx::set_err(p->ctx, KVX_ERR_INVALID_ARG, "layer %d outside [0, %d)", layer,
                            p->num_layers);
    if (!x)
        return kvx::set_err(p->ctx, KVX_ERR_INVALID_ARG, "%s is NULL", what);
    if (*stride == 0)
        *stride = packed;
    if (*stride < packed)
        return kvx::set_err(p->ctx, KVX_ERR_INVALID_ARG, "%s: stride %lld below %lld elements",
                            what, (long long)*stride, (long long)packed);
    if ((reinterpret_cast<uintptr_t>(x) & 15) || *stride % 8)
        return kvx::set_err(p->ctx, KVX_ERR_ALIGNMENT, "%s not 16-byte aligned (stride %lld)",
                            what, (long long)*stride);
    *stride *= 2;  // bytes
    return KVX_OK;
}

// The scales of an append: divided by where the cache has fewer bits than the new tokens.
inline kvx_status scales_check(const kvx_attn_plan *p, float k_scale, float v_scale)
{
    // Reciprocals of a 4-bit cache's factors stay normal numbers.
    const bool four = p->cfg.kv_type == KVX_TYPE_FP_FOUR;
    const float least = four ? 0x1p-100f : 0.0f, most = four ? 0x1p100f : HUGE_VALF;
    auto fits = [&](float x) { return x > 0.0f && x >= least && x <= most && std::isfinite(x); };
    if (p->cfg.kv_type != p->cfg.type && !(fits(k_scale) && fits(v_scale)))
        return kvx::set_err(p->ctx, KVX_ERR_INVALID_ARG, "k_scale %g, v_scale %g",
                            double(k_scale), double(v_scale));
    return KVX_OK;
}

}  // namespace

namespace kvx {

// Of a 4-bit cache: the kernels of a kind (kvx_attend_four.cu) for units cut into so many parts,
// and how a unit of theirs is made up, the groups of KV heads and the keys of a step.
Kernel four_kernel(const kvx_attn_cfg &c, int64_t token_bytes, int kind, int most_parts);
void four_units(const kvx_attn_cfg &c, int64_t token_bytes, int *groups, int *keys);

// kvx_append_rotated's launch; without rope and q, kvx_append_tokens into a 4-bit cache
// (kvx_rotate.cu).
kvx_status append_rotated(const kvx_attn_plan *p, int layer, const kvx_rope *rope, const void *q,
                          int64_t q_stride, void *q_out, int64_t q_out_stride, const void *k,
                          const void *v, int64_t k_stride, int64_t v_stride, float k_scale,
                          float v_scale, cudaStream_t s);

}  // namespace kvx
