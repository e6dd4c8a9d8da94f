// kvx_pages.cu -- page upkeep of a paged KV cache on the device: fork (share by count, copy),
// free and compact.  Entry points and kernels; the checks and packing are in
// kvx_cache_host.cpp.
//
// The one question these operators ask is "which pages are free": fork needs the i-th free
// page, compaction pairs the i-th live page past the front with the i-th free one in it.  Both
// are rank and select on the bitmap refs[p] > 0.  Every CTA builds that bitmap in its own
// shared memory (one pass over refs, which stays in L2; a fork stops as soon as it has seen
// enough free pages) and answers its own queries there, so a call is one launch with no
// device-wide wait, no list in global memory and no order-dependent atomics.  Nothing may
// change a page between free and live while another CTA still scans: such writes are left to
// the last CTA that has scanned.  Until then counts of live pages only go up, which no bitmap
// sees.  CTAs count themselves in refs, below zero at the first page that will turn live: a
// page whose count is not positive is free, so no bitmap sees that either, the last CTA's
// writes leave no trace of it, and calls share nothing but the pool they work on.
//
// Measured: copies of whole requests (6.7 GB read and written) 993 us, the rate of a device
// copy, and compaction (4.1 GB) 622 us, 98 % of it; one request forked into four (256 tails of
// 18 KB), with the free before it, 5.9 us, 64 children of a beam step (28 MB of tails) 11.9: two
// launches, the scan, one page lookup and one copy in a row.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "kvx_cache.h"
#include "kvx_ctx.h"

using kvx::ForkEntry;
using kvx::TableEntry;

namespace {

// Descriptors up to this size travel as a kernel parameter (the parameter space of a launch
// was 4 KB before CUDA 12.1 and a call stays within it); larger batches take a descriptor slot.
const int kInlineBytes = 3840;
// 12 warps of a CTA copy, 4 see to tables: 24 KiB of loads in flight per SM and 8 KiB to a
// job carry copies of whole requests at the rate of a device copy (6.77 TB/s); with 28 or 14
// warps, or 16 KiB jobs, they reached 91-96 % of it.
const int kThreads = 512;
const int kWarps = kThreads / 32;
const int kGranWords = 8;                // bitmap words per granule
const int kGranPages = 32 * kGranWords;  // pages per granule: one warp scans one at a time
const int kTableWarps = 4;               // of a CTA that also copies
const int64_t kSliceBytes = 8192;        // of a warp's job where there are many
const int kUnits = 8;                    // 16-byte loads in flight per lane, or half as many of 32

struct Inline {
    uint4 bytes[kInlineBytes / 16];
};

struct Args {
    const char *ext;         // descriptors in device memory, or NULL: in the Inline parameter
    int32_t inline_bytes;    // of them there
    int32_t *refs;
    unsigned int *status;
    int32_t *n_live;         // compact
    int32_t *remap;          // compact
    int64_t token_bytes;
    int64_t slice;           // bytes a warp copies per job
    int32_t off_entries;     // of the entries, after the slab pointers
    int32_t n_entries;
    int32_t n_slabs;
    int32_t page_size;
    int32_t num_pages;
    int32_t slices;          // jobs per (page, slab)
    int32_t wide;            // everything that is copied is 32-byte aligned
    int32_t table_warps;     // of each CTA, for tables; the others copy
};

// -------------------------------------------------------------------------------- device

__device__ __forceinline__ int ld_ref(const int32_t *p)
{
    return __ldcg(p);  // L2: another CTA's atomics change counts while this launch runs
}

// These kernels start while the one before them on the stream ends (programmatic dependent
// launch): they touch memory only past this wait for its completion, and let the next one
// start in the same way.
__device__ __forceinline__ void wait_for_earlier_work()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The call's descriptors where searching them is cheap: inline ones are brought into shared
// memory (at `to`; the caller's next barrier ends it).
__device__ __forceinline__ const char *descriptors(const Args &a, const Inline &in, char *to)
{
    if (a.ext)
        return a.ext;
    for (int i = threadIdx.x; i < a.inline_bytes / 16; i += kThreads)
        reinterpret_cast<uint4 *>(to)[i] = in.bytes[i];
    return to;
}

// The bitmap of one kind of page (free or live) with running totals per granule.
struct Bits {
    unsigned *words;   // [granules * kGranWords]
    int *before;       // [granules + 1]: set bits in earlier granules
    int granules;      // scanned
    int total;         // set bits found

    // Page of the i-th set bit, i < total.
    __device__ int select(int i) const
    {
        int lo = 0, hi = granules;  // before[lo] <= i < before[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before[mid] <= i)
                lo = mid;
            else
                hi = mid;
        }
        int k = i - before[lo], w = lo * kGranWords;
        for (int n; k >= (n = __popc(words[w])); ++w)
            k -= n;
        unsigned m = words[w];
        int bit = 0;
#pragma unroll
        for (int half = 16; half; half >>= 1) {
            const int n = __popc(m & ((1u << half) - 1));
            if (k >= n) {
                k -= n;
                m >>= half;
                bit += half;
            } else {
                m &= (1u << half) - 1;
            }
        }
        return w * 32 + bit;
    }

    // Set bits below page p, p <= 32 * kGranWords * granules.
    __device__ int rank(int p) const
    {
        int w = p >> 5, r = before[w / kGranWords];
        for (int i = w / kGranWords * kGranWords; i < w; ++i)
            r += __popc(words[i]);
        if (p & 31)
            r += __popc(words[w] & ((1u << (p & 31)) - 1));
        return r;
    }

    __device__ bool test(int p) const { return words[p >> 5] >> (p & 31) & 1; }
};

// Build the bitmap of pages whose (refs > 0) equals `live`, in rounds of one granule per warp,
// until `enough` bits are set or the pool ends.  All threads; ends with a barrier.
__device__ Bits scan_pages(const Args &a, bool live, int enough, unsigned *smem)
{
    __shared__ int round_count[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int all = (a.num_pages + kGranPages - 1) / kGranPages;
    Bits b;
    b.words = smem;
    b.before = reinterpret_cast<int *>(smem + all * kGranWords);
    int found = 0, g0 = 0;
    for (; g0 < all && found < enough; g0 += kWarps) {
        const int g = g0 + warp;
        int n = 0;
        if (g < all) {
            int v[kGranWords];
#pragma unroll
            for (int i = 0; i < kGranWords; ++i) {
                const int p = g * kGranPages + i * 32 + lane;
                v[i] = p < a.num_pages ? ld_ref(a.refs + p) : (live ? 0 : 1);
            }
#pragma unroll
            for (int i = 0; i < kGranWords; ++i) {
                const unsigned m = __ballot_sync(0xffffffffu, (v[i] > 0) == live);
                if (lane == i)
                    b.words[g * kGranWords + i] = m;
                n += __popc(m);
            }
        }
        if (lane == 0)
            round_count[warp] = n;
        __syncthreads();
        const int c = lane < kWarps ? round_count[lane] : 0;
        int incl = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d)
                incl += x;
        }
        if (warp == 0 && lane < kWarps && g0 + lane <= all)
            b.before[g0 + lane] = found + incl - c;
        found += __shfl_sync(0xffffffffu, incl, 31);
        __syncthreads();
    }
    b.granules = g0 < all ? g0 : all;
    b.total = found;
    if (threadIdx.x == 0)
        b.before[b.granules] = found;
    __syncthreads();
    return b;
}

// Arrival of this CTA's scan, by one thread, after a barrier that ends the scan; and, past a
// later barrier, whether it was the last CTA of the launch to arrive.  `count` is that of a
// free page, 0 before the launch.
__device__ void arrive(int32_t *count, int *last)
{
    __threadfence();
    *last = atomicSub(count, 1) == 1 - int(gridDim.x);
    __threadfence();
}

// Entry that owns flat index i: the last e with begin(e) <= i, begin of the sentinel > i.
template <class E, class F>
__device__ __forceinline__ int find_entry(const E *entries, int n, int i, F begin)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (begin(entries[mid]) <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

struct V32 {
    unsigned r[8];
};

__device__ __forceinline__ V32 ld_32(const V32 *p)
{
    V32 v;
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v.r[0]), "=r"(v.r[1]), "=r"(v.r[2]), "=r"(v.r[3]), "=r"(v.r[4]),
                   "=r"(v.r[5]), "=r"(v.r[6]), "=r"(v.r[7])
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void st_32(V32 *p, const V32 &v)
{
    asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
                 "r"(v.r[0]), "r"(v.r[1]), "r"(v.r[2]), "r"(v.r[3]), "r"(v.r[4]), "r"(v.r[5]),
                 "r"(v.r[6]), "r"(v.r[7])
                 : "memory");
}

// One warp copies `bytes` (a multiple of 32, addresses too) with kUnits / 2 32-byte loads in
// flight per lane.
__device__ __forceinline__ void warp_copy_32(const char *src, char *dst, int64_t bytes, int lane)
{
    const int kN = kUnits / 2;
    const V32 *s = reinterpret_cast<const V32 *>(src) + lane;
    V32 *d = reinterpret_cast<V32 *>(dst) + lane;
    int64_t rem = bytes / 32 - lane;
    for (; rem > 0; rem -= 32 * kN, s += 32 * kN, d += 32 * kN) {
        V32 r[kN];
#pragma unroll
        for (int u = 0; u < kN; ++u)
            if (32 * u < rem)
                r[u] = ld_32(s + 32 * u);
#pragma unroll
        for (int u = 0; u < kN; ++u)
            if (32 * u < rem)
                st_32(d + 32 * u, r[u]);
    }
}

// One warp copies `bytes` (a multiple of 16) with kUnits 16-byte loads in flight per lane.
__device__ __forceinline__ void warp_copy(const char *src, char *dst, int64_t bytes, int lane)
{
    const uint4 *s = reinterpret_cast<const uint4 *>(src) + lane;
    uint4 *d = reinterpret_cast<uint4 *>(dst) + lane;
    int64_t rem = bytes / 16 - lane;
    for (; rem > 32 * (kUnits - 1); rem -= 32 * kUnits, s += 32 * kUnits, d += 32 * kUnits) {
        uint4 r[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
            r[u] = __ldcs(s + 32 * u);
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
            __stcs(d + 32 * u, r[u]);
    }
    if (rem > 0) {
        uint4 r[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
            if (32 * u < rem)
                r[u] = __ldcs(s + 32 * u);
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
            if (32 * u < rem)
                __stcs(d + 32 * u, r[u]);
    }
}

// Copy slice `slice` of `tokens` tokens from page `from` to page `to` in slab `slab`.
__device__ __forceinline__ void copy_slice(const Args &a, const char *desc, int slab, int slice,
                                           int from, int to, int tokens, int lane)
{
    const int64_t bytes = int64_t(tokens) * a.token_bytes, at = slice * a.slice;
    if (at >= bytes)
        return;
    char *base = reinterpret_cast<char *const *>(desc)[slab];
    const int64_t page = int64_t(a.page_size) * a.token_bytes;
    const int64_t n = bytes - at < a.slice ? bytes - at : a.slice;
    if (a.wide)
        warp_copy_32(base + from * page + at, base + to * page + at, n, lane);
    else
        warp_copy(base + from * page + at, base + to * page + at, n, lane);
}

__global__ void __launch_bounds__(kThreads, 1)
kvx_fork_kernel(const Args a, const __grid_constant__ Inline in)
{
    extern __shared__ unsigned smem[];
    __shared__ int last;
    __shared__ Inline staged;
    const char *desc = descriptors(a, in, reinterpret_cast<char *>(&staged));
    const ForkEntry *e = reinterpret_cast<const ForkEntry *>(desc + a.off_entries);
    const int lane = threadIdx.x & 31;
    __syncthreads();
    const ForkEntry end = e[a.n_entries];
    wait_for_earlier_work();
    const Bits free = scan_pages(a, false, end.fresh_begin, smem);
    if (free.total < end.fresh_begin) {  // the same in every CTA: counts of live pages only grow
        if (blockIdx.x == 0 && threadIdx.x == 0)
            atomicOr(a.status, KVX_DEV_NO_FREE_PAGE);
        return;
    }
    if (end.fresh_begin > 0 && threadIdx.x == 0)
        arrive(a.refs + free.select(0), &last);

    // Pages past the scan do not turn live in this launch.
    auto is_free = [&](int p) {
        return p < free.granules * kGranPages ? free.test(p) : ld_ref(a.refs + p) <= 0;
    };

    // Tables, and the counts of shared pages, by the last warps of every CTA (by all, if there
    // is nothing to copy) beside the copies of the others.  There are up to 2^31 - 1 entries;
    // the step past the last of them fits in 32 bits without a sign.
    const int warp = threadIdx.x >> 5, copy_warps = kWarps - a.table_warps;
    const int table_threads = 32 * a.table_warps;
    for (unsigned i = blockIdx.x * table_threads + threadIdx.x - 32 * copy_warps;
         warp >= copy_warps && i < unsigned(end.page_begin); i += gridDim.x * table_threads) {
        const int x = find_entry(e, a.n_entries, i, [](const ForkEntry &f) { return f.page_begin; });
        const int j = i - e[x].page_begin;
        if (j >= e[x].full) {
            e[x].child[j] = free.select(e[x].fresh_begin + j - e[x].full);
        } else if (!e[x].grow) {
            int p = e[x].parent[j];
            unsigned bad = 0;
            if (unsigned(p) >= unsigned(a.num_pages))
                bad = KVX_DEV_PAGE_OUT_OF_RANGE;
            else if (is_free(p))
                bad = KVX_DEV_PAGE_NOT_HELD;
            if (bad) {
                atomicOr(a.status, bad);
                p = -1;
            } else {
                atomicAdd(a.refs + p, 1);
            }
            e[x].child[j] = p;
        }
    }
    // Copies: jobs in the order (page, slab, slice).
    const int64_t jobs = int64_t(end.copy_begin) * a.n_slabs * a.slices;
    for (int64_t job = int64_t(blockIdx.x) * copy_warps + warp; warp < copy_warps && job < jobs;
         job += int64_t(gridDim.x) * copy_warps) {
        const unsigned t = unsigned(job) / unsigned(a.slices);  // jobs < 2^31 (host)
        const int slice = int(unsigned(job) - t * a.slices);
        const int c = int(t / unsigned(a.n_slabs)), slab = int(t - unsigned(c) * a.n_slabs);
        const int x = find_entry(e, a.n_entries, c, [](const ForkEntry &f) { return f.copy_begin; });
        const int j = e[x].full + c - e[x].copy_begin;
        const int from = e[x].parent[j];
        unsigned bad = 0;
        if (unsigned(from) >= unsigned(a.num_pages))
            bad = KVX_DEV_PAGE_OUT_OF_RANGE;
        else if (is_free(from))
            bad = KVX_DEV_PAGE_NOT_HELD;
        if (bad) {
            if (lane == 0)
                atomicOr(a.status, bad);
            continue;
        }
        const int to = free.select(e[x].fresh_begin + j - e[x].full);
        copy_slice(a, desc, slab, slice, from, to,
                   min(a.page_size, e[x].shared - j * a.page_size), lane);
    }
    __syncthreads();
    if (end.fresh_begin > 0 && last)
        for (int i = threadIdx.x; i < end.fresh_begin; i += kThreads)
            a.refs[free.select(i)] = 1;
}

__global__ void __launch_bounds__(kThreads, 1)
kvx_free_kernel(const Args a, const __grid_constant__ Inline in)
{
    __shared__ Inline staged;
    const char *desc = descriptors(a, in, reinterpret_cast<char *>(&staged));
    const TableEntry *e = reinterpret_cast<const TableEntry *>(desc + a.off_entries);
    __syncthreads();
    const unsigned total = e[a.n_entries].page_begin;
    wait_for_earlier_work();
    for (unsigned i = blockIdx.x * kThreads + threadIdx.x; i < total; i += gridDim.x * kThreads) {
        const int x = find_entry(e, a.n_entries, i, [](const TableEntry &t) { return t.page_begin; });
        int32_t *at = e[x].pages + (i - e[x].page_begin);
        const int p = *at;
        unsigned bad = 0;
        if (unsigned(p) >= unsigned(a.num_pages)) {
            bad = KVX_DEV_PAGE_OUT_OF_RANGE;
        } else if (atomicSub(a.refs + p, 1) <= 0) {
            // Not held: taken back, so that however such entries interleave the count ends
            // at zero.
            atomicAdd(a.refs + p, 1);
            bad = KVX_DEV_PAGE_NOT_HELD;
        }
        if (bad)
            atomicOr(a.status, bad);
        *at = -1;
    }
}

__global__ void __launch_bounds__(kThreads, 1)
kvx_compact_kernel(const Args a, const __grid_constant__ Inline in)
{
    extern __shared__ unsigned smem[];
    __shared__ int last;
    __shared__ Inline staged;
    const char *desc = descriptors(a, in, reinterpret_cast<char *>(&staged));
    const TableEntry *e = reinterpret_cast<const TableEntry *>(desc + a.off_entries);
    const int lane = threadIdx.x & 31;
    wait_for_earlier_work();
    const Bits live = scan_pages(a, true, a.num_pages + 1, smem);
    const int n = live.total, front = live.rank(n), moves = n - front;
    // Page of the i-th free page below n: the smallest p with (p - rank(p)) pages free before
    // it and p free, by bisection over pages.
    auto hole = [&](int i) {
        int lo = 0, hi = live.granules;  // free before granule lo <= i
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (mid * kGranPages - live.before[mid] <= i)
                lo = mid;
            else
                hi = mid;
        }
        int k = i - (lo * kGranPages - live.before[lo]), w = lo * kGranWords;
        for (int z; k >= (z = 32 - __popc(live.words[w])); ++w)
            k -= z;
        unsigned m = ~live.words[w];
        int bit = 0;
#pragma unroll
        for (int half = 16; half; half >>= 1) {
            const int z = __popc(m & ((1u << half) - 1));
            if (k >= z) {
                k -= z;
                m >>= half;
                bit += half;
            } else {
                m &= (1u << half) - 1;
            }
        }
        return w * 32 + bit;
    };
    if (moves > 0 && threadIdx.x == 0)
        arrive(a.refs + hole(0), &last);
    if (a.n_live && blockIdx.x == 0 && threadIdx.x == 0)
        *a.n_live = n;

    const int warp = threadIdx.x >> 5, copy_warps = kWarps - a.table_warps;
    const int table_threads = 32 * a.table_warps;
    const unsigned mine = blockIdx.x * table_threads + threadIdx.x - 32 * copy_warps;
    const unsigned total = e[a.n_entries].page_begin;
    for (unsigned i = mine; warp >= copy_warps && i < total; i += gridDim.x * table_threads) {
        const int x = find_entry(e, a.n_entries, i, [](const TableEntry &t) { return t.page_begin; });
        int32_t *at = e[x].pages + (i - e[x].page_begin);
        const int p = *at;
        if (unsigned(p) >= unsigned(a.num_pages))
            atomicOr(a.status, KVX_DEV_PAGE_OUT_OF_RANGE);
        else if (!live.test(p))
            atomicOr(a.status, KVX_DEV_PAGE_NOT_HELD);
        else if (p >= n)
            *at = hole(live.rank(p) - front);
    }
    if (a.remap)
        for (int p = int(mine); warp >= copy_warps && p < a.num_pages;
             p += gridDim.x * table_threads)
            a.remap[p] = !live.test(p) ? -1 : p < n ? p : hole(live.rank(p) - front);

    const int64_t jobs = int64_t(moves) * a.n_slabs * a.slices;
    for (int64_t job = int64_t(blockIdx.x) * copy_warps + warp; warp < copy_warps && job < jobs;
         job += int64_t(gridDim.x) * copy_warps) {
        const unsigned t = unsigned(job) / unsigned(a.slices);
        const int slice = int(unsigned(job) - t * a.slices);
        const int c = int(t / unsigned(a.n_slabs)), slab = int(t - unsigned(c) * a.n_slabs);
        copy_slice(a, desc, slab, slice, live.select(front + c), hole(c), a.page_size, lane);
    }
    __syncthreads();
    if (moves > 0 && last)
        for (int i = threadIdx.x; i < moves; i += kThreads) {
            const int from = live.select(front + i);
            a.refs[hole(i)] = ld_ref(a.refs + from);
            a.refs[from] = 0;
        }
}

// ---------------------------------------------------------------------------------- host

size_t bitmap_bytes(int num_pages)
{
    const size_t granules = (size_t(num_pages) + kGranPages - 1) / kGranPages;
    return granules * kGranWords * 4 + (granules + kWarps + 1) * 4;
}

// Cut `units` pages of up to `page` bytes into slices so that every copying warp of the grid
// has one job, or, past that, jobs of about 8 KiB; no slice below 1 KiB.
void choose_slices(const kvx_ctx *ctx, int64_t units, int64_t page, Args *a)
{
    const int64_t warps = int64_t(ctx->num_sms) * (kWarps - kTableWarps);
    const int64_t fill = units > 0 ? std::max<int64_t>(1, warps / units) : 1;
    int64_t slice = std::max<int64_t>((page + fill - 1) / fill, 1024);
    if (units * page > 2 * kSliceBytes * warps)
        slice = std::min<int64_t>(slice, kSliceBytes);
    slice = (slice + 31) / 32 * 32;
    a->slice = slice;
    a->slices = int32_t((page + slice - 1) / slice);
}

struct Batch {
    Inline in;
    kvx::Slot *slot = nullptr;
    char *host = nullptr;
    size_t bytes = 0;
};

// Where a call's descriptors are packed: the launch's own parameter, or a context slot.
kvx_status begin_batch(kvx_ctx *ctx, size_t bytes, Batch *b)
{
    b->bytes = bytes;
    if (bytes <= size_t(kInlineBytes)) {
        b->host = reinterpret_cast<char *>(&b->in);
        return KVX_OK;
    }
    kvx_status st = kvx::acquire_slot(ctx, bytes, &b->slot);
    if (st == KVX_OK)
        b->host = b->slot->host;
    return st;
}

kvx_status launch_batch(kvx_ctx *ctx, void (*fn)(Args, Inline), Args a, Batch *b, int64_t ctas,
                        size_t smem, int64_t items, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    a.inline_bytes = b->slot ? 0 : int32_t((b->bytes + 15) / 16 * 16);
    if (b->slot) {
        a.ext = b->slot->dev;
        e = kvx::stage(ctx, *b->slot, b->bytes, 0, 0, s);
    }
    if (e != cudaSuccess)
        return kvx::cuda_err(ctx, e, "descriptor copy");
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(unsigned(ctas));
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = smem;  // up to what prepare_upkeep asked for
    lc.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    void *args[] = {&a, &b->in};
    e = cudaLaunchKernelExC(&lc, reinterpret_cast<const void *>(fn), args);
    if (e != cudaSuccess)
        return kvx::cuda_err(ctx, e, "kernel launch");
    if (b->slot)
        return kvx::finish_call(ctx, *b->slot, s, items, ctas, kThreads, b->bytes);
    ctx->last_items = items;
    ctx->last_ctas = int32_t(ctas);
    ctx->last_threads = kThreads;
    ctx->last_desc_bytes = int64_t(b->bytes);
    return KVX_OK;
}

Args common_args(kvx_ctx *ctx, const kvx_pool *pool, int32_t *refs, int n)
{
    Args a = {};
    a.refs = refs;
    a.status = ctx->status_dev;
    a.token_bytes = pool->token_bytes;
    a.n_entries = n;
    a.n_slabs = pool->num_layers * pool->kv_factor;
    a.off_entries = int32_t((size_t(a.n_slabs) * sizeof(char *) + 15) / 16 * 16);
    a.page_size = pool->page_size;
    a.num_pages = pool->num_pages;
    uintptr_t bits = uintptr_t(pool->token_bytes);
    for (int l = 0; l < pool->num_layers; ++l)
        for (int k = 0; k < pool->kv_factor; ++k)
            bits |= reinterpret_cast<uintptr_t>((k ? pool->v_pages : pool->k_pages)[l]);
    a.wide = bits % 32 == 0;
    return a;
}

kvx_status too_many_jobs(kvx_ctx *ctx, int64_t pages, const Args &a)
{
    return pages > INT32_MAX / (int64_t(a.n_slabs) * a.slices)
               ? kvx::set_err(ctx, KVX_ERR_CAPACITY, "%lld pages x %d slabs x %d slices exceed "
                              "2^31 copies", (long long)pages, a.n_slabs, a.slices)
               : KVX_OK;
}

}  // namespace

cudaError_t kvx::prepare_upkeep()
{
    const int smem = int(bitmap_bytes(KVX_MAX_UPKEEP_PAGES));
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kvx_fork_kernel),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kvx_compact_kernel),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return e;
}

extern "C" {

kvx_status kvx_fork_pages(kvx_ctx *ctx, const kvx_pool *pool, int32_t *refs,
                          const kvx_fork *forks, int n_forks, kvx_stream_t stream)
{
    if (!ctx)
        return KVX_ERR_INVALID_ARG;
    kvx::begin_call(ctx);
    kvx_status st = kvx::validate_upkeep(pool, refs, forks, n_forks, nullptr, 0, ctx->validation,
                                         true, ctx->err, sizeof ctx->err);
    if (st != KVX_OK)
        return st;
    kvx::DeviceGuard guard(ctx->device);
    if (!guard.ok)
        return kvx::set_err(ctx, KVX_ERR_CUDA, "cannot make device %d current", ctx->device);
    Args a = common_args(ctx, pool, refs, n_forks);
    Batch b;
    st = begin_batch(ctx, a.off_entries + (size_t(n_forks) + 1) * sizeof(ForkEntry), &b);
    if (st != KVX_OK)
        return st;
    kvx::pack_slabs(pool, reinterpret_cast<char **>(b.host));
    ForkEntry *e = reinterpret_cast<ForkEntry *>(b.host + a.off_entries);
    st = kvx::pack_forks(pool, forks, n_forks, e, ctx->err, sizeof ctx->err);
    if (st != KVX_OK)
        return st;
    const ForkEntry &end = e[n_forks];
    if (end.page_begin == 0)
        return KVX_OK;
    int64_t longest = 0;  // tokens of a page that is copied
    for (int i = 0; i < n_forks; ++i)
        if (e[i + 1].copy_begin > e[i].copy_begin)
            longest = std::max<int64_t>(longest, std::min(e[i].shared - e[i].full *
                                                          pool->page_size, pool->page_size));
    choose_slices(ctx, int64_t(end.copy_begin) * a.n_slabs,
                  std::max<int64_t>(longest, 1) * pool->token_bytes, &a);
    if ((st = too_many_jobs(ctx, end.copy_begin, a)) != KVX_OK)
        return st;
    a.table_warps = end.copy_begin ? kTableWarps : kWarps;
    const int64_t jobs = int64_t(end.copy_begin) * a.n_slabs * a.slices;
    const int copy_warps = std::max(1, kWarps - a.table_warps);
    const int64_t ctas = std::min<int64_t>(
        ctx->num_sms, std::max((jobs + copy_warps - 1) / copy_warps,
                               (int64_t(end.page_begin) + 32 * a.table_warps - 1) /
                                   (32 * a.table_warps)));
    return launch_batch(ctx, kvx_fork_kernel, a, &b, ctas, bitmap_bytes(pool->num_pages), jobs,
                        reinterpret_cast<cudaStream_t>(stream));
}

static kvx_status tables_call(kvx_ctx *ctx, const kvx_pool *pool, int32_t *refs,
                              const kvx_table *tables, int n_tables, int32_t *n_live,
                              int32_t *remap, bool compact, kvx_stream_t stream)
{
    if (!ctx)
        return KVX_ERR_INVALID_ARG;
    kvx::begin_call(ctx);
    kvx_status st = kvx::validate_upkeep(pool, refs, nullptr, 0, tables, n_tables,
                                         ctx->validation, true, ctx->err, sizeof ctx->err);
    if (st != KVX_OK)
        return st;
    if ((reinterpret_cast<uintptr_t>(n_live) | reinterpret_cast<uintptr_t>(remap)) & 3)
        return kvx::set_err(ctx, KVX_ERR_ALIGNMENT, "n_live or remap not 4-byte aligned");
    kvx::DeviceGuard guard(ctx->device);
    if (!guard.ok)
        return kvx::set_err(ctx, KVX_ERR_CUDA, "cannot make device %d current", ctx->device);
    Args a = common_args(ctx, pool, refs, n_tables);
    if (!compact)
        a.off_entries = a.n_slabs = 0;
    Batch b;
    st = begin_batch(ctx, a.off_entries + (size_t(n_tables) + 1) * sizeof(TableEntry), &b);
    if (st != KVX_OK)
        return st;
    if (compact)
        kvx::pack_slabs(pool, reinterpret_cast<char **>(b.host));
    TableEntry *e = reinterpret_cast<TableEntry *>(b.host + a.off_entries);
    st = kvx::pack_tables(tables, n_tables, e, ctx->err, sizeof ctx->err);
    if (st != KVX_OK)
        return st;
    const int64_t entries = e[n_tables].page_begin;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!compact) {
        if (entries == 0)
            return KVX_OK;
        const int64_t ctas = std::min<int64_t>(ctx->num_sms, (entries + kThreads - 1) / kThreads);
        return launch_batch(ctx, kvx_free_kernel, a, &b, ctas, 0, entries, s);
    }
    a.n_live = n_live;
    a.remap = remap;
    a.table_warps = kTableWarps;
    // How many pages move is known on the device only: at most half the pool.
    choose_slices(ctx, int64_t(pool->num_pages) * a.n_slabs / 4,
                  int64_t(pool->page_size) * pool->token_bytes, &a);
    if ((st = too_many_jobs(ctx, pool->num_pages / 2, a)) != KVX_OK)
        return st;
    return launch_batch(ctx, kvx_compact_kernel, a, &b, ctx->num_sms,
                        bitmap_bytes(pool->num_pages), entries, s);
}

kvx_status kvx_free_pages(kvx_ctx *ctx, const kvx_pool *pool, int32_t *refs,
                          const kvx_table *tables, int n_tables, kvx_stream_t stream)
{
    return tables_call(ctx, pool, refs, tables, n_tables, nullptr, nullptr, false, stream);
}

kvx_status kvx_compact_pages(kvx_ctx *ctx, const kvx_pool *pool, int32_t *refs,
                             const kvx_table *tables, int n_tables, int32_t *n_live,
                             int32_t *remap, kvx_stream_t stream)
{
    return tables_call(ctx, pool, refs, tables, n_tables, n_live, remap, true, stream);
}

}  // extern "C"
