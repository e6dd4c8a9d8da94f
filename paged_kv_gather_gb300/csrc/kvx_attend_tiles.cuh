// kvx_attend_tiles.cuh -- attention of more than 16 rows per KV head (prefill chunks, many
// drafted tokens): every key meets enough rows that the tensor cores bound the kernel.
// Included by kvx_attend.cu only.
#pragma once

#include "kvx_attend.cuh"

namespace {

// A CTA takes a block of 256 rows (new tokens x the heads that share a KV head, packed) of one
// KV head as two tiles of 128, 128 keys at a time.  Tensor memory holds, per tile, the scores
// S (128 columns) and the output O (D columns), 512 columns in all at D = 128; the weights P
// go back into the columns of S as the first operand of P V, so they never pass through
// shared memory.  Two warpgroups turn the scores of one tile each into weights, a thread per
// row, while the tensor cores work on the other tile: S0 -> P0 beside P1 V, S1 and so on.
// One warp issues the products; three warps bring K and V from the pages into a ring of
// shared-memory slots (K0, V0, K1, V1, ...).  Where a tile of keys is whole and a page holds
// eight keys or a power of two more, one of them fetches it with tensor copies, a run of keys
// inside a page each: with 16-byte copies by the threads of all three, the only way for other
// pages and ragged ends, the ring was what the kernel waited for.  An e4m3 cache is copied as
// it is into a stage of its own and from there converted to half precision in the ring.
//
// Shared-memory tiles are [D / 64][128 rows][64 elements] with the 16-byte chunks of a
// 128-byte line permuted by the row's low three bits, the layout the matrix instructions
// call 128-byte swizzle.  K and q are read along it, V across it (its rows are the summed
// index), so the same copy serves both.
//
// A step of 256 rows x 128 keys costs the tensor cores 2048 cycles and takes 2950 (units 128
// steps longer, at the clock sampled meanwhile; the tensor pipe is active 66-69 % of the
// cycles): each tile's own chain (scores out, maximum, weights, the second half of P V, the next
// scores) is 1490 + 1050 of them by counters in the kernel, and tensor memory is full at
// D = 128, so no third tile fills the gap.  With options a step takes 3710 (bias), 5060 (cap),
// 5300 (both) or 7820 cycles (scores past half the cap), with a cap the tensor pipe active 40 %
// and the FMA pipe 37 % of them: S is read, shaped and written back one
// block of 32 columns after the other, and read again for the weights.  Over an e4m3 cache,
// converted by three warps, it takes 3620; at D = 64 2270, of which 1024 are products.
// Measured: 2048 new tokens x 8 heads behind 32k tokens (2.13 TFLOP) 1.37 ms on its own and
// 1.45-1.5 ms in long runs under the power cap (cuBLAS sustains 1.70 PFLOP/s there).  A unit
// costs about 9000 cycles beside its steps (q in, first scores, O out), which is what short
// prompts pay: 2k tokens 36 us, 8k 373 us.
const int kTileThreads = 384;
const int kTileRows = 128;
const int kTileKeys = 128;
const int kBlockRows = 2 * kTileRows;
const int kLoaders = 96;
const int kLoaderWarps = kLoaders / 32;
const int kLoaderLag = 2;          // slots filled by 16-byte copies before the first is announced

// Barriers, by index: of the two tiles of rows first, then the loaders', the ring's, the end's.
enum {
    kBarQ = 0,      // q is in shared memory
    kBarS = 2,      // S is complete, and every product before it
    kBarP = 4,      // P of the first 64 keys is in tensor memory
    kBarP2 = 6,     // and of the others
    kBarO = 8,      // O is complete
    kBarKeys = 10,  // the loaders among themselves
    kBarFull = 11,
    kBarEmpty = 21,
    kBarEnd = 31,
    kBars = 32
};

template <int KV, int D>
struct TileShape {
    static const bool kEight = KV == KVX_TYPE_FP_EIGHT;
    static const int kTile = kTileRows * D * 2;              // bytes of a q, K or V tile
    static const int kSlots = (D == 128 ? 5 : 10) - kEight;
    static const int kOffRing = 2 * kTile;
    static const int kOffStage = kOffRing + kSlots * kTile;  // e4m3: [2][kTile / 2]
    static const int kOffKeys = kOffStage + kEight * kTile;  // int64 [2][kTileKeys]
    static const int kOffBars = kOffKeys + 2 * kTileKeys * 8;
    static const int kOffMisc = kOffBars + 8 * kBars;        // int[2]
    static const int kBytes = kOffMisc + 16;
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
    static const int kSlotFloats = kBlockRows * (D + 2);     // a partial result: O, m, l
};

__device__ __forceinline__ void mbar_init(unsigned bar, unsigned count)
{
    asm volatile("mbarrier.init.shared.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(unsigned bar)
{
    asm volatile("mbarrier.arrive.shared.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try(unsigned bar, unsigned phase)
{
    unsigned ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared.b64 p, [%1], %2; "
                 "selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(phase)
                 : "memory");
    return ok;
}

__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

// Wait for a phase of a barrier, for about a second at most; then, or once another wait of
// the CTA has run out, false.  The answer is the same for a whole warp.  Past the wait for
// earlier work, which every role of the CTA does before its first barrier, so that the second
// is this kernel's own, no thread waits in any other way before the last barrier: a wait that
// runs out ends the launch.
__device__ __forceinline__ bool mbar_wait(unsigned bar, unsigned phase, volatile int *gave_up,
                                          unsigned *status)
{
    bool ok = mbar_try(bar, phase);
    if (!__all_sync(0xffffffffu, ok)) {
        const uint64_t t0 = now_ns();
        for (;;) {
            for (int i = 0; i < 64 && !ok; ++i)
                ok = mbar_try(bar, phase);
            if (__all_sync(0xffffffffu, ok))
                return true;
            if (__any_sync(0xffffffffu, *gave_up != 0))
                return false;
            if (__any_sync(0xffffffffu, now_ns() - t0 > 1000000000ull)) {
                *gave_up = 1;
                atomicOr(status, KVX_DEV_WAIT_TIMEOUT);
                return false;
            }
        }
    }
    return true;
}

// The same for a thread on its own.
__device__ __forceinline__ bool mbar_wait_one(unsigned bar, unsigned phase, volatile int *gave_up,
                                              unsigned *status)
{
    if (mbar_try(bar, phase))
        return true;
    const uint64_t t0 = now_ns();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try(bar, phase))
                return true;
        if (*gave_up)
            return false;
        if (now_ns() - t0 > 1000000000ull) {
            *gave_up = 1;
            atomicOr(status, KVX_DEV_WAIT_TIMEOUT);
            return false;
        }
    }
}

// One thread of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    unsigned one;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }"
                 : "=r"(one)::"memory");
    return one;
}

__device__ __forceinline__ void fence_async_shared()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_commit(unsigned bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::
                     "r"(bar)
                 : "memory");
}

// D (tensor memory) = A B, or += with `add`; A in shared or tensor memory, B in shared.
__device__ __forceinline__ void tc_mma_ss(unsigned d, uint64_t a, uint64_t b, unsigned idesc,
                                          bool add)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; "
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a),
                 "l"(b), "r"(idesc), "r"(unsigned(add))
                 : "memory");
}

__device__ __forceinline__ void tc_mma_ts(unsigned d, unsigned a, uint64_t b, unsigned idesc,
                                          bool add)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; "
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a),
                 "l"(b), "r"(idesc), "r"(unsigned(add))
                 : "memory");
}

// 32 (16) consecutive columns of this thread's lane of tensor memory.
__device__ __forceinline__ void tc_ld32(float (&r)[32], unsigned addr)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
          "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
          "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]),
          "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]),
          "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tc_st32(unsigned addr, const float (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
        "%29, %30, %31, %32};" ::"r"(addr),
        "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]),
        "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]),
        "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]), "f"(r[19]), "f"(r[20]), "f"(r[21]),
        "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]), "f"(r[26]), "f"(r[27]), "f"(r[28]),
        "f"(r[29]), "f"(r[30]), "f"(r[31])
        : "memory");
}

__device__ __forceinline__ void tc_st16(unsigned addr, const unsigned (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

// The loads into r are complete; keeps uses of r behind the wait.
__device__ __forceinline__ void tc_wait_ld(float (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i)
        asm volatile("" : "+f"(r[i]));
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float max3_abs(float a, float b, float c)
{
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};

// The bits 0 .. n - 1 of 32.
__device__ __forceinline__ unsigned bits_below(int n)
{
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1;
}

// Two 32-bit numbers at a time.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ float2 halves_of(uint64_t x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}

__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void tc_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory operand with 128-byte swizzle: 8-row groups 1024 bytes apart; `lead` bytes
// between 64-element blocks where the operand is read across its lines.
__device__ __forceinline__ uint64_t tile_desc(unsigned addr, unsigned lead)
{
    return uint64_t((addr & 0x3ffff) >> 4) | uint64_t(lead >> 4) << 16 | uint64_t(1024 >> 4) << 32 |
           uint64_t(1) << 46 | uint64_t(2) << 61;
}

// kind::f16 with 32-bit accumulators, M = 128.
__host__ __device__ constexpr unsigned mma_idesc(int type, int n, bool b_across)
{
    return 1u << 4 | unsigned(type == KVX_TYPE_BFLOAT) << 7 | unsigned(type == KVX_TYPE_BFLOAT) << 10 |
           unsigned(b_across) << 16 | unsigned(n / 8) << 17 | unsigned(128 / 16) << 24;
}

// Byte offset of 16-byte chunk c of row r in a shared-memory tile.
__device__ __forceinline__ int tile_at(int r, int c)
{
    return (c >> 3) * (kTileRows * 128) + r * 128 + (((c ^ r) & 7) << 4);
}

// A box of a matrix in global memory into shared memory; completes on a barrier.
__device__ __forceinline__ void tensor_copy(unsigned dst, const CUtensorMap *map, int x, int y,
                                            unsigned bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void mbar_expect(unsigned bar, unsigned bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

// Walks a CTA's share of the line, or the units dealt to it; every role of the CTA steps through
// the same units.
struct Walk {
    const Attend &a;
    const Work &w;
    AttnStart at;
    AttnReq r;
    Keys keys;
    int row0, rows, todo;   // of the block; tiles of keys to do

    __device__ __forceinline__ Walk(const Attend &a_, const Work &w_, const AttnStart &at_)
        : a(a_), w(w_), at(at_)
    {
        if (!done())
            enter();
    }
    __device__ __forceinline__ bool done() const { return at.tiles <= 0; }
    // The CTAs that begin and end the unit.
    __device__ __forceinline__ int begun_by() const
    {
        return at.tile > 0 ? at.first : int(blockIdx.x);
    }
    __device__ __forceinline__ int ended_by() const
    {
        return at.tile + todo < keys.tiles ? at.last : int(blockIdx.x);
    }
    // Key that step i begins at.  Last keys first: where a bias favours near keys, the largest
    // score is then met early and O is hardly ever rescaled.
    __device__ __forceinline__ int key_of(int i) const
    {
        const int t = keys.tiles - 1 - at.tile - i;
        return (t < keys.first ? t : t + keys.skip) * kTileKeys;
    }
    __device__ __forceinline__ void enter()
    {
        r = at.req;
        const int all = r.n_new * a.group;
        row0 = at.block * kBlockRows;
        rows = min(kBlockRows, all - row0);
        keys.set<kTileKeys>(r, a.window, row0 / a.group, (row0 + rows - 1) / a.group);
        todo = int(min(int64_t(keys.tiles - at.tile), at.tiles));
    }
    __device__ __forceinline__ void next()
    {
        at.tiles -= todo;
        if (done()) {
            if (at.last == 0 || at.tile + todo < keys.tiles)
                return;
            at = w.starts[at.last];
            enter();
            return;
        }
        at.tile = 0;
        if (++at.head == a.kv_heads) {
            at.head = 0;
            if ((++at.block) * kBlockRows >= r.n_new * a.group) {
                at.block = 0;
                at.req = w.reqs[++at.request];
            }
        }
        enter();
    }
};

template <int TYPE, int KV, int D>
__global__ void __launch_bounds__(kTileThreads, 1)
kvx_attend_tiles_kernel(const Attend a, const Work w, const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap v_map)
{
    typedef TileShape<KV, D> T;
    typedef Elem<TYPE> E;
    constexpr bool kEight = KV == KVX_TYPE_FP_EIGHT;
    constexpr int kMath = kEight ? KVX_TYPE_HALF : TYPE;
    typedef Elem<kMath> P;
    char *smem = attend_smem;
    int *misc = reinterpret_cast<int *>(smem + T::kOffMisc);
    int &gave_up = misc[0];
    unsigned &tmem_base = reinterpret_cast<unsigned &>(misc[1]);
    const unsigned sm = smem_u32(smem);
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    auto bar = [&](int i) { return sm + T::kOffBars + 8 * i; };
    auto wait = [&](int i, unsigned phase) { return mbar_wait(bar(i), phase, &gave_up, a.status); };

    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(&tmem_base))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar(kBarQ + x), kTileRows);
            mbar_init(bar(kBarS + x), 1);
            mbar_init(bar(kBarP + x), kTileRows);
            mbar_init(bar(kBarP2 + x), kTileRows);
            mbar_init(bar(kBarO + x), 1);
        }
        mbar_init(bar(kBarKeys), kLoaders);
        mbar_init(bar(kBarEnd), 1);
        for (int i = 0; i < T::kSlots; ++i) {
            mbar_init(bar(kBarFull + i), kLoaderWarps);
            mbar_init(bar(kBarEmpty + i), 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const unsigned tmem = tmem_base;
    const AttnStart begin = w.starts[blockIdx.x];
    bool waited = false;  // for earlier work: the first unit's arithmetic goes before it

    if (warp == 8) {
        // ------------------------------------------------------------- matrix products
        // One thread does it all: the queue of products is a few deep, so every instruction
        // between the last of one batch and the first of the next shows once the weights of
        // the other tile are there in time.
        if (elect_one()) {
            wait_for_earlier_work();
            constexpr unsigned kDescS = mma_idesc(kMath, kTileKeys, false);
            constexpr unsigned kDescO = mma_idesc(kMath, D, true);
            const uint64_t q_desc = tile_desc(sm, 16);
            const uint64_t k_desc = tile_desc(sm + T::kOffRing, 16);
            const uint64_t v_desc = tile_desc(sm + T::kOffRing, kTileRows * 128);
            unsigned slot = 0, turn = 0;  // ring position and its phase
            unsigned q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
            bool ok = true;
            auto wait1 = [&](int i, unsigned phase) {
                return mbar_wait_one(bar(i), phase, &gave_up, a.status);
            };
            auto scores = [&](int x, unsigned s) {
                const uint64_t q = q_desc + x * (T::kTile >> 4), k = k_desc + s * (T::kTile >> 4);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint64_t step = ((i >> 2) * (kTileRows * 128) + (i & 3) * 32) >> 4;
                    tc_mma_ss(tmem + x * kTileKeys, q + step, k + step, kDescS, i > 0);
                }
                tc_commit(bar(kBarS + x));
            };
            auto advance = [&]() {
                if (++slot == T::kSlots) {
                    slot = 0;
                    turn ^= 1;
                }
            };
            for (Walk u(a, w, begin); ok && !u.done(); u.next()) {
                const int tiles = u.rows > kTileRows ? 2 : 1;
                for (int x = 0; ok && x < tiles; ++x) {
                    ok = wait1(kBarQ + x, q_phase[x]);
                    q_phase[x] ^= 1;
                }
                if (!ok || !(ok = wait1(kBarFull + slot, turn)))
                    break;
                tc_fence_after();
                for (int x = 0; x < tiles; ++x)
                    scores(x, slot);
                tc_commit(bar(kBarEmpty + slot));
                advance();
                for (int i = 0; i < u.todo; ++i) {
                    const unsigned v_slot = slot;
                    if (!(ok = wait1(kBarFull + slot, turn)))
                        break;
                    advance();
                    const bool more = i + 1 < u.todo;
                    if (more && !(ok = wait1(kBarFull + slot, turn)))
                        break;
                    const uint64_t v = v_desc + v_slot * (T::kTile >> 4);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (x >= tiles)
                            break;
                        // P V of the first 64 keys runs while the weights of the others are
                        // still being made.
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if (!(ok = wait1((half ? kBarP2 : kBarP) + x, p_phase[x])))
                                break;
                            tc_fence_after();
#pragma unroll
                            for (int k = half * (kTileKeys / 32); k < (half + 1) * (kTileKeys / 32);
                                 ++k)
                                tc_mma_ts(tmem + 2 * kTileKeys + x * D,
                                          tmem + x * kTileKeys + 8 * k, v + (k * 2048 >> 4),
                                          kDescO, k > 0 || i > 0);
                        }
                        if (!ok)
                            break;
                        p_phase[x] ^= 1;
                        if (more)
                            scores(x, slot);
                        else
                            tc_commit(bar(kBarO + x));
                    }
                    if (!ok)
                        break;
                    tc_commit(bar(kBarEmpty + v_slot));
                    if (more) {
                        tc_commit(bar(kBarEmpty + slot));
                        advance();
                    }
                }
            }
            if (!ok) {
                // Let what was issued run out before the memory it works on goes away.
                tc_commit(bar(kBarEnd));
                const uint64_t t0 = now_ns();
                while (!mbar_try(bar(kBarEnd), 0) && now_ns() - t0 < 1000000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp > 8) {
        // ------------------------------------------------------------- K and V
        const int lt = threadIdx.x - (kTileThreads - kLoaders);
        int64_t *offs = reinterpret_cast<int64_t *>(smem + T::kOffKeys);  // [2][kTileKeys]
        constexpr int kRow = D * (kEight ? 1 : 2), kChunks = kRow / 16;
        constexpr int kCopies = (kTileKeys * kChunks + kLoaders - 1) / kLoaders;  // per thread
        constexpr unsigned kPerTile = D / 64;  // tensor copies side by side
        unsigned slot = 0, turn = 0;
        unsigned filled = 0, announced = 0;    // slots of the stream so far
        bool ok = true;
        // This warp's part of slot number `announced` is in place.
        auto announce = [&]() {
            fence_async_shared();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(kBarFull + announced % T::kSlots));
            ++announced;
        };
        auto advance = [&]() {
            ++filled;
            if (++slot == T::kSlots) {
                slot = 0;
                turn ^= 1;
            }
        };
        // Copy this thread's chunks of 16 bytes of a tile, where each key lies at off[key].
        auto copy = [&](const char *base, const int64_t *off, unsigned dst) {
            int64_t o[kCopies];  // all at once: nothing moves across an asynchronous copy
#pragma unroll
            for (int b = 0; b < kCopies; ++b) {
                const int x = lt + b * kLoaders;
                o[b] = x < kTileKeys * kChunks ? off[x / kChunks] : -1;
            }
#pragma unroll
            for (int b = 0; b < kCopies; ++b) {
                const int x = lt + b * kLoaders, t = x / kChunks, c = x % kChunks;
                if (x < kTileKeys * kChunks)
                    cp_async16(dst + (kEight ? x * 16 : tile_at(t, c)),
                               base + (o[b] >= 0 ? o[b] : 0) + c * 16, o[b] >= 0);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        unsigned key_phase = 0;
        // e4m3: tile sides (K, V, K, V, ...) are copied one ahead of their conversion.
        bool staged = false;
        auto convert = [&]() {  // the staged side, number `filled` of the stream
            const char *src = smem + T::kOffStage + (filled & 1) * (T::kTile / 2);
            char *dst = smem + T::kOffRing + slot * T::kTile;
            uint4 in[kCopies];  // all at once: loads do not move up across stores
#pragma unroll
            for (int b = 0; b < kCopies; ++b) {
                const int x = lt + b * kLoaders;
                if (x < kTileKeys * kChunks)
                    in[b] = *reinterpret_cast<const uint4 *>(src + x * 16);
            }
#pragma unroll
            for (int b = 0; b < kCopies; ++b) {
                const int x = lt + b * kLoaders, t = x / kChunks, c = x % kChunks;
                if (x < kTileKeys * kChunks) {
                    uint4 h0, h1;
                    half4_of_e4m3(in[b].x, h0.x, h0.y);
                    half4_of_e4m3(in[b].y, h0.z, h0.w);
                    half4_of_e4m3(in[b].z, h1.x, h1.y);
                    half4_of_e4m3(in[b].w, h1.z, h1.w);
                    *reinterpret_cast<uint4 *>(dst + tile_at(t, 2 * c)) = h0;
                    *reinterpret_cast<uint4 *>(dst + tile_at(t, 2 * c + 1)) = h1;
                }
            }
            announce();
            advance();
        };
        for (Walk u(a, w, begin); ok && !u.done(); u.next()) {
            if (!waited)
                wait_for_earlier_work();
            waited = true;
            // The loaders are ahead of the warps that will read this unit's rows of q.
            for (int i = lt; i < u.rows * (D / 64); i += kLoaders) {
                const int packed = u.row0 + i / (D / 64), tok = packed / a.group;
                const char *q = a.q + int64_t(u.r.row_begin + tok) * a.q_stride +
                                (u.at.head * a.group + packed - tok * a.group) * (D * 2) +
                                i % (D / 64) * 128;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
            }
            const int64_t head_at = int64_t(u.at.head) * kRow;
            // A lane per tensor copy of a tile: run of keys `lane / kPerTile` and 64-element
            // block of the head `lane % kPerTile`; its page is looked up a tile ahead.
            const int run = a.box ? int(unsigned(lane) / kPerTile) * a.box : kTileKeys;
            auto page_of = [&](int i) {
                const int j = i < u.todo ? u.key_of(i) + run : 0;
                return i < u.todo && run < kTileKeys && u.keys.used(j)
                           ? u.r.table[a.page.div(j)] : -1;
            };
            int next = kEight ? -1 : page_of(0);
            // Page of key lt + b * kLoaders of tile i.
            auto key_page = [&](int i, int b) {
                const int t = lt + b * kLoaders;
                const int j = i < u.todo && t < kTileKeys ? u.key_of(i) + t : 0;
                return i < u.todo && t < kTileKeys && u.keys.used(j)
                           ? u.r.table[a.page.div(j)] : -1;
            };
            int later[2] = {-1, -1};
            for (int i = 0; ok && i < u.todo; ++i) {
                const int j0 = u.key_of(i);
                if (!kEight) {
                    const int page = next;
                    next = page_of(i + 1);
                    if (a.box && u.keys.whole<kTileKeys>(j0) &&
                        __all_sync(0xffffffffu, run >= kTileKeys ||
                                                    unsigned(page) < unsigned(a.num_pages))) {
                        const int j = j0 + run;
                        const int y = page * a.page_size + j - a.page.div(j) * a.page_size;
                        for (int side = 0; side < 2; ++side) {
                            if (!(ok = wait(kBarEmpty + slot, turn ^ 1)))
                                break;
                            if (lane == 0) {
                                if (warp == 9)
                                    mbar_expect(bar(kBarFull + slot), T::kTile);
                                else
                                    mbar_arrive(bar(kBarFull + slot));
                            }
                            __syncwarp();
                            if (warp == 9 && run < kTileKeys) {
                                const int block = int(unsigned(lane) % kPerTile);
                                tensor_copy(sm + T::kOffRing + slot * T::kTile +
                                                block * (kTileRows * 128) + run * 128,
                                            side ? &v_map : &k_map, u.at.head * D + block * 64, y,
                                            bar(kBarFull + slot));
                            }
                            ++announced;
                            advance();
                        }
                        continue;
                    }
                }
                // Where each key of the tile lies; -1: not used.
                int64_t *off = offs + key_phase * kTileKeys;
                int page[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    // Looked up a tile ahead where every tile comes this way.
                    page[b] = !a.box && i > 0 ? later[b] : key_page(i, b);
                    later[b] = a.box ? -1 : key_page(i + 1, b);
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int t = lt + b * kLoaders, j = j0 + t;
                    if (t < kTileKeys) {
                        int64_t o = -1;
                        if (u.keys.used(j)) {
                            if (unsigned(page[b]) < unsigned(a.num_pages))
                                o = (int64_t(page[b]) * a.page_size + j -
                                     a.page.div(j) * a.page_size) * a.token_bytes + head_at;
                            else
                                atomicOr(a.status, KVX_DEV_PAGE_OUT_OF_RANGE);
                        }
                        off[t] = o;
                    }
                }
                mbar_arrive(bar(kBarKeys));
                ok = wait(kBarKeys, key_phase);
                key_phase ^= 1;
                for (int side = 0; ok && side < 2; ++side) {
                    const char *base = side ? a.v : a.k;
                    if (kEight) {
                        // The stage that this side takes was converted two sides ago.
                        copy(base, off, sm + T::kOffStage +
                                            ((filled + staged) & 1) * (T::kTile / 2));
                        if (staged) {
                            asm volatile("cp.async.wait_group 1;" ::: "memory");
                            if ((ok = wait(kBarEmpty + slot, turn ^ 1)))
                                convert();
                        }
                        staged = true;
                        continue;
                    }
                    if (!(ok = wait(kBarEmpty + slot, turn ^ 1)))
                        break;
                    copy(base, off, sm + T::kOffRing + slot * T::kTile);
                    advance();
                    if (a.box) {  // alone between tiles that come by tensor copies
                        asm volatile("cp.async.wait_group 0;" ::: "memory");
                        announce();
                    } else if (filled - announced > kLoaderLag) {
                        asm volatile("cp.async.wait_group %0;" ::"n"(kLoaderLag) : "memory");
                        announce();
                    }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (ok && staged && (ok = wait(kBarEmpty + slot, turn ^ 1)))
            convert();
        while (ok && announced < filled)
            announce();
        if (!ok && warp == 9) {
            // Tensor copies may still be under way: see the slots filled last complete.
            const uint64_t t0 = now_ns();
            for (unsigned n = filled > T::kSlots ? filled - T::kSlots : 0; n < filled; ++n)
                while (!__all_sync(0xffffffffu,
                                   mbar_try(bar(kBarFull + n % T::kSlots), n / T::kSlots & 1)) &&
                       !__any_sync(0xffffffffu, now_ns() - t0 > 1000000000ull)) {
                }
        }
    } else {
        // ------------------------------------------------------------- weights
        const int x = warp >> 2;                        // tile of rows
        const int row = threadIdx.x & (kTileRows - 1);  // and row in it
        const unsigned lanes = unsigned(warp & 3) << 21;
        const unsigned ts = tmem + lanes + x * kTileKeys;
        const unsigned to = tmem + lanes + 2 * kTileKeys + x * D;
        const Score score(a);
        // Rows of q and out as a warp reads and writes them: kRowsAtOnce of its 32 at a time,
        // kRowChunks lanes to a row.
        constexpr int kRowChunks = D / 8, kRowsAtOnce = 32 / kRowChunks;
        const int sub_row = lane / kRowChunks, sub_chunk = lane % kRowChunks;
        const int warp_row = row & ~31;
        unsigned s_phase = 0, o_phase = 0;
        bool ok = true;
        for (Walk u(a, w, begin); ok && !u.done(); u.next()) {
            const bool mine = x == 0 || u.rows > kTileRows;  // the tile has rows
            const bool have = x * kTileRows + row < u.rows;
            const int packed = u.row0 + (have ? x * kTileRows + row : 0);
            const int tok = packed / a.group, head = u.at.head * a.group + packed - tok * a.group;
            const int pos = u.r.n_tokens - u.r.n_new + tok;
            const int64_t orow = u.r.row_begin + tok;
            if (!waited)
                wait_for_earlier_work();
            waited = true;
            const float slope = a.slopes ? a.slopes[head] * kLog2e : 0.0f;
            float row_factor = 1.0f;
            if (mine) {
                // q into shared memory.  A warp reads its 32 rows a few whole rows at a time:
                // with a row per thread, every load and store of the warp met 32 lines.
                const int64_t off = have ? orow * a.q_stride + head * (D * 2) : -1;
                char *dst = smem + x * T::kTile;
                uint4 v[kRowChunks];
#pragma unroll
                for (int t = 0; t < kRowChunks; ++t) {
                    const int64_t o = __shfl_sync(0xffffffffu, off, t * kRowsAtOnce + sub_row);
                    v[t] = o >= 0 ? reinterpret_cast<const uint4 *>(a.q + o)[sub_chunk]
                                  : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int t = 0; t < kRowChunks; ++t) {
                    if (kEight) {  // scaled by a power of two into half precision
                        const typename E::T *e = reinterpret_cast<const typename E::T *>(&v[t]);
                        float q[8], top = 0.0f, down, up;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            q[i] = E::load(e[i]);
                            top = fmaxf(top, fabsf(q[i]));
                        }
#pragma unroll
                        for (int d = 1; d < kRowChunks; d <<= 1)
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        unit_scale(top, &down, &up);
                        v[t] = make_uint4(P::pack(q[0] * down, q[1] * down),
                                          P::pack(q[2] * down, q[3] * down),
                                          P::pack(q[4] * down, q[5] * down),
                                          P::pack(q[6] * down, q[7] * down));
                        up = __shfl_sync(0xffffffffu, up, lane % kRowsAtOnce * kRowChunks);
                        if (lane / kRowsAtOnce == t)
                            row_factor = up;
                    }
                    *reinterpret_cast<uint4 *>(
                        dst + tile_at(warp_row + t * kRowsAtOnce + sub_row, sub_chunk)) = v[t];
                }
                fence_async_shared();
                mbar_arrive(bar(kBarQ + x));
            }
            float m = -INFINITY, l = 0.0f;
            if (mine) {
                // Scores stay products of q and k, with one factor to units of log 2, where
                // that factor is all there is to them.  The same for a whole warp: the loads
                // and stores of tensor memory below must not diverge.
                const float factor = score.factor * row_factor;
                // Under a cap, the terms of cap tanh(inner x) / x in x^2.
                const float inner = score.inner * row_factor;
                const float series_reach = tanh_reach(inner);
                uint64_t series[kTanhTerms];
                {
                    // Without a cap the first term alone is used, and is the factor itself.
                    float t = a.softcap > 0.0f ? score.cap * inner : factor * (1.0f / kTanh[0]);
#pragma unroll
                    for (int n = 0; n < kTanhTerms; ++n) {
                        series[n] = pair_of(t * kTanh[n], t * kTanh[n]);
                        t *= inner * inner;
                    }
                }
                const bool plain = !(a.softcap > 0.0f) && !a.slopes && a.scale > 1e-10f;
                for (int i = 0; i < u.todo; ++i) {
                    const int j0 = u.key_of(i);
                    ok = wait(kBarS + x, s_phase);
                    if (!ok)
                        break;
                    s_phase ^= 1;
                    tc_fence_after();
                    const bool all_seen = j0 + kTileKeys <= u.keys.prefix ||
                                          (j0 + kTileKeys - 1 <= u.keys.pmin &&
                                           (!a.window || j0 > u.keys.pmax - a.window));
                    // First pass: the largest score.  Scores that need more than one factor,
                    // or have hidden ones among them, are written back as they are to be used.
                    // Reading S twice costs less than the 128 registers of holding it.
                    const float unit = plain ? factor : 1.0f;
                    float top = -INFINITY;
                    if (plain && all_seen) {
                        float s[2][32], t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        tc_ld32(s[0], ts);
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            float(&z)[32] = s[b & 1];
                            tc_wait_ld(z);
                            if (b < 3)
                                tc_ld32(s[(b + 1) & 1], ts + 32 * (b + 1));
#pragma unroll
                            for (int k = 0; k < 32; k += 2)
                                t4[k >> 1 & 3] = max3(t4[k >> 1 & 3], z[k], z[k + 1]);
                        }
                        top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                    } else {
                        const int hi = pos - j0, pre = u.keys.prefix - j0;
                        const int lo = a.window ? hi - a.window + 1 : -j0;
                        // Where rows see no key after their own, -|i - j| is j - i.
                        const bool behind = a.slopes && u.keys.prefix <= u.keys.pmin + 1;
                        // Scores from products, two at a time: a factor or the cap's series, and a
                        // bias that grows by `step` from pair to pair (its rounding grows with the
                        // bias, that is, with how little such keys weigh).  Each combination is
                        // code of its own: as one with conditions, all of it is executed.
                        auto shape = [&](float(&z)[32], float away, auto capped, auto biased) {
                            const float z0 = slope * away, two = 2.0f * slope;
                            uint64_t bias = pair_of(z0, z0 + slope);
                            const uint64_t step = pair_of(two, two);
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const uint64_t x = pair_of(z[2 * k], z[2 * k + 1]);
                                uint64_t t = series[0];
                                if constexpr (decltype(capped)::value) {
                                    const uint64_t u = mul_pair(x, x);
                                    t = series[kTanhTerms - 1];
#pragma unroll
                                    for (int n = kTanhTerms - 2; n >= 0; --n)
                                        t = fma_pair(t, u, series[n]);
                                }
                                float2 y;
                                if constexpr (decltype(biased)::value) {
                                    y = halves_of(fma_pair(x, t, bias));
                                    bias = add_pair(bias, step);
                                } else {
                                    y = halves_of(mul_pair(x, t));
                                }
                                z[2 * k] = y.x;
                                z[2 * k + 1] = y.y;
                            }
                        };
                        auto adjust = [&](float(&z)[32], int b) {
                            const float away = float(32 * b - hi);  // j - i of z[0]
                            if (a.softcap > 0.0f) {
                                float most = 0.0f, more = 0.0f;
#pragma unroll
                                for (int k = 0; k < 32; k += 4) {
                                    most = max3_abs(most, z[k], z[k + 1]);
                                    more = max3_abs(more, z[k + 2], z[k + 3]);
                                }
                                most = fmaxf(most, more);
                                // Past the series' reach tanh is good to 2^-22 of 1, which
                                // the cap multiplies: less than what 32 bits make of products
                                // that large.
                                if (!__all_sync(0xffffffffu, most <= series_reach)) {
#pragma unroll
                                    for (int k = 0; k < 32; ++k)
                                        z[k] = score.cap * tanh_of_1(z[k] * inner);
                                    if (behind) {
#pragma unroll
                                        for (int k = 0; k < 32; ++k)
                                            z[k] += slope * (away + float(k));
                                    }
                                } else if (behind) {
                                    shape(z, away, Yes(), Yes());
                                } else {
                                    shape(z, away, Yes(), No());
                                }
                            } else if (behind) {
                                shape(z, away, No(), Yes());
                            } else if (!plain) {
                                shape(z, away, No(), No());
                            }
                            if (a.slopes && !behind) {
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    z[k] -= slope * fabsf(away + float(k));
                            }
                            if (!all_seen) {
                                const unsigned seen = (bits_below(hi + 1 - 32 * b) &
                                                       ~bits_below(lo - 32 * b)) |
                                                      bits_below(pre - 32 * b);
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    z[k] = seen >> k & 1 ? z[k] : -INFINITY;
                            }
                            float t4[2] = {top, -INFINITY};
#pragma unroll
                            for (int k = 0; k < 32; k += 2)
                                t4[k >> 1 & 1] = max3(t4[k >> 1 & 1], z[k], z[k + 1]);
                            top = fmaxf(t4[0], t4[1]);
                            tc_st32(ts + 32 * b, z);
                        };
                        float s0[32];
#pragma unroll 1
                        for (int b = 0; b < 4; ++b) {
                            tc_ld32(s0, ts + 32 * b);
                            tc_wait_ld(s0);
                            adjust(s0, b);
                        }
                        tc_wait_st();
                    }
                    top *= unit;
                    // The subtracted number may lag by up to 2^8 more than its room; O is
                    // rescaled only past that.  S of this step is complete, so P V of the last
                    // one is too.
                    const bool lift = top > m + (P::kRoom + 8.0f);
                    if (__any_sync(0xffffffffu, lift)) {
                        const float next = lift ? top - P::kRoom : m;
                        const float keep = lift ? exp2_(m - next) : 1.0f;
                        m = next;
                        l *= keep;
                        if (i > 0) {
#pragma unroll 1
                            for (int b = 0; b < D / 32; ++b) {
                                float o[32];
                                tc_ld32(o, to + 32 * b);
                                tc_wait_ld(o);
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    o[k] *= keep;
                                tc_st32(to + 32 * b, o);
                            }
                        }
                    }
                    // Second pass: weights.  P of columns 32 b .. + 31 takes columns 16 b .. + 15,
                    // which held scores that have been read.
                    const float base = m == -INFINITY ? 0.0f : m;
                    const uint64_t unit2 = pair_of(unit, unit), base2 = pair_of(-base, -base);
                    uint64_t sum[2] = {0, 0};
                    {
                        float s[2][32];
                        tc_ld32(s[0], ts);
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            float(&z)[32] = s[b & 1];
                            tc_wait_ld(z);
                            if (b < 3)
                                tc_ld32(s[(b + 1) & 1], ts + 32 * (b + 1));
                            unsigned p[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                float2 e = halves_of(
                                    fma_pair(pair_of(z[2 * k], z[2 * k + 1]), unit2, base2));
                                e.x = exp2_(e.x);
                                e.y = exp2_(e.y);
                                sum[k & 1] = add_pair(sum[k & 1], pair_of(e.x, e.y));
                                p[k] = P::pack(e.x, e.y);
                            }
                            tc_st16(ts + 16 * b, p);
                            if (b & 1) {
                                tc_wait_st();
                                tc_fence_before();
                                mbar_arrive(bar((b == 1 ? kBarP : kBarP2) + x));
                            }
                        }
                    }
                    const float2 sums = halves_of(add_pair(sum[0], sum[1]));
                    l += sums.x + sums.y;
                }
                if (!ok)
                    break;
                ok = wait(kBarO + x, o_phase);
                if (!ok)
                    break;
                o_phase ^= 1;
                tc_fence_after();
            }

            // The result, or this CTA's part of it.
            const int c0 = u.begun_by(), c1 = u.ended_by();
            // Rows go out by way of q's place in shared memory, which is free by now; each warp
            // uses its own rows of it.
            auto put = [&](int b, const float(&o)[32], float ll) {
                const float f = a.v_scale / ll;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<uint4 *>(smem + x * T::kTile + tile_at(row, 4 * b + k)) =
                        make_uint4(E::pack(o[8 * k] * f, o[8 * k + 1] * f),
                                   E::pack(o[8 * k + 2] * f, o[8 * k + 3] * f),
                                   E::pack(o[8 * k + 4] * f, o[8 * k + 5] * f),
                                   E::pack(o[8 * k + 6] * f, o[8 * k + 7] * f));
            };
            auto flush = [&](float mm, float ll) {
                const int64_t off = have ? orow * a.out_stride + head * (D * 2) : -1;
                __syncwarp();
#pragma unroll
                for (int t = 0; t < kRowChunks; ++t) {
                    const int r = t * kRowsAtOnce + sub_row;
                    const int64_t o = __shfl_sync(0xffffffffu, off, r);
                    if (o >= 0)
                        reinterpret_cast<uint4 *>(a.out + o)[sub_chunk] =
                            *reinterpret_cast<const uint4 *>(
                                smem + x * T::kTile + tile_at(warp_row + r, sub_chunk));
                }
                __syncwarp();
                if (have && a.lse)
                    a.lse[orow * a.q_heads + head] = mm * kLn2 + logf(ll);
            };
            // A part: [D / 4][256 rows][4] of O, then [256][m, l].
            const int prow = x * kTileRows + row;
            if (mine) {
                float *slot = w.partial +
                              (2 * int64_t(blockIdx.x) + (int(blockIdx.x) == c0)) * T::kSlotFloats;
#pragma unroll 1
                for (int b = 0; b < D / 32; ++b) {
                    float o[32];
                    tc_ld32(o, to + 32 * b);
                    tc_wait_ld(o);
                    if (c0 == c1) {
                        put(b, o, l);
                    } else if (have) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<float4 *>(slot + ((8 * b + k) * kBlockRows + prow) * 4) =
                                make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    }
                }
                if (c0 == c1)
                    flush(m, l);
                else if (have)
                    *reinterpret_cast<float2 *>(slot + kBlockRows * D + 2 * prow) = make_float2(m, l);
            }
        }
    }
    __syncthreads();
    if (warp == 8)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// The results of units that were cut: block (c, slice) joins, in order, the parts of the unit
// that CTA c began and did not end, for 32 of its rows.  A launch of its own puts every SM to
// this, where the last CTA of a unit would have read up to 150 parts of 128 KB alone (65 us
// against 37 for 64 new tokens behind 32k), and spares all of them a fence and a counter.
const int kJoinThreads = 256;
const int kJoinRows = 32;

template <int TYPE, int D>
__global__ void __launch_bounds__(kJoinThreads)
kvx_attend_join_kernel(const Attend a, const Work w)
{
    typedef Elem<TYPE> E;
    constexpr int kSlotFloats = kBlockRows * (D + 2);
    __shared__ uint2 out[kJoinRows][D / 4 + 1];
    const int c0 = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const AttnStart next = w.starts[c0 + 1];
    const int c1 = w.starts[c0].last;
    wait_for_earlier_work();
    if (next.tile == 0 || next.first != c0)
        return;
    const AttnReq &r = next.req;
    const int row0 = next.block * kBlockRows, rows = min(kBlockRows, r.n_new * a.group - row0);
    const int row = blockIdx.y * kJoinRows + lane;
    if (int(blockIdx.y) * kJoinRows >= rows)
        return;
    auto part = [&](int c) { return w.partial + (2 * int64_t(c) + (c == c0)) * kSlotFloats; };
    auto ml = [&](int c) {
        return __ldcg(reinterpret_cast<const float2 *>(part(c) + kBlockRows * D) + row);
    };
    float mm = -INFINITY, ll = 0.0f;
    float4 o[D / 32];
#pragma unroll
    for (int k = 0; k < D / 32; ++k)
        o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (row < rows) {
#pragma unroll 8
        for (int c = c0; c <= c1; ++c)
            mm = fmaxf(mm, ml(c).x);
#pragma unroll 4
        for (int c = c0; c <= c1; ++c) {
            float4 v[D / 32];
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
                v[k] = __ldcg(reinterpret_cast<const float4 *>(part(c)) +
                              (8 * k + warp) * kBlockRows + row);
            const float2 p = ml(c);
            const float f = p.x == -INFINITY ? 0.0f : exp2_(p.x - mm);
            ll += f * p.y;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                o[k].x += f * v[k].x;
                o[k].y += f * v[k].y;
                o[k].z += f * v[k].z;
                o[k].w += f * v[k].w;
            }
        }
        const float f = a.v_scale / ll;
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
            out[lane][8 * k + warp] =
                make_uint2(E::pack(o[k].x * f, o[k].y * f), E::pack(o[k].z * f, o[k].w * f));
    }
    __syncthreads();
    // Whole rows, 8 bytes to a lane.
    for (int i = threadIdx.x; i < kJoinRows * (D / 4); i += kJoinThreads) {
        const int sub = i / (D / 4), d = i % (D / 4), packed = row0 + blockIdx.y * kJoinRows + sub;
        if (blockIdx.y * kJoinRows + sub < rows) {
            const int tok = packed / a.group, head = next.head * a.group + packed - tok * a.group;
            reinterpret_cast<uint2 *>(a.out + (r.row_begin + tok) * a.out_stride +
                                      head * (D * 2))[d] = out[sub][d];
        }
    }
    if (a.lse && warp == 0 && row < rows) {
        const int packed = row0 + row, tok = packed / a.group;
        a.lse[int64_t(r.row_begin + tok) * a.q_heads + next.head * a.group + packed -
              tok * a.group] = mm * kLn2 + logf(ll);
    }
}

}  // namespace
