// kvx_attend_four.cuh -- attention of at most 16 rows per KV head (single new tokens, a few
// drafted ones) over a cache held in 4 bits.  Included by kvx_attend_four.cu only.
#pragma once

#include "kvx_attend.cuh"
#include "kvx_attend_rows.cuh"
#include "kvx_attend_tiles.cuh"

namespace {

// A head's key is 72 bytes at 128 elements, in two places of its token: too short a run for
// memory to serve well, one head at a time.  So a CTA takes a unit (request, group of up to
// eight KV heads) and streams whole tokens: one warp has runs of tokens brought into a ring of
// shared-memory stages, a bulk copy for each run inside a page and side; eight warps multiply,
// each a KV head of its own, or, where the group has fewer than eight heads, sharing a head's
// keys out among `split` warps.  Each keeps its running maximum, sum and output in registers;
// warps of one head join theirs in shared memory when the unit ends.
//
// Products are those of the other caches' kernel (S' = K Q', O' = V' P' on m16n8k16), in half
// precision, which holds code x scale exactly (6 bits, 2^-10 .. 2688); q is scaled by a power of
// two per row to at most 1, as there.  A thread's operands of K are 16 consecutive bytes of a
// key (32 elements, two scales), of V 8 bytes of four keys (one block, one scale each); pairs
// of codes become pairs of halves in one conversion, V's are then paired across keys by byte
// permutation.  Conversion, scaling and pairing are some 200 of the 337 instructions that a warp
// spends on 16 keys of a head; 32 keys go through each step so that what is not proportional to
// them (barriers, votes, addresses) is met half as often.
//
// Measured: 64 requests of 1k to 32k tokens, 4 KV heads of 7 rows, 69 us (298 MB, 4.3 TB/s; the
// same copies with nothing multiplied take 54, the device copy's rate would be 44); one request
// of 256k tokens, 8 heads, 62 us with the join (302 MB, 4.9 TB/s; 56 with nothing multiplied); 24
// requests of up to 64k, 16 rows a head, 149 us (535 MB, 3.6 TB/s; 95): there one CTA's eight
// warps hold 168 registers each and wait for their own latencies, issuing in 43 % of the cycles.
const int kFourWarps = 8;
const int kFourThreads = 32 * (kFourWarps + 1);
const int kFourStages = 8;    // at most
const int kFourKeys = 32;     // of a warp and step, two products' worth
const int kFourAhead = 3;     // stages that page ids are looked up before they are used

template <int N>
struct Looks {
    static constexpr int value = N;
};

struct FourShape {
    int heads, groups;  // KV heads of a group, groups
    int split;          // warps per head
    int keys;           // tokens of a stage
    int code_row, scale_at, scale_row;  // of a stage's side, in bytes
    int side;

    __host__ __device__ static FourShape of(int kv_heads, int D, int token_bytes)
    {
        FourShape f;
        f.groups = (kv_heads + kFourWarps - 1) / kFourWarps;
        f.heads = (kv_heads + f.groups - 1) / f.groups;
        f.split = f.heads > 4 ? 1 : f.heads > 2 ? 2 : f.heads > 1 ? 4 : 8;
        f.keys = kFourKeys * f.split;
        if (f.groups == 1) {
            f.code_row = f.scale_row = token_bytes;
            f.scale_at = kv_heads * (D / 2);
            f.side = f.keys * token_bytes;
        } else {
            // A group's codes, and the 16-byte units that its scales lie in.
            f.code_row = f.heads * (D / 2);
            f.scale_at = f.keys * f.code_row;
            f.scale_row = (f.heads * (D / 16) + 30) / 16 * 16;
            f.side = f.keys * (f.code_row + f.scale_row);
        }
        return f;
    }
};

template <int D, int NT>
__host__ __device__ constexpr int four_join_floats()  // a warp's result: O, m, l
{
    return 8 * NT * (D + 4 + 2);
}

template <int D, int NT>
__host__ __device__ constexpr int four_slot_floats()  // a partial result: [head][row] O, then m, l
{
    return kFourWarps * 8 * NT * (D + 2);
}

__host__ __device__ constexpr int four_ctas_per_sm(int NT) { return NT == 1 ? 2 : 1; }

// Dynamic shared memory of a CTA, at most: beside 1 KB of its own and 1 KB of the system's.
__host__ __device__ constexpr int four_room(int NT)
{
    return 226 * 1024 / four_ctas_per_sm(NT) - 2 * 1024;
}

// Shared memory in which warps of a head hand over their results.
template <int D, int NT>
__host__ __device__ inline int four_join_bytes(const FourShape &f)
{
    return f.heads * (f.split / 2) * four_join_floats<D, NT>() * 4;
}

template <int D, int NT>
__host__ __device__ inline int four_stages(const FourShape &f)
{
    const int n = (four_room(NT) - four_join_bytes<D, NT>(f)) / (2 * f.side);
    return n < kFourStages ? n : kFourStages;
}

template <int D, int NT>
inline size_t four_smem(const FourShape &f)
{
    return size_t(four_stages<D, NT>(f)) * 2 * f.side + four_join_bytes<D, NT>(f);
}

// As mma16816 in half precision; not volatile, so that products of K move among the conversions
// of V.
__device__ __forceinline__ void mma_half(float (&d)[4], const unsigned (&a)[4], unsigned b0,
                                         unsigned b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// `bytes` (a multiple of 16, addresses too) of global memory into shared memory; completes on a
// barrier.
__device__ __forceinline__ void bulk_copy(unsigned dst, const void *src, unsigned bytes,
                                          unsigned bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], "
                 "%2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// PLAIN: neither a cap nor a bias, whose code keeps the rest from staying in the instruction
// caches.
template <int TYPE, int D, int NT, bool PLAIN>
__global__ void __launch_bounds__(kFourThreads, four_ctas_per_sm(NT))
kvx_attend_four_kernel(const Attend a, const Work w)
{
    typedef Elem<TYPE> E;
    typedef Elem<KVX_TYPE_HALF> P;
    constexpr float kRoom = P::kRoom;
    constexpr int kSteps = D / 16, kRowsMax = 8 * NT, kMine = D / 8;  // elements of V per thread
    constexpr int kHalves = kFourKeys / 16;
    constexpr int kJoin = four_join_floats<D, NT>(), kSlot = four_slot_floats<D, NT>();
    __shared__ __align__(8) uint64_t bars[2 * kFourStages];
    __shared__ int gave_up;
    const FourShape f = FourShape::of(a.kv_heads, D, int(a.token_bytes));
    const int stages = four_stages<D, NT>(f);
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const unsigned ring = smem_u32(attend_smem), bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8 * s; };
    auto empty = [&](int s) { return bar0 + 8 * (kFourStages + s); };
    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kFourWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    AttnStart at = w.starts[blockIdx.x];
    Keys keys;
    int todo = 0;
    auto enter = [&]() {
        keys.set(at.req, a.window, 0, at.req.n_new - 1, f.keys);
        todo = int(min(int64_t(keys.tiles - at.tile), at.tiles));
    };
    // Last keys first, as in the other kernels.
    auto key_of = [&](int i) {
        const int t = keys.tiles - 1 - at.tile - i;
        return (t < keys.first ? t : t + keys.skip) * f.keys;
    };
    auto next_unit = [&]() {
        at.tiles -= todo;
        at.tile = 0;
        if (++at.head == f.groups) {
            at.head = 0;
            ++at.request;
            if (at.tiles > 0)
                at.req = w.reqs[at.request];
        }
    };
    int stage = 0;
    unsigned phase = 0;
    auto advance = [&]() {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    };
    bool ok = true;

    if (warp == kFourWarps) {
        // ------------------------------------------------------------- K and V
        wait_for_earlier_work();
        unsigned filled = 0;
        while (at.tiles > 0) {
            enter();
            const int head0 = at.head * f.heads, heads = min(f.heads, a.kv_heads - head0);
            const int scale_lo = head0 * (D / 16) / 16 * 16;
            const int scale_hi = ((head0 + heads) * (D / 16) + 15) / 16 * 16;
            const unsigned per_token = f.groups == 1
                                           ? unsigned(a.token_bytes)
                                           : unsigned(heads * (D / 2) + scale_hi - scale_lo);
            // A run of tokens inside a page and a stretch of used keys, from token t of a stage
            // of keys from j0: its length, 0 if none begins there, its page of the table and its
            // place in it.
            auto run_at = [&](int j0, int t, bool whole, int &nth, int &in) {
                const int j = j0 + t;
                nth = a.page.div(j);
                in = j - nth * a.page_size;
                int n = t < f.keys && (t == 0 || in == 0) ? min(f.keys - t, a.page_size - in) : 0;
                if (!whole) {
                    const int seen = j < keys.prefix && keys.prefix < keys.low
                                         ? keys.prefix : max(keys.prefix, keys.end);
                    n = t < f.keys && keys.used(j) && (t == 0 || in == 0 || !keys.used(j - 1))
                            ? min(min(f.keys - t, a.page_size - in), seen - j) : 0;
                }
                return n;
            };
            auto whole_at = [&](int j0) {
                return j0 + f.keys <= keys.prefix || (j0 >= keys.low && j0 + f.keys <= keys.end);
            };
            // Pages outside the pool: zeros, which nothing may be in flight beside.
            auto clear = [&](int t0, int n) {
                for (int x = 0; x < 2 * n; ++x) {
                    char *s = attend_smem + (stage * 2 + (x & 1)) * f.side;
                    const int t = t0 + x / 2;
                    for (int c = 0; c < f.code_row; c += 16)
                        *reinterpret_cast<uint4 *>(s + t * f.code_row + c) = make_uint4(0, 0, 0, 0);
                    for (int c = 0; f.groups > 1 && c < f.scale_row; c += 16)
                        *reinterpret_cast<uint4 *>(s + f.scale_at + t * f.scale_row + c) =
                            make_uint4(0, 0, 0, 0);
                }
            };
            // A group's part of n tokens from `src`, token by token.
            auto copy_group = [&](unsigned dst, int t, int n, int64_t src) {
                for (int r = 0; r < 2 * n; ++r) {
                    const char *s = (r & 1 ? a.v : a.k) + src + r / 2 * a.token_bytes;
                    const unsigned d = dst + (r & 1) * f.side;
                    bulk_copy(d + (t + r / 2) * f.code_row, s + head0 * (D / 2), heads * (D / 2),
                              full(stage));
                    bulk_copy(d + f.scale_at + (t + r / 2) * f.scale_row,
                              s + a.kv_heads * (D / 2) + scale_lo, scale_hi - scale_lo,
                              full(stage));
                }
            };
            // One warp does this for eight that multiply, so instructions count: at 300 a stage
            // it was what the kernel waited for.  A lane looks after tokens lane, lane + 32, ...
            // of a stage, LOOK of them, and has their page ids kFourAhead stages early.
            auto produce = [&](auto look) {
                constexpr int LOOK = decltype(look)::value;
                int ids[kFourAhead][LOOK];
                auto look_up = [&](int i, int (&id)[LOOK]) {
                    if (i >= todo)
                        return;
                    const int j0 = key_of(i);
                    const bool whole = whole_at(j0);
#pragma unroll
                    for (int b = 0; b < LOOK; ++b) {
                        int nth, in;
                        if (run_at(j0, lane + 32 * b, whole, nth, in))
                            id[b] = at.req.table[nth];
                    }
                };
#pragma unroll
                for (int q = 0; q < kFourAhead; ++q)
                    look_up(q, ids[q]);
#pragma unroll 1
                for (int i = 0; i < todo; ++i) {
                    const int j0 = key_of(i);
                    const bool whole = whole_at(j0);
                    int n[LOOK], in[LOOK], page[LOOK];
                    bool bad = false;
#pragma unroll
                    for (int b = 0; b < LOOK; ++b) {
                        int nth;
                        n[b] = run_at(j0, lane + 32 * b, whole, nth, in[b]);
                        page[b] = ids[0][b];
                        bad |= n[b] && unsigned(page[b]) >= unsigned(a.num_pages);
                    }
#pragma unroll
                    for (int q = 0; q + 1 < kFourAhead; ++q)
#pragma unroll
                        for (int b = 0; b < LOOK; ++b)
                            ids[q][b] = ids[q + 1][b];
                    look_up(i + kFourAhead, ids[kFourAhead - 1]);
                    if (ok)
                        ok = mbar_wait(empty(stage), phase ^ 1, &gave_up, a.status);
                    unsigned bytes = 2 * unsigned(f.keys) * per_token;
                    bad = __any_sync(0xffffffffu, bad);
                    if (bad || !whole) {
                        bytes = 0;
#pragma unroll
                        for (int b = 0; b < LOOK; ++b) {
                            if (n[b] && unsigned(page[b]) >= unsigned(a.num_pages)) {
                                atomicOr(a.status, KVX_DEV_PAGE_OUT_OF_RANGE);
                                clear(lane + 32 * b, n[b]);
                                n[b] = 0;
                            }
                            bytes += 2 * n[b] * per_token;
                        }
                        bytes = __reduce_add_sync(0xffffffffu, bytes);
                        fence_async_shared();
                        __syncwarp();
                    }
                    if (!ok)
                        continue;
                    if (lane == 0) {
                        if (bytes)
                            mbar_expect(full(stage), bytes);
                        else
                            mbar_arrive(full(stage));
                    }
                    __syncwarp();
                    const unsigned dst = ring + stage * 2 * f.side;
#pragma unroll
                    for (int b = 0; b < LOOK; ++b) {
                        if (n[b] == 0)
                            continue;
                        const int t = lane + 32 * b;
                        const int64_t src =
                            (int64_t(page[b]) * a.page_size + in[b]) * a.token_bytes;
                        if (f.groups == 1) {
                            const unsigned size = unsigned(n[b]) * per_token;
                            bulk_copy(dst + t * f.code_row, a.k + src, size, full(stage));
                            bulk_copy(dst + f.side + t * f.code_row, a.v + src, size, full(stage));
                        } else {
                            copy_group(dst, t, n[b], src);
                        }
                    }
                    ++filled;
                    advance();
                }
            };
            if (f.keys <= 32)
                produce(Looks<1>());
            else if (f.keys <= 64)
                produce(Looks<2>());
            else if (f.keys <= 128)
                produce(Looks<4>());
            else
                produce(Looks<8>());
            next_unit();
        }
        if (!ok) {
            // Copies may still be under way: see the stages filled last complete.
            const uint64_t t0 = now_ns();
            for (unsigned n = filled > unsigned(stages) ? filled - stages : 0; n < filled; ++n)
                while (!__all_sync(0xffffffffu, mbar_try(full(n % stages), n / stages & 1)) &&
                       !__any_sync(0xffffffffu, now_ns() - t0 > 1000000000ull)) {
                }
        }
        return;
    }

    // ----------------------------------------------------------------- products
    const int quad = lane >> 2, c = lane & 3;
    const int hh = warp / f.split, sub = warp - hh * f.split;  // head of the group, share of keys
    const Score score(a);
    float *join = reinterpret_cast<float *>(attend_smem + stages * 2 * f.side);
    wait_for_earlier_work();
    while (at.tiles > 0) {
        enter();
        const AttnReq r = at.req;
        const int rows = r.n_new * a.group, kv_head = at.head * f.heads + hh;
        const bool active = hh < f.heads && kv_head < a.kv_heads;
        // Byte of the group's first scale within a stage's 16-byte units of them.
        const int scale0 = f.groups == 1 ? 0 : at.head * f.heads * (D / 16) % 16;

        // From a stage's start: codes and scales of K of key quad, of V of key 2 c.
        const int t0 = sub * kFourKeys, in = hh * (D / 2), in_unit = scale0 + hh * (D / 16);
        const int k_code = (t0 + quad) * f.code_row + in + c * (D / 8);
        const int k_unit = f.scale_at + (t0 + quad) * f.scale_row + in_unit + c * (D / 64);
        const int v_code = f.side + (t0 + 2 * c) * f.code_row + in + quad * (D / 16);
        const int v_unit = f.side + f.scale_at + (t0 + 2 * c) * f.scale_row + in_unit +
                           quad * (D / 16) / 8;

        // q as the second operand, in the order in which a thread reads K: step s of quad thread
        // c takes elements (D / 4) c + 4 s .. + 3.
        unsigned qb[NT][kSteps][2];
        float factor[NT][2], slope[NT][2];
        int pos[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool have = active && quad + 8 * n < rows;
            const int row = have ? quad + 8 * n : 0, tok = row / a.group;
            const char *qp = a.q + int64_t(r.row_begin + tok) * a.q_stride +
                             ((active ? kv_head : 0) * a.group + row - tok * a.group) * (D * 2) +
                             c * (D / 2);
            uint4 u[kSteps / 2];
            float top = 0.0f, down, up;
#pragma unroll
            for (int s = 0; s < kSteps / 2; ++s) {
                u[s] = have ? reinterpret_cast<const uint4 *>(qp)[s] : make_uint4(0, 0, 0, 0);
                const typename E::T *e = reinterpret_cast<const typename E::T *>(&u[s]);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    top = fmaxf(top, fabsf(E::load(e[i])));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            unit_scale(top, &down, &up);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const typename E::T *e =
                    reinterpret_cast<const typename E::T *>(&u[s / 2]) + 4 * (s & 1);
                qb[n][s][0] = P::pack(E::load(e[0]) * down, E::load(e[1]) * down);
                qb[n][s][1] = P::pack(E::load(e[2]) * down, E::load(e[3]) * down);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int mine = 2 * c + e + 8 * n, t = mine < rows ? mine / a.group : 0;
                pos[n][e] = keys.pmin + t;
                factor[n][e] = __shfl_sync(0xffffffffu, up, 8 * c + 4 * e) *
                               (a.softcap > 0.0f ? score.inner : score.factor);
                slope[n][e] = a.slopes && active && mine < rows
                                  ? a.slopes[kv_head * a.group + mine - t * a.group] * kLog2e
                                  : 0.0f;
            }
        }

        // O': row quad + 8 half of block mt is element quad D / 8 + 2 mt + half.
        float o[NT][kSteps][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int t = 0; t < kSteps; ++t)
                o[n][t][0] = o[n][t][1] = o[n][t][2] = o[n][t][3] = 0.0f;
            m[n][0] = m[n][1] = 0.0f;
            l[n][0] = l[n][1] = 0.0f;
        }
        // Rows (the same for the lanes that share them) of which no key has been seen; and the
        // first keys of 32 that all rows see: from seen_lo to seen_hi, or up to seen_pre.
        unsigned fresh = (1u << 2 * NT) - 1;
        const int seen_hi = keys.pmin - kFourKeys + 1, seen_pre = keys.prefix - kFourKeys;
        const int seen_lo = a.window ? keys.pmax - a.window + 1 : 0;

#pragma unroll 1
        for (int i = 0; i < todo; ++i) {
            if (ok)
                ok = mbar_wait(full(stage), phase, &gave_up, a.status);
            const int j0 = key_of(i) + sub * kFourKeys;
            if (ok && active) {
                // This stage's K and V, at the thread's own codes and scales of its first key.
                const char *base = attend_smem + stage * 2 * f.side;
                // Scores of both halves: s[u][n][2 x + e] is key j0 + 16 u + quad + 8 x, row 8 n +
                // 2 c + e.
                float s[kHalves][NT][4];
#pragma unroll
                for (int u = 0; u < kHalves; ++u) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.0f;
                    unsigned code[2][D / 32], unit[2][2];  // unit: of the first and second block
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const char *ka = base + k_code + (16 * u + 8 * x) * f.code_row;
                        const char *sa = base + k_unit + (16 * u + 8 * x) * f.scale_row;
                        if (D == 128) {
                            const uint4 w4 = *reinterpret_cast<const uint4 *>(ka);
                            code[x][0] = w4.x, code[x][1] = w4.y;
                            code[x][D / 32 - 2] = w4.z, code[x][D / 32 - 1] = w4.w;
                            const unsigned two =
                                half2_of_e4m3(*reinterpret_cast<const uint16_t *>(sa));
                            unit[x][0] = __byte_perm(two, 0, 0x1010);
                            unit[x][1] = __byte_perm(two, 0, 0x3232);
                        } else {
                            const uint2 w2 = *reinterpret_cast<const uint2 *>(ka);
                            code[x][0] = w2.x, code[x][1] = w2.y;
                            unit[x][0] =
                                half2_of_e4m3(*reinterpret_cast<const uint8_t *>(sa) * 0x101u);
                            unit[x][1] = unit[x][0];
                        }
                    }
#pragma unroll
                    for (int g = 0; g < D / 32; ++g) {
                        unsigned h0[4], h1[4];
                        half8_of_e2m1(code[0][g], h0);
                        half8_of_e2m1(code[1][g], h1);
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            h0[y] = mul_half2(h0[y], unit[0][g / 2]);
                            h1[y] = mul_half2(h1[y], unit[1][g / 2]);
                        }
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const unsigned k[4] = {h0[2 * y], h1[2 * y], h0[2 * y + 1],
                                                   h1[2 * y + 1]};
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_half(s[u][n], k, qb[n][2 * g + y][0], qb[n][2 * g + y][1]);
                        }
                    }
                }

                // Scores less what is subtracted, m, which may lag behind the maximum, as in the
                // other kernel.
                const bool all_seen = (j0 <= seen_hi && j0 >= seen_lo) || j0 <= seen_pre;
                float top = -INFINITY;
                if (PLAIN && all_seen) {
#pragma unroll
                    for (int u = 0; u < kHalves; ++u)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                s[u][n][x] = fmaf(s[u][n][x], factor[n][x & 1], -m[n][x & 1]);
                            top = max3(top, s[u][n][0], s[u][n][1]);
                            top = max3(top, s[u][n][2], s[u][n][3]);
                        }
                } else {
#pragma unroll
                    for (int u = 0; u < kHalves; ++u)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const int e = x & 1, j = j0 + 16 * u + quad + 8 * (x >> 1);
                                float z = s[u][n][x] * factor[n][e];
                                if (!PLAIN) {
                                    if (a.softcap > 0.0f)
                                        z = score.cap * tanh_(z);
                                    z -= slope[n][e] * fabsf(float(pos[n][e] - j));
                                }
                                if (!(j < keys.prefix ||
                                      (j <= pos[n][e] &&
                                       (!a.window || pos[n][e] - j < a.window))))
                                    z = -INFINITY;
                                s[u][n][x] = z - m[n][e];
                                top = fmaxf(top, s[u][n][x]);
                            }
                }
                if (__any_sync(0xffffffffu, top > kRoom + 8.0f || fresh)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float most = -INFINITY;
#pragma unroll
                            for (int u = 0; u < kHalves; ++u)
                                most = max3(most, s[u][n][e], s[u][n][2 + e]);
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1)
                                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                            // A row's first keys set m, down as well as up.
                            const unsigned bit = 1u << (2 * n + e);
                            const bool first = fresh & bit && most > -INFINITY;
                            const float up = first         ? most - kRoom
                                             : fresh & bit ? 0.0f : fmaxf(most - kRoom, 0.0f);
                            const float keep = first ? 1.0f : exp2_(-up);
                            fresh &= ~(first ? bit : 0u);
                            m[n][e] += up;
#pragma unroll
                            for (int u = 0; u < kHalves; ++u) {
                                s[u][n][e] -= up;
                                s[u][n][2 + e] -= up;
                            }
                            l[n][e] *= keep;
#pragma unroll
                            for (int t = 0; t < kSteps; ++t) {
                                o[n][t][e] *= keep;
                                o[n][t][2 + e] *= keep;
                            }
                        }
                }
                // Weights as the second operand, for half-precision outputs in two numbers: rounded
                // once, weights of short contexts alone would be as far off as the output's type.
                constexpr int kParts = TYPE == KVX_TYPE_HALF ? 2 : 1;
                unsigned p[kParts][kHalves][NT][2];
#pragma unroll
                for (int u = 0; u < kHalves; ++u)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            s[u][n][x] = exp2_(s[u][n][x]);
                            l[n][x & 1] += s[u][n][x];
                        }
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const float lo = s[u][n][2 * b], hi = s[u][n][2 * b + 1];
                            const unsigned w = P::pack(lo, hi);
                            p[0][u][n][b] = transpose8x8(w);
                            if constexpr (kParts == 2) {
                                const __half *h = reinterpret_cast<const __half *>(&w);
                                p[1][u][n][b] = transpose8x8(
                                    P::pack(lo - P::load(h[0]), hi - P::load(h[1])));
                            }
                        }
                    }

                // V of keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9: elements quad D / 8 and on.  A key
                // that no row sees has no weight; its scale is 0 too, whatever memory holds.
#pragma unroll
                for (int u = 0; u < kHalves; ++u) {
                    unsigned v[4][D / 64], vu[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int t = 16 * u + (y & 1) + 8 * (y >> 1);
                        const char *va = base + v_code + t * f.code_row;
                        if (D == 128) {
                            const uint2 w2 = *reinterpret_cast<const uint2 *>(va);
                            v[y][0] = w2.x, v[y][D / 64 - 1] = w2.y;
                        } else {
                            v[y][0] = *reinterpret_cast<const unsigned *>(va);
                        }
                        vu[y] = *reinterpret_cast<const uint8_t *>(base + v_unit +
                                                                   t * f.scale_row);
                    }
                    if (!all_seen) {
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            if (!keys.used(j0 + 16 * u + 2 * c + (y & 1) + 8 * (y >> 1)))
                                vu[y] = 0;
                    }
                    const unsigned unit0 = half2_of_e4m3(vu[0] | vu[1] << 8);
                    const unsigned unit1 = half2_of_e4m3(vu[2] | vu[3] << 8);
#pragma unroll
                    for (int g = 0; g < D / 64; ++g) {
                        unsigned h[4][4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            half8_of_e2m1(v[y][g], h[y]);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const unsigned k[4] = {
                                mul_half2(__byte_perm(h[0][x], h[1][x], 0x5410), unit0),
                                mul_half2(__byte_perm(h[0][x], h[1][x], 0x7632), unit0),
                                mul_half2(__byte_perm(h[2][x], h[3][x], 0x5410), unit1),
                                mul_half2(__byte_perm(h[2][x], h[3][x], 0x7632), unit1)};
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int y = 0; y < kParts; ++y)
                                    mma_half(o[n][4 * g + x], k, p[y][u][n][0], p[y][u][n][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(empty(stage));
            advance();
        }

#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
        // A row without keys here has no weight in what follows.
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                m[n][e] = fresh >> (2 * n + e) & 1 ? -1e30f : m[n][e];
        // Join the warps of a head by halves: the upper half hands its results to the lower.
        // Warps past the group's heads have no part in it.
        for (int half = f.split / 2; half > 0 && hh < f.heads; half >>= 1) {
            float *area = join + (hh * (f.split / 2) + (sub & (half - 1))) * kJoin;
            if (sub >= half && sub < 2 * half) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 8 * n + 2 * c + e;
                        float *p = area + row * (D + 4) + quad * kMine;
#pragma unroll
                        for (int t = 0; t < kSteps; t += 2)
                            *reinterpret_cast<float4 *>(p + 2 * t) =
                                make_float4(o[n][t][e], o[n][t][2 + e], o[n][t + 1][e],
                                            o[n][t + 1][2 + e]);
                        if (quad == 0)
                            *reinterpret_cast<float2 *>(area + kRowsMax * (D + 4) + 2 * row) =
                                make_float2(m[n][e], l[n][e]);
                    }
            }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + hh), "r"(32 * f.split) : "memory");
            if (sub < half) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 8 * n + 2 * c + e;
                        const float *p = area + row * (D + 4) + quad * kMine;
                        const float2 other = *reinterpret_cast<const float2 *>(
                            area + kRowsMax * (D + 4) + 2 * row);
                        const float top = fmaxf(m[n][e], other.x);
                        const float x = exp2_(m[n][e] - top), y = exp2_(other.x - top);
                        m[n][e] = top;
                        l[n][e] = l[n][e] * x + other.y * y;
#pragma unroll
                        for (int t = 0; t < kSteps; t += 2) {
                            const float4 u = *reinterpret_cast<const float4 *>(p + 2 * t);
                            o[n][t][e] = o[n][t][e] * x + u.x * y;
                            o[n][t][2 + e] = o[n][t][2 + e] * x + u.y * y;
                            o[n][t + 1][e] = o[n][t + 1][e] * x + u.z * y;
                            o[n][t + 1][2 + e] = o[n][t + 1][2 + e] * x + u.w * y;
                        }
                    }
            }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + hh), "r"(32 * f.split) : "memory");
        }
        if (active && sub == 0) {
            const int c0 = at.tile > 0 ? at.first : int(blockIdx.x);
            const int c1 = at.tile + todo < keys.tiles ? at.last : int(blockIdx.x);
            float *slot = w.partial + (2 * int64_t(blockIdx.x) + (int(blockIdx.x) == c0)) * kSlot;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 8 * n + 2 * c + e;
                    if (row >= rows)
                        continue;
                    if (c0 != c1) {
                        float *p = slot + (hh * kRowsMax + row) * D + quad * kMine;
#pragma unroll
                        for (int t = 0; t < kSteps; t += 2)
                            *reinterpret_cast<float4 *>(p + 2 * t) =
                                make_float4(o[n][t][e], o[n][t][2 + e], o[n][t + 1][e],
                                            o[n][t + 1][2 + e]);
                        if (quad == 0)
                            *reinterpret_cast<float2 *>(slot + kFourWarps * kRowsMax * D +
                                                        2 * (hh * kRowsMax + row)) =
                                make_float2(m[n][e], l[n][e]);
                        continue;
                    }
                    const int tok = row / a.group, head = kv_head * a.group + row - tok * a.group;
                    const int64_t orow = r.row_begin + tok;
                    const float g = a.v_scale / l[n][e];
                    uint4 *out = reinterpret_cast<uint4 *>(a.out + orow * a.out_stride +
                                                           (head * D + quad * kMine) * 2);
#pragma unroll
                    for (int t = 0; t < kSteps; t += 4)
                        out[t / 4] = make_uint4(
                            E::pack(o[n][t][e] * g, o[n][t][2 + e] * g),
                            E::pack(o[n][t + 1][e] * g, o[n][t + 1][2 + e] * g),
                            E::pack(o[n][t + 2][e] * g, o[n][t + 2][2 + e] * g),
                            E::pack(o[n][t + 3][e] * g, o[n][t + 3][2 + e] * g));
                    if (a.lse && quad == 0)
                        a.lse[orow * a.q_heads + head] = m[n][e] * kLn2 + logf(l[n][e]);
                }
        }
        next_unit();
    }
}

// The results of units that were cut: block (i, head and row) joins the parts of one row of the
// i-th of them, its warps every so many parts each, four of them in flight.  One request of 256k
// tokens has a part in every CTA, 300 of 33 KB, which its last CTA would be reading alone for
// longer than the attention takes: 32 warps to a row then (one request of 8k tokens 12.1 us
// instead of 14.2 with eight), eight where there are few parts (64 requests 74 instead of 91).
const int kFourJoinWarps = 32;    // at most
const int kFourJoinFew = 8;       // where no unit has more than kFourManyParts
const int kFourManyParts = 24;

template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(32 * kFourJoinWarps)
kvx_attend_four_join_kernel(const Attend a, const Work w)
{
    typedef Elem<TYPE> E;
    constexpr int kSlot = four_slot_floats<D, NT>(), kRowsMax = 8 * NT, kEach = D / 32;
    constexpr int kBatch = 4;
    __shared__ float sum[kFourJoinWarps][D], ml[kFourJoinWarps][2];
    const int c0 = w.cuts[blockIdx.x], lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = blockDim.x >> 5;
    const AttnStart next = w.starts[c0 + 1];
    const int c1 = w.starts[c0].last;
    const FourShape f = FourShape::of(a.kv_heads, D, int(a.token_bytes));
    wait_for_earlier_work();
    const AttnReq &r = next.req;
    const int hh = blockIdx.y % f.heads, row = blockIdx.y / f.heads;
    const int kv_head = next.head * f.heads + hh;
    if (row >= r.n_new * a.group || kv_head >= a.kv_heads)
        return;
    float m = -1e30f, l = 0.0f, o[kEach] = {};
    const int at = hh * kRowsMax + row;
    for (int b = c0 + warp; b <= c1; b += kBatch * warps) {
        float2 p[kBatch];
        float v[kBatch][kEach];
#pragma unroll
        for (int y = 0; y < kBatch; ++y) {
            const int c = b + y * warps;
            const float *part = w.partial + (2 * int64_t(c) + (c == c0)) * kSlot;
            p[y] = make_float2(-1e30f, 0.0f);
            if (c <= c1)
                p[y] = __ldcg(
                    reinterpret_cast<const float2 *>(part + kFourWarps * kRowsMax * D) + at);
#pragma unroll
            for (int k = 0; k < kEach; ++k)
                v[y][k] = c <= c1 ? __ldcg(part + at * D + 32 * k + lane) : 0.0f;
        }
        float top = m;
#pragma unroll
        for (int y = 0; y < kBatch; ++y)
            top = fmaxf(top, p[y].x);
        const float keep = exp2_(m - top);
        m = top;
        l *= keep;
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            o[k] *= keep;
#pragma unroll
        for (int y = 0; y < kBatch; ++y) {
            const float x = exp2_(p[y].x - top);
            l += p[y].y * x;
#pragma unroll
            for (int k = 0; k < kEach; ++k)
                o[k] += v[y][k] * x;
        }
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        sum[warp][32 * k + lane] = o[k];
    if (lane == 0) {
        ml[warp][0] = m;
        ml[warp][1] = l;
    }
    __syncthreads();
    if (threadIdx.x >= D / 2)
        return;
    float mm = -1e30f, ll = 0.0f, lo = 0.0f, hi = 0.0f;
    for (int k = 0; k < warps; ++k)
        mm = fmaxf(mm, ml[k][0]);
#pragma unroll 4
    for (int k = 0; k < warps; ++k) {
        const float y = exp2_(ml[k][0] - mm);
        ll += ml[k][1] * y;
        lo += sum[k][2 * threadIdx.x] * y;
        hi += sum[k][2 * threadIdx.x + 1] * y;
    }
    const int tok = row / a.group, head = kv_head * a.group + row - tok * a.group;
    const int64_t orow = r.row_begin + tok;
    const float g = a.v_scale / ll;
    reinterpret_cast<unsigned *>(a.out + orow * a.out_stride + head * (D * 2))[threadIdx.x] =
        E::pack(lo * g, hi * g);
    if (a.lse && threadIdx.x == 0)
        a.lse[orow * a.q_heads + head] = mm * kLn2 + logf(ll);
}

}  // namespace
