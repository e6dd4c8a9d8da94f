// kvx_attend_rows.cuh -- attention of at most 16 rows per KV head (single new tokens, a few
// drafted ones): the cache is read once and each byte of it meets few rows, so what bounds the
// kernel is reading K and V.  Included by kvx_attend.cu, and by kvx_attend_four.cuh
// for what the kernels of few rows share.
#pragma once

#include "kvx_attend.cuh"

namespace {

// A CTA of eight warps takes a unit (request, KV head) 128 keys at a time, 16 to a warp.  Each
// warp streams its own keys through a private ring of shared-memory stages with asynchronous
// copies and keeps its own running maximum, sum and output in registers, so warps wait for
// nobody until the unit ends; then the eight results are joined in shared memory.
//
// The products are taken transposed, S' = K Q' and O' = V' P', on m16n8k16 matrix instructions:
// keys and head elements fill the 16 rows and the unit's rows (new tokens x heads that share
// the KV head) are the 8 columns, NT times.  With the unit's rows as the 16 instead, half of
// the work and of the accumulators went to rows that do not exist.  P' changes from result to
// operand by a transposition of 8 x 8 blocks between lanes.
//
// An e4m3 cache is multiplied in half precision, which holds every code exactly, whatever the
// type of q: q is first scaled by a power of two per row to at most 1.  That is exact for
// elements down to 2^-17 of full scale in bfloat16 (8 bits above half's last, 2^-24), to 2^-14
// in half; smaller ones are off by at most 2^-25 of it, which is what 32 bits make of products
// with the row's largest element.  The order of the 16 elements a matrix instruction sums over
// is free as long as both operands share it, and so is that of O's columns; they are chosen so
// that a thread's operands are 16 consecutive bytes of a key.
//
// Measured: 64 bf16 requests of 1k to 32k tokens, 8 KV heads, 321 us (2.2 GB, 6.9 TB/s; a copy
// reaches 6.8); 64 e4m3 requests, 4 KV heads, 92 us (552 MB, 5.9 TB/s, where the heads' runs
// of 128 bytes are what memory serves less well: neither more bytes in flight nor more warps
// change it); one request of 32k tokens 26 us (134 MB), of 512 tokens 5.4 us, of which three
// are a launch and the rest the chain page id, keys, products, join.
const int kRowWarps = 8;
const int kRowThreads = 32 * kRowWarps;
const int kRowKeys = 16;                      // keys per warp and step
const int kRowTile = kRowKeys * kRowWarps;
const int kRowMax = 16;                       // rows of a unit, NT = 2
const int kRowStages = 6;                     // at most
const int kJoinSums = 64 << 10;               // in the rings, past m and l of all parts

// Two CTAs share an SM where a stage of 16 keys is small enough that both rings, and the
// registers of NT = 1, leave them room: their joins then hide behind each other's streaming.
template <int KV, int D, int NT>
__host__ __device__ constexpr int row_ctas_per_sm()
{
    return NT == 1 && D * (KV == KVX_TYPE_FP_EIGHT ? 1 : 2) <= 128 ? 2 : 1;
}

template <int KV, int D, int NT>
__host__ __device__ constexpr int row_ring()  // bytes of a warp's ring
{
    return (24 << 10) / row_ctas_per_sm<KV, D, NT>();
}

template <int D, int NT>
__host__ __device__ constexpr int row_slot_floats()  // a partial result: O, m, l
{
    return 8 * NT * (D + 2);
}

template <int KV, int D, int NT>
constexpr size_t row_smem()
{
    return size_t(kRowWarps) * row_ring<KV, D, NT>() + kRowWarps * 8 * NT * 2 * 4;
}

__device__ __forceinline__ void ldmatrix4(unsigned (&r)[4], unsigned addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(unsigned (&r)[4], unsigned addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <int TYPE>
__device__ __forceinline__ void mma16816(float (&d)[4], const unsigned (&a)[4], unsigned b0,
                                         unsigned b1)
{
    if (TYPE == KVX_TYPE_HALF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four e4m3 codes (low byte first) as two pairs of half-precision numbers.
__device__ __forceinline__ void half4_of_e4m3(unsigned four, unsigned &lo, unsigned &hi)
{
    asm("{ .reg .b16 x, y; mov.b32 {x, y}, %2; cvt.rn.f16x2.e4m3x2 %0, x; "
        "cvt.rn.f16x2.e4m3x2 %1, y; }"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}

__device__ __forceinline__ unsigned transpose8x8(unsigned x)
{
    unsigned r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint4 lds16(unsigned addr)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(addr)
                 : "memory");
    return r;
}

__device__ __forceinline__ uint2 lds8(unsigned addr)
{
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr) : "memory");
    return r;
}

// Layout of a stage and of the matrix operands taken from it.  Rows of D elements lie back to
// back; 16-byte chunks are permuted within 128-byte lines so that the reads of a warp spread
// over all banks.
template <int KV, int D, int NT>
struct RowLayout {
    static const int kItem = KV == KVX_TYPE_FP_EIGHT ? 1 : 2;
    static const int kRow = D * kItem;                 // bytes of a key
    static const int kChunks = kRow / 16;
    static const int kSide = kRowKeys * kRow;          // bytes of K (or V) in a stage
    static const int kStage = 2 * kSide;
    static const int kRing = row_ring<KV, D, NT>();
    static const int kNumStages = kRing / kStage < kRowStages ? kRing / kStage : kRowStages;
    static const bool kEight = KV == KVX_TYPE_FP_EIGHT;

    // Byte offset of chunk c of key t.
    static __device__ __forceinline__ int k_at(int t, int c)
    {
        if (!kEight)  // ldmatrix reads one chunk column of eight keys
            return t * kRow + ((c ^ (t & 7)) << 4);
        if (D == 128)  // four chunks of two keys at a time
            return t * kRow + ((c ^ ((t & 1) << 2)) << 4);
        return t * kRow + (c << 4);
    }
    static __device__ __forceinline__ int v_at(int t, int c)
    {
        if (!kEight)
            return t * kRow + ((c ^ (t & 7)) << 4);
        const int x = t * kChunks + c;  // one or two chunks of every second key
        return ((x & ~7) | ((x & 7) ^ ((t >> 1 & 3) << 1))) << 4;
    }
    // Element of the head in row quad + 8 * half of block mt of O'.
    static __device__ __forceinline__ int element(int mt, int half, int quad)
    {
        return kEight ? quad * (D / 8) + 2 * mt + half : 16 * mt + 8 * half + quad;
    }
};

template <int TYPE, int KV, int D, int NT>
__global__ void __launch_bounds__(kRowThreads, row_ctas_per_sm<KV, D, NT>())
kvx_attend_rows_kernel(const Attend a, const Work w)
{
    typedef RowLayout<KV, D, NT> L;
    typedef Elem<TYPE> E;
    constexpr bool kEight = L::kEight;
    constexpr int kMath = kEight ? KVX_TYPE_HALF : TYPE;  // of the matrix products
    constexpr float kRoom = Elem<kMath>::kRoom;
    constexpr int kSteps = D / 16, kRowsMax = 8 * NT;
    constexpr int kSlot = row_slot_floats<D, NT>();
    char *smem = attend_smem;
    float *ml = reinterpret_cast<float *>(smem + kRowWarps * L::kRing);  // [warp][row][m, l]
    __shared__ int flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int quad = lane >> 2, c = lane & 3;
    const unsigned ring = smem_u32(smem) + warp * L::kRing;
    const Score score(a);
    const bool plain = !(a.softcap > 0.0f) && !a.slopes;

    AttnStart at = w.starts[blockIdx.x];
    bool waited = false;  // for earlier work: the first unit's arithmetic goes before it
    while (at.tiles > 0) {
        const AttnReq r = at.req;
        Keys keys;
        keys.set<kRowTile>(r, a.window, 0, r.n_new - 1);
        const int rows = r.n_new * a.group;
        const int todo = int(min(int64_t(keys.tiles - at.tile), at.tiles));

        // The warp's keys in step i of the unit's share; last keys first, so that a bias that
        // favours near keys does not raise the maximum step by step.
        auto first_key = [&](int i) {
            const int t = keys.tiles - 1 - at.tile - i;
            return (t < keys.first ? t : t + keys.skip) * kRowTile + warp * kRowKeys;
        };
        const int64_t head_at = int64_t(at.head) * L::kRow;
        // Page of key `lane` of step i, or -1; loaded one step before it is used.
        auto page_of = [&](int i) {
            const int j = first_key(i) + (lane & (kRowKeys - 1));
            return i < todo && keys.used(j) ? r.table[a.page.div(j)] : -1;
        };
        auto issue = [&](int i, int page) {
            if (i < todo) {
                const int j = first_key(i) + (lane & (kRowKeys - 1));
                int64_t off = -1;
                if (keys.used(j)) {
                    if (unsigned(page) < unsigned(a.num_pages))
                        off = (int64_t(page) * a.page_size + j - a.page.div(j) * a.page_size) *
                                  a.token_bytes + head_at;
                    else
                        atomicOr(a.status, KVX_DEV_PAGE_OUT_OF_RANGE);
                }
                const unsigned stage = ring + (i % L::kNumStages) * L::kStage;
#pragma unroll
                for (int x = 0; x < kRowKeys * L::kChunks / 32; ++x) {
                    const int t = (x * 32 + lane) / L::kChunks, ch = lane % L::kChunks;
                    const int64_t src = __shfl_sync(0xffffffffu, off, t);
                    const bool valid = src >= 0;
                    const int64_t s = (valid ? src : 0) + ch * 16;
                    cp_async16(stage + L::k_at(t, ch), a.k + s, valid);
                    cp_async16(stage + L::kSide + L::v_at(t, ch), a.v + s, valid);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };

        if (!waited)
            wait_for_earlier_work();
        waited = true;
        int page;
        {
            int first[L::kNumStages];  // pages of the first steps, looked up together
#pragma unroll
            for (int i = 0; i < L::kNumStages; ++i)
                first[i] = page_of(i);
#pragma unroll
            for (int i = 0; i < L::kNumStages - 1; ++i)
                issue(i, first[i]);
            page = first[L::kNumStages - 1];
        }

        // q as the second operand: row quad + 8 n in column quad, zero past the unit's rows.
        // Of the scores and O', a thread has columns 2 c and 2 c + 1.
        unsigned qb[NT][kSteps][2];
        float factor[NT][2], slope[NT][2];
        int pos[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool have = quad + 8 * n < rows;
            const int row = have ? quad + 8 * n : 0, tok = row / a.group;
            const char *qp = a.q + int64_t(r.row_begin + tok) * a.q_stride +
                             (at.head * a.group + row - tok * a.group) * (D * 2);
            float up = 1.0f;
            if (!kEight) {
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qb[n][s][i] = have ? *reinterpret_cast<const unsigned *>(
                                                 qp + 2 * (16 * s + 8 * i + 2 * c)) : 0u;
            } else {
                // Step s, quad thread c: elements 64 (s / 4) + 16 c + 4 (s % 4) .. + 3, as the
                // bytes of chunk 4 (s / 4) + c of a key.
                uint2 u[kSteps];
                float top = 0.0f, down;
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    u[s] = have ? *reinterpret_cast<const uint2 *>(
                                      qp + 2 * (64 * (s >> 2) + 16 * c + 4 * (s & 3)))
                                : make_uint2(0, 0);
                    const typename E::T *e = reinterpret_cast<const typename E::T *>(&u[s]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        top = fmaxf(top, fabsf(E::load(e[i])));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                unit_scale(top, &down, &up);
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const typename E::T *e = reinterpret_cast<const typename E::T *>(&u[s]);
                    qb[n][s][0] = Elem<kMath>::pack(E::load(e[0]) * down, E::load(e[1]) * down);
                    qb[n][s][1] = Elem<kMath>::pack(E::load(e[2]) * down, E::load(e[3]) * down);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int mine = 2 * c + e + 8 * n, t = mine < rows ? mine / a.group : 0;
                pos[n][e] = keys.pmin + t;
                factor[n][e] = __shfl_sync(0xffffffffu, up, 8 * c + 4 * e) *
                               (a.softcap > 0.0f ? score.inner : score.factor);
                slope[n][e] = a.slopes && mine < rows
                                  ? a.slopes[at.head * a.group + mine - t * a.group] * kLog2e
                                  : 0.0f;
            }
        }

        float o[NT][kSteps][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int t = 0; t < kSteps; ++t)
                o[n][t][0] = o[n][t][1] = o[n][t][2] = o[n][t][3] = 0.0f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
        }

#pragma unroll 1
        for (int i = 0; i < todo; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(L::kNumStages - 2) : "memory");
            __syncwarp();
            {
                const int next = page_of(i + L::kNumStages);
                issue(i + L::kNumStages - 1, page);
                page = next;
            }
            const int j0 = first_key(i);
            const unsigned ks = ring + (i % L::kNumStages) * L::kStage, vs = ks + L::kSide;

            // Scores: s[n][2 x + e] is key j0 + quad + 8 x, row 8 n + 2 c + e.
            float s[NT][4], odd[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                s[n][0] = s[n][1] = s[n][2] = s[n][3] = odd[n][0] = odd[n][1] = odd[n][2] =
                    odd[n][3] = 0.0f;
            if (!kEight) {
#pragma unroll
                for (int t = 0; t < kSteps; t += 2) {
                    unsigned k0[4], k1[4];
                    ldmatrix4(k0, ks + L::k_at(lane & 15, 2 * t + (lane >> 4)));
                    ldmatrix4(k1, ks + L::k_at(lane & 15, 2 * t + 2 + (lane >> 4)));
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16816<kMath>(s[n], k0, qb[n][t][0], qb[n][t][1]);
                        mma16816<kMath>(odd[n], k1, qb[n][t + 1][0], qb[n][t + 1][1]);
                    }
                }
            } else {
#pragma unroll
                for (int t = 0; t < kSteps / 4; ++t) {
                    const uint4 u0 = lds16(ks + L::k_at(quad, 4 * t + c));
                    const uint4 u1 = lds16(ks + L::k_at(quad + 8, 4 * t + c));
                    const unsigned x0[4] = {u0.x, u0.y, u0.z, u0.w};
                    const unsigned x1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        unsigned k[4];
                        half4_of_e4m3(x0[y], k[0], k[2]);
                        half4_of_e4m3(x1[y], k[1], k[3]);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816<kMath>(y & 1 ? odd[n] : s[n], k, qb[n][4 * t + y][0],
                                            qb[n][4 * t + y][1]);
                    }
                }
            }

            const bool all_seen = j0 + kRowKeys <= keys.prefix ||
                                  (j0 + kRowKeys - 1 <= keys.pmin &&
                                   (!a.window || j0 > keys.pmax - a.window));
            bool lift = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int e = x & 1;
                    float z = (s[n][x] + odd[n][x]) * factor[n][e];
                    if (!plain) {
                        if (a.softcap > 0.0f)
                            z = score.cap * tanh_(z);
                        z -= slope[n][e] * fabsf(float(pos[n][e] - j0 - quad - 8 * (x >> 1)));
                    }
                    if (!all_seen) {
                        const int j = j0 + quad + 8 * (x >> 1);
                        if (!(j < keys.prefix || (j <= pos[n][e] &&
                                                  (!a.window || pos[n][e] - j < a.window))))
                            z = -INFINITY;
                    }
                    s[n][x] = z;
                    lift |= z > m[n][e] + (kRoom + 8.0f);
                }
            // What is subtracted need not be the maximum (less kRoom): it may lag by up to
            // 2^8, which neither a 32-bit sum nor a weight in either 16-bit type minds.  So
            // lanes compare notes, and the output is rescaled, only past that.
            if (__any_sync(0xffffffffu, lift)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(s[n][e], s[n][2 + e]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1)
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        const float next = fmaxf(m[n][e], top - kRoom);
                        const float keep = next == -INFINITY ? 1.0f : exp2_(m[n][e] - next);
                        m[n][e] = next;
                        l[n][e] *= keep;
#pragma unroll
                        for (int t = 0; t < kSteps; ++t) {
                            o[n][t][e] *= keep;
                            o[n][t][2 + e] *= keep;
                        }
                    }
            }
            unsigned p[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float z[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int e = x & 1;
                    z[x] = exp2_(s[n][x] - (m[n][e] == -INFINITY ? 0.0f : m[n][e]));
                    l[n][e] += z[x];
                }
                p[n][0] = transpose8x8(Elem<kMath>::pack(z[0], z[1]));
                p[n][1] = transpose8x8(Elem<kMath>::pack(z[2], z[3]));
            }
            if (!kEight) {
#pragma unroll
                for (int t = 0; t < kSteps; ++t) {
                    unsigned v[4];
                    ldmatrix4_trans(v, vs + L::v_at((lane & 7) + 8 * (lane >> 4),
                                                    2 * t + (lane >> 3 & 1)));
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816<kMath>(o[n][t], v, p[n][0], p[n][1]);
                }
            } else {
                // Keys 2c, 2c + 1, 2c + 8, 2c + 9, elements quad * D / 8 and on.
                unsigned v[4][D / 32];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int t = 2 * c + (y & 1) + 8 * (y >> 1);
                    if (D == 128) {
                        const uint4 u = lds16(vs + L::v_at(t, quad));
                        v[y][0] = u.x, v[y][1] = u.y, v[y][D / 32 - 2] = u.z, v[y][D / 32 - 1] = u.w;
                    } else {
                        const uint2 u = lds8(vs + L::v_at(t, quad >> 1) + 8 * (quad & 1));
                        v[y][0] = u.x, v[y][1] = u.y;
                    }
                }
#pragma unroll
                for (int g = 0; g < D / 32; ++g)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const unsigned sel = half ? 0x7362 : 0x5140;  // x0 y0 x1 y1
                        unsigned k[4];
                        half4_of_e4m3(__byte_perm(v[0][g], v[1][g], sel), k[0], k[1]);
                        half4_of_e4m3(__byte_perm(v[2][g], v[3][g], sel), k[2], k[3]);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma16816<kMath>(o[n][2 * g + half], k, p[n][0], p[n][1]);
                    }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");

        // Join the warps' results in the rings' memory: [warp][row][D + 8].
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
                if (quad == 0)
                    *reinterpret_cast<float2 *>(ml + (warp * kRowsMax + 8 * n + 2 * c + e) * 2) =
                        make_float2(m[n][e], l[n][e]);
            }
        __syncthreads();
        float *join = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (8 * n + 2 * c + e < rows) {
                    float *p = join + (warp * kRowsMax + 8 * n + 2 * c + e) * (D + 8);
#pragma unroll
                    for (int t = 0; t < kSteps; ++t) {
                        p[L::element(t, 0, quad)] = o[n][t][e];
                        p[L::element(t, 1, quad)] = o[n][t][2 + e];
                    }
                }
        __syncthreads();

        const int c0 = at.tile > 0 ? at.first : int(blockIdx.x);
        const int c1 = at.tile + todo < keys.tiles ? at.last : int(blockIdx.x);
        float *slot = w.partial + (2 * int64_t(blockIdx.x) + (int(blockIdx.x) == c0)) * kSlot;
        auto write = [&](int row, int d, float4 v, float mm, float ll) {
            const int tok = row / a.group, head = at.head * a.group + row - tok * a.group;
            const int64_t orow = r.row_begin + tok;
            const float f = a.v_scale / ll;
            uint2 u = make_uint2(E::pack(v.x * f, v.y * f), E::pack(v.z * f, v.w * f));
            *reinterpret_cast<uint2 *>(a.out + orow * a.out_stride + (head * D + d) * 2) = u;
            if (a.lse && d == 0)
                a.lse[orow * a.q_heads + head] = mm * kLn2 + logf(ll);
        };
        for (int i = threadIdx.x; i < rows * (D / 4); i += kRowThreads) {
            const int row = i / (D / 4), d = i % (D / 4) * 4;
            float mm = -INFINITY, ll = 0.0f;
#pragma unroll
            for (int k = 0; k < kRowWarps; ++k)
                mm = fmaxf(mm, ml[(k * kRowsMax + row) * 2]);
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kRowWarps; ++k) {
                const float *p = ml + (k * kRowsMax + row) * 2;
                const float f = p[0] == -INFINITY ? 0.0f : exp2_(p[0] - mm);
                const float4 u = *reinterpret_cast<const float4 *>(
                    join + (k * kRowsMax + row) * (D + 8) + d);
                ll += f * p[1];
                v.x += f * u.x;
                v.y += f * u.y;
                v.z += f * u.z;
                v.w += f * u.w;
            }
            if (c0 == c1) {
                write(row, d, v, mm, ll);
            } else {
                *reinterpret_cast<float4 *>(slot + row * D + d) = v;
                if (d == 0)
                    *reinterpret_cast<float2 *>(slot + kRowsMax * D + 2 * row) =
                        make_float2(mm, ll);
            }
        }
        if (c0 != c1) {
            // The last CTA to arrive joins the parts, in order.
            __syncthreads();
            if (threadIdx.x == 0) {
                __threadfence();  // with the barrier before it, for all the CTA has written
                const unsigned n = atomicAdd(w.counters + c0, 1);
                flag = n == unsigned(c1 - c0);
                if (n == unsigned(c1 - c0))
                    w.counters[c0] = 0;
                __threadfence();
            }
            __syncthreads();
            if (flag) {
                const int parts = c1 - c0 + 1, items = rows * (D / 4);
                auto part = [&](int k) {
                    return w.partial + (2 * int64_t(c0 + k) + (k == 0)) * kSlot;
                };
                // Row i / (D / 4), four elements, over parts k0, k0 + step, ...; m and l of part
                // k's row by ml_of.
                auto joined = [&](int i, int k0, int step, auto ml_of, float &mm, float &ll) {
                    const int row = i / (D / 4), d = i % (D / 4) * 4;
                    mm = -INFINITY;
                    ll = 0.0f;
#pragma unroll 4
                    for (int k = 0; k < parts; ++k)
                        mm = fmaxf(mm, ml_of(k, row).x);
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
                    for (int k = k0; k < parts; k += step) {
                        const float4 u = __ldcg(reinterpret_cast<const float4 *>(
                            part(k) + row * D + d));
                        const float2 p = ml_of(k, row);
                        const float f = p.x == -INFINITY ? 0.0f : exp2_(p.x - mm);
                        ll += f * p.y;
                        v.x += f * u.x;
                        v.y += f * u.y;
                        v.z += f * u.z;
                        v.w += f * u.w;
                    }
                    return v;
                };
                auto ml_part = [&](int k, int row) {
                    return __ldcg(reinterpret_cast<const float2 *>(part(k) + kRowsMax * D) + row);
                };
                float mm, ll;
                if (parts <= 4 || items > kRowThreads / 2) {
                    for (int i = threadIdx.x; i < items; i += kRowThreads) {
                        const float4 v = joined(i, 0, 1, ml_part, mm, ll);
                        write(i / (D / 4), i % (D / 4) * 4, v, mm, ll);
                    }
                } else {
                    // Many parts of few rows: m and l of all of them by all threads first, and
                    // the threads that the rows leave over shared out over the parts (one
                    // request of 2k tokens 9.6 -> 8.5 us; with two parts the barriers cost
                    // more, 5.7 -> 6.1).
                    float2 *pml = reinterpret_cast<float2 *>(smem);               // [part][row]
                    float4 *sums = reinterpret_cast<float4 *>(smem + kJoinSums);  // [group][item]
                    float *sums_l = reinterpret_cast<float *>(sums + kRowThreads);
                    for (int i = threadIdx.x; i < parts * rows; i += kRowThreads)
                        pml[i] = ml_part(i / rows, i % rows);
                    __syncthreads();
                    const int groups = kRowThreads / items;
                    const int g = threadIdx.x / items, i = threadIdx.x - g * items;
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (g < groups) {
                        v = joined(i, g, groups,
                                   [&](int k, int row) { return pml[k * rows + row]; }, mm, ll);
                        sums[g * items + i] = v;
                        sums_l[g * items + i] = ll;
                    }
                    __syncthreads();
                    if (g == 0) {
                        for (int k = 1; k < groups; ++k) {
                            const float4 u = sums[k * items + i];
                            ll += sums_l[k * items + i];
                            v.x += u.x;
                            v.y += u.y;
                            v.z += u.z;
                            v.w += u.w;
                        }
                        write(i / (D / 4), i % (D / 4) * 4, v, mm, ll);
                    }
                }
            }
        }
        __syncthreads();  // the rings and ml are free for the next unit

        at.tiles -= todo;
        at.tile = 0;
        if (++at.head == a.kv_heads) {
            at.head = 0;
            ++at.request;
            if (at.tiles > 0)
                at.req = w.reqs[at.request];
        }
    }
}

}  // namespace
