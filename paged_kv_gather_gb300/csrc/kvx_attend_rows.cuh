// kvx_attend_rows.cuh -- attention of at most 16 rows per KV head (single new tokens, a few
// drafted ones): the cache is read once and each byte of it meets few rows, so what bounds the
// kernel is reading K and V.  Included by kvx_attend.cu only.
#pragma once

#include "kvx_attend.cuh"

namespace {

// A CTA of eight warps takes a unit (request, KV head) 128 keys at a time, 16 to a warp.  Each
// warp streams its own keys through a private ring of shared-memory stages with asynchronous
// copies and keeps its own running maximum, sum and output in registers, so warps wait for
// nobody until the unit ends; then the eight results are joined in shared memory.  Products
// run on m16n8k16 matrix instructions whose 16 rows hold the heads that share the KV head
// times the new tokens: rows left over cost nothing that is scarce here.
//
// An e4m3 cache is multiplied in half precision, which holds every code exactly, whatever the
// type of q: q is first scaled by a power of two per row to at most 1, which is exact for
// bfloat16 down to 2^-24 of the row's largest element.  The order of the 16 elements a matrix
// instruction sums over is free as long as both operands share it; K's is chosen so that a
// thread's operands are 16 consecutive bytes, and V's columns likewise.
const int kRowWarps = 8;
const int kRowThreads = 32 * kRowWarps;
const int kRowKeys = 16;                      // keys per warp and step
const int kRowTile = kRowKeys * kRowWarps;
const int kRowRing = 24 << 10;                // bytes of a warp's ring
const int kRowMax = 16;                       // rows of a unit
const int kRowStages = 6;                     // at most

template <int D>
__host__ __device__ constexpr int row_slot_floats() { return kRowMax * (D + 2); }  // a partial result: O, m, l

constexpr size_t row_smem()
{
    return size_t(kRowWarps) * kRowRing + kRowWarps * kRowMax * 2 * 4;
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

// Two e4m3 codes (low byte first) as two half-precision numbers.
__device__ __forceinline__ unsigned half2_of_e4m3(unsigned two)
{
    unsigned r;
    asm("{ .reg .b16 x; cvt.u16.u32 x, %1; cvt.rn.f16x2.e4m3x2 %0, x; }" : "=r"(r) : "r"(two));
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
template <int KV, int D>
struct RowLayout {
    static const int kItem = KV == KVX_TYPE_FP_EIGHT ? 1 : 2;
    static const int kRow = D * kItem;                 // bytes of a key
    static const int kChunks = kRow / 16;
    static const int kSide = kRowKeys * kRow;          // bytes of K (or V) in a stage
    static const int kStage = 2 * kSide;
    static const int kNumStages = kRowRing / kStage < kRowStages ? kRowRing / kStage : kRowStages;
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
    // Output column held in element e (0, 1) of accumulator nt by quad thread c.
    static __device__ __forceinline__ int column(int nt, int e, int c)
    {
        return kEight ? (2 * c + e) * (D / 8) + nt : nt * 8 + 2 * c + e;
    }
};

template <int TYPE, int KV, int D>
__global__ void __launch_bounds__(kRowThreads, 1)
kvx_attend_rows_kernel(const Attend a, const Work w)
{
    typedef RowLayout<KV, D> L;
    typedef Elem<TYPE> E;
    constexpr bool kEight = L::kEight;
    constexpr int kMath = kEight ? KVX_TYPE_HALF : TYPE;  // of the matrix products
    constexpr int kSteps = D / 16, kCols = D / 8;
    char *smem = attend_smem;
    float *ml = reinterpret_cast<float *>(smem + kRowWarps * kRowRing);  // [warp][row][m, l]
    __shared__ int flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int quad = lane >> 2, c = lane & 3;
    const unsigned ring = smem_u32(smem) + warp * kRowRing;
    const int64_t line0 = int64_t(blockIdx.x) * w.tiles / w.ctas;
    const int64_t line1 = (int64_t(blockIdx.x) + 1) * w.tiles / w.ctas;
    const Score score(a);

    AttnStart at = w.starts[blockIdx.x];
    int64_t line = line0;
    while (line < line1) {
        const AttnReq r = w.reqs[at.request];
        Keys keys;
        keys.set<kRowTile>(r, a.window, 0, r.n_new - 1);
        const int rows = r.n_new * a.group;
        const int64_t unit = line - at.tile;                   // the unit's first tile
        const int todo = int(min(int64_t(keys.tiles - at.tile), line1 - line));

        // q as matrix operands, zero in rows that are left over.
        unsigned qa[kSteps][4];
        float row_factor[2] = {1.0f, 1.0f}, slope[2] = {0.0f, 0.0f};
        int pos[2];
        {
            const char *qp[2];
            bool have[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = quad + 8 * x, tok = row / a.group, h = row - tok * a.group;
                have[x] = row < rows;
                pos[x] = keys.pmin + (have[x] ? tok : 0);
                const int head = at.head * a.group + (have[x] ? h : 0);
                qp[x] = a.q + int64_t(r.row_begin + (have[x] ? tok : 0)) * a.q_stride + head * D * 2;
                if (a.slopes)
                    slope[x] = a.slopes[head] * kLog2e;
            }
            if (!kEight) {
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        qa[s][i] = have[i & 1] ? *reinterpret_cast<const unsigned *>(
                                                     qp[i & 1] + 2 * (16 * s + 8 * (i >> 1) + 2 * c))
                                               : 0u;
            } else {
                // Step s, quad thread c: elements 64 (s / 4) + 16 c + 4 (s % 4) .. + 3, as the
                // bytes of chunk 4 (s / 4) + c of a key.
                float f[kSteps][2][4], top[2] = {0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint2 u = make_uint2(0, 0);
                        if (have[x])
                            u = *reinterpret_cast<const uint2 *>(
                                qp[x] + 2 * (64 * (s >> 2) + 16 * c + 4 * (s & 3)));
                        const typename E::T *e = reinterpret_cast<const typename E::T *>(&u);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            f[s][x][i] = E::load(e[i]);
                            top[x] = fmaxf(top[x], fabsf(f[s][x][i]));
                        }
                    }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
                    top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
                    float down;
                    unit_scale(top[x], &down, &row_factor[x]);
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        qa[s][x] = Elem<kMath>::pack(f[s][x][0] * down, f[s][x][1] * down);
                        qa[s][2 + x] = Elem<kMath>::pack(f[s][x][2] * down, f[s][x][3] * down);
                    }
                }
            }
        }

        float o[kCols][4];
#pragma unroll
        for (int n = 0; n < kCols; ++n)
            o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

        // The warp's keys in step i of the unit's share.
        auto first_key = [&](int i) {
            const int t = at.tile + i;
            return (t < keys.first ? t : t + keys.skip) * kRowTile + warp * kRowKeys;
        };
        const int64_t head_at = int64_t(at.head) * L::kRow;
        // Page of key `lane` of step i, or -1; loaded one step before it is used.
        auto page_of = [&](int i) {
            const int j = first_key(i) + (lane & (kRowKeys - 1));
            return i < todo && keys.used(j) ? __ldg(r.table + j / a.page_size) : -1;
        };
        auto issue = [&](int i, int page) {
            const int j = first_key(i) + (lane & (kRowKeys - 1));
            int64_t off = -1;
            if (i < todo && keys.used(j)) {
                if (unsigned(page) < unsigned(a.num_pages))
                    off = (int64_t(page) * a.page_size + j % a.page_size) * a.token_bytes + head_at;
                else
                    atomicOr(a.status, KVX_DEV_PAGE_OUT_OF_RANGE);
            }
            if (i < todo) {
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

        int page = page_of(0);
#pragma unroll 1
        for (int i = 0; i < L::kNumStages - 1; ++i) {
            const int next = page_of(i + 1);
            issue(i, page);
            page = next;
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

            // Scores: s[n][2 x + e] is row quad + 8 x, key j0 + 8 n + 2 c + e.
            float s[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
            if (!kEight) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int t = 0; t < kSteps; t += 2) {
                        unsigned b[4];
                        ldmatrix4(b, ks + L::k_at(8 * n + (lane & 7), 2 * t + (lane >> 3)));
                        mma16816<kMath>(s[n], qa[t], b[0], b[1]);
                        mma16816<kMath>(s[n], qa[t + 1], b[2], b[3]);
                    }
            } else {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int t = 0; t < kSteps / 4; ++t) {
                        const uint4 u = lds16(ks + L::k_at(8 * n + quad, 4 * t + c));
                        const unsigned x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            mma16816<kMath>(s[n], qa[4 * t + y], half2_of_e4m3(x[y] & 0xffffu),
                                            half2_of_e4m3(x[y] >> 16));
                    }
            }

            const bool all_seen = j0 + kRowKeys <= keys.prefix ||
                                  (j0 + kRowKeys - 1 <= keys.pmin &&
                                   (!a.window || j0 > keys.pmax - a.window));
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float z = s[n][2 * x + e] * row_factor[x];
                        z = a.softcap > 0.0f ? score.capped(z) : z * score.factor;
                        const int j = j0 + 8 * n + 2 * c + e;
                        if (a.slopes)
                            z -= slope[x] * fabsf(float(pos[x] - j));
                        if (!all_seen && !(j < keys.prefix ||
                                           (j <= pos[x] && (!a.window || pos[x] - j < a.window))))
                            z = -INFINITY;
                        s[n][2 * x + e] = z;
                        top[x] = fmaxf(top[x], z);
                    }
                top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
                top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
            }
            // The subtracted maximum may lag by up to 2^8, which neither a 32-bit sum nor a
            // weight in either 16-bit type minds; the output is rescaled only past that.
            if (__any_sync(0xffffffffu, top[0] > m[0] + 8.0f || top[1] > m[1] + 8.0f)) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float next = fmaxf(m[x], top[x]);
                    const float keep = next == -INFINITY ? 1.0f : exp2_(m[x] - next);
                    m[x] = next;
                    l[x] *= keep;
#pragma unroll
                    for (int n = 0; n < kCols; ++n) {
                        o[n][2 * x] *= keep;
                        o[n][2 * x + 1] *= keep;
                    }
                }
            }
            unsigned p[4];  // the weights as the first operand: keys are its columns
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float base = m[x] == -INFINITY ? 0.0f : m[x];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float p0 = exp2_(s[n][2 * x] - base), p1 = exp2_(s[n][2 * x + 1] - base);
                    l[x] += p0 + p1;
                    p[2 * n + x] = Elem<kMath>::pack(p0, p1);
                }
            }
            if (!kEight) {
#pragma unroll
                for (int n = 0; n < kCols; n += 2) {
                    unsigned b[4];
                    ldmatrix4_trans(b, vs + L::v_at(lane & 15, n + (lane >> 4)));
                    mma16816<kMath>(o[n], p, b[0], b[1]);
                    mma16816<kMath>(o[n + 1], p, b[2], b[3]);
                }
            } else {
                // Keys 2c, 2c + 1, 2c + 8, 2c + 9, columns quad * D / 8 and on.
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
                        const unsigned lo = __byte_perm(v[0][g], v[1][g], sel);
                        const unsigned hi = __byte_perm(v[2][g], v[3][g], sel);
                        const int n = 4 * g + 2 * half;
                        mma16816<kMath>(o[n], p, half2_of_e4m3(lo & 0xffffu),
                                        half2_of_e4m3(hi & 0xffffu));
                        mma16816<kMath>(o[n + 1], p, half2_of_e4m3(lo >> 16),
                                        half2_of_e4m3(hi >> 16));
                    }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");

        // Join the warps' results in the rings' memory: [warp][row][D + 8].
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
            if (c == 0) {
                float *p = ml + (warp * kRowMax + quad + 8 * x) * 2;
                p[0] = m[x];
                p[1] = l[x];
            }
        }
        __syncthreads();
        float *join = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (quad + 8 * x < rows) {
                float *p = join + (warp * kRowMax + quad + 8 * x) * (D + 8);
#pragma unroll
                for (int n = 0; n < kCols; ++n) {
                    p[L::column(n, 0, c)] = o[n][2 * x];
                    p[L::column(n, 1, c)] = o[n][2 * x + 1];
                }
            }
        __syncthreads();

        const int c0 = cta_of(w, unit), c1 = cta_of(w, unit + keys.tiles - 1);
        float *slot = w.partial + (2 * int64_t(blockIdx.x) + (int(blockIdx.x) == c0)) *
                                      row_slot_floats<D>();
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
                mm = fmaxf(mm, ml[(k * kRowMax + row) * 2]);
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kRowWarps; ++k) {
                const float *p = ml + (k * kRowMax + row) * 2;
                const float f = p[0] == -INFINITY ? 0.0f : exp2_(p[0] - mm);
                const float4 u = *reinterpret_cast<const float4 *>(
                    join + (k * kRowMax + row) * (D + 8) + d);
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
                if (d == 0) {
                    slot[kRowMax * D + 2 * row] = mm;
                    slot[kRowMax * D + 2 * row + 1] = ll;
                }
            }
        }
        if (c0 != c1) {
            // The last CTA to arrive joins the parts, in order.
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                const unsigned n = atomicAdd(w.counters + c0, 1);
                flag = n == unsigned(c1 - c0);
                if (n == unsigned(c1 - c0))
                    w.counters[c0] = 0;
                __threadfence();
            }
            __syncthreads();
            if (flag) {
                const int parts = c1 - c0 + 1;
                auto part = [&](int k) {
                    return w.partial + (2 * int64_t(c0 + k) + (k == 0)) * row_slot_floats<D>();
                };
                for (int i = threadIdx.x; i < rows * (D / 4); i += kRowThreads) {
                    const int row = i / (D / 4), d = i % (D / 4) * 4;
                    float mm = -INFINITY, ll = 0.0f;
#pragma unroll 8
                    for (int k = 0; k < parts; ++k)
                        mm = fmaxf(mm, __ldcg(part(k) + kRowMax * D + 2 * row));
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
                    for (int k = 0; k < parts; ++k) {
                        const float2 p = __ldcg(reinterpret_cast<const float2 *>(
                            part(k) + kRowMax * D + 2 * row));
                        const float4 u = __ldcg(reinterpret_cast<const float4 *>(
                            part(k) + row * D + d));
                        const float f = p.x == -INFINITY ? 0.0f : exp2_(p.x - mm);
                        ll += f * p.y;
                        v.x += f * u.x;
                        v.y += f * u.y;
                        v.z += f * u.z;
                        v.w += f * u.w;
                    }
                    write(row, d, v, mm, ll);
                }
            }
        }
        __syncthreads();  // the rings and ml are free for the next unit

        line += todo;
        at.tile = 0;
        if (++at.head == a.kv_heads) {
            at.head = 0;
            ++at.request;
        }
    }
}

}  // namespace
