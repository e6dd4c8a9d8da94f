// kvx_rotate.cu -- append of a step's new K and V to their pages with the position rotation on
// the way, and rotation of q; also the plain append into a 4-bit cache.
#include <cuda_runtime.h>

#include <cmath>

#include "kvx_attend_plan.h"

namespace {

struct Rotate {
    Step step;
    const char *src[3];       // q (or NULL), K, V
    int64_t stride[3];        // bytes between tokens
    char *q_out;
    int64_t q_out_stride;
    char *pool[2];
    int64_t token_bytes;      // of the cache
    const float *freqs;
    const int32_t *positions;
    float scale[2];           // of K and V
    float six[2];             // 1 / (6 scale)
    float magnitude;
    int32_t q_heads, kv_heads;  // q_heads 0: no q
    int32_t rotary, interleaved;
};

// An angle in units of 2^-64 turns wraps where it should, at whole turns, and is exact however
// large the position.  A frequency f = m 2^e (m of 24 bits) is f / (2 pi) turns per position:
// the product of m with 1 / (2 pi) in 64 bits, shifted.
const uint64_t kPerTurn = 0x28be60db9391054aull;  // 2^64 / (2 pi)

__device__ __forceinline__ uint64_t turns_of(float f)
{
    const unsigned bits = __float_as_uint(f);
    const int e = int(bits >> 23 & 255);
    const uint64_t m = e ? (bits & 0x7fffff) | 0x800000 : bits & 0x7fffff;
    const uint64_t lo = m * kPerTurn, hi = __umul64hi(m, kPerTurn);
    const int right = 150 - max(e, 1);  // f = m 2^-right
    uint64_t t;
    if (right >= 128)
        t = 0;
    else if (right >= 64)
        t = hi >> (right - 64);
    else if (right > 0)
        t = lo >> right | hi << (64 - right);
    else
        t = -right < 64 ? lo << -right : 0;
    return bits >> 31 ? 0 - t : t;
}

// Cosine and sine of `turns`: the nearest quarter taken off, then the power series, whose next
// terms are below 2^-25 at an eighth of a turn.  What x is rounded by is put right to first
// order, so that both are off by little more than their own last rounding.
__device__ __forceinline__ float2 cos_sin(uint64_t turns)
{
    const uint64_t quarter = (turns + (1ull << 61)) >> 62;
    const int rest = int(int64_t(turns - (quarter << 62)) >> 32);  // in 2^-32 turns
    constexpr double kStep = 6.283185307179586476925 / 4294967296.0;
    constexpr float kHi = float(kStep), kLo = float(kStep - double(kHi));
    const float f = float(rest), x = f * kHi;
    const float lo = fmaf(f, kHi, -x) + fmaf(f, kLo, float(rest - int(f)) * kHi);
    const float u = x * x;
    float s = 1.0f / 362880, c = 1.0f / 40320;
    s = fmaf(s, u, -1.0f / 5040);
    s = fmaf(s, u, 1.0f / 120);
    s = fmaf(s, u, -1.0f / 6);
    c = fmaf(c, u, -1.0f / 720);
    c = fmaf(c, u, 1.0f / 24);
    c = fmaf(c, u, -0.5f);
    s = fmaf(s * u, x, lo) + x;
    c = fmaf(c, u, -lo * x) + 1.0f;
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Eight numbers as e2m1 codes, the first in the low half of the low byte.
__device__ __forceinline__ unsigned e2m1_of_8(const float (&x)[8])
{
    unsigned r;
    asm("{ .reg .b8 a, b, c, d; cvt.rn.satfinite.e2m1x2.f32 a, %2, %1; "
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3; cvt.rn.satfinite.e2m1x2.f32 c, %6, %5; "
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7; mov.b32 %0, {a, b, c, d}; }"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

const int kRotateThreads = 256;

// A CTA takes a new token.  Moving q, K and V is what bounds it: 8.2k tokens of 32 + 8 heads 36.7
// us (203 MB, 5.5 TB/s, 82 % of a device copy's rate; 41.8 with the data asked for after the
// angles), 64 tokens 3.4 us, a launch and the chain table, angles, data.  The angles go to shared
// memory, then D / 16 lanes take a head, two units of eight elements each: units j and
// j + rotary / 16 where pairs lie half of rotary_dim apart, neighbours otherwise.  For a 4-bit
// cache the largest magnitude of a block is that of two units, which meet by way of two shuffles.
template <int TYPE, int KV, int D>
__global__ void __launch_bounds__(kRotateThreads)
kvx_append_rotated_kernel(const Rotate a)
{
    typedef Elem<TYPE> E;
    typedef typename E::T T;
    constexpr int kLanes = D / 16;
    __shared__ float2 turn[D / 2 + D / 16];  // a gap after each eight, for the banks
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x;
    const int pairs = a.rotary / 16;  // lanes of a head that rotate
    const int jobs = (a.q_heads + 2 * a.kv_heads) * kLanes;
    // What a job reads: its head, kind (0 q, 1 K, 2 V) and units of eight elements, which may lie
    // apart where they rotate.
    auto job_of = [&](int job, int &head, int &kind, int &u0, int &u1) {
        const int j = job % kLanes;
        head = job / kLanes;
        kind = 0;
        if (head >= a.q_heads) {
            head -= a.q_heads;
            kind = 1;
            if (head >= a.kv_heads) {
                head -= a.kv_heads;
                kind = 2;
            }
        }
        const bool apart = kind < 2 && j < pairs && !a.interleaved;
        u0 = apart ? j : 2 * j;
        u1 = apart ? j + pairs : 2 * j + 1;
    };
    auto load = [&](int job0, uint4 (&in)[2]) {
        int head, kind, u0, u1;
        job_of(min(job0 + lane, jobs - 1), head, kind, u0, u1);
        const uint4 *src = reinterpret_cast<const uint4 *>(a.src[kind] + row * a.stride[kind] +
                                                           head * (D * 2));
        in[0] = src[u0];
        in[1] = src[u1];
    };
    // Whole warps stay together, for the shuffles.  The data is on its way before anything else.
    const int job_first = threadIdx.x - lane;
    wait_for_earlier_work();
    uint4 in[2];
    load(job_first, in);
    const AttnReq q = a.step.reqs[request_of_row(a.step.reqs, a.step.n_req, row, lane)];
    const int pos = q.n_tokens - q.n_new + row - q.row_begin, nth = a.step.page.div(pos);
    const int page = q.table[nth];
    if (a.rotary) {
        const int at = a.positions ? a.positions[row] : pos;
        for (int i = threadIdx.x; i < a.rotary / 2; i += blockDim.x) {
            const float2 t = cos_sin(turns_of(a.freqs[i]) * uint64_t(int64_t(at)));
            turn[i + i / 8] = make_float2(t.x * a.magnitude, t.y * a.magnitude);
        }
        __syncthreads();
    }
    const bool held = unsigned(page) < unsigned(a.step.num_pages);
    if (!held && threadIdx.x == 0)
        atomicOr(a.step.status, KVX_DEV_PAGE_OUT_OF_RANGE);
    const int64_t slot = int64_t(held ? page : 0) * a.step.page_size + pos - nth * a.step.page_size;

    for (int job0 = job_first; job0 < jobs; job0 += blockDim.x) {
        uint4 later[2] = {in[0], in[1]};
        if (job0 + int(blockDim.x) < jobs)
            load(job0 + blockDim.x, later);
        const bool mine = job0 + lane < jobs;
        const int j = min(job0 + lane, jobs - 1) % kLanes;
        int head, kind, u0, u1;
        job_of(min(job0 + lane, jobs - 1), head, kind, u0, u1);
        const bool turned = kind < 2 && j < pairs, apart = turned && !a.interleaved;
        float x[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[i][k] = E::load(reinterpret_cast<const T *>(&in[i])[k]);
        if (apart) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 t = turn[9 * u0 + k];
                const float p = x[0][k], r = x[1][k];
                x[0][k] = p * t.x - r * t.y;
                x[1][k] = r * t.x + p * t.y;
            }
        } else if (turned) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    const int pair = 4 * (i ? u1 : u0) + k / 2;
                    const float2 t = turn[pair + pair / 8];
                    const float p = x[i][k], r = x[i][k + 1];
                    x[i][k] = p * t.x - r * t.y;
                    x[i][k + 1] = r * t.x + p * t.y;
                }
        }
        if (KV == TYPE || kind == 0) {
            if (turned) {  // the others keep their bytes
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    in[i] = make_uint4(E::pack(x[i][0], x[i][1]), E::pack(x[i][2], x[i][3]),
                                       E::pack(x[i][4], x[i][5]), E::pack(x[i][6], x[i][7]));
            }
        }
        float top[2] = {0.0f, 0.0f};
        if (KV == KVX_TYPE_FP_FOUR) {
            // The other half of a unit's block: unit u ^ 1, wherever it is held.
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    top[i] = max_nan(top[i], fabsf(x[i][k]));
            float both[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int other = (i ? u1 : u0) ^ 1;
                const bool far = kind < 2 && !a.interleaved && other < 2 * pairs;
                const int from = far ? other % max(pairs, 1) : other / 2;
                const bool second = far ? other >= pairs : other & 1;
                const float f0 = __shfl_sync(0xffffffffu, top[0], lane - j + from);
                const float f1 = __shfl_sync(0xffffffffu, top[1], lane - j + from);
                both[i] = max_nan(top[i], second ? f1 : f0);
            }
            top[0] = both[0];
            top[1] = both[1];
        }
        const uint4 out[2] = {in[0], in[1]};
        in[0] = later[0];
        in[1] = later[1];
        if (!mine)
            continue;
        if (kind == 0) {
            char *dst = a.q_out + row * a.q_out_stride + head * (D * 2);
            reinterpret_cast<uint4 *>(dst)[u0] = out[0];
            reinterpret_cast<uint4 *>(dst)[u1] = out[1];
            continue;
        }
        if (!held)
            continue;
        char *token = a.pool[kind - 1] + slot * a.token_bytes;
        const float scale = a.scale[kind - 1];
        if (KV == TYPE) {
            uint4 *dst = reinterpret_cast<uint4 *>(token + head * (D * 2));
            dst[u0] = out[0];
            dst[u1] = out[1];
        } else if (KV == KVX_TYPE_FP_EIGHT) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                unsigned r[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 lo = make_float2(x[i][4 * h] / scale, x[i][4 * h + 1] / scale);
                    const float2 hi = make_float2(x[i][4 * h + 2] / scale, x[i][4 * h + 3] / scale);
                    r[h] = __nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3) |
                           unsigned(__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3)) << 16;
                }
                reinterpret_cast<uint2 *>(token + head * D)[i ? u1 : u0] = make_uint2(r[0], r[1]);
            }
        } else {
            char *scales = token + a.kv_heads * (D / 2) + head * (D / 16);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int u = i ? u1 : u0;
                const unsigned unit = __nv_cvt_float_to_fp8(top[i] * a.six[kind - 1],
                                                            __NV_SATFINITE, __NV_E4M3);
                const float s = Elem<KVX_TYPE_HALF>::load(
                                    __half(__nv_cvt_fp8_to_halfraw(__nv_fp8_storage_t(unit),
                                                                   __NV_E4M3))) * scale;
                const float f = s > 0.0f ? 1.0f / s : 0.0f;
                float y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    y[k] = f > 0.0f ? x[i][k] * f : 0.0f;
                reinterpret_cast<unsigned *>(token + head * (D / 2))[u] = e2m1_of_8(y);
                if (!(u & 1))
                    scales[u / 2] = char(unit);
            }
        }
    }
}

template <int TYPE, int D>
const void *pick_append(int kv_type)
{
    return kv_type == KVX_TYPE_FP_FOUR
               ? reinterpret_cast<const void *>(
                     kvx_append_rotated_kernel<TYPE, KVX_TYPE_FP_FOUR, D>)
           : kv_type == KVX_TYPE_FP_EIGHT
               ? reinterpret_cast<const void *>(
                     kvx_append_rotated_kernel<TYPE, KVX_TYPE_FP_EIGHT, D>)
               : reinterpret_cast<const void *>(kvx_append_rotated_kernel<TYPE, TYPE, D>);
}

}  // namespace

kvx_status kvx::append_rotated(const kvx_attn_plan *p, int layer, const kvx_rope *rope,
                               const void *q, int64_t q_stride, void *q_out,
                               int64_t q_out_stride, const void *k, const void *v,
                               int64_t k_stride, int64_t v_stride, float k_scale, float v_scale,
                               cudaStream_t s)
{
    kvx_status st = io_check(p, layer, k, &k_stride, p->cfg.kv_heads, "k");
    if (st == KVX_OK)
        st = io_check(p, layer, v, &v_stride, p->cfg.kv_heads, "v");
    if (st == KVX_OK && q)
        st = io_check(p, layer, q, &q_stride, p->cfg.q_heads, "q");
    if (st == KVX_OK && q)
        st = io_check(p, layer, q_out, &q_out_stride, p->cfg.q_heads, "q_out");
    if (st == KVX_OK)
        st = scales_check(p, k_scale, v_scale);
    if (st != KVX_OK)
        return st;
    if (q && q == q_out && q_stride != q_out_stride)
        return kvx::set_err(p->ctx, KVX_ERR_INVALID_ARG, "q_out is q with another stride");
    kvx::DeviceGuard guard(p->ctx->device);
    if (!guard.ok)
        return kvx::set_err(p->ctx, KVX_ERR_CUDA, "cannot make device %d current",
                            p->ctx->device);
    Rotate a = {};
    a.step = step_of(p);
    a.src[0] = static_cast<const char *>(q);
    a.src[1] = static_cast<const char *>(k);
    a.src[2] = static_cast<const char *>(v);
    a.stride[0] = q_stride;
    a.stride[1] = k_stride;
    a.stride[2] = v_stride;
    a.q_out = static_cast<char *>(q_out);
    a.q_out_stride = q_out_stride;
    a.pool[0] = p->pools[2 * layer];
    a.pool[1] = p->pools[2 * layer + 1];
    a.token_bytes = p->token_bytes;
    a.scale[0] = k_scale;
    a.scale[1] = v_scale;
    a.six[0] = float(1.0 / (6.0 * double(k_scale)));
    a.six[1] = float(1.0 / (6.0 * double(v_scale)));
    a.q_heads = q ? p->cfg.q_heads : 0;
    a.kv_heads = p->cfg.kv_heads;
    if (rope) {
        a.freqs = rope->freqs;
        a.positions = rope->positions;
        a.magnitude = rope->magnitude;
        a.rotary = rope->rotary_dim;
        a.interleaved = rope->interleaved;
    }
    const bool half = p->cfg.type == KVX_TYPE_HALF;
    const void *fn = p->cfg.head_dim == 64
                         ? half ? pick_append<KVX_TYPE_HALF, 64>(p->cfg.kv_type)
                                : pick_append<KVX_TYPE_BFLOAT, 64>(p->cfg.kv_type)
                         : half ? pick_append<KVX_TYPE_HALF, 128>(p->cfg.kv_type)
                                : pick_append<KVX_TYPE_BFLOAT, 128>(p->cfg.kv_type);
    const int64_t jobs = (int64_t(a.q_heads) + 2 * a.kv_heads) * (p->cfg.head_dim / 16);
    const int64_t rounds = (jobs + kRotateThreads - 1) / kRotateThreads;  // shared out evenly
    const int threads = int((jobs + 32 * rounds - 1) / (32 * rounds) * 32);
    void *args[] = {&a};
    const cudaError_t e = launch_early(fn, dim3(unsigned(p->rows)), threads, 0, s, args);
    return e == cudaSuccess ? KVX_OK : kvx::cuda_err(p->ctx, e, "append launch");
}

extern "C" {

kvx_status kvx_append_rotated(const kvx_attn_plan *p, int layer, const kvx_rope *rope,
                              const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride,
                              const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                              float k_scale, float v_scale, kvx_stream_t stream)
{
    if (!p)
        return KVX_ERR_INVALID_ARG;
    const kvx_status st = kvx::validate_rope(rope, p->cfg.head_dim, p->ctx->err,
                                             sizeof p->ctx->err);
    if (st != KVX_OK)
        return st;
    if (p->rows == 0)
        return KVX_OK;
    return kvx::append_rotated(p, layer, rope, q, q_stride, q_out, q_out_stride, k, v, k_stride,
                               v_stride, k_scale, v_scale,
                               reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
