// kvx_attend.cu -- append and attention over the pages of a paged KV cache: plans, entry
// points and kernels.  The checks are in kvx_cache_host.cpp.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "kvx_cache.h"
#include "kvx_ctx.h"

using kvx::AttnReq;

struct kvx_attn_plan {
    kvx_ctx *ctx = nullptr;
    kvx_attn_cfg cfg = {};
    int32_t page_size = 0, num_pages = 0, num_layers = 0;
    int64_t token_bytes = 0;
    char **pools = nullptr;    // host: [2 * layer + kv]
    int capacity = 0;          // requests
    int n_req = 0;
    int64_t rows = 0;
    char *host = nullptr;      // pinned image of the device descriptors
    char *dev = nullptr;
    size_t bytes = 0;
    cudaEvent_t copied = nullptr;  // the last update's copy
};

namespace {

struct Step {
    const AttnReq *reqs;
    unsigned int *status;
    int32_t n_req;
    int32_t rows;
    int32_t page_size;
    int32_t num_pages;
};

template <int TYPE>
struct Elem;
template <>
struct Elem<KVX_TYPE_HALF> {
    typedef __half T;
    static __device__ float load(T x) { return __half2float(x); }
    static __device__ T store(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<KVX_TYPE_BFLOAT> {
    typedef __nv_bfloat16 T;
    static __device__ float load(T x) { return __bfloat162float(x); }
    static __device__ T store(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<KVX_TYPE_FP_EIGHT> {
    typedef __nv_fp8_e4m3 T;
    static __device__ float load(T x) { return float(x); }
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

// A warp per (new token, K or V).
template <int TYPE, int KV>
__global__ void __launch_bounds__(256)
kvx_append_kernel(const Append a)
{
    const int lane = threadIdx.x & 31;
    const int64_t job = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (job >= 2 * int64_t(a.step.rows))
        return;
    const int row = int(job >> 1), kv = int(job & 1);
    const AttnReq q = a.step.reqs[request_of_row(a.step.reqs, a.step.n_req, row, lane)];
    const int pos = q.n_tokens - q.n_new + row - q.row_begin;
    const int page = q.table[pos / a.step.page_size];
    if (unsigned(page) >= unsigned(a.step.num_pages)) {
        if (lane == 0)
            atomicOr(a.step.status, KVX_DEV_PAGE_OUT_OF_RANGE);
        return;
    }
    const char *src = a.src[kv] + row * a.stride[kv];
    char *dst = a.pool[kv] +
                (int64_t(page) * a.step.page_size + pos % a.step.page_size) * a.token_bytes;
    for (int u = lane; u < a.units; u += 32) {
        if (KV == TYPE) {
            reinterpret_cast<uint4 *>(dst)[u] = reinterpret_cast<const uint4 *>(src)[u];
        } else {
            typedef typename Elem<TYPE>::T T;
            alignas(16) T in[16];
            reinterpret_cast<uint4 *>(in)[0] = reinterpret_cast<const uint4 *>(src)[2 * u];
            reinterpret_cast<uint4 *>(in)[1] = reinterpret_cast<const uint4 *>(src)[2 * u + 1];
            alignas(16) unsigned char out[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                out[i] = __nv_cvt_float_to_fp8(Elem<TYPE>::load(in[i]) / a.scale[kv],
                                               __NV_SATFINITE, __NV_E4M3);
            reinterpret_cast<uint4 *>(dst)[u] = *reinterpret_cast<uint4 *>(out);
        }
    }
}

// ------------------------------------------------------------------------------- attend

struct Attend {
    Step step;
    const char *q;
    char *out;
    float *lse;
    int64_t q_stride, out_stride;  // bytes between tokens
    const char *k, *v;             // layer's pools
    int64_t token_bytes;
    const float *slopes;
    int32_t q_heads, kv_heads, window;
    float scale;                   // of q . k, with k_scale
    float softcap, v_scale;
};

// A warp per (row, query head), one key at a time.
template <int TYPE, int KV, int D>
__global__ void __launch_bounds__(128)
kvx_attend_kernel(const Attend a)
{
    typedef Elem<TYPE> E;
    typedef Elem<KV> C;
    const int lane = threadIdx.x & 31;
    const int64_t job = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (job >= int64_t(a.step.rows) * a.q_heads)
        return;
    const int row = int(job / a.q_heads), h = int(job % a.q_heads);
    const int kvh = h / (a.q_heads / a.kv_heads);
    const AttnReq r = a.step.reqs[request_of_row(a.step.reqs, a.step.n_req, row, lane)];
    const int pos = r.n_tokens - r.n_new + row - r.row_begin;
    const int low = a.window ? max(0, pos - a.window + 1) : 0;
    float q[D / 32], o[D / 32];
    const typename E::T *qp = reinterpret_cast<const typename E::T *>(a.q + row * a.q_stride) + h * D;
    for (int i = 0; i < D / 32; ++i) {
        q[i] = E::load(qp[lane + 32 * i]);
        o[i] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    const int end = max(pos + 1, r.prefix);
    for (int j = 0; j < end; ++j) {
        if (j >= r.prefix && j < low) {
            j = low - 1;
            continue;
        }
        const int page = r.table[j / a.step.page_size];
        if (unsigned(page) >= unsigned(a.step.num_pages)) {
            if (lane == 0)
                atomicOr(a.step.status, KVX_DEV_PAGE_OUT_OF_RANGE);
            continue;
        }
        const int64_t at = (int64_t(page) * a.step.page_size + j % a.step.page_size) * a.token_bytes;
        const typename C::T *k = reinterpret_cast<const typename C::T *>(a.k + at) + kvh * D;
        const typename C::T *v = reinterpret_cast<const typename C::T *>(a.v + at) + kvh * D;
        float s = 0.0f;
        for (int i = 0; i < D / 32; ++i)
            s += q[i] * C::load(k[lane + 32 * i]);
        for (int d = 16; d; d >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale;
        if (a.softcap > 0.0f)
            s = a.softcap * tanhf(s / a.softcap);
        if (a.slopes)
            s -= a.slopes[h] * fabsf(float(pos - j));
        const float m2 = fmaxf(m, s), keep = expf(m - m2), p = expf(s - m2);
        l = l * keep + p;
        for (int i = 0; i < D / 32; ++i)
            o[i] = o[i] * keep + p * C::load(v[lane + 32 * i]);
        m = m2;
    }
    typename E::T *op = reinterpret_cast<typename E::T *>(a.out + row * a.out_stride) + h * D;
    for (int i = 0; i < D / 32; ++i)
        op[lane + 32 * i] = E::store(o[i] / l * a.v_scale);
    if (a.lse && lane == 0)
        a.lse[job] = m + logf(l);
}

// ---------------------------------------------------------------------------------- host

kvx_status fill_plan(kvx_attn_plan *p, const kvx_request *reqs, int n_req, const int32_t *n_new,
                     const int32_t *prefix, cudaStream_t s)
{
    kvx_ctx *ctx = p->ctx;
    cudaError_t e = cudaEventSynchronize(p->copied);  // the image may still be being read
    if (e != cudaSuccess)
        return kvx::cuda_err(ctx, e, "waiting for the plan's last copy");
    AttnReq *out = reinterpret_cast<AttnReq *>(p->host);
    int64_t rows = 0;
    for (int r = 0; r < n_req; ++r) {
        out[r] = {reqs[r].page_table, reqs[r].n_tokens, n_new[r], prefix ? prefix[r] : 0,
                  int32_t(rows), {0, 0}};
        rows += n_new[r];
    }
    p->n_req = n_req;
    p->rows = rows;
    if (n_req) {
        e = cudaMemcpyAsync(p->dev, p->host, n_req * sizeof(AttnReq), cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess)
            e = cudaEventRecord(p->copied, s);
    }
    return e == cudaSuccess ? KVX_OK : kvx::cuda_err(ctx, e, "plan copy");
}

kvx_status io_check(const kvx_attn_plan *p, int layer, const void *x, int64_t *stride,
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

Step step_of(const kvx_attn_plan *p)
{
    return {reinterpret_cast<const AttnReq *>(p->dev), p->ctx->status_dev, p->n_req,
            int32_t(p->rows), p->page_size, p->num_pages};
}

const void *attend_kernel(const kvx_attn_cfg &c)
{
#define PICK(T, K)                                                                    \
    if (c.type == T && c.kv_type == K)                                                \
        return c.head_dim == 64 ? reinterpret_cast<const void *>(kvx_attend_kernel<T, K, 64>) \
                                : reinterpret_cast<const void *>(kvx_attend_kernel<T, K, 128>);
    PICK(KVX_TYPE_HALF, KVX_TYPE_HALF)
    PICK(KVX_TYPE_HALF, KVX_TYPE_FP_EIGHT)
    PICK(KVX_TYPE_BFLOAT, KVX_TYPE_BFLOAT)
    PICK(KVX_TYPE_BFLOAT, KVX_TYPE_FP_EIGHT)
#undef PICK
    return nullptr;
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
    p->page_size = pool->page_size;
    p->num_pages = pool->num_pages;
    p->num_layers = pool->num_layers;
    p->token_bytes = pool->token_bytes;
    p->capacity = n_req;
    p->bytes = std::max<size_t>(1, n_req) * sizeof(AttnReq);
    p->pools = new (std::nothrow) char *[2 * size_t(pool->num_layers)];
    if (!p->pools) {
        kvx_attn_plan_destroy(p);
        return kvx::set_err(ctx, KVX_ERR_CAPACITY, "out of host memory");
    }
    kvx::pack_slabs(pool, p->pools);
    cudaError_t e = cudaHostAlloc(reinterpret_cast<void **>(&p->host), p->bytes,
                                  cudaHostAllocDefault);
    if (e == cudaSuccess)
        e = cudaMalloc(reinterpret_cast<void **>(&p->dev), p->bytes);
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
        if (p->dev)
            cudaFree(p->dev);
        if (p->host)
            cudaFreeHost(p->host);
    }
    delete[] p->pools;
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
    kvx_status st = io_check(p, layer, k, &k_stride, p->cfg.kv_heads, "k");
    if (st == KVX_OK)
        st = io_check(p, layer, v, &v_stride, p->cfg.kv_heads, "v");
    if (st != KVX_OK)
        return st;
    if (p->cfg.kv_type == KVX_TYPE_FP_EIGHT &&
        !(k_scale > 0.0f && v_scale > 0.0f && std::isfinite(k_scale) && std::isfinite(v_scale)))
        return kvx::set_err(p->ctx, KVX_ERR_INVALID_ARG, "k_scale %g, v_scale %g",
                            double(k_scale), double(v_scale));
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
    const cudaError_t e = cudaLaunchKernel(fn, dim3(unsigned((2 * p->rows + 7) / 8)), dim3(256),
                                           args, 0, reinterpret_cast<cudaStream_t>(stream));
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
    Attend a = {step_of(p), static_cast<const char *>(q), static_cast<char *>(out), lse, q_stride,
                out_stride, p->pools[2 * layer], p->pools[2 * layer + 1], p->token_bytes,
                p->cfg.slopes, p->cfg.q_heads, p->cfg.kv_heads, p->cfg.window,
                p->cfg.scale * k_scale, p->cfg.softcap, v_scale};
    void *args[] = {&a};
    const int64_t jobs = p->rows * p->cfg.q_heads;
    const cudaError_t e = cudaLaunchKernel(attend_kernel(p->cfg), dim3(unsigned((jobs + 3) / 4)),
                                           dim3(128), args, 0,
                                           reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KVX_OK : kvx::cuda_err(p->ctx, e, "attention launch");
}

}  // extern "C"
