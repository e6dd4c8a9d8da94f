// kvx_attend.cuh -- what the attention kernels share: element types, a step's schedule,
// visibility of keys, and the scores' arithmetic.  Included by the units that
// attend, append or select.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kvx_cache.h"

using kvx::AttnReq;
using kvx::AttnStart;

namespace {

const float kLog2e = 1.4426950408889634f;
const float kLn2 = 0.6931471805599453f;

// Division of 0 <= n < 2^31 by a number fixed on the host: with L = ceil(log2 d), n / d =
// n m >> (31 + L) for m = floor(2^(31 + L) / d) + 1, whose error n (m - 2^(31+L) / d) stays
// below 2^31, less than what reaches the next multiple.
struct Divisor {
    uint32_t m, shift;

    static Divisor of(int d)
    {
        int L = 0;
        while ((int64_t(1) << L) < d)
            ++L;
        return {uint32_t((uint64_t(1) << (31 + L)) / uint64_t(d) + 1), uint32_t(31 + L)};
    }
    __device__ __forceinline__ int div(int n) const
    {
        return int(uint64_t(uint32_t(n)) * m >> shift);
    }
};

struct Attend {
    const char *q;
    char *out;
    float *lse;
    int64_t q_stride, out_stride;  // bytes between tokens
    const char *k, *v;             // the layer's pools
    int64_t token_bytes;
    const float *slopes;
    unsigned int *status;
    int32_t q_heads, kv_heads, group, window;
    int32_t page_size, num_pages;
    Divisor page;
    int32_t box;                   // keys per tensor copy, 0: the cache is not copied that way
    float scale;                   // of q . k, with k_scale
    float softcap, v_scale;
};

// The schedule of one kernel.  The keys that each unit of rows visits, cut into tiles, are
// laid end to end over all units, and every CTA takes an equal stretch of that line, whatever
// the lengths (AttnStart); or units are dealt to the CTAs one by one, each a share of its own.
// A unit that one CTA does not finish alone is joined from partial results: CTA c keeps one it
// began and did not finish in slot 2 c + 1, and one it took over from CTA c - 1 in slot 2 c.
struct Work {
    const AttnReq *reqs;       // of this kernel, those with rows
    const AttnStart *starts;   // [CTAs], and behind them the shares that follow those
    const int32_t *cuts;       // CTAs that begin a unit and do not finish it
    unsigned int *counters;    // [CTAs]: arrivals at the unit a CTA began, zero between launches
    float *partial;
};

// Kernels here start while the one before them on the stream ends (programmatic dependent
// launch).  Before this wait for its completion they touch nothing but the plan's descriptors,
// which only copies write, and no kernel starts early behind a copy; after it they let the
// next kernel start in the same way.  What an earlier kernel may have written (tables, q, new K
// and V, the pages) is never read through the read-only path: it may change while they run.
__device__ __forceinline__ void wait_for_earlier_work()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Keys that some row of a unit sees: [0, prefix) and [low, end); positions of its first and
// last row.  Tiles of T keys: tile i holds keys from T * (i < first ? i : i + skip), so that
// keys between prefix and low are passed over in whole tiles.
struct Keys {
    int prefix, low, end, pmin, pmax;
    int first, skip, tiles;

    template <int T>
    __device__ __forceinline__ void set(const AttnReq &r, int window, int row_lo, int row_hi)
    {
        set(r, window, row_lo, row_hi, T);
    }
    __device__ __forceinline__ void set(const AttnReq &r, int window, int row_lo, int row_hi,
                                        int T)
    {
        prefix = r.prefix;
        pmin = r.n_tokens - r.n_new + row_lo;
        pmax = r.n_tokens - r.n_new + row_hi;
        low = window ? max(0, pmin - window + 1) : 0;
        end = pmax + 1;
        kvx::key_tiles(prefix, low, end, T, &first, &skip, &tiles);
    }
    __device__ __forceinline__ bool used(int j) const
    {
        return j < prefix || (j >= low && j < end);
    }
    // Keys j .. j + T - 1 are all used.
    template <int T>
    __device__ __forceinline__ bool whole(int j) const
    {
        return j + T <= prefix || (j >= low && j + T <= end) ||
               (low <= prefix && j + T <= max(prefix, end));
    }
};

__device__ __forceinline__ float exp2_(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tanh x = x P(x^2) for |x| <= 1/2: P of degree 3 with the least largest relative error there
// (6e-7 in 32 bits; by weighted least squares iterated to it).  Scores rarely leave that range
// under a cap, and it takes no special-function instruction.  kTanh[i] goes with x^(2 i).
const int kTanhTerms = 4;
__device__ constexpr float kTanh[kTanhTerms] = {0.999999464f, -0.333263189f, 0.131902963f,
                                                -0.0444022268f};

// tanh by its definition, 1 - 2 / (exp(2 x) + 1): off by a few 2^-24 of 1 whatever x, where
// the hardware's approximate tanh is off by 2^-11.
__device__ __forceinline__ float tanh_of_1(float x)
{
    return 1.0f - __fdividef(2.0f, exp2_(x * (2.0f * kLog2e)) + 1.0f);
}

// And off by a few 2^-24 of itself: a cap far above the scores, whose tanh is then small,
// multiplies what that is off by.
__device__ __forceinline__ float tanh_(float x)
{
    const float u = x * x;
    float p = kTanh[kTanhTerms - 1];
#pragma unroll
    for (int n = kTanhTerms - 2; n >= 0; --n)
        p = fmaf(p, u, kTanh[n]);
    return fabsf(x) <= 0.5f ? x * p : tanh_of_1(x);
}

// Largest |z| up to which tanh(inner z) may be had from kTanh with the powers of `inner` in the
// coefficients: 1/2 / inner, and less where a cap far above the scores makes `inner` so small
// that they fall out of the normal numbers, x^6 and x^4 or all but 1 among them, and nothing
// may be missed that they would add.  1e18: z^2 is finite.
__device__ __forceinline__ float tanh_reach(float inner)
{
    inner = fabsf(inner);
    const float x = inner > 2e-6f ? 0.5f : inner > 1e-9f ? 0.015625f : 0.00048828125f;
    return inner > 0.0f && inner < 1e4f ? fminf(x / inner, 1e18f) : 0.0f;
}

// What turns q . k into a score in units of log 2.
struct Score {
    float factor;      // without a cap: scale * log2 e
    float cap, inner;  // with one: cap * log2 e, scale / softcap

    __device__ __forceinline__ explicit Score(const Attend &a)
        : factor(a.scale * kLog2e), cap(a.softcap * kLog2e),
          inner(a.softcap > 0.0f ? a.scale / a.softcap : 0.0f)
    {
    }
};

// 2^-e and 2^e with 2^e the power of two above `top` >= 0; e is kept to what leaves both
// normal numbers.
__device__ __forceinline__ void unit_scale(float top, float *down, float *up)
{
    const int e = min(max(int(__float_as_uint(top) >> 23) - 126, -60), 126);
    *down = __uint_as_float(unsigned(127 - e) << 23);
    *up = __uint_as_float(unsigned(127 + e) << 23);
}

// An element type, for q, new K and V and outputs, and for the products' operands.  Weights
// are exp2(score - subtracted), the subtracted number kRoom below the largest score when it is
// chosen and up to 8 more below it later.  Half precision has no weight below 2^-25, and what
// 2^-25 of the largest weight is lost of many keys adds up (128k keys 17 below the largest: 0.4 %
// of a result); made 2^7 larger, weights reach from 2^-32 to 2^15 of its 65504.
template <int TYPE>
struct Elem;
template <>
struct Elem<KVX_TYPE_HALF> {
    typedef __half T;
    static constexpr float kRoom = 7.0f;
    static __device__ __forceinline__ float load(T x) { return __half2float(x); }
    static __device__ __forceinline__ unsigned pack(float lo, float hi)
    {
        unsigned r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
};
template <>
struct Elem<KVX_TYPE_BFLOAT> {
    typedef __nv_bfloat16 T;
    static constexpr float kRoom = 0.0f;
    static __device__ __forceinline__ float load(T x) { return __bfloat162float(x); }
    static __device__ __forceinline__ unsigned pack(float lo, float hi)
    {
        unsigned r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
};

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

// Eight e2m1 codes (low half of the low byte first) as four pairs of half-precision numbers.
__device__ __forceinline__ void half8_of_e2m1(unsigned eight, unsigned (&h)[4])
{
    asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4; cvt.rn.f16x2.e2m1x2 %0, a; "
        "cvt.rn.f16x2.e2m1x2 %1, b; cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d; }"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(eight));
}

// The low two e4m3 codes as a pair of half-precision numbers.
__device__ __forceinline__ unsigned half2_of_e4m3(unsigned two)
{
    unsigned h;
    asm("{ .reg .b16 x, y; mov.b32 {x, y}, %1; cvt.rn.f16x2.e4m3x2 %0, x; }" : "=r"(h) : "r"(two));
    return h;
}

__device__ __forceinline__ unsigned mul_half2(unsigned a, unsigned b)
{
    unsigned r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// All of a kernel's dynamic shared memory; the matrix tiles in it start on 1024 bytes.
extern __shared__ __align__(1024) char attend_smem[];

__device__ __forceinline__ unsigned smem_u32(const void *p)
{
    return unsigned(__cvta_generic_to_shared(p));
}

// 16 bytes into shared memory, zeros if !valid.
__device__ __forceinline__ void cp_async16(unsigned dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}

}  // namespace
