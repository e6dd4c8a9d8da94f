// kvx_beams.cu -- selection of a beam search: the best continuations of every group over beams
// and vocabulary.  The checks are in kvx_cache_host.cpp, the reordering in kvx_pages.cu.
//
// The logits are read once.  A row (a beam's logits) is cut into parts that a CTA holds in
// registers: it takes the part's maximum and sum of exponentials, and its `picks` largest logits
// (equal ones by token).  Those all reach the `picks`-th largest of what 64 or 128 groups of
// threads have as their largest, and without ties hardly more than 1.4 times as many logits do: the
// CTA looks through the few threads' logits that reach it and ranks what it finds by counting.  A
// second kernel, a CTA per group, does the same with the parts' lists, by their sums in 64 bits.
// Where ties make candidates too many for a list (a row of one value, parts of one finite mask
// value), the largest are taken one after the other, which takes a part several us for each: 64
// groups of 8 beams with -1e9 for all but 1000 tokens of 128k, 16 picks, 613 us, with -infinity 37.
//
// Measured: 64 groups of 8 beams over 128k bf16 logits (a tenth of the beams done) 43 us, 118 MB:
// parts 35 (3.4 TB/s, issuing in 57 % of the cycles, DRAM 42 %: no unit's limit but the chain
// load, maximum, bar, sum, candidates, with a barrier after each), merge 7 (half of it the 64-bit
// pipe).  One group of 4 beams over 32k 6.8 us, two launches and their chains.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvx_attend.cuh"
#include "kvx_ctx.h"

namespace {

const int kSelThreads = 256;
const int kSelWarps = kSelThreads / 32;
const int kSelGroups = 64;     // of threads of the merge, KVX_MAX_PICKS at least
const int kMergeList = 512;    // continuations that are ranked, before ties are looked into
const int kMaxParts = 32;      // of a row: a lane each when they are merged
const int kMergeWarps = KVX_MAX_BEAMS / 2;
const int kMergeThreads = 32 * kMergeWarps;
static_assert(kMergeList == kMergeThreads, "a candidate per thread fits the list");

struct PartStats {
    float sum, more;  // of exp(logit - max), in two numbers
    float max, pad;
};

struct Select {
    const char *logits;
    int64_t stride;          // bytes from beam to beam
    const float *scores;
    const uint8_t *done;
    int32_t *parents, *tokens;
    float *out_scores;
    PartStats *stats;        // [beams][parts]
    uint64_t *keys;          // [beams][parts][picks], falling; 0: none
    int32_t n_groups, width, vocab, picks, parts, done_token;
};

template <int TYPE>
struct Logit {
    typedef typename Elem<TYPE>::T T;
    static __device__ __forceinline__ float load(T x) { return Elem<TYPE>::load(x); }
    static __device__ __forceinline__ T store(float x) { return T(x); }
    static __device__ __forceinline__ float larger(unsigned pair)
    {
        const T *x = reinterpret_cast<const T *>(&pair);
        return fmaxf(load(x[0]), load(x[1]));
    }
};
template <>
struct Logit<KVX_TYPE_FLOAT> {
    typedef float T;
    static __device__ __forceinline__ float load(float x) { return x; }
    static __device__ __forceinline__ float store(float x) { return x; }
    static __device__ __forceinline__ float larger(unsigned one) { return __uint_as_float(one); }
};

// Unsigned numbers in the order of floats; larger than 0 for all but -NaN.
__device__ __forceinline__ unsigned order_of(float x)
{
    const unsigned b = __float_as_uint(x);
    return b >> 31 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float float_of(unsigned order)
{
    return __uint_as_float(order >> 31 ? order & 0x7fffffffu : ~order);
}

// Keys fall with the logit (-0 is 0), then with the token.
__device__ __forceinline__ uint64_t key_of(float x, int token)
{
    return uint64_t(order_of(x + 0.0f)) << 32 | unsigned(~token);
}

// What continues a beam: 0 nothing (not where its score is NaN either), 1 its logits, 2 itself.
// Both are asked for at once.
__device__ __forceinline__ int kind_of(const Select &a, int beam)
{
    const float score = __ldcg(a.scores + beam);
    const int done = a.done ? __ldcg(a.done + beam) : 0;
    return !(score > -INFINITY) ? 0 : done ? 2 : 1;
}

// The larger of each of two logits, and the largest of a unit of 16 bytes; NaN is passed over.
template <int TYPE>
__device__ __forceinline__ unsigned max_pair(unsigned a, unsigned b)
{
    unsigned r;
    if (TYPE == KVX_TYPE_HALF)
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else if (TYPE == KVX_TYPE_BFLOAT)
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        r = __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    return r;
}

template <int TYPE>
__device__ __forceinline__ unsigned max_unit(const uint4 &u)
{
    return max_pair<TYPE>(max_pair<TYPE>(u.x, u.y), max_pair<TYPE>(u.z, u.w));
}

// The sum over a warp of what hi + lo holds, to about 2^-45 of it: 64-bit additions are slow here.
__device__ __forceinline__ float2 warp_sum(float hi, float lo)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, hi, d);
        lo += __shfl_xor_sync(0xffffffffu, lo, d);
        const float s = hi + other, part = s - hi;  // and what that sum is rounded by
        lo += (hi - (s - part)) + (other - part);
        hi = s;
    }
    return make_float2(hi, lo);
}

// A warp's sum of numbers in [0, 64.1] as integers, which are added in one operation each and in
// any order: in 2^-15, and what that leaves in 2^-38.
__device__ __forceinline__ int2 sum_of_warp(float x)
{
    constexpr float kUnit = 384.0f, kRest = 1.5f / 32768;  // numbers near these are that far apart
    const float whole = x + kUnit, rest = x - (whole - kUnit) + kRest;
    return make_int2(__reduce_add_sync(0xffffffffu, __float_as_int(whole) - __float_as_int(kUnit)),
                     __reduce_add_sync(0xffffffffu, __float_as_int(rest) - __float_as_int(kRest)));
}

template <int TYPE, int EACH, int GROUPS>
__global__ void __launch_bounds__(kSelThreads, EACH * sizeof(typename Logit<TYPE>::T) > 128 ? 2 : 4)
kvx_select_parts_kernel(const Select a)
{
    typedef Logit<TYPE> L;
    typedef typename L::T T;
    constexpr int kVec = 16 / sizeof(T), kVecs = EACH / kVec;
    constexpr int kPer = 4 / sizeof(T);   // logits of a word
    constexpr int kWords = EACH / kPer;  // words of a thread
    // Threads that have candidates, and candidates, at most, before ties are looked into.  Where
    // few tokens are left, or there are few, all of them may be candidates: those of fewer groups
    // than there are picks, eight to a thread.
    constexpr int kRows = GROUPS == 64 ? 96 : 128, kList = GROUPS == 64 ? 512 : 1024;
    __shared__ uint64_t list[kList];
    __shared__ uint4 rows[kRows][kVecs];
    __shared__ int owner[kRows];
    __shared__ uint4 tops[GROUPS / 4], maxima[kSelWarps / 4];  // order_of, of groups and warps
    __shared__ int2 sums[kSelWarps];
    __shared__ unsigned reach;  // the largest that `picks` of `tops` reach
    __shared__ int found, reached, odd;
    const int beam = blockIdx.x / a.parts, part = blockIdx.x - beam * a.parts;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_earlier_work();
    if (kind_of(a, beam) != 1)
        return;

    // 16-byte units of the row, the first and last of them partly outside it.
    const char *row = a.logits + beam * a.stride;
    const int skew = int((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const uint4 *units = reinterpret_cast<const uint4 *>(row - skew * sizeof(T));
    auto token_of = [&](int i) {  // of the i-th unit's first logit
        return ((part * kVecs + i) * kSelThreads + int(threadIdx.x)) * kVec - skew;
    };
    uint4 u[kVecs];
    const int first = part * kVecs * kSelThreads * kVec - skew;  // token of the part
    if (first >= 0 && first + kVecs * kSelThreads * kVec <= a.vocab) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            u[i] = __ldcs(units + (part * kVecs + i) * kSelThreads + threadIdx.x);
    } else {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int t = token_of(i);
            if (t >= 0 && t + kVec <= a.vocab) {
                u[i] = __ldcs(units + (t + skew) / kVec);
            } else {
                T *e = reinterpret_cast<T *>(&u[i]);
#pragma unroll
                for (int k = 0; k < kVec; ++k)
                    e[k] = t + k >= 0 && t + k < a.vocab ? reinterpret_cast<const T *>(row)[t + k]
                                                         : L::store(-INFINITY);
            }
        }
    }
    auto logit = [&](int i) {
        return L::load(reinterpret_cast<const T *>(&u[i / kVec])[i % kVec]);
    };

    float top, m, bar;
    constexpr int kLanes = kSelThreads / GROUPS;  // of a group
    for (bool again = false;; again = true) {
        unsigned pair = u[0].x;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            pair = max_pair<TYPE>(pair, max_unit<TYPE>(u[i]));
        top = L::larger(pair);
        top = top > -INFINITY ? top : -INFINITY;  // nor NaN, where there is nothing else
        float group = top;
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1)
            group = fmaxf(group, __shfl_xor_sync(0xffffffffu, group, d));
        const int mine = threadIdx.x / kLanes, sub = threadIdx.x % kLanes;
        const unsigned own = order_of(group);
        const unsigned most = __reduce_max_sync(0xffffffffu, own);
        if (sub == 0)
            reinterpret_cast<unsigned *>(tops)[mine] = own;
        if (lane == 0)
            reinterpret_cast<unsigned *>(maxima)[warp] = most;
        if (threadIdx.x == 0)
            found = reached = odd = 0, reach = 0;
        __syncthreads();
        // The largest of all, and how many groups' largest reach the own, by its threads together.
        unsigned all = 0;
#pragma unroll
        for (int k = 0; k < kSelWarps / 4; ++k) {
            const uint4 f = maxima[k];
            all = max(all, max(max(f.x, f.y), max(f.z, f.w)));
        }
        m = float_of(all);
        int rank = 0;
#pragma unroll
        for (int k = 0; k < GROUPS / 4 / kLanes; ++k) {
            const uint4 f = tops[k * kLanes + sub];
            rank += f.x >= own;
            rank += f.y >= own;
            rank += f.z >= own;
            rank += f.w >= own;
        }
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1)
            rank += __shfl_xor_sync(0xffffffffu, rank, d);
        const unsigned reaches = __reduce_max_sync(0xffffffffu, rank >= a.picks ? own : 0u);
        if (lane == 0)
            atomicMax(&reach, reaches);
        // A thread without a logit has no part in the sum (and -infinity less itself is NaN).
        float sum = 0.0f;
        if (top > -INFINITY) {
            // The exponents x log2 e - round(m log2 e) come out of one operation; what the
            // rounding moves them by is the same for all and goes into the sum at the end.  A
            // part of mask values alone may have them as large as the type goes: past 2^30 logits
            // are alike or at least 64 apart, and 2^(x - m) does as well, without overflow.
            const float unit = fabsf(m) > 0x1p30f ? 1.0f : kLog2e;
            const float base = m * unit, off = fmaf(m, unit, -base);
            const uint64_t less = pair_of(-base, -base), log2e = pair_of(unit, unit);
            uint64_t both[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < EACH; i += 2) {
                const float2 x = halves_of(fma_pair(pair_of(logit(i), logit(i + 1)), log2e, less));
                both[i >> 1 & 1] = add_pair(both[i >> 1 & 1], pair_of(exp2_(x.x), exp2_(x.y)));
            }
            const float2 x = halves_of(add_pair(both[0], both[1]));
            // The rounding, 64 at most, to first order where the second is below 2^-25.
            sum = (x.x + x.y) * (fabsf(off) < 0x1p-12f ? fmaf(off, -kLn2, 1.0f) : exp2f(-off));
        }
        // NaN, or +infinity, which the sum is NaN with too: taken out, once.
        if (!again && !(sum < INFINITY))
            odd = 1;
        const int2 s = sum_of_warp(sum);
        if (lane == 0)
            sums[warp] = s;
        __syncthreads();
        bar = float_of(reach);
        if (again || !odd)
            break;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            if (!(logit(i) < INFINITY))
                reinterpret_cast<T *>(&u[i / kVec])[i % kVec] = L::store(-INFINITY);
    }

    // Candidates: the logits that reach the bar.  The few threads that have some put all their
    // logits where the CTA looks through them together: each on its own, one divergent pass per
    // warp, took half of the kernel's time.
    if (top >= bar && top > -INFINITY) {
        const int at = atomicAdd(&reached, 1);
        if (at < kRows) {
            owner[at] = threadIdx.x;
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                rows[at][i] = u[i];
        }
    }
    __syncthreads();
    const int all_rows = reached;
    for (int i = threadIdx.x; i < min(all_rows, kRows) * kWords; i += kSelThreads) {
        const int r = i / kWords, w = i % kWords;
        const unsigned word = reinterpret_cast<const unsigned *>(rows[r])[w];
        if (L::larger(word) < bar)
            continue;
        const int token = ((part * kVecs + w / 4) * kSelThreads + owner[r]) * kVec - skew +
                          w % 4 * kPer;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const float x = L::load(reinterpret_cast<const T *>(&word)[k]);
            if (x >= bar && x > -INFINITY) {
                const int at = atomicAdd(&found, 1);
                if (at < kList)
                    list[at] = key_of(x, token + k);
            }
        }
    }
    __syncthreads();
    const int n = all_rows > kRows ? kList + 1 : found;
    uint64_t *out = a.keys + (int64_t(beam) * a.parts + part) * a.picks;
    constexpr int kRanked = 64, kSpread = kSelThreads / kRanked;  // candidates, threads to each
    if (n <= kRanked) {  // as usual: the other warps are done
        if (threadIdx.x < n) {
            const uint64_t key = list[threadIdx.x];
            int rank = 0;
#pragma unroll 4
            for (int k = 0; k < n; ++k)
                rank += list[k] > key;
            if (rank < a.picks)
                out[rank] = key;
        } else if (threadIdx.x < a.picks) {
            out[threadIdx.x] = 0;
        }
    } else if (n <= kList) {
        for (int i = threadIdx.x / kSpread; i < (n + kRanked - 1) / kRanked * kRanked;
             i += kRanked) {
            const uint64_t key = i < n ? list[i] : 0;
            int rank = 0;
            for (int k = threadIdx.x % kSpread; k < n; k += kSpread)
                rank += list[k] > key;
#pragma unroll
            for (int d = 1; d < kSpread; d <<= 1)
                rank += __shfl_xor_sync(0xffffffffu, rank, d);
            if (i < n && rank < a.picks && threadIdx.x % kSpread == 0)
                out[rank] = key;
        }
    } else {
        // Ties make them too many: one after the other, the largest of what the threads have left.
        uint64_t last = ~0ull;  // of this thread's, the one taken last
        uint64_t next = ~0ull;
        for (int r = 0; r < a.picks; ++r) {
            if (next == last) {
                // Read again: with registers of its own this would cost the usual case some.
                next = 0;
#pragma unroll 1
                for (int i = 0; i < EACH; ++i) {
                    const int token = token_of(i / kVec) + i % kVec;
                    if (token < 0 || token >= a.vocab)
                        continue;
                    const float x = L::load(reinterpret_cast<const T *>(row)[token]);
                    const uint64_t key = key_of(x, token);
                    if (x >= bar && x > -INFINITY && x < INFINITY && key < last && key > next)
                        next = key;
                }
            }
            const unsigned hi = __reduce_max_sync(0xffffffffu, unsigned(next >> 32));
            const unsigned lo = __reduce_max_sync(
                0xffffffffu, unsigned(next >> 32) == hi ? unsigned(next) : 0u);
            if (lane == 0)
                list[warp] = uint64_t(hi) << 32 | lo;
            __syncthreads();
            uint64_t best = 0;
#pragma unroll
            for (int i = 0; i < kSelWarps; ++i)
                best = max(best, list[i]);
            if (next == best)
                last = best;
            if (threadIdx.x == 0)
                out[r] = best;
            __syncthreads();
        }
    }
    if (warp == 0) {
        const int2 s = lane < kSelWarps ? sums[lane] : make_int2(0, 0);
        const int whole = __reduce_add_sync(0xffffffffu, s.x);  // up to 2^29
        const int rest = __reduce_add_sync(0xffffffffu, s.y);
        if (lane == 0)
            a.stats[int64_t(beam) * a.parts + part] = {
                float(whole & ~31) * 0x1p-15f,
                fmaf(float(rest), 0x1p-38f, float(whole & 31) * 0x1p-15f), m, 0.0f};
    }
}

// Unsigned numbers in the order of doubles, and back.
__device__ __forceinline__ uint64_t order_of(double x)
{
    const uint64_t b = uint64_t(__double_as_longlong(x));
    return b >> 63 ? ~b : b | 1ull << 63;
}

__device__ __forceinline__ double double_of(uint64_t order)
{
    return __longlong_as_double(int64_t(order >> 63 ? order & ~(1ull << 63) : ~order));
}

// log s to about 1e-9, for normal s >= 1: s = 2^e f with f in [3/4, 3/2), and
// log f = 2 artanh z by its power series, z = (f - 1) / (f + 1) with its rounding carried along.
// 64-bit arithmetic is slow here: a library logarithm per beam was a third of the merge.
__device__ __forceinline__ double log_of(double s)
{
    const uint64_t b = uint64_t(__double_as_longlong(s));
    const bool half = (b >> 51 & 1) != 0;  // f of the mantissa is 3/2 or more
    const int e = int(b >> 52) - 1023 + half;
    const double f = __longlong_as_double(int64_t((b & 0xfffffffffffffull) |
                                                  uint64_t(1023 - half) << 52));
    const double num = f - 1.0, den = f + 1.0;
    const float n0 = float(num), n1 = float(num - n0), d0 = float(den), d1 = float(den - d0);
    const float z = n0 / d0, z1 = (fmaf(-z, d0, n0) + (n1 - z * d1)) / d0, y = z * z;
    float p = 1.0f / 13;
    p = fmaf(p, y, 1.0f / 11);
    p = fmaf(p, y, 1.0f / 9);
    p = fmaf(p, y, 1.0f / 7);
    p = fmaf(p, y, 1.0f / 5);
    p = fmaf(p, y, 1.0f / 3);
    return e * 0.69314718055994530942 + (2.0 * z + double(2.0f * fmaf(z * y, p, z1)));
}

struct Continuation {
    uint64_t sum;  // order_of the sum
    int32_t token, beam;
};

// Norms first, a warp per beam.  A continuation's sum is (logit - m) + (score - log s) with the
// beam's largest logit m and s the sum of exp(logit - m): m + log s in one number would round
// log s away where m is a large mask value, and a beam of mask values alone has nothing else.
// Then the largest `picks` sums of all the beams' lists in the way of the parts' kernel: those that
// reach the `picks`-th largest of what 64 groups of threads have, ranked by counting.
//
// KEPT: candidates of a thread that stay in registers, and are on their way before the norms: all
// of them up to 4 (one group of 8 beams over 500k with 8 picks, 1984 candidates, 13.1 us; 14.4 with
// 2 kept; with 4 that are not there, of 1024, 10.9 instead of 10.5).  With one each the list holds
// all of them, and they stay in order, in as few warps as there can be, because their sums are
// 64-bit arithmetic.  More of them are spread: a thread's k-th is one of 64 in a row, another place
// in every row.  Lists are sorted, and a group of threads that had the same ranks of all of them
// would have a largest far below what it should be (16 beams, 32 picks: 380 candidates reached such
// a bar, 40 reach this one; 32 beams, 64 picks: 5000 and 180; one group of 16 beams over 500k with
// 32 picks 448 us and 60).  Rows turn by 64 / the golden ratio, which spreads the places that a
// group has had evenly, however many rows.
template <int KEPT>
__global__ void __launch_bounds__(kMergeThreads)
kvx_select_merge_kernel(const Select a)
{
    __shared__ Continuation list[kMergeList];
    __shared__ uint64_t tops[kSelGroups], bar;
    __shared__ double bases[KVX_MAX_BEAMS];   // score - log s, of a beam that is done the score
    __shared__ float largest[KVX_MAX_BEAMS];  // m
    __shared__ int state[KVX_MAX_BEAMS];  // 0: no continuations, 1: lists, 2: itself
    __shared__ int found;
    constexpr int kLanes = kMergeThreads / kSelGroups;
    const int group = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_earlier_work();
    // Candidate i: of beam b, key i - b per_beam of its parts' lists.
    constexpr bool kFew = KEPT == 1;
    constexpr int kTurn = 39;
    const int mine = threadIdx.x / kLanes, sub = threadIdx.x % kLanes;
    const int per_beam = a.parts * a.picks, all = a.width * per_beam;
    const int rounds = kFew ? 1 : (all + kMergeThreads - 1) / kMergeThreads;
    auto candidate = [&](int k) {
        const int r = k * kLanes + sub;
        return kFew ? int(threadIdx.x)
                   : r * kSelGroups + ((mine + kTurn * r) & (kSelGroups - 1));
    };
    const uint64_t *keys = a.keys + int64_t(group) * all;
    uint64_t kept[KEPT];
#pragma unroll
    for (int k = 0; k < KEPT; ++k) {
        const int i = candidate(k);
        kept[k] = i < all ? keys[i] : 0;
    }
    for (int b = warp; b < a.width; b += kMergeWarps) {
        const int beam = group * a.width + b;
        // Without logits that count there is nothing there, but it is asked for at once too.
        PartStats part = a.stats[int64_t(beam) * a.parts + min(lane, a.parts - 1)];
        const int kind = kind_of(a, beam);
        if (kind != 1 || lane >= a.parts)
            part = {0.0f, 0.0f, -INFINITY, 0.0f};
        const float m = float_of(__reduce_max_sync(0xffffffffu, order_of(part.max)));
        // exp(max - m): what the difference is rounded by goes in to first order.
        const double away = part.sum > 0.0f ? double(part.max) - m : 0.0;
        const float near = float(away);
        const double scaled = near < -200.0f ? 0.0  // and what follows may be 0 times infinity
                                             : (double(part.sum) + part.more) *
                                                   (double(expf(near)) * (1.0 + (away - near)));
        const float hi = float(scaled);
        const float2 s = warp_sum(hi, float(scaled - hi));
        if (lane == 0) {
            state[b] = kind;
            largest[b] = m;
            bases[b] = a.scores[beam] - (kind == 1 ? log_of(double(s.x) + s.y) : 0.0);
        }
    }
    if (threadIdx.x == 0)
        found = 0;
    __syncthreads();

    // The sum of candidate i with this key, as an ordered number; 0: there is none.
    auto sum_of = [&](int i, uint64_t key, int &b, int32_t &token) -> uint64_t {
        b = i / per_beam;
        if (state[b] == 2) {
            token = a.done_token;
            return i == b * per_beam ? order_of(bases[b]) : 0;
        }
        token = int32_t(~unsigned(key));
        return state[b] && key
                   ? order_of(bases[b] + (double(float_of(unsigned(key >> 32))) - largest[b])) : 0;
    };
    uint64_t sums[KEPT];
    int b;
    int32_t token;
    uint64_t top = 0;
#pragma unroll
    for (int k = 0; k < KEPT; ++k) {
        const int i = candidate(k);
        sums[k] = i < all ? sum_of(i, kept[k], b, token) : 0;
        top = max(top, sums[k]);
    }
    for (int k = KEPT; k < rounds; ++k) {
        const int i = candidate(k);
        if (i < all)
            top = max(top, sum_of(i, keys[i], b, token));
    }
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1)
        top = max(top, uint64_t(__shfl_xor_sync(0xffffffffu, top, d)));
    if (sub == 0)
        tops[mine] = top;
    __syncthreads();
    int rank = 0;
#pragma unroll
    for (int k = 0; k < kSelGroups / kLanes; ++k) {
        const uint64_t other = tops[k * kLanes + sub];
        rank += other > top || (other == top && k * kLanes + sub < mine);
    }
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1)
        rank += __shfl_xor_sync(0xffffffffu, rank, d);
    if (sub == 0 && rank == a.picks - 1)
        bar = top;
    __syncthreads();
    auto take = [&](uint64_t sum, int32_t token, int b) {
        const int at = atomicAdd(&found, 1);
        if (at < kMergeList)
            list[at] = {sum, token, b};
    };
#pragma unroll
    for (int k = 0; k < KEPT; ++k)
        if (sums[k] && sums[k] >= bar) {
            sum_of(candidate(k), kept[k], b, token);
            take(sums[k], token, b);
        }
    for (int k = KEPT; k < rounds; ++k) {
        const int i = candidate(k);
        const uint64_t sum = i < all ? sum_of(i, keys[i], b, token) : 0;
        if (sum && sum >= bar)
            take(sum, token, b);
    }
    __syncthreads();
    const int64_t out = int64_t(group) * a.picks;
    auto write = [&](int r, const Continuation &c) {
        a.parents[out + r] = c.beam;
        a.tokens[out + r] = c.token;
        a.out_scores[out + r] = float(double_of(c.sum));
    };
    // Larger sums first, equal ones by beam and then by token.
    auto ahead = [](const Continuation &x, const Continuation &y) {
        return x.sum != y.sum ? x.sum > y.sum
                              : x.beam != y.beam ? x.beam < y.beam : x.token < y.token;
    };
    const int n = found;
    if (kFew || n <= kMergeList) {
        for (int i = mine; i < (n + kSelGroups - 1) / kSelGroups * kSelGroups; i += kSelGroups) {
            int r = 0;
            for (int k = sub; i < n && k < n; k += kLanes)
                r += ahead(list[k], list[i]);
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1)
                r += __shfl_xor_sync(0xffffffffu, r, d);
            if (i < n && r < a.picks && sub == 0)
                write(r, list[i]);
        }
        for (int i = n + threadIdx.x; i < a.picks; i += kMergeThreads) {
            a.parents[out + i] = 0;
            a.tokens[out + i] = -1;
            a.out_scores[out + i] = -INFINITY;
        }
        return;
    }
    // Equal sums make them too many (and at least `picks`): one after the other, the first of what
    // the threads have left.
    Continuation last = {~0ull, -1, -1}, next = last;
    bool stale = true;
    for (int r = 0; r < a.picks; ++r) {
        if (stale) {
            next = {0, 0, INT32_MAX};
            for (int i = threadIdx.x; i < all; i += kMergeThreads) {
                Continuation c;
                c.sum = sum_of(i, keys[i], c.beam, c.token);
                if (c.sum && c.sum >= bar && ahead(last, c) && ahead(c, next))
                    next = c;
            }
        }
        Continuation best = next;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const Continuation c = {__shfl_xor_sync(0xffffffffu, best.sum, d),
                                    __shfl_xor_sync(0xffffffffu, best.token, d),
                                    __shfl_xor_sync(0xffffffffu, best.beam, d)};
            if (ahead(c, best))
                best = c;
        }
        if (lane == 0)
            list[warp] = best;
        __syncthreads();
        best = list[0];
        for (int i = 1; i < kMergeWarps; ++i)
            if (ahead(list[i], best))
                best = list[i];
        stale = next.beam == best.beam && next.token == best.token && next.sum == best.sum;
        if (stale)
            last = best;
        if (threadIdx.x == 0)
            write(r, best);
        __syncthreads();
    }
}

// Logits that a thread holds: 64, so that what a part costs besides its logits (half of the
// instructions at 32) is met seldom, and the merge has few lists; 8 where even those of one group
// leave the GPU nearly empty, and a row has at most 32 parts then, a lane each in the merge.  With
// 64 and 8, one group over 32k, as many picks as beams: 4 beams of fp32 7.1 and 6.6 us, of bf16 7.1
// and 7.1, 5 7.4 and 7.5, 7 8.3 and 9.3; over 50k 1 beam 7.3 and 6.3, 3 with 6 picks 7.7 and 7.1.
// Past the rule: 8 beams over 32k with 16 picks 10.4 and 13.1, 2 groups of 4 7.3 and 6.9, 8 groups
// 7.3 and 8.3, 16 groups of 8 11.9 and 19.5.  Between 10 and 16 parts it is either, by up to 1 us.
const int kEachMost = 64, kFewParts = 16;

int each_of(const kvx_select_cfg &c)
{
    const int64_t rows = int64_t(c.n_groups) * c.width;
    const int64_t large = (c.vocab + 7 + kEachMost * kSelThreads - 1) / (kEachMost * kSelThreads);
    const int64_t small = (c.vocab + 7 + 8 * kSelThreads - 1) / (8 * kSelThreads);
    return rows * large < kFewParts && small <= kMaxParts ? 8 : kEachMost;
}

int parts_of(const kvx_select_cfg &c, int each)
{
    return (c.vocab + 7 + each * kSelThreads - 1) / (each * kSelThreads);
}

// Up to this many picks a part's threads make 64 groups, past it 128: the nearer the picks are to
// the groups, the more logits reach the bar.  With 64 of 64 it is the smallest of the groups'
// largest, 300 logits of 175 threads reach it, and they are taken one after the other; with 64 of
// 128 it is 90 logits.  64 groups of 8 beams over 128k, 64 and 128 groups: 37.5 and 40.4 us with 4
// picks, 44.5 and 45.4 with 16, 52.4 and 50.4 with 24, 60.5 and 56 with 32, 2700 and 96 with 64.
const int kFewPicks = 16;

template <int TYPE, int EACH>
const void *parts_kernel(int picks)
{
    return picks > kFewPicks
               ? reinterpret_cast<const void *>(kvx_select_parts_kernel<TYPE, EACH, 128>)
               : reinterpret_cast<const void *>(kvx_select_parts_kernel<TYPE, EACH, 64>);
}

template <int TYPE>
const void *parts_kernel(int each, int picks)
{
    return each == 8 ? parts_kernel<TYPE, 8>(picks) : parts_kernel<TYPE, kEachMost>(picks);
}

const void *merge_kernel(int candidates)  // of a group
{
    return candidates <= kMergeThreads ? reinterpret_cast<const void *>(kvx_select_merge_kernel<1>)
           : candidates <= 2 * kMergeThreads
               ? reinterpret_cast<const void *>(kvx_select_merge_kernel<2>)
               : reinterpret_cast<const void *>(kvx_select_merge_kernel<4>);
}

cudaError_t launch(const void *fn, int64_t ctas, int threads, cudaStream_t s, void **args)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(unsigned(ctas));
    lc.blockDim = dim3(unsigned(threads));
    lc.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelExC(&lc, fn, args);
}

}  // namespace

extern "C" {

kvx_status kvx_select_workspace(kvx_ctx *ctx, const kvx_select_cfg *cfg, int64_t *bytes)
{
    if (!ctx || !bytes)
        return KVX_ERR_INVALID_ARG;
    *bytes = 0;
    const kvx_status st = kvx::validate_select(cfg, ctx->err, sizeof ctx->err);
    if (st != KVX_OK)
        return st;
    *bytes = int64_t(cfg->n_groups) * cfg->width * parts_of(*cfg, each_of(*cfg)) *
             int64_t(sizeof(PartStats) + cfg->picks * sizeof(uint64_t));
    return KVX_OK;
}

kvx_status kvx_select_beams(kvx_ctx *ctx, const kvx_select_cfg *cfg, const void *logits,
                            int64_t logits_stride, const float *scores, const uint8_t *done,
                            int32_t *parents, int32_t *tokens, float *out_scores, void *workspace,
                            kvx_stream_t stream)
{
    if (!ctx)
        return KVX_ERR_INVALID_ARG;
    kvx::begin_call(ctx);
    const kvx_status st = kvx::validate_select(cfg, ctx->err, sizeof ctx->err);
    if (st != KVX_OK)
        return st;
    if (!logits || !scores || !parents || !tokens || !out_scores || !workspace)
        return kvx::set_err(ctx, KVX_ERR_INVALID_ARG, "logits, scores, parents, tokens, "
                            "out_scores or workspace is NULL");
    const int item = cfg->type == KVX_TYPE_FLOAT ? 4 : 2;
    auto bits = [](const void *p) { return reinterpret_cast<uintptr_t>(p); };
    const uintptr_t words = bits(scores) | bits(parents) | bits(tokens) | bits(out_scores);
    if (bits(logits) % item || words & 3 || bits(workspace) & 15)
        return kvx::set_err(ctx, KVX_ERR_ALIGNMENT, "logits, scores, parents, tokens or "
                            "out_scores not aligned to their elements, or the workspace not to "
                            "16 bytes");
    if (logits_stride == 0)
        logits_stride = cfg->vocab;
    if (logits_stride < cfg->vocab)
        return kvx::set_err(ctx, KVX_ERR_INVALID_ARG, "logits: stride %lld below %d elements",
                            (long long)logits_stride, cfg->vocab);
    if (out_scores == scores && cfg->picks != cfg->width)
        return kvx::set_err(ctx, KVX_ERR_INVALID_ARG, "out_scores is scores, but picks %d is not "
                            "width %d", cfg->picks, cfg->width);
    kvx::DeviceGuard guard(ctx->device);
    if (!guard.ok)
        return kvx::set_err(ctx, KVX_ERR_CUDA, "cannot make device %d current", ctx->device);
    const int each = each_of(*cfg), parts = parts_of(*cfg, each);
    const int64_t beams = int64_t(cfg->n_groups) * cfg->width;
    if (beams * parts > INT32_MAX)
        return kvx::set_err(ctx, KVX_ERR_CAPACITY, "%lld beams of %d parts", (long long)beams,
                            parts);
    Select a = {static_cast<const char *>(logits), logits_stride * item, scores, done, parents,
                tokens, out_scores, static_cast<PartStats *>(workspace),
                reinterpret_cast<uint64_t *>(static_cast<PartStats *>(workspace) + beams * parts),
                cfg->n_groups, cfg->width, cfg->vocab, cfg->picks, parts, cfg->done_token};
    void *args[] = {&a};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int picks = cfg->picks;
    const void *fn = cfg->type == KVX_TYPE_HALF     ? parts_kernel<KVX_TYPE_HALF>(each, picks)
                     : cfg->type == KVX_TYPE_BFLOAT ? parts_kernel<KVX_TYPE_BFLOAT>(each, picks)
                                                    : parts_kernel<KVX_TYPE_FLOAT>(each, picks);
    cudaError_t e = launch(fn, beams * parts, kSelThreads, s, args);
    if (e == cudaSuccess)
        e = launch(merge_kernel(cfg->width * parts * picks), cfg->n_groups, kMergeThreads, s, args);
    if (e != cudaSuccess)
        return kvx::cuda_err(ctx, e, "selection launch");
    ctx->last_items = beams;
    ctx->last_ctas = int32_t(beams * parts);
    ctx->last_threads = kSelThreads;
    return KVX_OK;
}

}  // extern "C"
