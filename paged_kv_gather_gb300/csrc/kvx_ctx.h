// kvx_ctx.h -- the context behind kvx_ctx: descriptor slots, device status word, last launch
// and error text, with the helpers every entry point that uses a context shares.
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/kvx.h"

namespace kvx {

const int kSlots = 4;

struct Slot {
    char *host = nullptr;
    char *dev = nullptr;
    cudaEvent_t done = nullptr;    // recorded on the caller's stream after the kernel
    cudaEvent_t staged = nullptr;  // recorded on the copy stream after the descriptor copy
    bool used = false;
};

}  // namespace kvx

struct kvx_ctx {
    int device = 0;
    int num_sms = 0;
    int validation = 1;
    size_t slot_bytes = 0;
    kvx::Slot slots[kvx::kSlots];
    int next = 0;
    // Descriptor copies run here, beside the caller's stream, so that a call's copy overlaps
    // the previous call's kernel instead of sitting between two kernels.
    cudaStream_t copy_stream = nullptr;
    unsigned int *status_dev = nullptr;
    unsigned int *status_host = nullptr;
    int64_t last_items = 0;
    int32_t last_ctas = 0;
    int32_t last_threads = 0;
    int64_t last_desc_bytes = 0;
    char err[512] = {0};
};

namespace kvx {

inline kvx_status set_err(kvx_ctx *ctx, kvx_status st, const char *fmt, ...)
    __attribute__((format(printf, 3, 4)));

inline kvx_status set_err(kvx_ctx *ctx, kvx_status st, const char *fmt, ...)
{
    if (ctx) {
        va_list ap;
        va_start(ap, fmt);
        vsnprintf(ctx->err, sizeof ctx->err, fmt, ap);
        va_end(ap);
    }
    return st;
}

inline kvx_status cuda_err(kvx_ctx *ctx, cudaError_t e, const char *what)
{
    return set_err(ctx, KVX_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Copy a call's packed descriptors into its slot on the context's copy stream (zeroing
// `zero_bytes` at `zero_off` after them), and make the caller's stream wait for that.
// settle: the host waits for the copy first (a few microseconds), so that the caller's
// stream waits on an event that has already completed.  An overlapped launch needs that: a
// wait on a copy still in flight keeps it from starting before the kernel ahead of it ends,
// where a completed one does not.
inline cudaError_t stage(kvx_ctx *ctx, Slot &slot, size_t bytes, size_t zero_off, size_t zero_bytes,
                  cudaStream_t s, bool settle = false)
{
    cudaError_t e = cudaMemcpyAsync(slot.dev, slot.host, bytes, cudaMemcpyHostToDevice,
                                    ctx->copy_stream);
    if (e == cudaSuccess && zero_bytes)
        e = cudaMemsetAsync(slot.dev + zero_off, 0, zero_bytes, ctx->copy_stream);
    if (e == cudaSuccess)
        e = cudaEventRecord(slot.staged, ctx->copy_stream);
    if (e == cudaSuccess && settle)
        e = cudaEventSynchronize(slot.staged);
    if (e == cudaSuccess)
        e = cudaStreamWaitEvent(s, slot.staged, 0);
    return e;
}

// Keeps ctx->device current for the duration of a call and restores the caller's device.
struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) {
            prev = -1;
            ok = false;
            return;
        }
        if (prev != dev && cudaSetDevice(dev) != cudaSuccess)
            ok = false;
    }
    ~DeviceGuard()
    {
        int cur;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev)
            cudaSetDevice(prev);
    }
};

// Every call starts with an empty last-launch record, so a call that fails or moves
// nothing reports zeros.
inline void begin_call(kvx_ctx *ctx)
{
    ctx->last_items = 0;
    ctx->last_ctas = 0;
    ctx->last_threads = 0;
    ctx->last_desc_bytes = 0;
}

// Allow the page upkeep kernels the shared memory of the largest pool, on the current device:
// once, for every call of every context after it, so that no call lowers it under another
// thread's launch.
cudaError_t prepare_upkeep();

// The context's next descriptor slot, once the launch that last used it has finished.
inline kvx_status acquire_slot(kvx_ctx *ctx, size_t bytes, Slot **out)
{
    if (bytes > ctx->slot_bytes)
        return set_err(ctx, KVX_ERR_CAPACITY,
                       "descriptors need %zu bytes, the context holds %zu per call; create it "
                       "with a larger max_descriptor_bytes", bytes, ctx->slot_bytes);
    Slot &slot = ctx->slots[ctx->next];
    if (slot.used) {
        cudaError_t e = cudaEventSynchronize(slot.done);
        if (e != cudaSuccess)
            return cuda_err(ctx, e, "waiting for a descriptor buffer");
    }
    *out = &slot;
    return KVX_OK;
}

// After a launch: the slot stays busy until `s` passes this point; record the launch.
inline kvx_status finish_call(kvx_ctx *ctx, Slot &slot, cudaStream_t s, int64_t items, int64_t ctas,
                       int threads, size_t desc_bytes)
{
    cudaError_t e = cudaEventRecord(slot.done, s);
    if (e != cudaSuccess)
        return cuda_err(ctx, e, "event record");
    slot.used = true;
    ctx->next = (ctx->next + 1) % kSlots;
    ctx->last_items = items;
    ctx->last_ctas = int32_t(ctas);
    ctx->last_threads = threads;
    ctx->last_desc_bytes = int64_t(desc_bytes);
    return KVX_OK;
}

}  // namespace kvx
