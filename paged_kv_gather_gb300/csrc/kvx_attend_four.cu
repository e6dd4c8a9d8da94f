// kvx_attend_four.cu -- attention over a cache held in 4 bits: the kernels of few rows
// (kvx_attend_four.cuh) and of chunks (kvx_attend_tiles.cuh) for it.
#include <cuda_runtime.h>

#include "kvx_attend_plan.h"
#include "kvx_attend_four.cuh"

namespace {

template <int TYPE, int D, int NT>
Kernel few_rows(const kvx_attn_cfg &c, int64_t token_bytes, int most_parts)
{
    const FourShape f = FourShape::of(c.kv_heads, D, int(token_bytes));
    const bool plain = !(c.softcap > 0.0f) && !c.slopes;
    return {plain ? reinterpret_cast<const void *>(kvx_attend_four_kernel<TYPE, D, NT, true>)
                  : reinterpret_cast<const void *>(kvx_attend_four_kernel<TYPE, D, NT, false>),
            kFourThreads, four_ctas_per_sm(NT), four_smem<D, NT>(f), four_slot_floats<D, NT>(),
            reinterpret_cast<const void *>(kvx_attend_four_join_kernel<TYPE, D, NT>),
            32 * (most_parts > kFourManyParts ? kFourJoinWarps : kFourJoinFew), 0, f.heads,
            four_room(NT)};
}

template <int TYPE, int D>
Kernel kernel_of(const kvx_attn_cfg &c, int64_t token_bytes, int kind, int most_parts)
{
    if (kind == kRows)
        return few_rows<TYPE, D, 1>(c, token_bytes, most_parts);
    if (kind == kMoreRows)
        return few_rows<TYPE, D, 2>(c, token_bytes, most_parts);
    return {reinterpret_cast<const void *>(kvx_attend_tiles_kernel<TYPE, KVX_TYPE_FP_FOUR, D>),
            TileShape<KVX_TYPE_FP_FOUR, D>::kThreads, 1,
            size_t(TileShape<KVX_TYPE_FP_FOUR, D>::kBytes),
            TileShape<KVX_TYPE_FP_FOUR, D>::kSlotFloats,
            reinterpret_cast<const void *>(kvx_attend_join_kernel<TYPE, D>), kJoinThreads,
            kBlockRows / kJoinRows, 0, size_t(TileShape<KVX_TYPE_FP_FOUR, D>::kBytes)};
}

}  // namespace

Kernel kvx::four_kernel(const kvx_attn_cfg &c, int64_t token_bytes, int kind, int most_parts)
{
    const bool half = c.type == KVX_TYPE_HALF;
    if (c.head_dim == 64)
        return half ? kernel_of<KVX_TYPE_HALF, 64>(c, token_bytes, kind, most_parts)
                    : kernel_of<KVX_TYPE_BFLOAT, 64>(c, token_bytes, kind, most_parts);
    return half ? kernel_of<KVX_TYPE_HALF, 128>(c, token_bytes, kind, most_parts)
                : kernel_of<KVX_TYPE_BFLOAT, 128>(c, token_bytes, kind, most_parts);
}

void kvx::four_units(const kvx_attn_cfg &c, int64_t token_bytes, int *groups, int *keys)
{
    const FourShape f = FourShape::of(c.kv_heads, c.head_dim, int(token_bytes));
    *groups = f.groups;
    *keys = f.keys;
}
