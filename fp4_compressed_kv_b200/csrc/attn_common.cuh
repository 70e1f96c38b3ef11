// attn_common.cuh -- what the tensor-core attention kernels over 576-channel
// entries (attn_t128.cu, attn_tree_t128.cu) share: TMA loads of query and key
// rows and their tensor maps.
#pragma once

#include <cuda.h>

#include "kvc_internal.cuh"
#include "tc05_common.cuh"

namespace kvc {

// Tensor map of a bf16 tensor [rows][576] (attn_t128.cu); false if it cannot
// be made.
bool encode_rows576(CUtensorMap* m, const void* base, unsigned long long rows, unsigned box_rows);

namespace tc {

// TMA loads (non-multicast, into this CTA's shared memory)
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

}  // namespace tc
}  // namespace kvc
