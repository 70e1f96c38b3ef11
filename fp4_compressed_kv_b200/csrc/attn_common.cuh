// attn_common.cuh -- what the tensor-core attention kernels over 576-channel
// entries (attn_t128.cu, attn_tree.cu) share: TMA loads of query and key rows,
// their tensor maps, and the query tile's conversion to f16.
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
// The query tile of a record CTA, landed by TMA as bf16, converted in place to
// f16 with a per-head power of two that puts the row maximum in [2^14,
// 2^15); the head's softmax multiplier qs[h] absorbs it.  Thread t: head t/4,
// channels [144 (t%4), +144) as 18 16-byte pieces (the same swizzled
// positions the TMA wrote; a warp's accesses take the minimum 4 wavefronts).
__device__ __forceinline__ void convert_q_f16(uint32_t* status, float sm_log2, uint32_t sQ,
                                              uint32_t q_atom, float* qs, int tid) {
    const int h = tid >> 2, qq = tid & 3;
    uint4 v[18];
#pragma unroll
    for (int i = 0; i < 18; ++i) {
        const int c16 = 18 * qq + i;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                     : "r"(sQ + (c16 >> 3) * q_atom + swz(h, c16 & 7)));
    }
    uint32_t amax = 0;  // max |x| as fp32 bits (integer order = float order)
#pragma unroll
    for (int i = 0; i < 18; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            amax = max(amax, (w[k] << 16) & 0x7FFFFFFFu);
            amax = max(amax, w[k] & 0x7FFF0000u);
        }
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    int k = 0;
    if (amax >= 0x7F800000u) {
        if (qq == 0) set_status(status, KVC_DEV_NONFINITE);
    } else if (amax != 0) {
        const int e = (int)(amax >> 23) - 127;  // floor(log2 amax) for normal values
        k = min(max(e - 14, -60), 113);
    }
    const float mul = __uint_as_float((uint32_t)(127 - k) << 23);
    if (qq == 0) qs[h] = sm_log2 * __uint_as_float((uint32_t)(127 + k) << 23);
#pragma unroll
    for (int i = 0; i < 18; ++i) {
        const int c16 = 18 * qq + i;
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = pack_f16(__uint_as_float(w[j] << 16) * mul,
                            __uint_as_float(w[j] & 0xFFFF0000u) * mul);
        sts128(sQ + (c16 >> 3) * q_atom + swz(h, c16 & 7), o[0], o[1], o[2], o[3]);
    }
}

}  // namespace tc
}  // namespace kvc
