// attn_tree_t128.cu -- attention of a tree of drafted tokens on the
// 5th-generation tensor cores: 576-channel entries (512 latent + 64 RoPE),
// bf16 queries, a multiple of 16 heads.
//
// Method: "DeepSeek V1 到 V4.1-Flash，单 token 的 global KV 如何从 389,000 B
// 压缩到 890 B的？" (acejoy.com) part 3 breakthrough 2 and 4, as in attn_tree.cu
// (the mathematics) and attn_t128.cu (the products: keys are the MMA's M
// dimension, 128 keys against up to 64 heads; S^T = K Q^T and O^T += V^T P^T
// in tensor memory).  What differs from the single-token kernel:
//
//  * A node's keys are its raw rows (window rows and the drafted rows of its
//    path, gathered by 16-byte asynchronous copies) and then its records, in
//    chunks of 128.  Raw chunks run with bf16 operands against the query rows
//    as they landed; the query tile is then turned into f16 in place and the
//    record chunks run in f16, where every dequantised entry is exact.  Both
//    kinds add into the same fp32 accumulators.
//  * One K tile of 147 KB is all that fits beside the queries, so overlap is
//    made inside it: its latent channels are four pairs of 64-channel atoms,
//    and the PV products of channels 128 p ... are the only ones that read pair
//    p.  Their commit frees it for the next chunk's values while the other
//    products run, and the next chunk's QK starts on the first two pairs as
//    soon as they are filled.  Roles:
//      warps 0-7   softmax (thread = key, half of the heads each) and output
//      warps 8-15  loads: the next chunk's records are in registers while
//                  this one's are converted and stored; two groups of four
//                  warps take pairs 0, 2 and 1, 3, so that one's fences and
//                  waits lie under the other's stores (the stores to shared
//                  memory, 147 KB a chunk at 75 B a clock beside the
//                  products' reads, bound this part)
//      warp 16     issues the products and the queries' TMA
//      warp 17     walks the next node's path through the parents and asks
//                  for its selected records and queries into L2
//    so the tensor pipe waits only for the softmax of the chunk it works on.
//  * With many nodes a CTA takes node after node (the next node's queries,
//    path and records arrive while this one's last products run); with few,
//    the CTAs of a cluster split one node's chunks, push their partial sums
//    to the owners of the heads over distributed shared memory, and each
//    owner joins its heads' rows in split order.
//
// Bound: what one K tile serialises, at a clock that the load holds at 1.8 GHz.
// 32 x 8 nodes of 128 + 512 keys, two nodes a CTA: 84.5 K clocks, 47 us (52.5
// with a cold L2).  A record chunk takes 6.5 K of them: 1.8 softmax between QK
// and PV, 1.8 PV, 2.8 QK and the stores it waits for (a product is issued in 20
// clocks and takes 48, 60 with waits and commits: 4.1 K for the 68 of a chunk
// with nothing else on the multiprocessor; each reads 6 KB of operands); a
// node's raw chunk takes 8, its end and the next one's start 11.  The last nodes
// leave 40 of 148 multiprocessors idle.  Every variant spills 52 to 104 bytes a
// thread (96 registers at launch); in which role that costs time is not
// measured.
//
// Every wait on an mbarrier is bounded and no other barrier is used inside
// the roles; on expiry a role sets KVC_DEV_TIMEOUT and leaves, the others
// follow when their own waits expire, products and copies in flight get a last
// bounded wait, the tensor memory is freed.
#include <algorithm>
#include <cuda.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "kvc_internal.cuh"
#include "tc05_common.cuh"

namespace kvc {
namespace tree {

using namespace tc;

constexpr int D = 576, DV = 512, CK = 128, NATOM = 9;
constexpr int SOFT_WARPS = 8, LOAD_WARPS = 8, MMA_WARP = 16, PATH_WARP = 17;
constexpr int NT = 20 * 32;  // (whole warpgroups: registers are shared out by them)
constexpr uint32_t K_ATOM = CK * 128;  // 128 rows x 128 B
constexpr uint32_t OFF_Q = 0;
constexpr uint32_t OFF_K = NATOM * 64 * 128;            // 73,728
constexpr uint32_t OFF_P = OFF_K + 8 * K_ATOM;          // the RoPE atom, P^T after QK
constexpr uint32_t OFF_MISC = OFF_K + NATOM * K_ATOM;   // 221,184
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t S_COL = 0, O_COL = 256;
// A head's reference is put kTop (log2 units) below its largest logit and moved
// when one passes it by more than kMost: weights go up to 2^15, so that f16
// still has full precision for those 2^-21 of the largest (2^-32 of it below).
constexpr float kTop = 7.0f, kMost = 15.0f;
constexpr float kLn2 = 0.6931471805599453f;

struct Item {  // what the roles know of one node
    int c0, c1;     // this CTA's chunks: raw ones below nraw, then records
    int nraw;       // raw chunks
    int raw, skip;  // raw keys, and older ones out of the window
    int wl, depth, n;
};

struct Misc {
    float qs[2][64];               // softmax multiplier of the f16 queries, by item parity
    float wmax[2][2][4][32];       // chunk maxima: [parity][head half][quadrant][head]
    alignas(16) int over[2][2][4];  // a weight passes 2^kMost: [chunk parity][head half][quadrant]
    float4 sm[SOFT_WARPS][16];     // each softmax warp's multipliers and -references, two heads
    float fac[SOFT_WARPS][32];     // each softmax warp's rescale factors
    float lsum[2][4][32];          // sums of weights: [head half][quadrant][head]
    unsigned char valid[2][CK];    // keys of the chunk that count, by chunk parity
    short parents[kMaxTreeNodes];  // path warp's
    unsigned char up[2][kMaxTreeNodes];  // ancestors k steps up, by item parity
    Item item[2];
    uint64_t bars[22];
    uint32_t tmem;
    int failed;
    float ml[72 * 2];              // exchange: (m, l) of [split][head]
    float wts[72];                 // exchange: weights [head][split]
    uint32_t row_at[64], ml_at[64];  // exchange: owners' addresses
    float inv[64];
};
constexpr uint32_t SMEM_BYTES = OFF_MISC + sizeof(Misc) + 1024;  // + alignment slack
static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");

enum {
    B_FULL = 0,   // [2] pairs 0 and 1, the rest of the chunk is in place (8 warps)
    B_FREE = 2,   // [3] PV products of pair 0, pair 1, all pairs are done (commit)
    B_S = 5,      // QK done (commit)
    B_P = 6,      // P^T is in place (8 warps)
    B_Q = 7,      // query rows landed (TMA)
    B_Q16 = 8,    // queries in f16 (8 warps)
    B_MAX = 9,    // [2] chunk maxima of a head half (4 warps)
    B_INFO = 11,  // [2] item of that parity published
    B_ITEM = 13,  // [2] item of that parity finished by everyone (17 warps)
    B_SUM = 15,   // [2] sums of weights of a head half (4 warps)
    B_OVER = 17,  // [2] checks of a head half (4 warps)
    B_REDO = 19,  // [2] P^T of a head half is in place after all (4 warps)
    B_END = 21,
    N_BARS = 22
};

// A warpgroup's registers a thread.
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// A whole warp's bounded wait (tc::mbar_wait is a thread's): its lanes leave
// with one answer, by branches that the compiler knows to be warp-uniform, and
// each try may suspend the warp for up to 20 us.
__device__ __forceinline__ bool mbar_warp_wait(uint32_t addr, uint32_t parity, uint64_t limit_ns) {
    if (limit_ns == 0) return __all_sync(0xffffffffu, mbar_wait(addr, parity, 0));
    uint64_t t0 = 0;
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(addr), "r"(parity), "r"(20000u)
            : "memory");
        if (__all_sync(0xffffffffu, ok)) return true;
        const uint64_t now = global_ns();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, now - t0 > limit_ns)) return false;
    }
}
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(y) : "f"(x));
    return y;
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[N]) {
    if constexpr (N == 8) tmem_ld8(addr, r);
    else if constexpr (N == 16) tmem_ld16(addr, r);
    else tmem_ld32(addr, r);
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[N]) {
    if constexpr (N == 32) {
        tmem_st32(addr, r);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 8)
            asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(
                             addr + i),
                         "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]),
                         "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
                         : "memory");
        asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
    }
}
// One lane of a converged warp.  The product warp runs as a whole and elects a
// lane around each block of products: with warp-uniform operands a product is
// issued in 20 clocks, where one thread's own branch takes 47 to 68 and the
// products themselves 48.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc));
}
// (a, b) <- (a, b) * (k.x, k.y) + (k.z, k.w)
__device__ __forceinline__ void fma2(uint32_t& a, uint32_t& b, const float4& k) {
    asm("{\n\t.reg .b64 x, m, c;\n\t"
        "mov.b64 x, {%0, %1};\n\tmov.b64 m, {%2, %3};\n\tmov.b64 c, {%4, %5};\n\t"
        "fma.rn.f32x2 x, x, m, c;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+r"(a), "+r"(b)
        : "f"(k.x), "f"(k.y), "f"(k.z), "f"(k.w));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p));
}
// 16 bytes to shared memory, asynchronously; zeros without a source row.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
// Sums over a warp's lanes of N values each: lane l gets that of value l % N.
template <int N>
__device__ __forceinline__ float lane_sums(float (&v)[N], int lane) {
#pragma unroll
    for (int o = 16; o >= N; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
#pragma unroll
    for (int o = N / 2; o >= 1; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = lane & o ? v[i] : v[i + o], keep = lane & o ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    return v[0];
}

// The query tile, landed by TMA as bf16, turned into f16 in place with a power
// of two a head that puts the row's maximum in [2^14, 2^15); the head's softmax
// multiplier qs[h] takes it back.  Thread t: head t / 4, of each 64-channel
// atom the 16-byte pieces 2 (t % 4) and the next (eight lanes, two heads, cover
// the eight slots of a row).  The maxima are found before the last raw product
// is done with the tile, so that only the conversion itself waits for it; six
// pieces are in flight at a time.
struct QueryPart {
    unsigned char* at[2];
    float mul;
};
template <uint32_t q_atom>
__device__ __forceinline__ void query_scale(uint32_t* status, float sm_log2, unsigned char* tile,
                                            float* qs, int t, QueryPart& x) {
    const int h = t >> 2, qq = t & 3;
    unsigned char* row = tile + (h >> 3) * 1024 + (h & 7) * 128;
    x.at[0] = row + (((2 * qq) ^ (h & 7)) << 4);
    x.at[1] = row + (((2 * qq + 1) ^ (h & 7)) << 4);
    uint32_t amax = 0;  // max |x| as fp32 bits (integer order = float order)
#pragma unroll
    for (int i0 = 0; i0 < 18; i0 += 6) {
        uint4 v[6];
#pragma unroll
        for (int i = 0; i < 6; ++i)
            v[i] = *reinterpret_cast<const uint4*>(x.at[i & 1] + ((i0 + i) >> 1) * q_atom);
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                amax = max(amax, max((w[k] << 16) & 0x7FFFFFFFu, w[k] & 0x7FFF0000u));
        }
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    int k = 0;
    if (amax >= 0x7F800000u) {
        if (qq == 0) set_status(status, KVC_DEV_NONFINITE);
    } else if (amax != 0) {
        k = min(max((int)(amax >> 23) - 127 - 14, -60), 113);  // floor(log2 amax) - 14
    }
    x.mul = __uint_as_float((uint32_t)(127 - k) << 23);
    if (qq == 0) qs[h] = sm_log2 * __uint_as_float((uint32_t)(127 + k) << 23);
}
template <uint32_t q_atom>
__device__ __forceinline__ void queries_to_f16(const QueryPart& x) {
#pragma unroll
    for (int i0 = 0; i0 < 18; i0 += 6) {
        uint4 v[6];
#pragma unroll
        for (int i = 0; i < 6; ++i)
            v[i] = *reinterpret_cast<const uint4*>(x.at[i & 1] + ((i0 + i) >> 1) * q_atom);
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = pack_f16(__uint_as_float(w[j] << 16) * x.mul,
                                __uint_as_float(w[j] & 0xFFFF0000u) * x.mul);
            *reinterpret_cast<uint4*>(x.at[i & 1] + ((i0 + i) >> 1) * q_atom) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// A load warp's part of a chunk: 32 keys, two pairs, and the RoPE channels of 16
// keys.  Of a pair four lanes read the 64 code bytes of a record (eight keys at
// a time, four times), so that a load touches 8 lines and not 32: the loads,
// the stores and every barrier share one queue.  RoPE: two lanes a key.  Each
// item of 32 channels comes with the word of the record that holds its scales;
// its bytes are taken out at the store (taken out here, they would be waited
// for here).
template <int G>
struct Rec {
    uint4 code[2][4];
    uint32_t scale[2][4];
    uint4 rope;
    uint32_t rope_scale;
    // channel: the item's first, counted from the start of the groups
    static __device__ __forceinline__ uint32_t scales(const uint8_t* rec, int channel) {
        return __ldg(reinterpret_cast<const uint32_t*>(rec + 288) + (channel / G >> 2));
    }
    static __device__ __forceinline__ int shift(int channel) { return 8 * (channel / G & 3); }
    // idx: lane l holds key l's record.  A masked key (-1) reads `none` instead,
    // and its scales are taken as 0 at the store.
    __device__ __forceinline__ void load(const uint8_t* recs, int rb, int idx, const uint8_t* none,
                                         int grp, int lane) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = __shfl_sync(0xffffffffu, idx, 8 * u + (lane >> 2));
            const uint8_t* rec = k >= 0 ? recs + (size_t)k * rb : none;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int item = 4 * (grp + 2 * i) + (lane & 3);
                code[i][u] = ldg_nc(rec + 16 * item);
                scale[i][u] = scales(rec, 32 * item);
            }
        }
        load_rope(recs, rb, __shfl_sync(0xffffffffu, idx, 16 * grp + (lane >> 1)), none, lane);
    }
    __device__ __forceinline__ void load_rope(const uint8_t* recs, int rb, int k,
                                              const uint8_t* none, int lane) {
        const uint8_t* rec = k >= 0 ? recs + (size_t)k * rb : none;
        rope = ldg_nc(rec + 256 + 16 * (lane & 1));
        rope_scale = scales(rec, 512 + 32 * (lane & 1));
    }
};

// Item `code` (32 channels, 4 words) of a row into its 16-byte pieces; step k
// stores word k ^ 2 j at slot z ^ k (z holds the row's swizzle, the item's half
// of the atom and 2 j), so that eight lanes, two rows of items in two atoms
// (j = 0, 1), hit eight slots.
template <int G>
__device__ __forceinline__ void store_item(unsigned char* row, int z, int j, const uint4& code,
                                           uint32_t scale) {
    const uint32_t c[4] = {j ? code.z : code.x, j ? code.w : code.y, j ? code.x : code.z,
                           j ? code.y : code.w};
    uint32_t s2 = ue4m3_f16x2(scale & 0xFFu);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (G < 32) s2 = ue4m3_f16x2((scale >> (G == 8 ? 8 * (k ^ 2 * j) : 8 * ((k >> 1) ^ j))) & 0xFFu);
        uint32_t w[4];
        e2m1x8_scaled(c[k], s2, w);
        *reinterpret_cast<uint4*>(row + ((z ^ k) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int G, int HG>
__global__ void __launch_bounds__(NT, 1)
tree_t128_kernel(const __grid_constant__ CUtensorMap tm_q, TreeArgs a, int rb, int H, int K,
                 float sm_log2, int nsplit, unsigned long long wait_ns) {
    constexpr int NH = HG / 2;                        // heads of a softmax warp
    constexpr uint32_t Q_ATOM = (uint32_t)HG * 128u;  // packed atoms of HG rows
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (base - raw_base);
    const uint32_t sQ = base + OFF_Q, sK = base + OFF_K, sP = base + OFF_P;
    Misc& ms = *reinterpret_cast<Misc*>(smem + OFF_MISC);
    const uint32_t bars = smem_u32(ms.bars);
    auto bar = [&](int i) { return bars + 8u * i; };

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (known to be warp-uniform)
    const int split = blockIdx.x % nsplit;
    const int first = blockIdx.x / nsplit, step = gridDim.x / nsplit;
    const int nhg = H / HG, total = a.nodes * a.batch * nhg;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                         smem_u32(&ms.tmem)),
                     "r"(TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    if (tid == 0) {
        for (int i = 0; i < N_BARS; ++i) {
            const int count = i < B_FREE || i == B_P || i == B_Q16   ? 8
                              : i == B_MAX || i == B_MAX + 1         ? 4
                              : i == B_ITEM || i == B_ITEM + 1       ? 17
                              : i >= B_SUM && i < B_END              ? 4
                                                                     : 1;
            mbar_init(bar(i), count);
        }
        ms.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (nsplit > 1 && tid < HG) {  // where each head's owner takes this CTA's sums
        const int hpc = (HG + nsplit - 1) / nsplit;
        const int r = tid / hpc, hh = tid - r * hpc;
        const int nh_r = min(hpc, HG - r * hpc);
        uint32_t rk, rm;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rk) : "r"(sK), "r"(r));
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(rm)
                     : "r"(smem_u32(ms.ml)), "r"(r));
        ms.row_at[tid] = rk + (uint32_t)(split * nh_r + hh) * DV * 4;
        ms.ml_at[tid] = rm + (uint32_t)(split * nh_r + hh) * 8;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem;
    pdl_wait();

    bool ok = true;
    int gc = 0;  // chunks so far (phase of the chunk barriers)
    int mine = 0;           // exchange: this CTA's chunks of its one item
    float mref = -INFINITY, lv = 0.f;  // softmax warps: reference and sum of weights of head
                                       // lane (of the warp's half)
    auto warp_wait = [&](int i, int parity) { return mbar_warp_wait(bar(i), parity, wait_ns); };
    // The item's facts, once the path warp has published them.
    auto get_item = [&](int it, Item& x) {
        ok = warp_wait(B_INFO + (it & 1), (it >> 1) & 1);
        if (ok) x = ms.item[it & 1];
        return ok;
    };

    // Registers: 640 threads start with 96 each; while the roles run the last
    // warpgroup gives up 40 a thread and the two of the softmax take 16 each
    // (256 x 112 + 256 x 96 + 128 x 56 = 60,416 of 61,440).
    if (warp < SOFT_WARPS) {
        // ------------------------------------------------ softmax and output
        more_registers<112>();
        const int q = warp & 3, half = warp >> 2, hb = half * NH;
        const int s = q * 32 + lane;  // key of a chunk, tensor-memory lane
        const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16);
        unsigned char* prow = smem + OFF_P + (s >> 3) * 1024 + (s & 7) * 128;  // P^T of the key
        int it = 0, nsum = 0, nmax = 0, nover = 0;
        for (int w = first; w < total && ok; w += step, ++it) {
            Item x;
            if (!get_item(it, x)) break;
            mref = -INFINITY;
            lv = 0.f;
            // sums of this thread's key's weights (fp32, unrounded), added
            // over the lanes once at the end
            float l[NH];
#pragma unroll
            for (int i = 0; i < NH; ++i) l[i] = 0.f;
            for (int c = x.c0; c < x.c1; ++c, ++gc) {
                const bool raw = c < x.nraw;
                ok = warp_wait(B_S, gc & 1);
                if (!ok) break;
                tc_fence_after();
                const bool valid = ms.valid[gc & 1][s];
                const float mul = raw || lane >= NH ? sm_log2 : ms.qs[it & 1][hb + lane];
                uint32_t r[NH];
                auto logits = [&]() {
                    tmem_ld<NH>(ta + S_COL + hb, r);
                    tmem_wait_ld();
                    if (!__all_sync(0xffffffffu, valid))
#pragma unroll
                        for (int i = 0; i < NH; ++i) r[i] = valid ? r[i] : 0xFF800000u;  // -inf
                };
                auto factors = [&]() {
                    float* k = reinterpret_cast<float*>(&ms.sm[warp][lane >> 1]) + (lane & 1);
                    k[0] = mul;
                    k[2] = mref == -INFINITY ? 0.f : -mref;
                    __syncwarp();
                };
                // weights 2^(x - reference) of the key in place of its logits,
                // and P^T; returns the largest exponent
                auto weights = [&]() {
                    float mx = -INFINITY;
                    float4 f[2][4];  // (the next heads' factors: P^T's stores hold loads back)
#pragma unroll
                    for (int u = 0; u < 4; ++u) f[0][u] = ms.sm[warp][u];
#pragma unroll
                    for (int c8 = 0; c8 < NH / 8; ++c8) {
                        if (c8 + 1 < NH / 8)
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                f[(c8 + 1) & 1][u] = ms.sm[warp][4 * (c8 + 1) + u];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            uint32_t &p0 = r[8 * c8 + 2 * u], &p1 = r[8 * c8 + 2 * u + 1];
                            fma2(p0, p1, f[c8 & 1][u]);
                            mx = max3(mx, __uint_as_float(p0), __uint_as_float(p1));
                            p0 = __float_as_uint(ex2(__uint_as_float(p0)));
                            p1 = __float_as_uint(ex2(__uint_as_float(p1)));
                        }
                        uint32_t v[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float p0 = __uint_as_float(r[8 * c8 + 2 * u]);
                            const float p1 = __uint_as_float(r[8 * c8 + 2 * u + 1]);
                            v[u] = raw ? pack_bf16(p0, p1) : pack_f16(p0, p1);
                        }
                        *reinterpret_cast<uint4*>(prow + ((((hb >> 3) + c8) ^ (s & 7)) << 4)) =
                            make_uint4(v[0], v[1], v[2], v[3]);
                    }
                    return mx;
                };
                auto in_place = [&](int i) {
                    fence_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(i));
                };
                // The references of the earlier chunks nearly always serve: the
                // weights are made with them at once.  Where one of this head
                // half passes 2^kMost, the products are told to wait until the
                // half has done it over with the chunk's own maxima, as the
                // first chunk does.
                bool fresh = c == x.c0;
                logits();
                if (!fresh) {
                    if (c == x.nraw) factors();  // other multipliers from here on
                    // (a head without a key so far has no reference)
                    const bool over = __any_sync(
                        0xffffffffu, weights() > kMost || (lane < NH && mref == -INFINITY));
                    int(&ov)[4] = ms.over[gc & 1][half];
                    if (lane == 0) {
                        ov[q] = over;
                        mbar_arrive(bar(B_OVER + half));
                    }
                    in_place(B_P);
                    ok = warp_wait(B_OVER + half, nover++ & 1);
                    if (!ok) break;
                    fresh = ov[0] | ov[1] | ov[2] | ov[3];
                    if (fresh) logits();
                }
                if (fresh) {
                    // the chunk's maximum of every head: over the warp's keys,
                    // then over the four quadrants
                    float mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < NH; ++i) {
                        const float m = warp_max(__uint_as_float(r[i]));
                        if (lane == i) mx = m;
                    }
                    float(&wm)[4][32] = ms.wmax[nmax & 1][half];
                    wm[q][lane] = mx;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_MAX + half));
                    ok = warp_wait(B_MAX + half, nmax++ & 1);
                    if (!ok) break;
                    const float mc = mul * fmaxf(fmaxf(wm[0][lane], wm[1][lane]),
                                                 fmaxf(wm[2][lane], wm[3][lane]));
                    const float mo = mref;
                    if (mo == -INFINITY || mc > mo + kMost) mref = mc - kTop;
                    const float f = mo == -INFINITY ? 1.f : ex2(mo - mref);
                    ms.fac[warp][lane] = f;
                    factors();
                    if (__any_sync(0xffffffffu, lane < NH && c > x.c0 && f != 1.f)) {
                        // a reference moved: what the sums and accumulators
                        // hold of the earlier chunks is rescaled
                        ok = warp_wait(B_FREE + 2, (gc - 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int t = 0; t < 4; ++t) {
                            const uint32_t at = ta + O_COL + 64 * t + hb;
                            uint32_t o[NH];
                            tmem_ld<NH>(at, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < NH; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * ms.fac[warp][i]);
                            tmem_st<NH>(at, o);
                        }
#pragma unroll
                        for (int i = 0; i < NH; ++i) l[i] *= ms.fac[warp][i];
                        logits();
                    }
                    weights();
                    in_place(c == x.c0 ? B_P : B_REDO + half);
                }
#pragma unroll
                for (int i = 0; i < NH; ++i) l[i] += __uint_as_float(r[i]);
            }
            if (!ok) break;
            if (x.c1 > x.c0) {
                float(&ls)[4][32] = ms.lsum[half];
                ls[q][lane] = lane_sums<NH>(l, lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_SUM + half));
                ok = warp_wait(B_SUM + half, nsum++ & 1) && warp_wait(B_FREE + 2, (gc - 1) & 1);
                if (!ok) break;
                lv = (ls[0][lane] + ls[1][lane]) + (ls[2][lane] + ls[3][lane]);
                tc_fence_after();
                mine = 1;
            }
            if (nsplit == 1) {
                // ---- output: lane = channel of a tile; two lanes trade halves of
                // two heads so that a lane stores two channels of one head
                const int hg0 = (w % nhg) * HG, id = w / nhg;
                const int b = id / a.nodes, t = id - b * a.nodes;
                const size_t row = ((size_t)t * a.batch + b) * H + hg0 + hb;
                if (q == 0 && a.lse && lane < NH)
                    a.lse[row + lane] = lv == 0.f ? -INFINITY : (mref + __log2f(lv)) * kLn2;
                ms.fac[warp][lane] = lv == 0.f ? 0.f : 1.f / lv;
                __syncwarp();
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (row + (lane & 1)) * DV +
                                     q * 32 + (lane & ~1);
#pragma unroll 1
                for (int mt = 0; mt < 4; ++mt) {
                    uint32_t o[NH];
#pragma unroll
                    for (int i = 0; i < NH; ++i) o[i] = 0u;
                    if (x.c1 > x.c0) {
                        tmem_ld<NH>(ta + O_COL + 64 * mt + hb, o);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int i = 0; i < NH; i += 2) {
                        const float2 k = *reinterpret_cast<const float2*>(&ms.fac[warp][i]);
                        const float u = __uint_as_float(o[i]) * k.x;
                        const float v = __uint_as_float(o[i + 1]) * k.y;
                        const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? u : v, 1);
                        const uint32_t two = lane & 1 ? pack_bf16(got, v) : pack_bf16(u, got);
                        *reinterpret_cast<uint32_t*>(out + (size_t)i * DV + mt * 128) = two;
                    }
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_ITEM + (it & 1)));
        }
        fewer_registers<96>();
    } else if (warp < SOFT_WARPS + LOAD_WARPS) {
        // ------------------------------------------------------------- loads
        const int lw = warp - SOFT_WARPS;
        const int grp = lw >> 2;         // pairs grp and grp + 2
        const int row0 = (lw & 3) * 32;  // the warp's keys
        const int kq = lane >> 3;        // raw rows: eight lanes a row
        const int k8 = lane >> 2, j = (lane >> 1) & 1;  // records: four lanes a key
        const int z = (4 * (lane & 1)) ^ (2 * j) ^ k8;
        unsigned char* krow = smem + OFF_K + (row0 >> 3) * 1024 + k8 * 128 + j * K_ATOM;
        const int rkey = row0 + 16 * grp + (lane >> 1);  // RoPE: two lanes a key
        unsigned char* rrow = smem + OFF_K + 8 * K_ATOM + (rkey >> 3) * 1024 + (rkey & 7) * 128;
        auto filled = [&](int p) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_FULL + p));
        };
        int it = 0, nq = 0;
        if (first < total) {  // the first node's selection, while its path is walked
            const int id = first / nhg, b = id / a.nodes, t = id - b * a.nodes;
            const int32_t* sel = a.topk_idx + (size_t)(a.topk_shared ? b : t * a.batch + b) * K;
            for (int j = tid - SOFT_WARPS * 32; j < (K + 31) / 32; j += LOAD_WARPS * 32)
                prefetch_l2(sel + 32 * j);
        }
        for (int w = first; w < total && ok; w += step, ++it) {
            Item x;
            if (!get_item(it, x)) break;
            const int hg0 = (w % nhg) * HG, id = w / nhg;
            const int b = id / a.nodes, t = id - b * a.nodes;
            const int node = t * a.batch + b;
            const int32_t* sel = a.topk_idx + (a.topk_shared ? (size_t)b : (size_t)node) * K;
            const uint8_t* recs = a.records + (size_t)b * a.capacity * rb;
            // (a query row is longer than a record)
            const uint8_t* none = static_cast<const uint8_t*>(a.q);
            // record of key row0 + lane in chunk c, or -1
            auto pick = [&](int c) {
                const int j = (c - x.nraw) * CK + row0 + lane;
                if (j >= K || x.n < 0) return -1;
                const int idx = __ldg(sel + j);
                if (idx >= 0 && idx < x.n) return idx;
                if (idx != -1 && grp == 0 && hg0 == 0) set_status(a.status, KVC_DEV_BAD_INDEX);
                return -1;
            };
            Rec<G> rec;
            int cur = -1;
            const int cr = max(x.c0, x.nraw);  // first record chunk
            if (cr < x.c1) cur = pick(cr);
            // (behind the first node's raw copies: the index is on its way)
            const bool early = gc > 0 || x.c0 >= x.nraw;
            if (early && cr < x.c1) rec.load(recs, rb, cur, none, grp, lane);
            // ---- raw chunks
            int c = x.c0;
            for (; c < min(x.nraw, x.c1); ++c, ++gc) {
                // lane l finds row l of the warp's; eight lanes then copy 128
                // bytes of a row, four rows at a time
                const int j = c * CK + row0 + lane, r = x.skip + j;
                unsigned long long mine_row = 0;
                if (j < x.raw)
                    mine_row = reinterpret_cast<unsigned long long>(
                        r < x.wl ? static_cast<const __nv_bfloat16*>(a.window) +
                                       ((size_t)b * a.window_stride + r) * D
                                 : static_cast<const __nv_bfloat16*>(a.draft) +
                                       ((size_t)ms.up[it & 1][x.depth - 1 - (r - x.wl)] * a.batch + b) *
                                           D);
                const uint32_t piece = lane & 7;
                // `atoms` atoms from `atom` on, of rows first .. first + rows - 1
                auto copy = [&](int atom, int atoms, int first, int rows) {
#pragma unroll
                    for (int k = 0; k < rows / 4; ++k) {
                        const unsigned long long from =
                            __shfl_sync(0xffffffffu, mine_row, first + 4 * k + kq);
                        const __nv_bfloat16* src =
                            (from ? reinterpret_cast<const __nv_bfloat16*>(from)
                                  : static_cast<const __nv_bfloat16*>(a.draft)) + 64 * atom + 8 * piece;
                        const uint32_t dst =
                            sK + atom * K_ATOM + swz(row0 + first + 4 * k + kq, piece);
#pragma unroll
                        for (int i = 0; i < atoms; ++i)
                            cp16(dst + i * K_ATOM, src + 64 * i, from != 0);
                    }
                    cp_commit();
                };
                if (gc > 0) ok = warp_wait(B_FREE + grp, (gc - 1) & 1);
                if (!ok) break;
                if (grp == 0) ms.valid[gc & 1][row0 + lane] = mine_row != 0;
                copy(2 * grp, 2, 0, 32);
                if (gc > 0) {  // (it lands while the last products run)
                    cp_wait<0>();
                    filled(0);
                    ok = warp_wait(B_FREE + 2, (gc - 1) & 1);
                    if (!ok) break;
                }
                copy(2 * grp + 4, 2, 0, 32);
                copy(8, 1, 16 * grp, 16);
                if (!early && c == x.c0 && cr < x.c1) rec.load(recs, rb, cur, none, grp, lane);
                if (gc == 0) {
                    cp_wait<2>();
                    filled(0);
                }
                cp_wait<0>();
                filled(1);
            }
            if (!ok) break;
            // ---- the queries to f16, once the raw chunks' products have read them
            if (cr < x.c1) {
                ok = warp_wait(B_Q, nq & 1);
                if (!ok) break;
                const int ct = tid - SOFT_WARPS * 32;
                QueryPart part;
                if (ct < 4 * HG)
                    query_scale<Q_ATOM>(a.status, sm_log2, smem + OFF_Q, ms.qs[it & 1], ct, part);
                if (c > x.c0) ok = warp_wait(B_S, (gc - 1) & 1);
                if (!ok) break;
                if (ct < 4 * HG) queries_to_f16<Q_ATOM>(part);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_Q16));
            }
            if (x.c1 > x.c0) ++nq;
            // ---- record chunks
            for (; c < x.c1; ++c, ++gc) {
                const int next = c + 1 < x.c1 ? pick(c + 1) : -1;
                bool keep[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    keep[u] = __shfl_sync(0xffffffffu, cur, 8 * u + k8) >= 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int p = grp + 2 * i;
                    if (gc > 0) ok = warp_wait(B_FREE + (i ? 2 : grp), (gc - 1) & 1);
                    if (!ok) break;
                    if (i == 0 && grp == 0) ms.valid[gc & 1][row0 + lane] = cur >= 0;
                    const int shift = Rec<G>::shift(32 * (4 * p + (lane & 3)));
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        store_item<G>(krow + 2 * p * K_ATOM + u * 1024, z, j, rec.code[i][u],
                                      keep[u] ? rec.scale[i][u] >> shift : 0u);
                    if (i == 0) filled(0);
                }
                if (!ok) break;
                const bool live = __shfl_sync(0xffffffffu, cur, 16 * grp + (lane >> 1)) >= 0;
                store_item<G>(rrow, (4 * (lane & 1)) ^ (rkey & 7), 0, rec.rope,
                              live ? rec.rope_scale >> Rec<G>::shift(512 + 32 * (lane & 1)) : 0u);
                filled(1);
                // all loads behind the chunk's stores: issuing them takes a
                // thousand clocks, which lie under QK and the softmax here
                if (c + 1 < x.c1) rec.load(recs, rb, next, none, grp, lane);
                cur = next;
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_ITEM + (it & 1)));
        }
        cp_wait<0>();
    } else {
        fewer_registers<56>();
        if (warp == MMA_WARP) {
            // ---------------------------------------------------------- products
            int it = 0, nq = 0, n16 = 0, nredo0 = 0, nredo1 = 0;
            // operand descriptors; offsets are in units of 16 bytes
            const uint64_t kd = sdesc(sK, 16, 1024), qd = sdesc(sQ, 16, 1024);
            const uint64_t vd = sdesc(sK, K_ATOM, 1024), pd = sdesc(sP, K_ATOM, 1024);
            for (int w = first; w < total && ok; w += step, ++it) {
                Item x;
                if (!get_item(it, x)) break;
                if (x.c1 > x.c0) {
                    // every product that reads the query tile is done: its
                    // softmax was waited for
                    const int hg0 = (w % nhg) * HG, id = w / nhg;
                    const int b = id / a.nodes, t = id - b * a.nodes;
                    const int y = (t * a.batch + b) * H + hg0;
                    if (lane == 0) {
                        mbar_expect_tx(bar(B_Q), NATOM * Q_ATOM);
                        for (int at = 0; at < NATOM; ++at)
                            tma_load_2d(sQ + at * Q_ATOM, &tm_q, 64 * at, y, bar(B_Q));
                    }
                    __syncwarp();
                    ++nq;
                }
                for (int c = x.c0; c < x.c1; ++c, ++gc) {
                    const bool raw = c < x.nraw;
                    const uint32_t idQK = idesc_f16(128, HG, raw, 0, 0);
                    const uint32_t idPV = idesc_f16(128, 64, raw, 1, 1);
                    if (raw && c == x.c0) ok = warp_wait(B_Q, (nq - 1) & 1);
                    if (!raw && c == max(x.c0, x.nraw)) ok = warp_wait(B_Q16, n16++ & 1);
                    ok = ok && warp_wait(B_FULL, gc & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect()) {
#pragma unroll
                        for (int kk = 0; kk < 16; ++kk) {
                            const uint64_t ka = kd + (kk >> 2) * (K_ATOM >> 4) + (kk & 3) * 2;
                            const uint64_t qa = qd + (kk >> 2) * (Q_ATOM >> 4) + (kk & 3) * 2;
                            if (kk == 0) mma_f16(tmem + S_COL, ka, qa, idQK, 0);
                            else mma(tmem + S_COL, ka, qa, idQK);
                        }
                    }
                    __syncwarp();
                    ok = warp_wait(B_FULL + 1, gc & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect()) {
#pragma unroll
                        for (int kk = 16; kk < 36; ++kk)
                            mma(tmem + S_COL, kd + (kk >> 2) * (K_ATOM >> 4) + (kk & 3) * 2,
                                qd + (kk >> 2) * (Q_ATOM >> 4) + (kk & 3) * 2, idQK);
                        mma_commit(bar(B_S));
                    }
                    __syncwarp();
                    ok = warp_wait(B_P, gc & 1);
                    if (ok && c > x.c0) {  // a head half that does its weights over
                        const int4 o0 = *reinterpret_cast<const int4*>(ms.over[gc & 1][0]);
                        const int4 o1 = *reinterpret_cast<const int4*>(ms.over[gc & 1][1]);
                        if (o0.x | o0.y | o0.z | o0.w) ok = warp_wait(B_REDO, nredo0++ & 1);
                        if (ok && (o1.x | o1.y | o1.z | o1.w))
                            ok = warp_wait(B_REDO + 1, nredo1++ & 1);
                    }
                    if (!ok) break;
                    tc_fence_after();
                    if (elect()) {
#pragma unroll 1
                        for (int p = 0; p < 4; ++p) {
                            const uint32_t o = tmem + O_COL + 64 * p;
                            const uint64_t va = vd + p * (2 * K_ATOM >> 4);
                            mma_f16(o, va, pd, idPV, c > x.c0);
#pragma unroll
                            for (int kk = 1; kk < CK / 16; ++kk)
                                mma(o, va + kk * 128, pd + kk * 128, idPV);
                            if (p != 2) mma_commit(bar(B_FREE + (p < 2 ? p : 2)));
                        }
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (lane == 0) mbar_arrive(bar(B_ITEM + (it & 1)));
            }
            // Nothing of this CTA is in flight past here: the softmax waited for
            // the last products; after a timeout they and the queries' copies
            // are waited for now (the elected lane is the same throughout, so
            // its commit covers every product).
            if (!ok && elect()) {
                mma_commit(bar(B_END));
                mbar_wait(bar(B_END), 0, kCleanupWaitNs);
                if (nq > 0) mbar_wait(bar(B_Q), (nq - 1) & 1, kCleanupWaitNs);
            }
            __syncwarp();
        } else if (warp == PATH_WARP) {
            // -------------------------------------------------------------- path
            int it = 0;
            for (int w = first; w < total && ok; w += step, ++it) {
                if (it >= 2) ok = warp_wait(B_ITEM + (it & 1), ((it >> 1) - 1) & 1);
                if (!ok) break;
                const int id = w / nhg;
                const int b = id / a.nodes, t = id - b * a.nodes;
                const int n = a.n_entries[b];
                int wl = a.window_lens ? a.window_lens[b] : a.window_len;
                for (int i = lane; i <= t; i += 32) {
                    const int p = a.parents[(size_t)i * a.batch + b];
                    ms.parents[i] = (short)(p < -2 || p >= i ? -3 : p);
                }
                __syncwarp();
                if (lane == 0) {
                    const bool len_ok = n >= 0 && n <= a.capacity;
                    if (!len_ok || wl < 0 || wl > a.window_len) set_status(a.status, KVC_DEV_BAD_LENGTH);
                    if (wl < 0 || wl > a.window_len) wl = 0;
                    int depth = 0, at = t;
                    for (;;) {
                        ms.up[it & 1][depth++] = (unsigned char)at;
                        at = ms.parents[at];
                        if (at >= 0) continue;
                        if (at == -3) set_status(a.status, KVC_DEV_BAD_INDEX);
                        if (at != -1) depth = 0;
                        break;
                    }
                    Item x;
                    x.depth = depth;
                    x.wl = wl;
                    x.n = len_ok ? n : -1;
                    x.raw = depth ? min(a.window_stride, wl + depth) : 0;
                    x.skip = wl + depth - x.raw;
                    x.nraw = (x.raw + CK - 1) / CK;
                    const int chunks = depth ? x.nraw + (K + CK - 1) / CK : 0;
                    x.c0 = chunks * split / nsplit;
                    x.c1 = chunks * (split + 1) / nsplit;
                    ms.item[it & 1] = x;
                    mbar_arrive(bar(B_INFO + (it & 1)));
                }
                __syncwarp();
                if (it > 0) {  // (a CTA's first node is being loaded already)
                    const int node = t * a.batch + b;
                    const int32_t* sel = a.topk_idx + (a.topk_shared ? (size_t)b : (size_t)node) * K;
                    const uint8_t* recs = a.records + (size_t)b * a.capacity * rb;
                    const char* qrow = static_cast<const char*>(a.q) +
                                       ((size_t)node * H + (w % nhg) * HG) * D * 2;
                    for (int i = lane; i < (int)(NATOM * Q_ATOM) / 128; i += 32)
                        prefetch_l2(qrow + 128 * i);
                    for (int j = lane; j < K; j += 32) {
                        const int idx = __ldg(sel + j);
                        if (idx >= 0 && idx < min(n, a.capacity))
                            for (int o = 0; o < rb; o += 128)
                                prefetch_l2(recs + (size_t)idx * rb + o);
                    }
                }
            }
        }
        __syncwarp();
    }
    if (!ok && lane == 0) {
        ms.failed = 1;
        set_status(a.status, KVC_DEV_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    // (only now: a warp that waits for registers to be free takes issue slots
    // from the others of its scheduler)
    if (warp >= MMA_WARP) more_registers<96>();
    tc_fence_after();
    pdl_trigger();  // only the exchange is left: let the next kernel be scheduled

    if (nsplit > 1) {
        // ---- the CTAs of the cluster hold parts of one node: CTA r owns heads
        // [r hpc, (r + 1) hpc) of the group.  Each stores its unnormalised O
        // columns (a lane per channel) and (m, l) into the owners' freed K
        // tiles, rows [split][head] of 2 KB; every owner joins them in split
        // order.
        const int hpc = (HG + nsplit - 1) / nsplit;
        const int h_lo = split * hpc, nh = max(0, min(HG, h_lo + hpc) - h_lo);
        const bool have = !ms.failed;
        cluster_sync();  // every CTA of the cluster is past its last product
        if (warp < SOFT_WARPS) {
            const int q = warp & 3, hb = (warp >> 2) * NH;
            const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16);
            const bool any = have && mine;
            if (q == 0 && lane < NH)
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(ms.ml_at[hb + lane]),
                             "f"(any ? mref : -INFINITY), "f"(any ? lv : 0.f)
                             : "memory");
            if (any) {
#pragma unroll 1
                for (int mt = 0; mt < 4; ++mt) {
                    uint32_t o[NH];
                    tmem_ld<NH>(ta + O_COL + 64 * mt + hb, o);
                    tmem_wait_ld();
                    const uint32_t d4 = (mt * 128 + q * 32 + lane) * 4;
#pragma unroll
                    for (int i = 0; i < NH; ++i)
                        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(ms.row_at[hb + i] + d4),
                                     "r"(o[i])
                                     : "memory");
                }
            }
            tc_fence_before();
        }
        cluster_sync();  // every row and (m, l) has arrived
        const int hg0 = (first % nhg) * HG, id = first / nhg;
        const int b = id / a.nodes, t = id - b * a.nodes;
        const size_t row = ((size_t)t * a.batch + b) * H + hg0 + h_lo;
        if (tid < nh) {
            float2 ml[8];
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < nsplit) {
                    ml[r] = reinterpret_cast<const float2*>(ms.ml)[r * nh + tid];
                    M = fmaxf(M, ml[r].x);
                }
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < nsplit) {
                    // a split without a weight pushed no row, or one of zeros
                    const float wt = ml[r].y == 0.f ? 0.f : ex2(ml[r].x - M);
                    ms.wts[tid * nsplit + r] = wt;
                    if (ml[r].y != 0.f) L += wt * ml[r].y;
                }
            ms.inv[tid] = L == 0.f ? 0.f : 1.f / L;
            if (a.lse) a.lse[row + tid] = L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
        }
        __syncthreads();
        const float* rows = reinterpret_cast<const float*>(smem + OFF_K);
        for (int i = tid; i < nh * (DV / 4); i += NT) {
            const int hh = i / (DV / 4), q4 = i - hh * (DV / 4);
            float wt[8];
            float4 v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < nsplit) {
                    wt[r] = ms.wts[hh * nsplit + r];
                    v[r] = reinterpret_cast<const float4*>(rows + (r * nh + hh) * DV)[q4];
                }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < nsplit && wt[r] != 0.f) {
                    acc.x = fmaf(wt[r], v[r].x, acc.x);
                    acc.y = fmaf(wt[r], v[r].y, acc.y);
                    acc.z = fmaf(wt[r], v[r].z, acc.z);
                    acc.w = fmaf(wt[r], v[r].w, acc.w);
                }
            const float inv = ms.inv[hh];
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (row + hh) * DV + 4 * q4) =
                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem),
                     "r"(TMEM_COLS));
}

template <int G, int HG>
cudaError_t configure(int dev) {
    static bool done[64] = {};
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(
        tree_t128_kernel<G, HG>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

template <int G, int HG>
cudaError_t launch(const kvc_config& c, const Shape& sh, const TreeArgs& a, int nsplit, unsigned grid,
                   cudaStream_t s) {
    CUtensorMap tq = {};
    if (!encode_rows576(&tq, a.q, (unsigned long long)a.nodes * a.batch * c.n_heads, HG))
        return cudaErrorUnknown;
    int dev = 0;
    cudaGetDevice(&dev);
    cudaError_t e = configure<G, HG>(dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = nsplit;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const float sm_log2 = c.sm_scale * 1.4426950408889634f;
    trace_before("tree_t128", s);
    e = cudaLaunchKernelEx(&cfg, tree_t128_kernel<G, HG>, tq, a, sh.rb, c.n_heads, c.topk, sm_log2,
                           nsplit, device_wait_limit_ns());
    trace_after(s);
    return e;
}

template <int G>
cudaError_t launch_g(const kvc_config& c, const Shape& sh, const TreeArgs& a, int hg, int nsplit,
                     unsigned grid, cudaStream_t s) {
    if (hg == 64) return launch<G, 64>(c, sh, a, nsplit, grid, s);
    if (hg == 32) return launch<G, 32>(c, sh, a, nsplit, grid, s);
    return launch<G, 16>(c, sh, a, nsplit, grid, s);
}

// Clusters of `size` of these CTAs (one a multiprocessor) that can be resident
// at once on the current device; the kernel's variants have the same shape.
int max_clusters(int size) {
    static int cache[64][9] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return 0;
    if (cache[dev][size]) return cache[dev][size] > 0 ? cache[dev][size] : 0;
    configure<32, 64>(dev);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, tree_t128_kernel<32, 64>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    cache[dev][size] = n > 0 ? n : -1;
    return n;
}

}  // namespace tree

bool tree_t128_supported(const kvc_config& c, const Shape& sh) {
    const bool g_ok = sh.G == 8 || sh.G == 16 || sh.G == 32 || sh.G == 64 || sh.G == 128;
    return c.act_dtype == KVC_BF16 && c.scale_fmt == KVC_SCALE_UE4M3 && c.n_heads % 16 == 0 &&
           sh.D == tree::D && sh.Dv == tree::DV && g_ok;
}

cudaError_t launch_tree_t128(const kvc_config& c, const Shape& sh, const TreeArgs& a,
                             cudaStream_t s) {
    const int H = c.n_heads;
    const int chunks = (std::min(c.window, a.window_len + a.nodes) + tree::CK - 1) / tree::CK +
                       (c.topk + tree::CK - 1) / tree::CK;
    // Split of a node's keys over nsplit CTAs and of its heads into groups of hg:
    // the least of what follows, in microseconds as measured on one sequence's
    // node to 256 nodes of 5 chunks (64 heads; in brackets measured).  A CTA
    // that takes whole nodes: 10 + rounds x (chunks x c + 1) [1 node 33.8, 256
    // nodes 60.4]; a cluster that splits them: 5 + rounds x (chunks / nsplit x c
    // + e) [1 node over 5 CTAs 23.5, in groups of 16 heads 18.6], where a chunk
    // takes c = 4.5, 3.9, 3.6 and a start, exchange and end e = 14, 12, 10 for
    // 64, 32, 16 heads.
    int hg = 16, nsplit = 1;
    double best = 1e30;
    for (int g = 64; g >= 16; g /= 2) {
        if (H % g) continue;
        const long long items = (long long)a.nodes * a.batch * (H / g);
        const double ct = g == 64 ? 4.5 : g == 32 ? 3.9 : 3.6;
        const double et = g == 64 ? 14.0 : g == 32 ? 12.0 : 10.0;
        for (int ns = 1; ns <= std::min(8, std::max(1, chunks)); ++ns) {
            const long long fit = tree::max_clusters(ns);
            if (fit < 1) continue;
            const double rounds = (double)((items + fit - 1) / fit);
            const double cost = ns == 1 ? 10.0 + rounds * (chunks * ct + 1.0)
                                        : 5.0 + rounds * ((chunks + ns - 1) / ns * ct + et);
            if (cost < best) best = cost, hg = g, nsplit = ns;
        }
    }
    const long long items = (long long)a.nodes * a.batch * (H / hg);
    const unsigned grid =
        nsplit > 1 ? (unsigned)(items * nsplit)
                   : (unsigned)std::min<long long>(items, std::max(1, tree::max_clusters(1)));
    switch (sh.G) {
        case 8: return tree::launch_g<8>(c, sh, a, hg, nsplit, grid, s);
        case 16: return tree::launch_g<16>(c, sh, a, hg, nsplit, grid, s);
        case 32: return tree::launch_g<32>(c, sh, a, hg, nsplit, grid, s);
        case 64: return tree::launch_g<64>(c, sh, a, hg, nsplit, grid, s);
        default: return tree::launch_g<128>(c, sh, a, hg, nsplit, grid, s);
    }
}

}  // namespace kvc
