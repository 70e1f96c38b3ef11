// unpack.cu -- packed records and FP8 window rows read back as rows of
// values.
//
// Method: "DeepSeek V1 到 V4.1-Flash，单 token 的 global KV 如何从 389,000 B
// 压缩到 890 B的？" (acejoy.com) part 4 "P4 main KV" (an element is stored
// relative to its group's scale and multiplied back on use; the window stays
// in FP8).  v_c = E2M1(code_c) * scale_group(c), or E4M3(code_c) * scale_row.
//
// A record is read once (a quarter of what a bf16 row takes) and its row
// written once: the bound is HBM, and four fifths of its bytes are writes.  A
// thread keeps one place of a row, 8 channels (4 code bytes, one 16-byte store,
// two for fp32), and goes through rows, four of them in flight: what depends on
// the place alone (its scale's place above all) is found once, and a row's
// places are neighbouring threads, so accesses are contiguous.  Products of a
// code (two significant bits) and a UE4M3 scale (four) are exact in bf16; with
// fp32 scales they are rounded to fp32 and then to the row's type.  Measured (in
// a graph of twenty calls; "cold": on twenty caches, with L2 swept before):
// 500,000 records of 576 channels to bf16 in 113.4 us, cold 113.9, 6.4 TB/s; 85 %
// of the issue slots are taken then.  200,000 to fp32 in 110 us, 4.7 TB/s.
// Gathered, 32 x 512: 6.3 us, cold 7.8; 1,376 CTAs where 1,332 are resident (32 x
// 492 in 1,312 CTAs take 5.6).  FP8 window rows, a thread 8 channels of a row:
// 500,000 in 198 us, 4.4 TB/s (a 64-bit quotient a thread for the row's scale).
#include <algorithm>

#include "kvc_internal.cuh"

namespace kvc {
namespace {

constexpr int NT = 256;

__device__ __forceinline__ void put8(__nv_bfloat16* dst, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(v[2 * k + 1]), "f"(v[2 * k]));
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put8(float* dst, const float (&v)[8]) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Grid (tiles of rows, batch); block of `lanes` rows' places; a tile is
// lanes * U * rounds rows.
constexpr int U = 4;
template <typename T, bool UE4M3>
__global__ void __launch_bounds__(NT)
unpack_kernel(UnpackArgs a, Shape sh, int lanes, int rounds) {
    pdl_wait();
    const int b = blockIdx.y, np = sh.D >> 3, np_lat = sh.Dv >> 3;
    const int n = a.n_entries[b];
    const bool len_ok = n >= 0 && n <= a.capacity;
    if (!len_ok && blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, KVC_DEV_BAD_LENGTH);
    const int lane = threadIdx.x / np, c = threadIdx.x - lane * np;
    const int lg = 31 - __clz(sh.lpg);  // 8-channel pieces of a group: a power of two
    const int g = c < np_lat ? c >> lg : (sh.Dv + sh.G - 1) / sh.G + ((c - np_lat) >> lg);
    const uint8_t* base = a.records + (size_t)b * a.capacity * sh.rb;
    const int scale_at = sh.code_bytes + g * (UE4M3 ? 1 : 4);
    T* out = static_cast<T*>(a.out) + (size_t)b * a.n * sh.D + 8 * c;
    const int32_t* idx = a.idx ? a.idx + (size_t)b * a.n : nullptr;
    int j = blockIdx.x * (lanes * U * rounds) + lane;
    for (int round = 0; round < rounds; ++round, j += lanes * U) {
        uint32_t codes[U];
        float scale[U];
        int e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = j + lanes * u;
            e[u] = -1;
            if (row < a.n) e[u] = idx ? __ldg(idx + row) : a.first + row;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            codes[u] = 0u;
            scale[u] = 0.f;
            if (e[u] >= 0 && e[u] < n && len_ok) {
                const uint8_t* rec = base + (size_t)e[u] * sh.rb;
                codes[u] = __ldg(reinterpret_cast<const uint32_t*>(rec) + c);
                scale[u] = UE4M3 ? __uint_as_float(__ldg(rec + scale_at))
                                 : __ldg(reinterpret_cast<const float*>(rec + scale_at));
            } else if (idx && e[u] != -1 && len_ok && c == 0) {
                set_status(a.status, KVC_DEV_BAD_INDEX);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = j + lanes * u;
            float v[8];
            e2m1x8_values(codes[u],
                          UE4M3 ? e4m3_to_f32((uint8_t)__float_as_uint(scale[u])) : scale[u], v);
            if (row < a.n) put8(out + (size_t)row * sh.D, v);
        }
    }
}

// FP8 window rows: thread = 8 channels of a row.
template <typename T>
__global__ void __launch_bounds__(NT)
unpack_fp8_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales, long long n,
                  int np, T* __restrict__ rows) {
    pdl_wait();
    for (long long p = (long long)blockIdx.x * NT + threadIdx.x; p < n * np;
         p += (long long)gridDim.x * NT) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(codes) + p);
        const float s = __ldg(scales + p / np);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = e4m3s_to_f32(((k < 4 ? w.x : w.y) >> (8 * (k & 3))) & 0xFFu) * s;
        put8(rows + p * 8, v);
    }
}

}  // namespace

cudaError_t launch_unpack(const kvc_config& c, const Shape& sh, const UnpackArgs& a,
                          cudaStream_t s) {
    // rows at a time: as many as a block's threads hold places for; bf16 rows in
    // two rounds a tile once the grid fills the device anyway (1 round, 2 rounds:
    // 500,000 bf16 rows of 576 119.7, 113.4 us, 64,000 of them 17.6, 17.0; 200,000
    // fp32 rows 110.2, 116.6; 8 and 32 rounds of the bf16 rows 129, 150: short tiles
    // keep what runs at one time close together in memory)
    const int np = sh.D / 8, lanes = NT / np;
    const long long tiles = (long long)a.batch * ((a.n + lanes * U - 1) / (lanes * U));
    const int rounds = c.act_dtype == KVC_BF16 && tiles >= 148 * 16 ? 2 : 1;
    const int tile = lanes * U * rounds;
    const dim3 grid((a.n + tile - 1) / tile, a.batch);
    const bool u = c.scale_fmt == KVC_SCALE_UE4M3;
    trace_before("unpack", s);
    cudaError_t e;
    if (c.act_dtype == KVC_BF16)
        e = u ? launch_pdl(unpack_kernel<__nv_bfloat16, true>, grid, lanes * np, 0, s, a, sh, lanes, rounds)
              : launch_pdl(unpack_kernel<__nv_bfloat16, false>, grid, lanes * np, 0, s, a, sh, lanes, rounds);
    else
        e = u ? launch_pdl(unpack_kernel<float, true>, grid, lanes * np, 0, s, a, sh, lanes, rounds)
              : launch_pdl(unpack_kernel<float, false>, grid, lanes * np, 0, s, a, sh, lanes, rounds);
    trace_after(s);
    return e;
}

cudaError_t launch_unpack_fp8(const kvc_config& c, const Shape& sh, const uint8_t* codes,
                              const float* scales, long long n, void* rows, cudaStream_t s) {
    const int np = sh.D / 8;
    const unsigned grid = (unsigned)std::min<long long>((n * np + NT - 1) / NT, 148 * 64);
    trace_before("unpack_fp8", s);
    const cudaError_t e =
        c.act_dtype == KVC_BF16
            ? launch_pdl(unpack_fp8_kernel<__nv_bfloat16>, grid, NT, 0, s, codes, scales, n, np,
                         static_cast<__nv_bfloat16*>(rows))
            : launch_pdl(unpack_fp8_kernel<float>, grid, NT, 0, s, codes, scales, n, np,
                         static_cast<float*>(rows));
    trace_after(s);
    return e;
}

}  // namespace kvc
