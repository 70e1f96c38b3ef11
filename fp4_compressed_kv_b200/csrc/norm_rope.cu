// norm_rope.cu -- RMS norms of query and key rows for each head, with the
// position rotation of their RoPE channels in the same pass.
//
// Method: "DeepSeek V1 到 V4.1-Flash，单 token 的 global KV 如何从 389,000 B
// 压缩到 890 B的？" (acejoy.com) part 3 breakthrough 2 (an entry is 512 latent
// channels and 64 RoPE channels, shared by every head), part 4 "P4 main KV"
// (the RMS norm bounds the latent before it is quantised).
//
// Mathematics, for one row x of D channels and a norm over the first w of
// them:  y_c = x_c / sqrt(sum_{c < w} x_c^2 / w + eps) * g_c  (c < w; y = x
// behind them), then for each pair (a, b) of RoPE channels and its angle
// t = position * inv_freq:  (a cos t - b sin t, a sin t + b cos t).  Sums and
// products are fp32, rounded once to the row's type.  The angle is formed and
// reduced to [-pi, pi] in fp64: at position 10^6 the fp32 product alone would
// be off by 0.06.
//
// One row is read once and written once; nothing else moves more than a few
// per cent of that, so the bound is HBM (prompt) or the launch (a few rows).
// Eight lanes hold a row (piece l + 8 i of 8 latent channels in lane l: a
// warp's 16-byte accesses cover four runs of 128 bytes; RoPE channels in units
// of four pairs), so the sum is three shuffles and 512 + 64 channels fill
// every lane.  A warp takes four consecutive rows at a time and `run` such
// fours: heads of one token share its angles, one sine and cosine a lane.
// Measured (in a graph of twenty calls; "cold": on twenty sets of rows, with L2
// swept before): a prompt of 8192 tokens of 64 + 1 rows of 576 bf16 channels in
// 190 us, cold 193, 6.4 TB/s (0.98 of the measured copy rate), 4096 of fp32 195,
// cold 197; 4 tokens 3.6, cold 5.8.  Between them waves count: 96 registers let
// 740 CTAs of 16 rows be resident, so 180 tokens (732 CTAs) take 6.4 us and 184
// (748) 8.5, 256 (1,040) 10.1, cold 13.9.
#include "kvc_internal.cuh"

namespace kvc {
namespace {

constexpr int NT = 128;

// Eight channels held as loaded (16 bytes of bf16, 32 of fp32).
template <typename T>
struct Raw8 {  // (values: pairs of fp32 for the packed operations)
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* src) {
#pragma unroll
        for (int u = 0; u < (int)sizeof(T) / 2; ++u) w[u] = reinterpret_cast<const uint4*>(src)[u];
    }
    __device__ __forceinline__ void values(float2 (&v)[4]) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t x[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = make_float2(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xFFFF0000u));
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                v[2 * k] = make_float2(__uint_as_float(w[k].x), __uint_as_float(w[k].y));
                v[2 * k + 1] = make_float2(__uint_as_float(w[k].z), __uint_as_float(w[k].w));
            }
        }
    }
};
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float2 (&v)[4]) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(bf16x2(v[0].x, v[0].y), bf16x2(v[1].x, v[1].y),
                                                bf16x2(v[2].x, v[2].y), bf16x2(v[3].x, v[3].y));
}
__device__ __forceinline__ void store8(float* dst, const float2 (&v)[4]) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}
// Two fp32 products (and sums) by one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mov.b64 z, {%0, %1};\n\tfma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "+f"(c.x), "+f"(c.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return c;
}

// A rotation unit: four pairs (x, y) of RoPE channels, unit j holding pairs
// 4 j .. 4 j + 3, read and written by one lane only (so rows may be rotated in
// place).  Its channels are 8 j .. 8 j + 7 in the pairs layout, 4 j .. 4 j + 3
// and as many half the RoPE channels further on in the halves layout.
struct Unit {
    float x[4], y[4];
};
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    const float4 w = *reinterpret_cast<const float4*>(p);
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <typename T>  // rope: the row's first RoPE channel
__device__ __forceinline__ void load_unit(const T* rope, int j, int half, int pairs, Unit& u) {
    if (pairs) {
        float a[4], b[4];
        load4(rope + 8 * j, a);
        load4(rope + 8 * j + 4, b);
        u.x[0] = a[0], u.y[0] = a[1], u.x[1] = a[2], u.y[1] = a[3];
        u.x[2] = b[0], u.y[2] = b[1], u.x[3] = b[2], u.y[3] = b[3];
    } else {
        load4(rope + 4 * j, u.x);
        load4(rope + half + 4 * j, u.y);
    }
}
template <typename T>
__device__ __forceinline__ void store_unit(T* rope, int j, int half, int pairs, const Unit& u) {
    if (pairs) {
        const float a[4] = {u.x[0], u.y[0], u.x[1], u.y[1]}, b[4] = {u.x[2], u.y[2], u.x[3], u.y[3]};
        store4(rope + 8 * j, a);
        store4(rope + 8 * j + 4, b);
    } else {
        store4(rope + 4 * j, u.x);
        store4(rope + half + 4 * j, u.y);
    }
}
__device__ __forceinline__ float square_sum(const Unit& u) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fmaf(u.x[i], u.x[i], fmaf(u.y[i], u.y[i], s));
    return s;
}
// cos and sin of position * inv_freq: the product in whole turns, its turns
// taken off in fp64 (2^-53 of the angle), the rest of a turn to fp32.
__device__ __forceinline__ void turn(int pos, float freq, float& c, float& s) {
    const double turns = (double)pos * (double)freq * 0.15915494309189535;  // 1 / (2 pi)
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
}

// The angles of a token that a lane holds (its first rotation unit).
struct Angles {
    int tok = -1;
    float c[4], s[4];
};

// One row by a group of eight lanes (l: lane of the group): from src to dst,
// which may be the same; nothing is written without `live`.  All four groups of
// the warp call it together.  FULL: every lane has NPL pieces and one unit.
template <typename T, int NPL, bool FULL>  // NPL: pieces of 8 latent channels a lane holds
__device__ __forceinline__ void do_row(const NormRopeArgs& a, bool is_k, int tok, const T* src,
                                       T* dst, bool live, int l, unsigned group_mask, Angles& held) {
    const int np = a.latent >> 3, half = a.rope >> 1, units = a.rope >> 3;
    const float* gain = is_k ? a.k_gain : a.q_gain;
    const int width = is_k ? a.k_width : a.q_width;
    Raw8<T> raw[NPL];
    Unit first = {};
    src += 8 * l;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        if (FULL || l + 8 * i < np) raw[i].load(src + 64 * i);
    src += a.latent - 8 * l;  // from here on the row's RoPE channels
    if (FULL || l < units) load_unit(src, l, half, a.pairs, first);
    if (__any_sync(0xffffffffu, held.tok != tok)) {  // while the row is on its way
        const int pos = a.positions[tok];
        const bool same = __all_sync(0xffffffffu, __shfl_sync(0xffffffffu, tok, 0) == tok);
        if (same && units <= 8) {
            // a pair a lane; lane l of every group takes pairs 4 l .. 4 l + 3
            const int lane = threadIdx.x & 31;
            float c = 1.f, sn = 0.f;
            if (lane < half) turn(pos, __ldg(a.inv_freq + lane), c, sn);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                held.c[i] = __shfl_sync(0xffffffffu, c, 4 * l + i);
                held.s[i] = __shfl_sync(0xffffffffu, sn, 4 * l + i);
            }
        } else if (l < units) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                turn(pos, __ldg(a.inv_freq + 4 * l + i), held.c[i], held.s[i]);
        }
        held.tok = tok;
    }
    float inv = 1.f;
    if (width) {
        float2 s2[2] = {};
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (FULL || l + 8 * i < np) {
                float2 v[4];
                raw[i].values(v);
#pragma unroll
                for (int j = 0; j < 4; ++j) s2[j & 1] = fma2(v[j], v[j], s2[j & 1]);
            }
        float ss = (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
        if (width > a.latent) {
            ss += square_sum(first);
            if (!FULL)
                for (int j = l + 8; j < units; j += 8) {
                    Unit u;
                    load_unit(src, j, half, a.pairs, u);
                    ss += square_sum(u);
                }
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(group_mask, ss, o);
        inv = 1.0f / sqrtf(ss / (float)width + a.eps);
        if (l == 0 && live && !(ss < INFINITY && inv < INFINITY))
            set_status(a.status, KVC_DEV_NONFINITE);
    }
    if (!live) return;
    const float2 inv2 = make_float2(inv, inv);
    T* out = dst + 8 * l;
    if (width && gain) {
        const float* gl = gain + 8 * l;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            if (!FULL && l + 8 * i >= np) continue;
            float2 v[4];
            raw[i].values(v);
            const float4 g0 = __ldg(reinterpret_cast<const float4*>(gl + 64 * i));
            const float4 g1 = __ldg(reinterpret_cast<const float4*>(gl + 64 * i) + 1);
            v[0] = mul2(v[0], mul2(inv2, make_float2(g0.x, g0.y)));
            v[1] = mul2(v[1], mul2(inv2, make_float2(g0.z, g0.w)));
            v[2] = mul2(v[2], mul2(inv2, make_float2(g1.x, g1.y)));
            v[3] = mul2(v[3], mul2(inv2, make_float2(g1.z, g1.w)));
            store8(out + 64 * i, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            if (!FULL && l + 8 * i >= np) continue;
            float2 v[4];
            raw[i].values(v);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], inv2);  // (no norm: times 1)
            store8(out + 64 * i, v);
        }
    }
    for (int j = l; FULL ? j == l : j < units; j += 8) {
        Unit u = first;
        float c[4], s[4];
        if (FULL || j == l) {
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = held.c[i], s[i] = held.s[i];
        } else {  // more than 64 RoPE channels
            load_unit(src, j, half, a.pairs, u);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                turn(a.positions[tok], __ldg(a.inv_freq + 4 * j + i), c[i], s[i]);
        }
        if (width > a.latent) {
            Unit g;
            if (gain) {
                load_unit(gain + a.latent, j, half, a.pairs, g);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) g.x[i] = g.y[i] = 1.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) u.x[i] *= inv * g.x[i], u.y[i] *= inv * g.y[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = u.x[i], y = u.y[i];
            u.x[i] = x * c[i] - y * s[i];
            u.y[i] = x * s[i] + y * c[i];
        }
        store_unit(dst + a.latent, j, half, a.pairs, u);
    }
}

// Rows are numbered queries first, token by token, then keys; a warp takes
// rows 4 run w .. 4 run (w + 1) - 1, one of four to each group of eight lanes.
template <typename T, int NPL, bool FULL>
__global__ void __launch_bounds__(NT)
norm_rope_kernel(NormRopeArgs a, int run) {
    pdl_wait();
    const int l = threadIdx.x & 7, g = (threadIdx.x & 31) >> 3;
    const unsigned group_mask = 0xFFu << (threadIdx.x & 24);
    const long long nq = (long long)a.n_rows * a.q_heads;
    const long long total = nq + (a.k ? a.n_rows : 0);
    const long long w = (long long)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
    long long r = w * run * 4 + g;
    Angles held;
    for (int it = 0; it < run; ++it, r += 4) {
        if (r - g >= total) break;
        // (a group past the end reads the last row, so that all four stay together)
        const long long rr = min(r, total - 1);
        const bool is_k = rr >= nq;
        int tok, head = 0;
        if (is_k) {
            tok = (int)(rr - nq);
        } else if (nq < (1ll << 31)) {
            tok = (int)((unsigned)rr / (unsigned)a.q_heads);
            head = (int)((unsigned)rr - (unsigned)tok * (unsigned)a.q_heads);
        } else {
            tok = (int)(rr / a.q_heads);
            head = (int)(rr - (long long)tok * a.q_heads);
        }
        const T* src = is_k ? static_cast<const T*>(a.k) + tok * a.k_stride
                            : static_cast<const T*>(a.q) + tok * a.q_stride + (long long)head * a.D;
        T* dst = is_k ? static_cast<T*>(a.k_out) + (long long)tok * a.D
                      : static_cast<T*>(a.q_out) + ((long long)tok * a.q_heads + head) * a.D;
        do_row<T, NPL, FULL>(a, is_k, tok, src, dst, r < total, l, group_mask, held);
        __syncwarp();
    }
}

template <typename T, int NPL>
cudaError_t launch_n(const NormRopeArgs& a, cudaStream_t s) {
    const long long total = (long long)a.n_rows * (a.q_heads + (a.k ? 1 : 0));
    // fours of a warp: heads of a token share its angles, once the grid fills
    // the device several times over anyway (8192 tokens of 65 rows of 576 bf16
    // channels: runs of 1, 4, 16 take 193.1, 191.3, 196.0 us)
    int run = 1;
    while (run < 4 && total / (8 * run) >= 148ll * 16 * 4) run *= 2;
    const long long warps = (total + 4ll * run - 1) / (4ll * run);
    const unsigned grid = (unsigned)((warps + NT / 32 - 1) / (NT / 32));
    // every lane filled: no predicates (191.3 against 207.4 us there)
    const bool full = a.latent == 64 * NPL && a.rope == 64;
    trace_before("norm_rope", s);
    const cudaError_t e = full ? launch_pdl(norm_rope_kernel<T, NPL, true>, grid, NT, 0, s, a, run)
                               : launch_pdl(norm_rope_kernel<T, NPL, false>, grid, NT, 0, s, a, run);
    trace_after(s);
    return e;
}

template <typename T>
cudaError_t launch_t(const NormRopeArgs& a, cudaStream_t s) {
    const int npl = (a.latent / 8 + 7) / 8;
    if (npl <= 1) return launch_n<T, 1>(a, s);
    if (npl <= 2) return launch_n<T, 2>(a, s);
    if (npl <= 4) return launch_n<T, 4>(a, s);
    if (npl <= 8) return launch_n<T, 8>(a, s);
    return launch_n<T, 16>(a, s);
}

}  // namespace

cudaError_t launch_norm_rope(const kvc_config& c, const NormRopeArgs& a, cudaStream_t s) {
    return c.act_dtype == KVC_BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace kvc
