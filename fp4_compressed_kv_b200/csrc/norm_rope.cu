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
// every lane.  A group of eight lanes takes `rpg` consecutive rows: heads of
// one token share its angles.
#include "kvc_internal.cuh"

namespace kvc {
namespace {

constexpr int NT = 256;

// Eight channels held as loaded (16 bytes of bf16, 32 of fp32).
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* src) {
#pragma unroll
        for (int u = 0; u < (int)sizeof(T) / 2; ++u) w[u] = reinterpret_cast<const uint4*>(src)[u];
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t x[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = __uint_as_float(x[k] << 16);
                v[2 * k + 1] = __uint_as_float(x[k] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                v[4 * k] = __uint_as_float(w[k].x);
                v[4 * k + 1] = __uint_as_float(w[k].y);
                v[4 * k + 2] = __uint_as_float(w[k].z);
                v[4 * k + 3] = __uint_as_float(w[k].w);
            }
        }
    }
};
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]),
                                                bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* dst, const float (&v)[8]) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
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

template <typename T, int NPL>  // NPL: pieces of 8 latent channels a lane holds
__global__ void __launch_bounds__(NT)
norm_rope_kernel(NormRopeArgs a, int rpg) {
    // (no early launch of dependents: kvc_pack reads its tokens before it waits
    // for the kernel in front of it, and these rows may be its tokens)
    pdl_wait();
    const int l = threadIdx.x & 7;
    const unsigned group_mask = 0xFFu << (threadIdx.x & 24);
    const long long nq = (long long)a.n_rows * a.q_heads;
    const long long total = nq + (a.k ? a.n_rows : 0);
    const long long r0 = ((long long)blockIdx.x * (NT / 8) + (threadIdx.x >> 3)) * rpg;
    const int np = a.latent >> 3, half = a.rope >> 1, units = a.rope >> 3;
    int held = -1;  // token whose angles cs / sn hold (this lane's first unit)
    float cs[4], sn[4];
    for (long long r = r0; r < min(r0 + rpg, total); ++r) {
        const bool is_k = r >= nq;
        const int tok = is_k ? (int)(r - nq) : (int)(r / a.q_heads);
        const int head = is_k ? 0 : (int)(r - (long long)tok * a.q_heads);
        const T* src = is_k ? static_cast<const T*>(a.k) + tok * a.k_stride
                            : static_cast<const T*>(a.q) + tok * a.q_stride + (long long)head * a.D;
        T* dst = is_k ? static_cast<T*>(a.k_out) + (long long)tok * a.D
                      : static_cast<T*>(a.q_out) + ((long long)tok * a.q_heads + head) * a.D;
        const float* gain = is_k ? a.k_gain : a.q_gain;
        const int width = is_k ? a.k_width : a.q_width;
        Raw8<T> raw[NPL];
        Unit first = {};
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (l + 8 * i < np) raw[i].load(src + 8 * (l + 8 * i));
        if (l < units) load_unit(src + a.latent, l, half, a.pairs, first);
        if (held != tok && l < units) {  // while the row is on its way
            const int pos = a.positions[tok];
#pragma unroll
            for (int i = 0; i < 4; ++i) turn(pos, __ldg(a.inv_freq + 4 * l + i), cs[i], sn[i]);
            held = tok;
        }
        float inv = 1.f;
        if (width) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (l + 8 * i < np) {
                    float v[8];
                    raw[i].values(v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
                }
            if (width > a.latent) {
                ss += square_sum(first);
                for (int j = l + 8; j < units; j += 8) {
                    Unit u;
                    load_unit(src + a.latent, j, half, a.pairs, u);
                    ss += square_sum(u);
                }
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(group_mask, ss, o);
            inv = 1.0f / sqrtf(ss / (float)width + a.eps);
            if (l == 0 && !(ss < INFINITY)) set_status(a.status, KVC_DEV_NONFINITE);
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int piece = l + 8 * i;
            if (piece >= np) continue;
            float v[8];
            raw[i].values(v);
            if (width) {
                float g[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
                if (gain) {
                    const float4 g0 = __ldg(reinterpret_cast<const float4*>(gain + 8 * piece));
                    const float4 g1 = __ldg(reinterpret_cast<const float4*>(gain + 8 * piece) + 1);
                    g[0] = g0.x, g[1] = g0.y, g[2] = g0.z, g[3] = g0.w;
                    g[4] = g1.x, g[5] = g1.y, g[6] = g1.z, g[7] = g1.w;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= inv * g[j];
            }
            store8(dst + 8 * piece, v);
        }
        for (int j = l; j < units; j += 8) {
            Unit u = first;
            float c[4], s[4];
            if (j == l) {
#pragma unroll
                for (int i = 0; i < 4; ++i) c[i] = cs[i], s[i] = sn[i];
            } else {  // more than 64 RoPE channels
                load_unit(src + a.latent, j, half, a.pairs, u);
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
}

template <typename T>
cudaError_t launch_t(const NormRopeArgs& a, cudaStream_t s) {
    const long long total = (long long)a.n_rows * (a.q_heads + (a.k ? 1 : 0));
    // rows of one lane group: several heads of a token share its angles once
    // the grid fills the device anyway
    int rpg = 1;
    while (rpg < 8 && total / (rpg * 2) >= 148ll * 8 * (NT / 8)) rpg *= 2;
    const long long groups = (total + rpg - 1) / rpg;
    const unsigned grid = (unsigned)((groups + NT / 8 - 1) / (NT / 8));
    const int npl = (a.latent / 8 + 7) / 8;
    trace_before("norm_rope", s);
    cudaError_t e;
    if (npl <= 1) e = launch_pdl(norm_rope_kernel<T, 1>, grid, NT, 0, s, a, rpg);
    else if (npl <= 2) e = launch_pdl(norm_rope_kernel<T, 2>, grid, NT, 0, s, a, rpg);
    else if (npl <= 4) e = launch_pdl(norm_rope_kernel<T, 4>, grid, NT, 0, s, a, rpg);
    else if (npl <= 8) e = launch_pdl(norm_rope_kernel<T, 8>, grid, NT, 0, s, a, rpg);
    else e = launch_pdl(norm_rope_kernel<T, 16>, grid, NT, 0, s, a, rpg);
    trace_after(s);
    return e;
}

}  // namespace

cudaError_t launch_norm_rope(const kvc_config& c, const NormRopeArgs& a, cudaStream_t s) {
    return c.act_dtype == KVC_BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace kvc
