// attn_tree.cu -- attention of a tree of drafted tokens over the compressed
// cache: every node attends over its selected entries and the sliding window
// of its own path.
//
// Method: "DeepSeek V1 到 V4.1-Flash，单 token 的 global KV 如何从 389,000 B
// 压缩到 890 B的？" (acejoy.com) part 3 breakthrough 2 (one 512 + 64 channel
// entry for all heads, values = the latent channels), breakthrough 4 (the
// selected entries plus a 128-token window), as for one token in
// attn_t128.cu; here T tokens of a sequence at once, each behind its own
// ancestors.
//
// Mathematics, for node t of sequence b with path root = a_1, ..., a_d = t:
// its raw keys are the last W rows of (window rows of b, draft rows a_1 ..
// a_d), its records those of topk[t][b]; one softmax of sm_scale q.k over
// both, values the first latent channels.
#include "kvc_internal.cuh"

namespace kvc {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Path of node t, walked by one thread over the parents of its sequence:
// up[k] = the ancestor k steps up (up[0] = t).  Returns the depth (1 at a
// root), or 0 for an absent node (its own parent, or an ancestor's, is -2 or
// no parent at all: outside [-1, own index)).
__device__ __forceinline__ int tree_path(const int* parents, int t, int* up, uint32_t* status) {
    int d = 0, at = t;
    for (;;) {
        up[d++] = at;
        const int p = parents[at];
        if (p == -1) return d;
        if (p < -1 || p >= at) {
            if (p != -2) set_status(status, KVC_DEV_BAD_INDEX);
            return 0;
        }
        at = p;
    }
}

// Window rows of sequence b (0 .. window_len), from the device lengths if given.
__device__ __forceinline__ int tree_window_len(const TreeArgs& a, int b) {
    if (!a.window_lens) return a.window_len;
    const int w = a.window_lens[b];
    if (w < 0 || w > a.window_len) {
        set_status(a.status, KVC_DEV_BAD_LENGTH);
        return 0;
    }
    return w;
}

__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t m = c & 7u;  // magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6
    const float mag = m < 4u ? 0.5f * (float)m : (float)(1u << (m >> 1)) * (1.0f + 0.5f * (m & 1u)) * 0.5f;
    return (c & 8u) ? -mag : mag;
}
__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// ----------------------------------------------------------------------------
// Any shape: block (8 heads, node); a warp is one head, the keys go through
// shared memory as fp32 in chunks of 32.
constexpr int kChunk = 32;

template <typename T>
__global__ void __launch_bounds__(256)
tree_simt_kernel(TreeArgs a, Shape sh, int H, int K, float scale_log2, int ue4m3) {
    extern __shared__ __align__(16) float keys[];  // [kChunk][D]
    __shared__ int kind[kChunk];                   // record, -1, or -2 - raw key
    __shared__ int parents[kMaxTreeNodes], up[kMaxTreeNodes];
    __shared__ int s_depth, s_wl;
    pdl_wait();
    const int b = blockIdx.x / a.nodes, t = blockIdx.x - b * a.nodes;
    const int node = t * a.batch + b;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int h = blockIdx.y * 8 + w;
    const int D = sh.D, Dv = sh.Dv;
    for (int i = threadIdx.x; i < a.nodes; i += blockDim.x)
        parents[i] = a.parents[(size_t)i * a.batch + b];
    const int n = a.n_entries[b];
    const bool len_ok = n >= 0 && n <= a.capacity;
    __syncthreads();
    if (threadIdx.x == 0) {
        if (!len_ok) set_status(a.status, KVC_DEV_BAD_LENGTH);
        s_depth = tree_path(parents, t, up, a.status);
        s_wl = tree_window_len(a, b);
    }
    __syncthreads();
    const int depth = s_depth, wl = s_wl;
    const int raw = depth ? min(a.window_stride, wl + depth) : 0;  // raw keys of this node
    const int skip = wl + depth - raw;                              // older ones out of its window
    const int total = depth ? K + raw : 0;
    const int32_t* sel = a.topk_idx + (a.topk_shared ? (size_t)b : (size_t)node) * K;

    float q[32], o[32];
    float m = -INFINITY, l = 0.f;
    const T* qp = static_cast<const T*>(a.q) + ((size_t)node * H + (h < H ? h : 0)) * D;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int d = lane + 32 * i;
        q[i] = d < D ? as_f32(qp[d]) : 0.f;
        o[i] = 0.f;
    }
    for (int c = 0; c < total; c += kChunk) {
        if (threadIdx.x < kChunk) {
            const int j = c + threadIdx.x;
            int k = -1;
            if (j < K) {
                const int idx = sel[j];
                if (len_ok && idx >= 0 && idx < n) k = idx;
                else if (len_ok && idx != -1 && blockIdx.y == 0) set_status(a.status, KVC_DEV_BAD_INDEX);
            } else if (j < total) {
                k = -2 - (skip + j - K);
            }
            kind[threadIdx.x] = k;
        }
        __syncthreads();
        for (int p = threadIdx.x; p < kChunk * D; p += blockDim.x) {
            const int s = p / D, d = p - s * D;
            const int k = kind[s];
            float v = 0.f;
            if (k >= 0) {
                const uint8_t* rec = a.records + ((size_t)b * a.capacity + k) * sh.rb;
                const uint32_t code = (rec[d >> 1] >> ((d & 1) * 4)) & 15u;
                const int g = d < Dv ? (d >> 3) / sh.lpg
                                     : (Dv + sh.G - 1) / sh.G + ((d - Dv) >> 3) / sh.lpg;
                const float sc = ue4m3 ? e4m3_to_f32(rec[sh.code_bytes + g])
                                       : reinterpret_cast<const float*>(rec + sh.code_bytes)[g];
                v = e2m1_value(code) * sc;
            } else if (k <= -2) {
                const int r = -2 - k;
                const T* row = r < wl ? static_cast<const T*>(a.window) +
                                            ((size_t)b * a.window_stride + r) * D
                                      : static_cast<const T*>(a.draft) +
                                            ((size_t)up[depth - 1 - (r - wl)] * a.batch + b) * D;
                v = as_f32(row[d]);
            }
            keys[p] = v;
        }
        __syncthreads();
        if (h < H) {
            for (int s = 0; s < kChunk; ++s) {
                if (kind[s] == -1) continue;
                const float* kr = keys + s * D;
                float part = 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int d = lane + 32 * i;
                    if (d < D) part = fmaf(q[i], kr[d], part);
                }
#pragma unroll
                for (int off = 16; off >= 1; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
                const float x = part * scale_log2;
                const float mn = fmaxf(m, x);
                const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn);
                const float p = mn == -INFINITY ? 0.f : exp2f(x - mn);
                l = l * alpha + p;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int d = lane + 32 * i;
                    if (d < Dv) o[i] = fmaf(p, kr[d], o[i] * alpha);
                }
                m = mn;
            }
        }
        __syncthreads();
    }
    if (h >= H) return;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    T* op = static_cast<T*>(a.out) + ((size_t)node * H + h) * Dv;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int d = lane + 32 * i;
        if (d < Dv) put(op + d, l == 0.f ? 0.f : o[i] * inv);
    }
    if (lane == 0 && a.lse)
        a.lse[(size_t)node * H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

cudaError_t launch_tree_simt(const kvc_config& c, const Shape& sh, const TreeArgs& a,
                             cudaStream_t s) {
    const size_t smem = (size_t)kChunk * sh.D * sizeof(float);
    const bool bf = c.act_dtype == KVC_BF16;
    static bool attr_set[64][2] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev][bf]) {
        const cudaError_t e =
            bf ? cudaFuncSetAttribute(tree_simt_kernel<__nv_bfloat16>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, kChunk * 1024 * 4)
               : cudaFuncSetAttribute(tree_simt_kernel<float>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, kChunk * 1024 * 4);
        if (e != cudaSuccess) return e;
        attr_set[dev][bf] = true;
    }
    const dim3 grid((unsigned)a.nodes * a.batch, (c.n_heads + 7) / 8);
    const float scale_log2 = c.sm_scale * kLog2e;
    const int ue4m3 = c.scale_fmt == KVC_SCALE_UE4M3;
    trace_before("tree_simt", s);
    const cudaError_t e =
        bf ? launch_pdl(tree_simt_kernel<__nv_bfloat16>, grid, 256, smem, s, a, sh, c.n_heads,
                        c.topk, scale_log2, ue4m3)
           : launch_pdl(tree_simt_kernel<float>, grid, 256, smem, s, a, sh, c.n_heads, c.topk,
                        scale_log2, ue4m3);
    trace_after(s);
    return e;
}

}  // namespace

cudaError_t launch_tree(const kvc_config& c, const Shape& sh, const TreeArgs& a, cudaStream_t s) {
    return tree_t128_supported(c, sh) ? launch_tree_t128(c, sh, a, s) : launch_tree_simt(c, sh, a, s);
}

}  // namespace kvc
