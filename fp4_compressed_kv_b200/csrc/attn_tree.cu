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

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// ----------------------------------------------------------------------------
// Any shape: a block is one node and 8 heads, a warp a head.  Keys go through
// shared memory as fp32 in chunks of 32 (rows padded by 16 bytes, so that 32
// lanes read 16 bytes of 32 rows without a conflict): lane = key for the
// logits, 8 sums of D / 8 products, and the chunk's softmax is one warp
// maximum; lane = channel for the values, each key's weight by a shuffle.
// Bound by a block's chain of chunks: with 512 + 64 channels, 64 heads and 640
// keys, 4 nodes and 16 both take 247 us (cold L2 285), 20 chunks of 12.4 us.
// By count, about half of a chunk's 23 K clocks are its reads of shared memory (8
// warps of 576 + 144 for the logits, 512 for the values), the rest waits between;
// a node's 8 blocks each dequantise all of its keys.  The products alone would
// take 19 us for 16 nodes at the fp32 rate.  Small entries (fp32, 8 heads of 64 +
// 16 channels, 64 entries and 32 tokens): 4 nodes 9.9 us, cold 13.1; 256 nodes
// 12.8, cold 15.8 (with lane = channel for the logits too, five shuffles a key,
// cold and launched by itself, 72 and 88 us, where this takes 18.5 and 20.5).
constexpr int kChunk = 32;

// Eight channels of a raw row.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(x[k] << 16);
        v[2 * k + 1] = __uint_as_float(x[k] & 0xFFFF0000u);
    }
}

template <typename T, int NI>  // NI: latent channels of a lane
__global__ void __launch_bounds__(256)
tree_simt_kernel(TreeArgs a, Shape sh, int H, int K, float scale_log2, int ue4m3) {
    extern __shared__ __align__(16) float smem[];
    __shared__ int kind[kChunk];  // record, -1, or -2 - raw key
    __shared__ int parents[kMaxTreeNodes], up[kMaxTreeNodes];
    __shared__ int s_depth, s_wl;
    const int D = sh.D, Dv = sh.Dv, np = D >> 3, pitch = D + 4;
    float* keys = smem;                    // [kChunk][pitch]
    float* qs = smem + kChunk * pitch;     // [8][D]
    pdl_wait();
    const int b = blockIdx.x / a.nodes, t = blockIdx.x - b * a.nodes;
    const int node = t * a.batch + b;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int h = blockIdx.y * 8 + w;
    for (int i = threadIdx.x; i <= t; i += blockDim.x)
        parents[i] = a.parents[(size_t)i * a.batch + b];
    const int n = a.n_entries[b];
    const bool len_ok = n >= 0 && n <= a.capacity;
    if (h < H)
        for (int c = lane; c < np; c += 32) {
            float v[8];
            load8(static_cast<const T*>(a.q) + ((size_t)node * H + h) * D + 8 * c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) qs[w * D + 8 * c + i] = v[i];
        }
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
    const int np_lat = Dv >> 3, lat_groups = (Dv + sh.G - 1) / sh.G;

    float o[NI];
    float m = -INFINITY, l = 0.f;  // l: this lane's keys
#pragma unroll
    for (int i = 0; i < NI; ++i) o[i] = 0.f;
    for (int c0 = 0; c0 < total; c0 += kChunk) {
        if (threadIdx.x < kChunk) {
            const int j = c0 + threadIdx.x;
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
        for (int p = threadIdx.x; p < kChunk * np; p += blockDim.x) {
            const int s = p / np, c = p - s * np;
            const int k = kind[s];
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (k >= 0) {
                const uint8_t* rec = a.records + ((size_t)b * a.capacity + k) * sh.rb;
                const int g = c < np_lat ? c / sh.lpg : lat_groups + (c - np_lat) / sh.lpg;
                e2m1x8_values(__ldg(reinterpret_cast<const uint32_t*>(rec) + c),
                              ue4m3 ? e4m3_to_f32(__ldg(rec + sh.code_bytes + g))
                                    : __ldg(reinterpret_cast<const float*>(rec + sh.code_bytes) + g),
                              v);
            } else if (k <= -2) {
                const int r = -2 - k;
                load8((r < wl ? static_cast<const T*>(a.window) + ((size_t)b * a.window_stride + r) * D
                              : static_cast<const T*>(a.draft) +
                                    ((size_t)up[depth - 1 - (r - wl)] * a.batch + b) * D) +
                          8 * c,
                      v);
            }
            float4* dst = reinterpret_cast<float4*>(keys + s * pitch + 8 * c);
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        __syncthreads();
        if (h < H) {
            float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            const float4* kr = reinterpret_cast<const float4*>(keys + lane * pitch);
            const float4* qr = reinterpret_cast<const float4*>(qs + w * D);
#pragma unroll 2
            for (int c = 0; c < 2 * np; c += 2) {
                const float4 k0 = kr[c], k1 = kr[c + 1], q0 = qr[c], q1 = qr[c + 1];
                s[0] = fmaf(q0.x, k0.x, s[0]), s[1] = fmaf(q0.y, k0.y, s[1]);
                s[2] = fmaf(q0.z, k0.z, s[2]), s[3] = fmaf(q0.w, k0.w, s[3]);
                s[4] = fmaf(q1.x, k1.x, s[4]), s[5] = fmaf(q1.y, k1.y, s[5]);
                s[6] = fmaf(q1.z, k1.z, s[6]), s[7] = fmaf(q1.w, k1.w, s[7]);
            }
            float x = (((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]))) * scale_log2;
            if (kind[lane] == -1) x = -INFINITY;
            float mx = x;
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float mn = fmaxf(m, mx);
            const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn);
            const float p = x == -INFINITY ? 0.f : exp2f(x - mn);
            l = l * alpha + p;
            m = mn;
#pragma unroll
            for (int i = 0; i < NI; ++i) o[i] *= alpha;
#pragma unroll 4
            for (int j = 0; j < kChunk; ++j) {
                const float pj = __shfl_sync(0xffffffffu, p, j);
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int d = lane + 32 * i;
                    if (d < Dv) o[i] = fmaf(pj, keys[j * pitch + d], o[i]);
                }
            }
        }
        __syncthreads();
    }
    if (h >= H) return;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    const float inv = l > 0.f ? 1.f / l : 0.f;
    T* op = static_cast<T*>(a.out) + ((size_t)node * H + h) * Dv;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int d = lane + 32 * i;
        if (d < Dv) put(op + d, l == 0.f ? 0.f : o[i] * inv);
    }
    if (lane == 0 && a.lse)
        a.lse[(size_t)node * H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename T, int NI>
cudaError_t launch_simt(const kvc_config& c, const Shape& sh, const TreeArgs& a, cudaStream_t s) {
    const size_t smem = ((size_t)kChunk * (sh.D + 4) + 8 * sh.D) * sizeof(float);
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(
            tree_simt_kernel<T, NI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
            (kChunk * (1024 + 4) + 8 * 1024) * (int)sizeof(float));
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const dim3 grid((unsigned)a.nodes * a.batch, (c.n_heads + 7) / 8);
    trace_before("tree_simt", s);
    const cudaError_t e =
        launch_pdl(tree_simt_kernel<T, NI>, grid, 256, smem, s, a, sh, c.n_heads, c.topk,
                   c.sm_scale * kLog2e, (int)(c.scale_fmt == KVC_SCALE_UE4M3));
    trace_after(s);
    return e;
}

template <typename T>
cudaError_t launch_simt_t(const kvc_config& c, const Shape& sh, const TreeArgs& a, cudaStream_t s) {
    if (sh.Dv <= 64) return launch_simt<T, 2>(c, sh, a, s);
    if (sh.Dv <= 256) return launch_simt<T, 8>(c, sh, a, s);
    if (sh.Dv <= 512) return launch_simt<T, 16>(c, sh, a, s);
    return launch_simt<T, 32>(c, sh, a, s);
}

}  // namespace

cudaError_t launch_tree(const kvc_config& c, const Shape& sh, const TreeArgs& a, cudaStream_t s) {
    if (tree_t128_supported(c, sh)) return launch_tree_t128(c, sh, a, s);
    return c.act_dtype == KVC_BF16 ? launch_simt_t<__nv_bfloat16>(c, sh, a, s)
                                   : launch_simt_t<float>(c, sh, a, s);
}

}  // namespace kvc
