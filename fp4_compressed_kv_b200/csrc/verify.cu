// verify.cu -- a tree of drafted tokens verified against the target's
// probabilities from given random numbers.
//
// Mathematics.  Node 0 is the root (accepted), p_c and q_c the target's and
// the draft's probabilities behind node c.  At the deepest accepted node c its
// children are tried in index order, each drawn from q_c: child x is accepted
// where u m q(x) < r(x), with the residual r and its mass m starting at p_c
// and 1; a rejection replaces r by max(r - m q, 0) and m by its sum.  Since
// max(max(p - a q, 0) - b q, 0) = max(p - (a + b) q, 0) for a, b, q >= 0, the
// residual after any number of rejections is max(p - S q, 0) with S the sum of
// the masses so far: one running number, and one pass over the two rows for
// each rejection.  Without draft probabilities a child was chosen for certain
// (q(x) = 1): it is accepted where u m < r(x), and a rejection takes p(x) out
// of r and m.  The next token is drawn from the residual of the last accepted
// node: the lowest i whose running sum passes v times the whole sum.
//
// Everything that decides (products, masses, running sums) is fp64: the
// products of two fp32 numbers are exact and a border is moved by 10^-16 of
// the mass, where fp32 sums of 10^5 terms would move it past whole tokens.
//
// A sequence is one cluster of CTAs, each with a contiguous share of the
// vocabulary in chunks of 1024; sums of the shares are exchanged over
// distributed shared memory, so every CTA walks the tree alike.  What each
// node's walk looks up (token, parent, u, p(x), q(x)) is loaded by one thread
// a node at the start.  Bound: the rows of the last accepted node and of every
// node with a rejection, read from HBM.
#include "kvc_internal.cuh"

namespace kvc {
namespace {

constexpr int NT = 512, NW = NT / 32;
constexpr int CHUNK = 1024;   // vocabulary entries of one warp's share of a pass
constexpr int MAX_CLUSTER = 8;

__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// A probability as it counts: NaN, infinities and negative values are 0.
__device__ __forceinline__ float counts(float x, bool& bad) {
    const bool ok = x >= 0.f && x < INFINITY;
    bad |= !ok && !(x < 0.f && x > -INFINITY);
    return ok ? x : 0.f;
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ double warp_scan(double x, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Entries e .. e + 3 of a row as floats; past the vocabulary 0.
template <typename T, bool VEC>
__device__ __forceinline__ void load4(const T* row, int e, int vocab, float (&v)[4]) {
    if constexpr (VEC) {
        if (e + 4 <= vocab) {
            if constexpr (sizeof(T) == 4) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(row + e));
                v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
            } else {
                const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + e));
                v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
                v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = e + j < vocab ? as_f32(row[e + j]) : 0.f;
}

struct NodeFacts {
    int parent, token;
    float u, p, q;  // q: 1 without draft probabilities
};

// The residual of 4 entries: max(p - S q, 0), or p without the rejected tokens.
struct Residual {
    double S;
    const int* gone;  // rejected tokens (no draft probabilities)
    int n_gone;
};

// Residual values of a chunk's entries e = c0 + 4 lane + 128 i + j, summed
// into the warp's total; r receives them when given.
template <typename T, bool VEC>
__device__ __forceinline__ double chunk_pass(const T* p, const T* q, int c0, int vocab,
                                             const Residual& res, int lane, bool& bad, double* r) {
    double sum = 0.0;
    bool any_gone = false;
    for (int g = 0; g < res.n_gone; ++g)
        any_gone |= res.gone[g] >= c0 && res.gone[g] < c0 + CHUNK;
    float pv[8][4], qv[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        load4<T, VEC>(p, c0 + 4 * lane + 128 * i, vocab, pv[i]);
        if (q) load4<T, VEC>(q, c0 + 4 * lane + 128 * i, vocab, qv[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = c0 + 4 * lane + 128 * i + j;
            double x = (double)counts(pv[i][j], bad);
            if (q) x = fmax(fma(-res.S, (double)counts(qv[i][j], bad), x), 0.0);
            if (any_gone)
                for (int g = 0; g < res.n_gone; ++g)
                    if (res.gone[g] == e) x = 0.0;
            if (r) r[(e - c0) + ((e - c0) >> 5)] = x;
            sum += x;
        }
    return warp_sum(sum);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(NT)
verify_kernel(VerifyArgs a, int cluster, int chunks_per_cta) {
    extern __shared__ __align__(16) unsigned char smem[];
    NodeFacts* facts = reinterpret_cast<NodeFacts*>(smem);               // [nodes]
    int* gone = reinterpret_cast<int*>(facts + a.nodes);                 // [nodes]
    double* csum = reinterpret_cast<double*>(
        smem + ((a.nodes * (sizeof(NodeFacts) + 4) + 15) & ~(size_t)15));  // [chunks_per_cta]
    double* rbuf = csum + chunks_per_cta;                                // [CHUNK + CHUNK / 32]
    __shared__ double share[2][MAX_CLUSTER];  // every CTA's sum of the pass, by its parity
    __shared__ double wsum[NW];
    const int b = blockIdx.x / cluster, rank = blockIdx.x - b * cluster;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T* pb = static_cast<const T*>(a.p);
    const T* qb = static_cast<const T*>(a.q);
    bool bad = false;
    pdl_wait();
    for (int t = tid; t < a.nodes; t += NT) {
        NodeFacts f;
        f.parent = a.parents[(size_t)t * a.batch + b];
        f.token = a.tokens[(size_t)t * a.batch + b];
        f.u = a.u[(size_t)t * a.batch + b];
        f.p = 0.f;
        f.q = 1.f;
        const bool is_child = t > 0 && f.parent >= 0 && f.parent < t;
        if (t > 0 && !is_child && f.parent != -1 && f.parent != -2 && rank == 0)
            set_status(a.status, KVC_DEV_BAD_INDEX);
        if (!is_child) f.parent = -1;
        if (is_child && (f.token < 0 || f.token >= a.vocab)) {
            if (rank == 0) set_status(a.status, KVC_DEV_BAD_INDEX);
            f.parent = -1;
        } else if (is_child) {
            const size_t row = (size_t)f.parent * a.batch + b;
            f.p = counts(as_f32(pb[row * a.p_ld + f.token]), bad);
            if (qb) f.q = counts(as_f32(qb[row * a.q_ld + f.token]), bad);
        }
        if (t == 0) f.parent = a.parents[b] == -2 ? -2 : -1;
        facts[t] = f;
    }
    // the facts are in place, and every CTA of the cluster runs (its shared
    // memory may be written)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    const bool absent = facts[0].parent == -2;  // a sequence without a tree

    int cur = 0, n_path = 1, n_gone = 0, passes = 0;
    double S = 0.0, m = 1.0;
    bool summed = false;  // csum and share hold the residual of `cur` at S
    const int chunk_lo = rank * chunks_per_cta;
    const int n_chunks = min(chunks_per_cta, (a.vocab + CHUNK - 1) / CHUNK - chunk_lo);
    // One pass over this CTA's share of the residual; returns its whole mass.
    auto pass = [&](bool use_q) -> double {
        const size_t row = (size_t)cur * a.batch + b;
        const Residual res = {S, gone, n_gone};
        double mine = 0.0;
        for (int c = warp; c < n_chunks; c += NW) {
            const double s = chunk_pass<T, VEC>(pb + row * a.p_ld,
                                                use_q ? qb + row * a.q_ld : nullptr,
                                                (chunk_lo + c) * CHUNK, a.vocab, res, lane, bad,
                                                nullptr);
            if (lane == 0) csum[c] = s;
            mine += s;
        }
        if (lane == 0) wsum[warp] = mine;
        __syncthreads();
        const int par = passes & 1;
        ++passes;
        if (warp == 0) {
            double t = lane < NW ? wsum[lane] : 0.0;
            t = warp_sum(t);
            if (lane < cluster) {
                uint32_t dst;
                const uint32_t src = (uint32_t)__cvta_generic_to_shared(&share[par][rank]);
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(src), "r"(lane));
                asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(dst), "d"(t) : "memory");
            }
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                     "barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
        double sum = 0.0;
        for (int r = 0; r < cluster; ++r) sum += share[par][r];
        return sum;
    };

    if (rank == 0 && tid == 0 && !absent) a.path[(size_t)b * a.nodes] = 0;
    bool over = false;  // the residual is empty: no further sibling is tried
    if (!absent)
        for (int t = 1; t < a.nodes; ++t) {
            const NodeFacts f = facts[t];
            if (f.parent != cur || over) continue;
            double rx = (double)f.p;
            if (qb) {
                rx = fmax(fma(-S, (double)f.q, rx), 0.0);
            } else {
                for (int g = 0; g < n_gone; ++g)
                    if (gone[g] == f.token) rx = 0.0;
            }
            if ((double)f.u * m * (double)f.q < rx) {
                if (rank == 0 && tid == 0) a.path[(size_t)b * a.nodes + n_path] = t;
                cur = t;
                ++n_path;
                S = 0.0;
                m = 1.0;
                n_gone = 0;
                summed = false;
            } else if (qb) {
                S += m;
                m = pass(true);
                summed = true;
                over = !(m > 0.0);
            } else {
                m = fmax(m - rx, 0.0);
                __syncthreads();  // every thread has read the list
                if (tid == 0) gone[n_gone] = f.token;
                ++n_gone;
                __syncthreads();
            }
        }
    // the residual's sum at the last accepted node; an empty one gives way to
    // the target's own probabilities
    bool use_q = qb && S > 0.0;
    if (!absent) {
        if (!summed) m = pass(use_q);
        if (!(m > 0.0)) {
            n_gone = 0;
            use_q = false;
            m = pass(false);
        }
        // the CTA whose share the draw falls into (the last one with any mass
        // where rounding leaves none), its chunk, and the entry
        const double* sh = share[(passes - 1) & 1];
        const double target = (double)a.v[b] * m;
        double before = 0.0;
        int owner = -1;
        for (int r = 0; r < cluster; ++r) {
            if (!(sh[r] > 0.0)) continue;
            if (owner >= 0) before += sh[owner];
            owner = r;
            if (before + sh[r] > target) break;
        }
        if (owner < 0) {
            if (rank == 0 && tid == 0) {
                a.next[b] = -1;
                bad = true;
            }
        } else if (owner == rank && warp == 0) {
            int chunk = -1;
            double base = before;   // running sum in front of `chunk`
            double run = before;
            for (int c0 = 0; c0 < n_chunks; c0 += 32) {
                const double mine = c0 + lane < n_chunks ? csum[c0 + lane] : 0.0;
                const double upto = run + warp_scan(mine, lane);
                const unsigned hit = __ballot_sync(0xffffffffu, mine > 0.0 && upto > target);
                const unsigned pos = __ballot_sync(0xffffffffu, mine > 0.0);
                const int at = hit ? __ffs(hit) - 1 : (pos ? 31 - __clz(pos) : -1);
                if (at >= 0) {
                    chunk = c0 + at;
                    base = __shfl_sync(0xffffffffu, upto - mine, at);
                }
                if (hit) break;
                run = __shfl_sync(0xffffffffu, upto, 31);
            }
            const size_t row = (size_t)cur * a.batch + b;
            const Residual res = {S, gone, n_gone};
            const int c0 = (chunk_lo + chunk) * CHUNK;
            chunk_pass<T, VEC>(pb + row * a.p_ld, use_q ? qb + row * a.q_ld : nullptr, c0, a.vocab,
                               res, lane, bad, rbuf);
            __syncwarp();
            double mine = 0.0;
            for (int i = 0; i < 32; ++i) mine += rbuf[33 * lane + i];
            const double upto = base + warp_scan(mine, lane);
            const unsigned hit = __ballot_sync(0xffffffffu, mine > 0.0 && upto > target);
            const unsigned pos = __ballot_sync(0xffffffffu, mine > 0.0);
            const int at = hit ? __ffs(hit) - 1 : 31 - __clz(pos);
            if (lane == at) {
                double x = upto - mine;
                int found = 0;
                for (int i = 0; i < 32; ++i) {
                    const double r = rbuf[33 * lane + i];
                    if (!(r > 0.0)) continue;
                    found = i;
                    x += r;
                    if (x > target) break;
                }
                a.next[b] = c0 + 32 * lane + found;
            }
        }
    } else if (rank == 0 && tid == 0) {
        a.next[b] = -1;
    }
    if (rank == 0) {
        if (absent) n_path = 0;
        for (int t = n_path + tid; t < a.nodes; t += NT) a.path[(size_t)b * a.nodes + t] = -1;
        if (tid == 0) a.n_path[b] = n_path;
    }
    if (bad) set_status(a.status, KVC_DEV_NONFINITE);
    // no CTA leaves while another may still write its share
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

template <typename T, bool VEC>
cudaError_t launch_v(const VerifyArgs& a, cudaStream_t s) {
    const int chunks = (a.vocab + CHUNK - 1) / CHUNK;
    int cluster = 1;
    while (cluster < MAX_CLUSTER && cluster * 2 <= chunks && a.batch * cluster * 2 <= 148 * 4)
        cluster *= 2;
    const int per = (chunks + cluster - 1) / cluster;
    const size_t smem = ((a.nodes * (sizeof(NodeFacts) + 4) + 15) & ~(size_t)15) +
                        ((size_t)per + CHUNK + CHUNK / 32) * 8;
    int dev = 0;
    cudaGetDevice(&dev);
    static bool attr_set[64] = {};
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(
            verify_kernel<T, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.batch * cluster);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    trace_before("verify", s);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel<T, VEC>, a, cluster, per);
    trace_after(s);
    return e;
}

template <typename T>
cudaError_t launch_t(const VerifyArgs& a, cudaStream_t s) {
    // 16-byte (bf16: 8-byte) loads where every row starts on such a boundary
    const size_t al = 4 * sizeof(T);
    const bool vec = reinterpret_cast<uintptr_t>(a.p) % al == 0 && a.p_ld % 4 == 0 &&
                     (!a.q || (reinterpret_cast<uintptr_t>(a.q) % al == 0 && a.q_ld % 4 == 0));
    return vec ? launch_v<T, true>(a, s) : launch_v<T, false>(a, s);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int dtype, cudaStream_t s) {
    return dtype == KVC_BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace kvc
