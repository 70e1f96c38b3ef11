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
// of r and m, so m is 1 less the rejected probabilities and not the sum of what
// is left (which would take a pass over the row for each rejection): rows whose
// sum is not 1 keep that difference in m.  The next token is drawn from the
// residual of the last accepted node: the lowest i whose running sum passes v
// times the whole sum.
//
// Everything that decides is fp64: S q is rounded once, inside the multiply-add
// of the residual, u m q twice, masses and running sums once an addition.  That
// moves a border by 10^-16 of the mass (a sum of n terms by less than n / 2^53 of
// it), where fp32 sums of 10^5 terms would move it past whole tokens.  No value
// is converted: an fp32 pattern moved up by 29 bits is the same number times
// 2^-896 in fp64, subnormals and 0 included, so a pass works on residuals of
// that scale (two shifts an entry, where a conversion takes a warp 8 clocks) and
// scales their sum back.
//
// A sequence is one cluster of CTAs, each with a contiguous share of the
// vocabulary in blocks of 128 entries (more where a share has more than 1024
// of them), a block to a warp, two in flight; the sums of the shares are
// exchanged over distributed shared memory, so every CTA walks the tree alike.
// What each node's walk looks up (token, parent, u, p(x), q(x)) is loaded by
// one thread a node at the start.  Bound: the rows of the last accepted node
// and of every node with a rejection, read from HBM once and from the caches
// in later passes; small batches by the chain of a pass, two dependent loads
// and a cluster barrier for each rejection.  Measured (fp32, with draft rows, in
// a graph of twenty calls; "cold": on twenty sets of rows, with L2 swept
// before): one tree of 4 over 32,000 tokens 6.8 us, cold 8.8; 32 trees of 8 over
// 131,072 16.6 us, cold 21.6.
#include "kvc_internal.cuh"

namespace kvc {
namespace {

constexpr int NT = 512, NW = NT / 32;
constexpr int BLOCK = 128;  // vocabulary entries a warp sums at a time
constexpr int NB = 2;       // blocks of a warp in flight
constexpr int MAX_CLUSTER = 8, MAX_BLOCKS = 1024;
constexpr double kScaleUp = 0x1p896;

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

// Entries e .. e + 3 of a row as fp32 patterns; past the vocabulary 0.
template <typename T, bool VEC>
__device__ __forceinline__ void load4(const T* row, int e, int vocab, uint32_t (&v)[4]) {
    if constexpr (VEC) {
        if (e + 4 <= vocab) {
            if constexpr (sizeof(T) == 4) {
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + e));
                v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
            } else {
                const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + e));
                v[0] = w.x << 16, v[1] = w.x & 0xFFFF0000u;
                v[2] = w.y << 16, v[3] = w.y & 0xFFFF0000u;
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = e + j < vocab ? __float_as_uint(as_f32(row[e + j])) : 0u;
}
// A pattern as it counts: negative values, NaN and infinities are 0.
__device__ __forceinline__ uint32_t clean(uint32_t x, bool& bad) {
    bad |= (x & 0x7F800000u) == 0x7F800000u;
    return x < 0x7F800000u ? x : 0u;
}
__device__ __forceinline__ double scaled(uint32_t x) {  // value x 2^-896
    return __hiloint2double((int)(x >> 3), (int)(x << 29));
}

struct NodeFacts {
    int parent, token;
    float u, p, q;  // q: 1 without draft probabilities
};

// The residual max(p - S q, 0) (without q: p without the rejected tokens).
template <typename T>
struct Residual {
    const T* p;
    const T* q;  // or null
    double S;
    const int* gone;  // rejected tokens (no draft probabilities)
    int n_gone;
};

// N quads of entries e[i] .. e[i] + 3 of this lane as patterns, cleaned and
// without the rejected tokens (e[i] >= vocab: zeros).
template <typename T, bool VEC, int N>
__device__ __forceinline__ void load_quads(const Residual<T>& res, const int (&e)[N], int vocab,
                                           uint32_t (&pv)[N][4], uint32_t (&qv)[N][4], bool& bad) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) load4<T, VEC>(res.p, e[i], vocab, pv[i]);
    if (res.q)
#pragma unroll
        for (int i = 0; i < N; ++i) load4<T, VEC>(res.q, e[i], vocab, qv[i]);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!res.q) qv[i][j] = 0u;
            most = max(most, max(pv[i][j], qv[i][j]));
        }
    if (most >= 0x7F800000u)  // rare: something that is no finite probability
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                pv[i][j] = clean(pv[i][j], bad);
                qv[i][j] = clean(qv[i][j], bad);
            }
    for (int g = 0; g < res.n_gone; ++g) {
        const int t = res.gone[g];
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (t == e[i] + j) pv[i][j] = 0u;
    }
}
// Residual of one entry, times 2^-896.
__device__ __forceinline__ double residual(uint32_t p, uint32_t q, double S) {
    const double x = fma(-S, scaled(q), scaled(p));
    return x > 0.0 ? x : 0.0;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(NT, 2)
verify_kernel(VerifyArgs a, int cluster, int blocks_per_cta, int nsub) {
    extern __shared__ __align__(16) unsigned char smem[];
    NodeFacts* facts = reinterpret_cast<NodeFacts*>(smem);  // [nodes]
    int* gone = reinterpret_cast<int*>(facts + a.nodes);    // [nodes]
    double* bsum = reinterpret_cast<double*>(                // [blocks_per_cta], times 2^-896
        smem + ((a.nodes * (sizeof(NodeFacts) + 4) + 15) & ~(size_t)15));
    __shared__ double share[2][MAX_CLUSTER];  // every CTA's sum of the pass, by its parity
    const int b = blockIdx.x / cluster, rank = blockIdx.x - b * cluster;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T* pb = static_cast<const T*>(a.p);
    const T* qb = static_cast<const T*>(a.q);
    bool bad = false;
    pdl_wait();
    // (without a tree the sequence's tokens and rows are not looked at: they may
    // hold anything)
    const bool absent = a.parents[b] != -1;
    for (int t = tid; t < a.nodes; t += NT) {
        NodeFacts f;
        f.parent = a.parents[(size_t)t * a.batch + b];
        f.token = a.tokens[(size_t)t * a.batch + b];
        f.u = a.u[(size_t)t * a.batch + b];
        f.p = 0.f;
        f.q = 1.f;
        const bool is_child = t > 0 && f.parent >= 0 && f.parent < t;
        if (!is_child && f.parent != -1) {  // no node there
            if (f.parent != -2 && rank == 0) set_status(a.status, KVC_DEV_BAD_INDEX);
            f.parent = -2;
        }
        if (is_child && !absent && (f.token < 0 || f.token >= a.vocab)) {
            if (rank == 0) set_status(a.status, KVC_DEV_BAD_INDEX);
            f.parent = -1;
        } else if (is_child && !absent) {
            const size_t row = (size_t)f.parent * a.batch + b;
            f.p = counts(as_f32(pb[row * a.p_ld + f.token]), bad);
            if (qb) f.q = counts(as_f32(qb[row * a.q_ld + f.token]), bad);
        }
        facts[t] = f;
    }
    // the facts are in place, and every CTA of the cluster runs (its shared
    // memory may be written)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;\n" ::: "memory");

    int cur = 0, n_path = 1, n_gone = 0, passes = 0;
    double S = 0.0, m = 1.0;
    bool summed = false;  // bsum and share hold the residual of `cur` at S
    const int width = BLOCK * nsub;  // entries of a block
    const int first_block = rank * blocks_per_cta;
    const int n_blocks = min(blocks_per_cta, (a.vocab + width - 1) / width - first_block);
    auto residual_of = [&](bool use_q) {
        const size_t row = (size_t)cur * a.batch + b;
        return Residual<T>{pb + row * a.p_ld, use_q ? qb + row * a.q_ld : nullptr, use_q ? S : 0.0,
                           gone, n_gone};
    };
    // One pass over this CTA's share of the residual; returns its whole mass.
    auto pass = [&](bool use_q) -> double {
        const Residual<T> res = residual_of(use_q);
        for (int b0 = warp; b0 < n_blocks; b0 += NW * NB) {
            double s[NB] = {};
            for (int sub = 0; sub < nsub; ++sub) {
                int e[NB];
#pragma unroll
                for (int i = 0; i < NB; ++i)
                    e[i] = b0 + NW * i < n_blocks
                               ? (first_block + b0 + NW * i) * width + sub * BLOCK + 4 * lane
                               : a.vocab;
                uint32_t pv[NB][4], qv[NB][4];
                load_quads<T, VEC, NB>(res, e, a.vocab, pv, qv, bad);
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const double x = fma(-res.S, scaled(qv[i][j]), scaled(pv[i][j]));
                        if (x > 0.0) s[i] += x;
                    }
            }
            // block sums: lanes 16 k .. 16 k + 15 end with that of block k
            const double send = lane & 16 ? s[0] : s[1], keep = lane & 16 ? s[1] : s[0];
            s[0] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
            const int k = b0 + NW * (lane >> 4);
            if ((lane & 15) == 0 && k < n_blocks) bsum[k] = s[0];
        }
        __syncthreads();
        const int par = passes & 1;
        ++passes;
        if (warp == 0) {
            double t = 0.0;
            for (int k = lane; k < n_blocks; k += 32) t += bsum[k];
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
        return sum * kScaleUp;
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
        // where rounding leaves none), its block, and the entry; all of it at
        // the scale of the sums
        const double* sh = share[(passes - 1) & 1];
        double whole = 0.0;
        for (int r = 0; r < cluster; ++r) whole += sh[r];
        const double target = (double)a.v[b] * whole;
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
            // Among values in order, the first whose running sum passes the
            // target, or the last with any mass: `found`, with `base` the sum in
            // front of it.
            int found = -1;
            double base = before, run = before;
            auto step = [&](double mine, int first) {  // one value a lane
                const double upto = run + warp_scan(mine, lane);
                const unsigned hit = __ballot_sync(0xffffffffu, mine > 0.0 && upto > target);
                const unsigned pos = __ballot_sync(0xffffffffu, mine > 0.0);
                const int at = hit ? __ffs(hit) - 1 : (pos ? 31 - __clz(pos) : -1);
                if (at >= 0) {
                    found = first + at;
                    base = __shfl_sync(0xffffffffu, upto - mine, at);
                }
                run = __shfl_sync(0xffffffffu, upto, 31);
                return hit != 0;
            };
            for (int k = 0; k < n_blocks; k += 32)
                if (step(k + lane < n_blocks ? bsum[k + lane] : 0.0, k)) break;
            const int e0 = (first_block + found) * width;
            const Residual<T> res = residual_of(use_q);
            run = base;
            found = -1;
            double r[4], in_quad[4] = {};
            for (int sub = 0; sub < nsub; ++sub) {
                const int e[1] = {e0 + sub * BLOCK + 4 * lane};
                uint32_t pv[1][4], qv[1][4];
                load_quads<T, VEC, 1>(res, e, a.vocab, pv, qv, bad);
#pragma unroll
                for (int j = 0; j < 4; ++j) r[j] = residual(pv[0][j], qv[0][j], res.S);
                const int was = found;
                const bool done = step((r[0] + r[1]) + (r[2] + r[3]), 32 * sub);
                if (found != was)
#pragma unroll
                    for (int j = 0; j < 4; ++j) in_quad[j] = r[j];
                if (done) break;
            }
            if (lane == (found & 31)) {
                double x = base;
                int at = 0;
#pragma unroll
                for (int j = 3; j >= 0; --j)  // the last with any mass ...
                    if (in_quad[j] > 0.0) {
                        at = j;
                        break;
                    }
                for (int j = 0; j < 4; ++j) {  // ... unless the target is passed
                    x += in_quad[j];
                    if (in_quad[j] > 0.0 && x > target) {
                        at = j;
                        break;
                    }
                }
                a.next[b] = e0 + 4 * found + at;
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
    // CTAs of a sequence: while each keeps a block for every warp and all of
    // them run at once (two a multiprocessor).  1, 4, 8 of them: 32 trees of 8
    // over 131,072 tokens 69.0, 23.9, 18.5 us, one of 4 over 32,000 12.8, 7.0, 6.4.
    const int quads = (a.vocab + BLOCK - 1) / BLOCK;
    int cluster = 1;
    while (cluster < MAX_CLUSTER && quads >= 2 * cluster * NW && a.batch * cluster * 2 <= 148 * 2)
        cluster *= 2;
    int nsub = 1;
    while ((quads + nsub * cluster - 1) / (nsub * cluster) > MAX_BLOCKS) nsub *= 2;
    const int blocks = (quads + nsub - 1) / nsub;
    const int per = (blocks + cluster - 1) / cluster;
    const size_t smem = ((a.nodes * (sizeof(NodeFacts) + 4) + 15) & ~(size_t)15) + (size_t)per * 8;
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel<T, VEC>, a, cluster, per, nsub);
    trace_after(s);
    return e;
}

template <typename T>
cudaError_t launch_t(const VerifyArgs& a, cudaStream_t s) {
    // 16-byte (bf16: 8-byte) loads where every row starts on such a boundary
    // (32 trees of 8 over 131,072 fp32 tokens: 18.5 us, by single loads 19.3)
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
