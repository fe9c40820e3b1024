// Verification of drafted trees: speculative sampling from given uniform numbers.
//
// A cluster of CTAs walks one tree.  What a node's test needs besides its token's two probabilities (gathered for all nodes at the
// start) is the sum R of the residual r after each rejection: one pass over the vocabulary, a part of it to each CTA.  The walk
// itself is a few hundred instructions that every thread repeats, so it needs no exchange.  r is never stored: it is computed from
// the rows and the R of the node's rejections whenever it is needed.
// All of r and R are integers, in steps of 2^-50 of the largest value they may have: sums are exact, in any order, so that
// neither the split over CTAs nor the number of warps can change the sampled token.
// Bound by the latency of the chain: tokens, their probabilities, one or two passes (rows where the walk ends: 1 MB a tree of two
// rows of 131072 in 32 bits) and one search.
#include <algorithm>

#include "common.cuh"

namespace tq {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kRun = 256;          // elements of a run, whose sum is kept for the search
constexpr int kNodes = 1024;       // largest tree
constexpr int kVocab = 1 << 20;    // largest vocabulary
constexpr int kCluster = 8;        // most CTAs of a tree
constexpr u64 kOne = 1ull << 50;

struct VerifyArgs {
    const void* p;
    const void* q;
    int64_t p_stride, q_stride;
    const int32_t* tokens;
    const int32_t* parent;
    const float* u;
    const int32_t* n_tok;
    int32_t* path;
    int32_t* count;
    int32_t* next;
    uint32_t* err;
    int n, V, runs;  // runs: of each CTA
};

template <int DT>
TQ_DEVFN float load_p(const void* p, int64_t i) {
    if (DT == TQ_F32) return __ldg(reinterpret_cast<const float*>(p) + i);
    if (DT == TQ_BF16) return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + i) << 16);
    return __half2float(__ushort_as_half(__ldg(reinterpret_cast<const unsigned short*>(p) + i)));
}

// x in steps of 2^-50, rounded to nearest; below 0 and NaN: 0, above 1: 1.
TQ_DEVFN u64 fixed(float x) {
    const uint32_t b = __float_as_uint(x);
    if (b > 0x3f800000u) return x > 1.f ? kOne : 0ull;  // (above one's bits as integers: larger, negative or NaN)
    const int e = b >> 23;
    const u64 m = (u64)((b & 0x7fffffu) | (e ? 0x800000u : 0u)) << 28;  // x = m 2^(e - 178), a subnormal's is 0 below
    const int down = 127 - e;
    return down > 62 ? 0ull : ((m >> down) + 1) >> 1;
}

// The residual after `k` rejections of a node: R of each rejection before it, and the shift that brought its sum up to 2^49 .. 2^50.
struct Steps {
    u64 R[kNodes];
    int shift[kNodes];
};
// max(r - R q, 0) 2^shift, q and R in steps of 2^-50.
TQ_DEVFN u64 step_down(u64 r, u64 q, u64 R, int shift) {
    const u64 hi = __umul64hi(R, q), lo = R * q;
    const u64 rq = (hi << 14) | (lo >> 50);
    return r > rq ? (r - rq) << shift : 0ull;
}

TQ_DEVFN uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
TQ_DEVFN uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
TQ_DEVFN void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
TQ_DEVFN void store_remote(u64* local, uint32_t rank, u64 v) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(local)), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

TQ_DEVFN u64 warp_sum(u64 x) {
#pragma unroll
    for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(kFull, x, m);
    return x;
}
TQ_DEVFN u64 warp_prefix(u64 x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const u64 y = __shfl_up_sync(kFull, x, m);
        if (lane >= m) x += y;
    }
    return x;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) verify_tree_kernel(VerifyArgs a) {
    extern __shared__ u64 run_sum[];          // [runs]
    __shared__ float s_p[kNodes], s_q[kNodes], s_u[kNodes];  // of each node: its token's probabilities, its number
    __shared__ int s_parent[kNodes], s_token[kNodes], s_path[kNodes];
    __shared__ Steps steps;
    __shared__ u64 s_total[2][kCluster];      // by turns, so that one exchange needs one barrier
    __shared__ u64 s_part[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int b = blockIdx.x / size;
    const int64_t row0 = (int64_t)b * a.n;
    pdl_trigger();
    pdl_wait();
    const int used = a.n_tok ? min(max(a.n_tok[b], 0), a.n) : a.n;
    uint32_t wrong = 0;
    for (int i = tid; i < used; i += kThreads) {
        const int parent = a.parent[row0 + i], token = a.tokens[row0 + i];
        const bool ok = i > 0 && (uint32_t)parent < (uint32_t)i && (uint32_t)token < (uint32_t)a.V;
        if (i > 0 && !ok) wrong |= TQ_DEVERR_BAD_ID;
        s_parent[i] = ok ? parent : -1;
        s_token[i] = token;
        s_u[i] = a.u[row0 + i];
        // (fmaxf drops a NaN)
        s_p[i] = ok ? fminf(fmaxf(load_p<DT>(a.p, (row0 + parent) * a.p_stride + token), 0.f), 1.f) : 0.f;
        s_q[i] = ok && a.q ? fminf(fmaxf(load_p<DT>(a.q, (row0 + parent) * a.q_stride + token), 0.f), 1.f) : 1.f;
    }
    if (wrong && a.err && rank == 0) atomicOr(a.err, wrong);
    __syncthreads();

    const int first = (int)rank * a.runs;  // of this CTA's runs
    int turn = 0;
    // r of element x of the rows of `node`, after `k` rejections.
    auto residual = [&](const void* prow, const void* qrow, int x, int k, const int* gone) {
        u64 r = fixed(load_p<DT>(prow, x));
        if (a.q) {
            if (k) {
                const u64 q = fixed(load_p<DT>(qrow, x));
                for (int j = 0; j < k; ++j) r = step_down(r, q, steps.R[j], steps.shift[j]);
            }
        } else {
            for (int j = 0; j < k; ++j)
                if (x == gone[j]) r = 0;
        }
        return r;
    };
    // The sum of r over the vocabulary; run_sum holds this CTA's runs, `mine` and `before` its own total and that of the CTAs before.
    auto pass = [&](const void* prow, const void* qrow, int k, const int* gone, u64& mine, u64& before) {
        u64 sum = 0;
        for (int i = warp; i < a.runs; i += kWarps) {
            const int x0 = (first + i) * kRun;
            u64 r = 0;
#pragma unroll
            for (int c = 0; c < kRun / 32; ++c) {
                const int x = x0 + c * 32 + lane;
                if (x < a.V) r += residual(prow, qrow, x, k, gone);
            }
            r = warp_sum(r);
            if (lane == 0) run_sum[i] = r;
            sum += r;
        }
        if (lane == 0) s_part[warp] = sum;
        __syncthreads();
        mine = warp_sum(lane < kWarps ? s_part[lane] : 0ull);
        if (warp == 0 && lane < (int)size) store_remote(&s_total[turn][rank], lane, mine);
        cluster_sync();
        u64 all = 0;
        before = 0;
        for (uint32_t c = 0; c < size; ++c) {
            if (c < rank) before += s_total[turn][c];
            all += s_total[turn][c];
        }
        turn ^= 1;
        return all;
    };

    auto row_p = [&](int node) {
        return reinterpret_cast<const char*>(a.p) + (row0 + node) * a.p_stride * (DT == TQ_F32 ? 4 : 2);
    };
    auto row_q = [&](int node) {
        return reinterpret_cast<const char*>(a.q) + (row0 + node) * a.q_stride * (DT == TQ_F32 ? 4 : 2);
    };
    int* const gone = steps.shift;  // without q: the tokens of the rejected children
    int node = 0, length = 1, k = 0;
    u64 R = kOne, mine = 0, before = 0;
    bool summed = false;  // run_sum holds the sums of r as it is
    if (tid == 0) s_path[0] = 0;
    for (int i = 1; i < used; ++i) {
        if (s_parent[i] != node) continue;
        const int x = s_token[i];
        bool yes;
        u64 r = 0;
        if (k == 0) {
            yes = (double)s_u[i] * (double)s_q[i] < (double)s_p[i];  // (the product is exact)
        } else {
            r = fixed(s_p[i]);
            if (a.q) {
                const u64 q = fixed(s_q[i]);
                for (int j = 0; j < k; ++j) r = step_down(r, q, steps.R[j], steps.shift[j]);
            } else {
                for (int j = 0; j < k; ++j)
                    if (gone[j] == x) r = 0;
            }
            yes = (double)s_u[i] * (double)s_q[i] * (double)R < (double)r;
        }
        if (yes) {
            node = i;
            k = 0;
            R = kOne;
            summed = false;
            if (tid == 0) s_path[length] = i;
            ++length;
            continue;
        }
        __syncthreads();  // the last reads of steps
        if (a.q) {
            if (tid == 0) {
                steps.R[k] = R;
                steps.shift[k] = 0;
            }
            __syncthreads();
            R = pass(row_p(node), row_q(node), ++k, gone, mine, before);
            summed = true;
            const int up = R ? max(__clzll((long long)R) - 14, 0) : 0;
            if (up) {  // keep 2^-50 of what is left, however little that is
                __syncthreads();
                if (tid == 0) steps.shift[k - 1] = up;
                for (int j = tid; j < a.runs; j += kThreads) run_sum[j] <<= up;
                R <<= up;
                mine <<= up;
                before <<= up;
                __syncthreads();
            }
        } else {
            if (k == 0) r = fixed(s_p[i]);
            R = R > r ? R - r : 0;
            if (tid == 0) gone[k] = x;
            ++k;
            __syncthreads();
        }
    }
    if (used == 0) {
        length = 0;
    } else {
        if (!summed) R = pass(row_p(node), row_q(node), k, gone, mine, before);
        if (R == 0) {
            k = 0;
            R = pass(row_p(node), row_q(node), 0, gone, mine, before);
        }
    }
    __syncthreads();
    if (rank == 0) {
        for (int i = tid; i < a.n; i += kThreads) a.path[row0 + i] = i < length ? s_path[i] : -1;
        if (tid == 0) {
            a.count[b] = length;
            if (R == 0 || used == 0) a.next[b] = -1;
        }
    }
    if (used && R && warp == 0) {
        // the first token whose prefix sum passes u R: in this CTA where the threshold falls into its part
        const double want = (double)s_u[0] * (double)R;
        const u64 t = want > 0 ? min((u64)fmin(want, 9.0e18), R - 1) : 0;
        if (t >= before && t - before < mine) {
            u64 left = t - before;  // prefix sums within this CTA must pass it
            int run = 0;
            for (int i0 = 0; i0 < a.runs; i0 += 32) {
                const u64 own = i0 + lane < a.runs ? run_sum[i0 + lane] : 0, upto = warp_prefix(own);
                const unsigned hit = __ballot_sync(kFull, upto > left);
                if (hit) {
                    const int src = __ffs(hit) - 1;
                    left -= __shfl_sync(kFull, upto - own, src);
                    run = i0 + src;
                    break;
                }
                left -= __shfl_sync(kFull, upto, 31);
            }
            constexpr int kEach = kRun / 32;
            const int x0 = (first + run) * kRun + lane * kEach;
            u64 r[kEach], own = 0;
#pragma unroll
            for (int c = 0; c < kEach; ++c) {
                r[c] = x0 + c < a.V ? residual(row_p(node), row_q(node), x0 + c, k, gone) : 0;
                own += r[c];
            }
            const u64 upto = warp_prefix(own);
            const unsigned hit = __ballot_sync(kFull, upto > left);
            if (hit && lane == __ffs(hit) - 1) {
                u64 at = upto - own;
                int x = x0;
#pragma unroll
                for (int c = 0; c < kEach; ++c) {
                    if (at <= left) x = x0 + c;  // the sums before it do not pass the threshold
                    at += r[c];
                }
                a.next[b] = x;
            }
        }
    }
    cluster_sync();  // no CTA ends while another may still write its totals here
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" tq_status tq_verify_tree(const void* p, int64_t p_stride, const void* q, int64_t q_stride, tq_dtype dt, int32_t B,
                                    int32_t n, int32_t V, const int32_t* tokens, const int32_t* parent, const float* u,
                                    const int32_t* n_tok, int32_t* path, int32_t* count, int32_t* next, uint32_t* err,
                                    void* stream) {
    if (B < 0 || n < 0 || V < 0) return TQ_ERR_INVALID;
    if (!(dt == TQ_F32 || dt == TQ_BF16 || dt == TQ_F16)) return TQ_ERR_INVALID;
    if (n > kNodes || V > kVocab || B > (1 << 20)) return TQ_ERR_UNSUPPORTED;
    if (B == 0) return TQ_OK;
    if (n == 0 || V == 0) return TQ_ERR_INVALID;
    if (!p || !tokens || !parent || !u || !path || !count || !next) return TQ_ERR_INVALID;
    const size_t size = dt == TQ_F32 ? 4 : 2;
    if (p_stride < V || (q && q_stride < V) || p_stride > (1ll << 40) || (q && q_stride > (1ll << 40))) return TQ_ERR_INVALID;
    if (!aligned(p, size) || !aligned(q, size)) return TQ_ERR_INVALID;
    for (const void* x : {(const void*)tokens, (const void*)parent, (const void*)u, (const void*)n_tok, (const void*)path,
                          (const void*)count, (const void*)next})
        if (!aligned(x, 4)) return TQ_ERR_INVALID;
    VerifyArgs a{p, q, p_stride, q ? q_stride : 0, tokens, parent, u, n_tok, path, count, next, err, n, V, 0};
    const int runs = (V + kRun - 1) / kRun;
    // few trees: each over several CTAs, as long as each has two runs to a warp
    int size_c = 1;
    while (size_c < kCluster && B * size_c < 152 && runs >= 2 * kWarps * 2 * size_c) size_c *= 2;
    a.runs = (runs + size_c - 1) / size_c;
    void (*kernel)(VerifyArgs) = dt == TQ_F32 ? verify_tree_kernel<TQ_F32>
                                              : (dt == TQ_BF16 ? verify_tree_kernel<TQ_BF16> : verify_tree_kernel<TQ_F16>);
    const size_t smem = (size_t)a.runs * sizeof(u64);
    constexpr size_t kStatic = 40 * 1024;  // above the kernel's own arrays: the limit that is raised holds for both together
    if (ensure_smem((const void*)kernel, smem + kStatic) != cudaSuccess) return TQ_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(B * size_c));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = as_stream(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size_c;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
