// Verification of drafted trees: speculative sampling from given uniform numbers.
//
// A cluster of CTAs walks one tree.  What a node's test needs besides its token's two probabilities (gathered for all nodes at the
// start) is the sum R of the residual r after each rejection: one pass over the vocabulary, a part of it to each CTA, whose r stays in
// shared memory for the next pass and for the search.  (r - R q is the rest of the target for children drawn independently, with
// replacement, or for a single one.)  The walk itself is a few hundred instructions that every thread repeats, so
// it needs no exchange.
// All of r and R are integers, in steps of 2^-50, and tests and the search compare products of 112 and 88 bits: sums are exact, in any order, so
// that neither the split over CTAs nor the number of warps can change the sampled token.  (Sums in fp64 would be off by
// little, but this GPU adds two of them a clock and SM.)
// Bound by the latency of the chain: tokens, their probabilities (launch and walk 4 us), a pass and the search (1.5 to 3 us), and 3.7 us
// for each further rejection of a node, 54 instructions an element.  8 chains of 5 drafts over 131072 tokens, fp32: 10.1 us; 48
// trees of up to 23 drafts over 50001, bf16: 32 us.
#include <algorithm>

#include "common.cuh"

namespace tq {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kRun = 256;          // elements of a run, whose sum is kept for the search
constexpr int kNodes = 1024;       // largest tree
constexpr int kVocab = 1 << 20;    // largest vocabulary
constexpr int kCluster = 16;       // most CTAs of a tree (more than 8 have to be asked for)
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

// A probability's bits: below 0 and NaN 0, above 1 those of 1.
TQ_DEVFN uint32_t bits_of(float x) {
    const uint32_t b = __float_as_uint(x);  // (above one's bits as integers: larger, negative or NaN)
    return b > 0x3f800000u ? (x > 1.f ? 0x3f800000u : 0u) : b;
}
// x in steps of 2^-50, rounded to nearest (subnormal numbers are 0).
TQ_DEVFN u64 fixed(float x) {
    const uint32_t b = bits_of(x);
    const u64 m = (u64)((b & 0x7fffffu) | 0x800000u) << 28;  // x = m 2^(e - 178)
    return ((m >> min(127 - (int)(b >> 23), 63)) + 1) >> 1;
}
// max(r - R q, 0), R q rounded as `fixed` rounds (R = 1 gives q's own value): q's 24 bits times R's, shifted to steps of 2^-50.
TQ_DEVFN u64 step_down(u64 r, float q, u64 R) {
    const uint32_t b = bits_of(q), m = (b & 0x7fffffu) | 0x800000u;
    const u64 low = (u64)(uint32_t)R * m, high = (u64)(uint32_t)(R >> 32) * m + (low >> 32);  // R m = high 2^32 + the low word
    const u64 x = high << 10 | (uint32_t)low >> 22;                                           // R q = x 2^(e - 128)
    const u64 rq = ((x >> min(127 - (int)(b >> 23), 63)) + 1) >> 1;
    return r > rq ? r - rq : 0ull;
}

// u q < p, exactly: the sum's sign is not rounded (the powers of two keep it from underflow).
TQ_DEVFN bool below(float u, float q, float p) { return fmaf(u * 4294967296.f, q * 4294967296.f, -p * 18446744073709551616.f) < 0.f; }
// u q R < r, exactly, as integers: u and q are 24 bits and a power of two each.
TQ_DEVFN bool below(float u, float q, u64 R, u64 r) {
    if (!(u > 0.f)) return u <= 0.f && r > 0;  // (a NaN accepts nothing)
    const uint32_t bu = __float_as_uint(fminf(u, 2.f)), bq = __float_as_uint(q);
    const int eu = bu >> 23, eq = bq >> 23;
    const u64 m = (u64)((bu & 0x7fffffu) | (eu ? 0x800000u : 0u)) * ((bq & 0x7fffffu) | (eq ? 0x800000u : 0u));
    const u64 high = __umul64hi(m, R), low = m * R;  // u q R = (high 2^64 + low) 2^-s, below 2^112
    const int s = 300 - max(eu, 1) - max(eq, 1);     // 45 at least
    if (s >= 128) return r > 0;
    if (s > 64 && r >> (128 - s)) return true;  // r 2^s has more than 128 bits
    const u64 rh = s >= 64 ? r << (s - 64) : r >> (64 - s), rl = s >= 64 ? 0 : r << s;
    return high < rh || (high == rh && low < rl);
}

// u R without its fraction, exactly, for 0 <= u < 1 (R - 1 above, 0 below and for a NaN): an integer P passes u R where it is larger.
TQ_DEVFN u64 share(float u, u64 R) {
    if (!(u > 0.f)) return 0;
    if (u >= 1.f) return R - 1;
    const uint32_t b = __float_as_uint(u);
    const int e = b >> 23, s = 150 - max(e, 1);  // u = m 2^-s, s 24 at least
    const u64 m = (b & 0x7fffffu) | (e ? 0x800000u : 0u), high = __umul64hi(m, R), low = m * R;
    if (s >= 64) return s >= 128 ? 0 : high >> (s - 64);
    return high << (64 - s) | low >> s;
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
TQ_DEVFN void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
TQ_DEVFN void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
TQ_DEVFN void cluster_sync() {
    cluster_arrive();
    cluster_wait();
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

// KEPT: the residual lies in shared memory, an element of the CTA's part after another; else it is computed from the rows and all
// rejections of the node.
template <int DT, bool Q, bool KEPT>
__global__ void __launch_bounds__(kThreads) verify_tree_kernel(const __grid_constant__ VerifyArgs a) {
    extern __shared__ u64 shared[];
    u64* const run_sum = shared;                                  // [runs]
    u64* const kept = run_sum + a.runs;                           // [runs][kRun]
    u64* const s_R = kept + (KEPT ? (size_t)a.runs * kRun : 0);   // [n]: of each rejection of the node, R before it
    float* const s_p = reinterpret_cast<float*>(s_R + a.n);       // of each node: its token's probabilities, its number
    float *const s_q = s_p + a.n, *const s_u = s_q + a.n;
    int *const s_parent = reinterpret_cast<int*>(s_u + a.n), *const s_token = s_parent + a.n, *const s_path = s_token + a.n;
    int* const s_shift = s_path + a.n;         // of each rejection: how much finer its steps became; without q: its token
    __shared__ u64 s_total[2][kCluster];       // by turns, so that one exchange needs one barrier
    __shared__ u64 s_part[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int b = blockIdx.x / size;
    const int64_t row0 = (int64_t)b * a.n;
    pdl_trigger();
    cluster_arrive();
    pdl_wait();
    const int used = a.n_tok ? min(max(a.n_tok[b], 0), a.n) : a.n;
    uint32_t wrong = 0;
    for (int i = tid; i < a.n; i += kThreads) {
        const int parent = a.parent[row0 + i], token = a.tokens[row0 + i];
        const bool ok = i > 0 && i < used && (uint32_t)parent < (uint32_t)i && (uint32_t)token < (uint32_t)a.V;
        if (i > 0 && i < used && !ok) wrong |= TQ_DEVERR_BAD_ID;
        s_parent[i] = ok ? parent : -1;
        s_token[i] = token;
        s_u[i] = a.u[row0 + i];
        // (fmaxf drops a NaN)
        s_p[i] = ok ? fminf(fmaxf(load_p<DT>(a.p, (row0 + parent) * a.p_stride + token), 0.f), 1.f) : 0.f;
        s_q[i] = Q && ok ? fminf(fmaxf(load_p<DT>(a.q, (row0 + parent) * a.q_stride + token), 0.f), 1.f) : 1.f;
    }
    if (wrong && a.err && rank == 0) atomicOr(a.err, wrong);
    if (rank == 0 && tid == 0) a.next[b] = -1;  // until the search finds one, behind a pass's barrier of the cluster
    __syncthreads();
    cluster_wait();  // every CTA of the cluster has started: before that none may store into another's shared memory

    const int first = (int)rank * a.runs;  // of this CTA's runs
    int turn = 0, node = 0, length = 1, k = 0;  // k: rejections of the node
    u64 R = kOne, mine = 0, before = 0;         // of the whole vocabulary, this CTA's part, the parts before it
    auto row_p = [&](int at) { return reinterpret_cast<const char*>(a.p) + (row0 + at) * a.p_stride * (DT == TQ_F32 ? 4 : 2); };
    auto row_q = [&](int at) { return reinterpret_cast<const char*>(a.q) + (row0 + at) * a.q_stride * (DT == TQ_F32 ? 4 : 2); };
    // An element's residual after the node's k rejections, from its probabilities.
    auto residual = [&](float p, float q, int x) {
        u64 r = fixed(p);
        if (Q) {
            for (int j = 0; j < k; ++j) r = step_down(r, q, s_R[j]) << s_shift[j];
        } else {
            for (int j = 0; j < k; ++j)
                if (x == s_shift[j]) r = 0;
        }
        return r;
    };
    // The residual after k rejections, and its sums: from the rows, after a node's first rejection, or by one more step from what is kept.
    auto sums_of = [&](auto how) {
        constexpr bool AGAIN = decltype(how)::value == 2, FIRST = decltype(how)::value == 1;
        const char *prow = row_p(node), *qrow = row_q(node);
        const u64 R1 = R;
        u64 sum = 0;
        constexpr int N = kRun / 32, kTwo = 2;  // elements a lane, runs on their way at a time
        for (int i0 = warp; i0 < a.runs; i0 += kTwo * kWarps) {
            float p[kTwo][N], q[kTwo][N];
#pragma unroll
            for (int z = 0; z < kTwo; ++z) {
                const int i = i0 + z * kWarps, x0 = (first + i) * kRun + lane;
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    const int x = x0 + c * 32;
                    const bool in = i < a.runs && x < a.V;
                    p[z][c] = in && !AGAIN ? load_p<DT>(prow, x) : 0.f;
                    q[z][c] = Q && in && k ? load_p<DT>(qrow, x) : 0.f;
                }
            }
#pragma unroll
            for (int z = 0; z < kTwo; ++z) {
                const int i = i0 + z * kWarps;
                if (i >= a.runs) break;
                u64 r = 0;
                u64* const at = kept + (KEPT ? i * kRun + lane : 0);
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    u64 v;
                    if (AGAIN) {
                        v = step_down(at[c * 32], q[z][c], R1);
                    } else if (FIRST) {  // R is 1
                        const u64 f = fixed(p[z][c]), g = fixed(q[z][c]);
                        v = f > g ? f - g : 0;
                    } else {
                        v = residual(p[z][c], q[z][c], (first + i) * kRun + lane + c * 32);
                    }
                    if (KEPT) at[c * 32] = v;
                    r += v;
                }
                r = warp_sum(r);
                if (lane == 0) run_sum[i] = r;
                sum += r;
            }
        }
        return sum;
    };
    auto pass = [&]() {
        u64 sum;
        if (KEPT && Q && k > 1) sum = sums_of(std::integral_constant<int, 2>{});
        else if (Q && k == 1) sum = sums_of(std::integral_constant<int, 1>{});
        else sum = sums_of(std::integral_constant<int, 0>{});
        if (lane == 0) s_part[warp] = sum;
        __syncthreads();
        mine = warp_sum(lane < kWarps ? s_part[lane] : 0ull);
        if (warp == 0 && lane < (int)size) store_remote(&s_total[turn][rank], lane, mine);
        cluster_sync();
        R = before = 0;
        for (uint32_t c = 0; c < size; ++c) {
            if (c < rank) before += s_total[turn][c];
            R += s_total[turn][c];
        }
        turn ^= 1;
    };

    bool summed = false;  // run_sum and what is kept are those of r as it is
    if (tid == 0) s_path[0] = 0;
    for (int i = 1; i < used; ++i) {
        if (s_parent[i] != node) continue;
        bool yes;
        u64 r = 0;
        if (k == 0) {
            yes = below(s_u[i], s_q[i], s_p[i]);
        } else {
            r = residual(s_p[i], s_q[i], s_token[i]);
            yes = below(s_u[i], s_q[i], R, r);
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
        if (!Q && k == 0) r = fixed(s_p[i]);
        if (!KEPT || !Q || k == 0) __syncthreads();  // the last reads of the rejections
        if (tid == 0) {
            s_R[k] = R;
            s_shift[k] = Q ? 0 : s_token[i];
        }
        ++k;
        if (!KEPT || !Q) __syncthreads();  // (else they are read again behind the pass's barriers)
        if (Q) {
            pass();
            summed = true;
            if (R && R < 1ull << 34) {  // little is left: its steps are made finer, 2^-50 of it to 2^-49
                const int up = __clzll((long long)R) - 14;
                __syncthreads();
                if (tid == 0) s_shift[k - 1] = up;
                for (int j = tid; j < a.runs; j += kThreads) run_sum[j] <<= up;
                if (KEPT)
                    for (int j = tid; j < a.runs * kRun; j += kThreads) kept[j] <<= up;
                R <<= up;
                mine <<= up;
                before <<= up;
                __syncthreads();
            }
        } else {
            R = R > r ? R - r : 0;
        }
    }
    if (used == 0) {
        length = 0;
    } else {
        if (!summed) pass();
        if (R == 0) {
            k = 0;
            pass();
        }
    }
    __syncthreads();
    if (rank == 0) {
        for (int i = tid; i < a.n; i += kThreads) a.path[row0 + i] = i < length ? s_path[i] : -1;
        if (tid == 0) a.count[b] = length;
    }
    if (used && R && warp == 0) {
        // the first token whose prefix sum passes u R: in this CTA where the threshold falls into its part
        const u64 t = share(s_u[0], R);
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
                const int x = x0 + c;
                if (KEPT) r[c] = kept[run * kRun + lane * kEach + c];
                else r[c] = x < a.V ? residual(load_p<DT>(row_p(node), x), Q && k ? load_p<DT>(row_q(node), x) : 0.f, x) : 0;
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

template <int DT>
void (*kernel_of(bool q, bool kept))(VerifyArgs) {
    if (q) return kept ? verify_tree_kernel<DT, true, true> : verify_tree_kernel<DT, true, false>;
    return kept ? verify_tree_kernel<DT, false, true> : verify_tree_kernel<DT, false, false>;
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
    // Each tree over several CTAs, since it waits for the slowest of its passes: as many as four to an SM make, each with a run for
    // every warp (48 trees over 50001 tokens: 35 us with eight to a tree, 41 with four, although two of 64 registers by 512 threads are
    // resident on an SM, so that 384 CTAs come in two waves); sixteen where the trees are few (one tree,
    // 131072 tokens, five rejections: 23 us for 34; eight trees gain nothing).
    int size_c = 1;
    while (size_c < kCluster && B * size_c * 2 <= (size_c < 8 ? 4 * device_sms() : 64) && runs >= 32 * size_c) size_c *= 2;
    const size_t nodes = (size_t)n * (sizeof(u64) + 3 * sizeof(float) + 4 * sizeof(int));
    // The residual stays in shared memory where it fits (five rejections in each of 48 trees over 131072 tokens: 130 us in parts that
    // fit, 367 us in parts twice as large, computed anew in each pass).
    constexpr size_t kStatic = 1024;  // above the kernel's own arrays: the limit that is raised holds for both together
    size_t smem = 0;
    void (*kernel)(VerifyArgs) = nullptr;
    for (;; size_c = 8) {  // (once more where no cluster of 16 has a place)
        a.runs = (runs + size_c - 1) / size_c;
        const size_t sums = (size_t)a.runs * sizeof(u64);
        const bool kept = nodes + sums * (1 + kRun) <= 200 * 1024;
        smem = nodes + sums * (1 + (kept ? kRun : 0));
        kernel = dt == TQ_F32 ? kernel_of<TQ_F32>(q, kept) : (dt == TQ_BF16 ? kernel_of<TQ_BF16>(q, kept) : kernel_of<TQ_F16>(q, kept));
        if (ensure_smem((const void*)kernel, smem + kStatic) != cudaSuccess) return TQ_ERR_CUDA;
        if (clusters_fit((const void*)kernel, size_c, kThreads, smem)) break;
    }
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
