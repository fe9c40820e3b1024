// Attention of prompts over keys and values expanded from the latents, on the 5th-generation tensor cores.
//
// A CTA takes 256 query rows of a head and sequence, as two streams of 128, over the keys that they see, 128 at a time:
//   scores   S[128 x 128]  = Q (shared) . [K, Kr]^T (shared)   12 MMAs of K = 16; the rotary keys are the same for every head
//   weights  P = exp2(S f + bias), 16 bits, written over S in TMEM       one thread to a row
//   values   O[128 x 128] += P (TMEM) . V (shared)                       8 MMAs of K = 16
// One thread issues: values of a stream, then its next scores, then the same of the other stream, so that each stream's softmax
// runs beside the other's products.  TMEM is full: scores and sums of two streams.  Tokens come by tensor copies into a ring of eight
// units of 128 tokens by 64 elements; a step takes three for keys and two for values.  A row's running maximum follows only when
// a score passes it by a set amount, so O is seldom rescaled.
//
// Values of steps that some row sees in part are looked through by two guard warps: those past the sequence's end are zeroed, and
// those that are not finite, which become NaN in the rows that see them (a masked weight of 0 times NaN would reach the others).
// Every wait on an mbarrier is bounded; on expiry the CTA sets TQ_DEVERR_TIMEOUT, drains and frees TMEM.
#include <math.h>

#include <algorithm>

#include "latent.cuh"
#include "tensor.cuh"

namespace tq {
namespace {

using namespace tc;

constexpr int kRows = 128, kStreams = 2, kTile = kRows * kStreams, kTok = 128;
constexpr int kSoft = 4 * kStreams, kMma = kSoft, kCopy = kSoft + 1, kGuard = kSoft + 2, kWarps = kSoft + 4;  // 12: 168 registers
constexpr uint32_t kUnit = kTok * 128;  // bytes of 128 rows of 64 elements
constexpr int kUnits = 8, kQUnits = kHeadQuery / 64, kVUnits = kHeadValue / 64, kStep = kQUnits + kVUnits;
constexpr uint32_t kRing = kStreams * kQUnits * kUnit, kControl = kRing + kUnits * kUnit;
constexpr uint32_t kSmem = kControl + 1024 + 1024;  // the last for the start's alignment
static_assert(kUnits == 8 && kStep == 5, "the ring's reuse below");

struct PromptArgs {
    int64_t Tq, Tkv, kvh;
    const int32_t* q_starts;
    const int32_t* kv_starts;
    uint16_t* o;
    uint32_t* err;
    int B, H;
    bool causal;
    float scale2;  // scale * log2(e)
    long long wait_cycles;
};

// Of a CTA: its rows and keys as places of the packed arrays, and what its first row stands at.
struct Job {
    int q0, rows;   // rows in use
    int k0, keys;   // of the sequence
    int at;         // key of the first row's own place, less k0; the rows' are at + row (causal)
};
TQ_DEVFN bool span(const PromptArgs& a, int b, int& q0, int& q1, int& k0, int& k1) {
    q0 = a.q_starts[b], q1 = a.q_starts[b + 1], k0 = a.kv_starts[b], k1 = a.kv_starts[b + 1];
    return q0 >= 0 && q0 <= q1 && q1 <= a.Tq && k0 >= 0 && k0 <= k1 && k1 <= a.Tkv;
}
// Tile `at` of the batch, counted from the last (late rows of a sequence see most: they go first); rows 0 where there is none (one
// warp).
TQ_DEVFN Job find_job(const PromptArgs& a, int at, bool report) {
    const int lane = threadIdx.x & 31;
    Job j{};
    bool bad = false;
    for (int end = a.B; end > 0; end -= 32) {  // sequences end - 1, end - 2, ...
        const int b = end - 1 - lane;
        int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
        bool ok = b >= 0 && span(a, b, q0, q1, k0, k1);
        bad |= b >= 0 && !ok;
        const int tiles = ok ? (q1 - q0 + kTile - 1) / kTile : 0;
        int upto = tiles;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int x = __shfl_up_sync(kFull, upto, m);
            if (lane >= m) upto += x;
        }
        const unsigned hit = __ballot_sync(kFull, upto > at);
        if (hit && j.rows == 0) {
            const int src = __ffs(hit) - 1;
            const int tile = __shfl_sync(kFull, tiles, src) - 1 - (at - __shfl_sync(kFull, upto - tiles, src));
            q0 = __shfl_sync(kFull, q0, src), q1 = __shfl_sync(kFull, q1, src);
            k0 = __shfl_sync(kFull, k0, src), k1 = __shfl_sync(kFull, k1, src);
            j.q0 = q0 + tile * kTile;
            j.rows = min(kTile, q1 - j.q0);
            j.k0 = k0;
            j.keys = k1 - k0;
            j.at = j.keys - (q1 - q0) + tile * kTile;
            if (!report) break;
        }
        at -= __shfl_sync(kFull, upto, 31);
    }
    if (report && bad && a.err) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
    return j;
}
// Keys that row r of the job sees: the first `seen_by`.
TQ_DEVFN int seen_by(const PromptArgs& a, const Job& j, int r) { return a.causal ? min(max(j.at + r + 1, 0), j.keys) : j.keys; }
// Steps of stream t, and the first step that some row of it sees in part (or that passes the keys' end).
TQ_DEVFN int steps_of(const PromptArgs& a, const Job& j, int t) {
    const int last = min(j.rows, (t + 1) * kRows) - 1;
    return last < t * kRows ? 0 : (seen_by(a, j, last) + kTok - 1) / kTok;
}
TQ_DEVFN int whole_of(const PromptArgs& a, const Job& j, int t) { return seen_by(a, j, t * kRows) / kTok; }

struct Control {
    uint64_t q_full[kStreams], k_full[2], v_full[2], k_empty[2], v_empty[2], guarded[2];  // [2]: of even and odd steps
    uint64_t s_ready[kStreams], p_ready[kStreams], o_done[kStreams], drain;
    uint32_t odd[2][4];  // values of a step that are not finite
    Job job;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(Control) <= 1024, "control block");

template <bool BF>
__global__ void __launch_bounds__(32 * kWarps, 1)
    latent_prompt_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                         const __grid_constant__ CUtensorMap map_r) {
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t* const smem = raw + (base - smem_u32(raw));
    Control& c = *reinterpret_cast<Control*>(smem + kControl);
    volatile int* abort_flag = &c.abort;
    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31, h = blockIdx.y;

    pdl_trigger();
    if (warp == kMma) {
        if (lane == 0) {
            c.abort = 0;
            for (int i = 0; i < 2; ++i) {
                mbar_init(c.q_full + i, 1);
                mbar_init(c.k_full + i, 1);
                mbar_init(c.v_full + i, 1);
                mbar_init(c.k_empty + i, 1);
                mbar_init(c.v_empty + i, 3);  // the products and the guards
                mbar_init(c.guarded + i, 2);
                mbar_init(c.s_ready + i, 1);
                mbar_init(c.p_ready + i, 128);
                mbar_init(c.o_done + i, 1);
            }
            mbar_init(&c.drain, 1);
            fence_mbar_init();
        }
        __syncwarp();
        alloc512(&c.tmem);
    }
    pdl_wait();
    if (warp == kCopy) {
        const Job j = find_job(a, blockIdx.x, blockIdx.x == 0 && h == 0);
        if (lane == 0) c.job = j;
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = c.tmem;
    const Job j = c.job;
    const int n0 = steps_of(a, j, 0), n1 = steps_of(a, j, 1), n = max(n0, n1);
    // steps from here on are looked through by the guards
    const int part = min(n0 ? whole_of(a, j, 0) : n, n1 ? whole_of(a, j, 1) : n);

    if (warp == kCopy) {
        // ------------------------------------------------------------ tensor copies
        bool ok = true;
        int k_done = 0, v_done = 0;
        if (n && elected()) {
            for (int t = 0; t < kStreams; ++t) {
                mbar_expect_tx(c.q_full + t, kQUnits * kUnit);
                for (int d = 0; d < kQUnits; ++d)
                    tma_load_2d(base + (t * kQUnits + d) * kUnit, &map_q, h * kHeadQuery + d * 64, j.q0 + t * kRows, c.q_full + t);
            }
            for (int i = 0; i < n && ok; ++i) {
                const int e = i & 1, row = j.k0 + i * kTok, x = (int)(h * a.kvh);
                auto unit = [&](int u) { return base + kRing + ((i * kStep + u) % kUnits) * kUnit; };
                // its keys lie where the last keys and the values of two steps before did, its values where keys of the step before did
                if (i >= 2) ok = mbar_wait(c.v_empty + e, ((i - 2) >> 1) & 1, abort_flag, a.wait_cycles);
                if (!ok) break;
                mbar_expect_tx(c.k_full + e, kQUnits * kUnit);
                tma_load_2d(unit(0), &map_k, x, row, c.k_full + e);
                tma_load_2d(unit(1), &map_k, x + 64, row, c.k_full + e);
                tma_load_2d(unit(2), &map_r, 0, row, c.k_full + e);
                ++k_done;
                if (i >= 1) ok = mbar_wait(c.k_empty + (e ^ 1), ((i - 1) >> 1) & 1, abort_flag, a.wait_cycles);
                if (!ok) break;
                mbar_expect_tx(c.v_full + e, kVUnits * kUnit);
                tma_load_2d(unit(3), &map_v, x, row, c.v_full + e);
                tma_load_2d(unit(4), &map_v, x + 64, row, c.v_full + e);
                ++v_done;
            }
            // no copy may be in flight when the CTA ends (on an abort: nobody else has waited for them)
            for (int t = 0; t < kStreams; ++t) mbar_wait_drain(c.q_full + t, 0);
            for (int i = max(k_done - 2, 0); i < k_done; ++i) mbar_wait_drain(c.k_full + (i & 1), (i >> 1) & 1);
            for (int i = max(v_done - 2, 0); i < v_done; ++i) mbar_wait_drain(c.v_full + (i & 1), (i >> 1) & 1);
        }
        __syncwarp();
    } else if (warp == kMma) {
        // ------------------------------------------------------------ MMA issue
        if (elected()) {
            const uint64_t dq = desc(base, 16), dk = desc(base + kRing, 16), dv = desc(base + kRing, kUnit);
            auto scores = [&](int t, int i) {
                if (!mbar_wait(c.k_full + (i & 1), (i >> 1) & 1, abort_flag, a.wait_cycles)) return false;
                fence_after();
                constexpr uint32_t id = idesc(BF, kRows, kTok, 0);
#pragma unroll
                for (int d = 0; d < kQUnits; ++d) {
                    const uint64_t from = dk + (uint32_t)((i * kStep + d) % kUnits) * (kUnit / 16);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss(tmem + 256 * t, dq + (t * kQUnits + d) * (kUnit / 16) + 2 * k, from + 2 * k, id, (d | k) != 0);
                }
                commit(c.s_ready + t);
                if (t == 1 || i >= n1) commit(c.k_empty + (i & 1));  // the last to read these keys
                return true;
            };
            bool ok = true;
            if (n0) ok = mbar_wait(c.q_full, 0, abort_flag, a.wait_cycles) && scores(0, 0);
            if (n1 && ok) ok = mbar_wait(c.q_full + 1, 0, abort_flag, a.wait_cycles) && scores(1, 0);
            for (int i = 0; i < n && ok; ++i)
#pragma unroll
                for (int t = 0; t < kStreams; ++t) {
                    if (!ok || i >= (t ? n1 : n0)) continue;
                    ok = mbar_wait(c.v_full + (i & 1), (i >> 1) & 1, abort_flag, a.wait_cycles) &&
                         (i < part || mbar_wait(c.guarded + (i & 1), (i >> 1) & 1, abort_flag, a.wait_cycles)) &&
                         mbar_wait(c.p_ready + t, i & 1, abort_flag, a.wait_cycles);
                    if (!ok) break;
                    fence_after();
                    constexpr uint32_t id = idesc(BF, kRows, kHeadValue, 1);
                    // (its two units may lie at the ring's end and start: then each is a product of its own)
                    const uint32_t u = (uint32_t)(i * kStep + kQUnits) % kUnits;
                    const uint64_t from = dv + u * (kUnit / 16);
#pragma unroll
                    for (int k = 0; k < kTok / 16; ++k) {
                        if (u + 1 < kUnits) {
                            mma_ts(tmem + 256 * t + 128, tmem + 256 * t + 8 * k, from + 128 * k, id, (i | k) != 0);
                        } else {
                            mma_ts(tmem + 256 * t + 128, tmem + 256 * t + 8 * k, from + 128 * k, idesc(BF, kRows, 64, 1), (i | k) != 0);
                            mma_ts(tmem + 256 * t + 192, tmem + 256 * t + 8 * k, dv + 128 * k, idesc(BF, kRows, 64, 1), (i | k) != 0);
                        }
                    }
                    commit(c.o_done + t);
                    if (t == 1 || i >= n1) commit(c.v_empty + (i & 1));
                    if (i + 1 < (t ? n1 : n0)) ok = scores(t, i + 1);
                }
            commit(&c.drain);  // completes when every MMA issued above has finished
            if (!mbar_wait_drain(&c.drain, 0)) *abort_flag = 1;
        }
        __syncwarp();
    } else if (warp >= kGuard) {
        // ------------------------------------------------------------ guards: a thread to two tokens
        const int id = tid - kGuard * 32;
        bool ok = true;
        for (int i = 0; i < n && ok; ++i) {
            const int e = i & 1;
            ok = __all_sync(kFull, mbar_wait(c.v_full + e, (i >> 1) & 1, abort_flag, a.wait_cycles));
            if (!ok) break;
            if (i >= part) {
                bool wrote = false;
                for (int z = 0; z < 2; ++z) {
                    const int t = id + 64 * z;
                    uint8_t* rows[2];
                    for (int d = 0; d < 2; ++d) rows[d] = smem + kRing + ((i * kStep + kQUnits + d) % kUnits) * kUnit + t * 128;
                    bool odd = false, wipe = i * kTok + t >= j.keys;
                    constexpr uint32_t kTop = BF ? 0x7f80u : 0x7c00u;
                    for (int d = 0; d < 2 && !wipe; ++d)
#pragma unroll
                        for (int p = 0; p < 8; ++p) {
                            const uint4 v = *reinterpret_cast<const uint4*>(rows[d] + ((p + t) & 7) * 16);
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int q = 0; q < 4; ++q) odd |= (w[q] & kTop) == kTop || ((w[q] >> 16) & kTop) == kTop;
                        }
                    const uint32_t bits = __ballot_sync(kFull, odd);
                    if (lane == 0) c.odd[e][2 * z + warp - kGuard] = bits;
                    if (wipe || odd) {
                        wrote = true;
                        for (int d = 0; d < 2; ++d)
#pragma unroll
                            for (int p = 0; p < 8; ++p)
                                *reinterpret_cast<uint4*>(rows[d] + ((p + t) & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                if (wrote) fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(c.guarded + e);
                mbar_arrive(c.v_empty + e);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax: a thread to a row
        const int t = warp >> 2, row = t * kRows + (warp & 3) * 32 + lane, steps = t ? n1 : n0, whole = steps ? whole_of(a, j, t) : 0;
        const uint32_t at = tmem + 256 * t + ((uint32_t)(warp & 3) << 21), col_o = at + 128;
        const int seen = row < j.rows ? seen_by(a, j, row) : 0;
        const f2 ff = pk(a.scale2, a.scale2);
        float m = -INFINITY, sum = 0.f, bias = 0.f;
        bool ok = true;
        for (int i = 0; i < steps; ++i) {
            ok = __all_sync(kFull, mbar_wait(c.s_ready + t, i & 1, abort_flag, a.wait_cycles));
            if (!ok) break;
            fence_after();
            uint32_t s[128];
#pragma unroll
            for (int q = 0; q < 4; ++q) ld32(at + 32 * q, s + 32 * q);
            wait_ld();
#pragma unroll
            for (int k = 0; k < 64; ++k) {
                const float2 y = un(mul2(pk(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), ff));
                s[2 * k] = __float_as_uint(y.x);
                s[2 * k + 1] = __float_as_uint(y.y);
            }
            bool spoilt = false;
            if (i >= whole) {
                const int limit = seen - i * kTok;  // keys of this step that the row sees
#pragma unroll
                for (int k = 0; k < 128; ++k)
                    if (k >= limit) s[k] = __float_as_uint(-INFINITY);
            }
            if (i >= part) {
                ok = __all_sync(kFull, mbar_wait(c.guarded + (i & 1), (i >> 1) & 1, abort_flag, a.wait_cycles));
                if (!ok) break;
                const int limit = seen - i * kTok;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int bits = min(max(limit - 32 * w, 0), 32);
                    spoilt |= (c.odd[i & 1][w] & (bits == 32 ? ~0u : (1u << bits) - 1)) != 0;
                }
            }
            float x4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x4[k] = __uint_as_float(s[k]);
#pragma unroll
            for (int k = 4; k < 124; k += 8)
#pragma unroll
                for (int z = 0; z < 4; ++z) x4[z] = fmaxf(fmaxf(x4[z], __uint_as_float(s[k + z])), __uint_as_float(s[k + z + 4]));
#pragma unroll
            for (int k = 124; k < 128; ++k) x4[k & 3] = fmaxf(x4[k & 3], __uint_as_float(s[k]));
            const float top = fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3]));
            if (__any_sync(kFull, top - m > Weights<BF>::kSlack)) {
                // (each row by its own scores alone: its result must not hang on what its neighbours see)
                const float to_m = top - m > Weights<BF>::kSlack ? top : m, to = Weights<BF>::bias(to_m);
                const float r = m == -INFINITY ? 0.f : exp2_fast(to - bias);
                m = to_m;
                bias = to;
                sum *= r;
                if (i) {  // the sums so far, once the last product has written them
                    ok = __all_sync(kFull, mbar_wait(c.o_done + t, (i - 1) & 1, abort_flag, a.wait_cycles));
                    if (!ok) break;
                    fence_after();
#pragma unroll 1
                    for (int q = 0; q < 16; ++q) {
                        uint32_t o[8];
                        ld8(col_o + 8 * q, o);
                        wait_ld();
#pragma unroll
                        for (int z = 0; z < 8; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * r);
                        st8(col_o + 8 * q, o);
                    }
                }
            }
            // ---- weights; the sum takes them before their rounding
            const f2 bb = pk(bias, bias);
            f2 ls[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < 64; ++k) {
                const float2 y = un(add2(pk(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), bb));
                const float u = exp2_fast(y.x), v = exp2_fast(y.y);
                ls[k & 1] = add2(ls[k & 1], pk(u, v));
                s[k] = pack16<BF>(u, v);
                if ((k & 31) == 31) st32(at + (k & 32), s + (k & 32));
            }
            const float2 z = un(add2(ls[0], ls[1]));
            sum += z.x + z.y;
            if (spoilt) sum = NAN;
            wait_st();
            fence_before();
            mbar_arrive(c.p_ready + t);
        }
        if (ok && steps) {
            ok = __all_sync(kFull, mbar_wait(c.o_done + t, (steps - 1) & 1, abort_flag, a.wait_cycles));
            fence_after();
        }
        if (ok) {
            const float over = sum == 0.f ? 0.f : 1.f / sum;  // (a NaN sum stays one)
            uint16_t* out = a.o + ((int64_t)(j.q0 + row) * a.H + h) * kHeadValue;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                uint32_t o[32];
                if (steps) {
                    ld32(col_o + 32 * q, o);
                    wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[e] = pack16<BF>(__uint_as_float(o[2 * e]) * over, __uint_as_float(o[2 * e + 1]) * over);
                if (row < j.rows) {  // whole 32-byte sectors
                    stg256(reinterpret_cast<float*>(out + 32 * q), reinterpret_cast<const float*>(o));
                    stg256(reinterpret_cast<float*>(out + 32 * q + 16), reinterpret_cast<const float*>(o + 8));
                }
                __syncwarp();
            }
        }
    }

    fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag && a.err) atomicOr(a.err, TQ_DEVERR_TIMEOUT);
    if (warp == kMma) {
        fence_after();
        dealloc512(tmem);
    }
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" tq_status tq_latent_attend_prompt(const void* q, int64_t q_stride, const void* k, const void* v, int64_t kv_stride,
                                             int64_t kv_head_stride, const void* k_rope, int64_t k_rope_stride, tq_dtype dt,
                                             int32_t B, int32_t H, int64_t Tq, int64_t Tkv, const int32_t* q_starts,
                                             const int32_t* kv_starts, int32_t causal, float scale, void* o, uint32_t* err,
                                             void* stream) {
    if (B < 0 || H <= 0 || H > 65535 || Tq < 0 || Tkv < 0 || !isfinite(scale)) return TQ_ERR_INVALID;
    if (!(dt == TQ_BF16 || dt == TQ_F16 || dt == TQ_F32)) return TQ_ERR_INVALID;
    if (dt == TQ_F32 || Tq > 1ll << 30 || Tkv > 1ll << 30) return TQ_ERR_UNSUPPORTED;
    if (q_stride < (int64_t)H * kHeadQuery || kv_head_stride < kHeadKey || kv_stride < (H - 1) * kv_head_stride + kHeadKey ||
        k_rope_stride < kLatentRope || q_stride % 8 || kv_stride % 8 || kv_head_stride % 8 || k_rope_stride % 8)
        return TQ_ERR_INVALID;
    if (q_stride > 1ll << 32 || kv_stride > 1ll << 32 || k_rope_stride > 1ll << 32) return TQ_ERR_UNSUPPORTED;
    if (B == 0 || Tq == 0) return TQ_OK;
    if (!q || !o || !q_starts || !kv_starts || (Tkv && (!k || !v || !k_rope))) return TQ_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_rope, 16) || !aligned(o, 32) || !aligned(q_starts, 4) ||
        !aligned(kv_starts, 4))
        return TQ_ERR_INVALID;
    PromptArgs a{};
    a.Tq = Tq;
    a.Tkv = Tkv;
    a.kvh = kv_head_stride;
    a.q_starts = q_starts;
    a.kv_starts = kv_starts;
    a.o = reinterpret_cast<uint16_t*>(o);
    a.err = err;
    a.B = B;
    a.H = H;
    a.causal = causal != 0;
    a.scale2 = scale * 1.4426950408889634f;
    a.wait_cycles = wait_budget();
    const bool bf = dt == TQ_BF16;
    CUtensorMap mq, mk, mv, mr;
    const int64_t cols = (H - 1) * kv_head_stride + kHeadKey, keys = std::max<int64_t>(Tkv, 1);
    // (without keys no copy is made: any address serves)
    if (!tensor_map(&mq, bf, q, Tq, (int64_t)H * kHeadQuery, q_stride, kRows) ||
        !tensor_map(&mk, bf, Tkv ? k : q, keys, cols, kv_stride, kTok) || !tensor_map(&mv, bf, Tkv ? v : q, keys, cols, kv_stride, kTok) ||
        !tensor_map(&mr, bf, Tkv ? k_rope : q, keys, kLatentRope, k_rope_stride, kTok))
        return TQ_ERR_CUDA;
    const int64_t tiles = (Tq + kTile - 1) / kTile + B;  // at most
    if (tiles > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
    void (*kernel)(PromptArgs, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap) =
        bf ? latent_prompt_kernel<true> : latent_prompt_kernel<false>;
    if (ensure_smem((const void*)kernel, kSmem) != cudaSuccess) return TQ_ERR_CUDA;
    return launch_pdl(kernel, dim3((unsigned)std::min<int64_t>(tiles, Tq), (unsigned)H), dim3(32 * kWarps), kSmem, as_stream(stream), a, mq, mk, mv, mr);
}
