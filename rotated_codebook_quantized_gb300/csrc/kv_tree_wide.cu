// The cached context of tq_kv_attend_tree for more than 16 query rows to a kv head, on the 5th-generation tensor cores.
//
// A persistent CTA takes a run of 64-token steps.  Each step is decoded once into shared memory, as fp16 keys (K-major)
// and values (MN-major, so that neither needs a transpose), for one or two tiles of 128 query rows:
//   scores   S[128 x 64]   = Q (TMEM, fp16) . K^T (shared)          8 MMAs of K = 16
//   weights  P = exp2(S f - m), fp16, written over S in TMEM        one thread to a row
//   values   O[128 x 128] += P (TMEM) . V (shared)                  4 MMAs of K = 16
// Roles: four softmax warps to a tile, eight decoder warps (8 tokens of a step each, fed by their own cp.async rings), one
// thread issuing MMAs.  Operands from TMEM leave the shared-memory bandwidth to the decoders' table reads and stores and to
// the tensor cores' reads of K and V.  A row's running maximum follows only when a score passes it by 2^kSlack, so O is
// seldom rescaled.  Every wait on an mbarrier is bounded; on expiry the CTA sets TQ_DEVERR_TIMEOUT, drains and frees TMEM.
#include <math.h>

#include "kv_tree.cuh"

using namespace tq;
using namespace tq::tree;

namespace {

constexpr int kTok = 64;       // tokens of a step
constexpr int kUnit = 8;       // of a decoder warp
constexpr int kDec = kTok / kUnit;
constexpr int kStages = 3;     // decoded steps
constexpr int kDepth = 3;      // units of a decoder's ring: two in flight while one is decoded
constexpr uint32_t kTile = kTok * kPD * 2;  // bytes of a step's keys, or values
constexpr uint32_t kHalf = kTile / 2;       // of 64 of their dims (one 128-byte swizzled row a token)

// Shared addresses: the decode table starts at 64 K (see kv_tree.cu's kernel: one byte permute builds an entry's address),
// rings and barriers lie below it, the decoded steps above.
constexpr uint32_t kTable = 65536, kSteps = 131072, kEnd = kSteps + kStages * 2 * kTile;
constexpr uint32_t kStart = 1024 + 512;  // the system's first KB, then the static variables
constexpr uint32_t kFactors = kStart, kRings = kFactors + 256 * 4;
static_assert(kEnd <= 232448, "fits an SM");

template <int KL, int VL>
struct Unit {  // of a ring: 8 tokens' codes and scales
    static constexpr uint32_t kKRow = KvBook<KL>::kWords * 4, kVRow = KvBook<VL>::kWords * 4;
    static constexpr uint32_t kK = 0, kV = kUnit * kKRow, kKs = kV + kUnit * kVRow, kVs = kKs + 128, kBytes = kVs + 128;
    static_assert(kBytes % 16 == 0 && kRings + kDec * kDepth * kBytes <= kTable, "rings below the table");
};

TQ_DEVFN void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
TQ_DEVFN void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
TQ_DEVFN void tc_commit(uint64_t* b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(b))
                 : "memory");
}
// D (TMEM) (+)= A (TMEM) . B (shared, by descriptor); fp16 operands, fp32 sums.
TQ_DEVFN void tc_mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accum)
        : "memory");
}
// 128-byte swizzled tiles whose 8-row atoms lie 1024 bytes apart.  Keys: K-major rows of 64 dims (the leading offset is not
// used).  Values: MN-major, atoms of 64 dims by 8 tokens; the next 64 dims are kHalf bytes on (the leading offset).
TQ_DEVFN uint64_t desc(uint32_t addr, uint32_t leading) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(leading >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16: D fp32, A and B fp16, M = 128; B MN-major where mn is set.
constexpr uint32_t idesc(int n, int mn) {
    return (1u << 4) | ((uint32_t)mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

#define TQ_O8(i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), \
                 "=r"(v[i + 6]), "=r"(v[i + 7])
#define TQ_I8(i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), \
                 "r"(v[i + 7])
#define TQ_L32 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, " \
               "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31}"
// 32 columns of the warp's 32 TMEM lanes; the loads are complete after tc_wait_ld.
TQ_DEVFN void tc_ld32(uint32_t at, uint32_t* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " TQ_L32 ", [%32];"
                 : TQ_O8(0), TQ_O8(8), TQ_O8(16), TQ_O8(24)
                 : "r"(at)
                 : "memory");
}
TQ_DEVFN void tc_st32(uint32_t at, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " TQ_L32 ";" ::TQ_I8(0), TQ_I8(8), TQ_I8(16), TQ_I8(24), "r"(at)
        : "memory");
}
#undef TQ_O8
#undef TQ_I8
#undef TQ_L32
TQ_DEVFN void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
TQ_DEVFN void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
TQ_DEVFN void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <int T>
constexpr int kThreads = 32 * (4 * T + kDec + 1);

template <int KL, int VL, int T>
__global__ void __launch_bounds__(kThreads<T>, 1) kv_tree_wide_kernel(TreeArgs a) {
    using U = Unit<KL, VL>;
    constexpr int kSoft = 4 * T, kMma = kSoft + kDec, kRows = 128 * T;
    // TMEM columns: T = 1: sums, queries, two score buffers; T = 2: sums, queries, scores of each tile
    constexpr uint32_t kO = 0, kQ = 128 * T, kS = kQ + 64 * T;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* const space = smem - (uint32_t)__cvta_generic_to_shared(smem);  // shared address 0
    float* factors = reinterpret_cast<float*>(space + kFactors);            // [kRows] from a row's products to log2 scores
    // S and P alternate between two places: of the step's parity (T = 1), or of the tile (T = 2)
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], s_ready[2], p_ready[2], o_done[2], drain;
    __shared__ __align__(8) uint8_t valid[kStages][kDec];  // tokens of each unit of a decoded step, a bit each
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word, s_b;
    __shared__ Work s_before;
    __shared__ long long s_total;
    volatile int* abort_flag = &abort_word;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_trigger();
    if (warp == kMma) {
        if (lane == 0) {
            abort_word = 0;
            for (int s = 0; s < kStages; ++s) {
                mbar_init(full + s, 32 * kDec);
                mbar_init(empty + s, 1);
            }
            for (int s = 0; s < 2; ++s) {
                mbar_init(s_ready + s, 1);
                mbar_init(p_ready + s, 128);
                mbar_init(o_done + s, 1);
            }
            mbar_init(&drain, 1);
            fence_mbar_init();
        }
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 0) {
        Work w;
        long long total;
        count_work(a, 0, w, total);
        int b;
        find_run(a, blockIdx.x * steps_per_cta(a, total), w, b);
        if (lane == 0) {
            s_before = w;
            s_total = total;
            s_b = b;
        }
    }
    // The decode table, as in the 16-row kernel: row c of 256 bytes holds, a copy for each lane, the fp16 centroid of key
    // code c (or of both 4-bit codes of byte c) over a power of two, and in its upper half the pair of two 4-bit values.
    const int ek = exponent_above(fmaxf(fabsf(a.c.kcent[0]), fabsf(a.c.kcent[KL - 1])));
    const int ev = exponent_above(fmaxf(fabsf(a.c.vcent[0]), fabsf(a.c.vcent[VL - 1])));
    const float kd = exp2f((float)-ek), vd = exp2f((float)-ev);
    for (int c = warp; c < 256; c += kMma + 1) {
        uint32_t* row = reinterpret_cast<uint32_t*>(space + kTable + c * 256);
        row[lane] = KL == 256 ? pack_f16(a.c.kcent[c % KL] * kd, 0.f)
                              : pack_f16(a.c.kcent[(c & 15) % KL] * kd, a.c.kcent[(c >> 4) % KL] * kd);
        if (VL == 16) row[32 + lane] = pack_f16(a.c.vcent[(c & 15) % VL] * vd, a.c.vcent[(c >> 4) % VL] * vd);
    }
    uint32_t tl[2] = {0, 0}, th[2] = {0, 0};  // low and high bytes of an 8-level value book
    if (VL == 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t h = __half_as_ushort(__float2half_rn(a.c.vcent[i % VL] * vd));
            tl[i >> 2] |= (h & 255u) << (8 * (i & 3));
            th[i >> 2] |= (h >> 8) << (8 * (i & 3));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    const long long total = s_total, per = steps_per_cta(a, total);
    long long p = blockIdx.x * per;
    const long long pend = min(p + per, total);
    int b = s_b;
    long long base = s_before.steps;
    int ubase = s_before.units;
    uint32_t g = 0;  // steps of this CTA so far: the phase of every barrier
    const int ng = kPD >> a.c.lgroup;

    // decoder state that outlives a segment
    const int d = warp - kSoft;
    const uint32_t ring = kRings + (d > 0 ? d : 0) * kDepth * U::kBytes, ring_end = ring + kDepth * U::kBytes;

    while (p < pend) {
        int steps = seq_steps(a, b), tiles = seq_tiles(a, b);
        while (p >= base + (long long)steps * tiles * a.c.Hkv) {  // into the next sequence that has any
            base += (long long)steps * tiles * a.c.Hkv;
            ubase += tiles * a.c.Hkv;
            ++b;
            steps = seq_steps(a, b);
            tiles = seq_tiles(a, b);
        }
        const int unit = (int)((p - base) / steps);
        const int s0 = (int)(p - base - (long long)unit * steps);
        const int s1 = (int)min((long long)steps, s0 + (pend - p));
        const int h = unit / tiles, tile = unit - h * tiles;
        const int len = seq_len(a, b), rows = min(kRows, seq_live(a, b) * a.ratio - tile * kRows);

        // ---- decoders: the first copies are under way while the queries are turned
        const int32_t* tab = a.table + (int64_t)b * a.table_stride;
        auto page_of = [&](int st) {
            const int t = st * kTok + d * kUnit;
            return st < s1 && t < len ? __ldg(tab + (t >> a.c.lpage)) : -1;
        };
        int ahead = s0, page_next = -1;
        uint32_t fill = ring, counts = 0;  // four bits a step: valid tokens of the unit
        auto issue = [&]() {
            const int page = page_next, t = ahead * kTok + d * kUnit;
            page_next = page_of(ahead + 1);
            counts <<= 4;
            if (ahead < s1 && t < len) {
                if ((uint32_t)page < (uint32_t)a.c.pages) {
                    counts |= (uint32_t)min(len - t, kUnit);
                    const uint32_t row8 = (uint32_t)page * (uint32_t)(a.c.page_stride >> 3) +
                                          (uint32_t)h * (uint32_t)(a.c.head_stride >> 3) + ((t & ((1 << a.c.lpage) - 1)) >> 3);
                    const uint8_t* k = reinterpret_cast<const uint8_t*>(a.c.kcodes) + (uint64_t)row8 * (kUnit * U::kKRow) + lane * 16;
                    cp16(fill + U::kK + lane * 16, k);
                    if (KL == 256) cp16(fill + U::kK + lane * 16 + 512, k + 512);
                    if (lane < kUnit * (int)U::kVRow / 16)
                        cp16(fill + U::kV + lane * 16,
                             reinterpret_cast<const uint8_t*>(a.c.vcodes) + (uint64_t)row8 * (kUnit * U::kVRow) + lane * 16);
                    if ((lane & 7) < ng && lane < 16)
                        cp16(fill + (lane < 8 ? U::kKs : U::kVs) + (lane & 7) * 16,
                             reinterpret_cast<const uint8_t*>(lane < 8 ? a.c.kscales : a.c.vscales) +
                                 (uint64_t)row8 * (uint32_t)(kUnit * 2 * ng) + (lane & 7) * 16);
                } else if (lane == 0 && a.err) {
                    atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            ++ahead;
            fill = fill + U::kBytes == ring_end ? ring : fill + U::kBytes;
        };
        if (d >= 0 && d < kDec) {
            page_next = page_of(s0);
#pragma unroll
            for (int i = 0; i < kDepth - 1; ++i) issue();
        }

        // ---- queries: rotated, over a power of two of their own, fp16, through the decoded steps' memory into TMEM
        if (warp != kMma) {
#pragma unroll 2
            for (int row = warp; row < kRows; row += kMma) {
                float v[4] = {0.f, 0.f, 0.f, 0.f};
                if (row < rows) {
                    const int x = tile * kRows + row, i = x / a.ratio, gq = x - i * a.ratio;
                    const uint2 raw = *reinterpret_cast<const uint2*>(a.q + ((int64_t)b * a.n + i) * a.qs +
                                                                      (int64_t)(h * a.ratio + gq) * kPD + lane * 4);
                    const uint32_t sg = *reinterpret_cast<const uint32_t*>(a.c.signs + lane * 4);
                    v[0] = __uint_as_float(raw.x << 16) * (float)(int8_t)sg;
                    v[1] = __uint_as_float(raw.x & 0xffff0000u) * (float)(int8_t)(sg >> 8);
                    v[2] = __uint_as_float(raw.y << 16) * (float)(int8_t)(sg >> 16);
                    v[3] = __uint_as_float(raw.y & 0xffff0000u) * (float)(int8_t)(sg >> 24);
                    fwht_warp128(v);
                }
                float mx = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
                for (int m = 16; m; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, m));
                const int e = exponent_above(mx);
                const float dn = a.scale2 < 0.f ? -exp2f((float)-e) : exp2f((float)-e);  // the factor below is not negative
                // 16-byte pieces of a row are swapped by its number: the reader is a thread to a row
                *reinterpret_cast<uint2*>(space + kSteps + row * 256 + (((lane >> 1) ^ (row & 7)) << 4) + (lane & 1) * 8) =
                    make_uint2(pack_f16(v[0] * dn, v[1] * dn), pack_f16(v[2] * dn, v[3] * dn));
                if (lane == 0) factors[row] = exp2f((float)(e + ek)) * (kInvSqrtD * fabsf(a.scale2));
            }
        }
        __syncthreads();
        const int row = warp * 32 + lane;  // softmax threads: of the CTA's rows
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's TMEM lanes
        const uint32_t col_o = tmem + kO + (warp >> 2) * 128 + lanes;
        float f = 0.f;
        if (warp < kSoft) {
            f = factors[row];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t w[32];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint4 x = lds128(kSteps + row * 256 + (((8 * half + c) ^ (row & 7)) << 4));
                    w[4 * c] = x.x, w[4 * c + 1] = x.y, w[4 * c + 2] = x.z, w[4 * c + 3] = x.w;
                }
                tc_st32(tmem + kQ + (warp >> 2) * 64 + 32 * half + lanes, w);
            }
            tc_wait_st();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();

        if (warp == kMma) {
            // -------------------------------------------------------- MMA issue
            if (lane == 0) {
                auto scores = [&](uint32_t i, int t) {  // of the CTA's step i, tile t
                    const uint32_t at = kSteps + (i % kStages) * 2 * kTile, to = tmem + kS + 64 * (T == 1 ? i & 1 : t);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        tc_mma_ts(to, tmem + kQ + 64 * t + 8 * k, desc(at + (k >> 2) * kHalf, 16) + 2 * (k & 3), idesc(kTok, 0), k != 0);
                    tc_commit(s_ready + (T == 1 ? i & 1 : t));
                };
                auto values = [&](uint32_t i, int t, bool first) {
                    const uint32_t at = kSteps + (i % kStages) * 2 * kTile + kTile, from = tmem + kS + 64 * (T == 1 ? i & 1 : t);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_ts(tmem + kO + 128 * t, from + 8 * k, desc(at + 2048 * k, kHalf), idesc(kPD, 1), !first || k != 0);
                };
                auto wait_full = [&](uint32_t i) {
                    const bool ok = mbar_wait(full + i % kStages, (i / kStages) & 1, abort_flag, a.wait_cycles);
                    tc_fence_after();
                    return ok;
                };
                const uint32_t ge = g + (s1 - s0);
                bool ok = wait_full(g);
                if (ok)
                    for (int t = 0; t < T; ++t) scores(g, t);
                for (uint32_t i = g; i < ge && ok; ++i) {
                    if (T == 1 && i + 1 < ge) {
                        // the other score buffer still held the weights of step i - 1
                        ok = wait_full(i + 1) && (i == g || mbar_wait(o_done, (i - 1) & 1, abort_flag, a.wait_cycles));
                        if (!ok) break;
                        tc_fence_after();
                        scores(i + 1, 0);
                    }
                    for (int t = 0; t < T; ++t) {
                        ok = mbar_wait(p_ready + (T == 1 ? i & 1 : t), T == 1 ? (i >> 1) & 1 : i & 1, abort_flag, a.wait_cycles);
                        if (!ok) break;
                        tc_fence_after();
                        values(i, t, i == g);
                        tc_commit(o_done + t);
                        if (t == T - 1) tc_commit(empty + i % kStages);
                        if (T == 2 && i + 1 < ge) {
                            // the scores go where the weights were read from
                            ok = (t || wait_full(i + 1)) && mbar_wait(o_done + t, i & 1, abort_flag, a.wait_cycles);
                            if (!ok) break;
                            tc_fence_after();
                            scores(i + 1, t);
                        }
                    }
                }
            }
            __syncwarp();
        } else if (warp < kSoft) {
            // -------------------------------------------------------- softmax: a thread to a row
            const int t = warp >> 2;
            const bool idle = (warp & 3) * 32 + t * 128 >= rows;  // no row of this warp is in use
            float m = -INFINITY, l = 0.f, bias = 0.f;
            bool ok = true;
            for (uint32_t i = g; i < g + (s1 - s0) && ok; ++i) {
                const int buf = T == 1 ? i & 1 : t;
                const uint32_t at = tmem + kS + 64 * buf + lanes;
                // (the decoders' barrier has long completed; waiting on it too orders their `valid` before the read)
                ok = mbar_wait(s_ready + buf, T == 1 ? (i >> 1) & 1 : i & 1, abort_flag, a.wait_cycles) &&
                     mbar_wait(full + i % kStages, (i / kStages) & 1, abort_flag, a.wait_cycles);
                if (!__all_sync(kFull, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (!idle) {
                    uint32_t s[64];
                    tc_ld32(at, s);
                    tc_ld32(at + 32, s + 32);
                    tc_wait_ld();
                    const unsigned long long in = *reinterpret_cast<const unsigned long long*>(valid[i % kStages]);
                    if (in != ~0ull) {  // tokens past the end, or of a bad page
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!((in >> c) & 1)) s[c] = __float_as_uint(-INFINITY);
                    }
                    float x[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) x[c] = __uint_as_float(s[c]);
#pragma unroll
                    for (int c = 4; c < 64; ++c) x[c & 3] = fmaxf(x[c & 3], __uint_as_float(s[c]));
                    const float top = f * fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                    if (__any_sync(kFull, top > m + kSlack)) {
                        const float n = fmaxf(m, top), r = m == -INFINITY ? 0.f : fast_exp2(m - n);
                        m = n;
                        bias = m == -INFINITY ? 0.f : -m;
                        l *= r;
                        if (i != g) {  // the sums so far, once the last product has written them
                            ok = mbar_wait(o_done + t, (i - 1) & 1, abort_flag, a.wait_cycles);
                            if (!__all_sync(kFull, ok)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                uint32_t o[32];
                                tc_ld32(col_o + 32 * c, o);
                                tc_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * r);
                                tc_st32(col_o + 32 * c, o);
                            }
                        }
                    }
                    float ls[4] = {0.f, 0.f, 0.f, 0.f};
                    uint32_t w[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float u = fast_exp2(fmaf(__uint_as_float(s[2 * c]), f, bias));
                        const float v = fast_exp2(fmaf(__uint_as_float(s[2 * c + 1]), f, bias));
                        ls[c & 3] += u + v;
                        w[c] = pack_f16(u, v);
                    }
                    l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                    tc_st32(at, w);
                    tc_wait_st();
                }
                tc_fence_before();
                mbar_arrive(p_ready + buf);
            }
            // ---- the run's partial result of this tile
            if (ok) ok = mbar_wait(o_done + t, (g + (s1 - s0) - 1) & 1, abort_flag, a.wait_cycles);
            if (__all_sync(kFull, ok) && !idle) {
                tc_fence_after();
                const int64_t at = ((int64_t)blockIdx.x + ubase + unit) * kRows + row;
                const float vscale = exp2f((float)ev);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32];
                    tc_ld32(col_o + 32 * c, o);
                    tc_wait_ld();
                    if (row < rows) {
                        float4* to = reinterpret_cast<float4*>(a.part + at * kPD + 32 * c);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            to[e] = make_float4(__uint_as_float(o[4 * e]) * vscale, __uint_as_float(o[4 * e + 1]) * vscale,
                                                __uint_as_float(o[4 * e + 2]) * vscale, __uint_as_float(o[4 * e + 3]) * vscale);
                    }
                }
                if (row < rows) a.stat[at] = make_float2(m, l);
                tc_fence_before();
            }
        } else {
            // -------------------------------------------------------- decoders
            const int c = lane & 15, hi = lane >> 4;  // 8 dims of tokens hi, hi + 2, ...
            const uint32_t lane_k = lane * 4 | 0x100, lane_v = lane_k + 128;
            const uint32_t k_at = U::kK + hi * U::kKRow + c * (KL == 256 ? 8 : 4);
            const uint32_t ks_at = U::kKs + (hi * ng + ((8 * c) >> a.c.lgroup)) * 2, vs_at = ks_at + 128;
            // 3-bit values: 8 codes from code `from` of word w0, ten to a word
            const int w0 = (8 * c) / 10, from = (8 * c) % 10;
            const uint32_t v_at = U::kV + hi * U::kVRow + (VL == 8 ? w0 * 4 : c * 4);
            const uint32_t shr = 3 * from, mulr = 1u << (30 - 3 * from);
            // in a decoded step: 64 dims to a half, a 128-byte row to a token, its 16-byte pieces swapped by the token
            const uint32_t to = kSteps + (c >> 3) * kHalf + (d * kUnit + hi) * 128, piece = ((c & 7) ^ hi) * 16;
            uint32_t at = ring;
            bool ok = true;
            for (uint32_t i = g; i < g + (s1 - s0) && ok; ++i) {
                issue();
                asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
                __syncwarp();
                ok = mbar_wait(empty + i % kStages, ((i / kStages) & 1) ^ 1, abort_flag, a.wait_cycles);
                if (!__all_sync(kFull, ok)) {
                    ok = false;
                    break;
                }
                const uint32_t count = (counts >> (4 * (kDepth - 1))) & 15u;
                const uint32_t dst = to + (i % kStages) * 2 * kTile;
#pragma unroll
                for (int q = 0; q < kUnit / 2; ++q) {  // keys of tokens 2 q + hi
                    uint32_t s = lds16(at + ks_at + 4 * q * ng) * 0x10001u;
                    if (count < kUnit && 2 * q + hi >= (int)count) s = 0;  // what lies past the end may be anything
                    uint32_t w[4];
                    if constexpr (KL == 256) {
                        const uint2 x = lds64(at + k_at + 2 * q * U::kKRow);
                        w[0] = prmt(table<0>(x.x, lane_k), table<1>(x.x, lane_k), 0x5410);
                        w[1] = prmt(table<2>(x.x, lane_k), table<3>(x.x, lane_k), 0x5410);
                        w[2] = prmt(table<0>(x.y, lane_k), table<1>(x.y, lane_k), 0x5410);
                        w[3] = prmt(table<2>(x.y, lane_k), table<3>(x.y, lane_k), 0x5410);
                    } else {
                        const uint32_t x = lds32(at + k_at + 2 * q * U::kKRow);
                        w[0] = table<0>(x, lane_k), w[1] = table<1>(x, lane_k);
                        w[2] = table<2>(x, lane_k), w[3] = table<3>(x, lane_k);
                    }
                    sts128(dst + 256 * q + (piece ^ (32 * q)), mul2(w[0], s), mul2(w[1], s), mul2(w[2], s), mul2(w[3], s));
                }
#pragma unroll
                for (int q = 0; q < kUnit / 2; ++q) {  // values
                    uint32_t s = lds16(at + vs_at + 4 * q * ng) * 0x10001u;
                    if (count < kUnit && 2 * q + hi >= (int)count) s = 0;
                    uint32_t w[4];
                    if constexpr (VL == 8) {
                        const uint32_t x = (lds32(at + v_at + 2 * q * U::kVRow) >> shr) + lds32(at + v_at + 2 * q * U::kVRow + 4) * mulr;
                        const uint32_t y = (x & 0x0000ffffu) | ((x << 4) & 0xffff0000u);          // 12 bits to 16
                        const uint32_t z = (y & 0x00ff00ffu) | ((y << 2) & 0xff00ff00u);          // 6 to 8
                        const uint32_t sel = ((z & 0x0f0f0f0fu) | ((z << 1) & 0xf0f0f0f0u)) & 0x77777777u;  // 3 to 4: byte selectors
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t lo = prmt(tl[0], tl[1], sel >> (16 * e)), hb = prmt(th[0], th[1], sel >> (16 * e));
                            w[2 * e] = prmt(lo, hb, 0x5140);
                            w[2 * e + 1] = prmt(lo, hb, 0x7362);
                        }
                    } else {
                        const uint32_t x = lds32(at + v_at + 2 * q * U::kVRow);
                        w[0] = table<0>(x, lane_v), w[1] = table<1>(x, lane_v);
                        w[2] = table<2>(x, lane_v), w[3] = table<3>(x, lane_v);
                    }
                    sts128(dst + kTile + 256 * q + (piece ^ (32 * q)), mul2(w[0], s), mul2(w[1], s), mul2(w[2], s), mul2(w[3], s));
                }
                if (lane == 0) valid[i % kStages][d] = (uint8_t)((1u << count) - 1u);
                fence_async_smem();
                mbar_arrive(full + i % kStages);
                __syncwarp();  // the ring's place is free for the next copy
                at = at + U::kBytes == ring_end ? ring : at + U::kBytes;
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        if (*abort_flag) break;
        g += s1 - s0;
        p += s1 - s0;
    }

    if (warp == kMma && lane == 0) {
        tc_commit(&drain);  // completes when every MMA issued above has finished
        if (!mbar_wait_drain(&drain, 0)) *abort_flag = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag && a.err) atomicOr(a.err, TQ_DEVERR_TIMEOUT);
    if (warp == kMma) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <int KL, int VL, int T>
tq_status launch(const TreeArgs& a, cudaStream_t st) {
    constexpr size_t smem = kEnd - 1024;  // from the start of the dynamic part, wherever it is
    static const bool fits = [] {  // the system's part and the static variables end below kStart
        int dev = 0, reserved = 0;
        cudaFuncAttributes at{};
        return cudaGetDevice(&dev) == cudaSuccess &&
               cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev) == cudaSuccess &&
               cudaFuncGetAttributes(&at, (const void*)kv_tree_wide_kernel<KL, VL, T>) == cudaSuccess && reserved >= 1024 &&
               reserved + at.sharedSizeBytes <= kStart;
    }();
    if (!fits) return TQ_ERR_UNSUPPORTED;
    if (ensure_smem((const void*)kv_tree_wide_kernel<KL, VL, T>, smem) != cudaSuccess) return TQ_ERR_CUDA;
    kv_tree_wide_kernel<KL, VL, T><<<a.ctas, kThreads<T>, smem, st>>>(a);
    return launch_status();
}

template <int T>
tq_status by_books(int kl, int vl, const TreeArgs& a, cudaStream_t st) {
    if (kl == 256) return vl == 8 ? launch<256, 8, T>(a, st) : launch<256, 16, T>(a, st);
    return vl == 8 ? launch<16, 8, T>(a, st) : launch<16, 16, T>(a, st);
}

}  // namespace

namespace tq {
namespace tree {
tq_status launch_wide(int klevels, int vlevels, const TreeArgs& a, cudaStream_t st) {
    return a.trows == 128 ? by_books<1>(klevels, vlevels, a, st) : by_books<2>(klevels, vlevels, a, st);
}
}  // namespace tree
}  // namespace tq
