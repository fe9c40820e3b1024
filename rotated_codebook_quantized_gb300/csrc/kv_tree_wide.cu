// The cached context of tq_kv_attend_tree for more than 16 query rows to a kv head, on the 5th-generation tensor cores.
//
// kv_tree_turn_kernel rotates the query rows once.  Then a persistent CTA takes a run of 32-token steps.  Each step is decoded
// once into shared memory, as fp16 keys (K-major) and values (MN-major, so that neither needs a transpose), for one or two
// tiles of 128 query rows:
//   scores   S[128 x 32]   = Q (TMEM, fp16) . K^T (shared)          8 MMAs of K = 16
//   weights  P = exp2(S f + bias), fp16, written over S in TMEM     one thread to a row
//   values   O[128 x 128] += P (TMEM) . V (shared)                  2 MMAs of K = 16
// Two streams of four softmax warps each, with scores and sums of their own: the two tiles (T = 2), or the even and the odd
// steps of one tile (T = 1), joined at the end of the run.  A stream's scores alternate between two places, so that its
// exponentials run beside its products (one place: 1.9 times as long, the tensor cores and the softmax waiting for one
// another).  Decoder warps take units of 8 tokens in turn, each fed by a cp.async ring of its own; a thread to a stream issues
// its MMAs (an issue costs its thread about 30 cycles).
// Operands from TMEM leave the shared-memory bandwidth to the decoders' table reads and stores and to the tensor cores'
// reads of K and V.  A row's running maximum follows only when a score passes it by 2^kSlack, so O is seldom rescaled.
//
// Bound by the softmax's chain of latencies (1100 of 1290 cycles a step and stream; the products alone take 514) and by issue
// slots (62 % of them): 256 rows to each of 8 heads over 131072 tokens 146 us alone, 940 TFLOP/s, half of the measured bf16 rate
// (the call 156); 32 rows to each of 8 heads of 16 sequences of up to 8192 tokens: 64 us alone, 1.7 TB/s of codes and scales (the
// call 70).
// Every wait on an mbarrier is bounded; on expiry the CTA sets TQ_DEVERR_TIMEOUT, drains and frees TMEM.
#include <math.h>

#include "kv_tree.cuh"

using namespace tq;
using namespace tq::tree;

namespace {

constexpr int kTok = 32;       // tokens of a step
constexpr int kUnit = 8;       // of a unit, which one decoder warp decodes
constexpr int kUnits = kTok / kUnit;
constexpr int kStages = 6;     // decoded steps
constexpr int kDepth = 2;      // units of a decoder's ring: one in flight while one is decoded
constexpr uint32_t kTile = kTok * kPD * 2;  // bytes of a step's keys, or values
constexpr uint32_t kHalf = kTile / 2;       // of 64 of their dims (one 128-byte swizzled row a token)

// Shared addresses: the decode table starts at 64 K (see kv_tree.cu's kernel: one byte permute builds an entry's address),
// rings and barriers lie below it, the decoded steps above.
constexpr uint32_t kTable = 65536, kSteps = 131072, kEnd = kSteps + kStages * 2 * kTile;
constexpr uint32_t kStart = 1024 + 512;  // the system's first KB, then the static variables
constexpr uint32_t kOdd = kStart, kRings = kOdd + 2 * 128 * 4;
// Decoder warps.  Units go to them in turn over all of a CTA's steps, whatever stretches these belong to: a warp's units lie
// kDec / kUnits steps apart, a divisor of kStages, so it comes to the same places of decoded steps in every round and knows a
// place's phase.  (A place's barrier tells only odd from even phases: a warp that left a round of a place out could take a phase
// two back for the one it waits for, as other warps run ahead and the two streams free places out of order.)
constexpr int kDec = 12;
static_assert(kDec % kUnits == 0 && kStages % (kDec / kUnits) == 0, "every place in every round");
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
TQ_DEVFN void tc_ld8(uint32_t at, uint32_t* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : TQ_O8(0) : "r"(at) : "memory");
}
TQ_DEVFN void tc_st8(uint32_t at, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::TQ_I8(0), "r"(at) : "memory");
}
TQ_DEVFN void tc_st16(uint32_t at, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::TQ_I8(
            0),
        TQ_I8(8), "r"(at)
        : "memory");
}
#undef TQ_O8
#undef TQ_I8
#undef TQ_L32
TQ_DEVFN void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
TQ_DEVFN void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// One lane of the (converged) warp.  The compiler knows that a single thread passes, so that what it guards (MMA issue, whose
// operands are uniform registers) is straight code and not a loop over lanes.
TQ_DEVFN bool elected() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
template <int OFF>
TQ_DEVFN void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0+%5], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d), "n"(OFF)
                 : "memory");
}

constexpr int kSoft = 8, kMma = kSoft + kDec, kWarps = kMma + 2;  // 22 warps: 80 registers a thread

// The queries, rotated, over a power of two of their own, times the scale's mantissa, fp16: a warp to a row.  Of a tile of `trows`
// rows the 16-byte pieces
// [16][trows] lie together, a thread of the next kernel reading its row's; the power's exponent beside them.
__global__ void __launch_bounds__(256) kv_tree_turn_kernel(TreeArgs a, int tiles) {
    pdl_trigger();
    const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (at >= (int64_t)a.B * a.n * a.Hq) return;
    const int lane = threadIdx.x & 31;
    const int64_t token = at / a.Hq;
    const int hq = (int)(at - token * a.Hq), b = (int)(token / a.n), i = (int)(token - (int64_t)b * a.n);
    if (i >= seq_live(a, b)) return;
    const int h = hq / a.ratio, y = i * a.ratio + hq - h * a.ratio, tile = y / a.trows, row = y - tile * a.trows;
    const uint2 raw = *reinterpret_cast<const uint2*>(a.q + token * a.qs + (int64_t)hq * kPD + lane * 4);
    const uint32_t sg = *reinterpret_cast<const uint32_t*>(a.c.signs + lane * 4);
    float v[4] = {__uint_as_float(raw.x << 16) * (float)(int8_t)sg, __uint_as_float(raw.x & 0xffff0000u) * (float)(int8_t)(sg >> 8),
                  __uint_as_float(raw.y << 16) * (float)(int8_t)(sg >> 16),
                  __uint_as_float(raw.y & 0xffff0000u) * (float)(int8_t)(sg >> 24)};
    fwht_warp128(v);
    // magnitudes order as their bits
    const float top = __uint_as_float(__reduce_max_sync(
        kFull, max(max(__float_as_uint(fabsf(v[0])), __float_as_uint(fabsf(v[1]))),
                   max(__float_as_uint(fabsf(v[2])), __float_as_uint(fabsf(v[3]))))));
    const int e = exponent_above(top);
    const float d = query_factor(e, a.qmant);  // a negative scale's sign goes here
    const int64_t unit = ((int64_t)b * a.c.Hkv + h) * tiles + tile;
    uint8_t* to = reinterpret_cast<uint8_t*>(a.turned) + ((unit * 16 + (lane >> 1)) * a.trows + row) * 16 + (lane & 1) * 8;
    *reinterpret_cast<uint2*>(to) = make_uint2(pack_f16(v[0] * d, v[1] * d), pack_f16(v[2] * d, v[3] * d));
    if (lane == 0) a.power[unit * a.trows + row] = e;
}

TQ_DEVFN void stg256(float* p, const float* v) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
// A 16-byte asynchronous copy, where `on`.
template <int OFF>
TQ_DEVFN void cp16_if(uint32_t dst, const void* src, bool on) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n @p cp.async.cg.shared.global [%0+%3], [%1], 16;\n}\n" ::"r"(dst), "l"(src),
                 "r"((int)on), "n"(OFF)
                 : "memory");
}

template <int KL, int VL, int T>
__global__ void __launch_bounds__(32 * kWarps, 1) kv_tree_wide_kernel(TreeArgs a, int tiles) {
    using U = Unit<KL, VL>;
    constexpr int kRows = 128 * T, D = kDec;
    // TMEM columns: sums and scores of each stream, queries of each tile
    constexpr uint32_t kO = 0, kS = 256, kQ = 384;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* const space = smem - (uint32_t)__cvta_generic_to_shared(smem);  // shared address 0
    float* const odd = reinterpret_cast<float*>(space + kOdd);              // [2][128] levels and sums of the odd steps (T = 1)
    // full / empty: of a decoded step's place.  Of a place of a stream's scores: scores, weights, values written.  Of a stream:
    // queries written, and read for the last time.  Odd steps' statistics ready, and the sums they go with read (T = 1).
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], s_ready[2][2], p_ready[2][2], o_done[2][2], q_ready[2], q_free[2],
        odd_ready, odd_free, drain;
    __shared__ __align__(8) uint8_t valid[kStages][kUnits];  // tokens of each unit of a decoded step, a bit each
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    __shared__ Run s_run;
    volatile int* abort_flag = &abort_word;

    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;  // (the warp: known to be uniform)
    pdl_trigger();
    if (warp == kMma) {
        if (lane == 0) {
            abort_word = 0;
            for (int s = 0; s < kStages; ++s) {
                mbar_init(full + s, 32 * kUnits);
                mbar_init(empty + s, T);
            }
            for (int s = 0; s < 2; ++s) {
                for (int e = 0; e < 2; ++e) {
                    mbar_init(&s_ready[s][e], 1);
                    mbar_init(&p_ready[s][e], 128);
                    mbar_init(&o_done[s][e], 1);
                }
                mbar_init(q_ready + s, 128);
                mbar_init(q_free + s, 3 - T);
            }
            mbar_init(&odd_ready, 128);
            mbar_init(&odd_free, 128);
            mbar_init(&drain, 2);
            fence_mbar_init();
        }
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (warp == kMma + 1) {
        const Run run = find_run(a, blockIdx.x);
        if (lane == 0) s_run = run;
    }
    const int ek = exponent_above(fmaxf(fabsf(a.c.kcent[0]), fabsf(a.c.kcent[KL - 1])));
    const int ev = exponent_above(fmaxf(fabsf(a.c.vcent[0]), fabsf(a.c.vcent[VL - 1])));
    const float vd = exp2f((float)-ev);
    if (warp < kMma) build_table<KL, VL>(a.c, space + kTable, exp2f((float)-ek), vd, warp, kMma);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    Walk walk(s_run);
    Stretch x;
    uint32_t g = 0, seg = 0;  // steps and stretches of this CTA so far: the phases of every barrier
    // Each role walks the CTA's stretches on its own; the decoders run ahead into the next one.

    if (warp >= kMma) {
        // ------------------------------------------------------------ MMA issue, of one stream
        const int t = warp - kMma;
        if (elected()) {
            uint32_t done = 0;  // steps of this stream so far
            const uint32_t to_s = tmem + kS + 64 * t, to_o = tmem + kO + 128 * t, from_q = tmem + kQ + (T == 1 ? 0 : 64 * t);
            bool ok = true;
            while (ok && walk.next(a, x)) {
                const uint32_t ge = g + (x.s1 - x.s0), first = g + (T == 1 ? t : 0);
                ok = mbar_wait(q_ready + (T == 1 ? 0 : t), seg & 1, abort_flag, a.wait_cycles);
                // Scores of the CTA's step i, the stream's n-th, where the weights of its n-2nd were read from.
                auto scores = [&](uint32_t i, uint32_t n) {
                    const uint32_t stage = i % kStages, e = n & 1;
                    if (!mbar_wait(full + stage, (i / kStages) & 1, abort_flag, a.wait_cycles) ||
                        (n >= 2 && !mbar_wait(&o_done[t][e], ((n - 2) >> 1) & 1, abort_flag, a.wait_cycles)))
                        return false;
                    tc_fence_after();
                    const uint64_t dk = desc(kSteps, 16) + stage * (2 * kTile / 16);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        tc_mma_ts(to_s + kTok * e, from_q + 8 * k, dk + ((k >> 2) * (kHalf / 16) + 2 * (k & 3)), idesc(kTok, 0), k != 0);
                    tc_commit(&s_ready[t][e]);
                    return true;
                };
                if (ok && first < ge) ok = scores(first, done);
                for (uint32_t i = first; i < ge && ok; i += 3 - T, ++done) {
                    // the next scores first, so that they are there when the softmax is done with these; but a step that is
                    // not decoded yet is not waited for (its place may be this step's to free)
                    const uint32_t on = i + (3 - T), stage = i % kStages, e = done & 1;
                    const bool next = on < ge, early = next && mbar_peek(full + on % kStages, (on / kStages) & 1);
                    if (early) ok = scores(on, done + 1);
                    if (ok) ok = mbar_wait(&p_ready[t][e], (done >> 1) & 1, abort_flag, a.wait_cycles);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dv = desc(kSteps + kTile, kHalf) + stage * (2 * kTile / 16);
#pragma unroll
                    for (int k = 0; k < kTok / 16; ++k)
                        tc_mma_ts(to_o, to_s + kTok * e + 8 * k, dv + 128 * k, idesc(kPD, 1), i != first || k != 0);
                    tc_commit(&o_done[t][e]);
                    tc_commit(empty + stage);
                    if (next && !early) ok = scores(on, done + 1);
                }
                mbar_arrive(q_free + (T == 1 ? 0 : t));
                g = ge;
                ++seg;
            }
            tc_commit(&drain);  // completes when every MMA issued above has finished
        }
        __syncwarp();
    } else if (warp < kSoft) {
        // ------------------------------------------------------------ softmax: a thread to a row
        const int stream = warp >> 2, row = (T == 1 ? 0 : stream * 128) + (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's TMEM lanes
        const uint32_t col_o = tmem + kO + stream * 128 + lanes, at = tmem + kS + 64 * stream + lanes;
        uint32_t done = 0;  // steps of this stream so far
        bool ok = true;
        while (walk.next(a, x)) {
            const uint32_t first = g + (T == 1 ? stream : 0), ge = g + (x.s1 - x.s0);
            const bool idle = row - lane >= x.rows;  // no row of this warp is in use
            const bool writer = T == 2 || stream == 0;
            if (writer && seg) ok = __all_sync(kFull, mbar_wait(q_free + (T == 1 ? 0 : stream), (seg - 1) & 1, abort_flag, a.wait_cycles));
            if (!ok) break;
            float f = 0.f;  // from a row's products to log2 scores: not negative
            if (seg == 0) pdl_wait();  // the turned queries
            if (!idle) {
                const int64_t unit = ((int64_t)x.b * a.c.Hkv + x.h) * tiles + x.tile;
                const bool in = row < x.rows;
                if (writer) {
                    const uint4* src = a.turned + unit * 16 * kRows + row;
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        uint32_t w[32];
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const uint4 v = in ? src[(8 * half + c) * kRows] : make_uint4(0u, 0u, 0u, 0u);
                            w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
                        }
                        tc_st32(tmem + kQ + (T == 1 ? 0 : 64 * stream) + 32 * half + lanes, w);
                    }
                    tc_wait_st();
                }
                f = score_factor((in ? a.power[unit * kRows + row] : 0) + ek, a.qexp);
            }
            if (writer) {
                tc_fence_before();
                mbar_arrive(q_ready + (T == 1 ? 0 : stream));
            }
            float m = -INFINITY, l = 0.f, bias = 0.f;
            for (uint32_t i = first; i < ge; i += 3 - T) {
                const uint32_t e = done & 1;
                {
                    // (the decoders' barrier has long completed; waiting on it too, beside the load, orders `valid` before its read)
                    ok = __all_sync(kFull, mbar_wait(&s_ready[stream][e], (done >> 1) & 1, abort_flag, a.wait_cycles));
                    if (!ok) break;
                    tc_fence_after();
                    if (!idle) {
                        uint32_t s[32];
                        tc_ld32(at + kTok * e, s);
                        ok = __all_sync(kFull, mbar_wait(full + i % kStages, (i / kStages) & 1, abort_flag, a.wait_cycles));
                        const uint32_t in = *reinterpret_cast<const uint32_t*>(valid[i % kStages]);
                        tc_wait_ld();
                        if (!ok) break;
                        if (in != ~0u) {  // tokens past the end, or of a bad page
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!((in >> c) & 1)) s[c] = __float_as_uint(-INFINITY);
                        }
                        float x4[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) x4[c] = __uint_as_float(s[c]);
#pragma unroll
                        for (int c = 4; c < 28; c += 8)
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                x4[z] = fmaxf(fmaxf(x4[z], __uint_as_float(s[c + z])), __uint_as_float(s[c + z + 4]));
#pragma unroll
                        for (int c = 28; c < 32; ++c) x4[c & 3] = fmaxf(x4[c & 3], __uint_as_float(s[c]));
                        const float top = f * fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3]));
                        if (__any_sync(kFull, top - m > kSlack)) {
                            const float n = fmaxf(m, top), to = weight_bias(n), r = m == -INFINITY ? 0.f : fast_exp2(to - bias);
                            m = n;
                            bias = to;
                            l *= r;
                            if (i != first) {  // the sums so far, once the last product has written them
                                ok = __all_sync(kFull, mbar_wait(&o_done[stream][e ^ 1], ((done - 1) >> 1) & 1, abort_flag, a.wait_cycles));
                                if (!ok) break;
                                tc_fence_after();
#pragma unroll 1
                                for (int c = 0; c < 16; ++c) {
                                    uint32_t o[8];
                                    tc_ld8(col_o + 8 * c, o);
                                    tc_wait_ld();
#pragma unroll
                                    for (int z = 0; z < 8; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * r);
                                    tc_st8(col_o + 8 * c, o);
                                }
                            }
                        }
                        // (the sum takes the weights before their rounding to fp16, which moves one by 2^-11 of itself or, where it is
                        // subnormal, by 2^-32 of the maximum's at most)
                        const f2 ff = pk(f, f), bb = pk(bias, bias);
                        f2 ls[2] = {0, 0};
#pragma unroll
                        for (int c = 0; c < 16; ++c) {  // the weights take the scores' registers
                            const float2 y = un(fma2(pk(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), ff, bb));
                            const float u = fast_exp2(y.x), v = fast_exp2(y.y);
                            ls[c & 1] = add2(ls[c & 1], pk(u, v));
                            s[c] = pack_f16(u, v);
                        }
                        const float2 sum = un(add2(ls[0], ls[1]));
                        l += sum.x + sum.y;
                        tc_st16(at + kTok * e, s);
                        tc_wait_st();
                    }
                    tc_fence_before();
                    mbar_arrive(&p_ready[stream][e]);
                }
                if (!ok) break;
                ++done;
            }
            if (!ok) break;
            // ---- the stretch's partial result
            if (first < ge) {  // (the odd steps may be none)
                ok = __all_sync(kFull, mbar_wait(&o_done[stream][(done - 1) & 1], ((done - 1) >> 1) & 1, abort_flag, a.wait_cycles));
                if (!ok) break;
                tc_fence_after();
            }
            m = level(m, bias);
            float m1 = -INFINITY, l1 = 0.f;
            if (T == 1) {  // the even steps' warps add the odd steps' sums, which lie in the same TMEM lanes
                if (stream == 1) {
                    odd[row] = m;
                    odd[128 + row] = l;
                    tc_fence_before();
                    mbar_arrive(&odd_ready);
                    ok = __all_sync(kFull, mbar_wait(&odd_free, seg & 1, abort_flag, a.wait_cycles));
                } else {
                    ok = __all_sync(kFull, mbar_wait(&odd_ready, seg & 1, abort_flag, a.wait_cycles));
                    tc_fence_after();
                    m1 = odd[row];
                    l1 = odd[128 + row];
                }
                if (!ok) break;
            }
            if (writer) {
                if (!idle) {
                    const bool two = T == 1 && ge - g > 1;
                    const float n = two ? fmaxf(m, m1) : m;
                    // weight 1 for the higher level's own (also where both saw nothing); a NaN sum stays one
                    const float w0 = m == n ? 1.f : fast_exp2(m - n), w1 = m1 == n ? 1.f : fast_exp2(m1 - n);
                    const int64_t to = ((int64_t)blockIdx.x + x.unit) * kRows + row;
                    const float vscale = exp2f((float)ev);
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        uint32_t o[16], o1[16];
                        tc_ld8(col_o + 16 * c, o);
                        tc_ld8(col_o + 16 * c + 8, o + 8);
                        if (two) {
                            tc_ld8(col_o + 128 + 16 * c, o1);
                            tc_ld8(col_o + 136 + 16 * c, o1 + 8);
                        }
                        tc_wait_ld();
                        float z[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            z[k] = __uint_as_float(o[k]) * (w0 * vscale);
                            if (two) z[k] = fmaf(__uint_as_float(o1[k]), w1 * vscale, z[k]);
                        }
                        if (row < x.rows) {  // whole 32-byte sectors
                            float* out = a.part + to * kPD + 16 * c;
                            stg256(out, z);
                            stg256(out + 8, z + 8);
                        }
                    }
                    if (row < x.rows) a.stat[to] = make_float2(n, two ? l * w0 + l1 * w1 : l);
                }
                tc_fence_before();
                if (T == 1) mbar_arrive(&odd_free);
            }
            g = ge;
            ++seg;
        }
        // A CTA without work waits too: this grid must not end before the turn, or what comes after the call could meet it still
        // reading the queries and writing the workspace.
        if (seg == 0) pdl_wait();
    } else {
        // ------------------------------------------------------------ decoders: warp d takes units d, d + D, ... of the CTA's steps
        const int d = warp - kSoft, ng = kPD >> a.c.lgroup;
        uint32_t tl[2] = {0, 0}, th[2] = {0, 0};  // low and high bytes of an 8-level value book
        if (VL == 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t h = __half_as_ushort(__float2half_rn(a.c.vcent[i % VL] * vd));
                tl[i >> 2] |= (h & 255u) << (8 * (i & 3));
                th[i >> 2] |= (h >> 8) << (8 * (i & 3));
            }
        }
        const uint32_t ring = kRings + d * kDepth * U::kBytes, ring_end = ring + kDepth * U::kBytes;
        // (cache rows by the 8: 32-bit numbers)
        const uint32_t page8 = (uint32_t)(a.c.page_stride >> 3), head8 = (uint32_t)(a.c.head_stride >> 3);
        const uint32_t in_page = (1u << (a.c.lpage - 3)) - 1;
        const uint8_t* kc = reinterpret_cast<const uint8_t*>(a.c.kcodes) + lane * 16;
        const uint8_t* vc = reinterpret_cast<const uint8_t*>(a.c.vcodes) + lane * 16;
        const uint8_t* zc = reinterpret_cast<const uint8_t*>(lane < 8 ? a.c.kscales : a.c.vscales) + (lane & 7) * 16;
        const uint32_t z_at = (lane < 8 ? U::kKs : U::kVs) + (lane & 7) * 16;
        const bool copies_z = (lane & 7) < ng && lane < 16, copies_v = lane < kUnit * (int)U::kVRow / 16;
        bool ok = true;
        while (ok && walk.next(a, x)) {
            const int s0 = x.s0, s1 = x.s1, len = x.len, h = x.h;
            const int32_t* tab = a.table + (int64_t)x.b * a.table_stride;
        const int u0 = s0 * kUnits, u1 = min(s1 * kUnits, (len + kUnit - 1) / kUnit);  // units that hold tokens
        auto page_of = [&](int u) { return u < u1 ? __ldg(tab + (u >> (a.c.lpage - 3))) : 0; };
        // its first unit here: the first step of the CTA's count that is this warp's
        const int mine = (d + kDec - kUnits * (int)(g % (kDec / kUnits))) % kDec;
        int ahead = u0 + mine, page_next = 0;
        uint32_t fill = ring, counts = 0;  // four bits a unit: its valid tokens
        auto issue = [&]() {
            const int page = page_next, u = ahead;
            ahead += D;
            page_next = page_of(ahead);
            const bool in = u < u1, good = in && (uint32_t)page < (uint32_t)a.c.pages;
            counts = counts << 4 | (good ? (uint32_t)min(len - u * kUnit, kUnit) : 0u);
            const uint64_t row8 = (uint32_t)page * page8 + (uint32_t)h * head8 + (u & in_page);
            const uint8_t* k = kc + row8 * (kUnit * U::kKRow);
            cp16_if<U::kK>(fill + lane * 16, k, good);
            if (KL == 256) cp16_if<U::kK + 512>(fill + lane * 16, k + 512, good);
            cp16_if<U::kV>(fill + lane * 16, vc + row8 * (kUnit * U::kVRow), good && copies_v);
            cp16_if<0>(fill + z_at, zc + row8 * (uint32_t)(kUnit * 2 * ng), good && copies_z);
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (in && !good && lane == 0 && a.err) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
            fill = fill + U::kBytes == ring_end ? ring : fill + U::kBytes;
        };
            page_next = page_of(ahead);
#pragma unroll
            for (int i = 0; i < kDepth - 1; ++i) issue();
            const int c = lane & 15, hi = lane >> 4;  // 8 dims of tokens hi, hi + 2, ...
            const uint32_t lane_k = lane * 4 | 0x100, lane_v = lane_k + 128;
            const uint32_t k_at = U::kK + hi * U::kKRow + c * (KL == 256 ? 8 : 4);
            const uint32_t ks_at = U::kKs + (hi * ng + ((8 * c) >> a.c.lgroup)) * 2;  // the value's 128 on
            // 3-bit values: 8 codes from code `from` of word w0, ten to a word
            const int w0 = (8 * c) / 10, from = (8 * c) % 10;
            const uint32_t v_at = U::kV + hi * U::kVRow + (VL == 8 ? w0 * 4 : c * 4);
            const uint32_t shr = 3 * from, mulr = 1u << (30 - 3 * from);
            // in a decoded step: 64 dims to a half, a 128-byte row to a token, its 16-byte pieces swapped by the token
            const uint32_t to = kSteps + (c >> 3) * kHalf + hi * 128 + ((c & 7) ^ hi) * 16;
            uint32_t at = ring;
            // the unit's step, as a place among the decoded ones and the phase of its barriers
            uint32_t stage = (g + mine / kUnits) % kStages, phase = (g + mine / kUnits) / kStages & 1;
            for (int u = u0 + mine; u < s1 * kUnits; u += D) {
                issue();
                asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
                __syncwarp();
                const uint32_t count = (counts >> (4 * (kDepth - 1))) & 15u;
                if (count < kUnit) {  // what lies past the end may be anything: its scales are taken as zeros
                    for (uint32_t x = count * ng + lane; x < kUnit * ng; x += 32) {
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + U::kKs + 2 * x), "h"((uint16_t)0) : "memory");
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + U::kVs + 2 * x), "h"((uint16_t)0) : "memory");
                    }
                    __syncwarp();
                }
                constexpr int N = kUnit / 2;  // passes of two tokens
                uint32_t ks[N], vs[N], kw[N][2], vw[N];
                const uint32_t at_k = at + k_at, at_v = at + v_at;
                static_for<0, N>([&](auto qc) {
                    constexpr int q = decltype(qc)::value;
                    ks[q] = lds16(at + ks_at + 4 * q * ng);
                    vs[q] = lds16<128>(at + ks_at + 4 * q * ng);
                    if constexpr (KL == 256) {
                        const uint2 x = lds64<2 * q * U::kKRow>(at_k);
                        kw[q][0] = x.x;
                        kw[q][1] = x.y;
                    } else {
                        kw[q][0] = lds32<2 * q * U::kKRow>(at_k);
                    }
                    if constexpr (VL == 8)
                        vw[q] = (lds32<2 * q * U::kVRow>(at_v) >> shr) + lds32<2 * q * U::kVRow + 4>(at_v) * mulr;
                    else
                        vw[q] = lds32<2 * q * U::kVRow>(at_v);
                });
                ok = __all_sync(kFull, mbar_wait(empty + stage, phase ^ 1, abort_flag, a.wait_cycles));
                if (!ok) break;
                const uint32_t dst = to + (u & (kUnits - 1)) * (kUnit * 128) + stage * 2 * kTile;
                static_for<0, N>([&](auto qc) {  // keys of tokens 2 q + hi
                    constexpr int q = decltype(qc)::value;
                    const uint32_t s = ks[q] * 0x10001u;
                    uint32_t w[4];
                    if constexpr (KL == 256) {
                        const uint32_t x = kw[q][0], y = kw[q][1];
                        w[0] = prmt(table<0>(x, lane_k), table<1>(x, lane_k), 0x5410);
                        w[1] = prmt(table<2>(x, lane_k), table<3>(x, lane_k), 0x5410);
                        w[2] = prmt(table<0>(y, lane_k), table<1>(y, lane_k), 0x5410);
                        w[3] = prmt(table<2>(y, lane_k), table<3>(y, lane_k), 0x5410);
                    } else {
                        const uint32_t x = kw[q][0];
                        w[0] = table<0>(x, lane_k), w[1] = table<1>(x, lane_k);
                        w[2] = table<2>(x, lane_k), w[3] = table<3>(x, lane_k);
                    }
                    sts128<256 * q>(dst ^ (32 * q), mul2(w[0], s), mul2(w[1], s), mul2(w[2], s), mul2(w[3], s));
                });
                static_for<0, N>([&](auto qc) {  // values
                    constexpr int q = decltype(qc)::value;
                    const uint32_t s = vs[q] * 0x10001u, x = vw[q];
                    uint32_t w[4];
                    if constexpr (VL == 8) {
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
                        w[0] = table<0>(x, lane_v), w[1] = table<1>(x, lane_v);
                        w[2] = table<2>(x, lane_v), w[3] = table<3>(x, lane_v);
                    }
                    sts128<kTile + 256 * q>(dst ^ (32 * q), mul2(w[0], s), mul2(w[1], s), mul2(w[2], s), mul2(w[3], s));
                });
                if (lane == 0) valid[stage][u & (kUnits - 1)] = (uint8_t)((1u << count) - 1u);
                fence_async_smem();
                mbar_arrive(full + stage);
                __syncwarp();  // the ring's place is free for the next copy
                at = at + U::kBytes == ring_end ? ring : at + U::kBytes;
                stage += D / kUnits;
                if (stage >= kStages) stage -= kStages, phase ^= 1;
            }

            asm volatile("cp.async.wait_group 0;" ::: "memory");
            g += s1 - s0;
        }
    }

    if (warp >= kMma && elected()) {
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
    const int tiles = (a.n * a.ratio + a.trows - 1) / a.trows;
    kv_tree_turn_kernel<<<(unsigned)(((int64_t)a.B * a.n * a.Hq + 7) / 8), 256, 0, st>>>(a, tiles);
    const tq_status s = launch_status();
    if (s != TQ_OK) return s;
    // its prologue and first copies run beside the turn, which began after everything before it on the stream had ended
    return launch_pdl(kv_tree_wide_kernel<KL, VL, T>, dim3((unsigned)a.ctas), dim3(32 * kWarps), smem, st, a, tiles);
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
