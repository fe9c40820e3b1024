// Attention of drafted trees over the paged latent cache (the absorbed form), on the 5th-generation tensor cores.
//
// A cached row of 576 elements is the key of every head and its first 512 the value, so 64 query rows (heads of drafts) share
// each token that is read.  A persistent CTA takes a run of steps of 64 tokens; tokens come by tensor copies into a ring of four
// places of 32, one 128-byte swizzled row a token for each 64 elements, which serves as the K-major operand of
//   scores   S[64 x 64]   = Q (shared) . K^T     36 MMAs of K = 16
// and as the MN-major operand of
//   values   O[64 x 512] += P (shared) . V       2 x 4 MMAs of K = 16, N = 256
// M = 64 takes 16 of the 32 TMEM lanes of each warp: O's upper half of the elements lies in the other 16, so that O takes 256
// columns, and scores have two places of 64.  The scores of a step are issued before the values of the one before it, so the
// softmax of one runs beside the products of the other.  A row's running maximum follows only when a score passes it by 2^kSlack.
//
// Tokens past the end and drafts that hold something that is not finite are zeroed in shared memory by two guard warps (a
// masked weight of 0 times NaN would reach the rows that do not see it); only steps that have such tokens wait for them.
// Every wait on an mbarrier is bounded; on expiry the CTA sets TQ_DEVERR_TIMEOUT, drains and frees TMEM.
#include <math.h>

#include <algorithm>

#include "latent.cuh"
#include "tensor.cuh"

namespace tq {
namespace {

using namespace tc;

constexpr int kRows = 64, kTok = 64, kPlace = 32;  // query rows of a tile; tokens of a step, of a place of the ring
constexpr int kBlocks = kLatentRow / 64;           // 128-byte pieces of a row
constexpr int kMaxSms = 256;
constexpr int kSoft = 4, kMma = 4, kCopy = 5, kGuard = 6, kWarps = 8;
constexpr uint32_t kRingBlock = 2 * kTok * 128, kQBlock = kRows * 128;  // bytes of 64 elements of the ring's tokens, of the queries
constexpr uint32_t kQ = 0, kRing = kQ + kBlocks * kQBlock, kP = kRing + kBlocks * kRingBlock, kControl = kP + kRows * 128;
constexpr uint32_t kSmem = kControl + 1024 + 1024;  // the last for the start's alignment

struct AttendArgs {
    LatentArgs l;
    int ctas, pad, least;  // of the schedule: CTAs, places that beginning a unit weighs, fewest places of a run
    int fresh_box;         // rows of a copy of drafts
    float* part;           // [2 ctas][64][512]
    float2* stat;          // [2 ctas][64]: level and sum
    long long wait_cycles;
};

// ---------------------------------------------------------------- the batch's work, counted on the device

// A unit is a tile of 64 query rows of a sequence: `steps` of cached tokens, then of drafts.
struct Seq {
    int len, live, ctx, steps, tiles;
};
TQ_DEVFN Seq seq(const LatentArgs& a, int b) {
    Seq s;
    s.len = latent_len(a, b);
    s.live = latent_live(a, b);
    s.ctx = (s.len + kTok - 1) / kTok;
    s.steps = s.ctx + (a.fresh ? (s.live + kTok - 1) / kTok : 0);
    s.tiles = (int)(((int64_t)s.live * a.H + kRows - 1) / kRows);
    return s;
}
// Places on the axis that the CTAs divide: a unit with steps takes `pad` places, then one for each step.
TQ_DEVFN int places_of(const Seq& s, int pad) { return s.steps ? s.steps + pad : 0; }
TQ_DEVFN int pad_of(const AttendArgs& a, int steps) { return min(a.pad, steps / (4 * a.ctas)); }
TQ_DEVFN int per_cta(const AttendArgs& a, int total) { return max((total + a.ctas - 1) / a.ctas, a.least); }

// Of the whole batch (one warp): steps, and units that have any.
TQ_DEVFN void count_all(const AttendArgs& a, int& steps, int& busy) {
    int s = 0, u = 0;
    for (int b = threadIdx.x & 31; b < a.l.B; b += 32) {
        const Seq q = seq(a.l, b);
        s += q.steps * q.tiles;
        u += q.steps ? q.tiles : 0;
    }
    steps = __reduce_add_sync(kFull, s);
    busy = __reduce_add_sync(kFull, u);
}

struct Run {
    int at, end, pad, b, places;  // first place, end; places before sequence b, the last one that begins at or before it
};
TQ_DEVFN Run find_run(const AttendArgs& a, int cta) {
    const int lane = threadIdx.x & 31;
    int steps, busy;
    count_all(a, steps, busy);
    Run r{};
    r.pad = pad_of(a, steps);
    const int total = steps + busy * r.pad, per = per_cta(a, total);
    r.at = (int)min((int64_t)cta * per, (int64_t)total);
    r.end = (int)min((int64_t)r.at + per, (int64_t)total);
    for (int b0 = 0; b0 < a.l.B; b0 += 32) {
        int own = 0;
        if (b0 + lane < a.l.B) {
            const Seq q = seq(a.l, b0 + lane);
            own = q.tiles * places_of(q, r.pad);
        }
        int upto = own;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int x = __shfl_up_sync(kFull, upto, m);
            if (lane >= m) upto += x;
        }
        const unsigned hit = __ballot_sync(kFull, r.places + upto > r.at);
        if (hit) {
            const int src = __ffs(hit) - 1;
            r.places += __shfl_sync(kFull, upto - own, src);
            r.b = b0 + src;
            break;
        }
        r.places += __shfl_sync(kFull, upto, 31);
    }
    return r;
}

// A stretch of a run within one unit: steps s0 .. s1 - 1 of it.
struct Stretch {
    Seq s;
    int b, tile, s0, s1;
};
struct Walk {
    Run r;
    TQ_DEVFN explicit Walk(const Run& run) : r(run) {}
    TQ_DEVFN bool next(const LatentArgs& a, Stretch& x) {
        while (r.at < r.end) {
            x.s = seq(a, r.b);
            int own = places_of(x.s, r.pad);
            while (r.at >= r.places + own * x.s.tiles) {  // into the next sequence that has any
                r.places += own * x.s.tiles;
                x.s = seq(a, ++r.b);
                own = places_of(x.s, r.pad);
            }
            x.tile = (r.at - r.places) / own;
            const int at = r.at - r.places - x.tile * own, to = min(own, at + (r.end - r.at));
            r.at += to - at;
            if (to <= r.pad) continue;  // none of its steps
            x.b = r.b;
            x.s0 = max(at - r.pad, 0);
            x.s1 = to - r.pad;
            return true;
        }
        return false;
    }
};

struct Control {
    uint64_t full[4], empty[4];     // of the ring's places
    uint64_t guarded[2];            // of a step's tokens, where it has any to zero
    uint64_t s_ready[2];            // of the scores' places
    uint64_t p_ready, o_done, q_ready, drain;
    unsigned long long valid[2], odd[2];  // of a step's tokens: those that exist; drafts that are not finite
    Run run;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(Control) <= 1024, "control block");

// Tokens of a step that its products take: up to the last one that exists, in sixteens.
TQ_DEVFN int used_of(unsigned long long valid) { return valid ? (64 - __clzll((long long)valid) + 15) & ~15 : 16; }

template <bool BF>
__global__ void __launch_bounds__(32 * kWarps, 1)
    latent_attend_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap map_rows,
                         const __grid_constant__ CUtensorMap map_fresh) {
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t* const smem = raw + (base - smem_u32(raw));
    Control& c = *reinterpret_cast<Control*>(smem + kControl);
    volatile int* abort_flag = &c.abort;
    const LatentArgs& l = a.l;
    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;

    pdl_trigger();
    if (warp == kMma) {
        if (lane == 0) {
            c.abort = 0;
            for (int i = 0; i < 4; ++i) {
                mbar_init(c.full + i, 1);
                mbar_init(c.empty + i, i & 1 ? 1 : 3);  // the products; of a step's first place the guards too
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(c.guarded + i, 2);
                mbar_init(c.s_ready + i, 1);
            }
            mbar_init(&c.p_ready, 32 * kSoft);
            mbar_init(&c.o_done, 1);
            mbar_init(&c.q_ready, 32 * kSoft);
            mbar_init(&c.drain, 1);
            fence_mbar_init();
        }
        __syncwarp();
        alloc512(&c.tmem);
    }
    pdl_wait();
    if (warp == kCopy) {
        const Run run = find_run(a, blockIdx.x);
        if (lane == 0) c.run = run;
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = c.tmem, to_s = tmem + 256;
    Walk walk(c.run);
    Stretch x;
    uint32_t g = 0, seg = 0;  // steps and stretches of this CTA so far: the phases of every barrier
    // Each role walks the CTA's stretches on its own.

    if (warp == kCopy) {
        // ------------------------------------------------------------ tensor copies of the tokens
        const int box = min(1 << l.lpage, kPlace), boxes = kPlace / box;
        bool ok = true;
        uint32_t issued = 0;  // places of the ring filled so far
        while (ok && walk.next(l, x)) {
            const int32_t* table = l.table + (int64_t)x.b * l.table_stride;
            // page ids, a lane to a 16-token piece, of 8 steps and of the next 8
            auto look = [&](int s) {
                const int64_t t = (int64_t)s * kTok + lane * 16;
                return t < x.s.len ? table[t >> l.lpage] : -1;
            };
            int ids = 0, ids_next = look(x.s0);
            for (int s = x.s0; s < x.s1 && ok; ++s, ++g) {
                const uint32_t place = g & 1, phase = (g >> 1) & 1;
                const bool context = s < x.s.ctx;
                if (((s - x.s0) & 7) == 0) {
                    ids = ids_next;
                    ids_next = look(s + 8);
                }
                unsigned long long valid;
                if (context) {
                    const int mine = __shfl_sync(kFull, ids, ((s - x.s0) & 7) * 4 + (lane & 3));
                    const int count = min(max(x.s.len - (s * kTok + (lane & 3) * 16), 0), 16);
                    const bool good = (uint32_t)mine < (uint64_t)l.pages;
                    if (count > 0 && !good && lane < 4 && l.err) atomicOr(l.err, TQ_DEVERR_BAD_PAGE);
                    const uint32_t bits = lane < 4 && good ? (1u << count) - 1 : 0u;
                    const uint32_t lo = __shfl_sync(kFull, bits, 0) | __shfl_sync(kFull, bits, 1) << 16,
                                   hi = __shfl_sync(kFull, bits, 2) | __shfl_sync(kFull, bits, 3) << 16;
                    valid = (unsigned long long)hi << 32 | lo;
                } else {
                    const int count = min(x.s.live - (s - x.s.ctx) * kTok, kTok);
                    valid = count == 64 ? ~0ull : (1ull << count) - 1;
                }
                for (int h = 0; h < 2 && ok; ++h) {
                    const uint32_t at = place * 2 + h;
                    ok = __all_sync(kFull, mbar_wait(c.empty + at, phase ^ 1, abort_flag, a.wait_cycles));
                    if (!ok) break;
                    const uint32_t half = (uint32_t)(valid >> (32 * h));
                    const uint32_t dst = base + kRing + at * (kPlace * 128);
                    if (h == 0 && lane == 0) c.valid[place] = valid;
                    if (context) {
                        const int part = 2 * h;  // of the ids
                        int bytes = 0;
                        for (int p = 0; p < boxes; ++p)
                            if ((half >> (p * box)) & 1) bytes += box * 128 * kBlocks;
                        if (elected()) mbar_expect_tx(c.full + at, bytes);
                        __syncwarp();
                        for (int p = 0; p < boxes; ++p) {
                            const int id = __shfl_sync(kFull, ids, ((s - x.s0) & 7) * 4 + part + p * (box / 16));
                            const int t = s * kTok + h * kPlace + p * box;
                            const int row = (int)((int64_t)id * l.page_stride) + (t & ((1 << l.lpage) - 1));
                            if (((half >> (p * box)) & 1) && elected())
#pragma unroll 1
                                for (int d = 0; d < kBlocks; ++d)
                                    tma_load_2d(dst + d * kRingBlock + p * box * 128, &map_rows, d * 64, row, c.full + at);
                            __syncwarp();
                        }
                    } else if (elected()) {
                        const int t = (s - x.s.ctx) * kTok + h * kPlace, row = x.b * l.n + t;
                        const int copies = half ? (min(kPlace, x.s.live - t) + a.fresh_box - 1) / a.fresh_box : 0;
                        mbar_expect_tx(c.full + at, copies * a.fresh_box * 128 * kBlocks);
                        for (int p = 0; p < copies; ++p)
#pragma unroll 1
                            for (int d = 0; d < kBlocks; ++d)
                                tma_load_2d(dst + d * kRingBlock + p * a.fresh_box * 128, &map_fresh, d * 64, row + p * a.fresh_box,
                                            c.full + at);
                    }
                    __syncwarp();
                    ++issued;
                }
            }
        }
        // no copy may be in flight when the CTA ends (on an abort: nobody else has waited for them)
        for (int at = 0; at < 4; ++at) {
            const uint32_t fills = (issued + 3 - at) >> 2;
            if (fills) mbar_wait_drain(c.full + at, (fills - 1) & 1);
        }
    } else if (warp == kMma) {
        // ------------------------------------------------------------ MMA issue
        if (elected()) {
            bool ok = true;
            const uint64_t dq = desc(base + kQ, 16), dk = desc(base + kRing, 16), dv = desc(base + kRing, kRingBlock),
                           dp = desc(base + kP, 16);
            // Scores of step i, whose tokens are in.
            auto scores = [&](uint32_t i, bool context) {
                const uint32_t place = i & 1, phase = (i >> 1) & 1;
                if (!mbar_wait(c.full + 2 * place, phase, abort_flag, a.wait_cycles) ||
                    !mbar_wait(c.full + 2 * place + 1, phase, abort_flag, a.wait_cycles))
                    return false;
                const unsigned long long valid = c.valid[place];
                if ((valid != ~0ull || !context) && !mbar_wait(c.guarded + place, phase, abort_flag, a.wait_cycles)) return false;
                fence_after();
                const uint32_t id = idesc(BF, kRows, used_of(valid), 0);
                const uint64_t k0 = dk + place * (kTok * 128 / 16);
#pragma unroll 1
                for (int d = 0; d < kBlocks; ++d)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss(to_s + 64 * (i & 1), dq + d * (kQBlock / 16) + 2 * k, k0 + d * (kRingBlock / 16) + 2 * k, id,
                               (d | k) != 0);
                commit(c.s_ready + (i & 1));
                return true;
            };
            while (ok && walk.next(l, x)) {
                const uint32_t ge = g + (x.s1 - x.s0), first = g;
                ok = mbar_wait(&c.q_ready, seg & 1, abort_flag, a.wait_cycles) && scores(g, x.s0 < x.s.ctx);
                for (uint32_t i = g; i < ge && ok; ++i) {
                    const uint32_t place = i & 1;
                    // the next scores first, unless their tokens are still on their way (and may wait for this step's places)
                    const bool next = i + 1 < ge, ctx = x.s0 + (int)(i + 1 - first) < x.s.ctx;
                    const bool early = next && mbar_peek(c.full + 2 * (place ^ 1) + 1, ((i + 1) >> 1) & 1);
                    if (early) ok = scores(i + 1, ctx);
                    if (ok) ok = mbar_wait(&c.p_ready, i & 1, abort_flag, a.wait_cycles);
                    if (!ok) break;
                    fence_after();
                    const int used = used_of(c.valid[place]);
                    const uint64_t v0 = dv + place * (kTok * 128 / 16);
                    constexpr uint32_t id = idesc(BF, kRows, 256, 1);
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        if (k * 16 < used) {
                            const uint32_t more = i != first || k != 0;
                            mma_ss(tmem, dp + 2 * k, v0 + 128 * k, id, more);
                            mma_ss(tmem + (16u << 16), dp + 2 * k, v0 + 128 * k + 4 * (kRingBlock / 16), id, more);
                        }
                        if (k & 1) commit(c.empty + 2 * place + (k >> 1));
                    }
                    commit(&c.o_done);
                    if (next && !early) ok = scores(i + 1, ctx);
                }
                g = ge;
                ++seg;
            }
            commit(&c.drain);  // completes when every MMA issued above has finished
            if (!mbar_wait_drain(&c.drain, 0)) *abort_flag = 1;
        }
        __syncwarp();
    } else if (warp >= kGuard) {
        // ------------------------------------------------------------ guards: a thread to a token
        const int t = tid - kGuard * 32;
        bool ok = true;
        while (ok && walk.next(l, x)) {
            for (int s = x.s0; s < x.s1 && ok; ++s, ++g) {
                const uint32_t place = g & 1, phase = (g >> 1) & 1;
                const bool context = s < x.s.ctx;
                ok = __all_sync(kFull, mbar_wait(c.full + 2 * place, phase, abort_flag, a.wait_cycles) &&
                                           mbar_wait(c.full + 2 * place + 1, phase, abort_flag, a.wait_cycles));
                if (!ok) break;
                const unsigned long long valid = c.valid[place];
                uint8_t* row = smem + kRing + place * (kTok * 128) + t * 128;
                bool wipe = !((valid >> t) & 1) && t < used_of(valid), odd = false;
                if (!context && ((valid >> t) & 1)) {
                    constexpr uint32_t kTop = BF ? 0x7f80u : 0x7c00u;
                    for (int d = 0; d < kBlocks; ++d)
#pragma unroll
                        for (int p = 0; p < 8; ++p) {
                            const uint4 v = *reinterpret_cast<const uint4*>(row + d * kRingBlock + ((p + t) & 7) * 16);
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                odd |= (w[e] & kTop) == kTop || ((w[e] >> 16) & kTop) == kTop;
                        }
                    wipe |= odd;
                }
                const uint32_t bits = __ballot_sync(kFull, odd);
                if (lane == 0) reinterpret_cast<uint32_t*>(&c.odd[place])[warp - kGuard] = bits;
                if (wipe) {
                    for (int d = 0; d < kBlocks; ++d)
#pragma unroll
                        for (int p = 0; p < 8; ++p)
                            *reinterpret_cast<uint4*>(row + d * kRingBlock + ((p + t) & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    fence_async_smem();
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(c.guarded + place);
                    mbar_arrive(c.empty + 2 * place);
                }
            }
        }
    } else {
        // ------------------------------------------------------------ softmax: rows lane / 4 and lane / 4 + 8 of the warp's 16
        const uint32_t lanes = (uint32_t)warp << 21;
        const int words = (l.n + 63) / 64;
        uint8_t* const p_smem = smem + kP;
        bool ok = true;
        while (ok && walk.next(l, x)) {
            const uint32_t ge = g + (x.s1 - x.s0);
            const int64_t y0 = (int64_t)x.tile * kRows;
            const int rows = (int)min((int64_t)kRows, (int64_t)x.s.live * l.H - y0);
            // ---- the tile's queries (the last scores of the stretch before have been read, so its queries are free)
            for (int i = tid; i < kRows * (kLatentRow / 8); i += 32 * kSoft) {
                const int r = i / (kLatentRow / 8), piece = i - r * (kLatentRow / 8);
                const int64_t y = y0 + min(r, rows - 1);
                const int64_t token = y / l.H;
                const uint16_t* src = l.q + ((int64_t)x.b * l.n + token) * l.qs + (y - token * l.H) * kLatentRow + piece * 8;
                const uint32_t dst = base + kQ + (piece >> 3) * kQBlock + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(r < rows ? 16 : 0) : "memory");
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            mbar_arrive(&c.q_ready);
            float m[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, bias[2] = {0.f, 0.f};
            int draft[2];  // of the two rows
#pragma unroll
            for (int j = 0; j < 2; ++j) draft[j] = (int)((y0 + min(warp * 16 + (lane >> 2) + 8 * j, rows - 1)) / l.H);
            for (uint32_t i = g; i < ge; ++i) {
                const uint32_t place = i & 1;
                const int s = x.s0 + (int)(i - g);
                ok = __all_sync(kFull, mbar_wait(c.s_ready + place, (i >> 1) & 1, abort_flag, a.wait_cycles));
                if (!ok) break;
                fence_after();
                uint32_t v[32];
                ld16x64(to_s + 64 * place + lanes, v);
                // (its tokens' barriers have completed before the scores; waiting on them too orders `valid` before its read)
                ok = __all_sync(kFull, mbar_wait(c.full + 2 * place, (i >> 1) & 1, abort_flag, a.wait_cycles));
                if (!ok) break;
                unsigned long long see[2];
                see[0] = see[1] = c.valid[place];
                const bool whole = see[0] == ~0ull && s < x.s.ctx;
                const int used = used_of(see[0]);
                bool spoilt[2] = {false, false};
                if (s >= x.s.ctx) {
                    ok = __all_sync(kFull, mbar_wait(c.guarded + place, (i >> 1) & 1, abort_flag, a.wait_cycles));
                    if (!ok) break;
                    const unsigned long long odd = c.odd[place];
                    const int w = s - x.s.ctx;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        unsigned long long bits;
                        if (l.mask) bits = l.mask[((int64_t)x.b * l.n + draft[j]) * words + w];
                        else bits = draft[j] >= 64 * w + 63 ? ~0ull : draft[j] < 64 * w ? 0ull : (2ull << (draft[j] - 64 * w)) - 1;
                        see[j] &= bits;
                        spoilt[j] = (see[j] & odd) != 0;
                    }
                }
                wait_ld();
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 8; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int col = 8 * k + 2 * (lane & 3) + e;
                            float f = __uint_as_float(v[4 * k + 2 * j + e]) * l.scale2;
                            if (!whole && !((see[j] >> col) & 1)) f = -INFINITY;
                            v[4 * k + 2 * j + e] = __float_as_uint(f);
                            top[j] = fmaxf(top[j], f);
                        }
                if (__any_sync(kFull, top[0] - m[0] > kSlack || top[1] - m[1] > kSlack)) {
                    float r[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        top[j] = fmaxf(top[j], __shfl_xor_sync(kFull, top[j], 1));
                        top[j] = fmaxf(top[j], __shfl_xor_sync(kFull, top[j], 2));
                        // (each row by its own scores alone: its result must not hang on what its neighbours see)
                        const float n = top[j] - m[j] > kSlack ? top[j] : m[j], to = weight_bias(n);
                        r[j] = m[j] == -INFINITY ? 0.f : exp2_fast(to - bias[j]);
                        m[j] = n;
                        bias[j] = to;
                        sum[j] *= r[j];
                    }
                    if (i != g) {  // the sums so far, once the last product has written them
                        ok = __all_sync(kFull, mbar_wait(&c.o_done, (i - 1) & 1, abort_flag, a.wait_cycles));
                        if (!ok) break;
                        fence_after();
                        // row lane % 16 of O's two halves
                        const float lo = __shfl_sync(kFull, r[0], (lane & 7) * 4), hi = __shfl_sync(kFull, r[1], (lane & 7) * 4);
                        const float f = lane & 8 ? hi : lo;
#pragma unroll 1
                        for (int q = 0; q < 8; ++q) {
                            uint32_t o[32];
                            ld32(tmem + lanes + 32 * q, o);
                            wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            st32(tmem + lanes + 32 * q, o);
                        }
                        wait_st();
                    }
                }
                // ---- weights; the sum takes them before their rounding
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 8; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float p0 = exp2_fast(__uint_as_float(v[4 * k + 2 * j]) + bias[j]);
                        const float p1 = exp2_fast(__uint_as_float(v[4 * k + 2 * j + 1]) + bias[j]);
                        sum[j] += p0 + p1;
                        w[2 * k + j] = pack16<BF>(p0, p1);
                    }
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (spoilt[j]) sum[j] = NAN;
                if (i > 0) {  // the products before have read P
                    ok = __all_sync(kFull, mbar_wait(&c.o_done, (i - 1) & 1, abort_flag, a.wait_cycles));
                    if (!ok) break;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (8 * k < used)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int row = warp * 16 + (lane >> 2) + 8 * j;
                            *reinterpret_cast<uint32_t*>(p_smem + row * 128 + ((k ^ (row & 7)) << 4) + (lane & 3) * 4) = w[2 * k + j];
                        }
                fence_before();
                fence_async_smem();
                mbar_arrive(&c.p_ready);
            }
            if (!ok) break;
            // ---- the stretch's result: the rows themselves where it is the whole unit, else a partial result
            ok = __all_sync(kFull, mbar_wait(&c.o_done, (ge - 1) & 1, abort_flag, a.wait_cycles));
            if (!ok) break;
            fence_after();
            float level_[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sum[j] += __shfl_xor_sync(kFull, sum[j], 1);
                sum[j] += __shfl_xor_sync(kFull, sum[j], 2);
                level_[j] = level(m[j], bias[j]);
            }
            const int row = warp * 16 + (lane & 15), from = (lane & 7) * 4;
            const float s_lo = __shfl_sync(kFull, sum[0], from), s_hi = __shfl_sync(kFull, sum[1], from);
            const float l_lo = __shfl_sync(kFull, level_[0], from), l_hi = __shfl_sync(kFull, level_[1], from);
            const float total = lane & 8 ? s_hi : s_lo, lev = lane & 8 ? l_hi : l_lo;
            const bool all = x.s0 == 0 && x.s1 == x.s.steps, mine = row < rows;
            const int64_t slot = 2ll * blockIdx.x + (x.s0 == 0);
            const float over = total == 0.f ? 0.f : 1.f / total;  // (a NaN sum stays one)
            const int64_t y = y0 + min(row, rows - 1);
            uint16_t* out = l.o + ((int64_t)x.b * l.n * l.H + y) * kLatent + (lane >> 4) * 256;
            float* part = a.part + (slot * kRows + row) * kLatent + (lane >> 4) * 256;
            if (!all && mine && lane < 16) a.stat[slot * kRows + row] = make_float2(lev, total);
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {
                uint32_t o[32];
                ld32(tmem + lanes + 32 * q, o);
                wait_ld();
                if (mine && all) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t z[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            z[k] = pack16<BF>(__uint_as_float(o[8 * e + 2 * k]) * over, __uint_as_float(o[8 * e + 2 * k + 1]) * over);
                        *reinterpret_cast<uint4*>(out + 32 * q + 8 * e) = make_uint4(z[0], z[1], z[2], z[3]);
                    }
                } else if (mine) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) stg256(part + 32 * q + 8 * e, reinterpret_cast<const float*>(o) + 8 * e);
                }
                __syncwarp();
            }
            fence_before();
            g = ge;
            ++seg;
        }
    }

    fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag && l.err) atomicOr(l.err, TQ_DEVERR_TIMEOUT);
    if (warp == kMma) {
        fence_after();
        dealloc512(tmem);
    }
}

// What the CTAs left in parts, joined in their order; rows that see nothing, and drafts that are not in use, are zeros.  A CTA to
// `1 / gridDim.z` of the elements of a tile of 64 rows.
template <bool BF>
__global__ void __launch_bounds__(256) latent_join_kernel(AttendArgs a) {
    __shared__ int s_before, s_steps, s_busy;
    __shared__ float s_weight[kRows];
    pdl_trigger();
    pdl_wait();
    const LatentArgs& l = a.l;
    const int b = blockIdx.y, tile = blockIdx.x, tid = threadIdx.x;
    if (l.err && tile == 0 && blockIdx.z == 0 && tid == 0 && l.lens[b] != latent_len(l, b)) atomicOr(l.err, TQ_DEVERR_BAD_PAGE);
    const Seq s = seq(l, b);
    const int64_t y0 = (int64_t)tile * kRows;
    const int rows = (int)min((int64_t)kRows, (int64_t)l.n * l.H - y0);          // of the output
    const int live = (int)max(min((int64_t)rows, (int64_t)s.live * l.H - y0), (int64_t)0);
    const int width = kLatent / gridDim.z, e0 = blockIdx.z * width, pieces = width / 4;
    uint16_t* const out = l.o + ((int64_t)b * l.n * l.H + y0) * kLatent + e0;
    auto zero = [&](int from) {
        for (int i = from * pieces + tid; i < rows * pieces; i += 256)
            *reinterpret_cast<uint2*>(out + (int64_t)(i / pieces) * kLatent + (i % pieces) * 4) = make_uint2(0u, 0u);
    };
    if (live == 0 || s.steps == 0) {
        zero(0);
        return;
    }
    zero(live);
    if (tid < 32) {
        int steps, busy, before = 0;
        count_all(a, steps, busy);
        const int pad = pad_of(a, steps);
        for (int i = tid; i < b; i += 32) {
            const Seq q = seq(l, i);
            before += q.tiles * places_of(q, pad);
        }
        before = __reduce_add_sync(kFull, before);
        if (tid == 0) s_before = before, s_steps = steps, s_busy = busy;
    }
    __syncthreads();
    const int pad = pad_of(a, s_steps), per = per_cta(a, s_steps + s_busy * pad), own = s.steps + pad;
    const int begin = s_before + tile * own;                 // the unit's first place
    const int c0 = (begin + pad) / per, c1 = (begin + own - 1) / per;  // CTAs with steps of it
    if (c0 == c1) return;  // one CTA has written its rows
    // ---- weights of a row's parts: 2^level over the highest, over the sum
    auto slot_of = [&](int c) { return 2ll * c + (c == c0); };
    const int row = tid / 4;  // four threads to a row
    float top = -INFINITY, total = 0.f;
    if (row < live) {
        for (int c = c0; c <= c1; ++c) top = fmaxf(top, a.stat[slot_of(c) * kRows + row].x);
        for (int c = c0; c <= c1; ++c) {
            const float2 z = a.stat[slot_of(c) * kRows + row];
            total += z.y * (z.x == top ? 1.f : exp2_fast(z.x - top));
        }
    }
    const float over = total == 0.f ? 0.f : 1.f / total;
    if (row < live)
        for (int e = (tid & 3) * 4; e < width; e += 16) {
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = c0; c <= c1; ++c) {
                const float level = a.stat[slot_of(c) * kRows + row].x, w = level == top ? 1.f : exp2_fast(level - top);
                const float4 z = *reinterpret_cast<const float4*>(a.part + (slot_of(c) * kRows + row) * kLatent + e0 + e);
                o.x = fmaf(z.x, w, o.x);
                o.y = fmaf(z.y, w, o.y);
                o.z = fmaf(z.z, w, o.z);
                o.w = fmaf(z.w, w, o.w);
            }
            *reinterpret_cast<uint2*>(out + (int64_t)row * kLatent + e) =
                make_uint2(pack16<BF>(o.x * over, o.y * over), pack16<BF>(o.z * over, o.w * over));
        }
}

int sm_count() {
    static const int n = [] {
        int dev = 0, v = 0;
        return cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? v : 152;
    }();
    return n;
}

// Steps of the whole batch at most; 0 where there are too many.
int64_t most_steps(const tq_latent_pages_t* cache, int32_t B, int32_t n, int32_t H, int64_t max_len) {
    if (latent_check(cache) != TQ_OK || B <= 0 || n <= 0 || H <= 0 || H > 65535 || max_len < 0) return 0;
    const int64_t most = 1ll << 29;
    const int64_t tiles = ((int64_t)n * H + kRows - 1) / kRows, steps = (std::min<int64_t>(max_len, 1ll << 40) + kTok - 1) / kTok + (n + kTok - 1) / kTok;
    if ((int64_t)n * H > most || steps > most || tiles > most / B || tiles * B > most / steps) return 0;
    return tiles * B * steps;
}

template <bool BF>
tq_status launch(const AttendArgs& a, const CUtensorMap& rows, const CUtensorMap& fresh, cudaStream_t st) {
    if (ensure_smem((const void*)latent_attend_kernel<BF>, kSmem) != cudaSuccess) return TQ_ERR_CUDA;
    tq_status s = launch_pdl(latent_attend_kernel<BF>, dim3((unsigned)a.ctas), dim3(32 * kWarps), kSmem, st, a, rows, fresh);
    if (s != TQ_OK) return s;
    const int64_t tiles = ((int64_t)a.l.n * a.l.H + kRows - 1) / kRows;
    const int parts = tiles * a.l.B * 8 <= 2 * sm_count() ? 8 : tiles * a.l.B * 2 <= 2 * sm_count() ? 4 : 1;
    return launch_pdl(latent_join_kernel<BF>, dim3((unsigned)tiles, (unsigned)a.l.B, (unsigned)parts), dim3(256), 0, st, a);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" size_t tq_latent_attend_tree_workspace_bytes(const tq_latent_pages_t* cache, int32_t B, int32_t n, int32_t H,
                                                        int64_t max_len) {
    const int64_t steps = most_steps(cache, B, n, H, max_len);
    return (size_t)(2 * std::min<int64_t>(steps, kMaxSms)) * kRows * (kLatent * sizeof(float) + sizeof(float2));
}

extern "C" tq_status tq_latent_attend_tree(const tq_latent_pages_t* cache, const void* q, int64_t q_stride, int32_t B, int32_t n,
                                           int32_t H, const int32_t* table, int32_t table_stride, const int32_t* lens,
                                           int64_t max_len, const void* fresh, int64_t fresh_stride, const uint64_t* mask,
                                           const int32_t* n_tok, float scale, void* o, void* ws, size_t ws_bytes, uint32_t* err,
                                           void* stream) {
    const tq_status s = latent_check(cache);
    if (s != TQ_OK) return s;
    if (B < 0 || n < 0 || H <= 0 || H > 65535 || table_stride < 0 || max_len < 0 || !isfinite(scale)) return TQ_ERR_INVALID;
    if (max_len > (int64_t)table_stride * cache->page) return TQ_ERR_INVALID;
    if (q_stride < (int64_t)H * kLatentRow || q_stride % 8 || (fresh && (fresh_stride < kLatentRow || fresh_stride % 8)))
        return TQ_ERR_INVALID;
    if (B == 0 || n == 0) return TQ_OK;
    const int64_t steps = most_steps(cache, B, n, H, max_len);
    if (!steps || B > 65535) return TQ_ERR_UNSUPPORTED;
    if (q_stride > 1ll << 32 || fresh_stride > 1ll << 32) return TQ_ERR_UNSUPPORTED;
    const size_t need = tq_latent_attend_tree_workspace_bytes(cache, B, n, H, max_len);
    if (!q || !o || !lens || (max_len && !table) || !ws || ws_bytes < need) return TQ_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(fresh, 16) || !aligned(ws, 32) || !aligned(mask, 8) || !aligned(table, 4) ||
        !aligned(lens, 4) || !aligned(n_tok, 4))
        return TQ_ERR_INVALID;
    AttendArgs a{};
    a.l.rows = reinterpret_cast<const uint16_t*>(cache->rows);
    a.l.q = reinterpret_cast<const uint16_t*>(q);
    a.l.fresh = reinterpret_cast<const uint16_t*>(fresh);
    a.l.qs = q_stride;
    a.l.fs = fresh_stride;
    a.l.pages = cache->pages;
    a.l.page_stride = cache->page_stride;
    a.l.max_len = max_len;
    a.l.table = table;
    a.l.lens = lens;
    a.l.mask = mask;
    a.l.n_tok = n_tok;
    a.l.B = B;
    a.l.n = n;
    a.l.H = H;
    a.l.table_stride = table_stride;
    a.l.lpage = ilog2(cache->page);
    a.l.scale2 = scale * 1.4426950408889634f;
    a.l.o = reinterpret_cast<uint16_t*>(o);
    a.l.err = err;
    a.ctas = (int)std::min<int64_t>(steps, std::min(sm_count(), kMaxSms));
    a.pad = 2;
    a.least = 2;
    a.fresh_box = n <= 8 ? 8 : n <= 16 ? 16 : kPlace;  // (a divisor of a place)
    a.part = reinterpret_cast<float*>(ws);
    a.stat = reinterpret_cast<float2*>(a.part + 2ll * a.ctas * kRows * kLatent);
    a.wait_cycles = wait_budget();
    const bool bf = cache->dt == TQ_BF16;
    CUtensorMap rows, drafts;
    // (an empty pool has no page that a copy could reach)
    if (!tensor_map(&rows, bf, cache->pages ? cache->rows : q, std::max<int64_t>(cache->pages * cache->page_stride, 1), kLatentRow,
                    kLatentRow, std::min(cache->page, kPlace)) ||
        !tensor_map(&drafts, bf, fresh ? fresh : q, (int64_t)B * n, kLatentRow, fresh ? fresh_stride : kLatentRow, a.fresh_box))
        return TQ_ERR_CUDA;
    return bf ? launch<true>(a, rows, drafts, as_stream(stream)) : launch<false>(a, rows, drafts, as_stream(stream));
}
