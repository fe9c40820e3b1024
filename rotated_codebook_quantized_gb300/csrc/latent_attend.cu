// Attention of drafted trees over the paged latent cache (the absorbed form), on the 5th-generation tensor cores.
//
// A cached row of 576 elements is the key of every head and its first 512 the value, so 64 query rows (heads of drafts) share
// each token that is read.  A persistent CTA takes steps of 32 tokens; they come by tensor copies into a ring of five places, one 128-byte
// swizzled row a token for each 64 elements, which serves as the K-major operand of
//   scores   S[64 x 32]   = Q (TMEM; a third in shared memory) . K^T     36 MMAs of K = 16
// and as the MN-major operand of
//   values   O[64 x 512] += P (shared) . V                               2 x 2 MMAs of K = 16, N = 256
// M = 64 takes 16 of the 32 TMEM lanes of each warp: O's upper half of the elements lies in the other 16, so that O takes 256
// columns, six blocks of Q (in both halves of the lanes) 192 and two places of scores 64.  Q in shared memory as a whole would leave
// room for four steps (193 us for 204 over trees).  Scores and values are issued by a thread each: behind its own products a
// thread's next wait is held up, so that one for both leaves the tensor cores idle between them (1810 clocks a step for 1560).
// A row's running maximum follows only when a score passes it by a set amount.
//
// Tokens past the end and drafts that hold something that is not finite are zeroed in shared memory by two guard warps (a
// masked weight of 0 times NaN would reach the rows that do not see it); only steps that have such tokens wait for them.
// Every wait on an mbarrier is bounded; on expiry the CTA sets TQ_DEVERR_TIMEOUT, drains and frees TMEM.
//
// Up to 64 rows a sequence: bound by HBM, 1600 clocks a step of 1575 at the copy rate, and by its beginning and end: 32 ragged sequences
// of up to 16384 tokens, 64 heads: 69 us, 4.6 TB/s of 6.75 over the whole call (73 over others at each call); 64 rows over 131072
// tokens: 50 us.  More rows: by the products, 1090 of 1360 clocks a step (M = 64 runs at half rate): 512 rows over 65536 tokens, two sequences: 182 us, 800 TFLOP/s.
#include <math.h>

#include <algorithm>

#include "latent.cuh"
#include "tensor.cuh"

namespace tq {
namespace {

using namespace tc;

constexpr int kRows = 64, kTok = 32, kPlaces = 5;  // query rows of a tile; tokens of a step; steps in the ring
constexpr int kBlocks = kLatentRow / 64;           // 128-byte pieces of a row
constexpr int kFetch = 2;  // steps that the L2 cache is told of ahead (4: 2 % slower over ragged sequences, none: 7 % over trees)
constexpr int kMaxSms = 256;
constexpr int kSoft = 4, kMma = 4, kCopy = 6, kGuard = 7, kWarps = 9;
constexpr uint32_t kRingBlock = kPlaces * kTok * 128, kQBlock = kRows * 128;  // bytes of 64 elements of the ring's tokens, of the queries
constexpr int kQTmem = 6;  // blocks of the queries that lie in TMEM; the others in shared memory
constexpr uint32_t kQ = 0, kRing = kQ + (kBlocks - kQTmem) * kQBlock, kP = kRing + kBlocks * kRingBlock, kControl = kP + 2 * kQBlock;  // (a spare tile behind the weights)
constexpr uint32_t kSmem = kControl + 1024 + 1024;  // the last for the start's alignment

struct AttendArgs {
    LatentArgs l;
    int ctas, pad, least;  // of the schedule: CTAs, places that beginning a unit weighs, fewest places of a run
    int fresh_box;         // rows of a copy of drafts
    float* part;           // [2 ctas][64][512]
    float2* stat;          // [2 ctas][64]: level and sum
    int2* units;           // [B][tiles]: first and last CTA of each unit, written by the first
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
    s.tiles = s.steps ? (s.live * a.H + kRows - 1) / kRows : 0;  // (without steps there is nothing to do)
    return s;
}

// How the units are shared out.  Where there are no more of them than CTAs, each is cut into equal segments of at most `per` steps, as
// few steps as let every segment have a CTA of its own: the tiles of a sequence then read the same tokens at the same time, which
// the L2 cache holds for all but the first (two sequences of 65536 tokens and 8 tiles: 1.05 GB from memory in runs that cross
// tiles, 0.16 GB in segments).  Where there are more, a CTA takes a run of `per` places on an axis on which a unit has a place for
// each step and `pad` for its beginning.
struct Plan {
    int per, pad, total;  // pad < 0: segments; total: places
};
TQ_DEVFN int segments_of(int steps, int per) { return (steps + per - 1) / per; }
TQ_DEVFN int places_of(const Seq& s, const Plan& p) {
    return s.tiles * (p.pad < 0 ? segments_of(s.steps, p.per) : s.steps + p.pad);
}
TQ_DEVFN Plan make_plan(const AttendArgs& a) {  // (one warp)
    const int lane = threadIdx.x & 31;
    int steps = 0, units = 0, most = 0;
    for (int b = lane; b < a.l.B; b += 32) {
        const Seq q = seq(a.l, b);
        steps += q.steps * q.tiles;
        units += q.tiles;
        most = max(most, q.tiles ? q.steps : 0);
    }
    steps = __reduce_add_sync(kFull, steps);
    units = __reduce_add_sync(kFull, units);
    most = __reduce_max_sync(kFull, most);
    Plan p{};
    if (units > a.ctas) {
        p.pad = min(a.pad, steps / (4 * a.ctas));
        p.total = steps + units * p.pad;
        p.per = (p.total + a.ctas - 1) / a.ctas;
        return p;
    }
    p.pad = -1;
    int lo = min(max((steps + a.ctas - 1) / a.ctas, a.least), max(most, 1)), hi = max(most, 1);  // (with `most` there are as many as units)
    const Seq own = lane < a.l.B ? seq(a.l, lane) : Seq{};
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        int n = own.tiles * segments_of(own.steps, mid);
        for (int b = lane + 32; b < a.l.B; b += 32) {
            const Seq q = seq(a.l, b);
            n += q.tiles * segments_of(q.steps, mid);
        }
        if ((int)__reduce_add_sync(kFull, n) <= a.ctas) hi = mid;
        else lo = mid + 1;
    }
    p.per = lo;
    p.total = a.ctas;
    return p;
}

struct Run {
    Plan plan;
    int at, end, b, places;  // first place, end; places before sequence b, the last one that begins at or before it
};
TQ_DEVFN Run find_run(const AttendArgs& a, int cta) {
    const int lane = threadIdx.x & 31;
    Run r{};
    r.plan = make_plan(a);
    const int width = r.plan.pad < 0 ? 1 : r.plan.per;
    r.at = (int)min((int64_t)cta * width, (int64_t)r.plan.total);
    r.end = min(r.at + width, r.plan.total);
    bool found = false;
    for (int b0 = 0; b0 < a.l.B; b0 += 32) {
        const int own = b0 + lane < a.l.B ? places_of(seq(a.l, b0 + lane), r.plan) : 0;
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
            found = true;
            break;
        }
        r.places += __shfl_sync(kFull, upto, 31);
    }
    if (!found) r.end = r.at;  // past the last segment
    return r;
}

// A stretch of a run within one unit: steps s0 .. s1 - 1 of it.
struct Stretch {
    Seq s;
    int b, tile, s0, s1;
    int last;  // of the unit's CTAs, where this is the first
};
struct Walk {
    Run r;
    Walk() = default;
    TQ_DEVFN explicit Walk(const Run& run) : r(run) {}
    TQ_DEVFN bool next(const LatentArgs& a, Stretch& x) {
        while (r.at < r.end) {
            x.s = seq(a, r.b);
            int all = places_of(x.s, r.plan);
            while (r.at >= r.places + all) {  // into the next sequence that has any
                r.places += all;
                x.s = seq(a, ++r.b);
                all = places_of(x.s, r.plan);
            }
            const int own = all / x.s.tiles, pad = r.plan.pad;
            x.b = r.b;
            x.tile = (r.at - r.places) / own;
            const int at = r.at - r.places - x.tile * own;
            if (pad < 0) {  // segment `at` of `own`
                const int len = (x.s.steps + own - 1) / own;
                x.s0 = min(at * len, x.s.steps);
                x.s1 = min(x.s0 + len, x.s.steps);
                x.last = r.at + (x.s.steps + len - 1) / len - 1;  // (segments at the end may be empty)
                ++r.at;
            } else {
                const int to = min(own, at + (r.end - r.at));
                x.last = (r.at - at + own - 1) / r.plan.per;
                r.at += to - at;
                x.s0 = max(at - pad, 0);
                x.s1 = to - pad;
            }
            if (x.s0 < x.s1) return true;
        }
        return false;
    }
};

struct Control {
    uint64_t full[kPlaces], empty[kPlaces], guarded[kPlaces];  // of the ring's places
    uint64_t s_ready[2], p_ready[2], o_done[2], q_ready, drain;                              // [2]: of even and odd steps
    uint32_t valid[kPlaces], odd[kPlaces][2];  // of a step's tokens: those that exist; drafts that are not finite
    Walk walk;      // past the CTA's first stretch
    Stretch first;  // which it is
    uint32_t tmem;
    int some, abort;
};
static_assert(sizeof(Control) <= 1024, "control block");

// Tokens of a step that its products take: up to the last one that exists, in sixteens.
TQ_DEVFN int used_of(uint32_t valid) { return valid >> 16 ? 32 : 16; }

TQ_DEVFN void stg128(float* p, const uint32_t* v) {
    asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
// A partial result: 16-byte pieces [4 warps][8 x 32 elements][8][32 lanes], as the warps hold them, so that each store is one run of
// 512 bytes.  Piece e (4 elements) of a row lies at:
TQ_DEVFN int64_t part_at(int64_t slot, int row, int e) {
    const int lane = (row & 15) + (e >> 6) * 16, q = (e >> 3) & 7;
    return (slot * kRows * (kLatent / 4) + (((row >> 4) * 8 + q) * 8 + (e & 7)) * 32 + lane) * 4;
}

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
            for (int i = 0; i < kPlaces; ++i) {
                mbar_init(c.full + i, 1);
                mbar_init(c.empty + i, 3);  // the products and the guards
                mbar_init(c.guarded + i, 2);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(c.s_ready + i, 1);
                mbar_init(c.p_ready + i, 32 * kSoft);
                mbar_init(c.o_done + i, 1);
            }
            mbar_init(&c.q_ready, 32 * kSoft);
            mbar_init(&c.drain, 2);
            fence_mbar_init();
        }
        __syncwarp();
        alloc512(&c.tmem);
    } else if (warp == kCopy) {
        if (lane == 0) {
            prefetch_map(&map_rows);
            prefetch_map(&map_fresh);
        }
        pdl_wait();
        const Run run = find_run(a, blockIdx.x);
        if (lane == 0) {
            Walk walk(run);
            c.some = walk.next(l, c.first);
            c.walk = walk;
        }
        __syncwarp();
        // the first tile's queries, before the tokens' copies: they are what the products wait for
        const uint32_t lines = c.some ? min(kRows, c.first.s.live * l.H - c.first.tile * kRows) * kBlocks : 0;
        for (uint32_t i = lane; i < lines; i += 32) {
            const uint32_t y = c.first.tile * kRows + i / kBlocks, token = y / (uint32_t)l.H;
            const uint16_t* at = l.q + ((int64_t)c.first.b * l.n + token) * l.qs + (int64_t)(y - token * l.H) * kLatentRow + i % kBlocks * 64;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
        }
    }
    pdl_wait();
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = c.tmem, to_s = tmem + 256, to_q = tmem + 320;
    Walk walk = c.walk;
    Stretch x = c.first;
    bool some = c.some;
    uint32_t g = 0, seg = 0;  // steps and stretches of this CTA so far: the phases of every barrier
    // Each role walks the CTA's stretches on its own.

    if (warp == kCopy) {
        // ------------------------------------------------------------ tensor copies of the tokens
        const int box = min(1 << l.lpage, kTok), boxes = kTok / box;
        bool ok = true;
        uint32_t issued = 0;  // places filled so far
        for (; ok && some; some = walk.next(l, x)) {
            const int32_t* table = l.table + (int64_t)x.b * l.table_stride;
            // page ids, a lane to a 16-token piece, of 16 steps and of the next 16
            auto look = [&](int s) {
                const int64_t t = (int64_t)s * kTok + lane * 16;
                return t < x.s.len ? table[t >> l.lpage] : -1;
            };
            int ids = 0, ids_next = look(x.s0);
            // Step s (within the 16 that `from` holds, from s0 on) into the L2 cache: it then arrives while earlier ones are worked on, and
            // while the CTA waits for its queries.
            auto fetch = [&](int s, int s0, int from) {
                const int piece = 2 * (s - s0), id0 = __shfl_sync(kFull, from, piece & 31), id1 = __shfl_sync(kFull, from, (piece + 1) & 31);
                if (s >= min(x.s1, x.s.ctx)) return;
                if (lane < kBlocks && (uint32_t)id0 < (uint64_t)l.pages)
                    prefetch_2d(&map_rows, lane * 64, (int)((int64_t)id0 * l.page_stride) + ((s * kTok) & ((1 << l.lpage) - 1)));
                if (boxes == 2 && lane < kBlocks && (uint32_t)id1 < (uint64_t)l.pages)
                    prefetch_2d(&map_rows, lane * 64, (int)((int64_t)id1 * l.page_stride));
            };
            for (int k = 0; k < kFetch; ++k) fetch(x.s0 + k, x.s0, ids_next);
            for (int s = x.s0; s < x.s1 && ok; ++s, ++g) {
                const uint32_t place = g % kPlaces, phase = (g / kPlaces) & 1;
                const bool context = s < x.s.ctx;
                const int piece = 2 * ((s - x.s0) & 15);
                if (piece == 0) {
                    ids = ids_next;
                    ids_next = look(s + 16);
                }
                const int ahead = ((s - x.s0) & 15) + kFetch;
                fetch(s + kFetch, s + kFetch - (ahead & 15), ahead < 16 ? ids : ids_next);
                uint32_t valid;
                const int id0 = __shfl_sync(kFull, ids, piece), id1 = __shfl_sync(kFull, ids, piece + 1);
                if (context) {
                    const int count = x.s.len - s * kTok;  // at least 1
                    const bool good0 = (uint32_t)id0 < (uint64_t)l.pages, good1 = (uint32_t)id1 < (uint64_t)l.pages;
                    if ((!good0 || (count > 16 && !good1)) && lane == 0 && l.err) atomicOr(l.err, TQ_DEVERR_BAD_PAGE);
                    valid = count >= 32 ? ~0u : (1u << count) - 1;
                    valid &= (good0 ? 0xffffu : 0u) | (good1 ? 0xffff0000u : 0u);
                } else {
                    const int count = x.s.live - (s - x.s.ctx) * kTok;
                    valid = count >= 32 ? ~0u : (1u << count) - 1;
                }
                ok = __all_sync(kFull, mbar_wait(c.empty + place, phase ^ 1, abort_flag, a.wait_cycles));
                if (!ok) break;
                const uint32_t dst = base + kRing + place * (kTok * 128);
                if (elected()) {
                    c.valid[place] = valid;
                    if (context) {
                        const bool on0 = valid & 0xffffu, on1 = boxes == 2 && (valid >> 16);
                        // (pages of 32 tokens and more hold the whole step)
                        const int row0 = (int)((int64_t)id0 * l.page_stride) + ((s * kTok) & ((1 << l.lpage) - 1));
                        mbar_expect_tx(c.full + place, (on0 + on1) * box * 128 * kBlocks);
                        if (on0)
#pragma unroll
                            for (int d = 0; d < kBlocks; ++d) tma_load_2d(dst + d * kRingBlock, &map_rows, d * 64, row0, c.full + place);
                        if (on1)
#pragma unroll
                            for (int d = 0; d < kBlocks; ++d)
                                tma_load_2d(dst + d * kRingBlock + 16 * 128, &map_rows, d * 64, (int)((int64_t)id1 * l.page_stride),
                                            c.full + place);
                    } else {
                        const int t = (s - x.s.ctx) * kTok, copies = (min(kTok, x.s.live - t) + a.fresh_box - 1) / a.fresh_box;
                        mbar_expect_tx(c.full + place, copies * a.fresh_box * 128 * kBlocks);
                        for (int p = 0; p < copies; ++p)
#pragma unroll
                            for (int d = 0; d < kBlocks; ++d)
                                tma_load_2d(dst + d * kRingBlock + p * a.fresh_box * 128, &map_fresh, d * 64,
                                            x.b * l.n + t + p * a.fresh_box, c.full + place);
                    }
                }
                __syncwarp();
                ++issued;
            }
        }
        // no copy may be in flight when the CTA ends (on an abort: nobody else has waited for them)
        for (int at = 0; at < kPlaces; ++at) {
            const uint32_t fills = (issued + kPlaces - 1 - at) / kPlaces;
            if (fills) mbar_wait_drain(c.full + at, (fills - 1) & 1);
        }
    } else if (warp == kMma) {
        // ------------------------------------------------------------ MMA issue: scores
        if (elected()) {
            bool ok = true;
            const uint64_t dq = desc(base + kQ, 16), dk = desc(base + kRing, 16);
            for (; ok && some; some = walk.next(l, x), ++seg) {
                ok = mbar_wait(&c.q_ready, seg & 1, abort_flag, a.wait_cycles);
                if (!ok) break;  // (else it would issue on queries that are still being copied)
                for (int s = x.s0; s < x.s1; ++s, ++g) {
                    const uint32_t place = g % kPlaces, phase = (g / kPlaces) & 1;
                    ok = mbar_wait(c.full + place, phase, abort_flag, a.wait_cycles);
                    if (!ok) break;
                    const uint32_t valid = c.valid[place];
                    if (valid != ~0u || s >= x.s.ctx) ok = mbar_wait(c.guarded + place, phase, abort_flag, a.wait_cycles);
                    // the scores of two steps before have been read when their weights are there
                    if (ok && g > 1) ok = mbar_wait(c.p_ready + (g & 1), ((g - 2) >> 1) & 1, abort_flag, a.wait_cycles);
                    if (!ok) break;
                    fence_after();
                    const uint32_t id = idesc(BF, kRows, used_of(valid), 0), to = to_s + kTok * (g & 1);
                    const uint64_t k0 = dk + place * (kTok * 128 / 16);
#pragma unroll
                    for (int d = 0; d < kQTmem; ++d)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_ts(to, to_q + 32 * d + 8 * k, k0 + d * (kRingBlock / 16) + 2 * k, id, (d | k) != 0);
#pragma unroll
                    for (int d = kQTmem; d < kBlocks; ++d)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_ss(to, dq + (d - kQTmem) * (kQBlock / 16) + 2 * k, k0 + d * (kRingBlock / 16) + 2 * k, id, 1);
                    commit(c.s_ready + (g & 1));
                }
            }
            commit(&c.drain);  // completes when every MMA issued above has finished
        }
        __syncwarp();
    } else if (warp == kMma + 1) {
        // ------------------------------------------------------------ MMA issue: values
        if (elected()) {
            bool ok = true;
            const uint64_t dv = desc(base + kRing, kRingBlock), dp = desc(base + kP, 16);
            for (; ok && some; some = walk.next(l, x)) {
                for (int s = x.s0; s < x.s1; ++s, ++g) {
                    const uint32_t place = g % kPlaces;
                    ok = mbar_wait(c.p_ready + (g & 1), (g >> 1) & 1, abort_flag, a.wait_cycles);
                    if (!ok) break;
                    // (complete since before the scores; waiting on it too orders `valid` before its read)
                    ok = mbar_wait(c.full + place, (g / kPlaces) & 1, abort_flag, a.wait_cycles);
                    if (!ok) break;
                    fence_after();
                    const uint64_t v0 = dv + place * (kTok * 128 / 16), p0 = dp + 4 * (g & 1);
                    constexpr uint32_t id = idesc(BF, kRows, 256, 1);
                    const uint32_t more = s != x.s0;
                    const bool both = used_of(c.valid[place]) == 32;
                    mma_ss(tmem, p0, v0, id, more);
                    mma_ss(tmem + (16u << 16), p0, v0 + 4 * (kRingBlock / 16), id, more);
                    if (both) {
                        mma_ss(tmem, p0 + 2, v0 + 128, id, 1);
                        mma_ss(tmem + (16u << 16), p0 + 2, v0 + 128 + 4 * (kRingBlock / 16), id, 1);
                    }
                    commit(c.empty + place);
                    commit(c.o_done + (g & 1));
                }
            }
            commit(&c.drain);
        }
        __syncwarp();
    } else if (warp >= kGuard) {
        // ------------------------------------------------------------ guards: a warp to every other token
        bool ok = true;
        for (; ok && some; some = walk.next(l, x)) {
            for (int s = x.s0; s < x.s1 && ok; ++s, ++g) {
                const uint32_t place = g % kPlaces, phase = (g / kPlaces) & 1;
                const bool context = s < x.s.ctx;
                ok = __all_sync(kFull, mbar_wait(c.full + place, phase, abort_flag, a.wait_cycles));
                if (!ok) break;
                const uint32_t valid = c.valid[place];
                if (valid != ~0u || !context) {
                    uint8_t* const tokens = smem + kRing + place * (kTok * 128);
                    uint32_t odd = 0;  // (this warp's: the even or the odd tokens)
                    if (!context) {
                        constexpr uint32_t kTop = BF ? 0x7f807f80u : 0x7c007c00u;
                        const int count = 32 - __clz(valid);
                        for (int t = warp - kGuard; t < count; t += 2) {
                            bool bad = false;
#pragma unroll
                            for (int d = 0; d < 3; ++d) {  // 72 pieces of 16 bytes, in any order
                                const int piece = d * 32 + lane;
                                if (piece < kBlocks * 8) {
                                    const uint4 v = *reinterpret_cast<const uint4*>(tokens + (piece >> 3) * kRingBlock + t * 128 + (piece & 7) * 16);
                                    bad |= (__vcmpeq2(v.x & kTop, kTop) | __vcmpeq2(v.y & kTop, kTop) | __vcmpeq2(v.z & kTop, kTop) |
                                            __vcmpeq2(v.w & kTop, kTop)) != 0;
                                }
                            }
                            if (__any_sync(kFull, bad)) odd |= 1u << t;
                        }
                        if (lane == 0) c.odd[place][warp - kGuard] = odd;
                    }
                    const int used = used_of(valid);
                    bool wrote = false;
                    for (int t = warp - kGuard; t < used; t += 2)
                        if (!((valid & ~odd) >> t & 1)) {
                            wrote = true;
#pragma unroll
                            for (int d = 0; d < 3; ++d) {
                                const int piece = d * 32 + lane;
                                if (piece < kBlocks * 8)
                                    *reinterpret_cast<uint4*>(tokens + (piece >> 3) * kRingBlock + t * 128 + (piece & 7) * 16) =
                                        make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                    if (wrote) fence_async_smem();
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(c.guarded + place);
                    mbar_arrive(c.empty + place);
                }
            }
        }
    } else {
        // ------------------------------------------------------------ softmax: rows lane / 4 and lane / 4 + 8 of the warp's 16
        const uint32_t lanes = (uint32_t)warp << 21;
        const int words = (l.n + 63) / 64;
        const float f = fabsf(l.scale2);
        const f2 ff = pk(f, f);
        bool ok = true;
        for (; ok && some; some = walk.next(l, x)) {
            const uint32_t ge = g + (x.s1 - x.s0);
            const uint32_t y0 = x.tile * kRows;
            const int rows = min(kRows, x.s.live * l.H - (int)y0);
            if (x.s0 == 0 && tid == 0)  // (before any wait: the join takes these for indices)
                a.units[(int64_t)x.b * ((l.n * l.H + kRows - 1) / kRows) + x.tile] = make_int2(blockIdx.x, x.last);
            // ---- the tile's queries (the last scores of the stretch before have been read, so its queries are free)
            // Six blocks go to TMEM, whose lanes 16 .. 31 of a warp repeat its 16 rows (M = 64 wants A in both halves), by way of
            // shared memory: five where the others, the weights and a spare tile lie, then one beside the others.
            {
                const int r0 = warp * 16, r = r0 + (lane & 15);
                const uint16_t* src[4];  // eight lanes to a row, 16 bytes each
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t y = y0 + min(r0 + 4 * k + (lane >> 3), rows - 1), token = y / (uint32_t)l.H;
                    src[k] = l.q + ((int64_t)x.b * l.n + token) * l.qs + (int64_t)(y - token * l.H) * kLatentRow + (lane & 7) * 8;
                }
                auto bring = [&](int d, uint32_t tile) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = r0 + 4 * k + (lane >> 3);
                        const uint32_t dst = base + tile + row * 128 + (((lane ^ row) & 7) << 4);
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src[k] + d * 64) : "memory");
                    }
                };
                auto move = [&](int d, uint32_t tile) {
                    uint32_t v[32];
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        const uint4 z = *reinterpret_cast<const uint4*>(smem + tile + r * 128 + ((p ^ (r & 7)) << 4));
                        v[4 * p] = z.x, v[4 * p + 1] = z.y, v[4 * p + 2] = z.z, v[4 * p + 3] = z.w;
                    }
                    st32(to_q + 32 * d + lanes, v);
                };
                auto tile_of = [](int d) { return d < 3 ? kQ + d * kQBlock : kP + (d - 3) * kQBlock; };
#pragma unroll
                for (int d = 0; d < kQTmem - 1; ++d) bring(d, tile_of(d));
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
#pragma unroll 1
                for (int d = 0; d < kQTmem - 1; ++d) move(d, tile_of(d));
                __syncwarp();
                bring(kQTmem - 1, kP);
#pragma unroll
                for (int d = kQTmem; d < kBlocks; ++d) bring(d, kQ + (d - kQTmem) * kQBlock);
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                move(kQTmem - 1, kP);
                wait_st();
                __syncwarp();  // (its tile takes weights next)
                fence_before();
                fence_async_smem();
                mbar_arrive(&c.q_ready);
            }
            float m[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, bias[2] = {0.f, 0.f};
            int draft[2];  // of the two rows
#pragma unroll
            for (int j = 0; j < 2; ++j) draft[j] = (y0 + min(warp * 16 + (lane >> 2) + 8 * j, rows - 1)) / (uint32_t)l.H;
            for (uint32_t i = g; i < ge; ++i) {
                const uint32_t place = i % kPlaces, phase = (i / kPlaces) & 1;
                const int s = x.s0 + (int)(i - g);
                ok = __all_sync(kFull, mbar_wait(c.s_ready + (i & 1), (i >> 1) & 1, abort_flag, a.wait_cycles));
                if (!ok) break;
                fence_after();
                uint32_t v[16];  // of 8 columns k: element 4 k + 2 j + e is row j, column 8 k + 2 (lane % 4) + e
                ld16x32(to_s + kTok * (i & 1) + lanes, v);
                // (its tokens' barrier has completed before the scores; waiting on it too orders `valid` before its read)
                ok = __all_sync(kFull, mbar_wait(c.full + place, phase, abort_flag, a.wait_cycles));
                if (!ok) break;
                const uint32_t valid = c.valid[place];
                const bool whole = valid == ~0u && s < x.s.ctx;
                uint32_t see[2] = {valid, valid};
                bool spoilt[2] = {false, false};
                if (s >= x.s.ctx) {
                    ok = __all_sync(kFull, mbar_wait(c.guarded + place, phase, abort_flag, a.wait_cycles));
                    if (!ok) break;
                    const uint32_t odd = c.odd[place][0] | c.odd[place][1];
                    const int w = s - x.s.ctx;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t bits;
                        if (l.mask) bits = (uint32_t)(l.mask[((int64_t)x.b * l.n + draft[j]) * words + (w >> 1)] >> (32 * (w & 1)));
                        else bits = draft[j] >= 32 * w + 31 ? ~0u : draft[j] < 32 * w ? 0u : (2u << (draft[j] - 32 * w)) - 1;
                        see[j] &= bits;
                        spoilt[j] = (see[j] & odd) != 0;
                    }
                }
                wait_ld();
                float top[2] = {-INFINITY, -INFINITY};
                if (l.scale2 < 0)
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] ^= 0x80000000u;
                if (!whole)
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (!((see[(k >> 1) & 1] >> (8 * (k >> 2) + 2 * (lane & 3) + (k & 1))) & 1)) v[k] = __float_as_uint(-INFINITY);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    top[k & 1] = fmaxf(fmaxf(top[k & 1], __uint_as_float(v[2 * k])), __uint_as_float(v[2 * k + 1]));
                top[0] *= f;
                top[1] *= f;
                if (__any_sync(kFull, top[0] - m[0] > Weights<BF>::kSlack || top[1] - m[1] > Weights<BF>::kSlack)) {
                    float r[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        top[j] = fmaxf(top[j], __shfl_xor_sync(kFull, top[j], 1));
                        top[j] = fmaxf(top[j], __shfl_xor_sync(kFull, top[j], 2));
                        // (each row by its own scores alone: its result must not hang on what its neighbours see)
                        const float n = top[j] - m[j] > Weights<BF>::kSlack ? top[j] : m[j], to = Weights<BF>::bias(n);
                        r[j] = m[j] == -INFINITY ? 0.f : exp2_fast(to - bias[j]);
                        m[j] = n;
                        bias[j] = to;
                        sum[j] *= r[j];
                    }
                    if (i != g) {  // the sums so far, once the last product has written them
                        ok = __all_sync(kFull, mbar_wait(c.o_done + ((i - 1) & 1), ((i - 1) >> 1) & 1, abort_flag, a.wait_cycles));
                        if (!ok) break;
                        fence_after();
                        // row lane % 16 of O's two halves
                        const float lo = __shfl_sync(kFull, r[0], (lane & 7) * 4), hi = __shfl_sync(kFull, r[1], (lane & 7) * 4);
                        const float by = lane & 8 ? hi : lo;
#pragma unroll 1
                        for (int q = 0; q < 8; ++q) {
                            uint32_t o[32];
                            ld32(tmem + lanes + 32 * q, o);
                            wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
                            st32(tmem + lanes + 32 * q, o);
                        }
                        wait_st();
                    }
                }
                // ---- weights; the sum takes them before their rounding
                uint32_t w[8];
                const f2 bb[2] = {pk(bias[0], bias[0]), pk(bias[1], bias[1])};
                f2 ls[2] = {0, 0}, by = ff;
                if (__any_sync(kFull, huge(m[0]) || huge(m[1]))) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__fmul_rn(__uint_as_float(v[k]), f));
                    by = pk(1.f, 1.f);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 y = un(fma2(pk(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), by, bb[k & 1]));
                    const float p0 = exp2_fast(y.x), p1 = exp2_fast(y.y);
                    ls[k & 1] = add2(ls[k & 1], pk(p0, p1));
                    w[k] = pack16<BF>(p0, p1);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 z = un(ls[j]);
                    sum[j] += z.x + z.y;
                    if (spoilt[j]) sum[j] = NAN;
                }
                if (i > 1) {  // the products two steps before have read these weights' place
                    ok = __all_sync(kFull, mbar_wait(c.o_done + (i & 1), ((i - 2) >> 1) & 1, abort_flag, a.wait_cycles));
                    if (!ok) break;
                }
                uint8_t* const to = smem + kP + (warp * 16 + (lane >> 2)) * 128 + (lane & 3) * 4;
                const int half = 4 * (i & 1), turn = lane >> 2;  // (both rows are lane / 4 mod 8)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<uint32_t*>(to + (k & 1) * 1024 + (((half + (k >> 1)) ^ turn) << 4)) = w[k];
                fence_before();
                fence_async_smem();
                mbar_arrive(c.p_ready + (i & 1));
            }
            if (!ok) break;
            // ---- the stretch's result: the rows themselves where it is the whole unit, else a partial result
            ok = __all_sync(kFull, mbar_wait(c.o_done + ((ge - 1) & 1), ((ge - 1) >> 1) & 1, abort_flag, a.wait_cycles));
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
            const bool mine = row < rows;
            const int64_t slot = 2ll * blockIdx.x + (x.s0 == 0);
            if (x.s0 == 0 && x.s1 == x.s.steps) {
                const float over = total == 0.f ? 0.f : 1.f / total;  // (a NaN sum stays one)
                uint16_t* out = l.o + ((int64_t)x.b * l.n * l.H + y0 + min(row, rows - 1)) * kLatent + (lane >> 4) * 256;
#pragma unroll 1
                for (int q = 0; q < 8; ++q) {
                    uint32_t o[32];
                    ld32(tmem + lanes + 32 * q, o);
                    wait_ld();
                    if (mine) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t z[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                z[k] = pack16<BF>(__uint_as_float(o[8 * e + 2 * k]) * over, __uint_as_float(o[8 * e + 2 * k + 1]) * over);
                            *reinterpret_cast<uint4*>(out + 32 * q + 8 * e) = make_uint4(z[0], z[1], z[2], z[3]);
                        }
                    }
                    __syncwarp();
                }
            } else {
                if (lane < 16) a.stat[slot * kRows + row] = make_float2(lev, total);
                float* const part = a.part + (slot * kRows * (kLatent / 4) + (int64_t)warp * 2048 + lane) * 4;
#pragma unroll 2
                for (int q = 0; q < 8; ++q) {
                    uint32_t o[32];
                    ld32(tmem + lanes + 32 * q, o);
                    wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) stg128(part + (q * 8 + e) * 128, o + 4 * e);
                }
            }
            fence_before();
            g = ge;
            ++seg;
        }
    }

    if (warp == kMma && elected() && !mbar_wait_drain(&c.drain, 0)) *abort_flag = 1;
    __syncwarp();
    fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag && l.err) atomicOr(l.err, TQ_DEVERR_TIMEOUT);
    if (warp == kMma) {
        fence_after();
        dealloc512(tmem);
    }
}

// What the CTAs left in parts, joined in their order; rows that see nothing, and drafts that are not in use, are zeros.  A warp's lanes
// have the 512 bytes that a warp of the attention stored at a time, and the 512 after them: 8 elements of 16 rows and two halves;
// 128 such pieces make a tile.  SPLIT: the parts are dealt to the CTA's 8 warps, a CTA to a piece, where few units are in many parts
// (64 rows over 131072 tokens, one unit in 152 parts: the call 118 us without).
template <bool BF, bool SPLIT>
__global__ void __launch_bounds__(256) latent_join_kernel(const __grid_constant__ AttendArgs a) {
    constexpr int kJoin = 8, kAhead = 4;  // warps; parts on their way at a time
    __shared__ float s_sum[SPLIT ? kJoin : 1][10][32];
    pdl_trigger();
    pdl_wait();
    const LatentArgs& l = a.l;
    const int b = blockIdx.y, tile = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (l.err && tile == 0 && blockIdx.z == 0 && tid == 0 && l.lens[b] != latent_len(l, b)) atomicOr(l.err, TQ_DEVERR_BAD_PAGE);
    const Seq s = seq(l, b);
    const int64_t y0 = (int64_t)tile * kRows;
    const int rows = (int)max(min((int64_t)kRows, (int64_t)l.n * l.H - y0), (int64_t)0);  // of the output
    const int live = s.steps ? (int)max(min((int64_t)rows, (int64_t)s.live * l.H - y0), (int64_t)0) : 0;
    uint16_t* const out = l.o + ((int64_t)b * l.n * l.H + y0) * kLatent;
    for (int i = live * (kLatent / 8) + blockIdx.z * 256 + tid; i < rows * (kLatent / 8); i += gridDim.z * 256)
        *reinterpret_cast<uint4*>(out + (int64_t)i * 8) = make_uint4(0u, 0u, 0u, 0u);
    if (live == 0) return;
    const int2 unit = a.units[(int64_t)b * gridDim.x + tile];
    const int c0 = unit.x, c1 = unit.y;
    if (c0 < 0 || c1 < c0 || c1 >= a.ctas) {  // not written: a CTA gave up in a stretch before this unit, and has reported it
        for (int i = blockIdx.z * 256 + tid; i < live * (kLatent / 8); i += gridDim.z * 256)
            *reinterpret_cast<uint4*>(out + (int64_t)i * 8) = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    if (c0 == c1) return;  // one CTA has written its rows
    auto slot_of = [&](int c) { return 2ll * c + (c == c0); };
    for (int piece = SPLIT ? blockIdx.z : blockIdx.z * kJoin + warp; piece < 128; piece += SPLIT ? 128 : gridDim.z * kJoin) {
        const int row = (piece >> 5) * 16 + (lane & 15), e = (lane >> 4) * 64 + (piece & 31) * 2;
        float o[8] = {}, top = -INFINITY, total = 0.f;
        auto add = [&](float level, float sum, const float4 (&z)[2]) {
            // both to the higher level: weight 1 for its own (also where neither saw anything)
            const float n = fmaxf(top, level), w0 = top == n ? 1.f : exp2_fast(top - n), w1 = level == n ? 1.f : exp2_fast(level - n);
            top = n;
            total = total * w0 + sum * w1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                o[4 * h] = fmaf(o[4 * h], w0, z[h].x * w1);
                o[4 * h + 1] = fmaf(o[4 * h + 1], w0, z[h].y * w1);
                o[4 * h + 2] = fmaf(o[4 * h + 2], w0, z[h].z * w1);
                o[4 * h + 3] = fmaf(o[4 * h + 3], w0, z[h].w * w1);
            }
        };
        constexpr int kDeal = SPLIT ? kJoin : 1;
        for (int c = c0 + (SPLIT ? warp : 0); c <= c1; c += kAhead * kDeal) {
            float2 stat[kAhead];
            float4 z[kAhead][2];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int64_t slot = slot_of(min(c + k * kDeal, c1));
                stat[k] = a.stat[slot * kRows + row];
#pragma unroll
                for (int h = 0; h < 2; ++h) z[k][h] = *reinterpret_cast<const float4*>(a.part + part_at(slot, row, e + h));
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (c + k * kDeal <= c1) add(stat[k].x, stat[k].y, z[k]);
        }
        if (SPLIT) {
            s_sum[warp][8][lane] = top;
            s_sum[warp][9][lane] = total;
#pragma unroll
            for (int k = 0; k < 8; ++k) s_sum[warp][k][lane] = o[k];
            __syncthreads();
            if (warp) return;
            for (int w = 1; w < kJoin; ++w) {
                const float4 z[2] = {make_float4(s_sum[w][0][lane], s_sum[w][1][lane], s_sum[w][2][lane], s_sum[w][3][lane]),
                                     make_float4(s_sum[w][4][lane], s_sum[w][5][lane], s_sum[w][6][lane], s_sum[w][7][lane])};
                add(s_sum[w][8][lane], s_sum[w][9][lane], z);
            }
        }
        const float over = total == 0.f ? 0.f : 1.f / total;  // (a NaN sum stays one)
        if (row < live)
            *reinterpret_cast<uint4*>(out + (int64_t)row * kLatent + e * 4) =
                make_uint4(pack16<BF>(o[0] * over, o[1] * over), pack16<BF>(o[2] * over, o[3] * over),
                           pack16<BF>(o[4] * over, o[5] * over), pack16<BF>(o[6] * over, o[7] * over));
    }
}

// Steps of the whole batch at most; 0 where there are too many.
int64_t most_steps(const tq_latent_pages_t* cache, int32_t B, int32_t n, int32_t H, int64_t max_len) {
    if (latent_check(cache) != TQ_OK || B <= 0 || n <= 0 || H <= 0 || H > 65535 || max_len < 0) return 0;
    const int64_t most = 1ll << 27;  // (with the places of their beginnings below 2^31)
    const int64_t tiles = ((int64_t)n * H + kRows - 1) / kRows, steps = (std::min<int64_t>(max_len, 1ll << 40) + kTok - 1) / kTok + (n + kTok - 1) / kTok;
    if ((int64_t)n * H > most || steps > most || tiles > most / B || tiles * B > most / steps) return 0;
    return tiles * B * steps;
}

template <bool BF>
tq_status launch(const AttendArgs& a, const CUtensorMap& rows, const CUtensorMap& fresh, int64_t steps, cudaStream_t st) {  // steps: of a unit
    if (ensure_smem((const void*)latent_attend_kernel<BF>, kSmem) != cudaSuccess) return TQ_ERR_CUDA;
    tq_status s = launch_pdl(latent_attend_kernel<BF>, dim3((unsigned)a.ctas), dim3(32 * kWarps), kSmem, st, a, rows, fresh);
    if (s != TQ_OK) return s;
    const int64_t tiles = ((int64_t)a.l.n * a.l.H + kRows - 1) / kRows;
    const int64_t units = tiles * a.l.B;
    // The parts of a tile dealt to warps: where there are few tiles in many parts (64 rows over 131072 tokens: 50 us for 96; over 30000
    // tokens, 4 sequences 42 for 54, 8 sequences 63 for 67, 16 sequences 107 for 102).  Else 128 pieces to a tile, over more CTAs
    // where there are fewer tiles (32 ragged sequences of up to 16384: 71, 73, 79 and 130 us with 16, 8, 4 and one; 200 sequences of
    // up to 1500: 71, 69, 69 and 91).
    const bool split = units <= 8 && steps >= 64;
    const dim3 grid((unsigned)tiles, (unsigned)a.l.B, split ? 128 : units <= 64 ? 16 : units <= 256 ? 8 : units <= 1024 ? 2 : 1);
    return launch_pdl(split ? latent_join_kernel<BF, true> : latent_join_kernel<BF, false>, grid, dim3(256), 0, st, a);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" size_t tq_latent_attend_tree_workspace_bytes(const tq_latent_pages_t* cache, int32_t B, int32_t n, int32_t H,
                                                        int64_t max_len) {
    const int64_t steps = most_steps(cache, B, n, H, max_len);
    if (!steps) return 0;
    const int64_t tiles = ((int64_t)n * H + kRows - 1) / kRows;
    return (size_t)(2 * std::min<int64_t>(steps, kMaxSms)) * kRows * (kLatent * sizeof(float) + sizeof(float2)) +
           (size_t)(B * tiles) * sizeof(int2);
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
    a.l.scale2 = score_factor(scale);
    a.l.o = reinterpret_cast<uint16_t*>(o);
    a.l.err = err;
    a.ctas = (int)std::min<int64_t>(steps, std::min(device_sms(), kMaxSms));
    a.pad = 8;    // what beginning a unit costs (200 sequences of up to 1500 tokens: 65.5 us; 4: 69, 0: 78)
    a.least = 4;  // (a segment of fewer steps costs more to join than it saves: three contexts of up to 300 tokens 15.4 us; 1: 16.4)
    a.fresh_box = n <= 8 ? 8 : n <= 16 ? 16 : kTok;  // (a divisor of a step)
    a.part = reinterpret_cast<float*>(ws);
    a.stat = reinterpret_cast<float2*>(a.part + 2ll * a.ctas * kRows * kLatent);
    a.units = reinterpret_cast<int2*>(a.stat + 2ll * a.ctas * kRows);
    a.wait_cycles = wait_budget();
    const bool bf = cache->dt == TQ_BF16;
    CUtensorMap rows, drafts;
    // (an empty pool has no page that a copy could reach)
    if (!tensor_map(&rows, bf, cache->pages ? cache->rows : q, std::max<int64_t>(cache->pages * cache->page_stride, 1), kLatentRow,
                    kLatentRow, std::min(cache->page, kTok)) ||
        !tensor_map(&drafts, bf, fresh ? fresh : q, (int64_t)B * n, kLatentRow, fresh ? fresh_stride : kLatentRow, a.fresh_box))
        return TQ_ERR_CUDA;
    const int64_t own = (max_len + kTok - 1) / kTok;
    return bf ? launch<true>(a, rows, drafts, own, as_stream(stream)) : launch<false>(a, rows, drafts, own, as_stream(stream));
}
