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
// Bound by a step's chain: products 2560 clocks, the step 3400 to 3570 (scores 1030, softmax 1280, values 520 and their hand-overs; the
// next keys, asked for behind the last step's values, take 1700).  A thread to each stream's issue instead of one for both: 1045 us
// for 937.  8192 tokens over 64 heads: 906 us over the same inputs again, 931 over others, 1.48 PFLOP/s, 86 % of the
// measured sustained rate.
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
    int B, H, heads, ctas;  // heads: of a group
    bool causal;
    uint32_t* taken;  // jobs taken beyond each CTA's first; NULL: there are no others
    float* part;      // [CTAs][256 rows][128], where jobs may be cut; NULL: they are not
    float2* stat;     // [CTAs][256]: level and sum
    float scale2;     // scale * log2(e)
    long long wait_cycles;
};

// A job: a tile of a sequence and head.  Its rows and keys as places of the packed arrays.
struct Job {
    int q0, rows;  // rows in use; -1: no more jobs
    int k0, keys;  // of the sequence
    int at;        // key of the first row's own place, less k0; the rows' are at + row (causal)
    int head;
    bool cut;      // one of several parts: the result is a partial one
};
struct Span {
    int q0, q1, k0, k1, tiles;
    bool bad;
};
TQ_DEVFN Span span(const PromptArgs& a, int b) {
    Span s{};
    if (b >= a.B) return s;
    s.q0 = a.q_starts[b], s.q1 = a.q_starts[b + 1], s.k0 = a.kv_starts[b], s.k1 = a.kv_starts[b + 1];
    s.bad = !(s.q0 >= 0 && s.q0 <= s.q1 && s.q1 <= a.Tq && s.k0 >= 0 && s.k0 <= s.k1 && s.k1 <= a.Tkv);
    s.tiles = s.bad ? 0 : (s.q1 - s.q0 + kTile - 1) / kTile;
    return s;
}
// What f is to make of every sequence, 32 at a time, until it returns true (all by one warp; f has the span of sequence b + lane).
// `torn`: some starts are out of order.  A sequence whose queries begin below an earlier start is then left out as well, or
// sequences would lie on one another: rows written by two jobs, and more tiles than the host has counted.
template <class F>
TQ_DEVFN void each_span(const PromptArgs& a, bool torn, F&& f) {
    const int lane = threadIdx.x & 31;
    int top = 0;  // highest start so far, of those within the array
    for (int b = 0; b < a.B; b += 32) {
        Span s = span(a, b + lane);
        if (torn) {
            int upto = max(top, b + lane < a.B && s.q0 <= a.Tq ? s.q0 : 0);
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int x = __shfl_up_sync(kFull, upto, m);
                if (lane >= m) upto = max(upto, x);
            }
            if (b + lane < a.B && s.q0 < upto) s.bad = true, s.tiles = 0;
            top = __shfl_sync(kFull, upto, 31);
        }
        if (f(s, b)) return;
    }
}
// Tiles of a sequence that take more than `steps` steps: its last ones.
TQ_DEVFN int tiles_above(const PromptArgs& a, const Span& s, int steps) {
    if (steps < 0 || !s.tiles) return s.tiles;
    if (s.k1 - s.k0 <= steps * kTok) return 0;
    if (!a.causal) return s.tiles;
    // a tile whose last row is the e-th sees keys - queries + e of them
    return s.tiles - max(steps * kTok + (s.q1 - s.q0) - (s.k1 - s.k0), 0) / kTile;
}
// Few jobs over many keys (a chunk of a prompt late in a long one) are cut into parts along the keys, one to a CTA, and joined: 16
// tokens after 8000, 8 heads 29 us (whole: 105), 700 after 1300, 4 heads 27 (47), 256 after 744, 32 heads 26 (27).
constexpr int kLeast = 4, kParts = 32;  // fewest steps of a part, most parts
// Jobs go in groups of `heads` heads, whose keys and values the L2 cache holds; in a group those with the most steps first.  A CTA
// takes the next one when its copies of the last are under way (shared out beforehand, seven chunks of prompts left a quarter of the
// SMs' time idle).  A warp finds a job by a search of all sequences' lengths, which hides behind the job before while sequences are few: 60
// prompts of 64 tokens, 64 heads 121 us (floor 42), 250 of them 690 (175), and 1000 of 16 tokens 7.2 ms (0.18), 17 us a job.
struct Jobs {
    int tiles, most;  // of a head; steps of the longest
    int parts, per;   // into how many parts jobs are cut, of how many steps at most
    bool torn;        // some sequence is left out
    int64_t rows;     // of the sequences that are not
};
TQ_DEVFN Jobs count_jobs(const PromptArgs& a, bool report) {  // (one warp)
    int tiles = 0, most = 0;
    unsigned rows = 0;
    bool bad = false, torn = false;
    auto count = [&](const Span& s, int) {
        bad |= s.bad;
        tiles += s.tiles;
        if (s.tiles) rows += s.q1 - s.q0;
        if (s.tiles) most = max(most, (s.k1 - s.k0 + kTok - 1) / kTok);
        return false;
    };
    each_span(a, false, count);
    if (__any_sync(kFull, bad)) {
        torn = true;
        tiles = most = rows = 0;
        each_span(a, true, count);
        if (report && bad && a.err) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
    }
    Jobs j{(int)__reduce_add_sync(kFull, tiles), (int)__reduce_max_sync(kFull, most), 1, 0, torn,
           __reduce_add_sync(kFull, rows)};
    const int64_t all = (int64_t)j.tiles * a.H;
    if (a.part && all > 0) j.parts = (int)max(min((int64_t)(a.ctas / all), (int64_t)min(j.most / kLeast, kParts)), (int64_t)1);
    j.per = (j.most + j.parts - 1) / j.parts;
    return j;
}
TQ_DEVFN Job find_job(const PromptArgs& a, const Jobs& jobs, int64_t at) {  // (one warp)
    const int lane = threadIdx.x & 31;
    Job j{};
    j.rows = -1;
    if (at >= (int64_t)jobs.tiles * a.H * jobs.parts) return j;
    const int part = (int)(at % jobs.parts);
    at /= jobs.parts;
    const int group = (int)(at / ((int64_t)jobs.tiles * a.heads)), in = min(a.heads, a.H - group * a.heads);
    const int left = (int)(at - (int64_t)group * jobs.tiles * a.heads);
    j.head = group * a.heads + left % in;
    int rank = left / in;
    // the fewest steps s that no more than `rank` tiles pass
    auto above = [&](int steps) {
        int n = 0;
        each_span(a, jobs.torn, [&](const Span& s, int) {
            n += tiles_above(a, s, steps);
            return false;
        });
        return (int)__reduce_add_sync(kFull, n);
    };
    int lo = 0, hi = jobs.most;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (above(mid) <= rank) hi = mid;
        else lo = mid + 1;
    }
    rank -= above(lo);  // of the tiles of exactly lo steps, in order
    each_span(a, jobs.torn, [&](const Span& s, int) {
        const int over = tiles_above(a, s, lo), own = tiles_above(a, s, lo - 1) - over;
        int upto = own;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int x = __shfl_up_sync(kFull, upto, m);
            if (lane >= m) upto += x;
        }
        const unsigned hit = __ballot_sync(kFull, upto > rank);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int tile = __shfl_sync(kFull, s.tiles - over - 1 - (rank - (upto - own)), src);
            const int q0 = __shfl_sync(kFull, s.q0, src), q1 = __shfl_sync(kFull, s.q1, src);
            j.k0 = __shfl_sync(kFull, s.k0, src);
            j.keys = __shfl_sync(kFull, s.k1, src) - j.k0;
            j.q0 = q0 + tile * kTile;
            j.rows = min(kTile, q1 - j.q0);
            j.at = j.keys - (q1 - q0) + tile * kTile;
            return true;
        }
        rank -= __shfl_sync(kFull, upto, 31);
        return false;
    });
    if (jobs.parts > 1) {  // a part is a job over some of the keys: the rows stand as far before or behind them as they do
        const int from = part * jobs.per * kTok;
        j.cut = true;
        j.k0 += from;
        j.keys = min(max(j.keys - from, 0), jobs.per * kTok);
        j.at -= from;
    }
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

// Zeros in the rows that belong to no sequence: behind the last one, before the first, and those of sequences that are left out.  A
// warp of each CTA.
TQ_DEVFN void clear_rest(const PromptArgs& a, const Jobs& jobs) {
    if (jobs.rows == a.Tq) return;
    const int lane = threadIdx.x & 31;
    const int64_t pieces = (int64_t)a.H * (kHeadValue / 8);  // of 16 bytes, of a row
    auto clear = [&](int64_t from, int64_t to) {
        for (int64_t i = from * pieces + blockIdx.x * 32 + lane; i < to * pieces; i += gridDim.x * 32)
            *reinterpret_cast<uint4*>(a.o + i * 8) = make_uint4(0u, 0u, 0u, 0u);
    };
    int end = 0;  // of the sequence before
    each_span(a, jobs.torn, [&](const Span& s, int) {
        for (unsigned own = __ballot_sync(kFull, s.tiles > 0); own; own &= own - 1) {
            const int src = __ffs(own) - 1, q0 = __shfl_sync(kFull, s.q0, src);
            clear(end, q0);
            end = __shfl_sync(kFull, s.q1, src);
        }
        return false;
    });
    clear(end, a.Tq);
}

struct Control {
    uint64_t q_full[kStreams], q_empty[kStreams], k_full[2], v_full[2], k_empty[2], v_empty[2], guarded[2];  // [2]: even, odd steps
    uint64_t s_ready[kStreams], p_ready[kStreams], o_done[kStreams], job_full[2], job_empty[2], drain;
    uint32_t odd[2][4];  // values of a step that are not finite
    Job job[2];          // of even and odd jobs of the CTA
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(Control) <= 1024, "control block");

// A role's way through the CTA's jobs.
struct Way {
    Control& c;
    volatile int* abort_flag;
    long long wait_cycles;
    uint32_t n = 0;  // jobs so far
    Job j{};
    int n0 = 0, n1 = 0, steps = 0, part = 0;  // steps of the streams, of both, and those that need no guard
    TQ_DEVFN Way(Control& c, volatile int* abort_flag, long long wait_cycles) : c(c), abort_flag(abort_flag), wait_cycles(wait_cycles) {}
    TQ_DEVFN void see(const PromptArgs& a) {
        n0 = steps_of(a, j, 0);
        n1 = steps_of(a, j, 1);
        steps = max(n0, n1);
        part = min(n0 ? whole_of(a, j, 0) : steps, n1 ? whole_of(a, j, 1) : steps);
    }
    // The next job: false where there is none (`ok` false: the CTA gives up).
    TQ_DEVFN bool next(const PromptArgs& a, bool& ok) {
        ok = mbar_wait(c.job_full + (n & 1), (n >> 1) & 1, abort_flag, wait_cycles);
        if (!ok) return false;
        j = c.job[n & 1];
        if (j.rows < 0) return false;
        see(a);
        return true;
    }
    TQ_DEVFN void done() {  // (one thread of the warp)
        mbar_arrive(c.job_empty + (n & 1));
    }
};

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
    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;

    pdl_trigger();
    if (warp == kMma) {
        if (lane == 0) {
            c.abort = 0;
            for (int i = 0; i < 2; ++i) {
                mbar_init(c.q_full + i, 1);
                mbar_init(c.q_empty + i, 1);
                mbar_init(c.k_full + i, 1);
                mbar_init(c.v_full + i, 1);
                mbar_init(c.k_empty + i, 1);
                mbar_init(c.v_empty + i, 3);  // the products and the guards
                mbar_init(c.guarded + i, 2);
                mbar_init(c.s_ready + i, 1);
                mbar_init(c.p_ready + i, 128);
                mbar_init(c.o_done + i, 1);
                mbar_init(c.job_full + i, 1);
                mbar_init(c.job_empty + i, kWarps - 1);  // every warp but the one that finds them
            }
            mbar_init(&c.drain, 1);
            fence_mbar_init();
        }
        __syncwarp();
        alloc512(&c.tmem);
    } else if (warp == kCopy && lane == 0) {
        prefetch_map(&map_q);
        prefetch_map(&map_k);
        prefetch_map(&map_v);
        prefetch_map(&map_r);
    }
    pdl_wait();
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = c.tmem;
    Way w(c, abort_flag, a.wait_cycles);
    uint32_t g = 0;  // steps of the CTA so far: the ring's places and the phases of its barriers

    if (warp == kCopy) {
        // ------------------------------------------------------------ jobs and tensor copies
        const Jobs jobs = count_jobs(a, blockIdx.x == 0);
        bool ok = true;
        uint32_t k_done = 0, v_done = 0, q_done[kStreams] = {0, 0};
        for (; ok; ++w.n) {
            uint32_t at = blockIdx.x;
            if (w.n) {
                if (!a.taken) at = ~0u;
                else if (lane == 0) at = gridDim.x + atomicAdd(a.taken, 1u);
                at = __shfl_sync(kFull, at, 0);
            }
            w.j = find_job(a, jobs, at);
            if (w.n >= 2) ok = __all_sync(kFull, mbar_wait(c.job_empty + (w.n & 1), ((w.n - 2) >> 1) & 1, abort_flag, a.wait_cycles));
            if (!ok) break;
            if (lane == 0) {
                c.job[w.n & 1] = w.j;
                mbar_arrive(c.job_full + (w.n & 1));
            }
            __syncwarp();
            if (w.j.rows < 0) break;
            w.see(a);
            const int row0 = w.j.k0, x = (int)(w.j.head * a.kvh);
            for (int i = 0; i < w.steps && ok; ++i, ++g) {
                const uint32_t e = g & 1;
                const int row = row0 + i * kTok;
                auto unit = [&](uint32_t u) { return base + kRing + ((g * kStep + u) % kUnits) * kUnit; };
                // its keys lie where the last keys and the values of two steps before did, its values where keys of the step before did
                if (g >= 2) ok = __all_sync(kFull, mbar_wait(c.v_empty + e, ((g - 2) >> 1) & 1, abort_flag, a.wait_cycles));
                if (!ok) break;
                if (elected()) {
                    mbar_expect_tx(c.k_full + e, kQUnits * kUnit);
                    tma_load_2d(unit(0), &map_k, x, row, c.k_full + e);
                    tma_load_2d(unit(1), &map_k, x + 64, row, c.k_full + e);
                    tma_load_2d(unit(2), &map_r, 0, row, c.k_full + e);
                }
                __syncwarp();
                ++k_done;
                if (i == 0)  // the job's queries, once the last products of the job before have read theirs
                    for (int t = 0; t < kStreams && ok; ++t) {
                        if (!(t ? w.n1 : w.n0)) continue;
                        if (q_done[t])
                            ok = __all_sync(kFull, mbar_wait(c.q_empty + t, (q_done[t] - 1) & 1, abort_flag, a.wait_cycles));
                        if (!ok) break;
                        if (elected()) {
                            mbar_expect_tx(c.q_full + t, kQUnits * kUnit);
                            for (int d = 0; d < kQUnits; ++d)
                                tma_load_2d(base + (t * kQUnits + d) * kUnit, &map_q, w.j.head * kHeadQuery + d * 64,
                                            w.j.q0 + t * kRows, c.q_full + t);
                        }
                        __syncwarp();
                        ++q_done[t];
                    }
                if (g >= 1 && ok) ok = __all_sync(kFull, mbar_wait(c.k_empty + (e ^ 1), ((g - 1) >> 1) & 1, abort_flag, a.wait_cycles));
                if (!ok) break;
                if (elected()) {
                    mbar_expect_tx(c.v_full + e, kVUnits * kUnit);
                    tma_load_2d(unit(3), &map_v, x, row, c.v_full + e);
                    tma_load_2d(unit(4), &map_v, x + 64, row, c.v_full + e);
                }
                __syncwarp();
                ++v_done;
            }
        }
        // no copy may be in flight when the CTA ends (on an abort: nobody else has waited for them)
        for (int t = 0; t < kStreams; ++t)
            if (q_done[t]) mbar_wait_drain(c.q_full + t, (q_done[t] - 1) & 1);
        for (uint32_t i = k_done < 2 ? 0 : k_done - 2; i < k_done; ++i) mbar_wait_drain(c.k_full + (i & 1), (i >> 1) & 1);
        for (uint32_t i = v_done < 2 ? 0 : v_done - 2; i < v_done; ++i) mbar_wait_drain(c.v_full + (i & 1), (i >> 1) & 1);
        clear_rest(a, jobs);
    } else if (warp == kMma) {
        // ------------------------------------------------------------ MMA issue
        if (elected()) {
            const uint64_t dq = desc(base, 16), dk = desc(base + kRing, 16), dv = desc(base + kRing, kUnit);
            uint32_t p_seen[kStreams] = {0, 0}, q_seen[kStreams] = {0, 0};  // steps and jobs of the streams so far
            bool ok = true;
            for (; w.next(a, ok); ++w.n) {
                // Scores of stream t and the job's step i.
                auto scores = [&](int t, int i) {
                    const uint32_t at = g + i;
                    if (!mbar_wait(c.k_full + (at & 1), (at >> 1) & 1, abort_flag, a.wait_cycles)) return false;
                    fence_after();
                    constexpr uint32_t id = idesc(BF, kRows, kTok, 0);
#pragma unroll
                    for (int d = 0; d < kQUnits; ++d) {
                        const uint64_t from = dk + (uint32_t)((at * kStep + d) % kUnits) * (kUnit / 16);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_ss(tmem + 256 * t, dq + (t * kQUnits + d) * (kUnit / 16) + 2 * k, from + 2 * k, id, (d | k) != 0);
                    }
                    commit(c.s_ready + t);
                    if (t == 1 || i >= w.n1) commit(c.k_empty + (at & 1));  // the last to read these keys
                    if (i + 1 == (t ? w.n1 : w.n0)) commit(c.q_empty + t);
                    return true;
                };
#pragma unroll
                for (int t = 0; t < kStreams; ++t)
                    if (ok && (t ? w.n1 : w.n0)) {
                        ok = mbar_wait(c.q_full + t, q_seen[t] & 1, abort_flag, a.wait_cycles) && scores(t, 0);
                        ++q_seen[t];
                    }
                for (int i = 0; i < w.steps && ok; ++i)
#pragma unroll
                    for (int t = 0; t < kStreams; ++t) {
                        if (!ok || i >= (t ? w.n1 : w.n0)) continue;
                        const uint32_t at = g + i;
                        ok = mbar_wait(c.v_full + (at & 1), (at >> 1) & 1, abort_flag, a.wait_cycles) &&
                             (i < w.part || mbar_wait(c.guarded + (at & 1), (at >> 1) & 1, abort_flag, a.wait_cycles)) &&
                             mbar_wait(c.p_ready + t, p_seen[t] & 1, abort_flag, a.wait_cycles);
                        if (!ok) break;
                        fence_after();
                        constexpr uint32_t id = idesc(BF, kRows, kHeadValue, 1), half = idesc(BF, kRows, 64, 1);
                        // (its two units may lie at the ring's end and start: then each is a product of its own)
                        const uint32_t u = (at * kStep + kQUnits) % kUnits;
                        const uint64_t from = dv + u * (kUnit / 16);
#pragma unroll
                        for (int k = 0; k < kTok / 16; ++k) {
                            if (u + 1 < kUnits) {
                                mma_ts(tmem + 256 * t + 128, tmem + 256 * t + 8 * k, from + 128 * k, id, (i | k) != 0);
                            } else {
                                mma_ts(tmem + 256 * t + 128, tmem + 256 * t + 8 * k, from + 128 * k, half, (i | k) != 0);
                                mma_ts(tmem + 256 * t + 192, tmem + 256 * t + 8 * k, dv + 128 * k, half, (i | k) != 0);
                            }
                        }
                        ++p_seen[t];
                        commit(c.o_done + t);
                        if (t == 1 || i >= w.n1) commit(c.v_empty + (at & 1));
                        if (i + 1 < (t ? w.n1 : w.n0)) ok = scores(t, i + 1);
                    }
                if (!ok) break;
                g += w.steps;
                w.done();
            }
            commit(&c.drain);  // completes when every MMA issued above has finished
            if (!mbar_wait_drain(&c.drain, 0)) *abort_flag = 1;
        }
        __syncwarp();
    } else if (warp >= kGuard) {
        // ------------------------------------------------------------ guards: a thread to two tokens
        const int id = tid - kGuard * 32;
        bool ok = true;
        for (; __all_sync(kFull, w.next(a, ok)); ++w.n) {
            for (int i = 0; i < w.steps && ok; ++i, ++g) {
                const uint32_t e = g & 1;
                ok = __all_sync(kFull, mbar_wait(c.v_full + e, (g >> 1) & 1, abort_flag, a.wait_cycles));
                if (!ok) break;
                if (i >= w.part) {
                    bool wrote = false;
                    for (int z = 0; z < 2; ++z) {
                        const int t = id + 64 * z;
                        uint8_t* rows[2];
                        for (int d = 0; d < 2; ++d) rows[d] = smem + kRing + ((g * kStep + kQUnits + d) % kUnits) * kUnit + t * 128;
                        bool odd = false;
                        const bool wipe = i * kTok + t >= w.j.keys;
                        constexpr uint32_t kTop = BF ? 0x7f807f80u : 0x7c007c00u;
                        for (int d = 0; d < 2 && !wipe; ++d)
#pragma unroll
                            for (int p = 0; p < 8; ++p) {
                                const uint4 v = *reinterpret_cast<const uint4*>(rows[d] + ((p + t) & 7) * 16);
                                odd |= (__vcmpeq2(v.x & kTop, kTop) | __vcmpeq2(v.y & kTop, kTop) | __vcmpeq2(v.z & kTop, kTop) |
                                        __vcmpeq2(v.w & kTop, kTop)) != 0;
                            }
                        __syncwarp();
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
            if (!ok) break;
            if (lane == 0) w.done();
        }
    } else {
        // ------------------------------------------------------------ softmax: a thread to a row
        const int t = warp >> 2, row = t * kRows + (warp & 3) * 32 + lane;
        const uint32_t at = tmem + 256 * t + ((uint32_t)(warp & 3) << 21), col_o = at + 128;
        const float f = fabsf(a.scale2);
        const f2 ff = pk(f, f);
        uint32_t done = 0;  // steps of this stream so far
        bool ok = true;
        for (; __all_sync(kFull, w.next(a, ok)); ++w.n) {
            const Job j = w.j;
            const int steps = t ? w.n1 : w.n0, whole = steps ? whole_of(a, j, t) : 0, part = w.part;
            const int seen = row < j.rows ? seen_by(a, j, row) : 0;
            const uint32_t g1 = g + w.steps;
            if (lane == 0) w.done();
            float m = -INFINITY, sum = 0.f, bias = 0.f;
            for (int i = 0; i < steps; ++i, ++g, ++done) {
                ok = __all_sync(kFull, mbar_wait(c.s_ready + t, done & 1, abort_flag, a.wait_cycles));
                if (!ok) break;
                fence_after();
                uint32_t s[128];
#pragma unroll
                for (int q = 0; q < 4; ++q) ld32(at + 32 * q, s + 32 * q);
                wait_ld();
                if (a.scale2 < 0)
#pragma unroll
                    for (int k = 0; k < 128; ++k) s[k] ^= 0x80000000u;
                bool spoilt = false;
                if (i >= whole) {
                    const int limit = seen - i * kTok;  // keys of this step that the row sees
#pragma unroll
                    for (int k = 0; k < 128; ++k)
                        if (k >= limit) s[k] = __float_as_uint(-INFINITY);
                }
                if (i >= part) {
                    ok = __all_sync(kFull, mbar_wait(c.guarded + (g & 1), (g >> 1) & 1, abort_flag, a.wait_cycles));
                    if (!ok) break;
                    const int limit = seen - i * kTok;
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const int bits = min(max(limit - 32 * z, 0), 32);
                        spoilt |= (c.odd[g & 1][z] & (bits == 32 ? ~0u : (1u << bits) - 1)) != 0;
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
                const float top = f * fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3]));
                if (__any_sync(kFull, top - m > Weights<BF>::kSlack)) {
                    // (each row by its own scores alone: its result must not hang on what its neighbours see)
                    const float to_m = top - m > Weights<BF>::kSlack ? top : m, to = Weights<BF>::bias(to_m);
                    const float r = m == -INFINITY ? 0.f : exp2_fast(to - bias);
                    m = to_m;
                    bias = to;
                    sum *= r;
                    if (i) {  // the sums so far (the scores were issued behind the products that wrote them)
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
                f2 by = ff;
                if (__any_sync(kFull, huge(m))) {
#pragma unroll
                    for (int k = 0; k < 128; ++k) s[k] = __float_as_uint(__fmul_rn(__uint_as_float(s[k]), f));
                    by = pk(1.f, 1.f);
                }
                f2 ls[2] = {0, 0};
#pragma unroll
                for (int k = 0; k < 64; ++k) {
                    const float2 y = un(fma2(pk(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), by, bb));
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
            if (!ok) break;
            if (steps) {
                ok = __all_sync(kFull, mbar_wait(c.o_done + t, (done - 1) & 1, abort_flag, a.wait_cycles));
                if (!ok) break;
                fence_after();
            }
            if (j.cut) {  // 16-byte pieces [8 warps][4 x 32 elements][8][32 lanes]: each store is one run of 512 bytes
                a.stat[(int64_t)blockIdx.x * kTile + row] = make_float2(level(m, bias), sum);
                float* const part_to = a.part + ((int64_t)blockIdx.x * kTile * (kHeadValue / 4) + warp * 1024 + lane) * 4;
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
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<uint4*>(part_to + (q * 8 + e) * 128) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
                fence_before();
                g = g1;
                continue;
            }
            const float over = sum == 0.f ? 0.f : 1.f / sum;  // (a NaN sum stays one)
            uint16_t* out = a.o + ((int64_t)(j.q0 + row) * a.H + j.head) * kHeadValue;
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
            fence_before();
            g = g1;
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

// The parts of jobs, joined in their order: a warp to 8 elements of 32 rows.
template <bool BF>
__global__ void __launch_bounds__(256) latent_prompt_join_kernel(const __grid_constant__ PromptArgs a) {
    __shared__ Jobs s_jobs;
    __shared__ Job s_job;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == 0) {
        Jobs jobs = count_jobs(a, false);
        const int parts = jobs.parts, per = jobs.per;
        jobs.parts = 1;  // (the whole job, not one of its parts)
        const Job j = find_job(a, jobs, blockIdx.x);
        jobs.parts = parts, jobs.per = per;
        if (lane == 0) s_jobs = jobs, s_job = j;
    }
    __syncthreads();
    const Jobs jobs = s_jobs;
    const Job j = s_job;
    if (jobs.parts <= 1 || j.rows < 0) return;
    constexpr int kAhead = 4;
    const int piece = blockIdx.y * 8 + warp, row = (piece >> 4) * 32 + lane, e = (piece & 15) * 2;  // pieces of 4 elements e, e + 1
    if (row >= j.rows) return;
    // parts that hold keys that some row of the job sees: the others' levels are -infinity
    const int64_t slot0 = (int64_t)blockIdx.x * jobs.parts;
    float o[8] = {}, top = -INFINITY, total = 0.f;
    for (int c = 0; c < jobs.parts; c += kAhead) {
        float2 stat[kAhead];
        float4 z[kAhead][2];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t slot = slot0 + min(c + k, jobs.parts - 1);
            stat[k] = a.stat[slot * kTile + row];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                z[k][h] = *reinterpret_cast<const float4*>(
                    a.part + (slot * kTile * (kHeadValue / 4) + (row >> 5) * 1024 + (((e + h) >> 3) * 8 + ((e + h) & 7)) * 32 + lane) * 4);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (c + k >= jobs.parts) break;
            // both to the higher level: weight 1 for its own (also where neither saw anything)
            const float n = fmaxf(top, stat[k].x), w0 = top == n ? 1.f : exp2_fast(top - n),
                        w1 = stat[k].x == n ? 1.f : exp2_fast(stat[k].x - n);
            top = n;
            total = total * w0 + stat[k].y * w1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                o[4 * h] = fmaf(o[4 * h], w0, z[k][h].x * w1);
                o[4 * h + 1] = fmaf(o[4 * h + 1], w0, z[k][h].y * w1);
                o[4 * h + 2] = fmaf(o[4 * h + 2], w0, z[k][h].z * w1);
                o[4 * h + 3] = fmaf(o[4 * h + 3], w0, z[k][h].w * w1);
            }
        }
    }
    const float over = total == 0.f ? 0.f : 1.f / total;  // (a NaN sum stays one)
    *reinterpret_cast<uint4*>(a.o + ((int64_t)(j.q0 + row) * a.H + j.head) * kHeadValue + e * 4) =
        make_uint4(pack16<BF>(o[0] * over, o[1] * over), pack16<BF>(o[2] * over, o[3] * over), pack16<BF>(o[4] * over, o[5] * over),
                   pack16<BF>(o[6] * over, o[7] * over));
}

}  // namespace
}  // namespace tq

using namespace tq;

namespace {
constexpr int kMaxSms = 256;
// Tiles over all heads, at most; and whether they may be cut: half the SMs would be idle, and a sequence can have 8 steps.
int64_t most_jobs(int32_t B, int32_t H, int64_t Tq) { return std::min((Tq + kTile - 1) / kTile + B, Tq) * H; }
bool may_cut(int64_t jobs, int64_t Tkv, int sms) { return jobs * 2 <= sms && Tkv >= 2 * kLeast * kTok; }
}  // namespace

extern "C" size_t tq_latent_attend_prompt_workspace_bytes(int32_t B, int32_t H, int64_t Tq, int64_t Tkv) {
    if (B <= 0 || H <= 0 || Tq <= 0 || Tkv < 0 || Tq > 1ll << 30) return sizeof(uint32_t);
    return may_cut(most_jobs(B, H, Tq), Tkv, kMaxSms) ? (size_t)kMaxSms * kTile * (kHeadValue * sizeof(float) + sizeof(float2)) : sizeof(uint32_t);
}

extern "C" tq_status tq_latent_attend_prompt(const void* q, int64_t q_stride, const void* k, const void* v, int64_t kv_stride,
                                             int64_t kv_head_stride, const void* k_rope, int64_t k_rope_stride, tq_dtype dt,
                                             int32_t B, int32_t H, int64_t Tq, int64_t Tkv, const int32_t* q_starts,
                                             const int32_t* kv_starts, int32_t causal, float scale, void* o, void* ws,
                                             size_t ws_bytes, uint32_t* err, void* stream) {
    if (B < 0 || H <= 0 || H > 65535 || Tq < 0 || Tkv < 0 || !isfinite(scale)) return TQ_ERR_INVALID;
    if (!(dt == TQ_BF16 || dt == TQ_F16 || dt == TQ_F32)) return TQ_ERR_INVALID;
    if (dt == TQ_F32 || Tq > 1ll << 30 || Tkv > 1ll << 30) return TQ_ERR_UNSUPPORTED;
    if (q_stride < (int64_t)H * kHeadQuery || kv_head_stride < kHeadKey || kv_stride < (H - 1) * kv_head_stride + kHeadKey ||
        k_rope_stride < kLatentRope || q_stride % 8 || kv_stride % 8 || kv_head_stride % 8 || k_rope_stride % 8)
        return TQ_ERR_INVALID;
    // (a tensor copy's column is an int)
    if (q_stride > 1ll << 32 || kv_stride > 1ll << 32 || k_rope_stride > 1ll << 32 || (H - 1) * kv_head_stride + kHeadKey > 0x7fffffffll)
        return TQ_ERR_UNSUPPORTED;
    if (B == 0 || Tq == 0) return TQ_OK;
    if (!q || !o || !ws || ws_bytes < tq_latent_attend_prompt_workspace_bytes(B, H, Tq, Tkv) || !q_starts || !kv_starts || (Tkv && (!k || !v || !k_rope))) return TQ_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_rope, 16) || !aligned(o, 32) || !aligned(ws, 32) || !aligned(q_starts, 4) ||
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
    a.scale2 = score_factor(scale);
    a.wait_cycles = wait_budget();
    const bool bf = dt == TQ_BF16;
    CUtensorMap mq, mk, mv, mr;
    const int64_t cols = (H - 1) * kv_head_stride + kHeadKey, keys = std::max<int64_t>(Tkv, 1);
    // (without keys no copy is made: any address serves)
    if (!tensor_map(&mq, bf, q, Tq, (int64_t)H * kHeadQuery, q_stride, kRows) ||
        !tensor_map(&mk, bf, Tkv ? k : q, keys, cols, kv_stride, kTok) || !tensor_map(&mv, bf, Tkv ? v : q, keys, cols, kv_stride, kTok) ||
        !tensor_map(&mr, bf, Tkv ? k_rope : q, keys, kLatentRope, k_rope_stride, kTok))
        return TQ_ERR_CUDA;
    // heads of a group: as many as the L2 cache (129 MB) holds the keys and values of twice over (8192 tokens: 915 us with 16 to 96 MB, 958
    // ungrouped; seven chunks 99 us with 64 MB, 108 with 16)
    a.heads = (int)std::min<int64_t>(H, std::max<int64_t>(1, (64ll << 20) / (keys * (kHeadKey + kHeadValue) * 2)));
    const int64_t jobs = most_jobs(B, H, Tq);
    if (jobs > 1ll << 30) return TQ_ERR_UNSUPPORTED;
    void (*kernel)(PromptArgs, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap) =
        bf ? latent_prompt_kernel<true> : latent_prompt_kernel<false>;
    if (ensure_smem((const void*)kernel, kSmem) != cudaSuccess) return TQ_ERR_CUDA;
    if (jobs > std::min(device_sms(), kMaxSms)) {
        a.taken = reinterpret_cast<uint32_t*>(ws);
        if (cudaMemsetAsync(ws, 0, sizeof(uint32_t), as_stream(stream)) != cudaSuccess) return TQ_ERR_CUDA;
    }
    const int sms = std::min(device_sms(), kMaxSms);
    const bool cut = may_cut(jobs, Tkv, sms);
    a.ctas = (int)(cut ? sms : std::min<int64_t>(jobs, sms));
    if (cut) {
        a.part = reinterpret_cast<float*>(ws);
        a.stat = reinterpret_cast<float2*>(a.part + (int64_t)sms * kTile * kHeadValue);
    }
    const tq_status s = launch_pdl(kernel, dim3((unsigned)a.ctas), dim3(32 * kWarps), kSmem, as_stream(stream), a, mq, mk, mv, mr);
    if (s != TQ_OK || !cut) return s;
    return launch_pdl(bf ? latent_prompt_join_kernel<true> : latent_prompt_join_kernel<false>, dim3((unsigned)jobs, 16), dim3(256), 0,
                      as_stream(stream), a);
}
