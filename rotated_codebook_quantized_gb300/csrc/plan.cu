// Pages of a step on the device: what each sequence gives back and takes, and the slots and positions of its new tokens.
//
// One CTA moves the pages: prefix sums over the sequences (pages given, pages taken, tokens) fix every place on the stack, in the
// tables and among the packed tokens, so nothing depends on the order of threads.  Slots and positions come from a second launch
// over the whole GPU (from the same CTA: 11.1 us for 64 sequences planned and undone, 8.7 with it; 38 and 12 for 1000 of 16 tokens).
// Bound by latency: a chain of dependent loads (lengths, pages held, the stack, the tables), 4.5 us a call.  A sequence's padded row is
// one warp's: 65536 tokens of one sequence planned and undone 223 us, packed (a search of each token's sequence) 11 us.
#include <algorithm>

#include "common.cuh"

namespace tq {
namespace {

constexpr int kThreads = 1024;

struct PlanArgs {
    int32_t* table;
    int32_t* held;
    int32_t* free;
    int32_t* n_free;
    const int32_t* lens;
    const int32_t* n_new;
    const int32_t* path;
    int32_t* slots;
    int32_t* positions;
    int32_t* new_lens;
    int32_t* starts;
    uint32_t* err;
    int64_t pages, tokens;
    int batch, width, lpage, n;
};

// What a sequence asks for: pages given and taken, its tokens in the packed order.
struct Ask {
    int len, fresh, give, take;
    int64_t room;  // places among the packed tokens
    bool bad;
};
TQ_DEVFN Ask ask(const PlanArgs& a, int b) {
    Ask k{};
    if (b >= a.batch) return k;
    k.len = a.lens[b];
    k.fresh = a.n_new[b];
    const int held = a.held[b];
    const int64_t total = (int64_t)k.len + k.fresh;
    const int64_t need = (total + (1 << a.lpage) - 1) >> a.lpage;
    const int64_t rows = a.n ? a.n : a.tokens;
    k.room = k.fresh >= 0 && k.fresh <= rows ? k.fresh : 0;
    k.bad = k.len < 0 || k.fresh < 0 || k.fresh > rows || held < 0 || held > a.width || need > a.width;
    if (!k.bad) {
        k.give = max(held - (int)need, 0);
        k.take = max((int)need - held, 0);
    }
    return k;
}

// Inclusive prefix sum over the CTA's threads; `all` the total.  part: an entry of shared memory a warp.
TQ_DEVFN int64_t scan(int64_t x, int64_t* part, int64_t& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    auto prefix = [&](int64_t v) {
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t y = __shfl_up_sync(kFull, v, m);
            if (lane >= m) v += y;
        }
        return v;
    };
    x = prefix(x);
    if (lane == 31) part[warp] = x;
    __syncthreads();
    const int64_t upto = prefix(lane < warps ? part[lane] : 0);
    all = __shfl_sync(kFull, upto, 31);
    const int64_t before = __shfl_sync(kFull, upto, warp ? warp - 1 : 0);
    __syncthreads();
    return x + (warp ? before : 0);
}

// Last entry of the ascending at[0 .. n) that is not above x (at[0] <= x).
template <class T>
TQ_DEVFN int last_upto(const T* at, int n, int64_t x) {
    int lo = 0;
    for (int hi = n; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)at[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Slot of token `pos` of sequence b.
TQ_DEVFN int slot_of(const PlanArgs& a, int b, int64_t pos, bool& bad) {
    const int id = a.table[(int64_t)b * a.width + (pos >> a.lpage)];
    if ((uint32_t)id >= (uint64_t)a.pages) {
        bad = true;
        return -1;
    }
    return (id << a.lpage) + (int)(pos & ((1 << a.lpage) - 1));
}

// Slots and positions, by all threads of `warps` warps of which this is number `warp`.
TQ_DEVFN void write_slots(const PlanArgs& a, int64_t warp, int64_t warps) {
    const int lane = threadIdx.x & 31;
    bool bad = false;
    if (a.n) {
        for (int64_t b = warp; b < a.batch; b += warps) {
            const int len = a.lens[b], fresh = a.n_new[b];
            const int live = a.new_lens[b] == len ? 0 : fresh;  // (refused, or nothing new)
            int32_t* s = a.slots + b * a.n;
            int32_t* z = a.positions + b * a.n;
            for (int i = lane; i < a.n; i += 32) {
                const bool own = !a.path && i < live;
                s[i] = own ? slot_of(a, (int)b, (int64_t)len + i, bad) : -1;
                z[i] = own ? len + i : 0;
            }
            if (a.path) {
                __syncwarp();
                for (int i = lane; i < live; i += 32) {
                    const int to = a.path[b * a.n + i];
                    if ((uint32_t)to >= (uint32_t)a.n) {
                        bad = true;
                        continue;
                    }
                    s[to] = slot_of(a, (int)b, (int64_t)len + i, bad);
                    z[to] = len + i;
                }
            }
        }
    } else {
        const int64_t total = a.starts[a.batch];
        for (int64_t t = warp * 32 + lane; t < a.tokens; t += warps * 32) {
            int slot = -1, pos = 0;
            if (t < total) {
                const int b = last_upto(a.starts, a.batch + 1, t), len = a.lens[b];
                if (a.new_lens[b] != len) {
                    pos = len + (int)(t - a.starts[b]);
                    slot = slot_of(a, b, pos, bad);
                }
            }
            a.slots[t] = slot;
            a.positions[t] = pos;
        }
    }
    if (bad && a.err) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
}

// One round for each blockDim.x sequences; what a round finds is found again by the next pass over them.
__global__ void __launch_bounds__(kThreads) kv_plan_kernel(PlanArgs a) {
    __shared__ int64_t part[32];
    __shared__ int64_t before_me[kThreads];    // pages given, or asked for, by the round's sequences before each
    __shared__ int first[kThreads];            // the first of them: its place in the table; -1: a refused sequence
    __shared__ unsigned long long taken_most;  // pages asked for up to the last sequence that is served
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, step = blockDim.x;
    uint32_t wrong = 0;
    if (tid == 0) taken_most = 0;
    int64_t before = a.n_free[0];
    if (before < 0 || before > a.pages) {
        wrong |= TQ_DEVERR_BAD_PAGE;
        before = before < 0 ? 0 : a.pages;
    }
    // What sequence b asks for, and the first of its packed tokens; `room`: of the rounds before, and brought up to date.
    auto look = [&](int b, int64_t& start, int64_t& room) {
        Ask k = ask(a, b);
        start = 0;
        if (!a.n) {  // tokens that pass the end are no one's
            int64_t all;
            start = room + scan(k.room, part, all) - k.room;
            room += all;
            if (start + k.room > a.tokens) k.bad = true, k.give = k.take = 0;
        }
        return k;
    };
    // ---- what all of them give back
    int64_t given = 0, room = 0, start;
    for (int b0 = 0; b0 < a.batch; b0 += step) {
        int64_t all;
        scan(look(b0 + tid, start, room).give, part, all);
        given += all;
    }
    const int64_t top = before + given;
    if (top > a.pages) wrong |= TQ_DEVERR_BAD_PAGE;
    if (given) {
        int64_t done = 0;
        room = 0;
        for (int b0 = 0; b0 < a.batch; b0 += step) {
            int64_t all;
            const Ask k = look(b0 + tid, start, room);
            before_me[tid] = scan(k.give, part, all) - k.give;
            first[tid] = k.give ? a.held[b0 + tid] - k.give : 0;
            __syncthreads();
            const int n = min(step, a.batch - b0);
            for (int64_t j = tid; j < all; j += step) {
                const int i = last_upto(before_me, n, j);
                int32_t* e = a.table + (int64_t)(b0 + i) * a.width + first[i] + (j - before_me[i]);
                const int64_t to = top - 1 - (done + j);
                if (to < a.pages) a.free[to] = *e;
                *e = -1;
            }
            done += all;
            __syncthreads();
        }
    }
    // ---- what they take, and the new lengths
    const int64_t stack = min(top, a.pages);
    int64_t asked = 0;
    room = 0;
    for (int b0 = 0; b0 < a.batch; b0 += step) {
        int64_t all;
        const int b = b0 + tid;
        const Ask k = look(b, start, room);
        const int64_t upto = scan(k.take, part, all);
        const bool fits = k.take == 0 || asked + upto <= stack, served = !k.bad && fits;
        before_me[tid] = upto - k.take;
        if (b < a.batch) {
            const int held = a.held[b];
            first[tid] = served ? held : -1;
            if (served) a.held[b] = held + k.take - k.give;
            if (served && k.take) atomicMax(&taken_most, (unsigned long long)(asked + upto));
            a.new_lens[b] = served ? k.len + k.fresh : k.len;
            if (a.starts) a.starts[b] = (int)min(start, a.tokens);
            if (!served) wrong |= k.bad ? TQ_DEVERR_BAD_PAGE : TQ_DEVERR_NO_PAGE;
        }
        __syncthreads();
        const int n = min(step, a.batch - b0);
        for (int64_t j = tid; j < all; j += step) {
            const int i = last_upto(before_me, n, j);
            if (first[i] < 0) continue;
            const int id = a.free[stack - 1 - (asked + j)];
            if ((uint32_t)id >= (uint64_t)a.pages) wrong |= TQ_DEVERR_BAD_PAGE;
            a.table[(int64_t)(b0 + i) * a.width + first[i] + (j - before_me[i])] = id;
        }
        asked += all;
        __syncthreads();
    }
    if (tid == 0) {
        a.n_free[0] = (int)(stack - (int64_t)taken_most);
        if (a.starts) a.starts[a.batch] = (int)min(room, a.tokens);
    }
    if (wrong && a.err) atomicOr(a.err, wrong);
}

__global__ void __launch_bounds__(256) kv_plan_slots_kernel(PlanArgs a) {
    pdl_trigger();
    pdl_wait();
    write_slots(a, (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), (int64_t)gridDim.x * 8);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" tq_status tq_kv_plan(const tq_page_pool_t* pool, const int32_t* lens, const int32_t* n_new, const int32_t* path,
                                int32_t n, int64_t tokens, int32_t* slots, int32_t* positions, int32_t* new_lens,
                                int32_t* starts, uint32_t* err, void* stream) {
    if (!pool || pool->batch < 0 || pool->width < 0 || pool->pages < 0 || n < 0 || tokens < 0) return TQ_ERR_INVALID;
    if (!is_pow2(pool->page) || pool->page < 16 || pool->page > 256) return TQ_ERR_INVALID;
    if (pool->pages > 0x7fffffffll / pool->page || pool->batch > (1 << 20)) return TQ_ERR_UNSUPPORTED;
    if (n ? starts != nullptr : path != nullptr) return TQ_ERR_INVALID;
    const int64_t rows = n ? (int64_t)pool->batch * n : tokens;
    if (rows > 1ll << 30) return TQ_ERR_UNSUPPORTED;
    if (pool->batch == 0 && (n || tokens == 0)) return TQ_OK;
    if (!pool->n_free || (pool->pages && !pool->free)) return TQ_ERR_INVALID;
    if (pool->batch && (!pool->held || (pool->width && !pool->table) || !lens || !n_new || !new_lens)) return TQ_ERR_INVALID;
    if (!n && !starts) return TQ_ERR_INVALID;
    if (rows && (!slots || !positions)) return TQ_ERR_INVALID;
    for (const void* p : {(const void*)pool->table, (const void*)pool->held, (const void*)pool->free, (const void*)pool->n_free,
                          (const void*)lens, (const void*)n_new, (const void*)path, (const void*)slots, (const void*)positions,
                          (const void*)new_lens, (const void*)starts})
        if (!aligned(p, 4)) return TQ_ERR_INVALID;
    PlanArgs a{};
    a.table = pool->table;
    a.held = pool->held;
    a.free = pool->free;
    a.n_free = pool->n_free;
    a.lens = lens;
    a.n_new = n_new;
    a.path = path;
    a.slots = slots;
    a.positions = positions;
    a.new_lens = new_lens;
    a.starts = starts;
    a.err = err;
    a.pages = pool->pages;
    a.tokens = tokens;
    a.batch = pool->batch;
    a.width = pool->width;
    a.lpage = ilog2(pool->page);
    a.n = n;
    const int threads = a.batch <= 256 ? 256 : kThreads;  // (64 sequences planned and undone: 9.1 us; by 1024 threads 11.1)
    const tq_status s = launch_pdl(kv_plan_kernel, dim3(1), dim3(threads), 0, as_stream(stream), a);
    if (s != TQ_OK || rows == 0) return s;
    const int64_t warps = n ? pool->batch : (tokens + 31) / 32;
    return launch_pdl(kv_plan_slots_kernel, dim3((unsigned)std::min<int64_t>((warps + 7) / 8, device_sms() * 8)), dim3(256), 0,
                      as_stream(stream), a);
}
