// Attention of drafted trees over the paged cache: what its kernels share (arguments, the count of the work, fragments
// of decoded codes).
#pragma once

#include "common.cuh"
#include "kv_pages.cuh"
#include "tma.cuh"

namespace tq {
namespace tree {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInvSqrtD = 0.08838834764831845f;  // 1 / sqrt(128)
constexpr float kSlack = 8.0f;                      // a running maximum may be this far (log2) below the true one
// A row's weights are 2^(score + bias), bias = kLift - maximum: at most 2^15, inside fp16, and the smallest that fp16 holds is
// 2^-31 of the maximum's (without the lift 2^-24: 131072 tokens a little below that are 0.4 % of a sum).  Rounded down, so that it
// is never more than the lift, however large the maximum.  Sums belong to the bias: what is kept and joined is its negative.
constexpr float kLift = 7.0f;
static_assert(kSlack + kLift <= 15.0f, "weights fit fp16");
TQ_DEVFN float weight_bias(float m) { return m == -INFINITY ? 0.f : __fadd_rd(kLift, -m); }
TQ_DEVFN float level(float m, float bias) { return m == -INFINITY ? m : -bias; }  // that sums belong to: -infinity where there are none

struct TreeArgs {
    KvPages c;
    const __nv_bfloat16* q;
    const __nv_bfloat16* kn;
    const __nv_bfloat16* vn;
    int64_t qs, ks, vs, max_len;
    const int32_t* table;
    const int32_t* lens;
    const uint64_t* mask;
    const int32_t* n_tok;
    int B, n, Hq, ratio, table_stride;  // ratio: query heads per kv head
    // context launch: CTAs, query rows of a tile, tokens of a step, fewest steps of a run, steps that beginning a tile weighs
    int ctas, trows, stoks, least, pad;
    float scale2;                       // scale * log2(e)
    float qmant;                        // scale2 / sqrt(128) as qmant 2^qexp, 1 <= |qmant| <= 2 (or 0)
    int qexp;
    __nv_bfloat16* o;
    float2* stat;  // [slot][trows]: level (log2 units) and sum of a row
    float* part;   // [slot][trows][128]: weighted values, rotated
    uint4* turned;   // more than 16 rows: rotated queries [unit][16 pieces][trows] and their exponents
    int32_t* power;  // [unit][trows]
    uint32_t* err;
    long long wait_cycles;  // budget of each bounded wait
};

tq_status launch_wide(int klevels, int vlevels, const TreeArgs& a, cudaStream_t st);

// ---------------------------------------------------------------- the batch's work, counted on the device

TQ_DEVFN int seq_len(const TreeArgs& a, int b) {
    const int len = a.lens[b];
    return len < 0 ? 0 : (int)min((int64_t)len, a.max_len);
}
TQ_DEVFN int seq_live(const TreeArgs& a, int b) { return a.n_tok ? min(max(a.n_tok[b], 0), a.n) : a.n; }
TQ_DEVFN int seq_tiles(const TreeArgs& a, int b) { return (seq_live(a, b) * a.ratio + a.trows - 1) / a.trows; }
TQ_DEVFN int seq_steps(const TreeArgs& a, int b) { return (seq_len(a, b) + a.stoks - 1) / a.stoks; }

// A run is a stretch of an axis on which every tile of a sequence that has steps takes `pad` places, then one for each step: so
// that a run which begins another tile on its way has fewer steps to do.  Where runs are short (there are few steps for the
// CTAs), the pad is at most a quarter of a run's steps.  Counts fit 31 bits: the host checks their bound.
TQ_DEVFN int tile_pad(const TreeArgs& a, int steps) { return min(a.pad, steps / (4 * a.ctas)); }

// Places of one CTA's run: an equal share, and no fewer than `least`.
TQ_DEVFN int places_per_cta(const TreeArgs& a, int total) { return max((total + a.ctas - 1) / a.ctas, a.least); }

// Over the batch, and over the sequences before b (one warp): steps, units ((kv head, tile) pairs), and units that have steps.
struct Count {
    int steps, units, busy;
};
TQ_DEVFN void count_work(const TreeArgs& a, int b, Count& before, Count& all) {
    const int lane = threadIdx.x & 31;
    Count p{}, q{};
    for (int i = lane; i < a.B; i += 32) {
        const int units = seq_tiles(a, i) * a.c.Hkv, steps = seq_steps(a, i);
        q.steps += units * steps;
        q.units += units;
        q.busy += steps ? units : 0;
        if (i < b) {
            p.steps += units * steps;
            p.units += units;
            p.busy += steps ? units : 0;
        }
    }
    before = {__reduce_add_sync(kFull, p.steps), __reduce_add_sync(kFull, p.units), __reduce_add_sync(kFull, p.busy)};
    all = {__reduce_add_sync(kFull, q.steps), __reduce_add_sync(kFull, q.units), __reduce_add_sync(kFull, q.busy)};
}

// The run of CTA `run`: its first place `at`, places of a run and of all, the pad, and the last sequence b with at most `at`
// places before it, with the places and units before b (one warp).
struct Run {
    int at, per, total, pad, b, places, units;
};
TQ_DEVFN Run find_run(const TreeArgs& a, int run) {
    const int lane = threadIdx.x & 31;
    Run r{};
    int units = 0, steps = 0;  // of sequence b0 + lane
    auto read = [&](int b0) {
        const int i = b0 + lane;
        units = i < a.B ? seq_tiles(a, i) * a.c.Hkv : 0;
        steps = i < a.B ? seq_steps(a, i) : 0;
    };
    int all = 0, busy = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        read(b0);
        all += __reduce_add_sync(kFull, units * steps);
        busy += __reduce_add_sync(kFull, steps ? units : 0);
    }
    r.pad = tile_pad(a, all);
    r.total = all + busy * r.pad;
    r.per = places_per_cta(a, r.total);
    r.at = run * r.per;  // at most the total and a run more
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        if (a.B > 32) read(b0);
        const int own = steps ? units * (steps + r.pad) : 0;
        int s = own, u = units;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int x = __shfl_up_sync(kFull, s, m), y = __shfl_up_sync(kFull, u, m);
            if (lane >= m) {
                s += x;
                u += y;
            }
        }
        const unsigned hit = __ballot_sync(kFull, r.places + s > r.at);
        if (hit) {
            const int src = __ffs(hit) - 1;
            r.places += __shfl_sync(kFull, s - own, src);
            r.units += __shfl_sync(kFull, u - units, src);
            r.b = b0 + src;
            break;
        }
        r.places += __shfl_sync(kFull, s, 31);
        r.units += __shfl_sync(kFull, u, 31);
    }
    return r;
}

// A stretch of a run within one (sequence, kv head, tile): steps s0 .. s1 - 1 of it.
struct Stretch {
    int b, h, tile, unit, s0, s1, len, rows;  // unit: numbered over the batch; rows in use
};
struct Walk {
    int p, end, pad, b, places, units;  // places and units before sequence b
    TQ_DEVFN explicit Walk(const Run& r)
        : p(r.at), end(min(r.at + r.per, r.total)), pad(r.pad), b(r.b), places(r.places), units(r.units) {}
    TQ_DEVFN bool next(const TreeArgs& a, Stretch& x) {
        while (p < end) {
            int steps = seq_steps(a, b), tiles = seq_tiles(a, b), own = steps ? steps + pad : 0;
            while (p >= places + own * tiles * a.c.Hkv) {  // into the next sequence that has any
                places += own * tiles * a.c.Hkv;
                units += tiles * a.c.Hkv;
                ++b;
                steps = seq_steps(a, b);
                tiles = seq_tiles(a, b);
                own = steps ? steps + pad : 0;
            }
            const int unit = (p - places) / own, at = p - places - unit * own;
            const int to = min(own, at + (end - p));
            p += to - at;
            if (to <= pad) continue;  // no step of this tile
            x.b = b;
            x.h = unit / tiles;
            x.tile = unit - x.h * tiles;
            x.unit = units + unit;
            x.s0 = max(at - pad, 0);
            x.s1 = to - pad;
            x.len = seq_len(a, b);
            x.rows = min(a.trows, seq_live(a, b) * a.ratio - x.tile * a.trows);
            return true;
        }
        return false;
    }
};

// ---------------------------------------------------------------- fragments

TQ_DEVFN uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(s));
    return d;
}
TQ_DEVFN uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// D[16, 8] += A[16, 16] B[16, 8], fp32 sums.
TQ_DEVFN void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
TQ_DEVFN void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
TQ_DEVFN uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
using f2 = unsigned long long;  // two packed fp32
TQ_DEVFN f2 pk(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
TQ_DEVFN float2 un(f2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
TQ_DEVFN f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
TQ_DEVFN f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
TQ_DEVFN float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The decode table at shared address TABLE: row c of 256 bytes holds, a copy for each lane (bank = lane), the fp16 centroid
// of 8-bit key code c, or the centroids of the two 4-bit key codes of byte c, and in its upper half the pair of two 4-bit
// value codes, all over powers of two (kd, vd).  Written by all of the CTA's warps.
template <int KL, int VL>
TQ_DEVFN void build_table(const KvPages& c, uint8_t* table, float kd, float vd, int warp, int warps) {
    const int lane = threadIdx.x & 31;
    const float k16 = KL == 16 ? c.kcent[lane & 15] * kd : 0.f, v16 = VL == 16 ? c.vcent[lane & 15] * vd : 0.f;
    const int per = (256 + warps - 1) / warps, first = warp * per;  // rows of this warp: at most 32
    const float own = KL == 256 && first + lane < 256 ? c.kcent[first + lane] * kd : 0.f;
    for (int i = 0; i < per && first + i < 256; ++i) {
        const int row = first + i;
        uint32_t* to = reinterpret_cast<uint32_t*>(table + row * 256) + lane;
        to[0] = KL == 256 ? pack_f16(__shfl_sync(kFull, own, i), 0.f)
                          : pack_f16(__shfl_sync(kFull, k16, row & 15), __shfl_sync(kFull, k16, row >> 4));
        if (VL == 16) to[32] = pack_f16(__shfl_sync(kFull, v16, row & 15), __shfl_sync(kFull, v16, row >> 4));
    }
}
TQ_DEVFN void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Shared memory at a 32-bit address and an offset known to the compiler.
template <int OFF = 0>
TQ_DEVFN uint32_t lds32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1+%2];" : "=r"(v) : "r"(at), "n"(OFF));
    return v;
}
template <int OFF = 0>
TQ_DEVFN uint32_t lds16(uint32_t at) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1+%2];" : "=h"(v) : "r"(at), "n"(OFF));
    return v;
}
template <int OFF = 0>
TQ_DEVFN uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2+%3];" : "=r"(v.x), "=r"(v.y) : "r"(at), "n"(OFF));
    return v;
}
template <int OFF = 0>
TQ_DEVFN uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4+%5];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at), "n"(OFF));
    return v;
}
// The lane's entry of a table of 256-byte rows: the row is byte `c` of w (asm without volatile: the table
// does not change after it is built, so the compiler may order these reads as it likes).
template <int C>
TQ_DEVFN uint32_t table(uint32_t w, uint32_t lane_base) {
    uint32_t v;
    asm("{\n .reg .b32 a;\n prmt.b32 a, %1, %2, %3;\n ld.shared.u32 %0, [a];\n}\n"
        : "=r"(v)
        : "r"(w), "r"(lane_base), "n"(0x6504 | (C << 4)));
    return v;
}
// 2^-e just above x's magnitude, as an exponent: 0 for 0, infinities and NaN.
TQ_DEVFN int exponent_above(float x) {
    const int e = (__float_as_int(x) >> 23) & 255;
    return e == 0 || e == 255 ? 0 : e - 126;
}

// The scale's mantissa goes into the rotated queries, with their own power of two: what a row's element is multiplied by.
TQ_DEVFN float query_factor(int e, float qmant) { return exp2f((float)-e) * qmant; }
// From a row's products, of operands over 2^e together, to log2 scores: a power of two, so that a product times it is exact, and
// the highest score less itself is 0 however large it is.  Never 0, so that a masked score, -infinity times it, is no NaN; products
// are below 2^24, so a score that the bound changes stays below 2^-98.
TQ_DEVFN float score_factor(int e, int qexp) { return exp2f((float)min(max(e + qexp, -122), 127)); }

}  // namespace tree
}  // namespace tq
