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
    int ctas, trows, stoks, least;      // context launch: CTAs, query rows of a tile, tokens of a step, fewest steps of a run
    float scale2;                       // scale * log2(e)
    __nv_bfloat16* o;
    float2* stat;  // [slot][trows]: running maximum (log2 units) and sum of a row
    float* part;   // [slot][trows][128]: weighted values, rotated
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

struct Work {
    long long steps;  // steps of the sequences before this one
    int units;        // (kv head, tile) units of the sequences before this one
};

// Steps and units of the sequences before b, and of all (one warp).
TQ_DEVFN void count_work(const TreeArgs& a, int b, Work& before, long long& total) {
    const int lane = threadIdx.x & 31;
    long long s = 0, all = 0;
    int u = 0;
    for (int i = lane; i < a.B; i += 32) {
        const int units = seq_tiles(a, i) * a.c.Hkv;
        const long long w = (long long)units * seq_steps(a, i);
        all += w;
        if (i < b) {
            s += w;
            u += units;
        }
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        s += __shfl_xor_sync(kFull, s, m);
        all += __shfl_xor_sync(kFull, all, m);
        u += __shfl_xor_sync(kFull, u, m);
    }
    before = {s, u};
    total = all;
}

// Steps of one CTA's run: an equal share, and no fewer than `least`.
TQ_DEVFN long long steps_per_cta(const TreeArgs& a, long long total) {
    return max((total + a.ctas - 1) / a.ctas, (long long)a.least);
}

// Where the run that begins at step P0 starts: the last sequence with at most P0 steps before it (one warp).
TQ_DEVFN void find_run(const TreeArgs& a, long long P0, Work& before, int& b) {
    const int lane = threadIdx.x & 31;
    before = {0, 0};
    b = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int i = b0 + lane;
        const int u = i < a.B ? seq_tiles(a, i) * a.c.Hkv : 0;
        const long long s = i < a.B ? (long long)u * seq_steps(a, i) : 0;
        long long incl = s;
        int ui = u;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long x = __shfl_up_sync(kFull, incl, m);
            const int y = __shfl_up_sync(kFull, ui, m);
            if (lane >= m) {
                incl += x;
                ui += y;
            }
        }
        const unsigned hit = __ballot_sync(kFull, before.steps + incl > P0);
        if (hit) {
            const int src = __ffs(hit) - 1;
            before.steps += __shfl_sync(kFull, incl - s, src);
            before.units += __shfl_sync(kFull, ui - u, src);
            b = b0 + src;
            return;
        }
        before.steps += __shfl_sync(kFull, incl, 31);
        before.units += __shfl_sync(kFull, ui, 31);
    }
}

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
TQ_DEVFN float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
TQ_DEVFN void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
TQ_DEVFN uint32_t lds32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
TQ_DEVFN uint32_t lds16(uint32_t at) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
    return v;
}
TQ_DEVFN uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}
TQ_DEVFN uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
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

}  // namespace tree
}  // namespace tq
