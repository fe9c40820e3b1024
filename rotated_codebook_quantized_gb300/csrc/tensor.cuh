// tcgen05 (5th-generation tensor core) helpers of the latent attention kernels: descriptors, products, TMEM loads and stores.
#pragma once

#include <math.h>

#include "common.cuh"
#include "tma.cuh"

namespace tq {
namespace tc {

TQ_DEVFN void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
TQ_DEVFN void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
TQ_DEVFN void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
TQ_DEVFN void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
TQ_DEVFN void commit(uint64_t* b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(b)) : "memory");
}
// All 512 columns (one CTA to an SM), by one warp; the address comes through `slot` in shared memory.
TQ_DEVFN void alloc512(uint32_t* slot) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
TQ_DEVFN void dealloc512(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}
// One lane of the converged warp; the compiler knows that a single thread passes.
TQ_DEVFN bool elected() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// Shared tiles of 128-byte rows, 128-byte swizzled, in atoms of 8 rows (1024 bytes), consecutive atoms 1024 bytes apart.
// K-major (64 elements of K to a row): `leading` is not used.  MN-major (64 elements of M or N to a row, rows along K): the next 64
// elements of M or N lie `leading` bytes on.
TQ_DEVFN uint64_t desc(uint32_t addr, uint32_t leading) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(leading >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16: fp32 sums, A and B of one type (bf16 or fp16), B MN-major where mn is set.
constexpr __host__ __device__ uint32_t idesc(bool bf, int m, int n, int mn) {
    return (1u << 4) | ((bf ? 1u : 0u) << 7) | ((bf ? 1u : 0u) << 10) | ((uint32_t)mn << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}
// D (TMEM) (+)= A (shared) . B (shared).
TQ_DEVFN void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accum) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accum)
        : "memory");
}
// D (TMEM) (+)= A (TMEM) . B (shared).
TQ_DEVFN void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accum) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(accum)
        : "memory");
}

#define TQ_O8(i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), \
                 "=r"(v[i + 6]), "=r"(v[i + 7])
#define TQ_I8(i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), \
                 "r"(v[i + 7])
#define TQ_L32 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, " \
               "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31}"
// 32 columns of the warp's 32 TMEM lanes, a lane to a thread.  Loads are complete after wait_ld.
TQ_DEVFN void ld32(uint32_t at, uint32_t* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " TQ_L32 ", [%32];"
                 : TQ_O8(0), TQ_O8(8), TQ_O8(16), TQ_O8(24)
                 : "r"(at)
                 : "memory");
}
TQ_DEVFN void st32(uint32_t at, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " TQ_L32 ";" ::TQ_I8(0), TQ_I8(8), TQ_I8(16), TQ_I8(24), "r"(at)
        : "memory");
}
TQ_DEVFN void ld8(uint32_t at, uint32_t* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : TQ_O8(0) : "r"(at) : "memory");
}
TQ_DEVFN void st8(uint32_t at, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::TQ_I8(0), "r"(at) : "memory");
}
// 32 columns of 16 lanes: thread t has, of each 8 columns k, elements 4 k + {0, 1} of lane t / 4, columns 8 k + 2 (t % 4) + {0, 1},
// and 4 k + {2, 3} of lane t / 4 + 8.
TQ_DEVFN void ld16x32(uint32_t at, uint32_t* v) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : TQ_O8(0), TQ_O8(8)
                 : "r"(at)
                 : "memory");
}
#undef TQ_O8
#undef TQ_I8
#undef TQ_L32

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
TQ_DEVFN float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
TQ_DEVFN void stg256(float* p, const float* v) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
// A box's lines into the L2 cache.
TQ_DEVFN void prefetch_2d(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y)
                 : "memory");
}
TQ_DEVFN void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// Weights are rounded to the type of the values, since the tensor cores take both operands in one: each is off by half a step at most
// (bf16 2^-8 of it, fp16 2^-11); the row's sum takes them before.  Results come out 1.04 to 1.4 times as far from 64 bits as with
// fp32 weights and the one rounding at the end (32 x 64 rows, bf16, relative 2-norms: 1.83e-3 for 1.39e-3).
// A row's weights are 2^(f s + bias), f s the score in log2 and bias = kLift - maximum rounded down, the maximum a running one that may
// be kSlack (log2) below the true one before it follows.  fp16: at most 2^14, with half a step of the
// maximum's where the product is not rounded by itself; and the smallest that it holds is 2^-31 of the largest's.
// bf16 has fp32's range: there the maximum seldom follows after the first tokens (each time costs the rescaling of a row's
// sums, and the products wait for it), and sums stay below 2^37 times the largest value.
template <bool BF>
struct Weights {
    static constexpr float kSlack = BF ? 20.0f : 7.0f, kLift = BF ? 0.0f : 7.0f;
    TQ_DEVFN static float bias(float m) { return m == -INFINITY ? 0.f : __fadd_rd(kLift, -m); }
};
// A factor on scores that is never 0, so that a masked score, -infinity times it, is no NaN.
inline float score_factor(float scale) {
    const float f = scale * 1.4426950408889634f, least = 1.8807909613156600e-37f;  // 2^-122
    return f < 0 ? fminf(f, -least) : fmaxf(f, least);
}
// Maxima whose products have to be rounded before the bias is added: the product's own rounding no longer counts for little.
TQ_DEVFN bool huge(float m) { return fabsf(m) > 4194304.f && m != -INFINITY; }
// What sums of weights belong to, for joining them: -infinity where there are none.
TQ_DEVFN float level(float m, float bias) { return m == -INFINITY ? m : -bias; }

// A row-major matrix of 16-bit elements [rows][cols], rows `stride` elements apart, copied in 128-byte swizzled boxes of 64 columns by
// `box` rows; what lies outside is read as zeros.
inline bool tensor_map(CUtensorMap* map, bool bf, const void* base, int64_t rows, int64_t cols, int64_t stride, int box) {
    const EncodeFn encode = tensor_map_encoder();
    if (!encode) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t boxes[2] = {64, (cuuint32_t)box}, steps[2] = {1, 1};
    return encode(map, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims,
                  strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace tq
