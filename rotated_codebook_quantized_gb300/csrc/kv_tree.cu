// Attention of a tree of drafted tokens over the paged compressed cache: tq_kv_attend_tree.
//
// o = softmax(scale * q K^T) V over a sequence's cached tokens and, through an ancestor
// mask, over the drafted tokens.  As in tq_kv_attend the rotation moves off the cache:
// q . k = (R q) . (R k), and sum_t p_t v_t = R^T sum_t p_t (R v_t), one de-rotation per row.
//
// Up to 16 query rows to a kv head, two launches.  kv_tree_context_kernel: the cached tokens.  The work is cut into
// steps of 16 tokens of one (sequence, kv head, tile of query rows); one persistent CTA per SM takes an equal run of the
// steps of the whole batch, whatever the sequences' lengths, and leaves a partial result (maximum, sum, weighted values
// of the rows) wherever its run crosses into another tile.  kv_tree_finish_kernel: the drafted tokens, then the join of a
// tile's partial results, the de-rotation and the output.  More rows: kv_tree_wide.cu's two kernels take the place of the
// first.  (Up to a few thousand tokens those are as fast for few rows too: one row over 100 tokens of one sequence 12.7 us there
// and 13.8 here, over 65536 63 and 44.  A rule on lengths, which are on the device, is not worth the 1 us.)
//
// The context kernel is bound by instruction issue: a lane decodes 128 codes of a step by a table read or two byte
// permutes each (131072 tokens of 8 heads: 59 us alone, 3.5 TB/s of codes and scales, 52 % of the copy rate; the call 67).
#include <math.h>

#include <algorithm>

#include "kv_tree.cuh"

using namespace tq;
using namespace tq::tree;

namespace {

constexpr int kStep = 16;      // tokens of a step, rows of a tile
// The context kernel for tiles of up to ROWS query rows: warps, and steps of a warp's ring (all but one in flight).
// Up to 8 rows the keys and values are the A operands of the products and the rows the 8 columns of B, which halves
// the products and the registers of sums and lets 16 warps stay (32 heads on 8, one token over 131072: 67 us, the
// other form 82; over 100: 13.8 and 15.8).
template <int ROWS>
struct Ctx {
    static constexpr int kWarps = ROWS == 8 ? 16 : 12;  // 128 registers a thread; 168, of which 64 of sums and 32 of queries
    static constexpr int kDepth = ROWS == 8 ? 2 : 3;
    static constexpr int kLowWarps = ROWS == 8 ? 7 : 5;  // whose rings lie below the decode table
    static constexpr int kSums = 4 * ROWS;               // registers of sums
};
constexpr int kFinWarps = 8, kDraftWarps = 4;
constexpr int kFragPad = 33;  // floats of a fragment register over the lanes, padded

// One step of a ring: 16 tokens' codes and scales.
template <int KL, int VL>
struct Stage {
    static constexpr int kKRow = KvBook<KL>::kWords * 4;            // bytes of a key row
    static constexpr int kVRow = VL == 16 ? 80 : 52;                // of a value row: 4-bit rows (64) spread over the banks
    static constexpr int kK = 0, kV = kStep * kKRow, kKs = kV + kStep * kVRow, kVs = kKs + 256, kBytes = kVs + 256;
};
// Shared memory of the context kernel.  The decode table (256 rows of 256 bytes) starts at shared address
// 64 K, so that one byte permute builds the address of an entry (64 K + code * 256 + lane * 4); the rings of
// some warps lie below it, the others above.
constexpr uint32_t kTable = 65536, kTableEnd = 131072;
constexpr uint32_t kSmemStart = 1024 + 512;  // of the space below: the system's first KB, then the static variables
constexpr uint32_t kQueries = kSmemStart, kFactors = kQueries + kStep * kPD * 2, kRingsLow = kFactors + kStep * 4;
template <int KL, int VL, int ROWS>
constexpr uint32_t warp_region() {  // a warp's ring, and its fragments of the join over it
    const uint32_t ring = Ctx<ROWS>::kDepth * Stage<KL, VL>::kBytes, join = Ctx<ROWS>::kSums * kFragPad * 4 + ROWS * 8;
    return ((ring > join ? ring : join) + 127) / 128 * 128;
}
template <int KL, int VL, int ROWS>
constexpr uint32_t context_smem_end() {
    static_assert(kRingsLow % 16 == 0 && kRingsLow + Ctx<ROWS>::kLowWarps * warp_region<KL, VL, ROWS>() <= kTable, "rings below the table");
    return kTableEnd + (Ctx<ROWS>::kWarps - Ctx<ROWS>::kLowWarps) * warp_region<KL, VL, ROWS>();
}

// An 8 x 8 matrix of 16-bit elements, a fragment register, transposed.
TQ_DEVFN uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int KL, int VL, int ROWS>
__global__ void __launch_bounds__(32 * Ctx<ROWS>::kWarps, 1) kv_tree_context_kernel(TreeArgs a) {
    using S = Stage<KL, VL>;
    constexpr int kCtxWarps = Ctx<ROWS>::kWarps, kDepth = Ctx<ROWS>::kDepth, kLowWarps = Ctx<ROWS>::kLowWarps;
    constexpr bool kFew = ROWS == 8;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* const space = smem - (uint32_t)__cvta_generic_to_shared(smem);  // shared address 0
    __half* qh = reinterpret_cast<__half*>(space + kQueries);  // [16][128] rotated queries
    float* qf = reinterpret_cast<float*>(space + kFactors);    // [16] factor from a row's products to log2 scores
    auto region = [&](int w) {  // of a warp
        return w < kLowWarps ? kRingsLow + w * warp_region<KL, VL, ROWS>() : kTableEnd + (w - kLowWarps) * warp_region<KL, VL, ROWS>();
    };
    __shared__ Run s_run;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
    pdl_trigger();
    if (warp == kCtxWarps - 1) {  // beside the others, which build the table
        const Run run = find_run(a, blockIdx.x);
        if (lane == 0) s_run = run;
    }
    // The books as fp16 over a power of two just above their largest centroid, a copy for each lane
    // (bank = lane), so a decoded value over 2^e is at most its group's scale and never overflows fp16.
    const int ek = exponent_above(fmaxf(fabsf(a.c.kcent[0]), fabsf(a.c.kcent[KL - 1])));
    const int ev = exponent_above(fmaxf(fabsf(a.c.vcent[0]), fabsf(a.c.vcent[VL - 1])));
    const float kd = exp2f((float)-ek), vd = exp2f((float)-ev);
    if (warp < kCtxWarps - 1) build_table<KL, VL>(a.c, space + kTable, kd, vd, warp, kCtxWarps - 1);
    // An 8-level value book lives in four registers: low and high bytes of its fp16 centroids.
    uint32_t tl[2] = {0, 0}, th[2] = {0, 0};
    if (VL == 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t h = __half_as_ushort(__float2half_rn(a.c.vcent[i % VL] * vd));
            tl[i >> 2] |= (h & 255u) << (8 * (i & 3));
            th[i >> 2] |= (h >> 8) << (8 * (i & 3));
        }
    }
    __syncthreads();

    Walk walk(s_run);
    const int ng = kPD >> a.c.lgroup;
    const uint32_t ring = region(warp), ring_end = ring + kDepth * S::kBytes;
    // bytes 0 .. 2 of a table address beside the code: lane * 4 in byte 0, the table's 64 K in byte 2
    const uint32_t lane_k = lane * 4 | 0x100, lane_v = lane_k + 128;
    // rows by the 16 (all strides are whole 16s): 32 bits are enough
    const uint32_t page16 = (uint32_t)(a.c.page_stride >> 4), head16 = (uint32_t)(a.c.head_stride >> 4);
    const uint32_t in_page = (1u << (a.c.lpage - 4)) - 1;
    const uint8_t* kc = reinterpret_cast<const uint8_t*>(a.c.kcodes) + lane * 16;
    const uint8_t* vc = reinterpret_cast<const uint8_t*>(a.c.vcodes) + lane * 16;
    const uint8_t* zc = reinterpret_cast<const uint8_t*>(lane < 16 ? a.c.kscales : a.c.vscales) + (lane & 15) * 16;
    // places of the lane's 16-byte pieces in a stage.  128-byte key rows: chunks of odd rows swapped in pairs, so
    // that eight lanes of a read (two rows, every other chunk) meet all banks.
    const uint32_t dk = S::kK + (KL == 256 ? lane ^ ((lane >> 3) & 1) : lane) * 16;
    const uint32_t dv = S::kV + (VL == 16 ? (lane >> 2) * S::kVRow + (lane & 3) * 16 : lane * 16);
    const uint32_t dz = (lane < 16 ? S::kKs : S::kVs) + (lane & 15) * 16;
    const bool copies_z = (lane & 15) < 2 * ng;

    Stretch x;
    while (walk.next(a, x)) {
        const int b = x.b, h = x.h, tile = x.tile, s0 = x.s0, s1 = x.s1, len = x.len, rows = x.rows;

        // the first copies are under way while the queries are turned
        const int32_t* tab = a.table + (int64_t)b * a.table_stride;
        uint32_t okbits = 0;
        auto page_of = [&](int st) { return st < s1 ? __ldg(tab + (st >> (a.c.lpage - 4))) : 0; };
        int ahead = s0 + warp, page_next = page_of(ahead);  // next step to copy, and its page
        uint32_t fill = ring;                               // and its place
        auto issue = [&]() {
            const int page = page_next;
            const uint32_t row16 = (uint32_t)page * page16 + h * head16 + (ahead & in_page);
            page_next = page_of(ahead + kCtxWarps);
            okbits <<= 1;
            if (ahead < s1) {
                if ((uint32_t)page < (uint32_t)a.c.pages) {
                    okbits |= 1;
                    const uint8_t* k = kc + (uint64_t)row16 * (kStep * S::kKRow);
#pragma unroll
                    for (int x = 0; x < kStep * S::kKRow / 512; ++x) cp16(fill + dk + 512 * x, k + 512 * x);
                    const uint8_t* v = vc + (uint64_t)row16 * (kStep * KvBook<VL>::kWords * 4);
                    cp16(fill + dv, v);
                    if (VL == 16 || lane < kStep * KvBook<VL>::kWords / 4 - 32)
                        cp16(fill + dv + (VL == 16 ? 8 * S::kVRow : 512), v + 512);
                    if (copies_z) cp16(fill + dz, zc + (uint64_t)row16 * (uint32_t)(kStep * 2 * ng));
                } else if (lane == 0 && a.err) {
                    atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            ahead += kCtxWarps;
            fill = fill + S::kBytes == ring_end ? ring : fill + S::kBytes;
        };
#pragma unroll
        for (int it = 0; it < kDepth - 1; ++it) issue();

        // queries of the tile: rotated, over a power of two of their own, times the scale's mantissa, fp16
        for (int row = warp; row < ROWS; row += kCtxWarps) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (row < rows) {
                const int y = tile * kStep + row, i = y / a.ratio, g = y - i * a.ratio;
                const uint2 raw = *reinterpret_cast<const uint2*>(a.q + ((int64_t)b * a.n + i) * a.qs +
                                                                  (int64_t)(h * a.ratio + g) * kPD + lane * 4);
                const uint32_t sg = *reinterpret_cast<const uint32_t*>(a.c.signs + lane * 4);
                v[0] = __uint_as_float(raw.x << 16) * (float)(int8_t)sg;
                v[1] = __uint_as_float(raw.x & 0xffff0000u) * (float)(int8_t)(sg >> 8);
                v[2] = __uint_as_float(raw.y << 16) * (float)(int8_t)(sg >> 16);
                v[3] = __uint_as_float(raw.y & 0xffff0000u) * (float)(int8_t)(sg >> 24);
            }
            fwht_warp128(v);
            float mx = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
            for (int m = 16; m; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, m));
            const int e = exponent_above(mx);
            const float d = query_factor(e, a.qmant);  // takes the scale's sign: the factor below is not negative
            *reinterpret_cast<uint2*>(qh + row * kPD + lane * 4) =
                make_uint2(pack_f16(v[0] * d, v[1] * d), pack_f16(v[2] * d, v[3] * d));
            if (lane == 0) qf[row] = score_factor(e + ek, a.qexp);
        }
        __syncthreads();
        // Operand of product step s: the lane's row r (A: and r + 8), dims 32 j + 4 s .. + 3.  Any order
        // of the dims will do as long as the keys' follows it; this one gives a lane whole words of a key.
        uint32_t qa[8][4];  // up to 8 rows: B, two registers
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 lo = *reinterpret_cast<const uint4*>(qh + r * kPD + 32 * j + 8 * i);
            qa[2 * i][0] = lo.x, qa[2 * i][2] = lo.y, qa[2 * i + 1][0] = lo.z, qa[2 * i + 1][2] = lo.w;
            if (kFew) continue;
            const uint4 hi = *reinterpret_cast<const uint4*>(qh + (r + 8) * kPD + 32 * j + 8 * i);
            qa[2 * i][1] = hi.x, qa[2 * i][3] = hi.y, qa[2 * i + 1][1] = hi.z, qa[2 * i + 1][3] = hi.w;
        }
        // the lane's two rows: of scores and sums they are r and r + 8, or 2 j and 2 j + 1
        const float f0 = qf[kFew ? 2 * j : r], f1 = qf[kFew ? 2 * j + 1 : r + 8];

        constexpr int kTiles = kFew ? 8 : 16;
        float o[kTiles][4];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        // the two rows' running maxima (log2), the biases of their weights, and sums
        float m0 = -INFINITY, m1 = -INFINITY, b0 = 0.f, b1 = 0.f, l[4] = {0.f, 0.f, 0.f, 0.f};
        // scale places of the lane: keys' dims 32 j and 32 j + 16, values' dims 16 r
        const int gk0 = (32 * j) >> a.c.lgroup, gk1 = (32 * j + 16) >> a.c.lgroup, gv = (16 * r) >> a.c.lgroup;
        // 3-bit values: dims 16 r .. + 7 begin at code c0 of word w0 (ten to a word), dims 16 r + 8 .. at c1 of w1
        const int w0 = (16 * r) / 10, c0 = (16 * r) % 10, w1 = (16 * r + 8) / 10, c1 = (16 * r + 8) % 10;
        const uint32_t k_at = S::kK + r * S::kKRow + (KL == 256 ? 0 : j * 16);
        const uint32_t kx = KL == 256 ? ((2 * j) ^ (r & 1)) * 16 : 0;  // of the first 16 dims; the other's is ^ 16 (8-bit) or + 8
        const uint32_t ks0 = S::kKs + (r * ng + gk0) * 2, ks1 = S::kKs + (r * ng + gk1) * 2;
        const uint32_t vs_at = S::kVs + (2 * j * ng + gv) * 2;
        const uint32_t v_at = S::kV + 2 * j * S::kVRow + (VL == 8 ? 0 : r * 8);
        uint32_t st = ring;
#pragma unroll 1
        for (int step = s0 + warp; step < s1; step += kCtxWarps) {
            issue();
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
            __syncwarp();
            if ((okbits >> (kDepth - 1)) & 1) {
                const int left = len - step * kStep;  // tokens of the step
                // ---- products of the rows with tokens r (e = 0) and r + 8 (e = 1).  Up to 8 rows: the keys are the A operand, so
                // that one product takes the place of two.
                float sc[2][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) sc[e][0] = sc[e][1] = sc[e][2] = sc[e][3] = 0.f;
                uint32_t ks2[2][2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    ks2[e][0] = lds16(st + ks0 + 16 * e * ng) * 0x10001u;
                    ks2[e][1] = lds16(st + ks1 + 16 * e * ng) * 0x10001u;
                }
                auto key = [&](int e, int half, uint32_t (&k)[4][2]) {  // 16 dims of a token: four steps' operands
                    const uint32_t s2 = ks2[e][half];
                    if constexpr (KL == 256) {
                        const uint4 w4 = lds128(st + k_at + 8 * S::kKRow * e + (kx ^ (16 * half)));
                        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            k[i][0] = mul2(prmt(table<0>(w[i], lane_k), table<1>(w[i], lane_k), 0x5410), s2);
                            k[i][1] = mul2(prmt(table<2>(w[i], lane_k), table<3>(w[i], lane_k), 0x5410), s2);
                        }
                    } else {
                        const uint2 w2 = lds64(st + k_at + 8 * S::kKRow * e + 8 * half);
                        const uint32_t w[2] = {w2.x, w2.y};
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            k[2 * i][0] = mul2(table<0>(w[i], lane_k), s2);
                            k[2 * i][1] = mul2(table<1>(w[i], lane_k), s2);
                            k[2 * i + 1][0] = mul2(table<2>(w[i], lane_k), s2);
                            k[2 * i + 1][1] = mul2(table<3>(w[i], lane_k), s2);
                        }
                    }
                };
                if constexpr (kFew) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t k[2][4][2];
                        key(0, half, k[0]);
                        key(1, half, k[1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t ka[4] = {k[0][i][0], k[1][i][0], k[0][i][1], k[1][i][1]};
                            mma_f16(sc[0], ka, qa[4 * half + i][0], qa[4 * half + i][2]);
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint32_t k[4][2];
                            key(e, half, k);
#pragma unroll
                            for (int i = 0; i < 4; ++i) mma_f16(sc[e], qa[4 * half + i], k[i][0], k[i][1]);
                        }
                }
                if (left < kStep) {  // tokens past the end are left out: rows r and r + 8, or columns 8 e + 2 j + {0, 1}
#pragma unroll
                    for (int e = 0; e < (kFew ? 1 : 2); ++e)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if ((kFew ? r + 8 * (c >> 1) : 8 * e + 2 * j + (c & 1)) >= left) sc[e][c] = -INFINITY;
                }
                // log2 scores are products times f0 and f1, which are not negative
                const float x0 = f0 * (kFew ? fmaxf(sc[0][0], sc[0][2]) : fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1])));
                const float x1 = f1 * (kFew ? fmaxf(sc[0][1], sc[0][3]) : fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3])));
                // the maximum follows only when a score passes it by kSlack (a difference of near numbers is exact)
                if (__any_sync(kFull, x0 - m0 > kSlack || x1 - m1 > kSlack)) {
                    float n0 = x0, n1 = x1;
#pragma unroll
                    for (int m = kFew ? 4 : 1; m < (kFew ? 32 : 4); m <<= 1) {
                        n0 = fmaxf(n0, __shfl_xor_sync(kFull, n0, m));
                        n1 = fmaxf(n1, __shfl_xor_sync(kFull, n1, m));
                    }
                    n0 = fmaxf(n0, m0);
                    n1 = fmaxf(n1, m1);
                    const float c0 = weight_bias(n0), c1 = weight_bias(n1);
                    const float g0 = m0 == -INFINITY ? 0.f : fast_exp2(c0 - b0), g1 = m1 == -INFINITY ? 0.f : fast_exp2(c1 - b1);
                    m0 = n0;
                    m1 = n1;
                    b0 = c0;
                    b1 = c1;
                    l[0] *= g0;
                    l[kFew ? 1 : 2] *= g1;
#pragma unroll
                    for (int i = 0; i < kTiles; ++i) {
                        o[i][0] *= g0;
                        o[i][1] *= kFew ? g1 : g0;
                        o[i][2] *= kFew ? g0 : g1;
                        o[i][3] *= g1;
                    }
                }
                uint32_t pa[4];  // weights as the A operand: the score fragment is already in its order
                uint32_t pb[2];  // or as B, which takes a transpose
                if constexpr (kFew) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        pb[e] = transpose8(pack_f16(fast_exp2(fmaf(sc[0][2 * e], f0, b0)), fast_exp2(fmaf(sc[0][2 * e + 1], f1, b1))));
                    const uint32_t ones[4] = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
                    mma_f16(l, ones, pb[0], pb[1]);  // their sums: a product with ones
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        pa[2 * e] = pack_f16(fast_exp2(fmaf(sc[e][0], f0, b0)), fast_exp2(fmaf(sc[e][1], f0, b0)));
                        pa[2 * e + 1] = pack_f16(fast_exp2(fmaf(sc[e][2], f1, b1)), fast_exp2(fmaf(sc[e][3], f1, b1)));
                    }
                    mma_f16(l, pa, 0x3c003c00u, 0x3c003c00u);  // their sums: a product with ones
                }
                // dims 16 r + i and 16 r + i + 1 of tokens 2 j, 2 j + 1 (lo, hi [0]) and 2 j + 8, 2 j + 9 ([1])
                auto weigh = [&](int i, const uint32_t (&lo)[2], const uint32_t (&hi)[2]) {
                    if constexpr (kFew) {
                        const uint32_t va[4] = {lo[0], hi[0], lo[1], hi[1]};
                        mma_f16(o[i / 2], va, pb[0], pb[1]);
                    } else {
                        mma_f16(o[i], pa, lo[0], lo[1]);
                        mma_f16(o[i + 1], pa, hi[0], hi[1]);
                    }
                };
                // ---- weighted values: tokens 2 j, 2 j + 1 and 2 j + 8, 2 j + 9, dims 16 r + i in tile i
                uint32_t s2[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t at = st + vs_at + 16 * e * ng;
                    s2[e] = lds16(at) | (lds16(at + 2 * ng) << 16);
                }
                if (left < kStep) {  // a scale past the end may be anything
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        s2[e] &= (8 * e + 2 * j < left ? 0xffffu : 0u) | (8 * e + 2 * j + 1 < left ? 0xffff0000u : 0u);
                }
                if constexpr (VL == 8) {
                    uint32_t bits[2][2][2];  // [pair][token][dims 8 q .. + 7]: 24 bits, then whatever follows
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t at = st + v_at + (8 * e + x) * S::kVRow;
                            bits[e][x][0] = (lds32(at + 4 * w0) >> (3 * c0)) + lds32(at + 4 * w0 + 4) * (1u << (30 - 3 * c0));
                            bits[e][x][1] = (lds32(at + 4 * w1) >> (3 * c1)) + lds32(at + 4 * w1 + 4) * (1u << (30 - 3 * c1));
                        }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t v[8][2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t u[2];
#pragma unroll
                            for (int x = 0; x < 2; ++x) {  // two codes to a byte
                                const uint32_t b24 = bits[e][x][q];
                                const uint32_t t = (b24 & 0x0000ffffu) | ((b24 << 4) & 0xffff0000u);
                                u[x] = (t & 0x00ff00ffu) | ((t << 2) & 0xff00ff00u);
                            }
                            // selectors: nibbles (token a, token b) of dims 0, 2, 4, 6 and of dims 1, 3, 5, 7
                            const uint32_t ev0 = ((u[0] & 0x0f0f0f0fu) | ((u[1] << 4) & 0xf0f0f0f0u)) & 0x77777777u;
                            const uint32_t od0 = (((u[0] >> 3) & 0x0f0f0f0fu) | ((u[1] << 1) & 0xf0f0f0f0u)) & 0x77777777u;
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const uint32_t sel = (y & 1 ? od0 : ev0) >> (16 * (y >> 1));
                                const uint32_t lo = prmt(tl[0], tl[1], sel), hi = prmt(th[0], th[1], sel);
                                v[4 * (y >> 1) + (y & 1)][e] = mul2(prmt(lo, hi, 0x5140), s2[e]);
                                v[4 * (y >> 1) + (y & 1) + 2][e] = mul2(prmt(lo, hi, 0x7362), s2[e]);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 8; i += 2) weigh(8 * q + i, v[i], v[i + 1]);
                    }
                } else {
                    uint32_t w[2][2][2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint2 y = lds64(st + v_at + (8 * e + x) * S::kVRow);
                            w[e][x][0] = y.x;
                            w[e][x][1] = y.y;
                        }
                    static_for<0, 8>([&](auto yc) {  // byte y of the 16 dims: dims 2 y and 2 y + 1
                        constexpr int y = decltype(yc)::value;
                        uint32_t lo[2], hi[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t va = table<(y & 3)>(w[e][0][y >> 2], lane_v), vb = table<(y & 3)>(w[e][1][y >> 2], lane_v);
                            lo[e] = mul2(prmt(va, vb, 0x5410), s2[e]);
                            hi[e] = mul2(prmt(va, vb, 0x7632), s2[e]);
                        }
                        weigh(2 * y, lo, hi);
                    });
                }
            }
            __syncwarp();  // the ring slot is free for the next copy
            st = st + S::kBytes == ring_end ? ring : st + S::kBytes;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");

        // ---- join the warps: fragments through shared memory (over the rings)
        const int act = min(kCtxWarps, s1 - s0);
        auto frag = [&](int w) { return reinterpret_cast<float*>(space + region(w)); };                              // [kSums][33]
        auto ml = [&](int w) { return reinterpret_cast<float2*>(space + region(w) + Ctx<ROWS>::kSums * kFragPad * 4); };  // [ROWS]
        __syncwarp();
        if (warp < act) {
            float* f = frag(warp) + lane;
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) f[(4 * i + c) * kFragPad] = o[i][c];
            if ((kFew ? r : j) == 0) {
                ml(warp)[kFew ? 2 * j : r] = make_float2(level(m0, b0), l[0]);
                ml(warp)[kFew ? 2 * j + 1 : r + 8] = make_float2(level(m1, b1), l[kFew ? 1 : 2]);
            }
        }
        __syncthreads();
        const int64_t slot = (int64_t)blockIdx.x + x.unit;
        const float vscale = exp2f((float)ev);
        for (int e = threadIdx.x; e < rows * kPD; e += 32 * kCtxWarps) {
            const int row = e >> 7, d = e & 127, i = d & 15, nn = d >> 4;
            const int at = kFew ? (4 * (i >> 1) + 2 * (i & 1) + (row & 1)) * kFragPad + nn * 4 + (row >> 1)
                                : (4 * i + 2 * (row >> 3) + (nn & 1)) * kFragPad + (row & 7) * 4 + (nn >> 1);
            float M = -INFINITY;
            for (int w = 0; w < act; ++w) M = fmaxf(M, ml(w)[row].x);
            float L = 0.f, acc = 0.f;
            for (int w = 0; w < act; ++w) {
                const float2 s = ml(w)[row];
                const float g = s.x == -INFINITY ? 1.f : fast_exp2(s.x - M);  // nothing seen: zeros, or NaN scores
                L = fmaf(g, s.y, L);
                acc = fmaf(g, frag(w)[at], acc);
            }
            a.part[(slot * kStep + row) * kPD + d] = acc * vscale;
            if (d == 0) a.stat[slot * kStep + row] = make_float2(M, L);
        }
        __syncthreads();  // the rings and the queries are free
    }
}

// ---------------------------------------------------------------- drafted tokens, join, output

// Which of the drafts t0 .. t0 + 15 draft i of sequence b sees (t0 a multiple of 16, i < n): bit by bit.
TQ_DEVFN uint32_t sees(const TreeArgs& a, int b, int i, int t0, int live) {
    const uint32_t in = live - t0 >= kStep ? 0xffffu : (1u << max(live - t0, 0)) - 1u;
    if (!a.mask) return in & (i - t0 >= kStep - 1 ? 0xffffu : (1u << max(i - t0 + 1, 0)) - 1u);
    return in & (uint32_t)(a.mask[((int64_t)b * a.n + i) * ((a.n + 63) >> 6) + (t0 >> 6)] >> (t0 & 63));
}

// One CTA per (sequence, kv head, tile of 16 rows).  The drafted tokens come as they are: bf16 queries, keys
// and values on the tensor cores, exact but for the weights, which are split in two bf16 halves.
__global__ void __launch_bounds__(32 * kFinWarps) kv_tree_finish_kernel(TreeArgs a, int tiles_max, int parts) {
    __shared__ float frag[kDraftWarps][64][kFragPad];
    __shared__ float2 ml[kDraftWarps][kStep];
    __shared__ __align__(16) float joined[kFinWarps][kPD];
    __shared__ float2 jml[kFinWarps];
    __shared__ Count s_before, s_all;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
    const int part = blockIdx.x % parts, tb = blockIdx.x / parts;  // of a tile's rows; parts: 1, 2 or 4
    const int tile = tb % tiles_max, bh = tb / tiles_max, h = bh % a.c.Hkv, b = bh / a.c.Hkv;
    const int live = seq_live(a, b), all = a.n * a.ratio;
    const int row0 = part * (kStep / parts);
    const int rows = min(kStep / parts, all - tile * kStep - row0);  // rows of the output, from row0 of the tile
    if (rows <= 0) return;
    const int used = min(rows, live * a.ratio - tile * kStep - row0);  // of which in use (may be none)
    // A operand rows r and r + 8 of the tile
    const int x0 = tile * kStep + r, x1 = x0 + 8;
    const int i0 = x0 / a.ratio, i1 = x1 / a.ratio;
    const int dsteps = a.kn && used > 0 ? (live + kStep - 1) / kStep : 0;
    const int dact = min(dsteps, kDraftWarps);
    if (warp < dact) {
        uint32_t qa[8][4];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int x = y ? x1 : x0, i = y ? i1 : i0;
            const bool in = x < live * a.ratio;
            const uint4* src = reinterpret_cast<const uint4*>(a.q + ((int64_t)b * a.n + i) * a.qs +
                                                              (int64_t)(h * a.ratio + x - i * a.ratio) * kPD + 32 * j);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const uint4 v = in ? src[z] : make_uint4(0u, 0u, 0u, 0u);
                qa[2 * z][y] = v.x, qa[2 * z][2 + y] = v.y, qa[2 * z + 1][y] = v.z, qa[2 * z + 1][2 + y] = v.w;
            }
        }
        float o[16][4];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
#pragma unroll 1
        for (int st = warp; st < dsteps; st += kDraftWarps) {
            const int t0 = st * kStep;
            // everything that the step reads is under way before the first of it is used
            const uint32_t see[2] = {sees(a, b, min(i0, a.n - 1), t0, live), sees(a, b, min(i1, a.n - 1), t0, live)};
            uint4 vraw[2][2][2];  // values of tokens 2 j, 2 j + 1, 2 j + 8, 2 j + 9, dims 16 r .. + 15
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int t = t0 + 8 * e + 2 * j + y;
                        vraw[z][e][y] = t < live ? reinterpret_cast<const uint4*>(a.vn + ((int64_t)b * a.n + t) * a.vs +
                                                                                  (int64_t)h * kPD + 16 * r)[z]
                                                 : make_uint4(0u, 0u, 0u, 0u);
                    }
            float sc[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = t0 + 8 * e + r;
                sc[e][0] = sc[e][1] = sc[e][2] = sc[e][3] = 0.f;
                const uint4* src = reinterpret_cast<const uint4*>(a.kn + ((int64_t)b * a.n + t) * a.ks + (int64_t)h * kPD + 32 * j);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const uint4 v = t < live ? src[z] : make_uint4(0u, 0u, 0u, 0u);
                    mma_bf16(sc[e], qa[2 * z], v.x, v.y);
                    mma_bf16(sc[e], qa[2 * z + 1], v.z, v.w);
                }
            }
            float x[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    sc[e][c] = (see[c >> 1] >> (8 * e + 2 * j + (c & 1))) & 1 ? sc[e][c] * a.scale2 : -INFINITY;
                    x[c >> 1] = fmaxf(x[c >> 1], sc[e][c]);
                }
#pragma unroll
            for (int m = 1; m < 4; m <<= 1) {
                x[0] = fmaxf(x[0], __shfl_xor_sync(kFull, x[0], m));
                x[1] = fmaxf(x[1], __shfl_xor_sync(kFull, x[1], m));
            }
            const float n0 = fmaxf(m0, x[0]), n1 = fmaxf(m1, x[1]);
            const float g0 = m0 == -INFINITY ? 1.f : exp2f(m0 - n0), g1 = m1 == -INFINITY ? 1.f : exp2f(m1 - n1);
            m0 = n0;
            m1 = n1;
            l0 *= g0;
            l1 *= g1;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                o[i][0] *= g0;
                o[i][1] *= g0;
                o[i][2] *= g1;
                o[i][3] *= g1;
            }
            const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
            uint32_t ph[4], pl[4];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float wa = exp2f(sc[e][2 * y] - (y ? b1 : b0)), wb = exp2f(sc[e][2 * y + 1] - (y ? b1 : b0));
                    (y ? l1 : l0) += wa + wb;
                    sc[e][2 * y] = wa;
                    sc[e][2 * y + 1] = wb;
                    const __nv_bfloat162 hi = __floats2bfloat162_rn(wa, wb);
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(wa - __low2float(hi), wb - __high2float(hi));
                    ph[2 * e + y] = *reinterpret_cast<const uint32_t*>(&hi);
                    pl[2 * e + y] = *reinterpret_cast<const uint32_t*>(&lo);
                }
            // values that are not finite are taken out (0 times them would reach rows that do not see them) and added below
            // to the rows that do
            uint32_t bad = 0;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                uint32_t w[2][2][4];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint4 v = vraw[z][e][y];
                        w[e][y][0] = v.x, w[e][y][1] = v.y, w[e][y][2] = v.z, w[e][y][3] = v.w;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t inf = ((w[e][y][k] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
                            bad |= inf;
                            w[e][y][k] &= ~((inf >> 15) * 0xffffu);
                        }
                    }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t lo0 = prmt(w[0][0][k], w[0][1][k], 0x5410), lo1 = prmt(w[1][0][k], w[1][1][k], 0x5410);
                    const uint32_t hi0 = prmt(w[0][0][k], w[0][1][k], 0x7632), hi1 = prmt(w[1][0][k], w[1][1][k], 0x7632);
                    mma_bf16(o[8 * z + 2 * k], ph, lo0, lo1);
                    mma_bf16(o[8 * z + 2 * k], pl, lo0, lo1);
                    mma_bf16(o[8 * z + 2 * k + 1], ph, hi0, hi1);
                    mma_bf16(o[8 * z + 2 * k + 1], pl, hi0, hi1);
                }
            }
            if (__any_sync(kFull, bad != 0)) {
#pragma unroll
                for (int col = 0; col < kStep; ++col) {
                    const int t = t0 + col, from = (lane & ~3) | ((col & 7) >> 1);
                    const float w0 = __shfl_sync(kFull, sc[col >> 3][col & 1], from);
                    const float w1 = __shfl_sync(kFull, sc[col >> 3][2 + (col & 1)], from);
                    if (t < live) {
                        const bool see0 = (see[0] >> col) & 1, see1 = (see[1] >> col) & 1;
                        const __nv_bfloat16* v = a.vn + ((int64_t)b * a.n + t) * a.vs + (int64_t)h * kPD;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const float x = __bfloat162float(v[16 * (2 * j + y) + i]);
                                if (!isfinite(x)) {
                                    if (see0) o[i][y] += w0 * x;
                                    if (see1) o[i][2 + y] += w1 * x;
                                }
                            }
                    }
                }
            }
        }
        l0 += __shfl_xor_sync(kFull, l0, 1);
        l0 += __shfl_xor_sync(kFull, l0, 2);
        l1 += __shfl_xor_sync(kFull, l1, 1);
        l1 += __shfl_xor_sync(kFull, l1, 2);
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) frag[warp][4 * i + c][lane] = o[i][c];
        if (j == 0) {
            ml[warp][r] = make_float2(m0, l0);
            ml[warp][r + 8] = make_float2(m1, l1);
        }
    }
    if (blockIdx.x == 0 && a.err)
        for (int i = threadIdx.x; i < a.B; i += 32 * kFinWarps)
            if (a.lens[i] < 0 || a.lens[i] > a.max_len) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
    if (warp == kFinWarps - 1) {
        Count before, total;
        count_work(a, b, before, total);
        if (lane == 0) {
            s_before = before;
            s_all = total;
        }
    }
    const uint32_t sg = *reinterpret_cast<const uint32_t*>(a.c.signs + lane * 4);
    int share = 1;
    while (share * 2 * rows <= kFinWarps) share *= 2;  // warps of a row
    // A warp's rows: one of up to 8, or two (row and row + 8), whose reads go together.
    constexpr int kRowsOf = kStep / kFinWarps;
    auto row_of = [&](int k) { return warp / share + kFinWarps * k; };
    __syncthreads();
    // the drafts' results of the rows, joined while the context is under way
    float dm[kRowsOf], dl[kRowsOf], dv[kRowsOf][4];
#pragma unroll
    for (int k = 0; k < kRowsOf; ++k) {
        const int row = row0 + row_of(k);
        dm[k] = -INFINITY;
        dl[k] = dv[k][0] = dv[k][1] = dv[k][2] = dv[k][3] = 0.f;
        if (row_of(k) < used)
            for (int w = 0; w < dact; ++w) {
                const float2 st = ml[w][row];
                const float N = fmaxf(dm[k], st.x), g = dm[k] == -INFINITY ? 1.f : exp2f(dm[k] - N);
                const float f = st.x == -INFINITY ? 1.f : exp2f(st.x - N);  // nothing seen: zeros, or NaN sums
                dm[k] = N;
                dl[k] = fmaf(f, st.y, dl[k] * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = lane * 4 + e, i = d & 15, nn = d >> 4;
                    dv[k][e] = fmaf(f, frag[w][4 * i + 2 * (row >> 3) + (nn & 1)][(row & 7) * 4 + (nn >> 1)], dv[k][e] * g);
                }
            }
    }
    pdl_wait();  // the context's partial results

    // Partial results of this tile: runs first .. last, each at slot run + unit.  Warps share a row where rows are few.
    const int pad = tile_pad(a, s_all.steps), per = places_per_cta(a, s_all.steps + s_all.busy * pad);
    const int wide = tile * kStep / a.trows, row_at = tile * kStep + row0 - wide * a.trows;  // the context's tile, and the first row in it
    const int steps = seq_steps(a, b), of_seq = h * seq_tiles(a, b) + wide, unit = s_before.units + of_seq;
    const int at = s_before.steps + s_before.busy * pad + of_seq * (steps + pad) + pad;  // its first step's place
    const int first = used > 0 && steps ? at / per : 0;
    const int count = used > 0 && steps ? (at + steps - 1) / per - first + 1 : 0;
    // A lane reads a partial result's statistics, then all of them walk the weighted values.
    float M[kRowsOf], L[kRowsOf], v[kRowsOf][4];
    const int mine = (count - warp % share + share - 1) / share;  // partial results of this warp
    const int64_t slot0 = (int64_t)first + unit + warp % share;
#pragma unroll
    for (int k = 0; k < kRowsOf; ++k) {
        M[k] = -INFINITY;
        L[k] = v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0.f;
    }
    for (int x0 = 0; x0 < mine; x0 += 32) {
        float w[kRowsOf];
#pragma unroll
        for (int k = 0; k < kRowsOf; ++k) {
            const bool in = row_of(k) < used && x0 + lane < mine;
            const float2 st = in ? a.stat[(slot0 + (int64_t)(x0 + lane) * share) * a.trows + row_at + row_of(k)] : make_float2(-INFINITY, 0.f);
            float top = fmaxf(M[k], st.x);
#pragma unroll
            for (int m = 16; m; m >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, m));
            const float g = M[k] == -INFINITY ? 1.f : exp2f(M[k] - top);  // nothing so far: zeros, or NaN sums
            w[k] = st.x == -INFINITY ? 1.f : exp2f(st.x - top);
            float l = w[k] * st.y;
#pragma unroll
            for (int m = 16; m; m >>= 1) l += __shfl_xor_sync(kFull, l, m);
            M[k] = top;
            L[k] = fmaf(L[k], g, l);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[k][e] *= g;
        }
        const int n = min(32, mine - x0);
        constexpr int kBatch = 8;  // reads under way together: each takes about a thousand cycles
        for (int x1 = 0; x1 < n; x1 += kBatch) {
            float4 y[kBatch][kRowsOf];
#pragma unroll
            for (int z = 0; z < kBatch; ++z) {
                const float* src = a.part + ((slot0 + (int64_t)(x0 + min(x1 + z, n - 1)) * share) * a.trows + row_at) * kPD + lane * 4;
#pragma unroll
                for (int k = 0; k < kRowsOf; ++k)
                    y[z][k] = row_of(k) < used ? *reinterpret_cast<const float4*>(src + row_of(k) * kPD) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int z = 0; z < kBatch; ++z)
                if (x1 + z < n) {
#pragma unroll
                    for (int k = 0; k < kRowsOf; ++k) {
                        const float g = __shfl_sync(kFull, w[k], x1 + z);
                        v[k][0] = fmaf(g, y[z][k].x, v[k][0]);
                        v[k][1] = fmaf(g, y[z][k].y, v[k][1]);
                        v[k][2] = fmaf(g, y[z][k].z, v[k][2]);
                        v[k][3] = fmaf(g, y[z][k].w, v[k][3]);
                    }
                }
        }
    }
    if (share > 1) {  // the warps of a row (rows of at most half as many as warps: one to a warp)
        *reinterpret_cast<float4*>(&joined[warp][lane * 4]) = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
        if (lane == 0) jml[warp] = make_float2(M[0], L[0]);
        __syncthreads();
        if (warp % share) return;
        float N = -INFINITY;
        for (int x = 0; x < share; ++x) N = fmaxf(N, jml[warp + x].x);
        M[0] = N;
        L[0] = v[0][0] = v[0][1] = v[0][2] = v[0][3] = 0.f;
        for (int x = 0; x < share; ++x) {
            const float2 st = jml[warp + x];
            const float4 y = *reinterpret_cast<const float4*>(&joined[warp + x][lane * 4]);
            const float g = st.x == -INFINITY ? 1.f : exp2f(st.x - N);
            L[0] = fmaf(g, st.y, L[0]);
            v[0][0] = fmaf(g, y.x, v[0][0]);
            v[0][1] = fmaf(g, y.y, v[0][1]);
            v[0][2] = fmaf(g, y.z, v[0][2]);
            v[0][3] = fmaf(g, y.w, v[0][3]);
        }
    }
#pragma unroll
    for (int k = 0; k < kRowsOf; ++k) {
        const int row = row_of(k);
        if (row >= rows) continue;
        const float N = fmaxf(M[k], dm[k]);
        const float g = M[k] == -INFINITY ? 1.f : exp2f(M[k] - N), f = dm[k] == -INFINITY ? 1.f : exp2f(dm[k] - N);
        fwht_warp128(v[k]);
        L[k] = fmaf(f, dl[k], L[k] * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] = fmaf(f, dv[k][e], v[k][e] * (g * kInvSqrtD * (float)(int8_t)(sg >> (8 * e))));
        // no weight at all: zeros.  A NaN sum stays NaN.
        const float inv = L[k] == 0.f ? 0.f : 1.0f / L[k];
        const int x = tile * kStep + row0 + row, i = x / a.ratio;
        __nv_bfloat162 y[2];
        y[0] = row >= used ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(v[k][0] * inv, v[k][1] * inv);
        y[1] = row >= used ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(v[k][2] * inv, v[k][3] * inv);
        *reinterpret_cast<uint2*>(a.o + (((int64_t)b * a.n + i) * a.Hq + h * a.ratio + x - i * a.ratio) * kPD + lane * 4) =
            make_uint2(*reinterpret_cast<uint32_t*>(&y[0]), *reinterpret_cast<uint32_t*>(&y[1]));
    }
}

int sm_count() {
    static const int n = [] {
        int dev = 0, v = 0;
        cudaGetDevice(&dev);
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        return v > 0 ? v : 1;
    }();
    return n;
}

struct Plan {
    int64_t tiles, slots, turned;  // output tiles of 16 rows; partial results, rows of turned queries at most
    int ctas, trows, stoks, least, pad;
};

// Rows, tiles and steps of a call within 30 bits, which the kernels count in 32 (B, n, Hq and Hkv positive).
bool plan_fits(int32_t Hkv, int32_t B, int32_t n, int32_t Hq, int64_t max_len) {
    constexpr double kMost = 0x3fffffff;  // products are compared in doubles: they may pass 64 bits
    const int64_t rows = (int64_t)n * (Hq / Hkv);
    if (rows > 0x3fffffffll || max_len > 0x7fffffffll - 64) return false;
    const double heads = (double)Hkv * B, step = rows <= kStep ? kStep : 32, tile = rows <= kStep ? kStep : (rows <= 128 ? 128 : 256);
    return heads * ((rows + kStep - 1) / kStep) <= kMost && heads * ceil(rows / tile) * (ceil(max_len / step) + 24) <= kMost;
}

// Context launch and workspace of a call.  Runs (CTAs) and units both ascend along the work, so run + unit numbers every
// partial result once.  Up to 16 rows to a kv head go to the kernel above, more to the one that decodes a step once for
// 128 or 256 rows.  (32 rows over 131072 tokens of 8 heads: 146 us above, 106 there; 20 rows over 32768: 49 and 39.  256 rows
// over 131072 tokens: 202 us as two tiles of 128, 156 as one of 256; over 4096, where beginning a tile counts, 26 and 30.)
Plan make_plan(int32_t Hkv, int32_t B, int32_t n, int32_t Hq, int64_t max_len, int sms) {
    Plan p{};
    const int64_t rows = (int64_t)n * (Hq / Hkv);
    p.trows = rows <= kStep ? kStep : (rows <= 128 ? 128 : 256);
    p.stoks = p.trows == kStep ? kStep : 32;
    p.least = p.trows == kStep ? 4 : 2;
    // measured, beginning another tile within a run: about 4 us (16 rows, 128 rows) and 10 us (256 rows)
    p.pad = p.trows == kStep ? 24 : (p.trows == 128 ? 8 : 14);
    p.tiles = (rows + kStep - 1) / kStep;
    const int64_t units = (rows + p.trows - 1) / p.trows * Hkv * B, steps = max_len ? (max_len + p.stoks - 1) / p.stoks + p.pad : 0;
    p.ctas = (int)std::min<int64_t>(sms, (units * steps + p.least - 1) / p.least);
    p.slots = p.ctas ? units + p.ctas : 0;
    p.turned = p.ctas && p.trows != kStep ? units * p.trows : 0;
    return p;
}

// Scratch of a plan: partial results and their statistics, turned queries and their exponents, and 32 bytes of alignment.
size_t plan_bytes(const Plan& p) {
    return 32 + (size_t)p.slots * p.trows * (kPD * sizeof(float) + sizeof(float2)) + (size_t)p.turned * (kPD * 2 + 4);
}

template <int KL, int VL, int ROWS>
tq_status launch_context(const TreeArgs& a, cudaStream_t st) {
    constexpr size_t smem = context_smem_end<KL, VL, ROWS>() - 1024;  // from the start of the dynamic part, wherever it is
    static const bool fits = [] {  // the system's part and the static variables end below kSmemStart
        int dev = 0, reserved = 0;
        cudaFuncAttributes at{};
        return cudaGetDevice(&dev) == cudaSuccess &&
               cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev) == cudaSuccess &&
               cudaFuncGetAttributes(&at, (const void*)kv_tree_context_kernel<KL, VL, ROWS>) == cudaSuccess &&
               reserved >= 1024 && reserved + at.sharedSizeBytes <= kSmemStart;
    }();
    if (!fits) return TQ_ERR_UNSUPPORTED;
    if (ensure_smem((const void*)kv_tree_context_kernel<KL, VL, ROWS>, smem) != cudaSuccess) return TQ_ERR_CUDA;
    kv_tree_context_kernel<KL, VL, ROWS><<<a.ctas, 32 * Ctx<ROWS>::kWarps, smem, st>>>(a);
    return launch_status();
}

template <int ROWS>
tq_status launch_books(const tq_kv_pages_t* cache, const TreeArgs& a, cudaStream_t st) {
    if (cache->kcb.levels == 256)
        return cache->vcb.levels == 8 ? launch_context<256, 8, ROWS>(a, st) : launch_context<256, 16, ROWS>(a, st);
    return cache->vcb.levels == 8 ? launch_context<16, 8, ROWS>(a, st) : launch_context<16, 16, ROWS>(a, st);
}

constexpr int kMaxSms = 256;  // bound on the SMs that the workspace is sized for

}  // namespace

extern "C" size_t tq_kv_attend_tree_workspace_bytes(const tq_kv_pages_t* cache, int32_t B, int32_t n, int32_t Hq,
                                                    int64_t max_len) {
    if (kv_pages_check(cache, false) != TQ_OK || B <= 0 || n <= 0 || Hq <= 0 || Hq % cache->Hkv || max_len < 0) return 0;
    if (!plan_fits(cache->Hkv, B, n, Hq, max_len)) return 0;
    return plan_bytes(make_plan(cache->Hkv, B, n, Hq, max_len, kMaxSms));
}

extern "C" tq_status tq_kv_attend_tree(const tq_kv_pages_t* cache, const void* q, int64_t q_stride, tq_dtype dt,
                                       int32_t B, int32_t n, int32_t Hq, const int32_t* table, int32_t table_stride,
                                       const int32_t* lens, int64_t max_len, const void* k_new, int64_t k_stride,
                                       const void* v_new, int64_t v_stride, const uint64_t* mask,
                                       const int32_t* n_tok, float scale, void* o, void* ws, size_t ws_bytes,
                                       uint32_t* err, void* stream) {
    const tq_status ok = kv_pages_check(cache, false);
    if (ok != TQ_OK) return ok;
    if (dt != TQ_BF16) return dt == TQ_F32 || dt == TQ_F16 ? TQ_ERR_UNSUPPORTED : TQ_ERR_INVALID;
    if (B < 0 || n < 0 || Hq <= 0 || Hq > 65535 || Hq % cache->Hkv || max_len < 0 || table_stride < 0 || !isfinite(scale))
        return TQ_ERR_INVALID;
    if (max_len > (int64_t)table_stride * cache->page) return TQ_ERR_INVALID;
    if (q_stride < (int64_t)Hq * kPD || q_stride % 8) return TQ_ERR_INVALID;
    if (!k_new != !v_new) return TQ_ERR_INVALID;
    if (k_new && (k_stride < (int64_t)cache->Hkv * kPD || k_stride % 8 || v_stride < (int64_t)cache->Hkv * kPD || v_stride % 8))
        return TQ_ERR_INVALID;
    if (B == 0 || n == 0) return TQ_OK;
    if (!q || !o || !lens || !ws || (max_len && !table)) return TQ_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(ws, 16) ||
        !aligned(mask, 8) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(n_tok, 4) || !aligned(err, 4))
        return TQ_ERR_INVALID;
    if (!plan_fits(cache->Hkv, B, n, Hq, max_len)) return TQ_ERR_UNSUPPORTED;
    if (ws_bytes < tq_kv_attend_tree_workspace_bytes(cache, B, n, Hq, max_len)) return TQ_ERR_INVALID;
    // (the size above is for the most SMs; a plan for fewer takes no more, and is held to it)
    const Plan p = make_plan(cache->Hkv, B, n, Hq, max_len, std::min(sm_count(), kMaxSms));
    if (ws_bytes < plan_bytes(p)) return TQ_ERR_INVALID;
    // cache rows by the 8 are 32-bit numbers
    if ((cache->pages * cache->page_stride + cache->Hkv * cache->head_stride) / 8 > 0xffffffffll) return TQ_ERR_UNSUPPORTED;
    TreeArgs a{};
    a.c = kv_pages_view(cache);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.kn = static_cast<const __nv_bfloat16*>(k_new);
    a.vn = static_cast<const __nv_bfloat16*>(v_new);
    a.qs = q_stride;
    a.ks = k_stride;
    a.vs = v_stride;
    a.max_len = max_len;
    a.table = table;
    a.lens = lens;
    a.mask = mask;
    a.n_tok = n_tok;
    a.B = B;
    a.n = n;
    a.Hq = Hq;
    a.ratio = Hq / cache->Hkv;
    a.table_stride = table_stride;
    a.ctas = std::max(p.ctas, 1);
    a.trows = p.trows;
    a.stoks = p.stoks;
    a.least = p.least;
    a.pad = p.pad;
    a.wait_cycles = wait_budget();
    a.scale2 = scale * kLog2e;
    int qexp = 0;
    const double qmant = 2.0 * frexp((double)scale * kLog2e * kInvSqrtD, &qexp);
    a.qmant = (float)qmant;
    a.qexp = qexp - 1;
    a.o = static_cast<__nv_bfloat16*>(o);
    a.part = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(ws) + 31) & ~uintptr_t(31));  // 32-byte stores
    a.stat = reinterpret_cast<float2*>(a.part + (size_t)p.slots * p.trows * kPD);
    a.turned = reinterpret_cast<uint4*>(a.stat + (size_t)p.slots * p.trows);
    a.power = reinterpret_cast<int32_t*>(a.turned + (size_t)p.turned * 16);
    a.err = err;
    // A tile's rows go to up to four CTAs of the last launch where there are SMs for them: reading the partial results is
    // bound by each SM's share of the L2 (16 drafts of 32 heads on 8 over 32768 tokens: 43.1 us with one CTA to a tile, 41.1 with four).
    const int64_t all_tiles = p.tiles * cache->Hkv * B;
    const int parts = all_tiles * 4 <= sm_count() ? 4 : (all_tiles * 2 <= sm_count() ? 2 : 1);
    cudaStream_t st = as_stream(stream);
    if (p.ctas) {
        tq_status s;
        if (p.trows != kStep) s = launch_wide(cache->kcb.levels, cache->vcb.levels, a, st);
        else s = n * a.ratio <= 8 ? launch_books<8>(cache, a, st) : launch_books<16>(cache, a, st);
        if (s != TQ_OK) return s;
        return launch_pdl(kv_tree_finish_kernel, dim3((unsigned)(p.tiles * cache->Hkv * B * parts)), dim3(32 * kFinWarps), 0, st, a, (int)p.tiles, parts);
    }
    kv_tree_finish_kernel<<<(unsigned)(p.tiles * cache->Hkv * B * parts), 32 * kFinWarps, 0, st>>>(a, (int)p.tiles, parts);
    return launch_status();
}
