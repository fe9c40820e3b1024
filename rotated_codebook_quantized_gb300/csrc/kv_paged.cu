// The paged compressed KV cache written and read back: tq_kv_append, tq_kv_fetch.
//
// "How it works", "The KV cache", and "Running a 1T-Parameter Model on a Laptop",
// update_and_fetch: rotate, quantize, store; dequantize, de-rotate.  The arithmetic of a
// vector is tq_kv_quantize's; a token's row is found through its slot.
#include <math.h>

#include "common.cuh"
#include "kv_pages.cuh"
#include "rope.cuh"

using namespace tq;

namespace {

constexpr int kWarps = 8;

struct AppendArgs {
    KvPages c;
    const void* k;
    const void* v;
    int64_t ks, vs, T;
    const int32_t* slots;
    const int32_t* pos;
    const uint64_t* steps;
    int lrot, interleaved;  // log2 of the rotary length
    float factor;
    int dt;
    uint32_t* err;
};

// One warp per (token, head): K, then V.
template <int KL, int VL>
__global__ void __launch_bounds__(32 * kWarps) kv_append_kernel(AppendArgs a) {
    __shared__ float kt[256], vt[16];
    __shared__ uint8_t cd[kWarps][kPD];
    for (int i = threadIdx.x; i < KL - 1; i += blockDim.x) kt[i] = a.c.kthr[i];
    for (int i = threadIdx.x; i < VL - 1; i += blockDim.x) vt[i] = a.c.vthr[i];
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t vec = (int64_t)blockIdx.x * kWarps + warp;
    if (vec >= a.T * a.c.Hkv) return;
    const int64_t t = vec / a.c.Hkv;
    const int h = (int)(vec - t * a.c.Hkv);
    const int32_t slot = a.slots[t];
    if (slot < 0) return;
    if ((int64_t)slot >= a.c.pages << a.c.lpage) {
        if (lane == 0 && a.err) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
        return;
    }
    const int64_t row = a.c.row(slot, h);
    const int group = 1 << a.c.lgroup, lpg = group / 4;
    for (int which = 0; which < 2; ++which) {
        const int64_t src = t * (which ? a.vs : a.ks) + (int64_t)h * kPD;
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = load_as_float(which ? a.v : a.k, src + lane * 4 + i, a.dt);
        if (which == 0 && a.steps) {
            const int rotary = 1 << a.lrot, half = rotary / 2;
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = lane * 4 + i;
                const float o = a.interleaved ? x[i ^ 1] : __shfl_xor_sync(kFull, x[i], half / 4);
                const int pair = a.interleaved ? e >> 1 : e & (half - 1);
                const bool second = a.interleaved ? (i & 1) : (e & half);
                float sn = 0.f, cs = 1.f;
                if (e < rotary) {
                    rope_angle(a.pos[t], a.steps[pair], sn, cs);
                    sn *= second ? a.factor : -a.factor;
                    cs *= a.factor;
                }
                y[i] = e < rotary ? x[i] * cs + o * sn : x[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = y[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] *= (float)a.c.signs[lane * 4 + i];
        fwht_warp128(x);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] *= 0.08838834764831845f;  // 1 / sqrt(128)
            ss += x[i] * x[i];
        }
        for (int m = 1; m < lpg; m <<= 1) ss += __shfl_xor_sync(kFull, ss, m);
        const float s = sqrtf(ss / (float)group);
        uint16_t* scales = which ? a.c.vscales : a.c.kscales;
        if ((lane & (lpg - 1)) == 0)
            scales[(row << (7 - a.c.lgroup)) + lane / lpg] = __half_as_ushort(__float2half_rn(s));
        const float* thr = which ? vt : kt;
        const int n = (which ? VL : KL) - 1;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = s > 0.f ? x[i] / s : 0.f;
            int lo = 0, hi = n;  // thresholds strictly below u
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (thr[mid] < u) lo = mid + 1; else hi = mid;
            }
            cd[warp][lane * 4 + i] = (uint8_t)lo;
        }
        __syncwarp();
        const int bits = which ? KvBook<VL>::kBits : KvBook<KL>::kBits, cw = 32 / bits;
        const int words = which ? KvBook<VL>::kWords : KvBook<KL>::kWords;
        if (lane < words) {
            uint32_t w = 0;
            for (int i = 0; i < cw && lane * cw + i < kPD; ++i) w |= (uint32_t)cd[warp][lane * cw + i] << (bits * i);
            (which ? a.c.vcodes : a.c.kcodes)[row * words + lane] = w;
        }
    }
}

struct FetchArgs {
    KvPages c;
    const int32_t* slots;
    int64_t T;
    void* k;
    void* v;
    int dt;
    uint32_t* err;
};

// One warp per (token, head): K, then V.
template <int KL, int VL>
__global__ void __launch_bounds__(32 * kWarps) kv_fetch_kernel(FetchArgs a) {
    __shared__ float kl[KL], vl[VL];
    for (int i = threadIdx.x; i < KL; i += blockDim.x) kl[i] = a.c.kcent[i];
    for (int i = threadIdx.x; i < VL; i += blockDim.x) vl[i] = a.c.vcent[i];
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t vec = (int64_t)blockIdx.x * kWarps + warp;
    if (vec >= a.T * a.c.Hkv) return;
    const int64_t t = vec / a.c.Hkv;
    const int h = (int)(vec - t * a.c.Hkv);
    int32_t slot = a.slots[t];
    if ((int64_t)slot >= a.c.pages << a.c.lpage) {
        if (lane == 0 && a.err) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
        slot = -1;
    }
    const int64_t row = slot < 0 ? 0 : a.c.row(slot, h);
    for (int which = 0; which < 2; ++which) {
        void* out = which ? a.v : a.k;
        if (!out) continue;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (slot >= 0) {
            const int bits = which ? KvBook<VL>::kBits : KvBook<KL>::kBits, cw = 32 / bits;
            const uint32_t* w = (which ? a.c.vcodes : a.c.kcodes) + row * (which ? KvBook<VL>::kWords : KvBook<KL>::kWords);
            const uint16_t* sc = (which ? a.c.vscales : a.c.kscales) + (row << (7 - a.c.lgroup));
            const float s = half_bits_to_float(sc[(lane * 4) >> a.c.lgroup]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = lane * 4 + i;
                const uint32_t c = (w[d / cw] >> (bits * (d % cw))) & ((1u << bits) - 1u);
                x[i] = s * (which ? vl : kl)[c];
            }
        }
        fwht_warp128(x);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            store_from_float(out, vec * kPD + lane * 4 + i, a.dt,
                             x[i] * 0.08838834764831845f * (float)a.c.signs[lane * 4 + i]);
    }
}

// fn<KL, VL>() for the books of a cache.
template <class F>
tq_status by_books(const tq_kv_pages_t* c, F&& f) {
    if (c->kcb.levels == 256)
        return c->vcb.levels == 8 ? f(std::integral_constant<int, 256>{}, std::integral_constant<int, 8>{})
                                  : f(std::integral_constant<int, 256>{}, std::integral_constant<int, 16>{});
    return c->vcb.levels == 8 ? f(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{})
                              : f(std::integral_constant<int, 16>{}, std::integral_constant<int, 16>{});
}

}  // namespace

extern "C" tq_status tq_kv_append(const tq_kv_pages_t* cache, const void* k, int64_t k_stride, const void* v,
                                  int64_t v_stride, tq_dtype dt, int64_t T, const int32_t* slots,
                                  const tq_rope_t* rope, const int32_t* positions, uint32_t* err, void* stream) {
    const tq_status ok = kv_pages_check(cache, true);
    if (ok != TQ_OK) return ok;
    if (T < 0 || (dt != TQ_F32 && dt != TQ_BF16)) return TQ_ERR_INVALID;
    const int es = dt == TQ_F32 ? 4 : 2;
    const int64_t need = (int64_t)cache->Hkv * kPD;
    if (k_stride < need || v_stride < need || k_stride * es % 16 || v_stride * es % 16) return TQ_ERR_INVALID;
    if (rope) {
        if (!rope_ok(rope) || rope->dim != kPD || !positions) return TQ_ERR_INVALID;
        if (!(rope->rotary == 32 || rope->rotary == 64 || rope->rotary == 128)) return TQ_ERR_UNSUPPORTED;
    }
    if (T == 0) return TQ_OK;
    if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16)) return TQ_ERR_INVALID;
    AppendArgs a{};
    a.c = kv_pages_view(cache);
    a.k = k;
    a.v = v;
    a.ks = k_stride;
    a.vs = v_stride;
    a.T = T;
    a.slots = slots;
    if (rope) {
        a.pos = positions;
        a.steps = rope->steps;
        a.lrot = ilog2(rope->rotary);
        a.interleaved = rope->layout == TQ_ROPE_INTERLEAVED;
        a.factor = rope->factor;
    }
    a.dt = dt;
    a.err = err;
    const int64_t blocks = (T * cache->Hkv + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffll) return TQ_ERR_UNSUPPORTED;
    cudaStream_t st = as_stream(stream);
    return by_books(cache, [&](auto kl, auto vl) {
        kv_append_kernel<decltype(kl)::value, decltype(vl)::value><<<(unsigned)blocks, 32 * kWarps, 0, st>>>(a);
        return launch_status();
    });
}

extern "C" tq_status tq_kv_fetch(const tq_kv_pages_t* cache, const int32_t* slots, int64_t T, void* k, void* v,
                                 tq_dtype dt, uint32_t* err, void* stream) {
    const tq_status ok = kv_pages_check(cache, false);
    if (ok != TQ_OK) return ok;
    if (T < 0 || (dt != TQ_F32 && dt != TQ_BF16 && dt != TQ_F16)) return TQ_ERR_INVALID;
    if (T == 0 || (!k && !v)) return TQ_OK;
    if (!slots || !aligned(k, 16) || !aligned(v, 16)) return TQ_ERR_INVALID;
    FetchArgs a{};
    a.c = kv_pages_view(cache);
    a.slots = slots;
    a.T = T;
    a.k = k;
    a.v = v;
    a.dt = dt;
    a.err = err;
    const int64_t blocks = (T * cache->Hkv + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffll) return TQ_ERR_UNSUPPORTED;
    cudaStream_t st = as_stream(stream);
    return by_books(cache, [&](auto kl, auto vl) {
        kv_fetch_kernel<decltype(kl)::value, decltype(vl)::value><<<(unsigned)blocks, 32 * kWarps, 0, st>>>(a);
        return launch_status();
    });
}
