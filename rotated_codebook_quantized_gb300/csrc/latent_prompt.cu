// Attention of prompts over keys and values expanded from the latents.
#include <math.h>

#include "latent.cuh"

namespace tq {
namespace {

struct PromptArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* kr;
    int64_t qs, kvs, kvh, krs, Tq, Tkv;
    const int32_t* q_starts;
    const int32_t* kv_starts;
    uint16_t* o;
    uint32_t* err;
    int B, H;
    bool causal;
    float scale2;
};

// A warp to a query row, 8 rows to a CTA, which read keys and values 16 at a time into shared memory.
constexpr int kTok = 16;
template <bool BF>
__global__ void __launch_bounds__(256) latent_prompt_kernel(PromptArgs a) {
    __shared__ uint16_t ks[kTok][kHeadQuery], vs[kTok][kHeadValue];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
    const int64_t t0 = (int64_t)blockIdx.x * 8;
    for (int b = 0; b < a.B; ++b) {
        const int64_t q0 = a.q_starts[b], q1 = a.q_starts[b + 1], k0 = a.kv_starts[b], k1 = a.kv_starts[b + 1];
        if (q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tkv) {
            if (a.err && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
            continue;
        }
        if (q1 <= t0 || q0 >= t0 + 8) continue;
        const int64_t t = t0 + warp;
        const bool mine = t >= q0 && t < q1;
        const int64_t upto = a.causal ? t - q1 + k1 + 1 : k1, most = a.causal ? min(t0 + 8, q1) - q1 + k1 : k1;
        float q[6], o[4] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
        for (int c = 0; c < 6; ++c) q[c] = mine ? from16<BF>(a.q[t * a.qs + (int64_t)h * kHeadQuery + c * 32 + lane]) : 0.f;
        for (int64_t j0 = k0; j0 < most; j0 += kTok) {
            __syncthreads();
            for (int j = warp; j < kTok && j0 + j < most; j += 8) {
                const int64_t at = (j0 + j) * a.kvs + h * a.kvh;
                for (int c = lane; c < kHeadKey; c += 32) {
                    ks[j][c] = a.k[at + c];
                    vs[j][c] = a.v[at + c];
                }
                for (int c = lane; c < kLatentRope; c += 32) ks[j][kHeadKey + c] = a.kr[(j0 + j) * a.krs + c];
            }
            __syncthreads();
            for (int j = 0; j < kTok && mine && j0 + j < min(upto, most); ++j) {
                float s = 0.f;
#pragma unroll
                for (int c = 0; c < 6; ++c) s = fmaf(q[c], from16<BF>(ks[j][c * 32 + lane]), s);
#pragma unroll
                for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(kFull, s, k);
                s *= a.scale2;
                bool odd = false;
#pragma unroll
                for (int c = 0; c < 4; ++c) odd |= !isfinite(from16<BF>(vs[j][c * 32 + lane]));
                if (__any_sync(kFull, odd)) s = NAN;
                const float n = fmaxf(m, s), r = m == n ? 1.f : exp2f(m - n), p = s == -INFINITY ? 0.f : s == s ? exp2f(s - n) : NAN;
                m = n;
                l = l * r + p;
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] = fmaf(p, from16<BF>(vs[j][c * 32 + lane]), o[c] * r);
            }
        }
        if (mine)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                a.o[(t * a.H + h) * kHeadValue + c * 32 + lane] = to16<BF>(l == 0.f ? 0.f : o[c] / l);
    }
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" tq_status tq_latent_attend_prompt(const void* q, int64_t q_stride, const void* k, const void* v, int64_t kv_stride,
                                             int64_t kv_head_stride, const void* k_rope, int64_t k_rope_stride, tq_dtype dt,
                                             int32_t B, int32_t H, int64_t Tq, int64_t Tkv, const int32_t* q_starts,
                                             const int32_t* kv_starts, int32_t causal, float scale, void* o, uint32_t* err,
                                             void* stream) {
    if (B < 0 || H <= 0 || H > 65535 || Tq < 0 || Tkv < 0 || !isfinite(scale)) return TQ_ERR_INVALID;
    if (!(dt == TQ_BF16 || dt == TQ_F16 || dt == TQ_F32)) return TQ_ERR_INVALID;
    if (dt == TQ_F32 || Tq > 1ll << 30 || Tkv > 1ll << 30) return TQ_ERR_UNSUPPORTED;
    if (q_stride < (int64_t)H * kHeadQuery || kv_head_stride < kHeadKey || kv_stride < (H - 1) * kv_head_stride + kHeadKey ||
        k_rope_stride < kLatentRope || q_stride % 8 || kv_stride % 8 || kv_head_stride % 8 || k_rope_stride % 8)
        return TQ_ERR_INVALID;
    if (q_stride > 1ll << 32 || kv_stride > 1ll << 32 || k_rope_stride > 1ll << 32) return TQ_ERR_UNSUPPORTED;
    if (B == 0 || Tq == 0) return TQ_OK;
    if (!q || !o || !q_starts || !kv_starts || (Tkv && (!k || !v || !k_rope))) return TQ_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_rope, 16) || !aligned(o, 16) || !aligned(q_starts, 4) ||
        !aligned(kv_starts, 4))
        return TQ_ERR_INVALID;
    PromptArgs a{};
    a.q = reinterpret_cast<const uint16_t*>(q);
    a.k = reinterpret_cast<const uint16_t*>(k);
    a.v = reinterpret_cast<const uint16_t*>(v);
    a.kr = reinterpret_cast<const uint16_t*>(k_rope);
    a.qs = q_stride;
    a.kvs = kv_stride;
    a.kvh = kv_head_stride;
    a.krs = k_rope_stride;
    a.Tq = Tq;
    a.Tkv = Tkv;
    a.q_starts = q_starts;
    a.kv_starts = kv_starts;
    a.o = reinterpret_cast<uint16_t*>(o);
    a.err = err;
    a.B = B;
    a.H = H;
    a.causal = causal != 0;
    a.scale2 = scale * 1.4426950408889634f;
    const dim3 grid((unsigned)((Tq + 7) / 8), (unsigned)H);
    if (dt == TQ_BF16) latent_prompt_kernel<true><<<grid, 256, 0, as_stream(stream)>>>(a);
    else latent_prompt_kernel<false><<<grid, 256, 0, as_stream(stream)>>>(a);
    return launch_status();
}
