// The write of the paged latent cache.
#include <algorithm>

#include "latent.cuh"
#include "rope.cuh"

namespace tq {
namespace {

// Eight elements of 16 or 32 bits as floats.
template <int DT>
TQ_DEVFN void load8(const void* p, int64_t at, float (&v)[8]) {
    if (DT == TQ_F32) {
        const float4* s = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at);
        const float4 x = s[0], y = s[1];
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    } else {
        const uint4 x = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + at);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = from16<DT == TQ_BF16>((uint16_t)w[i]);
            v[2 * i + 1] = from16<DT == TQ_BF16>((uint16_t)(w[i] >> 16));
        }
    }
}

struct AppendArgs {
    const void* c;
    const void* k;
    int64_t cs, ks, T, pages, page_stride;
    const int32_t* slots;
    const int32_t* positions;
    uint4* rows;
    uint32_t* err;
    int lpage;
    tq_rope_t rope;  // steps NULL: none
};

// A thread to 8 elements of a row (16 bytes of the cache); bound by HBM for a prompt, by the launch for a step.
constexpr int kPieces = kLatentRow / 8, kLatentPieces = kLatent / 8;
template <int DT, bool BF>
__global__ void __launch_bounds__(256) latent_append_kernel(AppendArgs a) {
    pdl_trigger();
    pdl_wait();
    const int64_t total = a.T * kPieces, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t t = i / kPieces;
        const int piece = (int)(i - t * kPieces);
        const int slot = a.slots[t];
        if (slot < 0) continue;
        if ((slot >> a.lpage) >= a.pages) {
            if (piece == 0 && a.err) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
            continue;
        }
        float v[8];
        if (piece < kLatentPieces) {
            load8<DT>(a.c, t * a.cs + piece * 8, v);
        } else {
            const int e0 = (piece - kLatentPieces) * 8;
            load8<DT>(a.k, t * a.ks + e0, v);
            if (a.rope.steps) {
                const int rotary = a.rope.rotary, half = rotary >> 1, pos = a.positions[t];
                if (a.rope.layout == TQ_ROPE_INTERLEAVED) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        if (e0 + e >= rotary) break;
                        float sn, cs;
                        rope_angle(pos, a.rope.steps[(e0 + e) >> 1], sn, cs);
                        const float x = v[e], y = v[e + 1];
                        v[e] = a.rope.factor * (x * cs - y * sn);
                        v[e + 1] = a.rope.factor * (x * sn + y * cs);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int at = e0 + e;
                        if (at >= rotary) break;
                        const bool low = at < half;
                        const float other = load_as_float(a.k, t * a.ks + (low ? at + half : at - half), DT);
                        float sn, cs;
                        rope_angle(pos, a.rope.steps[low ? at : at - half], sn, cs);
                        v[e] = a.rope.factor * (low ? v[e] * cs - other * sn : other * sn + v[e] * cs);
                    }
                }
            }
        }
        const int64_t row = (int64_t)(slot >> a.lpage) * a.page_stride + (slot & ((1 << a.lpage) - 1));
        a.rows[row * kPieces + piece] =
            make_uint4(pack16<BF>(v[0], v[1]), pack16<BF>(v[2], v[3]), pack16<BF>(v[4], v[5]), pack16<BF>(v[6], v[7]));
    }
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" tq_status tq_latent_append(const tq_latent_pages_t* cache, const void* c, int64_t c_stride, const void* k_rope,
                                      int64_t k_stride, tq_dtype dt, int64_t T, const int32_t* slots, const tq_rope_t* rope,
                                      const int32_t* positions, uint32_t* err, void* stream) {
    const tq_status s = latent_check(cache);
    if (s != TQ_OK) return s;
    if (T < 0 || !(dt == TQ_F32 || dt == TQ_BF16 || dt == TQ_F16)) return TQ_ERR_INVALID;
    if (T > 1ll << 40) return TQ_ERR_UNSUPPORTED;
    const int piece = dt == TQ_F32 ? 4 : 8;
    if (c_stride < kLatent || k_stride < kLatentRope || c_stride % piece || k_stride % piece) return TQ_ERR_INVALID;
    if (c_stride > 1ll << 40 || k_stride > 1ll << 40 || (T && std::max(c_stride, k_stride) > (1ll << 60) / T)) return TQ_ERR_UNSUPPORTED;
    if (rope && (!rope_ok(rope) || rope->dim != kLatentRope)) return TQ_ERR_INVALID;
    if (T == 0) return TQ_OK;
    if (!c || !k_rope || !slots || (rope && !positions)) return TQ_ERR_INVALID;
    if (!aligned(c, 16) || !aligned(k_rope, 16) || !aligned(slots, 4) || !aligned(positions, 4)) return TQ_ERR_INVALID;
    AppendArgs a{};
    a.c = c;
    a.k = k_rope;
    a.cs = c_stride;
    a.ks = k_stride;
    a.T = T;
    a.pages = cache->pages;
    a.page_stride = cache->page_stride;
    a.slots = slots;
    a.positions = positions;
    a.rows = reinterpret_cast<uint4*>(cache->rows);
    a.err = err;
    a.lpage = ilog2(cache->page);
    if (rope) a.rope = *rope;
    const unsigned grid = (unsigned)std::min<int64_t>((T * kPieces + 255) / 256, 152 * 16);
    const bool bf = cache->dt == TQ_BF16;
    void (*kernel)(AppendArgs) =
        dt == TQ_F32 ? (bf ? latent_append_kernel<TQ_F32, true> : latent_append_kernel<TQ_F32, false>)
        : dt == TQ_BF16 ? (bf ? latent_append_kernel<TQ_BF16, true> : latent_append_kernel<TQ_BF16, false>)
                        : (bf ? latent_append_kernel<TQ_F16, true> : latent_append_kernel<TQ_F16, false>);
    return launch_pdl(kernel, dim3(grid), dim3(256), 0, as_stream(stream), a);
}
