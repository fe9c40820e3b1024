// The write of the paged latent cache.
#include <algorithm>

#include "latent.cuh"
#include "rope.cuh"

namespace tq {
namespace {

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

// Eight elements, asked for now and converted later.
template <int DT>
struct Eight {
    uint4 w[DT == TQ_F32 ? 2 : 1];
    TQ_DEVFN void load(const void* p, int64_t at) {
        const uint4* s = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) + at * (DT == TQ_F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (DT == TQ_F32 ? 2 : 1); ++i) w[i] = __ldcs(s + i);
    }
    template <bool BF>
    TQ_DEVFN uint4 packed() const {
        if (DT == (BF ? TQ_BF16 : TQ_F16)) return w[0];  // the cache's own type
        float v[8];
        if (DT == TQ_F32) {
            const uint32_t x[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[DT == TQ_F32].x, w[DT == TQ_F32].y, w[DT == TQ_F32].z, w[DT == TQ_F32].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(x[i]);
        } else {
            const uint32_t x[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = from16<DT == TQ_BF16>((uint16_t)x[i]);
                v[2 * i + 1] = from16<DT == TQ_BF16>((uint16_t)(x[i] >> 16));
            }
        }
        return make_uint4(pack16<BF>(v[0], v[1]), pack16<BF>(v[2], v[3]), pack16<BF>(v[4], v[5]), pack16<BF>(v[6], v[7]));
    }
};

// A warp to a token, a lane to 16 of its latent vector's elements and to a pair of its rotary key's, so that every lane has one sine and
// cosine.  (16-byte pieces dealt to threads one after another left those of the rotary keys, four sines each, to an eighth of
// them.)  Bound by HBM: 65536 tokens 27.8 us, 5.5 TB/s, where tokens and rows are others at each call, and 24 us over the same ones again,
// part of which the L2 cache still holds (there pieces took 48 us; four tokens to a warp at a time 23.3, and 10.0 for 8.5 over 32768
// tokens).  48 tokens: 1.5 us, the launch.
template <int DT, bool BF>
__global__ void __launch_bounds__(256) latent_append_kernel(AppendArgs a) {
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    // the lane's two elements of the rotary key
    const bool turned = a.rope.steps && lane < a.rope.rotary / 2;
    int e0 = 2 * lane, e1 = e0 + 1;
    if (a.rope.layout == TQ_ROPE_HALF && turned) e0 = lane, e1 = lane + a.rope.rotary / 2;
    pdl_wait();
    const uint64_t step = turned ? a.rope.steps[lane] : 0;
    for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < a.T; t += (int64_t)gridDim.x * 8) {
        const int slot = a.slots[t], pos = a.rope.steps ? a.positions[t] : 0;
        Eight<DT> c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) c[h].load(a.c, t * a.cs + h * 256 + lane * 8);
        const float x = load_as_float(a.k, t * a.ks + e0, DT), y = load_as_float(a.k, t * a.ks + e1, DT);
        if (slot < 0) continue;
        if ((slot >> a.lpage) >= a.pages) {
            if (lane == 0 && a.err) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
            continue;
        }
        const int64_t row = (int64_t)(slot >> a.lpage) * a.page_stride + (slot & ((1 << a.lpage) - 1));
        uint16_t* const to = reinterpret_cast<uint16_t*>(a.rows) + row * kLatentRow;
#pragma unroll
        for (int h = 0; h < 2; ++h) *reinterpret_cast<uint4*>(to + h * 256 + lane * 8) = c[h].template packed<BF>();
        float u = x, v = y;
        if (turned) {
            float sn, cs;
            rope_angle(pos, step, sn, cs);
            u = a.rope.factor * (x * cs - y * sn);
            v = a.rope.factor * (x * sn + y * cs);
        }
        if (e1 == e0 + 1 && !(e0 & 1)) {
            *reinterpret_cast<uint32_t*>(to + kLatent + e0) = pack16<BF>(u, v);
        } else {
            to[kLatent + e0] = to16<BF>(u);
            to[kLatent + e1] = to16<BF>(v);
        }
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
    const unsigned grid = (unsigned)std::min<int64_t>((T + 7) / 8, device_sms() * 8);
    const bool bf = cache->dt == TQ_BF16;
    void (*kernel)(AppendArgs) =
        dt == TQ_F32 ? (bf ? latent_append_kernel<TQ_F32, true> : latent_append_kernel<TQ_F32, false>)
        : dt == TQ_BF16 ? (bf ? latent_append_kernel<TQ_BF16, true> : latent_append_kernel<TQ_BF16, false>)
                        : (bf ? latent_append_kernel<TQ_F16, true> : latent_append_kernel<TQ_F16, false>);
    return launch_pdl(kernel, dim3(grid), dim3(256), 0, as_stream(stream), a);
}
