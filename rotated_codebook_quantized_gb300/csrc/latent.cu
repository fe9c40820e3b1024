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

// A warp to N tokens at a time, all of whose loads it has on their way: a lane to 16 of a latent vector's elements and to a pair of the
// rotary key's, so that every lane has one sine and cosine a token.  (16-byte pieces dealt to threads one after another left those of
// the rotary keys, four sines each, to an eighth of them: 48 us for 65536 tokens.)
template <int DT, bool BF, int N>
__global__ void __launch_bounds__(256) latent_append_kernel(AppendArgs a) {
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    // the lane's two elements of the rotary key
    const bool turned = a.rope.steps && lane < a.rope.rotary / 2;
    int e0 = 2 * lane, e1 = e0 + 1;
    if (a.rope.steps && a.rope.layout == TQ_ROPE_HALF && turned) e0 = lane, e1 = lane + a.rope.rotary / 2;
    pdl_wait();
    const uint64_t step = turned ? a.rope.steps[lane] : 0;
    const int64_t warps = (int64_t)gridDim.x * 8;
    for (int64_t t0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * N; t0 < a.T; t0 += warps * N) {
        int slot[N], pos[N];
        Eight<DT> c[N][2];
        float x[N], y[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t t = min(t0 + i, a.T - 1);
            slot[i] = t0 + i < a.T ? a.slots[t] : -1;
            pos[i] = a.rope.steps ? a.positions[t] : 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) c[i][h].load(a.c, t * a.cs + h * 256 + lane * 8);
            x[i] = load_as_float(a.k, t * a.ks + e0, DT);
            y[i] = load_as_float(a.k, t * a.ks + e1, DT);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (slot[i] < 0) continue;
            if ((slot[i] >> a.lpage) >= a.pages) {
                if (lane == 0 && a.err) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
                continue;
            }
            const int64_t row = (int64_t)(slot[i] >> a.lpage) * a.page_stride + (slot[i] & ((1 << a.lpage) - 1));
            uint16_t* const to = reinterpret_cast<uint16_t*>(a.rows) + row * kLatentRow;
#pragma unroll
            for (int h = 0; h < 2; ++h) *reinterpret_cast<uint4*>(to + h * 256 + lane * 8) = c[i][h].template packed<BF>();
            float u = x[i], v = y[i];
            if (turned) {
                float sn, cs;
                rope_angle(pos[i], step, sn, cs);
                u = a.rope.factor * (x[i] * cs - y[i] * sn);
                v = a.rope.factor * (x[i] * sn + y[i] * cs);
            }
            if (e1 == e0 + 1 && !(e0 & 1)) {
                *reinterpret_cast<uint32_t*>(to + kLatent + e0) = pack16<BF>(u, v);
            } else {
                to[kLatent + e0] = to16<BF>(u);
                to[kLatent + e1] = to16<BF>(v);
            }
        }
    }
}

template <int DT>
void (*append_of(bool bf, bool many))(AppendArgs) {
    if (bf) return many ? latent_append_kernel<DT, true, 4> : latent_append_kernel<DT, true, 1>;
    return many ? latent_append_kernel<DT, false, 4> : latent_append_kernel<DT, false, 1>;
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
    // four tokens a warp hide the loads' latency where there are warps enough; fewer tokens go one to a warp
    const bool many = T >= 8192, bf = cache->dt == TQ_BF16;
    const int64_t warps = many ? (T + 3) / 4 : T;
    const unsigned grid = (unsigned)std::min<int64_t>((warps + 7) / 8, 152 * 8);
    void (*kernel)(AppendArgs) =
        dt == TQ_F32 ? append_of<TQ_F32>(bf, many) : dt == TQ_BF16 ? append_of<TQ_BF16>(bf, many) : append_of<TQ_F16>(bf, many);
    return launch_pdl(kernel, dim3(grid), dim3(256), 0, as_stream(stream), a);
}
