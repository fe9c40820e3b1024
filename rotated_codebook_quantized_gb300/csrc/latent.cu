// The paged latent cache: its write, and attention over it in the absorbed form.
#include <math.h>

#include <algorithm>

#include "latent.cuh"
#include "rope.cuh"

namespace tq {
namespace {

// ---------------------------------------------------------------- write

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

// ---------------------------------------------------------------- attention, absorbed

// A warp to a query row, 8 rows of a sequence to a CTA, which read its tokens 16 at a time into shared memory.
constexpr int kTok = 16;
template <bool BF>
__global__ void __launch_bounds__(256) latent_attend_kernel(LatentArgs a) {
    __shared__ uint16_t rows[kTok][kLatentRow];
    __shared__ bool usable[kTok];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.y;
    const int64_t y = (int64_t)blockIdx.x * 8 + warp;
    const int i = (int)(y / a.H), h = (int)(y - (int64_t)i * a.H);
    const bool mine = i < latent_live(a, b);
    const int len = latent_len(a, b), words = (a.n + 63) / 64;
    if (a.err && threadIdx.x == 0 && blockIdx.x == 0 && a.lens[b] != len) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
    float q[18], o[16] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int c = 0; c < 18; ++c)
        q[c] = mine ? from16<BF>(a.q[((int64_t)b * a.n + i) * a.qs + (int64_t)h * kLatentRow + c * 32 + lane]) : 0.f;
    const int total = len + (a.fresh ? a.n : 0);
    for (int t0 = 0; t0 < total; t0 += kTok) {
        __syncthreads();
        for (int t = warp; t < kTok; t += 8) {
            const int at = t0 + t;
            const uint16_t* src = nullptr;
            if (at < len) {
                const int page = a.table[(int64_t)b * a.table_stride + (at >> a.lpage)];
                if ((uint32_t)page < (uint64_t)a.pages)
                    src = a.rows + ((int64_t)page * a.page_stride + (at & ((1 << a.lpage) - 1))) * kLatentRow;
                else if (a.err && lane == 0)
                    atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
            } else if (at < total) {
                src = a.fresh + ((int64_t)b * a.n + at - len) * a.fs;
            }
            if (lane == 0) usable[t] = src != nullptr;
            if (src)
                for (int c = lane; c < kLatentRow; c += 32) rows[t][c] = src[c];
        }
        __syncthreads();
        for (int t = 0; t < kTok && t0 + t < total; ++t) {
            bool see = mine && usable[t];
            const int j = t0 + t - len;
            if (see && j >= 0) see = a.mask ? (a.mask[((int64_t)b * a.n + i) * words + (j >> 6)] >> (j & 63)) & 1 : j <= i;
            if (!see) continue;
            float s = 0.f;
            bool odd = false;
#pragma unroll
            for (int c = 0; c < 18; ++c) {
                const float x = from16<BF>(rows[t][c * 32 + lane]);
                odd |= !isfinite(x);
                s = fmaf(q[c], x, s);
            }
#pragma unroll
            for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(kFull, s, k);
            s *= a.scale2;
            if (__any_sync(kFull, odd)) s = NAN;
            const float n = fmaxf(m, s), r = m == n ? 1.f : exp2f(m - n), p = s == -INFINITY ? 0.f : s == s ? exp2f(s - n) : NAN;
            m = n;
            l = l * r + p;
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] = fmaf(p, from16<BF>(rows[t][c * 32 + lane]), o[c] * r);
        }
    }
    if (i < a.n)
#pragma unroll
        for (int c = 0; c < 16; ++c)
            a.o[(((int64_t)b * a.n + i) * a.H + h) * kLatent + c * 32 + lane] = to16<BF>(l == 0.f ? 0.f : o[c] / l);
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

extern "C" size_t tq_latent_attend_tree_workspace_bytes(const tq_latent_pages_t* cache, int32_t B, int32_t n, int32_t H,
                                                        int64_t max_len) {
    if (latent_check(cache) != TQ_OK || B <= 0 || n <= 0 || H <= 0 || H > 65535 || max_len < 0) return 0;
    return 16;
}

extern "C" tq_status tq_latent_attend_tree(const tq_latent_pages_t* cache, const void* q, int64_t q_stride, int32_t B, int32_t n,
                                           int32_t H, const int32_t* table, int32_t table_stride, const int32_t* lens,
                                           int64_t max_len, const void* fresh, int64_t fresh_stride, const uint64_t* mask,
                                           const int32_t* n_tok, float scale, void* o, void* ws, size_t ws_bytes, uint32_t* err,
                                           void* stream) {
    const tq_status s = latent_check(cache);
    if (s != TQ_OK) return s;
    if (B < 0 || n < 0 || H <= 0 || H > 65535 || table_stride < 0 || max_len < 0 || !isfinite(scale)) return TQ_ERR_INVALID;
    if (max_len > (int64_t)table_stride * cache->page) return TQ_ERR_INVALID;
    if (q_stride < (int64_t)H * kLatentRow || q_stride % 8 || (fresh && (fresh_stride < kLatentRow || fresh_stride % 8)))
        return TQ_ERR_INVALID;
    if (B == 0 || n == 0) return TQ_OK;
    const size_t need = tq_latent_attend_tree_workspace_bytes(cache, B, n, H, max_len);
    if (!need || (int64_t)B * n > (1ll << 30) / H) return TQ_ERR_UNSUPPORTED;
    if (q_stride > 1ll << 40 || fresh_stride > 1ll << 40) return TQ_ERR_UNSUPPORTED;
    if (!q || !o || !lens || (max_len && !table) || !ws || ws_bytes < need) return TQ_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(fresh, 16) || !aligned(ws, 16) || !aligned(mask, 8) || !aligned(table, 4) ||
        !aligned(lens, 4) || !aligned(n_tok, 4))
        return TQ_ERR_INVALID;
    LatentArgs a{};
    a.rows = reinterpret_cast<const uint16_t*>(cache->rows);
    a.q = reinterpret_cast<const uint16_t*>(q);
    a.fresh = reinterpret_cast<const uint16_t*>(fresh);
    a.qs = q_stride;
    a.fs = fresh_stride;
    a.pages = cache->pages;
    a.page_stride = cache->page_stride;
    a.max_len = max_len;
    a.table = table;
    a.lens = lens;
    a.mask = mask;
    a.n_tok = n_tok;
    a.B = B;
    a.n = n;
    a.H = H;
    a.table_stride = table_stride;
    a.lpage = ilog2(cache->page);
    a.scale2 = scale * 1.4426950408889634f;
    a.o = reinterpret_cast<uint16_t*>(o);
    a.err = err;
    const dim3 grid((unsigned)(((int64_t)n * H + 7) / 8), (unsigned)B);
    if (cache->dt == TQ_BF16) latent_attend_kernel<true><<<grid, 256, 0, as_stream(stream)>>>(a);
    else latent_attend_kernel<false><<<grid, 256, 0, as_stream(stream)>>>(a);
    return launch_status();
}
