// Attention of a tree of drafted tokens over the paged compressed cache: tq_kv_attend_tree.
//
// o = softmax(scale * q K^T) V over a sequence's cached tokens and, through an ancestor
// mask, over the drafted tokens.  As in tq_kv_attend the rotation moves off the cache:
// q . k = (R q) . (R k), and sum_t p_t v_t = R^T sum_t p_t (R v_t), one de-rotation per row.
// The drafted tokens come as they are (bf16, not rotated), so their part is a partial
// result of its own, added after the de-rotation.
#include <math.h>

#include "common.cuh"
#include "kv_pages.cuh"

using namespace tq;

namespace {

constexpr int kChunk = 512;  // cached tokens per CTA
constexpr float kLog2e = 1.4426950408889634f;

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
    int B, n, Hq, table_stride, splits;  // splits: of the context; one more partial for the drafts
    float scale2;                        // scale * log2(e)
    __nv_bfloat16* o;
    float* part;  // [row][splits + 1][2 + 128]: (max, sum, weighted values)
    uint32_t* err;
};

// One CTA (4 warps) per row and context chunk; the last chunk index is the drafts.
template <int KL, int VL>
__global__ void __launch_bounds__(128) kv_tree_kernel(TreeArgs a) {
    __shared__ float kl[KL], vl[VL], qr[kPD], sc[kChunk], red[4];
    __shared__ int64_t rows[kChunk];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t r = blockIdx.x;
    const int hq = (int)(r % a.Hq), i = (int)(r / a.Hq % a.n), b = (int)(r / a.Hq / a.n);
    const int h = hq / (a.Hq / a.c.Hkv), split = blockIdx.y;
    float* dst = a.part + (r * (a.splits + 1) + split) * (2 + kPD);
    const int live = a.n_tok ? a.n_tok[b] : a.n;
    const bool drafts = split == a.splits;
    int64_t len = a.lens[b];
    if (len < 0 || len > a.max_len) {
        if (tid == 0 && a.err) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
        len = len < 0 ? 0 : a.max_len;
    }
    const int64_t t0 = (int64_t)split * kChunk;
    const int64_t end = drafts ? (a.kn ? a.n : 0) : min(len, t0 + kChunk);
    float m = -INFINITY, l = 0.f, acc = 0.f;
    if (i < live && (drafts ? end > 0 : t0 < end)) {
        for (int x = tid; x < KL; x += 128) kl[x] = a.c.kcent[x];
        for (int x = tid; x < VL; x += 128) vl[x] = a.c.vcent[x];
        const __nv_bfloat16* q = a.q + ((int64_t)b * a.n + i) * a.qs + (int64_t)hq * kPD;
        if (drafts) {
            qr[tid] = __bfloat162float(q[tid]) * a.scale2;
        } else if (warp == 0) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __bfloat162float(q[lane * 4 + e]) * (float)a.c.signs[lane * 4 + e];
            fwht_warp128(v);
#pragma unroll
            for (int e = 0; e < 4; ++e) qr[lane * 4 + e] = v[e] * (0.08838834764831845f * a.scale2);
        }
        __syncthreads();
        for (int64_t base = drafts ? 0 : t0; base < end; base += kChunk) {  // the drafts may take several rounds
            const int cnt = (int)min((int64_t)kChunk, end - base);
            for (int x = tid; x < cnt; x += 128) {
                const int64_t t = base + x;
                float s = -INFINITY;
                if (drafts) {
                    const bool see = t < live && (a.mask ? (a.mask[((int64_t)b * a.n + i) * ((a.n + 63) / 64) + t / 64] >> (t % 64)) & 1 : t <= i);
                    if (see) {
                        const __nv_bfloat16* k = a.kn + ((int64_t)b * a.n + t) * a.ks + (int64_t)h * kPD;
                        s = 0.f;
                        for (int d = 0; d < kPD; ++d) s = fmaf(qr[d], __bfloat162float(k[d]), s);
                    }
                } else {
                    const int page = a.table[(int64_t)b * a.table_stride + (t >> a.c.lpage)];
                    rows[x] = -1;
                    if (page >= 0 && page < a.c.pages) {
                        const int64_t row = (int64_t)page * a.c.page_stride + (int64_t)h * a.c.head_stride + (t & ((1 << a.c.lpage) - 1));
                        rows[x] = row;
                        const uint32_t* w = a.c.kcodes + row * KvBook<KL>::kWords;
                        const uint16_t* z = a.c.kscales + (row << (7 - a.c.lgroup));
                        s = 0.f;
                        for (int d = 0; d < kPD; ++d) {
                            const uint32_t c = (w[d / KvBook<KL>::kCW] >> (KvBook<KL>::kBits * (d % KvBook<KL>::kCW))) & (KL - 1);
                            s = fmaf(qr[d], kl[c] * half_bits_to_float(z[d >> a.c.lgroup]), s);
                        }
                    } else if (a.err) {
                        atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
                    }
                }
                sc[x] = s;
            }
            __syncthreads();
            float mx = -INFINITY;
            for (int x = lane; x < cnt; x += 32) mx = mx != mx ? mx : (sc[x] != sc[x] ? sc[x] : fmaxf(mx, sc[x]));
            for (int o = 16; o; o >>= 1) {
                const float y = __shfl_xor_sync(kFull, mx, o);
                mx = mx != mx ? mx : (y != y ? y : fmaxf(mx, y));
            }
            if (!(mx == -INFINITY)) {
                const float nm = mx != mx || m != m ? NAN : fmaxf(m, mx), f = m == -INFINITY ? 0.f : exp2f(m - nm);
                acc *= f;
                l *= f;
                m = nm;
                float sum = 0.f;
                for (int x = 0; x < cnt; ++x) {
                    const float p = sc[x] == -INFINITY ? 0.f : exp2f(sc[x] - nm);
                    if (sc[x] == -INFINITY) continue;  // not seen: its value never enters
                    sum += p;
                    if (drafts) {
                        acc = fmaf(p, __bfloat162float(a.vn[((int64_t)b * a.n + base + x) * a.vs + (int64_t)h * kPD + tid]), acc);
                    } else if (rows[x] >= 0) {
                        const uint32_t w = a.c.vcodes[rows[x] * KvBook<VL>::kWords + tid / KvBook<VL>::kCW];
                        const uint32_t c = (w >> (KvBook<VL>::kBits * (tid % KvBook<VL>::kCW))) & (VL - 1);
                        acc = fmaf(p, vl[c] * half_bits_to_float(a.c.vscales[(rows[x] << (7 - a.c.lgroup)) + (tid >> a.c.lgroup)]), acc);
                    }
                }
                l += sum;
            }
            __syncthreads();
        }
    }
    if (tid == 0) {
        dst[0] = m;
        dst[1] = l;
    }
    dst[2 + tid] = acc;
}

// Joins the partial results of a row: the context's, de-rotated, and the drafts'.  One warp per row.
__global__ void __launch_bounds__(128) kv_tree_join_kernel(TreeArgs a) {
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (r >= (int64_t)a.B * a.n * a.Hq) return;
    const int lane = threadIdx.x & 31;
    const float* p = a.part + r * (a.splits + 1) * (2 + kPD);
    float M = -INFINITY;
    bool bad = false;
    for (int s = 0; s <= a.splits; ++s) {
        const float m = p[s * (2 + kPD)];
        bad |= m != m;
        M = fmaxf(M, m);
    }
    float L = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s <= a.splits; ++s) {
        const float* x = p + s * (2 + kPD);
        if (x[0] == -INFINITY) continue;
        const float f = exp2f(x[0] - M);
        L = fmaf(f, x[1], L);
#pragma unroll
        for (int e = 0; e < 4; ++e) (s == a.splits ? d : v)[e] = fmaf(f, x[2 + lane * 4 + e], (s == a.splits ? d : v)[e]);
    }
    fwht_warp128(v);
    const float inv = bad ? NAN : (L > 0.f ? 1.0f / L : (L == 0.f ? 0.f : NAN));
#pragma unroll
    for (int e = 0; e < 4; ++e)
        a.o[r * kPD + lane * 4 + e] =
            __float2bfloat16_rn((v[e] * 0.08838834764831845f * (float)a.c.signs[lane * 4 + e] + d[e]) * inv);
}

int64_t context_splits(int64_t max_len) { return (max_len + kChunk - 1) / kChunk; }

}  // namespace

extern "C" size_t tq_kv_attend_tree_workspace_bytes(const tq_kv_pages_t* cache, int32_t B, int32_t n, int32_t Hq,
                                                    int64_t max_len) {
    if (kv_pages_check(cache, false) != TQ_OK || B <= 0 || n <= 0 || Hq <= 0 || max_len < 0) return 0;
    return (size_t)B * n * Hq * (context_splits(max_len) + 1) * (2 + kPD) * sizeof(float);
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
        !aligned(mask, 8))
        return TQ_ERR_INVALID;
    if (ws_bytes < tq_kv_attend_tree_workspace_bytes(cache, B, n, Hq, max_len)) return TQ_ERR_INVALID;
    const int64_t rows = (int64_t)B * n * Hq, splits = context_splits(max_len);
    if (rows > 0x7fffffffll || splits > 65534) return TQ_ERR_UNSUPPORTED;
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
    a.table_stride = table_stride;
    a.splits = (int)splits;
    a.scale2 = scale * kLog2e;
    a.o = static_cast<__nv_bfloat16*>(o);
    a.part = static_cast<float*>(ws);
    a.err = err;
    cudaStream_t st = as_stream(stream);
    const dim3 grid((unsigned)rows, (unsigned)splits + 1);
    if (cache->kcb.levels == 256 && cache->vcb.levels == 8) kv_tree_kernel<256, 8><<<grid, 128, 0, st>>>(a);
    else if (cache->kcb.levels == 256) kv_tree_kernel<256, 16><<<grid, 128, 0, st>>>(a);
    else if (cache->vcb.levels == 8) kv_tree_kernel<16, 8><<<grid, 128, 0, st>>>(a);
    else kv_tree_kernel<16, 16><<<grid, 128, 0, st>>>(a);
    const tq_status s = launch_status();
    if (s != TQ_OK) return s;
    kv_tree_join_kernel<<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(a);
    return launch_status();
}
