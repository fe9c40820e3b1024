// The paged latent cache: argument checks and addressing shared by its write and the attention over it.
#pragma once

#include "common.cuh"

namespace tq {

constexpr int kLatent = 512, kLatentRope = 64, kLatentRow = kLatent + kLatentRope;
constexpr int kHeadKey = 128, kHeadQuery = kHeadKey + kLatentRope, kHeadValue = 128;  // of the expanded form

inline tq_status latent_check(const tq_latent_pages_t* c) {
    if (!c || c->pages < 0 || !(c->dt == TQ_BF16 || c->dt == TQ_F16 || c->dt == TQ_F32)) return TQ_ERR_INVALID;
    if (c->latent != kLatent || c->rope != kLatentRope || c->dt == TQ_F32) return TQ_ERR_UNSUPPORTED;
    if (!is_pow2(c->page) || c->page < 16 || c->page > 256) return TQ_ERR_INVALID;
    if (c->page_stride < c->page) return TQ_ERR_INVALID;
    // slots and rows are int32 (a tensor copy's coordinate)
    if (c->pages > 0x7fffffffll / c->page || (c->pages && c->page_stride > 0x7fffffffll / c->pages)) return TQ_ERR_UNSUPPORTED;
    if ((c->pages && !c->rows) || !aligned(c->rows, 16)) return TQ_ERR_INVALID;
    return TQ_OK;
}

template <bool BF>
TQ_DEVFN float from16(uint16_t x) {
    return BF ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x));
}
template <bool BF>
TQ_DEVFN uint32_t pack16(float lo, float hi) {
    if (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool BF>
TQ_DEVFN uint16_t to16(float x) {
    return BF ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

struct LatentArgs {
    const uint16_t* rows;
    const uint16_t* q;
    const uint16_t* fresh;
    int64_t qs, fs, pages, page_stride, max_len;
    const int32_t* table;
    const int32_t* lens;
    const uint64_t* mask;
    const int32_t* n_tok;
    int B, n, H, table_stride, lpage;
    float scale2;  // scale * log2(e)
    uint16_t* o;
    uint32_t* err;
};
TQ_DEVFN int latent_len(const LatentArgs& a, int b) {
    const int len = a.lens[b];
    return len < 0 ? 0 : (int)min((int64_t)len, a.max_len);
}
TQ_DEVFN int latent_live(const LatentArgs& a, int b) { return a.n_tok ? min(max(a.n_tok[b], 0), a.n) : a.n; }

}  // namespace tq
