// The paged compressed cache: argument checks and addressing shared by its write, its
// read and the attention over it.
#pragma once

#include "common.cuh"

namespace tq {

constexpr int kPD = 128;  // head length of the cache
constexpr int64_t kMaxRows = 1ll << 48;    // rows that a cache's strides may span
constexpr int64_t kMaxTokens = 1ll << 40;  // of a call: times the kv heads they fit 63 bits

// Device view of a tq_kv_pages_t.
struct KvPages {
    uint32_t* kcodes;
    uint16_t* kscales;
    uint32_t* vcodes;
    uint16_t* vscales;
    const float* kcent;
    const float* vcent;
    const float* kthr;
    const float* vthr;
    const int8_t* signs;
    int Hkv, lgroup, lpage;  // log2 of group and page
    int64_t pages, page_stride, head_stride;

    // Cache row of a slot (page * page size + offset) and head.
    __device__ __forceinline__ int64_t row(int32_t slot, int h) const {
        return (int64_t)(slot >> lpage) * page_stride + (int64_t)h * head_stride + (slot & ((1 << lpage) - 1));
    }
};

inline tq_status kv_pages_check(const tq_kv_pages_t* c, bool write) {
    if (!c || c->Hkv <= 0 || c->Hkv > 65535 || c->pages < 0) return TQ_ERR_INVALID;
    if (c->D != kPD) return TQ_ERR_UNSUPPORTED;
    if (!(c->group == 16 || c->group == 32 || c->group == 64 || c->group == 128)) return TQ_ERR_INVALID;
    if (!is_pow2(c->page) || c->page < 16 || c->page > 256) return TQ_ERR_INVALID;
    if (c->pages > 0x7fffffffll / c->page) return TQ_ERR_UNSUPPORTED;  // slots are int32
    if (c->page_stride < c->page || c->head_stride < c->page || c->page_stride % 16 || c->head_stride % 16)
        return TQ_ERR_INVALID;
    // rows (and bytes) of the arrays fit 63 bits
    if ((c->pages && c->page_stride > kMaxRows / c->pages) || c->head_stride > kMaxRows / c->Hkv) return TQ_ERR_UNSUPPORTED;
    if (!c->rot.signs || !aligned(c->rot.signs, 16) || c->rot.dim != kPD || c->rot.block != kPD) return TQ_ERR_INVALID;
    if (!c->kcb.centroids || !c->vcb.centroids || (write && (!c->kcb.thresholds || !c->vcb.thresholds)))
        return TQ_ERR_INVALID;
    if (!host_codes_per_word(c->kcb.levels) || !host_codes_per_word(c->vcb.levels)) return TQ_ERR_INVALID;
    if (!(c->kcb.levels == 256 || c->kcb.levels == 16) || !(c->vcb.levels == 8 || c->vcb.levels == 16))
        return TQ_ERR_UNSUPPORTED;
    if (c->pages > 0 && (!c->kcodes || !c->kscales || !c->vcodes || !c->vscales)) return TQ_ERR_INVALID;
    if (!aligned(c->kcodes, 16) || !aligned(c->kscales, 16) || !aligned(c->vcodes, 16) || !aligned(c->vscales, 16))
        return TQ_ERR_INVALID;
    return TQ_OK;
}

inline KvPages kv_pages_view(const tq_kv_pages_t* c) {
    KvPages p{};
    p.kcodes = c->kcodes;
    p.kscales = c->kscales;
    p.vcodes = c->vcodes;
    p.vscales = c->vscales;
    p.kcent = c->kcb.centroids;
    p.vcent = c->vcb.centroids;
    p.kthr = c->kcb.thresholds;
    p.vthr = c->vcb.thresholds;
    p.signs = c->rot.signs;
    p.Hkv = c->Hkv;
    p.lgroup = ilog2(c->group);
    p.lpage = ilog2(c->page);
    p.pages = c->pages;
    p.page_stride = c->page_stride;
    p.head_stride = c->head_stride;
    return p;
}

// Words of a row and codes of a word of a book.
template <int LEVELS>
struct KvBook {
    static constexpr int kBits = LEVELS == 256 ? 8 : (LEVELS == 16 ? 4 : 3);
    static constexpr int kCW = 32 / kBits;
    static constexpr int kWords = (kPD + kCW - 1) / kCW;
};

}  // namespace tq
