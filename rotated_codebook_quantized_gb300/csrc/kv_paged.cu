// The paged compressed KV cache written and read back: tq_kv_append, tq_kv_fetch.
//
// "How it works", "The KV cache", and "Running a 1T-Parameter Model on a Laptop",
// update_and_fetch: rotate, quantize, store; dequantize, de-rotate.  The arithmetic of a
// vector is tq_kv_quantize's; a token's row is found through its slot.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "kv_pages.cuh"
#include "rope.cuh"

using namespace tq;

namespace {

// Both kernels: four lanes to a (token, kv head), key and value together; a warp takes eight consecutive tokens of a
// head, so that their cache rows are one run of bytes.  Lane l of four holds elements 32 m + 8 l + i (m < 4, i < 8) of
// both vectors, the key's in the low and the value's in the high half of a 64-bit pair: the Hadamard butterflies of
// both are one packed fp32 instruction, strides 1, 2, 4, 32, 64 stay in the lane and 8, 16 are two shuffles; rows are
// read and written 16 bytes a lane, 64 bytes in a piece.
constexpr int kWarps = 8;
constexpr int kVecs = 8;  // tokens of a warp
constexpr float kInvSqrtD = 0.08838834764831845f;  // 1 / sqrt(128)

using f2 = unsigned long long;  // (key, value) as packed fp32
TQ_DEVFN f2 pk(float k, float v) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(k), "f"(v));
    return r;
}
TQ_DEVFN float2 un(f2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
TQ_DEVFN f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
TQ_DEVFN f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
TQ_DEVFN f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Unnormalised Walsh-Hadamard transform of both vectors, x[8 m + i]; the strides ascend as in fwht_warp128, so the
// sums round the same way.
TQ_DEVFN void fwht_pair(f2 (&x)[32]) {
    const f2 minus = pk(-1.f, -1.f);
    auto inside = [&](int h) {  // stride h of x's own index
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (!(e & h)) {
                const f2 p = x[e], q = x[e + h];
                x[e] = add2(p, q);
                x[e + h] = fma2(q, minus, p);
            }
    };
    inside(1);
    inside(2);
    inside(4);
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
        const float sg = (threadIdx.x & m) ? -1.f : 1.f;
        const f2 sg2 = pk(sg, sg);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const float2 v = un(x[e]);
            x[e] = fma2(x[e], sg2, pk(__shfl_xor_sync(kFull, v.x, m), __shfl_xor_sync(kFull, v.y, m)));
        }
    }
    inside(8);
    inside(16);
}

// The lane's signs, both vectors': +-factor.
TQ_DEVFN float sign_of(uint2 w, int i, float factor) {
    return (int8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3))) < 0 ? -factor : factor;
}

// Eight elements from 16 (bf16) or 32 (f32) bytes of shared memory.
template <bool BF16>
TQ_DEVFN void load8(const uint8_t* p, float (&y)[8]) {
    if constexpr (BF16) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = __uint_as_float(v[i] << 16);
            y[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 128);
        y[0] = a.x, y[1] = a.y, y[2] = a.z, y[3] = a.w, y[4] = b.x, y[5] = b.y, y[6] = b.z, y[7] = b.w;
    }
}

TQ_DEVFN void store8(void* p, int64_t at, int dt, const float (&y)[8]) {
    if (dt == TQ_F32) {
        float4* f = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at);
        f[0] = make_float4(y[0], y[1], y[2], y[3]);
        f[1] = make_float4(y[4], y[5], y[6], y[7]);
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (dt == TQ_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------- write

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
    int heads;  // of a warp's unit
    int dt;
    uint32_t* err;
};

// A value's code, the number of thresholds strictly below it, through equal bins over [-4.5, 4.5] (what lies outside goes to
// the end bins): bin_of is the same float expression for thresholds and values, hence monotone, so code = (thresholds of
// lower bins) + (the bin's own < u) wherever a bin holds one threshold at most.  A Lloyd-Max book's are further apart than
// its bins are wide (keys: 0.0169 against 0.0088; values: 0.258 against 0.143); other books search their thresholds.
// Entries are (thresholds of lower bins, the bin's own or +infinity); kReps copies lie interleaved, a lane reading copy
// lane % kReps, which keeps the lanes of a read from the same banks.
template <int N, int REPS>
struct Bins {
    static constexpr int kN = N, kReps = REPS;
    float2 at[N * REPS];
};
using KeyBins = Bins<1024, 4>;
using ValueBins = Bins<64, 16>;
// The bin of x as the low bits of a float's: 2^23 + bin.  NaN goes to bin 0.
template <int N>
TQ_DEVFN uint32_t bin_bits(float x) {
    return __float_as_uint(fmaf(__saturatef(fmaf(x, 1.0f / 9.0f, 0.5f)), (float)(N - 1), 8388608.0f));
}
// Fills a table from its book (all threads of the CTA); false if two thresholds share a bin.  bin: scratch of a book's size.
template <class B>
TQ_DEVFN bool fill_bins(B& t, const float* thr, int n, uint16_t* bin) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) bin[i] = (uint16_t)(bin_bits<B::kN>(thr[i]) & 0xffffu);
    __syncthreads();
    for (int x = threadIdx.x; x < B::kN; x += blockDim.x) {
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (bin[mid] < x) lo = mid + 1; else hi = mid;
        }
        const float2 e = make_float2(__int_as_float(lo), lo < n && bin[lo] == x ? thr[lo] : INFINITY);
        for (int r = 0; r < B::kReps; ++r) t.at[x * B::kReps + r] = e;
    }
    bool apart = true;
    for (int i = threadIdx.x; i + 1 < n; i += blockDim.x) apart = apart && bin[i] < bin[i + 1];
    return __syncthreads_and(apart);
}
// The code of u, looked up: `own` is the lane's copy of entry 0.
template <class B>
TQ_DEVFN uint32_t bin_code(uint32_t own, float u) {
    float2 e;
    // bits * (bytes of an entry's copies) wraps to the entry's offset: 2^23's exponent bits leave at the top
    const uint32_t at = own + (bin_bits<B::kN>(u) - 0x4b000000u) * (uint32_t)(sizeof(float2) * B::kReps);
    asm("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(e.x), "=f"(e.y) : "r"(at));
    uint32_t below;  // all ones where the bin's own threshold is below u
    asm("set.lt.u32.f32 %0, %1, %2;" : "=r"(below) : "f"(e.y), "f"(u));
    return __float_as_uint(e.x) - below;
}

TQ_DEVFN int count_below(const float* t, int n, float u) {  // thresholds strictly below u
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t[mid] < u) lo = mid + 1; else hi = mid;
    }
    return lo;
}

// Rotary positions of the lane's key elements.  Half pairs lie 64, 32 or 16 elements apart: in the lane's own other
// rows (m + 2, m + 1) or two lanes on.
struct Turn {
    float cs[16], sn[16];
};
TQ_DEVFN void turn_angles(const AppendArgs& a, int32_t pos, int l, Turn& w) {
    const int half = 1 << (a.lrot - 1);
#pragma unroll
    for (int z = 0; z < 16; ++z) {
        // interleaved: pairs 16 m + 4 l + 0 .. 3 at z = 4 m + ..; half: pairs 32 m + 8 l + i at z = 8 m + i
        const int pair = a.interleaved ? 16 * (z >> 2) + 4 * l + (z & 3) : (32 * (z >> 3) + 8 * l + (z & 7)) & (half - 1);
        const bool in = a.interleaved ? pair < half : (z < 8 || a.lrot == 7);
        float s = 0.f, c = 1.f;
        if (in) rope_angle(pos, a.steps[pair], s, c);
        w.sn[z] = s * a.factor;
        w.cs[z] = c * a.factor;
    }
}
TQ_DEVFN void turn_keys(const AppendArgs& a, const Turn& w, int l, float (&k)[32]) {
    auto pair = [&](float& x, float& y, int z) {
        const float p = x * w.cs[z] - y * w.sn[z], q = x * w.sn[z] + y * w.cs[z];
        x = p;
        y = q;
    };
    if (a.interleaved) {
#pragma unroll
        for (int z = 0; z < 16; ++z)
            if ((z >> 2) < 1 << (a.lrot - 5)) pair(k[8 * (z >> 2) + 2 * (z & 3)], k[8 * (z >> 2) + 2 * (z & 3) + 1], z);
    } else if (a.lrot == 7) {
#pragma unroll
        for (int z = 0; z < 16; ++z) pair(k[z], k[z + 16], z);
    } else if (a.lrot == 6) {
#pragma unroll
        for (int z = 0; z < 8; ++z) pair(k[z], k[z + 8], z);
    } else {
#pragma unroll
        for (int z = 0; z < 8; ++z) {
            const float o = __shfl_xor_sync(kFull, k[z], 2);
            k[z] = l < 2 ? k[z] * w.cs[z] - o * w.sn[z] : o * w.sn[z] + k[z] * w.cs[z];
        }
    }
}

// Persistent warps; a unit is eight tokens of one head (of four heads where rotary angles are shared among them).  The next
// head's or unit's vectors are copied to the warp's own shared memory while the present ones are encoded.
//
// Bound by instruction issue and the shared-memory pipe (table reads, shuffles): 65536 tokens of 8 heads in bf16, 8 and 3
// bits, 151 us (2.5 TB/s, 37 % of the copy rate), with rotary positions 190 us.
template <int KL, int VL, bool BF16, bool ROPE>
__global__ void __launch_bounds__(32 * kWarps, 2) kv_append_kernel(AppendArgs a) {
    using KB = KvBook<KL>;
    using VB = KvBook<VL>;
    constexpr int kPiece = BF16 ? 16 : 32, kVec = 16 * kPiece;  // bytes of eight elements, of a vector
    extern __shared__ __align__(16) uint8_t smem[];
    KeyBins& kbins = *reinterpret_cast<KeyBins*>(smem);
    ValueBins& vbins = *reinterpret_cast<ValueBins*>(smem + (KL == 256 ? sizeof(KeyBins) : sizeof(ValueBins)));
    // 4-bit keys take a small table too
    ValueBins& k4bins = *reinterpret_cast<ValueBins*>(smem);
    f2* const signs = reinterpret_cast<f2*>(reinterpret_cast<uint8_t*>(&vbins) + sizeof(ValueBins));  // [4][34] of a lane's 32
    uint8_t* const stage = reinterpret_cast<uint8_t*>(signs + 4 * 34) + (threadIdx.x >> 5) * (2 * kVecs * kVec);  // K, then V
    __shared__ float kt[256], vt[16];
    __shared__ uint16_t scratch[256];
    __shared__ uint32_t vbits[kWarps][kVecs][17];  // 24-bit pieces of 3-bit codes
    for (int i = threadIdx.x; i < KL - 1; i += blockDim.x) kt[i] = a.c.kthr[i];
    for (int i = threadIdx.x; i < VL - 1; i += blockDim.x) vt[i] = a.c.vthr[i];
    if (threadIdx.x < kPD) {  // element 32 m + 8 l + i of lane l
        const int m = threadIdx.x >> 5, q = (threadIdx.x >> 3) & 3, i = threadIdx.x & 7;
        const float s = (float)a.c.signs[threadIdx.x];
        signs[q * 34 + 8 * m + i] = pk(s, s);
    }
    __syncthreads();
    bool fast;
    if constexpr (KL == 256) fast = fill_bins(kbins, kt, KL - 1, scratch);
    else fast = fill_bins(k4bins, kt, KL - 1, scratch);
    __syncthreads();
    fast = fill_bins(vbins, vt, VL - 1, scratch) && fast;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, vec = lane >> 2, l = lane & 3;
    const int lg = a.c.lgroup;
    const float per_group = 1.0f / (float)(1 << lg);
    const int parts = (a.c.Hkv + a.heads - 1) / a.heads;
    // units are 32-bit numbers (the host sees to it): their division is a few instructions
    const uint32_t units = (uint32_t)((a.T + kVecs - 1) / kVecs) * parts, stride = gridDim.x * kWarps;
    const uint32_t kown = (uint32_t)__cvta_generic_to_shared(smem) + (KL == 256 ? (lane % KeyBins::kReps) : (lane % ValueBins::kReps)) * 8;
    const uint32_t vown = (uint32_t)__cvta_generic_to_shared(&vbins) + (lane % ValueBins::kReps) * 8;
    // The lane's pieces of its vector.  bf16: 64 bytes of four lanes to a piece number, those of odd vectors swapped by pairs,
    // so that eight lanes of a read (two vectors) meet all banks.  f32: the two halves of a piece 128 bytes apart.
    auto piece_at = [&](int m) {
        return stage + vec * kVec + (BF16 ? (m ^ (vec & 1)) * 64 : (m >> 1) * 256 + ((m ^ vec) & 1) * 64) + l * 16;
    };
    auto copy = [&](int64_t t, int h, bool on) {  // token t's key and value of head h
        if (on) {
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                const uint8_t* src = reinterpret_cast<const uint8_t*>(which ? a.v : a.k) +
                                     (t * (which ? a.vs : a.ks) + (int64_t)h * kPD + 8 * l) * (kPiece / 8);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(piece_at(m) + which * kVecs * kVec);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src + m * 4 * kPiece) : "memory");
                    if (!BF16)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 128), "l"(src + m * 4 * kPiece + 16)
                                     : "memory");
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int64_t all = a.c.pages << a.c.lpage;
    uint32_t unit = blockIdx.x * kWarps + warp;
    int64_t t = 0, t_next = 0;  // the lane's token of the unit, and of the next one; their slots (-1: nothing to write)
    int h0 = 0, h0_next = 0;
    int32_t slot = -1, slot_next = -1;
    auto look = [&](uint32_t u) {
        const uint32_t tb = u / (uint32_t)parts;
        t_next = (int64_t)tb * kVecs + vec;
        h0_next = (int)(u - tb * (uint32_t)parts) * a.heads;
        slot_next = u < units && t_next < a.T ? a.slots[t_next] : -1;
    };
    look(unit);
    copy(t_next, h0_next, slot_next >= 0 && slot_next < all);
    for (; unit < units; unit += stride) {
        t = t_next;
        h0 = h0_next;
        slot = slot_next;
        look(unit + stride);
        const int h1 = min(h0 + a.heads, a.c.Hkv);
        if (slot >= all) {
            if (l == 0 && a.err) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
            slot = -1;
        }
        Turn w;
        if (ROPE) turn_angles(a, t < a.T ? a.pos[t] : 0, l, w);
        for (int h = h0; h < h1; ++h) {
            f2 x[32];
            {
                float k[32], v[32];
                asm volatile("cp.async.wait_group 0;" ::: "memory");  // the lane reads what it copied itself
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    float y[8], z[8];
                    load8<BF16>(piece_at(m), y);
                    load8<BF16>(piece_at(m) + kVecs * kVec, z);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        k[8 * m + i] = y[i];
                        v[8 * m + i] = z[i];
                    }
                }
                // the next head's, or the next unit's first
                if (h + 1 < h1) copy(t, h + 1, slot >= 0);
                else copy(t_next, h0_next, slot_next >= 0 && slot_next < all);
                if (ROPE) turn_keys(a, w, l, k);
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = mul2(pk(k[e], v[e]), signs[l * 34 + e]);
            }
            fwht_pair(x);
            const f2 r = pk(kInvSqrtD, kInvSqrtD);
            f2 ss[4];  // sums of squares of the groups that piece m belongs to
#pragma unroll
            for (int m = 0; m < 4; ++m) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[8 * m + i] = mul2(x[8 * m + i], r);
                    ss[m] = i ? fma2(x[8 * m + i], x[8 * m + i], ss[m]) : mul2(x[8 * m], x[8 * m]);
                }
                const float2 p = un(ss[m]);
                ss[m] = add2(ss[m], pk(__shfl_xor_sync(kFull, p.x, 1), __shfl_xor_sync(kFull, p.y, 1)));
                if (lg > 4) {
                    const float2 q = un(ss[m]);
                    ss[m] = add2(ss[m], pk(__shfl_xor_sync(kFull, q.x, 2), __shfl_xor_sync(kFull, q.y, 2)));
                }
            }
            if (lg > 5) {
                ss[0] = ss[1] = add2(ss[0], ss[1]);
                ss[2] = ss[3] = add2(ss[2], ss[3]);
            }
            if (lg > 6) ss[0] = ss[1] = ss[2] = ss[3] = add2(ss[0], ss[2]);
            const int64_t row = slot >= 0 ? a.c.row(slot, h) : 0;
            uint32_t hk[4], hv[4];  // fp16 scales
            uint32_t vpiece[4], kpiece[4][KL == 256 ? 2 : 1];
            auto encode = [&](auto fast_c) {
                constexpr bool FAST = decltype(fast_c)::value;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float2 q = un(ss[m]);
                    const float sk = sqrtf(q.x * per_group), sv = sqrtf(q.y * per_group);
                    hk[m] = __half_as_ushort(__float2half_rn(sk));
                    hv[m] = __half_as_ushort(__float2half_rn(sv));
                    const f2 inv = pk(sk > 0.f ? 1.0f / sk : 0.f, sv > 0.f ? 1.0f / sv : 0.f);
                    uint32_t kw[2] = {0, 0}, vw = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 u = un(mul2(x[8 * m + i], inv));
                        const uint32_t ck = FAST ? bin_code<std::conditional_t<KL == 256, KeyBins, ValueBins>>(kown, u.x)
                                                 : (uint32_t)count_below(kt, KL - 1, u.x);
                        const uint32_t cv = FAST ? bin_code<ValueBins>(vown, u.y) : (uint32_t)count_below(vt, VL - 1, u.y);
                        kw[KL == 256 ? i >> 2 : 0] += ck * (1u << (KB::kBits * (KL == 256 ? i & 3 : i)));
                        vw += cv * (1u << (VB::kBits * i));
                    }
                    kpiece[m][0] = kw[0];
                    if constexpr (KL == 256) kpiece[m][1] = kw[1];
                    vpiece[m] = vw;
                }
            };
            if (fast) encode(std::true_type{});
            else encode(std::false_type{});
            if (slot >= 0) {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    if constexpr (KL == 256)
                        *reinterpret_cast<uint2*>(a.c.kcodes + row * 32 + 8 * m + 2 * l) = make_uint2(kpiece[m][0], kpiece[m][1]);
                    else
                        a.c.kcodes[row * 16 + 4 * m + l] = kpiece[m][0];
                    if constexpr (VL == 16) a.c.vcodes[row * 16 + 4 * m + l] = vpiece[m];
                }
            }
            if constexpr (VL == 8) {  // ten codes to a word: word w takes codes 10 w .. + 9, from pieces 10 w / 8 and the next
#pragma unroll
                for (int m = 0; m < 4; ++m) vbits[warp][vec][4 * m + l] = vpiece[m];
                __syncwarp();
                if (slot >= 0) {
                    uint32_t* dst = a.c.vcodes + row * 13;
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const int wd = 4 * z + l;
                        if (wd < 13) {
                            const int first = 10 * wd, piece = first >> 3, off = 3 * (first & 7);
                            const uint32_t lo = vbits[warp][vec][piece] >> off;
                            const uint32_t hi = wd < 12 ? vbits[warp][vec][piece + 1] << (24 - off) : 0u;
                            dst[wd] = (lo | hi) & 0x3fffffffu;
                        }
                    }
                }
                __syncwarp();
            }
            if (slot >= 0) {
                const int64_t z = row << (7 - lg);
                if (lg == 5) {
                    if (l == 0) *reinterpret_cast<uint2*>(a.c.kscales + z) = make_uint2(hk[0] | hk[1] << 16, hk[2] | hk[3] << 16);
                    if (l == 1) *reinterpret_cast<uint2*>(a.c.vscales + z) = make_uint2(hv[0] | hv[1] << 16, hv[2] | hv[3] << 16);
                } else if (lg == 4) {
                    if (!(l & 1))
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            a.c.kscales[z + 2 * m + (l >> 1)] = (uint16_t)hk[m];
                            a.c.vscales[z + 2 * m + (l >> 1)] = (uint16_t)hv[m];
                        }
                } else if (l == 0) {
                    a.c.kscales[z] = (uint16_t)hk[0];
                    a.c.vscales[z] = (uint16_t)hv[0];
                    if (lg == 6) {
                        a.c.kscales[z + 1] = (uint16_t)hk[2];
                        a.c.vscales[z + 1] = (uint16_t)hv[2];
                    }
                }
            }
        }
    }
}

// Calls of few vectors, where latency counts: a warp to a key or value vector, four elements a lane, the thresholds
// searched.  Every load that does not wait for another is under way before the first is needed.
template <int KL, int VL>
__global__ void __launch_bounds__(32 * kWarps) kv_append_small_kernel(AppendArgs a) {
    __shared__ float thr[2][256];
    __shared__ uint8_t cd[kWarps][kPD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t job = (int64_t)blockIdx.x * kWarps + warp, vec = job >> 1;
    const int which = (int)(job & 1);
    const bool on = vec < a.T * a.c.Hkv;
    const int64_t t = vec / a.c.Hkv;
    const int h = (int)(vec - t * a.c.Hkv);
    int32_t slot = -1, pos = 0;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t sg = 0;
    if (on) {
        slot = a.slots[t];
        const int64_t src = t * (which ? a.vs : a.ks) + (int64_t)h * kPD + lane * 4;
        if (a.dt == TQ_BF16) {
            const uint2 r = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(which ? a.v : a.k) + src);
            x[0] = __uint_as_float(r.x << 16), x[1] = __uint_as_float(r.x & 0xffff0000u);
            x[2] = __uint_as_float(r.y << 16), x[3] = __uint_as_float(r.y & 0xffff0000u);
        } else {
            const float4 r = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(which ? a.v : a.k) + src);
            x[0] = r.x, x[1] = r.y, x[2] = r.z, x[3] = r.w;
        }
        sg = *reinterpret_cast<const uint32_t*>(a.c.signs + lane * 4);
        if (a.steps && which == 0) pos = a.pos[t];
    }
    if (threadIdx.x < KL - 1) thr[0][threadIdx.x] = a.c.kthr[threadIdx.x];
    if (threadIdx.x < VL - 1) thr[1][threadIdx.x] = a.c.vthr[threadIdx.x];
    __syncthreads();
    if (slot < 0) return;
    if ((int64_t)slot >= a.c.pages << a.c.lpage) {
        if (lane == 0 && a.err) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
        return;
    }
    if (a.steps && which == 0) {
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
                rope_angle(pos, a.steps[pair], sn, cs);
                sn *= second ? a.factor : -a.factor;
                cs *= a.factor;
            }
            y[i] = e < rotary ? x[i] * cs + o * sn : x[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = y[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] *= (float)(int8_t)(sg >> (8 * i));
    fwht_warp128(x);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] *= kInvSqrtD;
        ss += x[i] * x[i];
    }
    const int group = 1 << a.c.lgroup, lpg = group / 4;
    for (int m = 1; m < lpg; m <<= 1) ss += __shfl_xor_sync(kFull, ss, m);
    const float s = sqrtf(ss / (float)group), inv = s > 0.f ? 1.0f / s : 0.f;
    const int64_t row = a.c.row(slot, h);
    if ((lane & (lpg - 1)) == 0)
        (which ? a.c.vscales : a.c.kscales)[(row << (7 - a.c.lgroup)) + lane / lpg] = __half_as_ushort(__float2half_rn(s));
    const int n = (which ? VL : KL) - 1;
    const int bits = which ? KvBook<VL>::kBits : KvBook<KL>::kBits, cw = 32 / bits;
    uint32_t c4 = 0;  // the lane's four codes
#pragma unroll
    for (int i = 0; i < 4; ++i) c4 |= (uint32_t)count_below(thr[which], n, x[i] * inv) << (8 * i);
    reinterpret_cast<uint32_t*>(cd[warp])[lane] = c4;
    __syncwarp();
    const int words = which ? KvBook<VL>::kWords : KvBook<KL>::kWords;
    if (lane < words) {
        uint32_t w = 0;
        for (int i = 0; i < cw && lane * cw + i < kPD; ++i) w |= (uint32_t)cd[warp][lane * cw + i] << (bits * i);
        (which ? a.c.vcodes : a.c.kcodes)[row * words + lane] = w;
    }
}

// ---------------------------------------------------------------- read

struct FetchArgs {
    KvPages c;
    const int32_t* slots;
    int64_t T;
    void* k;
    void* v;
    int dt;
    uint32_t* err;
};

// Eight codes from bit 0 of a piece; 3-bit pieces span two words.
template <int LEVELS>
TQ_DEVFN void piece8(const uint32_t* words, int piece, uint32_t (&w)[2]) {
    if constexpr (LEVELS == 256) {
        const uint2 y = *reinterpret_cast<const uint2*>(words + 2 * piece);
        w[0] = y.x;
        w[1] = y.y;
    } else if constexpr (LEVELS == 16) {
        w[0] = words[piece];
        w[1] = 0;
    } else {
        const int first = (8 * piece) / 10, off = 3 * (8 * piece - 10 * first);
        const uint32_t lo = words[first] >> off;
        w[0] = off > 6 ? lo | (words[first + 1] << (30 - off)) : lo;
        w[1] = 0;
    }
}

// The key book in shared memory once (a copy for each lane, without bank conflicts, took as long: 118 us both).  Bound by
// instruction issue and latency at 16 warps an SM: 65536 tokens of 8 heads 118 us, 3.1 TB/s, 47 % of the copy rate.
template <int KL, int VL>
__global__ void __launch_bounds__(32 * kWarps, 2) kv_fetch_kernel(FetchArgs a) {
    __shared__ float kl[KL], vl[VL];
    for (int i = threadIdx.x; i < KL; i += blockDim.x) kl[i] = a.c.kcent[i];
    for (int i = threadIdx.x; i < VL; i += blockDim.x) vl[i] = a.c.vcent[i];
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, vec = lane >> 2, l = lane & 3;
    const int lg = a.c.lgroup;
    const uint32_t units = (uint32_t)((a.T + kVecs - 1) / kVecs) * a.c.Hkv, stride = gridDim.x * kWarps;  // 32-bit numbers
    const int64_t all = a.c.pages << a.c.lpage;
    uint32_t unit = blockIdx.x * kWarps + warp;
    int64_t t_next = 0;
    int h_next = 0;
    int32_t slot_next = -1;
    auto look = [&](uint32_t u) {  // the lane's token of a unit, and its slot (-1: none)
        const uint32_t tb = u / (uint32_t)a.c.Hkv;
        t_next = (int64_t)tb * kVecs + vec;
        h_next = (int)(u - tb * (uint32_t)a.c.Hkv);
        slot_next = u < units && t_next < a.T ? a.slots[t_next] : -1;
    };
    look(unit);
    for (; unit < units; unit += stride) {
        const int64_t t = t_next;
        const int h = h_next;
        int32_t slot = slot_next;
        look(unit + stride);
        if (slot >= all) {
            if (l == 0 && a.err) atomicOr(a.err, TQ_DEVERR_BAD_PAGE);
            slot = -1;
        }
        f2 x[32];
        if (slot >= 0) {
            const int64_t row = a.c.row(slot, h);
            const uint32_t* kw = a.c.kcodes + row * KvBook<KL>::kWords;
            const uint32_t* vw = a.c.vcodes + row * KvBook<VL>::kWords;
            const int64_t z = row << (7 - lg);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                uint32_t ck[2], cv[2];
                piece8<KL>(kw, 4 * m + l, ck);
                piece8<VL>(vw, 4 * m + l, cv);
                const int g = (32 * m + 8 * l) >> lg;
                const f2 s = pk(half_bits_to_float(a.c.kscales[z + g]), half_bits_to_float(a.c.vscales[z + g]));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t p = KL == 256 ? (ck[i >> 2] >> (8 * (i & 3))) & 255u : (ck[0] >> (4 * i)) & 15u;
                    const uint32_t q = (cv[0] >> (KvBook<VL>::kBits * i)) & (VL - 1);
                    x[8 * m + i] = mul2(pk(kl[p % KL], vl[q]), s);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = 0;
        }
        if (slot_next >= 0 && slot_next < all) {  // the next unit's rows on their way to L1 beside the transform: a lane to an array
            const int64_t row = a.c.row(slot_next, h_next);
            const void* p = l == 0 ? (const void*)(a.c.kcodes + row * KvBook<KL>::kWords)
                                   : (l == 1 ? (const void*)(a.c.vcodes + row * KvBook<VL>::kWords)
                                             : (const void*)((l == 2 ? a.c.kscales : a.c.vscales) + (row << (7 - lg))));
            asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
        }
        fwht_pair(x);
        if (t < a.T) {
            const int64_t at = (t * a.c.Hkv + h) * kPD;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint2 sg = *reinterpret_cast<const uint2*>(a.c.signs + 32 * m + 8 * l);
                float y[8], w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float s = sign_of(sg, i, kInvSqrtD);
                    const float2 u = un(x[8 * m + i]);
                    y[i] = u.x * s;
                    w[i] = u.y * s;
                }
                if (a.k) store8(a.k, at + 32 * m + 8 * l, a.dt, y);
                if (a.v) store8(a.v, at + 32 * m + 8 * l, a.dt, w);
            }
        }
    }
}

int sm_count() {
    static const int n = [] {
        int dev = 0, v = 0;
        cudaGetDevice(&dev);
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        return std::max(v, 1);
    }();
    return n;
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
    if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || !aligned(positions, 4) || !aligned(err, 4))
        return TQ_ERR_INVALID;
    if (T > kMaxTokens) return TQ_ERR_UNSUPPORTED;
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
    cudaStream_t st = as_stream(stream);
    // Up to 4096 (token, head) pairs a warp to each vector (8 pairs: 3.8 us, against 9.2 for the persistent kernel and its
    // tables; 4096: 7.7 and 8.5); past that the persistent kernel (8192: 8.6 us against 13.0; 524288: 150 against 647).
    if (T * cache->Hkv <= 4096) {
        const unsigned blocks = (unsigned)((T * cache->Hkv * 2 + kWarps - 1) / kWarps);
        return by_books(cache, [&](auto kl, auto vl) {
            kv_append_small_kernel<decltype(kl)::value, decltype(vl)::value><<<blocks, 32 * kWarps, 0, st>>>(a);
            return launch_status();
        });
    }
    // A warp's unit: eight tokens of one head; of four heads where rotary angles are shared among them (65536 tokens of 8
    // heads: 190 us, 226 with one) and there are units enough for every warp of two CTAs an SM.
    const int64_t blocks8 = (T + kVecs - 1) / kVecs, all = (int64_t)sm_count() * 2 * kWarps;
    a.heads = rope && blocks8 * ((cache->Hkv + 3) / 4) >= all ? std::min(4, cache->Hkv) : 1;
    const int64_t units = blocks8 * ((cache->Hkv + a.heads - 1) / a.heads);
    if (units > 0x3fffffffll) return TQ_ERR_UNSUPPORTED;
    const unsigned blocks = (unsigned)std::min<int64_t>((units + kWarps - 1) / kWarps, sm_count() * 2);
    return by_books(cache, [&](auto kl, auto vl) {
        constexpr int KL = decltype(kl)::value, VL = decltype(vl)::value;
        auto launch = [&](auto kernel, size_t vector) {
            const size_t smem = (KL == 256 ? sizeof(KeyBins) : sizeof(ValueBins)) + sizeof(ValueBins) + 4 * 34 * sizeof(f2) +
                                kWarps * 2 * kVecs * vector;
            if (ensure_smem((const void*)kernel, smem) != cudaSuccess) return TQ_ERR_CUDA;
            kernel<<<blocks, 32 * kWarps, smem, st>>>(a);
            return launch_status();
        };
        if (dt == TQ_BF16) return rope ? launch(kv_append_kernel<KL, VL, true, true>, 256) : launch(kv_append_kernel<KL, VL, true, false>, 256);
        return rope ? launch(kv_append_kernel<KL, VL, false, true>, 512) : launch(kv_append_kernel<KL, VL, false, false>, 512);
    });
}

extern "C" tq_status tq_kv_fetch(const tq_kv_pages_t* cache, const int32_t* slots, int64_t T, void* k, void* v,
                                 tq_dtype dt, uint32_t* err, void* stream) {
    const tq_status ok = kv_pages_check(cache, false);
    if (ok != TQ_OK) return ok;
    if (T < 0 || (dt != TQ_F32 && dt != TQ_BF16 && dt != TQ_F16)) return TQ_ERR_INVALID;
    if (T == 0 || (!k && !v)) return TQ_OK;
    if (!slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || !aligned(err, 4)) return TQ_ERR_INVALID;
    if (T > kMaxTokens) return TQ_ERR_UNSUPPORTED;
    FetchArgs a{};
    a.c = kv_pages_view(cache);
    a.slots = slots;
    a.T = T;
    a.k = k;
    a.v = v;
    a.dt = dt;
    a.err = err;
    const int64_t units = (T + kVecs - 1) / kVecs * cache->Hkv;
    if (units > 0x3fffffffll) return TQ_ERR_UNSUPPORTED;
    const unsigned blocks = (unsigned)std::min<int64_t>((units + kWarps - 1) / kWarps, sm_count() * 2);
    cudaStream_t st = as_stream(stream);
    return by_books(cache, [&](auto kl, auto vl) {
        constexpr int KL = decltype(kl)::value, VL = decltype(vl)::value;
        kv_fetch_kernel<KL, VL><<<blocks, 32 * kWarps, 0, st>>>(a);
        return launch_status();
    });
}
