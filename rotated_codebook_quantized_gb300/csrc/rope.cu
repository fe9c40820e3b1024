// Rotary positions: tq_rope_steps (host), tq_rope.
//
// Pair (a, b) of a token at position p turns by the angle p w: (a cos - b sin,
// a sin + b cos).  The angle is kept as a phase: w / (2 pi) as a 64-bit fraction of a
// turn, so that p * step mod 2^64 drops whole turns exactly and its top 32 bits are the
// angle in units of pi / 2^31 (error below 2^-24 pi at any position; p * w in fp32
// would be off by 0.004 rad at position 131072).
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "rope.cuh"

using namespace tq;

namespace {

struct RopeSide {
    const void* x;
    void* y;
    int64_t xs, ys;  // elements between tokens
    int heads;
};

struct RopeArgs {
    RopeSide side[2];
    const int32_t* pos;
    const uint64_t* steps;
    int64_t tokens;
    int dim, rotary;
    float factor, sgn;
};

// P consecutive elements as floats, moved in pieces of up to 16 bytes.
template <class T, int P>
struct alignas(sizeof(T) * P < 16 ? sizeof(T) * P : 16) Pack {
    T v[P];
};

// A thread owns P pairs of a token (or 2 P elements past the rotated part) and walks the heads with them: the
// sines and cosines are computed once for all of its heads.  Bound by bytes: every element is read and written
// once, 16 bytes at a time.
//
// P = 8 where rows and parts allow pieces of 8 elements, 1 elsewhere (any even rotary, any alignment).  32768
// tokens of 32 + 8 heads of 128, bf16: P = 1 241 us, P = 8 109 us (6.2 TB/s, 92 % of the copy rate).
template <class T, int P, bool INTERLEAVED>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs a, uint32_t total, int chunks, int turned, int walkers) {
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
    if (idx >= total) return;
    const uint32_t th = idx / (uint32_t)chunks;
    const int c = (int)(idx - th * (uint32_t)chunks);
    const uint32_t t = th / (uint32_t)walkers;
    const int h0 = (int)(th - t * (uint32_t)walkers), heads = a.side[0].heads + a.side[1].heads;
    const bool turns = c < turned;
    int ia, ib;  // first elements of the thread's two pieces
    if (!turns) {
        ia = a.rotary + (c - turned) * 2 * P;
        ib = ia + P;
    } else if (INTERLEAVED) {
        ia = 2 * P * c;
        ib = ia + P;
    } else {
        ia = P * c;
        ib = ia + a.rotary / 2;
    }
    float sn[P], cs[P];
    if (turns) {
        const int32_t pos = a.pos[t];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            rope_angle(pos, a.steps[P * c + i], sn[i], cs[i]);
            sn[i] *= a.sgn * a.factor;
            cs[i] *= a.factor;
        }
    }
    using V = Pack<T, P>;
    const bool second = turns || ib < a.dim;  // the last piece past the rotated part may be half
#pragma unroll 4
    for (int h = h0; h < heads; h += walkers) {
        const bool k = h >= a.side[0].heads;
        const int64_t at = (int64_t)(k ? h - a.side[0].heads : h) * a.dim;
        const T* x = reinterpret_cast<const T*>(k ? a.side[1].x : a.side[0].x) + (int64_t)t * (k ? a.side[1].xs : a.side[0].xs) + at;
        T* y = reinterpret_cast<T*>(k ? a.side[1].y : a.side[0].y) + (int64_t)t * (k ? a.side[1].ys : a.side[0].ys) + at;
        V va = *reinterpret_cast<const V*>(x + ia), vb{};
        if (second) vb = *reinterpret_cast<const V*>(x + ib);
        if (turns) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (INTERLEAVED && P > 1) {  // pair i: elements 2 i, 2 i + 1 of the two pieces
                    T& ra = 2 * i < P ? va.v[(2 * i) % P] : vb.v[(2 * i) % P];
                    T& rb = 2 * i < P ? va.v[(2 * i + 1) % P] : vb.v[(2 * i + 1) % P];
                    const float xa = (float)ra, xb = (float)rb;
                    ra = (T)(xa * cs[i] - xb * sn[i]);
                    rb = (T)(xa * sn[i] + xb * cs[i]);
                } else {
                    const float xa = (float)va.v[i], xb = (float)vb.v[i];
                    va.v[i] = (T)(xa * cs[i] - xb * sn[i]);
                    vb.v[i] = (T)(xa * sn[i] + xb * cs[i]);
                }
            }
        }
        *reinterpret_cast<V*>(y + ia) = va;
        if (second) *reinterpret_cast<V*>(y + ib) = vb;
    }
}

template <class T, int P>
tq_status launch_rope_p(RopeArgs a, int layout, bool inplace, int sms, cudaStream_t st) {
    const int heads = a.side[0].heads + a.side[1].heads, turned = a.rotary / 2 / P;
    // in place nothing past the rotated part moves
    const int chunks = turned + (inplace ? 0 : (a.dim - a.rotary + 2 * P - 1) / (2 * P));
    // Threads for about three full waves; what is left of the heads a thread walks.
    const int64_t want = (int64_t)sms * 2048 * 3, per = a.tokens * chunks;
    const int walkers = (int)std::max<int64_t>(1, std::min<int64_t>(heads, (want + per - 1) / per));
    const int64_t most = 0x7fffff00ll / ((int64_t)chunks * walkers);  // tokens of a launch: 32-bit thread numbers
    if (most < 1) return TQ_ERR_UNSUPPORTED;
    const int64_t tokens = a.tokens;
    for (int64_t t0 = 0; t0 < tokens; t0 += most) {
        RopeArgs b = a;
        b.tokens = std::min(most, tokens - t0);
        b.pos += t0;
        for (RopeSide& s : b.side)
            if (s.heads) {
                s.x = static_cast<const T*>(s.x) + t0 * s.xs;
                s.y = static_cast<T*>(s.y) + t0 * s.ys;
            }
        const uint32_t total = (uint32_t)(b.tokens * chunks * walkers);
        if (layout == TQ_ROPE_INTERLEAVED)
            rope_kernel<T, P, true><<<(total + 255) / 256, 256, 0, st>>>(b, total, chunks, turned, walkers);
        else
            rope_kernel<T, P, false><<<(total + 255) / 256, 256, 0, st>>>(b, total, chunks, turned, walkers);
        const tq_status s = launch_status();
        if (s != TQ_OK) return s;
    }
    return TQ_OK;
}

template <class T>
tq_status launch_rope(const RopeArgs& a, int layout, cudaStream_t st) {
    static const int sms = [] {
        int dev = 0, v = 0;
        cudaGetDevice(&dev);
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        return std::max(v, 1);
    }();
    bool wide = a.rotary % 16 == 0 && a.dim % 8 == 0, inplace = true;
    for (const RopeSide& s : a.side)
        if (s.heads) {
            wide = wide && aligned(s.x, 16) && aligned(s.y, 16) && s.xs * sizeof(T) % 16 == 0 && s.ys * sizeof(T) % 16 == 0;
            inplace = inplace && s.x == s.y;
        }
    return wide ? launch_rope_p<T, 8>(a, layout, inplace, sms, st) : launch_rope_p<T, 1>(a, layout, inplace, sms, st);
}

}  // namespace

extern "C" tq_status tq_rope_steps(int32_t rotary, double base, const tq_rope_scaling_t* scaling, uint64_t* steps,
                                   float* factor) {
    if (rotary < 2 || (rotary & 1) || !(base > 1.0) || !isfinite(base) || !steps) return TQ_ERR_INVALID;
    const int kind = scaling ? scaling->kind : TQ_ROPE_NONE;
    double f = 1.0;
    if (kind != TQ_ROPE_NONE) {
        if (kind != TQ_ROPE_LINEAR && kind != TQ_ROPE_BASE && kind != TQ_ROPE_PARTS) return TQ_ERR_INVALID;
        f = scaling->factor;
        if (!(f >= 1.0) || !isfinite(f)) return TQ_ERR_INVALID;
        if (kind == TQ_ROPE_PARTS && !(scaling->original > 0.0 && isfinite(scaling->original) && scaling->slow_turns >= 0.0 &&
                                       scaling->fast_turns > scaling->slow_turns && isfinite(scaling->fast_turns)))
            return TQ_ERR_INVALID;
    }
    if (kind == TQ_ROPE_BASE) base *= pow(f, (double)rotary / (double)std::max(rotary - 2, 1));
    if (!isfinite(base)) return TQ_ERR_INVALID;
    const double two_pi = 6.283185307179586476925286766559;
    for (int i = 0; i < rotary / 2; ++i) {
        double w = pow(base, -2.0 * i / rotary);
        if (kind == TQ_ROPE_LINEAR) w /= f;
        if (kind == TQ_ROPE_PARTS) {
            const double turns = scaling->original * w / two_pi;
            const double keep =
                std::min(1.0, std::max(0.0, (turns - scaling->slow_turns) / (scaling->fast_turns - scaling->slow_turns)));
            w *= keep + (1.0 - keep) / f;
        }
        steps[i] = (uint64_t)rint(w / two_pi * 18446744073709551616.0);  // w <= 1: below 2^62
    }
    if (factor) *factor = kind == TQ_ROPE_PARTS ? (float)(0.1 * log(f) + 1.0) : 1.0f;
    return TQ_OK;
}

extern "C" tq_status tq_rope(const tq_rope_t* rope, const int32_t* positions, int64_t tokens, tq_dtype dt,
                             int32_t inverse, const void* q, int64_t q_stride, int32_t Hq, void* yq, int64_t yq_stride,
                             const void* k, int64_t k_stride, int32_t Hkv, void* yk, int64_t yk_stride, void* stream) {
    if (!rope_ok(rope) || tokens < 0 || Hq < 0 || Hkv < 0 || Hq > 65536 || Hkv > 65536) return TQ_ERR_INVALID;
    if (dt != TQ_F32 && dt != TQ_BF16 && dt != TQ_F16) return TQ_ERR_INVALID;
    const int64_t dim = rope->dim;
    if (Hq && (q_stride < Hq * dim || yq_stride < Hq * dim)) return TQ_ERR_INVALID;
    if (Hkv && (k_stride < Hkv * dim || yk_stride < Hkv * dim)) return TQ_ERR_INVALID;
    if (tokens == 0 || Hq + Hkv == 0) return TQ_OK;
    if (!positions || !aligned(positions, 4) || (Hq && (!q || !yq)) || (Hkv && (!k || !yk))) return TQ_ERR_INVALID;
    if (tokens > (1ll << 40)) return TQ_ERR_UNSUPPORTED;  // threads are counted in 64 bits
    const size_t es = dt == TQ_F32 ? 4 : 2;
    if ((Hq && (!aligned(q, es) || !aligned(yq, es))) || (Hkv && (!aligned(k, es) || !aligned(yk, es))))
        return TQ_ERR_INVALID;
    if ((q && q == yq && q_stride != yq_stride) || (k && k == yk && k_stride != yk_stride)) return TQ_ERR_INVALID;
    RopeArgs a{};
    a.side[0] = {q, yq, q_stride, yq_stride, Hq};
    a.side[1] = {k, yk, k_stride, yk_stride, Hkv};
    a.pos = positions;
    a.steps = rope->steps;
    a.tokens = tokens;
    a.dim = rope->dim;
    a.rotary = rope->rotary;
    a.factor = rope->factor;
    a.sgn = inverse ? -1.0f : 1.0f;
    cudaStream_t st = as_stream(stream);
    if (dt == TQ_F32) return launch_rope<float>(a, rope->layout, st);
    if (dt == TQ_BF16) return launch_rope<__nv_bfloat16>(a, rope->layout, st);
    return launch_rope<__half>(a, rope->layout, st);
}
