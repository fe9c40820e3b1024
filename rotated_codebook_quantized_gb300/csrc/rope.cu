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

// One thread per pair: the simplest form.
template <class T, bool INTERLEAVED>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs a) {
    const int heads = a.side[0].heads + a.side[1].heads;
    const int half = a.rotary / 2, rest = a.dim - a.rotary, per = half + rest;
    const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= a.tokens * heads * per) return;
    const int c = (int)(idx % per);
    const int64_t th = idx / per;
    int h = (int)(th % heads);
    const int64_t t = th / heads;
    const RopeSide& s = h < a.side[0].heads ? a.side[0] : a.side[1];
    if (h >= a.side[0].heads) h -= a.side[0].heads;
    const T* x = reinterpret_cast<const T*>(s.x) + t * s.xs + (int64_t)h * a.dim;
    T* y = reinterpret_cast<T*>(s.y) + t * s.ys + (int64_t)h * a.dim;
    if (c >= half) {
        const int e = a.rotary + c - half;
        y[e] = x[e];
        return;
    }
    float sn, cs;
    rope_angle(a.pos[t], a.steps[c], sn, cs);
    sn *= a.sgn * a.factor;
    cs *= a.factor;
    const int ia = INTERLEAVED ? 2 * c : c, ib = INTERLEAVED ? 2 * c + 1 : c + half;
    const float va = (float)x[ia], vb = (float)x[ib];
    y[ia] = (T)(va * cs - vb * sn);
    y[ib] = (T)(va * sn + vb * cs);
}

template <class T>
tq_status launch_rope(const RopeArgs& a, int layout, cudaStream_t st) {
    const int64_t total = a.tokens * (a.side[0].heads + a.side[1].heads) * (a.rotary / 2 + a.dim - a.rotary);
    const int64_t blocks = (total + 255) / 256;
    if (blocks > 0x7fffffffll) return TQ_ERR_UNSUPPORTED;
    if (layout == TQ_ROPE_INTERLEAVED)
        rope_kernel<T, true><<<(unsigned)blocks, 256, 0, st>>>(a);
    else
        rope_kernel<T, false><<<(unsigned)blocks, 256, 0, st>>>(a);
    return launch_status();
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
    if (!positions || (Hq && (!q || !yq)) || (Hkv && (!k || !yk))) return TQ_ERR_INVALID;
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
