// Rotary angles, shared by tq_rope and the cache write.
#pragma once

#include "common.cuh"

namespace tq {

inline bool rope_ok(const tq_rope_t* r) {
    return r && r->steps && r->dim > 0 && r->dim <= 65536 && r->rotary >= 2 && !(r->rotary & 1) && r->rotary <= r->dim &&
           (r->layout == TQ_ROPE_HALF || r->layout == TQ_ROPE_INTERLEAVED) && aligned(r->steps, 8);
}

// sin and cos of position * step: the top 32 bits of the wrapped product are the angle
// over pi / 2^31, as a signed number in [-1, 1) times pi.
TQ_DEVFN void rope_angle(int32_t pos, uint64_t step, float& sn, float& cs) {
    const uint64_t phase = (uint64_t)(int64_t)pos * step;
    sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &sn, &cs);
}

}  // namespace tq
