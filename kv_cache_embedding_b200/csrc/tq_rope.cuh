// Angles of the rotary positions, shared by tq_rope and tq_kv8_append.
#pragma once

#include <stdint.h>

#include "tq.h"

namespace tq {

// cos and sin of a position's angle.  `turns` is the frequency in turns as a
// fraction of 2^64, so pos * turns modulo 2^64 is the fraction of a turn exactly
// (two's complement takes negative positions along); its top 32 bits leave an
// error of 2^-32 turn.  The nearest quarter turn is taken off in integers: what
// is left, within 1/8 turn, rounds to fp32 with an error below 2^-25 of itself.
__device__ __forceinline__ void rope_angle(uint64_t turns, int64_t pos, float& c, float& s) {
    const uint32_t t = (uint32_t)(((uint64_t)pos * turns) >> 32);
    const uint32_t q = (t + 0x20000000u) >> 30;           // quarter turns, 0..3
    const int32_t r = (int32_t)(t - (q << 30));           // [-2^29, 2^29): 1/8 turn
    float cr, sr;
    sincospif((float)r * 4.656612873077393e-10f, &sr, &cr);  // r 2^-31 half turns
    c = (q & 1u) ? sr : cr;
    s = (q & 1u) ? cr : sr;
    if (q == 1u || q == 2u) c = -c;
    if (q >= 2u) s = -s;
}

bool rope_valid(const tq_rope_params_t* r);

}  // namespace tq
