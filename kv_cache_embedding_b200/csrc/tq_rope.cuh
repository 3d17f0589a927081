// Angles of the rotary positions, shared by tq_rope and tq_kv8_append.
#pragma once

#include <stdint.h>

#include "tq.h"

namespace tq {

// cos and sin of a position's angle.  `turns` is the frequency in turns as a
// fraction of 2^64, so pos * turns modulo 2^64 is that frequency's fraction of a turn
// exactly (two's complement takes negative positions along); its top 32 bits leave an
// error of 2^-32 turn.  The nearest quarter turn is taken off in integers: what
// is left, within 1/8 turn, rounds to fp32 with an error below 2^-24 of itself.
__device__ __forceinline__ void rope_angle(uint64_t turns, int64_t pos, float& c, float& s) {
    const uint32_t t = (uint32_t)(((uint64_t)pos * turns) >> 32);
    const uint32_t q = (t + 0x20000000u) >> 30;           // quarter turns, 0..3
    const int32_t r = (int32_t)(t - (q << 30));           // [-2^29, 2^29): 1/8 turn
    // |x| <= pi / 4: Taylor's series, the terms left out below 2^-29 and 2^-33
    const float x = (float)r * 1.4629180792671596e-9f, z = x * x;  // 2 pi / 2^32
    const float sr = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), x);
    const float cr = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800, 1.f / 40320), -1.f / 720),
                                          1.f / 24), -0.5f), 1.f);
    c = (q & 1u) ? sr : cr;
    s = (q & 1u) ? cr : sr;
    if (q == 1u || q == 2u) c = -c;
    if (q >= 2u) s = -s;
}

bool rope_valid(const tq_rope_params_t* r);

}  // namespace tq
