// Rotary angles, shared by the kernels that rotate.
//
// A pair i turns by 2 pi u(pos * f_i), f_i a fraction of a turn for each
// position. f_i is held in 64 bits as step_i = round(f_i 2^64) mod 2^64: the
// product pos * step_i modulo 2^64 is then the angle modulo a turn without any
// rounding (an fp32 product would be off by up to 0.06 rad at position 10^6),
// and costs one integer multiplication. Its top 32 bits, taken as a signed
// fraction, lie in [-1/2, 1/2) of a turn; as fp32 they are off by at most
// 2^-25 of themselves, so the angle is off by at most 2^-25 pi.
#pragma once
#include <stdint.h>

namespace mla {

// cos and sin of the angle, times mscale.
__device__ __forceinline__ float2 rope_cos_sin(int64_t pos, int64_t step, float mscale) {
    const uint64_t turn = static_cast<uint64_t>(pos) * static_cast<uint64_t>(step);
    const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * mscale, s * mscale);
}

}  // namespace mla
