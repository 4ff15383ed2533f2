// fa_rope.cuh -- the rotation's arithmetic, shared by the kernels that rotate, so
// that they give the same bits.
#pragma once

#include <cuda_runtime.h>

namespace fa {

// Cosine and sine of position * frequency, the frequency in units of 2^-64
// turns: the product modulo a turn is a wrapping 64-bit product, exact for every
// position, and its top 32 bits are a signed fraction of a turn.
__device__ __forceinline__ void rope_angle(long long pos, unsigned long long freq, float amp, float& c, float& s) {
    const unsigned long long turn = static_cast<unsigned long long>(pos) * freq;
    sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    c *= amp;
    s *= amp;
}
// x c - y s, one rounding of the product y s and one of the sum.
__device__ __forceinline__ float rope_turn(float x, float y, float c, float s) {
    return __fmaf_rn(x, c, -__fmul_rn(y, s));
}

}  // namespace fa
