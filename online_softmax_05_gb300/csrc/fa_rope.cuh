// fa_rope.cuh -- the rotation's arithmetic, shared by the kernels that rotate, so
// that they give the same bits.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace fa {

// cos and sin of k / 256 turns, each as a sum of two fp32 numbers, from their
// Taylor series in double precision (over at most an eighth of a turn).
struct RopeTable {
    float4 v[256];  // (cos, its rest, sin, its rest)
};
constexpr RopeTable rope_table() {
    RopeTable t{};
    for (int k = 0; k < 256; ++k) {
        // octants: a in [0, 1/8] turn, cos and sin swapped and signed
        const int oct = k / 32, in = k % 32, m = oct % 2 ? 32 - in : in;
        const double a = m * (6.283185307179586476925286766559 / 256);
        double c = 1, s = a, term = a;  // term: a^n / n!
        for (int n = 2; n < 24; ++n) {
            term *= a / n;
            if (n % 2) s += n % 4 == 1 ? term : -term;
            else c += n % 4 == 0 ? term : -term;
        }
        const int q = (oct + 1) / 2;  // quarter turns that a is counted from
        double cc = c, ss = oct % 2 ? -s : s;  // of +-a
        for (int i = 0; i < q; ++i) {
            const double x = cc;
            cc = -ss;
            ss = x;
        }
        t.v[k].x = static_cast<float>(cc);
        t.v[k].y = static_cast<float>(cc - static_cast<double>(t.v[k].x));
        t.v[k].z = static_cast<float>(ss);
        t.v[k].w = static_cast<float>(ss - static_cast<double>(t.v[k].z));
    }
    return t;
}
static __device__ const RopeTable kRopeTable = rope_table();

// Cosine and sine of position * frequency, the frequency in units of 2^-64
// turns: the product modulo a turn is a wrapping 64-bit product, exact for every
// position.  It is split into k / 256 turns, whose cosine and sine are tabled, and
// a rest t of at most 0.0123 rad:
//   cos(k + t) = c + (c (cos t - 1) - s sin t),  sin(k + t) = s + (s (cos t - 1) + c sin t).
// The bracket's largest term carries its product's rounding along, so that it is
// off by some 1e-11 and the sum, rounded once, is nearly always the nearest fp32
// number (40000 random angles: all of them).  Rotated keys are rounded to bf16 and
// then to 16 codes, where fp32's own sine and cosine, an ulp off, turned some keys
// into another code than the formula's.
__device__ __forceinline__ void rope_angle(long long pos, unsigned long long freq, float amp, float& cos_out,
                                           float& sin_out) {
    const unsigned long long turn = static_cast<unsigned long long>(pos) * freq;
    const unsigned k = static_cast<unsigned>((turn + (1ull << 55)) >> 56);
    const long long rest = static_cast<long long>(turn - (static_cast<unsigned long long>(k) << 56));  // 2^-64 turns
    // t = (hi + lo) 2^-32 turns; hi has 24 bits
    const float hi = static_cast<float>(static_cast<int>(rest >> 32));
    const float lo = static_cast<float>(static_cast<uint32_t>(rest)) * 2.3283064365386963e-10f;  // 2^-32
    constexpr double kRad = 6.283185307179586476925286766559 / 4294967296.0;
    constexpr float kRadHi = static_cast<float>(kRad), kRadLo = static_cast<float>(kRad - static_cast<double>(kRadHi));
    const float t = hi * kRadHi;
    const float t_lo = fmaf(hi, kRadHi, -t) + fmaf(hi, kRadLo, lo * kRadHi);
    const float t2 = t * t;
    // sin t = t + sn, cos t = 1 + cm
    const float sn = fmaf(t * t2, fmaf(t2, 1.f / 120.f, -1.f / 6.f), t_lo);
    const float cm = t2 * fmaf(t2, 1.f / 24.f, -0.5f);
    const float4 e = kRopeTable.v[k & 255u];
    const float st = __fmul_rn(e.z, t), ct = __fmul_rn(e.x, t);  // not fused into the sums: their rest is added below
    const float c_low = fmaf(e.x, cm, e.y) - (fmaf(e.z, t, -st) + fmaf(e.z, sn, e.w * t));
    const float s_low = fmaf(e.z, cm, e.w) + (fmaf(e.x, t, -ct) + fmaf(e.x, sn, e.y * t));
    // the tabled value is 0 or above the product: the sum's rounding is exact this way
    const float c1 = e.x - st, s1 = e.z + ct;
    cos_out = (c1 + (((e.x - c1) - st) + c_low)) * amp;
    sin_out = (s1 + (((e.z - s1) + ct) + s_low)) * amp;
}
// x c - y s: both products and the sum rounded.
__device__ __forceinline__ float rope_turn(float x, float y, float c, float s) {
    return __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
}

}  // namespace fa
