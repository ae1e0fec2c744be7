// hga_turn.cuh -- cosine and sine of a rotary angle in fp32 and in 64 bits, for
// rotations whose results are kept in fp32 or rounded to codes.
#pragma once

#include "hga_common.cuh"

namespace hga {

// The angle position * inv_freq as a double product less n quarter turns: pi/2
// in two parts and fused multiply-adds, so the rest r, |r| <= pi/4, of that product
// is good to 2^-52 for any int32 position. (The product's own rounding is 2^-53 of
// the angle: 2^-22 near 2^31, 2^-37 at 2^16.) Returns n's low bits.
__device__ __forceinline__ int quarter_turns(double position, double inv_freq, double& r) {
    constexpr double kTwoOverPi = 0.63661977236758134308;
    constexpr double kPio2 = 1.57079632679489661923;          // nearest double
    constexpr double kPio2Rest = 6.12323399573676603587e-17;  // pi/2 - kPio2
    constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52: the sum's low bits are n
    const double a = position * inv_freq;
    const double t = fma(a, kTwoOverPi, kMagic);
    const double n = t - kMagic;
    r = fma(-n, kPio2, a);
    r = fma(-n, kPio2Rest, r);
    return __double2loint(t);
}

template <typename F>
__device__ __forceinline__ void by_quadrant(int q, F cr, F sr, F& c, F& s) {
    const F c0 = (q & 1) ? sr : cr, s0 = (q & 1) ? cr : sr;
    c = ((q + 1) & 2) ? -c0 : c0;
    s = (q & 2) ? -s0 : s0;
}

// cos / sin of position * inv_freq, each off by about one fp32 rounding of what the
// reduced angle has (2^-23.8 measured over the interval, before the rounding of r
// itself, whose rest is carried along); the product's rounding, above, comes on top
// at far positions. The Taylor series to r^9 and r^10; the next terms are
// below 2^-28. The fast rope_cs (2^-21.4) reduces to half a turn and takes the
// hardware's sine.
__device__ __forceinline__ void turn_cs(double position, double inv_freq, float& c, float& s) {
    double r;
    const int q = quarter_turns(position, inv_freq, r);
    const float x = (float)r, rest = (float)(r - (double)x);
    const float x2 = x * x;
    float ps = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
    ps = fmaf(x2, ps, 1.f / 120.f);
    ps = fmaf(x2, ps, -1.f / 6.f);
    float pc = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
    pc = fmaf(x2, pc, -1.f / 720.f);
    pc = fmaf(x2, pc, 1.f / 24.f);
    pc = fmaf(x2, pc, -0.5f);
    const float cr = 1.f + fmaf(x2, pc, -x * rest);
    const float sr = x + fmaf(x * x2, ps, rest * cr);
    by_quadrant(q, cr, sr, c, s);
}

// The same in 64 bits: Taylor series to r^13 and r^12, off by 2^-41 at most
// (r^14 / 14!) of what the reduced angle has, far below what moves a 4-bit code.
__device__ __forceinline__ void turn_cs64(double position, double inv_freq, double& c, double& s) {
    double x;
    const int q = quarter_turns(position, inv_freq, x);
    const double x2 = x * x;
    double ps = fma(x2, 1.0 / 6227020800.0, -1.0 / 39916800.0);
    ps = fma(x2, ps, 1.0 / 362880.0);
    ps = fma(x2, ps, -1.0 / 5040.0);
    ps = fma(x2, ps, 1.0 / 120.0);
    ps = fma(x2, ps, -1.0 / 6.0);
    double pc = fma(x2, 1.0 / 479001600.0, -1.0 / 3628800.0);
    pc = fma(x2, pc, 1.0 / 40320.0);
    pc = fma(x2, pc, -1.0 / 720.0);
    pc = fma(x2, pc, 1.0 / 24.0);
    pc = fma(x2, pc, -0.5);
    by_quadrant(q, fma(x2, pc, 1.0), fma(x * x2, ps, x), c, s);
}

}  // namespace hga
