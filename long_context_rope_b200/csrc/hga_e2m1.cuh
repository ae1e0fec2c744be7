// hga_e2m1.cuh -- the 4-bit key/value store: pages, codes and block scales.
//
// A page holds the rows of 16 tokens of one tensor (d = 128): the codes as
// four tiles of 32 dims, each 16 rows x 16 bytes, then 16 rows x 8 E4M3
// scales (one per 16 dims). Tiles, not whole rows: 16-byte pieces of a row
// that a kernel can place freely in shared memory.
#pragma once

#include "hga_common.cuh"

namespace hga {
namespace e2m1 {

constexpr int kBlock = 16;           // dims that share a scale
constexpr int kScales = 128 / kBlock;

// Byte offsets in a page.
__host__ __device__ constexpr int code_at(int row, int dim) {
    return (dim >> 5) * (kGroupRows * 16) + row * 16 + ((dim & 31) >> 1);
}
__host__ __device__ constexpr int scale_at(int row, int block) {
    return kE2m1Codes + row * kScales + block;
}

// Eight codes (bits 4i..4i+3 of w) to four f16 pairs; exact, as every E2M1
// number is an f16 number.
__device__ __forceinline__ void codes_to_f16x2(uint32_t w, uint32_t (&f)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
        : "r"(w));
}

// v * ts cut to fp32, its last bit set where anything was cut off: rounded on to bf16
// that is the product rounded once. (A product rounded to fp32 first may come to lie
// halfway between two bf16 numbers, and then go the wrong way.)
__device__ __forceinline__ float mul_to_odd(float v, float ts) {
    const float q = __fmul_rz(v, ts);
    const bool cut = __fmaf_ru(fabsf(v), ts, -fabsf(q)) > 0.f;  // rounded up: never lost
    return __uint_as_float(__float_as_uint(q) | (cut ? 1u : 0u));
}

// Eight floats to codes, nearest even, at most 6 in magnitude.
__device__ __forceinline__ uint32_t f32x8_to_codes(const float* q) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return w;
}

// The E4M3 code of x >= 0, nearest even, at most 448.
__device__ __forceinline__ uint32_t scale_code(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xffu;
}

// Two E4M3 codes (low and high byte) to an f16 pair, exact.
__device__ __forceinline__ uint32_t scales_to_f16x2(uint16_t x) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
    return r;
}

__device__ __forceinline__ float scale_value(uint32_t code) {
    const uint32_t h = scales_to_f16x2((uint16_t)code);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a),
                              *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// An f16 pair times the low (half 0) or high (half 1) element of c.
__device__ __forceinline__ uint32_t hmul2_half(uint32_t a, uint32_t c, int half) {
    const __half2 c2 = *reinterpret_cast<const __half2*>(&c);
    const __half2 d = half ? __high2half2(c2) : __low2half2(c2);
    return hmul2(a, *reinterpret_cast<const uint32_t*>(&d));
}

// The low half of every byte of a, and the high half of every byte of b.
__device__ __forceinline__ uint32_t select_nibbles(uint32_t a, uint32_t b) {
    return (a & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
}

// Maximum that is NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// The tensor scale with what a block's scale needs of it. slow: its quotients
// by an ordinary divide (a magnitude whose reciprocal or remainders could leave
// fp32's normal range).
struct TensorScale {
    float ts, six, inv_six;
    bool slow;
};

__device__ __forceinline__ TensorScale tensor_scale(float ts) {
    return {ts, 6.f * ts, __frcp_rn(6.f * ts), !(ts > 0x1p-80f && ts < 0x1p80f)};
}

// x / d, correctly rounded, with inv = 1 / d rounded: the product, then
// Markstein's correction by the exact remainder (whose sign is taken so that a
// zero keeps its own). Halfway quotients, exact ones among them, are met
// exactly. For normal d and inv, and |x / d| well inside fp32's range.
__device__ __forceinline__ float quotient(float x, float d, float inv) {
    const float q = x * inv;
    return fmaf(-fmaf(q, d, -x), inv, q);
}

// A block's scale by the rounding that hga_store_kv states: its code, S = its
// value times the tensor scale, 1 / S. none: all codes are 0 (a zero scale, or a
// NaN or an infinity in the block, whose scale is then NaN). slow: as above, or
// a saturated scale, whose quotients may be huge.
struct Scale {
    uint32_t code;
    float S, inv;
    bool none, slow;
};

__device__ __forceinline__ Scale block_scale(float amax, const TensorScale& t) {
    Scale r;
    const bool finite = amax < INFINITY;
    // at most 512 before the correction, so that it cannot overflow; anything
    // above 448 is 448
    const float q = fminf(amax * t.inv_six, 512.f);
    const float a = t.slow ? amax / t.six : fmaf(-fmaf(q, t.six, -amax), t.inv_six, q);
    r.code = finite ? scale_code(a) : 0x7fu;
    r.S = scale_value(r.code) * t.ts;
    r.none = !(r.S > 0.f);  // NaN too
    if (r.none && finite) r.code = 0u;
    r.slow = t.slow || r.code == 0x7eu;
    r.inv = __frcp_rn(r.S);
    return r;
}

// Eight elements' codes under a scale.
__device__ __forceinline__ uint32_t codes_of(const float* x, const Scale& s) {
    float q[8];
    if (s.slow) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = x[e] / s.S;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = quotient(x[e], s.S, s.inv);
    }
    return s.none ? 0u : f32x8_to_codes(q);
}

}  // namespace e2m1
}  // namespace hga
