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

// A block's scale by the rounding that hga_store_kv states: its code, S = its
// value times the tensor scale, 1 / S. none: all codes 0 (a zero scale, or a
// NaN or infinity in the block, whose scale is then NaN). slow: quotients by
// an ordinary divide (saturated scales, whose quotients may be huge, and
// magnitudes whose reciprocal or remainder could leave fp32's normal range).
struct Scale {
    uint32_t code;
    float S, inv;
    bool none, slow;
};

__device__ __forceinline__ Scale block_scale(float amax, float ts) {
    Scale r;
    const bool finite = amax < INFINITY;
    r.code = finite ? scale_code(amax / (6.f * ts)) : 0x7fu;
    r.S = scale_value(r.code) * ts;
    r.none = !(r.S > 0.f);  // NaN too
    if (r.none && finite) r.code = 0u;
    r.slow = r.code == 0x7eu || r.S < 0x1p-80f || r.S > 0x1p80f;
    r.inv = __frcp_rn(r.S);
    return r;
}

// x / S, correctly rounded: the product with the rounded reciprocal, then
// Markstein's correction by the exact remainder. Of bf16 elements and a
// power-of-two tensor scale the quotients that lie halfway between two codes
// are met exactly. (A divide per element made the store compute-bound.)
__device__ __forceinline__ float quotient(float x, const Scale& s) {
    if (s.none) return 0.f;
    if (s.slow) return x / s.S;
    const float q = x * s.inv;
    return copysignf(fmaf(fmaf(-q, s.S, x), s.inv, q), x);
}

}  // namespace e2m1
}  // namespace hga
