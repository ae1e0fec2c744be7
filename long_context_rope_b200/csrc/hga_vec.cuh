// hga_vec.cuh -- 16-byte vectors of key / query elements as fp32, and the
// store of summary values, shared by the rotation and summary kernels.
#pragma once

#include "hga_common.cuh"

namespace hga {

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    using Raw = uint4;  // one 16-byte vector as loaded
    static __device__ __forceinline__ Raw load_raw(const __nv_bfloat16* p) {
        return __ldg(reinterpret_cast<const uint4*>(p));
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float* f) { bf16x8_to_f32(r, f); }
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* f) {
        bf16x8_to_f32(*reinterpret_cast<const uint4*>(p), f);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
        *reinterpret_cast<uint4*>(p) = f32x8_to_bf16(f);
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    using Raw = float4;
    static __device__ __forceinline__ Raw load_raw(const float* p) {
        return __ldg(reinterpret_cast<const float4*>(p));
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float* f) {
        f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
    }
    static __device__ __forceinline__ void load(const float* p, float* f) {
        float4 v = *reinterpret_cast<const float4*>(p);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    }
    static __device__ __forceinline__ void store(float* p, const float* f) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
};

// n consecutive summary values (n = 4 or 8) written as fp32, or rounded to
// bf16 (nearest even) for bf16 summary tables.
__device__ __forceinline__ void store_sum(float* out, const float* v, int n) {
    for (int i = 0; i < n; i += 4)
        *reinterpret_cast<float4*>(out + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
__device__ __forceinline__ void store_sum(__nv_bfloat16* out, const float* v, int n) {
    if (n == 8) {
        *reinterpret_cast<uint4*>(out) = f32x8_to_bf16(v);
    } else {
        __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
        *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(h);
    }
}

}  // namespace hga
