// k_store.cu -- writing and reading the 4-bit key/value store.
//
// hga_store_kv: a row's 128 elements fall into 8 blocks of 16; a block's
// scale is the E4M3 number nearest amax / (6 * tensor scale) and its codes
// the E2M1 numbers nearest x / (scale * tensor scale). Keys may be rotated
// on the way, in 64 bits and rounded once to fp32: an error of the angle near
// a border between two codes would move the stored value by a third. hga_load_kv: code * scale (exact in f16) * tensor scale, rounded
// once to bf16. Both are memory-bound: 256 bytes of bf16 against 72 of the
// store per row and tensor.
#include "hga_e2m1.cuh"
#include "hga_kernels.h"

namespace hga {

namespace {

constexpr int kStoreThreads = 256;

__device__ __forceinline__ void load16(const __nv_bfloat16* x, float* f) {
    const uint4 a = *reinterpret_cast<const uint4*>(x);
    const uint4 b = *reinterpret_cast<const uint4*>(x + 8);
    bf16x8_to_f32(a, f);
    bf16x8_to_f32(b, f + 8);
}

// Thread (row, s): blocks s and s + 4 of the row's key, then of its value
// (dims 16s.. and 64 + 16s.., the two halves of the same rotary pairs).
__global__ void __launch_bounds__(kStoreThreads) store_kv_kernel(
    Params p, AxisMap am, const int32_t* __restrict__ pos, const __nv_bfloat16* __restrict__ k,
    const __nv_bfloat16* __restrict__ v, uint8_t* __restrict__ ks, uint8_t* __restrict__ vs,
    int64_t pos0, int64_t n_tokens, int64_t n_rows) {
    for (int64_t it = (int64_t)blockIdx.x * kStoreThreads + threadIdx.x; it < n_rows * 4;
         it += (int64_t)gridDim.x * kStoreThreads) {
        const int s = (int)(it & 3);
        const int64_t row = it >> 2, bh = row / n_tokens, t = row % n_tokens;
        const int64_t at = pos0 + t;
        const int64_t page = bh * p.kv_slab + (at / kGroupRows) * kE2m1Page;
        const int pr = (int)(at % kGroupRows);
        float a[16], b[16];
        load16(k + row * 128 + 16 * s, a);
        load16(k + row * 128 + 64 + 16 * s, b);
        if (am.n_axes > 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int i = 16 * s + e, ax = am.axis[i];
                if (ax >= 0) {
                    const double x =
                        pos ? (double)pos[((int64_t)ax * p.B + bh / p.Hkv) * n_tokens + t] : (double)at;
                    double c, sn;
                    sincos(x * p.inv_freq[i], &sn, &c);
                    const double ra = (double)a[e] * c - (double)b[e] * sn;
                    b[e] = (float)((double)a[e] * sn + (double)b[e] * c);
                    a[e] = (float)ra;
                }
            }
        }
        auto put = [&](uint8_t* store, float ts) {
            uint2 c0, c1;
            uint32_t s0, s1;
            e2m1::quantise16(a, ts, c0, s0);
            e2m1::quantise16(b, ts, c1, s1);
            uint8_t* pg = store + page;
            *reinterpret_cast<uint2*>(pg + e2m1::code_at(pr, 16 * s)) = c0;
            *reinterpret_cast<uint2*>(pg + e2m1::code_at(pr, 64 + 16 * s)) = c1;
            pg[e2m1::scale_at(pr, s)] = (uint8_t)s0;
            pg[e2m1::scale_at(pr, s + 4)] = (uint8_t)s1;
        };
        put(ks, p.k_scale);
        load16(v + row * 128 + 16 * s, a);
        load16(v + row * 128 + 64 + 16 * s, b);
        put(vs, p.v_scale);
    }
}

// Thread (row, tile): 32 dims of the key, then of the value.
__global__ void __launch_bounds__(kStoreThreads) load_kv_kernel(
    Params p, const uint8_t* __restrict__ ks, const uint8_t* __restrict__ vs,
    __nv_bfloat16* __restrict__ k, __nv_bfloat16* __restrict__ v, int64_t pos0, int64_t n_tokens,
    int64_t n_rows) {
    for (int64_t it = (int64_t)blockIdx.x * kStoreThreads + threadIdx.x; it < n_rows * 4;
         it += (int64_t)gridDim.x * kStoreThreads) {
        const int tile = (int)(it & 3);
        const int64_t row = it >> 2, bh = row / n_tokens, at = pos0 + row % n_tokens;
        const int64_t page = bh * p.kv_slab + (at / kGroupRows) * kE2m1Page;
        const int pr = (int)(at % kGroupRows);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint8_t* pg = (x ? vs : ks) + page;
            const float ts = x ? p.v_scale : p.k_scale;
            __nv_bfloat16* out = (x ? v : k) + row * 128 + 32 * tile;
            const uint4 c = *reinterpret_cast<const uint4*>(pg + e2m1::code_at(pr, 32 * tile));
            const uint16_t s2 = *reinterpret_cast<const uint16_t*>(pg + e2m1::scale_at(pr, 2 * tile));
            const uint32_t sc = e2m1::scales_to_f16x2(s2);
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t sd = i < 2 ? __byte_perm(sc, 0, 0x1010) : __byte_perm(sc, 0, 0x3232);
                uint32_t f[4];
                e2m1::codes_to_f16x2(w[i], f);
                float o[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t h = e2m1::hmul2(f[e], sd);
                    const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&h));
                    o[2 * e] = r.x * ts;
                    o[2 * e + 1] = r.y * ts;
                }
                *reinterpret_cast<uint4*>(out + 8 * i) = f32x8_to_bf16(o);
            }
        }
    }
}

unsigned grid_of(int64_t n_rows) {
    const int64_t blocks = (n_rows * 4 + kStoreThreads - 1) / kStoreThreads;
    return (unsigned)(blocks < 148 * 64 ? blocks : 148 * 64);
}

}  // namespace

cudaError_t launch_store_kv(const Params& p, const AxisMap& am, const int32_t* positions,
                            const void* k, const void* v, void* k_store, void* v_store,
                            int64_t pos0, int64_t n_tokens, cudaStream_t st) {
    using bf = __nv_bfloat16;
    const int64_t rows = (int64_t)p.B * p.Hkv * n_tokens;
    store_kv_kernel<<<grid_of(rows), kStoreThreads, 0, st>>>(
        p, am, positions, (const bf*)k, (const bf*)v, (uint8_t*)k_store, (uint8_t*)v_store, pos0,
        n_tokens, rows);
    return cudaGetLastError();
}

cudaError_t launch_load_kv(const Params& p, const void* k_store, const void* v_store, void* k,
                           void* v, int64_t pos0, int64_t n_tokens, cudaStream_t st) {
    using bf = __nv_bfloat16;
    const int64_t rows = (int64_t)p.B * p.Hkv * n_tokens;
    load_kv_kernel<<<grid_of(rows), kStoreThreads, 0, st>>>(
        p, (const uint8_t*)k_store, (const uint8_t*)v_store, (bf*)k, (bf*)v, pos0, n_tokens, rows);
    return cudaGetLastError();
}

}  // namespace hga
