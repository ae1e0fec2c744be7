// k_store.cu -- writing and reading the 4-bit key/value store.
//
// hga_store_kv: a row's 128 elements fall into 8 blocks of 16; a block's
// scale is the E4M3 number nearest amax / (6 * tensor scale) and its codes
// the E2M1 numbers nearest x / (scale * tensor scale). Keys may be rotated
// on the way, in 64 bits and rounded once to fp32: an error of the angle near
// a border between two codes would move the stored value by a third.
// hga_load_kv: code * scale (exact in f16) * tensor scale, rounded once to
// bf16. Both are memory-bound (256 bytes of bf16 against 72 of the store per
// row and tensor), so what counts is that every access of a warp covers whole
// sectors, with a few loads in flight per thread, and few instructions per
// element (a correctly rounded quotient in three). 64K tokens x 4 heads (172
// MB each way): written in 38 us, bound by instructions; read back in 31.5 us,
// 0.83 of the copy bandwidth (36 under a tensor scale of more than 18 bits, whose
// products take more instructions to round once). Keys rotated by positions on the
// way make that 121 us: every KV head makes a token's angles again, in 64 bits.
#include <string.h>

#include "hga_e2m1.cuh"
#include "hga_kernels.h"
#include "hga_turn.cuh"

namespace hga {

namespace {

using e2m1::kBlock;
using bf = __nv_bfloat16;

constexpr int kStoreThreads = 256;

// One launch's rows, those of `units` units from u0 on, d tokens each, numbered
// unit by unit; row / d by multiplication, (mulhi(row, m) + row) >> s with s =
// ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1 (Granlund and Montgomery),
// right for rows below 2^31.
constexpr int64_t kRowsPerLaunch = 1 << 22;  // 16 lanes each and a grid past them fit 31 bits
static_assert((int64_t)kMaxChunks * 8 * kGroupRows <= kRowsPerLaunch, "a unit fits one launch");

struct Rows {
    uint32_t d, m, s, n;  // n: rows
    int64_t u0;
    Rows(int64_t u0_, int64_t units, int64_t tokens)
        : d((uint32_t)tokens), s(0), n((uint32_t)(units * tokens)), u0(u0_) {
        while (((uint64_t)1 << s) < d) ++s;
        m = (uint32_t)(((uint64_t)1 << 32) * (((uint64_t)1 << s) - d) / d + 1);
    }
    __device__ __forceinline__ void find(uint32_t row, int64_t& unit, int& token) const {
        const uint32_t u = (__umulhi(row, m) + row) >> s;
        unit = u0 + u;
        token = (int)(row - u * d);
    }
};

// f(Rows) for each launch of a call.
template <typename F>
cudaError_t each_launch(int64_t units, int64_t n_tokens, F f) {
    const int64_t per = kRowsPerLaunch / n_tokens;
    for (int64_t u = 0; u < units; u += per) {
        f(Rows(u, units - u < per ? units - u : per, n_tokens));
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Where position `at` of unit bh is in a store: its page; *row: within it.
__device__ __forceinline__ int64_t page_of(const Params& p, int64_t bh, int at, int* row) {
    *row = at % kGroupRows;
    return bh * p.kv_slab + (int64_t)(at / kGroupRows) * kE2m1Page;
}

// Rows as they are. Item = (row, block): row * 8 + block, so eight lanes hold
// the eight blocks of a row; its scales are written four bytes at a time.
__device__ __forceinline__ void store_rows(const Params& p, const bf* src, uint8_t* store, float ts,
                                           int pos0, const Rows& rows) {
    const e2m1::TensorScale tensor = e2m1::tensor_scale(ts);
    const int blk = threadIdx.x & 7;
    const uint32_t n_items = rows.n * 8;
    // whole warps stay to the end: their lanes exchange scales
    for (uint32_t it = blockIdx.x * kStoreThreads + threadIdx.x; (it & ~31u) < n_items;
         it += gridDim.x * kStoreThreads) {
        const bool ok = it < n_items;
        int64_t bh;
        int t;
        rows.find(ok ? it >> 3 : 0, bh, t);
        const uint4* src16 =
            reinterpret_cast<const uint4*>(src + (bh * rows.d + t) * 128 + kBlock * blk);
        const uint4 r0 = src16[0], r1 = src16[1];
        const uint32_t w[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
        // the largest magnitude as bits; infinities and NaN are the largest
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        m = max(m >> 16, m & 0xffffu);
        const e2m1::Scale sc = e2m1::block_scale(__uint_as_float(m << 16), tensor);
        float x[kBlock];
        bf16x8_to_f32(r0, x);
        bf16x8_to_f32(r1, x + 8);
        int pr;
        uint8_t* pg = store + page_of(p, bh, pos0 + t, &pr);
        if (ok)
            *reinterpret_cast<uint2*>(pg + e2m1::code_at(pr, kBlock * blk)) =
                make_uint2(e2m1::codes_of(x, sc), e2m1::codes_of(x + 8, sc));
        uint32_t four = sc.code << (8 * (blk & 3));
        four |= __shfl_xor_sync(0xffffffffu, four, 1);
        four |= __shfl_xor_sync(0xffffffffu, four, 2);
        if (ok && (blk & 3) == 0) *reinterpret_cast<uint32_t*>(pg + e2m1::scale_at(pr, blk)) = four;
    }
}

// Keys rotated on the way. 16 lanes a row, each with 4 rotary pairs: dims
// 4l .. + 3 and 64 + 4l .. + 3. Item = (row, lane): row * 16 + lane.
__device__ __forceinline__ void store_rotated(const Params& p, const AxisMap& am,
                                              const int32_t* pos, const bf* k, uint8_t* ks,
                                              int pos0, const Rows& rows) {
    const e2m1::TensorScale tensor = e2m1::tensor_scale(p.k_scale);
    const int l = threadIdx.x & 15;
    const uint32_t n_items = rows.n * 16;
    // this lane's pairs, read once (the constant cache serves one index at a time)
    double freq[4];
    int axis[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        freq[e] = p.inv_freq[4 * l + e];
        axis[e] = am.axis[4 * l + e];
    }
    for (uint32_t it = blockIdx.x * kStoreThreads + threadIdx.x; (it & ~31u) < n_items;
         it += gridDim.x * kStoreThreads) {
        const bool ok = it < n_items;
        int64_t bh;
        int t;
        rows.find(ok ? it >> 4 : 0, bh, t);
        const int at = pos0 + t;
        const uint2* src8 =
            reinterpret_cast<const uint2*>(k + (bh * rows.d + t) * 128 + 4 * l);
        const uint2 lo = src8[0], hi = src8[16];
        const uint32_t wl[2] = {lo.x, lo.y}, wh[2] = {hi.x, hi.y};
        float x[2][4];  // dims 4l .. and 64 + 4l ..
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = __uint_as_float((e & 1) ? wl[e >> 1] & 0xffff0000u : wl[e >> 1] << 16);
            const float b = __uint_as_float((e & 1) ? wh[e >> 1] & 0xffff0000u : wh[e >> 1] << 16);
            x[0][e] = a;
            x[1][e] = b;
            if (axis[e] >= 0) {
                const double at_axis =
                    pos ? (double)pos[(axis[e] * (int64_t)p.B + bh / p.Hkv) * rows.d + t]
                        : (double)at;
                double c, sn;
                turn_cs64(at_axis, freq[e], c, sn);
                x[0][e] = (float)((double)a * c - (double)b * sn);
                x[1][e] = (float)((double)a * sn + (double)b * c);
            }
        }
        int pr;
        uint8_t* pg = ks + page_of(p, bh, at, &pr);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            float amax = 0.f;  // NaN if any element of the block is
#pragma unroll
            for (int e = 0; e < 4; ++e) amax = e2m1::max_nan(amax, fabsf(x[y][e]));
            amax = e2m1::max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = e2m1::max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const e2m1::Scale sc = e2m1::block_scale(amax, tensor);
            const float four[8] = {x[y][0], x[y][1], x[y][2], x[y][3], 0.f, 0.f, 0.f, 0.f};
            const uint32_t w = e2m1::codes_of(four, sc) & 0xffffu;
            // four lanes' 16 bits of codes to the first of them
            const uint32_t w1 = w | (__shfl_down_sync(0xffffffffu, w, 1) << 16);
            const uint32_t w2 = __shfl_down_sync(0xffffffffu, w1, 2);
            const int blk = 4 * y + (l >> 2);
            if (ok && (l & 3) == 0) {
                *reinterpret_cast<uint2*>(pg + e2m1::code_at(pr, kBlock * blk)) = make_uint2(w1, w2);
                pg[e2m1::scale_at(pr, blk)] = (uint8_t)sc.code;
            }
        }
    }
}

// grid.y = 0: keys, 1: values.
template <bool kRotate>
__global__ void __launch_bounds__(kStoreThreads) store_kv_kernel(
    const __grid_constant__ Params p, const __grid_constant__ AxisMap am,
    const int32_t* __restrict__ pos, const bf* __restrict__ k, const bf* __restrict__ v,
    uint8_t* __restrict__ ks, uint8_t* __restrict__ vs, int pos0, Rows rows) {
    if (blockIdx.y == 1)
        store_rows(p, v, vs, p.v_scale, pos0, rows);
    else if (kRotate)
        store_rotated(p, am, pos, k, ks, pos0, rows);
    else
        store_rows(p, k, ks, p.k_scale, pos0, rows);
}

// grid.y = 0: keys, 1: values. Item = (row, 8 dims): row * 16 + piece; a
// thread has kLoadItems of them in flight, a grid apart. kExact: code x block scale
// times either tensor scale is an fp32 number.
constexpr int kLoadItems = 4;

template <bool kExact>
__global__ void __launch_bounds__(kStoreThreads) load_kv_kernel(
    const __grid_constant__ Params p, const uint8_t* __restrict__ ks,
    const uint8_t* __restrict__ vs, bf* __restrict__ k, bf* __restrict__ v, int pos0,
    Rows rows) {
    const uint8_t* store = blockIdx.y ? vs : ks;
    bf* dst = blockIdx.y ? v : k;
    const float ts = blockIdx.y ? p.v_scale : p.k_scale;
    const int pc = threadIdx.x & 15;
    const uint32_t n_items = rows.n * 16, step = gridDim.x * kStoreThreads;
    for (uint32_t it = blockIdx.x * kStoreThreads + threadIdx.x; it < n_items;
         it += step * kLoadItems) {
        int64_t dst_row[kLoadItems];
        uint32_t w[kLoadItems];
        uint8_t sc[kLoadItems];
#pragma unroll
        for (int i = 0; i < kLoadItems; ++i) {
            const uint32_t x = it + step * i;
            if (x < n_items) {
                int64_t bh;
                int t;
                rows.find(x >> 4, bh, t);
                dst_row[i] = bh * rows.d + t;
                int pr;
                const uint8_t* pg = store + page_of(p, bh, pos0 + t, &pr);
                w[i] = *reinterpret_cast<const uint32_t*>(pg + e2m1::code_at(pr, 8 * pc));
                sc[i] = pg[e2m1::scale_at(pr, pc >> 1)];
            }
        }
#pragma unroll
        for (int i = 0; i < kLoadItems; ++i) {
            const uint32_t x = it + step * i;
            if (x < n_items) {
                const uint32_t s2 = e2m1::scales_to_f16x2((uint16_t)(sc[i] * 0x101u));
                uint32_t f[4];
                e2m1::codes_to_f16x2(w[i], f);
                float o[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t h = e2m1::hmul2(f[e], s2);
                    const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&h));
                    o[2 * e] = kExact ? r.x * ts : e2m1::mul_to_odd(r.x, ts);
                    o[2 * e + 1] = kExact ? r.y * ts : e2m1::mul_to_odd(r.y, ts);
                }
                *reinterpret_cast<uint4*>(dst + dst_row[i] * 128 + 8 * pc) = f32x8_to_bf16(o);
            }
        }
    }
}

// CTAs for `items` threads, at most 16 an SM.
unsigned grid_of(int64_t items) {
    const int64_t blocks = (items + kStoreThreads - 1) / kStoreThreads;
    return (unsigned)(blocks < 148 * 16 ? blocks : 148 * 16);
}

}  // namespace

cudaError_t launch_store_kv(const Params& p, const AxisMap& am, const int32_t* positions,
                            const void* k, const void* v, void* k_store, void* v_store,
                            int64_t pos0, int64_t n_tokens, cudaStream_t st) {
    const bool rotate = am.n_axes > 0;
    auto* kernel = rotate ? store_kv_kernel<true> : store_kv_kernel<false>;
    return each_launch((int64_t)p.B * p.Hkv, n_tokens, [&](const Rows& rows) {
        kernel<<<dim3(grid_of((int64_t)rows.n * (rotate ? 16 : 8)), 2), kStoreThreads, 0, st>>>(
            p, am, positions, (const bf*)k, (const bf*)v, (uint8_t*)k_store, (uint8_t*)v_store,
            (int)pos0, rows);
    });
}

// Code x block scale has 6 significant bits and is 2^-10 at least, so 18 bits of a
// tensor scale far above fp32's smallest are exact.
static bool exact_scale(float ts) {
    uint32_t bits;
    memcpy(&bits, &ts, sizeof(bits));
    return (bits & 0x3fu) == 0u && ts > 0x1p-100f;
}

cudaError_t launch_load_kv(const Params& p, const void* k_store, const void* v_store, void* k,
                           void* v, int64_t pos0, int64_t n_tokens, cudaStream_t st) {
    auto* kernel = exact_scale(p.k_scale) && exact_scale(p.v_scale) ? load_kv_kernel<true>
                                                                    : load_kv_kernel<false>;
    return each_launch((int64_t)p.B * p.Hkv, n_tokens, [&](const Rows& rows) {
        const int64_t threads = ((int64_t)rows.n * 16 + kLoadItems - 1) / kLoadItems;
        kernel<<<dim3(grid_of(threads), 2), kStoreThreads, 0, st>>>(
            p, (const uint8_t*)k_store, (const uint8_t*)v_store, (bf*)k, (bf*)v, (int)pos0, rows);
    });
}

}  // namespace hga
