// hga_decode_pages.cuh -- the attention half of single-token decode over the
// 4-bit store (HGA_KV_E2M1), shared by the decode attention kernel and the
// one-launch decode steps.
//
// One query token, gq <= 8 query heads of one KV head. Every warp takes pages
// of its own (16 keys: 1152 bytes of K and of V) through a private ring of
// shared-memory stages, filled with 16-byte asynchronous copies: a warp waits
// only for its own copies, so there is no producer, no barrier and no wait
// between warps until the end. (One producer thread with a bulk copy per page
// and tensor needed 600 cycles a page, 16 x 32K keys 18.5 us; 8 lanes that
// issue side by side 270.)
//
// Products are warp-level fp16 MMA (m16n8k16, fp32 accumulate): S^T[16 keys x
// 8 heads] = K Q^T and O^T[128 dims x 8 heads] += V^T P^T. Code x block scale
// has at most 6 significant bits and is exact in fp16. The MMA's k and m
// indices are permuted so that a lane's codes are contiguous and meet one or
// two block scales. Lane (g, t4):
//   keys    rows g and g + 8, dims 32 t4 .. + 31 (16 bytes of tile t4 each):
//           step kk multiplies dims 32 t4 + 4 kk + {0, 1} and {2, 3};
//   values  keys 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9, dims 16 g .. + 15 (8
//           bytes each): a shift and a select give bytes that hold one dim of
//           two keys, the pair that one convert instruction widens; output
//           row g of MMA tile mt is dim 16 g + mt, row g + 8 dim 16 g + 8 + mt.
// 16-byte piece (tile t, row r) of a page's codes lies at row r ^ swz(t) of
// its tile in shared memory, which frees both reads of bank conflicts.
//
// Online softmax in fp32 with a lazily raised maximum: the weights 2^(s - m)
// are computed against a maximum m that is raised (and the accumulators
// rescaled) only when a score exceeds it by more than 8; weights stay below
// 2^8, far inside fp16, and nearly every page is spared the maximum over
// lanes and the rescaling. Weights are rounded to fp16 and summed as rounded.
// A NaN score makes its head's weight, sum and output NaN.
#pragma once

#include "hga_decode_core.cuh"
#include "hga_e2m1.cuh"

namespace hga {
namespace dec {

constexpr int kPageStages = 3;                // pages in flight per warp
constexpr int kPagePair = 2 * kE2m1Page;      // K page, then V page
constexpr int kPageVecs = kE2m1Page / 16;     // 72 16-byte pieces
constexpr int kPageCopies = (2 * kPageVecs + 31) / 32;
constexpr float kRaise = 8.0f;

// kWarps: warps of the CTA that take pages.
template <int kWarps>
struct PageSmem {
    union {
        alignas(128) uint8_t page[kWarps][kPageStages][kPagePair];
        alignas(16) float part[kWarps][8][kOStride];  // per warp and head: O, reused
    } u;
    float m[kWarps][8], l[kWarps][8];          // per warp and head: max, sum
    alignas(16) Owned owned;                   // partials of the heads this CTA finalises
};

// Stores of pages, `slab` bytes from one sequence and KV head to the next.
struct PageSource {
    const uint8_t* k;
    const uint8_t* v;
    int64_t slab;
};

__host__ __device__ constexpr int64_t page_slab(int64_t rows) {
    return (rows + kGroupRows - 1) / kGroupRows * kE2m1Page;
}

// A lane's view of a block's page pair: K page + 16 lane and V page + 16 (lane -
// 8) (a base that is offset once costs one multiply-add per page and tensor).
struct PageRef {
    const uint8_t* k;
    const uint8_t* v;
};
__device__ __forceinline__ PageRef lane_pages(const uint8_t* k, const uint8_t* v) {
    const int lane = threadIdx.x & 31;
    return {k + 16 * lane, v + 16 * (lane - 8)};
}
__device__ __forceinline__ PageRef page_at(const PageRef& base, int page) {
    const int64_t at = (int64_t)page * kE2m1Page;
    return {base.k + at, base.v + at};
}

__device__ __forceinline__ int swz(int tile) { return 2 * tile + (tile & 1); }

// Where a tile's piece of row r starts.
__device__ __forceinline__ int code_piece(int tile, int r) {
    return tile * (kGroupRows * 16) + ((r ^ swz(tile)) << 4);
}

// Q^T as MMA B fragments in fp16, in the keys' permutation; heads >= gq are
// zero. Each head is scaled by a power of two to at most 2^15 first, so
// bf16's whole range is held; the inverse is in sc, the score factors (log2
// units) of heads 2 t4 and 2 t4 + 1.
__device__ __forceinline__ void load_q_pages(const Params& p, const __nv_bfloat16* q, int b, int h,
                                             uint32_t (&qf)[8][2], float (&sc)[2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const bool okh = g < p.gq;
    const __nv_bfloat16* qr =
        q + ((int64_t)b * p.q_len * p.Hq + (int64_t)h * p.gq + (okh ? g : 0)) * kD + 32 * t4;
    uint4 raw[4];
#pragma unroll
    for (int w = 0; w < 4; ++w)
        raw[w] = okh ? *reinterpret_cast<const uint4*>(qr + 8 * w) : make_uint4(0u, 0u, 0u, 0u);
    // the head's largest exponent (bf16 bits 14..7), over its four lanes
    uint32_t big = 0u;
#pragma unroll
    for (int w = 0; w < 4; ++w)
        for (uint32_t x : {raw[w].x, raw[w].y, raw[w].z, raw[w].w})
            big = max(big, max((x >> 23) & 0xffu, (x >> 7) & 0xffu));
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // 2^(14 - e) for a largest exponent e = big - 127, from 2^-113 to 2^100; 1
    // for infinities and NaN
    const int e = big == 255u ? 0 : min(141 - (int)big, 100);
    const float up = __int_as_float((e + 127) << 23);
    const float down = __int_as_float((127 - e) << 23);
    const float sc0 = 1.4426950408889634f / sqrtf((float)kD) * p.k_scale;
    sc[0] = sc0 * __shfl_sync(0xffffffffu, down, 8 * t4);
    sc[1] = sc0 * __shfl_sync(0xffffffffu, down, 8 * t4 + 4);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const __nv_bfloat162* h2 = reinterpret_cast<const __nv_bfloat162*>(&raw[w]);
        uint32_t f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __bfloat1622float2(h2[i]);
            const __half2 hv = __floats2half2_rn(v.x * up, v.y * up);
            f[i] = *reinterpret_cast<const uint32_t*>(&hv);
        }
        qf[2 * w][0] = f[0];
        qf[2 * w][1] = f[1];
        qf[2 * w + 1][0] = f[2];
        qf[2 * w + 1][1] = f[3];
    }
}

// The warp's asynchronous copies of a page pair into a stage: 72 pieces of K,
// then 72 of V, piece lane + 32 u to dst[u].
struct CopyPlan {
    uint32_t dst[kPageCopies];
};
__device__ __forceinline__ CopyPlan copy_plan() {
    const int lane = threadIdx.x & 31;
    CopyPlan c;
#pragma unroll
    for (int u = 0; u < kPageCopies; ++u) {
        const int i = lane + 32 * u, pc = i >= kPageVecs ? i - kPageVecs : i;
        c.dst[u] = (i >= kPageVecs ? kE2m1Page : 0) + (pc < 64 ? code_piece(pc >> 4, pc & 15) : pc * 16);
    }
    return c;
}
__device__ __forceinline__ void copy_pages(const CopyPlan& c, uint32_t stage, const PageRef& r) {
    static_assert(kPageVecs == 72 && kPageCopies == 5, "the split of the pieces over copies");
    const int lane = threadIdx.x & 31;
    ptx::cp_async16(stage + c.dst[0], r.k);
    ptx::cp_async16(stage + c.dst[1], r.k + 512);
    ptx::cp_async16(stage + c.dst[2], lane < 8 ? r.k + 1024 : r.v);
    ptx::cp_async16(stage + c.dst[3], r.v + 512);
    if (lane < 16) ptx::cp_async16(stage + c.dst[4], r.v + 1024);
}

// The warp's blocks 0 .. n - 1: page_of(i) their pages, pos_of(i) the position
// of their first token; qpos: the query's position. Keys after it are masked,
// and their values' scales read as zero (their rows may hold anything).
template <typename PageOf, typename PosOf>
__device__ __forceinline__ void consume_pages(const uint32_t (&qf)[8][2], const float (&sc)[2],
                                              uint8_t (*ring)[kPagePair], int n, int qpos,
                                              PageOf page_of, PosOf pos_of, WarpAcc& acc) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const CopyPlan plan = copy_plan();
    const uint32_t ring0 = ptx::smem_u32(ring[0]);
    float mz[2] = {0.f, 0.f};  // the maximum, 0 while there is none
    float top[2] = {-INFINITY, -INFINITY};  // the score above which it is raised
#pragma unroll
    for (int d = 0; d < kPageStages; ++d) {
        if (d < n) copy_pages(plan, ring0 + d * kPagePair, page_of(d));
        ptx::cp_async_commit();
    }
    // this lane's places in a stage: its key rows g (and g + 8, 128 bytes on) and
    // their scales; its value rows 2 t4 and 2 t4 + 1 (and 8 more) and theirs
    const int key_at = code_piece(t4, g), key_sc = e2m1::scale_at(g, 2 * t4);
    const int val_at[2] = {kE2m1Page + code_piece(g >> 1, 2 * t4) + 8 * (g & 1),
                           kE2m1Page + code_piece(g >> 1, 2 * t4 + 1) + 8 * (g & 1)};
    const int val_sc = kE2m1Page + e2m1::scale_at(2 * t4, g);
    int st = 0;  // the stage's offset in the ring
    for (int i = 0; i < n; ++i) {
        ptx::cp_async_wait<kPageStages - 1>();
        __syncwarp();
        const uint8_t* stage = ring[0] + st;
        const int kp = pos_of(i);
        float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
        {
            const uint4 w0 = *reinterpret_cast<const uint4*>(stage + key_at);
            const uint4 w1 = *reinterpret_cast<const uint4*>(stage + key_at + 128);
            const uint32_t c0 =
                e2m1::scales_to_f16x2(*reinterpret_cast<const uint16_t*>(stage + key_sc));
            const uint32_t c1 =
                e2m1::scales_to_f16x2(*reinterpret_cast<const uint16_t*>(stage + key_sc + 64));
            const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t f0[4], f1[4];
                e2m1::codes_to_f16x2(a0[w], f0);
                e2m1::codes_to_f16x2(a1[w], f1);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f0[e] = e2m1::hmul2_half(f0[e], c0, w >> 1);
                    f1[e] = e2m1::hmul2_half(f1[e], c1, w >> 1);
                }
                uint32_t x[4] = {f0[0], f1[0], f0[1], f1[1]};
                ptx::mma_16816_f16(s0, x, qf[2 * w][0], qf[2 * w][1]);
                uint32_t y[4] = {f0[2], f1[2], f0[3], f1[3]};
                ptx::mma_16816_f16(s1, y, qf[2 * w + 1][0], qf[2 * w + 1][1]);
            }
        }
        // this lane: keys g (elements 0, 1) and g + 8 (2, 3), heads 2 t4, 2 t4 + 1
        float s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = (s0[e] + s1[e]) * sc[e & 1];
        const bool partial = kp + kGroupRows - 1 > qpos;
        if (partial) {
            if (kp + g > qpos) s[0] = s[1] = -INFINITY;
            if (kp + g + 8 > qpos) s[2] = s[3] = -INFINITY;
        }
        const bool raise = fmaxf(s[0], s[2]) > top[0] || fmaxf(s[1], s[3]) > top[1];
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                float mb = fmaxf(s[hh], s[hh + 2]);
                mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 4));
                mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 8));
                mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 16));
                const float mn = fmaxf(acc.m[hh], mb);
                if (mn != -INFINITY) {
                    const float alpha = ptx::ex2_approx(acc.m[hh] - mn);  // 0 from -inf
                    acc.m[hh] = mz[hh] = mn;
                    top[hh] = mn + kRaise;
                    acc.l[hh] *= alpha;
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt) {
                        acc.o[mt][hh] *= alpha;
                        acc.o[mt][hh + 2] *= alpha;
                    }
                }
            }
        }
        uint32_t pb[2];
#pragma unroll
        for (int k8 = 0; k8 < 2; ++k8) {
            const __half2 h2 = __floats2half2_rn(ptx::ex2_approx(s[2 * k8] - mz[0]),
                                                 ptx::ex2_approx(s[2 * k8 + 1] - mz[1]));
            const float2 r = __half22float2(h2);
            acc.l[0] += r.x;
            acc.l[1] += r.y;
            // [keys x heads] to the B fragment's [heads x keys]
            pb[k8] = ptx::movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h2));
        }
        {
            uint2 w[4];         // keys 2 t4 + {0, 1, 8, 9}: dims 16 g .. + 15
            uint32_t c[4];      // their scale bytes
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                w[x] = *reinterpret_cast<const uint2*>(stage + val_at[x & 1] + 128 * (x >> 1));
                c[x] = stage[val_sc + 8 * (x & 1) + 64 * (x >> 1)];
            }
            if (partial) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (kp + 2 * t4 + (x & 1) + 8 * (x >> 1) > qpos) c[x] = 0u;
            }
            const uint32_t c0 = e2m1::scales_to_f16x2((uint16_t)(c[0] | (c[1] << 8)));
            const uint32_t c1 = e2m1::scales_to_f16x2((uint16_t)(c[2] | (c[3] << 8)));
            // f[keys' half][word][odd][i]: dim 8 word + 2 i + odd of both keys
            uint32_t f[2][2][2][4];
#pragma unroll
            for (int k8 = 0; k8 < 2; ++k8)
#pragma unroll
                for (int wd = 0; wd < 2; ++wd) {
                    const uint32_t a = wd ? w[2 * k8].y : w[2 * k8].x;
                    const uint32_t b = wd ? w[2 * k8 + 1].y : w[2 * k8 + 1].x;
                    e2m1::codes_to_f16x2(e2m1::select_nibbles(a, b << 4), f[k8][wd][0]);
                    e2m1::codes_to_f16x2(e2m1::select_nibbles(a >> 4, b), f[k8][wd][1]);
#pragma unroll
                    for (int o = 0; o < 2; ++o)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            f[k8][wd][o][e] = e2m1::hmul2(f[k8][wd][o][e], k8 ? c1 : c0);
                }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                const int o = mt & 1, e = mt >> 1;
                uint32_t x[4] = {f[0][0][o][e], f[0][1][o][e], f[1][0][o][e], f[1][1][o][e]};
                ptx::mma_16816_f16(acc.o[mt], x, pb[0], pb[1]);
            }
        }
        __syncwarp();  // every lane is done with the stage
        if (i + kPageStages < n) copy_pages(plan, ring0 + st, page_of(i + kPageStages));
        ptx::cp_async_commit();
        st = st == (kPageStages - 1) * kPagePair ? 0 : st + kPagePair;
    }
}

// Four output places 4 lane .. + 3 of a head (place mt * 16 + 8 y + g holds dim
// 16 g + 8 y + mt), normalised. A sum of 0: no visible key, zeros.
__device__ __forceinline__ void store_places(const Params& p, float4 num, float den,
                                             __nv_bfloat16* row) {
    const int lane = threadIdx.x & 31;
    const float inv = den == 0.f ? 0.f : p.v_scale / den;
    const float v[4] = {num.x, num.y, num.z, num.w};
    const int d0 = 64 * (lane & 1) + 8 * ((lane >> 1) & 1) + (lane >> 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) row[d0 + 16 * i] = __float2bfloat16_rn(v[i] * inv);
}

// All threads of the CTA: joins the partials of the CTA's warps, then of
// the cluster's CTAs (CTA n % CL finalises head n), and writes the output
// rows. Sums in warp and CTA order.
template <int kWarps>
__device__ __forceinline__ void merge_pages(PageSmem<kWarps>& sm, cg::cluster_group& cluster,
                                            const Params& p, const WarpAcc& acc, int b, int h,
                                            __nv_bfloat16* out) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const int CL = (int)cluster.num_blocks(), r = (int)cluster.block_rank();
    const int per = owned_per_cta(CL);
    __nv_bfloat16* orow = out + ((int64_t)b * p.q_len * p.Hq + (int64_t)h * p.gq) * kD;
    __syncthreads();  // every warp is done with its pages
    if (warp < kWarps) {
        float* o = sm.u.part[warp][2 * t4];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            float v = acc.l[hh];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            if (g == 0) {
                sm.m[warp][2 * t4 + hh] = acc.m[hh];
                sm.l[warp][2 * t4 + hh] = v;
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                o[hh * kOStride + mt * 16 + g] = acc.o[mt][hh];
                o[hh * kOStride + mt * 16 + 8 + g] = acc.o[mt][hh + 2];
            }
        }
    }
    __syncthreads();
    auto join = [&](int count, auto m_of, auto l_of, auto o_of, float& M, float4& num, float& den) {
        M = -INFINITY;
        for (int w = 0; w < count; ++w) M = fmaxf(M, m_of(w));
        num = make_float4(0.f, 0.f, 0.f, 0.f);
        den = 0.f;
        for (int w = 0; w < count; ++w) {
            const float mw = m_of(w);
            const float wt = mw == -INFINITY ? 0.f : ptx::ex2_approx(mw - M);
            const float4 o = o_of(w);
            num.x = fmaf(wt, o.x, num.x);
            num.y = fmaf(wt, o.y, num.y);
            num.z = fmaf(wt, o.z, num.z);
            num.w = fmaf(wt, o.w, num.w);
            den = fmaf(wt, l_of(w), den);
        }
    };
    float M, den;
    float4 num;
    // warp w: heads w, w + kWarps, ..
    for (int n = warp; warp < kWarps && n < p.gq; n += kWarps) {
        join(
            kWarps, [&](int w) { return sm.m[w][n]; }, [&](int w) { return sm.l[w][n]; },
            [&](int w) { return *reinterpret_cast<const float4*>(&sm.u.part[w][n][4 * lane]); }, M,
            num, den);
        if (CL == 1) {
            store_places(p, num, den, orow + n * kD);
        } else {
            Owned* dst = cluster.map_shared_rank(&sm.owned, n % CL);
            const int slot = r * per + n / CL;
            *reinterpret_cast<float4*>(&dst->o[slot][4 * lane]) = num;
            if (lane == 0) {
                dst->m[slot] = M;
                dst->l[slot] = den;
            }
        }
    }
    if (CL == 1) return;
    cluster.sync();  // every partial is in its owner's shared memory
    for (int k = warp; warp < kWarps && r + k * CL < p.gq; k += kWarps) {
        join(
            CL, [&](int c) { return sm.owned.m[c * per + k]; },
            [&](int c) { return sm.owned.l[c * per + k]; },
            [&](int c) {
                return *reinterpret_cast<const float4*>(&sm.owned.o[c * per + k][4 * lane]);
            },
            M, num, den);
        store_places(p, num, den, orow + (r + k * CL) * kD);
    }
}

}  // namespace dec
}  // namespace hga
