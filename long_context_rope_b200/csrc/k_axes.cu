// k_axes.cu -- rotary positions with several axes: the rotation, its inverse
// (the gradient), and the chunk / group key summaries of keys rotated so.
//
// Pair i = (dim i, dim i + d/2) of a token turns by the angle
// a = p[axis(i)] * theta_i, p the token's position on the pair's axis:
//   y_i = x_i cos a - x_{i+d/2} sin a,   y_{i+d/2} = x_i sin a + x_{i+d/2} cos a.
// The matrix is orthogonal, so the gradient of x is the rotation of y's by -a.
#include <type_traits>

#include "hga_kernels.h"
#include "hga_ptx.cuh"
#include "hga_turn.cuh"
#include "hga_vec.cuh"

namespace hga {

namespace {

// ---------------------------------------------------------------- rotation
// Memory-bound: x is read once and y written once with 16-byte accesses. The
// angles, which every row (head) of a token shares, cost a double reduction
// and two polynomials each: a CTA makes those of its `sites` (a site is one
// token of one sequence) once, spread over its threads, and keeps cos and sin
// in shared memory. Then a thread owns V pairs of one site in registers and
// turns rows of it, kBatch rows' loads in flight. Rows of a site: rr = r *
// n_heads + h, r < rep; thread (site, row lane, pair slice). 64K tokens x 32
// heads (1.07 GB) in 173 us in the same buffers again and again, 188 in others each
// time (6.2 and 5.7 TB/s); one token of 16 sequences x 32 heads in 3.0 us.
constexpr int kRopeThreads = 256;
constexpr int kBatch = 4;
constexpr int kRopeCtas = 3;
constexpr int kRopeAngles = kRopeThreads * 8;  // at most: sites x d/2

constexpr float kNoTurn = 2.f;  // in place of the cosine of a pair on no axis

// A row's V pairs (a_e, b_e) turned in place, a few elements at a time to keep
// registers few. kAll: every pair is rotated; else those on no axis are copied,
// infinities among them.
template <bool kAll>
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
    const float ya = a * c - b * s, yb = a * s + b * c;
    a = kAll || c != kNoTurn ? ya : a;
    b = kAll || c != kNoTurn ? yb : b;
}
template <typename T, bool kAll>
__device__ __forceinline__ void turn_row(float4& a, float4& b, const float* c, const float* s) {
    turn_pair<kAll>(a.x, b.x, c[0], s[0]);
    turn_pair<kAll>(a.y, b.y, c[1], s[1]);
    turn_pair<kAll>(a.z, b.z, c[2], s[2]);
    turn_pair<kAll>(a.w, b.w, c[3], s[3]);
}
template <bool kAll>
__device__ __forceinline__ void turn_bf16x2(uint32_t& a, uint32_t& b, const float* c,
                                            const float* s) {
    float a0 = __uint_as_float(a << 16), a1 = __uint_as_float(a & 0xffff0000u);
    float b0 = __uint_as_float(b << 16), b1 = __uint_as_float(b & 0xffff0000u);
    turn_pair<kAll>(a0, b0, c[0], s[0]);
    turn_pair<kAll>(a1, b1, c[1], s[1]);
    const __nv_bfloat162 ha = __floats2bfloat162_rn(a0, a1), hb = __floats2bfloat162_rn(b0, b1);
    a = *reinterpret_cast<const uint32_t*>(&ha);
    b = *reinterpret_cast<const uint32_t*>(&hb);
}
template <typename T, bool kAll>
__device__ __forceinline__ void turn_row(uint4& a, uint4& b, const float* c, const float* s) {
    turn_bf16x2<kAll>(a.x, b.x, c, s);
    turn_bf16x2<kAll>(a.y, b.y, c + 2, s + 2);
    turn_bf16x2<kAll>(a.z, b.z, c + 4, s + 4);
    turn_bf16x2<kAll>(a.w, b.w, c + 6, s + 6);
}

struct RopeShape {
    int64_t n_sites, n_tokens, rep;
    int n_heads;
    int lanes_log2;   // pair slices of a row: d/2 / V
    int rlanes_log2;  // row lanes: rows that a site's threads turn at once
    int64_t rows_cta; // rows per CTA (grid.y splits the rest)
};

template <typename T>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_axes_kernel(
    const __grid_constant__ Params p, const __grid_constant__ AxisMap am, RopeShape sh,
    const int32_t* __restrict__ pos, const T* x, T* y) {
    constexpr int V = Vec<T>::N;
    __shared__ alignas(16) float s_c[kRopeAngles], s_s[kRopeAngles];
    const int half = p.d / 2, tid = threadIdx.x;
    const int sites_log2 = 8 - sh.lanes_log2 - sh.rlanes_log2;
    const int64_t site0 = (int64_t)blockIdx.x << sites_log2;
    const int u = (tid & ((1 << sh.lanes_log2) - 1)) * V;
    const int rl = (tid >> sh.lanes_log2) & ((1 << sh.rlanes_log2) - 1);
    const int sl = tid >> (sh.lanes_log2 + sh.rlanes_log2);
    const int64_t site = site0 + sl;
    const bool have = site < sh.n_sites;
    const int64_t nb = site / sh.n_tokens, t = site % sh.n_tokens;
    const int64_t rows = sh.rep * sh.n_heads;
    const int step = 1 << sh.rlanes_log2;
    const int64_t r0 = (int64_t)blockIdx.y * sh.rows_cta;
    const int64_t r1 = r0 + sh.rows_cta < rows ? r0 + sh.rows_cta : rows;
    typename Vec<T>::Raw ra[kBatch], rb[kBatch];
    auto at = [&](int64_t rr) {
        const int64_t r = sh.rep == 1 ? 0 : rr / sh.n_heads, h = rr - r * sh.n_heads;
        return (((nb * sh.rep + r) * sh.n_tokens + t) * sh.n_heads + h) * p.d + u;
    };
    auto load = [&](int64_t rr) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int64_t ri = rr + (int64_t)i * step;
            if (have && ri < r1) {
                const T* src = x + at(ri);
                ra[i] = *reinterpret_cast<const typename Vec<T>::Raw*>(src);
                rb[i] = *reinterpret_cast<const typename Vec<T>::Raw*>(src + half);
            }
        }
    };
    load(r0 + rl);  // on their way while the angles are made
    {
        // a thread makes one pair's angles only: the pair's axis and frequency are
        // read once (their index differs from lane to lane, which the constant
        // cache serves one lane at a time)
        const int pair = tid & (half - 1), ax = am.axis[pair];
        const double freq = p.inv_freq[pair];
        for (int i = tid; i < half << sites_log2; i += kRopeThreads) {
            const int64_t si = site0 + i / half;
            float c = kNoTurn, sn = 0.f;
            if (ax >= 0 && si < sh.n_sites) turn_cs((double)pos[ax * sh.n_sites + si], freq, c, sn);
            s_c[i] = c;
            s_s[i] = sn * am.sign;
        }
    }
    __syncthreads();
    if (!have) return;
    float c[V], s[V];
    bool all = true;  // of the thread's pairs are rotated
#pragma unroll
    for (int e = 0; e < V; e += 4) {
        *reinterpret_cast<float4*>(c + e) = *reinterpret_cast<const float4*>(s_c + sl * half + u + e);
        *reinterpret_cast<float4*>(s + e) = *reinterpret_cast<const float4*>(s_s + sl * half + u + e);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) all &= c[e] != kNoTurn;
    for (int64_t rr = r0 + rl; rr < r1; rr += (int64_t)step * kBatch) {
        if (rr != r0 + rl) load(rr);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int64_t ri = rr + (int64_t)i * step;
            if (ri < r1) {
                if (all)
                    turn_row<T, true>(ra[i], rb[i], c, s);
                else
                    turn_row<T, false>(ra[i], rb[i], c, s);
                T* dst = y + at(ri);
                *reinterpret_cast<typename Vec<T>::Raw*>(dst) = ra[i];
                *reinterpret_cast<typename Vec<T>::Raw*>(dst + half) = rb[i];
            }
        }
    }
}

// --------------------------------------------------------------- summaries
// One CTA per chunk, sequence and run of `hp` KV heads, which share the
// chunk's angles: cos and sin of every token and pair, made once in shared
// memory. Warp g owns group g: lane (q, u) the V pairs u*V .. of its tokens
// q*R .. q*R + R - 1 (R = L/2 tokens for L lanes a row), so a warp's loads are
// whole rows, and a group's sums need only shuffles over q. The sums of all heads
// wait in shared memory for the end, where all threads turn them into means (a
// barrier and a tail per head took two thirds of a head's time). The chunk's sums
// go over the groups in order. Mean positions are sums of integers, exact to
// double rounding. A token's rows of the next head are loaded as soon as the
// current ones are unpacked. 64K tokens x 4 heads (145 MB with the rotated keys)
// in 43 us, 3.4 TB/s, and 33.5 without them. It waits, with neither the memory nor
// the issue slots at a limit (47% of those in its profile): first for table reads,
// shuffles and conversions (short scoreboard), at 16 warps an SM. (5 or 6 CTAs an SM,
// at 96 or 80 registers: 47.5, 60 us.)
//
// In the tables, 16-byte piece j of a row sits at j ^ (j >> 3), so that the
// eight lanes of a row read different banks.
__device__ __forceinline__ int table_at(int row, int pair, int half) {
    const int j = pair >> 2;
    return row * half + ((j ^ (j >> 3)) << 2) + (pair & 3);
}

template <typename T, int D>
struct SumShape {
    static constexpr int V = Vec<T>::N, kHalf = D / 2;
    static constexpr int L = kHalf / V;         // lanes of a row
    static constexpr int R = kGroupRows * L / 32;  // tokens of a lane
};

template <typename T, typename S, int D>
__global__ void __launch_bounds__(256, 2) summaries_axes_kernel(
    const __grid_constant__ Params p, const __grid_constant__ AxisMap am,
    const int32_t* __restrict__ pos, const T* __restrict__ k_raw, S* __restrict__ cs,
    S* __restrict__ gs, T* __restrict__ k_rot, int chunk_begin, int hp) {
    using Sh = SumShape<T, D>;
    constexpr int V = Sh::V, half = Sh::kHalf, L = Sh::L, R = Sh::R;
    // cos of C x half, then sin; cos and sin of the mean angles of G groups and the
    // chunk; per head the groups' sums, G x D (summaries_smem)
    extern __shared__ __align__(16) float s_table[];
    __shared__ int s_pos[HGA_MAX_AXES][8 * kGroupRows];   // groups_per_chunk <= 8
    __shared__ int64_t s_psum[HGA_MAX_AXES][8];
    const int G = p.G, tid = threadIdx.x, lane = tid & 31, g = tid >> 5;
    const int u = lane & (L - 1), q = lane / L;
    const int ch = chunk_begin + blockIdx.x;
    const int64_t b = blockIdx.y;
    const int64_t c0 = (int64_t)ch * p.C;
    const int n_rows = (int)(p.L - c0 < p.C ? p.L - c0 : p.C);  // >= 1
    const int h0 = blockIdx.z * hp, h1 = h0 + hp < p.Hkv ? h0 + hp : p.Hkv;
    const int row0 = kGroupRows * g + R * q;
    float* tc = s_table;
    float* ts = tc + p.C * half;
    float* s_mc = ts + p.C * half;
    float* s_ms = s_mc + (G + 1) * half;
    float* s_sum = s_ms + (G + 1) * half;

    typename Vec<T>::Raw raw_a[R], raw_b[R];
    const T* k_rows = k_raw + ((b * p.Hkv + h0) * (int64_t)p.L + c0 + row0) * D + u * V;
    auto load_row = [&](int m) {
        raw_a[m] = Vec<T>::load_raw(k_rows + m * D);
        raw_b[m] = Vec<T>::load_raw(k_rows + m * D + half);
    };
#pragma unroll
    for (int m = 0; m < R; ++m)
        if (row0 + m < n_rows) load_row(m);
    const int left = n_rows - kGroupRows * g;  // tokens of this group, if positive
    const int n_g = left <= 0 ? 0 : (left >= kGroupRows ? kGroupRows : left);
    for (int a = 0; a < am.n_axes; ++a) {
        int64_t v = 0;
        if (lane < n_g) {
            const int at = pos[((int64_t)a * p.B + b) * p.L + c0 + kGroupRows * g + lane];
            s_pos[a][kGroupRows * g + lane] = at;
            v = at;
        }
#pragma unroll
        for (int off = 1; off < kGroupRows; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (lane == 0) s_psum[a][g] = v;
    }
    __syncthreads();
    {
        // a thread makes one pair's angles at a time: the pair's axis and frequency
        // are read once (their index differs from lane to lane, which the constant
        // cache serves one lane at a time)
        const int n_thr = 32 * G, per = n_thr >= half ? n_thr / half : 1;
        const int stride = n_thr >= half ? per * half : n_thr;
        if (tid < stride) {
            for (int pair = tid % half; pair < half; pair += stride) {
                const int ax = am.axis[pair];
                const double freq = p.inv_freq[pair];
                const bool low = pair >= p.F;
                if (ax >= 0 && (!low || k_rot != nullptr))
#pragma unroll 2
                    for (int r = tid / half; r < n_rows; r += per)
                        turn_cs((double)s_pos[ax][r], freq, tc[table_at(r, pair, half)],
                                ts[table_at(r, pair, half)]);
                for (int i = tid / half; i <= G; i += per) {
                    // a high pair, or one on no axis, takes no part
                    float c = kNoTurn, sn = 0.f;
                    if (ax >= 0 && low) {
                        int64_t sum = 0;
                        int n = n_rows;
                        if (i < G) {
                            sum = s_psum[ax][i];
                            n = min(max(n_rows - kGroupRows * i, 1), kGroupRows);
                        } else {
                            for (int y = 0; y < G; ++y) sum += s_psum[ax][y];
                        }
                        turn_cs((double)sum / (double)n, freq, c, sn);
                    }
                    s_mc[i * half + pair] = c;
                    s_ms[i * half + pair] = sn;
                }
            }
        }
    }
    // bit e: pair u*V + e is rotated; token by token in the sums too
    unsigned turn = 0, each = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const bool on = am.axis[u * V + e] >= 0, low = u * V + e >= p.F;
        turn |= (on && (!low || k_rot != nullptr) ? 1u : 0u) << e;
        each |= (on && !low ? 1u : 0u) << e;
    }
    // the whole warp's pairs are rotated (the rotated keys are wanted), and each
    // lane's are all or none token by token in the sums: no select per pair
    constexpr unsigned kFull = (1u << V) - 1u;
    const bool plain =
        __all_sync(0xffffffffu, turn == kFull && (each == 0u || each == kFull)) != 0;
    __syncthreads();

    for (int h = h0; h < h1; ++h) {
        const int64_t bh = b * p.Hkv + h;
        k_rows += (int64_t)p.L * D;  // the next head's
        float acc0[V], acc1[V];
#pragma unroll
        for (int e = 0; e < V; ++e) acc0[e] = acc1[e] = 0.f;
        auto rows = [&](auto is_plain) {
            constexpr bool kPlain = decltype(is_plain)::value;
            const bool lane_in = each != 0u;
#pragma unroll
            for (int m = 0; m < R; ++m) {
                const int r = row0 + m;
                if (r >= n_rows) break;
                float a[V], bb[V], c[V], sn[V];
                Vec<T>::unpack(raw_a[m], a);
                Vec<T>::unpack(raw_b[m], bb);
                if (h + 1 < h1) load_row(m);
#pragma unroll
                for (int e = 0; e < V; e += 4) {
                    const int at = table_at(r, u * V + e, half);
                    *reinterpret_cast<float4*>(c + e) = *reinterpret_cast<const float4*>(tc + at);
                    *reinterpret_cast<float4*>(sn + e) = *reinterpret_cast<const float4*>(ts + at);
                }
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    // two pairs at a time
                    const float2 a2 = {a[e], a[e + 1]}, b2 = {bb[e], bb[e + 1]};
                    const float2 c2 = {c[e], c[e + 1]}, s2 = {sn[e], sn[e + 1]};
                    float2 ra = ptx::sub2(ptx::mul2(a2, c2), ptx::mul2(b2, s2));
                    float2 rb = ptx::fma2(a2, s2, ptx::mul2(b2, c2));
                    if (!kPlain) {
                        const bool on0 = (turn >> e) & 1u, on1 = (turn >> (e + 1)) & 1u;
                        ra = {on0 ? ra.x : a2.x, on1 ? ra.y : a2.y};
                        rb = {on0 ? rb.x : b2.x, on1 ? rb.y : b2.y};
                    }
                    const bool in0 = kPlain ? lane_in : (each >> e) & 1u;
                    const bool in1 = kPlain ? lane_in : (each >> (e + 1)) & 1u;
                    const float2 t0 =
                        ptx::add2({acc0[e], acc0[e + 1]}, {in0 ? ra.x : a2.x, in1 ? ra.y : a2.y});
                    const float2 t1 =
                        ptx::add2({acc1[e], acc1[e + 1]}, {in0 ? rb.x : b2.x, in1 ? rb.y : b2.y});
                    acc0[e] = t0.x;
                    acc0[e + 1] = t0.y;
                    acc1[e] = t1.x;
                    acc1[e + 1] = t1.y;
                    a[e] = ra.x;
                    a[e + 1] = ra.y;
                    bb[e] = rb.x;
                    bb[e + 1] = rb.y;
                }
                if (k_rot != nullptr) {
                    T* orow = k_rot + (bh * (int64_t)p.L + c0 + r) * D + u * V;
                    Vec<T>::store(orow, a);
                    Vec<T>::store(orow + half, bb);
                }
            }
        };
        if (plain)
            rows(std::true_type());
        else
            rows(std::false_type());
#pragma unroll
        for (int e = 0; e < V; ++e) {
#pragma unroll
            for (int off = L; off < 32; off <<= 1) {
                acc0[e] += __shfl_xor_sync(0xffffffffu, acc0[e], off);
                acc1[e] += __shfl_xor_sync(0xffffffffu, acc1[e], off);
            }
        }
        if (q == 0) {
            float* sums = s_sum + ((h - h0) * G + g) * D + u * V;
#pragma unroll
            for (int e = 0; e < V; e += 4) {
                *reinterpret_cast<float4*>(sums + e) = *reinterpret_cast<const float4*>(acc0 + e);
                *reinterpret_cast<float4*>(sums + half + e) = *reinterpret_cast<const float4*>(acc1 + e);
            }
        }
    }
    __syncthreads();
    // the means of every head's groups and chunk (sum i = G), turned by the mean
    // angle where the pair is low: V pairs a thread
    for (int x = tid; x < (h1 - h0) * (G + 1) * L; x += 32 * G) {
        const int slice = x % L, i = x / L % (G + 1), h = x / L / (G + 1);
        const float* sums = s_sum + (h * G + (i < G ? i : 0)) * D + slice * V;
        float a[V], bb[V];
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            *reinterpret_cast<float4*>(a + e) = *reinterpret_cast<const float4*>(sums + e);
            *reinterpret_cast<float4*>(bb + e) = *reinterpret_cast<const float4*>(sums + half + e);
        }
        if (i == G) {
            for (int y = 1; y < G; ++y)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    a[e] += sums[y * D + e];
                    bb[e] += sums[y * D + half + e];
                }
        }
        const int n = i == G ? n_rows : min(max(n_rows - kGroupRows * i, 0), kGroupRows);
        const float inv_n = n > 0 ? 1.0f / (float)n : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int pair = slice * V + e;
            a[e] *= inv_n;
            bb[e] *= inv_n;
            const float c = s_mc[i * half + pair], sn = s_ms[i * half + pair];
            if (c != kNoTurn && n > 0) {
                const float m0 = a[e], m1 = bb[e];
                a[e] = m0 * c - m1 * sn;
                bb[e] = m0 * sn + m1 * c;
            }
        }
        const int64_t bh = b * p.Hkv + h0 + h, chunk = bh * p.nC + ch;
        S* out = (i == G ? cs + chunk * D : gs + (chunk * G + i) * D) + slice * V;
        store_sum(out, a, V);
        store_sum(out + half, bb, V);
    }
}

// Bytes of the kernel's dynamic shared memory (at most 102 KB).
size_t summaries_smem(const Params& p, int hp) {
    return ((size_t)p.C * p.d + (size_t)(p.G + 1) * p.d + (size_t)hp * p.G * p.d) * sizeof(float);
}

}  // namespace

cudaError_t launch_rope_axes(const Params& p, const AxisMap& am, const int32_t* positions,
                             const void* x, void* y, int64_t n_batch, int64_t n_outer,
                             int64_t n_tokens, int n_heads, cudaStream_t st) {
    const int V = p.dtype == HGA_BF16 ? 8 : 4;
    const int lanes = p.d / 2 / V;
    RopeShape sh;
    sh.n_sites = n_batch * n_tokens;
    sh.n_tokens = n_tokens;
    sh.rep = n_outer / n_batch;
    sh.n_heads = n_heads;
    sh.lanes_log2 = sh.rlanes_log2 = 0;
    while ((1 << sh.lanes_log2) < lanes) ++sh.lanes_log2;
    const int64_t rows = sh.rep * n_heads;
    // Row lanes: up to 8 while each has a batch of rows, or two of them where one would
    // have more than a batch, or while the grid is short of two CTAs per SM; more than 8
    // only while there are fewer sites than a CTA would then take. (2 x 20000 tokens of 4
    // rows: 26.7 us with a batch a thread, 47.2 with a row. 6 and 7 rows in two lanes: 3 x
    // 4999 x 6 of d = 64 in fp32 11.7 us against 13.1, 2 x 9001 x 7 18.3 against 22.5; the
    // worst 65536 x 6 of d = 64 in fp32, 42.0 against 40.9.)
    auto more_lanes = [&] {
        const int64_t per_cta = (int64_t)1 << (8 - sh.lanes_log2 - sh.rlanes_log2);
        if (sh.rlanes_log2 >= 3) return per_cta > sh.n_sites;
        return (int64_t)(2 << sh.rlanes_log2) * kBatch <= rows ||
               (sh.rlanes_log2 == 0 && rows > kBatch) || sh.n_sites < 2 * 148 * per_cta;
    };
    while (sh.lanes_log2 + sh.rlanes_log2 < 8 && (2 << sh.rlanes_log2) <= rows && more_lanes())
        ++sh.rlanes_log2;
    // fewer where the last rows would leave more than an eighth of the lanes idle
    while (sh.rlanes_log2 > 0) {
        const int64_t rl = (int64_t)1 << sh.rlanes_log2, turns = (rows + rl - 1) / rl;
        if (8 * (turns * rl - rows) <= turns * rl) break;
        --sh.rlanes_log2;
    }
    const int sites_log2 = 8 - sh.lanes_log2 - sh.rlanes_log2;
    const int64_t bx = (sh.n_sites + (1 << sites_log2) - 1) >> sites_log2;
    // Rows per CTA: one a lane while the grid is short of two CTAs per SM (the
    // angles are made again, the call's latency counts), more up to all of a
    // site's rows once it fills the GPU.
    int64_t per = (int64_t)1 << sh.rlanes_log2;
    while (per < rows && bx * ((rows + per - 1) / per) > 2 * 148) per *= 2;
    while ((rows + per - 1) / per > 65535) per *= 2;
    sh.rows_cta = per;
    if (bx > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)bx, (unsigned)((rows + per - 1) / per));
    using bf = __nv_bfloat16;
    if (p.dtype == HGA_BF16)
        rope_axes_kernel<bf><<<grid, kRopeThreads, 0, st>>>(p, am, sh, positions, (const bf*)x,
                                                            (bf*)y);
    else
        rope_axes_kernel<float><<<grid, kRopeThreads, 0, st>>>(p, am, sh, positions,
                                                               (const float*)x, (float*)y);
    return cudaGetLastError();
}

cudaError_t launch_summaries_axes(const Params& p, const AxisMap& am, const int32_t* positions,
                                  const void* k_raw, void* chunk_sum, void* group_sum,
                                  void* k_rot, int chunk_begin, int chunk_end, cudaStream_t st) {
    using bf = __nv_bfloat16;
    // heads per CTA: all of them up to 8, halved while the grid is short of two
    // CTAs per SM: fewer heads share a chunk's angles less (237 chunks of 8 heads:
    // 24.8 us in 474 CTAs, 31.5 in 948)
    int hp = p.Hkv < 8 ? p.Hkv : 8;
    auto ctas = [&](int n) {
        return (int64_t)(chunk_end - chunk_begin) * p.B * ((p.Hkv + n - 1) / n);
    };
    while (hp > 1 && ctas(hp) < 2 * 148) hp = (hp + 1) / 2;
    const int groups = (p.Hkv + hp - 1) / hp;
    if (p.B > 65535 || groups > 65535) return cudaErrorInvalidValue;
    const dim3 grid(chunk_end - chunk_begin, p.B, groups);
    const size_t smem = summaries_smem(p, hp);
    auto run = [&](auto t, auto s, auto d) {
        using T = decltype(t);
        using S = decltype(s);
        auto* kernel = summaries_axes_kernel<T, S, decltype(d)::value>;
        const cudaError_t e = set_func_attr_once(
            (const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 104 * 1024);
        if (e != cudaSuccess) return e;
        kernel<<<grid, 32 * p.G, smem, st>>>(p, am, positions, (const T*)k_raw, (S*)chunk_sum,
                                            (S*)group_sum, (T*)k_rot, chunk_begin, hp);
        return cudaGetLastError();
    };
    auto by_dim = [&](auto t, auto s) {
        return p.d == 128 ? run(t, s, std::integral_constant<int, 128>())
                          : run(t, s, std::integral_constant<int, 64>());
    };
    if (p.dtype == HGA_BF16) return p.sum_bf16 ? by_dim(bf(), bf()) : by_dim(bf(), float());
    return p.sum_bf16 ? by_dim(float(), bf()) : by_dim(float(), float());
}

}  // namespace hga
