// k_axes.cu -- rotary positions with several axes: the rotation, its inverse
// (the gradient), and the chunk / group key summaries of keys rotated so.
//
// Pair i = (dim i, dim i + d/2) of a token turns by the angle
// a = p[axis(i)] * theta_i, p the token's position on the pair's axis:
//   y_i = x_i cos a - x_{i+d/2} sin a,   y_{i+d/2} = x_i sin a + x_{i+d/2} cos a.
// The matrix is orthogonal, so the gradient of x is the rotation of y's by -a.
#include "hga_kernels.h"
#include "hga_vec.cuh"

namespace hga {

namespace {

// ---------------------------------------------------------------- rotation
// Memory-bound: x is read once and y written once with 16-byte accesses; the
// angles cost a double product and reduction per (token, pair) and are the
// same for every row (head) of a token, so a thread forms those of its V
// pairs once and turns `rp` rows with them, kBatch rows' loads in flight.
// Rows of a token: rr = r * n_heads + h, r < rep; thread groups of d/2/V lanes
// take one token each. grid (tokens, sequences, row splits).
constexpr int kRopeThreads = 256;
constexpr int kBatch = 4;

template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_axes_kernel(
    Params p, AxisMap am, const int32_t* __restrict__ pos, const T* x, T* y, int64_t n_batch,
    int64_t n_tokens, int n_heads, int64_t rep, int rp, int lanes_log2) {
    constexpr int V = Vec<T>::N;
    const int half = p.d / 2;
    const int64_t idx = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
    const int64_t t = idx >> lanes_log2;
    const int u = (int)(idx & ((1 << lanes_log2) - 1)) * V;
    if (t >= n_tokens) return;
    const int64_t rows = rep * n_heads;
    for (int64_t nb = blockIdx.y; nb < n_batch; nb += gridDim.y) {
        float c[V], s[V];
        unsigned turn = 0;  // bit e: pair u + e is rotated
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int ax = am.axis[u + e];
            c[e] = 1.f;
            s[e] = 0.f;
            if (ax >= 0) {
                const int at = pos[((int64_t)ax * n_batch + nb) * n_tokens + t];
                rope_cs((double)at, p.inv_freq[u + e], c[e], s[e]);
                s[e] *= am.sign;
                turn |= 1u << e;
            }
        }
        for (int64_t r0 = (int64_t)blockIdx.z * rp; r0 < rows; r0 += (int64_t)gridDim.z * rp) {
            const int64_t r1 = r0 + rp < rows ? r0 + rp : rows;
            int h = (int)(r0 % n_heads);
            int64_t off = ((nb * rep + r0 / n_heads) * n_tokens + t) * n_heads + h;
            for (int64_t rr = r0; rr < r1; rr += kBatch) {
                int64_t o[kBatch];
                typename Vec<T>::Raw ra[kBatch], rb[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    o[i] = off * p.d + u;
                    if (rr + i < r1) {
                        ra[i] = *reinterpret_cast<const typename Vec<T>::Raw*>(x + o[i]);
                        rb[i] = *reinterpret_cast<const typename Vec<T>::Raw*>(x + o[i] + half);
                    }
                    ++off;
                    if (++h == n_heads) {  // the same token of the sequence's next row
                        h = 0;
                        off += (n_tokens - 1) * n_heads;
                    }
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    if (rr + i < r1) {
                        float a[V], b[V], ya[V], yb[V];
                        Vec<T>::unpack(ra[i], a);
                        Vec<T>::unpack(rb[i], b);
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            // an unrotated pair is copied, infinities among it
                            const bool on = (turn >> e) & 1u;
                            ya[e] = on ? a[e] * c[e] - b[e] * s[e] : a[e];
                            yb[e] = on ? a[e] * s[e] + b[e] * c[e] : b[e];
                        }
                        Vec<T>::store(y + o[i], ya);
                        Vec<T>::store(y + o[i] + half, yb);
                    }
                }
            }
        }
    }
}

// --------------------------------------------------------------- summaries
// One CTA per (sequence, KV head, chunk); thread (u, k, s) owns the V pairs
// u*V .. of group k's tokens 16k + 4s + {0..3}. The chunk's positions and the
// groups' and chunk's mean positions per axis sit in shared memory; sums of
// integers, so the means are exact to double rounding.
template <typename T, typename S>
__global__ void summaries_axes_kernel(Params p, AxisMap am, const int32_t* __restrict__ pos,
                                      const T* __restrict__ k_raw, S* __restrict__ cs,
                                      S* __restrict__ gs, T* __restrict__ k_rot, int chunk_begin) {
    constexpr int V = Vec<T>::N;
    constexpr int kMaxRows = 8 * kGroupRows;  // groups_per_chunk <= 8
    __shared__ int s_pos[HGA_MAX_AXES][kMaxRows];
    __shared__ double s_mean[HGA_MAX_AXES][9];  // of groups 0..7, and of the chunk
    const int half = p.d / 2;
    const int G = p.G;
    const int tid = threadIdx.x;
    const int s = tid & 3;             // token lane within the group
    const int k = (tid >> 2) % G;      // group within the chunk
    const int u = tid / (4 * G);       // pair slice
    const int ch = chunk_begin + blockIdx.x;
    const int64_t bh = blockIdx.y;
    const int64_t b = bh / p.Hkv;
    const int64_t c0 = (int64_t)ch * p.C;
    const int n_rows = (int)(p.L - c0 < p.C ? p.L - c0 : p.C);  // >= 1
    const T* base = k_raw + bh * (int64_t)p.L * p.d;

    typename Vec<T>::Raw raw_a[4], raw_b[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int64_t t = c0 + 16 * k + 4 * s + m;
        if (t < p.L) {
            raw_a[m] = Vec<T>::load_raw(base + t * p.d + u * V);
            raw_b[m] = Vec<T>::load_raw(base + t * p.d + half + u * V);
        }
    }
    for (int i = tid; i < am.n_axes * n_rows; i += blockDim.x) {
        const int a = i / n_rows, r = i % n_rows;
        s_pos[a][r] = pos[((int64_t)a * p.B + b) * p.L + c0 + r];
    }
    __syncthreads();
    for (int i = tid; i < am.n_axes * (G + 1); i += blockDim.x) {
        const int a = i / (G + 1), g = i % (G + 1);
        const int lo = g < G ? 16 * g : 0;
        const int hi = g < G && 16 * g + 16 < n_rows ? 16 * g + 16 : n_rows;
        int64_t sum = 0;
        for (int r = lo; r < hi; ++r) sum += s_pos[a][r];
        s_mean[a][g < G ? g : 8] = hi > lo ? (double)sum / (double)(hi - lo) : 0.0;
    }
    __syncthreads();

    float acc0[V], acc1[V];
    int ax[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        acc0[e] = acc1[e] = 0.f;
        ax[e] = am.axis[u * V + e];
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int r = 16 * k + 4 * s + m;
        if (r < n_rows) {
            float a[V], bb[V], ra[V], rb[V];
            Vec<T>::unpack(raw_a[m], a);
            Vec<T>::unpack(raw_b[m], bb);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int i = u * V + e;
                ra[e] = a[e];
                rb[e] = bb[e];
                if (ax[e] >= 0 && (i < p.F || k_rot != nullptr)) {
                    float c, sn;
                    rope_cs((double)s_pos[ax[e]][r], p.inv_freq[i], c, sn);
                    ra[e] = a[e] * c - bb[e] * sn;
                    rb[e] = a[e] * sn + bb[e] * c;
                }
                acc0[e] += i < p.F ? ra[e] : a[e];
                acc1[e] += i < p.F ? rb[e] : bb[e];
            }
            if (k_rot != nullptr) {
                T* orow = k_rot + (bh * (int64_t)p.L + c0 + r) * p.d;
                Vec<T>::store(orow + u * V, ra);
                Vec<T>::store(orow + half + u * V, rb);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            acc0[e] += __shfl_xor_sync(0xffffffffu, acc0[e], off);
            acc1[e] += __shfl_xor_sync(0xffffffffu, acc1[e], off);
        }
    }
    auto finish = [&](const float* s0, const float* s1, int g, int n, S* out) {
        float o0[V], o1[V];
        const float inv_n = n > 0 ? 1.0f / (float)n : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int i = u * V + e;
            const float m0 = s0[e] * inv_n, m1 = s1[e] * inv_n;
            o0[e] = m0;
            o1[e] = m1;
            if (n > 0 && i >= p.F && ax[e] >= 0) {
                float c, sn;
                rope_cs(s_mean[ax[e]][g], p.inv_freq[i], c, sn);
                o0[e] = m0 * c - m1 * sn;
                o1[e] = m0 * sn + m1 * c;
            }
        }
        store_sum(out + u * V, o0, V);
        store_sum(out + half + u * V, o1, V);
    };
    if (s == 0) {
        const int left = n_rows - 16 * k;
        finish(acc0, acc1, k, left <= 0 ? 0 : (left >= 16 ? 16 : left),
               gs + ((bh * p.nC + ch) * G + k) * (int64_t)p.d);
    }
    // chunk sums over the groups, in group order (G need not be a power of two)
    __shared__ float s_sum[8][128];
    if (s == 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            s_sum[k][u * V + e] = acc0[e];
            s_sum[k][half + u * V + e] = acc1[e];
        }
    }
    __syncthreads();
    if (s == 0 && k == 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            acc0[e] = acc1[e] = 0.f;
            for (int g = 0; g < G; ++g) {
                acc0[e] += s_sum[g][u * V + e];
                acc1[e] += s_sum[g][half + u * V + e];
            }
        }
        finish(acc0, acc1, 8, n_rows, cs + (bh * p.nC + ch) * (int64_t)p.d);
    }
}

}  // namespace

cudaError_t launch_rope_axes(const Params& p, const AxisMap& am, const int32_t* positions,
                             const void* x, void* y, int64_t n_batch, int64_t n_outer,
                             int64_t n_tokens, int n_heads, cudaStream_t st) {
    const int V = p.dtype == HGA_BF16 ? 8 : 4;
    const int lanes = p.d / 2 / V;
    int lanes_log2 = 0;
    while ((1 << lanes_log2) < lanes) ++lanes_log2;
    const int64_t rep = n_outer / n_batch, rows = rep * n_heads;
    // rows per thread: one while the call is small (latency), more once the
    // threads fill the GPU about four times over (the angles' cost is shared)
    const int64_t threads = n_batch * n_tokens * rows * lanes;
    int rp = 1;
    while (rp < 16 && threads / (2 * rp) >= (int64_t)148 * 2048 * 4) rp *= 2;
    const int64_t bx = (n_tokens * lanes + kRopeThreads - 1) / kRopeThreads;
    const int64_t bz = (rows + rp - 1) / rp;
    if (bx > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)bx, (unsigned)(n_batch < 65535 ? n_batch : 65535),
                    (unsigned)(bz < 65535 ? bz : 65535));
    using bf = __nv_bfloat16;
    if (p.dtype == HGA_BF16)
        rope_axes_kernel<bf><<<grid, kRopeThreads, 0, st>>>(p, am, positions, (const bf*)x, (bf*)y,
                                                            n_batch, n_tokens, n_heads, rep, rp,
                                                            lanes_log2);
    else
        rope_axes_kernel<float><<<grid, kRopeThreads, 0, st>>>(
            p, am, positions, (const float*)x, (float*)y, n_batch, n_tokens, n_heads, rep, rp,
            lanes_log2);
    return cudaGetLastError();
}

cudaError_t launch_summaries_axes(const Params& p, const AxisMap& am, const int32_t* positions,
                                  const void* k_raw, void* chunk_sum, void* group_sum,
                                  void* k_rot, int chunk_begin, int chunk_end, cudaStream_t st) {
    using bf = __nv_bfloat16;
    const int V = p.dtype == HGA_BF16 ? 8 : 4;
    const int threads = (p.d / 2 / V) * 4 * p.G;
    const dim3 grid(chunk_end - chunk_begin, p.B * p.Hkv);
    auto run = [&](auto t, auto s) {
        using T = decltype(t);
        using S = decltype(s);
        summaries_axes_kernel<T, S><<<grid, threads, 0, st>>>(
            p, am, positions, (const T*)k_raw, (S*)chunk_sum, (S*)group_sum, (T*)k_rot, chunk_begin);
    };
    if (p.dtype == HGA_BF16) {
        if (p.sum_bf16) run(bf(), bf()); else run(bf(), float());
    } else {
        if (p.sum_bf16) run(float(), bf()); else run(float(), float());
    }
    return cudaGetLastError();
}

}  // namespace hga
