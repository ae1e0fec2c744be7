// k_attend_tc_pages.cu -- prefill exact attention over the routed set of a 4-bit
// store (HGA_KV_E2M1) on the 5th-generation tensor cores.
//
// "Technische Samenvatting: Hierarchical Global Attention (HGA)"
// (gist.science), "Kernmechanisme" item 4: standard softmax over the bounded
// exact token set of each query chunk.
//
// The plan is that of k_attend_tc.cu (a persistent CTA per SM, units of two M
// tiles of 128 query rows that share every tile of 128 keys, S | S | O | O in
// TMEM, P back in TMEM over S), with the tiles made from pages instead of
// copied: four warps widen the codes of a page row to 16 bits, times their
// block scales, straight into the swizzled operand tiles. Code x block scale
// has at most 6 significant bits, so that is exact in either type. Keys become
// bf16, the queries' type: three more instructions per pair of elements than
// fp16, but queries in fp16 would have to be scaled row by row to keep bf16's
// range (571 against 577 us at the time, and a longer start of every unit, which
// copies that go past the registers shorten). Values become fp16, and so does P
// (at most kMaxSum).
//
// Sixteen warps in four warpgroups, which split the registers:
//   warps 0..3, 4..7  softmax of M tile A, B (152 registers a thread);
//   warp 8            TMEM owner and MMA issuer; warp 9 builds the block lists
//                     and fetches their query rows into L2; warps 10, 11 copy
//                     the query rows (104);
//   warps 12..15      tiles (104): thread r owns key row r of every K and V
//                     tile, whose next codes it holds in registers while it
//                     widens the current ones.
//
// Bound by the alternation of products and softmax within a unit (the tensor
// cores wait while a tile's weights are made; both M tiles in turn hide most of
// it) and by the start and end of units, 8000 cycles each: 32 heads over 4, the
// last 16K tokens of 32K in 533 us (887 TFLOP/s), 4K tokens in 114 us.
//
// Spans of few tokens (at most 8 heads per KV head) go to k_attend_pages.cu.
//
// An M tile holds 128 / gq whole tokens (all gq heads of each), so any number
// of query heads per KV head up to 128 is served; rows past that are idle.
//
// Rows after the span's last query, which may hold anything, read as zero. A
// row whose key or value has a NaN scale must make NaN what sees it and
// nothing else, but 0 x NaN would reach the queries that the causal rule
// hides it from: its key is made NaN (the scores that see it become NaN, the
// others are masked) and its value zero.
#include "hga_blocks.cuh"
#include "hga_e2m1.cuh"
#include "hga_kernels.h"
#include "hga_ptx.cuh"
#include "hga_tc.cuh"

namespace hga {

namespace {

using namespace tc;

constexpr int kThreads = 512;
constexpr float kMaxSum = 8192.f;  // of a tile's weights
constexpr int kSoftmaxRegs = 152, kControlRegs = 104, kTileRegs = 104;
static_assert(2 * kSoftmaxRegs + kControlRegs + kTileRegs <= 4 * 128,
              "the warpgroups share the registers of the launch, 128 a thread");
constexpr uint32_t kIdQk = ptx::idesc_bf16_f32(kRows, kTileKeys, 0, 0);
constexpr uint32_t kIdPv = ptx::idesc_f16_f32(kRows, kD, 0, 1);

struct Smem {
    alignas(1024) uint8_t q[2][kTile];
    alignas(1024) uint8_t k[2][kTile];
    alignas(1024) uint8_t v[2][kTile];
    uint64_t bar_q, q_empty, k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2], p_full[2], o_done[2], list_full[2], list_empty[2], drain;
    uint32_t tmem_base;
    int abort;
    int nb[2];                                        // per list buffer
    int blk_row[2][kMaxBlocks];
    int blk_pos[2][kMaxBlocks];
    int tile_last[2][kMaxBlocks / kBlocksPerTile];    // last key position of a tile, INT_MAX if partial
    alignas(16) uint8_t stage[8][32 * 64];            // per softmax warp: 32 rows x 32 output dims
};
static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "shared memory of one CTA");

// How query rows map to tokens: row r of an M tile is head r % gq of its token
// r / gq, T tokens per tile. For r < 128 and gq <= 128, r / gq is
// (r * magic) >> 16 with magic = ceil(65536 / gq): the excess is below
// 128 / 65536 < 1 / gq.
struct Rows {
    int T, magic, pairs;
};
__host__ __device__ __forceinline__ Rows rows_of(const Params& p) {
    Rows w;
    w.T = kRows / p.gq;
    w.magic = (65536 + p.gq - 1) / p.gq;
    w.pairs = (p.C + 2 * w.T - 1) / (2 * w.T);
    return w;
}

// One unit = (pair of M tiles, query chunk, sequence x KV head); false if no
// token of it is in the query span. Late chunks, which have the most keys,
// come first: of 512 units on 148 CTAs the fullest CTA has 14 percent less to
// do than in ascending order.
struct Unit {
    int tok, jj, b, h, j;  // tok: the unit's first token within the chunk
    int64_t bh;
};

__device__ __forceinline__ bool unit_at(const Params& p, const Rows& w, int u, Unit& un) {
    un.tok = u % w.pairs * 2 * w.T;
    const int rest = u / w.pairs, units = p.B * p.Hkv;
    un.jj = p.nQC - 1 - rest / units;
    un.bh = rest % units;
    un.b = (int)(un.bh / p.Hkv);
    un.h = (int)(un.bh % p.Hkv);
    un.j = p.j0 + un.jj;
    const int t0 = un.j * p.C + un.tok;
    const int t1 = min(t0 + 2 * w.T, (un.j + 1) * p.C);
    return t0 < p.q_begin + p.q_len && t1 > p.q_begin;
}

// This CTA's unit of round rd: every other round in reverse, so that the CTA
// with the heaviest unit of one round has the lightest of the next.
__device__ __forceinline__ int unit_in_round(int rd) {
    const int grid = (int)gridDim.x, b = (int)blockIdx.x;
    return rd * grid + ((rd & 1) ? grid - 1 - b : b);
}

// Row r of M tile x: its offset in rows of d from head 0 (of the KV head) of the
// chunk's first token, or -1 if it holds no query of the span. In a query span
// of under 2^31 rows a chunk's rows fit an int.
__device__ __forceinline__ int row_offset(const Params& p, const Rows& w, const Unit& un, int x,
                                          int r) {
    const int t = (r * w.magic) >> 16;
    const int tok = un.tok + x * w.T + t, pos = un.j * p.C + tok;
    const bool ok = t < w.T && tok < p.C && pos >= p.q_begin && pos < p.q_begin + p.q_len;
    return ok ? tok * p.Hq + (r - t * p.gq) : -1;
}

// A tile thread's share of a key or value tile: its row's codes.
struct RowCodes {
    uint4 c[4];
};

__device__ __forceinline__ void load_codes(RowCodes& r, const uint8_t* page, int row) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r.c[i] = __ldg(reinterpret_cast<const uint4*>(page + e2m1::code_at(row, 32 * i)));
}

// An f16 pair as a bf16 pair (exact for what code x scale can be).
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// Widen a row into its place in a tile, to bf16 or fp16: 16-byte chunk c (dims
// 8c .. + 7) of row r at panel c / 8, chunk (c % 8) ^ (r % 8).
template <bool kBf16>
__device__ __forceinline__ void widen_row(const RowCodes& rc, uint2 scales, uint8_t* tile, int r) {
    uint8_t* dst = tile + r * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t word = i < 2 ? scales.x : scales.y;
        const uint32_t sc = e2m1::scales_to_f16x2((uint16_t)((i & 1) ? word >> 16 : word));
        const uint32_t w[4] = {rc.c[i].x, rc.c[i].y, rc.c[i].z, rc.c[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t f[4];
            e2m1::codes_to_f16x2(w[e], f);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                f[z] = e2m1::hmul2_half(f[z], sc, e >> 1);
                if (kBf16) f[z] = f16x2_to_bf16x2(f[z]);
            }
            const int c = 4 * i + e;
            *reinterpret_cast<uint4*>(dst + (c >> 3) * kPanel + (((c & 7) ^ (r & 7)) << 4)) =
                make_uint4(f[0], f[1], f[2], f[3]);
        }
    }
}

// Asynchronous copies of a unit's query rows into their places in the operand
// tiles: 16 lanes a row, zeros for rows without a query. r: thread 0 .. 63.
__device__ __forceinline__ void copy_queries(const Params& p, const Rows& w, const Unit& un,
                                             const __nv_bfloat16* q, uint8_t (*tiles)[kTile],
                                             int r) {
    const int c = r & 15;
    const uint32_t dst = ptx::smem_u32(tiles[0]) + (c >> 3) * kPanel;
    const __nv_bfloat16* src = q + (((int64_t)un.b * p.q_len + (un.j * p.C - p.q_begin)) * p.Hq +
                                    (int64_t)un.h * p.gq) * kD + 8 * c;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll 4
        for (int i = 0; i < kRows / 4; ++i) {
            const int rr = (r >> 4) + 4 * i;
            const int off = row_offset(p, w, un, x, rr);
            ptx::cp_async16_or_zero(dst + x * kTile + rr * 128 + (((c & 7) ^ (rr & 7)) << 4),
                                    off >= 0 ? src + (int64_t)off * kD : q, off >= 0);
        }
}

// True if one of the row's eight scale codes is NaN.
__device__ __forceinline__ bool has_nan_scale(uint2 s) {
    return (__vcmpeq4(s.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(s.y & 0x7f7f7f7fu, 0x7f7f7f7fu)) !=
           0u;
}

__global__ void __launch_bounds__(kThreads, 1) attend_tc_pages_kernel(
    const __grid_constant__ Params p, const __nv_bfloat16* __restrict__ q,
    const uint8_t* __restrict__ ks, const uint8_t* __restrict__ vs,
    const int32_t* __restrict__ sel, const int32_t* __restrict__ nsel,
    __nv_bfloat16* __restrict__ out, int n_units) {
    extern __shared__ uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(align_smem_1024(smem_raw));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int span_end = p.q_begin + p.q_len;
    const Rows rows = rows_of(p);

    if (tid == 0) {
        sm.abort = 0;
        ptx::mbar_init(&sm.bar_q, 2);  // warps 10, 11
        ptx::mbar_init(&sm.q_empty, 1);
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(&sm.k_full[s], 4);
            ptx::mbar_init(&sm.k_empty[s], 1);
            ptx::mbar_init(&sm.v_full[s], 4);
            ptx::mbar_init(&sm.v_empty[s], 1);
            ptx::mbar_init(&sm.s_full[s], 1);
            ptx::mbar_init(&sm.p_full[s], 4);
            ptx::mbar_init(&sm.o_done[s], 1);
            ptx::mbar_init(&sm.list_full[s], 1);
            ptx::mbar_init(&sm.list_empty[s], 12);  // tile and softmax warps
        }
        ptx::mbar_init(&sm.drain, 1);
        ptx::fence_mbar_init();
    }
    if (warp == 8) {
        ptx::tmem_alloc(&sm.tmem_base, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    volatile int* abort = &sm.abort;
    auto n_tiles_of = [](int nb) { return (nb + kBlocksPerTile - 1) / kBlocksPerTile; };
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_bar(bar, parity, abort, p.wait_ns)) != 0;
    };

    if (warp >= 12) {
        // ------------------------------------------------------ tiles
        ptx::regs_dec<kTileRegs>();
        const int r = tid - 12 * 32;     // key row of a tile
        const int row = r & (kGroupRows - 1);
        int k = 0, g0 = 0;
        Unit un;
        bool ok = true;
        for (int rd = 0, u; ok && (u = unit_in_round(rd)) < n_units; ++rd) {
            if (!unit_at(p, rows, u, un)) continue;
            const int bf = k & 1;
            if (!wait_warp(&sm.list_full[bf], (k >> 1) & 1)) break;
            const int nb = sm.nb[bf], n = n_tiles_of(nb);
            const uint8_t* kbase = ks + un.bh * p.kv_slab;
            const uint8_t* vbase = vs + un.bh * p.kv_slab;
            // this row's page in tile t; the pad blocks of the last tile read a page that is there
            auto page_of = [&](int t, bool* live) {
                const int blk = t * kBlocksPerTile + (r >> 4);
                const int pos = sm.blk_pos[bf][blk < nb ? blk : 0];
                *live = blk < nb && pos + row < span_end;
                return (int64_t)(pos / kGroupRows) * kE2m1Page;
            };
            RowCodes kc, vc;
            uint2 sk, sv, sv_next;
            auto load_k = [&](int t) {
                bool live;
                const int64_t at = page_of(t, &live);
                load_codes(kc, kbase + at, row);
                const uint2 zero = make_uint2(0u, 0u);
                sk = live ? __ldg(reinterpret_cast<const uint2*>(kbase + at + e2m1::scale_at(row, 0)))
                          : zero;
                sv_next =
                    live ? __ldg(reinterpret_cast<const uint2*>(vbase + at + e2m1::scale_at(row, 0)))
                         : zero;
            };
            auto load_v = [&](int t) {
                bool live;
                load_codes(vc, vbase + page_of(t, &live), row);
            };
            auto arrive = [&](uint64_t* bar) {
                ptx::fence_async_shared();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar);
            };
            load_k(0);
            load_v(0);
            for (int t = 0; t < n; ++t) {
                const int g = g0 + t, s = g & 1;
                if (g >= 2 && !wait_warp(&sm.k_empty[s], ((g >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                sv = sv_next;
                if (has_nan_scale(sv)) {
                    sv = make_uint2(0u, 0u);
                    sk = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
                }
                widen_row<true>(kc, sk, sm.k[s], r);
                arrive(&sm.k_full[s]);
                if (t + 1 < n) load_k(t + 1);
                if (g >= 2 && !wait_warp(&sm.v_empty[s], ((g >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                widen_row<false>(vc, sv, sm.v[s], r);
                arrive(&sm.v_full[s]);
                if (t + 1 < n) load_v(t + 1);
            }
            if (!ok) break;
            if (lane == 0) ptx::mbar_arrive(&sm.list_empty[bf]);
            g0 += n;
            ++k;
        }
    } else if (warp >= 8) {
        ptx::regs_dec<kControlRegs>();
        if (warp == 9) {
            // -------------------------------------------------- block lists
            // builds the key-block list of this CTA's next units into a double buffer
            int k = 0;
            Unit un;
            for (int rd = 0, u; (u = unit_in_round(rd)) < n_units; ++rd) {
                if (!unit_at(p, rows, u, un)) continue;
                const int bf = k & 1;
                if (k >= 2 && !wait_warp(&sm.list_empty[bf], ((k >> 1) - 1) & 1)) break;
                const int64_t prob = un.bh * p.nQC + un.jj;
                const int nb = build_key_blocks_warp(p, un.j, sel + prob * p.kg, nsel + prob, false,
                                                     sm.blk_row[bf], sm.blk_pos[bf]);
                __syncwarp();
                for (int t = lane; t * kBlocksPerTile < nb; t += 32) {
                    int last = 0;
#pragma unroll
                    for (int i = 0; i < kBlocksPerTile; ++i) {
                        const int blk = t * kBlocksPerTile + i;
                        last = blk < nb ? max(last, sm.blk_pos[bf][blk] + kGroupRows - 1) : INT_MAX;
                    }
                    sm.tile_last[bf][t] = last;
                }
                __syncwarp();
                if (lane == 0) {
                    sm.nb[bf] = nb;
                    ptx::mbar_arrive(&sm.list_full[bf]);
                }
                // a token's heads are contiguous
                for (int i = lane; i < 2 * rows.T; i += 32) {
                    const int off = row_offset(p, rows, un, i / rows.T, i % rows.T * p.gq);
                    if (off >= 0)
                        ptx::bulk_prefetch_l2(
                            q + (((int64_t)un.b * p.q_len + (un.j * p.C - p.q_begin)) * p.Hq +
                                 (int64_t)un.h * p.gq + off) * kD,
                            (uint32_t)(p.gq * kD * 2));
                }
                ++k;
            }
        } else if (warp >= 10) {
            // -------------------------------------------------- queries
            int k = 0;
            Unit un;
            for (int rd = 0, u; (u = unit_in_round(rd)) < n_units; ++rd) {
                if (!unit_at(p, rows, u, un)) continue;
                if (k >= 1 && !wait_warp(&sm.q_empty, (k - 1) & 1)) break;
                copy_queries(p, rows, un, q, sm.q, tid - 10 * 32);
                ptx::cp_async_commit();
                ptx::cp_async_wait<0>();
                ptx::fence_async_shared();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sm.bar_q);
                ++k;
            }
        } else if (warp == 8 && lane == 0) {
            // -------------------------------------------------- MMA issuer
            const uint32_t q_s[2] = {ptx::smem_u32(sm.q[0]), ptx::smem_u32(sm.q[1])};
            int k = 0, g0 = 0;
            Unit un;
            bool ok = true;
            for (int rd = 0, u; ok && (u = unit_in_round(rd)) < n_units; ++rd) {
                if (!unit_at(p, rows, u, un)) continue;
                const int bf = k & 1;
                ok = wait_bar(&sm.list_full[bf], (k >> 1) & 1, abort, p.wait_ns);
                if (!ok) break;
                const int n = n_tiles_of(sm.nb[bf]);
                const int s0 = g0 & 1;
                ok = wait_bar(&sm.bar_q, k & 1, abort, p.wait_ns) &&
                     wait_bar(&sm.k_full[s0], (g0 >> 1) & 1, abort, p.wait_ns);
                if (!ok) break;
                ptx::tc_fence_after();
                // S_x of the previous unit was read and its P consumed by the PV
                // issued before on this in-order queue
                const uint32_t k0 = ptx::smem_u32(sm.k[s0]);
                issue_qk<kIdQk>(tmem + col_s(0), q_s[0], k0);
                ptx::umma_commit(&sm.s_full[0]);
                issue_qk<kIdQk>(tmem + col_s(1), q_s[1], k0);
                ptx::umma_commit(&sm.s_full[1]);
                if (n == 1) ptx::umma_commit(&sm.q_empty);
                ptx::umma_commit(&sm.k_empty[s0]);
                for (int t = 0; ok && t < n; ++t) {
                    const int g = g0 + t, s = g & 1, s1 = (g + 1) & 1;
                    const bool more = t + 1 < n;
                    ok = wait_bar(&sm.v_full[s], (g >> 1) & 1, abort, p.wait_ns) &&
                         (!more || wait_bar(&sm.k_full[s1], ((g + 1) >> 1) & 1, abort, p.wait_ns));
                    if (!ok) break;
                    const uint32_t v_s = ptx::smem_u32(sm.v[s]);
                    const uint32_t k_s1 = ptx::smem_u32(sm.k[s1]);
                    for (int x = 0; x < 2; ++x) {
                        // P_x of this tile; for t == 0 this also orders the
                        // PV that overwrites O_x after the same warps' epilogue
                        // of the previous unit read it
                        if (!wait_bar(&sm.p_full[x], g & 1, abort, p.wait_ns)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        issue_pv<kIdPv>(tmem + col_o(x), tmem + col_s(x), v_s, t > 0);
                        if (more) {
                            issue_qk<kIdQk>(tmem + col_s(x), q_s[x], k_s1);
                            ptx::umma_commit(&sm.s_full[x]);
                        } else {
                            ptx::umma_commit(&sm.o_done[x]);
                        }
                    }
                    if (!ok) break;
                    if (more && t + 2 == n) ptx::umma_commit(&sm.q_empty);  // last QK issued
                    ptx::umma_commit(&sm.v_empty[s]);
                    if (more) ptx::umma_commit(&sm.k_empty[s1]);
                }
                g0 += n;
                ++k;
            }
            // drain: every MMA issued above has completed before TMEM is freed
            ptx::umma_commit(&sm.drain);
            const uint64_t t0 = ptx::globaltimer_ns();
            while (!ptx::mbar_try_wait(&sm.drain, 0) &&
                   ptx::globaltimer_ns() - t0 < ptx::kDrainLimitNs) {
            }
        }
    } else {
        // ------------------------------------------------------ softmax
        ptx::regs_inc<kSoftmaxRegs>();
        const int x = warp >> 2;                        // M tile of this warpgroup
        const int q4 = warp & 3;                        // TMEM lane quarter
        const int r = q4 * 32 + lane;                   // row = TMEM lane
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const uint32_t s_addr = tmem + lane_off + col_s(x);
        const uint32_t o_addr = tmem + lane_off + col_o(x);
        const float sc = 1.4426950408889634f / sqrtf((float)kD) * p.k_scale;
        int k = 0, g0 = 0;
        Unit un;
        bool ok = true;
        for (int rd = 0, u; ok && (u = unit_in_round(rd)) < n_units; ++rd) {
            if (!unit_at(p, rows, u, un)) continue;
            const int bf = k & 1;
            if (!wait_warp(&sm.list_full[bf], (k >> 1) & 1)) {
                ok = false;
                break;
            }
            const int nb = sm.nb[bf];
            const int n = n_tiles_of(nb);
            const int tokx = un.j * p.C + un.tok + x * rows.T;  // the M tile's first position
            const int qpos = tokx + ((r * rows.magic) >> 16);
            float m_used = -INFINITY, l = 0.f;
            for (int t = 0; t < n; ++t) {
                const int g = g0 + t;
                if (!wait_warp(&sm.s_full[x], g & 1)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const int blk0 = t * kBlocksPerTile;
                const bool masked = sm.tile_last[bf][t] > tokx;
                // chunk c of 32 scores, masked: causal within the current chunk,
                // padding past the set
                auto mask = [&](int c, uint32_t (&s32)[32]) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int blk = blk0 + 2 * c + i;
                        const int see = blk < nb ? qpos - sm.blk_pos[bf][blk] : -1;
#pragma unroll
                        for (int e = 0; e < kGroupRows; ++e)
                            if (e > see) s32[16 * i + e] = __float_as_uint(-INFINITY);
                    }
                };
                // P = 2^(S*sc - m) in fp16, the next chunk of scores on its way while one
                // is worked on. m is the first tile's maximum; it is raised, to this
                // tile's, only where the weights sum to more than kMaxSum (seldom;
                // without that no weight is above it, far inside fp16). So no maximum
                // is taken elsewhere. The sum so far then shrinks by alpha, and the
                // tile's weights are made again.
                uint32_t pk[kTileKeys / 2];
                float2 lsum;
                float alpha = 1.f;
                bool rescale = false;
                for (bool raise = t == 0, last = false;;) {
                    if (raise) {
                        float mc = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t s32[32];
                            ptx::tmem_ld32(s_addr + 32 * c, s32);
                            ptx::tmem_wait_ld();
                            ptx::reg_fence<32>(s32);
                            if (masked) mask(c, s32);
                            float m4[4] = {mc, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
#pragma unroll
                                for (int y = 0; y < 4; ++y)
                                    m4[y] = ptx::fmax3(m4[y], __uint_as_float(s32[e + 2 * y]),
                                                       __uint_as_float(s32[e + 2 * y + 1]));
                            mc = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                        }
                        const float m_new = fmaxf(m_used, mc * sc);
                        if (m_new > m_used) {
                            alpha = ptx::ex2_approx(m_used - m_new);
                            m_used = m_new;
                        }
                        rescale = true;
                        last = true;  // NaN scores must not come back here
                    }
                    const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
                    float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    uint32_t buf[2][32];
                    ptx::tmem_ld32(s_addr, buf[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t(&s32)[32] = buf[c & 1];
                        ptx::tmem_wait_ld();
                        ptx::reg_fence<32>(s32);
                        if (c < 3) ptx::tmem_ld32(s_addr + 32 * (c + 1), buf[(c + 1) & 1]);
                        if (masked) mask(c, s32);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float a0, a1;
                            ptx::fma2_bc(__uint_as_float(s32[e]), __uint_as_float(s32[e + 1]), sc,
                                         neg_m, a0, a1);
                            const float2 w =
                                make_float2(ptx::ex2_approx(a0), ptx::ex2_approx(a1));
                            ls[(e >> 1) & 1] = ptx::add2(ls[(e >> 1) & 1], w);
                            const __half2 h2 = __floats2half2_rn(w.x, w.y);
                            pk[16 * c + e / 2] = *reinterpret_cast<const uint32_t*>(&h2);
                        }
                    }
                    lsum = ptx::add2(ls[0], ls[1]);
                    raise = lsum.x + lsum.y > kMaxSum || m_used == -INFINITY;
                    if (last || !__any_sync(0xffffffffu, raise)) break;
                    raise = true;
                }
                // tcgen05.ld/st are warp-collective: the whole warp rescales its
                // rows when any row needs it (rows that do not use alpha = 1).
                // PV of the previous tile has completed: S of this tile was issued
                // after it on the same (in-order) tensor-core queue.
                if (__any_sync(0xffffffffu, rescale && t >= 1)) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[32];
                        ptx::tmem_ld32(o_addr + 32 * c, o);
                        ptx::tmem_wait_ld();
                        ptx::reg_fence<32>(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        ptx::tmem_st32(o_addr + 32 * c, o);
                    }
                }
                l = l * alpha + (lsum.x + lsum.y);
                ptx::tmem_st32(s_addr, pk);
                ptx::tmem_st32(s_addr + 32, pk + 32);
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sm.p_full[x]);
            }
            if (!ok) break;
            if (lane == 0) ptx::mbar_arrive(&sm.list_empty[bf]);
            if (!wait_warp(&sm.o_done[x], k & 1)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            // a row that met a NaN score has NaN in O, whatever its sum
            const float inv = l > 0.f ? p.v_scale / l : 0.f;
            // where this lane's read-back rows go: row 8i + lane / 4 of the warp
            const int rr = lane >> 2, cc = lane & 3;
            __nv_bfloat16* obase =
                out + (((int64_t)un.b * p.q_len + (un.j * p.C - p.q_begin)) * p.Hq +
                       (int64_t)un.h * p.gq) * kD + 8 * cc;
            int off[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) off[i] = row_offset(p, rows, un, x, q4 * 32 + 8 * i + rr);
            // all of O in one round trip
            uint32_t o[kD];
#pragma unroll
            for (int c = 0; c < 4; ++c) ptx::tmem_ld32(o_addr + 32 * c, o + 32 * c);
            ptx::tmem_wait_ld();
            ptx::reg_fence<kD>(o);
            ptx::tc_fence_before();
            // Coalesced output: four rounds of 32 dims; each row's 64 bytes go
            // through this warp's staging area (16-byte chunks XOR-swizzled by
            // (row / 2) % 4) and come back as 8 rows x 4 chunks per store.
            uint8_t* stg = sm.stage[warp];
#pragma unroll
            for (int qd = 0; qd < 4; ++qd) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float f[8];
#pragma unroll
                    for (int z = 0; z < 8; ++z) f[z] = __uint_as_float(o[32 * qd + 8 * c + z]) * inv;
                    *reinterpret_cast<uint4*>(stg + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
                        f32x8_to_bf16(f);
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int R = 8 * i + rr;                       // row within the warp
                    const uint4 v = *reinterpret_cast<const uint4*>(stg + R * 64 + ((cc ^ ((R >> 1) & 3)) << 4));
                    if (off[i] >= 0) *reinterpret_cast<uint4*>(obase + (int64_t)off[i] * kD + 32 * qd) = v;
                }
                __syncwarp();
            }
            g0 += n;
            ++k;
        }
        ptx::tc_fence_before();
    }
    __syncthreads();
    if (*abort && tid == 0) raise_timeout(p);
    if (warp == 8) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

cudaError_t launch_attend_tc_pages(const Params& p, const void* q_rot, const KvSources& kv,
                                   const int32_t* sel_groups, const int32_t* n_sel_groups,
                                   void* out, cudaStream_t st) {
    const size_t smem = sizeof(Smem) + 1024;
    cudaError_t e = set_func_attr_once((const void*)attend_tc_pages_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return cudaErrorInvalidValue;
    const int64_t n_units = (int64_t)rows_of(p).pairs * p.nQC * p.B * p.Hkv;
    if (n_units > INT32_MAX - 65536) return cudaErrorInvalidValue;
    const int grid = (int)(n_units < sms ? n_units : sms);
    attend_tc_pages_kernel<<<grid, kThreads, smem, st>>>(
        p, (const __nv_bfloat16*)q_rot, (const uint8_t*)kv.k_res, (const uint8_t*)kv.v_res,
        sel_groups, n_sel_groups, (__nv_bfloat16*)out, (int)n_units);
    return cudaGetLastError();
}

}  // namespace hga
