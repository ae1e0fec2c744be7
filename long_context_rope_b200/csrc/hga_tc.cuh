// hga_tc.cuh -- what the two prefill attention kernels on the 5th-generation
// tensor cores share: tile sizes, the TMEM plan, the bounded wait and the MMA
// sequences.
#pragma once

#include "hga_common.cuh"
#include "hga_ptx.cuh"

namespace hga {
namespace tc {

constexpr int kD = 128;
constexpr int kRows = 128;                 // query rows per M tile
constexpr int kTileKeys = 128;             // keys per tile
constexpr int kBlocksPerTile = kTileKeys / kGroupRows;
constexpr int kPanel = 128 * 128;          // 128 rows x 128 bytes (64 16-bit elements)
constexpr int kTile = 2 * kPanel;          // 128 x 128 16-bit elements
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.0f;

__host__ __device__ constexpr uint32_t col_s(int x) { return (uint32_t)(x * 128); }
__host__ __device__ constexpr uint32_t col_o(int x) { return (uint32_t)(256 + x * 128); }

// Bounded wait shared by the roles of one CTA: gives up after the launch's
// wait limit or when another role of this CTA gave up (*abort); a give-up
// sets *abort so the other roles stop. Both are checked every 8 polls. The
// device error word is not consulted: an invalid selection entry (of this
// unit or any other, in this launch or an earlier one) never stops a wait.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         uint64_t limit_ns) {
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t i = 0;; ++i) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if ((i & 7u) == 7u && (*abort || ptx::globaltimer_ns() - t0 > limit_ns)) break;
    }
    *abort = 1;
    return false;
}

// S = Q K^T of one M tile and one key tile in shared memory; kId: the
// instruction descriptor.
template <uint32_t kId>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint32_t q_s, uint32_t k_s) {
#pragma unroll
    for (int kk = 0; kk < kD / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kPanel + (kk & 3) * 32;
        ptx::umma_f16(d_tmem, ptx::smem_desc_sw128(q_s + off, 16, 1024),
                      ptx::smem_desc_sw128(k_s + off, 16, 1024), kId, kk > 0);
    }
}

// O (+)= P V with P (16-bit) in TMEM columns [p_tmem, p_tmem + 64).
template <uint32_t kId>
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_s,
                                         bool accumulate) {
#pragma unroll
    for (int kk = 0; kk < kTileKeys / 16; ++kk)
        ptx::umma_f16_ts(d_tmem, p_tmem + kk * 8,
                         ptx::smem_desc_sw128(v_s + kk * 2048, kPanel, 1024), kId,
                         (accumulate || kk > 0) ? 1u : 0u);
}

}  // namespace tc
}  // namespace hga
