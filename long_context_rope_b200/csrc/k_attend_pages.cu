// k_attend_pages.cu -- exact attention of single tokens over the routed set of a
// 4-bit store (HGA_KV_E2M1): a decode step, or a span of few tokens.
//
// "Technische Samenvatting: Hierarchical Global Attention (HGA)"
// (gist.science), "Kernmechanisme" item 4: standard softmax over the bounded
// exact token set. Every page of the set is read once (2304 bytes for 16 keys
// and values), and the query heads of a KV head share each load (GQA).
//
// One cluster of CL CTAs of four warps per unit (token, sequence, KV head): CL as large as
// keeps every unit's cluster resident at once (four CTAs per SM), and no larger
// than gives every warp a page. Block i of the unit (forced blocks, then the
// routed list) goes to warp i mod 4 CL of the cluster, and each warp works out
// its own blocks from the list, so a CTA starts without a barrier. (CTAs of
// eight warps, two per SM: the same up to 296 units, where all are resident
// either way; two us more for 512 units of 108 pages, which then take two rounds of
// CTAs.) Bound by instructions, about 390 a page, at 16 warps an SM: 127 MB in
// 38 us.
// hga_decode_pages.cuh has the arithmetic and the joining of the partials.
#include <cooperative_groups.h>

#include <mutex>

#include "hga_blocks.cuh"
#include "hga_decode_pages.cuh"
#include "hga_kernels.h"

namespace cg = cooperative_groups;

namespace hga {

namespace {

using dec::kMaxCluster;
constexpr int kWarps = 4;
constexpr int kCtasPerSm = 4;  // at 120 registers a thread

struct PagesSmem : dec::PageSmem<kWarps> {
    int2 blk[kWarps][kMaxBlocks / kWarps];  // per warp: page (kSrcGathered: of the
                                                    // gathered buffer), first position
};

// The keys' chunks that are always visible to position qpos, up to its block:
// sinks [0, s_end), then [l_begin, j].
struct Forced {
    int s_end, l_begin, blocks;
};

__host__ __device__ __forceinline__ Forced forced_of(const Params& p, int qpos) {
    Forced f;
    const int j = qpos / p.C;
    f.s_end = p.n_sink < j + 1 ? p.n_sink : j + 1;
    f.l_begin = j - p.n_local > f.s_end ? j - p.n_local : f.s_end;
    // chunk j comes last; with a sink chunk j it is [0, s_end)'s
    const int chunks = f.s_end + (j + 1 - f.l_begin);
    f.blocks = (chunks - 1) * p.G + (qpos - j * p.C) / kGroupRows + 1;
    return f;
}

__global__ void __launch_bounds__(32 * kWarps, kCtasPerSm) attend_pages_kernel(
    const __grid_constant__ dec::PageSource res, const __grid_constant__ dec::PageSource gat,
    const __grid_constant__ Params p, const __nv_bfloat16* __restrict__ q,
    const int32_t* __restrict__ sel, const int32_t* __restrict__ nsel,
    __nv_bfloat16* __restrict__ out) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    PagesSmem& sm = *reinterpret_cast<PagesSmem*>(smem_raw);
    cg::cluster_group cluster = cg::this_cluster();
    ptx::cluster_started_arrive();
    const int CL = (int)cluster.num_blocks(), r = (int)cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tok = blockIdx.y / (p.B * p.Hu);
    // routing unit: (sequence, KV head) or (sequence, query head)
    const int64_t bh = blockIdx.y - tok * (p.B * p.Hu);
    const int b = (int)(bh / p.Hu), h = (int)(bh % p.Hu);
    const int64_t kvh = (int64_t)b * p.Hkv + h / (p.Hu / p.Hkv);  // its K/V row
    const int qpos = p.q_begin + tok, j = qpos / p.C;
    const int64_t prob = bh * p.nQC + (j - p.j0);
    q += (int64_t)tok * p.Hq * dec::kD;
    out += (int64_t)tok * p.Hq * dec::kD;
    const bool gathered = gat.k != nullptr;

    // ---- this warp's blocks; the count and the first 32 entries in one round trip
    const Forced f = forced_of(p, qpos);
    const int first = warp * CL + r, step = kWarps * CL;
    const int32_t* list = sel + prob * p.kg;
    auto entry = [&](int s) { return s >= 0 && s < p.kg ? list[s] : -1; };
    int s = first + step * lane - f.blocks;
    int gi = entry(s), prev = entry(s - 1);
    int n_list = nsel[prob];
    uint32_t qf[8][2];
    float sc[2];
    dec::load_q_pages(p, q, b, h, qf, sc);
    if (n_list < 0 || n_list > p.kg) {
        if (threadIdx.x == 0 && r == 0) raise_dev_error(p, kDevErrCount);
        n_list = n_list < 0 ? 0 : p.kg;
    }
    int n = 0;
    for (int i0 = first; i0 < f.blocks + n_list; i0 += step * 32) {
        const int i = i0 + step * lane;
        if (i0 != first) {
            s = i - f.blocks;
            gi = entry(s);
            prev = entry(s - 1);
        }
        int page = 0, pos = 0;
        bool ok = false;
        if (i < f.blocks) {
            const int w = i / p.G, gm = i % p.G;
            const int c = w < f.s_end ? w : f.l_begin + (w - f.s_end);
            pos = c * p.C + kGroupRows * gm;
            page = p.kv_layout == HGA_KV_WINDOWS ? i : pos / kGroupRows;
            ok = true;
        } else if (s < n_list) {
            const int c = gi >= 0 ? gi / p.G : -1;
            ok = gi >= 0 && c < j && !is_forced(p, j, c) && (s == 0 || gi > prev);
            if (!ok) raise_dev_error(p, kDevErrGroupIndex);
            pos = gi * kGroupRows;
            page = gathered ? (kSrcGathered | s) : gi;
        }
        const unsigned m = __ballot_sync(0xffffffffu, ok);
        if (ok) sm.blk[warp][n + __popc(m & ((1u << lane) - 1u))] = make_int2(page, pos);
        n += __popc(m);
    }
    __syncwarp();

    dec::WarpAcc acc;
    dec::acc_init(acc);
    const dec::PageRef rbase = dec::lane_pages(res.k + kvh * res.slab, res.v + kvh * res.slab);
    const dec::PageRef gbase = dec::lane_pages(gat.k + prob * gat.slab, gat.v + prob * gat.slab);
    dec::consume_pages(
        qf, sc, sm.u.page[warp], n, qpos,
        [&](int i) {
            const int page = sm.blk[warp][i].x;
            return dec::page_at((page & kSrcGathered) ? gbase : rbase, page & ~kSrcGathered);
        },
        [&](int i) { return sm.blk[warp][i].y; }, acc);
    ptx::cluster_started_wait();
    dec::merge_pages<kWarps>(sm, cluster, p, acc, b, h, out);
}

cudaLaunchConfig_t config_of(int cl, int64_t units, cudaLaunchAttribute* attr, cudaStream_t st) {
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(cl, (unsigned)units, 1);
    c.blockDim = dim3(32 * kWarps);
    c.dynamicSmemBytes = sizeof(PagesSmem);
    c.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cl;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    c.attrs = attr;
    c.numAttrs = 1;
    return c;
}

std::mutex g_pages_mu;

// The largest cluster size, at most `most`, of which all units' are resident at
// once. Per device, resident clusters of each size are asked for once.
int cluster_size(int most, int64_t units, int dev) {
    static int active_of[kMaxDevicesPerProcess][kMaxCluster + 1] = {};  // 0: not asked yet
    std::lock_guard<std::mutex> lock(g_pages_mu);
    int* active = active_of[dev];
    int cl = most;
    for (; cl > 1; --cl) {
        if (active[cl] == 0) {
            cudaLaunchAttribute a[1];
            const cudaLaunchConfig_t c = config_of(cl, 1, a, nullptr);
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, attend_pages_kernel, &c) != cudaSuccess) {
                cudaGetLastError();
                n = -1;
            }
            active[cl] = n < 1 ? -1 : n;
        }
        if (active[cl] >= units) break;
    }
    return cl;
}

}  // namespace

cudaError_t launch_attend_pages(const Params& p, const void* q_rot, const KvSources& kv,
                                const int32_t* sel_groups, const int32_t* n_sel_groups, void* out,
                                cudaStream_t st) {
    const int64_t res_rows = p.kv_layout == HGA_KV_WINDOWS
                                 ? (int64_t)(p.n_sink + p.n_local + 1) * p.C
                                 : (int64_t)p.L;
    const dec::PageSource res{(const uint8_t*)kv.k_res, (const uint8_t*)kv.v_res,
                              dec::page_slab(res_rows)};
    const dec::PageSource gat{(const uint8_t*)kv.k_gat, (const uint8_t*)kv.v_gat,
                              (int64_t)p.kg * kE2m1Page};
    int dev = 0, sms = 148;
    cudaError_t e = current_device_index(&dev);
    if (e != cudaSuccess) return e;
    e = set_func_attr_once((const void*)attend_pages_kernel,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(PagesSmem));
    if (e == cudaSuccess)
        e = set_func_attr_once((const void*)attend_pages_kernel,
                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t units = (int64_t)p.q_len * p.B * p.Hu;
    const int blocks = forced_of(p, p.q_begin + p.q_len - 1).blocks + p.kg;
    int64_t most = (int64_t)kCtasPerSm * sms / units;
    if (most > (blocks + kWarps - 1) / kWarps) most = (blocks + kWarps - 1) / kWarps;
    most = most < 1 ? 1 : (most > kMaxCluster ? kMaxCluster : most);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t c = config_of(cluster_size((int)most, units, dev), units, attr, st);
    return cudaLaunchKernelEx(&c, attend_pages_kernel, res, gat, p, (const __nv_bfloat16*)q_rot,
                              sel_groups, n_sel_groups, (__nv_bfloat16*)out);
}

}  // namespace hga
