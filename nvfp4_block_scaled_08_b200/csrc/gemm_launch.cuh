// gemm_launch.cuh -- host-side launch of one variant of the persistent GEMM kernel: its TMA
// descriptors, kernel arguments and launch attributes. Included by the translation units that
// instantiate variants (gemm.cu: the plain products, gemm_fused.cu: the fused epilogues).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>
#include <mutex>

#include "gemm_kernel.cuh"
#include "internal.h"

namespace nvfp4 {

constexpr int kMaxDevicesForAttr = 64;

// gemm.cu: largest number of clusters of `cs` CTAs (one CTA per SM, as every GEMM variant here
// uses over 100 KB of shared memory) that the current device runs at once; cached per
// device. Clusters are placed inside a GPC, so this is below num_sms / cs.
int max_active_clusters(int cs);

// gemm.cu: uint8 tensor of `rank` (2 ... 5) dims (innermost first: dims[0] bytes per row), strides of
// dims 1 .. rank-1 in bytes, box extents per dim; cached per (pointer, geometry, device).
bool get_map_nd(CUtensorMap* out, const void* ptr, int rank, const uint64_t* dims,
                const uint64_t* strides, const uint32_t* box, int swizzle);

// Shared-memory swizzles of a tensor map's box.
enum : int { kSwizzleNone = 0, kSwizzle128 = 1, kSwizzle64 = 2 };

// uint8 tensor of `rank` (2 or 3) dims {inner bytes, rows[, depth]} with row stride
// `stride1` and depth stride `stride2` (bytes); box {box0, box1[, 1]}.
inline bool get_map(CUtensorMap* out, const void* ptr, int rank, uint64_t d0, uint64_t d1,
                    uint64_t d2, uint64_t stride1, uint64_t stride2, uint32_t box0, uint32_t box1,
                    bool swizzle128)
{
    const uint64_t dims[3] = {d0, d1, d2};
    const uint64_t strides[2] = {stride1, stride2};
    const uint32_t box[3] = {box0, box1, 1};
    return get_map_nd(out, ptr, rank, dims, strides, box, swizzle128 ? kSwizzle128 : kSwizzleNone);
}

// The gate_up weights [E, 2I, row_bytes] viewed so that one box of 128 rows holds four groups of
// [16 gate rows j .. j + 15, the 16 up rows I + j .. I + j + 15]: dims (innermost first)
// {row_bytes, 16 rows, gate/up, I / 16 groups, E}, strides {row_bytes, I rows, 16 rows,
// 2I rows}, box {box0, 16, 2, groups, 1} (groups of 32 rows: 4 for a 128-row box).
inline bool get_map_swiglu(CUtensorMap* out, const void* ptr, uint64_t row_bytes, uint64_t I, uint64_t E,
                           uint32_t box0, bool swizzle128, uint32_t groups = 4)
{
    const uint64_t dims[5] = {row_bytes, 16, 2, I / 16, E};
    const uint64_t strides[4] = {row_bytes, I * row_bytes, 16 * row_bytes, 2 * I * row_bytes};
    const uint32_t box[5] = {box0, 16, 2, groups, 1};
    return get_map_nd(out, ptr, 5, dims, strides, box, swizzle128 ? kSwizzle128 : kSwizzleNone);
}

template <int BN, bool SWAP, bool GROUPED, bool SFT = false, bool SWIGLU = false, bool MX = false,
          bool PAIR = false, bool ACTQ = false, int EPI = kEpiPlain>
static cudaError_t run(const GemmPlan& plan, const GemmLaunch& L, cudaStream_t stream,
                       bool* encode_failed)
{
    using Cfg = GemmCfg<BN, SWAP, GROUPED, SFT, SWIGLU, MX, PAIR, ACTQ, EPI>;
    auto kern = nvfp4_gemm_kernel<Cfg>;
    // Opt in to the large dynamic shared memory once per device (not a stream operation,
    // so a later launch may be captured into a CUDA graph).
    static std::once_flag attr_once[kMaxDevicesForAttr];
    static cudaError_t attr_err[kMaxDevicesForAttr];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevicesForAttr) return cudaErrorInvalidDevice;
    std::call_once(attr_once[dev], [&] {
        attr_err[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Cfg::SMEM_BYTES);
    });
    if (attr_err[dev] != cudaSuccess) return attr_err[dev];

    const uint64_t kb = static_cast<uint64_t>(L.K / 2);    // packed bytes per row
    const uint64_t ks = static_cast<uint64_t>(L.K / 16);   // scale bytes per row
    CUtensorMap tp, tq, tsp, tsq, tq_half;
    EpiMaps<Cfg::EPI_SIDE> em;
    std::memset(&em, 0, sizeof(em));
    bool ok = true;
    GemmArgs a;
    std::memset(&a, 0, sizeof(a));
    a.cluster_size = 1;
    a.groups = 1;
    a.M = static_cast<int32_t>(L.M);
    a.N = static_cast<int32_t>(L.N);
    a.num_kstages = static_cast<int32_t>(L.K / 256);
    a.num_p_tiles = plan.p_tiles;
    a.out = L.out;
    a.out_dtype = L.out_dtype;
    a.alpha = L.alpha;
    a.err_word = L.err_word;
    a.b_ready = L.b_ready ? 1 : 0;
    if constexpr (GROUPED) {
        const uint64_t E = static_cast<uint64_t>(L.E);
        const uint64_t rows = static_cast<uint64_t>(L.total_rows);
        if constexpr (SWIGLU) {
            const uint64_t I = static_cast<uint64_t>(L.N / 2);
            ok &= get_map_swiglu(&tp, L.B, kb, I, E, 128, true);
            ok &= get_map_swiglu(&tsp, L.sfB, ks, I, E, 16, false);
            a.h_q = L.h_q;
            a.h_sf = L.h_sf;
            a.gs_h = L.gs_h;
            a.inter = static_cast<int32_t>(I);
        } else {
            ok &= get_map(&tp, L.B, 3, kb, L.N, E, kb, kb * L.N, 128, 128, true);
            ok &= get_map(&tsp, L.sfB, 3, ks, L.N, E, ks, ks * L.N, 16, 128, false);
        }
        ok &= get_map(&tq, L.A, 2, kb, rows, 1, kb, 0, 128, Cfg::QBOX, true);
        ok &= get_map(&tsq, L.sfA, 2, ks, rows, 1, ks, 0, 16, Cfg::QBOX, false);
        a.p_rows = a.N;
        a.q_rows = static_cast<int32_t>(L.total_rows);
        a.splits = 1;
        if constexpr (PAIR) a.num_p_tiles = static_cast<int32_t>((L.N + 255) / 256);   // weight tile pairs
        a.expert_offsets = L.offsets;
        a.num_experts = L.E;
        a.total_rows = static_cast<int32_t>(L.total_rows);
    } else {
        const uint8_t* P = SWAP ? L.B : L.A;
        const uint8_t* sP = SWAP ? L.sfB : L.sfA;
        const uint8_t* Q = SWAP ? L.A : L.B;
        const uint8_t* sQ = SWAP ? L.sfA : L.sfB;
        const uint64_t p_rows = static_cast<uint64_t>(SWAP ? L.N : L.M);
        const uint64_t q_rows = static_cast<uint64_t>(SWAP ? L.M : L.N);
        // GLU: the weight operand through its gate / up row groups
        constexpr bool GLU_P = Cfg::GLU && SWAP, GLU_Q = Cfg::GLU && !SWAP;
        const uint64_t I = static_cast<uint64_t>(L.N / 2);
        constexpr uint32_t QB = PAIR ? BN / 2 : BN;   // PAIR: half tiles
        if constexpr (GLU_P) ok &= get_map_swiglu(&tp, P, kb, I, 1, 128, true);
        else ok &= get_map(&tp, P, 2, kb, p_rows, 1, kb, 0, 128, 128, true);
        if constexpr (ACTQ) tq = tp;          // unused: the kernel quantises the activations itself
        else if constexpr (GLU_Q) ok &= get_map_swiglu(&tq, Q, kb, I, 1, 128, true, QB / 32);
        else ok &= get_map(&tq, Q, 2, kb, q_rows, 1, kb, 0, 128, QB, true);
        // PAIR, BN = 256: each CTA's 64 rows of a 256 x 128 half tile
        if constexpr (Cfg::NARROW && GLU_Q) ok &= get_map_swiglu(&tq_half, Q, kb, I, 1, 128, true, BN / 4 / 32);
        else if constexpr (Cfg::NARROW) ok &= get_map(&tq_half, Q, 2, kb, q_rows, 1, kb, 0, 128, BN / 4, true);
        if constexpr (Cfg::EPI_SIDE) {
            // the side input in boxes of 64 bytes x 32 rows
            const uint64_t esz = L.out_dtype == kOutF32 ? 4 : 2;
            const uint32_t box[2] = {64, 32};
            const uint64_t sd[2] = {(EPI == kEpiGluGrad ? I : static_cast<uint64_t>(L.N)) * esz, static_cast<uint64_t>(L.M)};
            if (L.side) ok &= get_map_nd(&em.side, L.side, 2, sd, sd, box, kSwizzle64);
        }
        if constexpr (EPI != kEpiPlain) {
            a.act_fn = L.act_fn;
            a.bias = L.bias;
            a.side = L.side;
            a.side_scale = L.side_scale;
            a.h_q = L.h_q;
            a.h_sf = L.h_sf;
            a.gs_h = L.gs_h;
            a.h_sf_tiled = L.h_sf_tiled ? 1 : 0;
            a.inter = static_cast<int32_t>(I);
        }
        if constexpr (PAIR) {
            // the tiled scales as rows of 256 bytes: a stage's run of one 128-row tile is
            // SFP_BYTES / 256 rows (past the last tile: zero fill)
            const uint64_t sp_rows = (p_rows + 127) / 128 * (L.K / (MX ? 64 : 32));
            const uint64_t sq_rows = (q_rows + 127) / 128 * (L.K / (MX ? 64 : 32));
            ok &= get_map(&tsp, sP, 2, 256, sp_rows, 1, 256, 0, 256, Cfg::SF_ROWS256, false);
            ok &= get_map(&tsq, sQ, 2, 256, sq_rows, 1, 256, 0, 256, Cfg::SF_ROWS256, false);
            a.sf_p = sP;
            a.sf_q = sQ;
            a.sf_kb4 = static_cast<int32_t>(L.K / (MX ? 128 : 64));
        } else if constexpr (SFT) {
            tsp = tp;                       // unused: the scales come by bulk copy
            tsq = tq;
            a.sf_p = sP;
            a.sf_q = sQ;
            a.sf_kb4 = static_cast<int32_t>(L.K / (MX ? 128 : 64));   // 512-byte blocks per 128 rows
        } else if (L.sf_8x4) {
            // rows of the map: 8-row groups of K / 2 bytes; a stage's box: 128 bytes of 128 / 8
            // (P) or BN / 8 (Q) groups, the same bytes as the row-major box
            const uint64_t gb = static_cast<uint64_t>(L.K / 2);
            ok &= get_map(&tsp, sP, 2, gb, (p_rows + 7) / 8, 1, gb, 0, 128, 128 / 8, false);
            ok &= get_map(&tsq, sQ, 2, gb, (q_rows + 7) / 8, 1, gb, 0, 128, BN / 8, false);
            a.sf_8x4 = 1;
        } else {
            ok &= get_map(&tsp, sP, 2, ks, p_rows, 1, ks, 0, 16, 128, false);
            ok &= get_map(&tsq, sQ, 2, ks, q_rows, 1, ks, 0, 16, BN, false);
        }
        a.p_rows = static_cast<int32_t>(p_rows);
        a.q_rows = static_cast<int32_t>(q_rows);
        if constexpr (ACTQ) {
            a.act = L.act;
            a.act_ld = L.act_ld;
            a.act_bf16 = L.act_bf16 ? 1 : 0;
            a.gs_b = L.gs_b;
            a.gs_out = L.gs_out;
            a.alpha_out = L.alpha_out;
        }
        a.num_q_tiles = plan.q_tiles;
        if constexpr (PAIR) a.num_p_tiles = (plan.p_tiles + 1) / 2;   // work items are P tile pairs
        a.splits = plan.splits;
        a.cluster_size = plan.cluster;
        a.groups = plan.groups;
        a.num_tiles = plan.num_tiles;
        a.band = plan.band;
        if (plan.groups > 1) {
            a.ws_counters = static_cast<uint32_t*>(L.ws);
            a.ws_partial = reinterpret_cast<float*>(static_cast<uint8_t*>(L.ws) + plan.ws_counter_bytes);
        }
    }
    if constexpr (!Cfg::NARROW) tq_half = tq;   // unused
    if (!ok) {
        *encode_failed = true;
        return cudaSuccess;
    }
    if constexpr (PAIR) {
        a.band = plan.pair_band;
        a.num_tiles = plan.pair_items;
        a.narrow_from = plan.narrow_from;
    }
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(PAIR ? plan.pair_grid : plan.grid), 1, 1);
    cfg.blockDim = dim3(kGemmThreads, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = stream;
    // programmatic dependent launch: the prologue overlaps the previous kernel's tail
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = static_cast<unsigned>(plan.cluster);
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    if constexpr (PAIR) attrs[1].val.clusterDim.x = 2;
    cfg.attrs = attrs;
    cfg.numAttrs = (PAIR || (!GROUPED && plan.cluster > 1)) ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, tp, tq, tsp, tsq, tq_half, a, em);
}

}  // namespace nvfp4
