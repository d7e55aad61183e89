// dense_gemm_pairsplit.cuh -- the dense products on CTA-pair tiles (256 x BN) with
// the reduction over K split over a cluster.
//
// Between about 129 rows and the sizes that fill the GPU with whole 256 x 256 tiles
// (dense_gemm_pair.cu).  An SM takes in 64 bytes a clock: a one-CTA 128 x 128
// tile asks for 32 KB each 256 clocks of MMA and runs at half speed (0.24 us a
// k-block).  A pair's tile halves B's share: 24 KB for the same work with BN = 128
// (0.21 us), 32 KB for twice the work with BN = 256 (0.30 us).  Measured: linear
// 1001 x 4096 x 2056 18.2 us with a residual (0.93 PFLOP/s), gated 256 x 7168 x
// 2048 18.3 us, weight gradient 777 x 1024 x 4096 8.6 us.  Tiles that do not fill
// the GPU are split over K: S pairs form a cluster of 2 S CTAs, each pair parks
// its fp32 accumulator in shared memory (the stages are free by then), and after
// a cluster barrier each CTA adds every S-th of its 128 rows over the S parked
// copies, in order, through distributed shared memory, and runs the epilogue.
//
// Roles and bounded waits as in dense_gemm_split.cuh, with BN columns; full is the
// even CTA's and counts both CTAs' bytes, empty and done are multicast commits to
// both.
#pragma once

#include <algorithm>
#include <atomic>

#include "dense_gemm.cuh"

namespace moe {

namespace {

constexpr int kPsThreads = 256;
constexpr int kPsA = kBM * kRowBytes;  // 16 KB: this CTA's 128 rows x 64 K, or two MN-major boxes

template <int BN>
struct PsCfg {
    static constexpr int B_BYTES = BN / 2 * kRowBytes;  // this CTA's half of B
    static constexpr int STAGE = kPsA + B_BYTES;
    static constexpr int STAGES = BN == 256 ? 6 : 8;
    static_assert(kBM * BN * 4 <= STAGES * STAGE, "the parked accumulator reuses the stages");
};

template <int KIND, int BN, int SPLITS>
constexpr size_t kPsSmem =
    1024 + static_cast<size_t>(PsCfg<BN>::STAGES) * PsCfg<BN>::STAGE + kResidualBytes<KIND, BN, SPLITS> + 256;

template <int KIND, int BN, int SPLITS>
__global__ void __launch_bounds__(kPsThreads)
dense_pairsplit_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                       const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                       const DenseArgs a) {
    using L = DenseLayout<KIND>;
    using C = PsCfg<BN>;
    constexpr int S = C::STAGES;
    constexpr int N_TILE = L::GATED ? BN / 2 : BN;  // output columns of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);  // identical offsets in all CTAs
    constexpr int RES = kResidualBytes<KIND, BN, SPLITS>;
    uint8_t* res = smem + S * C::STAGE;
    uint64_t* full = reinterpret_cast<uint64_t*>(res + RES);
    uint64_t* empty = full + S;
    uint64_t* done = empty + S;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* progress = abort_flag + 1;  // changes with every 256th k-block whose copy of A was issued
    volatile int never = 0;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank(), rank = crank & 1u, lead = crank & ~1u, part = crank >> 1;
    const bool leader = rank == 0;
    const uint16_t both = static_cast<uint16_t>(0x3u << lead);
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmA0);
        tma_prefetch_desc(&tmB0);
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        *progress = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, BN);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // tile: m fastest, so that concurrent clusters share the weight columns
    const int mt = (a.M + 2 * kBM - 1) / (2 * kBM), nt = (a.N + N_TILE - 1) / N_TILE;
    int tile = blockIdx.x / (2 * SPLITS);
    const int mat = tile / (mt * nt);
    tile -= mat * mt * nt;
    const int m0 = (tile % mt) * 2 * kBM + static_cast<int>(rank) * kBM, n0 = (tile / mt) * N_TILE;
    const int kbs = (a.K + kBK - 1) / kBK;  // k-blocks of one segment
    const int total = kbs * a.segs;
    const int k_lo = static_cast<int>(static_cast<long long>(total) * part / SPLITS);
    const int k_hi = static_cast<int>(static_cast<long long>(total) * (part + 1) / SPLITS);
    const uint32_t full_lead = mapa_shared(smem_u32(full), lead);
    pdl_wait();

    if (warp == 0) {  // copies of A; the even CTA's also announces the stage's bytes
        if (lane == 0) {
            bool withhold = a.dbg && (*a.dbg & MOE_DBG_WITHHOLD_FIRST_LOAD) && blockIdx.x == 0;
            uint32_t pending = 0, pend_parity = 0;
            int stage = 0, seg = k_lo / kbs, kb = k_lo - seg * kbs;
            uint32_t phase = 0;
            bool ok = true;
            for (int n = k_hi - k_lo; n > 0; --n) {
                if (!pipe_wait(&empty[stage], phase ^ 1u, abort_flag, a.err)) { ok = false; break; }
                if (withhold) {
                    withhold = false;  // test hook: this stage never fills
                } else {
                    const uint32_t bar = full_lead + 8u * stage;
                    uint8_t* sA = smem + stage * C::STAGE;
                    if (leader) {
                        mbar_arrive_expect_tx(&full[stage], 2 * C::STAGE);
                        pending |= 1u << stage;
                        pend_parity = (pend_parity & ~(1u << stage)) | (phase << stage);
                    }
                    const CUtensorMap* mA = (seg | mat) ? &tmA1 : &tmA0;
                    if constexpr (L::A_MN) {
                        tma_load_2d_pair(mA, bar, sA, m0, kb * kBK);
                        tma_load_2d_pair(mA, bar, sA + kMnBlockBytes, m0 + 64, kb * kBK);
                    } else {
                        tma_load_2d_pair(mA, bar, sA, kb * kBK, m0);
                    }
                }
                if ((n & 255) == 0) *progress = n;
                if (++kb == kbs) { kb = 0; ++seg; }
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
            for (int s = 0; s < S; ++s)
                if (pending & (1u << s)) drain_wait(&full[s], (pend_parity >> s) & 1u, a.err);
            if (!ok) settle_copies();
        }
    } else if (warp == 2) {  // copies of B
        if (lane == 0) {
            const int bcol = n0 + (L::GATED ? 0 : static_cast<int>(rank) * (BN / 2));
            int stage = 0, seg = k_lo / kbs, kb = k_lo - seg * kbs;
            uint32_t phase = 0;
            bool ok = true;
            for (int n = k_hi - k_lo; n > 0; --n) {
                if (!pipe_wait(&empty[stage], phase ^ 1u, abort_flag, a.err)) { ok = false; break; }
                const uint32_t bar = full_lead + 8u * stage;
                uint8_t* sB = smem + stage * C::STAGE + kPsA;
                const CUtensorMap* mB = L::GATED ? (rank ? &tmB1 : &tmB0) : (L::B_MN && seg ? &tmB1 : &tmB0);
                if constexpr (L::B_MN) {
                    tma_load_2d_pair(mB, bar, sB, bcol, kb * kBK);
                    if constexpr (BN == 256) tma_load_2d_pair(mB, bar, sB + kMnBlockBytes, bcol + 64, kb * kBK);
                } else {
                    tma_load_2d_pair(mB, bar, sB, kb * kBK, bcol);
                }
                if (++kb == kbs) { kb = 0; ++seg; }
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
            if (!ok) settle_copies();  // some may be of stages that were never announced
        }
    } else if (warp == 1) {
        if (leader) {
            constexpr uint32_t idesc = dense_idesc<KIND>(2 * kBM, BN);
            StageWalk w(full, S);
            for (int n = 0; n < k_hi - k_lo; ++n) {
                if (!w.wait(abort_flag, a.err)) break;
                tc_fence_after();
                const uint32_t sA = smem_u32(smem + w.stage * C::STAGE);
                const uint64_t ad = operand_desc<L::A_MN>(sA), bd = operand_desc<L::B_MN>(sA + kPsA);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)
                        umma_bf16_pair(tmem, ad + k * kDescStep<L::A_MN>, bd + k * kDescStep<L::B_MN>, idesc,
                                       (n | k) != 0 ? 1u : 0u);
                    umma_commit_pair_multicast(&empty[w.stage], both);
                }
                __syncwarp();
                w.advance();
            }
            if (elect_one()) umma_commit_pair_multicast(done, both);
            __syncwarp();
        }
        if (lane == 0) {
            // to the end whatever happened: TMEM is released below, nothing may be in flight
            idle_wait(done, 0, &never, progress, a.err);
        }
    }
    if constexpr (RES > 0) {
        if (warp >= 4 && a.residual) fetch_residual<BN, SPLITS>(a, res, m0, n0, static_cast<int>(part), threadIdx.x - 128);
    }
    __syncwarp();
    __syncthreads();  // the accumulator is complete (or the product was given up)
    const bool ok = *abort_flag == 0;
    tc_fence_after();
    const int q = warp & 3, half = warp >> 2;  // TMEM lanes 32 q .., columns of this half
    if constexpr (SPLITS == 1) {
        // nothing to join: from TMEM through the epilogue, 32 x 32 at a time
        if (ok) {
            WholeEpilogue<KIND, BN> e{a, smem + warp * kChunkBytes, m0, n0, q, half, lane, {}};
            if (RES == 0) e.fetch_ahead();
            e.run(mat, tmem, RES > 0 && a.residual ? res : nullptr);
        }
        __syncwarp();
        pdl_trigger();
        tc_fence_before();
        __syncthreads();
        cluster_sync_all();  // neither CTA leaves while the other may still signal it
        if (warp == 1) {
            tc_fence_after();
            tmem_dealloc_pair(tmem, BN);
        }
        return;
    }
    if (ok && m0 + q * 32 < a.M) park_rows<BN>(smem, tmem, q, half, lane);  // rows that exist
    __syncwarp();
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // every CTA's accumulator is parked and read from TMEM
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, BN);
    }

    join_parts<KIND, BN, SPLITS>(a, mat, smem, res, m0, n0, static_cast<int>(part), rank, 2);
    cluster_sync_all();  // no CTA leaves while another reads its shared memory or signals it
}

template <int KIND, int BN, int SPLITS>
cudaLaunchConfig_t ps_config(cudaLaunchAttribute (&attr)[2], cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * SPLITS);
    cfg.blockDim = dim3(kPsThreads);
    cfg.dynamicSmemBytes = kPsSmem<KIND, BN, SPLITS>;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * SPLITS;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cfg;
}

// Clusters the current device holds at once (kept per device).
template <int KIND, int BN, int SPLITS>
cudaError_t ps_prepare(int* clusters) {
    static std::atomic<unsigned long long> done{0};
    static int limit[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(dense_pairsplit_kernel<KIND, BN, SPLITS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kPsSmem<KIND, BN, SPLITS>));
        if (e != cudaSuccess) return e;
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = ps_config<KIND, BN, SPLITS>(attr, nullptr);
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, dense_pairsplit_kernel<KIND, BN, SPLITS>, &cfg);
        if (e != cudaSuccess) return e;
        limit[dev & 63] = n;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    *clusters = limit[dev & 63];
    return *clusters > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int KIND, int BN, int SPLITS>
cudaError_t ps_go(const CUtensorMap* m, const DenseArgs& a, cudaStream_t st, int* clusters) {
    if (clusters) return ps_prepare<KIND, BN, SPLITS>(clusters);
    int limit = 0;
    cudaError_t e = ps_prepare<KIND, BN, SPLITS>(&limit);
    if (e != cudaSuccess) return e;
    constexpr int n_tile = DenseLayout<KIND>::GATED ? BN / 2 : BN, m_tile = 2 * kBM;
    const long long tiles = static_cast<long long>((a.M + m_tile - 1) / m_tile) * ((a.N + n_tile - 1) / n_tile) * a.mats;
    if (tiles * 2 * SPLITS > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = ps_config<KIND, BN, SPLITS>(attr, st);
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * 2 * SPLITS));
    return cudaLaunchKernelEx(&cfg, dense_pairsplit_kernel<KIND, BN, SPLITS>, m[0], m[1], m[2], m[3], a);
}

}  // namespace

// clusters != NULL asks only for how many the device holds at once.
template <int KIND>
cudaError_t dense_pairsplit_pick(const CUtensorMap* m, const DenseArgs& a, int bn, int splits, cudaStream_t st,
                                 int* clusters) {
    if (bn == 128) {
        switch (splits) {
            case 1: return ps_go<KIND, 128, 1>(m, a, st, clusters);
            case 2: return ps_go<KIND, 128, 2>(m, a, st, clusters);
            case 4: return ps_go<KIND, 128, 4>(m, a, st, clusters);
            default: return cudaErrorInvalidConfiguration;
        }
    }
    switch (splits) {
        case 1: return ps_go<KIND, 256, 1>(m, a, st, clusters);
        case 2: return ps_go<KIND, 256, 2>(m, a, st, clusters);
        case 4: return ps_go<KIND, 256, 4>(m, a, st, clusters);
        default: return cudaErrorInvalidConfiguration;
    }
}

}  // namespace moe
