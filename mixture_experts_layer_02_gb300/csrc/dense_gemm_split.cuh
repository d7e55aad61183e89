// dense_gemm_split.cuh -- the dense products on one-CTA 128 x 128 tiles with the
// reduction over K split over a cluster.
//
// A product with few tiles (few tokens, or a small weight gradient) leaves most
// SMs idle when one CTA owns a whole tile.  Here a cluster of S CTAs shares a
// tile: CTA r multiplies k-blocks [r T / S, (r + 1) T / S), parks its fp32
// accumulator in its own shared memory (the operand stages are free by then)
// and, after a cluster barrier, adds its 1/S of the tile over the S parked
// accumulators in rank order through distributed shared memory and runs the
// epilogue on the sums.  No fp32 partials reach HBM, there is no second launch,
// and the order of the additions is fixed.
//
// Used for up to about 128 rows, where the weights come from HBM once and latency
// is the rest, and above that where its rounds come out better than a pair's.
//   - Time stamps at 256 x 4096 x 4096 (S = 2, 32 k-blocks a CTA) showed a TMA
//     round trip of 1.1 us: three 32 KB stages moved a k-block each 0.37 us, six
//     (one CTA an SM) and separate copy threads each 0.23 us.  That is what an SM
//     takes in (64 bytes a clock), whichever SM or L2 it comes from.
//   - With K in parts, 4 to 5 us follow the main loop: parking 0.5, barrier 0.6,
//     sums 1.4 (one latency of loads from other CTAs), epilogue 0.2 a row of quads,
//     barrier 0.6.  The loads are all in flight at once, rows are dealt to the CTAs
//     in turn (33 rows would otherwise leave the join to one of them), rows that do
//     not exist are neither parked nor read, and the residual waits in shared memory.
//   Measured: gated 100 x 2048 x 768 7.2 us, linear 64 x 7168 x 2048 11.1 us,
//   33 x 2048 x 2048 6.0 us.
//
// Warp roles: 0 copies A, 2 copies B (one thread issuing both took longer than a
// k-block's MMAs), 1 allocates TMEM and issues the MMAs; all eight
// park the accumulator (warp w reads TMEM lanes 32 (w % 4) .. and columns 64
// (w / 4) ..), join and run the epilogue.
//
// Every wait is bounded; whatever a role sees, every thread reaches
// both cluster barriers, so no CTA waits for one that left.
#pragma once

#include <algorithm>
#include <atomic>

#include "dense_gemm.cuh"

namespace moe {

namespace {

constexpr int kSplitBN = 128;
constexpr int kSplitStages = 6;
constexpr int kSplitThreads = 256;
constexpr int kOperandBytes = kBM * kRowBytes;  // 16 KB: 128 rows x 64 K, or two MN-major boxes
constexpr int kSplitStageBytes = 2 * kOperandBytes;
template <int KIND, int SPLITS>
constexpr size_t kSplitSmem = 1024 + kSplitStages * kSplitStageBytes + kResidualBytes<KIND, kSplitBN, SPLITS> + 128;
static_assert(kBM * kSplitBN * 4 <= kSplitStages * kSplitStageBytes, "the parked accumulator reuses the stages");

template <int KIND, int SPLITS>
__global__ void __launch_bounds__(kSplitThreads)
dense_split_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                   const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                   const DenseArgs a) {
    using L = DenseLayout<KIND>;
    constexpr int S = kSplitStages;
    constexpr int N_TILE = L::GATED ? kSplitBN / 2 : kSplitBN;  // output columns of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    constexpr int RES = kResidualBytes<KIND, kSplitBN, SPLITS>;
    uint8_t* res = smem + S * kSplitStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(res + RES);
    uint64_t* empty = full + S;
    uint64_t* done = empty + S;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int never = 0;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = SPLITS > 1 ? cluster_ctarank() : 0u;  // the k-part
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmA0);
        tma_prefetch_desc(&tmB0);
        if (L::GATED) tma_prefetch_desc(&tmB1);
    }

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kSplitBN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // tile: m fastest, so that concurrent CTAs share the weight columns
    const int mt = (a.M + kBM - 1) / kBM, nt = (a.N + N_TILE - 1) / N_TILE;
    int tile = blockIdx.x / SPLITS;
    const int mat = tile / (mt * nt);
    tile -= mat * mt * nt;
    const int m0 = (tile % mt) * kBM, n0 = (tile / mt) * N_TILE;
    const int kbs = (a.K + kBK - 1) / kBK;  // k-blocks of one segment
    const int total = kbs * a.segs;
    const int k_lo = static_cast<int>(static_cast<long long>(total) * rank / SPLITS);
    const int k_hi = static_cast<int>(static_cast<long long>(total) * (rank + 1) / SPLITS);
    pdl_wait();

    if (warp == 0) {  // copies of A, and the announcement of the stage's bytes
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
                    uint8_t* sA = smem + stage * kSplitStageBytes;
                    const CUtensorMap* mA = (seg | mat) ? &tmA1 : &tmA0;
                    mbar_arrive_expect_tx(&full[stage], kSplitStageBytes);
                    pending |= 1u << stage;
                    pend_parity = (pend_parity & ~(1u << stage)) | (phase << stage);
                    if constexpr (L::A_MN) {
                        tma_load_2d(mA, &full[stage], sA, m0, kb * kBK);
                        tma_load_2d(mA, &full[stage], sA + kMnBlockBytes, m0 + 64, kb * kBK);
                    } else {
                        tma_load_2d(mA, &full[stage], sA, kb * kBK, m0);
                    }
                }
                if (++kb == kbs) { kb = 0; ++seg; }
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
            for (int s = 0; s < S; ++s)
                if (pending & (1u << s)) drain_wait(&full[s], (pend_parity >> s) & 1u, a.err);
            if (!ok) settle_copies();
        }
    } else if (warp == 2) {  // copies of B
        if (lane == 0) {
            int stage = 0, seg = k_lo / kbs, kb = k_lo - seg * kbs;
            uint32_t phase = 0;
            bool ok = true;
            for (int n = k_hi - k_lo; n > 0; --n) {
                if (!pipe_wait(&empty[stage], phase ^ 1u, abort_flag, a.err)) { ok = false; break; }
                uint8_t* sB = smem + stage * kSplitStageBytes + kOperandBytes;
                if constexpr (L::GATED) {
                    tma_load_2d(&tmB0, &full[stage], sB, kb * kBK, n0);
                    tma_load_2d(&tmB1, &full[stage], sB + kOperandBytes / 2, kb * kBK, n0);
                } else if constexpr (L::B_MN) {
                    const CUtensorMap* mB = seg ? &tmB1 : &tmB0;
                    tma_load_2d(mB, &full[stage], sB, n0, kb * kBK);
                    tma_load_2d(mB, &full[stage], sB + kMnBlockBytes, n0 + 64, kb * kBK);
                } else {
                    tma_load_2d(&tmB0, &full[stage], sB, kb * kBK, n0);
                }
                if (++kb == kbs) { kb = 0; ++seg; }
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
            if (!ok) settle_copies();  // some may be of stages that were never announced
        }
    } else if (warp == 1) {
        constexpr uint32_t idesc = dense_idesc<KIND>(kBM, kSplitBN);
        StageWalk w(full, S);
        for (int n = 0; n < k_hi - k_lo; ++n) {
            if (!w.wait(abort_flag, a.err)) break;
            tc_fence_after();
            const uint32_t sA = smem_u32(smem + w.stage * kSplitStageBytes);
            const uint64_t ad = operand_desc<L::A_MN>(sA), bd = operand_desc<L::B_MN>(sA + kOperandBytes);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k)
                    umma_bf16(tmem, ad + k * kDescStep<L::A_MN>, bd + k * kDescStep<L::B_MN>, idesc, (n | k) != 0 ? 1u : 0u);
                umma_commit(&empty[w.stage]);
            }
            __syncwarp();
            w.advance();
        }
        if (elect_one()) umma_commit(done);
        __syncwarp();
        if (lane == 0) {
            // to the end whatever happened: TMEM is released below, nothing may be in flight
            idle_wait(done, 0, &never, &never, a.err);
        }
    }
    if constexpr (RES > 0) {
        if (warp >= 4 && a.residual) fetch_residual<kSplitBN, SPLITS>(a, res, m0, n0, static_cast<int>(rank), threadIdx.x - 128);
    }
    __syncwarp();
    __syncthreads();  // the accumulator is complete (or the product was given up)
    const bool ok = *abort_flag == 0;
    tc_fence_after();
    const int q = warp & 3, half = warp >> 2;  // TMEM lanes 32 q .., columns of this half
    if constexpr (SPLITS == 1) {
        // nothing to join: from TMEM through the epilogue, 32 x 32 at a time
        if (ok) {
            WholeEpilogue<KIND, kSplitBN> e{a, smem + warp * kChunkBytes, m0, n0, q, half, lane, {}};
            e.run(mat, tmem, RES > 0 && a.residual ? res : nullptr);
        }
        __syncwarp();
        pdl_trigger();
        tc_fence_before();
        __syncthreads();
        if (warp == 1) {
            tc_fence_after();
            tmem_dealloc(tmem, kSplitBN);
        }
        return;
    }
    if (ok && m0 + q * 32 < a.M) park_rows<kSplitBN>(smem, tmem, q, half, lane);  // rows that exist
    __syncwarp();
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kSplitBN);
    }
    cluster_sync_all();  // every CTA's accumulator is parked
    join_parts<KIND, kSplitBN, SPLITS>(a, mat, smem, res, m0, n0, static_cast<int>(rank), 0, 1);
    cluster_sync_all();  // no CTA leaves while another reads its shared memory
}

template <int KIND, int SPLITS>
cudaLaunchConfig_t split_config(cudaLaunchAttribute (&attr)[2], cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(SPLITS);
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = kSplitSmem<KIND, SPLITS>;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = SPLITS;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cfg;
}

// Clusters the current device holds at once (kept per device).
template <int KIND, int SPLITS>
cudaError_t split_prepare(int* clusters) {
    static std::atomic<unsigned long long> done{0};
    static int limit[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(dense_split_kernel<KIND, SPLITS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kSplitSmem<KIND, SPLITS>));
        if (e != cudaSuccess) return e;
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = split_config<KIND, SPLITS>(attr, nullptr);
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, dense_split_kernel<KIND, SPLITS>, &cfg);
        if (e != cudaSuccess) return e;
        limit[dev & 63] = n;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    *clusters = limit[dev & 63];
    return *clusters > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int KIND, int SPLITS>
cudaError_t split_go(const CUtensorMap* m, const DenseArgs& a, cudaStream_t st, int* clusters) {
    if (clusters) return split_prepare<KIND, SPLITS>(clusters);
    int limit = 0;
    cudaError_t e = split_prepare<KIND, SPLITS>(&limit);
    if (e != cudaSuccess) return e;
    constexpr int n_tile = DenseLayout<KIND>::GATED ? kSplitBN / 2 : kSplitBN;
    const long long tiles = static_cast<long long>((a.M + kBM - 1) / kBM) * ((a.N + n_tile - 1) / n_tile) * a.mats;
    if (tiles * SPLITS > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = split_config<KIND, SPLITS>(attr, st);
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * SPLITS));
    return cudaLaunchKernelEx(&cfg, dense_split_kernel<KIND, SPLITS>, m[0], m[1], m[2], m[3], a);
}

}  // namespace

// clusters != NULL asks only for how many the device holds at once.
template <int KIND>
cudaError_t dense_split_pick(const CUtensorMap* m, const DenseArgs& a, int splits, cudaStream_t st, int* clusters) {
    switch (splits) {
        case 1: return split_go<KIND, 1>(m, a, st, clusters);
        case 2: return split_go<KIND, 2>(m, a, st, clusters);
        case 4: return split_go<KIND, 4>(m, a, st, clusters);
        case 8: return split_go<KIND, 8>(m, a, st, clusters);
        default: return cudaErrorInvalidConfiguration;
    }
}

}  // namespace moe
