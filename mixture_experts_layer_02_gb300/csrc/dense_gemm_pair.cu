// dense_gemm_pair.cu -- the dense products on CTA pairs (tcgen05 cta_group::2),
// for products with enough tiles to occupy the GPU.
//
// A cluster of two CTAs on two SMs owns a 256 x 256 tile: each CTA loads its
// own 128 rows of A and its own half of B (for the gated product the even CTA
// holds the W1 rows and the odd one the W3 rows, so an accumulator row has the
// gate in columns 0..127 and the up projection in 128..255), and the even CTA
// issues the MMAs for both.  Two 256-column accumulators fill TMEM: the
// epilogue of a tile runs under the main loop of the next.
//
// The main loop.  A k-block is 512 clocks of MMA, and the threads that feed it
// have to be quicker than that: one thread issuing both operands' copies took
// 570 clocks a k-block (time stamps), the MMA issuer 480, of which 200 waited for
// the answer of a barrier that was complete.  So A and B have a copy thread each,
// the MMA warp walks the stages as a whole with the next barrier asked ahead
// (StageWalk), and no other warp polls during a main loop.  That took the tensor
// pipe from 89 to 95 .. 96 % of the active cycles: 505 us alone at 4096 x 4096 x
// 2 x 14336 keeping both projections (1.90 PFLOP/s), 576 to 587 us in a long run,
// where the board's power limit holds the clock near 1.5 GHz (1.65 PFLOP/s; a library
// product of 8192^3 runs at 1.71 there).  Asking L2 for later k-blocks ahead made
// every size 8 to 14 % slower.
//
// A last round that leaves pairs idle was dealt out along K over all of them (with
// fp32 fragments joined through memory): 273 instead of 297 us alone at 4096 x
// 14336 x 4096, but no gain in a long run, where power and not pairs is short,
// and slower at smaller sizes; it is not kept.
//
// Order of tiles: bands of 8 m-tiles, inside a band n by n, m innermost, so
// that the pairs working at one time share weight tiles and token rows in L2.
//
// Barriers as in grouped_gemm_2sm.cuh: full (even CTA, both CTAs' bytes),
// empty and tfull (multicast commits), tempty (even CTA, the 16 epilogue warps
// of both CTAs).  Every wait is bounded.  Warps: 0 copies A, 1 allocates TMEM and
// issues the MMAs, 2..9 epilogue, 10 copies B.
#include <algorithm>
#include <atomic>

#include "dense_gemm.cuh"

namespace moe {

namespace {

constexpr int kStages = 6;
constexpr int kOperand = kBM * kRowBytes;        // 16 KB: this CTA's half of an operand
constexpr int kStageBytes = 2 * kOperand;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (3 + kEpiWarps) * 32;  // A copies, MMA issuer, epilogue, B copies
constexpr int kBand = 8;
constexpr size_t kPairSmem = 1024 + static_cast<size_t>(kStages) * kStageBytes + kEpiWarps * kChunkBytes + (2 * kStages + 5) * 8 + 16;

// Tile t of the list, as its first row and column; mats products follow one another.
struct TilePlace {
    int mat, m0, n0;
};

__device__ __forceinline__ TilePlace place_tile(int t, int mt, int nt, int n_tile) {
    TilePlace w;
    w.mat = t / (mt * nt);
    t -= w.mat * mt * nt;
    const int band = t / (kBand * nt), in = t - band * kBand * nt;
    const int rows = min(kBand, mt - band * kBand);
    const int n = in / rows;
    w.m0 = (band * kBand + in - n * rows) * kPairTile;
    w.n0 = n * n_tile;
    return w;
}

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
dense_pair_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                  const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                  const DenseArgs a) {
    using L = DenseLayout<KIND>;
    constexpr int S = kStages;
    constexpr int N_TILE = L::GATED ? kPairTile / 2 : kPairTile;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    uint8_t* sA = smem;
    uint8_t* sB = smem + S * kOperand;
    uint64_t* full = reinterpret_cast<uint64_t*>(sB + S * kOperand + kEpiWarps * kChunkBytes);
    uint64_t* empty = full + S;
    uint64_t* tfull = empty + S;   // [2]
    uint64_t* tempty = tfull + 2;  // [2]
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* progress = abort_flag + 1;  // changes with every 256th k-block whose copy of A was issued

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();  // in the pair; its even CTA issues the MMAs
    const bool leader = rank == 0;
    constexpr uint16_t both = 0x3;
    uint32_t* err = a.err;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * kEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        *progress = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 2 * kPairTile);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int kbs = (a.K + kBK - 1) / kBK;
    const int total_kb = kbs * a.segs;
    const int mt = (a.M + kPairTile - 1) / kPairTile, nt = (a.N + N_TILE - 1) / N_TILE;
    const int tiles = mt * nt * a.mats, first = blockIdx.x / 2, step = gridDim.x / 2;
    const uint32_t full_lead = mapa_shared(smem_u32(full), 0);
    const uint32_t tempty_lead = mapa_shared(smem_u32(tempty), 0);
    pdl_wait();

    if (warp == 0) {  // copies of A; the even CTA's also announces the stage's bytes
        if (lane == 0) {
            bool withhold = a.dbg && (*a.dbg & MOE_DBG_WITHHOLD_FIRST_LOAD) && blockIdx.x == 0;
            uint32_t pending = 0, pend_parity = 0;
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = first; ok && tile < tiles; tile += step) {
                const TilePlace w = place_tile(tile, mt, nt, N_TILE);
                const int arow = w.m0 + static_cast<int>(rank) * kBM;
                for (int kb = 0; kb < total_kb; ++kb) {
                    if (!pipe_wait(&empty[stage], phase ^ 1u, abort_flag, err)) { ok = false; break; }
                    if (withhold) {
                        withhold = false;  // test hook: this stage never fills
                    } else {
                        const int seg = kb >= kbs ? 1 : 0, k0 = (kb - seg * kbs) * kBK;
                        const uint32_t bar = full_lead + 8u * stage;
                        uint8_t* dA = sA + stage * kOperand;
                        if (leader) {
                            mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
                            pending |= 1u << stage;
                            pend_parity = (pend_parity & ~(1u << stage)) | (phase << stage);
                        }
                        const CUtensorMap* mA = (seg | w.mat) ? &tmA1 : &tmA0;
                        if constexpr (L::A_MN) {
                            tma_load_2d_pair(mA, bar, dA, arow, k0);
                            tma_load_2d_pair(mA, bar, dA + kMnBlockBytes, arow + 64, k0);
                        } else {
                            tma_load_2d_pair(mA, bar, dA, k0, arow);
                        }
                    }
                    if ((kb & 255) == 255) *progress = kb;
                    if (++stage == S) { stage = 0; phase ^= 1u; }
                }
            }
            for (int s = 0; s < S; ++s)
                if (pending & (1u << s)) drain_wait(&full[s], (pend_parity >> s) & 1u, err);
            if (!ok) settle_copies();
        }
    } else if (warp == 2 + kEpiWarps) {  // copies of B
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = first; ok && tile < tiles; tile += step) {
                const TilePlace w = place_tile(tile, mt, nt, N_TILE);
                const int bcol = w.n0 + (L::GATED ? 0 : static_cast<int>(rank) * (kPairTile / 2));
                for (int kb = 0; kb < total_kb; ++kb) {
                    if (!pipe_wait(&empty[stage], phase ^ 1u, abort_flag, err)) { ok = false; break; }
                    const int seg = kb >= kbs ? 1 : 0, k0 = (kb - seg * kbs) * kBK;
                    const uint32_t bar = full_lead + 8u * stage;
                    uint8_t* dB = sB + stage * kOperand;
                    const CUtensorMap* mB = L::GATED ? (rank ? &tmB1 : &tmB0) : (L::B_MN && seg ? &tmB1 : &tmB0);
                    if constexpr (L::B_MN) {
                        tma_load_2d_pair(mB, bar, dB, bcol, k0);
                        tma_load_2d_pair(mB, bar, dB + kMnBlockBytes, bcol + 64, k0);
                    } else {
                        tma_load_2d_pair(mB, bar, dB, k0, bcol);
                    }
                    if (++stage == S) { stage = 0; phase ^= 1u; }
                }
            }
            if (!ok) settle_copies();  // some may be of stages that were never announced
        }
    } else if (warp == 1) {
        if (leader) {
            constexpr uint32_t idesc = dense_idesc<KIND>(kPairTile, kPairTile);
            StageWalk w(full, S);
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (int tile = first; ok && tile < tiles; tile += step) {
                ok = __all_sync(0xffffffffu, pipe_wait(&tempty[acc], acc_phase ^ 1u, abort_flag, err));
                if (!ok) break;
                __syncwarp();
                tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kPairTile);
                for (int kb = 0; kb < total_kb; ++kb) {
                    if (!w.wait(abort_flag, err)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t ad = operand_desc<L::A_MN>(smem_u32(sA + w.stage * kOperand));
                    const uint64_t bd = operand_desc<L::B_MN>(smem_u32(sB + w.stage * kOperand));
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k)
                            umma_bf16_pair(d, ad + k * kDescStep<L::A_MN>, bd + k * kDescStep<L::B_MN>, idesc,
                                           (kb | k) != 0 ? 1u : 0u);
                        umma_commit_pair_multicast(&empty[w.stage], both);
                    }
                    __syncwarp();
                    w.advance();
                }
                if (!ok) break;
                if (elect_one()) umma_commit_pair_multicast(&tfull[acc], both);
                __syncwarp();
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (elect_one()) umma_commit_pair_multicast(drain, both);
            __syncwarp();
        }
    } else {
        // epilogue warp (q, half): TMEM lanes 32 q .., accumulator columns [0, 128) or [128, 256);
        // gated: 64 gate columns and the 64 up columns that belong to them
        const int q = warp & 3, half = (warp - 2) >> 2;
        uint8_t* stage_smem = smem + S * kStageBytes + (warp - 2) * kChunkBytes;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int tile = first; tile < tiles; tile += step) {
            const TilePlace w = place_tile(tile, mt, nt, N_TILE);
            WholeEpilogue<KIND, kPairTile> e{a, stage_smem, w.m0 + static_cast<int>(rank) * kBM, w.n0, q, half, lane, {}};
            e.fetch_ahead();
            const bool ok = warp != 2 || lane != 0 || idle_wait(&tfull[acc], acc_phase, abort_flag, progress, err);
            __syncwarp();
            if (!named_barrier_and(1, kEpiWarps * 32, ok)) break;  // given up: by all of them
            tc_fence_after();
            e.run(w.mat, tmem_base + static_cast<uint32_t>(acc * kPairTile), nullptr);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty_lead + 8u * acc);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    }

    __syncwarp();
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    // The pair's MMAs wrote this CTA's TMEM: they have ended.  Asked for here, when
    // every role of the CTA is through: from the start of a launch the odd CTA would
    // poll under every main loop and give a product of more than kWaitLimitNs up.
    if (threadIdx.x == 32) drain_wait(drain, 0, err);
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while another of the cluster may still signal it
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 2 * kPairTile);
    }
}

template <int KIND>
cudaError_t pair_prepare(int* clusters) {
    static std::atomic<unsigned long long> done{0};
    static int limit[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(dense_pair_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kPairSmem));
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kPairSmem;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, dense_pair_kernel<KIND>, &cfg);
        if (e != cudaSuccess) return e;
        limit[dev & 63] = n;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    *clusters = limit[dev & 63];
    return *clusters > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int KIND>
cudaError_t pair_go(const CUtensorMap* m, const DenseArgs& a, int clusters, cudaStream_t st) {
    int limit = 0;
    cudaError_t e = pair_prepare<KIND>(&limit);
    if (e != cudaSuccess) return e;
    if (clusters > limit) return cudaErrorInvalidConfiguration;
    return launch_kernel(dense_pair_kernel<KIND>, dim3(2 * clusters), dim3(kThreads), kPairSmem, st, m[0], m[1], m[2],
                         m[3], a);
}

}  // namespace

cudaError_t dense_pair_limit(DenseKind kind, int* clusters) {
    switch (kind) {
        case DENSE_GATED: return pair_prepare<DENSE_GATED>(clusters);
        case DENSE_LINEAR: return pair_prepare<DENSE_LINEAR>(clusters);
        case DENSE_DGRAD: return pair_prepare<DENSE_DGRAD>(clusters);
        default: return pair_prepare<DENSE_WGRAD>(clusters);
    }
}

cudaError_t launch_dense_pair(DenseKind kind, const CUtensorMap* m, const DenseArgs& a, int clusters, cudaStream_t st) {
    switch (kind) {
        case DENSE_GATED: return pair_go<DENSE_GATED>(m, a, clusters, st);
        case DENSE_LINEAR: return pair_go<DENSE_LINEAR>(m, a, clusters, st);
        case DENSE_DGRAD: return pair_go<DENSE_DGRAD>(m, a, clusters, st);
        default: return pair_go<DENSE_WGRAD>(m, a, clusters, st);
    }
}

}  // namespace moe
