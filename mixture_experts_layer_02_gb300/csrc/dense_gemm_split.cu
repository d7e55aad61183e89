// dense_gemm_split.cu -- the dense products on one-CTA 128 x 128 tiles with the
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
// Warp roles: 0 TMA producer, 1 TMEM allocator and MMA issuer, 4..7 park the
// accumulator (warp q reads TMEM lanes 32 q ..), all eight warps the join and
// epilogue.  Three 32 KB stages, so that two CTAs fit an SM: a short k-range
// then overlaps its neighbour's prologue and epilogue.
//
// Every wait is bounded (mbar_wait); whatever a role sees, every thread reaches
// both cluster barriers, so no CTA waits for one that left.
#include <algorithm>
#include <atomic>

#include "dense_gemm.cuh"

namespace moe {

namespace {

constexpr int kSplitBN = 128;
constexpr int kSplitStages = 3;
constexpr int kSplitThreads = 256;
constexpr int kOperandBytes = kBM * kRowBytes;  // 16 KB: 128 rows x 64 K, or two MN-major boxes
constexpr int kSplitStageBytes = 2 * kOperandBytes;
constexpr int kParkLd = kSplitBN + 4;           // floats: 16-byte rows, quarter-warps on distinct banks
constexpr size_t kSplitSmem = 1024 + kSplitStages * kSplitStageBytes + 128;
static_assert(kBM * kParkLd * 4 <= kSplitStages * kSplitStageBytes, "the parked accumulator reuses the stages");

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t cluster_nctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// Eight consecutive floats of a parked accumulator, summed over the cluster in rank order.
__device__ __forceinline__ void joined_octet(uint32_t offset, uint32_t splits, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    for (uint32_t s = 0; s < splits; ++s) {
        const uint32_t p = mapa_shared(offset, s);
        const float4 a = ld_cluster_v4(p), b = ld_cluster_v4(p + 16);
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
}

template <int KIND>
__global__ void __launch_bounds__(kSplitThreads)
dense_split_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                   const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                   const DenseArgs a) {
    using L = DenseLayout<KIND>;
    constexpr int S = kSplitStages;
    constexpr int N_TILE = L::GATED ? kSplitBN / 2 : kSplitBN;  // output columns of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    float* park = reinterpret_cast<float*>(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * kSplitStageBytes);
    uint64_t* empty = full + S;
    uint64_t* done = empty + S;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank(), splits = cluster_nctarank();

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
    int tile = blockIdx.x / splits;
    const int mat = tile / (mt * nt);
    tile -= mat * mt * nt;
    const int m0 = (tile % mt) * kBM, n0 = (tile / mt) * N_TILE;
    const int kbs = (a.K + kBK - 1) / kBK;  // k-blocks of one segment
    const int total = kbs * a.segs;
    const int k_lo = static_cast<int>(static_cast<long long>(total) * rank / splits);
    const int k_hi = static_cast<int>(static_cast<long long>(total) * (rank + 1) / splits);
    pdl_wait();

    if (warp == 0) {
        if (lane == 0) {
            bool withhold = a.dbg && (*a.dbg & MOE_DBG_WITHHOLD_FIRST_LOAD) && blockIdx.x == 0;
            uint32_t pending = 0, pend_parity = 0;
            int stage = 0;
            uint32_t phase = 0;
            for (int kb = k_lo; kb < k_hi; ++kb) {
                if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, a.err)) break;
                if (withhold) {
                    withhold = false;  // test hook: this stage never fills
                } else {
                    const int seg = kb / kbs, k0 = (kb - seg * kbs) * kBK;
                    uint8_t* sA = smem + stage * kSplitStageBytes;
                    uint8_t* sB = sA + kOperandBytes;
                    const CUtensorMap* mA = (seg | mat) ? &tmA1 : &tmA0;
                    mbar_arrive_expect_tx(&full[stage], kSplitStageBytes);
                    pending |= 1u << stage;
                    pend_parity = (pend_parity & ~(1u << stage)) | (phase << stage);
                    if constexpr (L::A_MN) {
                        tma_load_2d(mA, &full[stage], sA, m0, k0);
                        tma_load_2d(mA, &full[stage], sA + kMnBlockBytes, m0 + 64, k0);
                    } else {
                        tma_load_2d(mA, &full[stage], sA, k0, m0);
                    }
                    if constexpr (L::GATED) {
                        tma_load_2d(&tmB0, &full[stage], sB, k0, n0);
                        tma_load_2d(&tmB1, &full[stage], sB + kOperandBytes / 2, k0, n0);
                    } else if constexpr (L::B_MN) {
                        const CUtensorMap* mB = seg ? &tmB1 : &tmB0;
                        tma_load_2d(mB, &full[stage], sB, n0, k0);
                        tma_load_2d(mB, &full[stage], sB + kMnBlockBytes, n0 + 64, k0);
                    } else {
                        tma_load_2d(&tmB0, &full[stage], sB, k0, n0);
                    }
                }
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
            for (int s = 0; s < S; ++s)
                if (pending & (1u << s)) drain_wait(&full[s], (pend_parity >> s) & 1u, a.err);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = dense_idesc<KIND>(kBM, kSplitBN);
            int stage = 0;
            uint32_t phase = 0;
            for (int kb = k_lo; kb < k_hi; ++kb) {
                if (!mbar_wait(&full[stage], phase, abort_flag, a.err)) break;
                tc_fence_after();
                const uint32_t sA = smem_u32(smem + stage * kSplitStageBytes);
                const uint64_t ad = operand_desc<L::A_MN>(sA), bd = operand_desc<L::B_MN>(sA + kOperandBytes);
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k)
                    umma_bf16(tmem, ad + k * kDescStep<L::A_MN>, bd + k * kDescStep<L::B_MN>, idesc,
                              (kb != k_lo || k != 0) ? 1u : 0u);
                umma_commit(&empty[stage]);
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
            umma_commit(done);
            drain_wait(done, 0, a.err);  // TMEM is released below: nothing may be in flight
        }
    } else if (warp >= 4) {
        bool ok = mbar_wait(done, 0, abort_flag, a.err);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        if (ok) {
            const int q = warp & 3;
            float* row = park + (q * 32 + lane) * kParkLd;
            const uint32_t t = tmem + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
            for (int c = 0; c < kSplitBN; c += 32) {
                uint32_t r[32];
                tmem_ld_32x32(t + c, r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<uint4*>(row + c + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
            }
        }
    }
    __syncwarp();
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kSplitBN);
    }
    cluster_sync_all();  // every CTA's accumulator is parked

    constexpr int OCTETS = N_TILE / 8;
    constexpr int ITEMS = kBM * OCTETS;
    const int it_lo = ITEMS * static_cast<int>(rank) / static_cast<int>(splits);
    const int it_hi = ITEMS * static_cast<int>(rank + 1) / static_cast<int>(splits);
    const uint32_t park0 = smem_u32(park);
    for (int it = it_lo + threadIdx.x; it < it_hi; it += kSplitThreads) {
        const int r = it / OCTETS, c = (it - r * OCTETS) * 8;
        if (m0 + r >= a.M || n0 + c >= a.N) continue;
        const uint32_t at = park0 + static_cast<uint32_t>(r * kParkLd + c) * 4u;
        float v[8];
        joined_octet(at, splits, v);
        if constexpr (L::GATED) {
            float u[8];
            joined_octet(at + 4u * N_TILE, splits, u);
            gated_octet(a, m0 + r, n0 + c, v, u);
        } else if constexpr (KIND == DENSE_LINEAR) {
            linear_octet(a, m0 + r, n0 + c, v);
        } else {
            *octet(mat ? a.out1 : a.out0, m0 + r, a.N, n0 + c) = pack_bf16x8(v);
        }
    }
    cluster_sync_all();  // no CTA leaves while another reads its shared memory
}

template <int KIND>
cudaError_t split_prepare() {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(dense_split_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSplitSmem));
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

template <int KIND>
cudaError_t split_go(const CUtensorMap* m, const DenseArgs& a, int splits, cudaStream_t st) {
    cudaError_t e = split_prepare<KIND>();
    if (e != cudaSuccess) return e;
    constexpr int n_tile = DenseLayout<KIND>::GATED ? kSplitBN / 2 : kSplitBN;
    const long long tiles = static_cast<long long>((a.M + kBM - 1) / kBM) * ((a.N + n_tile - 1) / n_tile) * a.mats;
    if (tiles * splits > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits));
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = kSplitSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, dense_split_kernel<KIND>, m[0], m[1], m[2], m[3], a);
}

}  // namespace

cudaError_t launch_dense_split(DenseKind kind, const CUtensorMap* m, const DenseArgs& a, int splits, cudaStream_t st) {
    switch (kind) {
        case DENSE_GATED: return split_go<DENSE_GATED>(m, a, splits, st);
        case DENSE_LINEAR: return split_go<DENSE_LINEAR>(m, a, splits, st);
        case DENSE_DGRAD: return split_go<DENSE_DGRAD>(m, a, splits, st);
        default: return split_go<DENSE_WGRAD>(m, a, splits, st);
    }
}

}  // namespace moe
