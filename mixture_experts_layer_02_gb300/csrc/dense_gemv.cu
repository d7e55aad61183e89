// dense_gemv.cu -- the gated and linear products of a few tokens: a stream of
// weight rows.
//
// At a few rows of x the weights are read once and everything else is small, so
// the time is the weights' bytes over the HBM rate plus a fixed latency.  A
// 128-row tensor-core tile spends that latency on shared memory, barriers and
// clusters: gated 1 x 7168 x 2048 took 20.8 us there and takes 9.6 here (58.7 MB,
// 6.1 TB/s), linear 8 x 2048 x 7168 16.6 and 5.9.  From about 20 rows on the
// blocks' reads of x from L2 outweigh that (the plan in dense_api.cu compares
// them).  The weights go from global memory straight into registers as the 16-row
// operand of mma.sync.m16n8k16 and the tokens are its 8 columns:
//
//   - a block owns 16 weight rows (gated: 8 rows of W1 and the same 8 of W3, so
//     a thread holds the gate and the up sum of one output in one fragment) and
//     its 8 warps take 64-wide steps of K in turn;
//   - lane (g, t) = (lane / 4, lane % 4) loads the 16-byte pieces at columns
//     32 j + 8 t of rows g and g + 8: every load instruction covers whole
//     sectors, and any K that is a multiple of 8 will do.  Which K element sits
//     in which fragment slot does not matter as long as x is loaded the same
//     way, so no element is ever moved between lanes;
//   - the loads of four steps are issued before the first is used: two blocks
//     an SM keep about 128 KB in flight.
//
// The 8 warps' sums are added in warp order through shared memory and run
// through the epilogue, so results do not change from run to run.
#include <algorithm>

#include "dense_gemm.cuh"

namespace moe {

namespace {

constexpr int kGemvWarps = 8;
constexpr int kGemvRows = 16;
// steps of 64 K loaded ahead, by groups of eight tokens: what 128 registers hold
template <int NT>
constexpr int kGemvBatch = NT <= 2 ? 4 : 2;

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Read once: not kept in L1.  A coherent load, like those of x below: weights and x
// may be what the launch before this one writes while this grid is resident, and
// the non-coherent path is for data that nothing writes in a grid's lifetime.
__device__ __forceinline__ uint4 ld_once(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// NT: groups of eight tokens.
template <bool GATED, int NT>
__global__ void __launch_bounds__(kGemvWarps * 32, 2)
dense_gemv_kernel(const uint16_t* x, const uint16_t* w, const uint16_t* w3, const DenseArgs a) {
    __shared__ float sums[kGemvWarps][NT * 8][kGemvRows + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int K = a.K;
    // rows past the last are read as the last one and not stored
    const int n0 = blockIdx.x * (GATED ? 8 : kGemvRows);
    const uint16_t* lo = w + static_cast<long long>(min(n0 + g, a.N - 1)) * K;
    const uint16_t* hi = GATED ? w3 + static_cast<long long>(min(n0 + g, a.N - 1)) * K
                               : w + static_cast<long long>(min(n0 + g + 8, a.N - 1)) * K;
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    constexpr int BATCH = kGemvBatch<NT>;
    const int steps = (K + 63) >> 6;
    // The first steps' weights start their way into L2 while the kernel before
    // this one drains (L2 is coherent: if it writes them, the loads see that).
    if (t == 0)
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int k = (warp + b * kGemvWarps) * 64;
            if (k < K) {
                asm volatile("prefetch.global.L2 [%0];" ::"l"(lo + k));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(hi + k));
            }
        }
    // The next launch may start once every block is past its wait, never before: a
    // chain of such launches would otherwise be resident several deep, and a grid
    // that started before its inputs' last writer could find older copies in L1.
    pdl_wait();
    pdl_trigger();

    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int s0 = warp; s0 < steps; s0 += kGemvWarps * BATCH) {
        uint4 wl[BATCH][2], wh[BATCH][2], xv[BATCH][NT][2];
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = (s0 + b * kGemvWarps) * 64 + j * 32 + t * 8;
                const bool in = k < K;
                wl[b][j] = in ? ld_once(lo + k) : zero;
                wh[b][j] = in ? ld_once(hi + k) : zero;
            }
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int k = (s0 + b * kGemvWarps) * 64 + j * 32 + t * 8, tok = i * 8 + g;
                    xv[b][i][j] = k < K && tok < a.M
                                      ? *reinterpret_cast<const uint4*>(x + static_cast<long long>(tok) * K + k)
                                      : zero;
                }
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    mma_16x8x16(acc[i], wl[b][j].x, wh[b][j].x, wl[b][j].y, wh[b][j].y, xv[b][i][j].x, xv[b][i][j].y);
                    mma_16x8x16(acc[i], wl[b][j].z, wh[b][j].z, wl[b][j].w, wh[b][j].w, xv[b][i][j].z, xv[b][i][j].w);
                }
    }
    // acc[i]: rows g (0, 1) and g + 8 (2, 3), tokens 8 i + 2 t and the next
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[warp][i * 8 + 2 * t + (j & 1)][g + (j >> 1) * 8] = acc[i][j];
    __syncthreads();

    constexpr int COLS = GATED ? 8 : kGemvRows;
    for (int it = threadIdx.x; it < NT * 8 * COLS; it += kGemvWarps * 32) {
        const int tok = it / COLS, c = it - tok * COLS, col = n0 + c;
        if (tok >= a.M || col >= a.N) continue;
        const long long at = static_cast<long long>(tok) * a.N + col;
        float z = 0.0f, u = 0.0f;
#pragma unroll
        for (int v = 0; v < kGemvWarps; ++v) {
            z += sums[v][tok][c];
            if (GATED) u += sums[v][tok][c + 8];
        }
        auto put = [&](uint16_t* p, float f) { p[at] = static_cast<uint16_t>(pack_bf16x2(f, 0.0f)); };
        if constexpr (GATED) {
            if (a.out1) put(a.out1, z);
            if (a.out2) put(a.out2, u);
            float v[1] = {z};
            act_values(a.fn, v);
            put(a.out0, v[0] * u);
        } else {
            if (a.bias) z += a.bias[col];
            if (a.out1) put(a.out1, z);
            float v[1] = {z};
            act_values(a.fn, v);
            z = v[0];
            if (a.residual) z += __uint_as_float(static_cast<uint32_t>(a.residual[at]) << 16);
            put(a.out0, z);
        }
    }
}

template <bool GATED, int NT>
cudaError_t gemv_go(const DenseOperands& o, const DenseArgs& a, cudaStream_t st) {
    const int rows = GATED ? 8 : kGemvRows;
    return launch_kernel(dense_gemv_kernel<GATED, NT>, dim3((a.N + rows - 1) / rows), dim3(kGemvWarps * 32), 0, st, o.a0,
                         o.b0, o.b1, a);
}

}  // namespace

cudaError_t launch_dense_gemv(DenseKind kind, const DenseOperands& o, const DenseArgs& a, cudaStream_t st) {
    const int nt = (a.M + 7) / 8;
    if (kind == DENSE_GATED)
        return nt <= 1 ? gemv_go<true, 1>(o, a, st) : (nt <= 2 ? gemv_go<true, 2>(o, a, st) : gemv_go<true, 4>(o, a, st));
    return nt <= 1 ? gemv_go<false, 1>(o, a, st) : (nt <= 2 ? gemv_go<false, 2>(o, a, st) : gemv_go<false, 4>(o, a, st));
}

}  // namespace moe
