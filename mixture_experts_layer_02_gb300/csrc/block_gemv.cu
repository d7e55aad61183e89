// block_gemv.cu -- the experts' product in e4m3 with a scale for each block of 128 for
// a few rows: a stream of weight rows (BLOCK_FWD of block_gemm.h).
//
// With a handful of rows an expert the weights are read once and everything else is
// small: the time is their bytes over the HBM rate plus a fixed latency, which 128-row
// tiles spend on shared memory, barriers and clusters.  The weights go from global
// memory straight into registers as the 16-row operand of mma.sync, an
// expert's rows are its 8 columns, eight at a time:
//
//   - KW of a block's 8 warps share 16 weight rows, each a run of the blocks along K;
//   - lane (g, t) = (lane / 4, lane % 4) loads the 16-byte pieces at 16 t and 64 + 16 t
//     of a block of rows g and g + 8: whole sectors, and any K that is a multiple of 16.
//     Which K element sits in which fragment slot does not matter as long as x is
//     loaded the same way;
//   - codes become f16 (exactly) on the way into mma.sync.m16n8k16, eight of which sum a
//     block's 128 products from zero; the partial sum is scaled and added in fp32, as in
//     the tiles.  The e4m3 form of mma.sync is taken apart into the same and converts x
//     again for each (2048 x 768, 128 experts, 64 rows: 24.6 us, 22.5 so);
//   - the loads of kBatch blocks are issued before the first is used.
//
// The KW warps' sums are added in warp order through shared memory.  Measured: one row of
// 7168 x 2048 7.9 us a call in a run (14.7 MB: 2.2 us of HBM; the call from Python takes
// 7.7); 64 rows of 128 experts, 2048 x 768, 20 us (78.8 MB: 11.7 us).  What remains there is
// latency: finding the expert, then eight batches of two blocks a warp; asking L2 for a
// warp's rows ahead or more warps with fewer registers were slower (24 to 31 us).
#include <algorithm>

#include "activation.cuh"
#include "block_gemm.h"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBatch = 2;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes as f16 (exact): the first two in lo, the others in hi.
__device__ __forceinline__ void to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}

// c += the products of four K codes of weight rows g and g + 8 and of this lane's row of x
__device__ __forceinline__ void mma_word(float (&c)[4], uint32_t wl, uint32_t wh, uint32_t xw) {
    uint32_t a0, a1, a2, a3, b0, b1;
    to_f16(wl, a0, a2);
    to_f16(wh, a1, a3);
    to_f16(xw, b0, b1);
    mma_f16(c, a0, a1, a2, a3, b0, b1);
}

// Read once: not kept in L1.  Coherent, as the launch before may still be writing.
__device__ __forceinline__ uint4 ld_once(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Block (i, j): weight rows 16 (8 / KW) i .. of the j-th expert that has rows.
template <int KW>
__global__ void __launch_bounds__(kThreads, 2)
block_gemv_kernel(const uint8_t* x, const uint8_t* w, const BlockArgs a) {
    constexpr int UNITS = kWarps / KW;
    __shared__ float sums[kWarps][8][17];
    __shared__ int s_warp[kWarps];
    __shared__ int s_expert[3];  // the expert, its first row, its rows (0: none)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    if (threadIdx.x == 0) s_expert[2] = 0;
    pdl_wait();
    pdl_trigger();  // two launches overlap at most: this one has waited for the one before
    if (a.offsets == nullptr) {
        if (threadIdx.x == 0) s_expert[0] = s_expert[1] = 0, s_expert[2] = a.rows;
        __syncthreads();
    } else {
        constexpr int PER = 1024 / kThreads;  // consecutive experts a thread
        const int e0 = threadIdx.x * PER;
        int at[PER + 1];
#pragma unroll
        for (int i = 0; i <= PER; ++i) at[i] = e0 + i <= a.E ? a.offsets[e0 + i] : 0;
        int n = 0;
        bool bad = threadIdx.x == 0 && at[0] != 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (e0 + i >= a.E) continue;
            bad |= at[i] > at[i + 1] || (e0 + i + 1 == a.E && at[i + 1] > a.rows);
            n += at[i + 1] > at[i];
        }
        int v = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += up;
        }
        if (lane == 31) s_warp[warp] = v;
        if (__syncthreads_or(bad)) {
            if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) record_error(a.err, MOE_DEVERR_BOUNDS);
            return;
        }
        int before = v - n;
        for (int i = 0; i < warp; ++i) before += s_warp[i];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (e0 + i >= a.E || at[i + 1] <= at[i]) continue;
            if (before++ == static_cast<int>(blockIdx.y)) s_expert[0] = e0 + i, s_expert[1] = at[i], s_expert[2] = at[i + 1] - at[i];
        }
        __syncthreads();
    }
    const int e = s_expert[0], row0 = s_expert[1], rows = s_expert[2];
    const int K = a.K, kbs = (K + kBlock - 1) / kBlock;
    const int part = warp % KW, f0 = (blockIdx.x * UNITS + warp / KW) * 16;
    // rows past the last are read as the last one and not stored
    const uint8_t* lo = w + (static_cast<long long>(e) * a.N + min(f0 + g, a.N - 1)) * K;
    const uint8_t* hi = w + (static_cast<long long>(e) * a.N + min(f0 + g + 8, a.N - 1)) * K;
    const int nb = (a.N + kBlock - 1) / kBlock;
    const float* sb = a.b_scale + (static_cast<long long>(e) * nb + min(f0, a.N - 1) / kBlock) * kbs;
    const int k0 = kbs * part / KW, k1 = f0 < a.N ? kbs * (part + 1) / KW : 0;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int r0 = 0; r0 < rows; r0 += 8) {
        const uint8_t* xr = r0 + g < rows ? x + static_cast<long long>(row0 + r0 + g) * K : nullptr;
        int index[2];  // rows of a_scale of this lane's two output columns
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = r0 + 2 * t + j;
            index[j] = r >= rows ? -1 : (a.a_index ? a.a_index[row0 + r] : row0 + r);
        }
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int kb = k0; kb < k1; kb += kBatch) {
            uint4 wl[kBatch][2], wh[kBatch][2], xv[kBatch][2];
            float s[kBatch][2];
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int k = (kb + b) * kBlock + j * 64 + t * 16;
                    const bool in = kb + b < k1 && k < K;
                    wl[b][j] = in ? ld_once(lo + k) : zero;
                    wh[b][j] = in ? ld_once(hi + k) : zero;
                    xv[b][j] = in && xr ? *reinterpret_cast<const uint4*>(xr + k) : zero;
                }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const float scale = kb + b < k1 ? sb[kb + b] : 0.0f;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const bool on = kb + b < k1 && index[j] >= 0 && index[j] < a.a_scale_rows;
                    s[b][j] = on ? scale * a.a_scale[static_cast<long long>(index[j]) * kbs + kb + b] : 0.0f;
                }
            }
            float p[kBatch][4] = {};  // the blocks' MMAs in turn: a block's eight wait for one another
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int b = 0; b < kBatch; ++b) mma_word(p[b], wl[b][j].x, wh[b][j].x, xv[b][j].x);
#pragma unroll
                for (int b = 0; b < kBatch; ++b) mma_word(p[b], wl[b][j].y, wh[b][j].y, xv[b][j].y);
#pragma unroll
                for (int b = 0; b < kBatch; ++b) mma_word(p[b], wl[b][j].z, wh[b][j].z, xv[b][j].z);
#pragma unroll
                for (int b = 0; b < kBatch; ++b) mma_word(p[b], wl[b][j].w, wh[b][j].w, xv[b][j].w);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = fmaf(s[b][i & 1], p[b][i], acc[i]);  // rows g, g + 8; columns 2 t, 2 t + 1
        }
        if (part == 0 && g == 0)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (r0 + 2 * t + j < rows && (index[j] < 0 || index[j] >= a.a_scale_rows)) record_error(a.err, MOE_DEVERR_BOUNDS);
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[warp][2 * t + (i & 1)][g + (i >> 1) * 8] = acc[i];
        __syncthreads();
        // eight rows x 16 UNITS columns, pairs of columns a thread
        for (int it = threadIdx.x; it < 8 * 8 * UNITS; it += kThreads) {
            const int r = it / (8 * UNITS), c = (it - r * 8 * UNITS) * 2, u = c >> 4;
            const int col = blockIdx.x * UNITS * 16 + c;
            if (r0 + r >= rows || col >= a.N) continue;
            float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
            for (int i = 0; i < KW; ++i) {
                v0 += sums[u * KW + i][r][c & 15];
                v1 += sums[u * KW + i][r][(c & 15) + 1];
            }
            *reinterpret_cast<uint32_t*>(a.out + static_cast<long long>(row0 + r0 + r) * a.N + col) = pack_bf16x2(v0, v1);
        }
        __syncthreads();
    }
}

template <int KW>
cudaError_t gemv_go(const uint8_t* x, const uint8_t* w, const BlockArgs& a, cudaStream_t st) {
    const int width = 16 * (kWarps / KW);
    const int experts = a.offsets ? std::min(a.E, a.rows) : 1;
    return launch_kernel(block_gemv_kernel<KW>, dim3((a.N + width - 1) / width, experts), dim3(kThreads), 0, st, x, w, a);
}

}  // namespace

cudaError_t launch_block_gemv(const uint8_t* x, const uint8_t* w, const BlockArgs& a, int warps, cudaStream_t st) {
    switch (warps) {
        case 1: return gemv_go<1>(x, w, a, st);
        case 2: return gemv_go<2>(x, w, a, st);
        case 4: return gemv_go<4>(x, w, a, st);
        default: return gemv_go<8>(x, w, a, st);
    }
}

}  // namespace moe
