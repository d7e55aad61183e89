// quant_block.cu -- e4m3 codes with one power-of-two scale for each block of 128:
//   rows      1 x 128 of an activation: the operand of a product over that dimension
//   tiles     128 x 128 of a weight
//   segments  1 x 128 and 128 x 1 of an activation from one read of it; the second
//             form runs down the rows of one expert at a time, whose segments then
//             start at multiples of 128 with zero rows behind them: the operands of
//             the weight gradient, which sums over an expert's rows
// The rule is the row quantiser's (quant.cu): scale = 2^k, k the smallest integer
// >= -126 with max|block| <= 448 2^k; x 2^-k is exact, so the e4m3 rounding is the
// only one.  A block's values stay in registers between the maximum and the codes:
// each is read once.  Coherent loads only: the launch before may still be writing the
// source when blocks start.
//
// Measured: rows 1001 x 7168 6.8 us (21.7 MB: 3.2 us of HBM, the rest start and tail of one
// wave); segments of 8186 x 4096 28.5 us (136 MB: 20 us), 23 without writing the second
// form: conversions, maxima and shuffles fill about half of the issue slots at 16 warps an
// SM.  The next piece's loads stand in registers meanwhile (without: 40 us, as with three
// blocks an SM, whose registers spill); one wave of blocks, as a block's way to its rows
// costs as much as a piece (35 us with a block for each).
#include <algorithm>

#include "quant.cuh"
#include "train.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

int sms() {
    int dev = 0, n = 152;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

__device__ __forceinline__ float scale_of(int k) { return __uint_as_float(static_cast<uint32_t>(127 + k) << 23); }
__device__ __forceinline__ float inverse_of(int k) { return __uint_as_float(static_cast<uint32_t>(127 - k) << 23); }

// Sixteen lanes a block of 128 values, HPR such groups a row, each with U blocks of it in
// flight; a thread block's 16 groups take 16 / HPR rows at a time.
template <int HPR>
__global__ void __launch_bounds__(kThreads)
quant_rows_block_kernel(const uint16_t* src, long long rows, int cols, int nb, uint8_t* q, float* scale) {
    constexpr int U = 4, RPB = kThreads / 16 / HPR;
    pdl_wait();
    const int sub = threadIdx.x & 15, group = threadIdx.x >> 4;
    for (long long r0 = static_cast<long long>(blockIdx.x) * RPB; r0 < rows; r0 += static_cast<long long>(gridDim.x) * RPB) {
        const long long r = r0 + group / HPR;
        const bool row = r < rows;
        // every lane of a warp takes the same number of turns (the shuffles are the whole warp's)
        for (int b0 = 0; b0 < nb; b0 += U * HPR) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int col = (b0 + u * HPR + group % HPR) * kBlock + sub * 8;
                v[u] = row && col < cols ? *reinterpret_cast<const uint4*>(src + r * cols + col) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                uint32_t m = absmax8(v[u]);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                const int b = b0 + u * HPR + group % HPR, col = b * kBlock + sub * 8;
                if (!row || b >= nb) continue;
                const int k = scale_exp_of(m);
                if (sub == 0) scale[r * nb + b] = scale_of(k);
                if (col < cols) *reinterpret_cast<uint2*>(q + r * cols + col) = to_e4m3x8(v[u], inverse_of(k));
            }
        }
    }
    pdl_trigger();
}

// One 128 x 128 block a turn: thread (y, x) of 16 x 16 holds rows y, y + 16, ... of an octet of columns.
__global__ void __launch_bounds__(kThreads)
quant_tiles_kernel(const uint16_t* src, long long tiles, int rows, int cols, int rb, int nb, uint8_t* q, float* scale) {
    __shared__ uint32_t s_max[2][kThreads / 32];
    pdl_wait();
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
    int turn = 0;
    for (long long i = blockIdx.x; i < tiles; i += gridDim.x, turn ^= 1) {
        const long long mr = i / nb, mat = mr / rb;
        const int row0 = static_cast<int>(mr - mat * rb) * kBlock;
        const int col = static_cast<int>(i - mr * nb) * kBlock + x * 8;
        const long long at = (mat * rows + row0 + y) * cols + col;
        uint4 v[8];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = row0 + y + 16 * j < rows && col < cols;
            v[j] = in ? *reinterpret_cast<const uint4*>(src + at + static_cast<long long>(16 * j) * cols) : make_uint4(0, 0, 0, 0);
            m = max(m, absmax8(v[j]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((threadIdx.x & 31) == 0) s_max[turn][threadIdx.x >> 5] = m;
        __syncthreads();  // the other half of s_max is rewritten a turn later, behind the next one
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = max(m, s_max[turn][w]);
        const int k = scale_exp_of(m);
        if (threadIdx.x == 0) scale[i] = scale_of(k);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (row0 + y + 16 * j < rows && col < cols)
                *reinterpret_cast<uint2*>(q + at + static_cast<long long>(16 * j) * cols) = to_e4m3x8(v[j], inverse_of(k));
    }
    pdl_trigger();
}

// A block takes 128 rows of one segment and every gridDim.y-th block of 128 columns.
__global__ void __launch_bounds__(kThreads, 2)
quant_segments_kernel(const QuantSegArgs a) {
    __shared__ __align__(16) uint32_t s_col[2][8][kBlock / 2];  // maxima of column pairs, by warp
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // which expert's rows start at padded block blockIdx.x: every warp finds it for itself, by a
    // running sum of the segments' blocks (barriers would cost more)
    int carry = 0, first = -1, n = -1;  // first row, rows; n < 0: nothing here
    bool bad = false;
#pragma unroll 4
    for (int e0 = 0; e0 < a.E; e0 += 32) {  // unrolled: the offsets' loads do not wait for one another
        const int e = e0 + lane;
        int lo = 0, len = 0;
        if (e < a.E) {
            lo = a.offsets ? a.offsets[e] : 0;
            const int hi = a.offsets ? a.offsets[e + 1] : a.rows;
            len = hi - lo;
            bad |= lo < 0 || hi < lo || hi > a.rows || (e == 0 && lo != 0);
        }
        const int mine = len > 0 ? (len + kBlock - 1) / kBlock : 0;
        int v = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += up;
        }
        const int b = static_cast<int>(blockIdx.x) - (carry + v - mine);
        const unsigned here = __ballot_sync(0xffffffffu, b >= 0 && b < mine);
        if (here) {
            const int from = __ffs(here) - 1;
            first = __shfl_sync(0xffffffffu, lo + b * kBlock, from);
            n = __shfl_sync(0xffffffffu, min(kBlock, len - b * kBlock), from);
        }
        carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (__any_sync(0xffffffffu, bad)) {  // offsets that are not a prefix sum within the rows: nothing is written
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) record_error(a.err, MOE_DEVERR_BOUNDS);
        return;
    }
    if (n < 0) return;  // behind the last segment
    const long long row0 = first, pad0 = static_cast<long long>(blockIdx.x) * kBlock;
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
    const int nb = (a.cols + kBlock - 1) / kBlock;
    uint4 next[8];
    auto fetch = [&](int cb) {  // rows y, y + 16, ... of an octet of columns
        const int col = cb * kBlock + x * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = y + 16 * j;
            next[j] = r < n && col < a.cols ? *reinterpret_cast<const uint4*>(a.src + (row0 + r) * a.cols + col) : make_uint4(0, 0, 0, 0);
        }
    };
    fetch(blockIdx.y);
    int turn = 0;
    for (int cb = blockIdx.y; cb < nb; cb += gridDim.y, turn ^= 1) {
        const int col = cb * kBlock + x * 8;
        const bool inside = col < a.cols;
        uint4 v[8];
        uint32_t c[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = next[j];
        fetch(cb + gridDim.y);  // past the last column: nothing is read
        // magnitudes, two to a register: the columns' maxima, and two rows' at a time
        uint32_t rowmax[4];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            uint32_t pm[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t m[4] = {v[j + i].x & 0x7fff7fffu, v[j + i].y & 0x7fff7fffu, v[j + i].z & 0x7fff7fffu, v[j + i].w & 0x7fff7fffu};
#pragma unroll
                for (int w = 0; w < 4; ++w) c[w] = __vmaxu2(c[w], m[w]);
                pm[i] = __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3]));
            }
            rowmax[j / 2] = __vmaxu2(__byte_perm(pm[0], pm[1], 0x5410), __byte_perm(pm[0], pm[1], 0x7632));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = __vmaxu2(c[i], __shfl_xor_sync(0xffffffffu, c[i], 16));
        if (lane < 16) *reinterpret_cast<uint4*>(&s_col[turn][warp][lane * 4]) = make_uint4(c[0], c[1], c[2], c[3]);
        if (a.q) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) rowmax[i] = __vmaxu2(rowmax[i], __shfl_xor_sync(0xffffffffu, rowmax[i], o));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = y + 16 * j, k = scale_exp_of((rowmax[j / 2] >> (16 * (j & 1))) & 0xffffu);
                if (r >= n) continue;
                if (x == 0) a.scale[(row0 + r) * nb + cb] = scale_of(k);
                if (inside) *reinterpret_cast<uint2*>(a.q + (row0 + r) * a.cols + col) = to_e4m3x8(v[j], inverse_of(k));
            }
        }
        __syncthreads();  // the other half of s_col is rewritten a turn later, behind the next one
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const uint4 m = *reinterpret_cast<const uint4*>(&s_col[turn][w][x * 4]);
            c[0] = __vmaxu2(c[0], m.x), c[1] = __vmaxu2(c[1], m.y), c[2] = __vmaxu2(c[2], m.z), c[3] = __vmaxu2(c[3], m.w);
        }
        if (!inside) continue;
        float s[8], back[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = scale_exp_of((c[i >> 1] >> (16 * (i & 1))) & 0xffffu);
            s[i] = scale_of(k);
            back[i] = inverse_of(k);
        }
        if (y == 0) {
            float4* p = reinterpret_cast<float4*>(a.scale_seg + pad0 / kBlock * a.cols + col);
            p[0] = make_float4(s[0], s[1], s[2], s[3]);
            p[1] = make_float4(s[4], s[5], s[6], s[7]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // rows behind the segment's last are zeros
            const uint32_t w4[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = fp8x2(bf16_lo(w4[i]) * back[2 * i], bf16_hi(w4[i]) * back[2 * i + 1]);
            *reinterpret_cast<uint2*>(a.q_seg + (pad0 + y + 16 * j) * a.cols + col) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
        }
    }
    pdl_trigger();
}

}  // namespace

cudaError_t launch_quant_rows_block(const uint16_t* src, long long rows, int cols, uint8_t* q, float* scale,
                                    cudaStream_t st) {
    const int nb = static_cast<int>(blocks_of(cols));
    auto go = [&](auto kernel, int hpr) {
        const int rpb = kThreads / 16 / hpr;
        const int grid = static_cast<int>(std::min<long long>((rows + rpb - 1) / rpb, static_cast<long long>(sms()) * 8));
        return launch_kernel(kernel, dim3(grid), dim3(kThreads), 0, st, src, rows, cols, nb, q, scale);
    };
    if (nb <= 4) return go(quant_rows_block_kernel<1>, 1);
    if (nb <= 16) return go(quant_rows_block_kernel<4>, 4);
    return go(quant_rows_block_kernel<16>, 16);
}

cudaError_t launch_quant_tiles(const uint16_t* src, long long mats, int rows, int cols, uint8_t* q, float* scale,
                               cudaStream_t st) {
    const int rb = static_cast<int>(blocks_of(rows)), nb = static_cast<int>(blocks_of(cols));
    const long long tiles = mats * rb * nb;
    const int grid = static_cast<int>(std::min<long long>(tiles, static_cast<long long>(sms()) * 6));
    return launch_kernel(quant_tiles_kernel, dim3(grid), dim3(kThreads), 0, st, src, tiles, rows, cols, rb, nb, q, scale);
}

cudaError_t launch_quant_segments(const QuantSegArgs& a, cudaStream_t st) {
    const int blocks = static_cast<int>(segment_rows_of(a.rows, a.E) / kBlock);
    const int nb = static_cast<int>(blocks_of(a.cols));
    // one wave: a block's way to its rows costs as much as a 128 x 128 piece of them
    const int slices = std::max(1, std::min(nb, sms() * 2 / std::max(1, blocks)));
    return launch_kernel(quant_segments_kernel, dim3(blocks, slices), dim3(kThreads), 0, st, a);
}

}  // namespace moe
