// rmsnorm.cu -- root-mean-square norm with the residual's addition and an e4m3
// output, and its gradient.
//
//   s = x + residual          (fp32; stored in bf16 as the new residual stream)
//   y_j = s_j w_j / sqrt(mean_j s_j^2 + eps)
//   q = e4m3(y 2^-k), scale = 2^k, k = the smallest integer >= -126 with
//       max|y| <= 448 2^k (the row rule of quant.cu, applied to the fp32 y, so
//       a code has been rounded once)
//
// Every row is read once and held in registers between its sums and its
// outputs.  The sum of squares and the row's maximum come out of ONE reduction:
// y_j is formed as fl(fl(s_j w_j) r) with r > 0 and rounding is monotone, so
// max|y| = fl(max|fl(s_j w_j)| r) exactly.
#include <algorithm>

#include "activation.cuh"
#include "dense.h"
#include "quant.cuh"

namespace moe {

// k from the fp32 bits of the row maximum (as scale_exp_of for bf16):
// 448 = 1.75 * 2^8, fraction field of 1.75 = 0x600000.
__device__ __forceinline__ int scale_exp_of_f32(uint32_t m) {
    const int ef = static_cast<int>(m >> 23);
    return (ef == 0) ? -126 : max(-126, ef - 127 - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0));
}

// Sum of `a` and maximum of `m` (bits of non-negative floats; a NaN is larger
// than any number) over the T threads of a row.  T = 32: one warp.
template <int T>
__device__ __forceinline__ void row_reduce(float& a, uint32_t& m, float* s_a, uint32_t* s_m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if constexpr (T > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) {
            s_a[warp] = a;
            s_m[warp] = m;
        }
        __syncthreads();
        a = 0.0f;
        m = 0;
#pragma unroll
        for (int w = 0; w < T / 32; ++w) {
            a += s_a[w];
            m = max(m, s_m[w]);
        }
        __syncthreads();  // the arrays are rewritten for the next row
    }
}

// T threads a row (32: eight rows in a block of 256), V 16-byte chunks a thread.
template <int T, int V>
__global__ void __launch_bounds__(T < 256 ? 256 : T)
rmsnorm_kernel(const NormArgs a) {
    __shared__ float s_a[T / 32];
    __shared__ uint32_t s_m[T / 32];
    constexpr int ROWS = T == 32 ? 8 : 1;
    const int lane = T == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int chunks = a.D >> 3;
    pdl_wait();
    const uint4* wrow = reinterpret_cast<const uint4*>(a.weight);
    const float inv_d = 1.0f / static_cast<float>(a.D);
    for (long long r = static_cast<long long>(blockIdx.x) * ROWS + (T == 32 ? threadIdx.x >> 5 : 0); r < a.rows;
         r += static_cast<long long>(gridDim.x) * ROWS) {
        const long long at = r * chunks;
        const uint4* xr = reinterpret_cast<const uint4*>(a.x) + at;
        const uint4* rr = reinterpret_cast<const uint4*>(a.residual) + at;
        uint4 xv[V], rv[V], wv[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = lane + i * T;
            const bool in = c < chunks;
            xv[i] = in ? xr[c] : make_uint4(0, 0, 0, 0);
            rv[i] = in && a.residual ? rr[c] : make_uint4(0, 0, 0, 0);
            wv[i] = in ? __ldg(wrow + c) : make_uint4(0, 0, 0, 0);
        }
        float sw[V][8];
        float sum = 0.0f;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float s[8], b[8], w[8];
            unpack_bf16x8(xv[i], s);
            unpack_bf16x8(rv[i], b);
            unpack_bf16x8(wv[i], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[j] += b[j];
                sum += s[j] * s[j];
                sw[i][j] = s[j] * w[j];
                top = max(top, __float_as_uint(sw[i][j]) & 0x7fffffffu);
            }
            const int c = lane + i * T;
            if (a.residual_out && c < chunks) reinterpret_cast<uint4*>(a.residual_out)[at + c] = pack_bf16x8(s);
        }
        row_reduce<T>(sum, top, s_a, s_m);
        const float rstd = 1.0f / sqrtf(sum * inv_d + a.eps);
        float inv = 0.0f;
        if (a.yq) {
            const int k = scale_exp_of_f32(__float_as_uint(__uint_as_float(top) * rstd) & 0x7fffffffu);
            inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);  // 2^-k
            if (lane == 0) a.y_scale[r] = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = lane + i * T;
            if (c >= chunks) continue;
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = sw[i][j] * rstd;
            if (a.y) reinterpret_cast<uint4*>(a.y)[at + c] = pack_bf16x8(y);
            if (a.yq) {
                const uint32_t p0 = fp8x2(y[0] * inv, y[1] * inv), p1 = fp8x2(y[2] * inv, y[3] * inv);
                const uint32_t p2 = fp8x2(y[4] * inv, y[5] * inv), p3 = fp8x2(y[6] * inv, y[7] * inv);
                reinterpret_cast<uint2*>(a.yq)[at + c] = make_uint2(p0 | (p1 << 16), p2 | (p3 << 16));
            }
        }
    }
    pdl_trigger();
}

namespace {

int sms() {
    int dev = 0, n = 152;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

template <int T, int V>
cudaError_t norm_go(const NormArgs& a, cudaStream_t st) {
    constexpr int rows = T == 32 ? 8 : 1, threads = T < 256 ? 256 : T;
    const long long want = (a.rows + rows - 1) / rows;
    const int grid = static_cast<int>(std::min<long long>(want, static_cast<long long>(sms()) * (2048 / threads)));
    return launch_kernel(rmsnorm_kernel<T, V>, dim3(grid), dim3(threads), 0, st, a);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t st) {
    if (a.rows <= 0) return cudaSuccess;
    const int chunks = a.D >> 3;
    if (chunks <= 32) return norm_go<32, 1>(a, st);
    if (chunks <= 64) return norm_go<32, 2>(a, st);
    if (chunks <= 128) return norm_go<32, 4>(a, st);
    if (chunks <= 256) return norm_go<256, 1>(a, st);
    if (chunks <= 512) return norm_go<256, 2>(a, st);
    if (chunks <= 1024) return norm_go<256, 4>(a, st);
    if (chunks <= 1024 * 2) return norm_go<1024, 2>(a, st);
    return norm_go<1024, 4>(a, st);
}

// ----------------------------------------------------------------------------
// Gradient.  With v = dy w and r = 1 / sqrt(mean s^2 + eps):
//   dx_j = r v_j - s_j r^3 mean_i(v_i s_i) (+ dresidual_j),   dw_j = sum over rows of dy_j s_j r.
// r is computed again from s, which is read anyway: one reduction gives both
// sums.  A block keeps its columns' dw sums in registers over all its rows and
// stores them once; a second kernel adds the blocks' rows in a fixed order, so
// the result does not change from run to run.
template <int T, int V>
__global__ void __launch_bounds__(T)
rmsnorm_bwd_kernel(const NormBwdArgs a) {
    __shared__ float s_a[T / 32], s_b[T / 32];
    const int chunks = a.D >> 3;
    const int warp = threadIdx.x >> 5;
    pdl_wait();
    const uint4* wrow = reinterpret_cast<const uint4*>(a.weight);
    const float inv_d = 1.0f / static_cast<float>(a.D);
    uint4 wv[V];
    float dw[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * T;
        wv[i] = c < chunks ? wrow[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    }
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const long long at = r * chunks;
        uint4 sv[V], dv[V], ev[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            const bool in = c < chunks;
            sv[i] = in ? reinterpret_cast<const uint4*>(a.s)[at + c] : make_uint4(0, 0, 0, 0);
            dv[i] = in ? reinterpret_cast<const uint4*>(a.dy)[at + c] : make_uint4(0, 0, 0, 0);
            ev[i] = in && a.dresidual ? reinterpret_cast<const uint4*>(a.dresidual)[at + c] : make_uint4(0, 0, 0, 0);
        }
        float s2 = 0.0f, sv_sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float s[8], d[8], w[8];
            unpack_bf16x8(sv[i], s);
            unpack_bf16x8(dv[i], d);
            unpack_bf16x8(wv[i], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s2 += s[j] * s[j];
                sv_sum += d[j] * w[j] * s[j];
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s2 += __shfl_xor_sync(0xffffffffu, s2, o);
            sv_sum += __shfl_xor_sync(0xffffffffu, sv_sum, o);
        }
        if ((threadIdx.x & 31) == 0) {
            s_a[warp] = s2;
            s_b[warp] = sv_sum;
        }
        __syncthreads();
        s2 = sv_sum = 0.0f;
#pragma unroll
        for (int w = 0; w < T / 32; ++w) {
            s2 += s_a[w];
            sv_sum += s_b[w];
        }
        __syncthreads();
        const float rstd = 1.0f / sqrtf(s2 * inv_d + a.eps);
        const float back = rstd * (rstd * (sv_sum * inv_d));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            float s[8], d[8], w[8], e[8], dx[8];
            unpack_bf16x8(sv[i], s);
            unpack_bf16x8(dv[i], d);
            unpack_bf16x8(wv[i], w);
            unpack_bf16x8(ev[i], e);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[i][j] += d[j] * (s[j] * rstd);
                dx[j] = rstd * (d[j] * w[j] - s[j] * back) + e[j];
            }
            if (c < chunks) reinterpret_cast<uint4*>(a.dx)[at + c] = pack_bf16x8(dx);
        }
    }
    if (a.dweight) {
        float4* p = reinterpret_cast<float4*>(a.partial + static_cast<long long>(blockIdx.x) * a.D);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            if (c >= chunks) continue;
            p[2 * c] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            p[2 * c + 1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
    pdl_trigger();
}

// 32 columns a block, 8 threads a column: thread y sums parts y, y + 8, ... in
// order, then the eight sums are added in order.
__global__ void __launch_bounds__(256)
column_sums_kernel(const float* __restrict__ partial, int parts, int cols, float* __restrict__ out) {
    __shared__ float s[8][33];
    pdl_wait();
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
    float v = 0.0f;
    if (col < cols)
#pragma unroll 4
        for (int p = y; p < parts; p += 8) v += partial[static_cast<long long>(p) * cols + col];
    s[y][threadIdx.x & 31] = v;
    __syncthreads();
    if (y == 0 && col < cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][threadIdx.x & 31];
        out[col] = v;
    }
    pdl_trigger();
}

cudaError_t launch_column_sums(const float* partial, int parts, int cols, float* out, cudaStream_t st) {
    return launch_kernel(column_sums_kernel, dim3((cols + 31) / 32), dim3(256), 0, st, partial, parts, cols, out);
}

int rmsnorm_bwd_parts(long long rows) { return static_cast<int>(std::min<long long>(std::max<long long>(rows, 1), 304)); }

namespace {

template <int T, int V>
cudaError_t norm_bwd_go(const NormBwdArgs& a, cudaStream_t st) {
    return launch_kernel(rmsnorm_bwd_kernel<T, V>, dim3(rmsnorm_bwd_parts(a.rows)), dim3(T), 0, st, a);
}

}  // namespace

cudaError_t launch_rmsnorm_bwd(const NormBwdArgs& a, cudaStream_t st) {
    if (a.rows <= 0) return cudaSuccess;
    const int chunks = a.D >> 3;
    cudaError_t e;
    if (chunks <= 128) e = norm_bwd_go<128, 1>(a, st);
    else if (chunks <= 256) e = norm_bwd_go<256, 1>(a, st);
    else if (chunks <= 512) e = norm_bwd_go<512, 1>(a, st);
    else if (chunks <= 1024) e = norm_bwd_go<512, 2>(a, st);
    else if (chunks <= 2048) e = norm_bwd_go<1024, 2>(a, st);
    else e = norm_bwd_go<1024, 4>(a, st);
    if (e != cudaSuccess || !a.dweight) return e;
    return launch_column_sums(a.partial, rmsnorm_bwd_parts(a.rows), a.D, a.dweight, st);
}

}  // namespace moe
