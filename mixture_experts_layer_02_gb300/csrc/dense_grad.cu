// dense_grad.cu -- the elementwise halves of the dense products' gradients.
//
//   gated   dg = dh u act'(g),  du = dh act(g)
//   linear  dz = dy act'(z),    dbias = sum over rows of dz
//
// One pass over the inputs in 16-byte words, bound by HBM.  dg, du and dz are
// rounded to bf16 once: they are operands of tensor-core products next, which
// take bf16.  dbias is summed from the unrounded fp32 values.
#include <algorithm>

#include "activation.cuh"
#include "dense.h"

namespace moe {

namespace {

constexpr int kGradThreads = 256;

int sms() {
    int dev = 0, n = 152;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

__global__ void __launch_bounds__(kGradThreads)
gated_grad_kernel(const uint4* __restrict__ dh, const uint4* __restrict__ g, const uint4* __restrict__ u, int fn,
                  long long chunks, uint4* __restrict__ dg, uint4* __restrict__ du) {
    pdl_wait();
    for (long long i = static_cast<long long>(blockIdx.x) * kGradThreads + threadIdx.x; i < chunks;
         i += static_cast<long long>(gridDim.x) * kGradThreads) {
        float h[8], a[8], b[8];
        unpack_bf16x8(dh[i], h);
        unpack_bf16x8(g[i], a);
        unpack_bf16x8(u[i], b);
        float slope[8];
        act_slopes(fn, a, slope);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            slope[j] *= h[j] * b[j];
            b[j] = h[j] * a[j];
        }
        dg[i] = pack_bf16x8(slope);
        du[i] = pack_bf16x8(b);
    }
    pdl_trigger();
}

// A block owns 256 columns (32 octets) of a range of rows; its 8 warps take
// the rows in turn.  The column sums stay in registers, are added over the
// warps in order, and one fp32 row a block goes to `partial`.
__global__ void __launch_bounds__(kGradThreads)
linear_grad_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ z, int fn, long long rows, int cols,
                   int parts, uint16_t* __restrict__ dz, float* __restrict__ partial) {
    __shared__ float s[8][32][9];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = (blockIdx.x * 32 + lane) * 8;
    const long long r0 = rows * blockIdx.y / parts, r1 = rows * (blockIdx.y + 1) / parts;
    float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (col < cols) {
#pragma unroll 2
        for (long long r = r0 + warp; r < r1; r += 8) {
            const long long at = r * cols + col;
            float d[8];
            unpack_bf16x8(*reinterpret_cast<const uint4*>(dy + at), d);
            if (fn != FN_NONE) {
                float v[8];
                unpack_bf16x8(*reinterpret_cast<const uint4*>(z + at), v);
                float slope[8];
                act_slopes(fn, v, slope);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] *= slope[j];
                *reinterpret_cast<uint4*>(dz + at) = pack_bf16x8(d);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += d[j];
        }
    }
    if (partial) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[warp][lane][j] = sum[j];
        __syncthreads();
        const int c = blockIdx.x * 256 + threadIdx.x;
        if (c < cols) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) v += s[w][threadIdx.x >> 3][threadIdx.x & 7];
            partial[static_cast<long long>(blockIdx.y) * cols + c] = v;
        }
    }
    pdl_trigger();
}

}  // namespace

cudaError_t launch_gated_grad(const uint16_t* dh, const uint16_t* g, const uint16_t* u, int fn, long long n,
                              uint16_t* dg, uint16_t* du, cudaStream_t st) {
    const long long chunks = n >> 3;
    const long long want = (chunks + kGradThreads - 1) / kGradThreads;
    const int grid = static_cast<int>(std::min<long long>(want, static_cast<long long>(sms()) * 8));
    return launch_kernel(gated_grad_kernel, dim3(grid), dim3(kGradThreads), 0, st, reinterpret_cast<const uint4*>(dh),
                         reinterpret_cast<const uint4*>(g), reinterpret_cast<const uint4*>(u), fn, chunks,
                         reinterpret_cast<uint4*>(dg), reinterpret_cast<uint4*>(du));
}

int linear_grad_parts(long long rows) {
    return static_cast<int>(std::min<long long>(64, std::max<long long>(1, (rows + 31) / 32)));
}

cudaError_t launch_linear_grad(const uint16_t* dy, const uint16_t* z, int fn, long long rows, int cols, uint16_t* dz,
                               float* dbias, float* partial, cudaStream_t st) {
    if (fn == FN_NONE && dbias == nullptr) return cudaSuccess;  // dz = dy
    const int parts = linear_grad_parts(rows);
    cudaError_t e = launch_kernel(linear_grad_kernel, dim3((cols + 255) / 256, parts), dim3(kGradThreads), 0, st, dy, z,
                                  fn, rows, cols, parts, dz, dbias ? partial : static_cast<float*>(nullptr));
    if (e != cudaSuccess || dbias == nullptr) return e;
    return launch_column_sums(partial, parts, cols, dbias, st);
}

}  // namespace moe
