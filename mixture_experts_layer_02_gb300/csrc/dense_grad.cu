// dense_grad.cu -- the elementwise halves of the dense products' gradients.
//
//   gated   dg = dh u act'(g),  du = dh act(g)
//   linear  dz = dy act'(z),    dbias = sum over rows of dz
//
// One pass over the inputs in 16-byte words, bound by HBM and, with GELU, by its
// arithmetic (777 x 4096 with the bias gradient 7.0 us, 4096 x 4096 24 us).  dg, du and dz are
// rounded to bf16 once: they are operands of tensor-core products next, which
// take bf16.  dbias is summed from the unrounded fp32 values.  Coherent loads only (no
// const __restrict__): the launch before may still be writing them when blocks start.
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
gated_grad_kernel(const uint4* dh, const uint4* g, const uint4* u, int fn, long long chunks, uint4* dg, uint4* du) {
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

// A cluster of eight blocks owns 64 columns (128-byte pieces of a row); each
// takes an eighth of the rows, 32 at a time.  The column sums stay in registers,
// are added over the rows of a block and then, through distributed shared
// memory, over the blocks in order: no partial sums in memory, no second launch
// (which took 3 us of the 10 at 777 x 4096).
constexpr int kGradParts = 8;

__global__ void __cluster_dims__(1, kGradParts, 1) __launch_bounds__(kGradThreads, 4)
linear_grad_kernel(const uint16_t* dy, const uint16_t* z, int fn, long long rows, int cols, uint16_t* dz,
                   float* dbias) {
    __shared__ float s_warp[kGradThreads / 32][64];
    __shared__ float s_part[64];
    pdl_wait();
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;  // octet of columns, row of 32
    const int col = blockIdx.x * 64 + tx * 8;
    const long long r0 = rows * blockIdx.y / kGradParts, r1 = rows * (blockIdx.y + 1) / kGradParts;
    float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    // the next row's loads are issued before this row's arithmetic
    uint4 dn = make_uint4(0, 0, 0, 0), zn = dn;
    auto fetch = [&](long long r) {
        if (r >= r1) return;
        dn = *reinterpret_cast<const uint4*>(dy + r * cols + col);
        if (fn != FN_NONE) zn = *reinterpret_cast<const uint4*>(z + r * cols + col);
    };
    if (col < cols) {
        fetch(r0 + ty);
        for (long long r = r0 + ty; r < r1; r += 32) {
            float d[8], v[8];
            unpack_bf16x8(dn, d);
            unpack_bf16x8(zn, v);
            fetch(r + 32);
            if (fn != FN_NONE) {
                float slope[8];
                act_slopes(fn, v, slope);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] *= slope[j];
                *reinterpret_cast<uint4*>(dz + r * cols + col) = pack_bf16x8(d);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += d[j];
        }
    }
    pdl_trigger();
    if (dbias == nullptr) return;  // the same for the whole cluster
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // the warp's four rows
        sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 8);
        sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 16);
    }
    if ((threadIdx.x & 31) < 8)
#pragma unroll
        for (int j = 0; j < 8; ++j) s_warp[threadIdx.x >> 5][tx * 8 + j] = sum[j];
    __syncthreads();
    if (threadIdx.x < 64) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kGradThreads / 32; ++w) v += s_warp[w][threadIdx.x];
        s_part[threadIdx.x] = v;
    }
    cluster_sync_all();
    const int c = blockIdx.x * 64 + static_cast<int>(threadIdx.x);
    if (cluster_ctarank() == 0 && threadIdx.x < 64 && c < cols) {
        float v = 0.0f;
#pragma unroll
        for (uint32_t p = 0; p < kGradParts; ++p) {
            float f;
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(f)
                         : "r"(mapa_shared(smem_u32(&s_part[threadIdx.x]), p))
                         : "memory");
            v += f;
        }
        dbias[c] = v;
    }
    cluster_sync_all();  // no block leaves while the first reads its sums
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

cudaError_t launch_linear_grad(const uint16_t* dy, const uint16_t* z, int fn, long long rows, int cols, uint16_t* dz,
                               float* dbias, cudaStream_t st) {
    if (fn == FN_NONE && dbias == nullptr) return cudaSuccess;  // dz = dy
    return launch_kernel(linear_grad_kernel, dim3((cols + 63) / 64, kGradParts), dim3(kGradThreads), 0, st, dy, z, fn, rows,
                         cols, dz, dbias);
}

}  // namespace moe
