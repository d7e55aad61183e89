// dense_gemm.cuh -- pieces shared by the dense tensor-core products: operand
// layouts, descriptors and the fused epilogues.
#pragma once

#include "activation.cuh"
#include "dense.h"
#include "gemm_common.cuh"

namespace moe {

// How a kind stores its operands.  K-major: rows m (or n), K contiguous, one
// TMA box of 64 K x R rows a k-block.  MN-major: rows k, M (or N) contiguous,
// one box of 64 columns x 64 k-rows (8 KB) for each 64 columns.  Nothing is
// transposed in memory: the gradient products read the weights, activations
// and incoming gradients as the forward pass stored them.
template <int KIND>
struct DenseLayout {
    static constexpr bool A_MN = KIND == DENSE_WGRAD;
    static constexpr bool B_MN = KIND == DENSE_DGRAD || KIND == DENSE_WGRAD;
    static constexpr bool GATED = KIND == DENSE_GATED;
};

constexpr int kMnBlockBytes = 64 * kRowBytes;  // one MN-major box: 64 k-rows of 64 columns

// Shared-memory descriptor of an MN-major operand written by TMA with 128-byte
// swizzle: each k-row holds 64 consecutive M/N elements (128 bytes), 8 k-rows
// are a 1024-byte swizzle atom (stride offset), the next 64 M/N elements start
// one box further (leading offset).  A step of 16 along K is two atoms.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(kMnBlockBytes >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
    return MN ? sw128_mnmajor_desc(saddr) : sw128_kmajor_desc(saddr);
}
// descriptor step (16-byte units) of one MMA's 16 K elements
template <bool MN>
constexpr uint64_t kDescStep = MN ? (2 * 1024) >> 4 : 32 >> 4;

template <int KIND>
__host__ __device__ constexpr uint32_t dense_idesc(int M, int N) {
    return idesc_bf16_f32(M, N) | (DenseLayout<KIND>::A_MN ? 1u << 15 : 0u) | (DenseLayout<KIND>::B_MN ? 1u << 16 : 0u);
}

// ---- fused epilogues: eight consecutive columns of one row ----
// n % 8 == 0 for every width, so an octet is inside or outside as a whole and
// every access is one aligned 16-byte word.
__device__ __forceinline__ uint4* octet(uint16_t* base, long long row, int ld, int col) {
    return reinterpret_cast<uint4*>(base + row * ld + col);
}
__device__ __forceinline__ const uint4* octet(const uint16_t* base, long long row, int ld, int col) {
    return reinterpret_cast<const uint4*>(base + row * ld + col);
}

// h = act(g) u from the fp32 accumulators (g and u are rounded only where they
// are stored for the backward pass).
__device__ __forceinline__ void gated_octet(const DenseArgs& a, long long row, int col, const float (&g)[8],
                                            const float (&u)[8]) {
    float h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = act_value(a.fn, g[j]) * u[j];
    *octet(a.out0, row, a.N, col) = pack_bf16x8(h);
    if (a.out1) *octet(a.out1, row, a.N, col) = pack_bf16x8(g);
    if (a.out2) *octet(a.out2, row, a.N, col) = pack_bf16x8(u);
}

// y = residual + act(acc + bias) in fp32, rounded once.
__device__ __forceinline__ void linear_octet(const DenseArgs& a, long long row, int col, float (&z)[8]) {
    if (a.bias) {
        const float4 b0 = __ldg(reinterpret_cast<const float4*>(a.bias + col));
        const float4 b1 = __ldg(reinterpret_cast<const float4*>(a.bias + col) + 1);
        z[0] += b0.x, z[1] += b0.y, z[2] += b0.z, z[3] += b0.w;
        z[4] += b1.x, z[5] += b1.y, z[6] += b1.z, z[7] += b1.w;
    }
    if (a.out1) *octet(a.out1, row, a.N, col) = pack_bf16x8(z);
    if (a.fn != FN_NONE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = act_value(a.fn, z[j]);
    }
    if (a.residual) {
        float r[8];
        unpack_bf16x8(*octet(a.residual, row, a.N, col), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] += r[j];
    }
    *octet(a.out0, row, a.N, col) = pack_bf16x8(z);
}

}  // namespace moe
