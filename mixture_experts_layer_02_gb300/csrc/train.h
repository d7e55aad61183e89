// train.h -- internal launch interfaces of the routed layer's training operators
// (gradients of the sort, the weighted sum and the router) and of the products in
// e4m3 with a scale for each block of 128.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// moe_workspace_size of these operations (train_api.cu); 0 for another name or invalid sizes.
size_t train_workspace_size(const char* op, int N, int D, int E, int Dff);

// ---- gradients of the weighted sum, the sort and the routing weights (routing_grad.cu) ----
// dy[inv[t,k]] = w[t,k] dout[t] and dw[t,k] = <dout[t], y[inv[t,k]]>, each where its pointer is set.
cudaError_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y, const int32_t* inv, const float* w, int N, int D,
                               int K, long long rows, uint16_t* dy, float* dw, uint32_t* err, cudaStream_t st);
// dx[t] = dresidual[t] + sum_k dx_perm[inv[t,k]]
cudaError_t launch_permute_bwd(const uint16_t* dx_perm, const int32_t* inv, const uint16_t* dresidual, int N, int D, int K,
                               long long rows, uint16_t* dx, uint32_t* err, cudaStream_t st);

// Gradient of the selected logits, scattered into dl [N, ld] bf16 (ld = E rounded up to 8,
// zero elsewhere) and, where dbias is set, summed over the tokens through `partial`
// [route_bwd_parts(N)][E].
constexpr int kRouteBwdTokens = 8;  // tokens a block: one a warp
inline long long route_bwd_parts(int N) { return (static_cast<long long>(N) + kRouteBwdTokens - 1) / kRouteBwdTokens; }
struct RouteBwdArgs {
    const float* dw;        // [N, K]
    const int32_t* ids;     // [N, K]
    const float* w;         // [N, K]
    const float* logits;    // [N, E], sigmoid scores only
    int N, E, K, ld;
    bool sigmoid;
    uint16_t* dl;           // [N, ld]
    float* partial;
    float* dbias;           // [E] or NULL
    uint32_t* err;
};
cudaError_t launch_route_bwd(const RouteBwdArgs& a, cudaStream_t st);

// ---- e4m3 with a scale for each block of 128 (quant_block.cu) ----
constexpr int kBlock = 128;  // values that share a scale, along each blocked dimension
inline long long blocks_of(long long n) { return (n + kBlock - 1) / kBlock; }
// Rows of a buffer whose segments start at multiples of 128, for any routing.
inline long long segment_rows_of(long long rows, int E) {
    return (rows + (kBlock - 1) * (rows < E ? rows : static_cast<long long>(E))) / kBlock * kBlock;
}
cudaError_t launch_quant_rows_block(const uint16_t* src, long long rows, int cols, uint8_t* q, float* scale,
                                    cudaStream_t st);
cudaError_t launch_quant_tiles(const uint16_t* src, long long mats, int rows, int cols, uint8_t* q, float* scale,
                               cudaStream_t st);
struct QuantSegArgs {
    const uint16_t* src;     // [rows, cols]
    const int32_t* offsets;  // [E + 1] or NULL: one segment
    int E, rows, cols;
    uint8_t* q;              // [rows, cols] or NULL
    float* scale;            // [rows, blocks]
    uint8_t* q_seg;          // [segment rows, cols]
    float* scale_seg;        // [segment rows / 128, cols]
    uint32_t* err;
};
cudaError_t launch_quant_segments(const QuantSegArgs& a, cudaStream_t st);

}  // namespace moe
