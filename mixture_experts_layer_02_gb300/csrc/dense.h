// dense.h -- internal launch interfaces of the dense operators (norm, gated
// product, linear product and their gradients).  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// ---- root-mean-square norm (rmsnorm.cu) ----
constexpr int kNormMaxD = 32768;

struct NormArgs {
    const uint16_t* x;         // [rows, D]
    const uint16_t* residual;  // [rows, D] or NULL
    const uint16_t* weight;    // [D]
    uint16_t* y;               // [rows, D] or NULL
    uint8_t* yq;               // [rows, D] or NULL
    float* y_scale;            // [rows], with yq
    uint16_t* residual_out;    // [rows, D] or NULL
    long long rows;
    int D;
    float eps;
};
cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t st);

struct NormBwdArgs {
    const uint16_t* dy;         // [rows, D]
    const uint16_t* s;          // [rows, D]
    const uint16_t* weight;     // [D]
    const uint16_t* dresidual;  // [rows, D] or NULL
    uint16_t* dx;               // [rows, D]
    float* dweight;             // [D] or NULL
    float* partial;             // [rmsnorm_bwd_parts(rows, D)][D]
    long long rows;
    int D;
    float eps;
    uint32_t* err;              // workspace error word
    const uint32_t* dbg;        // test flags
};
// Row groups whose dweight sums are kept apart (the workspace's size; the same on every device).
int rmsnorm_bwd_parts(long long rows, int D);
cudaError_t launch_rmsnorm_bwd(const NormBwdArgs& a, cudaStream_t st);

// ---- elementwise halves of the gradients (dense_grad.cu) ----
// dg = dh u act'(g), du = dh act(g) over n values (n % 8 == 0).
cudaError_t launch_gated_grad(const uint16_t* dh, const uint16_t* g, const uint16_t* u, int fn, long long n,
                              uint16_t* dg, uint16_t* du, cudaStream_t st);
// dz = dy act'(z) (FN_NONE: not stored) and, where dbias is set, dbias = the column sums of the unrounded dz.
cudaError_t launch_linear_grad(const uint16_t* dy, const uint16_t* z, int fn, long long rows, int cols, uint16_t* dz,
                               float* dbias, cudaStream_t st);

// ---- tensor-core products (dense_gemm*.cu) ----
// out[m, n] = sum_k A[m, k] B[n, k], bf16 operands, fp32 accumulation.  Each
// operand is stored either K-major (rows m or n, columns k) or MN-major (rows
// k, columns m or n).
//   DENSE_GATED   A = x, B0 = W1, B1 = W3 (both K-major): h = act(g) u, and g, u where set
//   DENSE_LINEAR  A = x, B0 = W (both K-major): y = residual + act(acc + bias), and z = acc + bias where set
//   DENSE_DGRAD   A0|A1 = the incoming gradients (K-major), B0|B1 = the weights (MN-major); segs = 1 or 2
//                 products summed into one output
//   DENSE_WGRAD   A0|A1 = the gradients (MN-major), B0 = x (MN-major); mats = 1 or 2 outputs
enum DenseKind { DENSE_GATED = 0, DENSE_LINEAR = 1, DENSE_DGRAD = 2, DENSE_WGRAD = 3 };

struct DenseArgs {
    int M, N, K;   // output rows and columns, K of one segment
    int segs;      // products summed into the output (DGRAD)
    int mats;      // outputs (WGRAD)
    int fn;
    const float* bias;          // [N] or NULL
    const uint16_t* residual;   // [M, N] or NULL
    uint16_t* out0;             // h, y, dx or dW
    uint16_t* out1;             // g, z or the second dW, or NULL
    uint16_t* out2;             // u or NULL
    uint32_t* err;              // workspace error word
    const uint32_t* dbg;        // test flags
};

struct DenseOperands {
    const uint16_t *a0, *a1, *b0, *b1;
};

// Tensor map of a row-major [rows, cols] bf16 matrix with boxes of 64 columns
// x box_rows rows, 128-byte swizzle (moe_api.cu); 0 or a moe_status.
int make_bf16_map(CUtensorMap* m, const void* base, long long rows, long long cols, int box_rows);

// moe_workspace_size of the dense operations (dense_api.cu); 0 for another name or invalid sizes.
size_t dense_workspace_size(const char* op, int N, int D, int F);

// Tiles with the reduction over K split over a cluster: bn = 0: one CTA per
// 128 x 128 tile and part of K (splits 1, 2, 4 or 8); bn = 128 or 256: a CTA pair
// per 256 x bn tile and part (splits 1, 2 or 4).  clusters != NULL: launch
// nothing, tell how many clusters the device holds at once.
cudaError_t dense_split_gated(const CUtensorMap*, const DenseArgs&, int splits, cudaStream_t, int* clusters);
cudaError_t dense_pairsplit_gated(const CUtensorMap*, const DenseArgs&, int bn, int splits, cudaStream_t, int* clusters);
cudaError_t dense_split_linear(const CUtensorMap*, const DenseArgs&, int splits, cudaStream_t, int* clusters);
cudaError_t dense_pairsplit_linear(const CUtensorMap*, const DenseArgs&, int bn, int splits, cudaStream_t, int* clusters);
cudaError_t dense_split_dgrad(const CUtensorMap*, const DenseArgs&, int splits, cudaStream_t, int* clusters);
cudaError_t dense_pairsplit_dgrad(const CUtensorMap*, const DenseArgs&, int bn, int splits, cudaStream_t, int* clusters);
cudaError_t dense_split_wgrad(const CUtensorMap*, const DenseArgs&, int splits, cudaStream_t, int* clusters);
cudaError_t dense_pairsplit_wgrad(const CUtensorMap*, const DenseArgs&, int bn, int splits, cudaStream_t, int* clusters);
inline cudaError_t dense_split(DenseKind kind, const CUtensorMap* m, const DenseArgs& a, int bn, int splits,
                               cudaStream_t st, int* clusters = nullptr) {
    switch (kind) {
        case DENSE_GATED:
            return bn ? dense_pairsplit_gated(m, a, bn, splits, st, clusters) : dense_split_gated(m, a, splits, st, clusters);
        case DENSE_LINEAR:
            return bn ? dense_pairsplit_linear(m, a, bn, splits, st, clusters) : dense_split_linear(m, a, splits, st, clusters);
        case DENSE_DGRAD:
            return bn ? dense_pairsplit_dgrad(m, a, bn, splits, st, clusters) : dense_split_dgrad(m, a, splits, st, clusters);
        default:
            return bn ? dense_pairsplit_wgrad(m, a, bn, splits, st, clusters) : dense_split_wgrad(m, a, splits, st, clusters);
    }
}

// A few rows (DENSE_GATED, DENSE_LINEAR; M <= kGemvMaxRows): one pass over the weights.
constexpr int kGemvMaxRows = 32;
cudaError_t launch_dense_gemv(DenseKind kind, const DenseOperands& o, const DenseArgs& a, cudaStream_t st);

// CTA pairs on 256 x 256 tiles, persistent: one pair a cluster.
constexpr int kPairTile = 256;
// clusters the device holds at once
cudaError_t dense_pair_limit(DenseKind kind, int* clusters);
cudaError_t launch_dense_pair(DenseKind kind, const CUtensorMap* maps, const DenseArgs& a, int clusters,
                              cudaStream_t st);

}  // namespace moe
