// dense_gemm_pairsplit_linear.cu -- the linear product on split pair tiles (dense_gemm_pairsplit.cuh).
#include "dense_gemm_pairsplit.cuh"

namespace moe {

cudaError_t dense_pairsplit_linear(const CUtensorMap* m, const DenseArgs& a, int bn, int splits, cudaStream_t st,
                                int* clusters) {
    return dense_pairsplit_pick<DENSE_LINEAR>(m, a, bn, splits, st, clusters);
}

}  // namespace moe
