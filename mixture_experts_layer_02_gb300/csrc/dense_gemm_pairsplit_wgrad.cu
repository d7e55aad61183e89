// dense_gemm_pairsplit_wgrad.cu -- the weight gradients on split pair tiles (dense_gemm_pairsplit.cuh).
#include "dense_gemm_pairsplit.cuh"

namespace moe {

cudaError_t dense_pairsplit_wgrad(const CUtensorMap* m, const DenseArgs& a, int bn, int splits, cudaStream_t st,
                                int* clusters) {
    return dense_pairsplit_pick<DENSE_WGRAD>(m, a, bn, splits, st, clusters);
}

}  // namespace moe
