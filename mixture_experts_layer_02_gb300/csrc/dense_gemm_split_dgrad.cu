// dense_gemm_split_dgrad.cu -- the input gradients on split one-CTA tiles (dense_gemm_split.cuh).
#include "dense_gemm_split.cuh"

namespace moe {

cudaError_t dense_split_dgrad(const CUtensorMap* m, const DenseArgs& a, int splits, cudaStream_t st, int* clusters) {
    return dense_split_pick<DENSE_DGRAD>(m, a, splits, st, clusters);
}

}  // namespace moe
