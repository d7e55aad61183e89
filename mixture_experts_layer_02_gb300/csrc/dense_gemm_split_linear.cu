// dense_gemm_split_linear.cu -- the linear product on split one-CTA tiles (dense_gemm_split.cuh).
#include "dense_gemm_split.cuh"

namespace moe {

cudaError_t dense_split_linear(const CUtensorMap* m, const DenseArgs& a, int splits, cudaStream_t st, int* clusters) {
    return dense_split_pick<DENSE_LINEAR>(m, a, splits, st, clusters);
}

}  // namespace moe
