// block_gemm_fwd.cu -- the block-scaled e4m3 product's BLOCK_FWD kernels (block_gemm.cuh).
#include "block_gemm.cuh"

namespace moe {

cudaError_t block_fwd(const BlockPlan& p, const CUtensorMap* maps, const BlockArgs* a, cudaStream_t st, int* clusters) {
    return block_pick<BLOCK_FWD>(p, maps, a, st, clusters);
}

}  // namespace moe
