// block_gemm.h -- launch interface of the products in e4m3 with a scale for each
// block of 128 (block_gemm.cuh).  Not part of the public ABI.
#pragma once

#include "train.h"

namespace moe {

//   BLOCK_FWD    y[r, f]     = sum over blocks b of D of sx[r, b] sw[e, f / 128, b] (x[r, b] . w[e, f, b])
//   BLOCK_DGRAD  dx[r, d]    = sum over blocks b of F of sdy[r, b] sw[e, b, d / 128] (dy[r, b] . w[e, b, d])
//   BLOCK_WGRAD  dw[e, f, d] = sum over blocks b of e's padded rows of sdy[b, f] sx[b, d] (dy[b, f] . x[b, d])
enum BlockKind { BLOCK_FWD = 0, BLOCK_DGRAD = 1, BLOCK_WGRAD = 2 };

struct BlockArgs {
    const int32_t* offsets;  // [E + 1] rows of each expert, or NULL: one expert with all rows
    int E, rows;
    int M, N, K;             // WGRAD: M = F, N = D and K by expert; else M by expert, N and K
    const float* a_scale;    // [scale rows, blocks of K]; WGRAD [segment rows / 128, M]
    const int32_t* a_index;  // [rows] row of a_scale, or NULL: the row itself
    int a_scale_rows;
    const float* b_scale;    // [E, blocks of F, blocks of D]; WGRAD [segment rows / 128, N]
    uint16_t* out;           // [rows, N]; WGRAD [E, M, N]
    uint32_t* err;
    const uint32_t* dbg;
};

// A tile kind: CTA pairs on 256 x 256 tiles, or one CTA on 128 x bn, with the sum
// over K in `splits` parts joined over a cluster (bn = 128; then at most one tile a
// cluster).  `tiles` bounds the number of tiles.
struct BlockPlan {
    int stream;  // not 0: no tiles but the stream of weight rows, with this many warps a row (FWD)
    bool pair;
    int bn, splits;
    long long tiles;
};
// Launches the product with the tensor maps of A and B (boxes of 128 x 128 bytes) and of
// the output (boxes of 32 rows x 64 bf16; read by pairs only); clusters != NULL: launches
// nothing, tells how many clusters of this kind the device holds at once (the maps and
// arguments may be NULL).
cudaError_t block_fwd(const BlockPlan&, const CUtensorMap* maps, const BlockArgs*, cudaStream_t, int* clusters);
cudaError_t block_dgrad(const BlockPlan&, const CUtensorMap* maps, const BlockArgs*, cudaStream_t, int* clusters);
cudaError_t block_wgrad(const BlockPlan&, const CUtensorMap* maps, const BlockArgs*, cudaStream_t, int* clusters);

// BLOCK_FWD of a few rows an expert as a stream of weight rows, `warps` (1, 2, 4 or 8)
// of a block's 8 sharing the same rows (block_gemv.cu).
cudaError_t launch_block_gemv(const uint8_t* x, const uint8_t* w, const BlockArgs& a, int warps, cudaStream_t st);

}  // namespace moe
