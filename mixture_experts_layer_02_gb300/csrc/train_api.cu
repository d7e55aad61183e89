// train_api.cu -- the C entry points of the routed layer's training operators and of
// the products in e4m3 with a scale for each block of 128 (include/moe.h): argument
// checks, workspace carving, the choice of kernel and the launches.
#include <algorithm>
#include <cstdlib>
#include <cstring>

#include "../../include/moe.h"
#include "api_checks.h"
#include "block_gemm.h"
#include "dense.h"

using namespace moe;

namespace {

constexpr long long kRowsLimit = 0x7fffffffLL - 4095;  // rounded up to whole tiles it stays below 2^31

moe_status check_experts(int E) {
    return E < 1 || E > 1024 ? refuse(MOE_ERR_INVALID_ARG, "E=%d outside 1..1024", E) : MOE_OK;
}

// assignments and rows of the sort's gradients
moe_status check_sort(int N, int D, int K, int rows) {
    if (N < 0) return refuse(MOE_ERR_INVALID_ARG, "N=%d < 0", N);
    if (K < 1 || K > 32) return refuse(MOE_ERR_INVALID_ARG, "K=%d outside 1..32", K);
    if (D < 8 || D % 8) return refuse(MOE_ERR_INVALID_ARG, "D=%d not a positive multiple of 8", D);
    if (rows < 0) return refuse(MOE_ERR_INVALID_ARG, "rows=%d < 0", rows);
    if (static_cast<long long>(N) * K > kRowsLimit) return refuse(MOE_ERR_INVALID_ARG, "N*K=%lld too large", static_cast<long long>(N) * K);
    if (static_cast<long long>(std::max(rows, N)) * D >= (1LL << 40)) return refuse(MOE_ERR_INVALID_ARG, "rows*D too large");
    return MOE_OK;
}

moe_status check_route(int N, int D, int E, int K) {
    moe_status s = check_experts(E);
    if (s == MOE_OK) s = check_sort(N, D, K, 0);
    if (s != MOE_OK) return s;
    if (K > E) return refuse(MOE_ERR_INVALID_ARG, "K=%d above E=%d", K, E);
    if (std::max(N, D) > kRowsLimit) return refuse(MOE_ERR_INVALID_ARG, "N=%d, D=%d too large", N, D);
    return MOE_OK;
}

// rows of codes whose width is a multiple of 16 bytes
moe_status check_codes(const char* name, int width) {
    if (width < 16 || width % 16) return refuse(MOE_ERR_INVALID_ARG, "%s=%d not a positive multiple of 16", name, width);
    if (width > (1 << 30)) return refuse(MOE_ERR_INVALID_ARG, "%s=%d above %d", name, width, 1 << 30);  // column numbers past the end stay in 32 bits
    return MOE_OK;
}

moe_status check_block(int rows, int D, int E, int F) {
    moe_status s = check_experts(E);
    if (s == MOE_OK) s = check_codes("D", D);
    if (s == MOE_OK) s = check_codes("F", F);
    if (s != MOE_OK) return s;
    if (rows < 0) return refuse(MOE_ERR_INVALID_ARG, "total_rows=%d < 0", rows);
    if (segment_rows_of(rows, E) > kRowsLimit) return refuse(MOE_ERR_INVALID_ARG, "total_rows=%d too large", rows);
    if (segment_rows_of(rows, E) * std::max(D, F) >= (1LL << 40) || static_cast<long long>(D) * F >= (1LL << 40) / E)
        return refuse(MOE_ERR_INVALID_ARG, "total_rows=%d, D=%d, E=%d, F=%d too large", rows, D, E, F);
    // tiles are numbered in 32 bits: the smallest, 128 x 128, of rows and of weight gradients
    if ((blocks_of(rows) + E) * blocks_of(std::max(D, F)) > kRowsLimit || E * blocks_of(D) * blocks_of(F) > kRowsLimit)
        return refuse(MOE_ERR_INVALID_ARG, "total_rows=%d, D=%d, E=%d, F=%d: too many tiles", rows, D, E, F);
    return MOE_OK;
}

int up8(int v) { return (v + 7) / 8 * 8; }

struct RouteLayout {
    size_t dl, partial, total;
};

RouteLayout route_layout(int N, int E) {
    RouteLayout l;
    l.dl = kWsHeaderBytes;
    l.partial = l.dl + up256(static_cast<size_t>(N) * up8(E) * 2);
    l.total = l.partial + up256(static_cast<size_t>(route_bwd_parts(N)) * E * sizeof(float));
    return l;
}

uint8_t* at(void* ws, size_t off) { return static_cast<uint8_t*>(ws) + off; }
uint32_t* error_word(void* ws) { return static_cast<uint32_t*>(ws); }

moe_status zero(void* p, size_t bytes, cudaStream_t st) {
    return p ? launched(cudaMemsetAsync(p, 0, bytes, st), "zero gradient") : MOE_OK;
}

int env_int(const char* name, int dflt) {
    const char* f = getenv(name);
    return f ? atoi(f) : dflt;
}

cudaError_t block(BlockKind kind, const BlockPlan& p, const CUtensorMap* maps, const BlockArgs* a, cudaStream_t st) {
    switch (kind) {
        case BLOCK_FWD: return block_fwd(p, maps, a, st, nullptr);
        case BLOCK_DGRAD: return block_dgrad(p, maps, a, st, nullptr);
        default: return block_wgrad(p, maps, a, st, nullptr);
    }
}

// Row tiles of `height` that the experts' segments have at most.
long long row_tiles(const BlockArgs& a, int height) {
    const long long some = std::min(a.rows, a.E);  // experts with rows, one at least
    return some + (a.rows - some) / height;
}

// The choice of kernel, from sizes that the host knows; times are microseconds on GB300.
//   stream      up to 8 rows, or up to 128 and one an expert on average: 7168 x 2048 and
//               one row 8, as tiles 11 to 24; 2048 x 768, 128 experts and 64 rows 21, tiles
//               25 to 27.  An expert's rows are taken in turns of eight, each of which reads
//               its weights again: tiles win from 16 rows an expert on (7168 x 2048 14
//               against 12), and 128 rows bound the turns of a batch that all goes to one.
//   pairs       where an expert fills most of a 256-row tile: 4096 x 4096 x 14336 by 8
//               experts (1024 rows each) 404, one-CTA tiles 441; at 128 rows each 119 both
//               ways, but 4096 x 7168 x 2048 by 256 experts (128 rows on average, ragged)
//               872 and 729, and 64 rows each 115 and 96.  The weight gradient's tiles are
//               whole whatever the rows (both gradients 4096^2 by 8 experts: 64 rows 92 and
//               100, 256 rows 133 and 162, 512 rows 197 and 217).
//   128 x 256   else, where its tiles fill most of the GPU: 2048 x 768, 128 experts, 16384
//               rows 61 against 65 for 128 x 128.
//   128 x 128   else, with K in up to four parts while its tiles leave SMs idle: 7168 x 2048
//               and 64 rows 16 in four parts, 20 in two, 28 whole.  The
//               weight gradient's K is an expert's rows, too short for parts to pay but with
//               one expert: 1024^2 by 4000 rows 31 whole and in two parts.
// MOE_BLOCK_KERNEL = 1 (128 x 128), 2 (128 x 256), 3 (pairs) or 4 (stream, FWD only), and
// MOE_BLOCK_SPLIT = parts of K (1) or warps a row (4), force a choice, for tuning and test
// coverage.
BlockPlan plan_block(BlockKind kind, const BlockArgs& a) {
    auto tiles = [&](int height, int width) {
        const long long n = (a.N + width - 1) / width;
        return kind == BLOCK_WGRAD ? a.E * ((a.M + height - 1) / static_cast<long long>(height)) * n : row_tiles(a, height) * n;
    };
    int kernel = env_int("MOE_BLOCK_KERNEL", 0);
    const bool kernel_set = kernel != 0;
    const int fixed = kernel_set ? env_int("MOE_BLOCK_SPLIT", 1) : 0;
    if (kernel == 4 && kind != BLOCK_FWD) kernel = 1;
    if (kernel == 0) {
        const int mean = a.rows / a.E;
        const bool high = (kind == BLOCK_WGRAD ? a.M : mean) >= 160;
        if (kind == BLOCK_FWD && (a.rows <= 8 || (mean <= 1 && a.rows <= 128))) kernel = 4;
        else if (high && tiles(2 * kBM, 256) >= 38) kernel = 3;
        else kernel = tiles(kBM, 256) >= 120 ? 2 : 1;
    }
    if (kernel == 4) {
        int warps = fixed;
        if (!warps) {  // enough warps for the GPU, each with a few blocks
            const long long units = static_cast<long long>(std::min(a.rows, a.E)) * ((a.N + 15) / 16);
            warps = 1;
            while (warps < 8 && units * warps < 152 * 12 && blocks_of(a.K) >= 4 * warps) warps *= 2;
        }
        return {warps, false, 0, 0, 0};
    }
    if (kernel == 3) return {0, true, 256, 1, tiles(2 * kBM, 256)};
    if (kernel == 2) return {0, false, 256, 1, tiles(kBM, 256)};
    int splits = kernel_set && fixed != 2 && fixed != 4 ? 1 : fixed;
    const long long n = tiles(kBM, 128), kbs = kind == BLOCK_WGRAD ? blocks_of(a.rows / a.E) : blocks_of(a.K);
    if (!splits) {
        splits = 1;
        while (splits < 4 && n * splits * 2 <= 152 && kbs >= 4 * splits) splits *= 2;
    }
    return {0, false, 128, splits, n};
}

moe_status product(BlockKind kind, const uint8_t* a_codes, long long a_rows, long long a_cols, const uint8_t* b_codes,
                   long long b_mats, long long b_rows, long long b_cols, const BlockArgs& a, cudaStream_t st) {
    const BlockPlan p = plan_block(kind, a);
    if (p.stream) return launched(launch_block_gemv(a_codes, b_codes, a, p.stream, st), "block-scaled product launch");
    CUtensorMap m[3];
    int e = make_byte_map(&m[0], a_codes, 1, a_rows, a_cols);
    if (e == 0) e = make_byte_map(&m[1], b_codes, b_mats, b_rows, b_cols);
    if (e == 0 && p.pair) e = make_bf16_out_map(&m[2], a.out, kind == BLOCK_WGRAD ? a.E : 1, a.M, a.N);
    if (e != 0) return static_cast<moe_status>(e);
    if (!p.pair) m[2] = m[0];
    return launched(block(kind, p, m, &a, st), "block-scaled product launch");
}

BlockArgs block_args(const int32_t* offsets, int E, int rows, void* ws) {
    BlockArgs a = {};
    a.offsets = offsets;
    a.E = E;
    a.rows = rows;
    a.err = error_word(ws);
    a.dbg = error_word(ws) + 1;
    return a;
}

}  // namespace

size_t moe::train_workspace_size(const char* op, int N, int D, int E, int F) {
    if (!strcmp(op, "route_backward")) return check_route(N, D, E, 1) == MOE_OK ? route_layout(N, E).total : 0;
    if (!strcmp(op, "grouped_linear_e4m3_block") || !strcmp(op, "grouped_linear_e4m3_block_backward"))
        return check_block(N, D, E, F) == MOE_OK ? kWsHeaderBytes : 0;
    return 0;
}

extern "C" {

moe_status moe_combine_backward(const moe_bf16* dout, const moe_bf16* y_perm, const int32_t* inv_perm, const float* topk_w,
                                int N, int D, int K, int rows, moe_bf16* dy_perm, float* dtopk_w, void* ws, size_t ws_bytes,
                                void* stream) {
    const moe_status s = check_sort(N, D, K, rows);
    if (s != MOE_OK) return s;
    MAY(y_perm);
    MAY(dy_perm);
    MAY(dtopk_w);
    if (N == 0) return MOE_OK;
    NEED(dout);
    NEED(inv_perm);
    NEED(topk_w);
    if (!dy_perm && !dtopk_w && rows) return refuse(MOE_ERR_INVALID_ARG, "no output: dy_perm and dtopk_w are NULL");
    if (dtopk_w && rows) NEED(y_perm);
    NEED_WS(kWsHeaderBytes);
    return launched(launch_combine_bwd(dout, y_perm, inv_perm, topk_w, N, D, K, rows, dy_perm, dtopk_w, error_word(ws),
                                       static_cast<cudaStream_t>(stream)),
                    "combine backward launch");
}

moe_status moe_permute_backward(const moe_bf16* dx_perm, const int32_t* inv_perm, const moe_bf16* dresidual, int N, int D,
                                int K, int rows, moe_bf16* dx, void* ws, size_t ws_bytes, void* stream) {
    const moe_status s = check_sort(N, D, K, rows);
    if (s != MOE_OK) return s;
    MAY(dresidual);
    if (N == 0) return MOE_OK;
    if (rows) NEED(dx_perm);
    NEED(inv_perm);
    NEED(dx);
    NEED_WS(kWsHeaderBytes);
    return launched(launch_permute_bwd(dx_perm, inv_perm, dresidual, N, D, K, rows, dx, error_word(ws),
                                       static_cast<cudaStream_t>(stream)),
                    "permute backward launch");
}

moe_status moe_route_backward(const float* dtopk_w, const int32_t* topk_ids, const float* topk_w, const float* logits,
                              const moe_bf16* x, const moe_bf16* w_gate, const moe_bf16* dresidual, int N, int D, int E,
                              int K, int mode, moe_bf16* dx, moe_bf16* dw_gate, float* dbias, void* ws, size_t ws_bytes,
                              void* stream) {
    moe_status s = check_route(N, D, E, K);
    if (s != MOE_OK) return s;
    if (mode != MOE_SCORE_SOFTMAX_TOPK && mode != MOE_SCORE_SIGMOID_NORM) return refuse(MOE_ERR_INVALID_ARG, "mode=%d", mode);
    MAY(dx);
    MAY(dw_gate);
    MAY(dbias);
    MAY(dresidual);
    if (!dx && !dw_gate && !dbias) return refuse(MOE_ERR_INVALID_ARG, "no output: dx, dw_gate and dbias are NULL");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (N == 0) {
        s = zero(dw_gate, static_cast<size_t>(E) * D * 2, st);
        return s == MOE_OK ? zero(dbias, static_cast<size_t>(E) * sizeof(float), st) : s;
    }
    NEED(dtopk_w);
    NEED(topk_ids);
    NEED(topk_w);
    if (mode == MOE_SCORE_SIGMOID_NORM) NEED(logits);
    if (dx) NEED(w_gate);
    if (dw_gate) NEED(x);
    const RouteLayout l = route_layout(N, E);
    NEED_WS(l.total);
    const int ld = up8(E);
    uint16_t* dl = reinterpret_cast<uint16_t*>(at(ws, l.dl));
    const RouteBwdArgs r = {dtopk_w, topk_ids, topk_w, logits, N, E, K, ld, mode == MOE_SCORE_SIGMOID_NORM, dl,
                            reinterpret_cast<float*>(at(ws, l.partial)), dbias, error_word(ws)};
    s = launched(launch_route_bwd(r, st), "route backward launch");
    DenseArgs a = {};
    a.segs = a.mats = 1;
    a.err = error_word(ws);
    a.dbg = error_word(ws) + 1;
    a.N = D;
    if (s == MOE_OK && dx) {  // dx = dresidual + dl w_gate
        a.M = N;
        a.K = E;
        a.residual = dresidual;
        a.out0 = dx;
        s = static_cast<moe_status>(dense_product(DENSE_DGRAD, {dl, nullptr, w_gate, nullptr, ld}, a, st));
    }
    if (s == MOE_OK && dw_gate) {  // dw_gate = dl^T x
        a.M = E;
        a.K = N;
        a.residual = nullptr;
        a.out0 = dw_gate;
        s = static_cast<moe_status>(dense_product(DENSE_WGRAD, {dl, nullptr, x, nullptr, ld}, a, st));
    }
    return s;
}

moe_status moe_quantize_e4m3_block(const moe_bf16* src, int mats, int rows, int cols, int block_rows, uint8_t* q, float* scale,
                                   void* stream) {
    if (mats < 0 || rows < 0) return refuse(MOE_ERR_INVALID_ARG, "mats=%d, rows=%d", mats, rows);
    if (block_rows != 1 && block_rows != kBlock) return refuse(MOE_ERR_INVALID_ARG, "block_rows=%d is neither 1 nor 128", block_rows);
    const moe_status s = check_codes("cols", cols);
    if (s != MOE_OK) return s;
    const long long all = static_cast<long long>(mats) * rows;
    if (all >= (1LL << 40) / cols || rows > kRowsLimit) return refuse(MOE_ERR_INVALID_ARG, "mats=%d, rows=%d, cols=%d too large", mats, rows, cols);
    if (all == 0) return MOE_OK;
    NEED(src);
    NEED(q);
    NEED(scale);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (block_rows == 1) return launched(launch_quant_rows_block(src, all, cols, q, scale, st), "block quantiser launch");
    return launched(launch_quant_tiles(src, mats, rows, cols, q, scale, st), "block quantiser launch");
}

long long moe_segment_rows(int total_rows, int E) {
    return total_rows < 0 || check_experts(E) != MOE_OK ? -1 : segment_rows_of(total_rows, E);
}

moe_status moe_quantize_e4m3_segments(const moe_bf16* src, const int32_t* expert_offsets, int total_rows, int cols, int E,
                                      uint8_t* q, float* scale, uint8_t* q_seg, float* scale_seg, void* ws, size_t ws_bytes,
                                      void* stream) {
    const moe_status s = check_block(total_rows, cols, E, 16);
    if (s != MOE_OK) return s;
    MAY(expert_offsets);
    MAY(q);
    MAY(scale);
    if ((q == nullptr) != (scale == nullptr)) return refuse(MOE_ERR_INVALID_ARG, "q and scale come together");
    if (!expert_offsets && E != 1) return refuse(MOE_ERR_INVALID_ARG, "expert_offsets is NULL with E=%d", E);
    if (total_rows == 0) return MOE_OK;
    NEED(src);
    NEED(q_seg);
    NEED(scale_seg);
    NEED_WS(kWsHeaderBytes);
    const QuantSegArgs a = {src, expert_offsets, E, total_rows, cols, q, scale, q_seg, scale_seg, error_word(ws)};
    return launched(launch_quant_segments(a, static_cast<cudaStream_t>(stream)), "segment quantiser launch");
}

moe_status moe_grouped_linear_e4m3_block(const uint8_t* xq, const float* x_scale, const int32_t* x_scale_index,
                                         int x_scale_rows, const int32_t* expert_offsets, int total_rows, const uint8_t* wq,
                                         const float* w_scale, int E, int D, int F, moe_bf16* y, void* ws, size_t ws_bytes,
                                         void* stream) {
    const moe_status s = check_block(total_rows, D, E, F);
    if (s != MOE_OK) return s;
    MAY(x_scale_index);
    MAY(expert_offsets);
    if (!expert_offsets && E != 1) return refuse(MOE_ERR_INVALID_ARG, "expert_offsets is NULL with E=%d", E);
    if (!x_scale_index && x_scale_rows < total_rows)
        return refuse(MOE_ERR_INVALID_ARG, "x_scale_rows=%d below total_rows=%d", x_scale_rows, total_rows);
    if (total_rows == 0) return MOE_OK;
    NEED(xq);
    NEED(x_scale);
    NEED(wq);
    NEED(w_scale);
    NEED(y);
    NEED_WS(kWsHeaderBytes);
    BlockArgs a = block_args(expert_offsets, E, total_rows, ws);
    a.M = total_rows;
    a.N = F;
    a.K = D;
    a.a_scale = x_scale;
    a.a_index = x_scale_index;
    a.a_scale_rows = x_scale_rows;
    a.b_scale = w_scale;
    a.out = y;
    return product(BLOCK_FWD, xq, total_rows, D, wq, E, F, D, a, static_cast<cudaStream_t>(stream));
}

moe_status moe_grouped_linear_e4m3_block_backward(const uint8_t* dyq, const float* dy_scale, const uint8_t* dyq_seg,
                                                  const float* dy_scale_seg, const uint8_t* xq_seg, const float* x_scale_seg,
                                                  const int32_t* expert_offsets, int total_rows, const uint8_t* wq,
                                                  const float* w_scale, int E, int D, int F, moe_bf16* dx, moe_bf16* dw,
                                                  void* ws, size_t ws_bytes, void* stream) {
    moe_status s = check_block(total_rows, D, E, F);
    if (s != MOE_OK) return s;
    MAY(expert_offsets);
    MAY(dx);
    MAY(dw);
    if (!expert_offsets && E != 1) return refuse(MOE_ERR_INVALID_ARG, "expert_offsets is NULL with E=%d", E);
    if (!dx && !dw) return refuse(MOE_ERR_INVALID_ARG, "no output: dx and dw are NULL");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (total_rows == 0) return zero(dw, static_cast<size_t>(E) * D * F * 2, st);
    NEED_WS(kWsHeaderBytes);
    if (dx) {
        NEED(dyq);
        NEED(dy_scale);
        NEED(wq);
        NEED(w_scale);
    }
    if (dw) {
        NEED(dyq_seg);
        NEED(dy_scale_seg);
        NEED(xq_seg);
        NEED(x_scale_seg);
    }
    if (dx) {
        BlockArgs a = block_args(expert_offsets, E, total_rows, ws);
        a.M = total_rows;
        a.N = D;
        a.K = F;
        a.a_scale = dy_scale;
        a.a_scale_rows = total_rows;
        a.b_scale = w_scale;
        a.out = dx;
        s = product(BLOCK_DGRAD, dyq, total_rows, F, wq, E, F, D, a, st);
    }
    if (s == MOE_OK && dw) {
        const long long seg = segment_rows_of(total_rows, E);
        BlockArgs a = block_args(expert_offsets, E, total_rows, ws);
        a.M = F;
        a.N = D;
        a.a_scale = dy_scale_seg;
        a.b_scale = x_scale_seg;
        a.out = dw;
        s = product(BLOCK_WGRAD, dyq_seg, seg, F, xq_seg, 1, seg, D, a, st);
    }
    return s;
}

}  // extern "C"
