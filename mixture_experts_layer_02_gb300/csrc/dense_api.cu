// dense_api.cu -- the C entry points of the dense operators (include/moe.h):
// argument checks, workspace carving, the choice of kernel and the launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <cstring>

#include "../../include/moe.h"
#include "api_checks.h"
#include "dense.h"

using namespace moe;

namespace {

// Largest size of a dimension: rounded up to whole tiles, or walked past its end by a
// batch of steps (up to 1600 columns, dense_gemv.cu), it stays below 2^31.
constexpr int kDimLimit = 0x7fffffff - 4095;

// rows * width stays below 2^40, tile counts below 2^31
moe_status check_widths(int N, int D, int F) {
    if (N < 0) return refuse(MOE_ERR_INVALID_ARG, "N=%d < 0", N);
    if (std::max({N, D, F}) > kDimLimit)
        return refuse(MOE_ERR_INVALID_ARG, "N=%d, D=%d, F=%d: above %d", N, D, F, kDimLimit);
    if (D < 8 || D % 8) return refuse(MOE_ERR_INVALID_ARG, "D=%d not a positive multiple of 8", D);
    if (F < 8 || F % 8) return refuse(MOE_ERR_INVALID_ARG, "F=%d not a positive multiple of 8", F);
    if (static_cast<long long>(N) * std::max(D, F) >= (1LL << 40) || static_cast<long long>(D) * F >= (1LL << 40))
        return refuse(MOE_ERR_INVALID_ARG, "N=%d, D=%d, F=%d too large", N, D, F);
    return MOE_OK;
}

moe_status check_fn(int fn) {
    return fn < MOE_FN_NONE || fn > MOE_FN_GELU_TANH ? refuse(MOE_ERR_INVALID_ARG, "fn=%d outside 0..4", fn) : MOE_OK;
}

moe_status check_norm(int N, int D, float eps) {
    if (N < 0) return refuse(MOE_ERR_INVALID_ARG, "N=%d < 0", N);
    if (D < 8 || D % 8) return refuse(MOE_ERR_INVALID_ARG, "D=%d not a positive multiple of 8", D);
    if (D > kNormMaxD) return refuse(MOE_ERR_UNSUPPORTED, "D=%d above %d", D, kNormMaxD);
    if (!(eps >= 0.0f) || eps > 1e30f) return refuse(MOE_ERR_INVALID_ARG, "eps=%g is not a finite number >= 0", eps);
    return MOE_OK;
}

// byte offsets of the backward workspaces (the header first)
struct BackwardLayout {
    size_t d0, d1, total;
};

BackwardLayout backward_layout(int N, int F, int grads) {
    BackwardLayout l;
    const size_t one = up256(static_cast<size_t>(N) * F * 2);
    l.d0 = kWsHeaderBytes;
    l.d1 = l.d0 + one;
    l.total = l.d0 + one * grads;
    return l;
}

uint8_t* at(void* ws, size_t off) { return static_cast<uint8_t*>(ws) + off; }

// ---- the choice of kernel ----
// Estimated microseconds of the product alone: rounds over the clusters that fit
// the device, each k-blocks (64 of K) times the time of one, plus first load, join
// and epilogue.  Fitted to times measured on GB300 over 33 to 4096 rows and K of 768
// to 16384; whole tiles and pairs again over 24 products of 64 to 1792 tiles and K of
// 2 to 14336, most within 10 %, the worst 21 % off (4096 x 2048 x 768 gated: 29.3 for
// 24.2).  What the estimates leave out is the same for every form: the activation,
// a kept pre-activation (1001 x 4096 x 2056 takes 18 us, with bias, GELU and z 22.7),
// and the clock under the power limit.
struct TileKind {
    int bn;                                // 0: one CTA, 128 x 128; else a pair, 256 x bn
    double whole_block, whole;             // K whole: a k-block, the rest of a round
    double block, joined;                  // K in parts
};
constexpr TileKind kSplitTiles[3] = {{0, 0.24, 3.6, 0.24, 4.5}, {128, 0.206, 5.0, 0.206, 7.2}, {256, 0.325, 5.1, 0.30, 10.3}};
constexpr double kJoinRows = 2.5, kJoinEight = 1.0;  // one-CTA tiles: a join of all 128 rows, of eight parts
// Persistent pairs.  Over several rounds they beat whole 256 x 256 tiles, whose
// epilogue no main loop hides (4096^3 92 against 105 us, 4096 x 14336 x 4096 304
// against 314); in one round the whole tile ends earlier where K is short (weight
// gradient 777 x 1024 x 4096: 8.6 against 9.2).
constexpr double kPairBlock = 0.308, kPairRound = 2.0, kPairOnce = 5.7;
// The streamed form (M <= kGemvMaxRows) reads x once a block of 16 weight rows:
// weights at the HBM rate, or weights and x at the L2 rate that 240 blocks and
// more reach, whichever takes longer.  MB a microsecond is TB a second.
constexpr double kHbmRate = 6.3, kGemvL2Rate = 10.0, kGemvBlocks = 240.0, kGemvOnce = 2.4;

struct Plan {
    int bn, splits;  // split tiles
    int pairs;       // persistent pairs instead, where not 0
    bool stream;     // the streamed form instead
};

int env_int(const char* name, int dflt) {
    const char* f = getenv(name);
    return f ? atoi(f) : dflt;
}

// MOE_DENSE_KERNEL = 1 (split tiles), 2 (persistent pairs) or 3 (streamed weights,
// where M allows), and with it MOE_DENSE_SPLIT = 10 * bn + splits force a choice, for
// tuning and test coverage.  Parts that K does not allow fall back to one-CTA tiles
// with K whole.
moe_status plan_product(DenseKind kind, const DenseArgs& a, int kblocks, Plan* p) {
    const int n2 = kind == DENSE_GATED ? 128 : 256;
    const int kernel = env_int("MOE_DENSE_KERNEL", 0);
    *p = {0, 1, 0, false};
    const bool forward = kind == DENSE_GATED || kind == DENSE_LINEAR;
    const double weights = 2e-6 * a.N * a.K * (kind == DENSE_GATED ? 2 : 1);  // MB
    // up to eight rows x is at most half of what the weights are: nothing came near the streamed form
    if (forward && ((a.M <= 8 && kernel == 0) || (a.M <= kGemvMaxRows && kernel == 3))) {
        p->stream = true;
        return MOE_OK;
    }
    const int fixed = kernel ? env_int("MOE_DENSE_SPLIT", -1) : -1;
    double best = 1e30;
    for (const TileKind& t : kSplitTiles) {
        const int rows = t.bn ? 2 * kBM : kBM, width = (t.bn ? t.bn : 128) / (kind == DENSE_GATED ? 2 : 1);
        const long long tiles = static_cast<long long>((a.M + rows - 1) / rows) * ((a.N + width - 1) / width) * a.mats;
        // every part of K has work: an empty one would add what its accumulator held before
        for (int s = 1; s <= (t.bn ? 4 : 8) && s <= kblocks; s *= 2) {
            if (fixed >= 0 && fixed != 10 * t.bn + s) continue;
            int limit = 0;
            const moe_status st = launched(dense_split(kind, nullptr, a, t.bn, s, nullptr, &limit), "dense split limit");
            if (st != MOE_OK) return st;
            const double block = s == 1 ? t.whole_block : t.block;
            double rest = s == 1 ? t.whole : t.joined;
            if (s > 1 && t.bn == 0) rest += kJoinRows * std::min(a.M, kBM) / kBM + (s == 8 ? kJoinEight : 0.0);
            const double rounds = static_cast<double>((tiles + limit - 1) / limit);
            const double c = std::max(rounds * kblocks * block / s, forward ? weights / kHbmRate : 0.0) + rounds * rest;
            if (c < best) {
                best = c;
                p->bn = t.bn;
                p->splits = s;
            }
        }
    }
    if (kernel == 1) return MOE_OK;
    if (forward && a.M <= kGemvMaxRows && kernel == 0) {
        const int blocks = (a.N + (kind == DENSE_GATED ? 7 : 15)) / (kind == DENSE_GATED ? 8 : 16);
        const double l2 = weights + 2e-6 * blocks * a.M * a.K;
        const double c = kGemvOnce + std::max(weights / kHbmRate, l2 / (kGemvL2Rate * std::min(1.0, blocks / kGemvBlocks)));
        if (c < best) {
            best = c;
            p->stream = true;
        }
    }
    int limit = 0;
    const moe_status st = launched(dense_pair_limit(kind, &limit), "dense pair limit");
    if (st != MOE_OK) return st;
    const long long tiles =
        static_cast<long long>((a.M + kPairTile - 1) / kPairTile) * ((a.N + n2 - 1) / n2) * a.mats;
    const double c = static_cast<double>((tiles + limit - 1) / limit) * (kblocks * kPairBlock + kPairRound) + kPairOnce;
    if (c < best || kernel == 2) {
        p->stream = false;
        p->pairs = static_cast<int>(std::min<long long>(tiles, limit));
    }
    return MOE_OK;
}

}  // namespace

// One product: tensor maps, the choice of kernel, the launch.
int moe::dense_product(DenseKind kind, const DenseOperands& o, const DenseArgs& a, cudaStream_t st) {
    const bool a_mn = kind == DENSE_WGRAD, b_mn = kind == DENSE_DGRAD || kind == DENSE_WGRAD;
    const int kblocks = (a.K + kBK - 1) / kBK * a.segs;
    Plan p;
    const moe_status planned = plan_product(kind, a, kblocks, &p);
    if (planned != MOE_OK) return planned;
    if (p.stream) return launched(launch_dense_gemv(kind, o, a, st), "dense product launch");
    // K-major boxes: 128 rows of A; of B what one CTA loads at a time
    const int b_rows = p.pairs ? 128 : (p.bn ? p.bn / 2 : (kind == DENSE_GATED ? 64 : 128));
    CUtensorMap m[4];
    auto map_a = [&](CUtensorMap* t, const uint16_t* q) {
        return a_mn ? make_bf16_map(t, q, a.K, a.M, 64, o.lda) : make_bf16_map(t, q, a.M, a.K, kBM, o.lda);
    };
    auto map_b = [&](CUtensorMap* t, const uint16_t* q) {
        return b_mn ? make_bf16_map(t, q, a.K, a.N, 64) : make_bf16_map(t, q, a.N, a.K, b_rows);
    };
    int s = map_a(&m[0], o.a0);
    if (s == 0 && o.a1) s = map_a(&m[1], o.a1);
    if (s == 0) s = map_b(&m[2], o.b0);
    if (s == 0 && o.b1) s = map_b(&m[3], o.b1);
    if (s != 0) return static_cast<moe_status>(s);
    if (!o.a1) m[1] = m[0];
    if (!o.b1) m[3] = m[2];
    if (!p.pairs) return launched(dense_split(kind, m, a, p.bn, p.splits, st), "dense product launch");
    return launched(launch_dense_pair(kind, m, a, p.pairs, st), "dense pair product launch");
}

namespace {

moe_status product(DenseKind kind, const DenseOperands& o, const DenseArgs& a, cudaStream_t st) {
    return static_cast<moe_status>(dense_product(kind, o, a, st));
}

DenseArgs args_of(int M, int N, int K, void* ws) {
    DenseArgs a = {};
    a.M = M;
    a.N = N;
    a.K = K;
    a.segs = a.mats = 1;
    a.err = static_cast<uint32_t*>(ws);
    a.dbg = static_cast<const uint32_t*>(ws) + 1;
    return a;
}

// A gradient of no rows is zero.
moe_status zero(void* p, size_t bytes, cudaStream_t st) {
    return p ? launched(cudaMemsetAsync(p, 0, bytes, st), "zero gradient") : MOE_OK;
}

}  // namespace

// Workspace bytes of a dense operation, 0 for another name or invalid sizes.
size_t moe::dense_workspace_size(const char* op, int N, int D, int F) {
    if (!strcmp(op, "rmsnorm_backward")) {
        if (check_norm(N, D, 0.0f) != MOE_OK) return 0;
        return kWsHeaderBytes + up256(static_cast<size_t>(rmsnorm_bwd_parts(N, D)) * D * sizeof(float));
    }
    const bool gated = !strcmp(op, "gated_linear_backward");
    if (!strcmp(op, "gated_linear") || !strcmp(op, "linear"))
        return check_widths(N, D, F) == MOE_OK ? kWsHeaderBytes : 0;
    if (!gated && strcmp(op, "linear_backward")) return 0;
    if (check_widths(N, D, F) != MOE_OK) return 0;
    return backward_layout(N, F, gated ? 2 : 1).total;
}

extern "C" {

moe_status moe_rmsnorm(const moe_bf16* x, const moe_bf16* residual, const moe_bf16* weight, int N, int D, float eps,
                       moe_bf16* y, uint8_t* yq, float* y_scale, moe_bf16* residual_out, void* stream) {
    moe_status s = check_norm(N, D, eps);
    if (s != MOE_OK) return s;
    if (N == 0) return MOE_OK;
    NEED(x);
    MAY(residual);
    NEED(weight);
    MAY(y);
    MAY(yq);
    MAY(y_scale);
    MAY(residual_out);
    if (!y && !yq && !residual_out) return refuse(MOE_ERR_INVALID_ARG, "no output: y, yq and residual_out are NULL");
    if ((yq == nullptr) != (y_scale == nullptr)) return refuse(MOE_ERR_INVALID_ARG, "yq and y_scale come together");
    const NormArgs a = {x, residual, weight, y, yq, y_scale, residual_out, N, D, eps};
    return launched(launch_rmsnorm(a, static_cast<cudaStream_t>(stream)), "rmsnorm launch");
}

moe_status moe_rmsnorm_backward(const moe_bf16* dy, const moe_bf16* s_in, const moe_bf16* weight,
                                const moe_bf16* dresidual, int N, int D, float eps, moe_bf16* dx, float* dweight,
                                void* ws, size_t ws_bytes, void* stream) {
    moe_status s = check_norm(N, D, eps);
    if (s != MOE_OK) return s;
    MAY(dweight);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (N == 0) return zero(dweight, static_cast<size_t>(D) * sizeof(float), st);
    NEED(dy);
    NEED(s_in);
    NEED(weight);
    MAY(dresidual);
    NEED(dx);
    NEED_WS(dense_workspace_size("rmsnorm_backward", N, D, 0));
    const NormBwdArgs a = {dy, s_in, weight, dresidual, dx, dweight, reinterpret_cast<float*>(at(ws, kWsHeaderBytes)),
                           N, D, eps, static_cast<uint32_t*>(ws), static_cast<const uint32_t*>(ws) + 1};
    return launched(launch_rmsnorm_bwd(a, st), "rmsnorm backward launch");
}

moe_status moe_gated_linear(const moe_bf16* x, const moe_bf16* w1, const moe_bf16* w3, int N, int D, int F, int fn,
                            moe_bf16* h, moe_bf16* g, moe_bf16* u, void* ws, size_t ws_bytes, void* stream) {
    moe_status s = check_widths(N, D, F);
    if (s == MOE_OK) s = check_fn(fn);
    if (s != MOE_OK) return s;
    if (N == 0) return MOE_OK;
    NEED(x);
    NEED(w1);
    NEED(w3);
    NEED(h);
    MAY(g);
    MAY(u);
    NEED_WS(kWsHeaderBytes);
    DenseArgs a = args_of(N, F, D, ws);
    a.fn = fn;
    a.out0 = h;
    a.out1 = g;
    a.out2 = u;
    return product(DENSE_GATED, {x, nullptr, w1, w3}, a, static_cast<cudaStream_t>(stream));
}

moe_status moe_gated_linear_backward(const moe_bf16* dh, const moe_bf16* x, const moe_bf16* w1, const moe_bf16* w3,
                                     const moe_bf16* g, const moe_bf16* u, int N, int D, int F, int fn, moe_bf16* dx,
                                     moe_bf16* dw1, moe_bf16* dw3, void* ws, size_t ws_bytes, void* stream) {
    moe_status s = check_widths(N, D, F);
    if (s == MOE_OK) s = check_fn(fn);
    if (s != MOE_OK) return s;
    MAY(dx);
    MAY(dw1);
    MAY(dw3);
    if ((dw1 == nullptr) != (dw3 == nullptr)) return refuse(MOE_ERR_INVALID_ARG, "dw1 and dw3 come together");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (N == 0) {
        const size_t bytes = static_cast<size_t>(D) * F * 2;
        s = zero(dw1, bytes, st);
        return s == MOE_OK ? zero(dw3, bytes, st) : s;
    }
    NEED(dh);
    NEED(x);
    NEED(w1);
    NEED(w3);
    NEED(g);
    NEED(u);
    const BackwardLayout l = backward_layout(N, F, 2);
    NEED_WS(l.total);
    uint16_t* dg = reinterpret_cast<uint16_t*>(at(ws, l.d0));
    uint16_t* du = reinterpret_cast<uint16_t*>(at(ws, l.d1));
    s = launched(launch_gated_grad(dh, g, u, fn, static_cast<long long>(N) * F, dg, du, st), "gated gradient launch");
    if (s == MOE_OK && dx) {
        DenseArgs a = args_of(N, D, F, ws);
        a.segs = 2;
        a.out0 = dx;
        s = product(DENSE_DGRAD, {dg, du, w1, w3}, a, st);
    }
    if (s == MOE_OK && dw1) {
        DenseArgs a = args_of(F, D, N, ws);
        a.mats = 2;
        a.out0 = dw1;
        a.out1 = dw3;
        s = product(DENSE_WGRAD, {dg, du, x, nullptr}, a, st);
    }
    return s;
}

moe_status moe_linear(const moe_bf16* x, const moe_bf16* w, const float* bias, const moe_bf16* residual, int N, int D,
                      int F, int fn, moe_bf16* y, moe_bf16* z, void* ws, size_t ws_bytes, void* stream) {
    moe_status s = check_widths(N, D, F);
    if (s == MOE_OK) s = check_fn(fn);
    if (s != MOE_OK) return s;
    if (N == 0) return MOE_OK;
    NEED(x);
    NEED(w);
    MAY(bias);
    MAY(residual);
    NEED(y);
    MAY(z);
    NEED_WS(kWsHeaderBytes);
    DenseArgs a = args_of(N, F, D, ws);
    a.fn = fn;
    a.bias = bias;
    a.residual = residual;
    a.out0 = y;
    a.out1 = z;
    return product(DENSE_LINEAR, {x, nullptr, w, nullptr}, a, static_cast<cudaStream_t>(stream));
}

moe_status moe_linear_backward(const moe_bf16* dy, const moe_bf16* x, const moe_bf16* w, const moe_bf16* z, int N,
                               int D, int F, int fn, moe_bf16* dx, moe_bf16* dw, float* dbias, void* ws,
                               size_t ws_bytes, void* stream) {
    moe_status s = check_widths(N, D, F);
    if (s == MOE_OK) s = check_fn(fn);
    if (s != MOE_OK) return s;
    MAY(dx);
    MAY(dw);
    MAY(dbias);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (N == 0) {
        s = zero(dw, static_cast<size_t>(D) * F * 2, st);
        return s == MOE_OK ? zero(dbias, static_cast<size_t>(F) * sizeof(float), st) : s;
    }
    NEED(dy);
    NEED(x);
    NEED(w);
    if (fn != MOE_FN_NONE) NEED(z);
    const BackwardLayout l = backward_layout(N, F, 1);
    NEED_WS(l.total);
    uint16_t* dz = reinterpret_cast<uint16_t*>(at(ws, l.d0));
    s = launched(launch_linear_grad(dy, z, fn, N, F, dz, dbias, st),
                 "linear gradient launch");
    const uint16_t* grad = fn == MOE_FN_NONE ? dy : dz;
    if (s == MOE_OK && dx) {
        DenseArgs a = args_of(N, D, F, ws);
        a.out0 = dx;
        s = product(DENSE_DGRAD, {grad, nullptr, w, nullptr}, a, st);
    }
    if (s == MOE_OK && dw) {
        DenseArgs a = args_of(F, D, N, ws);
        a.out0 = dw;
        s = product(DENSE_WGRAD, {grad, nullptr, x, nullptr}, a, st);
    }
    return s;
}

}  // extern "C"
