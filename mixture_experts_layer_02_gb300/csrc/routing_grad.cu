// routing_grad.cu -- gradients of the layer's routing: of the weighted sum back to
// token order (moe_combine), of the sort by expert (moe_permute) and of the routing
// weights (moe_route).
//
//   combine   dy[inv[t,k]] = w[t,k] dout[t],   dw[t,k] = <dout[t], y[inv[t,k]]>
//   permute   dx[t] = dresidual[t] + sum_k dx_perm[inv[t,k]]
//   route     c = sum_j w_j dw_j,  dl_k = w_k (dw_k - c), with sigmoid scores times
//             1 - sigmoid(l_k): d log w_k / d l_j = [j = k] - w_j for the softmax over
//             the chosen, and log s has the slope 1 - s
//
// The first two move rows and are bound by HBM.  Both go by assignments, so dout is
// read through L1/L2 by the K warps of a token that run side by side, each row of y
// once, and nothing is summed through atomics: the order of additions is fixed by the
// sizes.  Measured: combine 4096 x 7168, K = 8, 154 us (999 MB, 6.5 TB/s: 96 % of what a
// copy reaches); permute 4093 x 4096, K = 2, with residual 22.6 us (134 MB, 5.9 TB/s).  The
// router's gradient is two products of dl (256 experts: 15 GFLOP each): as sparse sums they
// would gather 470 MB of W_gate's rows through L2.  4096 x 7168 x 256: 58 us, of which dl 5,
// dx 33 and dW_gate 21.  Sums are fp32; dy and dx are rounded once.  Coherent loads only (no const
// __restrict__): the launch before may still be writing them when blocks start.
#include <algorithm>

#include "activation.cuh"
#include "train.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

int sms() {
    int dev = 0, n = 152;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

__device__ __forceinline__ const uint4* row_of(const uint16_t* base, long long row, int D) {
    return reinterpret_cast<const uint4*>(base + row * D);
}

// W warps an assignment.  A warp has U 16-byte pieces of both rows in flight.
template <int W>
__global__ void __launch_bounds__(kThreads)
combine_bwd_kernel(const uint16_t* dout, const uint16_t* y, const int32_t* inv, const float* w, long long assignments, int D,
                   int K, long long rows, uint16_t* dy, float* dw, uint32_t* err) {
    constexpr int U = 4;
    __shared__ float s_part[kWarps];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % W;
    const long long a = static_cast<long long>(blockIdx.x) * (kWarps / W) + warp / W;
    float sum = 0.0f;
    if (a < assignments) {
        const long long r = inv[a];
        if (r >= 0 && r < rows) {
            const uint4* g = row_of(dout, a / K, D);
            const uint4* v = dw ? row_of(y, r, D) : g;
            uint4* o = dy ? reinterpret_cast<uint4*>(dy + r * D) : nullptr;
            const float weight = w[a];
            const int chunks = D / 8;
            float acc[U] = {};
            for (int c0 = part * 32 + lane; c0 < chunks; c0 += U * W * 32) {
                uint4 gv[U], vv[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * W * 32;
                    gv[u] = c < chunks ? g[c] : make_uint4(0, 0, 0, 0);
                    if (dw) vv[u] = c < chunks ? v[c] : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * W * 32;
                    float gf[8];
                    unpack_bf16x8(gv[u], gf);
                    if (dw) {
                        float vf[8];
                        unpack_bf16x8(vv[u], vf);
#pragma unroll
                        for (int j = 0; j < 8; ++j) acc[u] = fmaf(gf[j], vf[j], acc[u]);
                    }
                    if (o && c < chunks) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) gf[j] *= weight;
                        o[c] = pack_bf16x8(gf);
                    }
                }
            }
            sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        } else if (r != -1 && part == 0 && lane == 0) {
            record_error(err, MOE_DEVERR_BOUNDS);
        }
    }
    pdl_trigger();
    if (dw == nullptr) return;  // the same for the whole grid
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if constexpr (W > 1) {
        if (lane == 0) s_part[warp] = sum;
        __syncthreads();
#pragma unroll
        for (int i = 1; i < W; ++i) sum += part == 0 ? s_part[warp + i] : 0.0f;
    }
    if (part == 0 && lane == 0 && a < assignments) dw[a] = sum;
}

// A warp takes a slice of a token's row: the K rows of an octet of columns are in
// flight together and summed in k order.
template <int KMAX>
__global__ void __launch_bounds__(kThreads)
permute_bwd_kernel(const uint16_t* dx_perm, const int32_t* inv, const uint16_t* dresidual, int N, int D, int K, int slices,
                   long long rows, uint16_t* dx, uint32_t* err) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (item >= static_cast<long long>(N) * slices) return;
    const long long t = item / slices;
    const int slice = static_cast<int>(item - t * slices);
    const int chunks = D / 8, per = (chunks + slices - 1) / slices;
    const int c0 = slice * per, c1 = min(chunks, c0 + per);
    int mine = -1;
    if (lane < K) {
        mine = inv[t * K + lane];
        if (mine < 0 || mine >= rows) {
            if (mine != -1 && slice == 0) record_error(err, MOE_DEVERR_BOUNDS);
            mine = -1;
        }
    }
    int r[KMAX];
#pragma unroll
    for (int k = 0; k < KMAX; ++k) r[k] = __shfl_sync(0xffffffffu, mine, k);
    for (int c = c0 + lane; c < c1; c += 32) {
        uint4 v[KMAX];
#pragma unroll
        for (int k = 0; k < KMAX; ++k)
            if (k < K && r[k] >= 0) v[k] = row_of(dx_perm, r[k], D)[c];
        float sum[8] = {};
        if (dresidual) unpack_bf16x8(row_of(dresidual, t, D)[c], sum);
#pragma unroll
        for (int k = 0; k < KMAX; ++k) {
            if (k >= K || r[k] < 0) continue;
            float f[8];
            unpack_bf16x8(v[k], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += f[j];
        }
        reinterpret_cast<uint4*>(dx + t * D)[c] = pack_bf16x8(sum);
    }
    pdl_trigger();
}

// A block owns eight tokens, a warp each.  Their rows of dl are built in shared memory in fp32 (a
// token may name an expert twice: its first lane adds up the others, in order),
// leave as bf16 (an operand of tensor-core products) and are summed over the
// tokens, unrounded and in order, for dbias.
__global__ void __launch_bounds__(kThreads)
route_bwd_kernel(const RouteBwdArgs a) {
    extern __shared__ float s_row[];  // [tokens][ld]
    for (int i = threadIdx.x; i < kRouteBwdTokens * a.ld; i += kThreads) s_row[i] = 0.0f;
    pdl_wait();
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    static_assert(kRouteBwdTokens == kWarps, "a warp a token");
    const int t0 = static_cast<int>(blockIdx.x) * kRouteBwdTokens, tokens = min(kRouteBwdTokens, a.N - t0);
    if (const int i = warp; i < tokens) {
        const long long t = t0 + i, at = t * a.K + lane;
        const bool on = lane < a.K;
        int id = on ? a.ids[at] : -1;
        const float w = on ? a.w[at] : 0.0f, d = on ? a.dw[at] : 0.0f;
        if (on && static_cast<unsigned>(id) >= static_cast<unsigned>(a.E)) {
            record_error(a.err, MOE_DEVERR_BOUNDS);
            id = -1;
        }
        float c = id >= 0 ? w * d : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
        float g = id >= 0 ? w * (d - c) : 0.0f;
        if (a.sigmoid && id >= 0) g /= 1.0f + expf(a.logits[t * a.E + id]);  // times 1 - sigmoid
        float sum = g;
        bool first = id >= 0;
        for (int k = 0; k < a.K; ++k) {
            const int other = __shfl_sync(0xffffffffu, id, k);
            const float v = __shfl_sync(0xffffffffu, g, k);
            if (other != id || k == lane) continue;
            if (k < lane) first = false;
            else sum += v;
        }
        if (first) s_row[i * a.ld + id] = sum;
    }
    __syncthreads();
    const int octets = a.ld / 8;
    for (int i = threadIdx.x; i < tokens * octets; i += kThreads) {
        const int r = i / octets, o = i - r * octets;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = s_row[r * a.ld + o * 8 + j];
        reinterpret_cast<uint4*>(a.dl + static_cast<long long>(t0 + r) * a.ld)[o] = pack_bf16x8(v);
    }
    if (a.dbias)
        for (int e = threadIdx.x; e < a.E; e += kThreads) {
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < kRouteBwdTokens; ++i) v += s_row[i * a.ld + e];  // rows past the last token are zero
            a.partial[static_cast<long long>(blockIdx.x) * a.E + e] = v;
        }
    pdl_trigger();
}

// 32 experts a block, 32 threads an expert: thread y sums parts y, y + 32, ... in
// order, then the 32 sums are added in order.
__global__ void __launch_bounds__(1024)
dbias_kernel(const float* partial, long long parts, int E, float* dbias) {
    __shared__ float s[32][33];
    pdl_wait();
    const int e = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
    float v = 0.0f;
    if (e < E)
#pragma unroll 4
        for (long long p = y; p < parts; p += 32) v += partial[p * E + e];
    s[y][threadIdx.x & 31] = v;
    __syncthreads();
    if (y == 0 && e < E) {
#pragma unroll
        for (int i = 1; i < 32; ++i) v += s[i][threadIdx.x & 31];
        dbias[e] = v;
    }
    pdl_trigger();
}

template <int W>
cudaError_t combine_bwd_go(const uint16_t* dout, const uint16_t* y, const int32_t* inv, const float* w, long long n, int D,
                           int K, long long rows, uint16_t* dy, float* dw, uint32_t* err, cudaStream_t st) {
    const long long per = kWarps / W;
    return launch_kernel(combine_bwd_kernel<W>, dim3(static_cast<unsigned>((n + per - 1) / per)), dim3(kThreads), 0, st, dout,
                         y, inv, w, n, D, K, rows, dy, dw, err);
}

}  // namespace

cudaError_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y, const int32_t* inv, const float* w, int N, int D,
                               int K, long long rows, uint16_t* dy, float* dw, uint32_t* err, cudaStream_t st) {
    // enough warps for the GPU, each with at least a whole step of its row
    const long long n = static_cast<long long>(N) * K, want = static_cast<long long>(sms()) * 32;
    if (n >= want || D <= 1024) return combine_bwd_go<1>(dout, y, inv, w, n, D, K, rows, dy, dw, err, st);
    if (2 * n >= want || D <= 2048) return combine_bwd_go<2>(dout, y, inv, w, n, D, K, rows, dy, dw, err, st);
    if (4 * n >= want || D <= 4096) return combine_bwd_go<4>(dout, y, inv, w, n, D, K, rows, dy, dw, err, st);
    return combine_bwd_go<8>(dout, y, inv, w, n, D, K, rows, dy, dw, err, st);
}

cudaError_t launch_permute_bwd(const uint16_t* dx_perm, const int32_t* inv, const uint16_t* dresidual, int N, int D, int K,
                               long long rows, uint16_t* dx, uint32_t* err, cudaStream_t st) {
    const long long want = static_cast<long long>(sms()) * 64;
    const int slices = static_cast<int>(std::max<long long>(1, std::min<long long>((want + N - 1) / N, D / 8 / 32)));
    const long long grid = (static_cast<long long>(N) * slices + kWarps - 1) / kWarps;
    auto kern = K <= 2 ? permute_bwd_kernel<2> : K <= 8 ? permute_bwd_kernel<8> : permute_bwd_kernel<32>;
    return launch_kernel(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, st, dx_perm, inv, dresidual, N, D, K,
                         slices, rows, dx, err);
}

cudaError_t launch_route_bwd(const RouteBwdArgs& a, cudaStream_t st) {
    const size_t smem = static_cast<size_t>(kRouteBwdTokens) * a.ld * sizeof(float);  // at most 32 KB
    const long long parts = route_bwd_parts(a.N);
    const cudaError_t e = launch_kernel(route_bwd_kernel, dim3(static_cast<unsigned>(parts)), dim3(kThreads), smem, st, a);
    if (e != cudaSuccess || !a.dbias) return e;
    return launch_kernel(dbias_kernel, dim3((a.E + 31) / 32), dim3(1024), 0, st, a.partial, parts, a.E, a.dbias);
}

}  // namespace moe
