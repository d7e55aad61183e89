// rmsnorm.cu -- root-mean-square norm with the residual's addition and an e4m3
// output, and its gradient.
//
//   s = x + residual          (fp32; stored in bf16 as the new residual stream)
//   y_j = s_j w_j / sqrt(mean_j s_j^2 + eps)
//   q = e4m3(y 2^-k), scale = 2^k, k = the smallest integer >= -126 with
//       max|y| <= 448 2^k (the row rule of quant.cu, applied to the fp32 y, so
//       a code has been rounded once)
//
// Bound by HBM: 40.7 us at 4096 x 7168 with residual, bf16 and e4m3 outputs (6.5
// TB/s), 2.4 us for one row.  Every row is read once and held in registers between
// its sums and its outputs; up to 1024 wide a warp takes a row, then a block of 256
// (to 8192) or 1024 threads.  The sum of squares and the row's maximum come out of ONE reduction:
// y_j is formed as fl(fl(s_j w_j) r) with r > 0 and rounding is monotone, so
// max|y| = fl(max|fl(s_j w_j)| r) exactly.
//
// Every global load here is a coherent one (no __ldg, no const __restrict__): the
// launch before may still be writing what this one reads when its blocks start.
#include <algorithm>
#include <atomic>

#include "activation.cuh"
#include "dense.h"
#include "quant.cuh"
#include "settle.cuh"

namespace moe {

// k from the fp32 bits of the row maximum (as scale_exp_of for bf16):
// 448 = 1.75 * 2^8, fraction field of 1.75 = 0x600000.
__device__ __forceinline__ int scale_exp_of_f32(uint32_t m) {
    const int ef = static_cast<int>(m >> 23);
    return (ef == 0) ? -126 : max(-126, ef - 127 - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0));
}

// Sum of `a` and maximum of `m` (bits of non-negative floats; a NaN is larger
// than any number) over the T threads of a row.  T = 32: one warp.
template <int T>
__device__ __forceinline__ void row_reduce(float& a, uint32_t& m, float* s_a, uint32_t* s_m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if constexpr (T > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) {
            s_a[warp] = a;
            s_m[warp] = m;
        }
        __syncthreads();
        a = 0.0f;
        m = 0;
#pragma unroll
        for (int w = 0; w < T / 32; ++w) {
            a += s_a[w];
            m = max(m, s_m[w]);
        }
        __syncthreads();  // the arrays are rewritten for the next row
    }
}

// The weight, which every row reads again, among rows that are read once: kept in
// L1 first.  Without the hint 42.5 instead of 41.2 us at 4096 x 7168.
__device__ __forceinline__ uint4 ld_kept(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.L1::evict_last.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// T threads a row (32: eight rows in a block of 256), V 16-byte chunks a thread.
template <int T, int V>
__global__ void __launch_bounds__(T < 256 ? 256 : T)
rmsnorm_kernel(const NormArgs a) {
    __shared__ float s_a[T / 32];
    __shared__ uint32_t s_m[T / 32];
    constexpr int ROWS = T == 32 ? 8 : 1;
    const int lane = T == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int chunks = a.D >> 3;
    pdl_wait();
    const uint4* wrow = reinterpret_cast<const uint4*>(a.weight);
    const float inv_d = 1.0f / static_cast<float>(a.D);
    for (long long r = static_cast<long long>(blockIdx.x) * ROWS + (T == 32 ? threadIdx.x >> 5 : 0); r < a.rows;
         r += static_cast<long long>(gridDim.x) * ROWS) {
        const long long at = r * chunks;
        const uint4* xr = reinterpret_cast<const uint4*>(a.x) + at;
        const uint4* rr = reinterpret_cast<const uint4*>(a.residual) + at;
        uint4 xv[V], rv[V], wv[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = lane + i * T;
            const bool in = c < chunks;
            xv[i] = in ? xr[c] : make_uint4(0, 0, 0, 0);
            rv[i] = in && a.residual ? rr[c] : make_uint4(0, 0, 0, 0);
            wv[i] = in ? ld_kept(wrow + c) : make_uint4(0, 0, 0, 0);
        }
        float sw[V][8];
        float sum = 0.0f;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float s[8], b[8], w[8];
            unpack_bf16x8(xv[i], s);
            unpack_bf16x8(rv[i], b);
            unpack_bf16x8(wv[i], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[j] += b[j];
                sum += s[j] * s[j];
                sw[i][j] = s[j] * w[j];
                top = max(top, __float_as_uint(sw[i][j]) & 0x7fffffffu);
            }
            const int c = lane + i * T;
            if (a.residual_out && c < chunks) reinterpret_cast<uint4*>(a.residual_out)[at + c] = pack_bf16x8(s);
        }
        row_reduce<T>(sum, top, s_a, s_m);
        const float rstd = 1.0f / sqrtf(sum * inv_d + a.eps);
        float inv = 0.0f;
        if (a.yq) {
            const int k = scale_exp_of_f32(__float_as_uint(__uint_as_float(top) * rstd) & 0x7fffffffu);
            inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);  // 2^-k
            if (lane == 0) a.y_scale[r] = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = lane + i * T;
            if (c >= chunks) continue;
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = sw[i][j] * rstd;
            if (a.y) reinterpret_cast<uint4*>(a.y)[at + c] = pack_bf16x8(y);
            if (a.yq) {
                const uint32_t p0 = fp8x2(y[0] * inv, y[1] * inv), p1 = fp8x2(y[2] * inv, y[3] * inv);
                const uint32_t p2 = fp8x2(y[4] * inv, y[5] * inv), p3 = fp8x2(y[6] * inv, y[7] * inv);
                reinterpret_cast<uint2*>(a.yq)[at + c] = make_uint2(p0 | (p1 << 16), p2 | (p3 << 16));
            }
        }
    }
    pdl_trigger();
}

namespace {

int sms() {
    int dev = 0, n = 152;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

template <int T, int V>
cudaError_t norm_go(const NormArgs& a, cudaStream_t st) {
    constexpr int rows = T == 32 ? 8 : 1, threads = T < 256 ? 256 : T;
    const long long want = (a.rows + rows - 1) / rows;
    const int grid = static_cast<int>(std::min<long long>(want, static_cast<long long>(sms()) * (2048 / threads)));
    return launch_kernel(rmsnorm_kernel<T, V>, dim3(grid), dim3(threads), 0, st, a);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t st) {
    if (a.rows <= 0) return cudaSuccess;
    const int chunks = a.D >> 3;
    if (chunks <= 32) return norm_go<32, 1>(a, st);
    if (chunks <= 64) return norm_go<32, 2>(a, st);
    if (chunks <= 128) return norm_go<32, 4>(a, st);
    if (chunks <= 256) return norm_go<256, 1>(a, st);
    if (chunks <= 512) return norm_go<256, 2>(a, st);
    if (chunks <= 1024) return norm_go<256, 4>(a, st);
    if (chunks <= 1024 * 2) return norm_go<1024, 2>(a, st);
    return norm_go<1024, 4>(a, st);
}

// ----------------------------------------------------------------------------
// Gradient.  With v = dy w and r = 1 / sqrt(mean s^2 + eps):
//   dx_j = r v_j - s_j r^3 mean_i(v_i s_i) (+ dresidual_j),   dw_j = sum over rows of dy_j s_j r.
// r is computed again from s, which is read anyway: one reduction gives both
// sums.  A group of threads keeps its columns' dw sums in registers over all
// its rows and stores them once; a second kernel adds the groups' rows in a
// fixed order, so the result does not change from run to run.
//
// Bound by HBM (8 bytes an element) once two things are out of the way.  A
// block that loads a row, reduces it and stores it leaves the memory idle in
// between: rows arrive by bulk copies into a ring of stages in shared memory,
// ahead of their use.  And 512 threads on one row spend more instructions on
// the reduction than on the row (2.3 us a row at 4096): here a group of T
// threads with up to 4 chunks each owns a row, several groups share a block,
// and each runs on its own ring and its own barrier, so one group's reduction
// overlaps another's arithmetic.  With two chunks a thread a row stays packed in
// registers over that barrier, which then frees its stage for the next copy;
// with four (rows above 8192; registers would spill: 46 us instead of 28 at
// 4093 x 4096) it is read from the stage again and the next row's barrier frees it.
// The arithmetic is done on pairs (fma.rn.f32x2), which halves it.  Measured: 4093
// x 4096 26.5 us (5.1 TB/s; the second kernel is 3 us of it), 16384 x 7168 140 us
// (6.7 TB/s).
struct NormBwdShape {
    int v;         // 16-byte chunks a thread: 1, 2 or 4
    int threads;   // T: threads of a group (a multiple of 32)
    int groups;    // per block
    int stages;    // rows of s, dy and dresidual each group holds
    int grid;      // blocks, and fp32 rows of dweight sums
};

constexpr int kNormBwdSms = 152;         // the grid does not depend on the device
constexpr int kNormBwdThreads = 512;
constexpr size_t kNormBwdSmem = 220 * 1024;

// Up to 16384 wide two rows a group fit the shared memory of an SM; a wider
// row (stages = 0) is loaded straight into registers.
NormBwdShape norm_bwd_shape(long long rows, int D) {
    NormBwdShape s;
    const int chunks = D >> 3;
    s.v = chunks <= 32 ? 1 : (chunks <= 1024 ? 2 : 4);
    s.threads = ((chunks + s.v - 1) / s.v + 31) / 32 * 32;
    s.groups = std::max(1, kNormBwdThreads / s.threads);
    s.stages = 0;
    if (s.threads <= kNormBwdThreads)
        s.stages = static_cast<int>(std::min<size_t>(8, kNormBwdSmem / (static_cast<size_t>(s.groups) * D * 2 * 3)));
    const long long steps = (std::max<long long>(rows, 1) + s.groups - 1) / s.groups;
    s.grid = static_cast<int>(std::min<long long>(steps, kNormBwdSms));
    return s;
}

__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w)); }

template <int V>
__global__ void __launch_bounds__(kNormBwdThreads, 1)
rmsnorm_bwd_ring_kernel(const NormBwdArgs a, const NormBwdShape sh) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 s_sum[2][kNormBwdThreads / 32];
    __shared__ uint64_t s_full[kNormBwdThreads / 32 * 8];
    __shared__ int s_abort;
    const int chunks = a.D >> 3, T = sh.threads, warps = T >> 5;
    const int group = threadIdx.x / T, lane = threadIdx.x - group * T;
    const uint32_t row_bytes = static_cast<uint32_t>(a.D) * 2;
    const int arrays = a.dresidual ? 3 : 2;
    uint64_t* full = s_full + group * sh.stages;
    uint8_t* mine = ring + static_cast<size_t>(group) * sh.stages * 3 * row_bytes;
    if (threadIdx.x == 0) {
        for (int i = 0; i < sh.groups * sh.stages; ++i) mbar_init(&s_full[i], 1);
        s_abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    pdl_wait();
    const long long row0 = static_cast<long long>(blockIdx.x) * sh.groups + group;
    const long long step = static_cast<long long>(gridDim.x) * sh.groups;
    auto fill = [&](long long i) {  // lane 0 of the group: row i of its list into its stage
        const long long r = row0 + i * step;
        if (r >= a.rows) return;
        const int st = static_cast<int>(i % sh.stages);
        uint8_t* at = mine + static_cast<size_t>(st) * 3 * row_bytes;
        mbar_arrive_expect_tx(&full[st], row_bytes * arrays);
        bulk_load_1d(at, a.s + r * a.D, row_bytes, &full[st]);
        bulk_load_1d(at + row_bytes, a.dy + r * a.D, row_bytes, &full[st]);
        if (a.dresidual) bulk_load_1d(at + 2 * row_bytes, a.dresidual + r * a.D, row_bytes, &full[st]);
    };
    if (lane == 0) {
        const bool first = row0 == 0;  // only this group reads the test hook: it is a load ahead of a copy
        for (int i = first ? 1 : 0; i < sh.stages; ++i) fill(i);
        if (first && !(*a.dbg & MOE_DBG_WITHHOLD_FIRST_LOAD)) fill(0);
    }
    uint4 wv[V];
    float2 dw[V][4];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int c = lane + k * T;
        wv[k] = c < chunks ? reinterpret_cast<const uint4*>(a.weight)[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[k][j] = make_float2(0.0f, 0.0f);
    }
    const float inv_d = 1.0f / static_cast<float>(a.D);
    int stage = 0;
    uint32_t phase = 0;
    // A wait that ran out is recorded and ends its group's copies: a stage is filled
    // again only after it was seen full.  The rows left are walked through all the same
    // (no wait takes time any more).
    long long i = 0;
    bool live = true;
    for (long long r = row0; r < a.rows; r += step, ++i) {
        live = mbar_wait(&full[stage], phase, &s_abort, a.err) && live;
        const uint4* ps = reinterpret_cast<const uint4*>(mine + static_cast<size_t>(stage) * 3 * row_bytes);
        const uint4* pd = ps + chunks;
        const uint4* pe = pd + chunks;
        constexpr bool KEEP = V <= 2;
        uint4 sv[V], dv[V], ev[V];
        float2 ss = make_float2(0.0f, 0.0f), vv = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = lane + k * T;
            const bool in = c < chunks;
            sv[k] = in ? ps[c] : make_uint4(0, 0, 0, 0);
            dv[k] = in ? pd[c] : make_uint4(0, 0, 0, 0);
            if (KEEP) ev[k] = in && arrays == 3 ? pe[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 s = bf16_pair(word_of(sv[k], j)), d = bf16_pair(word_of(dv[k], j));
                ss = fma2(s, s, ss);
                vv = fma2(mul2(d, bf16_pair(word_of(wv[k], j))), s, vv);
            }
        }
        float s2 = ss.x + ss.y, vs = vv.x + vv.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s2 += __shfl_xor_sync(0xffffffffu, s2, o);
            vs += __shfl_xor_sync(0xffffffffu, vs, o);
        }
        if (warps > 1) {
            float2* sums = s_sum[i & 1] + group * warps;  // two sets: the next row's sums overwrite none still being read
            if ((lane & 31) == 0) sums[lane >> 5] = make_float2(s2, vs);
            named_barrier_sync(1 + group, T);
            s2 = vs = 0.0f;
            for (int k = 0; k < warps; ++k) {
                const float2 p = sums[k];
                s2 += p.x;
                vs += p.y;
            }
        } else {
            __syncwarp();
        }
        if (lane == 0 && live) {
            if (KEEP) fill(i + sh.stages);  // every thread holds its part of this stage
            else if (i > 0) fill(i - 1 + sh.stages);  // every thread has left the previous row's stage
        }
        const float rstd = 1.0f / sqrtf(s2 * inv_d + a.eps);
        const float back = -rstd * (rstd * (vs * inv_d));
        const float2 r2 = make_float2(rstd, rstd), b2 = make_float2(back, back);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = lane + k * T;
            uint32_t o[4];
            if (!KEEP) {
                if (c >= chunks) continue;
                sv[k] = ps[c];
                dv[k] = pd[c];
                ev[k] = arrays == 3 ? pe[c] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 s = bf16_pair(word_of(sv[k], j)), d = bf16_pair(word_of(dv[k], j));
                dw[k][j] = fma2(d, mul2(s, r2), dw[k][j]);
                const float2 dx = fma2(r2, fma2(s, b2, mul2(d, bf16_pair(word_of(wv[k], j)))), bf16_pair(word_of(ev[k], j)));
                o[j] = pack_bf16x2(dx.x, dx.y);
            }
            if (c < chunks) reinterpret_cast<uint4*>(a.dx)[r * chunks + c] = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (++stage == sh.stages) { stage = 0; phase ^= 1u; }
    }
    if (s_abort) settle_copies();
    pdl_trigger();
    if (a.dweight) {  // the groups' sums, added in group order
        __syncthreads();  // no copy is in flight: every filled stage has been waited for
        float* all = reinterpret_cast<float*>(ring);
        if (group < sh.groups)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int c = lane + k * T;
                if (c >= chunks) continue;
                float4* p = reinterpret_cast<float4*>(all + static_cast<size_t>(group) * a.D + c * 8);
                p[0] = make_float4(dw[k][0].x, dw[k][0].y, dw[k][1].x, dw[k][1].y);
                p[1] = make_float4(dw[k][2].x, dw[k][2].y, dw[k][3].x, dw[k][3].y);
            }
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
            float v = all[c];
            for (int g = 1; g < sh.groups; ++g) v += all[static_cast<size_t>(g) * a.D + c];
            a.partial[static_cast<long long>(blockIdx.x) * a.D + c] = v;
        }
    }
}

// Rows wider than the ring takes: one block a row, loaded into registers.
template <int T, int V>
__global__ void __launch_bounds__(T)
rmsnorm_bwd_wide_kernel(const NormBwdArgs a) {
    __shared__ float s_a[T / 32], s_b[T / 32];
    const int chunks = a.D >> 3;
    const int warp = threadIdx.x >> 5;
    pdl_wait();
    const uint4* wrow = reinterpret_cast<const uint4*>(a.weight);
    const float inv_d = 1.0f / static_cast<float>(a.D);
    float dw[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const uint4* sr = reinterpret_cast<const uint4*>(a.s) + r * chunks;
        const uint4* dr = reinterpret_cast<const uint4*>(a.dy) + r * chunks;
        uint4 sv[V], dv[V];
        float s2 = 0.0f, vs = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            const bool in = c < chunks;
            sv[i] = in ? sr[c] : make_uint4(0, 0, 0, 0);
            dv[i] = in ? dr[c] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            float s[8], d[8], w[8];
            unpack_bf16x8(sv[i], s);
            unpack_bf16x8(dv[i], d);
            unpack_bf16x8(c < chunks ? wrow[c] : make_uint4(0, 0, 0, 0), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s2 += s[j] * s[j];
                vs += d[j] * w[j] * s[j];
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s2 += __shfl_xor_sync(0xffffffffu, s2, o);
            vs += __shfl_xor_sync(0xffffffffu, vs, o);
        }
        if ((threadIdx.x & 31) == 0) {
            s_a[warp] = s2;
            s_b[warp] = vs;
        }
        __syncthreads();
        s2 = vs = 0.0f;
#pragma unroll
        for (int w = 0; w < T / 32; ++w) {
            s2 += s_a[w];
            vs += s_b[w];
        }
        __syncthreads();
        const float rstd = 1.0f / sqrtf(s2 * inv_d + a.eps);
        const float back = rstd * (rstd * (vs * inv_d));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            if (c >= chunks) continue;
            float s[8], d[8], w[8], e[8], dx[8];
            unpack_bf16x8(sv[i], s);
            unpack_bf16x8(dv[i], d);
            unpack_bf16x8(wrow[c], w);
            unpack_bf16x8(a.dresidual ? reinterpret_cast<const uint4*>(a.dresidual)[r * chunks + c] : make_uint4(0, 0, 0, 0), e);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[i][j] += d[j] * (s[j] * rstd);
                dx[j] = rstd * (d[j] * w[j] - s[j] * back) + e[j];
            }
            reinterpret_cast<uint4*>(a.dx)[r * chunks + c] = pack_bf16x8(dx);
        }
    }
    pdl_trigger();
    if (a.dweight) {
        float4* p = reinterpret_cast<float4*>(a.partial + static_cast<long long>(blockIdx.x) * a.D);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * T;
            if (c >= chunks) continue;
            p[2 * c] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            p[2 * c + 1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
}

// 32 columns a block, 32 threads a column: thread y sums parts y, y + 32, ... in
// order, then the 32 sums are added in order.
__global__ void __launch_bounds__(1024)
column_sums_kernel(const float* partial, int parts, int cols, float* out) {
    __shared__ float s[32][33];
    pdl_wait();
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
    float v = 0.0f;
    if (col < cols)
#pragma unroll 8
        for (int p = y; p < parts; p += 32) v += partial[static_cast<long long>(p) * cols + col];
    s[y][threadIdx.x & 31] = v;
    __syncthreads();
    if (y == 0 && col < cols) {
#pragma unroll
        for (int i = 1; i < 32; ++i) v += s[i][threadIdx.x & 31];
        out[col] = v;
    }
    pdl_trigger();
}

int rmsnorm_bwd_parts(long long rows, int D) { return norm_bwd_shape(rows, D).grid; }

namespace {

template <int V>
cudaError_t ring_go(const NormBwdArgs& a, const NormBwdShape& s, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(rmsnorm_bwd_ring_kernel<V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kNormBwdSmem));
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    const size_t smem = static_cast<size_t>(s.stages) * s.groups * a.D * 2 * 3;
    return launch_kernel(rmsnorm_bwd_ring_kernel<V>, dim3(s.grid), dim3(s.threads * s.groups), smem, st, a, s);
}

}  // namespace

cudaError_t launch_rmsnorm_bwd(const NormBwdArgs& a, cudaStream_t st) {
    if (a.rows <= 0) return cudaSuccess;
    const NormBwdShape s = norm_bwd_shape(a.rows, a.D);
    cudaError_t e;
    if (s.stages < 1) e = launch_kernel(rmsnorm_bwd_wide_kernel<1024, 4>, dim3(s.grid), dim3(1024), 0, st, a);
    else if (s.v == 1) e = ring_go<1>(a, s, st);
    else if (s.v == 2) e = ring_go<2>(a, s, st);
    else e = ring_go<4>(a, s, st);
    if (e != cudaSuccess || !a.dweight) return e;
    return launch_kernel(column_sums_kernel, dim3((a.D + 31) / 32), dim3(1024), 0, st, a.partial, s.grid, a.D, a.dweight);
}

}  // namespace moe
