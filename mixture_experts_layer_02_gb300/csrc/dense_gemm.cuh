// dense_gemm.cuh -- pieces shared by the dense tensor-core products: operand
// layouts, descriptors and the fused epilogues.
#pragma once

#include "activation.cuh"
#include "dense.h"
#include "gemm_common.cuh"
#include "settle.cuh"

namespace moe {

// How a kind stores its operands.  K-major: rows m (or n), K contiguous, one
// TMA box of 64 K x R rows a k-block.  MN-major: rows k, M (or N) contiguous,
// one box of 64 columns x 64 k-rows (8 KB) for each 64 columns.  Nothing is
// transposed in memory: the gradient products read the weights, activations
// and incoming gradients as the forward pass stored them.
template <int KIND>
struct DenseLayout {
    static constexpr bool A_MN = KIND == DENSE_WGRAD;
    static constexpr bool B_MN = KIND == DENSE_DGRAD || KIND == DENSE_WGRAD;
    static constexpr bool GATED = KIND == DENSE_GATED;
};

constexpr int kMnBlockBytes = 64 * kRowBytes;  // one MN-major box: 64 k-rows of 64 columns

// Shared-memory descriptor of an MN-major operand written by TMA with 128-byte
// swizzle: each k-row holds 64 consecutive M/N elements (128 bytes), 8 k-rows
// are a 1024-byte swizzle atom (stride offset), the next 64 M/N elements start
// one box further (leading offset).  A step of 16 along K is two atoms.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(kMnBlockBytes >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
    return MN ? sw128_mnmajor_desc(saddr) : sw128_kmajor_desc(saddr);
}
// descriptor step (16-byte units) of one MMA's 16 K elements
template <bool MN>
constexpr uint64_t kDescStep = MN ? (2 * 1024) >> 4 : 32 >> 4;

template <int KIND>
__host__ __device__ constexpr uint32_t dense_idesc(int M, int N) {
    return idesc_bf16_f32(M, N) | (DenseLayout<KIND>::A_MN ? 1u << 15 : 0u) | (DenseLayout<KIND>::B_MN ? 1u << 16 : 0u);
}

// ---- waiting ----
// Waits on an mbarrier are polls, and polls of one SM queue up behind one
// another: with six to eight warps polling for the end of a main loop, each wait
// and each copy of its producer took about 370 clocks (time stamps), 730 a
// k-block of 256 to 512 clocks of MMA.  So during a main loop only its producer
// and its MMA issuer poll (pipe_wait); one thread waits for the accumulator,
// asleep between polls (idle_wait), and everybody else stands at a hardware
// barrier.  pipe_wait ends after kWaitLimitNs.  idle_wait spans a whole main loop,
// which a long K takes past any fixed limit: it ends kWaitLimitNs after the last
// change of `progress`, which follows this CTA's copies of A (each behind a bounded
// wait, so the changes end too).
__device__ __forceinline__ bool pipe_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err) {
    return mbar_wait(bar, parity, abort, err);
}

__device__ __forceinline__ bool idle_wait(uint64_t* bar, uint32_t parity, volatile int* abort, const volatile int* progress,
                                          uint32_t* err) {
    uint64_t t0 = globaltimer_ns();
    int seen = *progress;
    while (!mbar_test_wait(bar, parity)) {
        if (*abort) return false;
        if (*progress != seen) {
            seen = *progress;
            t0 = globaltimer_ns();
        }
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            record_error(err, MOE_DEVERR_TIMEOUT);
            return false;
        }
        __nanosleep(128);
    }
    return true;
}

// ---- issuing MMAs ----
// One lane of a converged warp, as a predicate the compiler knows to hold for a
// single thread: what the others compute alike stays in uniform registers, which
// the MMA instructions take their descriptors from.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// The MMA warp's walk over the stages, executed by all of its lanes.  A wait on
// an mbarrier that is complete still takes about 200 clocks to answer, so the
// next stage's barrier is asked before this stage's MMAs are issued.
struct StageWalk {
    uint64_t* full;
    int stages, stage;
    uint32_t phase;
    bool ready;  // the barrier of `stage` has been seen complete

    __device__ __forceinline__ StageWalk(uint64_t* f, int n) : full(f), stages(n), stage(0), phase(0), ready(false) {}
    // false: given up, by all lanes
    __device__ __forceinline__ bool wait(volatile int* abort, uint32_t* err) {
        const bool ok = ready || pipe_wait(&full[stage], phase, abort, err);
        if (!__all_sync(0xffffffffu, ok)) return false;
        __syncwarp();
        const int next = stage + 1 == stages ? 0 : stage + 1;
        ready = mbar_test_wait(&full[next], next == 0 ? phase ^ 1u : phase);
        return true;
    }
    __device__ __forceinline__ void advance() {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

// 32 accumulator columns of this thread's row, as floats.
__device__ __forceinline__ void tmem_row(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    tmem_ld_32x32(taddr, r);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}

// ---- a tile's accumulator joined over the k-parts of a cluster ----
// Each CTA parks its accumulator (128 rows x BN fp32) in shared memory, row by
// row, the 16-byte quads of a row permuted by its number: the parking threads
// (one row each) and the joining warps (whole rows) both use all banks, and a
// warp's load from another CTA is whole aligned lines.  Loads from other CTAs run
// at about 23 GB/s an SM whatever their shape, so a CTA's own copy is read as plain
// shared memory.
template <int BN>
__device__ __forceinline__ uint32_t park_at(int row, int quad) {
    return static_cast<uint32_t>(row * BN * 4 + ((quad ^ (row & 7)) << 4));
}

template <int BN>
__device__ __forceinline__ void park_rows(uint8_t* park, uint32_t tmem, int q, int half, int lane) {
    const int row = q * 32 + lane;
    const uint32_t t = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * (BN / 2));
#pragma unroll 1
    for (int c = 0; c < BN / 2; c += 32) {
        uint32_t r[32];
        tmem_ld_32x32(t + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(park + park_at<BN>(row, half * (BN / 8) + c / 4 + j)) =
                make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
    }
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Four consecutive columns of one row (every width is a multiple of 8, so a quad
// is inside or outside as a whole).
__device__ __forceinline__ uint2* quad_of(uint16_t* base, long long row, int ld, int col) {
    return reinterpret_cast<uint2*>(base + row * ld + col);
}
__device__ __forceinline__ uint2 pack_quad(const float (&v)[4]) {
    return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// h = act(g) u from the fp32 accumulators (g and u are rounded only where they
// are stored for the backward pass).
__device__ __forceinline__ void gated_quad(const DenseArgs& a, long long row, int col, float (&g)[4], const float (&u)[4]) {
    if (a.out1) *quad_of(a.out1, row, a.N, col) = pack_quad(g);
    if (a.out2) *quad_of(a.out2, row, a.N, col) = pack_quad(u);
    act_values(a.fn, g);
#pragma unroll
    for (int j = 0; j < 4; ++j) g[j] *= u[j];
    *quad_of(a.out0, row, a.N, col) = pack_quad(g);
}

// y = residual + act(acc + bias) in fp32, rounded once; `res` are the residual's four values.
__device__ __forceinline__ void linear_quad(const DenseArgs& a, long long row, int col, float (&z)[4], const uint2& res) {
    if (a.bias) {
        const float4 b = *reinterpret_cast<const float4*>(a.bias + col);
        z[0] += b.x, z[1] += b.y, z[2] += b.z, z[3] += b.w;
    }
    if (a.out1) *quad_of(a.out1, row, a.N, col) = pack_quad(z);
    act_values(a.fn, z);
    if (a.residual) {
        z[0] += __uint_as_float(res.x << 16), z[1] += __uint_as_float(res.x & 0xffff0000u);
        z[2] += __uint_as_float(res.y << 16), z[3] += __uint_as_float(res.y & 0xffff0000u);
    }
    *quad_of(a.out0, row, a.N, col) = pack_quad(z);
}

// ---- the residual of a split tile, fetched into shared memory under the main loop ----
// A CTA's rows of it (every SPLITS-th of 128) x BN columns, by four warps that have
// no other work then; read in the epilogue as it comes, it cost about 0.6 us a step.
// 16-byte pieces, permuted by the row.  0 bytes: no room (the whole 128 x 256 tile).
template <int KIND, int BN, int SPLITS>
constexpr int kResidualBytes = KIND == DENSE_LINEAR && kBM / SPLITS * BN * 2 <= 32768 ? kBM / SPLITS * BN * 2 : 0;

template <int BN>
__device__ __forceinline__ uint32_t residual_at(int local_row, int piece) {
    return static_cast<uint32_t>(local_row * BN * 2 + ((piece ^ (local_row & 15)) << 4));
}

template <int BN, int SPLITS>
__device__ __forceinline__ void fetch_residual(const DenseArgs& a, uint8_t* res, int m0, int n0, int part, int thread) {
    constexpr int PN = BN / 8;
#pragma unroll 4
    for (int it = thread; it < kBM / SPLITS * PN; it += 128) {
        const int i = it / PN, p = it % PN;
        const long long row = static_cast<long long>(m0) + i * SPLITS + part;
        const int col = n0 + p * 8;
        if (row < a.M && col < a.N)
            *reinterpret_cast<uint4*>(res + residual_at<BN>(i, p)) =
                *reinterpret_cast<const uint4*>(a.residual + row * a.N + col);
    }
}

// The share of CTA `part` of `SPLITS`: every SPLITS-th row, whose parked copies
// only this CTA reads.  Thread t of 256 takes quads t, t + 256, ... of those rows;
// `first` + k * `step` are the ranks of the k-parts, summed in order.  First the
// sums, in passes of up to sixteen loads, all issued before the first is used,
// each sum back into this CTA's own copy; then the epilogue over them in a rolled
// loop: its instructions run once a launch, and unrolled eight times they were
// fetched cold for longer than they worked.
template <int KIND, int BN, int SPLITS>
__device__ __forceinline__ void join_parts(const DenseArgs& a, int mat, uint8_t* park, const uint8_t* res, int m0, int n0,
                                           int part, uint32_t first, uint32_t step) {
    constexpr bool GATED = DenseLayout<KIND>::GATED;
    constexpr int HALVES = GATED ? 2 : 1;
    constexpr int QN = BN / 4 / HALVES;  // output quads of a row
    constexpr int ITEMS = kBM / SPLITS * QN;
    constexpr int MOST = 16 / (HALVES * SPLITS), ALL = (ITEMS + 255) / 256;
    constexpr int PER = MOST < ALL ? MOST : ALL;
    const uint32_t park0 = smem_u32(park);
    // item -> row of the tile (-1: none) and quad
    auto place = [&](int it, int& r, int& q) {
        r = it / QN * SPLITS + part;
        q = it % QN;
        if (it >= ITEMS || m0 + r >= a.M || n0 + q * 4 >= a.N) r = -1;
    };
#pragma unroll 1
    for (int base = 0; base < ITEMS; base += PER * 256) {
        float4 parts[PER][HALVES][SPLITS];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            int r, q;
            place(base + i * 256 + static_cast<int>(threadIdx.x), r, q);
            if (r < 0) continue;
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
#pragma unroll
                for (int s = 0; s < SPLITS; ++s) {
                    const uint32_t at = park_at<BN>(r, h * QN + q);
                    if (s == part) parts[i][h][s] = *reinterpret_cast<const float4*>(park + at);
                    else parts[i][h][s] = ld_cluster_v4(mapa_shared(park0 + at, first + s * step));
                }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            int r, q;
            place(base + i * 256 + static_cast<int>(threadIdx.x), r, q);
            if (r < 0) continue;
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                float4 v = parts[i][h][0];
#pragma unroll
                for (int s = 1; s < SPLITS; ++s) {
                    const float4 x = parts[i][h][s];
                    v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
                }
                *reinterpret_cast<float4*>(park + park_at<BN>(r, h * QN + q)) = v;
            }
        }
    }
#pragma unroll 1
    for (int it = threadIdx.x; it < ITEMS; it += 256) {
        int r, q;
        place(it, r, q);
        if (r < 0) continue;
        float v[HALVES][4];
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            const float4 x = *reinterpret_cast<const float4*>(park + park_at<BN>(r, h * QN + q));
            v[h][0] = x.x, v[h][1] = x.y, v[h][2] = x.z, v[h][3] = x.w;
        }
        const long long row = static_cast<long long>(m0) + r;
        const int col = n0 + q * 4;
        if constexpr (GATED) gated_quad(a, row, col, v[0], v[HALVES - 1]);
        else if constexpr (KIND == DENSE_LINEAR) linear_quad(a, row, col, v[0],
                                                            *reinterpret_cast<const uint2*>(
                                                                res + residual_at<BN>(r / SPLITS, q >> 1) + (q & 1) * 8));
        else *quad_of(mat ? a.out1 : a.out0, row, a.N, col) = pack_quad(v[0]);
    }
}

__device__ __forceinline__ uint4* octet(uint16_t* base, long long row, int ld, int col) {
    return reinterpret_cast<uint4*>(base + row * ld + col);
}
__device__ __forceinline__ const uint4* octet(const uint16_t* base, long long row, int ld, int col) {
    return reinterpret_cast<const uint4*>(base + row * ld + col);
}

// ---- fused epilogues: 32 rows x 32 columns of a warp ----
// tcgen05.ld leaves one accumulator row in each thread.  Stored as it lies, a
// warp's 16-byte store touches 32 rows at once, half a sector each; the kernel
// that keeps g and u was bound by that (83 us of 656 at 4096 x 4096 x 14336; they
// cost 25 to 37 of 580 now).  So a chunk goes through shared memory and leaves (and a
// residual enters) as 64-byte pieces of eight rows.  The 16-byte pieces of a row
// are permuted so that both directions use all banks.
constexpr int kChunkBytes = 32 * 128;  // 64-byte rows here, 128-byte rows in plain_chunk

struct RowChunk {
    uint8_t* smem;   // this warp's kChunkBytes
    long long row0;
    int col0, M, N, lane;

    __device__ __forceinline__ uint4* cell(int r, int p) const {
        return reinterpret_cast<uint4*>(smem + r * 64 + ((p ^ ((r >> 1) & 3)) << 4));
    }
    // rows i * 8 + lane / 4, piece lane % 4 of a [M, N] matrix (zeros outside)
    __device__ __forceinline__ void fetch(const uint16_t* base, uint4 (&v)[4]) const {
        const int col = col0 + (lane & 3) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long r = row0 + i * 8 + (lane >> 2);
            v[i] = r < M && col < N ? *octet(base, r, N, col) : make_uint4(0, 0, 0, 0);
        }
    }
    // what fetch read, as this thread's row
    __device__ __forceinline__ void to_row(uint4 (&v)[4]) const {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) *cell(i * 8 + (lane >> 2), lane & 3) = v[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = *cell(lane, i);
    }
    __device__ __forceinline__ void store(uint16_t* base, const float (&v)[32]) const {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *cell(lane, i) = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                        pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
        __syncwarp();
        const int col = col0 + (lane & 3) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long r = row0 + i * 8 + (lane >> 2);
            if (r < M && col < N) *octet(base, r, N, col) = *cell(i * 8 + (lane >> 2), lane & 3);
        }
    }
};

__device__ __forceinline__ void gated_chunk(const DenseArgs& a, const RowChunk& c, float (&g)[32], float (&u)[32]) {
    if (a.out1) c.store(a.out1, g);
    if (a.out2) c.store(a.out2, u);
    act_values(a.fn, g);
#pragma unroll
    for (int j = 0; j < 32; ++j) g[j] *= u[j];
    c.store(a.out0, g);
}

// `res`: the residual as RowChunk::fetch left it, or (own_row) this thread's row of it.
__device__ __forceinline__ void linear_chunk(const DenseArgs& a, const RowChunk& c, float (&z)[32], uint4 (&res)[4],
                                             bool own_row) {
    if (a.bias) {
#pragma unroll
        for (int o = 0; o < 4; ++o) {
            if (c.col0 + o * 8 >= a.N) break;
            const float4* b = reinterpret_cast<const float4*>(a.bias + c.col0 + o * 8);
            const float4 b0 = b[0], b1 = b[1];
            z[8 * o] += b0.x, z[8 * o + 1] += b0.y, z[8 * o + 2] += b0.z, z[8 * o + 3] += b0.w;
            z[8 * o + 4] += b1.x, z[8 * o + 5] += b1.y, z[8 * o + 6] += b1.z, z[8 * o + 7] += b1.w;
        }
    }
    if (a.out1) c.store(a.out1, z);
    act_values(a.fn, z);
    if (a.residual) {
        if (!own_row) c.to_row(res);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float r[8];
            unpack_bf16x8(res[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[8 * i + j] += r[j];
        }
    }
    c.store(a.out0, z);
}

// A gradient's 32 rows x 64 columns: 128-byte lines of four rows a store.
__device__ __forceinline__ void plain_chunk(uint8_t* smem, uint32_t taddr, uint16_t* base, long long row0, int col0, int M,
                                            int N, int lane) {
    uint32_t r[64];
    {
        uint32_t(&lo)[32] = *reinterpret_cast<uint32_t(*)[32]>(&r[0]);
        uint32_t(&hi)[32] = *reinterpret_cast<uint32_t(*)[32]>(&r[32]);
        tmem_ld_32x32(taddr, lo);
        tmem_ld_32x32(taddr + 32, hi);
        tmem_ld_wait();
    }
    auto cell = [&](int row, int p) { return reinterpret_cast<uint4*>(smem + row * 128 + ((p ^ (row & 7)) << 4)); };
    auto two = [&](int j) { return pack_bf16x2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])); };
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) *cell(lane, i) = make_uint4(two(8 * i), two(8 * i + 2), two(8 * i + 4), two(8 * i + 6));
    __syncwarp();
    const int col = col0 + (lane & 7) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long long row = row0 + i * 4 + (lane >> 3);
        if (row < M && col < N) *octet(base, row, N, col) = *cell(i * 4 + (lane >> 3), lane & 7);
    }
}

// The epilogue of a whole accumulator of 128 rows x BN columns by eight warps:
// warp (q, half) takes lanes 32 q .. and half of the output columns.  `res`: the
// tile's residual in shared memory (fetch_residual), or NULL: it is read here, a
// chunk ahead, the first one by the caller into `ahead` (fetch_ahead) before it
// waits for the accumulator.
template <int KIND, int BN>
struct WholeEpilogue {
    static constexpr bool GATED = DenseLayout<KIND>::GATED;
    static constexpr int COLS = GATED ? BN / 4 : BN / 2;  // output columns of a warp
    const DenseArgs& a;
    uint8_t* smem;  // this warp's kChunkBytes
    int m0, n0, q, half, lane;
    uint4 ahead[4];

    __device__ __forceinline__ RowChunk chunk(int c) const {
        return RowChunk{smem, static_cast<long long>(m0) + q * 32, n0 + half * COLS + c, a.M, a.N, lane};
    }
    __device__ __forceinline__ void fetch_ahead() {
        if (KIND == DENSE_LINEAR && a.residual) chunk(0).fetch(a.residual, ahead);
    }
    __device__ __forceinline__ void run(int mat, uint32_t tmem, const uint8_t* res) {
        const uint32_t t = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * COLS);
        if constexpr (KIND == DENSE_DGRAD || KIND == DENSE_WGRAD) {
#pragma unroll 1
            for (int c = 0; c < COLS; c += 64)
                plain_chunk(smem, t + c, mat ? a.out1 : a.out0, static_cast<long long>(m0) + q * 32, n0 + half * COLS + c, a.M,
                            a.N, lane);
        } else {
#pragma unroll 1
            for (int c = 0; c < COLS; c += 32) {
                float v[32];
                if constexpr (KIND == DENSE_LINEAR) {
                    uint4 piece[4];
                    if (res) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            piece[i] = *reinterpret_cast<const uint4*>(
                                res + residual_at<BN>(q * 32 + lane, (half * COLS + c) / 8 + i));
                    } else if (a.residual) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) piece[i] = ahead[i];
                        if (c + 32 < COLS) chunk(c + 32).fetch(a.residual, ahead);
                    }
                    tmem_row(t + c, v);
                    linear_chunk(a, chunk(c), v, piece, res != nullptr);
                } else {
                    float u[32];
                    tmem_row(t + c, v);
                    tmem_row(t + BN / 2 + c, u);
                    gated_chunk(a, chunk(c), v, u);
                }
            }
        }
    }
};

}  // namespace moe
