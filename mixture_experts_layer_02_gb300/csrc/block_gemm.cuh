// block_gemm.cuh -- products in e4m3 with a scale for each block of 128, grouped over
// the experts' segments, and their gradients (block_gemm.h has the formulas).
//
// A scale that changes along K cannot wait for the end of the sum: the tensor cores
// sum 128 products, the block's partial sum is scaled and added in fp32 on the CUDA
// cores, and so on.  So the accumulator lives in registers and TMEM holds a ring of
// partial sums: the MMA warp fills slot after slot (four MMAs of 32 a slot, the first
// one overwriting), and eight epilogue warps, one row a thread, read a slot, free it
// and add scale * partial with paired fp32 arithmetic.  The additions have a fixed
// order; the scales are any fp32 numbers.
//
// What bounds it.  A 256 x 256 x 128 step of a CTA pair is 512 clocks of MMA on each SM.
// Its 128 x 256 partial sums take 256 clocks to read from TMEM and 256 to add (WGRAD, with
// two scales a product, 512), on other pipes, but a slot is only refilled when all have
// read it: what counts is the way from a slot's MMAs through a barrier, two reads and a
// barrier back.  4096 tokens on 8 experts of 4096 x 14336: 400 us, 2.40 PFLOP/s, the tensor
// pipe active in 57 % of the cycles; the same loop without reading the slots runs in 332 us.  So a slot is freed as soon as a warp has its values in
// registers, no arrival waits for memory, and scales come through shared memory (kept by the
// epilogue's threads they cost spilled registers: 500 us).  Sixteen epilogue warps of 64
// columns: 441 for 420 us; reads of 32 columns one ahead: 448 to 523.  WGRAD of the same sizes
// has eight steps a tile: about 0.6 us each and 2 us a tile around them.  Its rows leave as
// tensor copies: both gradients 1020 us; as bulk copies of 256 bytes, 256 of them a tile,
// 1075, as 64-byte pieces by the epilogue's own stores 1128 (FWD 430 so, 411 with the copies).
// With 128 rows an expert the weights' stream is the limit (4096 x 7168 x 2048 by 256 experts:
// 728 us, 5.7 TB/s), and a warp whose 32 rows all lie behind the segment only frees its slots.
//
// Operands are read as stored, nothing is transposed in memory: FWD has both K-major,
// DGRAD the weights MN-major, WGRAD both MN-major, its K being an expert's rows from a
// multiple of 128 on with zero rows behind them (quant_block.cu).  Boxes are 128 x 128
// bytes; what lies outside a matrix reads as zeros, so K needs no multiple.
//
// Warps: 0 copies A, 1 issues the MMAs, 2 copies B, 3 allocates TMEM and brings a step's
// scales to shared memory, 4..11 epilogue.
// Registers are dealt out anew at the start: the epilogue's accumulators take 128.
// Barriers: full[s] the bytes of a stage (of both CTAs, on the even one's), empty[s]
// its MMAs are done, tfull[i] a slot and its scales are filled, tempty[i] a slot and sempty[i]
// its scales are read.
// Every wait is bounded (1 s); none spans more than one step of 128 along K.
#pragma once

#include <algorithm>
#include <atomic>

#include "activation.cuh"
#include "block_gemm.h"
#include "dense_gemm.cuh"

namespace moe {

namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 12 * 32;
constexpr int kBoxBytes = kBlock * kRowBytes;  // 128 rows of 128 bytes
constexpr int kMaxE = 1024;
constexpr int kCopyRegs = 72, kEpiRegs = 216;  // registers a thread of warps 0..3 and 4..11

template <int KIND, bool PAIR, int BN, int SPLITS>
struct BlockCfg {
    static constexpr bool A_MN = KIND == BLOCK_WGRAD;
    static constexpr bool B_MN = KIND != BLOCK_FWD;
    static constexpr int CTAS = PAIR ? 2 : 1;                  // that share a tile's MMAs
    static constexpr int ROWS = CTAS * kBM;                    // rows of a tile
    static constexpr int B_BOXES = PAIR ? 1 : BN / kBlock;     // of this CTA
    static constexpr int STAGE = (1 + B_BOXES) * kBoxBytes;
    static constexpr int SLOTS = 512 / BN;                     // partial sums in TMEM
    static constexpr int COLS = BN / 2;                        // accumulator columns of an epilogue warp
    // How the output leaves: one-CTA tiles in 64-byte pieces of eight rows, through 32 rows x
    // 32 columns of shared memory a warp.  Pairs keep all 32 rows x 128 columns there and let
    // them leave as two tensor copies under the next tile, for two stages less; rows at the
    // end of a segment, which a copy would not stop at, go by hand.
    static constexpr bool BULK = PAIR;
    static constexpr int PITCH = BULK ? COLS * 2 : 64;  // bytes of shared memory a row
    static constexpr int OUT = kEpiWarps * 32 * PITCH;
    static constexpr int STAGES = BULK ? 4 : 192 * 1024 / STAGE;
    static constexpr int CLUSTER = CTAS * SPLITS;
    // a slot's scales: FWD and DGRAD one of each row for either half of the columns, WGRAD
    // one of each row, then one of each column
    static constexpr int SCALES = A_MN ? kBM + BN : 2 * kBM;
    static constexpr size_t smem(int E) {
        return 1024 + STAGES * STAGE + OUT + SLOTS * SCALES * 4 + 48 * sizeof(uint64_t) + (2 * static_cast<size_t>(E) + 2) * sizeof(int) +
               (KIND == BLOCK_WGRAD ? E * sizeof(uint16_t) : 0);
    }
    static_assert(smem(kMaxE) <= 227 * 1024, "shared memory");
    static_assert(!BULK || (STAGES * STAGE) % 1024 == 0, "swizzled boxes start on 1024 bytes");
    static_assert(SPLITS == 1 || STAGES * STAGE >= kBM * 128 * 4, "the parked accumulator reuses the stages");
    static_assert(!PAIR || (BN == 256 && SPLITS == 1), "pairs own whole 256 x 256 tiles");
    static_assert(SPLITS == 1 || BN == 128, "parts of K are joined on 128 x 128 tiles");
};

__device__ __forceinline__ void load_box(const CUtensorMap* map, uint64_t* bar, void* dst, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// "This warp has read the slot", to the even CTA's barrier.  What it orders are TMEM
// reads, which the fence before it covers, and no memory: a release at cluster scope
// waits for every access in flight and took 1 us a step.
__device__ __forceinline__ void slot_arrive(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Wait for the tcgen05.ld that fills r; what uses r stays behind it.
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_landed(uint32_t (&r)[64]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31]), "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]),
                   "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]), "+r"(r[40]), "+r"(r[41]), "+r"(r[42]),
                   "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]), "+r"(r[48]), "+r"(r[49]),
                   "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]), "+r"(r[56]),
                   "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63])
                 :
                 : "memory");
}

// Descriptor of an MN-major byte operand: each k-row holds 128 consecutive M/N bytes,
// 8 k-rows are a 1024-byte swizzle atom (stride offset), the next 128 M/N bytes start
// one box further (leading offset).
template <bool MN>
__device__ __forceinline__ uint64_t byte_desc(uint32_t saddr) {
    uint64_t d = sw128_kmajor_desc(saddr);
    if (MN) d = (d & ~(static_cast<uint64_t>(0x3fff) << 16)) | static_cast<uint64_t>(kBoxBytes >> 4) << 16;
    return d;
}
// step of one MMA's 32 K bytes, in 16-byte units: 32 bytes of a row, or 32 rows
template <bool MN>
constexpr uint64_t kByteStep = MN ? 32 * kRowBytes / 16 : 2;

template <int KIND>
__host__ __device__ constexpr uint32_t block_idesc(int M, int N) {
    return idesc_e4m3_f32(M, N) | (KIND == BLOCK_WGRAD ? 1u << 15 : 0u) | (KIND != BLOCK_FWD ? 1u << 16 : 0u);
}

// A warp's walk over a ring of barriers, executed by all of its lanes.  A wait on an
// mbarrier that is complete still takes about 200 clocks to answer, so a stage's is asked
// before the MMAs of the one before are issued (AHEAD); a slot's, which is hardly ever
// complete a step ahead, is not (403 for 408 us at 4096 x 4096 x 14336 by 8 experts).
template <bool AHEAD>
struct BarrierWalk {
    uint64_t* bar;
    int n, at;
    uint32_t parity;
    bool ready;  // the barrier at `at` has been seen complete

    __device__ __forceinline__ BarrierWalk(uint64_t* b, int count, uint32_t first) : bar(b), n(count), at(0), parity(first), ready(false) {}
    // false: given up, by all lanes
    __device__ __forceinline__ bool wait(volatile int* abort, uint32_t* err) {
        const bool ok = ready || mbar_wait(&bar[at], parity, abort, err);
        if (!__all_sync(0xffffffffu, ok)) return false;
        __syncwarp();
        const int next = at + 1 == n ? 0 : at + 1;
        ready = AHEAD && mbar_test_wait(&bar[next], next == 0 ? parity ^ 1u : parity);
        return true;
    }
    __device__ __forceinline__ void advance() {
        if (++at == n) {
            at = 0;
            parity ^= 1u;
        }
    }
};

// A tile: expert, first output row and how many of its rows exist, first column, and
// where its K begins (WGRAD: 128-row blocks of the padded rows).
struct BlockTile {
    int e, row0, rows, n0, k0, kbs;
};

// Tiles are numbered expert by expert, inside an expert in bands of kPairBand row tiles,
// inside a band column by column, the band's row tiles innermost: what runs at a time
// shares weight columns and rows in L2.
struct TileList {
    const int *goff, *pre;  // segments; FWD, DGRAD: row tiles before an expert; WGRAD: 128-row blocks before it
    const uint16_t* ord;    // WGRAD: the experts' order
    int E, nt, mt, kbs, tile_rows, bn, M;

    template <int KIND>
    __device__ __forceinline__ BlockTile at(int t) const {
        BlockTile b;
        int rows = M, first = 0, tiles = mt;  // of this expert's output
        if constexpr (KIND == BLOCK_WGRAD) {
            const int i = t / (mt * nt);
            t -= i * mt * nt;
            b.e = ord[i];
            b.k0 = pre[b.e];
            b.kbs = (goff[b.e + 1] - goff[b.e] + kBlock - 1) / kBlock;
        } else {
            int lo = 0, hi = E - 1;
            while (lo < hi) {  // the last expert with pre * nt <= t
                const int mid = (lo + hi + 1) >> 1;
                if (pre[mid] * nt <= t) lo = mid; else hi = mid - 1;
            }
            t -= pre[lo] * nt;
            tiles = pre[lo + 1] - pre[lo];
            first = goff[lo];
            rows = goff[lo + 1] - first;
            b.e = lo;
            b.k0 = 0;
            b.kbs = kbs;
        }
        const int band = t / (kPairBand * nt), in = t - band * kPairBand * nt;
        const int high = min(kPairBand, tiles - band * kPairBand), n = in / high;
        const int m = band * kPairBand + in - n * high;
        b.row0 = first + m * tile_rows;
        b.rows = min(tile_rows, rows - m * tile_rows);
        b.n0 = n * bn;
        return b;
    }
};

// 32 lanes x 64 (or 32) consecutive fp32 columns, a row a thread.
__device__ __forceinline__ void tmem_ld_wide(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
        "}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
          "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
          "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
          "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
          "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_wide(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
        "}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// 16 lanes x 64 (or 32) consecutive fp32 columns in the layout of an MMA's accumulator:
// thread T gets columns 8 j + 2 (T % 4) and the next of rows T / 4 (r[4 j], r[4 j + 1]) and
// T / 4 + 8 (r[4 j + 2], r[4 j + 3]).
__device__ __forceinline__ void tmem_ld_frag64(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
        "}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_frag32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15"
        "}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Four 8 x 8 blocks of 16-bit values, in the same layout, to rows of 16 bytes: thread T
// has the address of row T % 8 of block T / 8.
__device__ __forceinline__ void st_blocks(void* row, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_u32(row)), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// A cell of 16 bytes of a warp's 32 rows x 32 columns, permuted so that both directions use all banks.
__device__ __forceinline__ uint4* chunk_cell(uint8_t* smem, int r, int piece) {
    return reinterpret_cast<uint4*>(smem + r * 64 + ((piece ^ ((r >> 1) & 3)) << 4));
}

// Stored as they lie, one row a thread, a 16-byte store would touch 32 rows at once.
__device__ __forceinline__ void store_chunk(uint8_t* smem, uint16_t* out, long long row0, int rows, int col0, int N, int lane) {
    const int col = col0 + (lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2);
        if (r < rows && col < N) *reinterpret_cast<uint4*>(out + (row0 + r) * N + col) = *chunk_cell(smem, r, lane & 3);
    }
}

// A box of 32 rows x 64 bf16 (128-byte swizzle) from shared to global memory, in the
// background; what lies outside the matrix is not written.
__device__ __forceinline__ void store_box(const CUtensorMap* map, const void* src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// This thread's copies have read shared memory; or have ended.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// The accumulator of one k-part, parked in shared memory: 128 rows of 128 fp32, the
// 16-byte quads of a row permuted by its number.
__device__ __forceinline__ uint32_t park_quad(int row, int quad) {
    return static_cast<uint32_t>(row * 512 + ((quad ^ (row & 7)) << 4));
}

__device__ __forceinline__ float4 ld_part(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

template <int KIND, bool PAIR, int BN, int SPLITS>
__global__ void __launch_bounds__(kThreads, 1)
block_gemm_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                  const __grid_constant__ CUtensorMap out_map, const BlockArgs args) {
    using C = BlockCfg<KIND, PAIR, BN, SPLITS>;
    constexpr int S = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);  // the same offset in every CTA of a cluster
    uint8_t* outs = smem + S * C::STAGE;
    float* scales = reinterpret_cast<float*>(outs + C::OUT);
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + C::SLOTS * C::SCALES);
    uint64_t* empty = full + S;
    uint64_t* tfull = empty + S;
    uint64_t* tempty = tfull + C::SLOTS;
    uint64_t* sempty = tempty + C::SLOTS;
    uint64_t* drain = tempty + 2 * C::SLOTS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* s_goff = reinterpret_cast<int*>(full + 48);  // [E + 1]
    int* s_pre = s_goff + args.E + 1;                 // [E + 1]
    uint16_t* s_ord = reinterpret_cast<uint16_t*>(s_pre + args.E + 1);  // [E], WGRAD: the experts, most rows first
    static_assert(2 * S + 3 * C::SLOTS + 1 + 1 <= 48, "barrier room");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = args.E;
    uint32_t* err = args.err;
    const uint32_t rank = C::CLUSTER > 1 ? cluster_ctarank() : 0u;
    const bool leader = !PAIR || rank == 0;
    const int part = SPLITS > 1 ? static_cast<int>(rank) : 0;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&a_map);
        tma_prefetch_desc(&b_map);
        if (C::BULK) tma_prefetch_desc(&out_map);
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < C::SLOTS; ++i) {
            mbar_init(&tfull[i], 2);  // the MMAs' commit, the scales
            mbar_init(&tempty[i], C::CTAS * kEpiWarps);
            mbar_init(&sempty[i], kEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 3) {
        if constexpr (PAIR) {
            tmem_alloc_pair(tmem_slot, 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, 512);
            tmem_relinquish();
        }
    }
    pdl_wait();
    for (int i = threadIdx.x; i <= E; i += kThreads) s_goff[i] = args.offsets ? args.offsets[i] : (i == 0 ? 0 : args.rows);
    __syncthreads();
    int bad = threadIdx.x == 0 && (s_goff[0] != 0 || s_goff[E] > args.rows);
    for (int i = threadIdx.x; i < E; i += kThreads) bad |= s_goff[i] > s_goff[i + 1];
    bad = __syncthreads_or(bad);
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) record_error(err, MOE_DEVERR_BOUNDS);
    // tiles of FWD and DGRAD cost the same; WGRAD's go by their expert's rows, the longest first
    // (above kSortMaxGroups experts in the experts' order)
    if constexpr (KIND == BLOCK_WGRAD)
        for (int e = threadIdx.x; e < E; e += kThreads) {
            int at = e;
            if (E <= kSortMaxGroups) {
                const int mine = s_goff[e + 1] - s_goff[e];
                at = 0;
                for (int o = 0; o < E; ++o) {
                    const int other = s_goff[o + 1] - s_goff[o];
                    at += (other > mine) | ((other == mine) & (o < e));
                }
            }
            s_ord[at] = static_cast<uint16_t>(e);
        }
    __syncthreads();
    if (warp == 0) {  // exclusive prefix of the experts' row tiles, or of their padded rows' blocks
        constexpr int UNIT = KIND == BLOCK_WGRAD ? kBlock : C::ROWS;
        int carry = 0;
        for (int base = 0; base < E; base += 32) {
            const int i = base + lane;
            int v = i < E ? (s_goff[i + 1] - s_goff[i] + UNIT - 1) / UNIT : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += up;
            }
            if (i < E) s_pre[i + 1] = carry + v;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) s_pre[0] = 0;
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (C::CLUSTER > 1) cluster_sync_all();  // every CTA's barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const TileList list = {s_goff, s_pre, s_ord, E, (args.N + BN - 1) / BN, (args.M + C::ROWS - 1) / C::ROWS,
                           (args.K + kBlock - 1) / kBlock, C::ROWS, BN, args.M};
    const int tiles = bad ? 0 : (KIND == BLOCK_WGRAD ? E * list.mt : s_pre[E]) * list.nt;
    const int first = blockIdx.x / C::CLUSTER, step = gridDim.x / C::CLUSTER;
    // this CTA's part of a tile's steps along K
    auto k_lo = [&](const BlockTile& b) { return SPLITS > 1 ? b.kbs * part / SPLITS : 0; };
    auto k_hi = [&](const BlockTile& b) { return SPLITS > 1 ? b.kbs * (part + 1) / SPLITS : b.kbs; };
    const uint32_t full_lead = PAIR ? mapa_shared(smem_u32(full), 0) : 0;

    if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        // epilogue warp (q, half): TMEM lanes 32 q .., columns half * COLS ..
        const int q = warp & 3, half = (warp - 4) >> 2;
        uint8_t* out_rows = outs + (warp - 4) * 32 * C::PITCH;
        const uint32_t tempty_lead = PAIR ? mapa_shared(smem_u32(tempty), 0) : 0;
        const uint32_t t_warp = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * C::COLS);
        const int in_tile = (PAIR ? static_cast<int>(rank) * kBM : 0) + q * 32;  // this warp's first row of the tile
        int slot = 0;
        uint32_t slot_phase = 0;
        bool ok = true;
        // Who holds what: in FWD and DGRAD a thread has one row, so that a step's two scales are
        // one number to it.  In WGRAD, where every column has its own, it has four rows (lane /
        // 4 and every 8th after it) and every fourth pair of columns: a quarter of the scales
        // to read from shared memory, which the MMAs' operands keep busy as well.
        constexpr int ROWS = KIND == BLOCK_WGRAD ? 4 : 1;
        const float* my_scales = scales + (KIND == BLOCK_WGRAD ? q * 32 + (lane >> 2) : half * kBM + q * 32 + lane);
        const float* my_columns = scales + kBM + half * C::COLS + (lane & 3) * 2;  // WGRAD
        float2 acc[C::COLS / 2];
        for (int t = first; ok && t < tiles; t += step) {
            const BlockTile b = list.at<KIND>(t);
            const int rows = min(32, b.rows - in_tile);  // of this warp; <= 0: none exist
#pragma unroll
            for (int i = 0; i < C::COLS / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
#pragma unroll 1
            for (int n = k_hi(b) - k_lo(b); n > 0; --n) {
                ok = __all_sync(0xffffffffu, mbar_wait(&tfull[slot], slot_phase, abort_flag, err));
                if (!ok) break;
                tc_fence_after();
                auto release = [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (PAIR) slot_arrive(tempty_lead + 8u * slot);
                        else mbar_arrive(&tempty[slot]);
                        if (KIND != BLOCK_WGRAD || rows <= 0) mbar_arrive(&sempty[slot]);
                    }
                };
                if (rows > 0) {
                    float s[ROWS];
#pragma unroll
                    for (int i = 0; i < ROWS; ++i) s[i] = my_scales[slot * C::SCALES + 8 * i];
                    const uint32_t t_slot = t_warp + static_cast<uint32_t>(slot * BN);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {  // half of the columns at a time
                        constexpr int W = C::COLS / 2;
                        uint32_t r[W];
                        if constexpr (KIND == BLOCK_WGRAD) {  // first rows 0..15, then 16..31
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t at = t_slot + c * W + (static_cast<uint32_t>(h * 16) << 16);
                                if constexpr (W == 64) tmem_ld_frag64(at, r + h * 32);
                                else tmem_ld_frag32(at, r + h * 16);
                            }
                        } else {
                            tmem_ld_wide(t_slot + c * W, r);
                        }
                        tmem_landed(r);
                        if (c == 1) release();  // all that this warp reads of the slot is in registers
                        if constexpr (KIND == BLOCK_WGRAD) {
#pragma unroll
                            for (int j = 0; j < W / 8; ++j) {
                                const float2 col = *reinterpret_cast<const float2*>(my_columns + slot * C::SCALES + c * W + j * 8);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {  // rows lane / 4 + 8 i
                                    const int at = (i >> 1) * (W / 2) + j * 4 + (i & 1) * 2;
                                    const float2 v = mul2(make_float2(__uint_as_float(r[at]), __uint_as_float(r[at + 1])), col);
                                    acc[c * (W / 2) + at / 2] = fma2(v, make_float2(s[i], s[i]), acc[c * (W / 2) + at / 2]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < W / 2; ++j)
                                acc[c * (W / 2) + j] = fma2(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])),
                                                            make_float2(s[0], s[0]), acc[c * (W / 2) + j]);
                        }
                    }
                    if constexpr (KIND == BLOCK_WGRAD) {  // the columns' scales are read to the end
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sempty[slot]);
                    }
                } else {
                    release();
                }
                if (++slot == C::SLOTS) { slot = 0; slot_phase ^= 1u; }
            }
            if (!ok) break;
            const int col0 = b.n0 + half * C::COLS;
            if constexpr (SPLITS == 1) {
                if (rows > 0) {
                    uint16_t* out = args.out + (KIND == BLOCK_WGRAD ? static_cast<long long>(b.e) * args.M * args.N : 0LL);
                    const long long row0 = static_cast<long long>(b.row0) + in_tile;
                    // the cell of 16 bytes that holds columns 8 p .. of row r
                    auto cell = [&](int r, int p) {
                        return C::BULK ? reinterpret_cast<uint4*>(out_rows + (p >> 3) * 4096 + sw128_offset(r, p & 7)) : chunk_cell(out_rows, r, p & 3);
                    };
                    if constexpr (C::BULK) bulk_wait_read();  // the last tile's
                    __syncwarp();
#pragma unroll
                    for (int p = 0; p < C::COLS / 8; ++p) {
                        if constexpr (KIND == BLOCK_WGRAD) {
                            constexpr int W = C::COLS / 2;
                            auto two = [&](int i) {
                                const float2 v = acc[p / (W / 8) * (W / 2) + (i >> 1) * (W / 4) + p % (W / 8) * 2 + (i & 1)];
                                return pack_bf16x2(v.x, v.y);
                            };
                            st_blocks(cell(lane, p), two(0), two(1), two(2), two(3));
                        } else {
                            const float2* v = &acc[p * 4];
                            *cell(lane, p) = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                                                        pack_bf16x2(v[3].x, v[3].y));
                        }
                        if constexpr (!C::BULK) {
                            if ((p & 3) == 3) {
                                __syncwarp();
                                store_chunk(out_rows, out, row0, rows, col0 + (p - 3) * 8, args.N, lane);
                                __syncwarp();
                            }
                        }
                    }
                    if constexpr (C::BULK) {
                        if (KIND == BLOCK_WGRAD || rows == 32) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane < C::COLS / 64 && col0 + lane * 64 < args.N)
                                store_box(&out_map, out_rows + lane * 4096, col0 + lane * 64, static_cast<int>(row0), KIND == BLOCK_WGRAD ? b.e : 0);
                            bulk_commit();
                        } else {
                            __syncwarp();
                            const int p = lane & 15;
#pragma unroll 4
                            for (int r = lane >> 4; r < rows; r += 2)
                                if (col0 + p * 8 < args.N) *reinterpret_cast<uint4*>(out + (row0 + r) * args.N + col0 + p * 8) = *cell(r, p);
                        }
                    }
                }
            } else if constexpr (KIND == BLOCK_WGRAD) {  // the stages are free: every copy of this CTA's part was waited for
#pragma unroll
                for (int i = 0; i < C::COLS / 2; ++i) {
                    // acc[i]: COLS / 2 columns, of them 16 rows at a time, then pairs of columns of rows lane / 4 and 8 further
                    constexpr int W = C::COLS / 2;
                    const int c = i / (W / 2), h = i / (W / 4) % 2, j = i % (W / 4);
                    const int r = (lane >> 2) + 8 * (j & 1) + 16 * h, col = half * C::COLS + c * W + (j >> 1) * 8 + (lane & 3) * 2;
                    if (r < rows) *reinterpret_cast<float2*>(smem + park_quad(in_tile + r, col >> 2) + (col & 2) * 4) = acc[i];
                }
            } else if (lane < rows) {
#pragma unroll
                for (int i = 0; i < C::COLS / 4; ++i)
                    *reinterpret_cast<float4*>(smem + park_quad(in_tile + lane, half * (C::COLS / 4) + i)) =
                        make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
            }
        }
        if constexpr (C::BULK) bulk_wait();  // shared memory is given back, and the rows are written
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
        // Copies: warp 0 A (it announces the stage's bytes), warp 2 B.  Each brings bytes of every
        // stage, rows that exist or not: a stage that is complete without one of its copiers could
        // be used up and filled again before that thread has seen it empty, which it then never
        // does.  (Only the rows that exist, in boxes of 32, were no faster: 736 us both ways at
        // 4096 x 7168 x 2048 by 256 experts.)
        if (warp == 0 || warp == 2) {
            if (lane == 0) {
                const bool is_a = warp == 0;
                bool withhold = is_a && args.dbg && (*args.dbg & MOE_DBG_WITHHOLD_FIRST_LOAD) && blockIdx.x == 0;
                uint32_t pending = 0, pend_parity = 0;
                int stage = 0;
                uint32_t phase = 0;
                bool ok = true;
                for (int t = first; ok && t < tiles; t += step) {
                    const BlockTile b = list.at<KIND>(t);
                    const int hi = k_hi(b);
                    for (int kb = k_lo(b); kb < hi; ++kb) {
                        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, err)) { ok = false; break; }
                        uint8_t* dst = smem + stage * C::STAGE;
                        const int k = (b.k0 + kb) * kBlock;
                        const uint32_t bar = full_lead + 8u * stage;
                        if (withhold) {
                            withhold = false;  // test hook: this stage never fills
                        } else if (is_a) {
                            if (leader) {
                                mbar_arrive_expect_tx(&full[stage], C::CTAS * C::STAGE);
                                pending |= 1u << stage;
                                pend_parity = (pend_parity & ~(1u << stage)) | (phase << stage);
                            }
                            const int row = b.row0 + (PAIR ? static_cast<int>(rank) * kBM : 0);
                            const int x = C::A_MN ? row : k, y = C::A_MN ? k : row;
                            if constexpr (PAIR) tma_load_3d_pair(&a_map, bar, dst, x, y, 0);
                            else load_box(&a_map, &full[stage], dst, x, y, 0);
                        } else {
#pragma unroll
                            for (int i = 0; i < C::B_BOXES; ++i) {
                                const int n = b.n0 + (PAIR ? static_cast<int>(rank) : i) * kBlock;
                                const int x = C::B_MN ? n : k, y = C::B_MN ? k : n, z = KIND == BLOCK_WGRAD ? 0 : b.e;
                                if constexpr (PAIR) tma_load_3d_pair(&b_map, bar, dst + kBoxBytes, x, y, z);
                                else load_box(&b_map, &full[stage], dst + (1 + i) * kBoxBytes, x, y, z);
                            }
                        }
                        if (++stage == S) { stage = 0; phase ^= 1u; }
                    }
                }
                for (int s = 0; s < S; ++s)
                    if (pending & (1u << s)) drain_wait(&full[s], (pend_parity >> s) & 1u, err);
                if (!ok) settle_copies();  // some may be of stages that were never announced
            }
        } else if (warp == 1) {
            if (leader) {
                constexpr uint32_t idesc = block_idesc<KIND>(C::ROWS, BN);
                BarrierWalk<true> stages(full, S, 0);
                BarrierWalk<false> slots(tempty, C::SLOTS, 1);
                bool ok = true;
                for (int t = first; ok && t < tiles; t += step) {
                    const BlockTile b = list.at<KIND>(t);
                    const int n = k_hi(b) - k_lo(b);
                    for (int kb = 0; kb < n; ++kb) {
                        ok = stages.wait(abort_flag, err) && slots.wait(abort_flag, err);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t d = tmem + static_cast<uint32_t>(slots.at * BN);
                        const uint64_t ad = byte_desc<C::A_MN>(smem_u32(smem + stages.at * C::STAGE));
                        const uint64_t bd = byte_desc<C::B_MN>(smem_u32(smem + stages.at * C::STAGE + kBoxBytes));
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if constexpr (PAIR) umma_e4m3_pair(d, ad + k * kByteStep<C::A_MN>, bd + k * kByteStep<C::B_MN>, idesc, k != 0);
                                else umma_e4m3(d, ad + k * kByteStep<C::A_MN>, bd + k * kByteStep<C::B_MN>, idesc, k != 0);
                            }
                            if constexpr (PAIR) {
                                umma_commit_pair_multicast(&tfull[slots.at], 0x3);
                                umma_commit_pair_multicast(&empty[stages.at], 0x3);
                            } else {
                                umma_commit(&tfull[slots.at]);
                                umma_commit(&empty[stages.at]);
                            }
                        }
                        __syncwarp();
                        stages.advance();
                        slots.advance();
                    }
                }
                if (elect_one()) {
                    if constexpr (PAIR) umma_commit_pair_multicast(drain, 0x3);
                    else umma_commit(drain);
                }
                __syncwarp();
            }
        } else {
            // scales: rows 4 lane .. of this CTA, and the columns; loaded kAhead steps before their use
            constexpr int kAhead = 2, COLS4 = BN / 128;  // WGRAD: column quads of a lane
            BarrierWalk<false> slots(sempty, C::SLOTS, 1);
            bool ok = true;
            const int nbs = (args.N + kBlock - 1) / kBlock;
            const int in_tile = (PAIR ? static_cast<int>(rank) * kBM : 0) + lane * 4;  // this lane's first row of the tile
            for (int t = first; ok && t < tiles; t += step) {
                const BlockTile b = list.at<KIND>(t);
                const int lo = k_lo(b), hi = k_hi(b);
                const float *sa[4], *sb[2];
                if constexpr (KIND == BLOCK_WGRAD) {
                    sa[0] = args.a_scale + static_cast<long long>(b.k0) * args.M + b.row0 + in_tile;
                    sb[0] = args.b_scale + static_cast<long long>(b.k0) * args.N + b.n0;
                } else {
                    int at[4];  // the row of a_scale, -1: no row
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = b.row0 + in_tile + i;
                        at[i] = in_tile + i >= b.rows ? -1 : (args.a_index ? args.a_index[r] : r);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool in = at[i] >= 0 && at[i] < args.a_scale_rows;
                        if (!in && in_tile + i < b.rows) record_error(err, MOE_DEVERR_BOUNDS);
                        sa[i] = in ? args.a_scale + static_cast<long long>(at[i]) * list.kbs : nullptr;
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // [blocks of F, blocks of D]: FWD walks along a row, DGRAD down a column
                        const int nb = min(b.n0 + h * C::COLS, args.N - 1) / kBlock;
                        sb[h] = args.b_scale + static_cast<long long>(b.e) * list.kbs * nbs + (KIND == BLOCK_FWD ? static_cast<long long>(nb) * list.kbs : nb);
                    }
                }
                float va[kAhead][4], vb[kAhead][KIND == BLOCK_WGRAD ? 4 * COLS4 : 2];
                auto load = [&](int u, int kb) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (KIND == BLOCK_WGRAD) va[u][i] = kb < hi && in_tile + i < b.rows ? sa[0][static_cast<long long>(kb) * args.M + i] : 0.0f;
                        else va[u][i] = kb < hi && sa[i] ? sa[i][kb] : 0.0f;
                    }
                    if constexpr (KIND == BLOCK_WGRAD) {
#pragma unroll
                        for (int c = 0; c < COLS4; ++c) {
                            const int col = c * 128 + lane * 4;
                            const float4 v = kb < hi && b.n0 + col < args.N
                                                 ? *reinterpret_cast<const float4*>(sb[0] + static_cast<long long>(kb) * args.N + col)
                                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            vb[u][4 * c] = v.x, vb[u][4 * c + 1] = v.y, vb[u][4 * c + 2] = v.z, vb[u][4 * c + 3] = v.w;
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) vb[u][h] = kb < hi ? sb[h][KIND == BLOCK_FWD ? kb : static_cast<long long>(kb) * nbs] : 0.0f;
                    }
                };
#pragma unroll
                for (int u = 0; u < kAhead; ++u) load(u, lo + u);
                for (int kb = lo; ok && kb < hi; kb += kAhead) {
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        if (kb + u >= hi) break;
                        ok = slots.wait(abort_flag, err);
                        if (!ok) break;
                        float* dst = scales + slots.at * C::SCALES;
                        if constexpr (KIND == BLOCK_WGRAD) {
                            *reinterpret_cast<float4*>(dst + lane * 4) = make_float4(va[u][0], va[u][1], va[u][2], va[u][3]);
#pragma unroll
                            for (int c = 0; c < COLS4; ++c)
                                *reinterpret_cast<float4*>(dst + kBM + c * 128 + lane * 4) =
                                    make_float4(vb[u][4 * c], vb[u][4 * c + 1], vb[u][4 * c + 2], vb[u][4 * c + 3]);
                        } else {
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                *reinterpret_cast<float4*>(dst + h * kBM + lane * 4) = make_float4(
                                    va[u][0] * vb[u][h], va[u][1] * vb[u][h], va[u][2] * vb[u][h], va[u][3] * vb[u][h]);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&tfull[slots.at]);
                        slots.advance();
                        load(u, kb + u + kAhead);
                    }
                }
            }
        }
    }

    __syncwarp();
    pdl_trigger();
    if constexpr (SPLITS > 1) {  // join the parts in rank order: CTA `part` takes every SPLITS-th row
        cluster_sync_all();
        if (warp >= 4 && first < tiles && !*abort_flag) {
            const BlockTile b = list.at<KIND>(first);
            const uint32_t park = smem_u32(smem);
            uint16_t* out = args.out + (KIND == BLOCK_WGRAD ? static_cast<long long>(b.e) * args.M * args.N : 0);
            const int items = (b.rows - part + SPLITS - 1) / SPLITS * 32;
            for (int it = threadIdx.x - 128; it < items; it += kEpiWarps * 32) {
                const int r = it / 32 * SPLITS + part, quad = it & 31, col = b.n0 + quad * 4;
                if (col >= args.N) continue;
                float4 v[SPLITS];
#pragma unroll
                for (int s = 0; s < SPLITS; ++s) v[s] = ld_part(mapa_shared(park + park_quad(r, quad), s));
#pragma unroll
                for (int s = 1; s < SPLITS; ++s) v[0].x += v[s].x, v[0].y += v[s].y, v[0].z += v[s].z, v[0].w += v[s].w;
                *reinterpret_cast<uint2*>(out + (static_cast<long long>(b.row0) + r) * args.N + col) =
                    make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[0].z, v[0].w));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 32) drain_wait(drain, 0, err);  // the MMAs that wrote this CTA's TMEM have ended
    __syncwarp();
    if constexpr (C::CLUSTER > 1) cluster_sync_all();  // no CTA leaves while another may still signal it or read its part
    else __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
}

template <int KIND, bool PAIR, int BN, int SPLITS>
cudaLaunchConfig_t block_config(int E, long long clusters, cudaLaunchAttribute (&attr)[2], cudaStream_t st) {
    using C = BlockCfg<KIND, PAIR, BN, SPLITS>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * C::CLUSTER));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::smem(E);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(C::CLUSTER), 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cfg;
}

template <int KIND, bool PAIR, int BN, int SPLITS>
cudaError_t block_prepare(int* clusters) {
    static std::atomic<unsigned long long> done{0};
    static int limit[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        auto kern = block_gemm_kernel<KIND, PAIR, BN, SPLITS>;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(BlockCfg<KIND, PAIR, BN, SPLITS>::smem(kMaxE)));
        if (e != cudaSuccess) return e;
        cudaFuncAttributes fa = {};  // the shares that setmaxnreg deals out must fit what the launch gets
        e = cudaFuncGetAttributes(&fa, kern);
        if (e != cudaSuccess) return e;
        if (fa.numRegs * kThreads < kCopyRegs * 128 + kEpiRegs * kEpiWarps * 32) return cudaErrorInvalidConfiguration;
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = block_config<KIND, PAIR, BN, SPLITS>(kMaxE, 1, attr, nullptr);
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        if (e != cudaSuccess) return e;
        limit[dev & 63] = n;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    *clusters = limit[dev & 63];
    return *clusters > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

// st_set: launch; else only tell how many clusters the device holds at once.
template <int KIND, bool PAIR, int BN, int SPLITS>
cudaError_t block_go(const BlockPlan& p, const CUtensorMap* maps, const BlockArgs* a, cudaStream_t st, int* clusters) {
    int limit = 0;
    cudaError_t e = block_prepare<KIND, PAIR, BN, SPLITS>(&limit);
    if (e != cudaSuccess) return e;
    if (clusters) {
        *clusters = limit;
        return cudaSuccess;
    }
    // a part of K is joined once, so its cluster has one tile; whole tiles are walked
    const long long n = SPLITS > 1 ? p.tiles : std::min<long long>(p.tiles, limit);
    if (n < 1 || n * BlockCfg<KIND, PAIR, BN, SPLITS>::CLUSTER > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = block_config<KIND, PAIR, BN, SPLITS>(a->E, n, attr, st);
    return cudaLaunchKernelEx(&cfg, block_gemm_kernel<KIND, PAIR, BN, SPLITS>, maps[0], maps[1], maps[2], *a);
}

}  // namespace

template <int KIND>
cudaError_t block_pick(const BlockPlan& p, const CUtensorMap* maps, const BlockArgs* a, cudaStream_t st, int* clusters) {
    if (p.pair) return block_go<KIND, true, 256, 1>(p, maps, a, st, clusters);
    if (p.bn == 256) return block_go<KIND, false, 256, 1>(p, maps, a, st, clusters);
    switch (p.splits) {
        case 1: return block_go<KIND, false, 128, 1>(p, maps, a, st, clusters);
        case 2: return block_go<KIND, false, 128, 2>(p, maps, a, st, clusters);
        case 4: return block_go<KIND, false, 128, 4>(p, maps, a, st, clusters);
        default: return cudaErrorInvalidConfiguration;
    }
}

}  // namespace moe
