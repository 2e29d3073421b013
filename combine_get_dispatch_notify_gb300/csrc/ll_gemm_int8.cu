// Experts' int8 products on the tensor cores (ep_ll_gemm_int8,
// ep_ll_gemm_swiglu_int8).
//
//   D[j][m] = sum_k w[j][k] a[m][k];  p[m][j] = as[m] ws[j] D[j][m]
//
// sm_103a's tensor cores take no int8, but every int8 value is an fp16 value, so the
// bytes cross memory as int8 and become fp16 on the SM: weights in registers on their way
// into TMEM, from where they are the tensor cores' first operand, an expert's rows on
// their way from one place of shared memory to another.  Products are exact and sums are
// fp32: exact too as long as they stay within 2^24, and beyond that short by a few parts in
// 10^6 at k = 7168, as the tensor cores add (ll_gemm_bf16.cu).  A byte b becomes a number without a
// conversion instruction: b + 128 in the low bits of 1024 makes the fp16 number 1152 + b.
//
// A pair of CTAs (one cluster, two SMs) owns a tile of two blocks of 256 weight
// rows x up to 128 rows of an expert, in steps of 32, and walks k in steps of 128.  Per CTA:
// a producer of weights and one of rows (TMA), four warps that convert each block's weights,
// four that convert the rows, on the pair's first CTA two that feed the tensor cores (a
// block each), eight that scale the sums and write them out.  For the gated product the blocks
// are the gate and the up matrix.  Its activations leave as fp32, because the scale of a row
// is known once the row is complete; a second kernel casts them.
//
// Measured, gated (7168 -> 2 x 2048, with the cast) and plain (2048 -> 7168).  One call by itself with its launch, caches
// emptied before it: 32 experts with about 1024 rows 1270 and 587 us (1.51 and 1.64 PFLOP/s; tensor pipe 65 % busy, more than
// half of the issue slots: the chain from bytes through TMEM to the tensor cores bounds it); 64 experts with about 64 rows 360
// and 177 us, 5.2 and 5.3 TB/s of weights; 8 experts with one row 62 and 41.  Both of them one after the other: 1926 to 1958 us,
// and 1975 to 2072 in long runs, where the power limit takes the clock from 2070 to 1940 MHz; 516 to 526; 75 to 77.  8 experts
// with one row in a captured graph: 46 and 27 us, of which 12 (5 of them the cast) and 7 at k = 128.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "ep.h"
#include "ep_device.cuh"
#include "ep_internal.h"
#include "gated.cuh"
#include "int8_cast.cuh"
#include "ll_gemm_fp8.cuh"
#include "row_tiles.cuh"
#include "tcgen05.cuh"

namespace ep {

namespace {

using gemm::Waits;

constexpr int kBlock = 256;               // weight rows of a block; each CTA has half
constexpr int kHalf = 128;
constexpr int kBlockK = 128;              // int8: one 128-byte swizzled row
constexpr int kWeightBytes = kHalf * kBlockK;          // a CTA's part of a block's step, 16 KB
constexpr int kRowStages = 4;             // of rows: one to each warp that converts them
constexpr int kRowSlots = 3;              // of batches of converted rows, in shared memory
constexpr int kBatchStages = 2;           // stages of rows of a batch
constexpr int kChunk = 16;                // rows of the smaller box of a
// What depends on the most rows of a tile, 128 or 64: with 64 the room that rows and sums leave holds more weights in
// flight and one more converted step of them.
template <int kTileRows>
struct Sizes {
    static constexpr int kStages = kTileRows == 128 ? 6 : 10;         // of weights, a block's step each
    static constexpr int kSlots = kTileRows == 128 ? 2 : 3;           // of converted steps of weights, in TMEM
    static constexpr int kRowBytes = kTileRows / 2 * kBlockK;         // a CTA's part of a stage of rows: one step of a full tile
    static constexpr int kBatchBytes = kBatchStages * 2 * kRowBytes;  // a batch of rows in fp16
    // steps of a stage of rows: as many as have room, by the rows of a tile (a multiple of 32)
    static __device__ __forceinline__ int stage_steps(int width) { return kTileRows / (width > 64 ? 128 : width > 32 ? 64 : 32); }
};
constexpr int kMostStages = 10, kMostSlots = 3;
constexpr int kWeightWarps = 8, kEpilogueWarps = 8;
constexpr int kRowWarps = 4;              // a stage of rows each
constexpr int kFirstEpilogue = 4 + kWeightWarps, kFirstRow = kFirstEpilogue + kEpilogueWarps;  // warps
constexpr int kRelay = kFirstRow + kRowWarps;
constexpr int kThreads = (kRelay + 4) * kWarp;  // whole warpgroups, whose registers are dealt out
static_assert(kRowWarps == kRowStages && kRowWarps == 4, "a warp owns a stage of rows");
constexpr int kTmemColumns = 512;
constexpr int kSlotColumns = kBlockK / 2;              // TMEM columns of a step of weights

struct Params {
    Int8GemmArgs g;
    int kb;
};

struct Shared {
    uint64_t raw_full[kMostStages];   // this CTA's weights have landed
    uint64_t raw_empty[kMostStages];  // its converting warps have read them
    uint64_t in_full[kRowStages];     // this CTA's rows have landed
    uint64_t in_empty[kRowStages];    // the warp that converts them has read them
    uint64_t go[kRowStages];          // the stage's batch has a slot
    uint64_t converted[kRowSlots];    // this CTA's part of a batch of rows is in shared memory
    uint64_t w_full[2][kMostSlots];   // leader's: a block's step is in both CTAs' TMEM
    uint64_t w_empty[2][kMostSlots];  // both: the MMAs that read it are done
    uint64_t rows_full[kRowSlots];    // leader's: a batch of rows is in both CTAs' shared memory
    uint64_t rows_empty[kRowSlots];   // both: both blocks' MMAs that read it are done
    uint64_t acc_full[2];             // both: a block's sums are in TMEM
    uint64_t acc_empty[2];            // leader's: the pair's epilogue warps have read them
    int first[kRowGroups + 2];        // tiles of rows before each group of 32 experts
    uint32_t tmem;
    Waits waits;
};

__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, Waits* w) {
    return gemm::wait_small(bar, parity, w);
}
// At cluster scope: what another CTA's threads wrote before they arrived is visible.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, Waits* w) {
    const long long start = globaltimer_ns();
    do {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait_cluster(bar, parity)) return true;
    } while (globaltimer_ns() - start < w->limit_us * 1000LL);
    *reinterpret_cast<volatile int*>(&w->ran_out) = 1;
    return false;
}

// Four int8 values (lowest byte first) -> two pairs of fp16.
__device__ __forceinline__ void widen(uint32_t v, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = v ^ 0x80808080u;  // + 128
    const __half2 back = __half2half2(__ushort_as_half(0x6480));  // 1152
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);  // 1024 + u
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), back);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), back);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}
// 16 bytes of a swizzled row of shared memory.
__device__ __forceinline__ uint4 row_piece(uint32_t tile, int row, int piece) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(tile + row * 128 + ((piece ^ (row & 7)) << 4)));
    return v;
}

// Several arrivals at once.
__device__ __forceinline__ void mbar_arrive_many(uint64_t* bar, uint32_t count) {
    asm volatile(
        "{\n\t.reg .b64 st;\n\t"
        "mbarrier.arrive.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(smem_addr(bar)),
        "r"(count)
        : "memory");
}

// Matrix m (8 columns x 8 rows, lane T: column T / 4, rows 2 (T % 4) and the next) for m = a, b, c, d -> 16 bytes of row
// lane / 4: the 8 columns of matrix lane % 4.
__device__ __forceinline__ uint4 rows_of_matrices(uint32_t a, uint32_t b, uint32_t c, uint32_t d, int lane) {
    const uint32_t in[4] = {a, b, c, d};
    uint32_t v[4];  // lane T: row T / 4, columns 2 (T % 4) and the next of matrix m
#pragma unroll
    for (int m = 0; m < 4; ++m)
        asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(v[m]) : "r"(in[m]));
    // 4 x 4 words between the four lanes of a row
#pragma unroll
    for (int s = 1; s <= 2; s *= 2) {
        const bool up = (lane & s) != 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t& lo = v[s == 1 ? 2 * i : i];
            uint32_t& hi = v[s == 1 ? 2 * i + 1 : i + 2];
            const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, s);
            if (up)
                lo = got;
            else
                hi = got;
        }
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

template <bool kSwiglu, int kTileRows>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ll_gemm_int8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                        const __grid_constant__ CUtensorMap map_a16, const Params p) {
    using S = Sizes<kTileRows>;
    constexpr int kStages = S::kStages, kSlots = S::kSlots, kRowBytes = S::kRowBytes, kBatchBytes = S::kBatchBytes;
    constexpr int kWeightColumns = 2 * kTileRows;  // TMEM columns: the weights, behind both accumulators
    static_assert(kWeightColumns + 2 * kSlots * kSlotColumns <= kTmemColumns && kStages <= kMostStages && kSlots <= kMostSlots, "");
    extern __shared__ uint8_t s_raw[];
    // swizzled tiles first, on a 1024-byte boundary, at the same offset in both CTAs
    uint8_t* s_stages = s_raw + ((1024u - (smem_addr(s_raw) & 1023u)) & 1023u);
    uint8_t* s_in = s_stages + kStages * kWeightBytes;
    uint8_t* s_rows = s_in + kRowStages * kRowBytes;
    Shared* s = reinterpret_cast<Shared*>(s_rows + kRowSlots * kBatchBytes);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / kWarp, 0), lane = threadIdx.x % kWarp;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s->raw_full[i], 1);
            mbar_init(&s->raw_empty[i], kWeightWarps / 2);
        }
        for (int i = 0; i < kSlots; ++i)
            for (int h = 0; h < 2; ++h) {
                mbar_init(&s->w_full[h][i], kWeightWarps);  // half of them, in both CTAs
                mbar_init(&s->w_empty[h][i], 1);
            }
        for (int i = 0; i < kRowStages; ++i) {
            mbar_init(&s->in_full[i], 1);
            mbar_init(&s->in_empty[i], 1);
            mbar_init(&s->go[i], 1);
        }
        for (int i = 0; i < kRowSlots; ++i) {
            mbar_init(&s->converted[i], kBatchStages);
            mbar_init(&s->rows_full[i], 2);
            mbar_init(&s->rows_empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->acc_full[i], 1);
            mbar_init(&s->acc_empty[i], kSwiglu ? 2 * kEpilogueWarps : kEpilogueWarps);  // of the pair
        }
        s->waits = Waits{0, p.g.stall.wait_limit_us};
        fence_mbarrier_init();
        prefetch_tensormap(&map_w);
        prefetch_tensormap(&map_a);
    }
    if (warp == 4) tmem_alloc_pair(&s->tmem, kTmemColumns);
    // The pair's barriers and TMEM are ready; the other half of this barrier, below, is behind the counts' way from memory (0.4
    // us a call saved).
    __syncwarp();
    cluster_arrive_release();
    griddep_wait();  // counts, rows and scales are complete from here on
    griddep_launch_dependents();
    RowTiles<kTileRows, false> walk{p.g.count, s->first, p.g.E, p.g.cap};
    const int columns = (p.g.n + kBlock - 1) / kBlock;
    if (warp == 1) walk.fill(s->first, lane, columns, pairs);
    tc_fence_before();
    __syncthreads();
    cluster_wait_acquire();
    tc_fence_after();
    const uint32_t tmem = s->tmem;
    walk.start();
    const int row_tiles = walk.row_tiles();
    const int blocks = kSwiglu ? 2 : blocks_of_tiles(row_tiles, columns, pairs);
    walk.tiles_n = kSwiglu ? columns : (columns + blocks - 1) / blocks;
    const int tiles = row_tiles * walk.tiles_n;
    // first output column of a tile (its second block may lie past the last one)
    const auto first_column = [&](const RowTile& t) { return t.col * (kSwiglu ? 1 : blocks) * kBlock; };
    // Steps of weights, all of the pair's tiles in turn.  Where tiles have two blocks, the first group of converting warps,
    // the first MMA warp and the first accumulator have the first block's and the second ones the second's.  Where
    // they have one, the groups take every other step, the first MMA warp does them all, and the accumulators take turns by
    // tile.  Either way unit number 2 i + g, in the order of the loads, is the i-th of group g.
    const uint32_t steps = tiles > pair ? static_cast<uint32_t>((tiles - pair + pairs - 1) / pairs) * p.kb : 0;
    // rows of a tile as the tensor cores take them
    const auto width = [&](const RowTile& t) { return (t.rows + 31) / 32 * 32; };

    if (warp < 4) regs_down<40>();
    if (warp == 0) {
        if (lane == 0) {
            // ---- producer: this CTA's half of the weights ----
            uint32_t it = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const RowTile tl = walk.at(t);
                const int w0 = first_column(tl) + static_cast<int>(rank) * kHalf;
                for (int u = 0; u < p.kb * blocks; ++u, ++it) {
                    const uint32_t st = it % kStages;
                    if (!(ok = wait_for(&s->raw_empty[st], it / kStages & 1 ^ 1, &s->waits))) break;
                    const int b = blocks == 2 ? u / 2 : u, i = blocks == 2 ? u % 2 : 0;
                    mbar_arrive_expect_tx(&s->raw_full[st], kWeightBytes);
                    tma_load_3d_alone(smem_addr(s_stages) + st * kWeightBytes, &map_w, b * kBlockK, kSwiglu ? w0 : w0 + i * kBlock,
                                      kSwiglu ? 2 * tl.e + i : tl.e, smem_addr(&s->raw_full[st]));
                }
            }
            // every stage has been read before the CTA may leave
            for (int i = 0; i < kStages && ok; ++i, ++it)
                ok = wait_for(&s->raw_empty[it % kStages], it / kStages & 1 ^ 1, &s->waits);
        }
    } else if (warp == 3) {
        if (lane == 0) {
            // ---- producer of rows: apart, because they have to be ahead of the weights ----
            uint32_t it = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const RowTile tl = walk.at(t);
                const int n = width(tl), a0 = tl.m0 + static_cast<int>(rank) * (n / 2), in_stage = S::stage_steps(n);
                for (int b0 = 0; b0 < p.kb; b0 += in_stage, ++it) {
                    const uint32_t st = it % kRowStages;
                    if (!(ok = wait_for(&s->in_empty[st], it / kRowStages & 1 ^ 1, &s->waits))) break;
                    const uint32_t bar = smem_addr(&s->in_full[st]);
                    uint32_t to = smem_addr(s_in) + st * kRowBytes;
                    const int steps = min(in_stage, p.kb - b0);
                    mbar_arrive_expect_tx(&s->in_full[st], steps * (n / 2) * kBlockK);
                    for (int b = b0; b < b0 + steps; ++b, to += n / 2 * kBlockK)
                        if (n == kTileRows)
                            tma_load_3d_alone(to, &map_a, b * kBlockK, a0, tl.e, bar);
                        else
                            for (int i = 0; i < n / 2; i += kChunk)
                                tma_load_3d_alone(to + i * kBlockK, &map_a16, b * kBlockK, a0 + i, tl.e, bar);
                }
            }
            for (int i = 0; i < kRowStages && ok; ++i, ++it)
                ok = wait_for(&s->in_empty[it % kRowStages], it / kRowStages & 1 ^ 1, &s->waits);
        }
    } else if (warp == 1 || warp == 2) {
        const uint32_t half = warp - 1;
        if (rank == 0 && half < static_cast<uint32_t>(blocks)) {
            // ---- MMA ----
            uint32_t batch = 0, it = 0;  // batches of rows and steps so far
            bool ok = true;
            for (uint32_t t = pair, i = 0; t < static_cast<uint32_t>(tiles) && ok; t += pairs, ++i) {
                if (pair == p.g.stall.pair && static_cast<int>(i) >= p.g.stall.tile) break;  // testing hook
                const int n = __shfl_sync(0xffffffffu, width(walk.at(t)), 0), in_batch = kBatchStages * S::stage_steps(n);
                const uint32_t idesc = f16_idesc(kBlock, n), step_bytes = kBatchBytes / in_batch;
                const uint32_t acc = blocks == 2 ? half : i & 1, before = blocks == 2 ? i : i / 2;  // its tiles before this one
                ok = __all_sync(0xffffffffu, wait_for(&s->acc_empty[acc], before & 1 ^ 1, &s->waits));
                for (int b = 0; b < p.kb && ok; ++b, ++it) {
                    const uint32_t rs = batch % kRowSlots, g = blocks == 2 ? half : it & 1, unit = blocks == 2 ? it : it / 2;
                    const uint32_t ws = unit % kSlots;
                    const int at = b % in_batch;
                    if (at == 0) ok = wait_cluster(&s->rows_full[rs], batch / kRowSlots & 1, &s->waits);
                    ok = ok && wait_for(&s->w_full[g][ws], unit / kSlots & 1, &s->waits);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const bool end = at + 1 == in_batch || b + 1 == p.kb;
                    uint64_t db = sw128_desc(smem_addr(s_rows) + rs * kBatchBytes + at * step_bytes);
                    asm volatile("" : "+l"(db));
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t a = tmem + kWeightColumns + (g * kSlots + ws) * kSlotColumns;
#pragma unroll
                        for (int k = 0; k < kBlockK / 16; ++k)
                            mma_f16_pair_tmem(tmem + acc * kTileRows, a + k * 8, db + k / 4 * (step_bytes >> 5) + k % 4 * 2, idesc,
                                              b > 0 || k > 0);
                        mma_commit_pair(smem_addr(&s->w_empty[g][ws]));
                        if (end) mma_commit_pair(smem_addr(&s->rows_empty[rs]));
                        if (end && blocks == 1) mma_commit_pair(smem_addr(&s->rows_empty[rs]));  // for the other warp
                        if (b + 1 == p.kb) mma_commit_pair(smem_addr(&s->acc_full[acc]));
                    }
                    __syncwarp();
                    if (end) ++batch;
                }
            }
        }
    } else if (warp >= 4 && warp < kFirstEpilogue) {
        // ---- weights: two groups of four warps; thread = one weight row, 128 bytes a step -> 64 columns of TMEM.  Arrivals are relaxed: what they
        // announce is in TMEM, which the tcgen05 waits and fences on both sides put in order ----
        regs_down<64>();
        const uint32_t g = (warp - 4) / 4, quarter = warp % 4;
        const int row = quarter * kWarp + lane;
        const uint32_t to = tmem + (quarter * kWarp << 16) + kWeightColumns + g * kSlots * kSlotColumns;
        const uint32_t full = mapa(smem_addr(&s->w_full[g][0]), 0);
        const uint32_t units = blocks == 2 ? steps : (steps + 1 - g) / 2;
        for (uint32_t u = 0; u < units; ++u) {
            const uint32_t st = (2 * u + g) % kStages, ws = u % kSlots;
            const bool ok = wait_for(&s->raw_full[st], (2 * u + g) / kStages & 1, &s->waits) &&
                            wait_for(&s->w_empty[g][ws], u / kSlots & 1 ^ 1, &s->waits);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const uint32_t from = smem_addr(s_stages) + st * kWeightBytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t v[32];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 x = row_piece(from, row, 4 * h + j);
                    widen(x.x, v[8 * j], v[8 * j + 1]);
                    widen(x.y, v[8 * j + 2], v[8 * j + 3]);
                    widen(x.z, v[8 * j + 4], v[8 * j + 5]);
                    widen(x.w, v[8 * j + 6], v[8 * j + 7]);
                }
                tmem_write(to + ws * kSlotColumns + h * 32, v);
            }
            // the bytes are in registers: their stage can be filled again while TMEM takes them
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->raw_empty[st]);
            tmem_write_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(full + ws * 8);
        }
    } else if (warp >= kRelay) {
        regs_down<48>();
        if (warp == kRelay && lane == 0) {
            // ---- relay: batches of rows, as this CTA's part of each is complete, announced to the pair's first CTA.  That
            // releases shared memory to the cluster, and an SM gets through one such release in some 1700 cycles
            // however many warps ask for one, where the tensor cores take 1024 for a full step: hence the batches ----
            const uint32_t full = mapa(smem_addr(&s->rows_full[0]), 0);
            uint32_t batch = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const int in_batch = kBatchStages * S::stage_steps(width(walk.at(t)));
                for (int b = 0; b < p.kb; b += in_batch, ++batch) {
                    const uint32_t rs = batch % kRowSlots;
                    if (!(ok = wait_for(&s->converted[rs], batch / kRowSlots & 1, &s->waits))) break;
                    mbar_arrive_cluster(full + rs * 8);
                }
            }
        } else if (warp == kRelay + 1 && lane == 0) {
            // ---- gate: each stage's converting warp told that the stage's batch has a slot.  A barrier tells phases apart by
            // one bit, so the warps, which take some of the stages, could not wait for all of the slots in turn ----
            uint32_t it = 0, batch = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const int in_stage = S::stage_steps(width(walk.at(t)));
                for (int b = 0, g = 0; b < p.kb; b += in_stage, ++g, ++it) {
                    const uint32_t st = it % kRowStages;
                    if (g % kBatchStages == 0) {
                        ok = wait_for(&s->rows_empty[batch % kRowSlots], batch / kRowSlots & 1 ^ 1, &s->waits);
                        ++batch;
                    }
                    if (!(ok = ok && wait_for(&s->in_empty[st], it / kRowStages & 1 ^ 1, &s->waits))) break;
                    mbar_arrive(&s->go[st]);
                }
            }
        }
    } else if (warp >= kFirstRow) {
        // ---- rows: a stage to each of four warps in turn, 128 bytes of a row -> two halves of 64 fp16 in swizzled rows ----
        regs_down<48>();
        const uint32_t st = warp - kFirstRow, from = smem_addr(s_in) + st * kRowBytes;  // the warp's stage
        uint32_t batches = 0, stages = 0;  // before this tile
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
            const int n = width(walk.at(t)), mine = n / 2, in_stage = S::stage_steps(n);  // mine: rows of this CTA
            const int all = (p.kb + in_stage - 1) / in_stage;                          // stages of this tile
            const uint32_t step_bytes = kBatchBytes / (kBatchStages * in_stage);
            for (int g = (st - stages) % kRowStages; g < all; g += kRowStages) {
                const uint32_t batch = batches + g / kBatchStages, rs = batch % kRowSlots, phase = (stages + g) / kRowStages & 1;
                ok = __all_sync(0xffffffffu, wait_for(&s->go[st], phase, &s->waits) && wait_for(&s->in_full[st], phase, &s->waits));
                if (!ok) break;
                const int lines = min(in_stage, p.kb - g * in_stage) * mine;
                const uint32_t slot = smem_addr(s_rows) + rs * kBatchBytes + g % kBatchStages * in_stage * step_bytes;
#pragma unroll 1
                for (int line = lane; line < lines; line += kWarp) {
                    const int step = in_stage == 1 ? 0 : line / mine, row = line - step * mine;
                    const uint32_t to = slot + step * step_bytes + row * 128;
#pragma unroll (kTileRows == 64 ? 2 : 8)
                    for (int j = 0; j < 8; ++j) {  // 16 values; steps are whole groups of eight rows apart, so `line` swizzles as `row`
                        const uint4 x = row_piece(from, line, j);
                        uint32_t v[8];
                        widen(x.x, v[0], v[1]);
                        widen(x.y, v[2], v[3]);
                        widen(x.z, v[4], v[5]);
                        widen(x.w, v[6], v[7]);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                             to + j / 4 * (step_bytes / 2) + (((j % 4 * 2 + h) ^ (row & 7)) << 4)),
                                         "r"(v[4 * h]), "r"(v[4 * h + 1]), "r"(v[4 * h + 2]), "r"(v[4 * h + 3])
                                         : "memory");
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s->in_empty[st]);
                    // a tile's last batch may be one stage short: its last stage arrives for that too
                    mbar_arrive_many(&s->converted[rs], g + 1 == all ? kBatchStages - g % kBatchStages : 1);
                }
            }
            batches += (all + kBatchStages - 1) / kBatchStages;
            stages += all;
        }
    } else if (warp >= kFirstEpilogue) {
        // ---- epilogue: lane = one output column, a quarter of a block's 128 to a warp ----
        regs_up<120>();
        const int half = (warp - kFirstEpilogue) / 4, quarter = warp % 4;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * kWarp) << 16);
        const uint32_t empty = mapa(smem_addr(&s->acc_empty[0]), 0);
        uint32_t acc_phase = 0;
        bool ok = true;
        const auto hand_back = [&](int h) {
            tc_fence_before();
            if (lane == 0) mbar_arrive_cluster_relaxed(empty + h * 8);
        };
        for (int t = pair, i = 0; t < tiles && ok; t += pairs, ++i) {
            const RowTile tl = walk.at(t);
            if (blocks == 1 && (i & 1) != half) continue;
            const int block = kSwiglu || blocks == 1 ? 0 : half;
            const int col = first_column(tl) + block * kBlock + static_cast<int>(rank) * kHalf + quarter * kWarp + lane;
            const bool on = col < p.g.n;
            const long long r0 = static_cast<long long>(tl.e) * p.g.cap + tl.m0;
            const float* ws = p.g.w_scales + static_cast<long long>(tl.e) * (kSwiglu ? 2 : 1) * p.g.n + col;
            const float s0 = on ? __ldg(ws) : 0.0f, s1 = on && kSwiglu ? __ldg(ws + p.g.n) : 0.0f;
            const int rows = tl.rows;
            float scale[kTileRows / 32];  // of row 32 i + lane
#pragma unroll
            for (int c = 0; c < kTileRows; c += 32) scale[c / 32] = c + lane < rows ? __ldg(p.g.a_scales + r0 + c + lane) : 0.0f;
            ok = wait_for(&s->acc_full[half], acc_phase, &s->waits);
            if (kSwiglu) ok = ok && wait_for(&s->acc_full[half ^ 1], acc_phase, &s->waits);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            acc_phase ^= 1;
            tc_fence_after();
            if (kSwiglu) {
                // 32 rows at a time, in turn for the two warps of a quarter.  Short calls find none of their instructions on the SM:
                // few rows go through a small loop (8 experts with one row, both products in turn 78 -> 73 us; 1024 rows 1332 -> 1429)
                constexpr int kPart = kTileRows == 64 ? 8 : 32;
#pragma unroll 1
                for (int c = half * 32; c < kTileRows; c += 64) {
                    float of_rows = scale[0];  // the scales of these rows
#pragma unroll
                    for (int k = 1; k < kTileRows / 32; ++k)
                        if (c == 32 * k) of_rows = scale[k];
#pragma unroll 1
                    for (int part = 0; part < 32; part += kPart) {
                        const int r = c + part;
                        uint64_t x[kPart / 2], y[kPart / 2];
                        if (r < rows) tmem_read2(lanes + r, lanes + kTileRows + r, x, y);
                        if (c + 64 >= kTileRows && part + kPart == 32) {
                            hand_back(0);
                            hand_back(1);
                        }
                        if (r >= rows) continue;
                        float* to = p.g.h + (r0 + r) * p.g.n + col;
#pragma unroll
                        for (int j = 0; j < kPart; ++j) {
                            const float as = __shfl_sync(0xffffffffu, of_rows, part + j);
                            const float2 a = unpack2(x[j / 2]), b = unpack2(y[j / 2]);
                            const float gate = (j & 1 ? a.y : a.x) * (as * s0), up = (j & 1 ? b.y : b.x) * (as * s1);
                            if (on && r + j < rows) to[static_cast<long long>(j) * p.g.n] = gated_unit<false>(gate, up);
                        }
                    }
                }
            } else {
                // All rows into registers, so that the accumulator is free while they are stored: as 8 x 8 matrices of
                // columns and rows, which are then transposed between the lanes so that each stores 16 bytes of a row.
                // (Columns stored by their lanes, 2 bytes each, took 9 us a tile, three quarters of its time at k = 512.)
                uint32_t v[kTileRows / 2];
                float ws[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) ws[m] = __shfl_sync(0xffffffffu, s0, 8 * m + lane / 4);
#pragma unroll
                for (int c = 0; c < kTileRows; c += 32)
                    if (c < rows) {
                        uint64_t x[16];
                        tmem_read_matrices(lanes + half * kTileRows + c, x);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float as0 = __shfl_sync(0xffffffffu, scale[c / 32], 8 * j + lane % 4 * 2);
                            const float as1 = __shfl_sync(0xffffffffu, scale[c / 32], 8 * j + lane % 4 * 2 + 1);
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const float2 d = unpack2(x[4 * j + m]);
                                const __nv_bfloat162 h = __floats2bfloat162_rn(d.x * (as0 * ws[m]), d.y * (as1 * ws[m]));
                                v[c / 2 + 4 * j + m] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                        }
                    }
                hand_back(half);
                const int to_col = col - lane + lane % 4 * 8;  // of this lane's 16 bytes
                uint16_t* to = static_cast<uint16_t*>(p.g.y) + r0 * p.g.n + to_col;
#pragma unroll
                for (int c = 0; c < kTileRows; c += 8)
                    if (c < rows) {
                        const uint4 w = rows_of_matrices(v[c / 2], v[c / 2 + 1], v[c / 2 + 2], v[c / 2 + 3], lane);
                        if (c + lane / 4 < rows && to_col < p.g.n) st_v4(to + static_cast<long long>(c + lane / 4) * p.g.n, w);
                    }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (s->waits.ran_out != 0) {
        // a wait ran out: let the copies and products still in flight land before shared memory and TMEM go
        const long long start = globaltimer_ns();
        while (globaltimer_ns() - start < 10000000LL) {
        }
        if (threadIdx.x == 0) flag_error(p.g.status, EP_DEV_TIMEOUT);
    }
    cluster_arrive_release();
    cluster_wait_acquire();
    tc_fence_after();
    if (warp == 4) tmem_dealloc_pair(tmem, kTmemColumns);
}

// ---- the gated product's rows, cast: a CTA to a row, which it holds in registers up to 4096 columns ----
constexpr int kCastThreads = 256;
constexpr int kCastPasses = 4;  // of four columns a thread

__global__ void __launch_bounds__(kCastThreads) cast_rows_kernel(const Int8GemmArgs p) {
    __shared__ uint32_t s_max[2][kCastThreads / kWarp];
    griddep_launch_dependents();
    griddep_wait();
    int turn = 0;
    for (long long r = blockIdx.x; r < static_cast<long long>(p.E) * p.cap; r += gridDim.x) {
        const int e = static_cast<int>(r / p.cap), m = static_cast<int>(r - static_cast<long long>(e) * p.cap);
        if (m >= __ldg(p.count + e)) continue;
        const float4* h = reinterpret_cast<const float4*>(p.h + r * p.n);
        const int pieces = p.n / 4, held = kCastThreads * kCastPasses;
        float4 v[kCastPasses];
        uint32_t most = 0;  // bits of the largest magnitude; NaN is above them all
        const auto larger = [&](const float4& x) {
            most = max(max(most, max(__float_as_uint(fabsf(x.x)), __float_as_uint(fabsf(x.y)))),
                       max(__float_as_uint(fabsf(x.z)), __float_as_uint(fabsf(x.w))));
        };
#pragma unroll
        for (int i = 0; i < kCastPasses; ++i) {
            const int c = i * kCastThreads + threadIdx.x;
            v[i] = c < pieces ? h[c] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int i = 0; i < kCastPasses; ++i) larger(v[i]);
        for (int c = held + threadIdx.x; c < pieces; c += kCastThreads) larger(h[c]);
        most = __reduce_max_sync(0xffffffffu, most);
        // two places take turns: passing this row's barrier says that the last one's maxima have been read
        if (threadIdx.x % kWarp == 0) s_max[turn][threadIdx.x / kWarp] = most;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kCastThreads / kWarp; ++i) most = max(most, s_max[turn][i]);
        turn ^= 1;
        const float scale = row_scale(__uint_as_float(most));
        const bool finite = most < 0x7f800000u;
        uint32_t* y = reinterpret_cast<uint32_t*>(static_cast<int8_t*>(p.y) + r * p.n);
        const auto cast = [&](const float4& x) {
            return finite ? pack_int8x4(x.x / scale, x.y / scale, x.z / scale, x.w / scale) : 0u;
        };
#pragma unroll
        for (int i = 0; i < kCastPasses; ++i) {
            const int c = i * kCastThreads + threadIdx.x;
            if (c < pieces) y[c] = cast(v[i]);
        }
        for (int c = held + threadIdx.x; c < pieces; c += kCastThreads) y[c] = cast(h[c]);
        if (threadIdx.x == 0) p.y_scales[r] = scale;
    }
}

template <bool kSwiglu, int kTileRows>
cudaError_t launch(const Int8GemmArgs& g, cudaStream_t stream) {
    using S = Sizes<kTileRows>;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const Params p = {g, (g.k + kBlockK - 1) / kBlockK};
    CUtensorMap w, a, a16;
    if (!gemm::make_map(&w, g.w, g.k, g.n, g.E * (kSwiglu ? 2 : 1), kHalf) ||
        !gemm::make_map(&a, g.a, g.k, g.cap, g.E, kTileRows / 2) || !gemm::make_map(&a16, g.a, g.k, g.cap, g.E, kChunk))
        return cudaErrorInvalidValue;
    const size_t smem = 1024 + S::kStages * kWeightBytes + kRowStages * S::kRowBytes + kRowSlots * S::kBatchBytes + sizeof(Shared);
    // an upper bound of the tiles: the counts are on the device
    const long long most = static_cast<long long>(g.E) * ((g.cap + kTileRows / 2 - 1) / (kTileRows / 2)) * ((g.n + kBlock - 1) / kBlock);
    const int pairs = static_cast<int>(most < sms / 2 ? most : sms / 2);
    return launch_pdl(ll_gemm_int8_kernel<kSwiglu, kTileRows>, dim3(2 * pairs), dim3(kThreads), smem, stream, 0, true, w, a, a16, p);
}

// Tiles of 64 rows where no expert can have more.  The host knows the capacity, not the rows, and a kernel's shared memory and
// TMEM are laid out for its tiles.  So few rows in buffers of a larger capacity go through tiles of 128, with fewer
// weights in flight and the epilogue of many rows: one row to each of 8 experts, both products, 75 us at a capacity of 16, 77 at
// 64, 85 at 72, 87 at 128 (16 tokens of 32 experts: 237, 239, 252, 254), and 101 (269) at 1280, where the cast also
// passes over 40960 rows' places.
template <bool kSwiglu>
cudaError_t launch(const Int8GemmArgs& g, cudaStream_t stream) {
    return g.cap <= 64 ? launch<kSwiglu, 64>(g, stream) : launch<kSwiglu, 128>(g, stream);
}

}  // namespace

cudaError_t launch_ll_gemm_int8(const Int8GemmArgs& g, cudaStream_t stream) {
    if (g.y_scales == nullptr) return launch<false>(g, stream);
    const cudaError_t e = launch<true>(g, stream);
    if (e != cudaSuccess) return e;
    const long long rows = static_cast<long long>(g.E) * g.cap;
    return launch_pdl(cast_rows_kernel, dim3(static_cast<unsigned>(rows < 4096 ? rows : 4096)), dim3(kCastThreads), 0,
                      stream, 0, false, g);
}

}  // namespace ep
