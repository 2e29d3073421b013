// Experts' bf16 products and their gradients on the tensor cores
// (ep_ll_gemm_bf16 and its neighbours).
//
//   kPlain, kSwiglu    D[j][m] = sum_c w[j][c] r[m][c]
//   kDgrad, kDswiglu   D[j][m] = sum_c w[c][j] r[m][c]
//   kWgrad             D[i][j] = sum_m r[m][i] a[m][j]    over an expert's rows
//
// A pair of CTAs (one cluster, two SMs) owns a tile of two blocks of 256 rows of the first
// operand x up to 256 rows of the second and walks the contraction in steps of 64: each
// CTA loads its own half of every block with swizzled TMA, two warps feed the pair's
// tensor cores (tcgen05.mma, K = 16), one for each block of 256, and the sums stay in TMEM
// until the tile is done.  Whether an operand's rows of memory run along the contraction
// or across it is settled by its descriptor: nothing is transposed in memory.
//
// In the forms over rows the weights are the first operand and an expert's rows the
// second, because that one's size goes in steps of 32: an expert's last rows cost
// the tensor cores what they are, not a whole tile.  The sums then lie transposed in
// TMEM (lane = output column) and go through 8 x 8 matrix stores into rows again.  For
// the gated product the two blocks are the gate and the up matrix, so both projections
// of an output meet in one thread.
//
// An expert's rows are the contraction of a weight gradient and may end inside a
// step of 64: its last 16 rows are then zeroed behind them in shared memory, in both
// operands, because what lies there may be a NaN.
//
// The tensor cores' fp32 sums come out short, as if what lies below a sum's last bit were cut off and not rounded: of n terms
// by about n 2^-30 of their magnitude (weight gradients of normal values, fp32, error against 64 bits: 4.7e-7 at 512 rows, 2.1e-6
// at 2048, 9.1e-6 at 8192, 3.8e-5 at 32768; the library's bf16 product gives the same).  A result in bf16 is rounded far more;
// fp32 gradients of long experts carry that error, because a second sum beside the first would take the room that the second
// block of a tile has.
//
// Bound by the tensor cores where experts have hundreds of rows, by the weights' bytes where they have few.  One call by itself
// with its launch, caches emptied before it, 32 experts with exactly 1024 rows, 7168 / 2048 (the longer times where the calls
// before brought the card to its power limit): gated 1026 to 1048 us (1.84 to 1.88 PFLOP/s; its loads alone take 653, its
// products without most of the loads 895), last product 549 to 564 (1.71 to 1.75), gradient through the activation 630 to 648
// (1.49 to 1.53), rows' gradient 1008 to 1087 (1.77 to 1.91), weight gradient in bf16 1057 to 1260 (1.53 to 1.82).  Rows that are not a multiple of 256 cost more than
// their share, because an expert's last tile reads all of its weights again: about 1024 rows, half of
// the experts with a few more, gated 1145 to 1199 us.  8 experts with one row: gated 74 us in a captured graph (6.4 TB/s), last
// product 38 (6.1); by themselves with their launches 94 and 55, and 113 to 117 the two of them among other calls.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ep.h"
#include "ep_device.cuh"
#include "ep_internal.h"
#include "gated.cuh"
#include "ll_gemm_fp8.cuh"
#include "row_tiles.cuh"
#include "tcgen05.cuh"

namespace ep {

namespace {

using gemm::Waits;

constexpr int kBlock = 256;                    // rows of a block of the first operand; each CTA has half
constexpr int kTileRows = 256;                 // most rows of the second operand
constexpr int kHalf = 128;
constexpr int kBlockK = 64;                    // bf16: one 128-byte swizzled row
constexpr int kBox = kBlockK * 128;            // 64 rows x 128 bytes, 8 KB
constexpr int kOperand = 2 * kBox;             // 128 rows of an operand
constexpr int kStageBytes = 3 * kOperand;      // two blocks of the first operand, one of the second
constexpr int kChunk = 16;                     // rows of the smaller box of the rows operand
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 128 + kEpilogueWarps * kWarp;  // producer, two MMA warps, relay | epilogue
constexpr int kTmemColumns = 512;
constexpr int kOutCols = 32, kOutRows = 32;    // of a warp's box of output
constexpr int kOutBytes = kOutCols * kOutRows * 2;

// Where gate and up come in on the way out, a stage is given up for twice the buffers of an epilogue warp.
template <Bf16Form kForm>
constexpr bool kWide = kForm == Bf16Form::kDswiglu;
constexpr int kMostStages = 4;

struct Params {
    Bf16GemmArgs g;
    int kb;                // steps of the contraction (forms over rows)
    int out_n;             // columns of the output (of each half of it)
    int tiles_m, tiles_n;  // kWgrad: tiles of output rows and columns
};

struct Shared {
    uint64_t full[kMostStages];    // leader's: both CTAs' bytes have landed
    uint64_t landed[kMostStages];  // kWgrad, each CTA's own: the bytes of a step that ends an expert's rows
    uint64_t empty[kMostStages];   // both: the MMAs that read the stage are done
    uint64_t acc_full[2];          // both: a block's sums are in TMEM
    uint64_t acc_empty[2];         // leader's: the pair's epilogue warps have read them
    uint64_t loaded[kEpilogueWarps][2];  // kDswiglu: gate and up are in the warp's buffers
    int first[kRowGroups + 2];     // tiles before each group of 32 experts
    uint32_t tmem;
    uint32_t asked;  // kWgrad: stages that this CTA's producer has asked for so far
    Waits waits;
};

__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, Waits* w) {
    return gemm::wait_for<true>(bar, parity, w);  // the limit is read only once a wait is slow
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

// For waits that may be for something many tiles ahead, which take as long as the call does: the limit is for the time in which
// the CTA's ring stands still, and begins again with every stage that its producer has asked for.
__device__ __forceinline__ bool wait_while_moving(uint64_t* bar, uint32_t parity, Waits* w, const uint32_t* asked) {
    long long start = 0;
    uint32_t seen = 0;
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (i % 64 != 0) continue;
        const long long now = globaltimer_ns();
        const uint32_t moved = *reinterpret_cast<const volatile uint32_t*>(asked);
        if (start == 0 || moved != seen) start = now;
        seen = moved;
        if (now - start > w->limit_us * 1000LL) break;
    }
    *reinterpret_cast<volatile int*>(&w->ran_out) = 1;
    return false;
}

// A place in the ring of stages.
template <int kStages>
struct Ring {
    uint32_t at = 0, phase;
    __device__ __forceinline__ explicit Ring(uint32_t first_phase) : phase(first_phase) {}
    __device__ __forceinline__ void next() {
        if (++at == kStages) {
            at = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ void skip(uint32_t steps) {
        const uint32_t to = at + steps;
        phase ^= to / kStages & 1;
        at = to % kStages;
    }
};

// One tile of either kind.
struct Tile {
    int e;
    int a0;      // first row of the first operand's first block (an output column; kWgrad: an output row)
    int blocks;  // that hold any
    int b0;      // kWgrad: first output column
    int m0;      // forms over rows: first row of the expert
    int rows;    // valid rows: of the tile; kWgrad: of the expert
};

// The tiles of this pair in turn.
template <Bf16Form kForm>
struct Tiles {
    static constexpr bool kWgrad = kForm == Bf16Form::kWgrad;
    const Params& p;
    RowTiles<kTileRows, kForm == Bf16Form::kSwiglu> walk;
    int blocks = 2;  // of a tile (1: a tile is one block, the two accumulators take turns)

    __device__ __forceinline__ Tile at(int t) {
        Tile r;
        if (kWgrad) {
            const int per = p.tiles_m * p.tiles_n, local = t - t / per * per;
            r.e = t / per;
            r.a0 = local / p.tiles_n * blocks * kBlock;
            r.b0 = local % p.tiles_n * kTileRows;
            r.rows = walk.rows_of(r.e);
            r.m0 = 0;
            r.blocks = min(blocks, (p.g.n - r.a0 + kBlock - 1) / kBlock);
        } else {
            const RowTile w = walk.at(t);
            r.e = w.e;
            r.m0 = w.m0;
            r.rows = w.rows;
            r.b0 = 0;
            if (kForm == Bf16Form::kSwiglu) {
                r.a0 = w.col * kBlock;
                r.blocks = 2;
            } else {
                r.a0 = w.col * blocks * kBlock;
                r.blocks = min(blocks, (p.out_n - r.a0 + kBlock - 1) / kBlock);
            }
        }
        return r;
    }
    // Steps of 64 of the contraction in a stage: two where a tile is one block and has up to 128 rows, so that as many bytes
    // of the weights are in flight as with two blocks (eight experts with one row each, 2048 -> 7168: 55 us, with
    // one step to a stage 60).
    __device__ __forceinline__ int in_stage(const Tile& t) const {
        return kForm != Bf16Form::kSwiglu && !kWgrad && blocks == 1 && t.rows <= kTileRows / 2 ? 2 : 1;
    }
    // Stages of a tile.
    __device__ __forceinline__ int stages(const Tile& t) const {
        return kWgrad ? (t.rows + kBlockK - 1) / kBlockK : (p.kb + in_stage(t) - 1) / in_stage(t);
    }
};
// The block that accumulator `half` has of the pair's tile number `i`, or -1.
__device__ __forceinline__ int block_of(const Tile& t, int blocks, int i, int half) {
    if (blocks == 2) return half < t.blocks ? half : -1;
    return (i & 1) == half ? 0 : -1;
}

__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
    const __nv_bfloat162 h = __float22bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <Bf16Form kForm, bool kOut16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ll_gemm_bf16_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                        const __grid_constant__ CUtensorMap map_b16, const __grid_constant__ CUtensorMap map_out,
                        const __grid_constant__ CUtensorMap map_gate_up, const Params p) {
    constexpr bool kWgrad = kForm == Bf16Form::kWgrad;
    constexpr bool kSwiglu = kForm == Bf16Form::kSwiglu, kDswiglu = kForm == Bf16Form::kDswiglu;
    constexpr bool kAcrossA = kWgrad || kForm == Bf16Form::kDgrad || kDswiglu;  // its rows of memory run across the contraction
    constexpr int kStages = kWide<kForm> ? 3 : 4;
    constexpr int kBufBytes = kWide<kForm> ? 4 * kOutBytes : 2 * kOutBytes;  // of an epilogue warp
    extern __shared__ uint8_t s_raw[];
    // stages first, on a 1024-byte boundary as the swizzle needs, at the same offset in both CTAs
    uint8_t* s_tiles = s_raw + ((1024u - (smem_addr(s_raw) & 1023u)) & 1023u);
    uint8_t* s_out = s_tiles + kStages * kStageBytes;
    Shared* s = reinterpret_cast<Shared*>(s_out + kEpilogueWarps * kBufBytes);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / kWarp, 0), lane = threadIdx.x % kWarp;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s->full[i], kWgrad ? 2 : 1);
            mbar_init(&s->landed[i], 1);
            mbar_init(&s->empty[i], 2);  // both blocks' MMAs
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->acc_full[i], 1);
            mbar_init(&s->acc_empty[i], kSwiglu || kDswiglu ? 2 * kEpilogueWarps : kEpilogueWarps);  // of the pair
        }
        for (int i = 0; i < kEpilogueWarps; ++i)
            for (int j = 0; j < 2; ++j) mbar_init(&s->loaded[i][j], 1);
        s->asked = 0;
        s->waits = Waits{0, p.g.stall.wait_limit_us};
        fence_mbarrier_init();
        prefetch_tensormap(&map_a);
        prefetch_tensormap(&map_b);
        prefetch_tensormap(&map_out);
    }
    if (warp == 4) tmem_alloc_pair(&s->tmem, kTmemColumns);
    // The pair's barriers and TMEM are ready; the other half of this barrier, below, is behind the counts' way from memory (0.4
    // us a call saved).
    __syncwarp();
    cluster_arrive_release();
    griddep_wait();  // counts, rows and weights are complete from here on
    griddep_launch_dependents();
    Tiles<kForm> list{p, RowTiles<kTileRows, kSwiglu>{p.g.count, s->first, p.g.E, p.g.cap}};
    const int columns = (p.out_n + kBlock - 1) / kBlock;
    if (!kWgrad && warp == 1) list.walk.fill(s->first, lane, columns, pairs);
    tc_fence_before();
    __syncthreads();
    cluster_wait_acquire();
    tc_fence_after();
    const uint32_t tmem = s->tmem;
    int tiles = p.g.E * p.tiles_m * p.tiles_n;
    if (!kWgrad) {
        list.walk.start();
        const int row_tiles = list.walk.row_tiles();
        if (!kSwiglu) list.blocks = blocks_of_tiles(row_tiles, columns, pairs);
        list.walk.tiles_n = kSwiglu ? columns : (columns + list.blocks - 1) / list.blocks;
        tiles = row_tiles * list.walk.tiles_n;
    }

    if (warp < 4) {
        regs_down<64>();
        if (warp == 0 && lane == 0) {
            // ---- producer ----
            Ring<kStages> st(1);  // a fresh barrier passes a wait for phase 1
            uint32_t asked = 0;
            bool ok = true;
            const uint32_t full = mapa(smem_addr(&s->full[0]), 0);
            for (int t = pair; t < tiles && ok; t += pairs) {
                const Tile tl = list.at(t);
                const int stages = list.stages(tl), in_stage = list.in_stage(tl);
                const int n = kWgrad ? kTileRows : (tl.rows + 31) / 32 * 32;  // rows of the second operand
                const int a0 = tl.a0 + static_cast<int>(rank) * kHalf;
                const int b0 = (kWgrad ? tl.b0 : tl.m0) + static_cast<int>(rank) * (n / 2);
                const uint32_t each = tl.blocks * kOperand + n / 2 * 128;  // bytes of a step, of each CTA
                for (int b = 0; b < stages; ++b) {
                    if (!(ok = wait_for(&s->empty[st.at], st.phase, &s->waits))) break;
                    uint32_t bar = full + st.at * sizeof(uint64_t);
                    const int steps = in_stage == 1 ? 1 : min(2, p.kb - 2 * b);
                    const uint32_t bytes = steps * each;
                    if (kWgrad && (tl.rows - b * kBlockK < kBlockK) && tl.rows % 16 != 0) {
                        bar = mapa(smem_addr(&s->landed[st.at]), rank);
                        mbar_arrive_expect_tx(&s->landed[st.at], bytes);
                    } else if (rank == 0) {
                        mbar_arrive_expect_tx(&s->full[st.at], 2 * bytes);
                        if (kWgrad) mbar_arrive(&s->full[st.at]);
                    }
                    uint32_t ta = smem_addr(s_tiles) + st.at * kStageBytes, tb = ta + 2 * kOperand;
                    for (int step = 0; step < steps; ++step, tb += kBox) {
                        const int c = (b * in_stage + step) * kBlockK;
                        for (int i = 0; i < tl.blocks; ++i, ta += kOperand) {
                            if (kSwiglu) {
                                tma_load_3d(ta, &map_a, c, a0, 2 * tl.e + i, bar);
                            } else if (kAcrossA) {
                                for (int j = 0; j < 2; ++j)
                                    tma_load_3d(ta + j * kBox, &map_a, a0 + i * kBlock + j * 64, c, tl.e, bar);
                            } else {
                                tma_load_3d(ta, &map_a, c, a0 + i * kBlock, tl.e, bar);
                            }
                        }
                        if (kWgrad) {
                            for (int j = 0; j < 2; ++j) tma_load_3d(tb + j * kBox, &map_b, b0 + j * 64, c, tl.e, bar);
                        } else if (n == kTileRows) {
                            tma_load_3d(tb, &map_b, c, b0, tl.e, bar);
                        } else {
                            for (int i = 0; i < n / 2; i += kChunk) tma_load_3d(tb + i * 128, &map_b16, c, b0 + i, tl.e, bar);
                        }
                    }
                    if (kWgrad) *reinterpret_cast<volatile uint32_t*>(&s->asked) = ++asked;
                    st.next();
                }
            }
            // every stage's last read is over before the CTA may leave
            for (int i = 0; i < kStages && ok; ++i, st.next()) ok = wait_for(&s->empty[st.at], st.phase, &s->waits);
        } else if ((warp == 1 || warp == 2) && rank == 0) {
            // ---- MMA: two warps feed the pair's tensor cores, one for each accumulator.  One accumulator's sums cross to
            // their epilogue warps, and it comes back, while the other one multiplies ----
            const int half = warp - 1;
            Ring<kStages> st(0);
            uint32_t acc_phase = 1;
            bool ok = true;
            for (int t = pair, i = 0; t < tiles && ok; t += pairs, ++i) {
                const Tile tl = list.at(t);
                if (pair == p.g.stall.pair && i >= p.g.stall.tile) break;  // testing hook
                const int stages = __shfl_sync(0xffffffffu, list.stages(tl), 0);
                const int in_stage = __shfl_sync(0xffffffffu, list.in_stage(tl), 0);
                if (stages == 0) continue;
                const int block = __shfl_sync(0xffffffffu, block_of(tl, list.blocks, i, half), 0);
                if (block < 0) {
                    // the other warp's tile: only this one's arrivals (a barrier tells phases apart by one bit, so a wait
                    // may not be left out)
                    for (int b = 0; b < stages && ok; ++b, st.next()) {
                        ok = __all_sync(0xffffffffu, wait_for(&s->full[st.at], st.phase, &s->waits));
                        if (ok && elect_one()) mma_commit_pair(smem_addr(&s->empty[st.at]));
                        __syncwarp();
                    }
                    continue;
                }
                const int rows = __shfl_sync(0xffffffffu, tl.rows, 0);
                const uint32_t idesc = bf16_idesc(kBlock, kWgrad ? kTileRows : (rows + 31) / 32 * 32, kAcrossA, kWgrad);
                const bool ragged = kWgrad && rows % 16 != 0;
                const int last = kWgrad ? (rows - (stages - 1) * kBlockK + 15) / 16 : kBlockK / 16;  // MMAs of the last step
                ok = __all_sync(0xffffffffu, wait_for(&s->acc_empty[half], acc_phase, &s->waits));
                acc_phase ^= 1;
                const uint32_t d = tmem + half * kTileRows;
                for (int b = 0; b < stages && ok; ++b) {
                    const bool end = b + 1 == stages;
                    const bool there = ragged && end ? wait_cluster(&s->full[st.at], st.phase, &s->waits)
                                                     : wait_for(&s->full[st.at], st.phase, &s->waits);
                    ok = __all_sync(0xffffffffu, there);
                    if (!ok) break;
                    const uint32_t to = smem_addr(s_tiles) + st.at * kStageBytes;
                    const uint32_t ta = to + block * kOperand, tb = to + 2 * kOperand;
                    uint64_t da = kAcrossA ? sw128_desc_mn(ta, kBox) : sw128_desc(ta);
                    uint64_t db = kWgrad ? sw128_desc_mn(tb, kBox) : sw128_desc(tb);
                    asm volatile("" : "+l"(da), "+l"(db));
                    tc_fence_after();
                    if (elect_one()) {
                        // 16 of the contraction: 32 bytes further inside the swizzled row, or 16 rows further
#pragma unroll
                        for (int k = 0; k < kBlockK / 16; ++k)
                            if (!kWgrad || !end || k < last)
                                mma_f16_pair(d, da + k * (kAcrossA ? 128 : 2), db + k * (kWgrad ? 128 : 2), idesc, b > 0 || k > 0);
                        if (!kWgrad && in_stage == 2 && 2 * b + 1 < p.kb) {
#pragma unroll
                            for (int k = 0; k < kBlockK / 16; ++k)
                                mma_f16_pair(d, da + (kOperand >> 4) + k * (kAcrossA ? 128 : 2), db + (kBox >> 4) + k * 2, idesc, true);
                        }
                        mma_commit_pair(smem_addr(&s->empty[st.at]));
                        if (end) mma_commit_pair(smem_addr(&s->acc_full[half]));
                    }
                    __syncwarp();
                    st.next();
                }
            }
        } else if (warp == 3 && kWgrad) {
            // ---- relay: the step that ends an expert's rows, zeroed behind the last of them.  Experts whose rows end with 16 are
            // passed over, so the next such step may be the call's last ----
            Ring<kStages> st(0);
            uint32_t phases = 0;  // of the landed barriers, a bit each
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const Tile tl = list.at(t);
                const int stages = list.stages(tl), left = tl.rows - (stages - 1) * kBlockK;
                if (tl.rows % 16 != 0) {
                    st.skip(stages - 1);
                    ok = __all_sync(0xffffffffu, wait_while_moving(&s->landed[st.at], phases >> st.at & 1, &s->waits, &s->asked));
                    if (!ok) break;
                    phases ^= 1u << st.at;
                    uint8_t* to = s_tiles + st.at * kStageBytes;
                    const int more = (left + 15) / 16 * 16 - left;
                    // whole rows of 128 bytes in each of the six boxes, so the swizzle does not matter
                    for (int i = lane; i < more * 48; i += kWarp)
                        *reinterpret_cast<uint4*>(to + i / 8 % 6 * kBox + (left + i / 48) * 128 + i % 8 * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(mapa(smem_addr(&s->full[st.at]), 0));
                    st.next();
                } else {
                    st.skip(stages);
                }
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue: four warps to an accumulator, a quarter of its 128 lanes each; gated: all of them read both ----
        regs_up<208>();
        const int half = (warp - 4) / 4, quarter = warp % 4;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * kWarp) << 16);
        const uint32_t empty = mapa(smem_addr(&s->acc_empty[0]), 0);
        const uint32_t buf = smem_addr(s_out + (warp - 4) * kBufBytes);
        uint32_t acc_phase = 0;
        bool ok = true;
        // kDswiglu: a tile of one block is shared by all eight warps, so where a block has four of its own they arrive twice
        const bool shared = kDswiglu && list.blocks == 1;
        const auto hand_back = [&](int h) {
            tc_fence_before();
            if (lane == 0) mbar_arrive_cluster_relaxed(empty + h * 8);
            if (kDswiglu && !shared && lane == 0) mbar_arrive_cluster_relaxed(empty + h * 8);
        };
        if (kWgrad) {
            // thread = one output row
            constexpr int kCols = 64;  // of one store in bf16: 128 bytes a row
            const auto store = [&](const uint4 (&v)[8], int x, int y, int e) {
                if (x >= p.g.k || y >= p.g.n) return;
                if (lane == 0) bulk_wait_read<0>();  // the store before has left the buffer
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 128 + ((j ^ (lane & 7)) << 4)),
                                 "r"(v[j].x), "r"(v[j].y), "r"(v[j].z), "r"(v[j].w)
                                 : "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&map_out, buf, x, y, e);
                    bulk_commit();
                }
            };
            for (int t = pair, i = 0; t < tiles && ok; t += pairs, ++i) {
                const Tile tl = list.at(t);
                const int block = block_of(tl, list.blocks, i, half);
                if (block < 0) continue;
                const bool any = tl.rows > 0;  // without rows the gradient is 0 and the tensor cores have nothing
                if (any) {
                    // the second accumulator may have been passed over for as many tiles as there are columns of them
                    ok = __all_sync(0xffffffffu, wait_while_moving(&s->acc_full[half], acc_phase, &s->waits, &s->asked));
                    if (!ok) break;
                    acc_phase ^= 1;
                    tc_fence_after();
                }
                const int y = tl.a0 + block * kBlock + static_cast<int>(rank) * kHalf + quarter * kWarp;
                const uint32_t d = lanes + half * kTileRows;
                if (kOut16) {
                    // all columns into registers, so that the accumulator is free while they are stored
                    uint4 v[kTileRows / kCols][8];
#pragma unroll
                    for (int c = 0; c < kTileRows; c += 32) {
                        uint64_t x[16];
                        if (any) tmem_read(d + c, x);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            reinterpret_cast<uint32_t*>(v)[c / 2 + j] = any ? pack_bf16(unpack2(x[j])) : 0u;
                    }
                    if (any) hand_back(half);
#pragma unroll
                    for (int c = 0; c < kTileRows / kCols; ++c) store(v[c], tl.b0 + c * kCols, y, tl.e);
                } else {
                    // From registers to memory: through shared memory, which the operands keep busy, 32 experts x 512 rows, 4096
                    // x 7168, took 1020 us, so 932.  Products and stores add up all the same (0.84 us a row and 500 us; the stores' bytes
                    // alone take 555), since both accumulators fill together and are handed back with their last columns.  Two
                    // neighbouring lanes trade pairs of columns, so that each stores 16 bytes and the four lanes of a row 64 in a line.
                    float* out = static_cast<float*>(p.g.out) + (static_cast<long long>(tl.e) * p.g.n + y + lane / 4) * p.g.k;
#pragma unroll 2
                    for (int c = 0; c < kTileRows; c += 32) {
                        uint64_t x[16];
                        if (any) tmem_read_matrices(d + c, x);
                        if (any && c + 32 == kTileRows) hand_back(half);
#pragma unroll
                        for (int j = 0; j < 4; j += 2) {
                            const int col = tl.b0 + c + 8 * (j + lane % 2) + lane % 4 / 2 * 4;
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const uint64_t lo = any ? x[4 * j + m] : 0, hi = any ? x[4 * j + 4 + m] : 0;
                                const uint64_t got = __shfl_xor_sync(0xffffffffu, lane % 2 ? lo : hi, 1);
                                const float2 first = unpack2(lane % 2 ? got : lo), second = unpack2(lane % 2 ? hi : got);
                                if (col < p.g.k && y + 8 * m + lane / 4 < p.g.n)
                                    *reinterpret_cast<float4*>(out + static_cast<long long>(8 * m) * p.g.k + col) =
                                        make_float4(first.x, first.y, second.x, second.y);
                            }
                        }
                    }
                }
            }
        } else {
            // Boxes of 32 rows x 32 output columns in rows of 64 swizzled bytes.  This lane's address for the 8 x 8
            // matrices of eight rows: matrix lane / 8 is 8 columns, 16 bytes.
            const auto address = [&](uint32_t box, int rows8) {
                const int r = rows8 * 8 + lane % 8;
                return box + r * 64 + ((lane / 8 ^ (r >> 1 & 3)) << 4);
            };
            // A box out to rows r0.. of the output: `which` of its halves where it has two (0 and 1, else -1).
            const auto send = [&](uint32_t box, const CUtensorMap* map, void* out, int which, int e, int row, int rows, int col) {
                fence_proxy_async_smem();
                __syncwarp();
                const long long r0 = static_cast<long long>(e) * p.g.cap + row;
                if (rows >= kOutRows) {
                    if (lane == 0) {
                        if (which >= 0)
                            tma_store_3d(map, box, col, which, static_cast<int>(r0));
                        else
                            tma_store_3d(map, box, col, row, e);
                        bulk_commit();
                    }
                } else {
                    // the expert's last rows, one by one: what lies behind them stays as it is
#pragma unroll
                    for (int i = 0; i < kOutRows; i += 8) {
                        const int r = i + lane / 4, c = col + lane % 4 * 8;
                        if (r < rows && c < p.out_n) {
                            uint4 v;
                            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                         : "r"(box + r * 64 + ((lane % 4 ^ (r >> 1 & 3)) << 4)));
                            const long long at = which >= 0 ? 2 * (r0 + r) + which : r0 + r;
                            st_v4(static_cast<uint16_t*>(out) + at * p.out_n + c, v);
                        }
                    }
                    fence_proxy_async_smem();  // before a copy may fill the box again
                    __syncwarp();
                    if (lane == 0) bulk_commit();  // an empty group: the waits count boxes
                }
            };
            uint32_t turn = 0;
            // The buffer that takes turns with the other one, once its last store has left it.
            const auto next_box = [&] {
                if (lane == 0) bulk_wait_read<1>();
                __syncwarp();
                return buf + (turn++ & 1) * kOutBytes;
            };
            // 32 rows x 32 columns packed as matrices, out.
            const auto put = [&](const uint32_t (&v)[16], const CUtensorMap* map, void* out, int which, const Tile& tl, int c,
                                 int col) {
                const uint32_t box = next_box();
#pragma unroll
                for (int j = 0; j < 4; ++j) store_matrices_trans(address(box, j), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                send(box, map, out, which, tl.e, tl.m0 + c, tl.rows - c, col);
            };
            uint32_t loads = 0;  // kDswiglu: boxes of gate and up asked for
            for (int t = pair, i = 0; t < tiles && ok; t += pairs, ++i) {
                const Tile tl = list.at(t);
                const int block = kSwiglu || shared ? 0 : block_of(tl, list.blocks, i, half);
                if (block < 0) continue;
                const int acc = shared ? i & 1 : half;
                const int col = tl.a0 + block * kBlock + static_cast<int>(rank) * kHalf + quarter * kWarp;
                const bool on = col < p.out_n;
                const auto load = [&](int c) {  // kDswiglu: gate and up of the rows from c on, into the next set of buffers
                    const int set = loads & 1;
                    ++loads;
                    if (lane == 0) {
                        bulk_wait_read<0>();  // what was stored from there has left
                        mbar_arrive_expect_tx(&s->loaded[warp - 4][set], 2 * kOutBytes);
                        const int r0 = static_cast<int>(static_cast<long long>(tl.e) * p.g.cap + tl.m0 + c);
                        for (int j = 0; j < 2; ++j)
                            tma_load_3d_alone(buf + set * 2 * kOutBytes + j * kOutBytes, &map_gate_up, col, j, r0,
                                              smem_addr(&s->loaded[warp - 4][set]));
                    }
                };
                // kDswiglu: the boxes of 32 rows that this warp has (shared: in turn for the two warps of a quarter), the first two
                // asked for ahead
                const int first = shared ? half * kOutRows : 0, stride = shared ? 2 * kOutRows : kOutRows;
                uint32_t now = loads;
                if (kDswiglu && on && first < tl.rows) {
                    load(first);
                    if (first + stride < tl.rows) load(first + stride);
                }
                ok = wait_for(&s->acc_full[acc], shared ? i >> 1 & 1 : acc_phase, &s->waits);
                if (kSwiglu) ok = ok && wait_for(&s->acc_full[half ^ 1], acc_phase, &s->waits);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                acc_phase ^= 1;
                tc_fence_after();
                if (!on || (kDswiglu && first >= tl.rows)) {
                    hand_back(acc);
                    if (kSwiglu) hand_back(half ^ 1);
                    continue;
                }
                if (kSwiglu) {
                    // boxes of 32 rows in turn for the two warps of a quarter
#pragma unroll 1
                    for (int c = half * kOutRows; c < tl.rows; c += 2 * kOutRows) {
                        uint32_t g[16], u[16], h[16];
                        uint64_t x[16], y[16];
                        tmem_read_matrices(lanes + c, x);
                        tmem_read_matrices(lanes + kTileRows + c, y);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 a = unpack2(x[j]), b = unpack2(y[j]);
                            h[j] = pack_bf16(make_float2(gated_unit<true>(a.x, b.x), gated_unit<true>(a.y, b.y)));
                            g[j] = pack_bf16(a);
                            u[j] = pack_bf16(b);
                        }
                        put(h, &map_out, p.g.out, -1, tl, c, col);
                        if (p.g.gate_up_out != nullptr) {
                            put(g, &map_gate_up, p.g.gate_up_out, 0, tl, c, col);
                            put(u, &map_gate_up, p.g.gate_up_out, 1, tl, c, col);
                        }
                    }
                    hand_back(0);
                    hand_back(1);
                } else if (kDswiglu) {
#pragma unroll 1
                    for (int c = first; c < tl.rows; c += stride, ++now) {
                        if (c > first && c + stride < tl.rows) load(c + stride);
                        const uint32_t box = buf + (now & 1) * 2 * kOutBytes;
                        uint64_t x[16];
                        tmem_read_matrices(lanes + acc * kTileRows + c, x);
                        if (c + stride >= tl.rows) hand_back(acc);
                        ok = __all_sync(0xffffffffu, wait_for(&s->loaded[warp - 4][now & 1], now >> 1 & 1, &s->waits));
                        if (!ok) break;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t g[4], u[4];
                            load_matrices_trans(address(box, j), g);
                            load_matrices_trans(address(box + kOutBytes, j), u);
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const float2 f = unpack2(x[4 * j + m]), a = unpack_bf16(g[m]), b = unpack_bf16(u[m]);
                                const float2 lo = gated_unit_gradient<true>(f.x, a.x, b.x), hi = gated_unit_gradient<true>(f.y, a.y, b.y);
                                g[m] = pack_bf16(make_float2(lo.x, hi.x));
                                u[m] = pack_bf16(make_float2(lo.y, hi.y));
                            }
                            __syncwarp();  // every lane has its values before they are overwritten
                            store_matrices_trans(address(box, j), g[0], g[1], g[2], g[3]);
                            store_matrices_trans(address(box + kOutBytes, j), u[0], u[1], u[2], u[3]);
                        }
                        for (int j = 0; j < 2; ++j)
                            send(box + j * kOutBytes, &map_out, p.g.out, j, tl.e, tl.m0 + c, tl.rows - c, col);
                    }
                    if (!ok) break;
                } else {
                    // all rows into registers, so that the accumulator is free while they are stored
                    uint32_t v[kTileRows / kOutRows][16];
#pragma unroll
                    for (int c = 0; c < kTileRows / kOutRows; ++c)
                        if (c * kOutRows < tl.rows) {
                            uint64_t x[16];
                            tmem_read_matrices(lanes + half * kTileRows + c * kOutRows, x);
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[c][j] = pack_bf16(unpack2(x[j]));
                        }
                    hand_back(half);
#pragma unroll
                    for (int c = 0; c < kTileRows / kOutRows; ++c)
                        if (c * kOutRows < tl.rows) put(v[c], &map_out, p.g.out, -1, tl, c * kOutRows, col);
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
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

// Map of the outputs of the forms over rows, boxes of 32 columns x 32 rows in 64 swizzled bytes a row: of
// [outer][rows][cols] bf16, or of [rows][2][cols].
bool make_out_map(CUtensorMap* map, const void* base, int cols, long long rows, int outer, bool halves) {
    const auto encode = gemm::encode_tiled();
    if (encode == nullptr) return false;
    const cuuint64_t row = static_cast<cuuint64_t>(cols) * 2, all = static_cast<cuuint64_t>(rows);
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), halves ? 2 : all, halves ? all : static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[2] = {row, halves ? 2 * row : row * all};
    const cuuint32_t box[3] = {kOutCols, halves ? 1u : kOutRows, halves ? kOutRows : 1u}, step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Bf16Form kForm, bool kOut16>
cudaError_t launch(const Bf16GemmArgs& g, cudaStream_t stream) {
    using gemm::make_map_bf16;
    constexpr bool kWgrad = kForm == Bf16Form::kWgrad, kSwiglu = kForm == Bf16Form::kSwiglu;
    constexpr bool kDswiglu = kForm == Bf16Form::kDswiglu;
    constexpr bool kTransposed = kForm == Bf16Form::kDgrad || kDswiglu;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const auto over = [](int v, int by) { return (v + by - 1) / by; };
    Params p = {};
    p.g = g;
    const int inner = kTransposed ? g.n : g.k;  // forms over rows: the contraction
    p.out_n = kWgrad || kTransposed ? g.k : g.n;
    p.kb = over(inner, kBlockK);
    p.tiles_m = over(g.n, 2 * kBlock);
    p.tiles_n = over(g.k, kTileRows);
    CUtensorMap a = {}, b = {}, b16 = {}, out = {}, gate_up = {};
    bool ok;
    if (kWgrad) {
        // without a capacity nothing is loaded, but a map needs an array
        const bool none = g.cap == 0;
        ok = make_map_bf16(&a, none ? g.out : g.rows, g.n, none ? 1 : g.cap, none ? 1 : g.E, kBlockK) &&
             make_map_bf16(&b, none ? g.out : g.other, g.k, none ? 1 : g.cap, none ? 1 : g.E, kBlockK) &&
             (!kOut16 || make_map_bf16(&out, g.out, g.k, g.n, g.E, kWarp));
    } else {
        const long long rows = static_cast<long long>(g.E) * g.cap;
        ok = make_map_bf16(&a, g.other, g.k, g.n, g.E * (kSwiglu ? 2 : 1), kTransposed ? kBlockK : kHalf) &&
             make_map_bf16(&b, g.rows, inner, g.cap, g.E, kHalf) && make_map_bf16(&b16, g.rows, inner, g.cap, g.E, kChunk) &&
             (kDswiglu ? make_out_map(&out, g.out, p.out_n, rows, 1, true) : make_out_map(&out, g.out, p.out_n, g.cap, g.E, false));
        const void* halves = kDswiglu ? static_cast<const void*>(g.gate_up) : g.gate_up_out;
        if (halves != nullptr) ok = ok && make_out_map(&gate_up, halves, p.out_n, rows, 1, true);
    }
    if (!ok) return cudaErrorInvalidValue;
    constexpr bool wide = kWide<kForm>;
    const size_t smem = 1024 + (wide ? 3 : 4) * kStageBytes + kEpilogueWarps * (wide ? 4 : 2) * kOutBytes + sizeof(Shared);
    // an upper bound of the tiles: the counts are on the device
    const long long most = static_cast<long long>(g.E) *
                           (kWgrad ? p.tiles_m * p.tiles_n : over(g.cap, kTileRows / 2) * over(p.out_n, kBlock));
    const int pairs = static_cast<int>(most < sms / 2 ? most : sms / 2);
    return launch_pdl(ll_gemm_bf16_kernel<kForm, kOut16>, dim3(2 * pairs), dim3(kThreads), smem, stream, 0, true, a, b, b16,
                      out, gate_up, p);
}

}  // namespace

cudaError_t launch_ll_gemm_bf16(const Bf16GemmArgs& g, cudaStream_t stream) {
    switch (g.form) {
        case Bf16Form::kPlain: return launch<Bf16Form::kPlain, true>(g, stream);
        case Bf16Form::kSwiglu: return launch<Bf16Form::kSwiglu, true>(g, stream);
        case Bf16Form::kDgrad: return launch<Bf16Form::kDgrad, true>(g, stream);
        case Bf16Form::kDswiglu: return launch<Bf16Form::kDswiglu, true>(g, stream);
        case Bf16Form::kWgrad: break;
    }
    return g.out_bf16 ? launch<Bf16Form::kWgrad, true>(g, stream) : launch<Bf16Form::kWgrad, false>(g, stream);
}

}  // namespace ep
