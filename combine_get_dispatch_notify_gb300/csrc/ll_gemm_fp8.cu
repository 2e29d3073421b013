// Experts' block-scaled e4m3 products on the tensor cores (ep_ll_gemm_fp8,
// ep_ll_gemm_swiglu_fp8): tiles of more than 128 rows.
//
//   p[m][n] = sum_b as[m][b] ws[n / 128][b] sum_{k in block b} a[m][k] w[n][k]
//
// A pair of CTAs (one cluster, two SMs) owns a tile of 256 rows x 256 weight
// rows and walks the k-blocks of 128.  A block's plain sums are made in TMEM, in
// two halves of 128 columns with an MMA warp each (a chain of four tcgen05.mma,
// K = 32 each) and two accumulators that take turns (2 x 2 x 128 columns, all of
// TMEM): one half multiplies while the epilogue warps read the other, scale it by
// as * ws and add it to fp32 sums in their registers.  That scaling is what
// hardware block scales cannot do for fp32 scales: 32768 FMAs of an SM per block.
//
// What bounds it: a block's products take the tensor core 512 cycles, its operands
// (32 KB to each SM; up to 49 bytes a cycle arrive from L2) 669, and the sixteen
// epilogue warps' instructions about 550 of the four schedulers; together they run at
// 860 cycles a block.  None of them is full: which waits of the chain from operands to
// sums make up the other 190 cycles has not been measured.  The tile is as large as TMEM and the registers for its sums
// allow: with a smaller one the operands would take longer still.  Measured, with
// the few-rows kernel's share: 32 experts with 1024 rows each, gated, 7168 -> 2 x 2048:
// 890 to 930 us over long blocks, from card to card, 2.1 to 2.2 PFLOP/s; 850 us in a burst of 30 calls
// (tensor pipe busy 54 %); 32768 rows in 32 experts by Zipf popularity, 2048 -> 7168: 440
// to 467 us, 2.1 to 2.2 PFLOP/s; 430 us in a burst.  One MMA of 256 columns in place of
// the halves took 791 us for the first and 481 for the second when the halves took 806
// and 460, bursts all; eight epilogue warps took 900 us and more for the first.
//
// Each CTA loads its own 128 rows of a and half of the weight rows with
// swizzled TMA; the weights cross HBM once per 256 rows, and only the 32-row
// chunks of a that hold rows are read.  For the gated product the weight rows
// are 128 of the gate matrix (loaded by the leader) and the same 128 of the up
// matrix (its peer), so gate and up of one output column meet in one thread.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ll_gemm_fp8.cuh"

namespace ep {
namespace gemm {

namespace {

constexpr int kTileN = 256;                    // weight rows of a pair's tile
constexpr int kHalf = kBoxRows;                // rows of a, and of w, that one CTA loads
constexpr int kTileBytes = kBoxBytes;          // one operand of a stage
template <bool kSwiglu>
constexpr int kStages = kSwiglu ? 6 : 4;       // four leave room for the output tile
constexpr int kMostStages = 6;
constexpr int kGroups = 4;                     // epilogue warpgroups, 64 columns of a tile each
constexpr int kSums = kTileN / kGroups;        // sums of an epilogue thread
constexpr int kGroupCols = kSums / 2;          // gated: columns of each of the tile's two weight blocks
constexpr int kThreads = 128 + 128 * kGroups;  // producer, two MMA warps, scale warp | epilogue
constexpr int kOutRow = 128;                   // bytes of one epilogue thread's bf16 results: 64 columns
constexpr int kOutBytes = kWarp * kOutRow;     // of a warp's
constexpr int kScaleSlots = 4;                 // of four k-blocks each
constexpr int kTileRing = 2 * kScaleSlots;     // more than slots: a tile is overwritten once the one after it is summed
constexpr int kHalfN = kTileN / 2;             // weight rows of one MMA: 64 of each CTA's 128; its TMEM columns

struct Barriers {
    uint64_t full[kMostStages];             // leader's: bytes of both CTAs have landed
    uint64_t empty[kMostStages];            // both: the MMAs that read the stage are done
    uint64_t acc_full[2][2];            // [half][buffer], both: a block's sums are in TMEM
    uint64_t acc_empty[2][2];           // leader's: the half's epilogue warps of the pair have read them
    uint64_t scale_full[kScaleSlots];   // both: the scales of four blocks are in shared memory
    uint64_t scale_empty[kScaleSlots];  // both: every epilogue warp is done with them
};

struct Shared {
    Barriers bar;
    float row_scale[kScaleSlots][4][kHalf];  // of each row of the CTA
    float2 w_scale[kScaleSlots][4];          // of the tile's two weight blocks
    Tile tile[kTileRing];                    // the tiles in turn, each handed over with its first scales
    float amax[2][kGroups][kHalf];           // [tile parity][warpgroup][row]
    int first[kMaxGroups + 2];               // tiles before each group of 32 experts
    uint32_t tmem;
    Waits waits;
};

// Row `row` of this CTA's half of the tile, in the packed rows of all experts.
__device__ __forceinline__ long long tile_row(const Tile& t, const Params& p, uint32_t rank, int row) {
    return static_cast<long long>(t.e) * p.g.cap + t.m0 + static_cast<int>(rank) * kHalf + row;
}

// Barrier of the four epilogue warps, one of each warpgroup, that have the same 32 rows.
__device__ __forceinline__ void quarter_sync(int quarter) {
    asm volatile("bar.sync %0, 128;" ::"r"(1 + quarter) : "memory");
}

template <bool kSwiglu, bool kStall>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ll_gemm_fp8_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_a128, const __grid_constant__ CUtensorMap map_w,
                       const __grid_constant__ CUtensorMap map_y, const Params p) {
    extern __shared__ uint8_t s_raw[];
    // stages first, on a 1024-byte boundary as the swizzle needs, at the same offset in both CTAs
    const uint32_t pad = (1024u - (smem_addr(s_raw) & 1023u)) & 1023u;
    uint8_t* s_tiles = s_raw + pad;
    constexpr int kStages = gemm::kStages<kSwiglu>;
    uint8_t* s_out = s_tiles + kStages * 2 * kTileBytes;  // of each epilogue warp (bf16 results)
    Shared* s = reinterpret_cast<Shared*>(s_out + (kSwiglu ? 0 : 4 * kGroups * kOutBytes));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / kWarp, 0), lane = threadIdx.x % kWarp;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const int cols = kSwiglu ? kTileN / 2 : kTileN;  // output columns of a tile

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s->bar.full[i], 1);
            mbar_init(&s->bar.empty[i], 2);  // both halves' MMAs
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s->bar.acc_full[i / 2][i % 2], 1);
            mbar_init(&s->bar.acc_empty[i / 2][i % 2], 4 * kGroups);  // half the epilogue warps, in both CTAs
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&s->bar.scale_full[i], 1);
            mbar_init(&s->bar.scale_empty[i], 4 * kGroups);
        }
        s->waits = Waits{0, p.g.wait_limit_us};
        fence_mbarrier_init();
        prefetch_tensormap(&map_a);
        prefetch_tensormap(&map_w);
        if (!kSwiglu) prefetch_tensormap(&map_y);
    }
    if (warp == 4) tmem_alloc_pair(&s->tmem, kTmemColumns);
    griddep_wait();  // counts, rows and scales are complete from here on
    griddep_launch_dependents();
    if (warp == 1) count_tiles<false>(s->first, p, lane);
    tc_fence_before();
    __syncthreads();
    cluster_arrive_release();
    cluster_wait_acquire();
    tc_fence_after();
    const uint32_t tmem = s->tmem;
    const int tiles = s->first[(p.g.E + kWarp - 1) / kWarp];
    const int mine = pair < tiles ? (tiles - pair + pairs - 1) / pairs : 0;  // tiles of this pair

    if (warp < 4) {
        regs_down<64>();
        if (warp == 0 && lane == 0) {
            // ---- producer: this CTA's rows of a and its half of the weight rows ----
            uint32_t st = 0, phase = 1;  // a fresh barrier passes a wait for phase 1
            Walk walk;
            bool ok = true;
            const uint32_t full = mapa(smem_addr(&s->bar.full[0]), 0);
            for (int t = pair; t < tiles && ok; t += pairs) {
                const Tile tl = tile_at<false>(t, walk, s->first, p, cols);
                const int chunks0 = (min(tl.rows, kHalf) + kChunk - 1) / kChunk;
                const int chunks1 = (min(max(tl.rows - kHalf, 0), kHalf) + kChunk - 1) / kChunk;
                const int chunks = rank == 0 ? chunks0 : chunks1;
                const uint32_t bytes = 2 * kTileBytes + (chunks0 + chunks1) * kChunk * kBlockK;
                const int wy = kSwiglu ? tl.n0 : tl.n0 + static_cast<int>(rank) * kHalf;
                const int wz = kSwiglu ? 2 * tl.e + static_cast<int>(rank) : tl.e;
                const int ay = tl.m0 + static_cast<int>(rank) * kHalf;
                for (int b = 0; b < p.kb; ++b) {
                    if (!(ok = wait_for<kStall>(&s->bar.empty[st], phase, &s->waits))) break;
                    if (rank == 0) mbar_arrive_expect_tx(&s->bar.full[st], bytes);
                    const uint32_t bar = full + st * sizeof(uint64_t);
                    const uint32_t ta = smem_addr(s_tiles) + st * 2 * kTileBytes;
                    tma_load_3d(ta + kTileBytes, &map_w, b * kBlockK, wy, wz, bar);
                    if (chunks == kHalf / kChunk)
                        tma_load_3d(ta, &map_a128, b * kBlockK, ay, tl.e, bar);
                    else
                        for (int c = 0; c < chunks; ++c)
                            tma_load_3d(ta + c * kChunk * kBlockK, &map_a, b * kBlockK, ay + c * kChunk, tl.e, bar);
                    if (++st == kStages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            // every stage's last read is over before the CTA may leave
            for (int i = 0; i < kStages && ok; ++i) {
                ok = wait_for<kStall>(&s->bar.empty[st], phase, &s->waits);
                if (++st == kStages) {
                    st = 0;
                    phase ^= 1;
                }
            }
        } else if ((warp == 1 || warp == 2) && rank == 0) {
            // ---- MMA: two warps feed the pair's tensor cores, one for each half of the tile's columns.  One half's
            // sums cross to its epilogue warps, and its accumulator comes back, while the other half multiplies ----
            constexpr uint32_t idesc = e4m3_idesc(kTileM, kHalfN);
            const uint32_t half = warp - 1;
            const int fed = kStall && half == 0 && pair == p.g.stall_cta ? min(mine, p.g.stall_tile) : mine;
            const uint32_t blocks = fed * p.kb;
            uint32_t st = 0, full_phase = 0, buf = 0, empty_phase = 1;
            for (uint32_t it = 0; it < blocks; ++it) {
                // everything but the accumulator's hand-back is settled before the wait for it: what follows that
                // wait is on the path of every block
                bool ok = wait_for<kStall>(&s->bar.full[st], full_phase, &s->waits);
                const uint32_t ta = smem_addr(s_tiles) + st * 2 * kTileBytes;
                uint64_t da = sw128_desc(ta), dw = sw128_desc(ta + kTileBytes + half * (kTileBytes / 2));
                asm volatile("" : "+l"(da), "+l"(dw));
                ok = ok && wait_for<kStall>(&s->bar.acc_empty[half][buf], empty_phase, &s->waits);
                if (!__all_sync(0xffffffffu, ok)) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kBlockK / 32; ++k)  // 32 bytes further inside the swizzled row
                        mma_e4m3_pair(tmem + (2 * half + buf) * kHalfN, da + 2 * k, dw + 2 * k, idesc, k > 0);
                    mma_commit_pair(smem_addr(&s->bar.acc_full[half][buf]));
                    mma_commit_pair(smem_addr(&s->bar.empty[st]));
                }
                __syncwarp();
                buf ^= 1;
                empty_phase ^= buf ^ 1;  // both buffers share a phase
                if (++st == kStages) {
                    st = 0;
                    full_phase ^= 1;
                }
            }
        }
        if (warp == 3) {
            // ---- scales: four rows a lane, four k-blocks at a time, handed over through shared memory ----
            uint32_t q = 0;  // slots so far
            Walk walk;
            bool ok = true;
            for (int i = 0; i < mine && ok; ++i) {
                const Tile tl = tile_at<false>(pair + i * pairs, walk, s->first, p, cols);
                const int left = tl.rows - static_cast<int>(rank) * kHalf;
                const float* as = p.g.a_scales + tile_row(tl, p, rank, lane) * p.kb;
                const long long step = static_cast<long long>(kWarp) * p.kb;
                const float* ws = weight_scales<kSwiglu>(tl, p, lane & 1);
                for (int b = 0; b < p.kb; b += 4, ++q) {
                    const uint32_t slot = q % kScaleSlots;
                    float4 a[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[j] = load_scales(as + j * step, b, p.kb, lane + j * kWarp < left);
                    const float4 w = load_scales(ws, b, p.kb, lane < 2);
                    const uint32_t phase = q / kScaleSlots & 1 ^ 1;  // a fresh barrier passes a wait for phase 1
                    ok = __all_sync(0xffffffffu, wait_for<kStall>(&s->bar.scale_empty[slot], phase, &s->waits));
                    if (!ok) break;
                    if (b == 0 && lane == 0) s->tile[i % kTileRing] = tl;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) s->row_scale[slot][k][lane + j * kWarp] = element(a[j], k);
                        if (lane < 2) reinterpret_cast<float*>(&s->w_scale[slot][k])[lane] = element(w, k);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s->bar.scale_full[slot]);
                }
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue: thread = one row.  Warpgroup g sums 64 columns: 32 g + [0, 32) of both weight blocks where
        // gate and up have to meet, else 64 (g / 2) + [0, 64) of block g % 2, which leave as whole lines ----
        regs_up<104>();
        // Columns of one TMEM read.  Sums, read and addresses have to fit 104 registers, or moves crowd the loop: gated
        // 794 us with 16 and 917 with 32 (32 experts, 1024 rows, 7168 -> 2 x 2048), plain 425 and 406 (32768 rows of
        // Zipf-distributed experts, 2048 -> 7168).
        constexpr int kRead = kSwiglu ? 16 : 32;
        const int g = (warp - 4) / 4, quarter = warp % 4;
        const int row = quarter * kWarp + lane;  // of this CTA's 128
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * kWarp) << 16) + g / 2 * kTileN +
                               g % 2 * (kSwiglu ? kGroupCols : kHalfN / 2);
        uint64_t* full = s->bar.acc_full[g / 2];
        const uint32_t empty = mapa(smem_addr(s->bar.acc_empty[g / 2]), 0);
        uint32_t it = 0, q = 0;  // blocks and slots so far
        for (int i = 0; i < mine; ++i) {
            // the tile comes with its first scales: walking here would hold up the sums, some 800 cycles a tile
            const uint32_t first = q % kScaleSlots;
            bool ok = __all_sync(0xffffffffu, wait_for<kStall>(&s->bar.scale_full[first], q / kScaleSlots & 1, &s->waits));
            const bool warp_on = quarter * kWarp < s->tile[i % kTileRing].rows - static_cast<int>(rank) * kHalf;
            uint64_t acc[kSums / 2];  // gated: the gates, then the ups
#pragma unroll
            for (int j = 0; j < kSums / 2; ++j) acc[j] = 0;
#pragma unroll 1
            for (int b = 0; ok && b < p.kb; ++b, ++it) {
                const uint32_t buf = it & 1, slot = q % kScaleSlots;
                ok = b == 0 || (b & 3) != 0 || wait_for<kStall>(&s->bar.scale_full[slot], q / kScaleSlots & 1, &s->waits);
                const float2 ws = s->w_scale[slot][b & 3];
                const float as = s->row_scale[slot][b & 3][row];
                ok = __all_sync(0xffffffffu, ok && wait_for<kStall>(&full[buf], (it / 2) & 1, &s->waits));
                if (!ok) break;
                tc_fence_after();
                if (warp_on) {
                    const uint32_t col = lanes + buf * kHalfN;
                    const uint64_t s0 = pair2(as * (kSwiglu || g % 2 == 0 ? ws.x : ws.y));
                    const uint64_t s1 = kSwiglu ? pair2(as * ws.y) : s0;
                    uint64_t x[kRead / 2];
#pragma unroll
                    for (int c = 0; c < kSums; c += kRead) {
                        tmem_read(col + (kSwiglu ? c / kGroupCols * (kHalfN / 2) + c % kGroupCols : c), x);
                        if (c + kRead == kSums) {  // the block's sums have left TMEM
                            tc_fence_before();
                            if (lane == 0) mbar_arrive_cluster_relaxed(empty + buf * 8);
                        }
#pragma unroll
                        for (int j = 0; j < kRead / 2; ++j) fma2(acc[c / 2 + j], x[j], c < kSums / 2 ? s0 : s1);
                    }
                } else {
                    tc_fence_before();
                    if (lane == 0) mbar_arrive_cluster_relaxed(empty + buf * 8);
                }
                if ((b & 3) == 3 || b + 1 == p.kb) {
                    __syncwarp();  // every lane has read the slot; the arrival hands it back: a release
                    if (lane == 0) mbar_arrive(&s->bar.scale_empty[slot]);
                    ++q;
                }
            }
            if (!ok) {
                // the quarter's other warps may still come to the barriers of this tile and the ones after it: each of
                // their own waits is bounded too, a barrier that this warp stays away from would not be
                if (kSwiglu)
                    for (; i < mine; ++i) quarter_sync(quarter);
                break;
            }
            const Tile tl = s->tile[i % kTileRing];
            const int left = tl.rows - static_cast<int>(rank) * kHalf;
            const bool valid = row < left;
            const long long r = tile_row(tl, p, rank, row);
            if (!kSwiglu) {
                const int col = tl.n0 + g % 2 * kHalf + g / 2 * (kHalfN / 2);
                uint4 v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {  // 8 columns
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __nv_bfloat162 h = __float22bfloat162_rn(unpack2(acc[4 * j + k]));
                        w[k] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    v[j] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (col < p.g.n && quarter * kWarp + kWarp <= left) {
                    // all 32 rows: through shared memory, in swizzled rows, and out by TMA while the next tile's blocks
                    // are summed (stores straight from here would hold them up: each touches 32 lines)
                    uint8_t* to = s_out + (warp - 4) * kOutBytes;
                    if (lane == 0) bulk_wait_read<0>();  // the last tile's store has left the buffer
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4*>(to + lane * kOutRow + ((j ^ (lane & 7)) << 4)) = v[j];
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&map_y, smem_addr(to), col, tl.m0 + static_cast<int>(rank) * kHalf + quarter * kWarp,
                                     tl.e);
                        bulk_commit();
                    }
                } else if (valid) {
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.g.y) + r * p.g.n + col;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (col + 8 * j < p.g.n) st_v4(out + 8 * j, v[j]);
                }
            } else if (!warp_on) {
                quarter_sync(quarter);
            } else {
                // h = gate / (1 + exp(-gate)) * up; columns past n have zero weights, so h = 0 there
                float h[kGroupCols];
                float amax = 0.0f;
#pragma unroll
                for (int j = 0; j < kGroupCols / 2; ++j) {
                    const float2 a = unpack2(acc[j]), u = unpack2(acc[kGroupCols / 2 + j]);
                    h[2 * j] = gated(a.x, u.x);
                    h[2 * j + 1] = gated(a.y, u.y);
                    amax = fmaxf(amax, fmaxf(fabsf(h[2 * j]), fabsf(h[2 * j + 1])));
                }
                // The other warpgroups have the rest of the block's 128 columns.  Every warp of the quarter comes to the
                // barrier on every tile, with rows or without: passing it for one tile says that the maxima of the tile
                // before have been read, so two places take turns.
                s->amax[i & 1][g][row] = amax;
                quarter_sync(quarter);
#pragma unroll
                for (int k = 0; k < kGroups; ++k) amax = fmaxf(amax, s->amax[i & 1][k][row]);
                const float scale = block_scale(amax);
                if (valid) {
                    const float inv = 1.0f / scale;
                    uint8_t* out = static_cast<uint8_t*>(p.g.y) + r * p.g.n;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {  // 16 columns
                        const int col = tl.n0 + g * kGroupCols + j * 16;
                        uint32_t v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v[k] = pack_e4m3x4(over_scale(h[j * 16 + k * 4], scale, inv), over_scale(h[j * 16 + k * 4 + 1], scale, inv),
                                               over_scale(h[j * 16 + k * 4 + 2], scale, inv), over_scale(h[j * 16 + k * 4 + 3], scale, inv));
                        if (col < p.g.n) st_v4(out + col, make_uint4(v[0], v[1], v[2], v[3]));
                    }
                    if (g == 0) p.g.y_scales[r * p.nb + tl.n0 / kScaleBlock] = scale;
                }
            }
        }
        if (!kSwiglu && lane == 0) bulk_wait_all();
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

template <bool kSwiglu, bool kStall>
cudaError_t launch_form(const GemmArgs& g, cudaStream_t stream) {
    Params p = {};
    p.g = g;
    p.kb = scale_blocks(g.k);
    p.nb = scale_blocks(g.n);
    const int cols = kSwiglu ? kTileN / 2 : kTileN;
    p.tiles_n = (g.n + cols - 1) / cols;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    CUtensorMap map_a, map_a128, map_w, map_y = {};
    if (!make_map(&map_a, g.a, g.k, g.cap, g.E, kChunk) || !make_map(&map_a128, g.a, g.k, g.cap, g.E, kHalf) ||
        !make_map(&map_w, g.w, g.k, g.n, g.E * (kSwiglu ? 2 : 1), kHalf) ||
        (!kSwiglu && !make_map_bf16(&map_y, g.y, g.n, g.cap, g.E, kWarp)))
        return cudaErrorInvalidValue;
    const size_t smem = 1024 + static_cast<size_t>(kStages<kSwiglu>) * 2 * kTileBytes +
                        (kSwiglu ? 0 : 4 * kGroups * kOutBytes) + sizeof(Shared);
    // an upper bound of the tiles: the counts are on the device
    const long long most = static_cast<long long>(g.E) * ((g.cap + kTileM - 1) / kTileM) * p.tiles_n;
    const int pairs = static_cast<int>(most < sms / 2 ? most : sms / 2);
    return launch_pdl(ll_gemm_fp8_kernel<kSwiglu, kStall>, dim3(2 * pairs), dim3(kThreads), smem, stream, 0, true, map_a,
                      map_a128, map_w, map_y, p);
}

cudaError_t launch(const GemmArgs& g, cudaStream_t stream) {
    const bool gated = g.y_scales != nullptr;
    if (g.stall) return gated ? launch_form<true, true>(g, stream) : launch_form<false, true>(g, stream);
    return gated ? launch_form<true, false>(g, stream) : launch_form<false, false>(g, stream);
}

}  // namespace
}  // namespace gemm

cudaError_t launch_ll_gemm_fp8(const GemmArgs& g, cudaStream_t stream) {
    // With up to 128 rows an expert there is nothing for the pairs.  Otherwise the few-rows kernel follows them: its
    // CTAs take over SMs as they run dry and wait there for the pairs' end.
    if (g.cap > gemm::kFewRows) {
        const cudaError_t e = gemm::launch(g, stream);
        if (e != cudaSuccess) return e;
    }
    return gemm::launch_few(g, stream);
}

}  // namespace ep
