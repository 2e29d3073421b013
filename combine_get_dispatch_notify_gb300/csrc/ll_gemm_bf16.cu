// Experts' bf16 products and their gradients on the tensor cores
// (ep_ll_gemm_bf16 and its neighbours).
//
//   rows forms   D[m][j] = sum_c r[m][c] w[j][c]    (kPlain, kSwiglu)
//                D[m][j] = sum_c r[m][c] w[c][j]    (kDgrad, kDswiglu)
//   kWgrad       D[i][j] = sum_m r[m][i] a[m][j]    over an expert's rows
//
// A pair of CTAs (one cluster, two SMs) owns a tile of 256 x 256 and walks the
// contraction in blocks of 64: each CTA loads its own 128 rows of the first operand
// and half of the second with swizzled TMA, one thread feeds the pair's tensor cores
// (tcgen05.mma, K = 16), and the sums stay in TMEM until the tile is done, in two
// accumulators that take turns so that one is read while the other is summed.
// Whether an operand's rows of memory run along the contraction or across it is
// settled by its descriptor: nothing is transposed in memory.  For the gated product
// the second operand is 128 rows of the gate matrix and the same 128 of the up matrix, so both
// projections of one column meet in one thread.
//
// An expert's rows are the contraction of a weight gradient and may end inside a
// block: the block's last step of 16 is then zeroed behind them in shared memory, in both
// operands, because what lies there may be a NaN.
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

constexpr int kTileM = 256;                        // of a pair; each CTA has half
constexpr int kTileN = 256;
constexpr int kHalf = 128;
constexpr int kBlockK = 64;                        // bf16: one 128-byte swizzled row
constexpr int kOperand = kHalf * kBlockK * 2;      // one operand of a CTA's stage, 16 KB
constexpr int kBox = kBlockK * 128;                // 64 rows x 128 bytes of an operand that runs across the contraction
constexpr int kChunk = 32;                         // rows of the smaller box of the rows operand
constexpr int kStages = 6;
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 128 + kEpilogueWarps * kWarp;  // producer, MMA, relay, spare | epilogue
constexpr int kOutRow = 128;                       // bytes of one epilogue thread's results
constexpr int kOutBytes = kWarp * kOutRow;         // of a warp's
constexpr int kTmemColumns = 512;

struct Params {
    Bf16GemmArgs g;
    int kb;                // blocks of the contraction (rows forms)
    int tiles_m, tiles_n;  // tiles_m: kWgrad
    int out_n;             // columns of the output (of each half of it)
};

struct Shared {
    uint64_t full[kStages];      // bytes have landed: leader's, of both CTAs (rows forms); each CTA's own (kWgrad)
    uint64_t ready[kStages];     // leader's, kWgrad: both CTAs' blocks are complete and zeroed behind the last row
    uint64_t empty[kStages];     // both: the MMAs that read the stage are done
    uint64_t acc_full[2];        // both: a tile's sums are in TMEM
    uint64_t acc_empty[2];       // leader's: the epilogue warps of the pair have read them
    int first[kRowGroups + 2];   // tiles before each group of 32 experts
    uint32_t tmem;
    Waits waits;
};

// Bounded waits, as gemm::wait_for, at cluster scope.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, Waits* w) {
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait_cluster(bar, parity)) return true;
    const long long start = globaltimer_ns();
    do {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait_cluster(bar, parity)) return true;
    } while (globaltimer_ns() - start < gemm::kWaitLimitNs);
    *reinterpret_cast<volatile int*>(&w->ran_out) = 1;
    return false;
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, Waits* w) {
    return gemm::wait_for<false>(bar, parity, w);
}

// A place in a ring of barriers.
template <int kSize>
struct Ring {
    uint32_t at = 0, phase;
    __device__ __forceinline__ explicit Ring(uint32_t first_phase) : phase(first_phase) {}
    __device__ __forceinline__ void next() {
        if (++at == kSize) {
            at = 0;
            phase ^= 1;
        }
    }
};

// Tile t of a weight gradient: expert, tile of rows, tile of columns.
struct WgradTile {
    int e, m, n, rows;
};
__device__ __forceinline__ WgradTile wgrad_tile(int t, const Params& p) {
    const int per = p.tiles_m * p.tiles_n, e = t / per, local = t - e * per;
    return WgradTile{e, local / p.tiles_n, local % p.tiles_n, min(max(__ldg(p.g.count + e), 0), p.g.cap)};
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <Bf16Form kForm, bool kOut16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ll_gemm_bf16_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_a32,
                        const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_out,
                        const __grid_constant__ CUtensorMap map_gate_up, const Params p) {
    constexpr bool kWgrad = kForm == Bf16Form::kWgrad;
    constexpr bool kSwiglu = kForm == Bf16Form::kSwiglu, kDswiglu = kForm == Bf16Form::kDswiglu;
    constexpr bool kAcrossB = kWgrad || kForm == Bf16Form::kDgrad || kDswiglu;  // b's rows run across the contraction
    extern __shared__ uint8_t s_raw[];
    // stages first, on a 1024-byte boundary as the swizzle needs, at the same offset in both CTAs
    uint8_t* s_tiles = s_raw + ((1024u - (smem_addr(s_raw) & 1023u)) & 1023u);
    uint8_t* s_out = s_tiles + kStages * 2 * kOperand;
    Shared* s = reinterpret_cast<Shared*>(s_out + kEpilogueWarps * kOutBytes);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / kWarp, 0), lane = threadIdx.x % kWarp;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s->full[i], 1);
            mbar_init(&s->ready[i], 2);
            mbar_init(&s->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->acc_full[i], 1);
            mbar_init(&s->acc_empty[i], 2 * kEpilogueWarps);
        }
        s->waits = Waits{0, 0};
        fence_mbarrier_init();
        prefetch_tensormap(&map_a);
        prefetch_tensormap(&map_b);
        prefetch_tensormap(&map_out);
    }
    if (warp == 4) tmem_alloc_pair(&s->tmem, kTmemColumns);
    griddep_wait();  // counts, rows and weights are complete from here on
    griddep_launch_dependents();
    RowTiles<kTileM> walk{p.g.count, s->first, p.g.E, p.g.cap, p.tiles_n};
    if (!kWgrad && warp == 1) walk.fill(s->first, lane);
    tc_fence_before();
    __syncthreads();
    cluster_arrive_release();
    cluster_wait_acquire();
    tc_fence_after();
    const uint32_t tmem = s->tmem;
    const int tiles = kWgrad ? p.g.E * p.tiles_m * p.tiles_n : walk.total();

    if (warp == 0) {
        if (lane == 0) {
            // ---- producer ----
            Ring<kStages> st(1);  // a fresh barrier passes a wait for phase 1
            bool ok = true;
            const uint32_t full = mapa(smem_addr(&s->full[0]), kWgrad ? rank : 0);
            for (int t = pair; t < tiles && ok; t += pairs) {
                int e, ax, ay, bx, kb = p.kb, chunks0 = 4, chunks1 = 4;
                if (kWgrad) {
                    const WgradTile tl = wgrad_tile(t, p);
                    e = tl.e;
                    ax = tl.m * kTileM + static_cast<int>(rank) * kHalf;
                    ay = 0;
                    bx = tl.n * kTileN;
                    kb = (tl.rows + kBlockK - 1) / kBlockK;
                } else {
                    const RowTile tl = walk.at(t);
                    e = tl.e;
                    ax = 0;
                    ay = tl.m0 + static_cast<int>(rank) * kHalf;
                    bx = tl.col * (kSwiglu ? kHalf : kTileN);
                    chunks0 = (min(tl.rows, kHalf) + kChunk - 1) / kChunk;
                    chunks1 = (min(max(tl.rows - kHalf, 0), kHalf) + kChunk - 1) / kChunk;
                }
                if (!kSwiglu) bx += static_cast<int>(rank) * kHalf;
                const int chunks = rank == 0 ? chunks0 : chunks1;
                const uint32_t bytes = kWgrad ? 2 * kOperand : 2 * kOperand + (chunks0 + chunks1) * kChunk * 128;
                for (int b = 0; b < kb; ++b) {
                    if (!(ok = wait_for(&s->empty[st.at], st.phase, &s->waits))) break;
                    if (kWgrad || rank == 0) mbar_arrive_expect_tx(&s->full[st.at], bytes);
                    const uint32_t bar = full + st.at * sizeof(uint64_t);
                    const uint32_t ta = smem_addr(s_tiles) + st.at * 2 * kOperand, tb = ta + kOperand;
                    const int c = b * kBlockK;
                    if (kAcrossB) {
                        for (int i = 0; i < 2; ++i) tma_load_3d(tb + i * kBox, &map_b, bx + i * 64, c, e, bar);
                    } else {
                        tma_load_3d(tb, &map_b, c, bx, kSwiglu ? 2 * e + static_cast<int>(rank) : e, bar);
                    }
                    if (kWgrad) {
                        for (int i = 0; i < 2; ++i) tma_load_3d(ta + i * kBox, &map_a, ax + i * 64, c, e, bar);
                    } else if (chunks == kHalf / kChunk) {
                        tma_load_3d(ta, &map_a, c, ay, e, bar);
                    } else {
                        for (int i = 0; i < chunks; ++i)
                            tma_load_3d(ta + i * kChunk * 128, &map_a32, c, ay + i * kChunk, e, bar);
                    }
                    st.next();
                }
            }
            // every stage's last read is over before the CTA may leave
            for (int i = 0; i < kStages && ok; ++i, st.next()) ok = wait_for(&s->empty[st.at], st.phase, &s->waits);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            // ---- MMA ----
            constexpr uint32_t idesc = bf16_idesc(kTileM, kTileN, kWgrad, kAcrossB);
            Ring<kStages> st(0);
            Ring<2> acc(1);
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                int kb = p.kb, last = kBlockK / 16;  // steps of the last block
                if (kWgrad) {
                    const int rows = __shfl_sync(0xffffffffu, wgrad_tile(t, p).rows, 0);
                    if (rows == 0) continue;
                    kb = (rows + kBlockK - 1) / kBlockK;
                    last = (rows - (kb - 1) * kBlockK + 15) / 16;
                }
                ok = __all_sync(0xffffffffu, wait_for(&s->acc_empty[acc.at], acc.phase, &s->waits));
                const uint32_t d = tmem + acc.at * kTileN;
                for (int b = 0; b < kb && ok; ++b) {
                    const bool landed = kWgrad ? wait_cluster(&s->ready[st.at], st.phase, &s->waits)
                                               : wait_for(&s->full[st.at], st.phase, &s->waits);
                    ok = __all_sync(0xffffffffu, landed);
                    if (!ok) break;
                    const uint32_t ta = smem_addr(s_tiles) + st.at * 2 * kOperand, tb = ta + kOperand;
                    uint64_t da = kWgrad ? sw128_desc_mn(ta, kBox) : sw128_desc(ta);
                    uint64_t db = kAcrossB ? sw128_desc_mn(tb, kBox) : sw128_desc(tb);
                    asm volatile("" : "+l"(da), "+l"(db));
                    tc_fence_after();
                    if (elect_one()) {
                        // a step of 16: 32 bytes further inside the swizzled row, or 16 rows further
#pragma unroll
                        for (int k = 0; k < kBlockK / 16; ++k)
                            if (!kWgrad || b + 1 < kb || k < last)
                                mma_f16_pair(d, da + k * (kWgrad ? 128 : 2), db + k * (kAcrossB ? 128 : 2), idesc,
                                             b > 0 || k > 0);
                        mma_commit_pair(smem_addr(&s->empty[st.at]));
                        if (b + 1 == kb) mma_commit_pair(smem_addr(&s->acc_full[acc.at]));
                    }
                    __syncwarp();
                    st.next();
                }
                acc.next();
            }
        }
    } else if (warp == 2) {
        if (kWgrad) {
            // ---- relay: each block as it lands, zeroed behind the expert's last row ----
            Ring<kStages> st(0);
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const int rows = wgrad_tile(t, p).rows, kb = (rows + kBlockK - 1) / kBlockK;
                for (int b = 0; b < kb; ++b) {
                    ok = __all_sync(0xffffffffu, wait_for(&s->full[st.at], st.phase, &s->waits));
                    if (!ok) break;
                    const int left = rows - b * kBlockK;
                    if (left < kBlockK && left % 16 != 0) {
                        const int end = (left + 15) / 16 * 16;
                        uint8_t* to = s_tiles + st.at * 2 * kOperand;
                        // whole rows of 128 bytes in each of the four boxes, so the swizzle does not matter
                        for (int i = lane; i < (end - left) * 32; i += kWarp) {
                            const int box = i / 8 % 4, row = left + i / 32;
                            *reinterpret_cast<uint4*>(to + box * kBox + row * 128 + i % 8 * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive_cluster(mapa(smem_addr(&s->ready[st.at]), 0));
                    st.next();
                }
            }
        }
    } else if (warp >= 4) {
        // ---- epilogue: thread = one row; four warps have one half of the tile's columns, four the other ----
        const int half = (warp - 4) / 4, quarter = warp % 4;
        const int row = static_cast<int>(rank) * kHalf + quarter * kWarp + lane;  // of the tile
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * kWarp) << 16);
        const uint32_t empty = mapa(smem_addr(&s->acc_empty[0]), 0);
        uint8_t* to = s_out + (warp - 4) * kOutBytes;
        const uint32_t to_addr = smem_addr(to);
        Ring<2> acc(0);
        // 128 bytes of this thread's row into the warp's box of shared memory, in swizzled rows
        const auto stage = [&](const uint4 (&v)[8]) {
            if (lane == 0) bulk_wait_read<0>();  // the last store has left the buffer
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4*>(to + lane * kOutRow + ((j ^ (lane & 7)) << 4)) = v[j];
            fence_proxy_async_smem();
            __syncwarp();
        };
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
            if (kWgrad) {
                const WgradTile tl = wgrad_tile(t, p);
                if (tl.rows > 0) {
                    ok = __all_sync(0xffffffffu, wait_for(&s->acc_full[acc.at], acc.phase, &s->waits));
                    if (!ok) break;
                    tc_fence_after();
                }
                const int y = tl.m * kTileM + static_cast<int>(rank) * kHalf + quarter * kWarp;
                constexpr int kCols = kOut16 ? 64 : 32;  // of one store
#pragma unroll 1
                for (int c = 0; c < kHalf; c += kCols) {
                    uint4 v[8];
                    uint32_t* w = reinterpret_cast<uint32_t*>(v);
#pragma unroll
                    for (int i = 0; i < kCols; i += 32) {
                        uint64_t x[16];
                        if (tl.rows > 0) {
                            tmem_read(lanes + acc.at * kTileN + half * kHalf + c + i, x);
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) x[j] = 0;
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 f = unpack2(x[j]);
                            if (kOut16) {
                                w[i / 2 + j] = pack_bf16(f.x, f.y);
                            } else {
                                w[2 * j] = __float_as_uint(f.x);
                                w[2 * j + 1] = __float_as_uint(f.y);
                            }
                        }
                    }
                    if (c + kCols == kHalf && tl.rows > 0) {
                        tc_fence_before();
                        if (lane == 0) mbar_arrive_cluster_relaxed(empty + acc.at * 8);
                    }
                    const int x0 = tl.n * kTileN + half * kHalf + c;
                    if (x0 >= p.g.k || y >= p.g.n) continue;
                    stage(v);
                    if (lane == 0) {
                        tma_store_3d(&map_out, to_addr, x0, y, tl.e);
                        bulk_commit();
                    }
                }
                if (tl.rows > 0) acc.next();
                continue;
            }
            const RowTile tl = walk.at(t);
            ok = __all_sync(0xffffffffu, wait_for(&s->acc_full[acc.at], acc.phase, &s->waits));
            if (!ok) break;
            tc_fence_after();
            const int y = tl.m0 + static_cast<int>(rank) * kHalf + quarter * kWarp;  // the warp's first row
            const bool whole = row - lane + kWarp <= tl.rows, valid = row < tl.rows;
            const long long r = static_cast<long long>(tl.e) * p.g.cap + y + lane;
            const uint32_t d = lanes + acc.at * kTileN;
            const auto hand_back = [&] {
                tc_fence_before();
                if (lane == 0) mbar_arrive_cluster_relaxed(empty + acc.at * 8);
            };
            if (row - lane >= tl.rows) {
                hand_back();
                acc.next();
                continue;
            }
            // 64 columns from `col` on of the output, or of half `which` of an output of two halves
            const auto put = [&](const uint4 (&v)[8], int col, bool halves, int which, const CUtensorMap* map, void* out) {
                if (col >= p.out_n) return;
                if (whole) {
                    stage(v);
                    if (lane == 0) {
                        if (halves)
                            tma_store_3d(map, to_addr, col, which, static_cast<int>(r));
                        else
                            tma_store_3d(map, to_addr, col, y, tl.e);
                        bulk_commit();
                    }
                } else if (valid) {
                    uint16_t* o = static_cast<uint16_t*>(out) + (halves ? 2 * r + which : r) * p.out_n + col;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (col + 8 * j < p.out_n) st_v4(o + 8 * j, v[j]);
                }
            };
            if (kSwiglu) {
                const int col = tl.col * kHalf + half * 64;
                uint4 vg[8], vu[8], vh[8];
#pragma unroll
                for (int i = 0; i < 64; i += 16) {
                    uint64_t g[8], u[8];
                    tmem_read16x2(d + half * 64 + i, d + kHalf + half * 64 + i, g, u);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 a = unpack2(g[j]), b = unpack2(u[j]);
                        reinterpret_cast<uint32_t*>(vg)[i / 2 + j] = pack_bf16(a.x, a.y);
                        reinterpret_cast<uint32_t*>(vu)[i / 2 + j] = pack_bf16(b.x, b.y);
                        reinterpret_cast<uint32_t*>(vh)[i / 2 + j] = pack_bf16(gated_unit(a.x, b.x), gated_unit(a.y, b.y));
                    }
                }
                hand_back();
                put(vh, col, false, 0, &map_out, p.g.out);
                if (p.g.gate_up_out != nullptr) {
                    put(vg, col, true, 0, &map_gate_up, p.g.gate_up_out);
                    put(vu, col, true, 1, &map_gate_up, p.g.gate_up_out);
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < kHalf; c += 64) {
                    const int col = tl.col * kTileN + half * kHalf + c;
                    if (kDswiglu) {
                        uint4 vg[8], vu[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            vg[j] = vu[j] = make_uint4(0, 0, 0, 0);
                            if (valid && col + 8 * j < p.out_n) {
                                vg[j] = ld_nc_v4(p.g.gate_up + 2 * r * p.out_n + col + 8 * j);
                                vu[j] = ld_nc_v4(p.g.gate_up + (2 * r + 1) * p.out_n + col + 8 * j);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 64; i += 32) {
                            uint64_t x[16];
                            tmem_read(d + half * kHalf + c + i, x);
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                uint32_t& wg = reinterpret_cast<uint32_t*>(vg)[i / 2 + j];
                                uint32_t& wu = reinterpret_cast<uint32_t*>(vu)[i / 2 + j];
                                const float2 f = unpack2(x[j]);
                                const float2 lo = gated_unit_gradient(f.x, __uint_as_float(wg << 16), __uint_as_float(wu << 16));
                                const float2 hi = gated_unit_gradient(f.y, __uint_as_float(wg & 0xffff0000u),
                                                                      __uint_as_float(wu & 0xffff0000u));
                                wg = pack_bf16(lo.x, hi.x);
                                wu = pack_bf16(lo.y, hi.y);
                            }
                        }
                        if (c + 64 == kHalf) hand_back();
                        put(vg, col, true, 0, &map_out, p.g.out);
                        put(vu, col, true, 1, &map_out, p.g.out);
                    } else {
                        uint4 v[8];
#pragma unroll
                        for (int i = 0; i < 64; i += 32) {
                            uint64_t x[16];
                            tmem_read(d + half * kHalf + c + i, x);
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float2 f = unpack2(x[j]);
                                reinterpret_cast<uint32_t*>(v)[i / 2 + j] = pack_bf16(f.x, f.y);
                            }
                        }
                        if (c + 64 == kHalf) hand_back();
                        put(v, col, false, 0, &map_out, p.g.out);
                    }
                }
            }
            acc.next();
        }
        if (lane == 0) bulk_wait_all();
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

// Map of [rows][2][cols] bf16, boxes of 64 columns of one half x 32 rows.
bool make_map_halves(CUtensorMap* map, const void* base, int cols, long long rows) {
    const auto encode = gemm::encode_tiled();
    if (encode == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), 2, static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(cols) * 4};
    const cuuint32_t box[3] = {64, 1, kWarp}, step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Bf16Form kForm, bool kOut16>
cudaError_t launch(const Bf16GemmArgs& g, cudaStream_t stream) {
    using gemm::make_map_bf16;
    constexpr bool kWgrad = kForm == Bf16Form::kWgrad, kSwiglu = kForm == Bf16Form::kSwiglu;
    constexpr bool kTransposed = kForm == Bf16Form::kDgrad || kForm == Bf16Form::kDswiglu;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const auto over = [](int v, int by) { return (v + by - 1) / by; };
    Params p = {};
    p.g = g;
    const int inner = kTransposed ? g.n : g.k;  // rows forms: the contraction
    p.out_n = kWgrad || kTransposed ? g.k : g.n;
    p.kb = over(inner, kBlockK);
    p.tiles_m = over(g.n, kTileM);
    p.tiles_n = over(p.out_n, kSwiglu ? kHalf : kTileN);
    CUtensorMap a = {}, a32 = {}, b = {}, out = {}, gate_up = {};
    bool ok;
    if (kWgrad) {
        if (g.cap > 0)  // without a capacity nothing is loaded
            ok = make_map_bf16(&a, g.rows, g.n, g.cap, g.E, kBlockK) && make_map_bf16(&b, g.other, g.k, g.cap, g.E, kBlockK);
        else
            ok = make_map_bf16(&a, g.out, g.k, g.n, g.E, kBlockK) && make_map_bf16(&b, g.out, g.k, g.n, g.E, kBlockK);
        ok = ok && (kOut16 ? make_map_bf16(&out, g.out, g.k, g.n, g.E, kWarp)
                           : gemm::make_map(&out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, g.out, g.k, g.n, g.E, kWarp));
    } else {
        ok = make_map_bf16(&a, g.rows, inner, g.cap, g.E, kHalf) && make_map_bf16(&a32, g.rows, inner, g.cap, g.E, kChunk) &&
             make_map_bf16(&b, g.other, g.k, g.n, g.E * (kSwiglu ? 2 : 1), kTransposed ? kBlockK : kHalf);
        const long long rows = static_cast<long long>(g.E) * g.cap;
        ok = ok && (kForm == Bf16Form::kDswiglu ? make_map_halves(&out, g.out, p.out_n, rows)
                                                : make_map_bf16(&out, g.out, p.out_n, g.cap, g.E, kWarp));
        if (g.gate_up_out != nullptr) ok = ok && make_map_halves(&gate_up, g.gate_up_out, p.out_n, rows);
    }
    if (!ok) return cudaErrorInvalidValue;
    const size_t smem = 1024 + kStages * 2 * kOperand + kEpilogueWarps * kOutBytes + sizeof(Shared);
    // an upper bound of the tiles: the counts are on the device
    const long long most = static_cast<long long>(g.E) * (kWgrad ? p.tiles_m : over(g.cap, kTileM)) * p.tiles_n;
    const int pairs = static_cast<int>(most < sms / 2 ? most : sms / 2);
    return launch_pdl(ll_gemm_bf16_kernel<kForm, kOut16>, dim3(2 * pairs), dim3(kThreads), smem, stream, 0, true, a, a32, b,
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
