// Experts' block-scaled e4m3 products on the tensor cores (ep_ll_gemm_fp8,
// ep_ll_gemm_swiglu_fp8).
//
//   p[m][n] = sum_b as[m][b] ws[n / 128][b] sum_{k in block b} a[m][k] w[n][k]
//
// A pair of CTAs (one cluster, two SMs) owns a tile of 256 rows x 256 weight
// rows and walks the k-blocks of 128.  One tcgen05.mma chain of four (K = 32
// each) leaves a block's plain sums in TMEM; two such accumulators (256
// columns each, all of TMEM) take turns, so the next block multiplies while
// the epilogue warps read this one, scale it by as * ws and add it to fp32
// sums in their registers.  That scaling is what hardware block scales cannot
// do for fp32 scales; it takes 32768 FMAs of an SM per block, half the time
// the tensor core needs for it.
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

#include "ep.h"
#include "ep_device.cuh"
#include "ep_internal.h"
#include "fp8_cast.cuh"
#include "tcgen05.cuh"

namespace ep {

namespace {

constexpr int kTileM = 256;                    // rows of a pair's tile, 128 per CTA
constexpr int kTileN = 256;                    // weight rows of a pair's tile
constexpr int kHalf = 128;                     // rows of a, and of w, that one CTA loads
constexpr int kChunk = 32;                     // rows of one TMA box of a
constexpr int kBlockK = kScaleBlock;           // 128 e4m3: one 128-byte swizzled row
constexpr int kTileBytes = kHalf * kBlockK;    // 16 KB, one operand of a stage
constexpr int kStages = 6;
constexpr int kGroups = 4;                     // epilogue warpgroups, 64 columns of a tile each
constexpr int kGroupCols = kHalf / kGroups;    // of each of the tile's two weight blocks
constexpr int kThreads = 128 + 128 * kGroups;  // producer, MMA, two scale warps | epilogue
constexpr int kEpilogueWarps = 4 * kGroups;
constexpr int kScaleSlots = 4;
constexpr int kAccColumns = kTileN;            // TMEM columns of one accumulator
constexpr int kTmemColumns = 512;
constexpr long long kWaitLimitNs = 2000000000LL;

struct Barriers {
    uint64_t full[kStages];   // leader's: bytes of both CTAs have landed
    uint64_t empty[kStages];  // both: the MMAs that read the stage are done
    uint64_t acc_full[2];     // both: a block's sums are in TMEM, its scales in shared memory
    uint64_t acc_empty[2];    // leader's: every epilogue warp of the pair has read them
};

struct Shared {
    Barriers bar;
    float2 scale[kScaleSlots][kHalf];   // of each row with the tile's two weight blocks
    float amax[2][kGroups][kHalf];      // [tile parity][warpgroup][row]
    int first[8192 / kWarp + 2];  // tiles before each group of 32 experts
    uint32_t tmem;
    int abort;
};

struct Params {
    GemmArgs g;
    int kb, nb, tiles_n;
};

// One wait of a role: false when the limit passes or another role gave up.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, Shared* s) {
    if (mbar_try_wait(bar, parity)) return true;
    long long start = 0;
    uint32_t polls = 0;
    while (!mbar_try_wait(bar, parity)) {
        if ((++polls & 63u) != 0) continue;
        if (*reinterpret_cast<volatile int*>(&s->abort) != 0) return false;
        const long long now = globaltimer_ns();
        if (start == 0) start = now;
        if (now - start > kWaitLimitNs) {
            *reinterpret_cast<volatile int*>(&s->abort) = 1;
            return false;
        }
    }
    return true;
}

// The pair's tiles: experts in order, then row tiles, then weight tiles.
// `first` holds the tiles before each group of 32 experts; a role walks on
// from the expert of its last tile.
struct Walk {
    int e = 0, before = 0;  // an expert, and the tiles before it
};
struct Tile {
    int e, m0, n0, rows;  // rows: valid rows of the expert from m0 on
};
__device__ __forceinline__ int expert_rows(const Params& p, int e) {
    return min(max(__ldg(p.g.count + e), 0), p.g.cap);
}
__device__ __forceinline__ Tile tile_at(int t, Walk& w, const int* first, const Params& p, int cols) {
    if (first[w.e / kWarp + 1] <= t) {
        int group = w.e / kWarp + 1;
        while (first[group + 1] <= t) ++group;
        w.e = group * kWarp;
        w.before = first[group];
    }
    Tile r;
    for (;;) {
        r.rows = expert_rows(p, w.e);
        const int n = (r.rows + kTileM - 1) / kTileM * p.tiles_n;
        if (w.before + n > t) break;
        w.before += n;
        ++w.e;
    }
    const int local = t - w.before;
    r.e = w.e;
    r.m0 = local / p.tiles_n * kTileM;
    r.n0 = local % p.tiles_n * cols;
    r.rows -= r.m0;
    return r;
}

// Row `row` of this CTA's half of the tile, in the packed rows of all experts.
__device__ __forceinline__ long long tile_row(const Tile& t, const Params& p, uint32_t rank, int row) {
    return static_cast<long long>(t.e) * p.g.cap + t.m0 + static_cast<int>(rank) * kHalf + row;
}
// Scales of the tile's two weight blocks: gate and up, or two neighbours (the
// last one twice when it has no neighbour; its columns are past n then).
template <bool kSwiglu>
__device__ __forceinline__ void weight_scales(const Tile& t, const Params& p, const float** w0, const float** w1) {
    const int block = t.n0 / kScaleBlock;
    *w0 = p.g.w_scales + (static_cast<long long>(t.e) * (kSwiglu ? 2 : 1) * p.nb + block) * p.kb;
    *w1 = *w0 + (kSwiglu ? static_cast<long long>(p.nb) * p.kb : (block + 1 < p.nb ? p.kb : 0));
}

__device__ __forceinline__ void store32(void* dst, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Four consecutive k-blocks' scales of a row or a weight block (0 past the end).
__device__ __forceinline__ float4 load_scales(const float* p, int b, int kb, bool on) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!on || b >= kb) return v;
    if (kb % 4 == 0) return __ldg(reinterpret_cast<const float4*>(p + b));  // rows on 16-byte boundaries
    v.x = __ldg(p + b);
    if (b + 1 < kb) v.y = __ldg(p + b + 1);
    if (b + 2 < kb) v.z = __ldg(p + b + 2);
    if (b + 3 < kb) v.w = __ldg(p + b + 3);
    return v;
}
__device__ __forceinline__ float element(const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// acc += s * (16 columns of TMEM).  Scalar FMAs: the packed form (fma.rn.f32x2)
// runs at the same rate on this part and costs moves to pair its operands.
__device__ __forceinline__ void add16(float* acc, uint32_t tmem, float s) {
    float x[16];
    tmem_read16(tmem, x);
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = fmaf(x[j], s, acc[j]);
}

template <bool kSwiglu>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ll_gemm_fp8_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                       const Params p) {
    extern __shared__ uint8_t s_raw[];
    // stages first, on a 1024-byte boundary as the swizzle needs, at the same offset in both CTAs
    const uint32_t pad = (1024u - (smem_addr(s_raw) & 1023u)) & 1023u;
    uint8_t* s_tiles = s_raw + pad;
    Shared* s = reinterpret_cast<Shared*>(s_tiles + kStages * 2 * kTileBytes);
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const int cols = kSwiglu ? kTileN / 2 : kTileN;  // output columns of a tile

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s->bar.full[i], 1);
            mbar_init(&s->bar.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->bar.acc_full[i], 3);  // the MMAs and two scale warps
            mbar_init(&s->bar.acc_empty[i], 2 * kEpilogueWarps);
        }
        s->abort = 0;
        fence_mbarrier_init();
        prefetch_tensormap(&map_a);
        prefetch_tensormap(&map_w);
    }
    if (warp == 4) tmem_alloc_pair(&s->tmem, kTmemColumns);
    griddep_launch_dependents();
    griddep_wait();  // counts, rows and scales are complete from here on
    const int groups = (p.g.E + kWarp - 1) / kWarp;
    if (warp == 1) {  // one warp counts the tiles
        int base = 0;
        for (int i = 0; i < groups; ++i) {
            if (lane == 0) s->first[i] = base;
            const int e = i * kWarp + lane;
            const int n = e < p.g.E ? (expert_rows(p, e) + kTileM - 1) / kTileM * p.tiles_n : 0;
            base += static_cast<int>(__reduce_add_sync(0xffffffffu, n));
        }
        if (lane == 0) s->first[groups] = base;
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive_release();
    cluster_wait_acquire();
    tc_fence_after();
    const uint32_t tmem = s->tmem;
    const int tiles = s->first[groups];

    if (warp < 4) {
        regs_down<64>();
        if (warp == 0 && lane == 0) {
            // ---- producer: this CTA's rows of a and its half of the weight rows ----
            uint32_t it = 0;
            Walk walk;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const Tile tl = tile_at(t, walk, s->first, p, cols);
                const int chunks0 = (min(tl.rows, kHalf) + kChunk - 1) / kChunk;
                const int chunks1 = (min(max(tl.rows - kHalf, 0), kHalf) + kChunk - 1) / kChunk;
                const int chunks = rank == 0 ? chunks0 : chunks1;
                const uint32_t bytes = 2 * kTileBytes + (chunks0 + chunks1) * kChunk * kBlockK;
                const int wy = kSwiglu ? tl.n0 : tl.n0 + static_cast<int>(rank) * kHalf;
                const int wz = kSwiglu ? 2 * tl.e + static_cast<int>(rank) : tl.e;
                const int ay = tl.m0 + static_cast<int>(rank) * kHalf;
                for (int b = 0; b < p.kb; ++b, ++it) {
                    const uint32_t st = it % kStages, use = it / kStages;
                    if (use > 0 && !(ok = wait_for(&s->bar.empty[st], (use - 1) & 1, s))) break;
                    if (rank == 0) mbar_arrive_expect_tx(&s->bar.full[st], bytes);
                    const uint32_t bar = mapa(smem_addr(&s->bar.full[st]), 0);
                    const uint32_t ta = smem_addr(s_tiles) + st * 2 * kTileBytes;
                    tma_load_3d(ta + kTileBytes, &map_w, b * kBlockK, wy, wz, bar);
                    for (int c = 0; c < chunks; ++c)
                        tma_load_3d(ta + c * kChunk * kBlockK, &map_a, b * kBlockK, ay + c * kChunk, tl.e, bar);
                }
            }
            // every stage's last read is over before the CTA may leave
            for (uint32_t i = it > kStages ? it - kStages : 0; i < it && ok; ++i)
                ok = wait_for(&s->bar.empty[i % kStages], (i / kStages) & 1, s);
        } else if (warp == 1 && lane == 0 && rank == 0) {
            // ---- MMA: one thread feeds the pair's tensor cores ----
            constexpr uint32_t idesc = e4m3_idesc(kTileM, kTileN);
            uint32_t it = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                for (int b = 0; b < p.kb; ++b, ++it) {
                    const uint32_t st = it % kStages, buf = it & 1, round = it / 2;
                    if (!(ok = wait_for(&s->bar.full[st], (it / kStages) & 1, s))) break;
                    if (round > 0 && !(ok = wait_for(&s->bar.acc_empty[buf], (round - 1) & 1, s))) break;
                    tc_fence_after();
                    const uint32_t ta = smem_addr(s_tiles) + st * 2 * kTileBytes;
                    const uint64_t da = sw128_desc(ta), dw = sw128_desc(ta + kTileBytes);
#pragma unroll
                    for (int k = 0; k < kBlockK / 32; ++k)  // 32 bytes further inside the swizzled row
                        mma_e4m3_pair(tmem + buf * kAccColumns, da + 2 * k, dw + 2 * k, idesc, k > 0);
                    mma_commit_pair(smem_addr(&s->bar.acc_full[buf]));
                    mma_commit_pair(smem_addr(&s->bar.empty[st]));
                }
            }
        }
        if (warp >= 2) {
            // ---- scales: a row's scale times each weight block's, for two rows a thread, four k-blocks at a time ----
            const int row = threadIdx.x - 64;
            uint32_t it = 0;
            Walk walk;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const Tile tl = tile_at(t, walk, s->first, p, cols);
                const int left = tl.rows - static_cast<int>(rank) * kHalf;
                const float* a0 = p.g.a_scales + tile_row(tl, p, rank, row) * p.kb;
                const float* a1 = a0 + 64LL * p.kb;
                const float *w0, *w1;
                weight_scales<kSwiglu>(tl, p, &w0, &w1);
                float4 na0 = load_scales(a0, 0, p.kb, row < left), na1 = load_scales(a1, 0, p.kb, row + 64 < left),
                       nw0 = load_scales(w0, 0, p.kb, true), nw1 = load_scales(w1, 0, p.kb, true);
                for (int b = 0; b < p.kb && ok; b += 4) {
                    const float4 va0 = na0, va1 = na1, vw0 = nw0, vw1 = nw1;
                    na0 = load_scales(a0, b + 4, p.kb, row < left);  // on their way while these are handed over
                    na1 = load_scales(a1, b + 4, p.kb, row + 64 < left);
                    nw0 = load_scales(w0, b + 4, p.kb, true);
                    nw1 = load_scales(w1, b + 4, p.kb, true);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (b + i >= p.kb) break;
                        // Sums of block it - 2 complete: its MMA waited for the reads of block it - 4, the slot's last user.
                        const uint32_t buf = it & 1;
                        ok = it < 2 || wait_for(&s->bar.acc_full[buf], (it / 2 - 1) & 1, s);
                        if (!__all_sync(0xffffffffu, ok)) {
                            ok = false;
                            break;
                        }
                        float2* slot = s->scale[it % kScaleSlots];
                        const float u = element(va0, i), v = element(va1, i), x = element(vw0, i), y = element(vw1, i);
                        slot[row] = make_float2(u * x, u * y);
                        slot[row + 64] = make_float2(v * x, v * y);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s->bar.acc_full[buf]);
                        ++it;
                    }
                }
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue: thread = one row; warpgroup g sums columns 32 g + [0, 32) of both weight blocks ----
        regs_up<104>();
        const int g = (warp - 4) / 4, quarter = warp % 4;
        const int row = quarter * kWarp + lane;  // of this CTA's 128
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * kWarp) << 16) + g * kGroupCols;
        const uint32_t empty = mapa(smem_addr(&s->bar.acc_empty[0]), 0);
        uint32_t it = 0, parity = 0;
        Walk walk;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs, parity ^= 1) {
            const Tile tl = tile_at(t, walk, s->first, p, cols);
            const int left = tl.rows - static_cast<int>(rank) * kHalf;
            const bool warp_on = quarter * kWarp < left;
            float acc[2 * kGroupCols];  // of the first weight block, then of the second
#pragma unroll
            for (int j = 0; j < 2 * kGroupCols; ++j) acc[j] = 0.0f;
#pragma unroll 1
            for (int b = p.kb; b > 0; --b, ++it) {
                const uint32_t buf = it & 1;
                ok = __all_sync(0xffffffffu, wait_for(&s->bar.acc_full[buf], (it / 2) & 1, s));
                if (!ok) break;
                tc_fence_after();
                if (warp_on) {
                    const float2 sc = s->scale[it % kScaleSlots][row];
                    const uint32_t col = lanes + buf * kAccColumns;
                    add16(acc, col, sc.x);
                    add16(acc + 16, col + 16, sc.x);
                    add16(acc + 32, col + kHalf, sc.y);
                    float x[16];
                    tmem_read16(col + kHalf + 16, x);
                    tc_fence_before();  // the block's sums have left TMEM
                    if (lane == 0) mbar_arrive_cluster_relaxed(empty + buf * 8);
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[48 + j] = fmaf(x[j], sc.y, acc[48 + j]);
                } else {
                    tc_fence_before();
                    if (lane == 0) mbar_arrive_cluster_relaxed(empty + buf * 8);
                }
            }
            if (!ok) {
                // the quarter's other warps may be waiting for this one's maxima
                if (kSwiglu && warp_on) asm volatile("bar.arrive %0, 128;" ::"r"(1 + quarter) : "memory");
                break;
            }
            const bool valid = row < left;
            const long long r = tile_row(tl, p, rank, row);
            if (!kSwiglu) {
                if (valid) {
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.g.y) + r * p.g.n;
                    const bool wide = p.g.n % 16 == 0;  // rows on 32-byte boundaries
#pragma unroll
                    for (int j = 0; j < 4; ++j) {  // 16 columns
                        const int col = tl.n0 + (j / 2) * kHalf + g * kGroupCols + (j % 2) * 16;
                        uint32_t v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const __nv_bfloat162 h =
                                __floats2bfloat162_rn(acc[j * 16 + 2 * i], acc[j * 16 + 2 * i + 1]);
                            v[i] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                        if (wide) {
                            if (col < p.g.n) store32(out + col, v);
                        } else {
                            if (col < p.g.n) st_v4(out + col, make_uint4(v[0], v[1], v[2], v[3]));
                            if (col + 8 < p.g.n) st_v4(out + col + 8, make_uint4(v[4], v[5], v[6], v[7]));
                        }
                    }
                }
            } else if (warp_on) {
                // h = gate / (1 + exp(-gate)) * up; columns past n have zero weights, so h = 0 there
                float amax = 0.0f;
#pragma unroll
                for (int j = 0; j < kGroupCols; ++j) {
                    acc[j] = __fdividef(acc[j], 1.0f + __expf(-acc[j])) * acc[kGroupCols + j];
                    amax = fmaxf(amax, fabsf(acc[j]));
                }
                // the other warpgroups have the rest of the block's 128 columns
                s->amax[parity][g][row] = amax;
                asm volatile("bar.sync %0, 128;" ::"r"(1 + quarter) : "memory");
#pragma unroll
                for (int i = 0; i < kGroups; ++i) amax = fmaxf(amax, s->amax[parity][i][row]);
                const float scale = block_scale(amax);
                if (valid) {
                    const float inv = 1.0f / scale;
                    uint8_t* out = static_cast<uint8_t*>(p.g.y) + r * p.g.n;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {  // 16 columns
                        const int col = tl.n0 + g * kGroupCols + j * 16;
                        uint32_t v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] = pack_e4m3x4(acc[j * 16 + i * 4] * inv, acc[j * 16 + i * 4 + 1] * inv,
                                               acc[j * 16 + i * 4 + 2] * inv, acc[j * 16 + i * 4 + 3] * inv);
                        if (col < p.g.n) st_v4(out + col, make_uint4(v[0], v[1], v[2], v[3]));
                    }
                    if (g == 0) p.g.y_scales[r * p.nb + tl.n0 / kScaleBlock] = scale;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (s->abort != 0) {
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

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder (no device work), looked up once.
EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

// Map of [outer][rows][k] bytes, boxes of `box_rows` rows x 128 bytes.
bool make_map(CUtensorMap* map, const void* base, int k, int rows, int outer, int box_rows) {
    const EncodeTiled encode = encode_tiled();
    if (encode == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(k) * rows};
    const cuuint32_t box[3] = {kBlockK, static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kSwiglu>
cudaError_t launch(const GemmArgs& g, cudaStream_t stream) {
    Params p = {};
    p.g = g;
    p.kb = scale_blocks(g.k);
    p.nb = scale_blocks(g.n);
    const int cols = kSwiglu ? kTileN / 2 : kTileN;
    p.tiles_n = (g.n + cols - 1) / cols;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    CUtensorMap map_a, map_w;
    if (!make_map(&map_a, g.a, g.k, g.cap, g.E, kChunk) ||
        !make_map(&map_w, g.w, g.k, g.n, g.E * (kSwiglu ? 2 : 1), kHalf))
        return cudaErrorInvalidValue;
    const size_t smem = 1024 + static_cast<size_t>(kStages) * 2 * kTileBytes + sizeof(Shared);
    // an upper bound of the tiles: the counts are on the device
    const long long most = static_cast<long long>(g.E) * ((g.cap + kTileM - 1) / kTileM) * p.tiles_n;
    const int pairs = static_cast<int>(most < sms / 2 ? most : sms / 2);
    return launch_pdl(ll_gemm_fp8_kernel<kSwiglu>, dim3(2 * pairs), dim3(kThreads), smem, stream, 0, true, map_a,
                      map_w, p);
}

}  // namespace

cudaError_t launch_ll_gemm_fp8(const GemmArgs& g, cudaStream_t stream) {
    return g.y_scales != nullptr ? launch<true>(g, stream) : launch<false>(g, stream);
}

}  // namespace ep
