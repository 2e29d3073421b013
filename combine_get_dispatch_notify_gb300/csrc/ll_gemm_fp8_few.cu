// Experts' block-scaled e4m3 products on the tensor cores, tiles of up to 128
// rows (serving's few tokens an expert, and the rest of a longer one).
//
// Here the weights are the tensor cores' row operand: one CTA works alone on 256
// weight rows (two blocks of 128, for the gated product gate and up of the same
// 128 columns) and the rows of a are the columns of its accumulators, 16 to 128
// of them as needed.  Such a tile is bound by the weights' bytes, so they are all
// that is read in full: 32 KB a k-block for each SM, with four stages in flight.  A
// row operand of a's few rows would multiply mostly padding, and its
// accumulators would fill TMEM two blocks deep whatever the row count.
//
//   D[n][m] = sum_{k in block} w[n][k] a[m][k];  acc[n][m] += (as[m] ws) * D[n][m]
//
// An epilogue thread owns one row of each weight block and every other 16
// columns, so a scale read from shared memory serves two products (the reads, 512
// bytes to the registers of a warp each, would else take as long as everything else),
// and gate and up of one output column meet in one thread.
//
// Measured, 7168 -> 2 x 2048 gated: 256 experts with 64 rows each 1.14 to 1.17 ms, 6.6 to 6.7 TB/s
// (the copy rate is 6.67); eight experts with one row each 42 us, 5.6 TB/s.  2048 ->
// 7168, 16 experts with 64 rows each: 44.5 us, 5.7 TB/s.  The short ones pay some 5 us for the
// launch, the first stages and a last round of tiles that not every SM has.  Towards
// 128 rows shared memory bounds it: operands in and out, and the scales' reads.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ll_gemm_fp8.cuh"

namespace ep {
namespace gemm {

namespace {

constexpr int kStages = 4;
constexpr int kStageBytes = 3 * kBoxBytes;  // two blocks of weight rows, up to 128 rows of a
constexpr int kThreads = 384;               // producer, MMA, scales, spare | two epilogue warpgroups
constexpr int kAccColumns = 256;            // TMEM columns of one buffer: both weight blocks, 128 each
constexpr int kScaleSlots = 3;              // of four k-blocks each
constexpr int kPart = 16;                   // rows of a, taken in turn by the two epilogue warpgroups
constexpr int kParts = kFewRows / kPart / 2;  // of one of them

struct Shared {
    uint64_t full[kStages];   // the stage's bytes have landed
    uint64_t empty[kStages];  // its MMAs are done
    uint64_t acc_full[2];     // a block's sums are in TMEM
    uint64_t acc_empty[2];    // every epilogue warp has read them
    uint64_t scale_full[kScaleSlots];
    uint64_t scale_empty[kScaleSlots];
    alignas(16) float row_scale[kScaleSlots][4][kFewRows];  // [k-block][row of a]
    float2 w_scale[kScaleSlots][4];                         // of the two weight blocks
    alignas(16) float amax[2][2][kPart][4];                 // [warpgroup][in turn][row of a][warp]
    int first[kMaxGroups + 2];
    uint32_t tmem;
    Waits waits;
};

// Barrier of an epilogue warpgroup.
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); }

// Whether `ok` holds in all its threads.
__device__ __forceinline__ bool group_all(int g, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.aligned.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(static_cast<uint32_t>(ok)), "r"(1 + g)
        : "memory");
    return all != 0;
}

template <bool kSwiglu, bool kStall>
__global__ void __launch_bounds__(kThreads, 1)
    ll_gemm_fp8_few_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                           const Params p) {
    extern __shared__ uint8_t s_raw[];
    uint8_t* s_tiles = s_raw + ((1024u - (smem_addr(s_raw) & 1023u)) & 1023u);  // as the swizzle needs
    Shared* s = reinterpret_cast<Shared*>(s_tiles + kStages * kStageBytes);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / kWarp, 0), lane = threadIdx.x % kWarp;
    constexpr int kCols = kSwiglu ? kBoxRows : 2 * kBoxRows;  // output columns of a tile

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s->full[i], 1);
            mbar_init(&s->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->acc_full[i], 1);
            mbar_init(&s->acc_empty[i], 8);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&s->scale_full[i], 1);
            mbar_init(&s->scale_empty[i], 8);
        }
        s->waits = Waits{0, p.g.wait_limit_us};
        fence_mbarrier_init();
        prefetch_tensormap(&map_a);
        prefetch_tensormap(&map_w);
    }
    if (warp == 4) tmem_alloc(&s->tmem, kTmemColumns);
    // Also behind the pairs: only a grid that has waited is promised the memory of the grids before it.  With the
    // inputs read while the pairs run, 32 experts with 1024 rows each, gated, 7168 -> 2 x 2048, took 884 us, now 900;
    // 32768 rows of Zipf-distributed experts, 2048 -> 7168, 452 and 450 us.
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 1) count_tiles<true>(s->first, p, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s->tmem;
    const int tiles = s->first[(p.g.E + kWarp - 1) / kWarp];
    const int cta = blockIdx.x, ctas = gridDim.x;

    if (warp < 4) {
        regs_down<88>();
        if (warp == 0 && lane == 0) {
            // ---- producer ----
            uint32_t st = 0, phase = 1;  // a fresh barrier passes a wait for phase 1
            Walk walk;
            bool ok = true;
            for (int t = cta; t < tiles && ok; t += ctas) {
                const Tile tl = tile_at<true>(t, walk, s->first, p, kCols);
                const int chunks = (tl.rows + kChunk - 1) / kChunk;
                const uint32_t bytes = 2 * kBoxBytes + chunks * kChunk * kBlockK;
                const int y1 = kSwiglu ? tl.n0 : tl.n0 + kBoxRows;
                const int z0 = kSwiglu ? 2 * tl.e : tl.e, z1 = kSwiglu ? z0 + 1 : z0;
                for (int b = 0; b < p.kb; ++b) {
                    if (!(ok = wait_for<kStall>(&s->empty[st], phase, &s->waits))) break;
                    const uint32_t bar = smem_addr(&s->full[st]), to = smem_addr(s_tiles) + st * kStageBytes;
                    mbar_arrive_expect_tx(&s->full[st], bytes);
                    tma_load_3d_alone(to, &map_w, b * kBlockK, tl.n0, z0, bar);
                    tma_load_3d_alone(to + kBoxBytes, &map_w, b * kBlockK, y1, z1, bar);
                    for (int c = 0; c < chunks; ++c)
                        tma_load_3d_alone(to + 2 * kBoxBytes + c * kChunk * kBlockK, &map_a, b * kBlockK,
                                          tl.m0 + c * kChunk, tl.e, bar);
                    if (++st == kStages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            // every stage's last read is over before the CTA may leave
            for (int i = 0; i < kStages && ok; ++i) {
                ok = wait_for<kStall>(&s->empty[st], phase, &s->waits);
                if (++st == kStages) {
                    st = 0;
                    phase ^= 1;
                }
            }
        } else if (warp == 1) {
            // ---- MMA ----
            uint32_t st = 0, full_phase = 0, buf = 0, empty_phase = 1;
            Walk walk;
            bool ok = true;
            const int end = kStall && cta == p.g.stall_cta ? min(tiles, cta + p.g.stall_tile * ctas) : tiles;
            for (int t = cta; t < end && ok; t += ctas) {
                const int rows = __shfl_sync(0xffffffffu, tile_at<true>(t, walk, s->first, p, kCols).rows, 0);
                const uint32_t idesc = e4m3_idesc(kBoxRows, (rows + 15) / 16 * 16);
                for (int b = 0; b < p.kb; ++b) {
                    ok = wait_for<kStall>(&s->full[st], full_phase, &s->waits);
                    const uint32_t at = smem_addr(s_tiles) + st * kStageBytes;
                    uint64_t dw = sw128_desc(at), da = sw128_desc(at + 2 * kBoxBytes);
                    asm volatile("" : "+l"(da), "+l"(dw));
                    ok = ok && wait_for<kStall>(&s->acc_empty[buf], empty_phase, &s->waits);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int k = 0; k < kBlockK / 32; ++k)  // 32 bytes further inside the swizzled row
                                mma_e4m3(tmem + buf * kAccColumns + h * kBoxRows, dw + h * (kBoxBytes >> 4) + 2 * k,
                                         da + 2 * k, idesc, k > 0);
                        mma_commit(smem_addr(&s->acc_full[buf]));
                        mma_commit(smem_addr(&s->empty[st]));
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
        } else if (warp == 2) {
            // ---- scales: four rows of a to a lane, four k-blocks at a time ----
            uint32_t slot = 0, phase = 1;
            Walk walk;
            bool ok = true;
            for (int t = cta; t < tiles && ok; t += ctas) {
                const Tile tl = tile_at<true>(t, walk, s->first, p, kCols);
                const float* as = p.g.a_scales + (static_cast<long long>(tl.e) * p.g.cap + tl.m0 + lane) * p.kb;
                const long long step = static_cast<long long>(kWarp) * p.kb;
                const float* ws = weight_scales<kSwiglu>(tl, p, lane & 1);
                for (int b = 0; b < p.kb; b += 4) {
                    float4 a[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[j] = load_scales(as + j * step, b, p.kb, lane + j * kWarp < tl.rows);
                    const float4 w = load_scales(ws, b, p.kb, lane < 2);
                    ok = __all_sync(0xffffffffu, wait_for<kStall>(&s->scale_empty[slot], phase, &s->waits));
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) s->row_scale[slot][i][lane + j * kWarp] = element(a[j], i);
                        if (lane < 2) reinterpret_cast<float*>(&s->w_scale[slot][i])[lane] = element(w, i);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s->scale_full[slot]);
                    if (++slot == kScaleSlots) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue: thread = one row of each weight block; warpgroup g has parts g, g + 2, ... of a's rows ----
        regs_up<208>();
        const int g = (warp - 4) / 4, quarter = warp % 4;
        const int row = quarter * kWarp + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * kWarp) << 16) + g * kPart;
        const uint32_t empty = mapa(smem_addr(s->acc_empty), 0);
        uint32_t it = 0, slot = 0, slot_phase = 0, turn = 0;
        Walk walk;
        bool ok = true;
        for (int t = cta; t < tiles && ok; t += ctas) {
            const Tile tl = tile_at<true>(t, walk, s->first, p, kCols);
            const int parts = (tl.rows + kPart - 1) / kPart;
            uint64_t acc[kParts][2][kPart / 2];
#pragma unroll
            for (int i = 0; i < kParts; ++i)
#pragma unroll
                for (int j = 0; j < kPart / 2; ++j) acc[i][0][j] = acc[i][1][j] = 0;
#pragma unroll 1
            for (int b = 0; b < p.kb; ++b, ++it) {
                const uint32_t buf = it & 1;
                ok = (b & 3) != 0 || wait_for<kStall>(&s->scale_full[slot], slot_phase, &s->waits);
                const ulonglong2* sc = reinterpret_cast<const ulonglong2*>(s->row_scale[slot][b & 3] + g * kPart);
                const float2 ws = s->w_scale[slot][b & 3];
                ok = __all_sync(0xffffffffu, ok && wait_for<kStall>(&s->acc_full[buf], (it / 2) & 1, &s->waits));
                if (!ok) break;
                tc_fence_after();
                const uint32_t col = lanes + buf * kAccColumns;
                const uint64_t w0 = pair2(ws.x), w1 = pair2(ws.y);
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    if (2 * i + g >= parts) break;
                    uint64_t x0[kPart / 2], x1[kPart / 2];
                    tmem_read16x2(col + 2 * i * kPart, col + 2 * i * kPart + kBoxRows, x0, x1);
#pragma unroll
                    for (int j = 0; j < kPart / 4; ++j) {
                        const ulonglong2 v = sc[i * (2 * kPart / 4) + j];
                        fma2(acc[i][0][2 * j], x0[2 * j], mul2(v.x, w0));
                        fma2(acc[i][0][2 * j + 1], x0[2 * j + 1], mul2(v.y, w0));
                        fma2(acc[i][1][2 * j], x1[2 * j], mul2(v.x, w1));
                        fma2(acc[i][1][2 * j + 1], x1[2 * j + 1], mul2(v.y, w1));
                    }
                }
                tc_fence_before();  // the block's sums have left TMEM
                if (lane == 0) mbar_arrive_cluster_relaxed(empty + buf * 8);
                if ((b & 3) == 3 || b + 1 == p.kb) {
                    __syncwarp();  // every lane has read the slot; the arrival hands it back: a release
                    if (lane == 0) mbar_arrive(&s->scale_empty[slot]);
                    if (++slot == kScaleSlots) {
                        slot = 0;
                        slot_phase ^= 1;
                    }
                }
            }
            ok = group_all(g, ok);  // every warp of the group comes here, also when a wait ran out
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                if (2 * i + g >= parts) break;
                const int m0 = (2 * i + g) * kPart;  // the part's first row, and how many are valid
                const int valid = tl.rows - m0;
                const long long r0 = static_cast<long long>(tl.e) * p.g.cap + tl.m0 + m0;
                const int n = tl.n0 + row;
                if (!kSwiglu) {
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.g.y) + r0 * p.g.n + n + w * kBoxRows;
                        const bool on = n + w * kBoxRows < p.g.n;
#pragma unroll
                        for (int j = 0; j < kPart / 2; ++j) {
                            const float2 v = unpack2(acc[i][w][j]);
                            if (on && 2 * j < valid) out[0] = __float2bfloat16_rn(v.x);
                            if (on && 2 * j + 1 < valid) out[p.g.n] = __float2bfloat16_rn(v.y);
                            out += 2LL * p.g.n;
                        }
                    }
                } else {
                    float h[kPart];
                    float mine = 0.0f;  // lane j: the largest of row j among the warp's 32 columns
#pragma unroll
                    for (int j = 0; j < kPart; ++j) {
                        const float2 a = unpack2(acc[i][0][j / 2]), u = unpack2(acc[i][1][j / 2]);
                        h[j] = gated(j % 2 == 0 ? a.x : a.y, j % 2 == 0 ? u.x : u.y);
                        const float m = h[j] == h[j] ? fabsf(h[j]) : 0.0f;
                        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
                        if (lane == j) mine = __uint_as_float(top);
                    }
                    // the other warps have the rest of the block's 128 columns; the buffers take turns, so one barrier
                    // a part is enough
                    float(*amax)[4] = s->amax[g][turn];
                    turn ^= 1;
                    if (lane < kPart) amax[lane][quarter] = mine;
                    group_sync(g);
                    const float4 m = *reinterpret_cast<const float4*>(amax[lane % kPart]);
                    const float scale = block_scale(fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w)));
                    const float inv = 1.0f / scale;
                    if (quarter == 0 && lane < kPart && lane < valid)
                        p.g.y_scales[(r0 + lane) * p.nb + tl.n0 / kScaleBlock] = scale;
                    uint8_t* out = static_cast<uint8_t*>(p.g.y) + r0 * p.g.n + n;
#pragma unroll
                    for (int j = 0; j < kPart; ++j) {
                        const float q = over_scale(h[j], __shfl_sync(0xffffffffu, scale, j), __shfl_sync(0xffffffffu, inv, j));
                        if (n < p.g.n && j < valid)
                            out[static_cast<long long>(j) * p.g.n] =
                                static_cast<uint8_t>(pack_e4m3x4(q, 0.0f, 0.0f, 0.0f));
                    }
                }
            }
        }
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
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tmem, kTmemColumns);
}

template <bool kSwiglu, bool kStall>
cudaError_t launch_form(const GemmArgs& g, cudaStream_t stream) {
    Params p = {};
    p.g = g;
    p.kb = scale_blocks(g.k);
    p.nb = scale_blocks(g.n);
    const int cols = kSwiglu ? kBoxRows : 2 * kBoxRows;
    p.tiles_n = (g.n + cols - 1) / cols;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    CUtensorMap map_a, map_w;
    if (!make_map(&map_a, g.a, g.k, g.cap, g.E, kChunk) ||
        !make_map(&map_w, g.w, g.k, g.n, g.E * (kSwiglu ? 2 : 1), kBoxRows))
        return cudaErrorInvalidValue;
    const size_t smem = 1024 + static_cast<size_t>(kStages) * kStageBytes + sizeof(Shared);
    const long long most = static_cast<long long>(g.E) * p.tiles_n;  // the counts are on the device
    return launch_pdl(ll_gemm_fp8_few_kernel<kSwiglu, kStall>, dim3(static_cast<unsigned>(most < sms ? most : sms)),
                      dim3(kThreads), smem, stream, 0, true, map_a, map_w, p);
}

}  // namespace

cudaError_t launch_few(const GemmArgs& g, cudaStream_t stream) {
    const bool gated = g.y_scales != nullptr;
    if (g.stall) return gated ? launch_form<true, true>(g, stream) : launch_form<false, true>(g, stream);
    return gated ? launch_form<true, false>(g, stream) : launch_form<false, false>(g, stream);
}

}  // namespace gemm
}  // namespace ep
