// What the two kernels of the experts' e4m3 products share: bounded waits, the
// walk over the experts' tiles, scale loads and tensor maps.
//
// An expert's rows are split between them: whole tiles of 256 rows, and a last
// one of more than 128, go to the kernel that works in pairs of SMs
// (ll_gemm_fp8.cu); a rest of up to 128 rows, which for few rows is all of them,
// goes to the kernel that puts the weights on the tensor cores' row side
// (ll_gemm_fp8_few.cu).  With k x n = 7168 x 2 x 2048, 64 rows to each of 76 experts take
// 357 us there and 415 us in pairs, 128 rows 412 and 463 us; with 2048 x 7168, 188 and
// 237 us, 214 and 235 us.  (32 experts, whose tiles fill the pairs' last round and
// not the single CTAs': 128 rows 215 and 193 us, 64 rows 177 and 188 us.)  More than 128
// rows would not fit its epilogue's registers.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "ep.h"
#include "ep_device.cuh"
#include "ep_internal.h"
#include "fp8_cast.cuh"
#include "tcgen05.cuh"

namespace ep {
namespace gemm {

constexpr int kTileM = 256;                  // rows of a pair's tile
constexpr int kFewRows = 128;                // most rows of a tile of the few-rows kernel
constexpr int kChunk = 32;                   // rows of the smaller TMA box of a
constexpr int kBlockK = kScaleBlock;         // 128 e4m3: one 128-byte swizzled row
constexpr int kBoxRows = 128;                // rows of the other TMA boxes
constexpr int kBoxBytes = kBoxRows * kBlockK;  // 16 KB
constexpr int kTmemColumns = 512;
constexpr int kMaxGroups = 8192 / kWarp;     // of 32 experts
constexpr long long kWaitLimitNs = 2000000000LL;

struct Params {
    GemmArgs g;
    int kb, nb, tiles_n;
};

// The CTA's bounded waits, in shared memory.
struct Waits {
    int ran_out;   // 1 once a wait has: the CTA's end then reports it
    int limit_us;  // with kStall
};
// One wait of a role: false when the limit passes.  The role then leaves, and the roles that wait on it do so when
// their own waits run out.  kStall: for the testing hook, whose limit is the caller's.  It is a form of the kernels of
// its own because the limit's register in every wait costs the pairs 4 to 20 % in moves and spills.
template <bool kStall>
__device__ __forceinline__ bool wait_slow(uint64_t* bar, uint32_t parity, Waits* w) {
    const long long start = globaltimer_ns(), limit = kStall ? w->limit_us * 1000LL : kWaitLimitNs;
    do {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
    } while (globaltimer_ns() - start < limit);
    *reinterpret_cast<volatile int*>(&w->ran_out) = 1;
    return false;
}
template <bool kStall>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, Waits* w) {
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return wait_slow<kStall>(bar, parity, w);
}

// The tiles of a kernel: experts in order, then row tiles, then weight tiles.
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
template <bool kFew>
__device__ __forceinline__ int row_tiles(int rows) {
    const int rest = rows % kTileM;
    if (kFew) return rest >= 1 && rest <= kFewRows ? 1 : 0;
    return rows / kTileM + (rest > kFewRows ? 1 : 0);
}
template <bool kFew>
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
        const int n = row_tiles<kFew>(r.rows) * p.tiles_n;
        if (w.before + n > t) break;
        w.before += n;
        ++w.e;
    }
    const int local = t - w.before;
    r.e = w.e;
    r.m0 = kFew ? r.rows / kTileM * kTileM : local / p.tiles_n * kTileM;
    r.n0 = local % p.tiles_n * cols;
    r.rows -= r.m0;
    return r;
}
// Fills `first` (one warp).
template <bool kFew>
__device__ __forceinline__ void count_tiles(int* first, const Params& p, int lane) {
    const int groups = (p.g.E + kWarp - 1) / kWarp;
    int base = 0;
    for (int i = 0; i < groups; ++i) {
        if (lane == 0) first[i] = base;
        const int e = i * kWarp + lane;
        const int n = e < p.g.E ? row_tiles<kFew>(expert_rows(p, e)) * p.tiles_n : 0;
        base += static_cast<int>(__reduce_add_sync(0xffffffffu, n));
    }
    if (lane == 0) first[groups] = base;
}

// Scales of the tile's weight block `which` (0 or 1): gate and up, or two
// neighbours (the last one again when it has no neighbour; those columns are past n).
template <bool kSwiglu>
__device__ __forceinline__ const float* weight_scales(const Tile& t, const Params& p, int which) {
    const long long first = static_cast<long long>(t.e) * (kSwiglu ? 2 : 1) * p.nb + t.n0 / kScaleBlock;
    const long long block = kSwiglu ? which * p.nb : min(which, p.nb - 1 - t.n0 / kScaleBlock);
    return p.g.w_scales + (first + block) * p.kb;
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
__device__ __forceinline__ float element(const float4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// h = gate / (1 + exp(-gate)) * up.  The quotient is made by an approximate reciprocal and corrected by its exact
// remainder (Markstein), to half an ulp; both sides are taken a quarter as large so that the reciprocal of a divisor near
// 2^128 is still a normal number.  __expf and __fdividef would be off by 2^-18 at gates of -80 and 0 below -87.3; the
// general division, 16 to 32 of them in a row, makes a whole product 4 to 14 % longer.
__device__ __forceinline__ float gated(float gate, float up) {
    const float n = 0.25f * gate, d = fmaf(0.25f, expf(-gate), 0.25f);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    const float q = n * r;
    const float c = fmaf(fmaf(-q, d, n), r, q);
    return (c == c ? c : q) * up;  // an infinite side leaves no remainder
}

// ---- host ----
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder (no device work), looked up once.
inline EncodeTiled encode_tiled() {
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

// Map of [outer][rows][cols], boxes of `box_rows` rows x 128 bytes.
inline bool make_map(CUtensorMap* map, CUtensorMapDataType type, int bytes, const void* base, int cols, int rows,
                     int outer, int box_rows) {
    const EncodeTiled encode = encode_tiled();
    if (encode == nullptr) return false;
    const cuuint64_t row = static_cast<cuuint64_t>(cols) * bytes;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[2] = {row, row * rows};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / bytes), static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode(map, type, 3, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline bool make_map(CUtensorMap* map, const void* base, int k, int rows, int outer, int box_rows) {
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, k, rows, outer, box_rows);
}
inline bool make_map_bf16(CUtensorMap* map, const void* base, int n, int rows, int outer, int box_rows) {
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, n, rows, outer, box_rows);
}

cudaError_t launch_few(const GemmArgs& g, cudaStream_t stream);

}  // namespace gemm
}  // namespace ep
