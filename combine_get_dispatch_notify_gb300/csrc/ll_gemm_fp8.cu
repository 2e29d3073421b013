// Experts' block-scaled e4m3 products (ep_ll_gemm_fp8, ep_ll_gemm_swiglu_fp8).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "ep.h"
#include "ep_device.cuh"
#include "ep_internal.h"
#include "fp8_cast.cuh"

namespace ep {

namespace {

constexpr int kRows = 16;      // rows of a tile
constexpr int kCols = 128;     // output columns of a tile: one scale block, one thread each

__device__ __forceinline__ void unpack_e4m3x4(uint32_t v, float* f) {
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(v)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(v >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
}

template <bool kSwiglu>
__global__ void __launch_bounds__(kCols) gemm_kernel(const GemmArgs p) {
    constexpr int kHalves = kSwiglu ? 2 : 1;
    __shared__ float s_a[kRows][kScaleBlock];
    __shared__ float s_scale[kRows];
    __shared__ float s_amax[kCols / kWarp][kRows];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, kb = scale_blocks(p.k), nb = scale_blocks(p.n);
    const int n = blockIdx.x * kCols + tid;
    const int e = blockIdx.z;
    const int rows = min(p.count[e], p.cap);
    for (int m0 = blockIdx.y * kRows; m0 < rows; m0 += gridDim.y * kRows) {
        float acc[kHalves][kRows];
        for (int h = 0; h < kHalves; ++h)
            for (int i = 0; i < kRows; ++i) acc[h][i] = 0.0f;
        for (int b = 0; b < kb; ++b) {
            __syncthreads();
            const int depth = min(kScaleBlock, p.k - b * kScaleBlock);
            for (int i = tid; i < kRows * kScaleBlock / 4; i += kCols) {
                const int r = i / (kScaleBlock / 4), c = i % (kScaleBlock / 4) * 4;
                uint32_t v = 0;
                if (m0 + r < rows && c < depth)
                    v = *reinterpret_cast<const uint32_t*>(
                        p.a + (static_cast<long long>(e) * p.cap + m0 + r) * p.k + b * kScaleBlock + c);
                unpack_e4m3x4(v, &s_a[r][c]);
            }
            if (tid < kRows)
                s_scale[tid] =
                    m0 + tid < rows ? p.a_scales[(static_cast<long long>(e) * p.cap + m0 + tid) * kb + b] : 0.0f;
            __syncthreads();
            if (n < p.n) {
                for (int h = 0; h < kHalves; ++h) {
                    const long long mat = static_cast<long long>(e) * kHalves + h;
                    const uint8_t* w = p.w + (mat * p.n + n) * p.k + b * kScaleBlock;
                    float part[kRows];
                    for (int i = 0; i < kRows; ++i) part[i] = 0.0f;
                    for (int c = 0; c < depth; c += 16) {
                        const uint4 v = *reinterpret_cast<const uint4*>(w + c);
                        float f[16];
                        unpack_e4m3x4(v.x, f);
                        unpack_e4m3x4(v.y, f + 4);
                        unpack_e4m3x4(v.z, f + 8);
                        unpack_e4m3x4(v.w, f + 12);
#pragma unroll
                        for (int i = 0; i < kRows; ++i)
#pragma unroll
                            for (int j = 0; j < 16; ++j) part[i] = fmaf(s_a[i][c + j], f[j], part[i]);
                    }
                    const float ws = p.w_scales[(mat * nb + blockIdx.x) * kb + b];
                    for (int i = 0; i < kRows; ++i) acc[h][i] = fmaf(s_scale[i] * ws, part[i], acc[h][i]);
                }
            }
        }
        if (!kSwiglu) {
            for (int i = 0; i < kRows; ++i)
                if (m0 + i < rows && n < p.n)
                    static_cast<__nv_bfloat16*>(p.y)[(static_cast<long long>(e) * p.cap + m0 + i) * p.n + n] =
                        __float2bfloat16_rn(acc[0][i]);
        } else {
            for (int i = 0; i < kRows; ++i) {
                acc[0][i] = acc[0][i] / (1.0f + expf(-acc[0][i])) * acc[kHalves - 1][i];
                float m = fabsf(acc[0][i]);
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                if (tid % kWarp == 0) s_amax[tid / kWarp][i] = m;
            }
            __syncthreads();
            for (int i = 0; i < kRows; ++i) {
                const float scale =
                    block_scale(fmaxf(fmaxf(s_amax[0][i], s_amax[1][i]), fmaxf(s_amax[2][i], s_amax[3][i])));
                const long long row = static_cast<long long>(e) * p.cap + m0 + i;
                if (m0 + i < rows && n < p.n) {
                    static_cast<uint8_t*>(p.y)[row * p.n + n] =
                        static_cast<uint8_t>(pack_e4m3x4(acc[0][i] / scale, 0.0f, 0.0f, 0.0f));
                    if (tid == 0) p.y_scales[row * nb + blockIdx.x] = scale;
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_ll_gemm_fp8(const GemmArgs& g, cudaStream_t stream) {
    const int want = (g.cap + kRows - 1) / kRows;
    const dim3 grid(static_cast<unsigned>(scale_blocks(g.n)), static_cast<unsigned>(want < 64 ? want : 64),
                    static_cast<unsigned>(g.E));
    return g.y_scales != nullptr ? launch_pdl(gemm_kernel<true>, grid, dim3(kCols), 0, stream, 0, false, g)
                                 : launch_pdl(gemm_kernel<false>, grid, dim3(kCols), 0, stream, 0, false, g);
}

}  // namespace ep
