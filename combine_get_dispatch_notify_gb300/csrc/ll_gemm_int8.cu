// Experts' int8 products (ep_ll_gemm_int8, ep_ll_gemm_swiglu_int8): 16 x 16 tiles
// in shared memory, then for the gated product a cast by rows.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ep.h"
#include "ep_device.cuh"
#include "ep_internal.h"
#include "int8_cast.cuh"
#include "gated.cuh"

namespace ep {

namespace {

constexpr int kTile = 16;

template <bool kSwiglu>
__global__ void ll_gemm_int8_kernel(const Int8GemmArgs p) {
    __shared__ float s_a[kTile][kTile + 1], s_b[2][kTile][kTile + 1];
    griddep_launch_dependents();
    griddep_wait();
    const int tx = threadIdx.x, ty = threadIdx.y;
    for (int e = blockIdx.z; e < p.E; e += gridDim.z) {
        const int M = min(max(__ldg(p.count + e), 0), p.cap);
        for (int m0 = blockIdx.y * kTile; m0 < M; m0 += gridDim.y * kTile)
            for (int n0 = blockIdx.x * kTile; n0 < p.n; n0 += gridDim.x * kTile) {
                float acc[2] = {0.0f, 0.0f};
                for (int k0 = 0; k0 < p.k; k0 += kTile) {
                    const int m = m0 + ty, j = n0 + ty, c = k0 + tx;
                    const long long w0 = (static_cast<long long>(kSwiglu ? 2 : 1) * e * p.n + j) * p.k + c;
                    const bool in = j < p.n && c < p.k;
                    s_a[ty][tx] = m < M && c < p.k ? p.a[(static_cast<long long>(e) * p.cap + m) * p.k + c] : 0;
                    s_b[0][ty][tx] = in ? p.w[w0] : 0;
                    s_b[1][ty][tx] = in && kSwiglu ? p.w[w0 + static_cast<long long>(p.n) * p.k] : 0;
                    __syncthreads();
#pragma unroll
                    for (int i = 0; i < kTile; ++i) {
                        acc[0] = fmaf(s_a[ty][i], s_b[0][tx][i], acc[0]);
                        acc[1] = fmaf(s_a[ty][i], s_b[1][tx][i], acc[1]);
                    }
                    __syncthreads();
                }
                const int m = m0 + ty, j = n0 + tx;
                if (m >= M || j >= p.n) continue;
                const long long row = static_cast<long long>(e) * p.cap + m;
                const float as = __ldg(p.a_scales + row);
                const float* ws = p.w_scales + static_cast<long long>(kSwiglu ? 2 : 1) * e * p.n + j;
                if (kSwiglu)
                    p.h[row * p.n + j] = gated_unit(acc[0] * (as * __ldg(ws)), acc[1] * (as * __ldg(ws + p.n)));
                else
                    static_cast<__nv_bfloat16*>(p.y)[row * p.n + j] = __float2bfloat16_rn(acc[0] * (as * __ldg(ws)));
            }
    }
}

// ---- the gated product's rows, cast ----
constexpr int kCastThreads = 128;

__global__ void __launch_bounds__(kCastThreads) cast_rows_kernel(const Int8GemmArgs p) {
    __shared__ uint32_t s_max[2][kCastThreads / kWarp];
    griddep_launch_dependents();
    griddep_wait();
    int turn = 0;
    for (long long r = blockIdx.x; r < static_cast<long long>(p.E) * p.cap; r += gridDim.x) {
        const int e = static_cast<int>(r / p.cap), m = static_cast<int>(r % p.cap);
        if (m >= __ldg(p.count + e)) continue;
        const float* h = p.h + r * p.n;
        uint32_t most = 0;  // bits of the largest magnitude; NaN is above them all
        for (int c = threadIdx.x * 4; c < p.n; c += kCastThreads * 4) {
            const float4 v = *reinterpret_cast<const float4*>(h + c);
            most = max(max(most, max(__float_as_uint(fabsf(v.x)), __float_as_uint(fabsf(v.y)))),
                       max(__float_as_uint(fabsf(v.z)), __float_as_uint(fabsf(v.w))));
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (threadIdx.x % kWarp == 0) s_max[turn][threadIdx.x / kWarp] = most;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kCastThreads / kWarp; ++i) most = max(most, s_max[turn][i]);
        turn ^= 1;
        const float scale = row_scale(__uint_as_float(most));
        const bool finite = most < 0x7f800000u;
        for (int c = threadIdx.x * 4; c < p.n; c += kCastThreads * 4) {
            const float4 v = *reinterpret_cast<const float4*>(h + c);
            const uint32_t q = finite ? pack_int8x4(v.x / scale, v.y / scale, v.z / scale, v.w / scale) : 0u;
            *reinterpret_cast<uint32_t*>(static_cast<int8_t*>(p.y) + r * p.n + c) = q;
        }
        if (threadIdx.x == 0) p.y_scales[r] = scale;
    }
}

}  // namespace

cudaError_t launch_ll_gemm_int8(const Int8GemmArgs& g, cudaStream_t stream) {
    const auto tiles = [](int v) { return static_cast<unsigned>(v < kTile * 1024 ? (v + kTile - 1) / kTile : 1024); };
    const dim3 grid(tiles(g.n), tiles(g.cap), static_cast<unsigned>(g.E)), block(kTile, kTile);
    if (g.y_scales == nullptr) return launch_pdl(ll_gemm_int8_kernel<false>, grid, block, 0, stream, 0, false, g);
    const cudaError_t e = launch_pdl(ll_gemm_int8_kernel<true>, grid, block, 0, stream, 0, false, g);
    if (e != cudaSuccess) return e;
    const long long rows = static_cast<long long>(g.E) * g.cap;
    return launch_pdl(cast_rows_kernel, dim3(static_cast<unsigned>(rows < 4096 ? rows : 4096)), dim3(kCastThreads), 0,
                      stream, 0, false, g);
}

}  // namespace ep
