// Experts' bf16 products and their gradients (ep_ll_gemm_bf16 and its
// neighbours): one kernel of 16 x 16 tiles in shared memory, fp32 sums, whose
// loads and last step differ by form.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ep.h"
#include "ep_device.cuh"
#include "ep_internal.h"
#include "gated.cuh"

namespace ep {

namespace {

constexpr int kTile = 16;

__device__ __forceinline__ float value(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16); }
__device__ __forceinline__ uint16_t bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

__global__ void ll_gemm_bf16_kernel(const Bf16GemmArgs p) {
    __shared__ float s_a[kTile][kTile + 1], s_b[2][kTile][kTile + 1];
    griddep_launch_dependents();
    griddep_wait();
    const bool wgrad = p.form == Bf16Form::kWgrad, swiglu = p.form == Bf16Form::kSwiglu;
    const bool transposed = p.form == Bf16Form::kDgrad || p.form == Bf16Form::kDswiglu;
    const int tx = threadIdx.x, ty = threadIdx.y;
    const long long n = p.n, k = p.k;
    for (int e = blockIdx.z; e < p.E; e += gridDim.z) {
        const int count = min(max(__ldg(p.count + e), 0), p.cap);
        const int M = wgrad ? p.n : count, N = wgrad || transposed ? p.k : p.n, K = wgrad ? count : transposed ? p.n : p.k;
        for (int m0 = blockIdx.y * kTile; m0 < M; m0 += gridDim.y * kTile)
            for (int n0 = blockIdx.x * kTile; n0 < N; n0 += gridDim.x * kTile) {
                float acc[2] = {0.0f, 0.0f};
                for (int k0 = 0; k0 < K; k0 += kTile) {
                    // row ty of a tile, element tx of the contraction
                    const int m = m0 + ty, j = n0 + ty, c = k0 + tx;
                    const long long row = static_cast<long long>(e) * p.cap;
                    float a = 0.0f, b0 = 0.0f, b1 = 0.0f;
                    if (m < M && c < K)
                        a = wgrad ? value(p.rows + (row + c) * n + m) : value(p.rows + (row + m) * (transposed ? n : k) + c);
                    if (j < N && c < K) {
                        if (wgrad)
                            b0 = value(p.other + (row + c) * k + j);
                        else if (transposed)
                            b0 = value(p.other + (e * n + c) * k + j);
                        else
                            b0 = value(p.other + ((swiglu ? 2 : 1) * e * n + j) * k + c);
                        if (swiglu) b1 = value(p.other + ((2LL * e + 1) * n + j) * k + c);
                    }
                    s_a[ty][tx] = a;
                    s_b[0][ty][tx] = b0;
                    s_b[1][ty][tx] = b1;
                    __syncthreads();
#pragma unroll
                    for (int i = 0; i < kTile; ++i) {
                        acc[0] = fmaf(s_a[ty][i], s_b[0][tx][i], acc[0]);
                        acc[1] = fmaf(s_a[ty][i], s_b[1][tx][i], acc[1]);
                    }
                    __syncthreads();
                }
                const int m = m0 + ty, j = n0 + tx;
                if (m >= M || j >= N) continue;
                const long long row = static_cast<long long>(e) * p.cap + m;
                uint16_t* out = static_cast<uint16_t*>(p.out);
                if (wgrad) {
                    const long long at = (e * n + m) * k + j;
                    if (p.out_bf16)
                        out[at] = bits(acc[0]);
                    else
                        static_cast<float*>(p.out)[at] = acc[0];
                } else if (swiglu) {
                    out[row * n + j] = bits(gated_unit(acc[0], acc[1]));
                    if (p.gate_up_out != nullptr) {
                        p.gate_up_out[row * 2 * n + j] = bits(acc[0]);
                        p.gate_up_out[row * 2 * n + n + j] = bits(acc[1]);
                    }
                } else if (p.form == Bf16Form::kDswiglu) {
                    const float2 d = gated_unit_gradient(acc[0], value(p.gate_up + row * 2 * k + j), value(p.gate_up + row * 2 * k + k + j));
                    out[row * 2 * k + j] = bits(d.x);
                    out[row * 2 * k + k + j] = bits(d.y);
                } else {
                    out[row * N + j] = bits(acc[0]);
                }
            }
    }
}

}  // namespace

cudaError_t launch_ll_gemm_bf16(const Bf16GemmArgs& g, cudaStream_t stream) {
    const bool wgrad = g.form == Bf16Form::kWgrad;
    const bool wide = wgrad || g.form == Bf16Form::kDgrad || g.form == Bf16Form::kDswiglu;
    const int M = wgrad ? g.n : g.cap, N = wide ? g.k : g.n;
    const auto tiles = [](int v) { return static_cast<unsigned>(v < kTile * 1024 ? (v + kTile - 1) / kTile : 1024); };
    return launch_pdl(ll_gemm_bf16_kernel, dim3(tiles(N), tiles(M), static_cast<unsigned>(g.E)), dim3(kTile, kTile), 0,
                      stream, 0, false, g);
}

}  // namespace ep
