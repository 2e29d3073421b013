// Gradient of the weighted combine (ep_ll_combine_backward): a team of threads
// takes one token, reads its gradient once and for each of its slots reads the
// expert's output row, adds up the dot product with it and writes the row's
// gradient.
//
//   grad_y[row] = bf16(w_k g);  grad_w[k] = <g, y[row]>
//
// Products and sums are fp32; the one rounding to fewer bits is grad_y's.  Bound by
// HBM: 2 H bytes of g a token, 2 H in and 2 H out a slot.  Slots are taken eight at a
// time, so that each piece of g is read once and eight loads are in flight a
// thread.  A team is a warp for short rows and four warps for long ones; the sums
// are joined in a fixed order.  2048 tokens x 7168 to 8 slots take 83 us, 32768 tokens
// 1199 us (6.7 TB/s, 98 % of the copy rate).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ep.h"
#include "ep_device.cuh"
#include "ep_internal.h"

namespace ep {

namespace {

constexpr int kThreads = 128;
constexpr int kSlots = 8;           // slots taken together
constexpr int kWarpChunks = 4 * kWarp;  // rows of up to 1024 columns go to one warp

struct Args {
    const uint16_t* grad;
    const uint16_t* y;
    const int64_t* topk_idx;
    const float* topk_w;
    const int32_t* slot_pos;
    uint16_t* grad_y;
    float* grad_w;
    int32_t* status;
    long long tokens;
    int K, E, H, cap;
};

__device__ __forceinline__ float2 bf16x2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ uint32_t scaled(uint32_t g, float w) {
    const float2 f = bf16x2(g);
    const __nv_bfloat162 h = __floats2bfloat162_rn(w * f.x, w * f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float acc) {
    const float2 x = bf16x2(a), y = bf16x2(b);
    return fmaf(x.y, y.y, fmaf(x.x, y.x, acc));
}

template <int kTeam>
__global__ void __launch_bounds__(kThreads) ll_combine_backward_kernel(const Args p) {
    constexpr int kTeams = kThreads / kTeam, kWarps = kTeam / kWarp;
    __shared__ long long s_row[kTeams][kSlots];
    __shared__ float s_wt[kTeams][kSlots];
    __shared__ float s_sum[kTeams][kSlots][kWarps];
    const int team = threadIdx.x / kTeam, tid = threadIdx.x % kTeam, lane = threadIdx.x % kWarp;
    const auto sync = [] {
        if (kWarps == 1)
            __syncwarp();
        else
            __syncthreads();
    };
    griddep_launch_dependents();
    griddep_wait();  // the gradient, the outputs and the row map are complete from here on
    const int chunks = p.H / 8;
    for (long long t = static_cast<long long>(blockIdx.x) * kTeams + team; t < p.tokens;
         t += static_cast<long long>(gridDim.x) * kTeams) {
        const uint16_t* g = p.grad + t * p.H;
        for (int k0 = 0; k0 < p.K; k0 += kSlots) {
            if (tid < kSlots) {
                long long row = -1;
                float w = 0.0f;
                if (k0 + tid < p.K) {
                    const long long e = __ldg(p.topk_idx + t * p.K + k0 + tid);
                    const int pos = __ldg(p.slot_pos + t * p.K + k0 + tid);
                    if (e >= 0 && pos >= 0) {
                        if (e >= p.E || pos >= p.cap) {
                            flag_error(p.status, EP_DEV_INCONSISTENT);
                        } else {
                            row = e * p.cap + pos;
                            w = __ldg(p.topk_w + t * p.K + k0 + tid);
                        }
                    }
                }
                s_row[team][tid] = row;
                s_wt[team][tid] = w;
            }
            sync();
            long long row[kSlots];
            float sum[kSlots];
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                row[i] = s_row[team][i];
                sum[i] = 0.0f;
            }
            for (int c = tid; c < chunks; c += kTeam) {
                const uint4 gv = ld_nc_v4(g + c * 8);
                uint4 v[kSlots];
#pragma unroll
                for (int i = 0; i < kSlots; ++i)
                    if (row[i] >= 0) v[i] = ld_nc_v4(p.y + row[i] * p.H + c * 8);
#pragma unroll
                for (int i = 0; i < kSlots; ++i) {
                    if (row[i] < 0) continue;
                    const float w = s_wt[team][i];
                    sum[i] = dot2(gv.x, v[i].x, sum[i]);
                    sum[i] = dot2(gv.y, v[i].y, sum[i]);
                    sum[i] = dot2(gv.z, v[i].z, sum[i]);
                    sum[i] = dot2(gv.w, v[i].w, sum[i]);
                    st_v4(p.grad_y + row[i] * p.H + c * 8,
                          make_uint4(scaled(gv.x, w), scaled(gv.y, w), scaled(gv.z, w), scaled(gv.w, w)));
                }
            }
            // Eight sums over 32 lanes: at each of three steps a lane keeps half of its sums and gives the other half
            // away, so lane l ends with sum l / 4, joined over two more steps.
#pragma unroll
            for (int half = kSlots / 2; half >= 1; half /= 2) {
                const bool upper = (lane & (half * 4)) != 0;
#pragma unroll
                for (int i = 0; i < half; ++i) {
                    const float give = upper ? sum[i] : sum[i + half], keep = upper ? sum[i + half] : sum[i];
                    sum[i] = keep + __shfl_xor_sync(0xffffffffu, give, half * 4);
                }
            }
            sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 2);
            sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 1);
            if (lane % 4 == 0) s_sum[team][lane / 4][tid / kWarp] = sum[0];
            sync();
            if (tid < kSlots && k0 + tid < p.K) {
                float total = 0.0f;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) total += s_sum[team][tid][i];
                p.grad_w[t * p.K + k0 + tid] = total;
            }
            sync();
        }
    }
}

template <int kTeam>
cudaError_t launch(const Args& p, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const long long want = (p.tokens + kThreads / kTeam - 1) / (kThreads / kTeam), most = sms * 8LL;
    return launch_pdl(ll_combine_backward_kernel<kTeam>, dim3(static_cast<unsigned>(want < most ? want : most)),
                      dim3(kThreads), 0, stream, 0, false, p);
}

}  // namespace

cudaError_t launch_ll_combine_backward(const Shape& sh, const uint16_t* grad, const uint16_t* y, int cap,
                                       const int64_t* topk_idx, const float* topk_w, const int32_t* slot_pos,
                                       uint16_t* grad_y, float* grad_topk_w, int32_t* status, cudaStream_t stream) {
    const Args p = {grad,   y,  topk_idx, topk_w, slot_pos, grad_y, grad_topk_w, status, static_cast<long long>(sh.R) * sh.T,
                    sh.K, sh.E, sh.H,     cap};
    return sh.H / 8 <= kWarpChunks ? launch<kWarp>(p, stream) : launch<kThreads>(p, stream);
}

}  // namespace ep
