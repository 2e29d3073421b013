// Router: scores, group and expert selection, weights (ep_route), and the
// gradient of the weights with respect to the logits (ep_route_backward).
// One warp works on one token; its E keys lie in shared memory.
#include <cfloat>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ep.h"
#include "ep_device.cuh"
#include "ep_internal.h"

namespace ep {

namespace {

constexpr int kRouteWarps = 4;
constexpr unsigned kFull = 0xffffffffu;
constexpr uint32_t kNone = 0u;  // key of an expert that cannot be taken

struct RouteArgs {
    const void* logits;
    const float* bias;
    int64_t* topk_idx;
    float* topk_w;
    int32_t* status;
    long long tokens;
    int E, K;
    RouteCfg rc;
};

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* p, long long i) {
    if (kBf16) return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p) + i)) << 16);
    return __ldg(static_cast<const float*>(p) + i);
}

// Largest finite value of the logits' type; its negative is the lowest one.
template <bool kBf16>
__device__ __forceinline__ float largest() {
    return kBf16 ? __uint_as_float(0x7f7f0000u) : FLT_MAX;
}

// Order-preserving map of a float onto uint32: -inf maps to 0x007fffff, so 0
// is free for "cannot be taken".  +0 and -0 are made one key.
__device__ __forceinline__ uint32_t key_of(float f) {
    const uint32_t b = __float_as_uint(f + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;

__device__ __forceinline__ float warp_max(float v) {
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Largest key of keys[lo, hi) and its lowest index (kNone, -1 when none is left).
__device__ __forceinline__ uint32_t warp_best(const uint32_t* keys, int lo, int hi, int lane, int& at) {
    uint32_t best = kNone;
    int idx = 0x7fffffff;
    for (int e = lo + lane; e < hi; e += kWarp)
        if (keys[e] > best) {
            best = keys[e];
            idx = e;
        }
    const uint32_t top = __reduce_max_sync(kFull, best);
    at = static_cast<int>(__reduce_min_sync(kFull, best == top && top != kNone ? idx : 0x7fffffff));
    return top;
}

template <bool kBf16>
__global__ void __launch_bounds__(kRouteWarps* kWarp) route_kernel(const RouteArgs p) {
    extern __shared__ uint32_t s_keys[];
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    uint32_t* keys = s_keys + static_cast<size_t>(warp) * p.E;
    griddep_launch_dependents();
    griddep_wait();  // the logits are complete from here on
    const int per_group = p.E / p.rc.G;
    const bool softmax = p.rc.score == 0;
    for (long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + warp; t < p.tokens;
         t += static_cast<long long>(gridDim.x) * kRouteWarps) {
        const long long base = t * p.E;
        bool nan = false;
        float m = -FLT_MAX;
        float sum = 0.0f;
        if (softmax) {
            for (int e = lane; e < p.E; e += kWarp) {
                const float l = load_logit<kBf16>(p.logits, base + e);
                if (l > -largest<kBf16>()) m = fmaxf(m, fminf(l, largest<kBf16>()));
            }
            m = warp_max(m);
            for (int e = lane; e < p.E; e += kWarp) {
                const float l = load_logit<kBf16>(p.logits, base + e);
                if (l > -largest<kBf16>()) sum += expf(fminf(l, largest<kBf16>()) - m);
            }
            sum = warp_sum(sum);
        }
        // softmax keeps the logits' order, so where a key is one score the logit serves
        const bool by_logit = softmax && p.bias == nullptr && (p.rc.group_top == 1 || p.rc.topk_groups == p.rc.G);
        auto score = [&](float l) {
            l = fminf(l, largest<kBf16>());
            return softmax ? expf(l - m) / sum : 1.0f / (1.0f + expf(-l));
        };
        for (int e = lane; e < p.E; e += kWarp) {
            const float l = load_logit<kBf16>(p.logits, base + e);
            uint32_t k = kNone;
            nan |= l != l;
            if (l > -largest<kBf16>()) {
                const float v = by_logit ? fminf(l, largest<kBf16>())
                                         : (p.bias != nullptr ? score(l) + __ldg(p.bias + e) : score(l));
                nan |= v != v;
                if (v > -INFINITY) k = key_of(v);
            }
            keys[e] = k;
        }
        if (__any_sync(kFull, nan) && lane == 0) flag_error(p.status, EP_DEV_INPUT);
        __syncwarp();
        if (p.rc.topk_groups < p.rc.G) {
            uint32_t mine = kNone;  // lane g holds the key of group g
            for (int g = 0; g < p.rc.G; ++g) {
                int at;
                uint32_t k = warp_best(keys, g * per_group, (g + 1) * per_group, lane, at);
                if (p.rc.group_top == 2 && k != kNone) {
                    // the second largest: the best one but for `at`
                    const uint32_t first = k;
                    __syncwarp();
                    if (lane == 0) keys[at] = kNone;
                    __syncwarp();
                    int at2;
                    const uint32_t second = warp_best(keys, g * per_group, (g + 1) * per_group, lane, at2);
                    __syncwarp();
                    if (lane == 0) keys[at] = first;
                    __syncwarp();
                    if (second != kNone) k = key_of(of_key(first) + of_key(second));
                }
                if (lane == g) mine = k;
            }
            unsigned kept = 0;
            for (int j = 0; j < p.rc.topk_groups; ++j) {
                const uint32_t top = __reduce_max_sync(kFull, mine);
                if (top == kNone) break;
                const int g = __ffs(__ballot_sync(kFull, mine == top)) - 1;
                kept |= 1u << g;
                if (lane == g) mine = kNone;
            }
            for (int e = lane; e < p.E; e += kWarp)
                if (!((kept >> (e / per_group)) & 1u)) keys[e] = kNone;
            __syncwarp();
        }
        int idx = -1;  // lane k holds slot k
        for (int k = 0; k < p.K; ++k) {
            int at;
            if (warp_best(keys, 0, p.E, lane, at) == kNone) break;
            if (lane == k) idx = at;
            __syncwarp();
            if (lane == 0) keys[at] = kNone;
            __syncwarp();
        }
        const float l = idx >= 0 ? load_logit<kBf16>(p.logits, base + idx) : 0.0f;
        float w = idx >= 0 ? score(l) : 0.0f;
        if (p.rc.renorm) {
            if (softmax) {
                const float top = warp_max(idx >= 0 ? fminf(l, largest<kBf16>()) : -FLT_MAX);
                w = idx >= 0 ? expf(fminf(l, largest<kBf16>()) - top) : 0.0f;
            }
            const float total = warp_sum(w);
            w = total > 0.0f ? w / total : 0.0f;
        }
        if (lane < p.K) {
            p.topk_idx[t * p.K + lane] = idx;
            p.topk_w[t * p.K + lane] = w * p.rc.scale;
        }
        __syncwarp();
    }
}

struct RouteBwdArgs {
    const void* logits;
    const int64_t* topk_idx;
    const float* grad_w;
    void* grad_logits;
    int32_t* status;
    long long tokens;
    int E, K;
    RouteCfg rc;
};

template <bool kBf16>
__global__ void __launch_bounds__(kRouteWarps* kWarp) route_backward_kernel(const RouteBwdArgs p) {
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    griddep_launch_dependents();
    griddep_wait();  // the logits, ids and gradients are complete from here on
    const bool softmax = p.rc.score == 0;
    const float hi = largest<kBf16>();
    for (long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + warp; t < p.tokens;
         t += static_cast<long long>(gridDim.x) * kRouteWarps) {
        const long long base = t * p.E;
        // lane k holds slot k
        long long id = lane < p.K ? __ldg(p.topk_idx + t * p.K + lane) : -1;
        if (id < -1 || id >= p.E) {
            flag_error(p.status, EP_DEV_INPUT);
            id = -1;
        }
        const int idx = static_cast<int>(id);
        float l = idx >= 0 ? load_logit<kBf16>(p.logits, base + idx) : -INFINITY;
        const bool on = l > -hi;  // a masked expert's score is 0 and stays 0
        l = fminf(l, hi);
        const float g = on ? __ldg(p.grad_w + t * p.K + lane) * p.rc.scale : 0.0f;
        float m = 0.0f, inv = 0.0f;
        const bool dense = softmax && !p.rc.renorm;
        if (dense) {
            m = -FLT_MAX;
            float sum = 0.0f;
            for (int e = lane; e < p.E; e += kWarp) {
                const float v = load_logit<kBf16>(p.logits, base + e);
                if (v > -hi) m = fmaxf(m, fminf(v, hi));
            }
            m = warp_max(m);
            for (int e = lane; e < p.E; e += kWarp) {
                const float v = load_logit<kBf16>(p.logits, base + e);
                if (v > -hi) sum += expf(fminf(v, hi) - m);
            }
            sum = warp_sum(sum);
            inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        }
        const float top = softmax && !dense ? warp_max(on ? l : -FLT_MAX) : 0.0f;
        float s;  // the kept score
        if (!softmax)
            s = on ? 1.0f / (1.0f + expf(-l)) : 0.0f;
        else if (dense)
            s = on ? expf(l - m) * inv : 0.0f;
        else
            s = on ? expf(l - top) : 0.0f;
        float ds = g;  // gradient of the kept score
        if (p.rc.renorm) {
            const float total = warp_sum(s);
            const float v = total > 0.0f ? s / total : 0.0f;
            const float c = g - warp_sum(v * g);
            ds = softmax ? c : (total > 0.0f ? c / total : 0.0f);
            if (softmax) s = v;
        }
        const float dot = dense ? warp_sum(s * ds) : 0.0f;
        const float own = softmax ? s * ds : s * (1.0f - s) * ds;  // this slot's part of its expert's gradient
        for (int e0 = 0; e0 < p.E; e0 += kWarp) {
            const int e = e0 + lane;
            float d = 0.0f;
            if (dense && e < p.E) {
                const float v = load_logit<kBf16>(p.logits, base + e);
                if (v > -hi) d = -expf(fminf(v, hi) - m) * inv * dot;
            }
            for (int k = 0; k < p.K; ++k) {
                const int ek = __shfl_sync(kFull, idx, k);
                const float gk = __shfl_sync(kFull, own, k);
                if (ek == e && ek >= 0) d += gk;
            }
            if (e < p.E) {
                if (kBf16)
                    static_cast<__nv_bfloat16*>(p.grad_logits)[base + e] = __float2bfloat16_rn(d);
                else
                    static_cast<float*>(p.grad_logits)[base + e] = d;
            }
        }
    }
}

}  // namespace

cudaError_t launch_route(const Shape& sh, const RouteCfg& rc, const void* logits, bool bf16, const float* bias,
                         int64_t* topk_idx, float* topk_w, int32_t* status, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const RouteArgs p = {logits, bias, topk_idx, topk_w, status, static_cast<long long>(sh.R) * sh.T, sh.E, sh.K, rc};
    const long long want = (p.tokens + kRouteWarps - 1) / kRouteWarps;
    const long long most = sms * 16LL;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    const size_t smem = sizeof(uint32_t) * kRouteWarps * static_cast<size_t>(sh.E);
    return bf16 ? launch_pdl(route_kernel<true>, grid, dim3(kRouteWarps * kWarp), smem, stream, 0, false, p)
                : launch_pdl(route_kernel<false>, grid, dim3(kRouteWarps * kWarp), smem, stream, 0, false, p);
}

cudaError_t launch_route_backward(const Shape& sh, const RouteCfg& rc, const void* logits, bool bf16,
                                  const int64_t* topk_idx, const float* grad_topk_w, void* grad_logits,
                                  int32_t* status, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const RouteBwdArgs p = {logits, topk_idx, grad_topk_w, grad_logits, status, static_cast<long long>(sh.R) * sh.T,
                            sh.E, sh.K, rc};
    const long long want = (p.tokens + kRouteWarps - 1) / kRouteWarps;
    const long long most = sms * 16LL;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    return bf16 ? launch_pdl(route_backward_kernel<true>, grid, dim3(kRouteWarps * kWarp), 0, stream, 0, false, p)
                : launch_pdl(route_backward_kernel<false>, grid, dim3(kRouteWarps * kWarp), 0, stream, 0, false, p);
}

}  // namespace ep
