// Router: scores, group and expert selection, weights (ep_route), and the
// gradient of the weights with respect to the logits (ep_route_backward).
// One warp works on one token.
//
// ep_route has three kernels.  route_lists_kernel, and route_bf16_kernel for
// bf16 logits whose order the keys keep (no bias, no groups), keep a lane's keys as
// one sorted list of 32-bit words in registers and take the K winners off the lists' heads;
// route_kernel keeps the keys in shared memory and covers what the lists do not
// (more than 512 experts, softmax scores with a bias or summed for groups).
// Where two of them could take a case, measured: 32768 tokens x 256 fp32 sigmoid
// keys in 8 groups 27 us with lists, 63 us in shared memory; 524288 x 256 bf16 logits
// 144 us in route_bf16_kernel (2.2 TB/s), 316 us in route_lists_kernel, 617 us in
// shared memory; 131072 x 256 bf16, sigmoid without a bias, 47 and 89 us.  The bytes
// alone would take 5 and 48 us of the first two: selection is bound by the integer
// pipe, which minima, maxima, compares and selects share at half rate (70 % busy in
// route_bf16_kernel, 57 % in route_lists_kernel, 260 instructions a token).
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

// Over the `W` neighbouring lanes around this one.
template <int W = kWarp>
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
template <int W = kWarp>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// Two sums over the warp in six exchanges: half the lanes go on with each.
__device__ __forceinline__ void warp_sum2(float& a, float& b, int lane) {
    const bool low = lane < kWarp / 2;
    float v = (low ? a : b) + __shfl_xor_sync(kFull, low ? b : a, kWarp / 2);
#pragma unroll
    for (int o = kWarp / 4; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    const float w = __shfl_xor_sync(kFull, v, kWarp / 2);
    a = low ? v : w;
    b = low ? w : v;
}

// ---------------------------------------------------------------------------
// Lists in registers.
//
// Lane i holds the N consecutive experts from i * N on.  A key becomes one word,
// its order-preserving bits cut to 32 - kIdxBits with the complemented index
// below them, so one unsigned maximum finds the largest key and, among equals,
// the lowest index.  Each lane sorts its words once; a round is then a
// redux.max over the list heads and one shift in the winner's lane.

template <int N>
__device__ __forceinline__ void sort_descending(uint32_t (&v)[N]) {
    // odd-even merge sort (Batcher)
#pragma unroll
    for (int p = 1; p < N; p <<= 1)
#pragma unroll
        for (int k = p; k >= 1; k >>= 1)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t hi = max(v[i + j], v[i + j + k]), lo = min(v[i + j], v[i + j + k]);
                        v[i + j] = hi;
                        v[i + j + k] = lo;
                    }
}

// Takes the largest words off the lists; lane r gets the r-th (0 past the end).
// A winner goes through shared memory, stored by the lane that had it: the
// integer pipe, half rate, is what bounds these kernels, and a select in every
// lane would use it twice a round.  kRounds > 0: that many rounds, unrolled, and
// round r shifts only what the rounds after it can still take; 0: `rounds` of
// them.
template <int N, int kRounds>
__device__ __forceinline__ uint32_t take(uint32_t (&w)[N], int rounds, int lane, uint32_t* slots) {
    if (kRounds > 0) {
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const uint32_t top = __reduce_max_sync(kFull, w[0]);
            const bool mine = w[0] == top;
            if (mine) slots[r] = top;
#pragma unroll
            for (int j = 0; j < N && j < kRounds - 1 - r; ++j) w[j] = mine ? (j + 1 < N ? w[(j + 1) % N] : 0u) : w[j];
        }
    } else {
        for (int r = 0; r < rounds; ++r) {
            const uint32_t top = __reduce_max_sync(kFull, w[0]);
            const bool mine = w[0] == top;
            if (mine) slots[r] = top;
#pragma unroll
            for (int j = 0; j < N; ++j) w[j] = mine ? (j + 1 < N ? w[(j + 1) % N] : 0u) : w[j];
        }
    }
    __syncwarp();
    const uint32_t win = lane < (kRounds > 0 ? kRounds : rounds) ? slots[lane] : 0u;
    __syncwarp();
    return win;
}

// The K largest of whole keys, ties to the lowest index: lane r gets the r-th one's expert (-1 past the end).
template <int N, typename Expert>
__device__ __forceinline__ int exact_rounds(uint32_t (&k)[N], int K, int lane, Expert expert) {
    int idx = -1;
    for (int r = 0; r < K; ++r) {
        uint32_t best = k[0];
        int at = 0;
#pragma unroll
        for (int j = 1; j < N; ++j)
            if (k[j] > best) {
                best = k[j];
                at = j;
            }
        const uint32_t top = __reduce_max_sync(kFull, best);
        if (top == kNone) break;
        const int from = static_cast<int>(
            __reduce_min_sync(kFull, best == top ? static_cast<uint32_t>(expert(at)) : 0xffffffffu));
        if (lane == r) idx = from;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (expert(j) == from) k[j] = kNone;
    }
    return idx;
}

// Sum over lanes [0, K) (the others hold 0), valid in those lanes.
template <int kFewK>
__device__ __forceinline__ float sum_kept(float v) {
    if (kFewK > 0) {  // K <= kFewK
#pragma unroll
        for (int o = 1; o < kFewK; o <<= 1) v += __shfl_xor_sync(kFull, v, o);
        return v;
    }
    return warp_sum(v);
}

// K up to this has its rounds unrolled, each shifting no more than the rest can take: 524288 x 256 bf16, K = 8, 148 us
// and 174 us in a loop; 32768 x 256 fp32 in groups 27 and 29 us.
constexpr int kFewK = 8;

// Where a warp's slots go; moved along with its tokens, so that no token needs a
// 64-bit product.
struct SlotOut {
    int64_t* idx;
    float* w;
    long long step;
    __device__ __forceinline__ SlotOut(const RouteArgs& p, long long t, long long tokens)
        : idx(p.topk_idx + t * p.K), w(p.topk_w + t * p.K), step(tokens * p.K) {}
    __device__ __forceinline__ void put(int slot, int i, float v) {
        idx[slot] = i;
        w[slot] = v;
    }
    __device__ __forceinline__ void move() {
        idx += step;
        w += step;
    }
};

__device__ __forceinline__ float sigmoid_exact(float l) { return 1.0f / (1.0f + expf(-l)); }

// ---- bf16 logits that are the keys themselves: the word holds the whole key ----
//
// Two logits are ordered by two instructions: a negative half flips all its
// bits, a positive one its sign.  In that order -inf, the lowest value and
// negative NaNs come last (up to kLowest16), +inf and positive NaNs first (from
// kInf16 on), so masked experts need no test.  Infinite and NaN logits, and zeros
// of either sign among the winners (equal keys with different bits), are rare:
// such a token runs once more over words cleaned one by one.
//
// A sigmoid without a bias keeps the logits' order, but two logits may share one
// fp32 sigmoid, and then the lower index comes first.  With neighbouring bf16 values at least
// 2^-9 |l| apart, sigmoids are more than four roundings apart where (1 - s) |l| > 2^-13,
// as it is for 2^-10 <= |l| with -80 <= l <= 11: such a winner is above every lower
// logit.  A token with another winner takes its rounds over exact sigmoids.
constexpr uint32_t kLowest16 = 0x0080u, kMinusInf16 = 0x007fu, kInf16 = 0xff80u, kLargest16 = 0xff7fu;
constexpr uint32_t kMinusZero16 = 0x7fffu, kZero16 = 0x8000u;

// 0xffff in each half whose sign is set.
__device__ __forceinline__ uint32_t half_signs(uint32_t v) {
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, 0xbb99;" : "=r"(r) : "r"(v));
    return r;
}

// a / b for a in [0, 1] and a sum b of 1 to 512: a quotient by an approximate reciprocal, corrected once by its exact
// remainder (Markstein), which makes it the nearest fp32 number but where a / b is within 2^-44 of halfway between two.  The
// general division's checks for sizes that do not occur here cost 524288 x 256 tokens 23 of 145 us.
__device__ __forceinline__ float over_sum(float a, float b) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b));
    const float q = a * r;
    return fmaf(fmaf(-q, b, a), r, q);
}

template <int N, bool kFew, bool kSigmoid>
__global__ void __launch_bounds__(kRouteWarps* kWarp) route_bf16_kernel(const RouteArgs p) {
    __shared__ uint32_t s_slots[kRouteWarps][kWarp];
    const int lane = threadIdx.x % kWarp, first = lane * N;
    uint32_t* slots = s_slots[threadIdx.x / kWarp];
    griddep_launch_dependents();
    griddep_wait();  // the logits are complete from here on
    const long long step = static_cast<long long>(gridDim.x) * kRouteWarps;
    long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + threadIdx.x / kWarp;
    const bool on = first < p.E;  // E is a multiple of N; lanes past it hold masked logits
    const uint16_t* src = static_cast<const uint16_t*>(p.logits) + t * p.E + first;
    SlotOut out(p, t, step);
    uint32_t next[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) next[i] = 0xff80ff80u;  // -inf
    auto load = [&]() {
        if (!on) return;
        if (N % 8 == 4 && N > 4) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(src) + i);
                next[(2 * i) % (N / 2)] = v.x;
                next[(2 * i + 1) % (N / 2)] = v.y;
            }
        } else if (N >= 8) {
#pragma unroll
            for (int i = 0; i < N / 8; ++i) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
                next[(4 * i) % (N / 2)] = v.x;
                next[(4 * i + 1) % (N / 2)] = v.y;
                next[(4 * i + 2) % (N / 2)] = v.z;
                next[(4 * i + 3) % (N / 2)] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) next[i] = __ldg(reinterpret_cast<const uint32_t*>(src) + i);
        }
    };
    if (t < p.tokens) load();
    for (; t < p.tokens; t += step, out.move()) {
        uint32_t raw[N / 2];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) raw[j] = next[j];
        src += step * p.E;
        if (t + step < p.tokens) load();
        uint32_t w[N];
        auto words = [&]() {
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const uint32_t o = raw[j] ^ (half_signs(raw[j]) | 0x80008000u);
                w[2 * j] = __byte_perm(o, 0xffffu - static_cast<uint32_t>(first + 2 * j), 0x1054);
                w[2 * j + 1] = __byte_perm(o, 0xffffu - static_cast<uint32_t>(first + 2 * j + 1), 0x3254);
            }
        };
        words();
        sort_descending<N>(w);
        bool special = w[0] >= (kInf16 << 16) || w[N - 1] < (kMinusInf16 << 16);
        uint32_t win = take<N, kFew ? kFewK : 0>(w, p.K, lane, slots);
        uint32_t o = win >> 16;
        auto value = [](uint32_t half) { return __uint_as_float((half & 0x8000u ? half ^ 0x8000u : half ^ 0xffffu) << 16); };
        bool kept = lane < p.K && o > kLowest16;
        float logit = value(o);
        int idx = kept ? static_cast<int>(0xffffu - (win & 0xffffu)) : -1;
        if (kSigmoid)
            special |= kept && !(logit >= -80.0f && logit <= 11.0f && fabsf(logit) >= 9.765625e-4f);
        else  // a zero among the winners: a kept one is always seen, and with none kept no zero matters
            special |= o - kMinusZero16 <= 1u;
        if (__any_sync(kFull, special)) {
            bool nan = false;
            if (kSigmoid) {
                const float lim = largest<true>();
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float l = __uint_as_float(j % 2 == 0 ? raw[j / 2] << 16 : raw[j / 2] & 0xffff0000u);
                    nan |= l != l;
                    w[j] = l > -lim ? key_of(sigmoid_exact(fminf(l, lim))) : kNone;
                }
                idx = exact_rounds<N>(w, p.K, lane, [&](int j) { return first + j; });
                kept = idx >= 0;
                logit = kept ? fminf(load_logit<true>(p.logits, t * p.E + idx), lim) : 0.0f;
            } else {
                words();
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    uint32_t c = w[j] >> 16;
                    nan |= c > kInf16 || c < kMinusInf16;
                    c = c > kInf16 || c <= kLowest16 ? 0u : c == kInf16 ? kLargest16 : c == kMinusZero16 ? kZero16 : c;
                    w[j] = c == 0u ? 0u : (c << 16) | (w[j] & 0xffffu);
                }
                sort_descending<N>(w);
                win = take<N, 0>(w, p.K, lane, slots);
                o = win >> 16;
                kept = lane < p.K && o > kLowest16;
                logit = value(o);
                idx = kept ? static_cast<int>(0xffffu - (win & 0xffffu)) : -1;
            }
            if (__any_sync(kFull, nan) && lane == 0) flag_error(p.status, EP_DEV_INPUT);
        }
        float weight;
        if (kSigmoid) {
            weight = kept ? sigmoid_exact(logit) : 0.0f;
            if (p.rc.renorm) {
                const float total = sum_kept<kFew ? kFewK : 0>(weight);
                weight = total > 0.0f ? weight / total : 0.0f;
            }
        } else {
            // softmax over the winners, the first of them the largest; or over all experts
            const float m = __shfl_sync(kFull, logit, 0);
            const float mine = kept ? expf(logit - m) : 0.0f;
            float total;
            if (p.rc.renorm) {
                total = sum_kept<kFew ? kFewK : 0>(mine);
            } else {
                total = 0.0f;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float l = __uint_as_float(j % 2 == 0 ? raw[j / 2] << 16 : raw[j / 2] & 0xffff0000u);
                    if (l > -largest<true>()) total += expf(fminf(l, largest<true>()) - m);
                }
                total = warp_sum(total);
            }
            weight = over_sum(mine, total);
        }
        if (lane < p.K) out.put(lane, idx, kept ? weight * p.rc.scale : 0.0f);
    }
}

// ---- fp32 keys: cut, and approximate for the sigmoid ----
//
// A sigmoid key is first taken from ex2.approx and rcp.approx, below 2^-20 off;
// the exact sigmoid, some 20 instructions, is computed for the K winners and not
// for E experts.  What comes out is proven token by token: every winner's exact
// key has to be out of the runner-up's reach (its cut and its approximation), and
// the last group kept out of reach of the first one dropped.  The winners'
// own order is settled by their exact keys.  A token that fails (about one in a
// hundred) takes its rounds over exact keys.  So does every token with a masked logit, after its
// first rounds: with eight of 256 fp32 experts masked in every row, 131072 tokens of softmax
// take 160 us and 32768 of sigmoids in 8 groups 72 us, where they take 70 and 31 without
// (each call timed alone; bf16 softmax, whose kernel needs no test, 41 with the mask).

__device__ __forceinline__ float approx_error() { return 9.5367431640625e-07f; }  // 2^-20

// The lane's logits (-inf past E).
template <bool kBf16, int N>
__device__ __forceinline__ void load_lane(const void* logits, long long base, int first, int E, bool vec,
                                          float (&l)[N]) {
    if (vec && first + N <= E && (kBf16 ? N % 8 == 0 : N % 4 == 0)) {
        if (kBf16) {
#pragma unroll
            for (int i = 0; i < N / 8; ++i) {
                const uint4 v =
                    __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(logits) + base + first) + i);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    l[(8 * i + 2 * j) % N] = __uint_as_float(w[j] << 16);
                    l[(8 * i + 2 * j + 1) % N] = __uint_as_float(w[j] & 0xffff0000u);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const float4 v =
                    __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(logits) + base + first) + i);
                l[(4 * i) % N] = v.x;
                l[(4 * i + 1) % N] = v.y;
                l[(4 * i + 2) % N] = v.z;
                l[(4 * i + 3) % N] = v.w;
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) l[j] = first + j < E ? load_logit<kBf16>(logits, base + first + j) : -INFINITY;
}

__device__ __forceinline__ float sigmoid_approx(float l, float& e) {  // e: exp(-l)
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// A group's key from its two largest ones (-inf: no expert can be taken).
__device__ __forceinline__ float group_value(uint32_t k1, uint32_t k2, int group_top) {
    if (k1 == kNone) return -INFINITY;
    return group_top == 2 && k2 != kNone ? of_key(k1) + of_key(k2) : of_key(k1);
}

// Largest and second largest key of the `seg` lanes around this one, from each lane's own two.
__device__ __forceinline__ void segment_merge2(int seg, uint32_t& k1, uint32_t& k2) {
    for (int o = 1; o < seg; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(kFull, k1, o), o2 = __shfl_xor_sync(kFull, k2, o);
        k2 = max(min(k1, o1), max(k2, o2));
        k1 = max(k1, o1);
    }
}
// The same from each lane's N keys.
template <int N>
__device__ __forceinline__ void segment_top2(const uint32_t (&k)[N], int seg, uint32_t& k1, uint32_t& k2) {
    k1 = k[0];
    k2 = kNone;
#pragma unroll
    for (int j = 1; j < N; ++j) {
        k2 = max(k2, min(k1, k[j]));
        k1 = max(k1, k[j]);
    }
    segment_merge2(seg, k1, k2);
}

// Whether this lane's group (value v) is one of the topk_groups largest, ties to
// the lowest.
__device__ __forceinline__ bool group_kept(float v, int G, int seg, int topk, int lane) {
    const int g = lane / seg;
    int above = 0;
    for (int i = 0; i < G; ++i) {
        const float d = __shfl_sync(kFull, v, i * seg) - v;  // every lane takes part; NaN between two infinities
        above += i < g ? !(d < 0.0f) : d > 0.0f;
    }
    return g < G && above < topk;
}

// kMode: 0 the logit is the key (softmax keeps its order), 1 sigmoid.
// kAny false: E is a multiple of N, lane i holds the experts from i * N on, groups
// are runs of `seg` lanes (a power of two).  kAny true: any E and any groups; lane
// i holds every 32nd expert from i on, and the groups' keys pass through a shared
// row from which `seg` lanes scan each group.
template <bool kBf16, int N, int kMode, bool kFew, bool kAny>
__global__ void __launch_bounds__(kRouteWarps* kWarp) route_lists_kernel(const RouteArgs p, int seg, int vec) {
    constexpr int kIdxBits = N <= 8 ? 8 : 9;
    constexpr uint32_t kIdxMask = (1u << kIdxBits) - 1u;
    constexpr float kCut = 1.0f / (1 << (23 - kIdxBits));  // of a key, lost below the index
    __shared__ uint32_t s_slots[kRouteWarps][kWarp];
    __shared__ uint32_t s_rows[kRouteWarps][kAny ? N * kWarp : 1];
    const int lane = threadIdx.x % kWarp;
    uint32_t* slots = s_slots[threadIdx.x / kWarp];
    uint32_t* row = s_rows[threadIdx.x / kWarp];
    const float lim = largest<kBf16>();
    griddep_launch_dependents();
    griddep_wait();  // the logits are complete from here on
    const long long step = static_cast<long long>(gridDim.x) * kRouteWarps;
    const bool groups = p.rc.topk_groups < p.rc.G;
    const int per_group = p.E / p.rc.G;
    auto expert = [&](int j) { return kAny ? lane + kWarp * j : lane * N + j; };
    auto has = [&](int j) { return expert(kAny ? j : 0) < p.E; };  // an expert there
    float bias[N];
    uint32_t group_bit[kAny ? N : 1];
    float largest_key = 1.0f;  // bound of the keys' magnitude
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (kMode == 1) {
            bias[j] = p.bias != nullptr && has(j) ? __ldg(p.bias + expert(j)) : 0.0f;
            largest_key = !(fabsf(bias[j]) < INFINITY) ? INFINITY : fmaxf(largest_key, 1.0f + fabsf(bias[j]));
        }
        if (kAny) group_bit[j % (kAny ? N : 1)] = has(j) ? 1u << (expert(j) / per_group) : 0u;
    }
    if (kMode == 1) largest_key = warp_max(largest_key);
    const bool odd_bias = !(largest_key < INFINITY);  // infinite or NaN: every token goes the exact way
    // two groups closer than this could be ordered wrongly: two approximate keys in each, their sum's roundings
    const float margin = kMode == 1 ? 4.0f * approx_error() + 4.76837158203125e-07f * largest_key : 0.0f;
    auto load = [&](long long base, float (&l)[N]) {
        if (kAny) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (has(j)) l[j] = load_logit<kBf16>(p.logits, base + expert(j));
        } else if (has(0)) {
            load_lane<kBf16, N>(p.logits, base, lane * N, p.E, vec != 0, l);
        }
    };
    // the two largest keys of the lane's group
    auto group_top2 = [&](const uint32_t (&k)[N], uint32_t& k1, uint32_t& k2) {
        if (kAny) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (has(j)) row[expert(j)] = k[j];
            __syncwarp();
            k1 = k2 = kNone;
            const int g = lane / seg;
            if (g < p.rc.G)
                for (int i = lane % seg; i < per_group; i += seg) {
                    const uint32_t v = row[g * per_group + i];
                    k2 = max(k2, min(k1, v));
                    k1 = max(k1, v);
                }
            __syncwarp();
            segment_merge2(seg, k1, k2);
        } else {
            segment_top2<N>(k, seg, k1, k2);
        }
    };
    // whether the lane's expert j is in a group kept, from the kept flags of the groups' lanes
    auto group_mask = [&](bool kept) { return kAny ? __reduce_or_sync(kFull, kept ? 1u << (lane / seg) : 0u) : 0u; };
    auto in_group = [&](int j, bool kept, uint32_t mask) {
        return kAny ? (mask & group_bit[j % (kAny ? N : 1)]) != 0u : kept;
    };
    long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + threadIdx.x / kWarp;
    float next[N];
#pragma unroll
    for (int j = 0; j < N; ++j) next[j] = 0.0f;
    long long base = t * p.E;
    const long long base_step = step * p.E;
    SlotOut out(p, t, step);
    if (t < p.tokens) load(base, next);
    for (; t < p.tokens; t += step, base += base_step, out.move()) {
        uint32_t k[N];
        float m = -FLT_MAX, total = 0.0f;
        if (kMode == 0 && !p.rc.renorm) {  // softmax over all experts
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (has(j) && next[j] > -lim) m = fmaxf(m, fminf(next[j], lim));
            m = warp_max(m);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (has(j) && next[j] > -lim) total += expf(fminf(next[j], lim) - m);
            total = warp_sum(total);
        }
        // Masked and NaN logits leave a NaN here, and so does any below -88 with the sigmoid: such a token goes the
        // exact way, so the keys below need no tests.
        float odd = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float v = next[j];
            if (kMode == 1) {
                float e;
                v = sigmoid_approx(v, e) + bias[j];
                odd = fmaf(e, 0.0f, odd);
            } else {
                odd = fmaf(v * 4.0f, 0.0f, odd);
            }
            k[j] = key_of(v);
        }
        if (t + step < p.tokens) load(base + base_step, next);
        bool bad = odd != odd || odd_bias || p.K == kWarp;  // with 32 winners no lane is left for the runner-up
        bool kept = true;
        uint32_t mask = 0xffffffffu;
        if (groups) {
            uint32_t k1, k2;
            group_top2(k, k1, k2);
            // one word a group, as for the experts; the last one kept has to be clear of the first one dropped
            const float v = p.rc.group_top == 2 ? of_key(k1) + of_key(k2) : of_key(k1);
            const bool mine = lane / seg < p.rc.G;
            const uint32_t word = mine ? (key_of(v) & ~31u) | (31u - static_cast<uint32_t>(lane / seg)) : 0u;
            uint32_t left = word, last = 0;
            for (int r = 0; r < p.rc.topk_groups; ++r) {
                last = __reduce_max_sync(kFull, left);
                if (left == last) left = 0;
            }
            kept = mine && word >= last;
            const float a = of_key(last & ~31u), b = of_key(__reduce_max_sync(kFull, left) & ~31u);
            bad |= !(a - b > margin + 3.814697265625e-06f * fabsf(b));  // the cut, 2^-18
            mask = group_mask(kept);
        }
#pragma unroll
        for (int j = 0; j < N; ++j)
            k[j] = has(j) && in_group(j, kept, mask) ? (k[j] & ~kIdxMask) | (kIdxMask - static_cast<uint32_t>(expert(j)))
                                                     : 0u;
        sort_descending<N>(k);
        const uint32_t win = take<N, kFew ? kFewK + 1 : 0>(k, min(p.K + 1, kWarp), lane, slots);  // lane K: the runner-up
        const uint32_t runner = __shfl_sync(kFull, win, p.K & 31);
        int idx = win != 0u && lane < p.K ? static_cast<int>(kIdxMask - (win & kIdxMask)) : -1;
        float logit = idx >= 0 ? fminf(load_logit<kBf16>(p.logits, base + idx), lim) : 0.0f;
        float s = kMode == 1 && idx >= 0 ? sigmoid_exact(logit) : 0.0f;
        const float key = kMode == 1 ? (idx >= 0 && p.bias != nullptr ? s + __ldg(p.bias + idx) : s) : logit;
        if (idx >= 0 && runner != 0u) {
            const float reach = of_key(runner & ~kIdxMask);
            bad |= !(key - reach > fabsf(reach) * kCut + approx_error());
        }
        int slot = lane;
        if (__any_sync(kFull, bad)) {  // rounds over exact keys
            bool nan = false;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float l = has(j) ? load_logit<kBf16>(p.logits, base + expert(j)) : -INFINITY;
                const float v = kMode == 1 ? sigmoid_exact(fminf(l, lim)) + bias[j] : fminf(l, lim);
                nan |= l != l || v != v;
                k[j] = l > -lim && v > -INFINITY ? key_of(v) : kNone;
            }
            if (__any_sync(kFull, nan) && lane == 0) flag_error(p.status, EP_DEV_INPUT);
            if (groups) {
                uint32_t k1, k2;
                group_top2(k, k1, k2);
                const bool in =
                    group_kept(group_value(k1, k2, p.rc.group_top), p.rc.G, seg, p.rc.topk_groups, lane);
                const uint32_t exact_mask = group_mask(in);
#pragma unroll
                for (int j = 0; j < N; ++j) k[j] = in_group(j, in, exact_mask) ? k[j] : kNone;
            }
            idx = exact_rounds<N>(k, p.K, lane, expert);
            logit = idx >= 0 ? fminf(load_logit<kBf16>(p.logits, base + idx), lim) : 0.0f;
            s = kMode == 1 && idx >= 0 ? sigmoid_exact(logit) : 0.0f;
        } else {
            const uint32_t mine = idx >= 0 ? key_of(key) : kNone;
            const uint32_t after = __shfl_down_sync(kFull, mine, 1);
            const int idx_after = __shfl_down_sync(kFull, idx, 1);
            const bool swapped = lane + 1 < p.K && (mine < after || (mine == after && idx_after >= 0 && idx > idx_after));
            if (__any_sync(kFull, swapped)) {  // order the winners by their exact keys
                int rank = 0;
                for (int j = 0; j < p.K; ++j) {
                    const uint32_t other = __shfl_sync(kFull, mine, j);
                    const int other_idx = __shfl_sync(kFull, idx, j);
                    rank += other > mine || (other == mine && (idx < 0 ? j < lane : other_idx >= 0 && other_idx < idx));
                }
                slot = rank;
            }
        }
        float wt = s;
        if (kMode == 0) {
            if (p.rc.renorm) m = warp_max(idx >= 0 ? logit : -FLT_MAX);
            wt = idx >= 0 ? expf(logit - m) : 0.0f;
        }
        if (p.rc.renorm) total = sum_kept<kFew ? kFewK : 0>(wt);
        if (kMode == 0 || p.rc.renorm) wt = total > 0.0f ? wt / total : 0.0f;
        if (lane < p.K) out.put(slot, idx, wt * p.rc.scale);
    }
}

// ---- keys in shared memory: any number of experts, any score ----
//
// Lane i owns every 32nd expert from i on: it brings their logits in, turns them
// into keys and knows the best of them (of those in groups kept).  A round takes the best
// of all; the warp then finds its owner's next best together, from a column of
// the padded rows.  Bound by the instructions spent on every key.  55512 tokens x 1536
// fp32, softmax, 8 groups: 186 us (1.8 TB/s); 32768 x 1024 bf16: 73 us; 32768 x 256 fp32
// softmax with bias and sums of two: 67 us.
__device__ __forceinline__ int padded(int e) { return e + (e >> 5); }  // rows of 33 words: columns without bank conflicts

template <bool kBf16>
__global__ void __launch_bounds__(kRouteWarps* kWarp) route_kernel(const RouteArgs p, int seg) {
    extern __shared__ uint32_t s_keys[];
    constexpr int kNowhere = 0x7fffffff, kRow = kWarp + 1;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    uint32_t* keys = s_keys + static_cast<size_t>(warp) * (padded(p.E) + 1);
    const float lim = largest<kBf16>();
    griddep_launch_dependents();
    griddep_wait();  // the logits are complete from here on
    const bool softmax = p.rc.score == 0, groups = p.rc.topk_groups < p.rc.G;
    const int per_group = p.E / p.rc.G;
    const float to_group = 1.0f / per_group;
    // softmax keeps the logits' order, so where a key is one score the logit serves; the scores are needed where
    // they are keys, or weights as they are
    const bool by_logit = softmax && p.bias == nullptr && (p.rc.group_top == 1 || !groups);
    const bool statistics = softmax && !(by_logit && p.rc.renorm);
    const long long step = static_cast<long long>(gridDim.x) * kRouteWarps;
    for (long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + warp; t < p.tokens; t += step) {
        const long long base = t * p.E;
        bool nan = false;
        float m = -FLT_MAX, sum = 0.0f;
        uint32_t* at = keys + lane;  // the lane's column
#pragma unroll 8
        for (int e = lane; e < p.E; e += kWarp, at += kRow) {
            const float l = load_logit<kBf16>(p.logits, base + e);
            if (statistics && l > -lim) m = fmaxf(m, fminf(l, lim));
            *at = __float_as_uint(l);
        }
        if (statistics) {
            m = redux_max(m);
            at = keys + lane;
#pragma unroll 4
            for (int e = lane; e < p.E; e += kWarp, at += kRow) {
                const float l = __uint_as_float(*at);
                if (l > -lim) sum += expf(fminf(l, lim) - m);
            }
            sum = warp_sum(sum);
        }
        auto score = [&](float l) {
            l = fminf(l, lim);
            return softmax ? expf(l - m) / sum : sigmoid_exact(l);
        };
        uint32_t best = kNone;  // of the lane's experts, and where it is
        int best_at = kNowhere;
        auto key = [&](float l, int e) {
            uint32_t k = kNone;
            nan |= l != l;
            if (l > -lim) {
                float v = by_logit ? fminf(l, lim) : score(l);
                if (p.bias != nullptr) v += __ldg(p.bias + e);
                nan |= v != v;
                if (v > -INFINITY) k = key_of(v);
            }
            if (k > best) {
                best = k;
                best_at = e;
            }
            return k;
        };
        at = keys + lane;
#pragma unroll 4
        for (int e = lane; e < p.E; e += kWarp, at += kRow) *at = key(__uint_as_float(*at), e);
        if (__any_sync(kFull, nan) && lane == 0) flag_error(p.status, EP_DEV_INPUT);
        uint32_t kept = 0xffffffffu;  // groups
        if (groups) {
            // `seg` lanes scan each group
            __syncwarp();
            uint32_t k1 = kNone, k2 = kNone;
            const int g = lane / seg;
            if (g < p.rc.G)
#pragma unroll 4
                for (int e = g * per_group + lane % seg; e < (g + 1) * per_group; e += seg) {
                    const uint32_t v = keys[padded(e)];
                    k2 = max(k2, min(k1, v));
                    k1 = max(k1, v);
                }
            __syncwarp();
            segment_merge2(seg, k1, k2);
            const bool in = group_kept(group_value(k1, k2, p.rc.group_top), p.rc.G, seg, p.rc.topk_groups, lane);
            kept = __reduce_or_sync(kFull, in ? 1u << g : 0u);
            best = kNone;
            best_at = kNowhere;
            for (uint32_t left = kept; left != 0u; left &= left - 1u) {
                const int lo = (__ffs(left) - 1) * per_group;
#pragma unroll 4
                for (int e = lo + ((lane - lo) & (kWarp - 1)); e < lo + per_group; e += kWarp) {
                    const uint32_t k = keys[padded(e)];
                    if (k > best) {
                        best = k;
                        best_at = e;
                    }
                }
            }
        }
        __syncwarp();
        int idx = -1;  // lane k holds slot k
        for (int k = 0; k < p.K; ++k) {
            const uint32_t top = __reduce_max_sync(kFull, best);
            if (top == kNone) break;
            const int at = static_cast<int>(__reduce_min_sync(kFull, best == top ? best_at : kNowhere));
            if (lane == k) idx = at;
            if (lane == 0) keys[padded(at)] = kNone;
            __syncwarp();
            uint32_t next = kNone;
            int next_at = kNowhere;
            for (int e = at % kWarp + kWarp * lane; e < p.E; e += kWarp * kWarp) {
                const uint32_t v = keys[padded(e)];
                // (e + 1/2) / per_group is far enough from a whole number for fp32
                if (v > next && (kept >> static_cast<int>((e + 0.5f) * to_group) & 1u)) {
                    next = v;
                    next_at = e;
                }
            }
            const uint32_t most = __reduce_max_sync(kFull, next);
            next_at = static_cast<int>(__reduce_min_sync(kFull, next == most && most != kNone ? next_at : kNowhere));
            if (lane == at % kWarp) {
                best = most;
                best_at = next_at;
            }
            __syncwarp();
        }
        const float l = idx >= 0 ? load_logit<kBf16>(p.logits, base + idx) : 0.0f;
        float w = 0.0f;
        if (softmax && p.rc.renorm) {
            const float top = warp_max(idx >= 0 ? fminf(l, lim) : -FLT_MAX);
            w = idx >= 0 ? expf(fminf(l, lim) - top) : 0.0f;
        } else if (idx >= 0) {
            w = score(l);
        }
        if (p.rc.renorm) {
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

// ---- gradient ----
//
// With s the scores, w = scale s / sum_kept(s) where they are renormalised, else scale s,
// and g the weights' gradient:
//
//   ds_k = (scale g_k - sum_j scale g_j v_j) / sum_kept(s), v = s / sum_kept(s)   or   scale g_k
//   sigmoid:                dl_k = s_k (1 - s_k) ds_k, 0 for the other experts
//   sigmoid, renormalised:  that is v_k (1 - s_k) (scale g_k - sum_j scale g_j v_j)
//   softmax, renormalised:  dl_k = v_k (scale g_k - sum_j scale g_j v_j), 0 for the others
//   softmax over all:       dl_e = [e kept] s_e ds_e - s_e sum_k s_k ds_k: dense

// A slot's expert and its incoming gradient.
struct Slot {
    long long id;
    float g;
};
__device__ __forceinline__ Slot load_slot(const RouteBwdArgs& p, long long t, int lane) {
    Slot s = {-1, 0.0f};
    if (lane < p.K) {
        s.id = __ldg(p.topk_idx + t * p.K + lane);
        s.g = __ldg(p.grad_w + t * p.K + lane);
    }
    return s;
}
// The slot's expert, -1 for none.
__device__ __forceinline__ int slot_expert(const RouteBwdArgs& p, const Slot& s) {
    if (s.id >= 0 && s.id < p.E) return static_cast<int>(s.id);
    if (s.id != -1) flag_error(p.status, EP_DEV_INPUT);
    return -1;
}
// What a slot adds to its expert's logit gradient, and (dense) what every expert then loses
// s_e times.  `W` lanes have a token's slots; `m` and `inv` are the dense softmax's
// maximum and reciprocal sum.
struct SlotGrad {
    float own, dot;
};
template <bool kBf16, bool kDense, int W>
__device__ __forceinline__ SlotGrad slot_gradient(const RouteBwdArgs& p, float l, float grad, float m, float inv) {
    const bool softmax = kDense || p.rc.score == 0;
    const float hi = largest<kBf16>();
    SlotGrad r;
    const bool on = l > -hi;  // a masked expert's score is 0 and stays 0
    l = fminf(l, hi);
    const float g = on ? grad * p.rc.scale : 0.0f;
    if (kDense) {
        const float s = on ? expf(l - m) * inv : 0.0f;
        r.own = s * g;
        r.dot = warp_sum<W>(r.own);
        return r;
    }
    float s = 0.0f, rest = 1.0f;  // the kept score; sigmoid: 1 - s, as s exp(-l) where the difference would lose digits
    if (softmax) {
        const float top = warp_max<W>(on ? l : -FLT_MAX);
        if (on) s = expf(l - top);
    } else if (on) {
        const float e = expf(-l);
        s = 1.0f / (1.0f + e);
        rest = e < 1.0f ? s * e : 1.0f - s;
    }
    float v = s, c = g;  // what the slot's weight is of `scale`, and its gradient
    if (p.rc.renorm) {
        const float total = warp_sum<W>(s);
        v = total > 0.0f ? s / total : 0.0f;
        c -= warp_sum<W>(v * g);
    }
    // v, not c, is divided by the sum: with every kept sigmoid small, c over the sum is no fp32 number
    r.dot = 0.0f;
    r.own = softmax ? v * c : v * rest * c;
    return r;
}

template <bool kBf16>
__device__ __forceinline__ void store_grad(void* out, long long i, float d) {
    if (kBf16)
        static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(d);
    else
        static_cast<float*>(out)[i] = d;
}

// One token's dense gradient, any E, any logits, repeated experts added up in slot order.
template <bool kBf16>
__device__ __noinline__ void backward_token(const RouteBwdArgs& p, long long t, int lane) {
    const float hi = largest<kBf16>();
    const long long base = t * p.E;
    float m = -FLT_MAX, sum = 0.0f;
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
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const Slot slot = load_slot(p, t, lane);
    const int idx = slot_expert(p, slot);
    const float l = idx >= 0 ? load_logit<kBf16>(p.logits, base + idx) : -INFINITY;
    const SlotGrad g = slot_gradient<kBf16, true, kWarp>(p, l, slot.g, m, inv);
    for (int e0 = 0; e0 < p.E; e0 += kWarp) {
        const int e = e0 + lane;
        float d = 0.0f;
        if (e < p.E) {
            const float v = load_logit<kBf16>(p.logits, base + e);
            if (v > -hi) d = -expf(fminf(v, hi) - m) * inv * g.dot;
        }
        for (int k = 0; k < p.K; ++k) {
            const int ek = __shfl_sync(kFull, idx, k);
            const float gk = __shfl_sync(kFull, g.own, k);
            if (ek == e && ek >= 0) d += gk;
        }
        if (e < p.E) store_grad<kBf16>(p.grad_logits, base + e, d);
    }
}

// Zeros elements [lo, hi) of an array on a 16-byte boundary.
template <bool kBf16>
__device__ __forceinline__ void zero_elements(void* out, long long lo, long long hi, int lane) {
    constexpr int kVec = kBf16 ? 8 : 4;
    const long long a = (lo + kVec - 1) / kVec, b = hi / kVec;  // whole vectors
    if (a >= b) {
        for (long long i = lo + lane; i < hi; i += kWarp) store_grad<kBf16>(out, i, 0.0f);
        return;
    }
    for (long long i = a + lane; i < b; i += kWarp) static_cast<uint4*>(out)[i] = make_uint4(0, 0, 0, 0);
    if (lo + lane < a * kVec) store_grad<kBf16>(out, lo + lane, 0.0f);
    if (b * kVec + lane < hi) store_grad<kBf16>(out, b * kVec + lane, 0.0f);
}

// Gradients that are zero but for the slots' experts (sigmoid, and softmax over
// the kept experts): W >= K lanes to a token, so a warp has 32 / W tokens at
// once.  Their rows, one after another in memory, are zeroed as vectors and the
// slots' parts stored on top.  It waits for the gathered logits: 131072 tokens x 256, K = 8, bf16 25 us,
// fp32 41 us, where whole sectors of what it moves would take 17 and 27 (DRAM at 44 % of its peak; a
// warp stalls 8.8 cycles on loads for each instruction).  With a whole warp to each token, and its row
// put together in shared memory, bf16 took 66 us.
template <bool kBf16, int W>
__global__ void __launch_bounds__(kRouteWarps* kWarp) route_backward_sparse_kernel(const RouteBwdArgs p) {
    constexpr int kTokens = kWarp / W;
    const int lane = threadIdx.x % kWarp, sub = lane / W;
    griddep_launch_dependents();
    griddep_wait();  // the logits, ids and gradients are complete from here on
    const long long step = static_cast<long long>(gridDim.x) * kRouteWarps * kTokens;
    auto load = [&](long long t) {
        return t < p.tokens ? load_slot(p, t, lane % W) : Slot{-1, 0.0f};
    };
    auto logit = [&](long long t, int idx) {
        return idx >= 0 ? load_logit<kBf16>(p.logits, t * p.E + idx) : -INFINITY;
    };
    // a group's logits are fetched one group ahead, its slots two
    long long t0 = (static_cast<long long>(blockIdx.x) * kRouteWarps + threadIdx.x / kWarp) * kTokens;
    Slot now = load(t0 + sub), next = load(t0 + step + sub);
    int idx = slot_expert(p, now);
    float l = logit(t0 + sub, idx);
    for (; t0 < p.tokens; t0 += step) {
        const Slot after = load(t0 + 2 * step + sub);
        const int next_idx = slot_expert(p, next);
        const float next_l = logit(t0 + step + sub, next_idx);
        zero_elements<kBf16>(p.grad_logits, t0 * p.E, min(t0 + kTokens, p.tokens) * p.E, lane);
        float own = slot_gradient<kBf16, false, W>(p, l, now.g, 0.0f, 0.0f).own;
        // the token's slots with the same expert: the first one gets their sum, in slot order
        const uint32_t key = idx >= 0 ? static_cast<uint32_t>(idx) * kTokens + sub : 0x80000000u + lane;
        const uint32_t same = __match_any_sync(kFull, key);
        if (__any_sync(kFull, (same & (same - 1u)) != 0u)) {
            float sum = 0.0f;
            for (int j = 0; j < kWarp; ++j) {
                const float v = __shfl_sync(kFull, own, j);
                if (same >> j & 1u) sum += v;
            }
            own = sum;
        }
        __syncwarp();  // after the zeros
        if (idx >= 0 && (same & ((1u << lane) - 1u)) == 0u)
            store_grad<kBf16>(p.grad_logits, (t0 + sub) * p.E + idx, own);
        __syncwarp();
        now = next;
        next = after;
        idx = next_idx;
        l = next_l;
    }
}

template <bool kBf16>
__global__ void __launch_bounds__(kRouteWarps* kWarp) route_backward_kernel(const RouteBwdArgs p) {
    griddep_launch_dependents();
    griddep_wait();  // the logits, ids and gradients are complete from here on
    const long long step = static_cast<long long>(gridDim.x) * kRouteWarps;
    for (long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + threadIdx.x / kWarp; t < p.tokens; t += step)
        backward_token<kBf16>(p, t, threadIdx.x % kWarp);
}

// Dense gradients of up to 512 experts.  With kVec rows are whole 16-byte vectors: lane i holds the N
// experts from i * N on and reads and writes them as vectors; else it holds every
// 32nd expert from i on.  It finds its slots' parts in a shared row that is zero
// but for them.  Bound by the instructions of a token, most of them the same for half the bytes.  Rows are brought into L2 three tokens ahead,
// because the warps that fit hold too few bytes in flight.  The exponentials are expf: __expf takes 49 us for the
// fp32 rows below, but its product x log2(e) alone is off by 2^-19 at scores of exp(-60).  A token with unusual
// logits, or with an expert in two slots, goes through backward_token.  W lanes have a token.  131072 tokens x 256:
// fp32 54 us (5.2 TB/s, 78 % of the copy rate), bf16 51 us; kVec off costs 2 % and 16 %.
// route_backward_kernel takes 282 us for the fp32 ones.
template <bool kBf16, int N, bool kVec, int W>
__global__ void __launch_bounds__(kRouteWarps* kWarp) route_backward_lanes_kernel(const RouteBwdArgs p) {
    __shared__ alignas(16) float s_rows[kRouteWarps][kWarp * N];
    constexpr int kTokens = kWarp / W;
    const int lane = threadIdx.x % kWarp, sub = lane / W, at = lane % W, first = at * N;
    float* row = s_rows[threadIdx.x / kWarp] + sub * (W * N);
    auto expert = [&](int j) { return kVec ? first + j : at + W * j; };
    auto has = [&](int j) { return expert(kVec ? 0 : j) < p.E; };  // kVec: E is a multiple of N
#pragma unroll
    for (int j = 0; j < N; ++j) row[first + j] = 0.0f;
    __syncwarp();
    griddep_launch_dependents();
    griddep_wait();  // the logits, ids and gradients are complete from here on
    const long long step = static_cast<long long>(gridDim.x) * kRouteWarps * kTokens;
    long long t = (static_cast<long long>(blockIdx.x) * kRouteWarps + threadIdx.x / kWarp) * kTokens + sub;
    auto load = [&](long long token, float (&l)[N]) {
        if (kVec) {
            if (has(0)) load_lane<kBf16, N>(p.logits, token * p.E, first, p.E, true, l);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (has(j)) l[j] = load_logit<kBf16>(p.logits, token * p.E + expert(j));
        }
    };
    constexpr int kAhead = 3;
    auto prefetch_row = [&](long long token) {
        constexpr int kLine = kBf16 ? 64 : 32;  // logits of 128 bytes
        if (at * kLine < p.E)
            prefetch_l2(static_cast<const char*>(p.logits) + (token * p.E + at * kLine) * (kBf16 ? 2 : 4));
    };
    float next[N];
#pragma unroll
    for (int j = 0; j < N; ++j) next[j] = 0.0f;
    Slot ahead = {-1, 0.0f};
    if (t < p.tokens) {
        load(t, next);
        ahead = load_slot(p, t, at);
    }
    for (; t - sub < p.tokens; t += step) {
        const Slot slot = ahead;
        const int idx = slot_expert(p, slot);
        const float l = idx >= 0 ? load_logit<kBf16>(p.logits, t * p.E + idx) : -INFINITY;
        if (W < kWarp) ahead = Slot{-1, 0.0f};
        if (t + step < p.tokens) ahead = load_slot(p, t + step, at);
        if (idx >= 0) row[idx] = __int_as_float(lane);  // of two slots with one expert, one keeps its mark
        float d[N];
        float m = -FLT_MAX, sum = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            d[j] = next[j];
            if (has(j)) m = fmaxf(m, d[j]);
        }
        if (t + step < p.tokens) load(t + step, next);
        if (t + kAhead * step < p.tokens) prefetch_row(t + kAhead * step);
        m = W == kWarp ? redux_max(m) : warp_max<W>(m);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            d[j] = has(j) ? expf(d[j] - m) : 0.0f;
            sum += d[j];
        }
        const float hi = largest<kBf16>();
        const float g = l > -hi ? slot.g * p.rc.scale : 0.0f;  // a masked expert's score is 0 and stays 0
        const float e = l > -hi ? expf(l - m) : 0.0f;
        float dot = e * g;
        if (W == kWarp) {
            warp_sum2(sum, dot, lane);
        } else {
            sum = warp_sum<W>(sum);
            dot = warp_sum<W>(dot);
        }
        const float inv = 1.0f / sum;
        // masked logits came out as 0; infinite or NaN ones as NaN, and with all masked m tells
        const bool odd = !(sum > 0.0f) || m <= -hi;
        __syncwarp();
        const bool twice = idx >= 0 && __float_as_int(row[idx]) != lane;
        bool done = false;  // nothing left to store
        if (W == kWarp) {
            if (__any_sync(kFull, odd || twice)) {
                backward_token<kBf16>(p, t, lane);
                if (idx >= 0) row[idx] = 0.0f;
                __syncwarp();
                continue;
            }
        } else {
            const bool on = t < p.tokens;
            const uint32_t slow = __ballot_sync(kFull, on && (odd || twice));
            const uint32_t mine = ((1u << (W % kWarp)) - 1u) << (sub * W);  // the token's lanes
            done = !on || (slow & mine) != 0u;
            for (int k = 0; slow != 0u && k < kTokens; ++k)
                if (__shfl_sync(kFull, slow & mine, k * W) != 0u) backward_token<kBf16>(p, t - sub + k, lane);
        }
        if (idx >= 0) row[idx] = e * g * inv;
        __syncwarp();
        const float c = inv * (inv * dot);
#pragma unroll
        for (int j = 0; j < N; ++j) d[j] = fmaf(-d[j], c, row[expert(j)]);
        __syncwarp();
        if (idx >= 0) row[idx] = 0.0f;
        __syncwarp();
        if (done) continue;
        if (!kVec) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (has(j)) store_grad<kBf16>(p.grad_logits, t * p.E + expert(j), d[j]);
            continue;
        }
        if (!has(0)) continue;
        if (kBf16) {
            uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.grad_logits) + t * p.E + first);
#pragma unroll
            for (int i = 0; i < N / 8; ++i) {
                uint32_t v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(d[8 * i + 2 * j], d[8 * i + 2 * j + 1]);
                    v[j] = *reinterpret_cast<const uint32_t*>(&h);
                }
                out[i] = make_uint4(v[0], v[1], v[2], v[3]);
            }
        } else {
            float4* out = reinterpret_cast<float4*>(static_cast<float*>(p.grad_logits) + t * p.E + first);
#pragma unroll
            for (int i = 0; i < N / 4; ++i)
                out[i] = make_float4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
        }
    }
}

// One resident CTA of warps for each place on the SMs, or fewer.
template <typename P, typename... Args>
cudaError_t launch_tokens(void (*kernel)(P, Args...), const P& p, int sms, cudaStream_t stream, Args... args) {
    const long long want = (p.tokens + kRouteWarps - 1) / kRouteWarps;
    const int resident = max_blocks_per_sm(reinterpret_cast<const void*>(kernel), kRouteWarps * kWarp, 0);
    if (resident <= 0) return cudaErrorInvalidValue;
    const long long most = static_cast<long long>(sms) * resident;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kRouteWarps * kWarp), 0,
                      stream, 0, false, p, args...);
}

template <int N>
cudaError_t launch_bf16(const RouteArgs& p, int sms, cudaStream_t stream) {
    if (p.rc.score == 1)
        return p.K <= kFewK ? launch_tokens(route_bf16_kernel<N, true, true>, p, sms, stream)
                            : launch_tokens(route_bf16_kernel<N, false, true>, p, sms, stream);
    return p.K <= kFewK ? launch_tokens(route_bf16_kernel<N, true, false>, p, sms, stream)
                        : launch_tokens(route_bf16_kernel<N, false, false>, p, sms, stream);
}

template <bool kBf16, int kMode, int N>
cudaError_t launch_lists_n(const RouteArgs& p, int seg, int vec, bool any, int sms, cudaStream_t stream) {
    if (any)
        return p.K <= kFewK
                   ? launch_tokens(route_lists_kernel<kBf16, N, kMode, true, true>, p, sms, stream, seg, vec)
                   : launch_tokens(route_lists_kernel<kBf16, N, kMode, false, true>, p, sms, stream, seg, vec);
    return p.K <= kFewK ? launch_tokens(route_lists_kernel<kBf16, N, kMode, true, false>, p, sms, stream, seg, vec)
                        : launch_tokens(route_lists_kernel<kBf16, N, kMode, false, false>, p, sms, stream, seg, vec);
}

template <bool kBf16, int kMode>
cudaError_t launch_lists(int n, const RouteArgs& p, int seg, int vec, bool any, int sms, cudaStream_t stream) {
    switch (n) {
        case 2: return launch_lists_n<kBf16, kMode, 2>(p, seg, vec, any, sms, stream);
        case 4: return launch_lists_n<kBf16, kMode, 4>(p, seg, vec, any, sms, stream);
        case 8: return launch_lists_n<kBf16, kMode, 8>(p, seg, vec, any, sms, stream);
        case 12: return launch_lists_n<kBf16, kMode, 12>(p, seg, vec, any, sms, stream);
        default: return launch_lists_n<kBf16, kMode, 16>(p, seg, vec, any, sms, stream);
    }
}

template <bool kBf16>
cudaError_t launch_sparse(const RouteBwdArgs& p, int sms, cudaStream_t stream) {
    if (p.K <= 8) return launch_tokens(route_backward_sparse_kernel<kBf16, 8>, p, sms, stream);
    if (p.K <= 16) return launch_tokens(route_backward_sparse_kernel<kBf16, 16>, p, sms, stream);
    return launch_tokens(route_backward_sparse_kernel<kBf16, 32>, p, sms, stream);
}

template <bool kBf16>
cudaError_t launch_backward(const RouteBwdArgs& p, int sms, cudaStream_t stream) {
    constexpr int kFewest = kBf16 ? 8 : 4;  // a 16-byte vector
    const bool vec = p.E % kFewest == 0;
    if (p.E <= kFewest * kWarp) {
        // short rows: as few lanes to a token as hold them and its slots, and the warp has several tokens (131072
        // tokens x 64 bf16, K = 8: 18 us, 51 us with a warp to each; x 72, K = 12: 35 and 51 us)
        if (vec && p.E <= kFewest * 8 && p.K <= 8)
            return launch_tokens(route_backward_lanes_kernel<kBf16, kFewest, true, 8>, p, sms, stream);
        if (vec && p.E <= kFewest * 16 && p.K <= 16)
            return launch_tokens(route_backward_lanes_kernel<kBf16, kFewest, true, 16>, p, sms, stream);
        if (vec) return launch_tokens(route_backward_lanes_kernel<kBf16, kFewest, true, 32>, p, sms, stream);
        if (p.E <= 2 * kWarp) return launch_tokens(route_backward_lanes_kernel<kBf16, 2, false, 32>, p, sms, stream);
        return launch_tokens(route_backward_lanes_kernel<kBf16, kFewest, false, 32>, p, sms, stream);
    }
    if (p.E <= 8 * kWarp)
        return p.E % 8 == 0 ? launch_tokens(route_backward_lanes_kernel<kBf16, 8, true, 32>, p, sms, stream)
                            : launch_tokens(route_backward_lanes_kernel<kBf16, 8, false, 32>, p, sms, stream);
    return p.E % 16 == 0 ? launch_tokens(route_backward_lanes_kernel<kBf16, 16, true, 32>, p, sms, stream)
                         : launch_tokens(route_backward_lanes_kernel<kBf16, 16, false, 32>, p, sms, stream);
}

}  // namespace

cudaError_t launch_route(const Shape& sh, const RouteCfg& rc, const void* logits, bool bf16, const float* bias,
                         int64_t* topk_idx, float* topk_w, int32_t* status, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const RouteArgs p = {logits, bias, topk_idx, topk_w, status, static_cast<long long>(sh.R) * sh.T, sh.E, sh.K, rc};
    const bool by_logit = rc.score == 0 && bias == nullptr && (rc.group_top == 1 || rc.topk_groups == rc.G);
    // experts of a lane: twelve up to 384, unless only sixteen divide them into runs (131072 x 384 bf16 softmax: 53 us
    // with twelve, 84 us with sixteen; fp32 87 and 126 us).  The strided forms (kAny) of twelve and sixteen spill 40 to
    // 128 bytes a thread where groups or sigmoids need registers beside the lists.
    const bool twelve = sh.E <= 384 && (sh.E % 12 == 0 || sh.E % 16 != 0);
    const int n = sh.E <= 64 ? 2 : sh.E <= 128 ? 4 : sh.E <= 256 ? 8 : twelve ? 12 : 16;
    if (sh.E <= 512 && (rc.score == 1 || by_logit)) {
        const bool grouped = rc.topk_groups < rc.G;
        if (bf16 && bias == nullptr && !grouped && sh.E % n == 0) {
            switch (n) {
                case 12: return launch_bf16<12>(p, sms, stream);
                case 2: return launch_bf16<2>(p, sms, stream);
                case 4: return launch_bf16<4>(p, sms, stream);
                case 8: return launch_bf16<8>(p, sms, stream);
                default: return launch_bf16<16>(p, sms, stream);
            }
        }
        // Runs of experts in a lane (vector loads, groups by shuffles) where E and the groups fall on lanes, else
        // every 32nd expert and groups through shared memory: 32768 x 256 sigmoid keys in 8 groups take 26 us in
        // runs, 32 us the other way.
        const int per_group = sh.E / rc.G;
        int seg = per_group / n;
        bool any = sh.E % n != 0 || (grouped && (per_group % n != 0 || (seg & (seg - 1)) != 0));
        if (any)
            for (seg = kWarp; seg * rc.G > kWarp;) seg /= 2;
        const int vec = (static_cast<long long>(sh.E) * (bf16 ? 2 : 4)) % 16 == 0;
        return bf16 ? (rc.score == 0 ? launch_lists<true, 0>(n, p, seg, vec, any, sms, stream)
                                     : launch_lists<true, 1>(n, p, seg, vec, any, sms, stream))
                    : (rc.score == 0 ? launch_lists<false, 0>(n, p, seg, vec, any, sms, stream)
                                     : launch_lists<false, 1>(n, p, seg, vec, any, sms, stream));
    }
    int seg = kWarp;  // lanes that scan a group
    while (seg * rc.G > kWarp) seg /= 2;
    const long long want = (p.tokens + kRouteWarps - 1) / kRouteWarps;
    const long long most = sms * 16LL;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    const size_t smem = sizeof(uint32_t) * kRouteWarps * static_cast<size_t>(sh.E + sh.E / 32 + 1);
    return bf16 ? launch_pdl(route_kernel<true>, grid, dim3(kRouteWarps * kWarp), smem, stream, 0, false, p, seg)
                : launch_pdl(route_kernel<false>, grid, dim3(kRouteWarps * kWarp), smem, stream, 0, false, p, seg);
}

cudaError_t launch_route_backward(const Shape& sh, const RouteCfg& rc, const void* logits, bool bf16,
                                  const int64_t* topk_idx, const float* grad_topk_w, void* grad_logits,
                                  int32_t* status, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const RouteBwdArgs p = {logits, topk_idx, grad_topk_w, grad_logits, status, static_cast<long long>(sh.R) * sh.T,
                            sh.E, sh.K, rc};
    if (rc.score != 0 || rc.renorm)
        return bf16 ? launch_sparse<true>(p, sms, stream) : launch_sparse<false>(p, sms, stream);
    if (sh.E <= 512) return bf16 ? launch_backward<true>(p, sms, stream) : launch_backward<false>(p, sms, stream);
    return bf16 ? launch_tokens(route_backward_kernel<true>, p, sms, stream)
                : launch_tokens(route_backward_kernel<false>, p, sms, stream);
}

}  // namespace ep
