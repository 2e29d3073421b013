// Low-latency dispatch that casts its rows to int8 (ep_ll_dispatch_int8): a team
// of threads holds a token's row, finds its largest magnitude, casts it once and
// writes it to each of the token's slots.
//
//   scale = max(amax, 2^-100) * (1 / 127) over the row;  q = round(x / scale)
//
// The quotient is fp32's division; the one rounding to fewer bits is the int8
// value's.  Bound by HBM: a token is read once and written K times at half its
// width, 2 H + K H bytes.  A scale needs the whole row, so a row is one team's:
// 32 threads hold up to 2048 columns in registers, 128 up to 8192, and what is
// longer is read a second time for its cast.  The cast row goes through shared
// memory and from there to every slot by one bulk copy each (16-byte stores by every
// thread: 416 us where this takes 383).  2048 tokens x 7168 to 8 slots take 31 us, 32768 tokens
// 376 to 383 us (6.1 to 6.3 TB/s, 91 to 93 % of the copy rate).
#include <cstdint>
#include <cuda_runtime.h>

#include "ep.h"
#include "ep_device.cuh"
#include "ep_internal.h"
#include "int8_cast.cuh"

namespace ep {

namespace {

constexpr int kThreads = 128;
constexpr int kLaneCols = 16;  // columns of a thread's pass: 32 B in, 16 B out
constexpr int kPasses = 4;     // passes held in registers

struct Args {
    const uint16_t* x;
    const int64_t* topk_idx;
    const int32_t* slot_pos;
    int8_t* recv_x;
    float* recv_scales;
    int32_t* src_info;
    long long tokens;
    int T, K, E, H, cap;
};

struct Piece {
    uint4 v[2];  // 16 bf16
};

__device__ __forceinline__ Piece load(const uint16_t* row, int col, int H) {
    Piece r;
    r.v[0] = r.v[1] = make_uint4(0, 0, 0, 0);
    if (col < H) {
        r.v[0] = ld_nc_v4(row + col);
        r.v[1] = ld_nc_v4(row + col + 8);
    }
    return r;
}

// Largest magnitude as bits, both halves apart: larger bits are larger magnitudes, and NaN is above them all.
__device__ __forceinline__ uint32_t max_bits(uint32_t m, const Piece& p) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        m = __vmaxu2(m, p.v[i].x & 0x7fff7fffu);
        m = __vmaxu2(m, p.v[i].y & 0x7fff7fffu);
        m = __vmaxu2(m, p.v[i].z & 0x7fff7fffu);
        m = __vmaxu2(m, p.v[i].w & 0x7fff7fffu);
    }
    return m;
}

__device__ __forceinline__ uint4 cast(const Piece& p, float scale) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4& v = p.v[i / 2];
        const uint32_t a = i % 2 == 0 ? v.x : v.z, b = i % 2 == 0 ? v.y : v.w;
        q[i] = pack_int8x4(__uint_as_float(a << 16) / scale, __uint_as_float(a & 0xffff0000u) / scale,
                           __uint_as_float(b << 16) / scale, __uint_as_float(b & 0xffff0000u) / scale);
    }
    return make_uint4(q[0], q[1], q[2], q[3]);
}

template <int kTeam>
__global__ void __launch_bounds__(kThreads) ll_dispatch_int8_kernel(const Args p) {
    constexpr int kTeams = kThreads / kTeam, kWarps = kTeam / kWarp;
    constexpr int kHeld = kTeam * kLaneCols * kPasses;
    __shared__ uint32_t s_max[2][kWarps];
    __shared__ alignas(128) uint8_t s_row[kTeams][2][kHeld];  // the team's cast rows: two take turns
    const int team = threadIdx.x / kTeam, tid = threadIdx.x % kTeam, lane = threadIdx.x % kWarp;
    const auto sync = [] {
        if (kWarps == 1)
            __syncwarp();
        else
            __syncthreads();
    };
    griddep_launch_dependents();
    griddep_wait();  // x, the ids and the row map are complete from here on
    int turn = 0;
    for (long long t = static_cast<long long>(blockIdx.x) * kTeams + team; t < p.tokens;
         t += static_cast<long long>(gridDim.x) * kTeams, turn ^= 1) {
        const uint16_t* x = p.x + t * p.H;
        Piece held[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) held[i] = load(x, (i * kTeam + tid) * kLaneCols, p.H);
        long long row = -1;  // lane k holds slot k's row
        if (lane < p.K) {
            const long long e = __ldg(p.topk_idx + t * p.K + lane);
            const int pos = __ldg(p.slot_pos + t * p.K + lane);
            if (e >= 0 && e < p.E && pos >= 0 && pos < p.cap) row = e * p.cap + pos;
        }
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) m = max_bits(m, held[i]);
        for (int col = kHeld + tid * kLaneCols; col < p.H; col += kTeam * kLaneCols) m = max_bits(m, load(x, col, p.H));
        m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
        // the copies out of this buffer, of the token before the last one, have read it
        if (tid < kWarp) bulk_wait_read<1>();
        // two places take turns: passing this token's barrier says that the last one's maxima have been read
        if (kWarps > 1 && lane == 0) s_max[turn][tid / kWarp] = m;
        sync();
        if (kWarps > 1) {
#pragma unroll
            for (int i = 0; i < kWarps; ++i) m = max(m, s_max[turn][i]);
        }
        const float scale = row_scale(__uint_as_float(m << 16));
        const bool finite = m < 0x7f80u;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        uint8_t* out = s_row[team][turn];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int col = (i * kTeam + tid) * kLaneCols;
            if (col < p.H) *reinterpret_cast<uint4*>(out + col) = finite ? cast(held[i], scale) : zero;
        }
        fence_proxy_async_smem();
        sync();
        if (tid < kWarp) {
            if (row >= 0) bulk_s2g(p.recv_x + row * p.H, out, min(p.H, kHeld));
            bulk_commit();
        }
        for (int col = kHeld + tid * kLaneCols; col - tid * kLaneCols < p.H; col += kTeam * kLaneCols) {
            const uint4 more = finite ? cast(load(x, col, p.H), scale) : zero;
            for (int k = 0; k < p.K; ++k) {
                const long long r = __shfl_sync(0xffffffffu, row, k);
                if (r >= 0 && col < p.H) st_v4(p.recv_x + r * p.H + col, more);
            }
        }
        if (tid < kWarp && row >= 0) {
            p.recv_scales[row] = scale;
            if (p.src_info != nullptr)
                reinterpret_cast<int2*>(p.src_info)[row] = make_int2(static_cast<int>(t / p.T), static_cast<int>(t % p.T));
        }
    }
    if (tid < kWarp) bulk_wait_all();
}

template <int kTeam>
cudaError_t launch(const Args& p, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const long long want = (p.tokens + kThreads / kTeam - 1) / (kThreads / kTeam), most = sms * 8LL;
    return launch_pdl(ll_dispatch_int8_kernel<kTeam>, dim3(static_cast<unsigned>(want < most ? want : most)),
                      dim3(kThreads), 0, stream, 0, true, p);
}

}  // namespace

cudaError_t launch_ll_dispatch_int8(const Shape& sh, const uint16_t* x, const int64_t* topk_idx,
                                    const int32_t* slot_pos, int cap, int8_t* recv_x, float* recv_x_scales,
                                    int32_t* recv_src_info, int32_t* status, cudaStream_t stream) {
    (void)status;  // nothing of this call can fail on the device
    const Args p = {x, topk_idx, slot_pos, recv_x, recv_x_scales, recv_src_info, static_cast<long long>(sh.R) * sh.T,
                    sh.T, sh.K, sh.E, sh.H, cap};
    return sh.H <= kWarp * kLaneCols * kPasses ? launch<kWarp>(p, stream) : launch<kThreads>(p, stream);
}

}  // namespace ep
