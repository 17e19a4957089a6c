// Multi-head scan, one token of every request: S <- a·S + (Δ·x) ⊗ B, y = (S·C + D·x)·silu(z), with
// the width-4 convolution and SiLU before it and the window's shift, in one launch.
//
// What bounds it is the state, read and written once (8·H·P·N bytes a request).  A CTA has a few
// rows of one head's state; its warps issue the state's loads first, convolve the CTA's x rows and
// the group's B and C (into shared memory) while those are in flight, then update and reduce in
// registers.  The heads of a group all read its B and C windows; the last of them shifts those.
// bf16, 61 requests of 64 heads of 64 x 128 states: 48 us, 5.5 TB/s (38.8 us at the copy rate); 256 of 80 heads of
// 64 x 64: 123 us (105), in fp32 with 8 groups 125 (107); 488 of 64 heads of 64 x 16, where the convolution's work per
// byte is largest, 75 (47).  Other state counts take 4-byte accesses: 64 heads of 64 x 24, 305 requests: 134 us (41); x 96,
// 81 requests: 116 (39); x 256, 30 requests: 65 (38).  One request of 24 heads: 4.6 us, the launch and one dependent
// chain of loads.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/selscan.h"
#include "heads_device.cuh"
#include "heads_params.h"
#include "heads_tc.h"
#include "internal.h"

namespace selscan {
namespace {

// One token of request b as a sequence.
__device__ __forceinline__ HeadsSeq step_seq(const HeadsParams& p, int b) {
    HeadsSeq s;
    s.slot = p.slots ? p.slots[b] : b;
    s.ok = s.slot < p.n_slots;
    s.row0 = b;
    s.len = 1;
    s.warm = s.slot >= 0;
    return s;
}

// LPR lanes share a row of the state, each with NV runs of W adjacent states (W = 4: 16-byte
// accesses, N = 4·LPR·NV; W = 1: any N up to 32·NV); a warp takes RPI = 32/LPR rows at once, U times.
template <typename TIO, int LPR, int NV, int W, int U, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, W == 4 ? 32 / WARPS : 1) heads_step_kernel(const HeadsParams p) {
    constexpr int RPI = 32 / LPR, RW = RPI * U, RC = RW * WARPS, NP = LPR * NV * W, kStepThreads = 32 * WARPS;
    __shared__ float sB[NP], sC[NP], sx[RC];
    __shared__ int last_reader;
    const int tiles = (p.P + RC - 1) / RC;
    int id = blockIdx.x;
    const int pt = id % tiles;
    id /= tiles;
    const int h = id % p.H, b = id / p.H;
    const HeadsSeq s = step_seq(p, b);
    if (!s.ok) {
        if (h == 0 && pt == 0 && threadIdx.x == 0 && p.err) atomicOr(p.err, kErrIndex);
        return;
    }
    const int g = h / (p.H / p.G), warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int p0 = pt * RC, np = min(RC, p.P - p0);
    const int cx = h * p.P + p0, cb = p.H * p.P + g * p.N, cc = cb + p.G * p.N;
    const int lr = lane % LPR, rr = lane / LPR;
    float* Sg = p.state + ((static_cast<int64_t>(max(s.slot, 0)) * p.H + h) * p.P + p0) * p.N;

    const int N = W == 4 ? NP : p.N;                                   // (whole rows of 16-byte runs)
    float* mine = Sg + static_cast<int64_t>(warp * RW + rr) * N + lr * W;
    float S[U][NV][W];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int row = warp * RW + u * RPI + rr;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int n = (j * LPR + lr) * W;
            const bool on = s.warm && row < np && n < N;
            const float* q = mine + u * RPI * N + j * LPR * W;
            if constexpr (W == 4) {
                const float4 v = on ? __ldcs(reinterpret_cast<const float4*>(q)) : make_float4(0.f, 0.f, 0.f, 0.f);
                S[u][j][0] = v.x; S[u][j][1] = v.y; S[u][j][2] = v.z; S[u][j][3] = v.w;
            } else {
                S[u][j][0] = on ? __ldcs(q) : 0.f;
            }
        }
    }
    for (int i = threadIdx.x; i < RC + 2 * NP; i += kStepThreads) {
        float* dst = i < RC ? &sx[i] : i < RC + NP ? &sB[i - RC] : &sC[i - RC - NP];
        const int k = i < RC ? i : (i - RC) % NP;
        const bool on = i < RC ? k < np : k < p.N;
        float v = 0.f;
        if (on) {
            const int c = i < RC ? cx + k : i < RC + NP ? cb + k : cc + k;
            const float* w = p.conv_w + static_cast<int64_t>(c) * 4;
            const float wk[4] = {w[0], w[1], w[2], w[3]}, bb = p.conv_b ? p.conv_b[c] : 0.f;
            const HeadsWindow win = heads_window(p, s, c);
            const float e = heads_sample<TIO>(p, s, win, c, 0);
            v = heads_conv(wk, bb, win.v[0], win.v[1], win.v[2], e);
            if (i < RC && s.slot >= 0) {           // an x channel: this CTA alone has its window
                float* q = p.window + (static_cast<int64_t>(s.slot) * p.C + c) * 3;
                q[0] = win.v[1];
                q[1] = win.v[2];
                q[2] = e;
            }
        }
        *dst = v;
    }
    const float dt = softplus(to_f32<TIO>(static_cast<const TIO*>(p.dt_raw)[s.row0 * p.dt_t + h]) +
                              (p.dt_bias ? p.dt_bias[h] : 0.f));
    const float a = ex2(dt * (-expf(p.A_log[h]) * kLog2e)), Dh = p.D ? p.D[h] : 0.f;
    __syncthreads();
    // the windows are read: said before the state's stores, which it would wait for, and looked at after them
    unsigned int* counter = p.arrivals + static_cast<int64_t>(b) * p.G + g;
    unsigned int said = 0u;
    if (s.slot >= 0 && threadIdx.x == kStepThreads - 1) said = heads_say_read(counter);
    float B[NV][W], C[NV][W];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < W; ++i) {
            B[j][i] = sB[(j * LPR + lr) * W + i];
            C[j][i] = sC[(j * LPR + lr) * W + i];
        }
    float acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int row = warp * RW + u * RPI + rr;
        const float dx = dt * sx[row];
        acc[u] = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                S[u][j][i] = fmaf(a, S[u][j][i], dx * B[j][i]);
                acc[u] = fmaf(S[u][j][i], C[j][i], acc[u]);
            }
        if (s.slot >= 0 && row < np)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int n = (j * LPR + lr) * W;
                if (n < N) {
                    float* q = mine + u * RPI * N + j * LPR * W;
                    if constexpr (W == 4)
                        __stcs(reinterpret_cast<float4*>(q), make_float4(S[u][j][0], S[u][j][1], S[u][j][2], S[u][j][3]));
                    else
                        __stcs(q, S[u][j][0]);
                }
            }
    }
    // sums over the lanes of a row: at each exchange a lane keeps half of its rows, so that the outputs of
    // the warp's rows end up in different lanes
    constexpr int kLeft = U > LPR ? U / LPR : 1, kSame = LPR > U ? LPR / U : 1;      // rows per lane; lanes with the same row
    int cnt = U, at = 0;
#pragma unroll
    for (int o = LPR / 2; o > 0; o /= 2) {
        if (cnt > 1) {
            cnt /= 2;
            const bool up = lr & o;
#pragma unroll
            for (int i = 0; i < U / 2; ++i)
                if (i < cnt) {
                    const float give = up ? acc[i] : acc[i + cnt];
                    acc[i] = (up ? acc[i + cnt] : acc[i]) + __shfl_xor_sync(0xffffffffu, give, o);
                }
            at += up ? cnt : 0;
        } else {
            acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
        }
    }
    if (lr % kSame == 0)
#pragma unroll
        for (int i = 0; i < kLeft; ++i) {
            const int row = warp * RW + (at + i) * RPI + rr;
            if (row < np) {
                const int c = cx + row;
                float v = fmaf(Dh, sx[row], acc[i]);
                if (p.z) v *= silu(to_f32<TIO>(static_cast<const TIO*>(p.z)[s.row0 * p.z_t + c]));
                static_cast<TIO*>(p.y)[s.row0 * p.y_t + c] = from_f32<TIO>(v);
            }
        }
    if (s.slot < 0) return;
    if (threadIdx.x == kStepThreads - 1) {
        last_reader = said == static_cast<unsigned int>((p.H / p.G) * tiles) - 1u;
        if (last_reader) *counter = 0u;
    }
    __syncthreads();
    if (last_reader)
        for (int k = threadIdx.x; k < 2 * p.N; k += kStepThreads)
            heads_keep_window<TIO>(p, s, k < p.N ? cb + k : cc + k - p.N);
}

template <typename TIO, int LPR, int NV, int W, int U, int WARPS>
cudaError_t launch_one(const HeadsParams& p, cudaStream_t stream) {
    constexpr int RC = (32 / LPR) * U * WARPS;
    const int64_t blocks = static_cast<int64_t>(p.n_seq) * p.H * ((p.P + RC - 1) / RC);
    heads_step_kernel<TIO, LPR, NV, W, U, WARPS><<<static_cast<unsigned>(blocks), 32 * WARPS, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename TIO>
cudaError_t launch_step_heads(const HeadsParams& p, cudaStream_t stream) {
    const bool vec = host::is_aligned(p.state, 16);
    // a CTA's convolution of the group's B and C is shared by its rows, so it has 64 of them, unless that
    // makes fewer CTAs than two to an SM: then 8 or 16
    const bool few = static_cast<int64_t>(p.n_seq) * p.H * ((p.P + 63) / 64) < 2 * heads_sm_count();
    if (vec && p.N == 128)
        return few ? launch_one<TIO, 32, 1, 4, 2, 4>(p, stream) : launch_one<TIO, 32, 1, 4, 8, 8>(p, stream);
    if (vec && p.N == 64)
        return few ? launch_one<TIO, 16, 1, 4, 2, 4>(p, stream) : launch_one<TIO, 16, 1, 4, 8, 4>(p, stream);
    if (vec && p.N == 32) return launch_one<TIO, 8, 1, 4, 4, 4>(p, stream);
    if (vec && p.N == 16) return launch_one<TIO, 4, 1, 4, 2, 4>(p, stream);
    if (p.N <= 64) return launch_one<TIO, 32, 2, 1, 8, 4>(p, stream);
    return launch_one<TIO, 32, 8, 1, 4, 4>(p, stream);
}

}  // namespace
}  // namespace selscan

using namespace selscan;
using namespace selscan::host;

extern "C" size_t ss_heads_step_workspace_size(int64_t batch, int64_t G) {
    return (batch <= 0 || G <= 0 || batch > INT32_MAX || G > (1 << 20)) ? 0 : heads_counter_bytes(batch, G);
}

extern "C" ss_status ss_heads_step(float* state, float* window, const void* xbc, const void* dt_raw, const void* z,
                                   const float* conv_w, const float* conv_b, const float* dt_bias, const float* A_log,
                                   const float* D, void* y, const int32_t* slots, int64_t batch, int64_t H, int64_t P,
                                   int64_t G, int64_t N, int64_t n_slots, const ss_heads_strides* strides, void* workspace,
                                   size_t workspace_bytes, void* stream_ptr) {
    HeadsParams p;
    bool bf16 = false, idle = false;
    const ss_status st = heads_check(p, strides, xbc, dt_raw, z, conv_w, conv_b, dt_bias, A_log, D, y, state, window,
                                     nullptr, slots, nullptr, batch, batch, H, P, G, N, n_slots, workspace,
                                     workspace_bytes, ss_heads_step_workspace_size(batch, G), &bf16, &idle);
    if (st != SS_OK || idle) return st;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    cudaError_t e = heads_counters(p, workspace, stream);
    if (e == cudaSuccess) e = bf16 ? launch_step_heads<__nv_bfloat16>(p, stream) : launch_step_heads<float>(p, stream);
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}
