// Backward of the causal depthwise conv1d + SiLU (ss_conv1d.cu).  With e = window ++ x and
// v_t = bias + Σ_k w_k e_{t+k}:
//   g_t = dout_t · silu'(v_t),  silu'(v) = σ(v) (1 + v (1 - σ(v)))      (g_t = dout_t without SiLU)
//   de_j = Σ_k w_k g_{j-k}  (dx_t = de_{t+3}; de_0..2 is the window's gradient),
//   dw_k = Σ_{b,t} g_t e_{t+k},  dbias = Σ_{b,t} g_t
//
// A stream of three elements per step and channel: what counts is how much of it is on its way.  A thread has 2
// channels (a packed pair) and a segment of steps; TMA brings the steps into a ring in shared memory (four stages of
// 8 KB a CTA, 6 CTAs an SM).  4 x 8192 x 5120 bf16: 175 us, 5.8 TB/s, 0.85 of the copy rate (3 stages and 8 CTAs 177, 6 and 4
// 173; loads into registers, the next steps' ahead, 315); 8 x 2048 x 1536 fp32: 56 us, 0.80; 45 steps: 6 us and 3 for the sums.
// It runs three steps past its segment, whose g belong to its last outputs.  The weight's gradients are sums in
// registers; every thread leaves its own in the workspace (a row of it per segment) and a second kernel adds the
// rows up in the same order every time.  Layouts that TMA does not take (rows or bases off 16 bytes) go by plain loads of
// single elements: 4 x 8192 x 5119 bf16 437 us, 0.34 of the copy rate; 5120 with x one element off 340; 8 x 2048 x 1535 fp32
// 65 us, 0.69.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/selscan.h"
#include "chained.cuh"
#include "column_sum.h"
#include "device_common.cuh"
#include "host_util.h"
#include "internal.h"

namespace selscan {
namespace {

constexpr int kConvK = SS_CONV_WIDTH;   // 4
constexpr int kSegMin = 8;
constexpr int kThreads = 128;
constexpr int kBlockChannels = 2 * kThreads;
constexpr int kBlocksPerSm = 6;
constexpr int kStages = 4;
template <typename T> constexpr int kSteps = 16 / sizeof(T);          // steps of a stage: 4 KB of x and of dout

struct ConvBwdParams {
    const void* dout;
    const void* x;
    const float* w;         // [Dm, 4]
    const float* bias;      // [Dm] or nullptr
    const float* win_in;    // [batch, Dm, 3] or nullptr
    const float* dwin_out;  // the same
    void* dx;
    float* dwin_in;         // or nullptr
    float* part;            // [batch · segs][ld]: dw [Dm, 4], then dbias [Dm]
    int64_t do_b, do_l, x_b, x_l, dx_b, dx_l, ld;
    int L, Dm, seg, nbd;
    unsigned int* err;
};
struct ConvBwdMaps {
    CUtensorMap x, dout;    // [batch, L, Dm], boxes of kSteps by kBlockChannels
};

__device__ __forceinline__ float2 load2(const float* q) { return *reinterpret_cast<const float2*>(q); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16* q) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(q);
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ void store2(float* q, float2 v) { __stcs(reinterpret_cast<float2*>(q), v); }
__device__ __forceinline__ void store2(__nv_bfloat16* q, float2 v) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    __stcs(reinterpret_cast<uint32_t*>(q), *reinterpret_cast<const uint32_t*>(&h));
}

__device__ __forceinline__ float2 silu_slope(float2 v) {
    const float2 s = rcp2(add2(splat2(1.f), ex2x2(mul2(v, splat2(-kLog2e)))));
    return mul2(s, fma2(v, fma2(s, splat2(-1.f), splat2(1.f)), splat2(1.f)));
}

// A thread's place: two channels (adjacent ones, or kThreads apart, so that a warp's are adjacent) and a segment.
struct Place {
    int seg, b, d0, d1, t0, t1, end;               // end: behind the steps whose g reach the segment's outputs
    bool one, two;                                 // channels that there are
};
__device__ __forceinline__ Place place_of(const ConvBwdParams& p, bool adjacent) {
    Place q;
    q.seg = static_cast<int>(blockIdx.x) / p.nbd;
    q.b = blockIdx.y;
    q.d0 = (static_cast<int>(blockIdx.x) - q.seg * p.nbd) * kBlockChannels + (adjacent ? 2 : 1) * static_cast<int>(threadIdx.x);
    q.d1 = q.d0 + (adjacent ? 1 : kThreads);
    q.one = q.d0 < p.Dm;
    q.two = q.d1 < p.Dm;
    q.t0 = q.seg * p.seg;
    q.t1 = min(q.t0 + p.seg, p.L);
    q.end = q.t1 + 3;
    return q;
}

// What a thread carries from step to step.
template <typename T, bool SILU> struct Pair {
    float2 w[kConvK], bs, e[3], g[3], dw[kConvK], db;      // e: the three samples before, g: of the three steps before
    template <typename F> static __device__ __forceinline__ float2 each(const Place& q, F&& f) {
        return make_float2(q.one ? f(q.d0) : 0.f, q.two ? f(q.d1) : 0.f);
    }
    static __device__ __forceinline__ float2 window(const ConvBwdParams& p, const Place& q, const float* w, int k) {
        return each(q, [&](int d) { return w[(static_cast<int64_t>(q.b) * p.Dm + d) * 3 + k]; });
    }
    __device__ __forceinline__ void start(const ConvBwdParams& p, const Place& q) {
#pragma unroll
        for (int k = 0; k < kConvK; ++k) {
            w[k] = each(q, [&](int d) { return p.w[static_cast<int64_t>(d) * kConvK + k]; });
            dw[k] = splat2(0.f);
        }
        bs = each(q, [&](int d) { return p.bias ? p.bias[d] : 0.f; });
        db = splat2(0.f);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const int t = q.t0 - 3 + j;
            e[j] = g[j] = splat2(0.f);
            if (t >= 0) e[j] = each(q, [&](int d) { return to_f32<T>(static_cast<const T*>(p.x)[q.b * p.x_b + t * p.x_l + d]); });
            else if (p.win_in) e[j] = window(p, q, p.win_in, 3 + t);
        }
    }
    // Step t: g_t (live: of a step that there is), its part in the weight's gradients (own: of the segment), and de
    // of three steps before.
    __device__ __forceinline__ float2 step(float2 xv, float2 gt, bool own, bool live) {
        if constexpr (SILU) gt = mul2(gt, silu_slope(fma2(w[3], xv, fma2(w[2], e[2], fma2(w[1], e[1], fma2(w[0], e[0], bs))))));
        if (!live) gt = splat2(0.f);
        if (own) {
            dw[0] = fma2(gt, e[0], dw[0]);
            dw[1] = fma2(gt, e[1], dw[1]);
            dw[2] = fma2(gt, e[2], dw[2]);
            dw[3] = fma2(gt, xv, dw[3]);
            db = add2(db, gt);
        }
        const float2 de = fma2(w[0], gt, fma2(w[1], g[2], fma2(w[2], g[1], mul2(w[3], g[0]))));
        g[0] = g[1];
        g[1] = g[2];
        g[2] = gt;
        e[0] = e[1];
        e[1] = e[2];
        e[2] = xv;
        return de;
    }
    // The same at a segment's ends: returns whether de is a step's of the segment; the window's goes where it belongs.
    __device__ __forceinline__ bool end_step(const ConvBwdParams& p, const Place& q, int t, float2 xv, float2 gt, float2* de) {
        *de = step(xv, gt, t < q.t1, t < p.L);
        const int j = t - 3;                       // the step (below 0: the window's entry) that de belongs to
        if (p.dwin_out && j >= p.L - 3) *de = add2(*de, window(p, q, p.dwin_out, j - (p.L - 3)));
        if (j >= q.t0) return true;
        if (j < 0 && p.dwin_in) {
            float* o = p.dwin_in + static_cast<int64_t>(q.b) * p.Dm * 3 + 3 + j;
            if (q.one) o[static_cast<int64_t>(q.d0) * 3] = de->x;
            if (q.two) o[static_cast<int64_t>(q.d1) * 3] = de->y;
        }
        return false;
    }
    __device__ __forceinline__ void leave(const ConvBwdParams& p, const Place& q) const {
        float* mine = p.part + (static_cast<int64_t>(q.b) * (gridDim.x / p.nbd) + q.seg) * p.ld;
        if (q.one) {
            *reinterpret_cast<float4*>(mine + 4 * static_cast<int64_t>(q.d0)) = make_float4(dw[0].x, dw[1].x, dw[2].x, dw[3].x);
            mine[4 * static_cast<int64_t>(p.Dm) + q.d0] = db.x;
        }
        if (q.two) {
            *reinterpret_cast<float4*>(mine + 4 * static_cast<int64_t>(q.d1)) = make_float4(dw[0].y, dw[1].y, dw[2].y, dw[3].y);
            mine[4 * static_cast<int64_t>(p.Dm) + q.d1] = db.y;
        }
    }
};

template <typename T, bool SILU>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) ss_conv1d_bwd_kernel(const ConvBwdParams p, const __grid_constant__ ConvBwdMaps m) {
    constexpr int U = kSteps<T>, kTile = U * kBlockChannels;
    __shared__ __align__(128) T tile[kStages][2][kTile];
    __shared__ uint64_t full[kStages];
    __shared__ int abort_flag;
    let_next_start();                              // (the sums' kernel: it waits for this one's end)
    const Place q = place_of(p, true);
    const int tid = threadIdx.x, c0 = q.d0 - 2 * tid, n = (q.end - q.t0 + U - 1) / U;
    auto issue = [&](int i) {                      // (steps and channels outside the tensor are zeros)
        const int s = i % kStages;
        mbar_expect_tx(&full[s], 2 * kTile * sizeof(T));
        tma_load_3d(tile[s][0], &m.x, &full[s], c0, q.t0 + i * U, q.b);
        tma_load_3d(tile[s][1], &m.dout, &full[s], c0, q.t0 + i * U, q.b);
    };
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
        abort_flag = 0;
        mbar_fence_init();
        for (int i = 0; i < min(n, kStages); ++i) issue(i);
    }
    Pair<T, SILU> c;
    c.start(p, q);
    __syncthreads();
    T* out = static_cast<T*>(p.dx) + q.b * p.dx_b + q.t0 * p.dx_l + q.d0;
    for (int i = 0; i < n; ++i) {
        const int s = i % kStages, tb = q.t0 + i * U;
        const bool ok = mbar_wait_bounded(&full[s], (i / kStages) & 1, &abort_flag, p.err);
        const T* xs = tile[s][0] + 2 * tid;
        const T* ds = tile[s][1] + 2 * tid;
        if (tb >= q.t0 + 3 && tb + U <= q.t1) {    // steps inside the segment, as all but its ends are
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float2 de = c.step(load2(xs + u * kBlockChannels), load2(ds + u * kBlockChannels), true, true);
                if (q.one) store2(out, de);
                out += p.dx_l;
            }
        } else {
            for (int u = 0; u < U && tb + u < q.end; ++u) {
                float2 de;
                if (c.end_step(p, q, tb + u, load2(xs + u * kBlockChannels), load2(ds + u * kBlockChannels), &de)) {
                    if (q.one) store2(out, de);
                    out += p.dx_l;
                }
            }
        }
        if (__syncthreads_or(!ok)) {               // a wait that ran out: copies in flight are over long before this
            for (int k = 0; k < 20; ++k) __nanosleep(1000000);
            break;
        }
        if (tid == 0 && i + kStages < n) issue(i + kStages);
    }
    c.leave(p, q);
}

template <typename T, bool SILU>
__global__ void __launch_bounds__(kThreads) ss_conv1d_bwd_plain_kernel(const ConvBwdParams p) {
    constexpr int U = 4;                           // steps whose loads are issued together
    let_next_start();
    const Place q = place_of(p, false);
    if (!q.one) return;                            // (an ended thread lets the next kernel start as well)
    Pair<T, SILU> c;
    c.start(p, q);
    const T* x = static_cast<const T*>(p.x) + q.b * p.x_b + q.t0 * p.x_l + q.d0;
    const T* dout = static_cast<const T*>(p.dout) + q.b * p.do_b + q.t0 * p.do_l + q.d0;
    T* out = static_cast<T*>(p.dx) + q.b * p.dx_b + q.t0 * p.dx_l + q.d0;
    for (int tb = q.t0; tb < q.end; tb += U) {
        T xs[U][2], ds[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool ok = tb + u < min(q.end, p.L);
            xs[u][0] = ok ? x[0] : from_f32<T>(0.f);
            xs[u][1] = ok && q.two ? x[kThreads] : from_f32<T>(0.f);
            ds[u][0] = ok ? dout[0] : from_f32<T>(0.f);
            ds[u][1] = ok && q.two ? dout[kThreads] : from_f32<T>(0.f);
            x += p.x_l;
            dout += p.do_l;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (tb + u >= q.end) break;
            float2 de;
            if (c.end_step(p, q, tb + u, make_float2(to_f32<T>(xs[u][0]), to_f32<T>(xs[u][1])),
                           make_float2(to_f32<T>(ds[u][0]), to_f32<T>(ds[u][1])), &de)) {
                out[0] = from_f32<T>(de.x);
                if (q.two) out[kThreads] = from_f32<T>(de.y);
                out += p.dx_l;
            }
        }
    }
    c.leave(p, q);
}

// Steps per thread for batch · ceil(L / seg) · nbd blocks when `slots` are resident at once: the length whose
// waves take the least time, a block taking seg + kSetup steps' worth (the three steps past its end, the
// weights, and the sums' way out).  For a number of waves the most segments that fit are the best, so only those are
// looked at (looking at every number of segments took 27 us of the host's time for 32768 steps of 768 channels).
constexpr int kSetup = 10, kMoreWaves = 8;
int segment_steps(int64_t batch, int64_t L, int64_t nbd, int64_t slots) {
    const int64_t per = batch * nbd, first = (per + slots - 1) / slots;
    int64_t best = L, best_cost = -1;
    for (int64_t waves = first; waves < first + kMoreWaves; ++waves) {
        const int64_t segs = std::min(waves * slots / per, std::max<int64_t>(L / kSegMin, 1));
        const int64_t seg = (L + segs - 1) / segs, blocks = per * ((L + seg - 1) / seg);
        const int64_t cost = (blocks + slots - 1) / slots * (seg + kSetup);
        if (best_cost < 0 || cost < best_cost) {
            best_cost = cost;
            best = seg;
        }
    }
    return static_cast<int>(best);
}

// The slots that the plan counts with: fixed, so that the workspace's size does not depend on the kernel.
int64_t plan_slots() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        sms = 152;
    }
    return kBlocksPerSm * static_cast<int64_t>(sms);
}

int64_t row_floats(int64_t Dm) { return (5 * Dm + 3) / 4 * 4; }

struct Plan {
    int64_t seg, segs, nbd;
};
Plan plan(int64_t batch, int64_t L, int64_t Dm) {
    Plan q;
    q.nbd = (Dm + kBlockChannels - 1) / kBlockChannels;
    q.seg = segment_steps(batch, L, q.nbd, plan_slots());
    q.segs = (L + q.seg - 1) / q.seg;
    return q;
}

// L == 0: the window passes through, so its gradient does, and the weights' are sums over nothing.
__global__ void window_grad_copy(const float* dwin_out, float* dwin_in, int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < n) dwin_in[i] = dwin_out ? dwin_out[i] : 0.f;
}

template <typename T, bool SILU>
cudaError_t launch(const ConvBwdParams& p, const ConvBwdMaps* m, dim3 grid, cudaStream_t stream) {
    if (m) ss_conv1d_bwd_kernel<T, SILU><<<grid, kThreads, 0, stream>>>(p, *m);
    else ss_conv1d_bwd_plain_kernel<T, SILU><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace
}  // namespace selscan

using namespace selscan;
using namespace selscan::host;

extern "C" size_t ss_conv1d_bwd_workspace_size(int64_t batch, int64_t L, int64_t Dm) {
    if (batch <= 0 || L <= 0 || Dm <= 0 || batch > 65535 || L > INT32_MAX - 64 || Dm > INT32_MAX / 8) return 0;
    const Plan q = plan(batch, L, Dm);
    return static_cast<size_t>(batch * q.segs * row_floats(Dm)) * 4;
}

extern "C" ss_status ss_conv1d_bwd(const void* dout, const void* x, const float* weight, const float* bias, const float* window_in,
                                   const float* dwindow_out, void* dx, float* dweight, float* dbias, float* dwindow_in, int64_t batch,
                                   int64_t L, int64_t Dm, int32_t silu, const ss_conv_grad_strides* strides, void* workspace,
                                   size_t workspace_bytes, void* stream_ptr) {
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    if (batch < 0 || L < 0 || Dm < 0) return SS_ERR_INVALID_ARG;
    ss_conv_grad_strides s;
    if (strides) {
        s = *strides;
    } else {
        std::memset(&s, 0, sizeof(s));
        s.io_dtype = SS_F32;
        s.dout_b = s.x_b = s.dx_b = L * Dm;
        s.dout_l = s.x_l = s.dx_l = Dm;
    }
    if (s.io_dtype != SS_F32 && s.io_dtype != SS_BF16) return SS_ERR_INVALID_ARG;
    if (Dm == 0) return SS_OK;
    if (batch > 65535 || L > INT32_MAX - 64 || Dm > INT32_MAX / 8) return SS_ERR_UNSUPPORTED;
    if (!weight || !dweight || !dbias) return SS_ERR_INVALID_ARG;
    const bool some = batch > 0 && L > 0, bf16 = s.io_dtype == SS_BF16;
    const int64_t es = bf16 ? 2 : 4;
    if (some && (!dout || !x || !dx)) return SS_ERR_INVALID_ARG;
    if (s.dout_b < 0 || s.dout_l < 0 || s.x_b < 0 || s.x_l < 0 || s.dx_b < 0 || s.dx_l < 0) return SS_ERR_INVALID_ARG;
    if (some && !distinct3(batch, s.dx_b, L, s.dx_l, Dm)) return SS_ERR_INVALID_ARG;      // dx: one word each
    const size_t need = some ? ss_conv1d_bwd_workspace_size(batch, L, Dm) : 0;
    if (some && (!workspace || workspace_bytes < need)) return SS_ERR_INVALID_ARG;
    const void* f[] = {weight, bias, window_in, dwindow_out, dweight, dbias, dwindow_in};
    for (const void* q : f)
        if (q && !is_aligned(q, 4)) return SS_ERR_MISALIGNED;
    const void* io[] = {dout, x, dx};
    if (some)
        for (const void* q : io)
            if (!is_aligned(q, es)) return SS_ERR_MISALIGNED;
    if (some && !is_aligned(workspace, 256)) return SS_ERR_MISALIGNED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SS_ERR_CUDA;
    for (const void* q : f)
        if (q && !dev_ptr(q, dev)) return SS_ERR_INVALID_ARG;
    if (some) {
        for (const void* q : io)
            if (!dev_ptr(q, dev)) return SS_ERR_INVALID_ARG;
        if (!dev_ptr(workspace, dev)) return SS_ERR_INVALID_ARG;
    }
    // outputs meet nothing else
    const int64_t wn = Dm * (kConvK - 1);
    auto win = [&](const float* q) { return range3(q, 1, batch, wn, 0, wn, 4); };
    const Range in[] = {range3(some ? dout : nullptr, batch, L, Dm, s.dout_b, s.dout_l, es), range3(some ? x : nullptr, batch, L, Dm, s.x_b, s.x_l, es),
                        range3(weight, 1, Dm, kConvK, 0, kConvK, 4), range3(bias, 1, 1, Dm, 0, 0, 4), win(window_in),
                        win(dwindow_out)};
    const Range out[] = {range3(some ? dx : nullptr, batch, L, Dm, s.dx_b, s.dx_l, es), range3(dweight, 1, Dm, kConvK, 0, kConvK, 4),
                         range3(dbias, 1, 1, Dm, 0, 0, 4), win(dwindow_in), range3(some ? workspace : nullptr, 1, 1, static_cast<int64_t>(need), 0, 0, 1)};
    for (int i = 0; i < 5; ++i) {
        for (const Range& r : in)
            if (meet(out[i], r)) return SS_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return SS_ERR_INVALID_ARG;
    }
    if (!some) {
        bool ok = cudaMemsetAsync(dweight, 0, Dm * kConvK * 4, stream) == cudaSuccess && cudaMemsetAsync(dbias, 0, Dm * 4, stream) == cudaSuccess;
        if (ok && batch > 0 && dwindow_in) {
            window_grad_copy<<<static_cast<unsigned>((batch * wn + 255) / 256), 256, 0, stream>>>(dwindow_out, dwindow_in, batch * wn);
            ok = cudaGetLastError() == cudaSuccess;
        }
        return ok ? SS_OK : SS_ERR_CUDA;
    }
    const Plan q = plan(batch, L, Dm);
    if (q.segs * q.nbd > INT32_MAX || batch * q.segs > INT32_MAX) return SS_ERR_UNSUPPORTED;
    ConvBwdParams p;
    p.dout = dout; p.x = x; p.w = weight; p.bias = bias; p.win_in = window_in; p.dwin_out = dwindow_out; p.dx = dx;
    p.dwin_in = dwindow_in; p.part = static_cast<float*>(workspace);
    p.do_b = s.dout_b; p.do_l = s.dout_l; p.x_b = s.x_b; p.x_l = s.x_l; p.dx_b = s.dx_b; p.dx_l = s.dx_l; p.ld = row_floats(Dm);
    p.L = static_cast<int>(L); p.Dm = static_cast<int>(Dm); p.seg = static_cast<int>(q.seg); p.nbd = static_cast<int>(q.nbd);
    p.err = device_error_word();
    // TMA: rows and bases on 16-byte boundaries; a pair of outputs is one store
    ConvBwdMaps m;
    const int steps = 16 / static_cast<int>(es);
    const bool tma = Dm % 2 == 0 && is_aligned(dx, 2 * es) && s.dx_l % 2 == 0 && (batch == 1 || s.dx_b % 2 == 0) &&
                     make_tile_map(&m.x, x, bf16, Dm, L, batch, s.x_l, s.x_b, kBlockChannels, steps) &&
                     make_tile_map(&m.dout, dout, bf16, Dm, L, batch, s.dout_l, s.dout_b, kBlockChannels, steps);
    const dim3 grid(static_cast<unsigned>(q.segs * q.nbd), static_cast<unsigned>(batch));
    const ConvBwdMaps* maps = tma ? &m : nullptr;
    const cudaError_t k = bf16 ? (silu ? launch<__nv_bfloat16, true>(p, maps, grid, stream) : launch<__nv_bfloat16, false>(p, maps, grid, stream))
                               : (silu ? launch<float, true>(p, maps, grid, stream) : launch<float, false>(p, maps, grid, stream));
    if (k != cudaSuccess) return SS_ERR_CUDA;
    const cudaError_t e = launch_column_sum(p.part, static_cast<int>(batch * q.segs), p.ld, 5 * p.Dm, 4 * p.Dm, dweight, dbias, stream);
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}
