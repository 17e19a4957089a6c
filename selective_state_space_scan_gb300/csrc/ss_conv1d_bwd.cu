// Backward of the causal depthwise conv1d + SiLU (ss_conv1d.cu).  With e = window ++ x and
// v_t = bias + Σ_k w_k e_{t+k}:
//   g_t = dout_t · silu'(v_t),  silu'(v) = σ(v) (1 + v (1 - σ(v)))      (g_t = dout_t without SiLU)
//   de_j = Σ_k w_k g_{j-k}  (dx_t = de_{t+3}; de_0..2 is the window's gradient),
//   dw_k = Σ_{b,t} g_t e_{t+k},  dbias = Σ_{b,t} g_t
//
// A stream of three elements per step and channel.  A thread has 2 channels (a packed pair) and a segment of steps;
// the next steps' loads are in flight while it works on some, and a warp covers 64 channels of a step.  It runs
// three steps past its segment, whose g belong to its last outputs.  The weight's gradients are sums in registers;
// every thread leaves its own in the workspace (a row of it per segment) and a second kernel adds the rows up in
// the same order every time.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/selscan.h"
#include "column_sum.h"
#include "device_common.cuh"
#include "host_util.h"

namespace selscan {
namespace {

constexpr int kConvK = SS_CONV_WIDTH;   // 4
constexpr int kSegMin = 8;
constexpr int kThreads = 256;
constexpr int kBlockChannels = 2 * kThreads;
constexpr int kBlocksPerSm = 3;

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
};

// 2 channels of one step as loaded.  VEC: adjacent ones; else kThreads apart, so that a warp's are adjacent.
template <typename T, bool VEC> struct Chan2;
template <> struct Chan2<float, true> {
    float2 v;
    __device__ __forceinline__ void load(const float* q, bool) { v = __ldcs(reinterpret_cast<const float2*>(q)); }
    __device__ __forceinline__ float2 get() const { return v; }
    __device__ __forceinline__ void zero() { v = make_float2(0.f, 0.f); }
};
template <> struct Chan2<__nv_bfloat16, true> {
    uint32_t v;
    __device__ __forceinline__ void load(const __nv_bfloat16* q, bool) { v = __ldcs(reinterpret_cast<const uint32_t*>(q)); }
    __device__ __forceinline__ float2 get() const { return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); }
    __device__ __forceinline__ void zero() { v = 0u; }
};
template <typename T> struct Chan2<T, false> {
    T v[2];
    __device__ __forceinline__ void load(const T* q, bool two) {
        v[0] = q[0];
        v[1] = two ? q[kThreads] : from_f32<T>(0.f);
    }
    __device__ __forceinline__ float2 get() const { return make_float2(to_f32<T>(v[0]), to_f32<T>(v[1])); }
    __device__ __forceinline__ void zero() { v[0] = v[1] = from_f32<T>(0.f); }
};
template <typename T, bool VEC>
__device__ __forceinline__ void store2(T* q, bool two, float2 v) {
    if constexpr (VEC && sizeof(T) == 4) {
        __stcs(reinterpret_cast<float2*>(q), v);
    } else if constexpr (VEC) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
        __stcs(reinterpret_cast<uint32_t*>(q), *reinterpret_cast<const uint32_t*>(&h));
    } else {
        q[0] = from_f32<T>(v.x);
        if (two) q[kThreads] = from_f32<T>(v.y);
    }
}

__device__ __forceinline__ float2 silu_slope(float2 v) {
    const float2 s = rcp2(add2(splat2(1.f), ex2x2(mul2(v, splat2(-kLog2e)))));
    return mul2(s, fma2(v, fma2(s, splat2(-1.f), splat2(1.f)), splat2(1.f)));
}

template <typename T, bool VEC, bool SILU>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) ss_conv1d_bwd_kernel(const ConvBwdParams p) {
    constexpr int U = VEC && sizeof(T) == 2 ? 8 : 4;      // steps whose loads are issued together
    const int seg = static_cast<int>(blockIdx.x) / p.nbd, b = blockIdx.y;
    const int base = (static_cast<int>(blockIdx.x) - seg * p.nbd) * kBlockChannels;
    const int d0 = base + (VEC ? 2 * threadIdx.x : threadIdx.x);
    if (d0 >= p.Dm) return;
    const int d1 = d0 + (VEC ? 1 : kThreads);
    const bool two = VEC || d1 < p.Dm;
    const int t0 = seg * p.seg, t1 = min(t0 + p.seg, p.L);
    const T* x = static_cast<const T*>(p.x) + b * p.x_b + d0;
    const T* dout = static_cast<const T*>(p.dout) + b * p.do_b + d0;
    T* dx = static_cast<T*>(p.dx) + b * p.dx_b + d0;

    auto each = [&](auto&& f) { return make_float2(f(d0), two ? f(d1) : 0.f); };            // f(channel)
    auto window = [&](const float* w, int k) {
        return each([&](int d) { return w[(static_cast<int64_t>(b) * p.Dm + d) * 3 + k]; });
    };
    float2 w[kConvK];
#pragma unroll
    for (int k = 0; k < kConvK; ++k) w[k] = each([&](int d) { return p.w[static_cast<int64_t>(d) * kConvK + k]; });
    const float2 bs = each([&](int d) { return p.bias ? p.bias[d] : 0.f; });
    // the three samples before the segment, and g of the three steps before
    float2 e[3], g[3], dw[kConvK], db = splat2(0.f);
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const int t = t0 - 3 + j;
        e[j] = g[j] = splat2(0.f);
        if (t >= 0) {
            Chan2<T, VEC> q;
            q.load(x + t * p.x_l, two);
            e[j] = q.get();
        } else if (p.win_in) {
            e[j] = window(p.win_in, 3 + t);
        }
    }
#pragma unroll
    for (int k = 0; k < kConvK; ++k) dw[k] = splat2(0.f);

    const int end = t1 + 3, have = min(end, p.L);  // the steps whose g reach the segment's outputs; those there are
    const T* xq = x + t0 * p.x_l;
    const T* dq = dout + t0 * p.do_l;
    auto load = [&](int tb, Chan2<T, VEC> (&xs)[U], Chan2<T, VEC> (&ds)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (tb + u < have) {
                xs[u].load(xq, two);
                ds[u].load(dq, two);
            } else {
                xs[u].zero();
                ds[u].zero();
            }
            xq += p.x_l;
            dq += p.do_l;
        }
    };
    // Step t: g_t (live: of a step that there is), its part in the weight's gradients (own: of the segment), and de of
    // three steps before.
    auto step = [&](float2 xv, float2 gt, bool own, bool live) {
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
    };
    T* out = dx + t0 * p.dx_l;
    Chan2<T, VEC> xs[U], ds[U];
    load(t0, xs, ds);
    for (int tb = t0; tb < end; tb += U) {
        Chan2<T, VEC> xn[U], dn[U];
        load(tb + U, xn, dn);
        if (tb >= t0 + 3 && tb + U <= t1) {        // steps inside the segment, as all but its ends are
#pragma unroll
            for (int u = 0; u < U; ++u) {
                store2<T, VEC>(out, two, step(xs[u].get(), ds[u].get(), true, true));
                out += p.dx_l;
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = tb + u, j = t - 3;   // j: the step (below 0: the window's entry) that de belongs to
                if (t >= end) break;
                float2 de = step(xs[u].get(), ds[u].get(), t < t1, t < p.L);
                if (p.dwin_out && j >= p.L - 3) de = add2(de, window(p.dwin_out, j - (p.L - 3)));
                if (j >= t0) {
                    store2<T, VEC>(out, two, de);
                    out += p.dx_l;
                } else if (j < 0 && p.dwin_in) {
                    float* q = p.dwin_in + static_cast<int64_t>(b) * p.Dm * 3 + 3 + j;
                    q[static_cast<int64_t>(d0) * 3] = de.x;
                    if (two) q[static_cast<int64_t>(d1) * 3] = de.y;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xs[u] = xn[u];
            ds[u] = dn[u];
        }
    }
    float* mine = p.part + (static_cast<int64_t>(b) * (gridDim.x / p.nbd) + seg) * p.ld;
    *reinterpret_cast<float4*>(mine + 4 * static_cast<int64_t>(d0)) = make_float4(dw[0].x, dw[1].x, dw[2].x, dw[3].x);
    mine[4 * static_cast<int64_t>(p.Dm) + d0] = db.x;
    if (two) {
        *reinterpret_cast<float4*>(mine + 4 * static_cast<int64_t>(d1)) = make_float4(dw[0].y, dw[1].y, dw[2].y, dw[3].y);
        mine[4 * static_cast<int64_t>(p.Dm) + d1] = db.y;
    }
}

// Steps per thread for batch · ceil(L / seg) · nbd blocks when `slots` are resident at once: the length whose
// waves take the least time, a block taking seg + kSetup steps' worth (the three steps past its end, the
// weights, and the sums' way out).
constexpr int kSetup = 10;
int segment_steps(int64_t batch, int64_t L, int64_t nbd, int64_t slots) {
    int64_t best = L, best_cost = -1;
    for (int64_t segs = 1; segs <= std::max<int64_t>(L / kSegMin, 1); ++segs) {
        const int64_t seg = (L + segs - 1) / segs, blocks = batch * ((L + seg - 1) / seg) * nbd;
        const int64_t cost = (blocks + slots - 1) / slots * (seg + kSetup);
        if (best_cost < 0 || cost < best_cost) {
            best_cost = cost;
            best = seg;
        }
        if (blocks > 8 * slots) break;
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

template <typename T>
void (*kernel_of(bool vec, bool silu))(ConvBwdParams) {
    if (vec) return silu ? ss_conv1d_bwd_kernel<T, true, true> : ss_conv1d_bwd_kernel<T, true, false>;
    return silu ? ss_conv1d_bwd_kernel<T, false, true> : ss_conv1d_bwd_kernel<T, false, false>;
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
    const int64_t va = 2 * es;                     // bytes of 2 channels
    auto wide = [&](const void* a, int64_t sb, int64_t sl) {
        return is_aligned(a, va) && (sl * es) % va == 0 && (batch == 1 || (sb * es) % va == 0);
    };
    const bool vec = Dm % 2 == 0 && wide(dout, s.dout_b, s.dout_l) && wide(x, s.x_b, s.x_l) && wide(dx, s.dx_b, s.dx_l);
    void (*kern)(ConvBwdParams) = bf16 ? kernel_of<__nv_bfloat16>(vec, silu != 0) : kernel_of<float>(vec, silu != 0);
    kern<<<dim3(static_cast<unsigned>(q.segs * q.nbd), static_cast<unsigned>(batch)), kThreads, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return SS_ERR_CUDA;
    const cudaError_t e = launch_column_sum(p.part, static_cast<int>(batch * q.segs), p.ld, 5 * p.Dm, 4 * p.Dm, dweight, dbias, stream);
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}
