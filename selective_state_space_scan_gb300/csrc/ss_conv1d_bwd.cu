// Backward of the causal depthwise conv1d + SiLU (ss_conv1d.cu).  With e = window ++ x and
// v_t = bias + Σ_k w_k e_{t+k}:
//   g_t = dout_t · silu'(v_t),  silu'(v) = σ(v) (1 + v (1 - σ(v)))      (g_t = dout_t without SiLU)
//   de_j = Σ_k w_k g_{j-k}  (dx_t = de_{t+3}; de_0..2 is the window's gradient),
//   dw_k = Σ_{b,t} g_t e_{t+k},  dbias = Σ_{b,t} g_t
//
// A stream of three elements per step and channel.  As in the forward kernel, a thread has 4 channels (as two
// packed pairs) and a segment of steps, with several steps' loads in flight; it runs three steps past its
// segment, whose g belong to its last outputs.  The weight's gradients are sums in registers; every thread
// leaves its own in the workspace (a row of it per segment) and a second kernel adds the rows up in the same
// order every time.
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
constexpr int kThreads = 128;
constexpr int kBlockChannels = 4 * kThreads;

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

// 4 channels of one step as loaded.  VEC: adjacent ones; else kThreads apart, so that a warp's are adjacent.
template <typename T, bool VEC> struct Chan4;
template <> struct Chan4<float, true> {
    float4 v;
    __device__ __forceinline__ void load(const float* q, int) { v = __ldcs(reinterpret_cast<const float4*>(q)); }
    __device__ __forceinline__ float2 lo() const { return make_float2(v.x, v.y); }
    __device__ __forceinline__ float2 hi() const { return make_float2(v.z, v.w); }
    __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <> struct Chan4<__nv_bfloat16, true> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* q, int) { v = __ldcs(reinterpret_cast<const uint2*>(q)); }
    static __device__ __forceinline__ float2 pair(uint32_t u) { return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }
    __device__ __forceinline__ float2 lo() const { return pair(v.x); }
    __device__ __forceinline__ float2 hi() const { return pair(v.y); }
    __device__ __forceinline__ void zero() { v = make_uint2(0u, 0u); }
};
template <typename T> struct Chan4<T, false> {
    T v[4];
    __device__ __forceinline__ void load(const T* q, int n) {
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = c < n ? q[c * kThreads] : from_f32<T>(0.f);
    }
    __device__ __forceinline__ float2 lo() const { return make_float2(to_f32<T>(v[0]), to_f32<T>(v[1])); }
    __device__ __forceinline__ float2 hi() const { return make_float2(to_f32<T>(v[2]), to_f32<T>(v[3])); }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = from_f32<T>(0.f);
    }
};
template <typename T, bool VEC>
__device__ __forceinline__ void store4(T* q, int n, float2 lo, float2 hi) {
    if constexpr (VEC && sizeof(T) == 4) {
        __stcs(reinterpret_cast<float4*>(q), make_float4(lo.x, lo.y, hi.x, hi.y));
    } else if constexpr (VEC) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(lo.x, lo.y), b = __floats2bfloat162_rn(hi.x, hi.y);
        __stcs(reinterpret_cast<uint2*>(q), make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b)));
    } else {
        const float v[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < n) q[c * kThreads] = from_f32<T>(v[c]);
    }
}

__device__ __forceinline__ float2 silu_slope(float2 v) {
    const float2 s = rcp2(add2(splat2(1.f), ex2x2(mul2(v, splat2(-kLog2e)))));
    return mul2(s, fma2(v, fma2(s, splat2(-1.f), splat2(1.f)), splat2(1.f)));
}

template <typename T, bool VEC, bool SILU>
__global__ void __launch_bounds__(kThreads, 4) ss_conv1d_bwd_kernel(const ConvBwdParams p) {
    constexpr int U = sizeof(T) == 2 ? 8 : 4;      // steps whose loads are issued together
    const int seg = static_cast<int>(blockIdx.x) / p.nbd, b = blockIdx.y;
    const int base = (static_cast<int>(blockIdx.x) - seg * p.nbd) * kBlockChannels;
    const int d0 = base + (VEC ? 4 * threadIdx.x : threadIdx.x);
    constexpr int kStep = VEC ? 1 : kThreads;      // from one of the thread's channels to the next
    if (d0 >= p.Dm) return;
    const int nc = VEC ? 4 : min(4, (p.Dm - d0 + kThreads - 1) / kThreads);
    const int t0 = seg * p.seg, t1 = min(t0 + p.seg, p.L);
    const T* x = static_cast<const T*>(p.x) + b * p.x_b + d0;
    const T* dout = static_cast<const T*>(p.dout) + b * p.do_b + d0;
    T* dx = static_cast<T*>(p.dx) + b * p.dx_b + d0;

    auto chan = [&](int c) { return d0 + c * kStep; };
    float2 w[2][kConvK], bs[2];
    auto each = [&](auto&& f) {                    // f(channel) for the two pairs
        float2 r[2];
        r[0].x = f(0);
        r[0].y = nc > 1 ? f(1) : 0.f;
        r[1].x = nc > 2 ? f(2) : 0.f;
        r[1].y = nc > 3 ? f(3) : 0.f;
        return make_float4(r[0].x, r[0].y, r[1].x, r[1].y);
    };
#pragma unroll
    for (int k = 0; k < kConvK; ++k) {
        const float4 f = each([&](int c) { return p.w[static_cast<int64_t>(chan(c)) * kConvK + k]; });
        w[0][k] = make_float2(f.x, f.y);
        w[1][k] = make_float2(f.z, f.w);
    }
    {
        const float4 f = each([&](int c) { return p.bias ? p.bias[chan(c)] : 0.f; });
        bs[0] = make_float2(f.x, f.y);
        bs[1] = make_float2(f.z, f.w);
    }
    // the three samples before the segment
    float2 e[3][2];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const int t = t0 - 3 + j;
        if (t >= 0) {
            Chan4<T, VEC> q;
            q.load(x + t * p.x_l, nc);
            e[j][0] = q.lo();
            e[j][1] = q.hi();
        } else {
            const float4 f = each([&](int c) { return p.win_in ? p.win_in[(static_cast<int64_t>(b) * p.Dm + chan(c)) * 3 + 3 + t] : 0.f; });
            e[j][0] = make_float2(f.x, f.y);
            e[j][1] = make_float2(f.z, f.w);
        }
    }
    float2 g[3][2], dw[2][kConvK], db[2];          // g of the three steps before
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        db[h] = g[0][h] = g[1][h] = g[2][h] = splat2(0.f);
#pragma unroll
        for (int k = 0; k < kConvK; ++k) dw[h][k] = splat2(0.f);
    }
    const int end = t1 + 3;                        // the steps whose g reach the segment's outputs
    for (int tb = t0; tb < end; tb += U) {
        Chan4<T, VEC> xs[U], ds[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = tb + u;
            if (t < min(end, p.L)) {
                xs[u].load(x + t * p.x_l, nc);
                ds[u].load(dout + t * p.do_l, nc);
            } else {
                xs[u].zero();
                ds[u].zero();
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = tb + u;
            if (t >= end) break;
            const float2 xv[2] = {xs[u].lo(), xs[u].hi()}, dv[2] = {ds[u].lo(), ds[u].hi()};
            float2 de[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float2 gt = dv[h];
                if constexpr (SILU) {
                    const float2 v = fma2(w[h][3], xv[h], fma2(w[h][2], e[2][h], fma2(w[h][1], e[1][h], fma2(w[h][0], e[0][h], bs[h]))));
                    gt = mul2(gt, silu_slope(v));
                }
                if (t >= p.L) gt = splat2(0.f);
                if (t < t1) {
                    dw[h][0] = fma2(gt, e[0][h], dw[h][0]);
                    dw[h][1] = fma2(gt, e[1][h], dw[h][1]);
                    dw[h][2] = fma2(gt, e[2][h], dw[h][2]);
                    dw[h][3] = fma2(gt, xv[h], dw[h][3]);
                    db[h] = add2(db[h], gt);
                }
                de[h] = fma2(w[h][0], gt, fma2(w[h][1], g[2][h], fma2(w[h][2], g[1][h], mul2(w[h][3], g[0][h]))));
                g[0][h] = g[1][h];
                g[1][h] = g[2][h];
                g[2][h] = gt;
                e[0][h] = e[1][h];
                e[1][h] = e[2][h];
                e[2][h] = xv[h];
            }
            const int j = t - 3;                   // the step (below 0: the window's entry) that de belongs to
            if (p.dwin_out && j >= p.L - 3) {
                const float4 f = each([&](int c) { return p.dwin_out[(static_cast<int64_t>(b) * p.Dm + chan(c)) * 3 + j - (p.L - 3)]; });
                de[0] = add2(de[0], make_float2(f.x, f.y));
                de[1] = add2(de[1], make_float2(f.z, f.w));
            }
            if (j >= t0) {
                store4<T, VEC>(dx + j * p.dx_l, nc, de[0], de[1]);
            } else if (j < 0 && p.dwin_in) {
                const float v[4] = {de[0].x, de[0].y, de[1].x, de[1].y};
                for (int c = 0; c < nc; ++c) p.dwin_in[(static_cast<int64_t>(b) * p.Dm + chan(c)) * 3 + 3 + j] = v[c];
            }
        }
    }
    float* mine = p.part + (static_cast<int64_t>(b) * (gridDim.x / p.nbd) + seg) * p.ld;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (c >= nc) break;
        const int h = c / 2;
        const bool y = c & 1;
        float4 f = y ? make_float4(dw[h][0].y, dw[h][1].y, dw[h][2].y, dw[h][3].y) : make_float4(dw[h][0].x, dw[h][1].x, dw[h][2].x, dw[h][3].x);
        *reinterpret_cast<float4*>(mine + 4 * static_cast<int64_t>(chan(c))) = f;
        mine[4 * static_cast<int64_t>(p.Dm) + chan(c)] = y ? db[h].y : db[h].x;
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
    return 4 * static_cast<int64_t>(sms);
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
    const int64_t va = 4 * es;                     // bytes of 4 channels
    auto wide = [&](const void* a, int64_t sb, int64_t sl) {
        return is_aligned(a, va) && (sl * es) % va == 0 && (batch == 1 || (sb * es) % va == 0);
    };
    const bool vec = Dm % 4 == 0 && wide(dout, s.dout_b, s.dout_l) && wide(x, s.x_b, s.x_l) && wide(dx, s.dx_b, s.dx_l);
    void (*kern)(ConvBwdParams) = bf16 ? kernel_of<__nv_bfloat16>(vec, silu != 0) : kernel_of<float>(vec, silu != 0);
    kern<<<dim3(static_cast<unsigned>(q.segs * q.nbd), static_cast<unsigned>(batch)), kThreads, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return SS_ERR_CUDA;
    const cudaError_t e = launch_column_sum(p.part, static_cast<int>(batch * q.segs), p.ld, 5 * p.Dm, 4 * p.Dm, dweight, dbias, stream);
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}
