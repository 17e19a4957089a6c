// Residual addition and layer norm, forward and backward.
//   r = x + residual,  xh = (r - mean) · rstd,  y = xh · weight + bias
//   a = dy · weight,   dr_in = rstd · (a - mean(a) - xh · mean(a · xh)) + dr,
//   dweight = Σ_rows dy · xh,  dbias = Σ_rows dy
//
// Streams, like ss_norm.cu: a row stays in the registers of the CTA that has it (8 columns a thread and
// run), and the next row's loads are in flight.  Both passes need one exchange among the warps: forward,
// each warp gives the sum and the squares about its own mean, which combine without cancellation
// (Σ (r - m)² = Σ_w [M2_w + n_w (m_w - m)²]); backward, the two sums over a.
// A thread has the same columns in every row, so the weight's gradients are sums in registers; each CTA
// leaves its own in the workspace and a second kernel adds them up, in the same order every time.
// 32768 rows of 2560, bf16 with an fp32 residual: forward 147 us for 1.0 GB, backward 197 us for 1.34 GB, both at the
// copy rate, the sums 5 us.  64 rows of 768: 3.5 us each, the launch and a few trips to memory.
// Rows or bases off 16 bytes, and widths that are no whole runs, are read and written by single elements: 32768 rows of 2559
// 325 and 318 us (2560 through the binding 156 and 209); bf16 alone, without a residual, 261 and 276 (105 and 136).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/selscan.h"
#include "chained.cuh"
#include "column_sum.h"
#include "device_common.cuh"
#include "host_util.h"
#include "row_runs.cuh"

namespace selscan {
namespace {

constexpr int kMaxWarps = 16;

struct LnParams {
    const void* x;          // backward: dy
    const void* res;        // or nullptr; backward: r
    const void* dr;         // backward, or nullptr
    const float* w;
    const float* b;         // or nullptr
    void* y;                // backward: dx, or nullptr
    void* res_out;          // or nullptr; backward: dresidual
    float* mean;            // backward: read
    float* rstd;
    float* part;            // backward: [grid][2][D]
    int64_t x_r, res_r, dr_r, y_r, res_out_r;
    int D;
    int64_t rows;
    float eps, inv_d;
};

// One thread's 8 columns of run k.  VEC: adjacent (16-byte accesses); else a warp's lanes have adjacent ones.
template <bool VEC> struct Cols {
    int D, nt, tid;
    __device__ __forceinline__ int at(int k, int i) const { return VEC ? (k * nt + tid) * kRun + i : (k * kRun + i) * nt + tid; }
    __device__ __forceinline__ bool has(int k, int i) const { return at(k, i) < D; }
    // Columns of warp w.
    __device__ __forceinline__ int of_warp(int w, int runs) const {
        int n = 0;
        for (int j = 0; j < (VEC ? runs : runs * kRun); ++j) {
            const int per = VEC ? kRun : 1;
            n += min(max(D - (j * nt + w * 32) * per, 0), 32 * per);
        }
        return n;
    }
};

template <typename T, bool VEC> struct ColsRaw;
template <typename T> struct ColsRaw<T, true> {
    Raw<T, true> raw;
    __device__ __forceinline__ void load(const T* row, const Cols<true>& c, int k) {
        raw.load(row + c.at(k, 0), row && c.has(k, 0) ? kRun : 0);
    }
    __device__ __forceinline__ void get(float v[kRun]) const { raw.get(v); }
};
template <typename T> struct ColsRaw<T, false> {
    T raw[kRun];
    __device__ __forceinline__ void load(const T* row, const Cols<false>& c, int k) {
#pragma unroll
        for (int i = 0; i < kRun; ++i) raw[i] = row && c.has(k, i) ? row[c.at(k, i)] : from_f32<T>(0.f);
    }
    __device__ __forceinline__ void get(float v[kRun]) const {
#pragma unroll
        for (int i = 0; i < kRun; ++i) v[i] = to_f32<T>(raw[i]);
    }
};
template <typename T, bool VEC>
__device__ __forceinline__ void store_cols(T* row, const Cols<VEC>& c, int k, const float v[kRun]) {
    if constexpr (VEC) {
        if (c.has(k, 0)) store_run<T, true>(row + c.at(k, 0), kRun, v);
    } else {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
            if (c.has(k, i)) row[c.at(k, i)] = from_f32<T>(v[i]);
    }
}
template <bool VEC>
__device__ __forceinline__ void load_weights(const float* w, const Cols<VEC>& c, int k, float v[kRun]) {
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 f = c.has(k, 0) ? __ldg(reinterpret_cast<const float4*>(w + c.at(k, 0)) + i) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kRun; ++i) v[i] = c.has(k, i) ? __ldg(w + c.at(k, i)) : 0.f;
    }
}

// Whether the registers hold the next row's loads beside a row (else a row is loaded when its turn comes).
template <bool VEC, int K> constexpr bool kAhead = VEC ? K < 4 : K < 2;

__device__ __forceinline__ float warp_sum(float v, int lanes = 32) {
    for (int o = lanes / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename TIO, typename TR, bool VEC, int K>
__global__ void __launch_bounds__(512) layernorm_kernel(const LnParams p) {
    __shared__ float2 part[2][kMaxWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    const Cols<VEC> c{p.D, static_cast<int>(blockDim.x), static_cast<int>(threadIdx.x)};
    const float n_mine = static_cast<float>(c.of_warp(warp, K));
    const float n_lane = lane < warps ? static_cast<float>(c.of_warp(lane, K)) : 0.f;
    const float inv_mine = n_mine > 0.f ? 1.f / n_mine : 0.f, inv_lane = n_lane > 0.f ? 1.f / n_lane : 0.f;
    ColsRaw<TIO, VEC> rx[K];
    ColsRaw<TR, VEC> rr[K];
    auto load_row = [&](int64_t row) {
        const TIO* x = static_cast<const TIO*>(p.x) + row * p.x_r;
        const TR* res = p.res ? static_cast<const TR*>(p.res) + row * p.res_r : nullptr;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            rx[k].load(x, c, k);
            rr[k].load(res, c, k);
        }
    };
    if (kAhead<VEC, K>) load_row(blockIdx.x);
    int turn = 0;                                  // rows take the two sets of partial results in turn
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        if (!kAhead<VEC, K>) load_row(row);
        float r[K][kRun], sum = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float b[kRun];
            rx[k].get(r[k]);
            rr[k].get(b);
#pragma unroll
            for (int i = 0; i < kRun; ++i) sum += r[k][i] += b[i];
        }
        if (kAhead<VEC, K> && row + gridDim.x < p.rows) load_row(row + gridDim.x);          // on its way while this row is worked on
        if (p.res_out) {
            TR* ro = static_cast<TR*>(p.res_out) + row * p.res_out_r;
#pragma unroll
            for (int k = 0; k < K; ++k) store_cols<TR, VEC>(ro, c, k, r[k]);
        }
        sum = warp_sum(sum);
        const float m_w = sum * inv_mine;
        float m2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                const float d = c.has(k, i) ? r[k][i] - m_w : 0.f;
                m2 = fmaf(d, d, m2);
            }
        m2 = warp_sum(m2);
        if (lane == 0) part[turn][warp] = make_float2(sum, m2);
        __syncthreads();
        const float2 q = lane < warps ? part[turn][lane] : make_float2(0.f, 0.f);
        const float mean = __shfl_sync(0xffffffffu, warp_sum(q.x, kMaxWarps), 0) * p.inv_d;
        const float dm = q.x * inv_lane - mean;
        const float var = __shfl_sync(0xffffffffu, warp_sum(fmaf(n_lane * dm, dm, q.y), kMaxWarps), 0) * p.inv_d;
        const float rstd = rsqrtf(var + p.eps);
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        TIO* y = static_cast<TIO*>(p.y) + row * p.y_r;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[kRun], b[kRun];
            load_weights<VEC>(p.w, c, k, w);
            if (p.b) {
                load_weights<VEC>(p.b, c, k, b);
            } else {
#pragma unroll
                for (int i = 0; i < kRun; ++i) b[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < kRun; ++i) r[k][i] = fmaf((r[k][i] - mean) * rstd, w[i], b[i]);
            store_cols<TIO, VEC>(y, c, k, r[k]);
        }
    }
}

template <typename TIO, typename TR, bool VEC, int K>
__global__ void __launch_bounds__(512) layernorm_bwd_kernel(const LnParams p) {
    __shared__ float2 part[2][kMaxWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    const Cols<VEC> c{p.D, static_cast<int>(blockDim.x), static_cast<int>(threadIdx.x)};
    ColsRaw<TIO, VEC> rdy[K];
    ColsRaw<TR, VEC> rr[K], rdr[K];
    let_next_start();                              // (the sums' kernel: it waits for this one's end)
    float next_mean, next_rstd;
    auto load_row = [&](int64_t row) {
        const TIO* dy = static_cast<const TIO*>(p.x) + row * p.x_r;
        const TR* r = static_cast<const TR*>(p.res) + row * p.res_r;
        const TR* dr = p.dr ? static_cast<const TR*>(p.dr) + row * p.dr_r : nullptr;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            rdy[k].load(dy, c, k);
            rr[k].load(r, c, k);
            rdr[k].load(dr, c, k);
        }
        next_mean = __ldg(p.mean + row);
        next_rstd = __ldg(p.rstd + row);
    };
    float dw[K][kRun], db[K][kRun];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < kRun; ++i) dw[k][i] = db[k][i] = 0.f;
    if (kAhead<VEC, K>) load_row(blockIdx.x);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        if (!kAhead<VEC, K>) load_row(row);
        const float mean = next_mean, rstd = next_rstd;
        float a[K][kRun], xh[K][kRun], d0[K][kRun];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[kRun];
            rdy[k].get(a[k]);
            rr[k].get(xh[k]);
            rdr[k].get(d0[k]);
            load_weights<VEC>(p.w, c, k, w);
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                xh[k][i] = (xh[k][i] - mean) * rstd;
                dw[k][i] = fmaf(a[k][i], xh[k][i], dw[k][i]);
                db[k][i] += a[k][i];
                a[k][i] *= w[i];
                s1 += a[k][i];                     // (zero where there is no column)
                s2 = fmaf(a[k][i], xh[k][i], s2);
            }
        }
        if (kAhead<VEC, K> && row + gridDim.x < p.rows) load_row(row + gridDim.x);
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (lane == 0) part[turn][warp] = make_float2(s1, s2);
        __syncthreads();
        const float2 q = lane < warps ? part[turn][lane] : make_float2(0.f, 0.f);
        s1 = __shfl_sync(0xffffffffu, warp_sum(q.x, kMaxWarps), 0) * p.inv_d;
        s2 = __shfl_sync(0xffffffffu, warp_sum(q.y, kMaxWarps), 0) * p.inv_d;
        TIO* dx = p.y ? static_cast<TIO*>(p.y) + row * p.y_r : nullptr;
        TR* dres = p.res_out ? static_cast<TR*>(p.res_out) + row * p.res_out_r : nullptr;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < kRun; ++i) a[k][i] = fmaf(fmaf(-xh[k][i], s2, a[k][i] - s1), rstd, d0[k][i]);
            if (dx) store_cols<TIO, VEC>(dx, c, k, a[k]);
            if (dres) store_cols<TR, VEC>(dres, c, k, a[k]);
        }
    }
    float* mine = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < kRun; ++i)
            if (c.has(k, i)) {
                mine[c.at(k, i)] = dw[k][i];
                mine[p.D + c.at(k, i)] = db[k][i];
            }
}

template <typename TIO, typename TR, bool VEC, int K>
cudaError_t launch_k(const LnParams& p, bool bwd, int threads, int64_t max_grid, int* grid_out, cudaStream_t stream) {
    void (*kern)(const LnParams) = bwd ? layernorm_bwd_kernel<TIO, TR, VEC, K> : layernorm_kernel<TIO, TR, VEC, K>;
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && p.rows > sms) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0);
    if (e != cudaSuccess) return e;
    // as many CTAs as fit at once, each with its share of the rows (an SM has room for one at least)
    const int64_t grid = std::min({p.rows, static_cast<int64_t>(sms) * std::max(per_sm, 1), max_grid});
    *grid_out = static_cast<int>(grid);
    kern<<<static_cast<unsigned>(grid), threads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename TIO, typename TR, bool VEC>
cudaError_t launch_v(const LnParams& p, bool bwd, int64_t max_grid, int* grid, cudaStream_t stream) {
    const int runs = (p.D + kRun - 1) / kRun, k = runs <= 512 ? 1 : runs <= 1024 ? 2 : 4;
    const int threads = ((runs + k - 1) / k + 31) / 32 * 32;
    if (k == 1) return launch_k<TIO, TR, VEC, 1>(p, bwd, threads, max_grid, grid, stream);
    if (k == 2) return launch_k<TIO, TR, VEC, 2>(p, bwd, threads, max_grid, grid, stream);
    return launch_k<TIO, TR, VEC, 4>(p, bwd, threads, max_grid, grid, stream);
}

cudaError_t launch(const LnParams& p, bool io_bf16, bool res_bf16, bool vec, bool bwd, int64_t max_grid, int* grid, cudaStream_t s) {
    using B = __nv_bfloat16;
    auto go = [&](auto tio, auto tr) {
        using I = decltype(tio);
        using R = decltype(tr);
        return vec ? launch_v<I, R, true>(p, bwd, max_grid, grid, s) : launch_v<I, R, false>(p, bwd, max_grid, grid, s);
    };
    return io_bf16 ? (res_bf16 ? go(B(), B()) : go(B(), 0.f)) : (res_bf16 ? go(0.f, B()) : go(0.f, 0.f));
}

using host::dev_ptr;
using host::is_aligned;
using host::meet;
using host::Range;
using host::range3;

// A [rows, D] operand of a call.
struct Mat {
    const void* q;
    int64_t stride, es;
    bool out;
};

// The checks that both calls share; `same` (an output, or -1) may lie exactly on input `on`.
ss_status check(const Mat* m, int n, int64_t rows, int64_t D, const void* const* f32, const int64_t* f32_n, int nf, int first_out_f32,
                int same, int on) {
    for (int i = 0; i < n; ++i) {
        if (!m[i].q) continue;
        if (m[i].stride < 0 || (m[i].out && rows > 1 && m[i].stride < D)) return SS_ERR_INVALID_ARG;
    }
    for (int i = 0; i < n; ++i)
        if (m[i].q && !is_aligned(m[i].q, m[i].es)) return SS_ERR_MISALIGNED;
    for (int i = 0; i < nf; ++i)
        if (f32[i] && !is_aligned(f32[i], 4)) return SS_ERR_MISALIGNED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SS_ERR_CUDA;
    for (int i = 0; i < n; ++i)
        if (m[i].q && !dev_ptr(m[i].q, dev)) return SS_ERR_INVALID_ARG;
    for (int i = 0; i < nf; ++i)
        if (f32[i] && !dev_ptr(f32[i], dev)) return SS_ERR_INVALID_ARG;
    auto mat = [&](int i) { return range3(m[i].q, 1, rows, D, 0, m[i].stride, m[i].es); };
    auto vec = [&](int i) { return range3(f32[i], 1, 1, f32_n[i], 0, 0, 4); };
    for (int i = 0; i < n; ++i) {
        if (!m[i].out) continue;
        for (int j = 0; j < n; ++j) {
            if (j == i || (m[j].out && j < i)) continue;
            if (i == same && j == on && m[i].q == m[j].q && (m[i].stride == m[j].stride || rows == 1)) continue;
            if (meet(mat(i), mat(j))) return SS_ERR_INVALID_ARG;
        }
        for (int j = 0; j < nf; ++j)
            if (meet(mat(i), vec(j))) return SS_ERR_INVALID_ARG;
    }
    for (int i = first_out_f32; i < nf; ++i) {
        for (int j = 0; j < n; ++j)
            if (meet(vec(i), mat(j))) return SS_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (meet(vec(i), vec(j))) return SS_ERR_INVALID_ARG;
    }
    return SS_OK;
}

// 16-byte accesses: whole runs, rows and bases on that boundary.
bool wide(const Mat* m, int n, int64_t rows, int64_t D, const float* w, const float* b) {
    bool ok = D % kRun == 0 && is_aligned(w, 16) && (!b || is_aligned(b, 16));
    for (int i = 0; i < n; ++i) ok = ok && (!m[i].q || (is_aligned(m[i].q, 16) && (rows == 1 || (m[i].stride * m[i].es) % 16 == 0)));
    return ok;
}

bool type_ok(int32_t t) { return t == SS_F32 || t == SS_BF16; }
int64_t size_of(int32_t t) { return t == SS_BF16 ? 2 : 4; }

// CTAs of the backward kernel at most (8 to an SM): what the workspace has room for.
int64_t bwd_max_grid(int64_t rows) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        sms = 152;
    }
    return std::min<int64_t>(rows, 8 * static_cast<int64_t>(sms));
}

}  // namespace
}  // namespace selscan

using namespace selscan;

extern "C" ss_status ss_add_layernorm(const void* x, const void* residual, const float* weight, const float* bias, void* residual_out,
                                      void* y, float* mean, float* rstd, int64_t rows, int64_t D, float eps,
                                      const ss_norm_strides* strides, void* stream) {
    if (rows < 0 || D < 0) return SS_ERR_INVALID_ARG;
    if (D > SS_NORM_MAX || rows > INT32_MAX) return SS_ERR_UNSUPPORTED;
    ss_norm_strides s;
    if (strides) {
        s = *strides;
    } else {
        std::memset(&s, 0, sizeof(s));
        s.io_dtype = s.res_dtype = SS_F32;
        s.x_r = s.res_r = s.res_out_r = s.y_r = D;
    }
    if (!type_ok(s.io_dtype) || !type_ok(s.res_dtype) || !(eps >= 0.f)) return SS_ERR_INVALID_ARG;
    if (rows == 0 || D == 0) return SS_OK;
    if (!x || !weight || !y) return SS_ERR_INVALID_ARG;
    const int64_t xe = size_of(s.io_dtype), re = size_of(s.res_dtype);
    const Mat m[] = {{x, s.x_r, xe, false}, {residual, s.res_r, re, false}, {residual_out, s.res_out_r, re, true}, {y, s.y_r, xe, true}};
    const void* f[] = {weight, bias, mean, rstd};
    const int64_t fn[] = {D, D, rows, rows};
    const ss_status st = check(m, 4, rows, D, f, fn, 4, 2, 2, 1);
    if (st != SS_OK) return st;
    LnParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = x; p.res = residual; p.w = weight; p.b = bias; p.y = y; p.res_out = residual_out; p.mean = mean; p.rstd = rstd;
    p.x_r = s.x_r; p.res_r = s.res_r; p.y_r = s.y_r; p.res_out_r = s.res_out_r;
    p.D = static_cast<int>(D); p.rows = rows; p.eps = eps; p.inv_d = 1.f / static_cast<float>(D);
    int grid = 0;
    const cudaError_t e = launch(p, s.io_dtype == SS_BF16, s.res_dtype == SS_BF16, wide(m, 4, rows, D, weight, bias), false, rows, &grid,
                                 static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

extern "C" size_t ss_add_layernorm_bwd_workspace_size(int64_t rows, int64_t D) {
    if (rows <= 0 || D <= 0 || D > SS_NORM_MAX || rows > INT32_MAX) return 0;
    return static_cast<size_t>(bwd_max_grid(rows)) * 2 * static_cast<size_t>(D) * 4;
}

extern "C" ss_status ss_add_layernorm_bwd(const void* dy, const void* dr, const void* r, const float* weight, const float* mean,
                                          const float* rstd, void* dx, void* dresidual, float* dweight, float* dbias, int64_t rows,
                                          int64_t D, const ss_norm_grad_strides* strides, void* workspace, size_t workspace_bytes,
                                          void* stream) {
    if (rows < 0 || D < 0) return SS_ERR_INVALID_ARG;
    if (D > SS_NORM_MAX || rows > INT32_MAX) return SS_ERR_UNSUPPORTED;
    ss_norm_grad_strides s;
    if (strides) {
        s = *strides;
    } else {
        std::memset(&s, 0, sizeof(s));
        s.io_dtype = s.res_dtype = SS_F32;
        s.dy_r = s.dr_r = s.r_r = s.dx_r = s.dres_r = D;
    }
    if (!type_ok(s.io_dtype) || !type_ok(s.res_dtype)) return SS_ERR_INVALID_ARG;
    if (D == 0) return SS_OK;
    if (!dweight || !dbias) return SS_ERR_INVALID_ARG;
    cudaStream_t st_ = static_cast<cudaStream_t>(stream);
    const int64_t ye = size_of(s.io_dtype), re = size_of(s.res_dtype);
    if (rows == 0) {                                          // the sums over no rows
        if (!is_aligned(dweight, 4) || !is_aligned(dbias, 4)) return SS_ERR_MISALIGNED;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return SS_ERR_CUDA;
        if (!dev_ptr(dweight, dev) || !dev_ptr(dbias, dev)) return SS_ERR_INVALID_ARG;
        const bool ok = cudaMemsetAsync(dweight, 0, D * 4, st_) == cudaSuccess && cudaMemsetAsync(dbias, 0, D * 4, st_) == cudaSuccess;
        return ok ? SS_OK : SS_ERR_CUDA;
    }
    if (!dy || !r || !weight || !mean || !rstd) return SS_ERR_INVALID_ARG;
    const size_t need = ss_add_layernorm_bwd_workspace_size(rows, D);
    if (!workspace || workspace_bytes < need) return SS_ERR_INVALID_ARG;
    if (!is_aligned(workspace, 256)) return SS_ERR_MISALIGNED;
    const Mat m[] = {{dy, s.dy_r, ye, false}, {dr, s.dr_r, re, false}, {r, s.r_r, re, false}, {dx, s.dx_r, ye, true},
                     {dresidual, s.dres_r, re, true}};
    const void* f[] = {weight, mean, rstd, dweight, dbias, workspace};
    const int64_t fn[] = {D, rows, rows, D, D, static_cast<int64_t>(need / 4)};
    const ss_status st = check(m, 5, rows, D, f, fn, 6, 3, 4, 1);
    if (st != SS_OK) return st;
    LnParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = dy; p.res = r; p.dr = dr; p.w = weight; p.y = dx; p.res_out = dresidual;
    p.mean = const_cast<float*>(mean); p.rstd = const_cast<float*>(rstd); p.part = static_cast<float*>(workspace);
    p.x_r = s.dy_r; p.res_r = s.r_r; p.dr_r = s.dr_r; p.y_r = s.dx_r; p.res_out_r = s.dres_r;
    p.D = static_cast<int>(D); p.rows = rows; p.inv_d = 1.f / static_cast<float>(D);
    int grid = 0;
    cudaError_t e = launch(p, s.io_dtype == SS_BF16, s.res_dtype == SS_BF16, wide(m, 5, rows, D, weight, nullptr), true, bwd_max_grid(rows),
                           &grid, st_);
    if (e != cudaSuccess) return SS_ERR_CUDA;
    e = launch_column_sum(p.part, grid, 2 * p.D, 2 * p.D, p.D, dweight, dbias, st_);
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}
