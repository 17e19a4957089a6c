// Residual addition and root-mean-square norm, y in the input's type or in 8 bits with scales.
//   r = x + residual,  y = r · rsqrt(mean r² + eps) · weight;
//   8 bits: scale = max(max |y|, 1e-30) / 448 over a block of columns (or the row), e4m3(y / scale).
//
// A stream: every element is read once and written once, so a row stays in the registers of the
// CTA that has it between its sum of squares and its output.  A thread has K runs of 8 adjacent
// columns (16-byte accesses for bf16), run k·threads + thread, so a warp covers 256 adjacent
// columns and the maximum over a block of 32 to 256 columns is a shuffle among 4 to 32 lanes.
// A CTA takes a share of the rows and has the next one's loads in flight.  32768 rows of 2560, bf16 with an fp32
// residual, e4m3 out: 142 us, 6.5 TB/s, 0.96 of the copy rate; 1000 rows 7.6 us; 61 rows 2.6 us (one trip to
// memory and the launch).
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/selscan.h"
#include "device_common.cuh"
#include "host_util.h"
#include "row_runs.cuh"

namespace selscan {
namespace {

constexpr float kF8Max = 448.f;        // largest finite e4m3
constexpr float kAmaxMin = 1e-30f;     // keeps 1/scale finite

struct NormParams {
    const void* x;
    const void* res;        // or nullptr
    const float* w;
    void* res_out;          // or nullptr
    void* y;
    float* scale;
    int64_t x_r, res_r, res_out_r, y_r;
    int D, block;           // block 0: the row
    int nblocks;
    int64_t rows;
    float eps, inv_d;
};

// The codes of v / scale (round to nearest even; at most 448 by the choice of scale).  The quotient is
// v·(1/scale) and one correction by its remainder: as good as rounded once, so that a value near the
// middle of two codes goes where a division would put it.  (An infinite scale has no remainder: v / scale is 0,
// NaN for an infinite v.)
template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* q, int n, const float v[kRun], float scale) {
    const float inv = 1.f / scale, back = scale == INFINITY ? 0.f : scale;
    uint32_t lo[4];
    auto quotient = [&](float x) {
        const float f = x * inv;
        return fmaf(fmaf(-f, back, x), inv, f);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i)
        lo[i] = __nv_cvt_float2_to_fp8x2(make_float2(quotient(v[2 * i]), quotient(v[2 * i + 1])), __NV_SATFINITE, __NV_E4M3);
    if constexpr (VEC) {
        __stcs(reinterpret_cast<uint2*>(q), make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16));
    } else {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
            if (i < n) q[i] = static_cast<uint8_t>(lo[i / 2] >> (8 * (i & 1)));
    }
}

// Magnitudes as whole numbers: their order is that of the floats, with NaN above infinity, so a
// NaN survives the maximum.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ float scale_of(uint32_t amax) {
    const float a = __uint_as_float(amax);
    return (a < kAmaxMin ? kAmaxMin : a) / kF8Max;
}

template <typename TIO, typename TR, bool F8, bool VEC, int K>
__global__ void __launch_bounds__(512) norm_kernel(const NormParams p) {
    __shared__ float part[2][16];
    __shared__ uint32_t pmax[2][16];
    const int tid = threadIdx.x, nt = blockDim.x, warp = tid / 32, lane = tid % 32;
    Raw<TIO, VEC> rx[K];
    Raw<TR, VEC> rr[K];
    auto load_row = [&](int64_t row) {
        const TIO* x = static_cast<const TIO*>(p.x) + row * p.x_r;
        const TR* res = p.res ? static_cast<const TR*>(p.res) + row * p.res_r : nullptr;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * nt + tid) * kRun;
            rx[k].load(x + c, p.D - c);
            rr[k].load(res + c, res ? p.D - c : 0);
        }
    };
    load_row(blockIdx.x);
    int turn = 0;                                  // rows take the two sets of partial results in turn
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        float r[K][kRun];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float b[kRun];
            rx[k].get(r[k]);
            rr[k].get(b);
#pragma unroll
            for (int i = 0; i < kRun; ++i) r[k][i] += b[i];
        }
        if (row + gridDim.x < p.rows) load_row(row + gridDim.x);          // on its way while this row is worked on
        if (p.res_out) {
            TR* ro = static_cast<TR*>(p.res_out) + row * p.res_out_r;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * nt + tid) * kRun;
                const int n = min(kRun, p.D - c);
                if (n > 0) store_run<TR, VEC>(ro + c, n, r[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < kRun; ++i) sum = fmaf(r[k][i], r[k][i], sum);
#pragma unroll
        for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) part[turn][warp] = sum;
        __syncthreads();
        sum = lane < nt / 32 ? part[turn][lane] : 0.f;                   // (at most 16 warps)
#pragma unroll
        for (int o = 8; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sum = __shfl_sync(0xffffffffu, sum, 0);
        const float rstd = rsqrtf(fmaf(sum, p.inv_d, p.eps));
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * nt + tid) * kRun;
            const int n = min(kRun, p.D - c);
            if (n > 0) {
                float w[kRun];
                if constexpr (VEC) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 f = __ldg(reinterpret_cast<const float4*>(p.w + c) + i);
                        w[4 * i] = f.x; w[4 * i + 1] = f.y; w[4 * i + 2] = f.z; w[4 * i + 3] = f.w;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kRun; ++i) w[i] = i < n ? p.w[c + i] : 0.f;
                }
#pragma unroll
                for (int i = 0; i < kRun; ++i) r[k][i] = i < n ? r[k][i] * rstd * w[i] : 0.f;
            }
        }
        if constexpr (!F8) {
            TIO* y = static_cast<TIO*>(p.y) + row * p.y_r;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * nt + tid) * kRun;
                const int n = min(kRun, p.D - c);
                if (n > 0) store_run<TIO, VEC>(y + c, n, r[k]);
            }
        } else {
            uint8_t* y = static_cast<uint8_t*>(p.y) + row * p.y_r;
            float* scale = p.scale + row * p.nblocks;
            uint32_t m[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                m[k] = 0u;
#pragma unroll
                for (int i = 0; i < kRun; ++i) m[k] = max(m[k], mag_bits(r[k][i]));
            }
            if (p.block == 0) {
                uint32_t a = m[0];
#pragma unroll
                for (int k = 1; k < K; ++k) a = max(a, m[k]);
                a = __reduce_max_sync(0xffffffffu, a);
                if (lane == 0) pmax[turn][warp] = a;
                __syncthreads();
                a = __reduce_max_sync(0xffffffffu, lane < nt / 32 ? pmax[turn][lane] : 0u);
                const float sc = scale_of(a);
                if (tid == 0) scale[0] = sc;
#pragma unroll
                for (int k = 0; k < K; ++k) m[k] = __float_as_uint(sc);
            } else {
                const int lanes = p.block / kRun;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    for (int o = lanes / 2; o > 0; o /= 2) m[k] = max(m[k], __shfl_xor_sync(0xffffffffu, m[k], o));
                    const float sc = scale_of(m[k]);
                    const int c = (k * nt + tid) * kRun;
                    if (c < p.D && lane % lanes == 0) scale[c / p.block] = sc;
                    m[k] = __float_as_uint(sc);
                }
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * nt + tid) * kRun;
                const int n = min(kRun, p.D - c);
                if (n > 0) store_codes<VEC>(y + c, n, r[k], __uint_as_float(m[k]));
            }
        }
    }
}

template <typename TIO, typename TR, bool F8, bool VEC, int K>
cudaError_t launch_norm_k(const NormParams& p, cudaStream_t stream) {
    const int runs = (p.D + kRun - 1) / kRun;
    const int threads = ((runs + K - 1) / K + 31) / 32 * 32;
    void (*kern)(const NormParams) = norm_kernel<TIO, TR, F8, VEC, K>;
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && p.rows > sms) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0);
    if (e != cudaSuccess) return e;
    // as many CTAs as fit at once, each with its share of the rows (an SM has room for one at least)
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(p.rows, static_cast<int64_t>(sms) * std::max(per_sm, 1)));
    kern<<<grid, threads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename TIO, typename TR, bool F8, bool VEC>
cudaError_t launch_norm(const NormParams& p, cudaStream_t stream) {
    const int runs = (p.D + kRun - 1) / kRun;
    if (runs <= 512) return launch_norm_k<TIO, TR, F8, VEC, 1>(p, stream);
    if (runs <= 1024) return launch_norm_k<TIO, TR, F8, VEC, 2>(p, stream);
    return launch_norm_k<TIO, TR, F8, VEC, 4>(p, stream);
}

template <typename TIO, typename TR>
cudaError_t launch_typed(const NormParams& p, bool f8, bool vec, cudaStream_t s) {
    if (f8) return vec ? launch_norm<TIO, TR, true, true>(p, s) : launch_norm<TIO, TR, true, false>(p, s);
    return vec ? launch_norm<TIO, TR, false, true>(p, s) : launch_norm<TIO, TR, false, false>(p, s);
}

using host::dev_ptr;
using host::is_aligned;
using host::meet;
using host::Range;
using host::range3;

ss_status add_rmsnorm(const void* x, const void* residual, const float* weight, void* residual_out, void* y, bool f8,
                      float* scale, int64_t rows, int64_t D, int64_t block, float eps, const ss_norm_strides* strides,
                      void* stream) {
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
    if ((s.io_dtype != SS_F32 && s.io_dtype != SS_BF16) || (s.res_dtype != SS_F32 && s.res_dtype != SS_BF16))
        return SS_ERR_INVALID_ARG;
    if (f8 && block != 0 && block != 32 && block != 64 && block != 128 && block != 256) return SS_ERR_UNSUPPORTED;
    if (!(eps >= 0.f)) return SS_ERR_INVALID_ARG;
    if (rows == 0 || D == 0) return SS_OK;
    if (!x || !weight || !y || (f8 && !scale)) return SS_ERR_INVALID_ARG;
    const int64_t xe = s.io_dtype == SS_BF16 ? 2 : 4, re = s.res_dtype == SS_BF16 ? 2 : 4, ye = f8 ? 1 : xe;
    const int64_t nb = f8 ? (block ? (D + block - 1) / block : 1) : 0;
    if (s.x_r < 0 || (residual && s.res_r < 0)) return SS_ERR_INVALID_ARG;
    if (rows > 1 && (s.y_r < D || (residual_out && s.res_out_r < D))) return SS_ERR_INVALID_ARG;
    if (!is_aligned(x, xe) || !is_aligned(y, ye) || !is_aligned(weight, 4) || (residual && !is_aligned(residual, re)) ||
        (residual_out && !is_aligned(residual_out, re)) || (f8 && !is_aligned(scale, 4)))
        return SS_ERR_MISALIGNED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SS_ERR_CUDA;
    const void* all[] = {x, residual, weight, residual_out, y, f8 ? scale : nullptr};
    for (const void* q : all)
        if (q && !dev_ptr(q, dev)) return SS_ERR_INVALID_ARG;
    const Range rx = range3(x, 1, rows, D, 0, s.x_r, xe), rr = range3(residual, 1, rows, D, 0, s.res_r, re),
                rw = range3(weight, 1, 1, D, 0, 0, 4), ro = range3(residual_out, 1, rows, D, 0, s.res_out_r, re),
                ry = range3(y, 1, rows, D, 0, s.y_r, ye), rs = range3(scale, 1, rows, nb, 0, nb, 4);
    if (meet(ry, rx) || meet(ry, rr) || meet(ry, rw) || meet(ry, ro) || meet(ro, rx) || meet(ro, rw))
        return SS_ERR_INVALID_ARG;
    if (f8 && (meet(rs, rx) || meet(rs, rr) || meet(rs, rw) || meet(rs, ro) || meet(rs, ry))) return SS_ERR_INVALID_ARG;
    if (meet(ro, rr) && !(residual_out == residual && (s.res_out_r == s.res_r || rows == 1))) return SS_ERR_INVALID_ARG;

    NormParams p;
    p.x = x; p.res = residual; p.w = weight; p.res_out = residual_out; p.y = y; p.scale = scale;
    p.x_r = s.x_r; p.res_r = s.res_r; p.res_out_r = s.res_out_r; p.y_r = s.y_r;
    p.D = static_cast<int>(D); p.block = f8 ? static_cast<int>(block) : 0; p.nblocks = static_cast<int>(nb);
    p.rows = rows; p.eps = eps; p.inv_d = 1.f / static_cast<float>(D);
    // 16-byte accesses (8-byte ones for the codes): whole runs, rows and bases on that boundary
    auto wide = [&](const void* q, int64_t stride, int64_t es, int64_t a) {
        return !q || (is_aligned(q, a) && (rows == 1 || (stride * es) % a == 0));
    };
    const bool vec = D % kRun == 0 && is_aligned(weight, 16) && wide(x, s.x_r, xe, 16) && wide(residual, s.res_r, re, 16) &&
                     wide(residual_out, s.res_out_r, re, 16) && wide(y, s.y_r, ye, f8 ? 8 : 16);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool xb = s.io_dtype == SS_BF16, rb = s.res_dtype == SS_BF16;
    const cudaError_t e = xb ? (rb ? launch_typed<__nv_bfloat16, __nv_bfloat16>(p, f8, vec, st)
                                   : launch_typed<__nv_bfloat16, float>(p, f8, vec, st))
                             : (rb ? launch_typed<float, __nv_bfloat16>(p, f8, vec, st)
                                   : launch_typed<float, float>(p, f8, vec, st));
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

}  // namespace
}  // namespace selscan

extern "C" ss_status ss_add_rmsnorm(const void* x, const void* residual, const float* weight, void* residual_out, void* y,
                                    int64_t rows, int64_t D, float eps, const ss_norm_strides* strides, void* stream) {
    return selscan::add_rmsnorm(x, residual, weight, residual_out, y, false, nullptr, rows, D, 0, eps, strides, stream);
}

extern "C" ss_status ss_add_rmsnorm_f8(const void* x, const void* residual, const float* weight, void* residual_out,
                                       uint8_t* y8, float* scale, int64_t rows, int64_t D, int64_t block, float eps,
                                       const ss_norm_strides* strides, void* stream) {
    return selscan::add_rmsnorm(x, residual, weight, residual_out, y8, true, scale, rows, D, block, eps, strides, stream);
}
