// Runs of 8 adjacent columns of a row, as the norm kernels read and write them (16-byte accesses for bf16).
#pragma once

#include <cuda_runtime.h>

#include "device_common.cuh"

namespace selscan {

constexpr int kRun = 8;

// 8 adjacent elements as loaded; `n` of them exist.  VEC: n is 8 or none, and the address 16-byte aligned.
template <typename T, bool VEC> struct Raw {
    static constexpr int kWords = sizeof(T) == 2 ? 1 : 2;
    uint4 u[kWords];
    __device__ __forceinline__ void load(const T* q, int n) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                u[i] = n > 0 ? __ldcs(reinterpret_cast<const uint4*>(q) + i) : make_uint4(0u, 0u, 0u, 0u);
        } else {
            T v[kRun];
#pragma unroll
            for (int i = 0; i < kRun; ++i) v[i] = i < n ? q[i] : from_f32<T>(0.f);
            if constexpr (sizeof(T) == 2) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = static_cast<uint32_t>(__bfloat16_as_ushort(v[2 * i])) | static_cast<uint32_t>(__bfloat16_as_ushort(v[2 * i + 1])) << 16;
                u[0] = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    u[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                                      __float_as_uint(v[4 * i + 3]));
            }
        }
    }
    __device__ __forceinline__ void get(float v[kRun]) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t a[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(a[i] << 16);
                v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[4 * i] = __uint_as_float(u[i].x);
                v[4 * i + 1] = __uint_as_float(u[i].y);
                v[4 * i + 2] = __uint_as_float(u[i].z);
                v[4 * i + 3] = __uint_as_float(u[i].w);
            }
        }
    }
};
template <typename T, bool VEC>
__device__ __forceinline__ void store_run(T* q, int n, const float v[kRun]) {
    if constexpr (VEC && sizeof(T) == 2) {
        uint32_t a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            a[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        __stcs(reinterpret_cast<uint4*>(q), make_uint4(a[0], a[1], a[2], a[3]));
    } else if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            __stcs(reinterpret_cast<float4*>(q) + i, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
    } else {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
            if (i < n) q[i] = from_f32<T>(v[i]);
    }
}

}  // namespace selscan
