// The next token of every row: temperature, top-k, top-p, min-p, then an exponential race with
// given random numbers.
//
// With l_max the row's largest logit, w = exp((l - l_max)/T).  Tokens are ordered by one whole
// number each, the logit's bits (made monotone) above the complement of the index, so there are no
// ties and the top-k and top-p sets are "every token from some number up".  That number is found
// without sorting the row: a histogram over d = (l_max - l)/T (counts, and weights in fixed point,
// whose sums do not depend on the order of the atomics) names the bin it is in; the bin's tokens,
// a few hundred as a rule, are collected in shared memory and ranked against each other.  A bin
// with more tokens than that (equal logits, or the tail beyond exp(-22)) is narrowed by further
// histograms over the ordering number itself.  The last pass runs the race over what stays and
// reads the noise of those tokens alone.
//
// A CTA has a row; its passes after the first read the logits from L2.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cstdint>

#include "../../include/selscan.h"
#include "device_common.cuh"
#include "host_util.h"

namespace selscan {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kCap = 1024;               // most tokens ranked against each other
constexpr int kIndexBits = 20;           // SS_SAMPLE_MAX
constexpr int kOrderBits = 32 + kIndexBits;
constexpr float kReach = 22.1807098f;    // ln 2^32: a weight below exp(-kReach) has no mass in fixed point
constexpr float kMassOne = 2147483648.f; // a weight of 1

static_assert(SS_SAMPLE_MAX == 1 << kIndexBits, "the ordering number holds every index");

struct SampleParams {
    const void* logits;
    const float* noise;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* tokens;
    int64_t logits_r, noise_r;
    int V;
};

__device__ __forceinline__ float tidy(float l) {           // NaN as -inf, +inf as the largest number
    return l != l ? -INFINITY : fminf(l, FLT_MAX);
}
__device__ __forceinline__ uint64_t order_of(float l, int i) {
    const uint32_t b = __float_as_uint(l + 0.f);           // -0 as +0: they are equal logits
    const uint32_t m = b & 0x80000000u ? ~b : b | 0x80000000u;
    return static_cast<uint64_t>(m) << kIndexBits | static_cast<uint32_t>((1 << kIndexBits) - 1 - i);
}
__device__ __forceinline__ int index_of(uint64_t order) {
    return (1 << kIndexBits) - 1 - static_cast<int>(order & ((1u << kIndexBits) - 1u));
}
__device__ __forceinline__ float logit_of(uint64_t order) {
    const uint32_t m = static_cast<uint32_t>(order >> kIndexBits);
    return __uint_as_float(m & 0x80000000u ? m & 0x7fffffffu : ~m);
}

template <typename T> struct Pack;
template <> struct Pack<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void load(const float* q, float v[4]) {
        const float4 f = *reinterpret_cast<const float4*>(q);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    }
};
template <> struct Pack<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void load(const __nv_bfloat16* q, float v[8]) {
        const uint4 u = *reinterpret_cast<const uint4*>(q);
        const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(a[i] << 16);
            v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        }
    }
};

// f(index, logit) for every token of the row: 16-byte loads between the first and the last
// 16-byte boundary of the row, single ones around them.
template <typename T, typename F>
__device__ __forceinline__ void each_token(const T* row, int V, F&& f) {
    constexpr int W = Pack<T>::n;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    const int head = min(V, off ? W - off : 0);
    const int body = (V - head) / W;
    const int tail0 = head + body * W;
    if (static_cast<int>(threadIdx.x) < head) f(static_cast<int>(threadIdx.x), tidy(to_f32<T>(row[threadIdx.x])));
    if (static_cast<int>(threadIdx.x) < V - tail0)
        f(tail0 + static_cast<int>(threadIdx.x), tidy(to_f32<T>(row[tail0 + threadIdx.x])));
#pragma unroll 2
    for (int b = threadIdx.x; b < body; b += kThreads) {
        float v[W];
        Pack<T>::load(row + head + b * W, v);
#pragma unroll
        for (int j = 0; j < W; ++j) f(head + b * W + j, tidy(v[j]));
    }
}

struct Shared {
    uint32_t count[kBins], lo[kBins], hi[kBins];   // a bin's tokens, and their mass as hi·2^32 + lo
    uint64_t cand[kCap];
    uint32_t cmass[kCap];
    uint64_t warp64[kWarps];
    uint32_t warp32[kWarps];
    uint64_t mass_above;      // of the bins before the found one
    uint32_t count_above;
    int bin;
    uint32_t ncand;
    uint64_t cut;
};

__device__ __forceinline__ uint64_t block_max(Shared& s, uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
        v = v > w ? v : w;
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) s.warp64[threadIdx.x / 32] = v;
    __syncthreads();
    v = s.warp64[threadIdx.x % 32];
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
        v = v > w ? v : w;
    }
    return v;
}

__device__ __forceinline__ void clear_bins(Shared& s) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = s.lo[i] = s.hi[i] = 0u;
    __syncthreads();
}
__device__ __forceinline__ void add_to_bin(Shared& s, int bin, uint32_t mass) {
    atomicAdd(&s.count[bin], 1u);
    if (mass) {
        const uint32_t old = atomicAdd(&s.lo[bin], mass);
        if (old + mass < old) atomicAdd(&s.hi[bin], 1u);      // the carry
    }
}
__device__ __forceinline__ uint64_t bin_mass(const Shared& s, int bin) {
    return static_cast<uint64_t>(s.hi[bin]) << 32 | s.lo[bin];
}

// The first bin at which the running count, begun at `count`, reaches `k` (by_mass false), or the
// running mass, begun at `mass`, reaches `target` (by_mass true); the last bin if none does.  Leaves
// it in s.bin, with the count and mass before it.
__device__ void find_bin(Shared& s, bool by_mass, uint32_t k, double target, uint32_t count, uint64_t mass) {
    static_assert(kBins == 2 * kThreads, "two bins a thread");
    const int b = 2 * threadIdx.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    __syncthreads();
    if (threadIdx.x == 0) s.bin = kBins;
    const uint32_t c0 = s.count[b], c1 = s.count[b + 1];
    const uint64_t m0 = bin_mass(s, b), m1 = bin_mass(s, b + 1);
    uint32_t ci = c0 + c1;
    uint64_t mi = m0 + m1;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t cu = __shfl_up_sync(0xffffffffu, ci, o);
        const uint64_t mu = __shfl_up_sync(0xffffffffu, mi, o);
        if (lane >= o) {
            ci += cu;
            mi += mu;
        }
    }
    __syncthreads();
    if (lane == 31) {
        s.warp32[warp] = ci;
        s.warp64[warp] = mi;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        count += s.warp32[w];
        mass += s.warp64[w];
    }
    const uint32_t cb = count + ci - c0 - c1;               // before bin b
    const uint64_t mb = mass + mi - m0 - m1;
    const bool r0 = by_mass ? static_cast<double>(mb + m0) >= target : cb + c0 >= k;
    const bool r1 = by_mass ? static_cast<double>(mb + m0 + m1) >= target : cb + c0 + c1 >= k;
    if (r0) atomicMin(&s.bin, b);
    else if (r1 || threadIdx.x == kThreads - 1) atomicMin(&s.bin, b + 1);
    __syncthreads();
    if (s.bin == b) {
        s.count_above = cb;
        s.mass_above = mb;
    } else if (s.bin == b + 1) {
        s.count_above = cb + c0;
        s.mass_above = mb + m0;
    }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p) {
    __shared__ Shared s;
    const int64_t r = blockIdx.x;
    const T* row = static_cast<const T*>(p.logits) + r * p.logits_r;
    const float* noise = p.noise + r * p.noise_r;
    const int V = p.V;

    uint64_t top = 0;
    each_token(row, V, [&](int i, float l) {
        const uint64_t o = order_of(l, i);
        top = o > top ? o : top;
    });
    top = block_max(s, top);
    const float lmax = logit_of(top);
    const float temp = p.temperature ? p.temperature[r] : 1.f;
    if (lmax == -INFINITY || temp <= 0.f) {
        if (threadIdx.x == 0) p.tokens[r] = lmax == -INFINITY ? -1 : index_of(top);
        return;
    }
    const float inv_t = fminf(1.f / (temp > 0.f ? temp : 1.f), 1e35f);   // finite times any reach
    const float c2 = inv_t * kLog2e;
    const int k = p.top_k && p.top_k[r] > 0 && p.top_k[r] < V ? p.top_k[r] : V;
    const float tp = p.top_p && p.top_p[r] < 1.f ? p.top_p[r] : 2.f;
    const float mp = p.min_p ? p.min_p[r] : 0.f;

    auto weight = [&](float l) { return l == -INFINITY ? 0.f : ex2((l - lmax) * c2); };
    const float per_bin = inv_t * (kBins / kReach);
    auto bin_of = [&](float l) { return static_cast<int>(fminf((lmax - l) * per_bin, kBins - 1.f)); };
    auto mass_of = [&](float l) { return __float2uint_rn(weight(l) * kMassOne); };

    // What stays: bins before `bin`, and in it the tokens whose number is at least `cut`.
    int bin = kBins;
    uint64_t cut = 0;
    if (k < V || tp < 2.f) {
        clear_bins(s);
        each_token(row, V, [&](int, float l) { add_to_bin(s, bin_of(l), mass_of(l)); });
        __syncthreads();

        // Collects the tokens of bin `b` that hold the k-th token (by_mass false) or the one at which
        // the mass reaches `target`, narrowing while there are more than kCap of them; `count` and
        // `mass` become those of the tokens above the collected ones.
        bool narrowed = false;
        auto collect = [&](int b, bool by_mass, uint32_t kk, double target, uint32_t& count, uint64_t& mass, uint32_t n) {
            uint64_t lo = 0;
            int bits = kOrderBits;                           // candidates: numbers lo .. lo + 2^bits - 1
            while (n > kCap) {
                const int shift = bits > 11 ? bits - 11 : 0;
                narrowed = true;
                __syncthreads();
                clear_bins(s);
                each_token(row, V, [&](int i, float l) {
                    if (bin_of(l) != b) return;
                    const uint64_t o = order_of(l, i) - lo;
                    if (o >> bits) return;
                    add_to_bin(s, kBins - 1 - static_cast<int>(o >> shift), mass_of(l));
                });
                __syncthreads();
                find_bin(s, by_mass, kk, target, count, mass);
                count = s.count_above;
                mass = s.mass_above;
                n = s.count[s.bin];
                lo += static_cast<uint64_t>(kBins - 1 - s.bin) << shift;
                bits = shift;
            }
            __syncthreads();
            if (threadIdx.x == 0) s.ncand = 0u;
            __syncthreads();
            each_token(row, V, [&](int i, float l) {
                if (bin_of(l) != b) return;
                const uint64_t o = order_of(l, i);
                if ((o - lo) >> bits) return;
                const uint32_t at = atomicAdd(&s.ncand, 1u);
                if (at < kCap) {
                    s.cand[at] = o;
                    s.cmass[at] = mass_of(l);
                }
            });
            __syncthreads();
        };
        // Over the collected tokens, with `count` and `mass` above them: the smallest number whose
        // token is among the first kk and has less than `target` above it (or is the row's first).
        auto smallest_kept = [&](uint32_t kk, double target, uint32_t count, uint64_t mass, uint64_t* kept_mass) {
            __syncthreads();
            if (threadIdx.x == 0) s.cut = ~0ull;
            __syncthreads();
            const int n = min(static_cast<int>(s.ncand), kCap);
            uint64_t sum = 0;
            for (int i = threadIdx.x; i < n; i += kThreads) {
                const uint64_t o = s.cand[i];
                uint32_t c = count;
                uint64_t m = mass;
                for (int j = 0; j < n; ++j)
                    if (s.cand[j] > o) {
                        ++c;
                        m += s.cmass[j];
                    }
                if ((c < kk && static_cast<double>(m) < target) || o == top) {
                    atomicMin(reinterpret_cast<unsigned long long*>(&s.cut), o);
                    sum = m + s.cmass[i];                    // largest at the smallest number
                }
            }
            sum = block_max(s, sum);
            if (kept_mass) *kept_mass = sum;
            __syncthreads();
            return s.cut;
        };

        uint32_t count = 0;
        uint64_t mass = 0;
        const double all = 1e300;
        double target = all;                                 // never below 1: the first token stays
        if (k < V) {
            find_bin(s, false, k, 0.0, 0u, 0ull);
            bin = s.bin;
            count = s.count_above;
            mass = s.mass_above;
            uint64_t kept = mass;
            collect(bin, false, k, 0.0, count, mass, s.count[bin]);
            cut = smallest_kept(k, all, count, mass, &kept);
            if (tp < 2.f) target = fmax(static_cast<double>(tp) * static_cast<double>(kept), 1.0);
        } else {
            // the whole mass: a target that no bin reaches leaves the last one
            find_bin(s, true, 0u, all, 0u, 0ull);
            target = fmax(static_cast<double>(tp) * static_cast<double>(s.mass_above + bin_mass(s, s.bin)), 1.0);
        }
        if (tp < 2.f) {
            const int kbin = bin;
            if (narrowed) {                                  // the bins hold something else by now
                __syncthreads();
                clear_bins(s);
                each_token(row, V, [&](int, float l) { add_to_bin(s, bin_of(l), mass_of(l)); });
                __syncthreads();
            }
            find_bin(s, true, 0u, target, 0u, 0ull);
            const int b = s.bin;
            if (b < kbin) {
                bin = b;
                count = s.count_above;
                mass = s.mass_above;
                collect(b, true, 0u, target, count, mass, s.count[b]);
                cut = smallest_kept(V, target, count, mass, nullptr);
            } else if (narrowed) {                           // the same bin, but elsewhere in it
                bin = kbin;
                find_bin(s, false, k, 0.0, 0u, 0ull);
                count = s.count_above;
                mass = s.mass_above;
                collect(kbin, true, 0u, target, count, mass, s.count[kbin]);
                const uint64_t pcut = smallest_kept(V, target, count, mass, nullptr);
                cut = pcut > cut ? pcut : cut;
            } else {
                cut = smallest_kept(k, target, count, mass, nullptr);
            }
        }
    }

    uint64_t best = 0;
    each_token(row, V, [&](int i, float l) {
        const int b = bin < kBins ? bin_of(l) : 0;
        if (b > bin) return;
        const uint64_t o = order_of(l, i);
        if (b == bin && o < cut) return;
        const float w = weight(l);
        if (!(w >= mp) && o != top) return;
        float key = w * rcp_approx(noise[i]);
        if (!(key >= 0.f)) key = 0.f;
        const uint64_t v = static_cast<uint64_t>(__float_as_uint(key)) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
        best = v > best ? v : best;
    });
    best = block_max(s, best);
    if (threadIdx.x == 0) p.tokens[r] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(best));
}

}  // namespace
}  // namespace selscan

using namespace selscan;
using namespace selscan::host;

extern "C" ss_status ss_sample(const void* logits, const float* noise, const float* temperature, const int32_t* top_k,
                               const float* top_p, const float* min_p, int32_t* tokens, int64_t rows, int64_t V,
                               int32_t io_dtype, int64_t logits_r, int64_t noise_r, void* stream_ptr) {
    if (rows < 0 || V < 1) return SS_ERR_INVALID_ARG;
    if (V > SS_SAMPLE_MAX || rows > INT32_MAX) return SS_ERR_UNSUPPORTED;
    if (io_dtype != SS_F32 && io_dtype != SS_BF16) return SS_ERR_INVALID_ARG;
    if (logits_r < 0 || noise_r < 0) return SS_ERR_INVALID_ARG;
    if (rows == 0) return SS_OK;
    if (!logits || !noise || !tokens) return SS_ERR_INVALID_ARG;
    const int64_t es = io_dtype == SS_BF16 ? 2 : 4;
    const void* f4[] = {noise, temperature, top_k, top_p, min_p, tokens};
    if (!is_aligned(logits, es)) return SS_ERR_MISALIGNED;
    for (const void* q : f4)
        if (q && !is_aligned(q, 4)) return SS_ERR_MISALIGNED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SS_ERR_CUDA;
    if (!dev_ptr(logits, dev)) return SS_ERR_INVALID_ARG;
    for (const void* q : f4)
        if (q && !dev_ptr(q, dev)) return SS_ERR_INVALID_ARG;
    const Range out = range3(tokens, 1, 1, rows, 0, 0, 4);
    const Range in[] = {range3(logits, 1, rows, V, 0, logits_r, es), range3(noise, 1, rows, V, 0, noise_r, 4),
                        range3(temperature, 1, 1, rows, 0, 0, 4), range3(top_k, 1, 1, rows, 0, 0, 4),
                        range3(top_p, 1, 1, rows, 0, 0, 4), range3(min_p, 1, 1, rows, 0, 0, 4)};
    for (const Range& q : in)
        if (meet(out, q)) return SS_ERR_INVALID_ARG;
    const SampleParams p{logits, noise, temperature, top_k, top_p, min_p, tokens, logits_r, noise_r, static_cast<int>(V)};
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    if (io_dtype == SS_BF16) sample_kernel<__nv_bfloat16><<<static_cast<unsigned>(rows), kThreads, 0, stream>>>(p);
    else sample_kernel<float><<<static_cast<unsigned>(rows), kThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}
