// Divergence from a teacher's distribution over its top logits, and its gradient.  Per row, with student logits
// z [V], teacher logits t_k at ids_k (k < K) and a temperature τ:
//   p = softmax_k(t / τ),  q = softmax_v(z / τ),  loss = Σ_k p_k (log p_k - log q_{ids_k})
//   dz_v = dloss / τ · (q_v - Σ_{k: ids_k = v} p_k)
//
// The vocabulary is the traffic, and it is read once: a row is shared out to the CTAs of a cluster so that each
// keeps its slice (64 KB) in shared memory from the running maximum and sum to the gradient.  Bulk copies bring it,
// three CTAs to an SM while a slice has no more than 64256 bytes (the entries' arrays take 12.5 KB besides; larger ones
// leave two), so that an SM has some 190 KB under way or in use while its CTAs are at different points of their
// chain (entries, row, exchange of the sums, stores: some 11 us), and each CTA has a later one's slice fetched into L2.
// 4096 rows with 64 entries each, bf16: 128000 columns 376 us, 0.82 of the copy rate; 129280 502 and 131072 484, 0.62 and 0.65,
// as 65536 (0.64) and other slices of 64 KB; 2048 rows of 64000 and of 65536 fp32: 184 and 234 us.
// With a tenth of the rows without entries 352 us, 5.7 TB/s, 0.84.  Measured besides: without the fetch ahead 370 (one
// CTA of an SM further 361, four 414), slices of 32 KB in registers 663, of 32 KB in shared memory 438 (against 390 then),
// clusters that take rows in turn with the next one on its way 522, the cluster's own barrier for the exchange 428 (it
// waits for stores).  What of a longer row does not fit is read again from L2.  An entry's values lie in shared memory as
// well; their columns get their gradient after the row's stream, rounded once, duplicates summed.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/selscan.h"
#include "device_common.cuh"
#include "heads_device.cuh"
#include "host_util.h"
#include "internal.h"

namespace selscan {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 64 * 1024 + 512;             // bytes of a slice that a CTA holds at most
constexpr int kBatch = 4;                          // vectors that a thread works on at a time
constexpr int kMaxK = SS_DISTILL_MAX_K;
constexpr int kMaxCluster = 8;
constexpr int kAhead = 2;                          // CTAs of an SM: how far ahead slices are fetched into L2

struct DistillParams {
    const void* logits;
    const int32_t* ids;
    const void* teacher;
    const float* dloss;
    float* loss;
    void* dlogits;
    int64_t logits_r, ids_r, teacher_r, dlogits_r, dloss_r;
    int64_t rows;
    int V, K, slice, cap, ahead;                          // slice: columns of a CTA (a multiple of 8); cap: vectors it holds
    bool teacher_bf16;
    float inv_t;                                   // 1 / τ
    unsigned int* err;
};

struct DistillShared {
    int4 id[kMaxK / 4];                            // the entries' columns, -1: not there
    float t[kMaxK], z[kMaxK];                      // their logits: teacher's, student's
    float2 stat[kWarps], entry[kWarps];
    float part[kWarps];
    float2 sums[kMaxCluster];                      // (max, sum) of the slices of the cluster's CTAs, which they send here
    uint64_t full, sent;
    int abort;
};

template <typename T> struct Vec16;                // 16 bytes of a row
template <> struct Vec16<float> {
    static constexpr int n = 4;
    // The largest value (of a NaN and a number the number).
    template <int B> static __device__ __forceinline__ float max(const uint4 (&u)[B]) {
        float b = -INFINITY;
#pragma unroll
        for (int k = 0; k < B; ++k)
            b = fmaxf(b, fmaxf(fmaxf(__uint_as_float(u[k].x), __uint_as_float(u[k].y)), fmaxf(__uint_as_float(u[k].z), __uint_as_float(u[k].w))));
        return b;
    }
    static __device__ __forceinline__ void get(const uint4& u, float (&v)[4]) {
        v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y); v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <> struct Vec16<__nv_bfloat16> {
    static constexpr int n = 8;
    template <int B> static __device__ __forceinline__ float max(const uint4 (&u)[B]) {
        auto h = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); };
        __nv_bfloat162 b = h(u[0].x);
#pragma unroll
        for (int k = 0; k < B; ++k) b = __hmax2(b, __hmax2(__hmax2(h(u[k].x), h(u[k].y)), __hmax2(h(u[k].z), h(u[k].w))));
        return fmaxf(__low2float(b), __high2float(b));
    }
    static __device__ __forceinline__ void get(const uint4& u, float (&v)[8]) {
        const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(a[i] << 16);
            v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&v)[8]) {
        uint32_t a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            a[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(a[0], a[1], a[2], a[3]);
    }
};

// A running maximum m and the sum s of exp2((z - m) c).
struct Running {
    float m = -INFINITY, s = 0.f;
    // (-inf as the maximum so far: nothing but -inf seen, whose weights are zero)
    static __device__ __forceinline__ float base(float m) { return m == -INFINITY ? 0.f : m; }
    // n vectors (of the type T, what is behind them is not read)
    template <typename T, int B> __device__ __forceinline__ void take(const uint4 (&u)[B], float c) {
        constexpr int N = Vec16<T>::n;
        const float b = Vec16<T>::max(u);
        if (b > m) {
            s *= ex2((m - b) * c);
            m = b;
        }
        const float2 off = splat2(-base(m)), c2 = splat2(c);
        float2 a = splat2(0.f), a2 = a;
#pragma unroll
        for (int k = 0; k < B; ++k) {
            float v[N];
            Vec16<T>::get(u[k], v);
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                a = add2(a, ex2x2(mul2(add2(make_float2(v[i], v[i + 1]), off), c2)));
                a2 = add2(a2, ex2x2(mul2(add2(make_float2(v[i + 2], v[i + 3]), off), c2)));
            }
        }
        a = add2(a, a2);
        s += a.x + a.y;
    }
    __device__ __forceinline__ void one(float v, float c) {
        if (v > m) {
            s *= ex2((m - v) * c);
            m = v;
        }
        s += ex2((v - base(m)) * c);
    }
    // Over groups of LANES lanes.
    template <int LANES> __device__ __forceinline__ void join_lanes(float c) {
        float n = m;
#pragma unroll
        for (int o = LANES / 2; o > 0; o /= 2) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
        s *= ex2((m - base(n)) * c);
        m = n;
#pragma unroll
        for (int o = LANES / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    }
};

// Two floats into a CTA's shared memory, which its barrier counts (addresses of the cluster's window).
__device__ __forceinline__ void send_f32x2(uint32_t to, float2 v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to), "f"(v.x), "f"(v.y), "r"(bar)
                 : "memory");
}

template <typename T, bool GRAD>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillParams p) {
    constexpr int N = Vec16<T>::n;
    extern __shared__ __align__(128) uint4 held[];
    __shared__ DistillShared sh;
    uint32_t rank = 0, size = 1;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / size;
    const T* z = static_cast<const T*>(p.logits) + row * p.logits_r;
    const float c = kLog2e * p.inv_t;

    if (tid == 0) {
        mbar_init(&sh.full, 1);
        mbar_init(&sh.sent, 1);
        sh.abort = 0;
        mbar_fence_init();
    }
    // (after thread 0's part: what it sets up is there for the cluster once all have arrived)
    __syncwarp();
    if (size > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    // the teacher's entries, in every CTA of the row
    Running e;
    int32_t* sid = reinterpret_cast<int32_t*>(sh.id);
    for (int k = tid; k < (p.K + 3) / 4 * 4; k += kThreads) {           // (a multiple of 4: the last ones are not there)
        const int id = k < p.K ? p.ids[row * p.ids_r + k] : -1;
        const bool ok = id >= 0 && id < p.V;
        if (id >= p.V && rank == 0 && p.err) atomicOr(p.err, kErrIndex);
        float t = -INFINITY;
        if (ok)
            t = p.teacher_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.teacher)[row * p.teacher_r + k])
                               : static_cast<const float*>(p.teacher)[row * p.teacher_r + k];
        sh.t[k] = t;
        sid[k] = ok ? id : -1;
        e.one(t, c);                               // (-inf and what is not there: no weight)
    }
    const bool some = __syncthreads_or(e.s != 0.f);        // (NaN: a row with a NaN)

    const int lo = static_cast<int>(rank) * p.slice, hi = min(lo + p.slice, p.V);
    // columns up to the first 16-byte boundary, whole vectors, and what is left
    const int head = min(hi, lo + static_cast<int>(((16 - reinterpret_cast<uintptr_t>(z + lo) % 16) % 16) / sizeof(T)));
    const int vecs = hi > head ? (hi - head) / N : 0, tail = head + vecs * N;
    const uint4* zv = reinterpret_cast<const uint4*>(z + head);
    const int mine = min(vecs, p.cap);
    // the slice that a CTA of the next wave will want, on its way to L2 (if its row begins with an entry)
    if (tid == kThreads - 32) {
        const int64_t later = row + p.ahead / size;
        if (later < p.rows && p.K > 0 && p.ids[later * p.ids_r] >= 0) {
            const T* q = static_cast<const T*>(p.logits) + later * p.logits_r + lo;
            q += (16 - reinterpret_cast<uintptr_t>(q) % 16) % 16 / sizeof(T);
            if (mine > 1)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(__cvta_generic_to_global(q)), "r"((mine - 1) * 16) : "memory");
        }
    }
    bool ok = true;
    Running r;
    if (some) {
        if (tid == 0 && mine > 0) {
            mbar_expect_tx(&sh.full, static_cast<uint32_t>(mine) * 16u);
            bulk_load(held, zv, static_cast<uint32_t>(mine) * 16u, &sh.full);
        }
        for (int k = tid; k < p.K; k += kThreads) sh.z[k] = sid[k] >= 0 ? to_f32<T>(z[sid[k]]) : 0.f;
        if (tid / 32 * 32 < p.K) {                 // (a warp that has entries)
            e.join_lanes<32>(c);
            if (tid % 32 == 0) sh.entry[tid / 32] = make_float2(e.m, e.s);
        }
        if (lo + tid < head) r.one(to_f32<T>(z[lo + tid]), c);
        if (tail + tid < hi) r.one(to_f32<T>(z[tail + tid]), c);
        if (mine > 0) ok = mbar_wait_bounded(&sh.full, 0, &sh.abort, p.err);
        constexpr int kAll = kBatch * kThreads;
        int k = tid;
        for (; k + kAll - kThreads < mine; k += kAll) {
            uint4 u[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) u[j] = held[k + j * kThreads];
            r.take<T>(u, c);
        }
        for (; k < mine; k += kThreads) {
            const uint4 u[1] = {held[k]};
            r.take<T>(u, c);
        }
#pragma unroll 4
        for (k = mine + tid; k < vecs; k += kThreads) {
            const uint4 u[1] = {zv[k]};
            r.take<T>(u, c);
        }
        r.join_lanes<32>(c);
        if (tid % 32 == 0) sh.stat[tid / 32] = make_float2(r.m, r.s);
        __syncthreads();
        const float2 q = sh.stat[tid % kWarps], qe = tid % kWarps * 32 < p.K ? sh.entry[tid % kWarps] : make_float2(-INFINITY, 0.f);
        r.m = q.x; r.s = q.y; e.m = qe.x; e.s = qe.y;
        r.join_lanes<kWarps>(c);
        e.join_lanes<kWarps>(c);
        if (size > 1) {                            // (a row's CTAs agree on whether it has any weight)
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");              // the others' barriers exist
            if (tid == 0) mbar_expect_tx(&sh.sent, size * 8u);
            if (tid < static_cast<int>(size))
                send_f32x2(peer_smem_addr(&sh.sums[rank], tid), make_float2(r.m, r.s), peer_smem_addr(&sh.sent, tid));
            ok = mbar_wait_bounded<true>(&sh.sent, 0, &sh.abort, p.err) && ok;
            const float2 v = tid % 32 < static_cast<int>(size) ? sh.sums[tid % 32] : make_float2(-INFINITY, 0.f);
            r.m = v.x;
            r.s = v.y;
            r.join_lanes<kMaxCluster>(c);
            r.m = __shfl_sync(0xffffffffu, r.m, 0);
            r.s = __shfl_sync(0xffffffffu, r.s, 0);
        }
    }
    const float m = Running::base(r.m), inv_s = 1.f / r.s;
    const float mt = Running::base(e.m), inv_pt = 1.f / e.s;

    if (rank == 0) {
        float sum = 0.f;
        if (some) {
            for (int k = tid; k < p.K; k += kThreads) {
                const float w = ex2((sh.t[k] - mt) * c) * inv_pt;
                if (w != 0.f) sum += w * ((sh.t[k] - mt) - (sh.z[k] - m)) * p.inv_t;
            }
#pragma unroll
            for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (tid % 32 == 0) sh.part[tid / 32] = sum;
            __syncthreads();
        }
        if (tid == 0) {
            sum = 0.f;
            if (some) {
                for (int i = 0; i < kWarps; ++i) sum += sh.part[i];
                sum += logf(r.s) - logf(e.s);
            }
            p.loss[row] = sum;
        }
    }
    if constexpr (GRAD) {
        T* d = static_cast<T*>(p.dlogits) + row * p.dlogits_r;
        const float g = some ? p.dloss[row * p.dloss_r] * p.inv_t : 0.f;
        const float gs = g * inv_s;
        const float2 off = splat2(-m), c2 = splat2(c), gs2 = splat2(gs);
        auto grad = [&](float v) { return some ? ex2((v - m) * c) * gs : 0.f; };
        // (a row of dlogits that lies otherwise against the 16 bytes is written element by element)
        const bool same = reinterpret_cast<uintptr_t>(d + head) % 16 == 0;
        const T first_z = some && lo + tid < head ? z[lo + tid] : from_f32<T>(0.f), last_z = some && tail + tid < hi ? z[tail + tid] : from_f32<T>(0.f);
        uint4* dv = reinterpret_cast<uint4*>(d + head);
        auto value = [&](const uint4& u, float (&v)[N]) {
            Vec16<T>::get(u, v);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float2 o = mul2(ex2x2(mul2(add2(make_float2(v[i], v[i + 1]), off), c2)), gs2);
                v[i] = o.x;
                v[i + 1] = o.y;
            }
        };
        if (!some) {
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            if (same)
                for (int k = tid; k < vecs; k += kThreads) __stcs(dv + k, zero);
            else
                for (int k = head + tid; k < tail; k += kThreads) d[k] = from_f32<T>(0.f);
        } else if (same) {
            float v[N];
            int k = tid;
            for (; k + (kBatch - 1) * kThreads < mine; k += kBatch * kThreads) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    value(held[k + j * kThreads], v);
                    __stcs(dv + k + j * kThreads, Vec16<T>::put(v));
                }
            }
            for (; k < mine; k += kThreads) {
                value(held[k], v);
                __stcs(dv + k, Vec16<T>::put(v));
            }
#pragma unroll 4
            for (k = mine + tid; k < vecs; k += kThreads) {
                value(__ldcs(zv + k), v);
                __stcs(dv + k, Vec16<T>::put(v));
            }
        } else {
            for (int k = tid; k < vecs; k += kThreads) {
                float v[N];
                value(k < mine ? held[k] : __ldcs(zv + k), v);
#pragma unroll
                for (int i = 0; i < N; ++i) d[head + k * N + i] = from_f32<T>(v[i]);
            }
        }
        if (lo + tid < head) d[lo + tid] = from_f32<T>(grad(to_f32<T>(first_z)));
        if (tail + tid < hi) d[tail + tid] = from_f32<T>(grad(to_f32<T>(last_z)));
        if (some) {
            // the entries' own columns in this slice, after all others: the first of equal ones has them all
            __syncthreads();
            for (int k = tid; k < p.K; k += kThreads) {
                const int id = sid[k];
                if (id < lo || id >= hi) continue;
                float w = 0.f;
                bool first = true;
                for (int i = 0; i < p.K; i += 4) {
                    const int4 o = sh.id[i / 4];
                    if (o.x != id && o.y != id && o.z != id && o.w != id) continue;
                    const int at[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (at[j] == id) {
                            first = first && i + j >= k;
                            w += ex2((sh.t[i + j] - mt) * c);
                        }
                }
                if (first) d[id] = from_f32<T>(g * (ex2((sh.z[k] - m) * c) * inv_s - w * inv_pt));
            }
        }
    }
    if (!ok)                                       // a wait that ran out: copies in flight are over long before this
        for (int i = 0; i < 20; ++i) __nanosleep(1000000);
    // (a CTA ends when it has everyone's sums, and its own have reached everyone: nobody ends before)
    if (!some && size > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// CTAs for a row: so many that each holds its slice, and more where the rows alone leave SMs idle, as long as each keeps
// some 8 KB (one row of 50257 fp32 5.8 us in 8 CTAs, 6.6 in 4; 300 rows of 32000 bf16 9.1 in one each, 9.9 in two).
int cluster_of(int64_t rows, int64_t row_bytes, int sms) {
    int n = 1;
    while (n < kMaxCluster && (row_bytes > n * static_cast<int64_t>(kHeld) || (rows * n < sms && row_bytes / (2 * n) >= 8192))) n *= 2;
    return n;
}

using host::dev_ptr;
using host::is_aligned;
using host::meet;
using host::Range;
using host::range3;

template <typename T, bool GRAD>
cudaError_t launch(const DistillParams& p, int cluster, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.rows * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.cap) * 16;
    cfg.stream = stream;
    // (cheap, and the same from every thread that calls)
    const cudaError_t e = cudaFuncSetAttribute(distill_kernel<T, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, distill_kernel<T, GRAD>, p);
}

ss_status distill(const float* dloss, const void* logits, const int32_t* ids, const void* teacher, float* loss, void* dlogits, bool grad,
                  int64_t rows, int64_t V, int64_t K, float temperature, const ss_distill_strides* strides, void* stream) {
    if (rows < 0 || V < 1 || K < 0 || !(temperature >= 1e-30f && temperature <= 1e30f)) return SS_ERR_INVALID_ARG;      // (1 / τ is a normal float)
    if (V > SS_DISTILL_MAX_V || K > SS_DISTILL_MAX_K || rows > INT32_MAX / kMaxCluster) return SS_ERR_UNSUPPORTED;
    ss_distill_strides s;
    if (strides) {
        s = *strides;
    } else {
        std::memset(&s, 0, sizeof(s));
        s.io_dtype = s.teacher_dtype = SS_F32;
        s.logits_r = s.dlogits_r = V;
        s.ids_r = s.teacher_r = K;
        s.dloss_r = 1;
    }
    if ((s.io_dtype != SS_F32 && s.io_dtype != SS_BF16) || (s.teacher_dtype != SS_F32 && s.teacher_dtype != SS_BF16)) return SS_ERR_INVALID_ARG;
    if (rows == 0) return SS_OK;
    if (!logits || !loss || (K > 0 && (!ids || !teacher)) || (grad && (!dloss || !dlogits))) return SS_ERR_INVALID_ARG;
    if (s.logits_r < 0 || s.ids_r < 0 || s.teacher_r < 0 || (grad && s.dloss_r < 0)) return SS_ERR_INVALID_ARG;
    if (grad && rows > 1 && s.dlogits_r < V) return SS_ERR_INVALID_ARG;
    const int64_t es = s.io_dtype == SS_BF16 ? 2 : 4, te = s.teacher_dtype == SS_BF16 ? 2 : 4;
    if (!is_aligned(logits, es) || !is_aligned(loss, 4) || (K > 0 && (!is_aligned(ids, 4) || !is_aligned(teacher, te))) ||
        (grad && (!is_aligned(dloss, 4) || !is_aligned(dlogits, es))))
        return SS_ERR_MISALIGNED;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return SS_ERR_CUDA;
    const void* all[] = {logits, K > 0 ? ids : nullptr, K > 0 ? teacher : nullptr, loss, grad ? dloss : nullptr, grad ? dlogits : nullptr};
    for (const void* q : all)
        if (q && !dev_ptr(q, dev)) return SS_ERR_INVALID_ARG;
    const Range rl = range3(logits, 1, rows, V, 0, s.logits_r, es), ri = range3(ids, 1, rows, K, 0, s.ids_r, 4),
                rt = range3(teacher, 1, rows, K, 0, s.teacher_r, te), ro = range3(loss, 1, 1, rows, 0, 0, 4),
                rg = range3(grad ? dloss : nullptr, 1, rows, 1, 0, s.dloss_r, 4), rd = range3(grad ? dlogits : nullptr, 1, rows, V, 0, s.dlogits_r, es);
    if (meet(ro, rl) || meet(ro, ri) || meet(ro, rt) || meet(ro, rg) || meet(ro, rd)) return SS_ERR_INVALID_ARG;
    if (meet(rd, ri) || meet(rd, rt) || meet(rd, rg)) return SS_ERR_INVALID_ARG;
    if (meet(rd, rl) && !(dlogits == logits && (s.dlogits_r == s.logits_r || rows == 1))) return SS_ERR_INVALID_ARG;

    DistillParams p;
    p.logits = logits; p.ids = ids; p.teacher = teacher; p.dloss = dloss; p.loss = loss; p.dlogits = dlogits;
    p.logits_r = s.logits_r; p.ids_r = s.ids_r; p.teacher_r = s.teacher_r; p.dlogits_r = s.dlogits_r; p.dloss_r = s.dloss_r;
    p.rows = rows; p.V = static_cast<int>(V); p.K = static_cast<int>(K);
    p.teacher_bf16 = s.teacher_dtype == SS_BF16;
    p.inv_t = 1.f / temperature;
    p.err = device_error_word();
    p.ahead = kAhead * sms;
    const int cluster = cluster_of(rows, V * es, sms);
    p.slice = static_cast<int>(((V + cluster - 1) / cluster + 7) / 8 * 8);
    p.cap = static_cast<int>(std::min<int64_t>(p.slice * es, kHeld) / 16);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool b = s.io_dtype == SS_BF16;
    const cudaError_t e = grad ? (b ? launch<__nv_bfloat16, true>(p, cluster, st) : launch<float, true>(p, cluster, st))
                               : (b ? launch<__nv_bfloat16, false>(p, cluster, st) : launch<float, false>(p, cluster, st));
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

}  // namespace
}  // namespace selscan

extern "C" ss_status ss_distill(const void* logits, const int32_t* ids, const void* teacher, float* loss, int64_t rows, int64_t V,
                                int64_t K, float temperature, const ss_distill_strides* strides, void* stream) {
    return selscan::distill(nullptr, logits, ids, teacher, loss, nullptr, false, rows, V, K, temperature, strides, stream);
}

extern "C" ss_status ss_distill_grad(const float* dloss, const void* logits, const int32_t* ids, const void* teacher, float* loss,
                                     void* dlogits, int64_t rows, int64_t V, int64_t K, float temperature,
                                     const ss_distill_strides* strides, void* stream) {
    return selscan::distill(dloss, logits, ids, teacher, loss, dlogits, true, rows, V, K, temperature, strides, stream);
}
