// The next token of every row: temperature, top-k, top-p, min-p, then an exponential race with
// given random numbers.
//
// With l_max the row's largest logit, w = exp((l - l_max)/T).  Tokens are ordered by one whole
// number each, the logit's bits (made monotone) above the complement of the index, so there are no
// ties and the top-k and top-p sets are "every token from some number up".  Weights are summed in
// fixed point, so that no sum depends on the order of its terms.
//
// A row is shared by the CTAs of a cluster (up to 8), each with a slice; they exchange what they find
// through distributed shared memory.  The first pass takes the maximum, per thread and then of the row.
//   - A small top_k: the k-th largest of the threads' maxima is a lower bound of the k-th largest
//     logit, and only little more than k logits reach it.  They are collected, ranked against each
//     other, and the race is among them: two passes over the logits, none over the noise.
//   - Otherwise, with a top_k or top_p: a histogram over d = (l_max - l)/T (weights, and counts where
//     they matter) names the bin that the last token to stay is in; the bin's tokens, a few hundred as
//     a rule, are collected and ranked against each other.  A bin with more of them (equal logits, or the
//     tail beyond exp(-22)) is narrowed by further histograms over the ordering number itself.
//   - The last pass runs the race over what stays and reads the noise of those tokens alone.
//
// 192 rows of 128000 bf16 logits (147 MB with the noise, 22 us at the copy rate), GPU time with nothing in L2
// from the call before: greedy 20 us; top_k 50 43 us; no filter 54 us (the race: an exp2 and a reciprocal a token);
// top_p 0.9 152 us (three more passes, each waiting for L2 more than for its arithmetic); every row with settings of
// its own 86 us (greedy and top_k rows need little of the noise).  One row of 50257: 4.3, 9.8, 8.0 and 24 us, the
// passes' latency and the cluster's syncs.
// Measured (the same inputs call after call: top_p 146, settings of its own 74) and not taken: light tokens summed in registers instead of the histogram (146 to 161 us: the atomic
// adds are not what bounds the pass), numbers stored to the peers instead of loaded from them (top_p 2% faster,
// top_k 3% slower), the race over single tokens that pass the cut instead of whole packs (146 to 190 us).
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cstdint>

#include "../../include/selscan.h"
#include "device_common.cuh"
#include "host_util.h"

namespace selscan {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kCap = 1024;               // most tokens ranked against each other
constexpr int kIndexBits = 19;           // SS_SAMPLE_MAX
constexpr int kMaxSlice = 1 << 16;       // most tokens per CTA
static_assert(SS_SAMPLE_MAX <= kMaxCluster * kMaxSlice, "the largest row fits a cluster");
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
    uint32_t cluster;        // CTAs per row
    int slice;               // tokens per CTA (whole 16-byte runs)
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
    // (fmaxf passes over NaN)
    static __device__ __forceinline__ float largest(const float* q) {
        const float4 f = *reinterpret_cast<const float4*>(q);
        return fmaxf(fmaxf(fmaxf(f.x, f.y), fmaxf(f.z, f.w)), -INFINITY);
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
    static __device__ __forceinline__ float largest(const __nv_bfloat16* q) {
        const uint4 u = *reinterpret_cast<const uint4*>(q);
        const __nv_bfloat162 m = __hmax2(__hmax2(*reinterpret_cast<const __nv_bfloat162*>(&u.x), *reinterpret_cast<const __nv_bfloat162*>(&u.y)),
                                         __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&u.z), *reinterpret_cast<const __nv_bfloat162*>(&u.w)));
        const float2 f = __bfloat1622float2(m);
        return fmaxf(fmaxf(f.x, f.y), -INFINITY);
    }
};

// f(index, logit) for every token of the row: 16-byte loads between the first and the last
// 16-byte boundary of the row, single ones around them.  A thread's indexes increase.
template <typename T, typename F>
__device__ __forceinline__ void each_token(const T* row, int V, F&& f) {
    constexpr int W = Pack<T>::n;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    const int head = min(V, off ? W - off : 0);
    const int body = (V - head) / W;
    const int tail0 = head + body * W;
    if (static_cast<int>(threadIdx.x) < head) f(static_cast<int>(threadIdx.x), tidy(to_f32<T>(row[threadIdx.x])));
#pragma unroll 2
    for (int b = threadIdx.x; b < body; b += kThreads) {
        float v[W];
        Pack<T>::load(row + head + b * W, v);
#pragma unroll
        for (int j = 0; j < W; ++j) f(head + b * W + j, tidy(v[j]));
    }
    if (static_cast<int>(threadIdx.x) < V - tail0)
        f(tail0 + static_cast<int>(threadIdx.x), tidy(to_f32<T>(row[tail0 + threadIdx.x])));
}

// f(index, weight, noise) for every token that stays, in the order of each_token.  The noise of a pack is
// read as a whole where its alignment allows: with the logits, two packs at a time, where every token may
// stay (`eager`), else if one of its tokens does.
template <typename T, typename S, typename Wt, typename F>
__device__ __forceinline__ void each_token_and_noise(const T* row, const float* noise, int V, bool eager, S&& stays, Wt&& weight,
                                                     F&& f) {
    constexpr int W = Pack<T>::n;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    const int head = min(V, off ? W - off : 0);
    const int body = (V - head) / W;
    const int tail0 = head + body * W;
    const bool wide = (reinterpret_cast<uintptr_t>(noise + head) & 15u) == 0;
    auto one = [&](int i) {
        const float l = tidy(to_f32<T>(row[i])), w = weight(l);
        if (stays(i, l, w)) f(i, w, noise[i]);
    };
    auto load_noise = [&](int i, float (&e)[W]) {
        if (wide) {
#pragma unroll
            for (int j = 0; j < W; j += 4) Pack<float>::load(noise + i + j, e + j);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) e[j] = noise[i + j];
        }
    };
    if (static_cast<int>(threadIdx.x) < head) one(static_cast<int>(threadIdx.x));
    int b = threadIdx.x;
    if (eager)
        for (; b + kThreads < body; b += 2 * kThreads) {
            float v[2][W], e[2][W];
#pragma unroll
            for (int k = 0; k < 2; ++k) Pack<T>::load(row + head + (b + k * kThreads) * W, v[k]);
#pragma unroll
            for (int k = 0; k < 2; ++k) load_noise(head + (b + k * kThreads) * W, e[k]);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const int i = head + (b + k * kThreads) * W + j;
                    const float l = tidy(v[k][j]), w = weight(l);
                    if (stays(i, l, w)) f(i, w, e[k][j]);
                }
        }
    for (; b < body; b += kThreads) {
        const int i = head + b * W;
        float v[W], e[W];
        Pack<T>::load(row + i, v);
        bool on[W], any = false;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float l = tidy(v[j]);
            v[j] = weight(l);
            on[j] = stays(i + j, l, v[j]);
            any = any || on[j];
        }
        if (!any) continue;
        load_noise(i, e);
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (on[j]) f(i + j, v[j], e[j]);
    }
    if (static_cast<int>(threadIdx.x) < V - tail0) one(tail0 + static_cast<int>(threadIdx.x));
}

// f(index, logit) for every token whose logit is `bound` or more (not NaN).
template <typename T, typename F>
__device__ __forceinline__ void each_token_from(const T* row, int V, float bound, F&& f) {
    constexpr int W = Pack<T>::n;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    const int head = min(V, off ? W - off : 0);
    const int body = (V - head) / W;
    const int tail0 = head + body * W;
    auto one = [&](int i) {
        const float l = tidy(to_f32<T>(row[i]));
        if (l >= bound) f(i, l);
    };
    if (static_cast<int>(threadIdx.x) < head) one(static_cast<int>(threadIdx.x));
    if (static_cast<int>(threadIdx.x) < V - tail0) one(tail0 + static_cast<int>(threadIdx.x));
#pragma unroll 4
    for (int b = threadIdx.x; b < body; b += kThreads)
        if (Pack<T>::largest(row + head + b * W) >= bound)
            for (int j = 0; j < W; ++j) one(head + b * W + j);
}

// f(index of the pack's first token, the pack's largest logit) for every pack: the same tokens by the same
// threads as each_token's, in increasing order of the index for each of them but the tail.
template <typename T, typename F>
__device__ __forceinline__ void each_pack(const T* row, int V, F&& f) {
    constexpr int W = Pack<T>::n;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    const int head = min(V, off ? W - off : 0);
    const int body = (V - head) / W;
    const int tail0 = head + body * W;
    if (static_cast<int>(threadIdx.x) < head) f(static_cast<int>(threadIdx.x), tidy(to_f32<T>(row[threadIdx.x])));
#pragma unroll 4
    for (int b = threadIdx.x; b < body; b += kThreads) f(head + b * W, fminf(Pack<T>::largest(row + head + b * W), FLT_MAX));
    if (static_cast<int>(threadIdx.x) < V - tail0)
        f(tail0 + static_cast<int>(threadIdx.x), tidy(to_f32<T>(row[tail0 + threadIdx.x])));
}
// The ordering number of the first token from `at` on that has logit `best` (the pack at `at` has one).
template <typename T>
__device__ __forceinline__ uint64_t first_of_pack(const T* row, int V, int at, float best, int i0) {
    for (int j = at; j < V && j < at + Pack<T>::n; ++j)
        if (tidy(to_f32<T>(row[j])) == best) return order_of(best, i0 + j);
    return 0;
}

struct Shared {
    uint32_t count[kBins], lo[kBins], hi[kBins];   // a bin's tokens, and their mass as hi·2^16 + lo
    uint64_t mine[kCap];                           // tokens that this CTA has collected
    uint64_t cand[kCap];                           // those of the whole cluster, and their masses
    uint32_t cmass[kCap];
    uint64_t slot[2][kMaxCluster];                 // a number from every CTA
    uint64_t last[kMaxCluster];                    // and the last one, at the first CTA
    uint64_t warp64[kWarps];
    uint32_t warp32[kWarps];
    uint64_t mass_above;                           // of the bins before the found one
    uint32_t count_above, share_count;
    uint64_t share_mass;
    int bin;
    uint32_t ncand;                                // collected here
    uint64_t cut;
};

__device__ __forceinline__ uint32_t ld_peer_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t ld_peer_u64(uint32_t addr) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

// The largest of the block's numbers, for all its threads.
__device__ __forceinline__ uint64_t block_max(Shared& s, uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
        v = v > w ? v : w;
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) s.warp64[threadIdx.x / 32] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v = s.warp64[w] > v ? s.warp64[w] : v;
    return v;
}
// The cluster that has a row.  Every thread of every CTA makes the same calls in the same order.
struct Team {
    Shared& s;
    uint32_t rank, size;
    int turn;                                      // alternates between the two sets of slots
    __device__ __forceinline__ void sync() const {
        if (size > 1) cluster_sync_all();
        else __syncthreads();
    }
    // A CTA's shared memory may be touched by its peers once it is known to run: each says so as it begins
    // and waits for the others after its first pass, by when they have.
    __device__ __forceinline__ void begin() const {
        if (size > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    }
    __device__ __forceinline__ void begun() const {
        if (size > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    // The largest of the CTAs' numbers (the same for all threads of a CTA).
    __device__ __forceinline__ uint64_t max_over(uint64_t v) {
        if (size == 1) return v;
        turn ^= 1;
        if (threadIdx.x == 0) s.slot[turn][rank] = v;
        sync();
        for (uint32_t r = 0; r < size; ++r) {
            const uint64_t w = ld_peer_u64(peer_smem_addr(&s.slot[turn][r], r));
            v = w > v ? w : v;
        }
        return v;                                  // (the next use of these slots is two syncs away)
    }
};

__device__ __forceinline__ void clear_bins(Shared& s) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = s.lo[i] = s.hi[i] = 0u;
    __syncthreads();
}
__device__ __forceinline__ void add_to_bin(Shared& s, int bin, uint32_t mass, bool counted) {
    if (counted) atomicAdd(&s.count[bin], 1u);
    // halves of 16 bits, which kMaxSlice tokens do not carry out of; most weights have no upper half
    if (mass & 0xffffu) atomicAdd(&s.lo[bin], mass & 0xffffu);
    if (mass >> 16) atomicAdd(&s.hi[bin], mass >> 16);
}

// A thread's share of the bins over the cluster's histograms: kBins / size of them belong to each CTA, in
// order of the ranks, and EACH = 8 / size adjacent ones to a thread.  All loads are issued before the first
// sum: each is a trip to another SM.
constexpr int kBinsThread = kBins / kThreads;
struct Bins {
    uint32_t c[kBinsThread];
    uint64_t m[kBinsThread];
    int n, first;                                              // how many, and the first's number
};
template <int EACH>
__device__ __forceinline__ void load_share(const Team& team, Bins& h) {
    constexpr int SIZE = kBinsThread / EACH;
    Shared& s = team.s;
    h.n = EACH;
    h.first = (static_cast<int>(team.rank) * kThreads + static_cast<int>(threadIdx.x)) * EACH;
    uint32_t v[SIZE][EACH][3];
#pragma unroll
    for (int r = 0; r < SIZE; ++r) {
        const uint32_t pc = SIZE > 1 ? peer_smem_addr(&s.count[h.first], r) : smem_addr(&s.count[h.first]);
#pragma unroll
        for (int j = 0; j < EACH; ++j)
#pragma unroll
            for (int k = 0; k < 3; ++k) v[r][j][k] = ld_peer_u32(pc + 4 * j + k * static_cast<uint32_t>(sizeof(s.count)));
    }
#pragma unroll
    for (int j = 0; j < kBinsThread; ++j) {
        h.c[j] = 0u;
        h.m[j] = 0ull;
        if (j < EACH)
#pragma unroll
            for (int r = 0; r < SIZE; ++r) {
                h.c[j] += v[r][j < EACH ? j : 0][0];
                h.m[j] += (static_cast<uint64_t>(v[r][j < EACH ? j : 0][2]) << 16) + v[r][j < EACH ? j : 0][1];
            }
    }
}
__device__ __forceinline__ void load_bins(const Team& team, Bins& h) {
    if (team.size == 1) load_share<8>(team, h);
    else if (team.size == 2) load_share<4>(team, h);
    else if (team.size == 4) load_share<2>(team, h);
    else load_share<1>(team, h);
}

// Sums of the CTAs' shares, exchanged.  Histograms are complete when every CTA has called.  Returns the mass
// of all bins; `h` is this thread's share.
__device__ uint64_t sum_bins(Team& team, Bins& h) {
    Shared& s = team.s;
    team.sync();
    load_bins(team, h);
    uint32_t c = 0;
    uint64_t m = 0;
#pragma unroll
    for (int j = 0; j < kBinsThread; ++j) {
        c += h.c[j];
        m += h.m[j];
    }
    c = __reduce_add_sync(0xffffffffu, c);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) m += __shfl_xor_sync(0xffffffffu, m, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) {
        s.warp32[threadIdx.x / 32] = c;
        s.warp64[threadIdx.x / 32] = m;
    }
    __syncthreads();
    c = 0;
    m = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        c += s.warp32[w];
        m += s.warp64[w];
    }
    if (threadIdx.x == 0) {
        s.share_count = c;
        s.share_mass = m;
    }
    team.sync();
    uint64_t all = 0;
    for (uint32_t r = 0; r < team.size; ++r)
        all += team.size > 1 ? ld_peer_u64(peer_smem_addr(&s.share_mass, r)) : s.share_mass;
    return all;
}

// After sum_bins: the first bin at which the running count, begun at `count`, reaches `k` (by_mass false),
// or the running mass, begun at `mass`, reaches `target` (by_mass true); the last bin if none does.  Leaves
// it in s.bin, with what is before it, in every CTA.  Histograms may be cleared after it.
__device__ void find_bin(Team& team, const Bins& h, bool by_mass, uint32_t k, uint64_t target, uint32_t count, uint64_t mass) {
    Shared& s = team.s;
    // the CTA whose share it is in
    uint32_t owner = 0;
    for (; owner < team.size; ++owner) {
        const uint32_t c = team.size > 1 ? ld_peer_u32(peer_smem_addr(&s.share_count, owner)) : s.share_count;
        const uint64_t m = team.size > 1 ? ld_peer_u64(peer_smem_addr(&s.share_mass, owner)) : s.share_mass;
        if (owner == team.size - 1 || (by_mass ? mass + m >= target : count + c >= k)) break;
        count += c;
        mass += m;
    }
    if (owner == team.rank) {
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
        uint32_t ci = 0;
        uint64_t mi = 0;
#pragma unroll
        for (int j = 0; j < kBinsThread; ++j) {
            ci += h.c[j];
            mi += h.m[j];
        }
        const uint32_t ct = ci;
        const uint64_t mt = mi;
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
        if (threadIdx.x == 0) s.bin = kBins;
        if (lane == 31) {
            s.warp32[warp] = ci;
            s.warp64[warp] = mi;
        }
        __syncthreads();
        for (int w = 0; w < warp; ++w) {
            count += s.warp32[w];
            mass += s.warp64[w];
        }
        uint32_t cb = count + ci - ct, c_at = 0;                 // before this thread's bins
        uint64_t mb = mass + mi - mt, m_at = 0;
        int mine = kBins;
#pragma unroll
        for (int j = 0; j < kBinsThread; ++j) {
            const bool end = threadIdx.x == kThreads - 1 && j == h.n - 1;
            if (mine == kBins && j < h.n && (end || (by_mass ? mb + h.m[j] >= target : cb + h.c[j] >= k))) {
                mine = h.first + j;
                c_at = cb;
                m_at = mb;
            }
            cb += h.c[j];
            mb += h.m[j];
        }
        if (mine < kBins) atomicMin(&s.bin, mine);
        __syncthreads();
        if (mine < kBins && s.bin == mine) {
            s.count_above = c_at;
            s.mass_above = m_at;
        }
    }
    team.sync();
    if (owner != team.rank && threadIdx.x == 0) {
        s.bin = static_cast<int>(ld_peer_u32(peer_smem_addr(&s.bin, owner)));
        s.count_above = ld_peer_u32(peer_smem_addr(&s.count_above, owner));
        s.mass_above = ld_peer_u64(peer_smem_addr(&s.mass_above, owner));
    }
    team.sync();
}

// The number of tokens that the CTAs have collected, all of which are then in s.cand with their masses;
// more than kCap: too many.  (The cluster syncs before it collects again, or ends.)
template <typename M>
__device__ uint32_t gather(Team& team, M&& mass_of) {
    Shared& s = team.s;
    team.sync();
    uint32_t c[kMaxCluster], n = 0;
    bool fits = true;
#pragma unroll
    for (uint32_t r = 0; r < kMaxCluster; ++r)
        c[r] = r >= team.size ? 0u : team.size > 1 ? ld_peer_u32(peer_smem_addr(&s.ncand, r)) : s.ncand;
#pragma unroll
    for (uint32_t r = 0; r < kMaxCluster; ++r) {
        fits = fits && c[r] <= kCap;
        n += c[r];
    }
    if (!fits || n > kCap) return kCap + 1;
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
        uint32_t r = 0, at = i;
#pragma unroll
        for (uint32_t q = 0; q < kMaxCluster - 1; ++q)
            if (r == q && at >= c[q]) {
                at -= c[q];
                r = q + 1;
            }
        const uint64_t o = ld_peer_u64(team.size > 1 ? peer_smem_addr(&s.mine[at], r) : smem_addr(&s.mine[at]));
        s.cand[i] = o;
        s.cmass[i] = mass_of(logit_of(o));
    }
    __syncthreads();
    return n;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(const SampleParams p) {
    __shared__ Shared s;
    Team team{s, 0u, p.cluster, 0};
    if (p.cluster > 1) team.rank = cluster_ctarank();
    team.begin();
    const int64_t r = blockIdx.x / p.cluster;
    const float* noise = p.noise + r * p.noise_r;
    const int V = p.V, i0 = min(V, static_cast<int>(team.rank) * p.slice), n_slice = min(V - i0, p.slice);
    const T* slice = static_cast<const T*>(p.logits) + r * p.logits_r + i0;

    // the row's largest logit, and the first of its indexes; each thread's own for the bound of top_k
    uint64_t own = 0;
    {
        float best = -INFINITY;
        int at = -1;
        each_pack(slice, n_slice, [&](int i, float l) {
            if (l > best) {
                best = l;
                at = i;
            }
        });
        if (at >= 0) own = first_of_pack(slice, n_slice, at, best, i0);
    }
    __syncwarp();                                              // (the barrier takes whole warps)
    team.begun();
    const float temp = p.temperature ? p.temperature[r] : 1.f;
    const float mp = p.min_p ? p.min_p[r] : 0.f;
    const int k = p.top_k && p.top_k[r] > 0 && p.top_k[r] < V ? p.top_k[r] : V;
    const bool first_only = temp <= 0.f || !(mp <= 1.f);       // greedy, or no weight reaches min_p
    const bool small_k = !first_only && k <= static_cast<int>(team.size * kThreads) / 2 && k <= kCap / 2;
    float lmax;
    float tops[kMaxCluster];                                   // maxima of this thread's namesakes in all CTAs
    if (small_k) {
        // every thread's maximum, everywhere (in the place of the counts, which this path does not need)
        static_assert(kMaxCluster * kThreads <= kBins, "a count's place for every thread");
        const float mine = own ? logit_of(own) : -INFINITY;
        if (team.size > 1) {
            for (uint32_t q = 0; q < team.size; ++q)
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer_smem_addr(&s.count[team.rank * kThreads + threadIdx.x], q)),
                             "f"(mine) : "memory");
        } else {
            s.count[threadIdx.x] = __float_as_uint(mine);
        }
        team.sync();
        lmax = -INFINITY;
#pragma unroll
        for (uint32_t q = 0; q < kMaxCluster; ++q) {
            tops[q] = q < team.size ? __uint_as_float(s.count[q * kThreads + threadIdx.x]) : -INFINITY;
            lmax = fmaxf(lmax, tops[q]);
        }
        const uint64_t top = block_max(s, lmax > -INFINITY ? order_of(lmax, 0) : 0ull);
        lmax = top ? logit_of(top) : -INFINITY;
    } else {
        const uint64_t top = team.max_over(block_max(s, own));
        lmax = top ? logit_of(top) : -INFINITY;
        if (first_only && top != 0) {
            if (team.rank == 0 && threadIdx.x == 0) p.tokens[r] = index_of(top);
            team.sync();                                       // (a peer may still read this CTA's slots)
            return;
        }
    }
    if (lmax == -INFINITY) {                                   // nothing there
        if (team.rank == 0 && threadIdx.x == 0) p.tokens[r] = -1;
        team.sync();
        return;
    }
    const float inv_t = fminf(1.f / (temp > 0.f ? temp : 1.f), 1e35f);   // finite times any reach
    const float c2 = inv_t * kLog2e;
    const float tp = p.top_p && p.top_p[r] < 1.f ? p.top_p[r] : 2.f;
    const uint64_t all = ~0ull;

    // top_p of a mass, rounded up and at least 1 (the first token stays), in whole numbers: doubles are slow here
    const uint64_t tq = tp > 0.f && tp < 1.f ? static_cast<uint64_t>(tp * 18446744073709551616.f) : 0ull;      // exact
    auto share_of = [&](uint64_t mass) {
        const uint64_t v = __umul64hi(mass, tq) + (mass * tq != 0 ? 1 : 0);
        return v > 0 ? v : static_cast<uint64_t>(1);
    };
    auto weight = [&](float l) { return l == -INFINITY ? 0.f : ex2((l - lmax) * c2); };
    const float per_bin = inv_t * (kBins / kReach);
    // (rounded by adding 2^23: monotone in l, and cheaper than a conversion)
    auto bin_of = [&](float l) { return __float_as_int(fminf((lmax - l) * per_bin, kBins - 1.f) + 8388608.f) & (kBins - 1); };
    auto mass_of = [&](float l) { return __float2uint_rn(weight(l) * kMassOne); };
    auto race = [&](float e, float w) {                        // the race's key, larger is better; NaN as 0
        const float key = w * rcp_approx(e);
        return key >= 0.f ? key : 0.f;
    };
    auto numbered = [&](float key, int i) {                    // the lower index among equals
        return static_cast<uint64_t>(__float_as_uint(key)) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
    };
    // the best of the CTAs' best, at the first of them (peers may read this CTA's memory up to that sync)
    auto finish = [&](uint64_t best) {
        best = block_max(s, best);
        if (threadIdx.x == 0) {
            if (team.size > 1)
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(peer_smem_addr(&s.last[team.rank], 0)), "l"(best) : "memory");
            else
                s.last[0] = best;
        }
        team.sync();
        if (team.rank == 0 && threadIdx.x == 0) {
            for (uint32_t q = 0; q < team.size; ++q) best = s.last[q] > best ? s.last[q] : best;
            p.tokens[r] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(best));
        }
    };
    auto keep = [&](float l, int i) {
        const uint32_t at = atomicAdd(&s.ncand, 1u);
        if (at < kCap) s.mine[at] = order_of(l, i);
    };
    auto start_collecting = [&](bool again) {                 // again: peers may still read the last list
        if (again) team.sync();
        __syncthreads();
        if (threadIdx.x == 0) s.ncand = 0u;
        __syncthreads();
    };
    // rank of collected token i: how many come before it, and their mass
    auto rank = [&](int n, uint64_t o, uint32_t& c, uint64_t& m) {
        for (int j = 0; j < n; ++j)
            if (s.cand[j] > o) {
                ++c;
                m += s.cmass[j];
            }
    };

    if (small_k) {
        // A bound that at least k of the maxima reach, and not many more: down from the largest logit by
        // doubled steps, then by halves.  Where that does not get there, all logits are collected.
        auto reach = [&](float t) {
            uint32_t c = 0;
#pragma unroll
            for (uint32_t q = 0; q < kMaxCluster; ++q) c += tops[q] >= t ? 1u : 0u;
            c = __reduce_add_sync(0xffffffffu, c);
            __syncthreads();
            if (threadIdx.x % 32 == 0) s.warp32[threadIdx.x / 32] = c;
            __syncthreads();
            c = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) c += s.warp32[w];
            return static_cast<int>(c);
        };
        float bound = -FLT_MAX, near = 0.f, far = 1.f;         // distances from the largest: too few, enough
        int c = 0;
        for (; far < 1e30f; far *= 4.f) {
            c = reach(lmax - far);
            if (c >= k) break;
            near = far;
        }
        if (c >= k) {
            bound = lmax - far;
            for (int i = 0; i < 24 && c > k + 64; ++i) {
                const float mid = 0.5f * (near + far);
                const int n = reach(lmax - mid);
                if (n >= k) {
                    far = mid;
                    c = n;
                    bound = lmax - mid;
                } else {
                    near = mid;
                }
            }
        }
        start_collecting(false);
        each_token_from(slice, n_slice, bound, [&](int i, float l) { keep(l, i0 + i); });
        const int n = static_cast<int>(gather(team, mass_of));
        if (n <= kCap) {
            // every CTA ranks a share of them
            const int at = static_cast<int>(team.rank * kThreads + threadIdx.x), step = static_cast<int>(team.size * kThreads);
            const int mine_n = (n + step - 1) / step;            // at most 4
            uint32_t c[4];
            uint64_t m[4], sum = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                c[q] = 0;
                m[q] = 0;
                const int i = at + q * step;
                if (q < mine_n && i < n) rank(n, s.cand[i], c[q], m[q]);
                if (q < mine_n && i < n && c[q] < static_cast<uint32_t>(k)) sum = max(sum, m[q] + s.cmass[i]);
            }
            // the mass of the first k: up to and with the last of them
            uint64_t target = all;
            if (tp < 2.f) target = share_of(team.max_over(block_max(s, sum)));
            uint64_t best = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = at + q * step;
                if (q < mine_n && i < n && c[q] < static_cast<uint32_t>(k) && m[q] < target) {
                    const float w = weight(logit_of(s.cand[i]));
                    const uint64_t v = numbered(race(noise[index_of(s.cand[i])], w), index_of(s.cand[i]));
                    if (w >= mp) best = v > best ? v : best;
                }
            }
            finish(best);
            return;
        }
    }

    // What stays: bins before `bin`, and in it the tokens whose number is at least `cut`.
    int bin = kBins;
    uint64_t cut = 0;
    if (k < V || tp < 2.f) {
        // Collects the tokens of bin `b` that hold the k-th token (by_mass false) or the one at which the mass
        // reaches `target`, narrowing while there are more than kCap of them; `count` and `mass` become those
        // of the tokens above the collected ones.  Returns how many there are.
        bool narrowed = false;
        auto collect = [&](int b, bool by_mass, uint32_t kk, uint64_t target, uint32_t& count, uint64_t& mass) {
            uint64_t lo = 0;
            int bits = kOrderBits;                             // candidates: numbers lo .. lo + 2^bits - 1
            for (;;) {
                start_collecting(true);
                each_token(slice, n_slice, [&](int i, float l) {
                    if (bin_of(l) == b && (order_of(l, i0 + i) - lo) >> bits == 0) keep(l, i0 + i);
                });
                const uint32_t n = gather(team, mass_of);
                if (n <= kCap) return static_cast<int>(n);
                const int shift = bits > 11 ? bits - 11 : 0;
                narrowed = true;
                clear_bins(s);
                each_token(slice, n_slice, [&](int i, float l) {
                    if (bin_of(l) != b) return;
                    const uint64_t o = order_of(l, i0 + i) - lo;
                    if (o >> bits) return;
                    add_to_bin(s, kBins - 1 - static_cast<int>(o >> shift), mass_of(l), true);
                });
                Bins h;
                sum_bins(team, h);
                find_bin(team, h, by_mass, kk, target, count, mass);
                count = s.count_above;
                mass = s.mass_above;
                lo += static_cast<uint64_t>(kBins - 1 - s.bin) << shift;
                bits = shift;
            }
        };
        // Over the n collected tokens, with `count` and `mass` above them: the smallest number whose token is
        // among the first kk and has less than `target` above it.
        auto smallest_kept = [&](int n, uint32_t kk, uint64_t target, uint32_t count, uint64_t mass, uint64_t* kept_mass) {
            __syncthreads();
            if (threadIdx.x == 0) s.cut = ~0ull;
            __syncthreads();
            uint64_t sum = 0;
            for (int i = threadIdx.x; i < n; i += kThreads) {
                uint32_t c = count;
                uint64_t m = mass;
                rank(n, s.cand[i], c, m);
                if (c < kk && m < target) {
                    atomicMin(reinterpret_cast<unsigned long long*>(&s.cut), s.cand[i]);
                    sum = max(sum, m + s.cmass[i]);              // largest at the smallest number
                }
            }
            sum = block_max(s, sum);
            if (kept_mass) *kept_mass = sum;
            __syncthreads();
            return s.cut;
        };
        auto histogram = [&](bool counted) {
            clear_bins(s);
            each_token(slice, n_slice, [&](int, float l) { add_to_bin(s, bin_of(l), mass_of(l), counted); });
        };

        uint32_t count = 0;
        uint64_t mass = 0;
        int n = 0;
        uint64_t target = all;                                   // never below 1: the first token stays
        team.sync();
        histogram(k < V);
        Bins h;
        const uint64_t whole = sum_bins(team, h);
        if (k < V) {
            find_bin(team, h, false, k, 0ull, 0u, 0ull);
            bin = s.bin;
            count = s.count_above;
            mass = s.mass_above;
            uint64_t kept = mass;
            n = collect(bin, false, k, 0ull, count, mass);
            cut = smallest_kept(n, k, all, count, mass, &kept);
            if (tp < 2.f) target = share_of(kept);
        } else {
            target = share_of(whole);
        }
        if (tp < 2.f) {
            const int kbin = bin;
            if (narrowed) {                                    // the bins hold something else by now
                histogram(k < V);
                sum_bins(team, h);
            } else if (k < V) {
                load_bins(team, h);
            }
            find_bin(team, h, true, 0u, target, 0u, 0ull);
            const int b = s.bin;
            if (b < kbin) {
                bin = b;
                count = s.count_above;
                mass = s.mass_above;
                n = collect(b, true, 0u, target, count, mass);
                cut = smallest_kept(n, V, target, count, mass, nullptr);
            } else if (narrowed) {                             // the same bin, but elsewhere in it
                find_bin(team, h, false, k, 0ull, 0u, 0ull);
                count = s.count_above;
                mass = s.mass_above;
                n = collect(kbin, true, 0u, target, count, mass);
                const uint64_t pcut = smallest_kept(n, V, target, count, mass, nullptr);
                cut = pcut > cut ? pcut : cut;
            } else {
                cut = smallest_kept(n, k, target, count, mass, nullptr);
            }
        }
    }

    float best = -1.f;
    int at = 0;
    auto stays = [&](int i, float l, float w) {
        const int b = bin < kBins ? bin_of(l) : 0;
        return !(b > bin || (b == bin && order_of(l, i0 + i) < cut)) && w >= mp;
    };
    each_token_and_noise(slice, noise + i0, n_slice, bin == kBins && mp <= 0.f, stays, weight, [&](int i, float w, float e) {
        const float key = race(e, w);
        if (key > best) {                                      // (a thread's indexes increase)
            best = key;
            at = i;
        }
    });
    finish(best >= 0.f ? numbered(best, i0 + at) : 0ull);
}

template <typename T>
cudaError_t launch_sample(const SampleParams& p, int64_t rows, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * p.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T>, p);
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
    // as many CTAs to a row as keep at least 2048 tokens each, up to six to an SM over all rows: a row's
    // passes take as long as its slices (one row of 50257: 38 us with one CTA of 1024 threads).  Four to an SM run
    // at once; with no more than those (the same inputs call after call) 192 rows of 128000 take 135 instead of 146 us if all have a top_p, but 96
    // instead of 74 if every row has settings of its own, when the longest rows are what the call waits for.
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return SS_ERR_CUDA;
    int cluster = 1;
    while (cluster < kMaxCluster && (V > cluster * static_cast<int64_t>(kMaxSlice) ||
                                     (V / (2 * cluster) >= 2048 && rows * 2 * cluster <= 6 * static_cast<int64_t>(sms))))
        cluster *= 2;
    const int slice = static_cast<int>(((V + cluster - 1) / cluster + 7) / 8 * 8);
    const SampleParams p{logits, noise, temperature, top_k, top_p, min_p, tokens, logits_r, noise_r, static_cast<int>(V),
                         static_cast<uint32_t>(cluster), slice};
    if (rows * cluster > INT32_MAX) return SS_ERR_UNSUPPORTED;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    const cudaError_t e = io_dtype == SS_BF16 ? launch_sample<__nv_bfloat16>(p, rows, stream) : launch_sample<float>(p, rows, stream);
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}
