// Device helpers of the multi-head scan's kernels.
#pragma once

#include "device_common.cuh"
#include "heads_params.h"

namespace selscan {

// Error bit beside those of device_common.cuh: a slot or row range in device memory is out of range (its
// sequence is skipped).
constexpr unsigned int kErrIndex = 4u;

// Where a sequence's rows and its cached state are.
struct HeadsSeq {
    int64_t row0;       // first row of xbc
    int len;            // rows
    int slot;           // < 0: none
    bool warm;          // starts from the slot's contents (else from zeros)
    bool ok;            // indexes in range (else the sequence is skipped)
};

__device__ __forceinline__ HeadsSeq heads_seq(const HeadsParams& p, int seq) {
    HeadsSeq s;
    const int64_t a = p.cu[seq], b = p.cu[seq + 1];
    s.slot = p.slots ? p.slots[seq] : seq;
    s.ok = a >= 0 && b >= a && b <= p.tokens && s.slot < p.n_slots;
    s.row0 = a;
    s.len = static_cast<int>(b - a);
    s.warm = s.slot >= 0 && !(p.fresh && p.fresh[seq] != 0);
    return s;
}

// The three samples of channel c before a sequence's first row.
struct HeadsWindow {
    float v[kHeadsConv - 1];
};
__device__ __forceinline__ HeadsWindow heads_window(const HeadsParams& p, const HeadsSeq& s, int c) {
    HeadsWindow w = {{0.f, 0.f, 0.f}};
    if (s.warm) {
        const float* q = p.window + (static_cast<int64_t>(s.slot) * p.C + c) * 3;
        w.v[0] = q[0];
        w.v[1] = q[1];
        w.v[2] = q[2];
    }
    return w;
}

// Sample t (may be negative: from the window) of channel c of a sequence.
template <typename TIO>
__device__ __forceinline__ float heads_sample(const HeadsParams& p, const HeadsSeq& s, const HeadsWindow& w, int c, int t) {
    if (t >= 0) return to_f32<TIO>(static_cast<const TIO*>(p.xbc)[(s.row0 + t) * p.xbc_t + c]);
    return t == -1 ? w.v[2] : t == -2 ? w.v[1] : w.v[0];
}

// Leaves the last three samples of channel c in its slot's window: the slot's old ones are read
// before any is written, so the thread that calls this owns the channel's window.
template <typename TIO>
__device__ __forceinline__ void heads_keep_window(const HeadsParams& p, const HeadsSeq& s, int c) {
    const HeadsWindow w = heads_window(p, s, c);
    const float a = heads_sample<TIO>(p, s, w, c, s.len - 3), b = heads_sample<TIO>(p, s, w, c, s.len - 2),
                d = heads_sample<TIO>(p, s, w, c, s.len - 1);
    float* q = p.window + (static_cast<int64_t>(s.slot) * p.C + c) * 3;
    q[0] = a;
    q[1] = b;
    q[2] = d;
}

__device__ __forceinline__ float heads_conv(const float w[4], float b, float e0, float e1, float e2, float e3) {
    return silu(fmaf(w[3], e3, fmaf(w[2], e2, fmaf(w[1], e1, fmaf(w[0], e0, b)))));
}

// heads_conv of two channels; w[k] their weights of sample k.
__device__ __forceinline__ float2 heads_conv2(const float2 w[4], float2 b, float2 e0, float2 e1, float2 e2, float2 e3) {
    return silu2(fma2(w[3], e3, fma2(w[2], e2, fma2(w[1], e1, fma2(w[0], e0, b)))));
}

// Sum over the block's threads before this one, and over all of them.
__device__ __forceinline__ int block_prefix(int v, int* total, int* scratch) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) before += scratch[w];
        all += scratch[w];
    }
    *total = all;
    return before + x - v;
}

// Sequences lie one behind the other: one that starts below an earlier entry of cu_seqlens is skipped.  So no
// row belongs to two of them, and there are no more chunks and segments than the workspace was planned for.
// For blockDim.x adjacent sequences at a time, from the first on, by all threads: whether this thread's
// sequence starts at or behind every entry before its own; `largest` (0 at first) is what carries over.
__device__ __forceinline__ bool heads_in_order(const HeadsParams& p, int seq, int& largest, int* scratch) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int start = seq < p.n_seq ? p.cu[seq] : 0;
    int x = start;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x = max(x, y);
    }
    int before = __shfl_up_sync(0xffffffffu, x, 1);
    before = lane == 0 ? largest : max(before, largest);
    __syncthreads();
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    for (int w = 0; w < warps; ++w) {
        if (w < warp) before = max(before, scratch[w]);
        largest = max(largest, scratch[w]);
    }
    return start >= before;
}

// The heads of a group share its B and C channels.  Each CTA that reads their windows says so on the
// group's counter once all its threads have (behind a barrier), and the one that finds itself the last
// may overwrite them; it puts the counter back to zero.
__device__ __forceinline__ unsigned int heads_say_read(unsigned int* counter) {
    unsigned int before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    return before;
}

}  // namespace selscan
