// Parameters of the multi-head scan's kernels (ss_heads_fwd.cu, ss_heads_step.cu) and the host
// checks that the two entry points share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/selscan.h"
#include "host_util.h"

namespace selscan {

constexpr int kHeadsConv = SS_CONV_WIDTH;      // samples under the convolution's kernel

struct HeadsParams {
    const void* xbc;        // [tokens, C]
    const void* dt_raw;     // [tokens, H]
    const void* z;          // [tokens, H·P] or nullptr
    void* y;                // [tokens, H·P]
    const float* conv_w;    // [C, 4]
    const float* conv_b;    // [C] or nullptr
    const float* dt_bias;   // [H] or nullptr
    const float* A_log;     // [H]
    const float* D;         // [H] or nullptr
    float* state;           // [n_slots, H, P, N]
    float* window;          // [n_slots, C, 3]
    const int32_t* cu;      // [n_seq + 1] (prompts)
    const int32_t* slots;   // [n_seq] or nullptr
    const int32_t* fresh;   // [n_seq] or nullptr (prompts)
    unsigned int* arrivals; // [n_seq, G], zero between calls
    unsigned int* err;
    int64_t xbc_t, dt_t, z_t, y_t;
    int64_t tokens;
    int n_seq, H, P, G, N, C, n_slots;
};

// The counters of the B and C windows' readers (one per sequence and group) are at the front of every
// workspace, in a part that nothing else uses, so that they are zero between calls of any sizes.
// Calls with more of them than that part holds clear theirs, behind it.
constexpr int64_t kHeadsCounters = 16384;
constexpr size_t kHeadsCounterBytes = kHeadsCounters * 4;

namespace host {

inline size_t heads_counter_bytes(int64_t n_seq, int64_t G) {
    const int64_t n = n_seq * G;
    return kHeadsCounterBytes + (n > kHeadsCounters ? (static_cast<size_t>(n) * 4 + 255) / 256 * 256 : 0);
}
inline cudaError_t heads_counters(HeadsParams& p, void* workspace, cudaStream_t stream) {
    const int64_t n = static_cast<int64_t>(p.n_seq) * p.G;
    p.arrivals = static_cast<unsigned int*>(workspace);
    if (n <= kHeadsCounters) return cudaSuccess;
    p.arrivals += kHeadsCounters;
    return cudaMemsetAsync(p.arrivals, 0, static_cast<size_t>(n) * 4, stream);
}

// Checks what ss_heads_fwd and ss_heads_step share and fills p (without cu, fresh, arrivals).
// `idle` is set when there is nothing to do.
ss_status heads_check(HeadsParams& p, const ss_heads_strides* strides, const void* xbc, const void* dt_raw, const void* z,
                      const float* conv_w, const float* conv_b, const float* dt_bias, const float* A_log, const float* D,
                      void* y, float* state, float* window, const int32_t* cu, const int32_t* slots, const int32_t* fresh,
                      int64_t n_seq, int64_t tokens, int64_t H, int64_t P, int64_t G, int64_t N, int64_t n_slots,
                      const void* workspace, size_t workspace_bytes, size_t need, bool* bf16, bool* idle);

}  // namespace host
}  // namespace selscan
