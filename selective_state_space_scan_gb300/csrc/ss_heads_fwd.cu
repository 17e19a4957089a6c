// Multi-head selective scan with its causal convolution, over packed prompts.
//
// Per head and token: S <- a·S + (Δ·x) ⊗ B (P × N), y = S·C + D·x, gated by silu(z), where x, B
// and C come out of a width-4 causal convolution and a SiLU.
//
// heads_seq_kernel walks the tokens in order, the recurrence as it is written.  A CTA has 16 rows
// of one head's state of one sequence, a warp 4 of them with its 32 lanes along N, all in
// registers; 16 tokens at a time the CTA convolves its x channels and the group's B and C into
// shared memory, then every warp takes the tokens one by one.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/selscan.h"
#include "heads_device.cuh"
#include "heads_params.h"
#include "heads_tc.h"
#include "internal.h"

namespace selscan {
namespace {

constexpr int kSeqThreads = 128;
constexpr int kSeqRowsWarp = 4;
constexpr int kSeqRows = kSeqRowsWarp * kSeqThreads / 32;   // rows of the state per CTA
constexpr int kSeqT = 16;                                   // tokens per round

template <typename TIO, int NL>
__global__ void __launch_bounds__(kSeqThreads) heads_seq_kernel(const HeadsParams p) {
    constexpr int NP = 32 * NL;
    __shared__ float sB[kSeqT][NP], sC[kSeqT][NP], sx[kSeqT][kSeqRows], sy[kSeqT][kSeqRows], sdt[kSeqT], sa[kSeqT];
    const int tiles = (p.P + kSeqRows - 1) / kSeqRows;
    int id = blockIdx.x;
    const int pt = id % tiles;
    id /= tiles;
    const int h = id % p.H, seq = id / p.H;
    const HeadsSeq s = heads_seq(p, seq);
    if (!s.ok) {
        if (h == 0 && pt == 0 && threadIdx.x == 0 && p.err) atomicOr(p.err, kErrIndex);
        return;
    }
    const int g = h / (p.H / p.G), warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int p0 = pt * kSeqRows, np = min(kSeqRows, p.P - p0);
    const int cx = h * p.P + p0, cb = p.H * p.P + g * p.N, cc = cb + p.G * p.N;
    const float A2 = -expf(p.A_log[h]) * kLog2e, bias = p.dt_bias ? p.dt_bias[h] : 0.f, Dh = p.D ? p.D[h] : 0.f;
    float* Sg = p.state + ((static_cast<int64_t>(max(s.slot, 0)) * p.H + h) * p.P + p0) * p.N;

    float S[kSeqRowsWarp][NL];
#pragma unroll
    for (int r = 0; r < kSeqRowsWarp; ++r)
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int row = warp * kSeqRowsWarp + r, n = lane + 32 * j;
            S[r][j] = (s.warm && row < np && n < p.N) ? Sg[static_cast<int64_t>(row) * p.N + n] : 0.f;
        }

    for (int t0 = 0; t0 < s.len; t0 += kSeqT) {
        const int nt = min(kSeqT, s.len - t0);
        // x, B and C of the round's tokens; lanes past np and N hold zeros
        for (int i = threadIdx.x; i < kSeqRows + 2 * NP; i += kSeqThreads) {
            float* dst = i < kSeqRows ? &sx[0][i] : i < kSeqRows + NP ? &sB[0][i - kSeqRows] : &sC[0][i - kSeqRows - NP];
            const int pitch = i < kSeqRows ? kSeqRows : NP;
            const int k = i < kSeqRows ? i : (i - kSeqRows) % NP;
            const bool on = i < kSeqRows ? k < np : k < p.N;
            const int c = i < kSeqRows ? cx + k : i < kSeqRows + NP ? cb + k : cc + k;
            if (!on) {
                for (int t = 0; t < nt; ++t) dst[t * pitch] = 0.f;
                continue;
            }
            const float* w = p.conv_w + static_cast<int64_t>(c) * 4;
            const float wk[4] = {w[0], w[1], w[2], w[3]}, b = p.conv_b ? p.conv_b[c] : 0.f;
            HeadsWindow win = {{0.f, 0.f, 0.f}};
            if (t0 < 3) win = heads_window(p, s, c);
            float e0 = heads_sample<TIO>(p, s, win, c, t0 - 3), e1 = heads_sample<TIO>(p, s, win, c, t0 - 2),
                  e2 = heads_sample<TIO>(p, s, win, c, t0 - 1);
#pragma unroll 4
            for (int t = 0; t < nt; ++t) {
                const float e3 = heads_sample<TIO>(p, s, win, c, t0 + t);
                dst[t * pitch] = heads_conv(wk, b, e0, e1, e2, e3);
                e0 = e1;
                e1 = e2;
                e2 = e3;
            }
        }
        if (threadIdx.x < nt) {
            const float r = to_f32<TIO>(static_cast<const TIO*>(p.dt_raw)[(s.row0 + t0 + threadIdx.x) * p.dt_t + h]);
            const float dt = softplus(r + bias);
            sdt[threadIdx.x] = dt;
            sa[threadIdx.x] = ex2(dt * A2);
        }
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            const float a = sa[t], dt = sdt[t];
            float acc[kSeqRowsWarp];
#pragma unroll
            for (int r = 0; r < kSeqRowsWarp; ++r) acc[r] = 0.f;
            float dx[kSeqRowsWarp];
#pragma unroll
            for (int r = 0; r < kSeqRowsWarp; ++r) dx[r] = dt * sx[t][warp * kSeqRowsWarp + r];
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                const float B = sB[t][lane + 32 * j], C = sC[t][lane + 32 * j];
#pragma unroll
                for (int r = 0; r < kSeqRowsWarp; ++r) {
                    S[r][j] = fmaf(a, S[r][j], dx[r] * B);
                    acc[r] = fmaf(S[r][j], C, acc[r]);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o /= 2)
#pragma unroll
                for (int r = 0; r < kSeqRowsWarp; ++r) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
            if (lane == 0)
#pragma unroll
                for (int r = 0; r < kSeqRowsWarp; ++r) sy[t][warp * kSeqRowsWarp + r] = acc[r];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < nt * kSeqRows; i += kSeqThreads) {
            const int t = i / kSeqRows, k = i % kSeqRows;
            if (k < np) {
                const int64_t row = s.row0 + t0 + t;
                float v = fmaf(Dh, sx[t][k], sy[t][k]);
                if (p.z) v *= silu(to_f32<TIO>(static_cast<const TIO*>(p.z)[row * p.z_t + cx + k]));
                static_cast<TIO*>(p.y)[row * p.y_t + cx + k] = from_f32<TIO>(v);
            }
        }
        __syncthreads();
    }
    if (s.slot < 0) return;
#pragma unroll
    for (int r = 0; r < kSeqRowsWarp; ++r)
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int row = warp * kSeqRowsWarp + r, n = lane + 32 * j;
            if (row < np && n < p.N) Sg[static_cast<int64_t>(row) * p.N + n] = S[r][j];
        }
    for (int k = threadIdx.x; k < np; k += kSeqThreads) heads_keep_window<TIO>(p, s, cx + k);
    if (heads_last_reader(p.arrivals + static_cast<int64_t>(seq) * p.G + g, (p.H / p.G) * tiles))
        for (int k = threadIdx.x; k < 2 * p.N; k += kSeqThreads)
            heads_keep_window<TIO>(p, s, k < p.N ? cb + k : cc + k - p.N);
}

template <typename TIO>
cudaError_t launch_seq(const HeadsParams& p, cudaStream_t stream) {
    const int64_t blocks = static_cast<int64_t>(p.n_seq) * p.H * ((p.P + kSeqRows - 1) / kSeqRows);
    const unsigned grid = static_cast<unsigned>(blocks);
    if (p.N <= 32) heads_seq_kernel<TIO, 1><<<grid, kSeqThreads, 0, stream>>>(p);
    else if (p.N <= 64) heads_seq_kernel<TIO, 2><<<grid, kSeqThreads, 0, stream>>>(p);
    else if (p.N <= 128) heads_seq_kernel<TIO, 4><<<grid, kSeqThreads, 0, stream>>>(p);
    else heads_seq_kernel<TIO, 8><<<grid, kSeqThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

namespace host {

ss_status heads_check(HeadsParams& p, const ss_heads_strides* strides, const void* xbc, const void* dt_raw, const void* z,
                      const float* conv_w, const float* conv_b, const float* dt_bias, const float* A_log, const float* D,
                      void* y, float* state, float* window, const int32_t* cu, const int32_t* slots, const int32_t* fresh,
                      int64_t n_seq, int64_t tokens, int64_t H, int64_t P, int64_t G, int64_t N, int64_t n_slots,
                      const void* workspace, size_t workspace_bytes, size_t need, bool* bf16, bool* idle) {
    *idle = false;
    if (n_seq < 0 || tokens < 0 || H < 0 || G < 0 || n_slots < 0) return SS_ERR_INVALID_ARG;
    if (P < 1 || P > SS_HEADS_MAX || N < 1 || N > SS_HEADS_MAX) return SS_ERR_UNSUPPORTED;
    if (H > 0 && (G < 1 || H % G != 0)) return SS_ERR_INVALID_ARG;
    if (H > (1 << 20) || n_seq > INT32_MAX || n_slots > INT32_MAX || tokens > INT32_MAX) return SS_ERR_UNSUPPORTED;
    const int64_t C = H * P + 2 * G * N;
    ss_heads_strides st;
    if (strides) {
        st = *strides;
    } else {
        std::memset(&st, 0, sizeof(st));
        st.io_dtype = SS_F32;
        st.xbc_t = C;
        st.dt_t = H;
        st.z_t = st.y_t = H * P;
    }
    if (st.io_dtype != SS_F32 && st.io_dtype != SS_BF16) return SS_ERR_INVALID_ARG;
    if (n_seq == 0 || H == 0) {
        *idle = true;
        return SS_OK;
    }
    *bf16 = st.io_dtype == SS_BF16;
    const int64_t es = *bf16 ? 2 : 4;
    if (!conv_w || !A_log) return SS_ERR_INVALID_ARG;
    if (tokens > 0 && (!xbc || !dt_raw || !y)) return SS_ERR_INVALID_ARG;
    if (n_slots > 0 && (!state || !window)) return SS_ERR_INVALID_ARG;
    if (!slots && n_seq > n_slots) return SS_ERR_INVALID_ARG;
    if (st.xbc_t < 0 || st.dt_t < 0 || st.y_t < 0 || (z && st.z_t < 0)) return SS_ERR_INVALID_ARG;
    if (tokens > 1 && st.y_t < H * P) return SS_ERR_INVALID_ARG;      // y: one address for each element
    if (n_seq * H > INT32_MAX / P) return SS_ERR_UNSUPPORTED;         // the grid's limit
    const void* f4[] = {conv_w, conv_b, dt_bias, A_log, D, state, window, cu, slots, fresh};
    for (const void* q : f4)
        if (q && !is_aligned(q, 4)) return SS_ERR_MISALIGNED;
    const void* io[] = {xbc, dt_raw, z, y};
    for (const void* q : io)
        if (q && !is_aligned(q, es)) return SS_ERR_MISALIGNED;
    if (need) {
        if (!workspace || workspace_bytes < need) return SS_ERR_INVALID_ARG;
        if (!is_aligned(workspace, 256)) return SS_ERR_MISALIGNED;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SS_ERR_CUDA;
    for (const void* q : f4)
        if (q && !dev_ptr(q, dev)) return SS_ERR_INVALID_ARG;
    for (const void* q : io)
        if (q && !dev_ptr(q, dev)) return SS_ERR_INVALID_ARG;
    if (need && !dev_ptr(workspace, dev)) return SS_ERR_INVALID_ARG;
    // what is written meets nothing that is read, nor another output
    const Range out[] = {range3(y, 1, tokens, H * P, 0, st.y_t, es), range3(state, 1, n_slots, H * P * N, 0, H * P * N, 4),
                         range3(window, 1, n_slots, C * 3, 0, C * 3, 4), range3(workspace, 1, 1, need, 0, 0, 1)};
    const Range in[] = {range3(xbc, 1, tokens, C, 0, st.xbc_t, es), range3(dt_raw, 1, tokens, H, 0, st.dt_t, es),
                        range3(z, 1, tokens, H * P, 0, st.z_t, es), range3(conv_w, 1, C, 4, 0, 4, 4),
                        range3(conv_b, 1, 1, C, 0, 0, 4), range3(dt_bias, 1, 1, H, 0, 0, 4),
                        range3(A_log, 1, 1, H, 0, 0, 4), range3(D, 1, 1, H, 0, 0, 4),
                        range3(cu, 1, 1, n_seq + 1, 0, 0, 4), range3(slots, 1, 1, n_seq, 0, 0, 4),
                        range3(fresh, 1, 1, n_seq, 0, 0, 4)};
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : in)
            if (meet(out[i], r)) return SS_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return SS_ERR_INVALID_ARG;
    }
    p = HeadsParams{};
    p.xbc = xbc; p.dt_raw = dt_raw; p.z = z; p.y = y;
    p.conv_w = conv_w; p.conv_b = conv_b; p.dt_bias = dt_bias; p.A_log = A_log; p.D = D;
    p.state = state; p.window = window; p.cu = cu; p.slots = slots; p.fresh = fresh;
    p.err = device_error_word();
    p.xbc_t = st.xbc_t; p.dt_t = st.dt_t; p.z_t = st.z_t; p.y_t = st.y_t;
    p.tokens = tokens;
    p.n_seq = static_cast<int>(n_seq); p.H = static_cast<int>(H); p.P = static_cast<int>(P);
    p.G = static_cast<int>(G); p.N = static_cast<int>(N); p.C = static_cast<int>(C);
    p.n_slots = static_cast<int>(n_slots);
    return SS_OK;
}

}  // namespace host
}  // namespace selscan

using namespace selscan;
using namespace selscan::host;

extern "C" size_t ss_heads_workspace_size(int64_t n_seq, int64_t tokens, int64_t H, int64_t P, int64_t G, int64_t N,
                                          int32_t io_dtype) {
    if (n_seq <= 0 || tokens < 0 || H <= 0 || G <= 0 || P < 1 || P > SS_HEADS_MAX || N < 1 || N > SS_HEADS_MAX ||
        H % G != 0 || n_seq > INT32_MAX || (io_dtype != SS_F32 && io_dtype != SS_BF16))
        return 0;
    return heads_tc_takes(n_seq, tokens, H, P, G, N, io_dtype == SS_BF16)
               ? kHeadsCounterBytes + heads_tc_plan(n_seq, tokens, H, P, G, N).bytes
               : heads_counter_bytes(n_seq, G);
}

extern "C" ss_status ss_heads_fwd(const void* xbc, const void* dt_raw, const void* z, const float* conv_w,
                                  const float* conv_b, const float* dt_bias, const float* A_log, const float* D, void* y,
                                  float* state, float* window, const int32_t* cu_seqlens, const int32_t* slots,
                                  const int32_t* fresh, int64_t n_seq, int64_t tokens, int64_t H, int64_t P, int64_t G,
                                  int64_t N, int64_t n_slots, const ss_heads_strides* strides, void* workspace,
                                  size_t workspace_bytes, void* stream_ptr) {
    HeadsParams p;
    bool bf16 = false, idle = false;
    if (n_seq > 0 && !cu_seqlens) return SS_ERR_INVALID_ARG;
    const size_t need =
        ss_heads_workspace_size(n_seq, tokens, H, P, G, N, strides ? strides->io_dtype : static_cast<int32_t>(SS_F32));
    const ss_status st = heads_check(p, strides, xbc, dt_raw, z, conv_w, conv_b, dt_bias, A_log, D, y, state, window,
                                     cu_seqlens, slots, fresh, n_seq, tokens, H, P, G, N, n_slots, workspace,
                                     workspace_bytes, need, &bf16, &idle);
    if (st != SS_OK || idle) return st;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    cudaError_t e;
    if (heads_tc_takes(n_seq, tokens, H, P, G, N, bf16)) {
        e = launch_heads_tc(p, static_cast<uint8_t*>(workspace) + kHeadsCounterBytes, bf16, stream);
    } else {
        e = heads_counters(p, workspace, stream);
        if (e == cudaSuccess) e = bf16 ? launch_seq<__nv_bfloat16>(p, stream) : launch_seq<float>(p, stream);
    }
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}
