// Multi-head selective scan with its causal convolution, over packed prompts.
//
// Per head and token: S <- a·S + (Δ·x) ⊗ B (P × N), y = S·C + D·x, gated by silu(z), where x, B
// and C come out of a width-4 causal convolution and a SiLU.
//
// heads_seq_kernel walks the tokens in order, the recurrence as it is written, all of it in fp32.  A CTA
// has 64 rows of one head's state of one sequence.  A thread has 8 or 16 states of two or four rows in registers,
// LPR lanes share a row; 16 tokens at a time the CTA convolves its x channels and the group's B and C
// into shared memory (their samples are loaded a round ahead), then every warp takes the tokens one by
// one.  For longer sequences heads_bc_kernel convolves B and C once for all heads of a group beforehand,
// and the rounds come as bulk copies into two buffers.  What bounds it is the FMA pipe: three operations
// per state and token, 195 cycles of an SM for 64 x 128 states.
// Long sequences of few heads are cut in segments: a first pass leaves each segment's state from zero
// and its decay, the second starts every segment from the state that enters it.
// 8 prompts of up to 1024 tokens, 24 heads of 64 x 64 states, fp32: 154 us (8.7 us of memory traffic; cut in
// segments, 1.7 times the recurrence's work); one of 32768 tokens, 24 heads of 64 x 128: 1605 us.  Eight prompts of
// 512 tokens, 48 heads of 64 x 128: 274 us, the FMA pipe at 62%.  bf16, 4 prompts of 2048 tokens, 24 heads of 64 x 256,
// which come here whatever their length: 1058 us (13 of traffic; 64 x 128 on the tensor cores 122).  One of 45 tokens,
// 24 heads: 20 us, 24 CTAs on 152 SMs with one chain of 45 steps each.  bf16 prompts take the tensor cores
// (ss_heads_tc.cu) from where a cost rule there says so.
// fp32 ones do not: operands of two bf16 (three products) leave 4e-6 of a state.  (Three parts and six products have
// not been tried.)
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "../../include/selscan.h"
#include "heads_device.cuh"
#include "heads_params.h"
#include "heads_tc.h"
#include "internal.h"

namespace selscan {
namespace {

constexpr int kSeqRows = 64;                                // rows of the state per CTA
constexpr int kSeqT = 16;                                   // tokens per round
constexpr int kPreTokens = 96;                              // mean length from which B and C are convolved beforehand

struct SeqParams {
    HeadsParams p;
    int seg;                // tokens per segment (a multiple of kSeqT)
    int64_t units;          // upper bound of the segments
    float* seg_state;       // [units, H, P, N]: what a segment leaves from zero
    float* seg_decay;       // [units, H]: its log2 decay
    float* bc;              // [G, tokens][B | C], each padded with zeros to all lanes' states
    uint8_t* in_order;      // [n_seq] whether a sequence lies behind all before it; nullptr: every CTA looks itself
};

// Sequences from which on one small launch looks at their order for all CTAs, each of which would read all entries
// before its own.  24 heads, looked at by every CTA and beforehand: 64 sequences of 8 tokens (64 x 128, bf16) 93 and
// 94 us, 256 of 4 300 and 300, 400 of 4 465 and 455; 2048 of 2 (64 x 64, fp32) 1306 and 1192.
constexpr int kOrderFrom = 256;
constexpr int kOrderThreads = 1024;

// The same by all threads of a CTA for one sequence.  (Not inlined: the recurrence is scheduled worse with it.)
__device__ __noinline__ bool heads_behind_all(const int32_t* cu, int seq) {
    bool below = false;
    for (int j = threadIdx.x; j < seq; j += blockDim.x) below |= cu[j] > cu[seq];
    return !__syncthreads_or(below);
}

__global__ void __launch_bounds__(kOrderThreads) heads_order_kernel(const SeqParams q) {
    __shared__ int scratch[kOrderThreads / 32];
    int largest = 0;
    for (int s0 = 0; s0 < q.p.n_seq; s0 += blockDim.x) {
        const int seq = s0 + static_cast<int>(threadIdx.x);
        const bool ok = heads_in_order(q.p, seq, largest, scratch);
        if (seq < q.p.n_seq) q.in_order[seq] = ok;
    }
}

enum class SeqPass { kWhole, kStates, kSegments };

// Parity of the last phase of buffer `b` of two, after `loads` copies into them in turn (more than b).
constexpr uint32_t last_parity(int loads, int b) { return ((loads - 1 - b) >> 1) & 1; }
static_assert(last_parity(1, 0) == 0 && last_parity(2, 1) == 0 && last_parity(3, 0) == 1 && last_parity(3, 1) == 0 &&
              last_parity(4, 0) == 1 && last_parity(4, 1) == 1 && last_parity(5, 0) == 0 && last_parity(5, 1) == 1, "copies 0, 2, 4 and 1, 3, 5");

constexpr int kBcThreads = 256, kBcToks = 32;               // tokens per block (and thread)

// B and C of all tokens, convolved.  Grid (kBcToks tokens of a sequence, group).
template <typename TIO>
__global__ void __launch_bounds__(kBcThreads) heads_bc_kernel(const SeqParams q, int np) {
    const HeadsParams& p = q.p;
    __shared__ int scratch[kBcThreads / 32], found[2];
    const int tid = threadIdx.x, id = blockIdx.x, g = blockIdx.y;
    if (tid == 0) found[0] = -1;
    __syncthreads();
    int base = 0, largest = 0;
    for (int s0 = 0; s0 < p.n_seq && found[0] < 0; s0 += kBcThreads) {
        const bool in_order = heads_in_order(p, s0 + tid, largest, scratch);
        int n = 0;
        if (s0 + tid < p.n_seq && in_order) {
            const HeadsSeq c = heads_seq(p, s0 + tid);
            n = c.ok ? max(1, (c.len + kBcToks - 1) / kBcToks) : 0;
        }
        int total;
        const int at = base + block_prefix(n, &total, scratch);
        if (id >= at && id < at + n) {
            found[0] = s0 + tid;
            found[1] = id - at;
        }
        base += total;
        __syncthreads();
    }
    if (found[0] < 0) return;
    const HeadsSeq s = heads_seq(p, found[0]);
    const int first = found[1] * kBcToks;
    const TIO* x = static_cast<const TIO*>(p.xbc) + s.row0 * p.xbc_t;
    for (int k = tid; k < 2 * np && first < s.len; k += kBcThreads) {
        const int n = k % np;
        const bool on = n < p.N;
        const int c = p.H * p.P + (k >= np ? p.G * p.N : 0) + g * p.N + (on ? n : 0);
        const HeadsWindow win = first == 0 ? heads_window(p, s, c) : HeadsWindow{{0.f, 0.f, 0.f}};
        const float* w = p.conv_w + static_cast<int64_t>(c) * 4;
        const float wk[4] = {w[0], w[1], w[2], w[3]}, b = p.conv_b ? p.conv_b[c] : 0.f;
        float e0 = heads_sample<TIO>(p, s, win, c, first - 3), e1 = heads_sample<TIO>(p, s, win, c, first - 2),
              e2 = heads_sample<TIO>(p, s, win, c, first - 1);
        float* out = q.bc + (g * p.tokens + s.row0 + first) * (2 * np) + k;
        for (int j0 = 0; j0 < kBcToks && first + j0 < s.len; j0 += 8) {
            TIO raw[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                raw[j] = first + j0 + j < s.len ? x[static_cast<int64_t>(first + j0 + j) * p.xbc_t + c] : from_f32<TIO>(0.f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float e3 = to_f32<TIO>(raw[j]);
                const float v = heads_conv(wk, b, e0, e1, e2, e3);
                if (first + j0 + j < s.len) out[static_cast<int64_t>(j0 + j) * (2 * np)] = on ? v : 0.f;
                e0 = e1;
                e1 = e2;
                e2 = e3;
            }
        }
    }
    if (found[1] == 0 && s.slot >= 0) {                     // this block alone reads these channels' windows
        __syncthreads();
        const int cb = p.H * p.P + g * p.N, cc = cb + p.G * p.N;
        for (int k = tid; k < 2 * p.N; k += kBcThreads) heads_keep_window<TIO>(p, s, k < p.N ? cb + k : cc + k - p.N);
    }
}

// Rows per thread.  B and C of a token go to every thread that has a row, 128 bytes a cycle of an SM, which
// is what bounds two rows a thread (290 cycles for 64 x 128 states); with four, and fewer threads, the FMA
// pipe does.  Where B and C are convolved here the threads are needed for that.
constexpr int seq_rows(int lpr, int ns, bool pre) { return pre && lpr * ns >= 32 ? 4 : 2; }
constexpr int seq_threads(int lpr, int ns, bool pre) { return kSeqRows / seq_rows(lpr, ns, pre) * lpr; }

// Lanes that share a row and states of a lane, for N up to 16, 32, 64, 128 and 256.  16 states to a lane make the
// fewest loads of B and C, but up to 32 states they leave a CTA one warp, which also has to convolve and write:
// 16 prompts of 512 tokens, 40 heads of 64 rows, fp32: 16 states 247 us with 1 x 16, 158 with 2 x 8, 157 with
// 4 x 4 (4 prompts of 2048: 284, 194, 243); 32 states 324 with 2 x 16, 216 with 4 x 8; 64 states 301 with 4 x 16, 302
// with 8 x 8, 366 with 16 x 4; 128 states 456 with 8 x 16, 531 with 16 x 8.
struct SeqLanes {
    int lpr, ns;
};
constexpr SeqLanes kSeqLanes[] = {{2, 8}, {4, 8}, {4, 16}, {8, 16}, {16, 16}};

// PRE: B and C come convolved from heads_bc_kernel.
template <typename TIO, int LPR, int NS, SeqPass PASS, bool PRE>
__global__ void __launch_bounds__(seq_threads(LPR, NS, PRE)) heads_seq_kernel(const SeqParams q) {
    constexpr int NT = seq_threads(LPR, NS, PRE), RPT = seq_rows(LPR, NS, PRE), RT = kSeqRows / RPT, NP = NS * LPR;
    constexpr int U = 8 / RPT;                              // tokens whose sums over lanes are taken together
    constexpr int CH = PRE ? kSeqRows : kSeqRows + 2 * NP;  // channels convolved here
    constexpr int XT = PRE && NT > kSeqRows ? kSeqT * kSeqRows / NT : kSeqT;      // tokens per thread and channel
    constexpr int CPT = (CH * (kSeqT / XT) + NT - 1) / NT;  // channels per thread
    constexpr int OPT = kSeqT * kSeqRows / NT;              // outputs per thread and round
    constexpr bool kOut = PASS != SeqPass::kStates;
    __shared__ __align__(128) float sbc[PRE ? 2 : 1][kSeqT][2 * NP];
    __shared__ float sx[kSeqT][kSeqRows], sy[kSeqT][kSeqRows];
    __shared__ float sdt[kSeqT], sa[kSeqT];
    __shared__ uint64_t full[2];
    __shared__ int abort_flag, loads;                       // loads: thread 0's copies so far
    __shared__ int scratch[NT / 32], found[2];
    const HeadsParams& p = q.p;
    const int tid = threadIdx.x, tiles = (p.P + kSeqRows - 1) / kSeqRows;
    const int64_t id = blockIdx.x;
    const int pt = static_cast<int>(id % tiles), h = static_cast<int>(id / tiles % p.H);
    int64_t unit = id / tiles / p.H;
    int seq = static_cast<int>(unit), seg = 0, nsegs = 1;
    if (PASS != SeqPass::kWhole) {                          // the sequence that this segment is of
        if (tid == 0) found[0] = -1;
        __syncthreads();
        int base = 0, largest = 0;
        const bool reports = id == 0;                       // (and looks at all sequences)
        for (int s0 = 0; s0 < p.n_seq && (reports || found[0] < 0); s0 += NT) {
            const bool in_order = heads_in_order(p, s0 + tid, largest, scratch);
            int n = 0;
            if (s0 + tid < p.n_seq) {
                const HeadsSeq c = heads_seq(p, s0 + tid);
                const bool ok = c.ok && in_order;
                n = ok ? max(1, (c.len + q.seg - 1) / q.seg) : 0;
                if (!ok && reports && p.err) atomicOr(p.err, kErrIndex);
            }
            int total;
            const int at = base + block_prefix(n, &total, scratch);
            if (unit >= at && unit < at + n) {
                found[0] = s0 + tid;
                found[1] = static_cast<int>(unit) - at;
            }
            base += total;
            __syncthreads();
        }
        if (found[0] < 0) return;
        seq = found[0];
        seg = found[1];
    }
    const bool in_order = PASS != SeqPass::kWhole || (q.in_order ? q.in_order[seq] != 0 : heads_behind_all(p.cu, seq));
    const HeadsSeq s = heads_seq(p, seq);
    if (!s.ok || !in_order) {
        if (h == 0 && pt == 0 && tid == 0 && p.err) atomicOr(p.err, kErrIndex);
        return;
    }
    if (PASS != SeqPass::kWhole) nsegs = max(1, (s.len + q.seg - 1) / q.seg);
    const int64_t unit0 = unit - seg;
    const int first = PASS == SeqPass::kWhole ? 0 : seg * q.seg;
    const int end = PASS == SeqPass::kWhole ? s.len : min(s.len, first + q.seg);
    const bool last = seg == nsegs - 1;
    if (PASS == SeqPass::kStates && nsegs == 1) return;

    const int g = h / (p.H / p.G), lr = tid % LPR, rp = tid / LPR;       // rows rp, rp + RT, ..
    const int p0 = pt * kSeqRows, np = min(kSeqRows, p.P - p0);
    const int cx = h * p.P + p0, cb = p.H * p.P + g * p.N, cc = cb + p.G * p.N;
    const float A2 = -expf(p.A_log[h]) * kLog2e, bias = p.dt_bias ? p.dt_bias[h] : 0.f, Dh = p.D ? p.D[h] : 0.f;

    const int rounds = (end - first + kSeqT - 1) / kSeqT;
    auto load_bc = [&](int r) {                             // (one thread, in order) round r into its buffer
        const int t0 = first + r * kSeqT;
        loads = r + 1;
        const uint32_t bytes = static_cast<uint32_t>(min(kSeqT, end - t0)) * (2 * NP * 4);
        mbar_expect_tx(&full[r & 1], bytes);
        bulk_load(&sbc[PRE ? r & 1 : 0][0][0], q.bc + (g * p.tokens + s.row0 + t0) * (2 * NP), bytes, &full[r & 1]);
    };
    // (the first pass only passes on the last segment's starting state: no rounds, and no copies that the
    // block would leave in flight)
    const bool runs = !(PASS == SeqPass::kStates && last);
    if (PRE && runs) {
        if (tid == 0) {
            mbar_init(&full[0], 1);
            mbar_init(&full[1], 1);
            mbar_fence_init();
            abort_flag = loads = 0;
        }
        // rows that no copy has reached yet meet Δ = 0: they have to be numbers
        for (int i = tid; i < 2 * kSeqT * 2 * NP; i += NT) (&sbc[0][0][0])[i] = 0.f;
        tma_store_fence();
        __syncthreads();
        if (tid == 0) {
            if (rounds > 0) load_bc(0);
            if (rounds > 1) load_bc(1);
        }
    }

    // this thread's channels (the tokens of a round shared among the threads of a channel), their weights
    // and their samples from three before on
    int chan[CPT];
    float w[CPT][4], cbias[CPT], win[CPT][3];
    TIO raw[CPT][XT + 3];
    const int my_t = PRE && NT > kSeqRows ? tid / kSeqRows * XT : 0;
    const TIO* xg = static_cast<const TIO*>(p.xbc) + s.row0 * p.xbc_t;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int i = PRE && NT > kSeqRows ? tid % kSeqRows : tid + k * NT;
        const int j = i < kSeqRows ? i : i < kSeqRows + NP ? i - kSeqRows : i - kSeqRows - NP;
        const bool on = i < CH && (i < kSeqRows ? j < np : j < p.N) && (kOut || i < kSeqRows + NP);
        chan[k] = !on ? -1 : i < kSeqRows ? cx + j : i < kSeqRows + NP ? cb + j : cc + j;
    }
    auto load_round = [&](int t0) {
#pragma unroll
        for (int k = 0; k < CPT; ++k)
#pragma unroll
            for (int t = 0; t < XT + 3; ++t) {
                const int at = t0 + my_t + t - 3;
                raw[k][t] = (chan[k] >= 0 && at >= 0 && at < end) ? xg[static_cast<int64_t>(at) * p.xbc_t + chan[k]] : from_f32<TIO>(0.f);
            }
    };
    if (runs && first < end) load_round(first);
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = max(chan[k], 0);
        HeadsWindow v = {{0.f, 0.f, 0.f}};
        if (chan[k] >= 0 && first == 0) v = heads_window(p, s, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[k][i] = chan[k] >= 0 ? p.conv_w[static_cast<int64_t>(c) * 4 + i] : 0.f;
        cbias[k] = (chan[k] >= 0 && p.conv_b) ? p.conv_b[c] : 0.f;
#pragma unroll
        for (int i = 0; i < 3; ++i) win[k][i] = v.v[i];
    }

    // The state that enters (see ss_heads_tc.cu: the second pass over a cut sequence must not read its
    // slot, which the first pass puts in the place of the last segment).
    float2 S[RPT][NS / 2];
    auto at_state = [&](float* base, int64_t k) { return base + ((k * p.H + h) * p.P + p0) * p.N; };
    auto each_state = [&](float* base, auto&& f) {          // f(element, its address) for this thread's
#pragma unroll
        for (int r = 0; r < RPT; ++r)
#pragma unroll
            for (int j = 0; j < NS / 2; ++j) {
                const int row = rp + RT * r, n = (j / 2 * LPR + lr) * 4 + (j & 1) * 2;
                if (row < np && n < p.N) f(S[r][j].x, base + static_cast<int64_t>(row) * p.N + n);
                if (row < np && n + 1 < p.N) f(S[r][j].y, base + static_cast<int64_t>(row) * p.N + n + 1);
            }
    };
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
        for (int j = 0; j < NS / 2; ++j) S[r][j] = make_float2(0.f, 0.f);
    float* slot_state = at_state(p.state, max(s.slot, 0));
    if (s.warm && (PASS == SeqPass::kStates ? seg == 0 || last : nsegs == 1))
        each_state(slot_state, [](float& v, const float* f) { v = *f; });
    if (!runs) {
        each_state(at_state(q.seg_state, unit), [](float& v, float* f) { *f = v; });
        return;
    }
    if (PASS == SeqPass::kSegments && nsegs > 1) {
        if (seg == 0) each_state(at_state(q.seg_state, unit0 + nsegs - 1), [](float& v, const float* f) { v = *f; });
        for (int j = 0; j < seg; ++j) {
            const float d = ex2(q.seg_decay[(unit0 + j) * p.H + h]);
            each_state(at_state(q.seg_state, unit0 + j), [d](float& v, const float* f) { v = fmaf(d, v, *f); });
        }
    }
    float decay_sum = 0.f, dt_next = 0.f;
    auto load_dt = [&](int t0) {
        return (tid < kSeqT && t0 + tid < end)
                   ? to_f32<TIO>(static_cast<const TIO*>(p.dt_raw)[(s.row0 + t0 + tid) * p.dt_t + h]) : 0.f;
    };
    if (first < end) dt_next = load_dt(first);

    for (int t0 = first; t0 < end; t0 += kSeqT) {
        const int nt = min(kSeqT, end - t0);
        const int round = (t0 - first) / kSeqT;
        float (*bc)[2 * NP] = sbc[PRE ? round & 1 : 0];
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int i = PRE && NT > kSeqRows ? tid % kSeqRows : tid + k * NT;
            float* dst = i < kSeqRows ? &sx[0][i] : &bc[0][i - kSeqRows];          // (B, then C)
            const int pitch = i < kSeqRows ? kSeqRows : 2 * NP;
            if (i < CH) {
                float e[3];
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    const int at = t0 + my_t + j - 3;
                    e[j] = at >= 0 ? to_f32<TIO>(raw[k][j]) : at == -1 ? win[k][2] : at == -2 ? win[k][1] : win[k][0];
                }
#pragma unroll
                for (int t = 0; t < XT; ++t) {
                    const float e3 = to_f32<TIO>(raw[k][t + 3]);
                    dst[(my_t + t) * pitch] = heads_conv(w[k], cbias[k], e[0], e[1], e[2], e3);
                    e[0] = e[1];
                    e[1] = e[2];
                    e[2] = e3;
                }
            }
        }
        if (tid < kSeqT) {                                  // past the end: Δ = 0, which changes nothing
            const float dt = tid < nt ? softplus(dt_next + bias) : 0.f;
            sdt[tid] = dt;
            sa[tid] = ex2(dt * A2);
            decay_sum += dt * A2;
        }
        if (t0 + kSeqT < end) {
            load_round(t0 + kSeqT);
            dt_next = load_dt(t0 + kSeqT);
        }
        TIO gate[OPT];                                      // z of this round's outputs, loaded ahead of their use
        if (kOut && p.z) {
#pragma unroll
            for (int k = 0; k < OPT; ++k) {
                const int i = tid + k * NT, t = i / kSeqRows, c = i % kSeqRows;
                gate[k] = (t < nt && c < np) ? static_cast<const TIO*>(p.z)[(s.row0 + t0 + t) * p.z_t + cx + c] : from_f32<TIO>(0.f);
            }
        }
        if (PRE) mbar_wait_bounded(&full[round & 1], (round >> 1) & 1, &abort_flag, p.err);
        __syncthreads();
#pragma unroll 1
        for (int t4 = 0; t4 < nt; t4 += U) {
            float2 a[U], d[RPT][U], y[RPT][U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t4 + u;
                const float dt = sdt[t];
                a[u] = splat2(sa[t]);
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    d[r][u] = splat2(dt * sx[t][rp + RT * r]);
                    y[r][u] = make_float2(0.f, 0.f);
                }
            }
            // four states at a time through all of the tokens, so that their loads are together
#pragma unroll
            for (int j = 0; j < NS / 4; ++j) {
                float4 B[U], C[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    B[u] = *reinterpret_cast<const float4*>(&bc[t4 + u][(j * LPR + lr) * 4]);
                    if (kOut) C[u] = *reinterpret_cast<const float4*>(&bc[t4 + u][NP + (j * LPR + lr) * 4]);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float2 b0 = make_float2(B[u].x, B[u].y), b1 = make_float2(B[u].z, B[u].w);
#pragma unroll
                    for (int r = 0; r < RPT; ++r) {
                        S[r][2 * j] = fma2(a[u], S[r][2 * j], mul2(d[r][u], b0));
                        S[r][2 * j + 1] = fma2(a[u], S[r][2 * j + 1], mul2(d[r][u], b1));
                        if (kOut) {
                            const float2 c0 = make_float2(C[u].x, C[u].y), c1 = make_float2(C[u].z, C[u].w);
                            y[r][u] = fma2(S[r][2 * j + 1], c1, fma2(S[r][2 * j], c0, y[r][u]));
                        }
                    }
                }
            }
            if (kOut) {
                // sums over the lanes of a row: at each exchange a lane keeps half of the values
                float v[RPT * U];
#pragma unroll
                for (int r = 0; r < RPT; ++r)
#pragma unroll
                    for (int u = 0; u < U; ++u) v[r * U + u] = y[r][u].x + y[r][u].y;
                int n = RPT * U, at = 0;
#pragma unroll
                for (int o = LPR / 2; o > 0; o /= 2) {
                    if (n > 1) {
                        n /= 2;
                        const bool up = lr & o;
#pragma unroll
                        for (int i = 0; i < n; ++i) {
                            const float give = up ? v[i] : v[i + n];
                            v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, give, o);
                        }
                        at += up ? n : 0;
                    } else {
                        v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
                    }
                }
#pragma unroll
                for (int i = 0; i < n; ++i) sy[t4 + (at + i) % U][rp + RT * ((at + i) / U)] = v[i];
            }
        }
        __syncthreads();
        if (PRE && tid == 0 && round + 2 < rounds && !abort_flag) load_bc(round + 2);
        if (kOut) {
#pragma unroll
            for (int k = 0; k < OPT; ++k) {
                const int i = tid + k * NT, t = i / kSeqRows, c = i % kSeqRows;
                if (t < nt && c < np) {
                    float y = fmaf(Dh, sx[t][c], sy[t][c]);
                    if (p.z) y *= silu(to_f32<TIO>(gate[k]));
                    static_cast<TIO*>(p.y)[(s.row0 + t0 + t) * p.y_t + cx + c] = from_f32<TIO>(y);
                }
            }
            __syncthreads();
        }
    }
    if (PRE && abort_flag && tid == 0) {                    // copies in flight land before the block ends
        const long long c0 = clock64();
        auto landed = [&](int b) { return loads <= b || mbar_try_wait(&full[b], last_parity(loads, b)); };
        while (!(landed(0) && landed(1)) && clock64() - c0 < (1ll << 28)) {
        }
    }
    if (PASS == SeqPass::kStates) {
        each_state(at_state(q.seg_state, unit), [](float& v, float* f) { *f = v; });
#pragma unroll
        for (int o = 8; o > 0; o /= 2) decay_sum += __shfl_xor_sync(0xffffffffu, decay_sum, o);      // the first 16 lanes hold it
        if (pt == 0 && tid == 0) q.seg_decay[unit * p.H + h] = decay_sum;
        return;
    }
    if (s.slot < 0) return;
    if (last) each_state(slot_state, [](float& v, float* f) { *f = v; });
    if (seg > 0) return;
    // the CTAs of a sequence's first segment read its windows: the x channels' are this CTA's own, those of
    // B and C the group's, whose last reader shifts them
    __syncthreads();
    for (int k = tid; k < np; k += NT) heads_keep_window<TIO>(p, s, cx + k);
    if (PRE) return;
    __shared__ int last_reader;
    if (tid == 0) {
        unsigned int* counter = p.arrivals + static_cast<int64_t>(seq) * p.G + g;
        last_reader = heads_say_read(counter) == static_cast<unsigned int>((p.H / p.G) * tiles) - 1u;
        if (last_reader) *counter = 0u;
    }
    __syncthreads();
    if (last_reader)
        for (int k = tid; k < 2 * p.N; k += NT) heads_keep_window<TIO>(p, s, k < p.N ? cb + k : cc + k - p.N);
}

// Tokens per segment (0: whole sequences), for sequences of equal length: a segmented call does about 1.7
// times the work and has one more launch (10 us, about 60 tokens' time), and pays where the CTAs of
// whole sequences leave the SMs fewer than 16 warps; past a dozen
// segments what a segment gathers of those before it costs more than that brings.
struct SeqPlan {
    int seg, np;            // np: states padded
    bool pre;               // B and C convolved beforehand
    int64_t units, chunks;  // upper bounds
    size_t off_state, off_decay, off_bc, off_order, bytes;
    bool order;             // the sequences' order is looked at beforehand
};
std::atomic<int> g_force_pre{0};

SeqPlan seq_plan(int64_t n_seq, int64_t tokens, int64_t H, int64_t P, int64_t G, int64_t N) {
    SeqPlan plan{};
    const int64_t ctas = n_seq * H * ((P + kSeqRows - 1) / kSeqRows);
    const SeqLanes lanes = kSeqLanes[N <= 16 ? 0 : N <= 32 ? 1 : N <= 64 ? 2 : N <= 128 ? 3 : 4];
    const int64_t mean = tokens / std::max<int64_t>(n_seq, 1);
    const int forced = g_force_pre.load();
    plan.pre = N <= 128 && G <= 65535 && (forced ? forced == 2 : mean >= kPreTokens);
    const int64_t room = heads_sm_count() * 16 / std::max(seq_threads(lanes.lpr, lanes.ns, plan.pre) / 32, 1);
    const int64_t k = std::min({room / std::max<int64_t>(ctas, 1), mean / 64, static_cast<int64_t>(12)});
    plan.units = n_seq;
    plan.np = lanes.lpr * lanes.ns;
    plan.chunks = tokens / kBcToks + n_seq;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 255) / 256 * 256;
        return here;
    };
    if (k >= 3) {
        plan.seg = static_cast<int>((mean / k + kSeqT - 1) / kSeqT * kSeqT);
        plan.units = tokens / plan.seg + n_seq;
        plan.off_state = take(static_cast<size_t>(plan.units) * H * P * N * 4);
        plan.off_decay = take(static_cast<size_t>(plan.units) * H * 4);
    }
    if (plan.pre) plan.off_bc = take(static_cast<size_t>(tokens) * G * 2 * plan.np * 4);
    plan.order = plan.seg == 0 && n_seq >= kOrderFrom;
    if (plan.order) plan.off_order = take(static_cast<size_t>(n_seq));
    plan.bytes = at;
    return plan;
}

template <typename TIO, int LPR, int NS, bool PRE>
cudaError_t launch_seq_pre(const SeqParams& q, unsigned grid, cudaStream_t stream) {
    if (q.seg == 0) {
        heads_seq_kernel<TIO, LPR, NS, SeqPass::kWhole, PRE><<<grid, seq_threads(LPR, NS, PRE), 0, stream>>>(q);
        return cudaGetLastError();
    }
    heads_seq_kernel<TIO, LPR, NS, SeqPass::kStates, PRE><<<grid, seq_threads(LPR, NS, PRE), 0, stream>>>(q);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    heads_seq_kernel<TIO, LPR, NS, SeqPass::kSegments, PRE><<<grid, seq_threads(LPR, NS, PRE), 0, stream>>>(q);
    return cudaGetLastError();
}

template <typename TIO, int LPR, int NS>
cudaError_t launch_seq_lanes(const SeqParams& q, const SeqPlan& plan, cudaStream_t stream) {
    const int64_t per_unit = static_cast<int64_t>(q.p.H) * ((q.p.P + kSeqRows - 1) / kSeqRows);
    const unsigned grid = static_cast<unsigned>(q.units * per_unit);
    if constexpr (LPR * NS <= 128) {                               // (two buffers of more states do not fit)
        if (plan.pre) {
            const dim3 bc(static_cast<unsigned>(plan.chunks), static_cast<unsigned>(q.p.G));
            heads_bc_kernel<TIO><<<bc, kBcThreads, 0, stream>>>(q, plan.np);
            const cudaError_t e = cudaGetLastError();
            return e != cudaSuccess ? e : launch_seq_pre<TIO, LPR, NS, true>(q, grid, stream);
        }
    }
    return launch_seq_pre<TIO, LPR, NS, false>(q, grid, stream);
}

template <typename TIO>
cudaError_t launch_seq(const HeadsParams& p, uint8_t* workspace, cudaStream_t stream) {
    const SeqPlan plan = seq_plan(p.n_seq, p.tokens, p.H, p.P, p.G, p.N);
    const SeqParams q{p, plan.seg, plan.units, reinterpret_cast<float*>(workspace + plan.off_state),
                      reinterpret_cast<float*>(workspace + plan.off_decay), reinterpret_cast<float*>(workspace + plan.off_bc),
                      plan.order ? workspace + plan.off_order : nullptr};
    if (plan.units * p.H * ((p.P + kSeqRows - 1) / kSeqRows) > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (plan.order) {
        heads_order_kernel<<<1, std::min(kOrderThreads, (p.n_seq + 31) / 32 * 32), 0, stream>>>(q);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    constexpr const SeqLanes* w = kSeqLanes;
    if (p.N <= 16) return launch_seq_lanes<TIO, w[0].lpr, w[0].ns>(q, plan, stream);
    if (p.N <= 32) return launch_seq_lanes<TIO, w[1].lpr, w[1].ns>(q, plan, stream);
    if (p.N <= 64) return launch_seq_lanes<TIO, w[2].lpr, w[2].ns>(q, plan, stream);
    if (p.N <= 128) return launch_seq_lanes<TIO, w[3].lpr, w[3].ns>(q, plan, stream);
    return launch_seq_lanes<TIO, w[4].lpr, w[4].ns>(q, plan, stream);
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
               : heads_counter_bytes(n_seq, G) + seq_plan(n_seq, tokens, H, P, G, N).bytes;
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
        uint8_t* behind = static_cast<uint8_t*>(workspace) + heads_counter_bytes(n_seq, G);
        if (e == cudaSuccess) e = bf16 ? launch_seq<__nv_bfloat16>(p, behind, stream) : launch_seq<float>(p, behind, stream);
    }
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

// Test hook: whether the token-by-token path convolves B and C beforehand (1 no, 2 yes, 0 by length).  Returns
// the previous value.
extern "C" int ss__force_heads_pre(int pre) { return selscan::g_force_pre.exchange(pre); }
