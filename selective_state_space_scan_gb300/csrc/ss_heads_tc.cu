// Multi-head selective scan over packed prompts on the tensor cores: 128 tokens at a time.
//
// With one decay per head the recurrence over a chunk of tokens is three matrix products.  Let a_t be
// the log2 decay of token t, l_t its running sum within the chunk, and S the state that enters:
//   Y   = exp2(l_t) (C_t · S) + Σ_{s<=t} exp2(l_t - l_s) Δ_s (C_t · B_s) x_s,   y = Y + D x
//   S'  = exp2(l_end) S + Σ_s exp2(l_end - l_s) Δ_s B_s ⊗ x_s
// heads_prep_kernel convolves B and C once per chunk and group and leaves them as shared-memory
// images of bf16 operand tiles: B as a sum of two bf16 (hi + lo), C rounded.  heads_tc_kernel walks
// the chunks of one sequence (or of a segment of it) for two tiles of 64 rows of the state (two heads,
// as a rule), a warpgroup for each:
//   scores C·Bᵀ, and C·S of both tiles        while the warpgroups convolve x, as tiles of x and of
//                                             x scaled for the state (hi + lo)
//   the state's products, hi·hi + hi·lo + lo·hi   while they turn scores into P (decay, Δ, mask)
//   P·x on top of exp2(l)·(C·S), P read from tensor memory
// The state itself stays in registers, fp32: what the chunk adds comes out of tensor memory.
//
// Rounding: the state's operands carry 16 bits each, so a state is off by about 1e-6 of what was added
// to it.  y is rounded to bf16 in the end; the factors C, S, P and x of its sums are rounded to bf16
// before the products, each error as large as that last one, and D·x is not.
// A decay is only ever the exp2 of a sum of steps between its two tokens, never a quotient, and such
// sums are taken over the steps themselves, so strong decays neither overflow nor cancel.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/selscan.h"
#include "heads_device.cuh"
#include "heads_params.h"
#include "heads_tc.h"
#include "internal.h"
#include "tc_device.cuh"

namespace selscan {
namespace {

constexpr int kQ = kHeadsChunk;                    // tokens per chunk (128: rows of the products)
constexpr int kTile = kHeadsTile;                  // rows of the state per tile (64)
constexpr uint32_t kBlock = kQ * kTcRow;           // a tile's block: 128 rows of 64 bf16
constexpr int kPrepThreads = 256;
constexpr int kTcThreads = 256;                    // two warpgroups, one per tile

// ---- where the chunks and segments of the sequences are

// Chunks of sequence `seq`: at least one, so that an empty sequence is visited too; none if its
// indexes are out of range.
__device__ __forceinline__ int chunks_of(const HeadsParams& p, int seq) {
    if (seq >= p.n_seq) return 0;
    const HeadsSeq s = heads_seq(p, seq);
    return s.ok ? max(1, (s.len + kQ - 1) / kQ) : 0;
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

// ---- B and C

// Four channels as loaded: bf16 pairs, or floats.  `n` of them exist; VEC: all or none, one aligned access.
template <typename TIO, bool VEC> struct Quad4;
template <bool VEC> struct Quad4<__nv_bfloat16, VEC> {
    uint2 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* q, int n) {
        u = make_uint2(0u, 0u);
        if constexpr (VEC) {
            if (n > 0) u = *reinterpret_cast<const uint2*>(q);
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(q);
            if (n > 0) u.x = h[0];
            if (n > 1) u.x |= static_cast<uint32_t>(h[1]) << 16;
            if (n > 2) u.y = h[2];
            if (n > 3) u.y |= static_cast<uint32_t>(h[3]) << 16;
        }
    }
    __device__ __forceinline__ float4 get() const { return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y)); }
    static __device__ __forceinline__ void store(__nv_bfloat16* q, int n, float4 v) {
        if constexpr (VEC) {
            if (n > 0) *reinterpret_cast<uint2*>(q) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        } else {
            if (n > 0) q[0] = from_f32<__nv_bfloat16>(v.x);
            if (n > 1) q[1] = from_f32<__nv_bfloat16>(v.y);
            if (n > 2) q[2] = from_f32<__nv_bfloat16>(v.z);
            if (n > 3) q[3] = from_f32<__nv_bfloat16>(v.w);
        }
    }
};

// Grid (chunk, group, B or C).  Block (0, 0, 0) also writes the tables of where chunks and segments
// begin, and reports indexes out of range.
template <typename TIO, bool VEC>
__global__ void __launch_bounds__(kPrepThreads) heads_prep_kernel(const HeadsTcParams q) {
    const HeadsParams& p = q.p;
    __shared__ int scratch[kPrepThreads / 32], found[2];
    const int tid = threadIdx.x, id = blockIdx.x, g = blockIdx.y;
    const bool first = id == 0 && g == 0 && blockIdx.z == 0;
    if (tid == 0) found[0] = -1;
    __syncthreads();
    int base = 0, sbase = 0;
    for (int s0 = 0; s0 < p.n_seq; s0 += kPrepThreads) {
        const int seq = s0 + tid, n = chunks_of(p, seq);
        int total;
        const int at = base + block_prefix(n, &total, scratch);
        if (id >= at && id < at + n) {
            found[0] = seq;
            found[1] = id - at;
        }
        if (first) {
            const int ns = (n + q.seg_chunks - 1) / q.seg_chunks;
            int stotal;
            const int sat = sbase + block_prefix(ns, &stotal, scratch);
            if (seq < p.n_seq) {
                q.chunk_base[seq] = at;
                q.seg_base[seq] = sat;
                if (n == 0 && p.err) atomicOr(p.err, kErrIndex);
            }
            sbase += stotal;
        }
        base += total;
        __syncthreads();
        if (!first && found[0] >= 0) break;
    }
    if (first && tid == 0) q.seg_base[p.n_seq] = sbase;
    __syncthreads();
    if (found[0] < 0) return;
    const int seq = found[0], chunk = found[1], which = blockIdx.z;
    const HeadsSeq s = heads_seq(p, seq);
    const int c0 = p.H * p.P + (which ? p.G * p.N : 0) + g * p.N;      // first channel
    const int quads = q.nb * 16, qd = tid % quads, rows = kQ * quads / kPrepThreads, r0 = (tid / quads) * rows;
    const int ch = qd * 4, n = min(4, p.N - ch), t0 = chunk * kQ;
    uint8_t* img = q.images + (static_cast<int64_t>(id) * p.G + g) * (3 * q.nb * static_cast<int64_t>(kBlock));
    uint8_t* hi = img + (which ? 2 * q.nb * kBlock : 0) + (qd / 16) * kBlock;
    uint8_t* lo = img + q.nb * kBlock + (qd / 16) * kBlock;            // B only
    const TIO* x = static_cast<const TIO*>(p.xbc) + s.row0 * p.xbc_t + c0 + ch;
    constexpr int kRows = 8;                                           // a round: its loads are issued together
    Quad4<TIO, VEC> raw[kRows];
    auto load_round = [&](int r) {
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const int t = t0 + r0 + r + j;
            raw[j].load(x + t * p.xbc_t, t < s.len ? n : 0);
        }
    };
    load_round(0);
    float w[4][4], b[4];
    float4 e[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[i][k] = i < n ? p.conv_w[static_cast<int64_t>(c0 + ch + i) * 4 + k] : 0.f;
        b[i] = (i < n && p.conv_b) ? p.conv_b[c0 + ch + i] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const int t = t0 + r0 + j - 3;
        Quad4<TIO, VEC> f;
        f.load(x + static_cast<int64_t>(max(t, 0)) * p.xbc_t, (t >= 0 && t < s.len) ? n : 0);
        e[j] = f.get();
        if (t < 0) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) v[i] = heads_window(p, s, c0 + ch + i).v[j];      // t = j - 3
            e[j] = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
    for (int r = 0; r < rows; r += kRows) {
        if (r > 0) load_round(r);
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const bool on = t0 + r0 + r + j < s.len;
            const float4 f = raw[j].get();
            float u[4];
            u[0] = heads_conv(w[0], b[0], e[0].x, e[1].x, e[2].x, f.x);
            u[1] = heads_conv(w[1], b[1], e[0].y, e[1].y, e[2].y, f.y);
            u[2] = heads_conv(w[2], b[2], e[0].z, e[1].z, e[2].z, f.z);
            u[3] = heads_conv(w[3], b[3], e[0].w, e[1].w, e[2].w, f.w);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (!on || i >= n) u[i] = 0.f;
            const uint32_t off = tc_chunk(r0 + r + j, (qd % 16) / 2) + (qd & 1) * 8;
            const uint2 h = make_uint2(pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]));
            *reinterpret_cast<uint2*>(hi + off) = h;
            if (which == 0)
                *reinterpret_cast<uint2*>(lo + off) = make_uint2(pack_bf16(u[0] - bf16_lo(h.x), u[1] - bf16_hi(h.x)),
                                                                 pack_bf16(u[2] - bf16_lo(h.y), u[3] - bf16_hi(h.y)));
            e[0] = e[1];
            e[1] = e[2];
            e[2] = f;
        }
    }
    // the first chunk's block alone reads these channels' windows: it shifts them
    if (chunk == 0 && s.slot >= 0) {
        __syncthreads();
        for (int k = tid; k < p.N; k += kPrepThreads) heads_keep_window<TIO>(p, s, c0 + k);
    }
}

// ---- the scan

constexpr uint32_t kImage = 2 * kBlock;            // B hi, B lo or C in shared memory (N up to 128)
constexpr uint32_t kTileBytes = 4 * kBlock;        // per tile: x, x scaled hi, x scaled lo, state
constexpr int kFacs = 192;                         // decay factors of the blocks off the diagonal
struct TcTables {
    float tail[kQ];                                // Δ_s · decay from s to the chunk's end
    float fac[kFacs];                              // Δ_s · decay from s to the start of a later block of 32
    float total[4];                                // log2 decay of the blocks of 32
};
struct TcShared {
    uint64_t bar_bc, bar_cs, bar_st, bar_pv[2];
    uint32_t tmem;
    int abort;
    TcTables tab[2];
};
constexpr uint32_t kTcSmem = 3 * kImage + 2 * kTileBytes + sizeof(TcShared);
static_assert(kTcSmem <= 232448, "227 KB of shared memory per CTA");

// Columns of tensor memory: scores, C·S and then y of both tiles, what the chunk adds to the state of
// both tiles, P of both tiles (two bf16 a column).
constexpr uint32_t kColScore = 0, kColY = 128, kColS = 256, kColP = 384, kTmemCols = 512;

// Warpgroup-wide barrier (its four warps).
__device__ __forceinline__ void wg_sync(int wg) { named_barrier(1 + wg, 128); }

// STATE_ONLY: the first pass over a sequence cut in segments: the state that each segment but the last
// leaves from zero, and its decay; no outputs.
template <typename TIO, bool VEC, bool STATE_ONLY>
__global__ void __launch_bounds__(kTcThreads, 1) heads_tc_kernel(const HeadsTcParams q) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const HeadsParams& p = q.p;
    uint8_t* img = smem;                                               // B hi, B lo, C
    TcShared& sh = *reinterpret_cast<TcShared*>(smem + 3 * kImage + 2 * kTileBytes);
    const int tid = threadIdx.x, wg = tid / 128, t = tid % 128, warp = t / 32, lane = t % 32;
    uint8_t* tile = smem + 3 * kImage + wg * kTileBytes;
    uint8_t *sX = tile, *sXh = tile + kBlock, *sXl = tile + 2 * kBlock, *sS = tile + 3 * kBlock;
    float* stage = reinterpret_cast<float*>(sXh);                      // y, over x scaled (hi and lo)

    const int unit = blockIdx.x / q.pairs, pair = blockIdx.x % q.pairs;
    if (unit >= q.seg_base[p.n_seq]) return;
    int seq = 0;
    for (int a = 0, b = p.n_seq; b - a > 1;) {                          // the sequence with seg_base <= unit
        const int m = (a + b) / 2;
        if (q.seg_base[m] <= unit) a = m;
        else b = m;
        seq = a;
    }
    // (a skipped sequence has no segments: the last of equal bases is the one that has them)
    const HeadsSeq s = heads_seq(p, seq);
    const int seg = unit - q.seg_base[seq], nchunks = (s.len + kQ - 1) / kQ;
    const int ch0 = seg * q.seg_chunks, ch1 = min(nchunks, ch0 + q.seg_chunks);
    const bool last = ch1 >= nchunks;
    // the tile: tiles of a group are numbered head by head, two of them to a CTA
    const int ppg = q.pairs / p.G, g = pair / ppg, tiles = (p.P + kTile - 1) / kTile, per_group = (p.H / p.G) * tiles;
    const int tl = (pair % ppg) * 2 + wg;
    const bool on = tl < per_group;
    const int h = g * (p.H / p.G) + (on ? tl / tiles : 0), p0 = on ? (tl % tiles) * kTile : 0, np = on ? min(kTile, p.P - p0) : 0;
    const int cx = h * p.P + p0, gtile = h * tiles + p0 / kTile;

    // the state that enters: thread = state n, registers = rows of the tile.  A sequence in one segment
    // takes its slot's state.  One in several must not read the slot here (the last segment's CTA may
    // have written it already): the first pass runs segment 0 from it and puts a copy in the place of the
    // last segment, which that pass does not run.
    float S[kTile];
    const float* slot_state =
        p.state + (static_cast<int64_t>(max(s.slot, 0)) * p.H + h) * p.P * p.N + static_cast<int64_t>(p0) * p.N + t;
    auto segment = [&](int j) { return static_cast<int64_t>(q.seg_base[seq] + j) * q.gtiles + gtile; };
    auto segment_state = [&](int j) { return reinterpret_cast<float4*>(q.seg_state + segment(j) * (kQ * kTile)) + t; };
    auto add_segment = [&](int j, float d) {
        const float4* l = segment_state(j);
#pragma unroll
        for (int i = 0; i < kTile / 4; ++i) {
            const float4 v = l[i * kQ];
            S[4 * i] = fmaf(d, S[4 * i], v.x);
            S[4 * i + 1] = fmaf(d, S[4 * i + 1], v.y);
            S[4 * i + 2] = fmaf(d, S[4 * i + 2], v.z);
            S[4 * i + 3] = fmaf(d, S[4 * i + 3], v.w);
        }
    };
    auto keep_segment = [&](int j) {
        float4* l = segment_state(j);
#pragma unroll
        for (int i = 0; i < kTile / 4; ++i) l[i * kQ] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
    };
    const int nsegs = max(1, (nchunks + q.seg_chunks - 1) / q.seg_chunks);
    const bool from_slot = s.warm && t < p.N && (STATE_ONLY ? seg == 0 || last : nsegs == 1);
#pragma unroll
    for (int i = 0; i < kTile; ++i) S[i] = (from_slot && i < np) ? slot_state[static_cast<int64_t>(i) * p.N] : 0.f;
    if (STATE_ONLY && last) {
        if (on && nsegs > 1) keep_segment(nsegs - 1);
        return;
    }
    if (!STATE_ONLY && on && nsegs > 1) {
        if (seg == 0) add_segment(nsegs - 1, 0.f);
        for (int j = 0; j < seg; ++j) add_segment(j, ex2(q.seg_decay[segment(j)]));      // in order
    }
    if (tid == 0) {
        mbar_init(&sh.bar_bc, 1);
        mbar_init(&sh.bar_cs, 1);
        mbar_init(&sh.bar_st, 1);
        mbar_init(&sh.bar_pv[0], 1);
        mbar_init(&sh.bar_pv[1], 1);
        mbar_fence_init();
        sh.abort = 0;
    }
    __syncwarp();
    if (tid / 32 == 0) tc_alloc(&sh.tmem, kTmemCols);
    if (q.nb == 1)                                                     // states 64 to 127: zeros in B's tiles
        for (int i = tid; i < static_cast<int>(kBlock / 16); i += kTcThreads) {
            *reinterpret_cast<uint4*>(img + kBlock + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(img + kImage + kBlock + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
    const uint8_t* src = q.images + (static_cast<int64_t>(q.chunk_base[seq]) * p.G + g) * (3 * q.nb * static_cast<int64_t>(kBlock));
    const int64_t src_step = static_cast<int64_t>(p.G) * 3 * q.nb * kBlock;
    const uint32_t part = q.nb * kBlock;
    auto load_bc = [&](int c) {
        mbar_expect_tx(&sh.bar_bc, (STATE_ONLY ? 2 : 3) * part);
        const uint8_t* f = src + c * src_step;
        bulk_load(img, f, part, &sh.bar_bc);
        bulk_load(img + kImage, f + part, part, &sh.bar_bc);
        if (!STATE_ONLY) bulk_load(img + 2 * kImage, f + 2 * part, part, &sh.bar_bc);
    };

    auto store_state_tile = [&]() {                                    // S rounded, for C·S
#pragma unroll
        for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(sS + tc_chunk(t, c)) =
                make_uint4(pack_bf16(S[8 * c], S[8 * c + 1]), pack_bf16(S[8 * c + 2], S[8 * c + 3]),
                           pack_bf16(S[8 * c + 4], S[8 * c + 5]), pack_bf16(S[8 * c + 6], S[8 * c + 7]));
    };
    if (!STATE_ONLY) store_state_tile();
    tma_store_fence();                                                 // (generic writes, for the tensor cores)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem, lanes = static_cast<uint32_t>(warp) << 21;      // this warp's lanes: 32·warp << 16
    if (tid == 0 && ch0 < ch1) load_bc(ch0);

    const float A2 = on ? -expf(p.A_log[h]) * kLog2e : 0.f, dbias = (on && p.dt_bias) ? p.dt_bias[h] : 0.f;
    const float Dh = (on && p.D) ? p.D[h] : 0.f;
    // x: a thread has 4 channels of 16 tokens
    const int qd = t % 16, tg = t / 16, nq = min(4, np - 4 * qd);
    float cw[4][4], cb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int k = 0; k < 4; ++k) cw[i][k] = i < nq ? p.conv_w[static_cast<int64_t>(cx + 4 * qd + i) * 4 + k] : 0.f;
        cb[i] = (i < nq && p.conv_b) ? p.conv_b[cx + 4 * qd + i] : 0.f;
    }
    const int row0 = tg * 16;
    const TIO* xg = static_cast<const TIO*>(p.xbc) + s.row0 * p.xbc_t + cx + 4 * qd;
    const TIO* zg = p.z ? static_cast<const TIO*>(p.z) + s.row0 * p.z_t + cx + 4 * qd : nullptr;
    TIO* yg = static_cast<TIO*>(p.y) + s.row0 * p.y_t + cx + 4 * qd;
    Quad4<TIO, VEC> raw[19];                                           // samples row0 - 3 .. row0 + 15 of a chunk
    auto load_x = [&](int c) {
#pragma unroll
        for (int j = 0; j < 19; ++j) {
            const int tk = c * kQ + row0 + j - 3;
            raw[j].load(xg + static_cast<int64_t>(max(tk, 0)) * p.xbc_t, (tk >= 0 && tk < s.len) ? nq : 0);
        }
    };
    const TIO* dg = static_cast<const TIO*>(p.dt_raw) + s.row0 * p.dt_t + h;
    if (ch0 < ch1) load_x(ch0);
    float decay_sum = 0.f;
    volatile int* abort = &sh.abort;
    TcTables& tab = sh.tab[wg];

    auto wait = [&](uint64_t* bar, uint32_t parity) {                  // for a product's completion
        mbar_wait_bounded(bar, parity, abort, p.err);
        __syncwarp();
        tc_fence_after();
    };

    for (int c = ch0; c < ch1; ++c) {
        const int tok0 = c * kQ, nt = min(kQ, s.len - tok0);
        const uint32_t ph = (c - ch0) & 1;
        // scores and C·S: the tiles are there, S was written before the last barrier
        if (tid == 0) {
            mbar_wait_bounded(&sh.bar_bc, ph, abort, p.err);
            if (!STATE_ONLY) {
                tc_fence_after();
                const uint32_t b = smem_addr(img), cc = b + 2 * kImage, st = smem_addr(smem + 3 * kImage + 3 * kBlock);
                for (int k = 0; k < 4 * q.nb; ++k) {
                    const uint32_t at = (k / 4) * kBlock + (k % 4) * 32;
                    tc_mma(tmem + kColScore, tc_desc(cc + at, 16, 1024), tc_desc(b + at, 16, 1024), tc_idesc(128, 128, false, false),
                           k > 0);
                }
                for (int k = 0; k < 4 * q.nb; ++k)
                    tc_mma(tmem + kColY, tc_desc(cc + (k / 4) * kBlock + (k % 4) * 32, 16, 1024),
                           tc_desc(st + k * 2048, kTileBytes, 1024), tc_idesc(128, 128, false, true), k > 0);
                tc_commit(&sh.bar_cs);
            }
        }
        __syncwarp();
        // time steps: thread = token
        float dt = 0.f;
        if (on && t < nt) dt = softplus(to_f32<TIO>(dg[static_cast<int64_t>(tok0 + t) * p.dt_t]) + dbias);
        const float a = dt * A2;
        float l = a, r = __shfl_down_sync(0xffffffffu, a, 1);          // sums up to t, and after t, in the block of 32
        if (lane == 31) r = 0.f;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const float u = __shfl_up_sync(0xffffffffu, l, o), d = __shfl_down_sync(0xffffffffu, r, o);
            if (lane >= o) l += u;
            if (lane + o < 32) r += d;
        }
        if (lane == 31) tab.total[warp] = l;
        wg_sync(wg);
        float before = 0.f, all = 0.f, after = r;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float v = tab.total[w];
            all += v;
            if (w < warp) before += v;
            if (w > warp) {
                if (!STATE_ONLY) tab.fac[(w - 1) * w / 2 * 32 + t] = dt * ex2(after);   // blocks 1, 2, 3 at 0, 32, 96
                after += v;
            }
        }
        tab.tail[t] = dt * ex2(after);
        decay_sum += all;
        wg_sync(wg);
        // x, through the convolution
        uint2 xlo[16];                                                 // what bf16 leaves of it, for D·x
        float4 e0 = raw[0].get(), e1 = raw[1].get(), e2 = raw[2].get();
        if (c == 0 && tg == 0 && s.warm) {
            float v[3][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                HeadsWindow w = {{0.f, 0.f, 0.f}};
                if (i < nq) w = heads_window(p, s, cx + 4 * qd + i);
                v[0][i] = w.v[0];
                v[1][i] = w.v[1];
                v[2][i] = w.v[2];
            }
            e0 = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
            e1 = make_float4(v[1][0], v[1][1], v[1][2], v[1][3]);
            e2 = make_float4(v[2][0], v[2][1], v[2][2], v[2][3]);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int row = row0 + j;
            const float m = tab.tail[row];
            const float4 f = raw[j + 3].get();
            float u[4];
            u[0] = heads_conv(cw[0], cb[0], e0.x, e1.x, e2.x, f.x);
            u[1] = heads_conv(cw[1], cb[1], e0.y, e1.y, e2.y, f.y);
            u[2] = heads_conv(cw[2], cb[2], e0.z, e1.z, e2.z, f.z);
            u[3] = heads_conv(cw[3], cb[3], e0.w, e1.w, e2.w, f.w);
            e0 = e1;
            e1 = e2;
            e2 = f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (row >= nt || i >= nq) u[i] = 0.f;
            const uint32_t off = tc_chunk(row, qd / 2) + (qd & 1) * 8;
            if (!STATE_ONLY) {
                const uint2 x = make_uint2(pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]));
                *reinterpret_cast<uint2*>(sX + off) = x;
                xlo[j] = make_uint2(pack_bf16(u[0] - bf16_lo(x.x), u[1] - bf16_hi(x.x)),
                                    pack_bf16(u[2] - bf16_lo(x.y), u[3] - bf16_hi(x.y)));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] *= m;
            const uint2 hi = make_uint2(pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]));
            *reinterpret_cast<uint2*>(sXh + off) = hi;
            *reinterpret_cast<uint2*>(sXl + off) = make_uint2(pack_bf16(u[0] - bf16_lo(hi.x), u[1] - bf16_hi(hi.x)),
                                                              pack_bf16(u[2] - bf16_lo(hi.y), u[3] - bf16_hi(hi.y)));
        }
        if (c + 1 < ch1) load_x(c + 1);
        tma_store_fence();
        __syncthreads();
        // what the chunk adds to the state, both tiles side by side
        if (tid == 0) {
            tc_fence_after();
            const uint32_t b = smem_addr(img), x = smem_addr(smem + 3 * kImage + kBlock);
            for (int k = 0; k < 8; ++k) {
                const uint64_t bh = tc_desc(b + k * 2048, kBlock, 1024), bl = tc_desc(b + kImage + k * 2048, kBlock, 1024);
                const uint64_t xh = tc_desc(x + k * 2048, kTileBytes, 1024), xl = tc_desc(x + kBlock + k * 2048, kTileBytes, 1024);
                constexpr uint32_t id = tc_idesc(128, 128, true, true);
                tc_mma(tmem + kColS, bh, xl, id, k > 0);
                tc_mma(tmem + kColS, bl, xh, id, true);
                tc_mma(tmem + kColS, bh, xh, id, true);
            }
            tc_commit(&sh.bar_st);
        }
        __syncwarp();
        if (!STATE_ONLY) {
            wait(&sh.bar_cs, ph);
            // exp2(l)·(C·S)
            const float carry = ex2(before + l);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t v[32];
                tc_ld32(tmem + lanes + kColY + wg * 64 + k * 32, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * carry);
                tc_st32(tmem + lanes + kColY + wg * 64 + k * 32, v);
            }
            // P: thread = row t; the blocks of 32 columns before its own by a product of two decays, its own
            // by the decay itself, the ones after it zero
            const float mine = ex2(l);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t o[16];
                if (j <= warp) {
                    uint32_t v[32];
                    tc_ld32(tmem + lanes + kColScore + j * 32, v);
                    if (j < warp) {
                        const float4* f = reinterpret_cast<const float4*>(&tab.fac[(warp - 1) * warp / 2 * 32 + j * 32]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 w = f[i];
                            o[2 * i] = pack_bf16(__uint_as_float(v[4 * i]) * w.x * mine, __uint_as_float(v[4 * i + 1]) * w.y * mine);
                            o[2 * i + 1] = pack_bf16(__uint_as_float(v[4 * i + 2]) * w.z * mine, __uint_as_float(v[4 * i + 3]) * w.w * mine);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float ls = __shfl_sync(0xffffffffu, l, i), ds = __shfl_sync(0xffffffffu, dt, i);
                            const float w = __uint_as_float(v[i]) * ds * ex2(l - ls);
                            v[i] = i <= lane ? __float_as_uint(w) : 0u;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = pack_bf16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = 0u;
                }
                tc_st16(tmem + lanes + kColP + wg * 64 + j * 16, o);
            }
            tc_wait_st();
            tc_fence_before();
            wg_sync(wg);
            if (t == 0) {
                tc_fence_after();
                const uint32_t x = smem_addr(sX);
                for (int k = 0; k < 8; ++k)
                    tc_mma_ta(tmem + kColY + wg * 64, tmem + kColP + wg * 64 + k * 8, tc_desc(x + k * 2048, 16, 1024),
                              tc_idesc(128, 64, false, true), true);
                tc_commit(&sh.bar_pv[wg]);
            }
            __syncwarp();
        }
        Quad4<TIO, VEC> gate[16];
        if (!STATE_ONLY && zg)
#pragma unroll
            for (int j = 0; j < 16; ++j)
                gate[j].load(zg + static_cast<int64_t>(tok0 + row0 + j) * p.z_t, row0 + j < nt ? nq : 0);
        // the state
        wait(&sh.bar_st, ph);
        if (tid == 0 && c + 1 < ch1 && !*abort) load_bc(c + 1);          // the products that read B and C are done
        __syncwarp();
        {
            const float d = ex2(all);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t v[32];
                tc_ld32(tmem + lanes + kColS + wg * 64 + k * 32, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) S[32 * k + i] = fmaf(d, S[32 * k + i], __uint_as_float(v[i]));
            }
        }
        if (!STATE_ONLY) {
            store_state_tile();
            wait(&sh.bar_pv[wg], ph);
            // y: rows out of tensor memory, through shared memory, so that 16 threads write a token's 64 channels
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t v[32];
                tc_ld32(tmem + lanes + kColY + wg * 64 + k * 32, v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(stage + t * kTile + (((8 * k + i) ^ (t & 7)) << 2)) =
                        make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
            wg_sync(wg);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int row = row0 + j;
                float4 v = *reinterpret_cast<const float4*>(stage + row * kTile + ((qd ^ (row & 7)) << 2));
                const uint2 x = *reinterpret_cast<const uint2*>(sX + tc_chunk(row, qd / 2) + (qd & 1) * 8);
                v.x = fmaf(Dh, bf16_lo(x.x) + bf16_lo(xlo[j].x), v.x);
                v.y = fmaf(Dh, bf16_hi(x.x) + bf16_hi(xlo[j].x), v.y);
                v.z = fmaf(Dh, bf16_lo(x.y) + bf16_lo(xlo[j].y), v.z);
                v.w = fmaf(Dh, bf16_hi(x.y) + bf16_hi(xlo[j].y), v.w);
                if (zg) {
                    const float4 z = gate[j].get();
                    v.x *= silu(z.x);
                    v.y *= silu(z.y);
                    v.z *= silu(z.z);
                    v.w *= silu(z.w);
                }
                Quad4<TIO, VEC>::store(yg + static_cast<int64_t>(tok0 + row) * p.y_t, row < nt ? nq : 0, v);
            }
            tma_store_fence();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    if (*abort && tid == 0) {                                          // a copy in flight lands before the block ends
        const long long t0 = clock64();
        while (!mbar_try_wait(&sh.bar_bc, (ch1 - ch0 - 1) & 1) && clock64() - t0 < (1ll << 28)) {
        }
    }
    if (STATE_ONLY) {
        if (on) {
            keep_segment(seg);
            if (t == 0) q.seg_decay[segment(seg)] = decay_sum;
        }
    } else if (s.slot >= 0) {
        if (last && on && t < p.N) {
            float* f = const_cast<float*>(slot_state);
#pragma unroll
            for (int i = 0; i < kTile; ++i)
                if (i < np) f[static_cast<int64_t>(i) * p.N] = S[i];
        }
        // the first segment's CTA alone reads its x channels' windows: it shifts them
        if (seg == 0)
            for (int k = t; k < np; k += 128) heads_keep_window<TIO>(p, s, cx + k);
    }
    __syncthreads();
    if (tid / 32 == 0) tc_dealloc(tmem, kTmemCols);
}

// Segments per sequence, for sequences of equal length, in units of a chunk's time: a segment costs a
// first pass of about 0.45 of a full one (no scores, no outputs) and a prologue, the whole call two
// launches; what it buys is CTAs, one to an SM.
int segments_for(int64_t n_seq, int64_t chunks, int64_t pairs, int64_t sms) {
    auto waves = [&](int64_t ctas) { return (ctas + sms - 1) / sms; };
    int best = 1;
    double cost = static_cast<double>(waves(n_seq * pairs)) * static_cast<double>(chunks + 1);
    for (int k = 2; k <= 64 && k <= chunks; ++k) {
        const double len = static_cast<double>((chunks + k - 1) / k);
        const double c = waves(n_seq * pairs * k) * (len + 1.5) + waves(n_seq * pairs * (k - 1)) * (0.45 * len + 1.0) + 2.0;
        if (c < cost) {
            cost = c;
            best = k;
        }
    }
    return best;
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 152;
    }
    return n;
}

size_t padded(size_t n) { return (n + 255) / 256 * 256; }

template <typename TIO, bool VEC>
cudaError_t launch_typed(const HeadsTcParams& q, const HeadsTcPlan& plan, cudaStream_t stream) {
    static_assert(sizeof(TIO) == 2, "bf16 operands of the products carry bf16 inputs");
    const dim3 prep(static_cast<unsigned>(plan.chunks), static_cast<unsigned>(q.p.G), 2u);
    heads_prep_kernel<TIO, VEC><<<prep, kPrepThreads, 0, stream>>>(q);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(plan.segments * plan.pairs);
    if (plan.split) {
        e = cudaFuncSetAttribute(heads_tc_kernel<TIO, VEC, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
        if (e != cudaSuccess) return e;
        heads_tc_kernel<TIO, VEC, true><<<grid, kTcThreads, kTcSmem, stream>>>(q);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    e = cudaFuncSetAttribute(heads_tc_kernel<TIO, VEC, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
    if (e != cudaSuccess) return e;
    heads_tc_kernel<TIO, VEC, false><<<grid, kTcThreads, kTcSmem, stream>>>(q);
    return cudaGetLastError();
}

}  // namespace

// bf16 activations, up to 128 states, and more than 16 tokens a sequence on average: below that the
// token-by-token kernel is faster (about 1 us a token against 5 us a chunk and a second launch).
bool heads_tc_takes(int64_t n_seq, int64_t tokens, int64_t H, int64_t P, int64_t G, int64_t N, bool bf16) {
    (void)P;
    if (!bf16 || N > 128 || tokens <= 16 * n_seq || G > 65535) return false;
    const HeadsTcPlan plan = heads_tc_plan(n_seq, tokens, H, P, G, N);
    return plan.segments * plan.pairs <= INT32_MAX && plan.chunks <= INT32_MAX;
}

HeadsTcPlan heads_tc_plan(int64_t n_seq, int64_t tokens, int64_t H, int64_t P, int64_t G, int64_t N) {
    HeadsTcPlan plan{};
    const int64_t tiles = (P + kHeadsTile - 1) / kHeadsTile;
    plan.nb = N > 64 ? 2 : 1;
    plan.gtiles = static_cast<int>(H * tiles);
    plan.pairs = static_cast<int>(G * ((H / G * tiles + 1) / 2));
    plan.chunks = tokens / kHeadsChunk + n_seq;
    const int64_t mean = (tokens / n_seq + kHeadsChunk - 1) / kHeadsChunk;
    const int k = segments_for(n_seq, std::max<int64_t>(mean, 1), plan.pairs, sm_count());
    plan.split = k > 1;
    plan.seg_chunks = plan.split ? static_cast<int>((mean + k - 1) / k) : INT32_MAX / 2;
    plan.segments = (plan.split ? plan.chunks / plan.seg_chunks : 0) + n_seq;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += padded(n);
        return here;
    };
    plan.off_images = take(static_cast<size_t>(plan.chunks) * G * 3 * plan.nb * kBlock);
    plan.off_chunk_base = take(static_cast<size_t>(n_seq) * 4);
    plan.off_seg_base = take(static_cast<size_t>(n_seq + 1) * 4);
    const size_t states = plan.split ? static_cast<size_t>(plan.segments) * plan.gtiles : 0;
    plan.off_state = take(states * kQ * kTile * 4);
    plan.off_decay = take(states * 4);
    plan.bytes = at;
    return plan;
}

cudaError_t launch_heads_tc(const HeadsParams& p, void* workspace, bool bf16, cudaStream_t stream) {
    if (!bf16) return cudaErrorInvalidValue;
    const HeadsTcPlan plan = heads_tc_plan(p.n_seq, p.tokens, p.H, p.P, p.G, p.N);
    uint8_t* w = static_cast<uint8_t*>(workspace);
    HeadsTcParams q{};
    q.p = p;
    q.images = w + plan.off_images;
    q.chunk_base = reinterpret_cast<int32_t*>(w + plan.off_chunk_base);
    q.seg_base = reinterpret_cast<int32_t*>(w + plan.off_seg_base);
    q.seg_state = reinterpret_cast<float*>(w + plan.off_state);
    q.seg_decay = reinterpret_cast<float*>(w + plan.off_decay);
    q.seg_chunks = plan.seg_chunks;
    q.pairs = plan.pairs;
    q.gtiles = plan.gtiles;
    q.nb = plan.nb;
    // four channels in one access: z, x, B, C and y of every head and group on that boundary
    auto wide = [&](const void* base, int64_t stride) { return host::is_aligned(base, 8) && stride % 4 == 0; };
    const bool vec = p.P % 4 == 0 && p.N % 4 == 0 && wide(p.xbc, p.xbc_t) && wide(p.z, p.z_t) && wide(p.y, p.y_t);
    return vec ? launch_typed<__nv_bfloat16, true>(q, plan, stream) : launch_typed<__nv_bfloat16, false>(q, plan, stream);
}

}  // namespace selscan
