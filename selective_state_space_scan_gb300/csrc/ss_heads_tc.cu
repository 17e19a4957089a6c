// Multi-head selective scan over packed prompts on the tensor cores: 128 tokens at a time.
//
// With one decay per head the recurrence over a chunk of tokens is three matrix products.  Let a_t be
// the log2 decay of token t, l_t its running sum within the chunk, and S the state that enters:
//   Y   = exp2(l_t) (C_t · S) + Σ_{s<=t} exp2(l_t - l_s) Δ_s (C_t · B_s) x_s,   y = Y + D x
//   S'  = exp2(l_end) S + Σ_s exp2(l_end - l_s) Δ_s B_s ⊗ x_s
// heads_prep_kernel convolves B and C once per chunk and group and leaves them as shared-memory
// images of bf16 operand tiles: B as a sum of two bf16 (hi + lo), C rounded.  heads_tc_kernel walks
// the chunks of one sequence (or of a segment of it) for two tiles of 64 rows of the state (two heads,
// as a rule), two warpgroups for each:
//   scores C·Bᵀ (C·hi + C·lo), and C·S        while the warpgroups convolve x, as tiles of x and of
//                                             x scaled for the state (hi + lo)
//   the state's products, hi·hi + hi·lo + lo·hi   while they turn scores into P (decay, Δ, mask)
//   P·x on top of exp2(l)·(C·S), P read from tensor memory
// The state itself stays in registers, fp32: what the chunk adds comes out of tensor memory.
//
// Rounding: the state's operands carry 16 bits each and the product of their low parts is left out, so a state
// is off by about 4e-6 of its norm (in fp32: 1e-6).  y is rounded to bf16 in the end; the factors C, S, P and x of
// its sums are rounded to bf16 before the products, each error as large as that last one, and D·x is not.  B is
// not either (hi + lo in the scores too): where one token's step outweighs all others', the error of its score is that
// of every output behind it, and C·B cancels.  y of such prompts is off by 3e-3 to 4.8e-3 (with B in one bf16 by
// up to 5.7e-3; the second product costs 0.15 us a chunk), of others by 2e-3, 1.7e-3 of which are its own rounding.
// A decay is the exp2 of the sum of the steps between its two tokens, never a quotient.  From one block of 32
// tokens to another, and to the chunk's end, these sums are taken over the steps themselves; within a block (P's
// diagonal) as the difference of two running sums, whose steps are cut at 2^-128, where a decay is zero whatever else
// it meets: the sums stay above -4096, whose ten roundings leave a decay behind strong steps off by less than 1e-3
// (not cut, a single step of 1e5 leaves y off by 4e-2, one of 1e6 by 0.35).
// P is zero above the diagonal, and zero times an infinity or NaN is NaN: such x are zeros in P·x, and their channel's
// outputs from that token on are set to NaN (as the recurrence leaves them) after it.
//
// What bounds it is the chain within a chunk (loads, convolution, products, P, products, outputs), with one
// CTA of 16 warps on an SM: two tiles' operands and accumulators fill its shared and tensor memory.  Four
// sequences of 8192 tokens, 80 heads of 64 x 128 states, bf16, gated: 770 us, 11.4 us a chunk and SM, at 42% of
// the issue slots, 17% of the tensor pipe and 15% of the memory's peak (153 us are the copy rate's): no unit is full,
// and global loads in the middle of the chain are the longest stall.  One document of 32768 tokens, 24 heads: 397 us
// in two passes (47 at the copy rate).  Token by token (see ss_heads_fwd.cu) the FMA pipe alone would take 1.7 and
// 0.5 ms.
// Measured (against 715 to 735 us then) and not taken: one tile per product (N = 64), which shared memory's bandwidth
// bounds (940 us), a warp for issuing alone (96 registers a thread, spills), x or z a chunk ahead in registers
// (841), waves of 2 or 8 chunks (no gain), equal ranges of chunks for every CTA (three times as long).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstdlib>

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
constexpr int kTcThreads = 512;                    // two warpgroups per tile

// ---- where the chunks and segments of the sequences are

// Chunks of sequence `seq`: at least one, so that an empty sequence is visited too; none if its
// indexes are out of range or out of order.
__device__ __forceinline__ int chunks_of(const HeadsParams& p, int seq, bool in_order) {
    if (seq >= p.n_seq || !in_order) return 0;
    const HeadsSeq s = heads_seq(p, seq);
    return s.ok ? max(1, (s.len + kQ - 1) / kQ) : 0;
}

// ---- B and C

// Four channels of a row as loaded, `n` of them existing, and where they begin in their first word.
// VEC: all or none, in one aligned access of 8 bytes.  Otherwise rows begin anywhere: the aligned words
// that hold the channels are loaded (a third one only where the row begins inside a word) and shifted into
// place at use.  A word that holds a channel that exists is readable as a whole; what else it holds belongs
// to channels past the last, whose columns reach no result.
template <bool VEC> struct Quad4;
template <> struct Quad4<true> {
    uint2 u;
    static __device__ __forceinline__ uint32_t shift(const __nv_bfloat16*) { return 0u; }
    __device__ __forceinline__ void load(const __nv_bfloat16* q, int n, uint32_t) {
        u = make_uint2(0u, 0u);
        if (n > 0) u = *reinterpret_cast<const uint2*>(q);
    }
    __device__ __forceinline__ uint2 bits(uint32_t) const { return u; }
};
template <> struct Quad4<false> {
    uint32_t w[3];
    static __device__ __forceinline__ uint32_t shift(const __nv_bfloat16* q) {
        return (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q)) & 2u) * 8u;
    }
    __device__ __forceinline__ void load(const __nv_bfloat16* q, int n, uint32_t sh) {
        const uint32_t* f = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(q) & ~static_cast<uintptr_t>(3));
        w[0] = w[1] = w[2] = 0u;
        if (n > 0) {
            const int words = (n + (sh ? 1 : 0) + 1) / 2;
            w[0] = f[0];
            if (words > 1) w[1] = f[1];
            if (words > 2) w[2] = f[2];
        }
    }
    __device__ __forceinline__ uint2 bits(uint32_t sh) const {
        return make_uint2(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh));
    }
};
__device__ __forceinline__ float4 quad_floats(uint2 u) { return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y)); }

// The same in the scan, where 16 lanes of a warp hold a row of a tile's 64 channels and a thread holds many
// rows: without VEC a lane loads the two words at its channels and takes the third from the lane after it;
// the last lane's third words of all rows (up to 16) are spread over the lanes of the row (load_tail).
// Sequences of 8192 tokens, 128 states, time over chunks per SM: 11.6 us with VEC (4, 76 heads), 15.9 at rows of
// 4-byte boundaries (8, 38 heads), 17.9 at any (4, 77 heads).  At 4-byte boundaries three words a row and thread (276
// bytes of spills) took 16.7 where this took 14.7 then, and one access per channel 22.6.
template <bool VEC> struct Row4 : Quad4<true> {
    __device__ __forceinline__ uint2 bits(uint32_t, uint32_t, int, int) const { return u; }
};
template <> struct Row4<false> {
    uint32_t w0, w1;
    __device__ __forceinline__ void load(const __nv_bfloat16* q, int n, uint32_t sh) {
        const uint32_t* f = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(q) & ~static_cast<uintptr_t>(3));
        const int m = n + (sh ? 1 : 0);            // channels from the first word's beginning (n < 0: no such row)
        w0 = m > 0 ? f[0] : 0u;
        w1 = m > 2 ? f[1] : 0u;
    }
    // all lanes at once; qd: the lane's place in its row, j: the row's number
    __device__ __forceinline__ uint2 bits(uint32_t sh, uint32_t tails, int qd, int j) const {
        const uint32_t next = __shfl_down_sync(0xffffffffu, w0, 1, 16), tail = __shfl_sync(0xffffffffu, tails, j, 16);
        return make_uint2(__funnelshift_r(w0, w1, sh), __funnelshift_r(w1, qd == 15 ? tail : next, sh));
    }
};
// The word that begins with channel 63 of row j, for lane j; q: channel 0 of row 0.  (Where rows begin at words it
// is not used.)
template <bool VEC>
__device__ __forceinline__ uint32_t load_tail(const __nv_bfloat16* q, int64_t stride, bool on, int j) {
    if (VEC || !on) return 0u;
    const __nv_bfloat16* f = q + j * stride + 63;
    return Quad4<false>::shift(f) == 0 ? *reinterpret_cast<const uint32_t*>(f) : 0u;
}

// Stores the first n of four channels; wide: every head's quads of y are on boundaries of 8 bytes.
template <bool VEC>
__device__ __forceinline__ void quad_store(__nv_bfloat16* q, int n, bool wide, float2 a, float2 b) {
    const uint2 u = make_uint2(pack_bf16(a.x, a.y), pack_bf16(b.x, b.y));
    if (VEC || (wide && (n & 3) == 0)) {
        if (n > 0) *reinterpret_cast<uint2*>(q) = u;
        return;
    }
    uint16_t* h = reinterpret_cast<uint16_t*>(q);
    if (n >= 4 && Quad4<false>::shift(q) == 0) {
        reinterpret_cast<uint32_t*>(q)[0] = u.x;
        reinterpret_cast<uint32_t*>(q)[1] = u.y;
    } else if (n >= 4) {
        h[0] = static_cast<uint16_t>(u.x);
        *reinterpret_cast<uint32_t*>(h + 1) = __funnelshift_r(u.x, u.y, 16);
        h[3] = static_cast<uint16_t>(u.y >> 16);
    } else {
        if (n > 0) h[0] = static_cast<uint16_t>(u.x);
        if (n > 1) h[1] = static_cast<uint16_t>(u.x >> 16);
        if (n > 2) h[2] = static_cast<uint16_t>(u.y);
    }
}

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
    int base = 0, sbase = 0, largest = 0;
    for (int s0 = 0; s0 < p.n_seq; s0 += kPrepThreads) {
        const int seq = s0 + tid, n = chunks_of(p, seq, heads_in_order(p, seq, largest, scratch));
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
    if (first && tid == 0) {
        q.seg_base[p.n_seq] = sbase;
        q.chunk_base[p.n_seq] = base;
    }
    if (first)
        for (int i = tid; i < q.nflags; i += kPrepThreads) q.flags[i] = 0u;
    __syncthreads();
    if (found[0] < 0) return;
    const int seq = found[0], chunk = found[1], which = blockIdx.z;
    if (g == 0 && which == 0 && chunk % q.seg_chunks == 0) {
        // the segment's place among all: after those of lower number, and those of its number in sequences before
        const int seg = chunk / q.seg_chunks;
        int at = 0, up_to = 0;
        for (int s0 = 0; s0 < p.n_seq; s0 += kPrepThreads) {
            const bool in_order = heads_in_order(p, s0 + tid, up_to, scratch);
            const int n = (chunks_of(p, s0 + tid, in_order) + q.seg_chunks - 1) / q.seg_chunks;
            int total;
            block_prefix(min(n, seg) + (n > seg && s0 + tid < seq ? 1 : 0), &total, scratch);
            at += total;
        }
        if (tid == 0) {
            q.order[2 * at] = seq;
            q.order[2 * at + 1] = seg;
        }
    }
    const HeadsSeq s = heads_seq(p, seq);
    const int c0 = p.H * p.P + (which ? p.G * p.N : 0) + g * p.N;      // first channel
    const int quads = q.nb * 16, qd = tid % quads, rows = kQ * quads / kPrepThreads, r0 = (tid / quads) * rows;
    const int ch = qd * 4, n = min(4, p.N - ch), t0 = chunk * kQ;
    uint8_t* img = q.images + (static_cast<int64_t>(id) * p.G + g) * (3 * q.nb * static_cast<int64_t>(kBlock));
    uint8_t* hi = img + (which ? 2 * q.nb * kBlock : 0) + (qd / 16) * kBlock;
    uint8_t* lo = img + q.nb * kBlock + (qd / 16) * kBlock;            // B only
    const TIO* x = static_cast<const TIO*>(p.xbc) + s.row0 * p.xbc_t + c0 + ch;
    constexpr int kRows = 8;                                           // a round: its loads are issued together
    Quad4<VEC> raw[kRows];
    const uint32_t sh0 = Quad4<VEC>::shift(x), sh1 = Quad4<VEC>::shift(x + p.xbc_t);    // of even rows, and of odd ones
    auto load_round = [&](int r) {
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const int t = t0 + r0 + r + j;
            raw[j].load(x + t * p.xbc_t, t < s.len ? n : 0, t & 1 ? sh1 : sh0);
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
        Quad4<VEC> f;
        const uint32_t sh = t & 1 ? sh1 : sh0;
        f.load(x + static_cast<int64_t>(max(t, 0)) * p.xbc_t, (t >= 0 && t < s.len) ? n : 0, sh);
        e[j] = quad_floats(f.bits(sh));
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
            const float4 f = quad_floats(raw[j].bits(j & 1 ? sh1 : sh0));      // (a round begins at an even row)
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
constexpr float kLeastDecay = -128.f;              // log2 of a step's decay at least: ex2 of it is zero, as of all below
constexpr int kFacs = 192;                         // decay factors of the blocks off the diagonal
constexpr uint32_t kNoBad = 0x01010101u * kQ;
constexpr int kToks = 8;                           // tokens per thread in the convolution and the output
struct alignas(16) TcTables {                      // (read in runs of four floats)
    float tail[kQ];                                // Δ_s · decay from s to the chunk's end
    float fac[kFacs];                              // Δ_s · decay from s to the start of a later block of 32
    float total[4];                                // log2 decay of the blocks of 32
    uint32_t bad[kTile / 4];                       // a channel's first token that is not finite (a byte each; kQ: none)
};
struct TcShared {
    uint64_t bc;                                   // B and C have arrived
    uint64_t cs, st, pv[2];                        // products complete: scores and C·S; state; P·x of a tile
    uint64_t x_ready, p_ready[2], y_free;          // operands written: x tiles; P; S (and the last y read)
    uint64_t drain[2];                             // everything a tile's issuer has issued (after a wait that ran out)
    uint32_t tmem;
    int abort;
    uint32_t loads;                                // of B and C so far (its issuer's alone)
    TcTables tab[2];
};
constexpr uint32_t kTcSmem = 3 * kImage + 2 * kTileBytes + sizeof(TcShared);
static_assert(offsetof(TcTables, fac) % 16 == 0 && offsetof(TcTables, bad) % 16 == 0 && offsetof(TcShared, tab) % 16 == 0, "16-byte loads");
static_assert(kTcSmem <= 232448, "227 KB of shared memory per CTA");

// Columns of tensor memory: scores, C·S and then y of both tiles, what the chunk adds to the state of
// both tiles, P of both tiles (two bf16 a column).
constexpr uint32_t kColScore = 0, kColY = 128, kColS = 256, kColP = 384, kTmemCols = 512;

enum class Pass {
    kWaves,       // one launch: the segments in the order of their place in their sequence, dealt out to
                  // the CTAs; a segment takes the state that the one before it left
    kStates,      // time split, first pass: the state that each segment but the last leaves; no outputs
    kSegments     // time split, second pass: every segment from the state that enters it
};

// Consecutive chunks of one sequence for one pair of tiles.
struct Piece {
    int seq, seg, pair, ch0, ch1, nchunks;   // nchunks: of the sequence, at least 1
};

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// One arrival per warp, after the writes of all its lanes.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}

// Whether all are finite, of bf16 pairs: times zero and summed they are zero or NaN.
__device__ __forceinline__ bool all_finite(const uint2 (&v)[kToks]) {
    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
    __nv_bfloat162 a = zero, b = zero;
#pragma unroll
    for (int j = 0; j < kToks; ++j) {
        a = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v[j].x), zero, a);
        b = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v[j].y), zero, b);
    }
    a = __hadd2(a, b);
    return (*reinterpret_cast<const uint32_t*>(&a) & 0x7fff7fffu) == 0u;
}

// Waits (with a limit, longer than any chain of segments takes) until *flag has reached n.
__device__ __forceinline__ void wait_flag(const unsigned int* flag, unsigned int n, volatile int* abort, unsigned int* err) {
    const long long t0 = clock64();
    for (;;) {
        unsigned int v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
        if (v >= n || *abort) return;
        if (clock64() - t0 > (1ll << 34)) {
            *abort = 1;
            if (err) atomicOr(err, kErrWaitTimeout);
            return;
        }
    }
}

template <typename TIO, bool VEC, Pass PASS>
__global__ void __launch_bounds__(kTcThreads, 1) heads_tc_kernel(const HeadsTcParams q) {
    constexpr bool kOut = PASS != Pass::kStates;
    extern __shared__ __align__(1024) uint8_t smem[];
    const HeadsParams& p = q.p;
    uint8_t* img = smem;                                               // B hi, B lo, C
    TcShared& sh = *reinterpret_cast<TcShared*>(smem + 3 * kImage + 2 * kTileBytes);
    volatile int* abort = &sh.abort;
    const int tid = threadIdx.x;

    // this CTA's pieces: a segment for a pair of tiles each.  Pairs run fastest, so that the CTAs at work
    // read the same rows of the tokens (a tile's share of a row is 128 bytes).
    const int64_t items = static_cast<int64_t>(q.seg_base[p.n_seq]) * q.pairs;
    if (blockIdx.x >= items) return;
    auto each_piece = [&](auto&& f) {
        for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
            Piece c;
            const int u = static_cast<int>(i / q.pairs);
            c.pair = static_cast<int>(i - static_cast<int64_t>(u) * q.pairs);
            c.seq = q.order[2 * u];
            c.seg = q.order[2 * u + 1];
            c.nchunks = q.chunk_base[c.seq + 1] - q.chunk_base[c.seq];
            c.ch0 = c.seg * q.seg_chunks;
            c.ch1 = min(c.nchunks, c.ch0 + q.seg_chunks);
            if (PASS == Pass::kStates && c.nchunks <= q.seg_chunks) continue;      // one segment: nothing to prepare
            f(c);
        }
    };

    if (tid == 0) {
        mbar_init(&sh.bc, 1);
        mbar_init(&sh.cs, 1);
        mbar_init(&sh.st, 1);
        mbar_init(&sh.pv[0], 1);
        mbar_init(&sh.pv[1], 1);
        mbar_init(&sh.x_ready, 16);
        mbar_init(&sh.p_ready[0], 8);
        mbar_init(&sh.p_ready[1], 8);
        mbar_init(&sh.y_free, 16);
        mbar_init(&sh.drain[0], 1);
        mbar_init(&sh.drain[1], 1);
        sh.loads = 0u;
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
    tma_store_fence();                                                 // (generic writes, for the tensor cores)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const int ppg = q.pairs / p.G, tiles = (p.P + kTile - 1) / kTile, per_group = (p.H / p.G) * tiles;
    uint32_t it = 0;                                                   // chunks so far: the barriers' phases

    {
        // two warpgroups to a tile: both have all 128 tokens (or states) as their lanes, and half of the
        // columns each
        const int wg = tid / 256, hf = (tid / 128) & 1, t = tid % 128, warp = t / 32, lane = t % 32;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp) << 21);        // this warp's lanes: 32·warp << 16
        uint8_t* tile = smem + 3 * kImage + wg * kTileBytes;
        uint8_t *sX = tile, *sXh = tile + kBlock, *sXl = tile + 2 * kBlock, *sS = tile + 3 * kBlock;
        float* stage = reinterpret_cast<float*>(sXh);                  // y, over x scaled (hi and lo)
        TcTables& tab = sh.tab[wg];
        auto tile_sync = [&]() { named_barrier(1 + wg, 256); };
        auto wait = [&](uint64_t* bar, uint32_t parity) {              // for a product's completion
            mbar_sleep_bounded(bar, parity, abort, p.err);
            __syncwarp();
            tc_fence_after();
        };
        // The products are issued by threads of the warps that have no block of P on or below the diagonal:
        // P·x of a tile by the tile's own, all others by the first tile's.
        const bool issue_pv = hf == 1 && t == 0, issue = issue_pv && wg == 0;
        const uint32_t b_at = smem_addr(img), c_at = b_at + 2 * kImage, x_at = smem_addr(smem + 3 * kImage);
        // the convolution and the output: a thread has 4 channels of 8 tokens
        const int qd = t % 16, row0 = (hf * 8 + t / 16) * kToks;

        each_piece([&](const Piece& c) {
            const HeadsSeq s = heads_seq(p, c.seq);
            const int ch1 = min(c.ch1, (s.len + kQ - 1) / kQ);
            const bool begins = c.ch0 == 0, ends = c.ch1 >= c.nchunks;
            // the tile: tiles of a group are numbered head by head, two of them to a CTA
            const int g = c.pair / ppg, tl = (c.pair % ppg) * 2 + wg;
            const bool on = tl < per_group;
            const int h = g * (p.H / p.G) + (on ? tl / tiles : 0), p0 = on ? (tl % tiles) * kTile : 0;
            const int np = on ? min(kTile, p.P - p0) : 0, cx = h * p.P + p0, gtile = h * tiles + p0 / kTile;
            const int nq = np > 0 ? min(4, np - 4 * qd) : -1;

            const uint8_t* src =
                q.images + (static_cast<int64_t>(q.chunk_base[c.seq]) * p.G + g) * (3 * q.nb * static_cast<int64_t>(kBlock));
            auto load_bc = [&](int ch) {
                const uint32_t part = q.nb * kBlock;
                const uint8_t* f = src + static_cast<int64_t>(ch) * p.G * 3 * part;
                ++sh.loads;
                mbar_expect_tx(&sh.bc, (kOut ? 3 : 2) * part);
                bulk_load(img, f, part, &sh.bc);
                bulk_load(img + kImage, f + part, part, &sh.bc);
                if (kOut) bulk_load(img + 2 * kImage, f + 2 * part, part, &sh.bc);
            };
            const TIO* xg = static_cast<const TIO*>(p.xbc) + s.row0 * p.xbc_t + cx + 4 * qd;
            Row4<VEC> raw[kToks + 3];                                  // samples row0 - 3 .. of a chunk
            // where they begin in a word: row0 - 3 and every second row, and the others
            const uint32_t sh0 = Quad4<VEC>::shift(xg - p.xbc_t), sh1 = Quad4<VEC>::shift(xg);
            uint32_t raw_tail = 0u;
            auto load_x = [&](int ch) {
                const int tk = ch * kQ + row0 - 3;
                const TIO* f = xg + static_cast<int64_t>(tk) * p.xbc_t;
                raw_tail = load_tail<VEC>(f - 4 * qd, p.xbc_t, np >= kTile && qd < kToks + 3 && tk + qd >= 0 && tk + qd < s.len, qd);
#pragma unroll
                for (int j = 0; j < kToks + 3; ++j) {
                    raw[j].load(f, (tk + j >= 0 && tk + j < s.len) ? nq : -1, j & 1 ? sh1 : sh0);
                    f += p.xbc_t;
                }
            };
            const TIO* dg = static_cast<const TIO*>(p.dt_raw) + s.row0 * p.dt_t + h;
            auto load_dt = [&](int ch) {
                const int tk = ch * kQ + t;
                return (on && tk < s.len) ? to_f32<TIO>(dg[static_cast<int64_t>(tk) * p.dt_t]) : 0.f;
            };
            float dt_next = 0.f;
            // x and z of a chunk into L2, a chunk ahead of their loads: one thread per row of 128 bytes, half
            // the threads for x and half for z
            auto prefetch = [&](int ch) {
                const int tk = ch * kQ + t;
                if (np <= 0 || tk >= s.len) return;
                const TIO* f = hf == 0 ? static_cast<const TIO*>(p.xbc) + (s.row0 + tk) * p.xbc_t + cx
                                       : static_cast<const TIO*>(p.z) + (s.row0 + tk) * p.z_t + cx;
                if (hf == 0 || (kOut && p.z)) asm volatile("prefetch.global.L2 [%0];" ::"l"(f));
            };
            if (c.ch0 < ch1) {
                prefetch(c.ch0);
                dt_next = load_dt(c.ch0);
                // (the last piece's products are complete: this thread has waited for them)
                if (issue && !(PASS == Pass::kStates && ends) && !*abort) load_bc(c.ch0);
            }

            // The state that enters: thread = state n, registers = rows hf·32 .. of the tile.
            // A time-split sequence must not read its slot in the second pass (the last segment's CTA may
            // have written it already): the first pass runs segment 0 from it and puts a copy in the place
            // of the last segment, which that pass does not run.
            float S[32];
            float* slot_state = p.state + ((static_cast<int64_t>(max(s.slot, 0)) * p.H + h) * p.P + p0 + hf * 32) * p.N + t;
            const int my_rows = np - hf * 32;
            auto segment = [&](int j) { return static_cast<int64_t>(q.seg_base[c.seq] + j) * q.gtiles + gtile; };
            auto saved = [&](float* base, int64_t at) {                // [16][128][4] floats per tile
                return reinterpret_cast<float4*>(base + at * (kQ * kTile)) + hf * 8 * kQ + t;
            };
            auto add_saved = [&](const float4* l, float d) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 v = __ldcg(l + i * kQ);
                    S[4 * i] = fmaf(d, S[4 * i], v.x);
                    S[4 * i + 1] = fmaf(d, S[4 * i + 1], v.y);
                    S[4 * i + 2] = fmaf(d, S[4 * i + 2], v.z);
                    S[4 * i + 3] = fmaf(d, S[4 * i + 3], v.w);
                }
            };
            auto save = [&](float4* l) {
#pragma unroll
                for (int i = 0; i < 8; ++i) __stcg(l + i * kQ, make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]));
            };
            const int seg = c.seg, nsegs = (c.nchunks + q.seg_chunks - 1) / q.seg_chunks;
            const int64_t chain = (static_cast<int64_t>(c.seq) * q.pairs + c.pair) * 2 + wg;
            const bool from_slot = s.warm && t < p.N &&
                                   (PASS == Pass::kStates ? begins || ends : PASS == Pass::kWaves ? begins : nsegs == 1);
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = (from_slot && i < my_rows) ? slot_state[static_cast<int64_t>(i) * p.N] : 0.f;
            if (PASS == Pass::kStates && ends) {
                if (on) save(saved(q.seg_state, segment(nsegs - 1)));
                return;
            }
            if (PASS == Pass::kSegments && on && nsegs > 1) {
                if (seg == 0) add_saved(saved(q.seg_state, segment(nsegs - 1)), 0.f);
                for (int j = 0; j < seg; ++j) add_saved(saved(q.seg_state, segment(j)), ex2(q.seg_decay[segment(j)]));
            }
            if (PASS == Pass::kWaves && !begins) {                      // what the segment before left
                if (t == 0 && hf == 0) wait_flag(q.flags + chain, seg, abort, p.err);
                tile_sync();
                add_saved(saved(q.handover, chain), 0.f);
            }
            auto state_tile = [&]() {                                   // S rounded, for C·S
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<uint4*>(sS + tc_chunk(t, hf * 4 + k)) =
                        make_uint4(pack_bf16(S[8 * k], S[8 * k + 1]), pack_bf16(S[8 * k + 2], S[8 * k + 3]),
                                   pack_bf16(S[8 * k + 4], S[8 * k + 5]), pack_bf16(S[8 * k + 6], S[8 * k + 7]));
            };
            if (kOut && c.ch0 < ch1) {
                state_tile();
                tma_store_fence();
                warp_arrive(&sh.y_free);
            }

            const float A2 = on ? -expf(p.A_log[h]) * kLog2e : 0.f, dbias = (on && p.dt_bias) ? p.dt_bias[h] : 0.f;
            const float Dh = (on && p.D) ? p.D[h] : 0.f;
            auto load_weights = [&](float2 (&wk)[2][4], float2 (&wb)[2]) {
                float4 f[4];
                float b[4];
                const float* w = p.conv_w + static_cast<int64_t>(cx + 4 * qd) * 4;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (VEC || q.wide_w)
                        f[i] = i < nq ? *reinterpret_cast<const float4*>(w + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
                    else
                        f[i] = i < nq ? make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3])
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
                    b[i] = (i < nq && p.conv_b) ? p.conv_b[cx + 4 * qd + i] : 0.f;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    wk[i][0] = make_float2(f[2 * i].x, f[2 * i + 1].x);
                    wk[i][1] = make_float2(f[2 * i].y, f[2 * i + 1].y);
                    wk[i][2] = make_float2(f[2 * i].z, f[2 * i + 1].z);
                    wk[i][3] = make_float2(f[2 * i].w, f[2 * i + 1].w);
                    wb[i] = make_float2(b[2 * i], b[2 * i + 1]);
                }
            };
            float decay_sum = 0.f, last_all = 0.f;
            // S <- decay · S + what a chunk added, from its place in tensor memory
            auto update = [&](float all, uint32_t col) {
                const float2 d = splat2(ex2(all));
                uint32_t v[32];
                tc_ld32(lanes + col + wg * 64 + hf * 32, v);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float2 n = fma2(d, make_float2(S[i], S[i + 1]), make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])));
                    S[i] = n.x;
                    S[i + 1] = n.y;
                }
            };

            for (int ch = c.ch0; ch < ch1; ++ch, ++it) {
                const uint32_t ph = it & 1;
                // The first pass has two sets of scaled tiles, accumulators and barriers, and takes a chunk's
                // products in while it convolves the next.  (A tile is at most one chunk ahead of the other: it
                // reaches a set again only behind the products of the set's last chunk.)
                const uint32_t set = kOut ? 0u : ph, set_ph = kOut ? ph : (it >> 1) & 1;
                uint8_t *th = set ? sX : sXh, *tl = set ? sS : sXl;
                uint64_t *st = set ? &sh.cs : &sh.st, *x_ready = set ? &sh.y_free : &sh.x_ready;
                const int tok0 = ch * kQ, nt = min(kQ, s.len - tok0);
                if (kOut && issue) {                                    // scores, and C·S of both tiles
                    mbar_sleep_bounded(&sh.bc, ph, abort, p.err);
                    // (both tiles read one set of scores: the other's P says that it has read the last ones)
                    if (it > 0) mbar_sleep_bounded(&sh.p_ready[1], ph ^ 1, abort, p.err);
                    tc_fence_after();
                    for (int k = 0; k < 4 * q.nb; ++k) {
                        const uint32_t at = (k / 4) * kBlock + (k % 4) * 32;
                        tc_mma(tmem + kColScore, tc_desc(c_at + at, 16, 1024), tc_desc(b_at + kImage + at, 16, 1024),
                               tc_idesc(128, 128, false, false), k > 0);
                        tc_mma(tmem + kColScore, tc_desc(c_at + at, 16, 1024), tc_desc(b_at + at, 16, 1024),
                               tc_idesc(128, 128, false, false), true);
                    }
                    mbar_sleep_bounded(&sh.y_free, ph, abort, p.err);
                    tc_fence_after();
                    for (int k = 0; k < 4 * q.nb; ++k)
                        tc_mma(tmem + kColY, tc_desc(c_at + (k / 4) * kBlock + (k % 4) * 32, 16, 1024),
                               tc_desc(x_at + 3 * kBlock + k * 2048, kTileBytes, 1024), tc_idesc(128, 128, false, true), k > 0);
                    tc_commit(&sh.cs);
                }
                __syncwarp();
                load_x(ch);
                if (ch + 1 < ch1) prefetch(ch + 1);
                float2 wk[2][4], wb[2];
                load_weights(wk, wb);
                // time steps: thread = token (both warpgroups of a tile compute them all)
                const float dt = (on && t < nt) ? softplus(dt_next + dbias) : 0.f;
                const float a = dt * A2 < kLeastDecay ? kLeastDecay : dt * A2;
                float l = a, r = __shfl_down_sync(0xffffffffu, a, 1);   // sums up to t, and after t, in the block of 32
                if (lane == 31) r = 0.f;
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const float u = __shfl_up_sync(0xffffffffu, l, o), d = __shfl_down_sync(0xffffffffu, r, o);
                    if (lane >= o) l += u;
                    if (lane + o < 32) r += d;
                }
                if (lane == 31 && hf == 0) tab.total[warp] = l;
                tile_sync();                                            // (also: the last chunk's y is out of its stage)
                float before = 0.f, all = 0.f, after = r;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float v = tab.total[w];
                    all += v;
                    if (w < warp) before += v;
                    if (w > warp) {
                        if (kOut && hf == 0) tab.fac[(w - 1) * w / 2 * 32 + t] = dt * ex2(after);   // blocks 1, 2, 3 at 0, 32, 96
                        after += v;
                    }
                }
                if (hf == 0) tab.tail[t] = dt * ex2(after);
                if (kOut && hf == 0 && t < kTile / 4) tab.bad[t] = kNoBad;
                decay_sum += all;
                // x, through the convolution
                float4 e0 = quad_floats(raw[0].bits(sh0, raw_tail, qd, 0)), e1 = quad_floats(raw[1].bits(sh1, raw_tail, qd, 1)),
                       e2 = quad_floats(raw[2].bits(sh0, raw_tail, qd, 2));
                if (ch == 0 && row0 == 0 && s.warm) {
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
                tile_sync();
                if (!kOut && issue && ch > c.ch0) {                     // B of this chunk, once the last one's products are complete
                    mbar_sleep_bounded(set ? &sh.st : &sh.cs, ((it - 1) >> 1) & 1, abort, p.err);
                    if (!*abort) load_bc(ch);
                }
                __syncwarp();
                // (rows past the sequence's end hold silu(conv_b): their Δ is zero, so nothing reads them)
                uint2 xlo[kToks];                                       // what bf16 leaves of x, for D·x
#pragma unroll
                for (int j = 0; j < kToks; ++j) {
                    const int row = row0 + j;
                    const float2 m = splat2(tab.tail[row]);
                    const float4 f = quad_floats(raw[j + 3].bits(j & 1 ? sh0 : sh1, raw_tail, qd, j + 3));
                    const float2 u0 = heads_conv2(wk[0], wb[0], make_float2(e0.x, e0.y), make_float2(e1.x, e1.y),
                                                  make_float2(e2.x, e2.y), make_float2(f.x, f.y));
                    const float2 u1 = heads_conv2(wk[1], wb[1], make_float2(e0.z, e0.w), make_float2(e1.z, e1.w),
                                                  make_float2(e2.z, e2.w), make_float2(f.z, f.w));
                    e0 = e1;
                    e1 = e2;
                    e2 = f;
                    const uint32_t off = tc_chunk(row, qd / 2) + (qd & 1) * 8;
                    if (kOut) {
                        const uint2 x = make_uint2(pack_bf16(u0.x, u0.y), pack_bf16(u1.x, u1.y));
                        *reinterpret_cast<uint2*>(sX + off) = x;
                        xlo[j] = make_uint2(pack_rest(u0, x.x), pack_rest(u1, x.y));
                    }
                    const float2 t0 = mul2(u0, m), t1 = mul2(u1, m);
                    const uint2 x = make_uint2(pack_bf16(t0.x, t0.y), pack_bf16(t1.x, t1.y));
                    *reinterpret_cast<uint2*>(th + off) = x;
                    *reinterpret_cast<uint2*>(tl + off) = make_uint2(pack_rest(t0, x.x), pack_rest(t1, x.y));
                }
                if (kOut && !all_finite(xlo)) {
                    uint32_t from = kNoBad;
#pragma unroll 1
                    for (int j = 0; j < kToks; ++j) {
                        uint16_t* x = reinterpret_cast<uint16_t*>(sX + tc_chunk(row0 + j, qd / 2) + (qd & 1) * 8);
#pragma unroll 1
                        for (int i = 0; i < 4; ++i)
                            if ((x[i] & 0x7f80u) == 0x7f80u) {
                                x[i] = 0;
                                from = __vminu4(from, ~(0xffu << 8 * i) | static_cast<uint32_t>(row0 + j) << 8 * i);
                            }
                    }
                    uint32_t was = tab.bad[qd], seen;
                    do {
                        seen = was;
                        was = atomicCAS(&tab.bad[qd], seen, __vminu4(seen, from));
                    } while (was != seen);
                }
                tma_store_fence();
                warp_arrive(x_ready);
                if (issue) {                                            // what the chunk adds to the state, both tiles side by side
                    if (!kOut) mbar_sleep_bounded(&sh.bc, ph, abort, p.err);
                    mbar_sleep_bounded(x_ready, set_ph, abort, p.err);
                    tc_fence_after();
                    const uint32_t xh_at = x_at + (set ? 0 : kBlock), xl_at = x_at + (set ? 3 : 2) * kBlock;
                    const uint32_t to = tmem + (set ? kColY : kColS);
                    for (int k = 0; k < 8; ++k) {
                        const uint64_t bh = tc_desc(b_at + k * 2048, kBlock, 1024), bl = tc_desc(b_at + kImage + k * 2048, kBlock, 1024);
                        const uint64_t xh = tc_desc(xh_at + k * 2048, kTileBytes, 1024), xl = tc_desc(xl_at + k * 2048, kTileBytes, 1024);
                        constexpr uint32_t id = tc_idesc(128, 128, true, true);
                        tc_mma(to, bh, xl, id, k > 0);
                        tc_mma(to, bl, xh, id, true);
                        tc_mma(to, bh, xh, id, true);
                    }
                    tc_commit(st);
                }
                __syncwarp();
                if (kOut) {
                    wait(&sh.cs, ph);
                    // exp2(l)·(C·S)
                    {
                        const float2 carry = splat2(ex2(before + l));
                        uint32_t v[32];
                        tc_ld32(lanes + kColY + wg * 64 + hf * 32, v);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 y = mul2(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), carry);
                            v[i] = __float_as_uint(y.x);
                            v[i + 1] = __float_as_uint(y.y);
                        }
                        tc_st32(lanes + kColY + wg * 64 + hf * 32, v);
                    }
                    // P: thread = row t; the blocks of 32 columns before its own by a product of two decays, its own
                    // by the decay itself, the ones after it zero.  One warpgroup has blocks 0 and 3, the other 1 and 2.
                    const float2 mine = splat2(ex2(l));
                    const float back = l - lg2_approx(dt);              // exp2(l_t - back_s) = Δ_s · decay from s to t
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int j = hf == 0 ? 3 * k : 1 + k;
                        uint32_t o[16];
                        if (j <= warp) {
                            uint32_t v[32];
                            tc_ld32(lanes + kColScore + j * 32, v);
                            if (j < warp) {
                                const float4* f = reinterpret_cast<const float4*>(&tab.fac[(warp - 1) * warp / 2 * 32 + j * 32]);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const float4 w = f[i];
                                    const float2 a0 = mul2(mul2(make_float2(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])),
                                                                make_float2(w.x, w.y)), mine);
                                    const float2 a1 = mul2(mul2(make_float2(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])),
                                                                make_float2(w.z, w.w)), mine);
                                    o[2 * i] = pack_bf16(a0.x, a0.y);
                                    o[2 * i + 1] = pack_bf16(a1.x, a1.y);
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    const float w = __uint_as_float(v[i]) * ex2(l - __shfl_sync(0xffffffffu, back, i));
                                    v[i] = i <= lane ? __float_as_uint(w) : 0u;
                                }
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = pack_bf16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = 0u;
                        }
                        tc_st16(lanes + kColP + wg * 64 + j * 16, o);
                    }
                    tc_wait_st();
                    tc_fence_before();
                    warp_arrive(&sh.p_ready[wg]);
                    if (issue_pv) {
                        mbar_sleep_bounded(&sh.p_ready[wg], ph, abort, p.err);
                        tc_fence_after();
                        for (int k = 0; k < 8; ++k)
                            tc_mma_ta(tmem + kColY + wg * 64, tmem + kColP + wg * 64 + k * 8,
                                      tc_desc(x_at + wg * kTileBytes + k * 2048, 16, 1024), tc_idesc(128, 64, false, true), true);
                        tc_commit(&sh.pv[wg]);
                    }
                    __syncwarp();
                }
                // the state
                if (kOut) {
                    wait(st, set_ph);
                    if (issue && ch + 1 < ch1 && !*abort) load_bc(ch + 1);   // the products that read B and C are complete
                    __syncwarp();
                    update(all, kColS);
                } else {
                    if (ch > c.ch0) {
                        wait(set ? &sh.st : &sh.cs, ((it - 1) >> 1) & 1);
                        update(last_all, set ? kColS : kColY);
                    }
                    last_all = all;
                }
                if (ch + 1 < ch1) dt_next = load_dt(ch + 1);
                if (kOut) {
                    if (ch + 1 < ch1) state_tile();
                    Row4<VEC> gate[kToks];
                    uint32_t zsh0 = 0u, zsh1 = 0u, gate_tail = 0u;
                    if (p.z) {
                        const TIO* z = static_cast<const TIO*>(p.z) + (s.row0 + tok0 + row0) * p.z_t + cx + 4 * qd;
                        zsh0 = Quad4<VEC>::shift(z);
                        zsh1 = Quad4<VEC>::shift(z + p.z_t);
                        gate_tail = load_tail<VEC>(z - 4 * qd, p.z_t, np >= kTile && qd < kToks && row0 + qd < nt, qd);
#pragma unroll
                        for (int j = 0; j < kToks; ++j) {
                            gate[j].load(z, row0 + j < nt ? nq : -1, j & 1 ? zsh1 : zsh0);
                            z += p.z_t;
                        }
                    }
                    wait(&sh.pv[wg], ph);
                    if (tab.bad[qd] != kNoBad)                          // NaN through D·x
#pragma unroll 1
                        for (int j = 0; j < 4 * kToks; ++j)
                            if (row0 + j / 4 >= static_cast<int>(tab.bad[qd] >> 8 * (j % 4) & 0xffu))
                                reinterpret_cast<uint16_t*>(sX + tc_chunk(row0 + j / 4, qd / 2) + (qd & 1) * 8)[j % 4] = 0x7fffu;
                    __syncwarp();
                    // y: rows out of tensor memory, through shared memory, so that 16 threads write a token's 64 channels
                    {
                        uint32_t v[32];
                        tc_ld32(lanes + kColY + wg * 64 + hf * 32, v);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4*>(stage + t * kTile + (((8 * hf + i) ^ (t & 7)) << 2)) =
                                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                    if (ch + 1 < ch1) {                                 // the next C·S may begin
                        tma_store_fence();
                        tc_fence_before();
                        warp_arrive(&sh.y_free);
                    }
                    tile_sync();
                    TIO* y = static_cast<TIO*>(p.y) + (s.row0 + tok0 + row0) * p.y_t + cx + 4 * qd;
#pragma unroll
                    for (int j = 0; j < kToks; ++j) {
                        const int row = row0 + j;
                        const float4 v = *reinterpret_cast<const float4*>(stage + row * kTile + ((qd ^ (row & 7)) << 2));
                        const uint2 x = *reinterpret_cast<const uint2*>(sX + tc_chunk(row, qd / 2) + (qd & 1) * 8);
                        const float2 Dd = splat2(Dh);
                        float2 y0 = fma2(Dd, add2(unpack2(x.x), unpack2(xlo[j].x)), make_float2(v.x, v.y));
                        float2 y1 = fma2(Dd, add2(unpack2(x.y), unpack2(xlo[j].y)), make_float2(v.z, v.w));
                        if (p.z) {
                            const float4 z = quad_floats(gate[j].bits(j & 1 ? zsh1 : zsh0, gate_tail, qd, j));
                            y0 = mul2(y0, silu2(make_float2(z.x, z.y)));
                            y1 = mul2(y1, silu2(make_float2(z.z, z.w)));
                        }
                        quad_store<VEC>(y, row < nt ? nq : 0, q.wide_y, y0, y1);
                        y += p.y_t;
                    }
                }
            }
            if (PASS == Pass::kStates) {
                if (c.ch0 < ch1) {
                    const uint32_t set = (it - 1) & 1;
                    wait(set ? &sh.cs : &sh.st, ((it - 1) >> 1) & 1);
                    update(last_all, set ? kColY : kColS);
                }
                if (on) {
                    save(saved(q.seg_state, segment(seg)));
                    if (t == 0 && hf == 0) q.seg_decay[segment(seg)] = decay_sum;
                }
                return;
            }
            if (!ends && PASS == Pass::kWaves) {                        // for the segment after this one
                save(saved(q.handover, chain));
                __threadfence();
                tile_sync();
                if (t == 0 && hf == 0)
                    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(q.flags + chain), "r"(static_cast<unsigned>(seg) + 1u) : "memory");
            }
            if (s.slot < 0) return;
            if (ends && on && t < p.N)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (i < my_rows) slot_state[static_cast<int64_t>(i) * p.N] = S[i];
            // the CTA that begins the sequence alone reads its x channels' windows: it shifts them
            if (begins) {
                tile_sync();
                for (int k = hf * 128 + t; k < np; k += 256) heads_keep_window<TIO>(p, s, cx + k);
            }
        });
        if (issue_pv && *abort) {                // products and copies in flight are over before the block ends (or a limit)
            tc_commit(&sh.drain[wg]);
            const long long t0 = clock64();
            while (!(mbar_try_wait(&sh.drain[wg], 0u) &&
                     (wg > 0 || sh.loads == 0u || mbar_try_wait(&sh.bc, (sh.loads - 1u) & 1u))) &&
                   clock64() - t0 < (1ll << 28)) {
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid / 32 == 0) tc_dealloc(tmem, kTmemCols);
}

// Segments per sequence of the time split (1: none), for sequences of equal length (the host does not know them:
// one of 32768 tokens among fifteen of 100, 24 heads, is not cut and takes 2.66 ms, alone 0.41), in units of a
// chunk's time.  Without it no more CTAs run than there are chains (sequences times pairs of tiles).  With it a
// segment costs a first pass of about 0.45 of a full one (no scores, no outputs) and a prologue, the
// whole call one more launch.
int segments_for(int64_t chains, int64_t chunks, int64_t sms) {
    auto waves = [&](int64_t ctas) { return (ctas + sms - 1) / sms; };
    int best = 1;
    double cost = static_cast<double>(chains * chunks) / static_cast<double>(std::min(chains, sms)) + 1.0;
    for (int k = 2; k <= 64 && k <= chunks; ++k) {
        const double len = static_cast<double>((chunks + k - 1) / k);
        const double c = waves(chains * k) * (len + 1.5) + waves(chains * (k - 1)) * (0.45 * len + 1.0) + 2.0;
        if (c < cost) {
            cost = c;
            best = k;
        }
    }
    return best;
}

std::atomic<int> g_force_path{0}, g_force_chunks{0};

// Chunks per segment of the waves: short ones, so that the last wave leaves little idle, unless there
// are so many chains that whole sequences do as well.
constexpr int kWaveChunks = 4;
constexpr int kManyChains = 8;           // per SM

size_t padded(size_t n) { return (n + 255) / 256 * 256; }

template <typename TIO, bool VEC, Pass PASS>
cudaError_t launch_pass(const HeadsTcParams& q, unsigned grid, cudaStream_t stream) {
    void (*kern)(const HeadsTcParams) = heads_tc_kernel<TIO, VEC, PASS>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
    if (e != cudaSuccess) return e;
    if (PASS == Pass::kWaves) {                       // CTAs wait for one another: all of them at once
        void* args[] = {const_cast<HeadsTcParams*>(&q)};
        return cudaLaunchCooperativeKernel(reinterpret_cast<void*>(kern), dim3(grid), dim3(kTcThreads), args, kTcSmem, stream);
    }
    kern<<<grid, kTcThreads, kTcSmem, stream>>>(q);
    return cudaGetLastError();
}

template <typename TIO, bool VEC>
cudaError_t launch_typed(const HeadsTcParams& q, const HeadsTcPlan& plan, cudaStream_t stream) {
    static_assert(sizeof(TIO) == 2, "bf16 operands of the products carry bf16 inputs");
    const dim3 prep(static_cast<unsigned>(plan.chunks), static_cast<unsigned>(q.p.G), 2u);
    heads_prep_kernel<TIO, VEC><<<prep, kPrepThreads, 0, stream>>>(q);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (!plan.split) return launch_pass<TIO, VEC, Pass::kWaves>(q, static_cast<unsigned>(plan.ctas), stream);
    const unsigned grid = static_cast<unsigned>(plan.segments * plan.pairs);
    e = launch_pass<TIO, VEC, Pass::kStates>(q, grid, stream);
    return e != cudaSuccess ? e : launch_pass<TIO, VEC, Pass::kSegments>(q, grid, stream);
}

}  // namespace

int heads_sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 152;
    }
    return n;
}

// bf16 activations, up to 128 states, and sequences long enough (on average) that the products' fixed
// costs pay, by what both paths measure, in us: token by token 7 + 0.28 a token of 128 states (0.18 of 16) as
// long as the CTAs are few, and 0.28 (0.1 of 16) per 170 CTAs beyond; here 12 + 10 a chunk up to 110 chains,
// whatever the states.  (128 states: one sequence of 45 tokens, 24 heads: 19 against 22; 8 of 32: 23 against 23;
// 16 of 24, 80 heads: 80 against 71.  40 sequences of 60 tokens, 40 heads: 16 states 51 against 81, 128 states 251
// against 89.)  It knows the mean length alone: the lengths themselves are in device memory.  Not for heads of fewer than 256 states: the operands' error is one of the terms, and in so few
// sums one may cancel (1.1e-5 of a state of 1 x 1, 4e-6 of one of 64 x 128; fp32 has neither), while a tile has
// 64 x 128 whatever the head has.
bool heads_tc_takes(int64_t n_seq, int64_t tokens, int64_t H, int64_t P, int64_t G, int64_t N, bool bf16) {
    if (!bf16 || N > 128 || P * N < 256 || G > 65535 || n_seq < 1 || tokens < 1) return false;
    const HeadsTcPlan plan = heads_tc_plan(n_seq, tokens, H, P, G, N);
    if (plan.segments * plan.pairs > INT32_MAX || plan.chunks > INT32_MAX) return false;
    if (const int forced = g_force_path.load()) return forced == 2;
    const double mean = static_cast<double>(tokens) / static_cast<double>(n_seq), chunks = std::ceil(mean / kHeadsChunk);
    const double part = static_cast<double>(N) / 128.0, ctas = static_cast<double>(n_seq) * plan.gtiles;
    const double seq = 7.0 + mean * std::max(0.16 + 0.12 * part, (0.07 + 0.21 * part) * ctas / 170.0);
    const double tc = 12.0 + 10.0 * chunks * std::max(1.0, static_cast<double>(n_seq) * plan.pairs / 110.0);
    return tc < seq;
}

HeadsTcPlan heads_tc_plan(int64_t n_seq, int64_t tokens, int64_t H, int64_t P, int64_t G, int64_t N) {
    HeadsTcPlan plan{};
    const int64_t tiles = (P + kHeadsTile - 1) / kHeadsTile;
    plan.nb = N > 64 ? 2 : 1;
    plan.gtiles = static_cast<int>(H * tiles);
    plan.pairs = static_cast<int>(G * ((H / G * tiles + 1) / 2));
    plan.chunks = tokens / kHeadsChunk + n_seq;
    const int64_t mean = (tokens / n_seq + kHeadsChunk - 1) / kHeadsChunk;
    const int sms = heads_sm_count();
    const int64_t chains = n_seq * plan.pairs;
    const int k = segments_for(chains, std::max<int64_t>(mean, 1), sms);
    const int forced = g_force_chunks.load();
    plan.split = forced ? forced > 0 : k > 1;
    const bool whole = !forced && !plan.split && chains > kManyChains * sms;
    plan.seg_chunks = plan.split ? static_cast<int>((mean + k - 1) / k) : whole ? INT32_MAX / 2 : kWaveChunks;
    if (forced) plan.seg_chunks = std::abs(forced);
    plan.segments = plan.chunks / plan.seg_chunks + n_seq;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += padded(n);
        return here;
    };
    plan.off_images = take(static_cast<size_t>(plan.chunks) * G * 3 * plan.nb * kBlock);
    plan.off_chunk_base = take(static_cast<size_t>(n_seq + 1) * 4);
    plan.off_seg_base = take(static_cast<size_t>(n_seq + 1) * 4);
    const size_t states = plan.split ? static_cast<size_t>(plan.segments) * plan.gtiles : 0;
    plan.off_state = take(states * kQ * kTile * 4);
    plan.off_decay = take(states * 4);
    plan.ctas = static_cast<int>(std::min<int64_t>(chains, sms));
    plan.chains = plan.split || whole ? 0 : static_cast<int>(chains);
    plan.off_handover = take(static_cast<size_t>(plan.chains) * 2 * kQ * kTile * 4);
    plan.off_flags = take(static_cast<size_t>(plan.chains) * 2 * 4);
    plan.off_order = take(static_cast<size_t>(plan.segments) * 8);
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
    q.handover = reinterpret_cast<float*>(w + plan.off_handover);
    q.flags = reinterpret_cast<unsigned int*>(w + plan.off_flags);
    q.nflags = 2 * plan.chains;
    q.order = reinterpret_cast<int32_t*>(w + plan.off_order);
    q.seg_chunks = plan.seg_chunks;
    q.pairs = plan.pairs;
    q.gtiles = plan.gtiles;
    q.nb = plan.nb;
    // four channels in one access: z, x, B, C and y of every head and group on that boundary
    auto wide = [&](const void* base, int64_t stride) { return host::is_aligned(base, 8) && stride % 4 == 0; };
    q.wide_w = host::is_aligned(p.conv_w, 16);
    q.wide_y = p.P % 4 == 0 && wide(p.y, p.y_t);
    const bool vec = p.N % 4 == 0 && q.wide_w && wide(p.xbc, p.xbc_t) && wide(p.z, p.z_t) && q.wide_y;
    return vec ? launch_typed<__nv_bfloat16, true>(q, plan, stream) : launch_typed<__nv_bfloat16, false>(q, plan, stream);
}

}  // namespace selscan

// Test hooks.  The path of ss_heads_fwd: 1 token by token, 2 products (where it can), 0 by size.  Chunks per
// segment of the products' path: n > 0 a time split, n < 0 waves of -n, 0 by size.  Return the previous value.
extern "C" int ss__force_heads_path(int path) { return selscan::g_force_path.exchange(path); }
extern "C" int ss__force_heads_chunks(int chunks) { return selscan::g_force_chunks.exchange(chunks); }
