// Softmax cross entropy over a vocabulary, from the rows of the last layer and the output embedding, and its
// gradients, without keeping the logits:
//   l_tv = hidden_t · weight_v,  lse_t = log Σ_v exp(l_tv),  loss_t = lse_t - l_{t,target_t}
//   dl_tv = (exp(l_tv - lse_t) - [v = target_t]) · dloss_t,  dhidden = dl · weight,  dweight = dlᵀ · hidden
//
// Four matrix products of tokens x D x V, and those are the bound: hand-written tcgen05 products of 256 x 256
// tiles by pairs of CTAs (tc_pair.cuh).  Rows without a target are left out before the first product: the others
// are gathered into rows of their own, and the products' sizes come from their count in device memory.
//   forward    the logits' tiles go from tensor memory into a maximum and a sum per row and half tile
//   backward   the logits again, piece by piece of the vocabulary; a piece's dl is kept in fp16 (in the workspace:
//              kPieceBytes of it), then both products over it in one launch: dweight's rows of the piece, whole, and
//              dhidden as sums in fp32 that grow from piece to piece
// Operands.  bf16 logits of the forward pass: as they are.  The backward pass takes bf16 tensors in fp16 as a rule, scaled
// by one power of two per tensor so that the largest value lies below 2^15, and dl has 11 bits instead of bf16's 8 (in bf16
// its rounding would add to the gradients' error as much as their own does: 2.9e-3 instead of 1.7e-3).  dl's power of two is
// its row's, from the row's dloss, and the rows of hidden that dweight sums over have the rest of it: one power for all would
// leave a token of dloss 2^-20 beside 1 with no more than a bit of its softmax at 128000 columns.  With few tokens, where the
// traffic is the bound, it takes bf16 tensors as they are and dl as the sum of two bf16: half more products, but weight is
// not copied.  A float32 value is the sum of two scaled fp16 (22 bits), and a product the three products of these that count
// (K three times as long; three parts of bf16 would take six).
//
// One persistent CTA pair per two SMs: a warp that loads (TMA, stages of 2 x 16 KB), one that issues, eight that empty
// the other of two accumulators meanwhile and send results off by TMA.  Launches by themselves, against 1888 TFLOP/s of a
// library product: the loss of 8191 tokens, 2560 x 50257, 1.07 ms (1980 TFLOP/s); for 3482 tokens, 2048 x 64000 (a piece),
// dl 0.50 ms (1840), both products over it 1.01 (1810).  Behind one another they run at the power limit, some 15% slower.
// With few tokens weight's traffic is the bound: 64 tokens, 2048 x 128000, loss 91 us (5.8 TB/s), dl 101, dhidden 83 (6.3),
// but dweight 131 (524 MB out), whose tiles of one step of K are the chain from accumulator to store.  Tiles of 256 x 256
// by one CTA each would read twice as much from L2 (some 28 TB/s); stores by the threads that hold the sums cost 8%,
// accumulators in local memory (an indexed choice among them) 30%.
#include <cuda_fp16.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "../../include/selscan.h"
#include "chained.cuh"
#include "heads_device.cuh"
#include "host_util.h"
#include "internal.h"
#include "tc_pair.cuh"
#include "xent_params.h"

namespace selscan {
namespace {

constexpr int kTile = 256;                        // rows and columns of a pair's tile
constexpr int kHalf = kTile / 2;                  // rows of a CTA's operand tiles
constexpr int kStep = 64;                         // of K per stage
// Stages of operands, and a warp's boxes for what leaves, in 227 KB of shared memory.  The loss leaves nothing; dl for few
// tokens leaves little of what is read, and the more is on its way the better.
constexpr int kBoxesOf(Product p, Form f) { return p == Product::kLoss ? 0 : p == Product::kGrad && f == Form::kRaw ? 1 : 2; }
constexpr int kStagesOf(Product p, Form f) { return 7 - kBoxesOf(p, f); }
constexpr int kMaxStages = 7;
constexpr uint32_t kOperand = kHalf * kStep * 2;  // bytes of one operand's tile
constexpr uint32_t kStageBytes = 2 * kOperand;
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = (kEpiWarps + 2) * 32;
// Tiles of rows that share a sweep over the vocabulary (8191 tokens, 2560 x 50257: 8 of them 1.29 ms, 16 1.25, 32, all, 1.235).
constexpr int kGroup = 32;
constexpr uint32_t kAccCols = 256;
constexpr unsigned int kInfBits = 0x7f800000u;
// Steps of K that one accumulator takes before its sums go into registers.  The tensor core cuts each addition of
// 16 products off at 2^-23 of the sum instead of rounding it, so a long chain is off by its length times half of
// that, to one side: 560 additions gave a dhidden off by 1e-5, 64 in a row 1e-6.  The registers' own additions
// round.  Results in fp32 take 16 (32 the loss) in a row, those that end in bf16 64.
template <Product P, Form F> constexpr int kChain = F == Form::kSplit ? 4 : P == Product::kLoss ? 8 : 16;

// The products of parts that a product takes, small ones first: kSplit's, then kOut's of kRaw (dl's low part, its high one).
template <Product P, Form F> constexpr int kSegs = F == Form::kSplit ? 3 : F == Form::kRaw && P == Product::kOut ? 2 : 1;
__constant__ int8_t kPartA[2][3] = {{0, 1, 0}, {1, 0, 0}};
__constant__ int8_t kPartB[2][3] = {{1, 0, 0}, {0, 0, 0}};
// Those of dhidden's when dl's two parts are in the rows of a pair's two CTAs: one for each part of weight, the small one first.
template <Form F> constexpr int kSegsPaired = F == Form::kSplit ? 2 : 1;
constexpr int kDlParts(Form f) { return f == Form::kHalf ? 1 : 2; }

// Exponent n of the power of two that a tensor's values are divided by, from the bits of its largest finite one: what
// is left is below 2^15.  2^n and 2^-n are normal floats.
__device__ __forceinline__ int scale_exp(unsigned int bits) { return min(max(static_cast<int>(bits >> 23) - 127 - 14, -126), 126); }
__device__ __forceinline__ float pow2(int n) { return __int_as_float((n + 127) << 23); }
// dl's, a row's own: its dloss sets how large it is, and one dloss may be a small part of another.  dweight sums over
// the rows, so the rows of hidden that it takes are scaled by what a row's exponent lacks to `most`, that of the largest
// finite dloss (a dloss that is not finite counts as that one).
__device__ __forceinline__ int row_exp(float g, int most) { return min(scale_exp(__float_as_uint(g) & 0x7fffffffu), most); }
// Whether every row's is the largest one's, as with one dloss for all (rows of no dloss aside, whose dl is zero): dweight
// takes hidden as the logits do then (4096 tokens, 2048 x 128000: 0.8% less than with rows of its own).
__device__ __forceinline__ bool one_exp(const unsigned int* range) { return scale_exp(kInfBits - range[kRangeL]) >= scale_exp(range[kRangeG]); }
// weight's, which is packed before its largest value is known: that of values below 2^7, unless they turn out larger or
// all below 2^-4 (they are packed again then).
// What is kept: fp16 ends at steps of 2^-24, so a tensor scaled by its own largest value (2^14 and more) is off by 2^-39 of
// that at most, and bf16 is exact down to 2^-31 of it; weights scaled by the guess (the largest 2^3 or more) by 2^-28, and
// exact down to 2^-20.
constexpr int kGuess = -7;
__device__ __forceinline__ int weight_exp(unsigned int bits) {
    const int e = static_cast<int>(bits >> 23) - 127;
    return e >= -4 && e < 7 ? kGuess : scale_exp(bits);
}
// 2^n for n of -252 to 252 as a product of two floats (the second 1 where one is enough).
struct Pow2x2 {
    float a, b;
    __device__ __forceinline__ explicit Pow2x2(int n) {
        const int h = min(max(n, -126), 126);
        a = pow2(h);
        b = pow2(n - h);
    }
};

// A unit of work: a tile and a range of steps of K (each of them kSegs products of parts).
struct Unit {
    int job, m, n, k0, k1, split;
};

// How a kernel's units are numbered.  kOut has two products: job 0 dweight (rows: the piece of the vocabulary), job 1
// dhidden (rows: the tokens) in slices of K.
struct Work {
    int mt0, mt1, nt, steps0, steps1, per, first;
    int n0, total;                                // units of the job that is first, and of both (fewer than 2^31: the host sees to it)
    int full;                                     // of the first job that every pair has
    int extra;                                    // pairs that have one unit of the first job more than the others
    int fill, filled;                             // units of the second job that each of the others has meanwhile, and all of these
};

struct GemmShared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
    Work work;                                    // (here and not in registers, which the accumulators take up)
    int rows, ex, ew, eg;                         // rows that have a target; the operands' scales
    bool one;                                     // dl has one scale (see one_exp)
    uint32_t tmem;
    int abort;
};
constexpr uint32_t kBox = 32 * 128;                // bytes of a warp's store: 32 rows of 128
constexpr size_t gemm_smem(Product p, Form f) {
    return kStagesOf(p, f) * kStageBytes + kEpiWarps * kBoxesOf(p, f) * kBox + sizeof(GemmShared) + 1024;
}
template <Product P, Form F>
__device__ __forceinline__ Work make_work(const XentParams& p, int rows, int pairs) {
    Work w = {};
    const int dt = (p.D + kTile - 1) / kTile, vt = (p.Vp + kTile - 1) / kTile, rt = (rows + kTile - 1) / kTile;
    if (P != Product::kOut) {
        w.mt0 = rt;
        w.nt = vt;
        w.steps0 = (p.D + kStep - 1) / kStep;
        w.n0 = w.total = rt * vt;
        w.full = w.n0 / pairs;
        w.extra = w.n0 % pairs;
        return w;
    }
    w.mt0 = vt;
    w.mt1 = rt;
    w.nt = dt;
    w.steps0 = (rows + kStep - 1) / kStep;
    w.steps1 = (p.Vp + kStep - 1) / kStep;
    w.per = (w.steps1 + p.splits - 1) / p.splits;
    const int l0 = w.steps0 * kSegs<P, F>, l1 = w.per * (p.paired ? kSegsPaired<F> : kSegs<P, F>);
    w.first = l1 > l0 ? 1 : 0;                    // the longer units first, so that the shorter ones fill up
    const int a = vt * dt, b = rt * dt * p.splits;
    w.n0 = w.first ? b : a;
    w.total = a + b;
    w.full = w.n0 / pairs;
    w.extra = w.n0 % pairs;
    w.fill = w.extra > 0 ? max(l0, l1) / max(min(l0, l1), 1) : 0;
    w.filled = static_cast<int>(min(static_cast<int64_t>(w.fill) * (pairs - w.extra), static_cast<int64_t>(w.total - w.n0)));
    return w;
}
// The i-th unit of a pair of CTAs, or -1: units of the first job in turn, then those of the second, of which the
// pairs that have one of the first less get as many more as that one's length allows.
__device__ __forceinline__ int nth_unit(const Work& w, int pair, int pairs, int i) {
    const int n = w.full + (pair < w.extra ? 1 : 0);
    if (i < n) return pair + i * pairs;
    i -= n;
    const int others = pairs - w.extra;
    int at;
    if (pair < w.extra) {
        at = w.filled + others + pair + i * pairs;
    } else if (i < w.fill && pair - w.extra + i * others < w.filled) {
        at = pair - w.extra + i * others;
    } else {
        i -= (w.filled - (pair - w.extra) + others - 1) / others;
        at = w.filled + pair - w.extra + i * pairs;
    }
    return at < w.total - w.n0 ? w.n0 + at : -1;
}
template <Product P>
__device__ __forceinline__ Unit unit_of(const Work& w, int i) {
    Unit u;
    if (P != Product::kOut) {
        // the row tiles of a group take each tile of the vocabulary at the same time: it is read once
        const int per_group = kGroup * w.nt, g = i / per_group, r = i - g * per_group;
        const int size = min(kGroup, w.mt0 - g * kGroup);
        u.job = 0;
        u.m = g * kGroup + r % size;
        u.n = r / size;
        u.k0 = 0;
        u.k1 = w.steps0;
        u.split = 0;
        return u;
    }
    u.job = i < w.n0 ? w.first : 1 - w.first;
    const int at = i < w.n0 ? i : i - w.n0, r = at / w.nt;
    u.n = at - r * w.nt;
    const int mt = u.job ? w.mt1 : w.mt0;
    u.split = u.job ? r / mt : 0;
    u.m = r - u.split * mt;
    u.k0 = u.job ? u.split * w.per : 0;
    u.k1 = u.job ? min(u.k0 + w.per, w.steps1) : w.steps0;
    return u;
}

// Whether a unit's tile has dl's high part in one CTA's rows and its low part in the other's (each a slice of sums).
template <Product P, Form F>
__device__ __forceinline__ bool is_paired(const XentParams& p, const Unit& u) {
    return P == Product::kOut && F != Form::kHalf && u.job && p.paired;
}

__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ void store16(void* q, uint4 v) { *reinterpret_cast<uint4*>(q) = v; }

__device__ __forceinline__ uint32_t half_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// 8 values to fp16, and (SPLIT) what is left of them to the second part.
template <bool SPLIT>
__device__ __forceinline__ void store_half8(__half* q, int64_t part, const float2 (&f)[4]) {
    __half2 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __float22half2_rn(f[i]);
    store16(q, make_uint4(half_bits(h[0]), half_bits(h[1]), half_bits(h[2]), half_bits(h[3])));
    if constexpr (SPLIT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __float22half2_rn(fma2(__half22float2(h[i]), splat2(-1.f), f[i]));
        store16(q + part, make_uint4(half_bits(h[0]), half_bits(h[1]), half_bits(h[2]), half_bits(h[3])));
    }
}

// A warp's 32 rows of 128 bytes (a lane has a row) to a tensor, by way of its own part of shared memory: as rows of
// their own they would be stores of 16 bytes to 32 lines at a time, which took the L1 half of its time beside the
// operands.  What lies outside the tensor is not written.  ADD: onto what is there.
__device__ __forceinline__ void fill_box(uint8_t* box, const uint32_t (&w)[32]) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        store16(box + tc_chunk(lane, j), make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
}
template <bool ADD, int BOXES>
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint8_t* boxes, uint32_t& turn, const uint32_t (&w)[32], int col, int row, int part) {
    const int lane = threadIdx.x % 32;
    uint8_t* box = boxes + turn * kBox;
    if (BOXES > 1) turn ^= 1u;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(BOXES - 1) : "memory");      // the box's last store has left this memory
    __syncwarp();
    fill_box(box, w);
    tma_store_fence();
    __syncwarp();
    if (lane == 0) {
        if constexpr (ADD) pair_tma_add(map, box, col, row, part);
        else tma_store_3d(map, box, col, row, part);
        tma_store_commit();
    }
}

template <Product P, Form F>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1) xent_gemm_kernel(const __grid_constant__ XentParams p) {
    constexpr int kStages = kStagesOf(P, F), kBoxes = kBoxesOf(P, F);
    extern __shared__ uint8_t raw[];
    uint8_t* tiles = raw + (1024 - smem_addr(raw) % 1024) % 1024;
    GemmShared& sh = *reinterpret_cast<GemmShared*>(tiles + kStages * kStageBytes + kEpiWarps * kBoxes * kBox);
    volatile int* abort = &sh.abort;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x / 2, clusters = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 2 * kEpiWarps);
        }
        sh.abort = 0;
        mbar_fence_init();
    }
    if (warp == 0) pair_alloc(&sh.tmem, 2 * kAccCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync_all();                            // the peer's barriers exist
    const uint32_t tmem = sh.tmem;
    constexpr int kTable = F == Form::kSplit ? 0 : 1, kSegsHere = kSegs<P, F>;
    wait_for_earlier();
    if (threadIdx.x == 0) {
        sh.rows = *p.count;
        sh.work = make_work<P, F>(p, sh.rows, clusters);
        sh.ex = sh.ew = sh.eg = 0;                 // (operands as they are)
        sh.one = true;
        if constexpr (F != Form::kRaw) {
            sh.ex = scale_exp(p.range[kRangeX]);
            sh.ew = weight_exp(p.range[kRangeW + p.piece]);
            if constexpr (P != Product::kLoss) sh.eg = scale_exp(p.range[kRangeG]);
            if constexpr (P == Product::kOut) sh.one = one_exp(p.range);
        }
    }
    __syncthreads();
    const Work& work = sh.work;

    if (warp == kEpiWarps) {
        // ---------------------------------------------------------------- loads, by one thread of each CTA
        if (lane == 0) {
            uint32_t full0[kStages];
#pragma unroll
            for (int i = 0; i < kStages; ++i) full0[i] = peer_smem_addr(&sh.full[i], 0);
            int st = 0;
            uint32_t ph = 0;
            for (int t = 0, i; (i = nth_unit(work, cluster, clusters, t)) >= 0 && !*abort; ++t) {
                const Unit u = unit_of<P>(work, i);
                const CUtensorMap* ma = u.job ? &p.a1 : &p.a0;
                const CUtensorMap* mb = u.job ? &p.b1 : P == Product::kOut && F != Form::kRaw && !sh.one ? &p.b2 : &p.b0;
                // dweight: both operands have K (the tokens) along rows; dhidden: weight has K (the vocabulary) along rows
                const bool a_mn = P == Product::kOut && u.job == 0, b_mn = P == Product::kOut;
                const bool both = is_paired<P, F>(p, u);
                const int am = both ? 0 : u.m * kTile + static_cast<int>(rank) * kHalf, bn = u.n * kTile + static_cast<int>(rank) * kHalf;
                const int segs = both ? kSegsPaired<F> : kSegsHere;
                bool go = true;
                for (int kc = u.k0; kc < u.k1 && go; kc += kChain<P, F>)
                    for (int seg = 0; seg < segs && go; ++seg) {
                        const int pa = both ? static_cast<int>(rank) : kSegsHere > 1 ? kPartA[kTable][seg] : 0;
                        const int pb = both ? segs - 1 - seg : kSegsHere > 1 ? kPartB[kTable][seg] : 0;
                        for (int k = kc; k < min(kc + kChain<P, F>, u.k1); ++k) {
                            go = mbar_wait_bounded(&sh.empty[st], ph ^ 1, abort, p.err);
                            if (!go) break;
                            if (rank == 0) mbar_expect_tx(&sh.full[st], 2 * kStageBytes);
                            uint8_t* sa = tiles + st * kStageBytes;
                            uint8_t* sb = sa + kOperand;
                            const int kk = k * kStep;
                            if (a_mn) {
                                pair_tma_load(sa, ma, full0[st], am, kk, pa);
                                pair_tma_load(sa + kOperand / 2, ma, full0[st], am + 64, kk, pa);
                            } else {
                                pair_tma_load(sa, ma, full0[st], kk, am, pa);
                            }
                            if (b_mn) {
                                pair_tma_load(sb, mb, full0[st], bn, kk, pb);
                                pair_tma_load(sb + kOperand / 2, mb, full0[st], bn + 64, kk, pb);
                            } else {
                                pair_tma_load(sb, mb, full0[st], kk, bn, pb);
                            }
                            if (++st == kStages) {
                                st = 0;
                                ph ^= 1;
                            }
                        }
                    }
            }
            // the products' last arrivals on this CTA's barriers are in before it ends
            for (int i = 0; i < kStages; ++i) {
                if (!mbar_wait_bounded(&sh.empty[st], ph ^ 1, abort, p.err)) break;
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
    } else if (warp == kEpiWarps + 1) {
        // ---------------------------------------------------------------- products, by one thread of CTA 0
        if (lane == 0 && rank == 0) {
            const uint32_t at = smem_addr(tiles);
            int st = 0;
            uint32_t ph = 0;
            int turn = 0;
            bool go = true;
            for (int t = 0, i; go && (i = nth_unit(work, cluster, clusters, t)) >= 0; ++t) {
                const Unit u = unit_of<P>(work, i);
                const bool a_mn = P == Product::kOut && u.job == 0, b_mn = P == Product::kOut;
                constexpr uint32_t kBf16 = 1u << 7 | 1u << 10;                          // operand types (else fp16)
                const uint32_t idesc = tc_idesc(256, 256, a_mn, b_mn) & ~(F == Form::kRaw ? 0u : kBf16);
                const uint32_t la = a_mn ? kOperand / 2 : 16, lb = b_mn ? kOperand / 2 : 16, ka = a_mn ? 2048 : 32, kb = b_mn ? 2048 : 32;
                for (int kc = u.k0; kc < u.k1 && go; kc += kChain<P, F>, ++turn) {
                    const uint32_t d = tmem + (turn & 1) * kAccCols;
                    const int n = (min(kc + kChain<P, F>, u.k1) - kc) * (is_paired<P, F>(p, u) ? kSegsPaired<F> : kSegsHere);
                    go = mbar_wait_bounded(&sh.acc_empty[turn & 1], ((turn >> 1) & 1) ^ 1, abort, p.err);
                    tc_fence_after();
                    for (int k = 0; k < n && go; ++k) {
                        go = mbar_wait_bounded(&sh.full[st], ph, abort, p.err);
                        if (!go) break;
                        tc_fence_after();
                        const uint32_t a = at + st * kStageBytes, b = a + kOperand;
#pragma unroll
                        for (int j = 0; j < kStep / 16; ++j)
                            pair_mma(d, tc_desc(a + j * ka, la, 1024), tc_desc(b + j * kb, lb, 1024), idesc, k > 0 || j > 0);
                        pair_commit(&sh.empty[st]);
                        if (++st == kStages) {
                            st = 0;
                            ph ^= 1;
                        }
                    }
                    pair_commit(&sh.acc_full[turn & 1]);
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- accumulators, by eight warps of each CTA
        const int quarter = warp % 4, half = warp / 4;
        const uint32_t empty0 = peer_smem_addr(&sh.acc_empty[0], 0), empty1 = peer_smem_addr(&sh.acc_empty[1], 0);
        uint8_t* boxes = tiles + kStages * kStageBytes + warp * kBoxes * kBox;     // (taken in turn)
        uint32_t box = 0u;
        int turn = 0;
        bool go = true;
        for (int t = 0, i; (i = nth_unit(work, cluster, clusters, t)) >= 0; ++t) {
            const Unit u = unit_of<P>(work, i);
            const int rows = sh.rows;
            const int row = u.m * kTile + static_cast<int>(rank) * kHalf + quarter * 32 + lane;
            const int col0 = u.n * kTile + half * kHalf;
            // what the row's end needs is on its way meanwhile
            int tgt = -1;
            float lse = 0.f, g = 0.f;
            if (P != Product::kOut && row < rows) {
                tgt = p.tgt[row] - p.v0 - col0;
                if constexpr (P == Product::kGrad) {
                    lse = p.lse[row];
                    g = p.g[row];
                }
            }
            if constexpr (P == Product::kOut && F != Form::kRaw) {
                const int at = is_paired<P, F>(p, u) ? quarter * 32 + lane : row;
                if (u.job && at < rows) g = p.g[at];
            }
            float acc[kHalf];                      // a thread has half a row of the tile
#pragma unroll
            for (int j = 0; j < kHalf; ++j) acc[j] = 0.f;
#pragma unroll 1
            for (int kc = u.k0; kc < u.k1; kc += kChain<P, F>, ++turn) {
                go = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.acc_full[turn & 1], (turn >> 1) & 1, abort, p.err));
                if (!go) break;
                tc_fence_after();
                const uint32_t at = tmem + (turn & 1) * kAccCols + half * kHalf + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
                for (int c = 0; c < kHalf; c += 16) {
                    uint32_t r[16];
                    tc_ld16(at + c, r);
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float2 v = add2(make_float2(acc[c + j], acc[c + j + 1]), make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])));
                        acc[c + j] = v.x;
                        acc[c + j + 1] = v.y;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) pair_arrive(turn & 1 ? empty1 : empty0);
            }
            if (!go) break;
            if constexpr (P == Product::kLoss) {
                if constexpr (F == Form::kSplit) {
                    const Pow2x2 f(sh.ex + sh.ew);
#pragma unroll
                    for (int j = 0; j < kHalf; ++j) acc[j] = acc[j] * f.a * f.b;
                }
                float m = -INFINITY, s = 0.f;
#pragma unroll
                for (int c = 0; c < kHalf; c += 32) {
                    const int n = p.Vp - col0 - c;
                    if (n <= 0) break;
                    float b = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        acc[c + j] = j < n ? acc[c + j] : -INFINITY;
                        b = fmaxf(b, acc[c + j]);
                    }
                    if (b > m) {
                        s *= ex2((m - b) * kLog2e);
                        m = b;
                    }
                    const float2 off = splat2(-base_of(m)), l2e = splat2(kLog2e);
                    float2 a = splat2(0.f);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) a = add2(a, ex2x2(mul2(add2(make_float2(acc[c + j], acc[c + j + 1]), off), l2e)));
                    s += a.x + a.y;
                    if (tgt >= c && tgt < c + 32) {
                        // (a choice written in C++ becomes an indexed array, and the accumulator with it local memory)
                        float l = 0.f;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            asm("{\n .reg .pred q;\n setp.eq.s32 q, %1, %2;\n @q mov.f32 %0, %3;\n}" : "+f"(l) : "r"(tgt - c), "r"(j), "f"(acc[c + j]));
                        p.tl[row] = l;
                    }
                }
                if (row < rows) p.part[(static_cast<int64_t>(p.tile0 + u.n) * 2 + half) * p.ld_part + row] = make_float2(m, s);
            } else if constexpr (P == Product::kGrad) {
                const bool ok = row < rows, all_ok = __all_sync(0xffffffffu, ok);
                if constexpr (F != Form::kRaw) g *= pow2(-row_exp(g, sh.eg));
                const Pow2x2 f(sh.ex + sh.ew);
                const float2 off = splat2(-lse), f2 = splat2(f.a), l2e = splat2(kLog2e), g2 = splat2(g);
                if (f.b != 1.f) {
#pragma unroll
                    for (int j = 0; j < kHalf; ++j) acc[j] *= f.b;
                }
#pragma unroll
                for (int c = 0; c < kHalf; c += 64) {
                    if (col0 + c >= p.Vp) break;
                    uint32_t hi[32], lo[kDlParts(F) > 1 ? 32 : 1];
#pragma unroll
                    for (int q = 0; q < 64; q += 8) {
                        float2 e[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            e[j] = ex2x2(mul2(fma2(make_float2(acc[c + q + 2 * j], acc[c + q + 2 * j + 1]), f2, off), l2e));
                        if (tgt >= c + q && tgt < c + q + 8) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                e[j].x -= tgt - c - q == 2 * j ? 1.f : 0.f;
                                e[j].y -= tgt - c - q == 2 * j + 1 ? 1.f : 0.f;
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            e[j] = mul2(e[j], g2);
                            if (!all_ok && !ok) e[j] = splat2(0.f);      // (a row past the last may hold anything)
                            if constexpr (F == Form::kRaw) {
                                hi[q / 2 + j] = pack_bf16(e[j].x, e[j].y);
                                lo[q / 2 + j] = pack_rest(e[j], hi[q / 2 + j]);
                            } else {
                                const __half2 h = __float22half2_rn(e[j]);
                                hi[q / 2 + j] = half_bits(h);
                                if constexpr (F == Form::kSplit) lo[q / 2 + j] = half_bits(__float22half2_rn(fma2(__half22float2(h), splat2(-1.f), e[j])));
                            }
                        }
                    }
                    store_box<false, kBoxes>(&p.s0, boxes, box, hi, col0 + c, row - lane, 0);
                    if constexpr (kDlParts(F) > 1) store_box<false, kBoxes>(&p.s0, boxes, box, lo, col0 + c, row - lane, 1);
                }
            } else {
                constexpr bool F32 = F == Form::kSplit;
                if constexpr (F != Form::kRaw) {
                    const Pow2x2 f(u.job ? row_exp(g, sh.eg) + sh.ew : sh.eg + sh.ex);
#pragma unroll
                    for (int j = 0; j < kHalf; ++j) acc[j] = acc[j] * f.a * f.b;
                }
                if (u.job || (F32 && p.dw_wide)) {
                    // rows of 32 floats
                    const bool both = is_paired<P, F>(p, u);
                    const int row0 = both ? quarter * 32 : row - lane, slice = both ? 2 * u.split + static_cast<int>(rank) : u.split;
#pragma unroll
                    for (int c = 0; c < kHalf; c += 32) {
                        if (col0 + c >= p.D) break;
                        uint32_t w[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(acc[c + j]);
                        if (!u.job) store_box<false, kBoxes>(&p.s0, boxes, box, w, col0 + c, row - lane, 0);
                        else if (p.add) store_box<true, kBoxes>(&p.s1, boxes, box, w, col0 + c, row0, slice);
                        else store_box<false, kBoxes>(&p.s1, boxes, box, w, col0 + c, row0, slice);
                    }
                } else if (!F32 && p.dw_wide) {
                    // Both boxes are filled at once: few tokens make this the whole of a unit's time.  Each is a group
                    // of its own, box 0 the older one, as store_box counts them: the dhidden unit that may follow
                    // takes box 0 when one group is still pending.
                    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < kHalf; c += 64) {
                        uint32_t w[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) w[j] = pack_bf16(acc[c + 2 * j], acc[c + 2 * j + 1]);
                        fill_box(boxes + c / 64 * kBox, w);
                    }
                    tma_store_fence();
                    __syncwarp();
                    if (lane == 0) {
                        if (col0 < p.D) tma_store_3d(&p.s0, boxes, col0, row, 0);
                        tma_store_commit();
                        if (col0 + 64 < p.D) tma_store_3d(&p.s0, boxes + kBox, col0 + 64, row, 0);
                        tma_store_commit();
                    }
                    box = 0u;
                } else if (row < p.Vp) {
                    // (rows off 16 bytes, which TMA does not store: a lane has a row, element by element.  64 tokens,
                    // 2047 x 128000: the backward pass 3.5 ms in bf16 and 2.8 in fp32, against 0.32 and 1.0 at 2048)
                    using T = std::conditional_t<F32, float, __nv_bfloat16>;
                    T* out = static_cast<T*>(p.dw) + static_cast<int64_t>(p.v0 + row) * p.ld_dw + col0;
#pragma unroll
                    for (int j = 0; j < kHalf; ++j)
                        if (j < p.D - col0) out[j] = from_f32<T>(acc[j]);
                }
            }
        }
        if (lane == 0) tma_store_wait_all();
    }
    __syncthreads();
    // (after a wait that ran out: copies and products in flight are over long before this)
    if (*abort)
        for (int i = 0; i < 20; ++i) __nanosleep(1000000);
    tc_fence_before();
    cluster_sync_all();                            // nobody reads or signals the peer's memory any more
    tc_fence_after();
    if (warp == 0) pair_dealloc(tmem, 2 * kAccCols);
}

// ------------------------------------------------------------------------------------------ before and after

constexpr int kPrepThreads = 256;

// Columns [c, c + 8) of a row as an operand: bf16 as it is (RAW), or fp16 times `scale`, in two parts for fp32.
// Columns of D and more are zero.  `also`: the same times `shift`, another power of two.
template <typename T, bool RAW>
__device__ __forceinline__ void pack8(const T* row, __half* out, int64_t part, int c, int D, bool wide, float scale, unsigned int* most = nullptr,
                                      __half* also = nullptr, float shift = 1.f) {
    float v[8];
    if (wide && c + 8 <= D) {
        if constexpr (sizeof(T) == 2) {
            const uint4 u = *reinterpret_cast<const uint4*>(row + c);
            if constexpr (RAW) {
                store16(out + c, u);
                return;
            }
            const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf16_lo(a[i]);
                v[2 * i + 1] = bf16_hi(a[i]);
            }
        } else {
            const float4 a = *reinterpret_cast<const float4*>(row + c), b = *reinterpret_cast<const float4*>(row + c + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < D ? to_f32<T>(row[c + i]) : 0.f;
    }
    if constexpr (RAW) {
        store16(out + c, make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])));
    } else {
        if (most) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const unsigned int bits = __float_as_uint(v[i]) & 0x7fffffffu;
                *most = max(*most, bits < kInfBits ? bits : 0u);
            }
        }
        float2 f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = make_float2(v[2 * i] * scale, v[2 * i + 1] * scale);
        store_half8<sizeof(T) == 4>(out + c, part, f);
        if (also) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], splat2(shift));
            store_half8<sizeof(T) == 4>(also + c, part, f);
        }
    }
}

// Magnitudes as bits, whose order is the floats': the larger of m and v's, if that is finite.
__device__ __forceinline__ unsigned int max_finite(unsigned int m, float v) {
    const unsigned int bits = __float_as_uint(v) & 0x7fffffffu;
    return max(m, bits < kInfBits ? bits : 0u);
}
// The block's largest to *out.
__device__ __forceinline__ void block_max(unsigned int m, unsigned int* part, unsigned int* out) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        m = __reduce_max_sync(0xffffffffu, threadIdx.x < kPrepThreads / 32 ? part[threadIdx.x] : 0u);
        if (threadIdx.x == 0 && m) atomicMax(out, m);
    }
    __syncthreads();
}

// Largest finite magnitudes of hidden's rows with a target and of their dloss, and the smallest one of dloss but zero; a warp
// has a row at a time.
template <typename T>
__global__ void __launch_bounds__(kPrepThreads) xent_range_kernel(const PrepParams p) {
    __shared__ unsigned int part[kPrepThreads / 32];
    constexpr int kWarps = kPrepThreads / 32, N = 16 / sizeof(T), U = 4;
    const int lane = threadIdx.x % 32, vecs = p.wide ? p.D / N : 0;
    unsigned int m = 0u, g = 0u, l = 0u;
    let_next_start();
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32; t < p.T; t += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int v = p.targets[t];
        if (v < 0 || v >= p.V) continue;
        const T* row = static_cast<const T*>(p.hidden) + t * p.hidden_t;
        for (int i = lane; i < vecs; i += 32 * U) {
            uint4 u[U];
#pragma unroll
            for (int k = 0; k < U; ++k) u[k] = i + 32 * k < vecs ? reinterpret_cast<const uint4*>(row)[i + 32 * k] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const uint32_t a[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    m = max_finite(m, sizeof(T) == 2 ? bf16_lo(a[j]) : __uint_as_float(a[j]));
                    if constexpr (sizeof(T) == 2) m = max_finite(m, bf16_hi(a[j]));
                }
            }
        }
        for (int c = vecs * N + lane; c < p.D; c += 32) m = max_finite(m, to_f32<T>(row[c]));
        if (p.dloss && lane == 0) {
            const unsigned int one = max_finite(0u, p.dloss[t * p.dloss_t]);
            g = max(g, one);
            if (one) l = max(l, kInfBits - one);
        }
    }
    block_max(m, part, &p.range[kRangeX]);
    block_max(g, part, &p.range[kRangeG]);
    block_max(l, part, &p.range[kRangeL]);
}

// The rows that have a target, gathered in order: row i of x is row rows[i] of hidden.  A block has `per` rows of
// hidden, at most one to a thread, and counts the targets before them itself.
template <typename T, bool BWD, bool RAW>
__global__ void __launch_bounds__(kPrepThreads) xent_gather_kernel(const PrepParams p) {
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int kWarps = kPrepThreads / 32;
    constexpr bool kScaled = BWD && !RAW;
    __shared__ int before[kWarps], own[kWarps], to[kPrepThreads];
    __shared__ float shift[kScaled ? kPrepThreads : 1];
    bool own_rows = false;                         // dweight takes rows of its own
    let_next_start();
    if constexpr (!RAW) wait_for_earlier();        // (else it is the call's first)
    const float scale = RAW ? 1.f : pow2(-scale_exp(p.range[kRangeX]));
    if constexpr (kScaled) own_rows = !one_exp(p.range);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.per;
    const int n = static_cast<int>(min(static_cast<int64_t>(p.per), p.T - first));
    auto has = [&](int v) { return v >= 0 && v < p.V; };
    int count = 0;
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < first; t += kPrepThreads) count += has(p.targets[t]);
    count = __reduce_add_sync(0xffffffffu, count);
    const int mine = static_cast<int>(threadIdx.x) < n ? p.targets[first + threadIdx.x] : -1;
    const unsigned int some = __ballot_sync(0xffffffffu, has(mine));
    if (lane == 0) {
        before[warp] = count;
        own[warp] = __popc(some);
    }
    __syncthreads();
    int at = 0, total = 0;
    for (int i = 0; i < kWarps; ++i) {
        total += before[i] + own[i];
        at += before[i] + (i < warp ? own[i] : 0);
    }
    at += __popc(some & ((1u << lane) - 1u));
    if (has(mine)) {
        const int64_t t = first + threadIdx.x;
        to[threadIdx.x] = at;
        p.rows[at] = static_cast<int>(t);
        p.tgt[at] = mine;
        if constexpr (BWD) {
            const float g = p.dloss[t * p.dloss_t];
            p.lse_c[at] = p.lse[t];
            p.g_c[at] = g;
            if constexpr (kScaled) {
                const int most = scale_exp(p.range[kRangeG]);
                shift[threadIdx.x] = pow2(max(row_exp(g, most) - most, -126));
            }
        }
    } else if (static_cast<int>(threadIdx.x) < n) {
        to[threadIdx.x] = -1;
        if constexpr (!BWD) {
            p.loss_out[first + threadIdx.x] = p.lse_out[first + threadIdx.x] = 0.f;
            if (mine >= p.V && p.err) atomicOr(p.err, kErrIndex);
        }
    }
    __syncthreads();
    const int chunks = (p.D + 255) / 256;          // of a row, one to a warp at a time
    for (int q = warp; q < n * chunks; q += kWarps) {
        const int r = q / chunks, c0 = (q - r * chunks) * 256;
        const int64_t t = first + r;
        const int i = to[r];
        if (i >= 0) {
            if (c0 + lane * 8 < p.D)
                pack8<T, RAW>(static_cast<const T*>(p.hidden) + t * p.hidden_t, p.x + static_cast<int64_t>(i) * p.ld_x, p.x_part, c0 + lane * 8, p.D,
                              p.wide, scale, nullptr, own_rows ? p.xg + static_cast<int64_t>(i) * p.ld_x : nullptr, own_rows ? shift[r] : 1.f);
        } else if constexpr (BWD) {
            T* d = static_cast<T*>(p.dhidden) + t * p.dhidden_t;
            for (int c = c0 + lane; c < min(c0 + 256, p.D); c += 32) d[c] = from_f32<T>(0.f);
        }
    }
    if (first + n == p.T) {
        if (threadIdx.x == 0) *p.count = total;
        // the rest of the last step of K over the tokens counts for nothing, but must be finite
        __half* x = own_rows ? p.xg : p.x;
        const int end = (total + kStep - 1) / kStep * kStep, vecs = static_cast<int>(p.ld_x / 8);
        if (BWD)
            for (int q = 0; q < (F32 ? 2 : 1); ++q)
                for (int i = threadIdx.x; i < (end - total) * vecs; i += kPrepThreads)
                    store16(x + q * p.x_part + (total + i / vecs) * p.ld_x + i % vecs * 8, make_uint4(0u, 0u, 0u, 0u));
    }
}

// Rows of weight as operands of the products.  The scale is a guess, and *range gets the largest finite magnitude;
// AGAIN: the same with the scale that this asks for, if the guess was wrong.
template <typename T, bool RAW, bool AGAIN>
__global__ void __launch_bounds__(kPrepThreads) xent_pack_kernel(const T* w, int64_t stride, __half* out, int64_t ld, int64_t part, int64_t n, int D,
                                                                 bool wide, unsigned int* range) {
    __shared__ unsigned int most[kPrepThreads / 32];
    const int vecs = static_cast<int>(ld / 8);
    let_next_start();
    wait_for_earlier();
    int e = kGuess;
    if constexpr (AGAIN) {
        e = weight_exp(*range);
        if (e == kGuess) return;
    }
    const float scale = RAW ? 1.f : pow2(-e);
    unsigned int m = 0u;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x; i < n * vecs; i += static_cast<int64_t>(gridDim.x) * kPrepThreads) {
        const int64_t r = i / vecs;
        pack8<T, RAW>(w + r * stride, out + r * ld, part, static_cast<int>(i - r * vecs) * 8, D, wide, scale, RAW || AGAIN ? nullptr : &m);
    }
    if constexpr (!RAW && !AGAIN) block_max(m, most, range);
}

// lse and loss from the maxima and sums of the half tiles; a block has 8 rows, and 128 threads share a row's.
constexpr int kJoinThreads = 1024, kJoinRows = 8;
__global__ void __launch_bounds__(kJoinThreads) xent_join_kernel(const float2* part, int64_t ld, int halves, const int* count, const int* rows,
                                                                 const float* tl, float* loss, float* lse) {
    constexpr int kShares = kJoinThreads / kJoinRows, U = 8;
    __shared__ float2 s[kJoinRows][kJoinThreads / 32];
    wait_for_earlier();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, n = *count;
    const int mine = threadIdx.x % kJoinRows, row = blockIdx.x * kJoinRows + mine;
    float m = -INFINITY, sum = 0.f;
    auto join = [&](float2 q) {
        const float b = fmaxf(m, q.x), o = base_of(b);
        sum = sum * ex2((m - o) * kLog2e) + q.y * ex2((q.x - o) * kLog2e);
        m = b;
    };
    auto join_lane = [&](int o) { join(make_float2(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, sum, o))); };
    if (blockIdx.x * kJoinRows >= n) return;
    for (int i = threadIdx.x / kJoinRows; i < halves; i += kShares * U) {
        float2 q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = row < n && i + u * kShares < halves ? part[(i + u * kShares) * ld + row] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u) join(q[u]);
    }
    join_lane(8);
    join_lane(16);
    if (lane < kJoinRows) s[mine][warp] = make_float2(m, sum);
    __syncthreads();
    if (warp >= kJoinRows) return;
    // a warp has a row now
    m = s[warp][lane].x;
    sum = s[warp][lane].y;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) join_lane(o);
    const int i = blockIdx.x * kJoinRows + warp;
    if (lane == 0 && i < n) {
        const float v = m + logf(sum);
        const int t = rows[i];
        lse[t] = v;
        loss[t] = v - tl[i];
    }
}

// dhidden's rows from their sums; a thread has 4 columns at a time.
template <typename T>
__global__ void __launch_bounds__(kPrepThreads) xent_scatter_kernel(const float* dx, int64_t split_stride, int splits, int64_t ld, const int* count,
                                                                    const int* rows, T* dhidden, int64_t stride, int D) {
    wait_for_earlier();
    const int n = *count, quads = (D + 3) / 4;
    for (int64_t q = static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x; q < static_cast<int64_t>(n) * quads;
         q += static_cast<int64_t>(gridDim.x) * kPrepThreads) {
        const int i = static_cast<int>(q / quads), c = static_cast<int>(q - static_cast<int64_t>(i) * quads) * 4;
        const float* from = dx + i * ld + c;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int s = 0; s < splits; ++s) {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(from + s * split_stride));
            v = make_float4(v.x + a.x, v.y + a.y, v.z + a.z, v.w + a.w);
        }
        T* out = dhidden + static_cast<int64_t>(rows[i]) * stride + c;
        const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < D) out[j] = from_f32<T>(w[j]);
    }
}

// ------------------------------------------------------------------------------------------------ host

using host::dev_ptr;
using host::is_aligned;
using host::meet;
using host::Range;
using host::range3;

// Bytes of dl (and of a packed piece of weight) at a time: 4096 tokens, 2048 x 128000 take 4.89 ms with 128 MB, 4.78 with
// 256, 4.77 with 512 and 4.72 with 2 GB (one piece).  At least kMinPiece columns, however many tokens: below, a piece's
// sums of dhidden, read and written again, cost as much as its products.
constexpr int64_t kPieceBytes = 512 << 20;
constexpr int64_t kMinPiece = 4096;
constexpr int64_t kMaxSplits = 32;
// Tokens up to which the backward pass takes bf16 operands as they are.  2048 x 128000, us as they are and in fp16:
// 64 tokens 325 and 468, 256 tokens 513 and 533, 512 tokens 886 and 736; 768 x 50257: 77 and 104, 105 and 113, 173 and 146.
constexpr int64_t kRawTokens = 256;
constexpr int64_t kMinSteps = 16;                 // of K to a slice of dhidden's sums

int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 152;
    }
    return sms;
}

// Where everything lies in the workspace.
struct Layout {
    int64_t parts, dl_parts, segs, ld_x, tpad, piece, pieces, splits, slices, ld_dl, ld_dx, halves;
    Form form;
    bool packed;                                  // weight, piece by piece
    bool paired;                                  // dhidden: dl's two parts as the rows of a pair's two CTAs
    size_t count, range, rows, tgt, lse, g, tl, part, x, xg, w, dl, dx, total;
};

// Time of one launch of both products over a piece, in steps of K, when dhidden's are cut in `splits`: units as
// nth_unit hands them out, each some steps longer for its end.
int64_t out_cost(int64_t T, int64_t D, int64_t Vp, int64_t segs, int64_t segs1, bool paired, int64_t splits, int64_t pairs) {
    constexpr int64_t kEnd = 4;
    const int64_t dt = (D + kTile - 1) / kTile;
    const int64_t len[2] = {(T + kStep - 1) / kStep * segs, ((Vp + kStep - 1) / kStep + splits - 1) / splits * segs1};
    const int64_t n[2] = {(Vp + kTile - 1) / kTile * dt, (T + kTile - 1) / kTile * dt * splits};
    const int first = len[1] > len[0] ? 1 : 0;
    const int64_t a = n[first], b = n[1 - first], la = len[first] + kEnd, lb = len[1 - first] + kEnd;
    const int64_t extra = a % pairs, others = pairs - extra, filled = extra ? std::min(len[first] / std::max<int64_t>(len[1 - first], 1) * others, b) : 0;
    // the pair that is last with each kind of load
    const int64_t rounds = (b - filled + pairs - 1) / pairs, rest = (b - filled) - (rounds - 1) * pairs;
    const int64_t with_extra = (a / pairs + (extra ? 1 : 0)) * la + (rounds - (extra && rest <= others ? 1 : 0)) * lb;
    const int64_t without = a / pairs * la + ((filled + others - 1) / others + rounds) * lb;
    // a slice of sums more: its bytes out and in again, some 2 MB of them to a step's time (0.3 us at 6.8 TB/s)
    return std::max(with_extra, without) + splits * (paired ? 2 : 1) * round_up(T, kStep) * D * 8 / (2 << 20);
}

Layout layout(int64_t T, int64_t V, int64_t D, bool f32, bool in_place, bool bwd) {
    Layout q;
    std::memset(&q, 0, sizeof(q));
    q.form = f32 ? Form::kSplit : bwd && T > kRawTokens ? Form::kHalf : Form::kRaw;
    const bool packed = q.packed = q.form != Form::kRaw || !in_place;
    q.parts = f32 ? 2 : 1;
    q.dl_parts = kDlParts(q.form);
    q.segs = f32 ? kSegs<Product::kOut, Form::kSplit> : q.form == Form::kRaw ? kSegs<Product::kOut, Form::kRaw> : 1;
    // (the low part would take another pass over weight's tiles: backward of 64 tokens, 2048 x 128000 bf16 429 us, 357
    // paired, fp32 1175 and 1074; 128 tokens, 768 x 50257 bf16 93 and 88)
    q.paired = bwd && q.form != Form::kHalf && T <= kHalf;
    q.ld_x = round_up(D, 8);
    q.tpad = round_up(T, kTile);
    const int64_t per_col = std::max(bwd ? q.tpad * 2 * q.dl_parts : 0, packed ? q.ld_x * 2 * q.parts : 0);
    q.piece = V;
    if (per_col > 0) {
        const int64_t most = std::max(kPieceBytes / per_col / kTile * kTile, kMinPiece);
        const int64_t n = (V + most - 1) / most;               // pieces of like widths
        q.piece = std::min(V, round_up((V + n - 1) / n, kTile));
    }
    q.pieces = (V + q.piece - 1) / q.piece;
    q.halves = 0;
    for (int64_t v = 0; v < V; v += q.piece) q.halves += 2 * ((std::min(q.piece, V - v) + kTile - 1) / kTile);
    q.ld_dl = round_up(q.piece, 8);
    q.ld_dx = round_up(D, 4);
    q.splits = 1;
    if (bwd) {
        const int64_t pairs = sm_count() / 2, segs1 = !q.paired ? q.segs : f32 ? kSegsPaired<Form::kSplit> : kSegsPaired<Form::kRaw>;
        int64_t best = -1;
        for (int64_t s = 1; s <= kMaxSplits && (s == 1 || (q.piece / kStep / s >= kMinSteps && s * q.tpad * q.ld_dx * 4 <= kPieceBytes)); ++s) {
            const int64_t c = out_cost(T, D, q.piece, q.segs, segs1, q.paired, s, pairs);
            if (best < 0 || c < best) {
                best = c;
                q.splits = s;
            }
        }
    }
    q.slices = q.splits * (q.paired ? 2 : 1);
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t o = at;
        at += static_cast<size_t>(round_up(bytes, 1024));
        return o;
    };
    q.count = take(4);
    q.range = take(4 * (kRangeW + q.pieces));
    q.rows = take(4 * q.tpad);
    q.tgt = take(4 * q.tpad);
    if (bwd) {
        q.lse = take(4 * q.tpad);
        q.g = take(4 * q.tpad);
    } else {
        q.tl = take(4 * q.tpad);
        q.part = take(8 * q.tpad * q.halves);
    }
    q.x = take(2 * q.parts * q.tpad * q.ld_x);
    if (bwd && q.form != Form::kRaw) q.xg = take(2 * q.parts * q.tpad * q.ld_x);
    if (packed) q.w = take(2 * q.parts * q.piece * q.ld_x);
    if (bwd) {
        q.dl = take(2 * q.dl_parts * q.tpad * q.ld_dl);
        q.dx = take(4 * q.slices * q.tpad * q.ld_dx);
    }
    q.total = at;
    return q;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* q = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(q);
    });
    return fn;
}

// [parts][rows][cols], boxes of 128 bytes by `box_rows` rows, 128-byte swizzle, zeros outside.  (Which 16-bit type it
// is does not matter to a copy; fp32 is added in its type.)
bool make_map(CUtensorMap* m, const void* base, int64_t es, int64_t cols, int64_t rows, int64_t parts, int64_t ld, int64_t part, int box_rows) {
    auto enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(parts)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * es), static_cast<cuuint64_t>((parts > 1 ? part : rows * ld) * es)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(box_rows), 1}, one[3] = {1, 1, 1};
    return enc(m, es == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of CTAs that fit on the device at once.
template <Product P, Form F>
cudaError_t launch_gemm_as(const XentParams& p, int64_t units, cudaStream_t stream) {
    static std::atomic<int> known[64] = {};
    auto* kern = xent_gemm_kernel<P, F>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int pairs = dev < 64 ? known[dev].load() : 0;
    if (pairs == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(gemm_smem(P, F)));
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * sm_count());
        cfg.blockDim = dim3(kGemmThreads);
        cfg.dynamicSmemBytes = gemm_smem(P, F);
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg);
        if (e != cudaSuccess) return e;
        if (pairs < 1) return cudaErrorInvalidConfiguration;
        if (dev < 64) known[dev].store(pairs);
    }
    const unsigned grid = 2 * static_cast<unsigned>(std::min<int64_t>(pairs, std::max<int64_t>(units, 1)));
    return launch_chained(kern, dim3(grid), dim3(kGemmThreads), gemm_smem(P, F), stream, p);
}
template <Product P>
cudaError_t launch_gemm(const XentParams& p, Form form, int64_t units, cudaStream_t stream) {
    if (form == Form::kSplit) return launch_gemm_as<P, Form::kSplit>(p, units, stream);
    if constexpr (P != Product::kLoss)
        if (form == Form::kHalf) return launch_gemm_as<P, Form::kHalf>(p, units, stream);
    return launch_gemm_as<P, Form::kRaw>(p, units, stream);
}

struct Call {
    const void* hidden;
    const void* weight;
    const int32_t* targets;
    const float* dloss;
    const float* lse_in;
    float* loss;
    float* lse;
    void* dhidden;
    void* dweight;
    bool bwd;
};

bool loads_in_place(const void* weight, int64_t stride, int32_t io) {
    return io == SS_BF16 && is_aligned(weight, 16) && stride % 8 == 0 && stride * 2 < (int64_t(1) << 40);
}

ss_status xent(const Call& c, int64_t T, int64_t V, int64_t D, const ss_xent_strides* strides, void* workspace, size_t workspace_bytes,
               void* stream_ptr) {
    if (T < 0 || V < 1 || D < 1) return SS_ERR_INVALID_ARG;
    if (T > SS_XENT_MAX_TOKENS || V > SS_XENT_MAX_V || D > SS_XENT_MAX_D) return SS_ERR_UNSUPPORTED;
    ss_xent_strides s;
    if (strides) {
        s = *strides;
    } else {
        std::memset(&s, 0, sizeof(s));
        s.io_dtype = SS_F32;
        s.hidden_t = s.weight_v = s.dhidden_t = s.dweight_v = D;
        s.dloss_t = 1;
    }
    if (s.io_dtype != SS_F32 && s.io_dtype != SS_BF16) return SS_ERR_INVALID_ARG;
    const bool f32 = s.io_dtype == SS_F32;
    const int64_t es = f32 ? 4 : 2;
    if (!c.bwd && T == 0) return SS_OK;
    if (s.hidden_t < 0 || s.weight_v < D) return SS_ERR_INVALID_ARG;
    if (T > 0 && (!c.hidden || !c.weight || !c.targets)) return SS_ERR_INVALID_ARG;
    if (c.bwd) {
        if (!c.dweight || s.dweight_v < D || s.dloss_t < 0 || (T > 1 && s.dhidden_t < D)) return SS_ERR_INVALID_ARG;
        if (T > 0 && (!c.dloss || !c.lse_in || !c.dhidden)) return SS_ERR_INVALID_ARG;
    } else if (!c.loss || !c.lse) {
        return SS_ERR_INVALID_ARG;
    }
    const bool in_place = loads_in_place(c.weight, s.weight_v, s.io_dtype);
    const Layout q = layout(std::max<int64_t>(T, 1), V, D, f32, in_place, c.bwd);
    if (T > 0 && (!workspace || workspace_bytes < q.total)) return SS_ERR_INVALID_ARG;
    const void* words[] = {c.targets, c.dloss, c.lse_in, c.loss, c.lse};
    for (const void* a : words)
        if (a && !is_aligned(a, 4)) return SS_ERR_MISALIGNED;
    const void* elems[] = {c.hidden, c.weight, c.dhidden, c.dweight};
    for (const void* a : elems)
        if (a && !is_aligned(a, es)) return SS_ERR_MISALIGNED;
    if (T > 0 && !is_aligned(workspace, 256)) return SS_ERR_MISALIGNED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SS_ERR_CUDA;
    for (const void* a : words)
        if (a && T > 0 && !dev_ptr(a, dev)) return SS_ERR_INVALID_ARG;
    for (const void* a : elems)
        if (a && (T > 0 || a == c.dweight) && !dev_ptr(a, dev)) return SS_ERR_INVALID_ARG;
    if (T > 0 && !dev_ptr(workspace, dev)) return SS_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream_ptr);
    if (T == 0)                                    // sums over no tokens
        return cudaMemset2DAsync(c.dweight, static_cast<size_t>(s.dweight_v * es), 0, static_cast<size_t>(D * es), static_cast<size_t>(V), st) ==
                       cudaSuccess
                   ? SS_OK
                   : SS_ERR_CUDA;
    const Range in[] = {range3(c.hidden, 1, T, D, 0, s.hidden_t, es), range3(c.weight, 1, V, D, 0, s.weight_v, es), range3(c.targets, 1, 1, T, 0, 0, 4),
                        range3(c.dloss, 1, T, 1, 0, s.dloss_t, 4), range3(c.lse_in, 1, 1, T, 0, 0, 4)};
    const Range out[] = {range3(c.loss, 1, 1, T, 0, 0, 4), range3(c.lse, 1, 1, T, 0, 0, 4), range3(c.dhidden, 1, T, D, 0, s.dhidden_t, es),
                         range3(c.dweight, 1, V, D, 0, s.dweight_v, es), range3(workspace, 1, 1, static_cast<int64_t>(q.total), 0, 0, 1)};
    for (int i = 0; i < 5; ++i) {
        for (const Range& r : in)
            if (meet(out[i], r)) return SS_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return SS_ERR_INVALID_ARG;
    }

    char* ws = static_cast<char*>(workspace);
    auto f32_at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
    __half* x = reinterpret_cast<__half*>(ws + q.x);
    __half* xg = reinterpret_cast<__half*>(ws + q.xg);
    __half* w = reinterpret_cast<__half*>(ws + q.w);
    __half* dl = reinterpret_cast<__half*>(ws + q.dl);
    const int64_t x_part = q.tpad * q.ld_x, w_part = q.piece * q.ld_x, dl_part = q.tpad * q.ld_dl;
    auto wide = [&](const void* a, int64_t stride) { return is_aligned(a, 16) && (stride * es) % 16 == 0; };

    PrepParams g;
    std::memset(&g, 0, sizeof(g));
    g.hidden = c.hidden; g.hidden_t = s.hidden_t; g.targets = c.targets; g.T = T; g.V = V; g.D = static_cast<int>(D);
    g.per = static_cast<int>(std::min<int64_t>(kPrepThreads, std::max<int64_t>(1, T / 1024)));
    g.x = x; g.xg = xg; g.ld_x = q.ld_x; g.x_part = x_part; g.wide = wide(c.hidden, T > 1 ? s.hidden_t : 0);
    g.count = reinterpret_cast<int*>(ws + q.count); g.rows = reinterpret_cast<int*>(ws + q.rows); g.tgt = reinterpret_cast<int*>(ws + q.tgt);
    g.lse = c.lse_in; g.dloss = c.dloss; g.dloss_t = s.dloss_t; g.lse_c = f32_at(q.lse); g.g_c = f32_at(q.g);
    g.dhidden = c.dhidden; g.dhidden_t = s.dhidden_t; g.loss_out = c.loss; g.lse_out = c.lse;
    g.err = device_error_word();
    g.range = reinterpret_cast<unsigned int*>(ws + q.range);
    const bool raw = q.form == Form::kRaw;
    if (!raw) {
        if (cudaMemsetAsync(g.range, 0, 4 * (kRangeW + q.pieces), st) != cudaSuccess) return SS_ERR_CUDA;
        const unsigned grid = static_cast<unsigned>(std::min<int64_t>((T + kPrepThreads / 32 - 1) / (kPrepThreads / 32), 8 * sm_count()));
        if (f32) xent_range_kernel<float><<<grid, kPrepThreads, 0, st>>>(g);
        else xent_range_kernel<__nv_bfloat16><<<grid, kPrepThreads, 0, st>>>(g);
        if (cudaGetLastError() != cudaSuccess) return SS_ERR_CUDA;
    }
    using B = __nv_bfloat16;
    void (*gather)(PrepParams) = f32   ? (c.bwd ? xent_gather_kernel<float, true, false> : xent_gather_kernel<float, false, false>)
                                 : raw ? (c.bwd ? xent_gather_kernel<B, true, true> : xent_gather_kernel<B, false, true>)
                                       : xent_gather_kernel<B, true, false>;
    const dim3 gather_grid(static_cast<unsigned>((T + g.per - 1) / g.per)), prep(kPrepThreads);
    if (raw) gather<<<gather_grid, prep, 0, st>>>(g);
    const cudaError_t ge = raw ? cudaGetLastError() : launch_chained(gather, gather_grid, prep, 0, st, g);
    if (ge != cudaSuccess) return SS_ERR_CUDA;

    XentParams p;
    std::memset(&p, 0, sizeof(p));
    p.count = g.count; p.tgt = g.tgt; p.D = static_cast<int>(D); p.range = g.range; p.err = g.err;
    p.part = reinterpret_cast<float2*>(ws + q.part); p.ld_part = q.tpad; p.tl = f32_at(q.tl);
    p.lse = g.lse_c; p.g = g.g_c;
    p.dw = c.dweight; p.ld_dw = s.dweight_v; p.dw_wide = c.bwd && wide(c.dweight, s.dweight_v);
    p.dx = f32_at(q.dx); p.ld_dx = q.ld_dx; p.dx_split = q.tpad * q.ld_dx; p.splits = static_cast<int>(q.splits); p.paired = q.paired;
    const int64_t rows = round_up(T, kStep);
    const int64_t mt = (T + kTile - 1) / kTile, dt = (D + kTile - 1) / kTile;
    for (int64_t v0 = 0; v0 < V; v0 += q.piece) {
        const int64_t Vp = std::min(q.piece, V - v0), vt = (Vp + kTile - 1) / kTile;
        const void* wp = static_cast<const char*>(c.weight) + v0 * s.weight_v * es;
        int64_t ld_w = s.weight_v;
        if (q.packed) {
            const unsigned grid = static_cast<unsigned>(std::min<int64_t>((Vp * q.ld_x / 8 + kPrepThreads - 1) / kPrepThreads, 16 * sm_count()));
            const bool ww = wide(wp, s.weight_v);
            auto pack = [&](auto* kern, auto* from) {
                return launch_chained(kern, dim3(grid), prep, 0, st, from, s.weight_v, w, q.ld_x, w_part, Vp, p.D, ww, g.range + kRangeW + p.piece);
            };
            const B* wb = static_cast<const B*>(wp);
            const float* wf = static_cast<const float*>(wp);
            cudaError_t e = f32 ? pack(xent_pack_kernel<float, false, false>, wf)
                                : raw ? pack(xent_pack_kernel<B, true, false>, wb) : pack(xent_pack_kernel<B, false, false>, wb);
            if (e == cudaSuccess && !raw) e = f32 ? pack(xent_pack_kernel<float, false, true>, wf) : pack(xent_pack_kernel<B, false, true>, wb);
            if (e != cudaSuccess) return SS_ERR_CUDA;
            wp = w;
            ld_w = q.ld_x;
        }
        p.v0 = static_cast<int>(v0);
        p.Vp = static_cast<int>(Vp);
        // logits: rows of x and of weight, K along the columns.  (The maps have T rows up to a step of K, not whole
        // tiles of them: what is behind costs no traffic, which for few tokens would be most of it.)
        if (!make_map(&p.a0, x, 2, D, rows, q.parts, q.ld_x, x_part, kHalf) || !make_map(&p.b0, wp, 2, D, Vp, q.parts, ld_w, w_part, kHalf))
            return SS_ERR_CUDA;
        if (!c.bwd) {
            if (launch_gemm<Product::kLoss>(p, q.form, mt * vt, st) != cudaSuccess) return SS_ERR_CUDA;
            p.tile0 += static_cast<int>(vt);
            ++p.piece;
            continue;
        }
        if (!make_map(&p.s0, dl, 2, Vp, rows, q.dl_parts, q.ld_dl, dl_part, 32)) return SS_ERR_CUDA;
        if (launch_gemm<Product::kGrad>(p, q.form, mt * vt, st) != cudaSuccess) return SS_ERR_CUDA;
        // dweight: dl and x with the tokens along rows; dhidden: dl with K along columns, weight with K along rows
        char* dw = static_cast<char*>(c.dweight) + v0 * s.dweight_v * es;
        if (!make_map(&p.a0, dl, 2, Vp, rows, q.dl_parts, q.ld_dl, dl_part, kStep) || !make_map(&p.b0, x, 2, D, rows, q.parts, q.ld_x, x_part, kStep) ||
            (!raw && !make_map(&p.b2, xg, 2, D, rows, q.parts, q.ld_x, x_part, kStep)) ||
            !make_map(&p.a1, dl, 2, Vp, rows, q.dl_parts, q.ld_dl, dl_part, kHalf) || !make_map(&p.b1, wp, 2, D, Vp, q.parts, ld_w, w_part, kStep) ||
            !make_map(&p.s1, p.dx, 4, D, rows, q.slices, q.ld_dx, p.dx_split, 32) ||
            (p.dw_wide && !make_map(&p.s0, dw, es, D, Vp, 1, s.dweight_v, 0, 32)))
            return SS_ERR_CUDA;
        p.add = v0 > 0;
        if (launch_gemm<Product::kOut>(p, q.form, vt * dt + mt * dt * q.splits, st) != cudaSuccess) return SS_ERR_CUDA;
        ++p.piece;
    }
    const unsigned rows_grid = static_cast<unsigned>(std::min<int64_t>((T * ((D + 3) / 4) + kPrepThreads - 1) / kPrepThreads, 8 * sm_count()));
    cudaError_t e;
    if (!c.bwd)
        e = launch_chained(xent_join_kernel, dim3(static_cast<unsigned>((T + kJoinRows - 1) / kJoinRows)), dim3(kJoinThreads), 0, st, p.part, q.tpad,
                           static_cast<int>(q.halves), g.count, g.rows, p.tl, c.loss, c.lse);
    else if (f32)
        e = launch_chained(xent_scatter_kernel<float>, dim3(rows_grid), prep, 0, st, p.dx, p.dx_split, static_cast<int>(q.slices), p.ld_dx, g.count, g.rows,
                           static_cast<float*>(c.dhidden), s.dhidden_t, p.D);
    else
        e = launch_chained(xent_scatter_kernel<__nv_bfloat16>, dim3(rows_grid), prep, 0, st, p.dx, p.dx_split, static_cast<int>(q.slices), p.ld_dx, g.count, g.rows,
                           static_cast<__nv_bfloat16*>(c.dhidden), s.dhidden_t, p.D);
    return e == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

}  // namespace
}  // namespace selscan

using namespace selscan;

extern "C" size_t ss_linear_xent_workspace_size(int64_t tokens, int64_t V, int64_t D, int32_t io_dtype, int32_t backward) {
    if (tokens <= 0 || V < 1 || D < 1 || tokens > SS_XENT_MAX_TOKENS || V > SS_XENT_MAX_V || D > SS_XENT_MAX_D ||
        (io_dtype != SS_F32 && io_dtype != SS_BF16))
        return 0;
    const bool f32 = io_dtype == SS_F32;
    return std::max(layout(tokens, V, D, f32, false, backward != 0).total, layout(tokens, V, D, f32, true, backward != 0).total);
}

extern "C" ss_status ss_linear_xent(const void* hidden, const void* weight, const int32_t* targets, float* loss, float* lse, int64_t tokens,
                                    int64_t V, int64_t D, const ss_xent_strides* strides, void* workspace, size_t workspace_bytes, void* stream) {
    Call c = {};
    c.hidden = hidden; c.weight = weight; c.targets = targets; c.loss = loss; c.lse = lse;
    return xent(c, tokens, V, D, strides, workspace, workspace_bytes, stream);
}

extern "C" ss_status ss_linear_xent_bwd(const float* dloss, const void* hidden, const void* weight, const int32_t* targets, const float* lse,
                                        void* dhidden, void* dweight, int64_t tokens, int64_t V, int64_t D, const ss_xent_strides* strides,
                                        void* workspace, size_t workspace_bytes, void* stream) {
    Call c = {};
    c.hidden = hidden; c.weight = weight; c.targets = targets; c.dloss = dloss; c.lse_in = lse; c.dhidden = dhidden; c.dweight = dweight;
    c.bwd = true;
    return xent(c, tokens, V, D, strides, workspace, workspace_bytes, stream);
}
