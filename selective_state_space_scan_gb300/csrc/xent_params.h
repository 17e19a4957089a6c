// Parameters of the cross entropy's kernels (ss_linear_xent.cu).
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace selscan {

enum class Product { kLoss, kGrad, kOut };

// What the operands of the products are:
//   kRaw    bf16 tensors as they are; dl as the sum of two bf16
//   kHalf   bf16 tensors in fp16, scaled by a power of two (exact), dl in one fp16
//   kSplit  fp32 tensors, and dl, as sums of two scaled fp16
enum class Form { kRaw, kHalf, kSplit };

// Largest finite magnitudes that the scales follow from; weight has one for each piece of the vocabulary.
// kRangeL: the smallest one of dloss but zero, as its distance from infinity's bits.
enum { kRangeX = 0, kRangeG = 1, kRangeL = 2, kRangeW = 3 };

struct XentParams {
    // operands of the products as [part][row][col]; kOut's second product has the maps a1 and b1
    CUtensorMap a0, b0, a1, b1;
    CUtensorMap b2;             // kOut: hidden with the rows' shares of dloss, for dweight where these are unlike
    CUtensorMap s0, s1;         // where results go: dl (kGrad), dweight's rows of the piece and dhidden's sums (kOut)
    const int* count;           // rows that have a target
    const int* tgt;             // [count] their targets
    int D, v0, Vp;              // the piece: columns v0 .. v0 + Vp of the vocabulary
    const unsigned int* range;  // bits of the largest magnitudes (scaled operands); kRangeW: the first piece's
    int piece;                  // the piece's number
    unsigned int* err;
    // kLoss
    float2* part;               // [half tile][ld_part] maximum and sum of a row
    float* tl;                  // [count] logit of the target
    int64_t ld_part;
    int tile0;                  // tiles of the pieces before
    // kGrad
    const float* lse;           // [count]
    const float* g;             // [count] gradient of the loss
    // kOut
    void* dw;
    int64_t ld_dw;
    bool dw_wide;               // rows begin on 16-byte boundaries: stored by s0
    float* dx;                  // [slice][row][ld_dx]
    int64_t ld_dx, dx_split;
    int splits;                 // slices of K that dhidden is summed in (paired: each of them twice, of dl's parts)
    bool paired;                // dl's high part is in one CTA's rows of a tile, its low part in the other's
    bool add;                   // dx has the earlier pieces' sums
};

struct PrepParams {
    const void* hidden;
    const int32_t* targets;
    int64_t hidden_t, T, V;
    int D, per;
    bool wide;                  // rows of hidden begin on 16-byte boundaries
    __half* x;                  // [part][row][ld_x] (bf16 where the operands are raw)
    __half* xg;                 // backward, scaled operands: the same times the rows' shares of the largest dloss, where these are unlike
    int64_t ld_x, x_part;
    int* count;
    int* rows;                  // [count] row of hidden
    int* tgt;
    unsigned int* err;
    unsigned int* range;        // zeros before xent_range_kernel
    float* loss_out;            // forward: zeros in rows without a target
    float* lse_out;
    const float* lse;           // backward
    const float* dloss;
    int64_t dloss_t;
    float* lse_c;
    float* g_c;
    void* dhidden;
    int64_t dhidden_t;
};

}  // namespace selscan
