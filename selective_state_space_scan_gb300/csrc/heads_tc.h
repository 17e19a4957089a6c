// The tensor-core path of ss_heads_fwd (ss_heads_tc.cu): its parameters, workspace and launch.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "heads_params.h"

namespace selscan {

constexpr int kHeadsChunk = 128;        // tokens per chunk
constexpr int kHeadsTile = 64;          // rows of the state per tile

struct HeadsTcParams {
    HeadsParams p;
    uint8_t* images;                    // [chunks, G][B hi, B lo, C][nb] blocks of 128 × 64 bf16
    int32_t* chunk_base;                // [n_seq + 1] first chunk of a sequence
    int32_t* seg_base;                  // [n_seq + 1] first segment of a sequence
    float* seg_state;                   // [segments, gtiles][16][128][4]: what a segment leaves from zero
    float* seg_decay;                   // [segments, gtiles]: its log2 decay
    int32_t* order;                     // [segments][sequence, segment], by the segment's number
    float* handover;                    // [n_seq, pairs, 2][16][128][4]: the state between two segments
    unsigned int* flags;                // [n_seq, pairs, 2]: segments done
    int nflags;
    int seg_chunks;                     // chunks per segment
    int pairs;                          // pairs of tiles, over all groups
    int gtiles;                         // tiles, over all heads
    int nb;                             // blocks of 64 states
    bool wide_w, wide_y;                // conv_w on a boundary of 16 bytes; the quads of y on boundaries of 8
};

struct HeadsTcPlan {
    int64_t chunks, segments;           // upper bounds over all lengths that make up `tokens`
    int seg_chunks, pairs, gtiles, nb, ctas, chains;
    size_t off_images, off_chunk_base, off_seg_base, off_state, off_decay, off_handover, off_flags, off_order,
        bytes;                          // in the workspace
    bool split;
};

int heads_sm_count();                   // of the current device
// Whether the tensor-core path takes these sizes.
bool heads_tc_takes(int64_t n_seq, int64_t tokens, int64_t H, int64_t P, int64_t G, int64_t N, bool bf16);
HeadsTcPlan heads_tc_plan(int64_t n_seq, int64_t tokens, int64_t H, int64_t P, int64_t G, int64_t N);
cudaError_t launch_heads_tc(const HeadsParams& p, void* workspace, bool bf16, cudaStream_t stream);

}  // namespace selscan
