// The products of the vocabulary head's loss and gradients (head_gemm.cu), all
// over the compact rows: the tokens that have a target, in token order.
#pragma once

#include "rowvec.cuh"
#include "tc.cuh"

namespace spco {

// Written by the head's first kernel, read by every later one.
struct HeadState {
    int rows;            // tokens with a target
    unsigned blocks_done;
    float inv_count;     // 1 / rows for the mean, 1 for the sum
};

enum HeadJobKind : int {
    HEAD_STATS = 0,  // logits tile -> each row's maximum and its sum of exponentials without the target's
    HEAD_PROB = 1,   // logits tile -> softmax - onehot, bf16, into a piece's buffer
    HEAD_DH = 2,     // dh partial sums (+)= piece . W
    HEAD_DW = 3,     // dw = factor * piece^T . H
};

struct HeadJob {
    int kind;
    int piece;   // which of the two piece buffers
    int v0;      // first vocabulary row of the piece
    int width;   // its vocabulary rows
    int splits;  // HEAD_DH: parts of the piece's rows, each with its own sums
    int add;     // HEAD_DH: add to what the sums hold
};

constexpr int kHeadJobs = 3;

struct HeadGemm {
    CUtensorMap tm_h, tm_w, tm_p[2];
    HeadJob job[kHeadJobs];
    int jobs;
    int vocab, dim;
    int row_cap;               // rows of the compact buffers (a multiple of the tile height)
    int piece_ld;              // columns of a piece buffer
    const HeadState *state;
    const int *target;         // [row_cap]
    float2 *stats;             // [2 * ceil(vocab / 256)][row_cap]
    const float4 *norm;        // [row_cap]: largest logit, 1 / sum, softmax - 1 at the target
    bf16 *piece[2];            // [row_cap][piece_ld]
    float *dh;                 // [splits][row_cap][dh_ld]
    int dh_ld;
    void *dw;                  // [vocab][dim]
    int dw_bf16, dw_add, dw_vec;
    float grad_scale;
};

constexpr int kHeadTileM = 128, kHeadTileN = 256;

int head_gemm(const HeadGemm &g, int max_tiles, const char *name, cudaStream_t st);

}  // namespace spco
