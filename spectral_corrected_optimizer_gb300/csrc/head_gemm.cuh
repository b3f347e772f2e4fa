// The products of the vocabulary head's loss and gradients (head_gemm.cu), all
// over the compact rows: the tokens that have a target, in token order.
#pragma once

#include "rowvec.cuh"
#include "tc_pair.cuh"

namespace spco {

// Written by the head's first kernel, read by every later one.
struct HeadState {
    int rows;            // tokens with a target
    unsigned blocks_done;
    float inv_count;     // 1 / rows for the mean, 1 for the sum
};

// What the products need of a compact row of h.
struct HeadRow {
    float target_logit;
    float log2e;  // times a tensor-core logit: the logit in log2 (row_log2e)
};

// What turns a row's logits into probabilities: 2^(logit in log2 - m) * inv.  m is a
// whole number, so the exponent is rounded once, to its own size; joined with the
// logarithm of the sum in one fp32 value, a row whose logits are near 1e5 would lose
// 3e-3 of every probability.
struct HeadNorm {
    float m, inv;
    float target;  // softmax - 1 at the target
};

enum HeadJobKind : int {
    HEAD_STATS = 0,  // logits tile -> each row's scale and sum of exponentials without the target's
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

// The compact rows of h and the pieces are stored in column blocks: 64 columns
// of all rows, then the next 64 ([columns / 64][row_cap][64]), so that every box
// the products load or store is one contiguous range of memory.
struct HeadGemm {
    CUtensorMap tm_h_k, tm_w_k, tm_p_k[2];  // boxes of 64 k x 128 rows
    CUtensorMap tm_h, tm_w, tm_p[2];        // boxes of 64 columns x 64 k
    CUtensorMap tm_p_st[2];                 // stores: boxes of 64 columns x 32 rows
    CUtensorMap tm_dh, tm_dw;               // stores: 32 fp32 or 64 bf16 columns x 32 rows
    HeadJob job[kHeadJobs];
    int jobs;
    int vocab, dim;
    int row_cap;               // rows of the compact buffers (a multiple of the tile height)
    const HeadState *state;
    const int *target;         // [row_cap]
    const HeadRow *rows;       // [row_cap]
    float2 *stats;             // [2 * ceil(vocab / 256)][row_cap]: r and the part's sum relative to 2^r
    const HeadNorm *norm;      // [row_cap]
    void *dw;                  // [vocab][dim]
    int dw_bf16, dw_add;
    int dw_tma;                // dw is stored through tm_dw
    float grad_scale;
};

constexpr int kHeadTileM = 256, kHeadTileN = 256;

int head_gemm(const HeadGemm &g, int max_tiles, const char *name, cudaStream_t st);

}  // namespace spco
