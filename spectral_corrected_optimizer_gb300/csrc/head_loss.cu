// Softmax cross entropy of the vocabulary head and its gradients
// (include/stage_ends.h): the last stage of the training pipeline.
//
//   l_i = h_i W^T,  row_loss_i = log sum_v exp(l_iv) - l_i,target,
//   d = (softmax(l) - onehot) * factor,  dh = d W,  dW = d^T h
//
// Order of the work (N tokens with a target, V rows of W, width D):
//   1. the tokens that have a target are counted and listed, their rows of h
//      copied together: a token without one costs nothing afterwards;
//   2. one product over the whole vocabulary leaves a reference exponent and the
//      sum of exponentials relative to it of each row and 128 logits; they are
//      joined into the row's loss and normalisation (2 N V D flops);
//   3. for each piece of the vocabulary, logits are formed again and turned
//      into softmax - onehot of the piece (bf16, 2 N V D flops), which feeds
//      the two gradient products (4 N V D).  A launch runs piece i's
//      probabilities beside piece i-1's products, so two piece buffers exist
//      and no [N][V] tensor does.  dh sums up in fp32 over the pieces.
// The products are in head_gemm.cu.
//
// A piece's logits are formed twice, 8 N V D operations where keeping [N][V] would take
// 6: that is the price of not keeping them, and of rounding a probability once (bf16,
// normalised) instead of twice.  Measured on a GB300: 8192 tokens, a tenth without a
// target, V = 128256, D = 2048: 9.25 ms (9.0 before the power limit sets in), 1.68
// PFLOP/s; loss alone of 2048 tokens 650 us (579); of one token over 32001 x 4096 62 us
// (W once: 39 us; its 126 tiles lie on 76 pairs of SMs, 83 %, and three launches); loss
// and gradients of 333 tokens, half without a target, over 50001 x 1000 126 us.
#include <algorithm>
#include <cstring>
#include <string>

#include "head_gemm.cuh"

namespace spco {
namespace {

// log2(e) and what its fp32 value lacks
constexpr float kLog2e = 1.4426950408889634f, kLog2eRest = (float)(1.4426950408889634074 - (double)kLog2e);
constexpr float kLn2 = 0.6931471805599453f;

// ---- the rows that have a target ---------------------------------------------------------

// 8 bf16 values of a row from column 8 v, zero behind dim
__device__ __forceinline__ uint4 row_vec(const uint16_t *row, int v, int dim, bool vec) {
    if (vec) return __ldg(reinterpret_cast<const uint4 *>(row) + v);
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = v * 8 + i < dim ? row[v * 8 + i] : 0u;
    return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}

__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float s) {
    return fmaf(hi_f(a), hi_f(b), fmaf(lo_f(a), lo_f(b), s));
}

// The tensor cores cut off, rather than round, what falls below the last place of
// each of the dim / 16 sums on the way to a logit, which leaves it short in the
// mean.  In units of 2^-24 dim / 32 of the logit, measured for dim 512 to 65536: 0.38
// to 0.54 over normal values with and without a common direction (standard deviation
// 0.15 to 0.4); 0.7 to 2.9 where all products have one sign; 0 where the sums are
// exact.  Half a unit, dim 2^-30, is given back in the factor of the exponent: the
// loss of one token at 32001 x 4096 is 2e-8 to 5e-7 off, 1.2e-6 without.  16 products
// of which h holds only zeros cut nothing off and do not count, so a logit of a few
// values of h is left as it is.  Where dense h and w make exact sums (small whole
// numbers), the logits other than the target's come out dim 2^-30 of themselves too far
// from 0, as inexact ones would come out too near it without the factor.
__device__ __forceinline__ float row_log2e(int blocks) {  // of 16 values of h, not all 0
    return kLog2e + fmaf(kLog2e, (float)max(blocks - 1, 0) * 0x1p-26f, kLog2eRest);
}
// how many of the 16 blocks of a warp's 32 pieces (8 values) hold anything but zeros
__device__ __forceinline__ int blocks_of(uint4 a) {
    const unsigned b = __ballot_sync(0xffffffffu, ((a.x | a.y | a.z | a.w) & 0x7fff7fffu) != 0);
    return __popc((b | b >> 1) & 0x55555555u);
}

constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;

__device__ __forceinline__ bool has_target(int64_t id, int64_t ignore, int vocab) {
    return id != ignore && id >= 0 && id < vocab;
}

// Targets among each kStretch neighbouring tokens.
constexpr int kStretch = 4096;
template <typename ID>
__global__ void __launch_bounds__(kRowThreads) head_count_kernel(const ID *__restrict__ targets, int64_t ignore,
                                                                 int vocab, int *__restrict__ counts) {
    const ID *from = targets + (int64_t)blockIdx.x * kStretch;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kStretch; i += kRowThreads)
        n += __syncthreads_count(has_target((int64_t)from[i + threadIdx.x], ignore, vocab));
    if (threadIdx.x == 0) counts[blockIdx.x] = n;
}

// Lists the tokens with a target in token order (row_of[r] = token of row r,
// at[t] = row of token t or -1, target[r]) and copies their rows of h together,
// in column blocks of 64 (zero behind dim).  Each block takes `share`
// neighbouring tokens (at most one per thread), counts the targets in front of
// them itself -- the ids come from L2, a kernel of its own for the list would
// cost more; among many tokens whole stretches come counted (counts, null for
// few) -- and then copies its rows, a warp per row.  The last blocks append the
// zero rows up to the next multiple of 64.
//
// On the way the logit of each row's target is formed as an fp32 dot product:
// the loss is the difference between it and the log-sum-exp, and a tensor core's
// logit is off by more than fp32's rounding (row_log2e).
constexpr int kPadBlocks = 8;
template <typename ID>
__global__ void __launch_bounds__(kRowThreads) head_rows_kernel(const ID *__restrict__ targets, int64_t ignore, int tokens,
                                                        int vocab, int mean, int share, int own_blocks, const int *counts,
                                                        const uint16_t *__restrict__ h,
                                                        const uint16_t *__restrict__ w, int dim, int row_cap, int h_vec,
                                                        int w_vec, HeadState *state, int *__restrict__ row_of,
                                                        int *__restrict__ at, int *__restrict__ target,
                                                        uint16_t *__restrict__ out, HeadRow *__restrict__ head_row,
                                                        float *__restrict__ row_loss, unsigned *flag) {
    __shared__ int red[2][kRowWarps], own_token[kRowThreads], own_target[kRowThreads];
    __shared__ float dots[kRowWarps];
    __shared__ int held[kRowWarps];
    grid_dependency_launch();
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int pad = (int)blockIdx.x - own_blocks;  // >= 0: a block of zero rows, which counts all targets
    const int t0 = pad >= 0 ? tokens : (int)blockIdx.x * share, t1 = min(t0 + share, tokens);
    int before = 0, first = 0;  // tokens in front of `first` are in counts
    if (counts) {
        const int whole = t0 / kStretch;
        for (int i = threadIdx.x; i < whole; i += kRowThreads) before += counts[i];
        first = whole * kStretch;
    }
#pragma unroll 4
    for (int t = first + threadIdx.x; t < t0; t += kRowThreads) before += has_target((int64_t)targets[t], ignore, vocab);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    const int t = t0 + threadIdx.x;
    const int64_t id = t < t1 ? (int64_t)targets[t] : ignore;
    const bool has = has_target(id, ignore, vocab);
    if (id != ignore && !has) atomicExch(flag, kSiteTarget);
    const unsigned ballot = __ballot_sync(0xffffffffu, has);
    if (lane == 0) {
        red[0][wp] = before;
        red[1][wp] = __popc(ballot);
    }
    __syncthreads();
    before = 0;
    int count = 0, k = __popc(ballot & ((1u << lane) - 1u));
#pragma unroll
    for (int i = 0; i < kRowWarps; ++i) {
        before += red[0][i];
        if (i < wp) k += red[1][i];
        count += red[1][i];
    }
    if (t < t1) at[t] = has ? before + k : -1;
    if (has) {
        row_of[before + k] = t;
        target[before + k] = (int)id;
        own_token[k] = t;
        own_target[k] = (int)id;
    } else if (t < t1) {
        row_loss[t] = 0.f;
    }
    __syncthreads();
    const int vecs = (dim + 63) / 64 * 8;
    const int copy = pad >= 0 ? (before + 63) / 64 * 64 - before : count;
    if (pad == -1 && threadIdx.x == 0) {
        const int rows = before + count;
        state->rows = rows;
        state->blocks_done = 0;
        state->inv_count = mean ? 1.f / (float)max(rows, 1) : 1.f;
    }
    // one token per block: its row is shared by all warps
    if (share == 1 && pad < 0) {
        if (count == 0) return;
        const uint16_t *hr = h + (int64_t)own_token[0] * dim, *wr = w + (int64_t)own_target[0] * dim;
        float s = 0.f;
        int n = 0;
        for (int v0 = wp * 32; v0 < vecs; v0 += kRowThreads) {
            const int v = v0 + lane;
            uint4 a = make_uint4(0, 0, 0, 0);
            if (v * 8 < dim) {
                a = row_vec(hr, v, dim, h_vec);
                const uint4 b = row_vec(wr, v, dim, w_vec);
                s += dot2(a.x, b.x, dot2(a.y, b.y, dot2(a.z, b.z, dot2(a.w, b.w, 0.f))));
            }
            if (v < vecs) reinterpret_cast<uint4 *>(out + ((int64_t)(v / 8) * row_cap + before) * 64)[v % 8] = a;
            n += blocks_of(a);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) {
            dots[wp] = s;
            held[wp] = n;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kRowWarps; ++i) {
                s += dots[i];
                n += held[i];
            }
            head_row[before] = HeadRow{s, row_log2e(n)};
        }
        return;
    }
    for (int i = max(pad, 0) * kRowWarps + wp; i < copy; i += (pad >= 0 ? kPadBlocks : 1) * kRowWarps) {
        const int r = before + i;
        const uint16_t *hr = i < count ? h + (int64_t)own_token[i] * dim : nullptr;
        const uint16_t *wr = i < count ? w + (int64_t)own_target[i] * dim : nullptr;
        float s = 0.f;
        int n = 0;
#pragma unroll 4
        for (int v0 = 0; v0 < vecs; v0 += 32) {
            const int v = v0 + lane;
            uint4 a = make_uint4(0, 0, 0, 0);
            if (hr && v * 8 < dim) {
                a = row_vec(hr, v, dim, h_vec);
                const uint4 b = row_vec(wr, v, dim, w_vec);
                s += dot2(a.x, b.x, dot2(a.y, b.y, dot2(a.z, b.z, dot2(a.w, b.w, 0.f))));
            }
            if (v < vecs) reinterpret_cast<uint4 *>(out + ((int64_t)(v / 8) * row_cap + r) * 64)[v % 8] = a;
            n += blocks_of(a);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0 && i < count) head_row[r] = HeadRow{s, row_log2e(n)};
    }
}

// Rows of W with ld values each: the tensor copies need rows of 16-byte multiples.
__global__ void __launch_bounds__(256) head_pad_kernel(const uint16_t *__restrict__ src, int64_t rows, int dim, int ld,
                                                       uint16_t *__restrict__ dst) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int v = threadIdx.x; v < ld / 8; v += blockDim.x)
            reinterpret_cast<uint4 *>(dst + r * ld)[v] = row_vec(src + r * dim, v, dim, false);
}

// ---- joining the row statistics ------------------------------------------------------------

// (m, s) <- (m, s) joined with a part: sums relative to 2^m, m whole numbers, so
// the factors are exact powers of two
__device__ __forceinline__ void join(float &m, float &s, float2 x) {
    const float top = fmaxf(m, x.x), ref = top == -INFINITY ? 0.f : top;
    s = s * exp2f(m - ref) + x.y * exp2f(x.x - ref);
    m = top;
}

// ROWS rows per block, LANES threads per row: each joins every LANES-th part, then
// a warp per row joins what its threads hold by halves.  The parts' sums
// leave the target out: S of them, relative to 2^r, and e = 2^(target's logit in
// log2 - r) give softmax - 1 = -S / (S + e) and the loss log(1 + S / e) without
// the cancellation that a well-predicted token (S small) would meet in 1 - p and
// in lse - l.  The last block to finish adds up the blocks' loss sums, in block
// order.
// Bound by the latency of a thread's reads while the blocks fit on the SMs at once:
// 8 rows per block then, 126 us for 333 tokens over 50001 x 1000 where 32 take 129;
// by the width of the reads when they do not: 32 rows then, 26 us for 8192 tokens
// and 1002 parts where 8 take 49.
constexpr int kLseThreads = 1024, kLseFew = 8, kLseMany = 32;
template <int ROWS>
__global__ void __launch_bounds__(kLseThreads) head_lse_kernel(const float2 *stats, int parts, int row_cap,
                                                       const HeadRow *head_row,
                                                       const int *row_of, HeadState *state,
                                                       HeadNorm *__restrict__ norm, float *__restrict__ row_loss,
                                                       float *__restrict__ block_loss, float *__restrict__ loss) {
    constexpr int LANES = kLseThreads / ROWS;
    __shared__ float sm[LANES][ROWS + 1], ss[LANES][ROWS + 1], row_sum[ROWS];
    grid_dependency_launch();
    grid_dependency_wait();
    const int rows = state->rows, row0 = blockIdx.x * ROWS, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float m = -INFINITY, s = 0.f;
    {
        const int c = threadIdx.x % ROWS, first = threadIdx.x / ROWS;
        if (row0 + c < rows) {
#pragma unroll 8
            for (int p = first; p < parts; p += LANES) join(m, s, stats[(int64_t)p * row_cap + row0 + c]);
        }
        sm[first][c] = m;
        ss[first][c] = s;
    }
    __syncthreads();
    if (w < ROWS) {  // warp w has row w of the block
        m = sm[lane][w];
        s = ss[lane][w];
#pragma unroll
        for (int i = 32; i < LANES; i += 32) join(m, s, make_float2(sm[i + lane][w], ss[i + lane][w]));
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
            join(m, s, make_float2(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o)));
        if (lane == 0) {
            const int row = row0 + w;
            float l = 0.f;
            if (row < rows) {
                // the target's logit in log2, to twice fp32's digits: hi + lo
                const float lt = head_row[row].target_logit, hi = lt * kLog2e;
                const float lo = fmaf(lt, kLog2e, -hi) + lt * kLog2eRest;
                // log2 of 2^r / e^target; a target's logit of -inf (or one that overflows in log2) leaves no term
                const bool none = hi == -INFINITY;
                const float above = none ? INFINITY : (m - hi) - lo;
                const float total = s + exp2f(-above);
                norm[row] = HeadNorm{m, 1.f / total, -s / total};
                // 2^30 S stays far from overflow; beyond it log(total) is no longer a small correction
                l = above < 30.f ? log1pf(s * exp2f(above))
                    : none       ? (m + log2f(total)) * kLn2 - lt
                                 : (above + log2f(total)) * kLn2;
                row_loss[row_of[row]] = l;
            }
            row_sum[w] = l;
        }
    }
    __syncthreads();
    if (w != 0) return;
    float l = lane < ROWS ? row_sum[lane] : 0.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    int last = 0;
    if (lane == 0) {
        block_loss[blockIdx.x] = l;
        __threadfence();
        last = atomicAdd(&state->blocks_done, 1u) == gridDim.x - 1;
    }
    if (!__shfl_sync(0xffffffffu, last, 0)) return;
    __threadfence();
    l = 0.f;
#pragma unroll 8
    for (int b = lane; b < (int)gridDim.x; b += 32) l += __ldcg(block_loss + b);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) *loss = l * state->inv_count;
}

// dh[t] = factor * sum over the parts of the token's row; zero without a target.
// The sums' rows are read from where dh's 16-byte pieces begin (VEC: column 0).
template <bool VEC>
__global__ void __launch_bounds__(256) head_dh_kernel(const Span<const float> sums, int parts, int row_cap, int ld,
                                                      const int *at, const HeadState *state,
                                                      float grad_scale, int tokens, int dim, const Span<bf16> dh) {
    grid_dependency_wait();
    const float factor = grad_scale * state->inv_count;
    for (int t = blockIdx.x; t < tokens; t += gridDim.x) {
        const int r = at[t];
        const int64_t row = dh.lo + (int64_t)t * dim;
        const int first = VEC ? 0 : -(int)(row & 7);
        for (int col = first + (int)threadIdx.x * 8; col < dim; col += blockDim.x * 8) {
            float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (r >= 0) {
#pragma unroll 4
                for (int p = 0; p < parts; ++p) {
                    float x[8];
                    const int64_t at = ((int64_t)p * row_cap + r) * ld + col;
                    if (VEC) load8(sums.p + at, x);
                    else load_any(sums, at, x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) a[i] += x[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) a[i] *= factor;
            }
            if (VEC) store8(dh.p + row + col, a);
            else store_any(dh, row + col, row, row + dim, a);
        }
    }
}

// ---- plan ------------------------------------------------------------------------------------

// Bytes of one piece buffer.  Each piece adds to dh once and ends a launch, so few
// large ones are better, although a piece of 256 MB does not stay in L2: 8192 tokens
// over 128256 x 2048 take 9.27 ms with 256 or 192 MB, 9.38 with 128, 9.6 with 64; 16384
// 21.3 ms with 256, 21.4 with 192, 21.8 with 128 or less.  But at least 4096 vocabulary
// rows, so that adding up dh stays small beside the products.
constexpr int64_t kPieceBytes = 256 << 20;
constexpr int kPieceMin = 4096;

struct HeadPlan {
    int row_cap, ld, parts, piece, pieces, splits, dh_ld;
    int64_t off_state, off_counts, off_row_of, off_at, off_target, off_head_row, off_norm, off_block_loss, off_stats,
        off_h, off_w, off_p0, off_p1, off_dh, bytes;
};

HeadPlan plan_head(int64_t tokens, int64_t vocab, int32_t dim, bool grad) {
    HeadPlan p{};
    p.row_cap = (int)round_up(std::max<int64_t>(tokens, 1), kHeadTileM);
    p.ld = (int)round_up(dim, 8);
    p.parts = (int)(2 * ceil_div(vocab, kHeadTileN));
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += round_up(bytes, 1024);
        return here;
    };
    const int64_t cap = p.row_cap;
    p.off_state = take(sizeof(HeadState));
    p.off_counts = take(tokens / kStretch * 4);
    p.off_row_of = take(cap * 4);
    p.off_at = take(cap * 4);
    p.off_target = take(cap * 4);
    p.off_head_row = take(cap * sizeof(HeadRow));
    p.off_norm = take(cap * sizeof(HeadNorm));
    p.off_block_loss = take(ceil_div(cap, kLseFew) * 4);
    p.off_stats = take((int64_t)p.parts * cap * 8);
    p.off_h = take(cap * round_up(dim, 64) * 2);
    p.off_w = p.ld != dim ? take(vocab * p.ld * 2) : 0;
    if (grad) {
        const int64_t all = round_up(vocab, kHeadTileN);
        const int64_t fit = kPieceBytes / (cap * 2) / kHeadTileN * kHeadTileN;
        p.piece = (int)std::min(all, std::max<int64_t>(fit, kPieceMin));
        p.pieces = (int)ceil_div(vocab, p.piece);
        // few rows: the long sum over the vocabulary is split until every pair of SMs has a tile (one
        // token over 128256 x 2048 424 us, 850 unsplit; 167 over 50001 x 1000 145 and 342; 2048 over
        // 32001 x 1000 369 and 379)
        p.dh_ld = (int)round_up(dim, 32);
        const int64_t tiles = (cap / kHeadTileM) * ceil_div(dim, kHeadTileN);
        const int64_t blocks = ceil_div(std::min<int64_t>(vocab, p.piece), 64);
        p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(num_sms() / 2 / tiles, blocks / 8));
        p.off_p0 = take(cap * p.piece * 2);
        p.off_p1 = p.pieces > 1 ? take(cap * p.piece * 2) : p.off_p0;
        p.off_dh = take((int64_t)p.splits * cap * p.dh_ld * 4);
    }
    p.bytes = at;
    return p;
}

int check_sizes(int64_t tokens, int64_t vocab, int32_t dim, const char *what) {
    if (tokens < 0 || tokens > (int64_t)1 << 24)
        return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": tokens outside [0, 2^24]");
    if (vocab < 1 || vocab > (int64_t)1 << 24)
        return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": vocab outside [1, 2^24]");
    if (dim < 1 || dim > 1 << 16) return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": dim outside [1, 65536]");
    if (round_up(tokens, kHeadTileM) * ceil_div(dim, 64) > INT32_MAX)
        return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": tokens x dim above 2^37");
    return SPECOPTIM_OK;
}

struct HeadCall {
    const void *h, *w, *targets;
    int32_t id_bytes;
    int64_t ignore, tokens, vocab;
    int32_t dim, mean;
    float *loss, *row_loss;
    char *ws;
    int64_t ws_bytes;
    cudaStream_t st;
};

int check_call(const HeadCall &c, const HeadPlan &p, const std::string &what) {
    if (c.id_bytes != 4 && c.id_bytes != 8) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": id_bytes must be 4 or 8");
    if (!c.w || !c.loss || !c.ws || (c.tokens > 0 && (!c.h || !c.targets || !c.row_loss)))
        return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": null pointer");
    if (!aligned_to(c.h, 2) || !aligned_to(c.targets, c.id_bytes) || !aligned_to(c.loss, 4) ||
        !aligned_to(c.row_loss, 4) || !aligned16(c.w) || !aligned16(c.ws))
        return fail(SPECOPTIM_ERR_MISALIGNED, what + ": w and the workspace must be 16-byte aligned, the rest to its elements");
    if (c.ws_bytes < p.bytes)
        return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": the workspace is smaller than " + what + "_workspace() says");
    return SPECOPTIM_OK;
}

// From so many tokens on their targets are counted in stretches first; below, each block counts
// all of those in front of it, which grows with the square of the tokens but saves the launch (width
// 8, listing / count + listing: 32768 tokens 22 / 6 + 15 us, 65536 35 / 7 + 22, 2^20 1056 / 8 + 207).
constexpr int kCountTokens = 1 << 16;

// Steps 1 and 2: afterwards loss, row_loss and the rows' norms exist.
int run_loss(const HeadCall &c, const HeadPlan &p, bool grad, HeadGemm *g) {
    std::memset(g, 0, sizeof(*g));
    HeadState *state = reinterpret_cast<HeadState *>(c.ws + p.off_state);
    int *row_of = reinterpret_cast<int *>(c.ws + p.off_row_of), *at = reinterpret_cast<int *>(c.ws + p.off_at);
    int *target = reinterpret_cast<int *>(c.ws + p.off_target);
    HeadRow *head_row = reinterpret_cast<HeadRow *>(c.ws + p.off_head_row);
    HeadNorm *norm = reinterpret_cast<HeadNorm *>(c.ws + p.off_norm);
    uint16_t *hc = reinterpret_cast<uint16_t *>(c.ws + p.off_h);
    const uint16_t *w = static_cast<const uint16_t *>(c.w);
    const int tokens = (int)c.tokens, vocab = (int)c.vocab;
    // tokens per block: one each while there are SMs for them, at most one per thread
    const int share = std::max(1, std::min(kRowThreads, tokens / (num_sms() * 4)));
    const int blocks = (int)std::max<int64_t>(1, ceil_div(tokens, share));
    const bool w_vec = c.dim % 8 == 0, h_vec = w_vec && aligned16(c.h);
    int *counts = tokens >= kCountTokens ? reinterpret_cast<int *>(c.ws + p.off_counts) : nullptr;
    auto rows = [&](auto id) {
        using ID = decltype(id);
        if (counts)
            SPCO_LAUNCH("head_count", c.st,
                        head_count_kernel<ID><<<tokens / kStretch, kRowThreads, 0, c.st>>>(
                            static_cast<const ID *>(c.targets), c.ignore, vocab, counts));
        SPCO_LAUNCH("head_rows", c.st,
                    head_rows_kernel<ID><<<blocks + (grad ? kPadBlocks : 0), kRowThreads, 0, c.st>>>(
                        static_cast<const ID *>(c.targets), c.ignore, tokens, vocab, c.mean, share, blocks, counts,
                        static_cast<const uint16_t *>(c.h), w, c.dim, p.row_cap, h_vec, w_vec, state, row_of, at, target,
                        hc, head_row, c.row_loss, stage_flag_ptr()));
    };
    if (c.id_bytes == 8) rows(int64_t{});
    else rows(int32_t{});
    if (p.ld != c.dim) {
        uint16_t *wc = reinterpret_cast<uint16_t *>(c.ws + p.off_w);
        SPCO_LAUNCH("head_pad", c.st,
                    head_pad_kernel<<<(unsigned)std::min<int64_t>(c.vocab, num_sms() * 16),
                                  (unsigned)std::min<int64_t>(256, round_up(p.ld / 8, 32)), 0, c.st>>>(
                        w, c.vocab, c.dim, p.ld, wc));
        w = wc;
    }
    SPECOPTIM_LAUNCHED("head_rows_kernel");
    const int64_t h_lines = ceil_div(c.dim, 64) * p.row_cap;
    if (int rc = make_tmap_2d_bf16(&g->tm_h_k, hc, h_lines, 64, 64, 128)) return rc;
    if (int rc = make_tmap_2d_bf16(&g->tm_w_k, w, c.vocab, p.ld, p.ld, 128)) return rc;
    if (int rc = make_tmap_2d_bf16(&g->tm_h, hc, h_lines, 64, 64, 64)) return rc;
    if (int rc = make_tmap_2d_bf16(&g->tm_w, w, c.vocab, p.ld, p.ld, 64)) return rc;
    g->vocab = vocab;
    g->dim = c.dim;
    g->row_cap = p.row_cap;
    g->state = state;
    g->target = target;
    g->rows = head_row;
    g->stats = reinterpret_cast<float2 *>(c.ws + p.off_stats);
    g->norm = norm;
    g->jobs = 1;
    g->job[0] = HeadJob{HEAD_STATS, 0, 0, vocab, 1, 0};
    const int64_t tiles = (int64_t)(p.row_cap / kHeadTileM) * (p.parts / 2);
    if (int rc = head_gemm(*g, (int)std::min<int64_t>(tiles, INT32_MAX), "head_stats", c.st)) return rc;
    cudaError_t e = cudaSuccess;
    const int lse_rows = p.row_cap / kLseFew <= 2 * num_sms() ? kLseFew : kLseMany;  // two blocks an SM
    auto *lse = lse_rows == kLseFew ? &head_lse_kernel<kLseFew> : &head_lse_kernel<kLseMany>;
    SPCO_LAUNCH("head_lse", c.st,
                e = launch_dependent(lse, dim3(p.row_cap / lse_rows), dim3(kLseThreads), 0, c.st, g->stats, p.parts,
                                     p.row_cap, head_row, row_of, state, norm, c.row_loss,
                                     reinterpret_cast<float *>(c.ws + p.off_block_loss), c.loss));
    SPECOPTIM_CUDA(e);
    return SPECOPTIM_OK;
}

}  // namespace
}  // namespace spco

using namespace spco;

extern "C" int64_t head_loss_workspace(int64_t tokens, int64_t vocab, int32_t dim) {
    int64_t bytes = -1;
    entry([&]() -> int {
        if (int rc = check_sizes(tokens, vocab, dim, "head_loss")) return rc;
        bytes = plan_head(tokens, vocab, dim, false).bytes;
        return SPECOPTIM_OK;
    });
    return bytes;
}

extern "C" int64_t head_loss_grad_workspace(int64_t tokens, int64_t vocab, int32_t dim) {
    int64_t bytes = -1;
    entry([&]() -> int {
        if (int rc = check_sizes(tokens, vocab, dim, "head_loss_grad")) return rc;
        bytes = plan_head(tokens, vocab, dim, true).bytes;
        return SPECOPTIM_OK;
    });
    return bytes;
}

extern "C" int head_loss(const void *h, const void *w, const void *targets, int32_t id_bytes, int64_t ignore_index,
                         int64_t tokens, int64_t vocab, int32_t dim, int32_t mean, float *loss, float *row_loss,
                         void *workspace, int64_t workspace_bytes, void *stream) {
    return entry([&]() -> int {
        if (int rc = check_sizes(tokens, vocab, dim, "head_loss")) return rc;
        const HeadPlan p = plan_head(tokens, vocab, dim, false);
        const HeadCall c{h, w, targets, id_bytes, ignore_index, tokens, vocab, dim, mean, loss, row_loss,
                         static_cast<char *>(workspace), workspace_bytes, static_cast<cudaStream_t>(stream)};
        if (int rc = check_call(c, p, "head_loss")) return rc;
        if (int rc = bind_device()) return rc;
        HeadGemm g;
        return run_loss(c, p, false, &g);
    });
}

extern "C" int head_loss_grad(const void *h, const void *w, const void *targets, int32_t id_bytes,
                              int64_t ignore_index, int64_t tokens, int64_t vocab, int32_t dim, int32_t mean,
                              float grad_scale, float *loss, float *row_loss, void *dh, void *dw, int32_t dw_type,
                              int32_t accumulate, void *workspace, int64_t workspace_bytes, void *stream) {
    return entry([&]() -> int {
        if (int rc = check_sizes(tokens, vocab, dim, "head_loss_grad")) return rc;
        const HeadPlan p = plan_head(tokens, vocab, dim, true);
        const HeadCall c{h, w, targets, id_bytes, ignore_index, tokens, vocab, dim, mean, loss, row_loss,
                         static_cast<char *>(workspace), workspace_bytes, static_cast<cudaStream_t>(stream)};
        if (int rc = check_call(c, p, "head_loss_grad")) return rc;
        if (!dw || (tokens > 0 && !dh)) return fail(SPECOPTIM_ERR_INVALID_ARG, "head_loss_grad: null pointer");
        if (!type_ok(dw_type))
            return fail(SPECOPTIM_ERR_INVALID_ARG, "head_loss_grad: dw_type must be STAGE_BF16 or STAGE_FP32");
        if (!aligned_to(dh, 2) || !aligned_to(dw, type_bytes(dw_type)))
            return fail(SPECOPTIM_ERR_MISALIGNED, "head_loss_grad: dh and dw must be aligned to their elements");
        if (int rc = bind_device()) return rc;
        HeadGemm g;
        if (int rc = run_loss(c, p, true, &g)) return rc;
        const int64_t p_lines = (int64_t)(p.piece / 64) * p.row_cap;
        for (int b = 0; b < std::min(p.pieces, 2); ++b) {
            char *piece = c.ws + (b ? p.off_p1 : p.off_p0);
            if (int rc = make_tmap_2d_bf16(&g.tm_p_k[b], piece, p_lines, 64, 64, 128)) return rc;
            if (int rc = make_tmap_2d_bf16(&g.tm_p[b], piece, p_lines, 64, 64, 64)) return rc;
            if (int rc = make_tmap_2d_bf16(&g.tm_p_st[b], piece, p_lines, 64, 64, 32)) return rc;
        }
        float *dh_sums = reinterpret_cast<float *>(c.ws + p.off_dh);
        if (int rc = make_tmap_2d(&g.tm_dh, dh_sums, (int64_t)p.splits * p.row_cap, p.dh_ld, p.dh_ld, 32, 32)) return rc;
        g.dw = dw;
        g.dw_bf16 = dw_type == STAGE_BF16;
        g.dw_add = accumulate != 0;
        g.dw_tma = aligned16(dw) && dim * type_bytes(dw_type) % 16 == 0 && !(g.dw_bf16 && g.dw_add);
        if (g.dw_tma && g.dw_bf16) {
            if (int rc = make_tmap_2d_bf16(&g.tm_dw, dw, vocab, dim, dim, 32)) return rc;
        } else if (g.dw_tma) {
            if (int rc = make_tmap_2d(&g.tm_dw, static_cast<float *>(dw), vocab, dim, dim, 32, 32)) return rc;
        }
        g.grad_scale = grad_scale;
        const int64_t m_tiles = p.row_cap / kHeadTileM, d_tiles = ceil_div(dim, kHeadTileN);
        for (int i = 0; i <= p.pieces; ++i) {
            g.jobs = 0;
            int64_t tiles = 0;
            if (i < p.pieces) {
                const int v0 = i * p.piece, width = (int)std::min<int64_t>(p.piece, vocab - v0);
                g.job[g.jobs++] = HeadJob{HEAD_PROB, i & 1, v0, width, 1, 0};
                tiles += m_tiles * ceil_div(width, kHeadTileN);
            }
            if (i > 0) {
                const int v0 = (i - 1) * p.piece, width = (int)std::min<int64_t>(p.piece, vocab - v0);
                g.job[g.jobs++] = HeadJob{HEAD_DH, (i - 1) & 1, v0, width, p.splits, i > 1};
                g.job[g.jobs++] = HeadJob{HEAD_DW, (i - 1) & 1, v0, width, 1, 0};
                tiles += m_tiles * d_tiles * p.splits + ceil_div(width, kHeadTileM) * d_tiles;
            }
            if (int rc = head_gemm(g, (int)std::min<int64_t>(tiles, INT32_MAX), "head_grad", c.st)) return rc;
        }
        if (tokens > 0) {
            const int threads = (int)std::min<int64_t>(256, round_up(ceil_div(dim, 8), 32));
            const int grid = (int)std::min<int64_t>(tokens, num_sms() * 16);
            const bool vec = dim % 8 == 0 && aligned16(dh);
            auto *k = vec ? &head_dh_kernel<true> : &head_dh_kernel<false>;
            cudaError_t e = cudaSuccess;
            SPCO_LAUNCH("head_dh", c.st,
                        e = launch_dependent(k, dim3(grid), dim3(threads), 0, c.st,
                                             Span<const float>(dh_sums, (int64_t)p.splits * p.row_cap * p.dh_ld),
                                             p.splits, p.row_cap, p.dh_ld, reinterpret_cast<const int *>(c.ws + p.off_at),
                                             g.state, grad_scale, (int)tokens, dim,
                                             Span<bf16>(static_cast<bf16 *>(dh), tokens * dim)));
            SPECOPTIM_CUDA(e);
        }
        return SPECOPTIM_OK;
    });
}
