// Losses over the log-probabilities of packed sequences (include/finetune.h): paired
// preferences, and the clipped policy ratio with a KL term; both with their gradient.
//
// What a launch is cut by depends on how many sequences there are and how long:
//   few short ones     one cluster of up to 8 CTAs, each with sequences of its own, which joins
//                      the loss through distributed shared memory: one launch
//   many short pairs   a block takes a pair: it sums over both sequences, half of its warps for
//                      each, and writes their gradient
//   long pairs         2^n slices of a pair, some 1024 tokens each: a launch sums over the
//                      slices, the next joins them and writes the gradient
//   many sequences     the policy's tokens need of one another only a count and an advantage,
//   (policy loss)      so its tiles of 512 tokens lie wherever memory is cut; a launch in front
//                      counts the mask and tells each tile the sequence that it begins in
// A last launch of one block joins the losses, in their order.
//
// A thread works on 4 neighbouring tokens at a time, cut at multiples of 4 of the
// arrays: 16-byte loads wherever a sequence begins.
//
// Scores are differences of sums of thousands of terms, so the sums are kept in
// two floats (value and what its roundings lost): 2^-44 instead of 2^-24 of the
// largest partial sum.  The ratio's clipping is decided on logp - old_logp in two
// floats against log(1 + clip_high) and log(1 - clip_low) in two floats: at the
// bound the gradient jumps, and a rounding of the ratio would move tokens over it.
//
// Measured on a GB300, in a CUDA graph, inputs out of L2 (copy bandwidth 6.78 TB/s):
//   1024 pairs of 2 x 2048 tokens on average, prompts masked: 26 us (floor 8.1): slices 16 us, of
//     which the 38 MB that they read are 6, and the fill 9; a block's chain of offsets, loads,
//     sums and a barrier is what takes the time (warps wait 12 of 27 cycles for loads, 6 at
//     barriers).  By a block for each pair, whatever its length: 34; by clusters: 28.
//   2048 rollouts of 2048 tokens, KL term, one advantage each: 30 us (floor 10.5), 13.3 million
//     instructions, issue slots 47 % busy; by a block for each sequence 47.
//   64 pairs of 2 x 8192 9.6 us, 2048 pairs of 2 x 100 8.5, one pair of 45 tokens 3.4;
//   64 rollouts of 4096 tokens 8.8, 7 of 331 5.3.
// fp64 sums of the losses alone had cost 5 us: a warp's addition takes 15 cycles here.
// At the blocks an SM that their bounds ask for, the slices spill 16 bytes a thread (44 where the
// arrays are not aligned) and the tiles 20 (4).
#include <algorithm>
#include <cmath>
#include <string>

#include "../../include/finetune.h"
#include "f32x2.cuh"
#include "rowvec.cuh"
#include "tc_pair.cuh"

namespace spco {
namespace {

constexpr int kFewThreads = 128, kManyThreads = 512;  // of a block
constexpr int kMaxCluster = 8;
constexpr int kTile = 512, kTileThreads = 128;  // tokens of a tile: 4 per thread
constexpr int kTileBlocks = 7;                  // an SM holds at once
constexpr int kUnit = 1024;                     // tokens of a unit where there are no sequences
constexpr int kMaxBlocksPerSm = 64;  // of a launch: the hardware hands blocks out as others end, which evens out long units

// ---- two floats ----------------------------------------------------------------------------

struct Two {
    float hi, lo;
};
// a + b and what the rounding lost (nothing that can be used where the sum is not finite)
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ void add(Two &a, const Two &b) {
    const Two t = two_sum(a.hi, b.hi);
    a.hi = t.hi;
    a.lo += t.lo + b.lo;
}
__device__ __forceinline__ Two finished(const Two &a) { return {a.hi, fabsf(a.hi) < INFINITY ? a.lo : 0.f}; }
__device__ __forceinline__ Two shuffled(const Two &a, int o) {
    return {__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
}
template <typename V> __device__ __forceinline__ V warp_add(V v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ Two times(const Two &a, float b) {
    const float p = a.hi * b;
    return {p, fmaf(a.lo, b, fmaf(a.hi, b, -p))};
}
__device__ __forceinline__ Two divided(const Two &a, float b) {
    const float q = a.hi / b;
    return {q, (fmaf(-q, b, a.hi) + a.lo) / b};
}
__device__ __forceinline__ float value(const Two &a) { return fabsf(a.hi) < INFINITY ? a.hi + a.lo : a.hi; }

// the same for two sums at once
struct Two2 {
    F2 hi, lo;
};
__device__ __forceinline__ Two2 two_sum(F2 a, F2 b) {
    const F2 s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}

// exp(x) - 1 - x for |x| < 1, by its series, whose next term is below 2^-24 of the first one: neither this nor
// x + this loses digits, and both cost less than expm1f does.
__device__ __forceinline__ float exp_rest(float x) {
    float p = 1.f / 3628800.f;
    p = fmaf(p, x, 1.f / 362880.f);
    p = fmaf(p, x, 1.f / 40320.f);
    p = fmaf(p, x, 1.f / 5040.f);
    p = fmaf(p, x, 1.f / 720.f);
    p = fmaf(p, x, 1.f / 120.f);
    p = fmaf(p, x, 1.f / 24.f);
    p = fmaf(p, x, 1.f / 6.f);
    p = fmaf(p, x, 0.5f);
    return p * x * x;
}
// exp(x) - 1 and exp(x) of any x, out of line: they are rare, and their copies would crowd the instruction cache
__device__ __noinline__ float exp_above(float x) { return expm1f(x); }
__device__ __noinline__ float exp_below(float x) { return expf(x); }

// ---- the tokens ----------------------------------------------------------------------------

struct Sequences {
    const void *offsets;  // null: units of kUnit tokens each
    int wide;             // 8-byte offsets
    int count, tokens;
    const uint8_t *mask;
    unsigned *flag;

    __device__ __forceinline__ int64_t raw(int i) const {
        return wide ? static_cast<const int64_t *>(offsets)[i] : (int64_t)static_cast<const int32_t *>(offsets)[i];
    }
    // where sequence i begins, within the tokens
    __device__ __forceinline__ int begin(int i) const {
        if (!offsets) return (int)min((int64_t)i * kUnit, (int64_t)tokens);
        return (int)min((uint64_t)raw(i), (uint64_t)tokens);
    }
    // whether the offsets i .. i + n keep the rule; without sequences it is the only one's to lie within the tokens
    __device__ __forceinline__ void check(int i, int n) const {
        if (!offsets) return;
        bool good = raw(i) >= 0 && raw(i + n) <= tokens;
        for (int k = 0; k < n; ++k) good = good && raw(i + k) <= raw(i + k + 1);
        if (!good) atomicExch(flag, kSiteOffset);
    }
};

// Pieces of 4 tokens that [a, b) touches, cut at multiples of 4 of the arrays: [first, last).
struct Pieces {
    int first, last;
    __device__ __forceinline__ Pieces(int a, int b) : first(a / 4), last(a < b ? (b - 1) / 4 + 1 : a / 4) {}
};

// x[t .. t + 3], t = 4 piece; 0 behind the end
template <bool VEC> __device__ __forceinline__ float4 load4(const float *x, int piece, int tokens) {
    if (VEC && piece < tokens / 4) return reinterpret_cast<const float4 *>(x)[piece];
    const int t = piece * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < tokens) v.x = x[t];
    if (t + 1 < tokens) v.y = x[t + 1];
    if (t + 2 < tokens) v.z = x[t + 2];
    if (t + 3 < tokens) v.w = x[t + 3];
    return v;
}
// Those of the piece's tokens that lie in [a, b) and count: a byte each that is not 0.
template <bool VEC> __device__ __forceinline__ unsigned counting(const uint8_t *mask, int piece, int a, int b, int tokens) {
    const int t = piece * 4;
    const int lo = max(a - t, 0), hi = min(b - t, 4);  // 0 .. 4, the piece touches [a, b)
    const unsigned in = (0xffffffffu << (8 * lo)) & (0xffffffffu >> (8 * (4 - hi)));
    if (!mask) return in;
    if (VEC && piece < tokens / 4) return in & reinterpret_cast<const unsigned *>(mask)[piece];
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i >= lo && i < hi) m |= (unsigned)mask[t + i] << (8 * i);
    return m;
}
__device__ __forceinline__ bool counts(unsigned m, int i) { return (m & (0xffu << (8 * i))) != 0; }

// v to those of the piece's tokens that lie in [a, b)
template <bool VEC> __device__ __forceinline__ void store4(float *x, int piece, int a, int b, float4 v) {
    const int t = piece * 4;
    if (VEC && t >= a && t + 4 <= b) {
        reinterpret_cast<float4 *>(x)[piece] = v;
        return;
    }
    if (t >= a && t < b) x[t] = v.x;
    if (t + 1 >= a && t + 1 < b) x[t + 1] = v.y;
    if (t + 2 >= a && t + 2 < b) x[t + 2] = v.z;
    if (t + 3 >= a && t + 3 < b) x[t + 3] = v.w;
}

__device__ __forceinline__ int nonzero_bytes(unsigned w) {
    return __popc((((w & 0x7f7f7f7fu) + 0x7f7f7f7fu) | w) & 0x80808080u);
}
// tokens that count in [a, b), this thread's share: 16 at a time where the mask allows it
__device__ __forceinline__ int count_tokens(const uint8_t *mask, int a, int b, int64_t at, int64_t step) {
    const uintptr_t from = reinterpret_cast<uintptr_t>(mask + a), to = reinterpret_cast<uintptr_t>(mask + b);
    const uintptr_t v0 = (from + 15) & ~uintptr_t(15), v1 = to & ~uintptr_t(15);
    int n = 0;
    if (v0 >= v1) {
        for (int64_t t = a + at; t < b; t += step) n += mask[t] != 0;
        return n;
    }
    const int64_t vecs = (int64_t)(v1 - v0) / 16;
    const uint4 *v = reinterpret_cast<const uint4 *>(v0);
#pragma unroll 4
    for (int64_t i = at; i < vecs; i += step) {
        const uint4 m = v[i];
        n += (nonzero_bytes(m.x) + nonzero_bytes(m.y)) + (nonzero_bytes(m.z) + nonzero_bytes(m.w));
    }
    const int head = (int)(v0 - from), tail = (int)(to - v1);  // at most 15 each
    if (at < head) n += mask[a + at] != 0;
    if (at < tail) n += mask[b - 1 - at] != 0;
    return n;
}

// zeros for the tokens in front of the first sequence and behind the last one, by the launch's first blocks
template <int THREADS> __device__ __forceinline__ void zero_outside(const Sequences &q, int sequences, float *dlogp) {
    constexpr int kBlocks = 64;
    if (!q.offsets || blockIdx.x >= kBlocks) return;
    const int a = q.begin(0), b = max(a, q.begin(sequences));
    if (sequences == 0 && blockIdx.x == 0 && threadIdx.x == 0) q.check(0, 0);
    const int64_t at = (int64_t)blockIdx.x * THREADS + threadIdx.x, step = (int64_t)min((int)gridDim.x, kBlocks) * THREADS;
    for (int64_t t = at; t < a; t += step) dlogp[t] = 0.f;
    for (int64_t t = b + at; t < q.tokens; t += step) dlogp[t] = 0.f;
}

__device__ __forceinline__ float load_peer(const float *p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(p, rank)) : "memory");
    return v;
}
// every thread of the cluster's CTAs
__device__ __forceinline__ void sync_ctas() {
    __syncwarp();
    cluster_sync();
}

// x - a, rounded once
__device__ __forceinline__ float below(float x, const Two &a) {
    Two t = two_sum(x, -a.hi);
    t.lo -= a.lo;
    return value(t);
}

// ---- preference ----------------------------------------------------------------------------

struct Preference {
    Sequences q;
    const float *logp, *ref;
    float *dlogp, *pair_loss, *rewards, *loss;
    float4 *scores;  // [pairs][slices][2]: hi, lo and count of a slice
    int pairs, slice_bits;  // 2^slice_bits slices of a pair
    int alone;       // the launch is one cluster, which forms the loss too
    int kind, average;
    float beta, smoothing, weight, loss_weight;  // weight: grad_scale / pairs or grad_scale
};

// What a thread, a warp or a block has of a sequence.
struct Score {
    Two sum;
    int count;
};

// A sequence of a pair, and the pieces of it that a block has to do with.
struct Part {
    int from, to, first, last;
};
__device__ __forceinline__ Part part_of(const Preference &a, int p, int side, int slice) {
    const int a0 = a.q.begin(2 * p), a1 = max(a0, a.q.begin(2 * p + 1)), a2 = max(a1, a.q.begin(2 * p + 2));
    const int from = side ? a1 : a0, to = side ? a2 : a1;
    const Pieces pieces(from, to);
    const int64_t n = pieces.last - pieces.first;
    return {from, to, pieces.first + (int)(n * slice >> a.slice_bits), pieces.first + (int)(n * (slice + 1) >> a.slice_bits)};
}

template <bool VEC> __device__ __forceinline__ Score score_of(const Preference &a, const Part &part, int at, int step) {
    constexpr int U = 2;
    F2 sum = pair(0.f, 0.f), lost = sum;
    int count = 0;
    for (int p0 = part.first + at; p0 < part.last; p0 += step * U) {
        float4 x[U], r[U];
        unsigned m[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int piece = p0 + u * step;
            m[u] = 0;
            if (piece >= part.last) continue;
            m[u] = counting<VEC>(a.q.mask, piece, part.from, part.to, a.q.tokens);
            x[u] = load4<VEC>(a.logp, piece, a.q.tokens);
            r[u] = a.ref ? load4<VEC>(a.ref, piece, a.q.tokens) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!m[u]) continue;
            const float d0 = counts(m[u], 0) ? x[u].x - r[u].x : 0.f, d1 = counts(m[u], 1) ? x[u].y - r[u].y : 0.f;
            const float d2 = counts(m[u], 2) ? x[u].z - r[u].z : 0.f, d3 = counts(m[u], 3) ? x[u].w - r[u].w : 0.f;
            const Two2 once = two_sum(sum, pair(d0, d1)), twice = two_sum(once.hi, pair(d2, d3));
            sum = twice.hi;
            lost = lost + (once.lo + twice.lo);
            if (a.average) count += nonzero_bytes(m[u]);
        }
    }
    const float2 hi = both(sum), lo = both(lost);
    Score v{{hi.x, lo.x}, count};
    add(v.sum, Two{hi.y, lo.y});
    return v;
}
// Sums over lanes that differ in the bits below `lanes`.
__device__ __forceinline__ void lanes_add(Score &v, int lanes) {
    for (int o = lanes / 2; o >= 1; o >>= 1) {
        add(v.sum, shuffled(v.sum, o));
        v.count += __shfl_xor_sync(0xffffffffu, v.count, o);
    }
}
// The block's sums, the first half of its warps having one sequence and the second half the other: to warp 0's
// lanes 0 and WARPS / 2.  One barrier.
template <int WARPS> __device__ __forceinline__ void block_scores(Score &v, Score *warps_of) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    lanes_add(v, 32);
    if (lane == 0) warps_of[warp] = v;
    __syncthreads();
    if (warp) return;
    v = warps_of[lane % WARPS];
    lanes_add(v, WARPS / 2);
}

struct Outcome {
    Two reward[2], delta;
    float slope[2];  // of the loss by each sequence's tokens
};
__device__ __forceinline__ Outcome outcome_of(const Preference &a, const Score &chosen, const Score &other) {
    Outcome o;
    o.reward[0] = times(finished(chosen.sum), a.beta);
    o.reward[1] = times(finished(other.sum), a.beta);
    if (a.average) {
        o.reward[0] = divided(o.reward[0], (float)max(chosen.count, 1));
        o.reward[1] = divided(o.reward[1], (float)max(other.count, 1));
    }
    o.delta = o.reward[0];
    add(o.delta, Two{-o.reward[1].hi, -o.reward[1].lo});
    const float d = value(o.delta);
    float slope;
    if (a.kind == PREFERENCE_LOGISTIC) {
        const float up = 1.f / (1.f + expf(-d)), down = 1.f / (1.f + expf(d));
        slope = a.smoothing * up - (1.f - a.smoothing) * down;
    } else if (a.kind == PREFERENCE_HINGE) {
        const float gap = below(1.f, o.delta);
        slope = gap <= 0.f ? 0.f : gap == gap ? -1.f : gap;  // NaN stays
    } else {
        slope = -2.f * (below(0.5f, o.delta) / a.beta) / a.beta;
    }
    slope *= a.beta * a.weight;
    o.slope[0] = a.average ? slope / (float)max(chosen.count, 1) : slope;
    o.slope[1] = a.average ? -slope / (float)max(other.count, 1) : -slope;
    return o;
}
// Writes what is known of a pair; its loss.
__device__ __forceinline__ float report(const Preference &a, int p, const Outcome &o) {
    const float d = value(o.delta);
    float l;
    if (a.kind == PREFERENCE_LOGISTIC) {
        const float soft = log1pf(expf(-fabsf(d)));
        l = (1.f - a.smoothing) * (soft + fmaxf(-d, 0.f));
        if (a.smoothing > 0.f) l += a.smoothing * (soft + fmaxf(d, 0.f));
    } else if (a.kind == PREFERENCE_HINGE) {
        const float gap = below(1.f, o.delta);
        l = gap <= 0.f ? 0.f : gap;
    } else {
        const float gap = below(0.5f, o.delta) / a.beta;
        l = gap * gap;
    }
    a.pair_loss[p] = l;
    a.rewards[2 * p] = value(o.reward[0]);
    a.rewards[2 * p + 1] = value(o.reward[1]);
    a.q.check(2 * p, 2);
    return l;
}

template <bool VEC> __device__ __forceinline__ void fill(const Preference &a, const Part &part, float g, int at, int step) {
#pragma unroll 4
    for (int piece = part.first + at; piece < part.last; piece += step) {
        const unsigned m = counting<VEC>(a.q.mask, piece, part.from, part.to, a.q.tokens);
        store4<VEC>(a.dlogp, piece, part.from, part.to, make_float4(counts(m, 0) ? g : 0.f, counts(m, 1) ? g : 0.f,
                                                                    counts(m, 2) ? g : 0.f, counts(m, 3) ? g : 0.f));
    }
}

// Short sequences: a block sums over a pair and writes its gradient.
template <int THREADS, bool VEC> __global__ void __launch_bounds__(THREADS, 1024 / THREADS) preference_kernel(const Preference a) {
    constexpr int HALF = THREADS / 2, WARPS = THREADS / 32;
    __shared__ Score warps_of[2][WARPS];
    __shared__ float slope_of[2][2], joined;
    const int side = threadIdx.x / HALF, at = threadIdx.x % HALF;
    grid_dependency_launch();
    zero_outside<THREADS>(a.q, 2 * a.pairs, a.dlogp);
    float loss = 0.f;  // thread 0
    int parity = 0;
    for (int p = blockIdx.x; p < a.pairs; p += gridDim.x, parity ^= 1) {
        const Part part = part_of(a, p, side, 0);
        Score v = score_of<VEC>(a, part, at, HALF);
        block_scores<WARPS>(v, warps_of[parity]);
        Outcome o;
        if (threadIdx.x < 32) {
            const Score other{{__shfl_sync(0xffffffffu, v.sum.hi, WARPS / 2), __shfl_sync(0xffffffffu, v.sum.lo, WARPS / 2)},
                              __shfl_sync(0xffffffffu, v.count, WARPS / 2)};
            if (threadIdx.x == 0) {
                o = outcome_of(a, v, other);
                slope_of[parity][0] = o.slope[0];
                slope_of[parity][1] = o.slope[1];
            }
        }
        __syncthreads();
        fill<VEC>(a, part, slope_of[parity][side], at, HALF);
        if (threadIdx.x == 0) loss += report(a, p, o);
    }
    if (!a.alone) return;
    if (threadIdx.x == 0) joined = loss;
    sync_ctas();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        loss = 0.f;
        for (int c = 0; c < (int)gridDim.x; ++c) loss += load_peer(&joined, c);
        *a.loss = loss * a.loss_weight;
    }
    sync_ctas();  // no CTA leaves while its loss is read
}

// Long sequences are cut into slices, so that the longest one does not end last: a launch sums over the slices, the
// next one joins a pair's slices in their order, in every block that has one of them to fill.
// More blocks an SM with fewer loads each: 1024 pairs of 2 x 2048 tokens take 26 us, 31 with 8 blocks and twice the loads;
// a warp for each slice and no barriers 28.
constexpr int kSliceThreads = 128, kSliceBlocks = 12;
template <bool VEC> __global__ void __launch_bounds__(kSliceThreads, kSliceBlocks) preference_slices_kernel(const Preference a) {
    constexpr int HALF = kSliceThreads / 2, WARPS = kSliceThreads / 32;
    __shared__ Score warps_of[WARPS];
    const int p = blockIdx.x >> a.slice_bits, slice = blockIdx.x & ((1 << a.slice_bits) - 1);
    grid_dependency_launch();
    Score v = score_of<VEC>(a, part_of(a, p, threadIdx.x / HALF, slice), threadIdx.x % HALF, HALF);
    block_scores<WARPS>(v, warps_of);
    if (threadIdx.x == 0 || threadIdx.x == WARPS / 2)
        a.scores[(int64_t)blockIdx.x * 2 + (threadIdx.x != 0)] = make_float4(v.sum.hi, v.sum.lo, __int_as_float(v.count), 0.f);
}
template <bool VEC> __global__ void __launch_bounds__(kSliceThreads, kSliceBlocks) preference_fill_kernel(const Preference a) {
    constexpr int HALF = kSliceThreads / 2;
    __shared__ float slope_of[2];
    const int slices = 1 << a.slice_bits, p = blockIdx.x >> a.slice_bits, slice = blockIdx.x & (slices - 1), side = threadIdx.x / HALF;
    const Part part = part_of(a, p, side, slice);
    grid_dependency_wait();
    grid_dependency_launch();
    zero_outside<kSliceThreads>(a.q, 2 * a.pairs, a.dlogp);
    Outcome o;
    if (threadIdx.x < 32) {  // 16 lanes for each sequence
        Score v{};
        for (int c = threadIdx.x & 15; c < slices; c += 16) {
            const float4 x = a.scores[((int64_t)p * slices + c) * 2 + (threadIdx.x >> 4)];
            add(v.sum, Two{x.x, x.y});
            v.count += __float_as_int(x.z);
        }
        lanes_add(v, 16);
        const Score other{{__shfl_sync(0xffffffffu, v.sum.hi, 16), __shfl_sync(0xffffffffu, v.sum.lo, 16)},
                          __shfl_sync(0xffffffffu, v.count, 16)};
        if (threadIdx.x == 0) {
            o = outcome_of(a, v, other);
            slope_of[0] = o.slope[0];
            slope_of[1] = o.slope[1];
        }
    }
    __syncthreads();
    fill<VEC>(a, part, slope_of[side], threadIdx.x % HALF, HALF);
    if (threadIdx.x == 0 && slice == 0) report(a, p, o);
}

// ---- policy --------------------------------------------------------------------------------

struct Policy {
    Sequences q;
    const float *logp, *old, *ref, *advantages;
    float *dlogp, *partial, *parts, *loss;
    // by the preparing launch, where there is one: tokens that count by block; of the sequence that each tile begins in
    // its number, its end, its advantage and the weight of its tokens; that weight of each sequence
    int *counted;
    int4 *first_of;
    float *weight_of;
    int counting_blocks, tiles;
    int per_sequence, reduction;
    float kl_coef, grad_scale, edge_high, edge_low;  // edges: the bounds' distance from 1
    Two log_high, log_low;   // log(1 + clip_high), log(1 - clip_low)
};

// sum over the block, to all threads
template <int WARPS> __device__ __forceinline__ int block_add(int v, int *red) {
    v = warp_add(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v += red[w];
    return v;
}

// A piece's inputs.
struct Tokens {
    float4 logp, old, ref, advantage;
};
template <bool VEC> __device__ __forceinline__ Tokens load_tokens(const Policy &a, int piece, float one) {
    Tokens t;
    t.logp = load4<VEC>(a.logp, piece, a.q.tokens);
    t.old = load4<VEC>(a.old, piece, a.q.tokens);
    t.ref = a.ref ? load4<VEC>(a.ref, piece, a.q.tokens) : t.logp;
    t.advantage = a.per_sequence ? make_float4(one, one, one, one) : load4<VEC>(a.advantages, piece, a.q.tokens);
    return t;
}

// Weighted sums over a thread's tokens: gains, divergences, clipped ones.
struct Seen {
    float gain, kl, clipped;
};

// How far logp - old lies above the bound that a gain of that sign takes.
__device__ __forceinline__ float beyond(const Policy &a, bool up, const Two &d) {
    return (d.hi - (up ? a.log_high.hi : a.log_low.hi)) + (d.lo - (up ? a.log_high.lo : a.log_low.lo));
}

// A piece's gradient, and what its tokens add to the sums; m says which of them count.
__device__ __forceinline__ float4 four_tokens(const Policy &a, unsigned m, const Tokens &t, float4 weight, Seen &seen) {
    if (!m) return make_float4(0.f, 0.f, 0.f, 0.f);
    const float lp[4] = {t.logp.x, t.logp.y, t.logp.z, t.logp.w}, old[4] = {t.old.x, t.old.y, t.old.z, t.old.w};
    const float ref[4] = {t.ref.x, t.ref.y, t.ref.z, t.ref.w}, w[4] = {weight.x, weight.y, weight.z, weight.w};
    float adv[4] = {t.advantage.x, t.advantage.y, t.advantage.z, t.advantage.w};
    Two d[4];
    float q[4], ratio[4], kl[4], dkl[4], g[4];  // ratio: its distance from 1
    bool near = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        d[i] = two_sum(lp[i], -old[i]);
        ratio[i] = d[i].hi + exp_rest(d[i].hi);
        near = near && fabsf(d[i].hi) < 1.f;
        if (a.ref) {
            q[i] = ref[i] - lp[i];
            kl[i] = exp_rest(q[i]);
            dkl[i] = q[i] + kl[i];
            near = near && fabsf(q[i]) < 1.f;
        }
    }
    if (!near) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!(fabsf(d[i].hi) < 1.f)) {
                d[i] = finished(d[i]);
                // A + A (r - 1) would round what is left of A to A's last place: A r goes on as an advantage whose
                // ratio is 1.  Its sign is A's, and where it vanishes neither bound is near
                if (d[i].hi <= -1.f && (adv[i] >= 0.f || !(beyond(a, false, d[i]) < 0.f))) {
                    adv[i] *= exp_below(d[i].hi);
                    ratio[i] = 0.f;
                } else {
                    // 0 times a ratio that overflows would be NaN
                    ratio[i] = adv[i] == 0.f && d[i].hi >= 1.f ? 0.f : exp_above(d[i].hi);
                }
            }
            if (a.ref && !(fabsf(q[i]) < 1.f)) {
                dkl[i] = exp_above(q[i]);
                kl[i] = dkl[i] - q[i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool here = counts(m, i), up = adv[i] >= 0.f;
        const float past = beyond(a, up, d[i]);
        const bool clipped = up ? past > 0.f : past < 0.f;
        // A r as A + A (r - 1): the sum over many tokens whose advantages cancel has no bias from the last place
        // of the exponential
        const float gain = fmaf(adv[i], clipped ? (up ? a.edge_high : a.edge_low) : ratio[i], adv[i]);
        float slope = clipped ? 0.f : -gain;
        // without a coefficient the divergence is only watched: 0 times one that overflows would be NaN
        if (a.kl_coef != 0.f) slope = fmaf(-a.kl_coef, dkl[i], slope);
        g[i] = here ? slope * w[i] * a.grad_scale : 0.f;
        const float wh = here ? w[i] : 0.f;
        seen.gain = fmaf(here ? gain : 0.f, w[i], seen.gain);
        if (a.ref) seen.kl = fmaf(here ? kl[i] : 0.f, w[i], seen.kl);
        seen.clipped += clipped ? wh : 0.f;
    }
    return make_float4(g[0], g[1], g[2], g[3]);
}
// The block's sums, to threads 0 .. 2: -gain, kl, clipped.
template <int WARPS> __device__ __forceinline__ float block_sums(const Seen &seen, float (*red)[3]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float v[3] = {warp_add(-seen.gain), warp_add(seen.kl), warp_add(seen.clipped)};
    if (lane == 0)
        for (int i = 0; i < 3; ++i) red[warp][i] = v[i];
    __syncthreads();
    float s = 0.f;
    if (threadIdx.x < 3)
        for (int w = 0; w < WARPS; ++w) s += red[w][threadIdx.x];
    return s;
}

// Few sequences: one cluster, each CTA takes sequences of its own, and the CTAs join their losses at the end.
template <int THREADS, bool VEC> __global__ void __launch_bounds__(THREADS, 1) policy_few_kernel(const Policy a) {
    constexpr int U = 2, WARPS = THREADS / 32;
    __shared__ int red[WARPS];
    __shared__ float sums_of[WARPS][3], joined[3];
    zero_outside<THREADS>(a.q, a.q.count, a.dlogp);
    float weight = 1.f;  // of a token
    if (a.reduction == POLICY_TOKEN_MEAN) {
        const int b0 = a.q.offsets ? a.q.begin(0) : 0, b1 = a.q.offsets ? max(b0, a.q.begin(a.q.count)) : a.q.tokens;
        const int n = a.q.mask ? block_add<WARPS>(count_tokens(a.q.mask, b0, b1, threadIdx.x, THREADS), red) : b1 - b0;
        weight = 1.f / (float)max(n, 1);
    }
    Seen seen{0.f, 0.f, 0.f};
    const int units = a.q.offsets ? a.q.count : (a.q.tokens + kUnit - 1) / kUnit;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const int b0 = a.q.begin(u), b1 = max(b0, a.q.begin(u + 1));
        if (a.reduction == POLICY_SEQUENCE_MEAN) {
            const int n = a.q.mask ? block_add<WARPS>(count_tokens(a.q.mask, b0, b1, threadIdx.x, THREADS), red) : b1 - b0;
            weight = 1.f / ((float)max(n, 1) * (float)a.q.count);
        }
        const float one = a.per_sequence ? a.advantages[u] : 0.f;
        const Pieces pieces(b0, b1);
        for (int p0 = pieces.first + (int)threadIdx.x; p0 < pieces.last; p0 += THREADS * U) {
            Tokens t[U];
            unsigned m[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (p0 + k * THREADS >= pieces.last) continue;
                m[k] = counting<VEC>(a.q.mask, p0 + k * THREADS, b0, b1, a.q.tokens);
                t[k] = load_tokens<VEC>(a, p0 + k * THREADS, one);
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (p0 + k * THREADS >= pieces.last) continue;
                const float4 g = four_tokens(a, m[k], t[k], make_float4(weight, weight, weight, weight), seen);
                store4<VEC>(a.dlogp, p0 + k * THREADS, b0, b1, g);
            }
        }
        if (threadIdx.x == 0) a.q.check(u, 1);
    }
    const float s = block_sums<WARPS>(seen, sums_of);
    if (threadIdx.x < 3) joined[threadIdx.x] = s;
    sync_ctas();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        float v[3] = {0.f, 0.f, 0.f};
        for (int i = 0; i < 3; ++i) {
            for (int c = 0; c < (int)gridDim.x; ++c) v[i] += load_peer(&joined[i], c);
            a.parts[i] = v[i];
        }
        *a.loss = a.kl_coef != 0.f ? fmaf(a.kl_coef, v[1], v[0]) : v[0];
    }
    sync_ctas();  // no CTA leaves while its sums are read
}

// Many sequences: tiles of kTile tokens, wherever sequences begin, so that no block has more to do than another.
// This launch goes before: the first counting_blocks blocks count the tokens of all sequences, the others
// tell each tile the sequence that it begins in and each sequence its tokens' weight.
constexpr int kPrepareThreads = 128;
__global__ void __launch_bounds__(kPrepareThreads) policy_prepare_kernel(const Policy a) {
    __shared__ int red[kPrepareThreads / 32];
    grid_dependency_launch();
    if ((int)blockIdx.x < a.counting_blocks) {
        const int from = a.q.offsets ? a.q.begin(0) : 0, to = a.q.offsets ? max(from, a.q.begin(a.q.count)) : a.q.tokens;
        const int n = block_add<kPrepareThreads / 32>(
            count_tokens(a.q.mask, from, to, (int64_t)blockIdx.x * kPrepareThreads + threadIdx.x,
                         (int64_t)a.counting_blocks * kPrepareThreads), red);
        if (threadIdx.x == 0) a.counted[blockIdx.x] = n;
        return;
    }
    const int first = blockIdx.x - a.counting_blocks, blocks = gridDim.x - a.counting_blocks;
    for (int s = first; s < a.q.count; s += blocks) {
        const int from = a.q.begin(s), to = max(from, a.q.begin(s + 1));
        // tiles that begin in the sequence, in front of the first or behind the last one
        const int t0 = s == 0 ? 0 : (from + kTile - 1) / kTile;
        const int t1 = s == a.q.count - 1 ? a.tiles : (to + kTile - 1) / kTile;
        float weight = 0.f;
        if (a.reduction == POLICY_SEQUENCE_MEAN) {
            const int n = a.q.mask ? block_add<kPrepareThreads / 32>(count_tokens(a.q.mask, from, to, threadIdx.x, kPrepareThreads), red)
                                   : to - from;
            weight = 1.f / ((float)max(n, 1) * (float)a.q.count);
            if (threadIdx.x == 0) a.weight_of[s] = weight;
        }
        const int4 what = make_int4(s, to, __float_as_int(a.per_sequence ? a.advantages[s] : 0.f), __float_as_int(weight));
        for (int t = t0 + (int)threadIdx.x; t < t1; t += kPrepareThreads) a.first_of[t] = what;
        if (threadIdx.x == 0) a.q.check(s, 1);
    }
}

template <bool VEC> __global__ void __launch_bounds__(kTileThreads, kTileBlocks) policy_tiles_kernel(const Policy a) {
    static_assert(kTile == 4 * kTileThreads, "a piece per thread");
    __shared__ float sums_of[kTileThreads / 32][3];
    const int lane = threadIdx.x & 31;
    const bool lookup = a.per_sequence || a.reduction == POLICY_SEQUENCE_MEAN;
    grid_dependency_wait();
    grid_dependency_launch();
    int b0 = 0, b1 = a.q.tokens;
    if (a.q.offsets) {
        b0 = a.q.begin(0);
        b1 = max(b0, a.q.begin(a.q.count));
        if (a.q.count == 0 && blockIdx.x == 0 && threadIdx.x == 0) a.q.check(0, 0);
        if (!lookup && !a.counting_blocks)  // else the launch in front did
            for (int64_t s = (int64_t)blockIdx.x * kTileThreads + threadIdx.x; s < a.q.count; s += (int64_t)gridDim.x * kTileThreads)
                a.q.check((int)s, 1);
    }
    float same = 1.f;
    if (a.reduction == POLICY_TOKEN_MEAN) {
        int n = 0;
#pragma unroll 4
        for (int i = lane; i < a.counting_blocks; i += 32) n += a.counted[i];
        n = a.counting_blocks ? warp_add(n) : b1 - b0;
        same = 1.f / (float)max(n, 1);
    }
    Seen seen{0.f, 0.f, 0.f};
    // the next tile's values are on their way while one is worked on
    struct Next {
        Tokens t;
        unsigned m;
        int4 first;
    };
    auto fetch = [&](int tile) {
        Next n;
        n.m = 0;
        if (tile >= a.tiles) return n;
        const int piece = tile * kTileThreads + (int)threadIdx.x, at = piece * 4;
        if (at < b1 && at + 4 > b0) {
            n.m = counting<VEC>(a.q.mask, piece, b0, b1, a.q.tokens);
            n.t = load_tokens<VEC>(a, piece, 0.f);
        }
        if (lookup) n.first = a.first_of[tile];
        return n;
    };
    Next next = fetch(blockIdx.x);
    for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        Next now = next;
        next = fetch(tile + gridDim.x);
        const int piece = tile * kTileThreads + (int)threadIdx.x, at = piece * 4;
        float4 weight = make_float4(same, same, same, same);
        if (lookup) {
            float w = a.reduction == POLICY_SEQUENCE_MEAN ? __int_as_float(now.first.w) : same, v = __int_as_float(now.first.z);
            float ws[4] = {w, w, w, w}, vs[4] = {v, v, v, v};
            if (now.m && at + 4 > now.first.y) {
                // the piece lies in a later sequence or goes on in one: the last that begins at or in front of it, within
                // bounds whatever the offsets were
                const int most = a.q.count - 1, s1 = tile + 1 < a.tiles ? min(max(a.first_of[tile + 1].x, 0), most) : most;
                int s = min(max(now.first.x, 0), s1), hi = s1;
                while (s < hi) {
                    const int mid = (s + hi + 1) / 2;
                    if (a.q.begin(mid) <= at) s = mid;
                    else hi = mid - 1;
                }
                int end = at;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (at + i >= end) {
                        if (i) ++s;
                        for (end = s < s1 ? a.q.begin(s + 1) : b1; s < s1 && at + i >= end; end = s < s1 ? a.q.begin(s + 1) : b1) ++s;
                        if (a.reduction == POLICY_SEQUENCE_MEAN) w = a.weight_of[s];
                        if (a.per_sequence) v = a.advantages[s];
                        if (s == s1) end = INT32_MAX;
                    }
                    ws[i] = w;
                    vs[i] = v;
                }
            }
            weight = make_float4(ws[0], ws[1], ws[2], ws[3]);
            if (a.per_sequence) now.t.advantage = make_float4(vs[0], vs[1], vs[2], vs[3]);
        }
        if (at < a.q.tokens) store4<VEC>(a.dlogp, piece, 0, a.q.tokens, four_tokens(a, now.m, now.t, weight, seen));
    }
    const float sum = block_sums<kTileThreads / 32>(seen, sums_of);
    if (threadIdx.x < 3) a.partial[(int64_t)blockIdx.x * 4 + threadIdx.x] = sum;
}

// parts[k] = weight * sum of from[0 .. count)[k], loss = parts[0] + kl_coef parts[1], in two floats (a warp's addition
// in fp64 takes 15 cycles here) and a fixed order.  KINDS values of each of `count`: 1, or 3 of 4.
constexpr int kJoinThreads = 1024;
template <int KINDS> __global__ void __launch_bounds__(kJoinThreads) loss_join_kernel(const float *from, int count, float weight,
                                                                                      float kl_coef, float *parts, float *loss) {
    __shared__ Two red[KINDS][kJoinThreads / 32];
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Two v[KINDS] = {};
#pragma unroll 4
    for (int i = threadIdx.x; i < count; i += kJoinThreads) {
        if (KINDS == 1) {
            add(v[0], Two{from[i], 0.f});
        } else {
            const float4 x = reinterpret_cast<const float4 *>(from)[i];
            add(v[0], Two{x.x, 0.f});
            add(v[KINDS > 1 ? 1 : 0], Two{x.y, 0.f});
            add(v[KINDS > 2 ? 2 : 0], Two{x.z, 0.f});
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
        for (int k = 0; k < KINDS; ++k) add(v[k], shuffled(v[k], o));
    if (lane == 0)
        for (int k = 0; k < KINDS; ++k) red[k][warp] = v[k];
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int k = 0; k < KINDS; ++k) v[k] = red[k][lane];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
        for (int k = 0; k < KINDS; ++k) add(v[k], shuffled(v[k], o));
    if (lane) return;
    for (int k = 0; k < KINDS; ++k) v[k] = times(finished(v[k]), weight);
    if (KINDS == 3) {
        for (int k = 0; k < KINDS; ++k) parts[k] = value(v[k]);
        if (kl_coef != 0.f) add(v[0], times(v[KINDS > 1 ? 1 : 0], kl_coef));
    }
    *loss = value(v[0]);
}

// ---- launches ------------------------------------------------------------------------------

// Few units of few tokens: one cluster, which needs no launch to join its losses.
bool alone(int units, int64_t tokens) { return units <= kMaxCluster && tokens <= (int64_t)std::max(units, 1) * 2048; }
int cluster_of(int units) { return units <= 1 ? 1 : units <= 2 ? 2 : units <= 4 ? 4 : kMaxCluster; }

// Slices of a pair, as a power of two: some 1024 tokens of an average one.  0: a block takes a pair.
int slice_bits_of(int64_t pairs, int64_t tokens) {
    if (pairs == 0 || alone((int)pairs, tokens)) return 0;
    int bits = 0;
    while (bits < 6 && tokens / pairs > (1024 << bits) && pairs << bits < 1 << 15) ++bits;
    return bits;
}

template <typename... P, typename... A>
cudaError_t launch_cluster(void (*kernel)(P...), int blocks, int threads, cudaStream_t st, A &&...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = blocks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

constexpr int64_t kMost = (int64_t)1 << 30;  // sequences and tokens, so that indexes fit 32 bits

int check_common(int64_t count, int64_t tokens, const void *logp, const void *offsets, int32_t offset_bytes, bool need_offsets,
                 const float *loss, const float *dlogp, const void *workspace, const std::string &what) {
    if (count < 0 || count > kMost) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": sequences outside [0, 2^30]");
    if (tokens < 0 || tokens > kMost) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": tokens outside [0, 2^30]");
    if (offset_bytes != 4 && offset_bytes != 8) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": offset_bytes must be 4 or 8");
    if (!loss || (need_offsets && !offsets) || (tokens > 0 && (!logp || !dlogp)))
        return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": null pointer");
    if (!aligned_to(logp, 4) || !aligned_to(offsets, offset_bytes) || !aligned_to(loss, 4) || !aligned_to(dlogp, 4) ||
        !aligned16(workspace))
        return fail(SPECOPTIM_ERR_MISALIGNED, what + ": pointers must be aligned to their elements, the workspace to 16 bytes");
    return SPECOPTIM_OK;
}

bool all_aligned16(std::initializer_list<const void *> p, const void *mask) {
    for (const void *x : p)
        if (!aligned16(x)) return false;
    return aligned_to(mask, 4);
}

// scores of the slices; none where a block has a pair
int64_t preference_bytes(int64_t pairs, int64_t tokens) {
    const int bits = slice_bits_of(pairs, tokens);
    return bits ? (pairs << bits) * 2 * 16 : 0;
}
// partial sums of the blocks
int64_t partial_bytes() { return (int64_t)num_sms() * kTileBlocks * 16; }
// and of the policy loss: counts, each tile's first sequence, each sequence's weight
constexpr int kMostCounts = 512;
int64_t policy_bytes(bool by_offsets, int64_t sequences, int64_t tokens) {
    if (alone((int)(by_offsets ? sequences : ceil_div(tokens, kUnit)), tokens)) return 0;
    return partial_bytes() + 16 * ceil_div(tokens, kTile) + 4 * (kMostCounts + sequences);
}

// log(x) in two floats
Two log_two(double x) {
    const double l = std::log(x);
    const float hi = (float)l;
    return {hi, std::isfinite(l) ? (float)(l - (double)hi) : 0.f};
}

}  // namespace
}  // namespace spco

using namespace spco;

extern "C" int64_t preference_loss_workspace(int64_t pairs, int64_t tokens) {
    int64_t bytes = -1;
    entry([&]() -> int {
        if (pairs < 0 || pairs > kMost / 2 || tokens < 0 || tokens > kMost)
            return fail(SPECOPTIM_ERR_INVALID_ARG, "preference_loss: pairs outside [0, 2^29] or tokens outside [0, 2^30]");
        bytes = preference_bytes(pairs, tokens);
        return SPECOPTIM_OK;
    });
    return bytes;
}

extern "C" int preference_loss(const float *logp, const float *ref_logp, const uint8_t *mask, const void *offsets,
                               int32_t offset_bytes, int64_t pairs, int64_t tokens, int32_t kind, float beta,
                               float smoothing, int32_t average, int32_t mean, float grad_scale, float *loss,
                               float *pair_loss, float *rewards, float *dlogp, void *workspace, int64_t workspace_bytes,
                               void *stream) {
    return entry([&]() -> int {
        const std::string what = "preference_loss";
        if (pairs < 0 || pairs > kMost / 2) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": pairs outside [0, 2^29]");
        if (int rc = check_common(2 * pairs, tokens, logp, offsets, offset_bytes, true, loss, dlogp, workspace, what)) return rc;
        if (kind != PREFERENCE_LOGISTIC && kind != PREFERENCE_HINGE && kind != PREFERENCE_SQUARE)
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": kind must be PREFERENCE_LOGISTIC, _HINGE or _SQUARE");
        if (!(beta > 0.f) || !std::isfinite(beta)) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": beta must be positive");
        if (!(smoothing >= 0.f && smoothing <= 0.5f) || (smoothing != 0.f && kind != PREFERENCE_LOGISTIC))
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": smoothing must lie in [0, 0.5], and be 0 but for the logistic loss");
        if (!std::isfinite(grad_scale)) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": grad_scale must be finite");
        if (pairs > 0 && (!pair_loss || !rewards)) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": null pointer");
        if (!aligned_to(ref_logp, 4) || !aligned_to(pair_loss, 4) || !aligned_to(rewards, 4))
            return fail(SPECOPTIM_ERR_MISALIGNED, what + ": pointers must be aligned to their elements");
        const int64_t need = preference_bytes(pairs, tokens);
        if (need && !workspace) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": null pointer");
        if (workspace_bytes < need)
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": the workspace is smaller than preference_loss_workspace() says");
        if (int rc = bind_device()) return rc;
        const float part = mean ? 1.f / (float)std::max<int64_t>(pairs, 1) : 1.f;
        const bool one = alone((int)pairs, tokens);
        const int bits = slice_bits_of(pairs, tokens);
        const Preference a{{offsets, offset_bytes == 8, (int)(2 * pairs), (int)tokens, mask, stage_flag_ptr()},
                           logp, ref_logp, dlogp, pair_loss, rewards, loss, static_cast<float4 *>(workspace), (int)pairs, bits,
                           one, kind, average != 0, beta, smoothing, grad_scale * part, part};
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        const bool vec = all_aligned16({logp, ref_logp, dlogp}, mask);
        cudaError_t e = cudaSuccess;
        if (one) {
            const bool many = tokens > pairs * 512;
            auto *k = many ? (vec ? &preference_kernel<kManyThreads, true> : &preference_kernel<kManyThreads, false>)
                           : (vec ? &preference_kernel<kFewThreads, true> : &preference_kernel<kFewThreads, false>);
            SPCO_LAUNCH("preference_loss", st,
                        e = launch_cluster(k, cluster_of((int)pairs), many ? kManyThreads : kFewThreads, st, a));
            SPECOPTIM_CUDA(e);
            return SPECOPTIM_OK;
        }
        if (bits == 0) {
            auto *k = vec ? &preference_kernel<kFewThreads, true> : &preference_kernel<kFewThreads, false>;
            const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>(pairs, num_sms() * kMaxBlocksPerSm));
            SPCO_LAUNCH("preference_loss", st, k<<<blocks, kFewThreads, 0, st>>>(a));
            SPECOPTIM_LAUNCHED("preference_kernel");
        } else {
            const unsigned blocks = (unsigned)(pairs << bits);
            auto *k = vec ? &preference_slices_kernel<true> : &preference_slices_kernel<false>;
            SPCO_LAUNCH("preference_slices", st, k<<<blocks, kSliceThreads, 0, st>>>(a));
            SPECOPTIM_LAUNCHED("preference_slices_kernel");
            auto *f = vec ? &preference_fill_kernel<true> : &preference_fill_kernel<false>;
            SPCO_LAUNCH("preference_loss", st, e = launch_dependent(f, dim3(blocks), dim3(kSliceThreads), 0, st, a));
            SPECOPTIM_CUDA(e);
        }
        SPCO_LAUNCH("loss_join", st,
                    e = launch_dependent(loss_join_kernel<1>, dim3(1), dim3(kJoinThreads), 0, st, pair_loss, (int)pairs, part, 0.f,
                                         static_cast<float *>(nullptr), loss));
        SPECOPTIM_CUDA(e);
        return SPECOPTIM_OK;
    });
}

extern "C" int64_t policy_loss_workspace(int64_t sequences, int64_t tokens) {
    int64_t bytes = -1;
    entry([&]() -> int {
        if (sequences < 0 || sequences > kMost || tokens < 0 || tokens > kMost)
            return fail(SPECOPTIM_ERR_INVALID_ARG, "policy_loss: sequences or tokens outside [0, 2^30]");
        // one sequence may stand for none
        bytes = std::max(policy_bytes(true, sequences, tokens), sequences == 1 ? policy_bytes(false, 1, tokens) : 0);
        return SPECOPTIM_OK;
    });
    return bytes;
}

extern "C" int policy_loss(const float *logp, const float *old_logp, const float *ref_logp, const uint8_t *mask,
                           const float *advantages, int32_t per_sequence, const void *offsets, int32_t offset_bytes,
                           int64_t sequences, int64_t tokens, double clip_low, double clip_high, float kl_coef,
                           int32_t reduction, float grad_scale, float *loss, float *parts, float *dlogp, void *workspace,
                           int64_t workspace_bytes, void *stream) {
    return entry([&]() -> int {
        const std::string what = "policy_loss";
        if (int rc = check_common(sequences, tokens, logp, offsets, offset_bytes, false, loss, dlogp, workspace, what)) return rc;
        if (reduction != POLICY_TOKEN_MEAN && reduction != POLICY_SEQUENCE_MEAN && reduction != POLICY_SUM)
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": reduction must be POLICY_TOKEN_MEAN, _SEQUENCE_MEAN or _SUM");
        if (!(clip_low >= 0. && clip_low <= 1.) || !(clip_high >= 0.))
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": clip_low must lie in [0, 1], clip_high be >= 0");
        if (!std::isfinite(kl_coef) || !std::isfinite(grad_scale))
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": kl_coef and grad_scale must be finite");
        if (kl_coef != 0.f && !ref_logp && tokens > 0)
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": kl_coef needs ref_logp");
        if (!offsets && (sequences != 1 || per_sequence))
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": without offsets sequences is 1 and advantages are the tokens'");
        if (!parts || (tokens > 0 && !old_logp) || ((per_sequence ? sequences : tokens) > 0 && !advantages))
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": null pointer");
        if (!aligned_to(old_logp, 4) || !aligned_to(ref_logp, 4) || !aligned_to(advantages, 4) || !aligned_to(parts, 4))
            return fail(SPECOPTIM_ERR_MISALIGNED, what + ": pointers must be aligned to their elements");
        const int64_t need = policy_bytes(offsets != nullptr, sequences, tokens);
        if (need && !workspace) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": null pointer");
        if (workspace_bytes < need)
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": the workspace is smaller than policy_loss_workspace() says");
        if (int rc = bind_device()) return rc;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        if (!offsets && reduction == POLICY_SEQUENCE_MEAN) reduction = POLICY_TOKEN_MEAN;
        const int tiles = (int)ceil_div(tokens, kTile), units = (int)(offsets ? sequences : ceil_div(tokens, kUnit));
        const bool vec = all_aligned16({logp, old_logp, ref_logp, dlogp, per_sequence ? nullptr : advantages}, mask);
        float *partial = static_cast<float *>(workspace);
        int4 *first_of = reinterpret_cast<int4 *>(static_cast<char *>(workspace) + partial_bytes());
        int *counted = reinterpret_cast<int *>(first_of + tiles);
        Policy a{{offsets, offset_bytes == 8, (int)sequences, (int)tokens, mask, stage_flag_ptr()},
                 logp, old_logp, ref_logp, advantages, dlogp, partial, parts, loss, counted, first_of,
                 reinterpret_cast<float *>(counted + kMostCounts), 0, tiles, per_sequence != 0, reduction, kl_coef,
                 grad_scale, (float)clip_high, (float)-clip_low, log_two(1. + clip_high), log_two(1. - clip_low)};
        cudaError_t e = cudaSuccess;
        if (alone(units, tokens)) {
            const bool many = tokens > (int64_t)units * 512;
            auto *k = many ? (vec ? &policy_few_kernel<kManyThreads, true> : &policy_few_kernel<kManyThreads, false>)
                           : (vec ? &policy_few_kernel<kFewThreads, true> : &policy_few_kernel<kFewThreads, false>);
            SPCO_LAUNCH("policy_loss", st, e = launch_cluster(k, cluster_of(units), many ? kManyThreads : kFewThreads, st, a));
            SPECOPTIM_CUDA(e);
            return SPECOPTIM_OK;
        }
        if (mask && reduction == POLICY_TOKEN_MEAN)
            a.counting_blocks = (int)std::max<int64_t>(1, std::min<int64_t>(kMostCounts, ceil_div(tokens, kPrepareThreads * 64)));
        // without sequences the tiles have nothing to look up
        const bool lookup = per_sequence || reduction == POLICY_SEQUENCE_MEAN;
        const int64_t by_sequence = lookup || (offsets && a.counting_blocks) ? std::min<int64_t>(sequences, num_sms() * 32) : 0;
        const bool prepared = a.counting_blocks + by_sequence > 0;
        if (prepared) {
            SPCO_LAUNCH("policy_prepare", st,
                        policy_prepare_kernel<<<(unsigned)(a.counting_blocks + by_sequence), kPrepareThreads, 0, st>>>(a));
            SPECOPTIM_LAUNCHED("policy_prepare_kernel");
        }
        const int blocks = std::max(1, std::min(tiles, num_sms() * kTileBlocks));
        auto *k = vec ? &policy_tiles_kernel<true> : &policy_tiles_kernel<false>;
        if (prepared) {
            SPCO_LAUNCH("policy_loss", st, e = launch_dependent(k, dim3(blocks), dim3(kTileThreads), 0, st, a));
            SPECOPTIM_CUDA(e);
        } else {
            SPCO_LAUNCH("policy_loss", st, k<<<blocks, kTileThreads, 0, st>>>(a));
            SPECOPTIM_LAUNCHED("policy_tiles_kernel");
        }
        SPCO_LAUNCH("loss_join", st,
                    e = launch_dependent(loss_join_kernel<3>, dim3(1), dim3(kJoinThreads), 0, st, partial, blocks, 1.f, kl_coef, parts,
                                         loss));
        SPECOPTIM_CUDA(e);
        return SPECOPTIM_OK;
    });
}
