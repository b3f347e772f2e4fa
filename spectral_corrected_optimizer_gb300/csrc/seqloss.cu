// Losses over the log-probabilities of packed sequences (include/finetune.h): paired
// preferences, and the clipped policy ratio with a KL term; both with their gradient.
//
// A unit of work is a pair, or a sequence.  A cluster of 1 to 8 CTAs takes a unit:
// it sums over the unit's tokens, the CTAs exchange their sums through distributed
// shared memory, and each writes the gradient of its tokens.  So a unit's tokens
// are read once from memory (the second reading, of the mask alone or of what
// the sums needed, comes from L1 or L2), nothing waits on another cluster, and few
// long sequences still use many SMs.  Each cluster leaves one partial of the loss;
// a last launch of one block adds the partials in their order.
//
// A thread works on 4 neighbouring tokens at a time, cut at multiples of 4 of the
// arrays: 16-byte loads wherever a sequence begins.
//
// Scores are differences of sums of thousands of terms, so the sums are kept in
// two floats (value and what its roundings lost): 2^-44 instead of 2^-24 of the
// largest partial sum.  The ratio's clipping is decided on logp - old_logp in two
// floats against log(1 + clip_high) and log(1 - clip_low) in two floats: at the
// bound the gradient jumps, and a rounding of the ratio would move tokens over it.
#include <algorithm>
#include <cmath>
#include <string>

#include "../../include/finetune.h"
#include "rowvec.cuh"
#include "tc_pair.cuh"

namespace spco {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kTile = 4096;       // tokens of a unit where there are no sequences
constexpr int kBlocksPerSm = 8;

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

// exp(x) - 1 and exp(x) - 1 - x.  Below 1 by the series of the latter, whose next term is below 2^-24 of the
// first one; neither loses digits then, nor costs what expm1f does.
struct Exp {
    float above, rest;
};
__device__ __forceinline__ Exp exp_of(float x) {
    float p = 1.f / 3628800.f;
    p = fmaf(p, x, 1.f / 362880.f);
    p = fmaf(p, x, 1.f / 40320.f);
    p = fmaf(p, x, 1.f / 5040.f);
    p = fmaf(p, x, 1.f / 720.f);
    p = fmaf(p, x, 1.f / 120.f);
    p = fmaf(p, x, 1.f / 24.f);
    p = fmaf(p, x, 1.f / 6.f);
    p = fmaf(p, x, 0.5f);
    Exp e;
    e.rest = p * x * x;
    e.above = x + e.rest;
    if (!(fabsf(x) < 1.f)) {
        e.above = expm1f(x);
        e.rest = e.above - x;
    }
    return e;
}

// ---- the tokens ----------------------------------------------------------------------------

struct Sequences {
    const void *offsets;  // null: units of kTile tokens
    int wide;             // 8-byte offsets
    int count, tokens;
    const uint8_t *mask;
    unsigned *flag;

    __device__ __forceinline__ int64_t raw(int i) const {
        return wide ? static_cast<const int64_t *>(offsets)[i] : (int64_t)static_cast<const int32_t *>(offsets)[i];
    }
    // where sequence i begins, within the tokens
    __device__ __forceinline__ int begin(int i) const {
        if (!offsets) return (int)min((int64_t)i * kTile, (int64_t)tokens);
        return (int)min(max(raw(i), (int64_t)0), (int64_t)tokens);
    }
    // whether the offsets i .. i + n keep the rule
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
    const int64_t t = (int64_t)piece * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < tokens) v.x = x[t];
    if (t + 1 < tokens) v.y = x[t + 1];
    if (t + 2 < tokens) v.z = x[t + 2];
    if (t + 3 < tokens) v.w = x[t + 3];
    return v;
}
// Those of the piece's tokens that lie in [a, b) and count: a byte each that is not 0.
template <bool VEC> __device__ __forceinline__ unsigned counting(const uint8_t *mask, int piece, int a, int b, int tokens) {
    const int64_t t = (int64_t)piece * 4;
    const int lo = (int)max(a - t, (int64_t)0), hi = (int)min(b - t, (int64_t)4);  // 0 .. 4, the piece touches [a, b)
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
    const int64_t t = (int64_t)piece * 4;
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

// zeros for the tokens in front of the first sequence and behind the last one
__device__ __forceinline__ void zero_outside(const Sequences &q, int sequences, float *dlogp) {
    if (!q.offsets) return;
    const int a = q.begin(0), b = max(a, q.begin(sequences));
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
    for (int64_t t = at; t < a; t += step) dlogp[t] = 0.f;
    for (int64_t t = b + at; t < q.tokens; t += step) dlogp[t] = 0.f;
}

__device__ __forceinline__ float load_peer(const float *p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ int load_peer(const int *p, uint32_t rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, rank)) : "memory");
    return v;
}
// every thread of the cluster's CTAs
__device__ __forceinline__ void sync_ctas() {
    __syncwarp();
    cluster_sync();
}

// How the CTAs of a launch share the units: `ctas` of a cluster take one together; or, few units (alone), the
// launch is one cluster, each CTA has units of its own and the CTAs join their losses at the end.
struct Share {
    int ctas, alone;
};

// ---- preference ----------------------------------------------------------------------------

struct Preference {
    Sequences q;
    const float *logp, *ref;
    float *dlogp, *pair_loss, *rewards, *partial, *loss;
    Share share;
    int pairs;
    int kind, average;
    float beta, smoothing, weight, loss_weight;  // weight: grad_scale / pairs or grad_scale
};

// What a CTA, or a warp, has of a sequence.
struct Score {
    Two sum;
    int count;
};

// Half of the CTA's warps have the chosen sequence, half the other one.
template <bool VEC> __global__ void __launch_bounds__(kThreads, 5) preference_kernel(const Preference a) {
    constexpr int HALF = kThreads / 2, U = 2;
    __shared__ Score warps_of[2][kWarps], own[2][2];
    __shared__ float slope_of[2][2], joined;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, side = threadIdx.x / HALF;
    const bool split = a.share.ctas > 1;
    const int rank = split ? (int)cluster_rank() : 0;
    const int cluster = blockIdx.x / a.share.ctas, clusters = gridDim.x / a.share.ctas;
    const int at = rank * HALF + threadIdx.x % HALF, step = a.share.ctas * HALF;
    grid_dependency_launch();
    zero_outside(a.q, 2 * a.pairs, a.dlogp);
    float loss = 0.f;  // thread 0 of rank 0
    int parity = 0;
    for (int p = cluster; p < a.pairs; p += clusters, parity ^= 1) {
        const int a0 = a.q.begin(2 * p), a1 = max(a0, a.q.begin(2 * p + 1)), a2 = max(a1, a.q.begin(2 * p + 2));
        if (rank == 0 && threadIdx.x == 0) a.q.check(2 * p, 2);
        const int from = side ? a1 : a0, to = side ? a2 : a1;
        const Pieces pieces(from, to);
        Score v{};
        for (int p0 = pieces.first + at; p0 < pieces.last; p0 += step * U) {
            float4 x[U], r[U];
            unsigned m[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int piece = p0 + u * step;
                m[u] = 0;
                if (piece >= pieces.last) continue;
                m[u] = counting<VEC>(a.q.mask, piece, from, to, a.q.tokens);
                x[u] = load4<VEC>(a.logp, piece, a.q.tokens);
                r[u] = a.ref ? load4<VEC>(a.ref, piece, a.q.tokens) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!m[u]) continue;
                const float d0 = counts(m[u], 0) ? x[u].x - r[u].x : 0.f, d1 = counts(m[u], 1) ? x[u].y - r[u].y : 0.f;
                const float d2 = counts(m[u], 2) ? x[u].z - r[u].z : 0.f, d3 = counts(m[u], 3) ? x[u].w - r[u].w : 0.f;
                Two t = two_sum(d0, d1);
                add(t, two_sum(d2, d3));
                add(v.sum, t);
                if (a.average) v.count += nonzero_bytes(m[u]);
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) add(v.sum, shuffled(v.sum, o));
        if (a.average) v.count = warp_add(v.count);
        if (lane == 0) warps_of[parity][warp] = v;
        __syncthreads();
        if (warp == 0) {
            // lanes 0 and 4 end with the two sequences' sums
            v = warps_of[parity][lane % kWarps];
#pragma unroll
            for (int o = kWarps / 4; o >= 1; o >>= 1) {
                add(v.sum, shuffled(v.sum, o));
                v.count += __shfl_xor_sync(0xffffffffu, v.count, o);
            }
            if (split && (lane == 0 || lane == kWarps / 2)) own[parity][lane != 0] = v;
        }
        if (split) {
            sync_ctas();  // the other CTAs' sums are there
            if (warp == 0) {
                v = Score{};
                if (lane == 0 || lane == kWarps / 2)
                    for (int c = 0; c < a.share.ctas; ++c) {
                        const Score &o = own[parity][lane != 0];
                        add(v.sum, Two{load_peer(&o.sum.hi, c), load_peer(&o.sum.lo, c)});
                        v.count += load_peer(&o.count, c);
                    }
            }
        }
        if (warp == 0) {
            v.sum = finished(v.sum);
            const Score second{{__shfl_sync(0xffffffffu, v.sum.hi, kWarps / 2), __shfl_sync(0xffffffffu, v.sum.lo, kWarps / 2)},
                               __shfl_sync(0xffffffffu, v.count, kWarps / 2)};
            if (lane == 0) {
                const double number0 = (double)max(v.count, 1), number1 = (double)max(second.count, 1);
                double r0 = (double)a.beta * ((double)v.sum.hi + (double)v.sum.lo);
                double r1 = (double)a.beta * ((double)second.sum.hi + (double)second.sum.lo);
                if (a.average) {
                    r0 /= number0;
                    r1 /= number1;
                }
                const double delta = r0 - r1;
                const float d = (float)delta;
                float l, slope;
                if (a.kind == PREFERENCE_LOGISTIC) {
                    const float soft = log1pf(expf(-fabsf(d))), up = 1.f / (1.f + expf(-d)), down = 1.f / (1.f + expf(d));
                    l = (1.f - a.smoothing) * (soft + fmaxf(-d, 0.f));
                    if (a.smoothing > 0.f) l += a.smoothing * (soft + fmaxf(d, 0.f));
                    if (d != d) l = d;  // fmaxf drops it
                    slope = a.smoothing * up - (1.f - a.smoothing) * down;
                } else if (a.kind == PREFERENCE_HINGE) {
                    const float gap = (float)(1. - delta);
                    l = gap <= 0.f ? 0.f : gap;  // NaN stays
                    slope = gap <= 0.f ? 0.f : gap == gap ? -1.f : gap;
                } else {
                    const float gap = (float)((delta - 0.5) / (double)a.beta);
                    l = gap * gap;
                    slope = 2.f * gap / a.beta;
                }
                slope *= a.beta * a.weight;
                slope_of[parity][0] = a.average ? slope / (float)max(v.count, 1) : slope;
                slope_of[parity][1] = a.average ? -slope / (float)max(second.count, 1) : -slope;
                if (rank == 0) {
                    a.pair_loss[p] = l;
                    a.rewards[2 * p] = (float)r0;
                    a.rewards[2 * p + 1] = (float)r1;
                    loss += l;
                }
            }
        }
        __syncthreads();
        const float g = slope_of[parity][side];
#pragma unroll 4
        for (int piece = pieces.first + at; piece < pieces.last; piece += step) {
            const unsigned m = counting<VEC>(a.q.mask, piece, from, to, a.q.tokens);
            store4<VEC>(a.dlogp, piece, from, to, make_float4(counts(m, 0) ? g : 0.f, counts(m, 1) ? g : 0.f, counts(m, 2) ? g : 0.f,
                                                              counts(m, 3) ? g : 0.f));
        }
    }
    if (a.share.alone) {
        if (threadIdx.x == 0) joined = loss;
        sync_ctas();
        if (cluster == 0 && threadIdx.x == 0) {
            loss = 0.f;
            for (int c = 0; c < clusters; ++c) loss += load_peer(&joined, c);
            *a.loss = loss * a.loss_weight;
        }
    } else if (rank == 0 && threadIdx.x == 0) {
        reinterpret_cast<float4 *>(a.partial)[cluster] = make_float4(loss, 0.f, 0.f, 0.f);
    }
    if (split || a.share.alone) sync_ctas();  // no CTA leaves while its sums are read
}

// ---- policy --------------------------------------------------------------------------------

struct Policy {
    Sequences q;
    const float *logp, *old, *ref, *advantages;
    float *dlogp, *partial, *parts, *loss;
    const int *counted;      // valid tokens by block of the counting launch; null: none was made
    int counting_blocks;
    Share share;
    int units;
    int per_sequence, reduction, count_here;
    float kl_coef, grad_scale, edge_high, edge_low;  // edges: the bounds' distance from 1
    Two log_high, log_low;   // log(1 + clip_high), log(1 - clip_low)
};

// sum over the block, to all threads
__device__ __forceinline__ int block_add(int v, int *red) {
    v = warp_add(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w];
    return v;
}

// Tokens that count in all sequences together, by block.
__global__ void __launch_bounds__(kThreads) policy_count_kernel(const Sequences q, int *__restrict__ counted) {
    __shared__ int red[kWarps];
    grid_dependency_launch();
    const int a = q.offsets ? q.begin(0) : 0, b = q.offsets ? max(a, q.begin(q.count)) : q.tokens;
    const int n = block_add(count_tokens(q.mask, a, b, (int64_t)blockIdx.x * kThreads + threadIdx.x,
                                         (int64_t)gridDim.x * kThreads), red);
    if (threadIdx.x == 0) counted[blockIdx.x] = n;
}

template <bool VEC> __global__ void __launch_bounds__(kThreads, 4) policy_kernel(const Policy a) {
    constexpr int U = 2;
    __shared__ int red[kWarps], own[2];
    __shared__ float sums_of[kWarps][3], joined[3];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool split = a.share.ctas > 1;
    const int rank = split ? (int)cluster_rank() : 0;
    const int cluster = blockIdx.x / a.share.ctas, clusters = gridDim.x / a.share.ctas;
    const int at = rank * kThreads + threadIdx.x, step = a.share.ctas * kThreads;
    grid_dependency_wait();
    grid_dependency_launch();
    zero_outside(a.q, a.q.count, a.dlogp);
    float weight = 1.f;  // of a token
    if (a.reduction == POLICY_TOKEN_MEAN) {
        const int b0 = a.q.offsets ? a.q.begin(0) : 0, b1 = a.q.offsets ? max(b0, a.q.begin(a.q.count)) : a.q.tokens;
        int n = b1 - b0;
        if (a.counted) {
            n = 0;
            for (int i = threadIdx.x; i < a.counting_blocks; i += kThreads) n += a.counted[i];
            n = block_add(n, red);
        } else if (a.count_here) {
            n = block_add(count_tokens(a.q.mask, b0, b1, threadIdx.x, kThreads), red);
        }
        weight = 1.f / (float)max(n, 1);
    }
    float total[3] = {0.f, 0.f, 0.f};
    int parity = 0;
    for (int u = cluster; u < a.units; u += clusters, parity ^= 1) {
        const int b0 = a.q.begin(u), b1 = max(b0, a.q.begin(u + 1));
        if (rank == 0 && threadIdx.x == 0) a.q.check(u, 1);
        if (a.reduction == POLICY_SEQUENCE_MEAN) {
            int n = b1 - b0;
            if (a.q.mask) {
                n = block_add(count_tokens(a.q.mask, b0, b1, at, step), red);
                if (split) {
                    if (threadIdx.x == 0) own[parity] = n;
                    sync_ctas();
                    n = 0;
                    for (int k = 0; k < a.share.ctas; ++k) n += load_peer(&own[parity], k);
                }
            }
            weight = 1.f / ((float)max(n, 1) * (float)a.q.count);
        }
        const float scaled = weight * a.grad_scale, one = a.per_sequence ? a.advantages[u] : 0.f;
        float sum[3] = {0.f, 0.f, 0.f};
        const Pieces pieces(b0, b1);
        for (int p0 = pieces.first + at; p0 < pieces.last; p0 += step * U) {
            float4 x[U], o[U], r[U], w[U];
            unsigned m[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int piece = p0 + k * step;
                m[k] = 0;
                if (piece >= pieces.last) continue;
                m[k] = counting<VEC>(a.q.mask, piece, b0, b1, a.q.tokens);
                x[k] = load4<VEC>(a.logp, piece, a.q.tokens);
                o[k] = load4<VEC>(a.old, piece, a.q.tokens);
                if (a.ref) r[k] = load4<VEC>(a.ref, piece, a.q.tokens);
                w[k] = a.per_sequence ? make_float4(one, one, one, one) : load4<VEC>(a.advantages, piece, a.q.tokens);
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int piece = p0 + k * step;
                if (piece >= pieces.last) continue;
                float g[4] = {0.f, 0.f, 0.f, 0.f};
                if (m[k]) {
                    const float lp[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, lo[4] = {o[k].x, o[k].y, o[k].z, o[k].w};
                    const float lr[4] = {r[k].x, r[k].y, r[k].z, r[k].w}, ad[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool here = counts(m[k], i), gains = ad[i] >= 0.f;
                        const Two d = finished(two_sum(lp[i], -lo[i]));
                        const float past = (d.hi - (gains ? a.log_high.hi : a.log_low.hi)) + (d.lo - (gains ? a.log_high.lo : a.log_low.lo));
                        const bool clipped = gains ? past > 0.f : past < 0.f;
                        // A r as A + A (r - 1): the sum over many tokens whose advantages cancel has no
                        // bias from the last place of the exponential
                        const float above = clipped ? (gains ? a.edge_high : a.edge_low) : exp_of(d.hi).above;
                        const float gain = fmaf(ad[i], above, ad[i]);
                        float slope = clipped ? 0.f : -gain, kl = 0.f;
                        if (a.ref) {
                            const Exp e = exp_of(lr[i] - lp[i]);
                            kl = e.rest;
                            slope = fmaf(-a.kl_coef, e.above, slope);
                        }
                        g[i] = here ? slope * scaled : 0.f;
                        sum[0] -= here ? gain : 0.f;
                        sum[1] += here ? kl : 0.f;
                        sum[2] += here && clipped ? 1.f : 0.f;
                    }
                }
                store4<VEC>(a.dlogp, piece, b0, b1, make_float4(g[0], g[1], g[2], g[3]));
            }
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) total[i] = fmaf(weight, sum[i], total[i]);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        total[i] = warp_add(total[i]);
        if (lane == 0) sums_of[warp][i] = total[i];
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        float s = 0.f;
        for (int w = 0; w < kWarps; ++w) s += sums_of[w][threadIdx.x];
        if (a.share.alone) joined[threadIdx.x] = s;
        else a.partial[(int64_t)blockIdx.x * 4 + threadIdx.x] = s;
    }
    if (a.share.alone) {
        sync_ctas();
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            float s[3] = {0.f, 0.f, 0.f};
            for (int i = 0; i < 3; ++i) {
                for (int c = 0; c < (int)gridDim.x; ++c) s[i] += load_peer(&joined[i], c);
                a.parts[i] = s[i];
            }
            *a.loss = a.kl_coef != 0.f ? fmaf(a.kl_coef, s[1], s[0]) : s[0];
        }
    }
    if (split || a.share.alone) sync_ctas();  // no CTA leaves while its sums are read
}

// parts[k] = weight * sum of partial[0 .. blocks)[k], loss = parts[0] + kl_coef parts[1]; in fp64, joined in a fixed order
constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads) loss_join_kernel(const float *partial, int blocks, float weight, float kl_coef,
                                                                 float *parts, float *loss) {
    __shared__ double red[kJoinThreads / 32][3];
    grid_dependency_wait();
    double v[3] = {0., 0., 0.};
#pragma unroll 4
    for (int i = threadIdx.x; i < blocks; i += kJoinThreads) {
        const float4 x = reinterpret_cast<const float4 *>(partial)[i];
        v[0] += (double)x.x;
        v[1] += (double)x.y;
        v[2] += (double)x.z;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        v[k] = warp_add(v[k]);
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5][k] = v[k];
    }
    __syncthreads();
    if (threadIdx.x >= 32) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] = warp_add(threadIdx.x < kJoinThreads / 32 ? red[threadIdx.x][k] : 0.) * (double)weight;
    if (threadIdx.x) return;
    if (parts) {
        parts[0] = (float)v[0];
        parts[1] = (float)v[1];
        parts[2] = (float)v[2];
    }
    *loss = (float)(kl_coef != 0.f ? v[0] + (double)kl_coef * v[1] : v[0]);
}

// ---- launches ------------------------------------------------------------------------------

// CTAs for a unit: as many as the SMs have room for beside the other units', while each still has some
// 1024 tokens (a unit may be a few times longer than the average).  Few units of few tokens: one cluster, which
// needs no launch to join its losses.
Share share_of(int units, int64_t tokens) {
    if (units <= kMaxCluster && tokens <= (int64_t)units * kThreads * 8) return {1, 1};
    int c = 1;
    while (c < kMaxCluster && units * c * 2 <= 2 * num_sms() && tokens / std::max(units, 1) > (int64_t)c * kThreads * 4) c *= 2;
    return {c, 0};
}
int blocks_of(int units, const Share &s) {
    if (s.alone) return units <= 1 ? 1 : units <= 2 ? 2 : units <= 4 ? 4 : kMaxCluster;
    return s.ctas * std::max(1, std::min(units, num_sms() * kBlocksPerSm / s.ctas));
}
// blocks that count tokens, and from how many tokens on (below, every block counts all of them)
constexpr int64_t kCountHere = 32768;
int counting_blocks(int64_t tokens) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(num_sms() * 2, ceil_div(tokens, kThreads * 32)));
}

template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), int blocks, const Share &share, bool dependent, cudaStream_t st, A &&...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = share.alone ? blocks : share.ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

constexpr int64_t kMost = (int64_t)1 << 30;  // sequences and tokens, so that indexes fit 32 bits

int check_common(int64_t count, int64_t tokens, const void *logp, const void *offsets, int32_t offset_bytes, bool need_offsets,
                 const float *loss, const float *dlogp, const void *workspace, const std::string &what) {
    if (count < 0 || count > kMost) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": sequences outside [0, 2^30]");
    if (tokens < 0 || tokens > kMost) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": tokens outside [0, 2^30]");
    if (offset_bytes != 4 && offset_bytes != 8) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": offset_bytes must be 4 or 8");
    if (!loss || !workspace || (need_offsets && !offsets) || (tokens > 0 && (!logp || !dlogp)))
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

int64_t workspace_of() { return (int64_t)num_sms() * (kBlocksPerSm * 16 + 2 * 4); }

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
        bytes = workspace_of();
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
        if (int rc = bind_device()) return rc;
        if (workspace_bytes < workspace_of())
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": the workspace is smaller than preference_loss_workspace() says");
        const Share share = share_of((int)pairs, tokens);
        const int blocks = blocks_of((int)pairs, share);
        const float part = mean ? 1.f / (float)std::max<int64_t>(pairs, 1) : 1.f;
        const Preference a{{offsets, offset_bytes == 8, (int)(2 * pairs), (int)tokens, mask, stage_flag_ptr()},
                           logp, ref_logp, dlogp, pair_loss, rewards, static_cast<float *>(workspace), loss, share, (int)pairs,
                           kind, average != 0, beta, smoothing, grad_scale * part, part};
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        auto *k = all_aligned16({logp, ref_logp, dlogp}, mask) ? &preference_kernel<true> : &preference_kernel<false>;
        cudaError_t e = cudaSuccess;
        SPCO_LAUNCH("preference_loss", st, e = launch_clusters(k, blocks, share, false, st, a));
        SPECOPTIM_CUDA(e);
        if (share.alone) return SPECOPTIM_OK;
        SPCO_LAUNCH("loss_join", st,
                    e = launch_dependent(loss_join_kernel, dim3(1), dim3(kJoinThreads), 0, st, a.partial, blocks / share.ctas, part,
                                         0.f, static_cast<float *>(nullptr), loss));
        SPECOPTIM_CUDA(e);
        return SPECOPTIM_OK;
    });
}

extern "C" int64_t policy_loss_workspace(int64_t sequences, int64_t tokens) {
    int64_t bytes = -1;
    entry([&]() -> int {
        if (sequences < 0 || sequences > kMost || tokens < 0 || tokens > kMost)
            return fail(SPECOPTIM_ERR_INVALID_ARG, "policy_loss: sequences or tokens outside [0, 2^30]");
        bytes = workspace_of();
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
        if (int rc = bind_device()) return rc;
        if (workspace_bytes < workspace_of())
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": the workspace is smaller than policy_loss_workspace() says");
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        if (!offsets && reduction == POLICY_SEQUENCE_MEAN) reduction = POLICY_TOKEN_MEAN;
        const int units = (int)(offsets ? sequences : ceil_div(tokens, kTile));
        const Share share = offsets || units <= kMaxCluster ? share_of(units, tokens) : Share{1, 0};
        const int blocks = blocks_of(units, share);
        const bool vec = all_aligned16({logp, old_logp, ref_logp, dlogp, per_sequence ? nullptr : advantages}, mask);
        const Sequences q{offsets, offset_bytes == 8, (int)sequences, (int)tokens, mask, stage_flag_ptr()};
        float *partial = static_cast<float *>(workspace);
        int *counted = reinterpret_cast<int *>(partial + (int64_t)num_sms() * kBlocksPerSm * 4);
        const bool counting = mask && reduction == POLICY_TOKEN_MEAN, apart = counting && tokens > kCountHere;
        cudaError_t e = cudaSuccess;
        if (apart) {
            SPCO_LAUNCH("policy_count", st, policy_count_kernel<<<counting_blocks(tokens), kThreads, 0, st>>>(q, counted));
            SPECOPTIM_LAUNCHED("policy_count_kernel");
        }
        const Policy a{q, logp, old_logp, ref_logp, advantages, dlogp, partial, parts, loss, apart ? counted : nullptr,
                       counting_blocks(tokens), share, units, per_sequence != 0, reduction, counting && !apart, kl_coef,
                       grad_scale, (float)clip_high, (float)-clip_low, log_two(1. + clip_high), log_two(1. - clip_low)};
        auto *k = vec ? &policy_kernel<true> : &policy_kernel<false>;
        SPCO_LAUNCH("policy_loss", st, e = launch_clusters(k, blocks, share, apart, st, a));
        SPECOPTIM_CUDA(e);
        if (share.alone) return SPECOPTIM_OK;
        SPCO_LAUNCH("loss_join", st,
                    e = launch_dependent(loss_join_kernel, dim3(1), dim3(kJoinThreads), 0, st, partial, blocks, 1.f, kl_coef, parts,
                                         loss));
        SPECOPTIM_CUDA(e);
        return SPECOPTIM_OK;
    });
}
