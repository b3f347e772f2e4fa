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
#include "f32x2.cuh"
#include "rowvec.cuh"
#include "tc_pair.cuh"

namespace spco {
namespace {

constexpr int kFewThreads = 128, kMiddleThreads = 256, kManyThreads = 512;  // of a block
constexpr int kMaxCluster = 8;
constexpr int kTile = 1024, kTileThreads = 128;  // tokens of a tile (and of a unit where there are no sequences)
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

// exp(x) - 1 and exp(x) - 1 - x.  Below 1 by the series of the latter, whose next term is below 2^-24 of the
// first one; neither loses digits then, nor costs what expm1f does.
struct Exp {
    F2 above, rest;
};
__device__ __forceinline__ Exp exp_of(F2 x) {
    const auto both_of = [](float c) { return pair(c, c); };
    F2 p = both_of(1.f / 3628800.f);
    p = fma2(p, x, both_of(1.f / 362880.f));
    p = fma2(p, x, both_of(1.f / 40320.f));
    p = fma2(p, x, both_of(1.f / 5040.f));
    p = fma2(p, x, both_of(1.f / 720.f));
    p = fma2(p, x, both_of(1.f / 120.f));
    p = fma2(p, x, both_of(1.f / 24.f));
    p = fma2(p, x, both_of(1.f / 6.f));
    p = fma2(p, x, both_of(0.5f));
    Exp e;
    e.rest = p * x * x;
    e.above = x + e.rest;
    const float2 v = both(x);
    if (!(fabsf(v.x) < 1.f && fabsf(v.y) < 1.f)) {
        float2 above = both(e.above), rest = both(e.rest);
        if (!(fabsf(v.x) < 1.f)) {
            above.x = expm1f(v.x);
            rest.x = above.x - v.x;
        }
        if (!(fabsf(v.y) < 1.f)) {
            above.y = expm1f(v.y);
            rest.y = above.y - v.y;
        }
        e = {pair(above.x, above.y), pair(rest.x, rest.y)};
    }
    return e;
}

// ---- the tokens ----------------------------------------------------------------------------

struct Sequences {
    const void *offsets;  // null: units of kTile tokens each
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
    const int64_t at = (int64_t)blockIdx.x * THREADS + threadIdx.x, step = (int64_t)min((int)gridDim.x, kBlocks) * THREADS;
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
template <int THREADS, bool VEC> __global__ void __launch_bounds__(THREADS, 1024 / THREADS) preference_kernel(const Preference a) {
    constexpr int HALF = THREADS / 2, WARPS = THREADS / 32, U = 4;
    __shared__ Score warps_of[2][WARPS], own[2][2];
    __shared__ float slope_of[2][2], joined;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, side = threadIdx.x / HALF;
    const bool split = a.share.ctas > 1;
    const int rank = split ? (int)cluster_rank() : 0;
    const int cluster = blockIdx.x / a.share.ctas, clusters = gridDim.x / a.share.ctas;
    const int at = rank * HALF + threadIdx.x % HALF, step = a.share.ctas * HALF;
    grid_dependency_launch();
    zero_outside<THREADS>(a.q, 2 * a.pairs, a.dlogp);
    float loss = 0.f;  // thread 0 of rank 0
    Two r0{}, r1{}, delta{};  // thread 0: the pair's rewards and their difference
    int parity = 0;
    for (int p = cluster; p < a.pairs; p += clusters, parity ^= 1) {
        const int a0 = a.q.begin(2 * p), a1 = max(a0, a.q.begin(2 * p + 1)), a2 = max(a1, a.q.begin(2 * p + 2));
        const int from = side ? a1 : a0, to = side ? a2 : a1;
        const Pieces pieces(from, to);
        Score v{};
        F2 sum = pair(0.f, 0.f), lost = sum;
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
                const Two2 once = two_sum(sum, pair(d0, d1)), twice = two_sum(once.hi, pair(d2, d3));
                sum = twice.hi;
                lost = lost + (once.lo + twice.lo);
                if (a.average) v.count += nonzero_bytes(m[u]);
            }
        }
        const float2 hi = both(sum), lo = both(lost);
        v.sum = {hi.x, lo.x};
        add(v.sum, Two{hi.y, lo.y});
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) add(v.sum, shuffled(v.sum, o));
        if (a.average) v.count = warp_add(v.count);
        if (lane == 0) warps_of[parity][warp] = v;
        __syncthreads();
        if (warp == 0) {
            // lanes 0 and WARPS / 2 end with the two sequences' sums
            v = warps_of[parity][lane % WARPS];
#pragma unroll
            for (int o = WARPS / 4; o >= 1; o >>= 1) {
                add(v.sum, shuffled(v.sum, o));
                v.count += __shfl_xor_sync(0xffffffffu, v.count, o);
            }
            if (split && (lane == 0 || lane == WARPS / 2)) own[parity][lane != 0] = v;
        }
        if (split) {
            sync_ctas();  // the other CTAs' sums are there
            if (warp == 0) {
                v = Score{};
                if (lane == 0 || lane == WARPS / 2)
                    for (int c = 0; c < a.share.ctas; ++c) {
                        const Score &o = own[parity][lane != 0];
                        add(v.sum, Two{load_peer(&o.sum.hi, c), load_peer(&o.sum.lo, c)});
                        v.count += load_peer(&o.count, c);
                    }
            }
        }
        if (warp == 0) {
            v.sum = finished(v.sum);
            const Score second{{__shfl_sync(0xffffffffu, v.sum.hi, WARPS / 2), __shfl_sync(0xffffffffu, v.sum.lo, WARPS / 2)},
                               __shfl_sync(0xffffffffu, v.count, WARPS / 2)};
            if (lane == 0) {
                r0 = times(v.sum, a.beta);
                r1 = times(second.sum, a.beta);
                if (a.average) {
                    r0 = divided(r0, (float)max(v.count, 1));
                    r1 = divided(r1, (float)max(second.count, 1));
                }
                delta = r0;
                add(delta, Two{-r1.hi, -r1.lo});
                const float d = value(delta);
                float slope;
                if (a.kind == PREFERENCE_LOGISTIC) {
                    const float up = 1.f / (1.f + expf(-d)), down = 1.f / (1.f + expf(d));
                    slope = a.smoothing * up - (1.f - a.smoothing) * down;
                } else if (a.kind == PREFERENCE_HINGE) {
                    const float gap = below(1.f, delta);
                    slope = gap <= 0.f ? 0.f : gap == gap ? -1.f : gap;  // NaN stays
                } else {
                    slope = -2.f * (below(0.5f, delta) / a.beta) / a.beta;
                }
                slope *= a.beta * a.weight;
                slope_of[parity][0] = a.average ? slope / (float)max(v.count, 1) : slope;
                slope_of[parity][1] = a.average ? -slope / (float)max(second.count, 1) : -slope;
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
        // what nobody waits for
        if (rank == 0 && threadIdx.x == 0) {
            const float d = value(delta);
            float l;
            if (a.kind == PREFERENCE_LOGISTIC) {
                const float soft = log1pf(expf(-fabsf(d)));
                l = (1.f - a.smoothing) * (soft + fmaxf(-d, 0.f));
                if (a.smoothing > 0.f) l += a.smoothing * (soft + fmaxf(d, 0.f));
            } else if (a.kind == PREFERENCE_HINGE) {
                const float gap = below(1.f, delta);
                l = gap <= 0.f ? 0.f : gap;
            } else {
                const float gap = below(0.5f, delta) / a.beta;
                l = gap * gap;
            }
            a.pair_loss[p] = l;
            a.rewards[2 * p] = value(r0);
            a.rewards[2 * p + 1] = value(r1);
            loss += l;
            a.q.check(2 * p, 2);
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
    // by the preparing launch, where there is one: tokens that count by block, the sequence that each tile begins in,
    // the weight of each sequence's tokens
    int *counted, *first_of;
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
    F2 gain, kl, clipped;
};

// Two tokens: their gradient over grad_scale; here: whether they count.
__device__ __forceinline__ F2 two_tokens(const Policy &a, bool here0, bool here1, F2 logp, F2 old, F2 ref, F2 advantage, F2 weight,
                                         Seen &seen) {
    const float2 adv = both(advantage), wt = both(weight);
    const bool up0 = adv.x >= 0.f, up1 = adv.y >= 0.f;
    Two2 d = two_sum(logp, old * pair(-1.f, -1.f));
    const float2 hi = both(d.hi), left = both(d.lo);
    d.lo = pair(fabsf(hi.x) < INFINITY ? left.x : 0.f, fabsf(hi.y) < INFINITY ? left.y : 0.f);
    const float2 past = both((d.hi - pair(up0 ? a.log_high.hi : a.log_low.hi, up1 ? a.log_high.hi : a.log_low.hi)) +
                             (d.lo - pair(up0 ? a.log_high.lo : a.log_low.lo, up1 ? a.log_high.lo : a.log_low.lo)));
    const bool clip0 = up0 ? past.x > 0.f : past.x < 0.f, clip1 = up1 ? past.y > 0.f : past.y < 0.f;
    // A r as A + A (r - 1): the sum over many tokens whose advantages cancel has no bias from the last place of
    // the exponential
    const float2 free = both(exp_of(d.hi).above);
    const F2 above = pair(clip0 ? (up0 ? a.edge_high : a.edge_low) : free.x, clip1 ? (up1 ? a.edge_high : a.edge_low) : free.y);
    const float2 gain = both(fma2(advantage, above, advantage));
    F2 slope = pair(clip0 ? 0.f : -gain.x, clip1 ? 0.f : -gain.y);
    seen.gain = fma2(pair(here0 ? gain.x : 0.f, here1 ? gain.y : 0.f), weight, seen.gain);
    seen.clipped = seen.clipped + pair(here0 && clip0 ? wt.x : 0.f, here1 && clip1 ? wt.y : 0.f);
    if (a.ref) {
        const Exp e = exp_of(ref - logp);
        const float2 kl = both(e.rest);
        seen.kl = fma2(pair(here0 ? kl.x : 0.f, here1 ? kl.y : 0.f), weight, seen.kl);
        slope = fma2(pair(-a.kl_coef, -a.kl_coef), e.above, slope);
    }
    const float2 out = both(slope * weight);
    return pair(here0 ? out.x : 0.f, here1 ? out.y : 0.f);
}
// A piece: m says which tokens count.
__device__ __forceinline__ float4 four_tokens(const Policy &a, unsigned m, const Tokens &t, float4 weight, Seen &seen) {
    if (!m) return make_float4(0.f, 0.f, 0.f, 0.f);
    const F2 scale = pair(a.grad_scale, a.grad_scale);
    const float2 g0 = both(scale * two_tokens(a, counts(m, 0), counts(m, 1), pair(t.logp.x, t.logp.y), pair(t.old.x, t.old.y),
                                              pair(t.ref.x, t.ref.y), pair(t.advantage.x, t.advantage.y),
                                              pair(weight.x, weight.y), seen));
    const float2 g1 = both(scale * two_tokens(a, counts(m, 2), counts(m, 3), pair(t.logp.z, t.logp.w), pair(t.old.z, t.old.w),
                                              pair(t.ref.z, t.ref.w), pair(t.advantage.z, t.advantage.w),
                                              pair(weight.z, weight.w), seen));
    return make_float4(g0.x, g0.y, g1.x, g1.y);
}
// The block's sums, to threads 0 .. 2: -gain, kl, clipped.
template <int WARPS> __device__ __forceinline__ float block_sums(const Seen &seen, float (*red)[3]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float v[3] = {warp_add(-sum2(seen.gain)), warp_add(sum2(seen.kl)), warp_add(sum2(seen.clipped))};
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
    Seen seen{pair(0.f, 0.f), pair(0.f, 0.f), pair(0.f, 0.f)};
    const int units = a.q.offsets ? a.q.count : a.tiles;
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
        for (int t = t0 + (int)threadIdx.x; t < t1; t += kPrepareThreads) a.first_of[t] = s;
        if (a.reduction == POLICY_SEQUENCE_MEAN) {
            const int n = a.q.mask ? block_add<kPrepareThreads / 32>(count_tokens(a.q.mask, from, to, threadIdx.x, kPrepareThreads), red)
                                   : to - from;
            if (threadIdx.x == 0) a.weight_of[s] = 1.f / ((float)max(n, 1) * (float)a.q.count);
        }
        if (threadIdx.x == 0) a.q.check(s, 1);
    }
}

template <bool VEC> __global__ void __launch_bounds__(kTileThreads, 8) policy_tiles_kernel(const Policy a) {
    constexpr int U = kTile / 4 / kTileThreads;
    __shared__ float sums_of[kTileThreads / 32][3];
    const int lane = threadIdx.x & 31;
    const bool lookup = a.per_sequence || a.reduction == POLICY_SEQUENCE_MEAN;
    grid_dependency_wait();
    grid_dependency_launch();
    int b0 = 0, b1 = a.q.tokens;
    if (a.q.offsets) {
        b0 = a.q.begin(0);
        b1 = max(b0, a.q.begin(a.q.count));
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
    Seen seen{pair(0.f, 0.f), pair(0.f, 0.f), pair(0.f, 0.f)};
    for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const int p0 = tile * (kTile / 4) + (int)threadIdx.x;
        Tokens t[U];
        unsigned m[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int piece = p0 + k * kTileThreads, at = piece * 4;
            m[k] = 0;
            if (at >= b1 || at + 4 <= b0) continue;
            m[k] = counting<VEC>(a.q.mask, piece, b0, b1, a.q.tokens);
            t[k] = load_tokens<VEC>(a, piece, 0.f);
        }
        int s0 = 0, s1 = 0;
        if (lookup) {
            s0 = min(max(a.first_of[tile], 0), a.q.count - 1);
            s1 = tile + 1 < a.tiles ? min(max(a.first_of[tile + 1], s0), a.q.count - 1) : a.q.count - 1;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int piece = p0 + k * kTileThreads, at = piece * 4;
            if (at >= a.q.tokens) continue;
            float4 weight = make_float4(same, same, same, same);
            if (lookup && m[k]) {
                int lo = s0, hi = s1;  // the last sequence that begins at or in front of the piece
                while (lo < hi) {
                    const int mid = (lo + hi + 1) / 2;
                    if (a.q.begin(mid) <= at) lo = mid;
                    else hi = mid - 1;
                }
                float w[4], v[4];
                int s = lo, end = a.q.begin(s + 1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    while (s < s1 && at + i >= end) end = a.q.begin(++s + 1);
                    w[i] = a.reduction == POLICY_SEQUENCE_MEAN ? a.weight_of[s] : same;
                    v[i] = a.per_sequence ? a.advantages[s] : 0.f;
                }
                weight = make_float4(w[0], w[1], w[2], w[3]);
                if (a.per_sequence) t[k].advantage = make_float4(v[0], v[1], v[2], v[3]);
            }
            const float4 g = four_tokens(a, m[k], t[k], weight, seen);
            store4<VEC>(a.dlogp, piece, 0, a.q.tokens, g);
        }
    }
    const float sum = block_sums<kTileThreads / 32>(seen, sums_of);
    if (threadIdx.x < 3) a.partial[(int64_t)blockIdx.x * 4 + threadIdx.x] = sum;
}

// parts[k] = weight * sum of partial[0 .. blocks)[k], loss = parts[0] + kl_coef parts[1], in two floats (a warp's
// addition in fp64 takes 15 cycles here) and a fixed order
constexpr int kJoinThreads = 1024;
__global__ void __launch_bounds__(kJoinThreads) loss_join_kernel(const float *partial, int blocks, float weight, float kl_coef,
                                                                 float *parts, float *loss) {
    __shared__ Two red[3][kJoinThreads / 32];
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Two v[3] = {};
#pragma unroll 4
    for (int i = threadIdx.x; i < blocks; i += kJoinThreads) {
        const float4 x = reinterpret_cast<const float4 *>(partial)[i];
        add(v[0], Two{x.x, 0.f});
        add(v[1], Two{x.y, 0.f});
        add(v[2], Two{x.z, 0.f});
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
        for (int k = 0; k < 3; ++k) add(v[k], shuffled(v[k], o));
    if (lane == 0)
        for (int k = 0; k < 3; ++k) red[k][warp] = v[k];
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] = red[k][lane];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
        for (int k = 0; k < 3; ++k) add(v[k], shuffled(v[k], o));
    if (lane) return;
    for (int k = 0; k < 3; ++k) v[k] = times(finished(v[k]), weight);
    if (parts)
        for (int k = 0; k < 3; ++k) parts[k] = value(v[k]);
    if (kl_coef != 0.f) add(v[0], times(v[1], kl_coef));
    *loss = value(v[0]);
}

// ---- launches ------------------------------------------------------------------------------

// Threads of a block and CTAs for a unit.  A unit's chain of loads, sums and stores is what takes the time, and the
// longest unit ends last: as many threads for each as the SMs hold for all of them at once, and 1024 tokens or more
// for a CTA.  Few units of few tokens: one cluster, which needs no launch to join its losses.
struct Cut {
    Share share;
    int threads;
};
Cut cut_of(int units, int64_t tokens) {
    const int64_t length = tokens / std::max(units, 1), room = (int64_t)num_sms() * 2048;
    if (units <= kMaxCluster && length <= 2048) return {{1, 1}, length > 512 ? kManyThreads : kFewThreads};
    int threads = kFewThreads, c = 1;
    while (threads < kManyThreads && (int64_t)units * threads * 2 <= room && length > (int64_t)threads * 4) threads *= 2;
    while (c < kMaxCluster && (int64_t)units * c * threads * 4 <= room && length > (int64_t)c * threads * 8) c *= 2;
    return {{c, 0}, threads};
}
int blocks_of(int units, const Share &s) {
    if (s.alone) return units <= 1 ? 1 : units <= 2 ? 2 : units <= 4 ? 4 : kMaxCluster;
    return s.ctas * std::max(1, std::min(units, num_sms() * kMaxBlocksPerSm / s.ctas));
}
template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), int blocks, const Cut &cut, cudaStream_t st, A &&...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(cut.threads);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cut.share.alone ? blocks : cut.share.ctas;
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

// partial sums of the blocks
int64_t partial_bytes() { return (int64_t)num_sms() * kMaxBlocksPerSm * 16; }
// and of the policy loss: counts, each tile's first sequence, each sequence's weight
constexpr int kMostCounts = 512;
int64_t policy_bytes(int64_t sequences, int64_t tokens) {
    return partial_bytes() + 4 * (kMostCounts + ceil_div(tokens, kTile) + sequences);
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
        bytes = partial_bytes();
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
        if (workspace_bytes < partial_bytes())
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": the workspace is smaller than preference_loss_workspace() says");
        const Cut cut = cut_of((int)pairs, tokens);
        const Share share = cut.share;
        const int blocks = blocks_of((int)pairs, share);
        const float part = mean ? 1.f / (float)std::max<int64_t>(pairs, 1) : 1.f;
        const Preference a{{offsets, offset_bytes == 8, (int)(2 * pairs), (int)tokens, mask, stage_flag_ptr()},
                           logp, ref_logp, dlogp, pair_loss, rewards, static_cast<float *>(workspace), loss, share, (int)pairs,
                           kind, average != 0, beta, smoothing, grad_scale * part, part};
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        const bool vec = all_aligned16({logp, ref_logp, dlogp}, mask);
        auto pick = [&](auto threads) {
            constexpr int THREADS = decltype(threads)::value;
            return vec ? &preference_kernel<THREADS, true> : &preference_kernel<THREADS, false>;
        };
        auto *k = cut.threads == kFewThreads      ? pick(std::integral_constant<int, kFewThreads>{})
                  : cut.threads == kMiddleThreads ? pick(std::integral_constant<int, kMiddleThreads>{})
                                                  : pick(std::integral_constant<int, kManyThreads>{});
        cudaError_t e = cudaSuccess;
        SPCO_LAUNCH("preference_loss", st, e = launch_clusters(k, blocks, cut, st, a));
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
        bytes = policy_bytes(sequences, tokens);
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
        if (workspace_bytes < policy_bytes(sequences, tokens))
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": the workspace is smaller than policy_loss_workspace() says");
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        if (!offsets && reduction == POLICY_SEQUENCE_MEAN) reduction = POLICY_TOKEN_MEAN;
        const int tiles = (int)ceil_div(tokens, kTile), units = offsets ? (int)sequences : tiles;
        const bool vec = all_aligned16({logp, old_logp, ref_logp, dlogp, per_sequence ? nullptr : advantages}, mask);
        float *partial = static_cast<float *>(workspace);
        int *counted = reinterpret_cast<int *>(static_cast<char *>(workspace) + partial_bytes());
        Policy a{{offsets, offset_bytes == 8, (int)sequences, (int)tokens, mask, stage_flag_ptr()},
                 logp, old_logp, ref_logp, advantages, dlogp, partial, parts, loss, counted, counted + kMostCounts,
                 reinterpret_cast<float *>(counted + kMostCounts + tiles), 0, tiles, per_sequence != 0, reduction, kl_coef,
                 grad_scale, (float)clip_high, (float)-clip_low, log_two(1. + clip_high), log_two(1. - clip_low)};
        cudaError_t e = cudaSuccess;
        const Cut cut = cut_of(units, tokens);
        if (cut.share.alone) {
            auto *k = cut.threads == kManyThreads ? (vec ? &policy_few_kernel<kManyThreads, true> : &policy_few_kernel<kManyThreads, false>)
                               : (vec ? &policy_few_kernel<kFewThreads, true> : &policy_few_kernel<kFewThreads, false>);
            SPCO_LAUNCH("policy_loss", st, e = launch_clusters(k, blocks_of(units, cut.share), cut, st, a));
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
        const int blocks = std::max(1, std::min(tiles, num_sms() * kMaxBlocksPerSm));
        auto *k = vec ? &policy_tiles_kernel<true> : &policy_tiles_kernel<false>;
        if (prepared) {
            SPCO_LAUNCH("policy_loss", st, e = launch_dependent(k, dim3(blocks), dim3(kTileThreads), 0, st, a));
            SPECOPTIM_CUDA(e);
        } else {
            SPCO_LAUNCH("policy_loss", st, k<<<blocks, kTileThreads, 0, st>>>(a));
            SPECOPTIM_LAUNCHED("policy_tiles_kernel");
        }
        SPCO_LAUNCH("loss_join", st,
                    e = launch_dependent(loss_join_kernel, dim3(1), dim3(kJoinThreads), 0, st, partial, blocks, 1.f, kl_coef, parts,
                                         loss));
        SPECOPTIM_CUDA(e);
        return SPECOPTIM_OK;
    });
}
