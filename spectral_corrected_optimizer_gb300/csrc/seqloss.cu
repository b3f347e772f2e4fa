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
constexpr int kUnroll = 4;        // pieces of 4 tokens that a thread has in flight
constexpr int kMaxCluster = 8;
constexpr int kTile = 4096;       // tokens of a unit where there are no sequences
constexpr int kBlocksPerSm = 8;

// ---- two floats ----------------------------------------------------------------------------

struct Two {
    float hi, lo;
};
// a + b and what the rounding lost (0 where the sum is not finite)
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = a + b, t = s - a;
    const float e = (a - (s - t)) + (b - t);
    return {s, fabsf(s) < INFINITY ? e : 0.f};
}
__device__ __forceinline__ void add(Two &a, float x) {
    const Two t = two_sum(a.hi, x);
    a.hi = t.hi;
    a.lo += t.lo;
}
__device__ __forceinline__ void add(Two &a, const Two &b) {
    const Two t = two_sum(a.hi, b.hi);
    a.hi = t.hi;
    a.lo += t.lo + b.lo;
}
__device__ __forceinline__ void warp_add(Two &a) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        add(a, Two{__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)});
}
__device__ __forceinline__ int warp_add(int v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---- the tokens ----------------------------------------------------------------------------

struct Sequences {
    const void *offsets;  // null: units of kTile tokens
    int wide;             // 8-byte offsets
    int64_t count, tokens;
    const uint8_t *mask;
    unsigned *flag;

    __device__ __forceinline__ int64_t raw(int64_t i) const {
        return wide ? static_cast<const int64_t *>(offsets)[i] : (int64_t)static_cast<const int32_t *>(offsets)[i];
    }
    // where sequence i begins, within the tokens
    __device__ __forceinline__ int64_t begin(int64_t i) const {
        if (!offsets) return min(i * kTile, tokens);
        return min(max(raw(i), (int64_t)0), tokens);
    }
    // whether the offsets i .. i + n keep the rule
    __device__ __forceinline__ void check(int64_t i, int n) const {
        if (!offsets) return;
        bool good = raw(i) >= 0 && raw(i + n) <= tokens;
        for (int k = 0; k < n; ++k) good = good && raw(i + k) <= raw(i + k + 1);
        if (!good) atomicExch(flag, kSiteOffset);
    }
};

// x[t .. t + 3], t a multiple of 4; 0 behind the end
template <bool VEC> __device__ __forceinline__ float4 load4(const float *x, int64_t t, int64_t tokens) {
    if (VEC && t + 4 <= tokens) return *reinterpret_cast<const float4 *>(x + t);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < tokens) v.x = x[t];
    if (t + 1 < tokens) v.y = x[t + 1];
    if (t + 2 < tokens) v.z = x[t + 2];
    if (t + 3 < tokens) v.w = x[t + 3];
    return v;
}
// which of the tokens t .. t + 3 lie in [a, b) and count, as bits
template <bool VEC> __device__ __forceinline__ unsigned valid4(const uint8_t *mask, int64_t t, int64_t a, int64_t b, int64_t tokens) {
    unsigned in = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) in |= (unsigned)(t + i >= a && t + i < b) << i;
    if (!mask || !in) return in;
    if (VEC && t + 4 <= tokens) {
        const unsigned m = *reinterpret_cast<const unsigned *>(mask + t);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!(m >> (8 * i) & 0xffu)) in &= ~(1u << i);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((in >> i & 1u) && !mask[t + i]) in &= ~(1u << i);
    }
    return in;
}
// v to those of the tokens t .. t + 3 that lie in [a, b)
template <bool VEC> __device__ __forceinline__ void store4(float *x, int64_t t, int64_t a, int64_t b, float4 v) {
    if (VEC && t >= a && t + 4 <= b) {
        *reinterpret_cast<float4 *>(x + t) = v;
        return;
    }
    if (t >= a && t < b) x[t] = v.x;
    if (t + 1 >= a && t + 1 < b) x[t + 1] = v.y;
    if (t + 2 >= a && t + 2 < b) x[t + 2] = v.z;
    if (t + 3 >= a && t + 3 < b) x[t + 3] = v.w;
}

// zeros for the tokens in front of the first sequence and behind the last one
__device__ __forceinline__ void zero_outside(const Sequences &q, int64_t sequences, float *dlogp) {
    if (!q.offsets) return;
    const int64_t a = q.begin(0), b = max(a, q.begin(sequences));
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
// every thread of the CTAs that share a unit's sums
__device__ __forceinline__ void sync_ctas(int ctas) {
    if (ctas == 1) return;
    __syncwarp();
    cluster_sync();
}

// ---- preference ----------------------------------------------------------------------------

struct Preference {
    Sequences q;
    const float *logp, *ref;
    float *dlogp, *pair_loss, *rewards, *partial, *loss;
    int64_t pairs;
    int kind, average, ctas;
    float beta, smoothing, weight, loss_weight;  // weight: grad_scale / pairs or grad_scale
};

// What a CTA has of a pair: both sequences' sums and tokens.
struct PairSums {
    Two sum[2];
    int count[2];
};

template <bool VEC> __global__ void __launch_bounds__(kThreads) preference_kernel(const Preference a) {
    __shared__ PairSums warps_of[2][kWarps], own[2];
    __shared__ float slope_of[2][2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = a.ctas > 1 ? (int)cluster_rank() : 0;
    const int64_t cluster = blockIdx.x / a.ctas, clusters = gridDim.x / a.ctas;
    const int64_t at = (int64_t)rank * kThreads + threadIdx.x, step = (int64_t)a.ctas * kThreads;
    grid_dependency_launch();
    zero_outside(a.q, 2 * a.pairs, a.dlogp);
    float loss = 0.f;  // thread 0 of rank 0
    int parity = 0;
    for (int64_t p = cluster; p < a.pairs; p += clusters, parity ^= 1) {
        const int64_t a0 = a.q.begin(2 * p), a1 = max(a0, a.q.begin(2 * p + 1)), a2 = max(a1, a.q.begin(2 * p + 2));
        if (rank == 0 && threadIdx.x == 0) a.q.check(2 * p, 2);
        PairSums v{};
        const int64_t first = a0 / 4, last = (a2 + 3) / 4;
        for (int64_t p0 = first + at; p0 < last; p0 += step * kUnroll) {
            float4 x[kUnroll], r[kUnroll];
            unsigned in[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t t = (p0 + u * step) * 4;
                in[u] = 0;
                if (p0 + u * step >= last) continue;
                in[u] = valid4<VEC>(a.q.mask, t, a0, a2, a.q.tokens);
                x[u] = load4<VEC>(a.logp, t, a.q.tokens);
                r[u] = a.ref ? load4<VEC>(a.ref, t, a.q.tokens) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (!in[u]) continue;
                const int64_t t = (p0 + u * step) * 4;
                const float d[4] = {x[u].x - r[u].x, x[u].y - r[u].y, x[u].z - r[u].z, x[u].w - r[u].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool here = in[u] >> i & 1u, second = t + i >= a1;
                    add(v.sum[0], here && !second ? d[i] : 0.f);
                    add(v.sum[1], here && second ? d[i] : 0.f);
                    v.count[0] += here && !second;
                    v.count[1] += here && second;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            warp_add(v.sum[k]);
            v.count[k] = warp_add(v.count[k]);
        }
        if (lane == 0) warps_of[parity][warp] = v;
        __syncthreads();
        if (threadIdx.x == 0) {
            v = warps_of[parity][0];
            for (int w = 1; w < kWarps; ++w)
                for (int k = 0; k < 2; ++k) {
                    add(v.sum[k], warps_of[parity][w].sum[k]);
                    v.count[k] += warps_of[parity][w].count[k];
                }
            own[parity] = v;
        }
        sync_ctas(a.ctas);  // the other CTAs' sums are there
        if (threadIdx.x == 0) {
            PairSums all{};
            for (int c = 0; c < a.ctas; ++c) {
                const PairSums &o = own[parity];
                for (int k = 0; k < 2; ++k) {
                    if (a.ctas > 1) {
                        add(all.sum[k], Two{load_peer(&o.sum[k].hi, c), load_peer(&o.sum[k].lo, c)});
                        all.count[k] += load_peer(&o.count[k], c);
                    } else {
                        all = o;
                    }
                }
            }
            double reward[2];
            float share[2];
            for (int k = 0; k < 2; ++k) {
                share[k] = a.average ? 1.f / (float)max(all.count[k], 1) : 1.f;
                const double s = (double)all.sum[k].hi + (double)all.sum[k].lo;
                reward[k] = (double)a.beta * (a.average ? s / (double)max(all.count[k], 1) : s);
            }
            const double delta = reward[0] - reward[1];
            const float d = (float)delta;
            float l, slope;
            if (a.kind == PREFERENCE_LOGISTIC) {
                const float soft = log1pf(expf(-fabsf(d))), up = 1.f / (1.f + expf(-d)), down = 1.f / (1.f + expf(d));
                // a weight of 0 takes no part, however large its term
                l = (1.f - a.smoothing) * (soft + fmaxf(-d, 0.f));
                if (a.smoothing > 0.f) l += a.smoothing * (soft + fmaxf(d, 0.f));
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
            slope_of[parity][0] = slope * a.beta * a.weight * share[0];
            slope_of[parity][1] = -slope * a.beta * a.weight * share[1];
            if (rank == 0) {
                a.pair_loss[p] = l;
                a.rewards[2 * p] = (float)reward[0];
                a.rewards[2 * p + 1] = (float)reward[1];
                loss += l;
            }
        }
        __syncthreads();
        const float g0 = slope_of[parity][0], g1 = slope_of[parity][1];
        for (int64_t piece = first + at; piece < last; piece += step) {
            const int64_t t = piece * 4;
            const unsigned in = valid4<VEC>(a.q.mask, t, a0, a2, a.q.tokens);
            float g[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = in >> i & 1u ? (t + i < a1 ? g0 : g1) : 0.f;
            store4<VEC>(a.dlogp, t, a0, a2, make_float4(g[0], g[1], g[2], g[3]));
        }
    }
    if (rank == 0 && threadIdx.x == 0) {
        if (clusters == 1) *a.loss = loss * a.loss_weight;
        else a.partial[cluster] = loss;
    }
    sync_ctas(a.ctas);  // no CTA leaves while its sums are read
}

// ---- policy --------------------------------------------------------------------------------

struct Policy {
    Sequences q;
    const float *logp, *old, *ref, *advantages;
    float *dlogp, *partial, *parts, *loss;
    const int *counts;       // valid tokens by block of the counting launch; null: none was made
    int counted;             // its blocks
    int64_t units;
    int per_sequence, reduction, ctas, count_here;
    float kl_coef, grad_scale, edge_high, edge_low;  // edges: the bounds' distance from 1
    Two log_high, log_low;   // log(1 + clip_high), log(1 - clip_low)
};

// tokens that count in [a, b), by this thread's share
template <bool VEC>
__device__ __forceinline__ int count_tokens(const Sequences &q, int64_t a, int64_t b, int64_t at, int64_t step) {
    int n = 0;
#pragma unroll 4
    for (int64_t piece = a / 4 + at; piece < (b + 3) / 4; piece += step)
        n += __popc(valid4<VEC>(q.mask, piece * 4, a, b, q.tokens));
    return n;
}
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
template <bool VEC> __global__ void __launch_bounds__(kThreads) policy_count_kernel(const Sequences q, int64_t sequences, int *__restrict__ counts) {
    __shared__ int red[kWarps];
    grid_dependency_launch();
    const int64_t a = q.offsets ? q.begin(0) : 0, b = q.offsets ? max(a, q.begin(sequences)) : q.tokens;
    const int n = block_add(count_tokens<VEC>(q, a, b, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads), red);
    if (threadIdx.x == 0) counts[blockIdx.x] = n;
}

// exp(q) - q - 1: by its series where the difference would lose digits (|q| < 1/2: the
// next term is below 2^-24 of the first)
__device__ __forceinline__ float kl_of(float q, float e) {
    float p = 1.f / 362880.f;
    p = fmaf(p, q, 1.f / 40320.f);
    p = fmaf(p, q, 1.f / 5040.f);
    p = fmaf(p, q, 1.f / 720.f);
    p = fmaf(p, q, 1.f / 120.f);
    p = fmaf(p, q, 1.f / 24.f);
    p = fmaf(p, q, 1.f / 6.f);
    p = fmaf(p, q, 0.5f);
    return fabsf(q) < 0.5f ? p * q * q : e - q;
}

template <bool VEC> __global__ void __launch_bounds__(kThreads) policy_kernel(const Policy a) {
    __shared__ int red[kWarps], own[2];
    __shared__ float sums_of[kWarps][3];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = a.ctas > 1 ? (int)cluster_rank() : 0;
    const int64_t cluster = blockIdx.x / a.ctas, clusters = gridDim.x / a.ctas;
    const int64_t at = (int64_t)rank * kThreads + threadIdx.x, step = (int64_t)a.ctas * kThreads;
    grid_dependency_wait();
    grid_dependency_launch();
    zero_outside(a.q, a.q.count, a.dlogp);
    float weight = 1.f;  // of a token
    if (a.reduction == POLICY_TOKEN_MEAN) {
        int64_t n = 0;
        if (a.counts || a.count_here) {
            const int64_t b0 = a.q.offsets ? a.q.begin(0) : 0, b1 = a.q.offsets ? max(b0, a.q.begin(a.q.count)) : a.q.tokens;
            int c = 0;
            if (a.counts) {
                for (int i = threadIdx.x; i < a.counted; i += kThreads) c += a.counts[i];
            } else {
                c = count_tokens<VEC>(a.q, b0, b1, threadIdx.x, kThreads);
            }
            n = block_add(c, red);
        } else {
            n = a.q.offsets ? max(a.q.begin(a.q.count) - a.q.begin(0), (int64_t)0) : a.q.tokens;
        }
        weight = 1.f / (float)max(n, (int64_t)1);
    }
    float total[3] = {0.f, 0.f, 0.f};
    int parity = 0;
    for (int64_t u = cluster; u < a.units; u += clusters, parity ^= 1) {
        const int64_t b0 = a.q.begin(u), b1 = max(b0, a.q.begin(u + 1));
        if (rank == 0 && threadIdx.x == 0) a.q.check(u, 1);
        if (a.reduction == POLICY_SEQUENCE_MEAN) {
            int64_t n = b1 - b0;
            if (a.q.mask) {
                int c = block_add(count_tokens<VEC>(a.q, b0, b1, at, step), red);
                if (a.ctas > 1) {
                    if (threadIdx.x == 0) own[parity] = c;
                    sync_ctas(a.ctas);
                    c = 0;
                    for (int k = 0; k < a.ctas; ++k) c += load_peer(&own[parity], k);
                }
                n = c;
            }
            weight = 1.f / ((float)max(n, (int64_t)1) * (float)a.q.count);
        }
        const float scaled = weight * a.grad_scale, shared_advantage = a.per_sequence ? a.advantages[u] : 0.f;
        float sum[3] = {0.f, 0.f, 0.f};
        const int64_t first = b0 / 4, last = (b1 + 3) / 4;
        for (int64_t p0 = first + at; p0 < last; p0 += step * kUnroll) {
            float4 x[kUnroll], o[kUnroll], r[kUnroll], w[kUnroll];
            unsigned in[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int64_t t = (p0 + k * step) * 4;
                in[k] = 0;
                if (p0 + k * step >= last) continue;
                in[k] = valid4<VEC>(a.q.mask, t, b0, b1, a.q.tokens);
                x[k] = load4<VEC>(a.logp, t, a.q.tokens);
                o[k] = load4<VEC>(a.old, t, a.q.tokens);
                if (a.ref) r[k] = load4<VEC>(a.ref, t, a.q.tokens);
                w[k] = a.per_sequence ? make_float4(shared_advantage, shared_advantage, shared_advantage, shared_advantage)
                                      : load4<VEC>(a.advantages, t, a.q.tokens);
            }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                if (p0 + k * step >= last) continue;
                const float lp[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, lo[4] = {o[k].x, o[k].y, o[k].z, o[k].w};
                const float lr[4] = {r[k].x, r[k].y, r[k].z, r[k].w}, ad[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
                float g[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool here = in[k] >> i & 1u, gains = ad[i] >= 0.f;
                    const Two d = two_sum(lp[i], -lo[i]), edge = gains ? a.log_high : a.log_low;
                    const float past = (d.hi - edge.hi) + (d.lo - edge.lo);
                    const bool clipped = gains ? past > 0.f : past < 0.f;
                    // A r as A + A (r - 1): expm1 is exact to its own size, so the sum over many
                    // tokens whose advantages cancel has no bias from exp's last place
                    const float above = clipped ? (gains ? a.edge_high : a.edge_low) : expm1f(d.hi);
                    const float gain = fmaf(ad[i], above, ad[i]);
                    float slope = clipped ? 0.f : -gain, kl = 0.f;
                    if (a.ref) {
                        const float q = lr[i] - lp[i], e = expm1f(q);
                        kl = kl_of(q, e);
                        slope = fmaf(-a.kl_coef, e, slope);
                    }
                    g[i] = here ? slope * scaled : 0.f;
                    sum[0] -= here ? gain : 0.f;
                    sum[1] += here ? kl : 0.f;
                    sum[2] += here && clipped ? 1.f : 0.f;
                }
                store4<VEC>(a.dlogp, (p0 + k * step) * 4, b0, b1, make_float4(g[0], g[1], g[2], g[3]));
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
        a.partial[(int64_t)threadIdx.x * gridDim.x + blockIdx.x] = s;
    }
    sync_ctas(a.ctas);  // no CTA leaves while its count is read
}

// sums[k] = weight * sum of partial[k][0 .. blocks), loss = sums[0] + kl_coef sums[1]
__global__ void __launch_bounds__(kThreads) loss_join_kernel(const float *partial, int kinds, int blocks, float weight,
                                                             float kl_coef, float *sums, float *loss) {
    __shared__ double red[kWarps][3];
    grid_dependency_wait();
    for (int k = 0; k < kinds; ++k) {
        double v = 0.;
        for (int i = threadIdx.x; i < blocks; i += kThreads) v += (double)partial[(int64_t)k * blocks + i];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5][k] = v;
    }
    __syncthreads();
    if (threadIdx.x) return;
    double s[3] = {0., 0., 0.};
    for (int k = 0; k < kinds; ++k) {
        for (int w = 0; w < kWarps; ++w) s[k] += red[w][k];
        s[k] *= (double)weight;
        if (sums) sums[k] = (float)s[k];
    }
    *loss = (float)(kl_coef != 0.f ? s[0] + (double)kl_coef * s[1] : s[0]);
}

// ---- launches ------------------------------------------------------------------------------

// CTAs for a unit: as many as the SMs have room for beside the other units', while each still has some
// 1024 tokens (a unit may be a few times longer than the average).
int ctas_of(int64_t units, int64_t tokens) {
    int c = 1;
    while (c < kMaxCluster && units * c * 2 <= 2 * num_sms() && tokens / std::max<int64_t>(units, 1) > (int64_t)c * kThreads * 4) c *= 2;
    return c;
}
int clusters_of(int64_t units, int ctas) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(units, (int64_t)num_sms() * kBlocksPerSm / ctas));
}
// blocks that count tokens, and from how many tokens on (below, every block counts all of them)
constexpr int64_t kCountHere = 32768;
int count_blocks(int64_t tokens) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(num_sms() * 2, ceil_div(tokens, kThreads * 32)));
}

template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), int blocks, int ctas, bool dependent, cudaStream_t st, A &&...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

int check_common(int64_t count, int64_t tokens, const void *logp, const void *offsets, int32_t offset_bytes, bool need_offsets,
                 const float *loss, const float *dlogp, const void *workspace, const std::string &what) {
    if (count < 0 || count > (int64_t)1 << 30) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": sequences outside [0, 2^30]");
    if (tokens < 0 || tokens > (int64_t)1 << 40) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": tokens outside [0, 2^40]");
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

int64_t workspace_of() { return round_up((int64_t)num_sms() * kBlocksPerSm * 3 * 4, 16) + (int64_t)num_sms() * 2 * 4; }

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
        if (pairs < 0 || pairs > (int64_t)1 << 29 || tokens < 0 || tokens > (int64_t)1 << 40)
            return fail(SPECOPTIM_ERR_INVALID_ARG, "preference_loss: pairs outside [0, 2^29] or tokens outside [0, 2^40]");
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
        if (pairs < 0 || pairs > (int64_t)1 << 29) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": pairs outside [0, 2^29]");
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
        const int ctas = ctas_of(pairs, tokens), clusters = clusters_of(pairs, ctas), blocks = clusters * ctas;
        const float share = mean ? 1.f / (float)std::max<int64_t>(pairs, 1) : 1.f;
        const Preference a{{offsets, offset_bytes == 8, 2 * pairs, tokens, mask, stage_flag_ptr()},
                           logp, ref_logp, dlogp, pair_loss, rewards, static_cast<float *>(workspace), loss, pairs, kind,
                           average != 0, ctas, beta, smoothing, grad_scale * share, share};
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        auto *k = all_aligned16({logp, ref_logp, dlogp}, mask) ? &preference_kernel<true> : &preference_kernel<false>;
        cudaError_t e = cudaSuccess;
        SPCO_LAUNCH("preference_loss", st, e = launch_clusters(k, blocks, ctas, false, st, a));
        SPECOPTIM_CUDA(e);
        if (clusters == 1) return SPECOPTIM_OK;
        SPCO_LAUNCH("loss_join", st,
                    e = launch_dependent(loss_join_kernel, dim3(1), dim3(kThreads), 0, st, a.partial, 1, clusters, share, 0.f,
                                         static_cast<float *>(nullptr), loss));
        SPECOPTIM_CUDA(e);
        return SPECOPTIM_OK;
    });
}

extern "C" int64_t policy_loss_workspace(int64_t sequences, int64_t tokens) {
    int64_t bytes = -1;
    entry([&]() -> int {
        if (sequences < 0 || sequences > (int64_t)1 << 30 || tokens < 0 || tokens > (int64_t)1 << 40)
            return fail(SPECOPTIM_ERR_INVALID_ARG, "policy_loss: sequences outside [0, 2^30] or tokens outside [0, 2^40]");
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
        const int64_t units = offsets ? sequences : ceil_div(tokens, kTile);
        const int ctas = offsets ? ctas_of(units, tokens) : 1, clusters = clusters_of(units, ctas), blocks = clusters * ctas;
        const bool vec = all_aligned16({logp, old_logp, ref_logp, dlogp, per_sequence ? nullptr : advantages}, mask);
        const Sequences q{offsets, offset_bytes == 8, sequences, tokens, mask, stage_flag_ptr()};
        float *partial = static_cast<float *>(workspace);
        int *counts = reinterpret_cast<int *>(static_cast<char *>(workspace) +
                                              round_up((int64_t)num_sms() * kBlocksPerSm * 3 * 4, 16));
        const bool counting = mask && reduction == POLICY_TOKEN_MEAN, apart = counting && tokens > kCountHere;
        const int counted = count_blocks(tokens);
        cudaError_t e = cudaSuccess;
        if (apart) {
            auto *k = vec ? &policy_count_kernel<true> : &policy_count_kernel<false>;
            SPCO_LAUNCH("policy_count", st, k<<<counted, kThreads, 0, st>>>(q, sequences, counts));
            SPECOPTIM_LAUNCHED("policy_count_kernel");
        }
        const Policy a{q, logp, old_logp, ref_logp, advantages, dlogp, partial, parts, loss, apart ? counts : nullptr, counted,
                       units, per_sequence != 0, reduction, ctas, counting && !apart, kl_coef, grad_scale,
                       (float)clip_high, (float)-clip_low, log_two(1. + clip_high), log_two(1. - clip_low)};
        auto *k = vec ? &policy_kernel<true> : &policy_kernel<false>;
        SPCO_LAUNCH("policy_loss", st, e = launch_clusters(k, blocks, ctas, apart, st, a));
        SPECOPTIM_CUDA(e);
        SPCO_LAUNCH("loss_join", st,
                    e = launch_dependent(loss_join_kernel, dim3(1), dim3(kThreads), 0, st, partial, 3, blocks, 1.f, kl_coef,
                                         parts, loss));
        SPECOPTIM_CUDA(e);
        return SPECOPTIM_OK;
    });
}
