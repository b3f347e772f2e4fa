// The global norm of many tensors and clipping (include/finetune.h).
//
//   norm = sqrt(sum (scale g)^2) or max |scale g|,
//   out  = g scale (norm > max_norm ? max_norm / norm : 1)
//
// The tensors' addresses and sizes travel in the launch's parameters (no copy to
// the device that a captured graph would repeat), up to kMany tensors a launch.
// Their memory is cut into chunks of 16 KB; a block takes neighbouring chunks,
// whatever tensors they lie in, so many small tensors cost what one large one
// does, and loads a chunk while it works on the one in front.  Each block leaves one
// partial; a second launch adds the partials in their order, in every block that
// scales values by the result.  Where one launch does not take all tensors, a launch
// of one block adds the partials of all of them, once for the launches that scale: each
// block of each launch would add them again, work that grows with the square of the
// tensors (100000 of 10 values 14.5 ms so, 0.80 with the join).
//
// Measured on a GB300 (copy bandwidth 6.78 TB/s, reading alone 7.4):
//   norm of 1e9 bytes 142 us, 7.0 TB/s (89 % of the DRAM's cycles); of the 1B model's 4.9 GB of fp32
//     gradients 700 us;
//   the same clipped into other buffers 2.21 ms: 14.8 GB, read twice and written once, at 6.7 TB/s;
//   one layer's bf16 gradients (122 MB) into fp32 89 us, 5.5 TB/s; 33 for the norm and 62 for the
//     scaling where each launch is timed by itself; 4e6 fp32 values 14 us;
//   2.5e8 fp32 values in place 473 us, into another buffer 470, bf16 248 and 246.
// Values that lie otherwise between two 16-byte boundaries than where they are written to (bf16 into
// fp32: between 16 and 32) are written one by one: 2.5e8 fp32 values 711 us, bf16 780, bf16 into fp32
// 1141 (334 where they lie alike), fp32 into bf16 538 (383).  Buffers of their own lie alike.
// The norm of squares spills 20 bytes a thread (4 of the other norm).
// Reading the chunks from the back, what the norm's launch left in L2 first, gained nothing.
#include <algorithm>
#include <cstring>
#include <string>
#include <vector>

#include "../../include/finetune.h"
#include "rowvec.cuh"

namespace spco {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPieces = 4;                         // of 16 bytes, per thread and chunk
constexpr int kChunk = kThreads * kPieces;         // pieces of a chunk
constexpr int kFew = 64, kMany = 1024;             // tensors of a launch
constexpr int kBlocksPerSm = 4;

// Tensors of one launch, as the 16-byte pieces of memory that they lie in: src[i] may begin inside its first piece.
// first[i]: chunks in front of tensor i.
template <int CAP> struct Table {
    int count, blocks;
    const void *src[CAP];
    int64_t size[CAP];
    int first[CAP + 1];
    uint8_t type[CAP];
};
template <int CAP> struct Outs {
    void *dst[CAP];
    uint8_t type[CAP];
};
static_assert(sizeof(Table<kMany>) + sizeof(Outs<kMany>) + 64 <= 32764, "parameters of a launch");

// The tensor that chunk c lies in.
template <int CAP> __device__ __forceinline__ int tensor_of(const Table<CAP> &t, int c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
// Where a block's chunks begin among the launch's.
template <int CAP> __device__ __forceinline__ int chunk_begin(const Table<CAP> &t, int block) {
    return (int)((int64_t)t.first[t.count] * block / t.blocks);
}

// |b| or a, whichever is larger; NaN if one of them is
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
    return m;
}

// One tensor as pieces: values [0, size) lie at values [head, head + size) from `base`.
template <typename T> struct Pieces {
    static constexpr int V = 16 / (int)sizeof(T);
    const T *base;
    int64_t head, end;
    __device__ __forceinline__ Pieces(const void *src, int64_t size) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(src);
        base = reinterpret_cast<const T *>(a & ~uintptr_t(15));
        head = (int64_t)((a & 15) / sizeof(T));
        end = head + size;
    }
    // of `count` chunks from `chunk` on, those that are whole: [lo, hi), counted from `chunk`
    __device__ __forceinline__ void whole_chunks(int chunk, int count, int &lo, int &hi) const {
        const int64_t chunk_values = (int64_t)kChunk * V;
        lo = chunk == 0 && head ? 1 : 0;
        hi = (int)min((int64_t)count, end / chunk_values - chunk);
        hi = max(lo, hi);
        lo = min(lo, count);
        hi = min(hi, count);
    }
    __device__ __forceinline__ bool whole(int64_t piece) const { return piece * V >= head && (piece + 1) * V <= end; }
    // zeros where the tensor has no values
    __device__ __forceinline__ uint4 load(int64_t piece) const {
        if (whole(piece)) return reinterpret_cast<const uint4 *>(base)[piece];
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t at = piece * V + i;
            if (at < head || at >= end) continue;
            if (sizeof(T) == 4) w[i % 4] = reinterpret_cast<const uint32_t *>(base)[at];
            else w[i / 2 % 4] |= (uint32_t)reinterpret_cast<const uint16_t *>(base)[at] << (16 * (i & 1));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
__device__ __forceinline__ void piece_values(uint4 u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void piece_values(uint4 u, float (&v)[8]) {
    v[0] = lo_f(u.x); v[1] = hi_f(u.x); v[2] = lo_f(u.y); v[3] = hi_f(u.y);
    v[4] = lo_f(u.z); v[5] = hi_f(u.z); v[6] = lo_f(u.w); v[7] = hi_f(u.w);
}

// A chunk's pieces of this thread.
struct Loaded {
    uint4 u[kPieces];
};
__device__ __forceinline__ Loaded load_whole(const uint4 *p) {
    Loaded r;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) r.u[k] = p[k * kThreads];
    return r;
}
template <typename T> __device__ __forceinline__ Loaded load_part(const Pieces<T> &p, int64_t first) {
    Loaded r;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) r.u[k] = p.load(first + k * kThreads);
    return r;
}

// f(tensor, its first chunk here, how many) for each tensor that chunks [c0, c1) lie in.  The table is read once a
// tensor: an indexed read of a launch's parameters takes some 100 cycles.
template <int CAP, typename F> __device__ __forceinline__ void each_tensor(const Table<CAP> &t, int c0, int c1, F &&f) {
    if (c0 >= c1) return;
    for (int i = tensor_of(t, c0), c = c0; c < c1; ++i) {
        const int end = min(c1, t.first[i + 1]);
        f(i, c - t.first[i], end - c);
        c = end;
    }
}

// What a thread has added up: squares in two floats, squares beyond their range, the largest magnitude.
struct Sums {
    float sum, lost, most;
    double far;
};
// A square leaves fp32's range from 2^64 on and loses digits below 2^-50; where a thread's values reach 2^40 or stay
// below 2^-50, it squares them in 64 bits.  Otherwise a chunk's squares, at most 32, are added in fp32 and the chunks in
// two floats (sums of 2^44 values stay below 2^128): fp64 additions take 15 cycles for a warp's.
template <typename T, int KIND> __device__ __forceinline__ void take(const Loaded &x, Sums &a) {
    constexpr int V = 16 / (int)sizeof(T);
    float top = 0.f, s = 0.f;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        float v[V];
        piece_values(x.u[k], v);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            top = max_nan(top, v[i]);
            if (KIND == NORM_L2) s = fmaf(v[i], v[i], s);
        }
    }
    a.most = max_nan(a.most, top);
    if (KIND != NORM_L2) return;
    if (top < 0x1p40f && (top > 0x1p-50f || top == 0.f)) {
        const float t = a.sum + s, u = t - a.sum;
        a.lost += (a.sum - (t - u)) + (s - u);
        a.sum = t;
    } else {
        // unrolled: pieces that a loop variable picks would live in local memory, for all chunks
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            float v[V];
            piece_values(x.u[k], v);
#pragma unroll
            for (int i = 0; i < V; ++i) a.far = fma((double)v[i], (double)v[i], a.far);
        }
    }
}

// Neighbouring chunks of one tensor; the whole ones in a loop of their own, which loads a chunk while it takes the one in
// front (a load behind a choice of ways would be waited for where the ways meet).
template <int KIND, typename T> __device__ __forceinline__ void take_run(const Pieces<T> &p, int chunk, int count, Sums &a) {
    int lo, hi;
    p.whole_chunks(chunk, count, lo, hi);
    const int64_t first = (int64_t)chunk * kChunk + threadIdx.x;
    const auto part = [&](int from, int to) {
        for (int c = from; c < to; ++c) take<T, KIND>(load_part(p, first + (int64_t)c * kChunk), a);
    };
    part(0, lo);
    if (lo < hi) {
        const uint4 *q = reinterpret_cast<const uint4 *>(p.base) + first + (int64_t)lo * kChunk;
        Loaded x = load_whole(q);
        for (int n = hi - lo - 1; n > 0; --n) {
            q += kChunk;
            const Loaded y = load_whole(q);
            take<T, KIND>(x, a);
            x = y;
        }
        take<T, KIND>(x, a);
    }
    part(hi, count);
}

// What a thread or a block leaves: squares in two floats (or the largest magnitude) and those beyond their range.
struct __align__(16) Part {
    float sum, lost;
    double far;
};
template <int KIND> __device__ __forceinline__ void join(Part &a, const Part &b) {
    if (KIND == NORM_MAX) {
        a.sum = max_nan(a.sum, b.sum);
        return;
    }
    const float t = a.sum + b.sum, u = t - a.sum;
    a.lost += b.lost + ((a.sum - (t - u)) + (b.sum - u));
    a.sum = t;
}
// Over the block, to all threads; in a fixed order.
template <int KIND> __device__ __forceinline__ Part block_join(Part v, Part *red) {
    const bool far = KIND == NORM_L2 && __syncthreads_or(v.far != 0.);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        join<KIND>(v, Part{__shfl_xor_sync(0xffffffffu, v.sum, o), __shfl_xor_sync(0xffffffffu, v.lost, o), 0.});
        if (far) v.far += __shfl_xor_sync(0xffffffffu, v.far, o);
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < kWarps; ++i) {
        join<KIND>(v, red[i]);
        if (far) v.far += red[i].far;
    }
    return v;
}

template <int CAP, int KIND>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) norm_parts_kernel(const __grid_constant__ Table<CAP> t, Part *__restrict__ parts) {
    __shared__ Part red[kWarps];
    grid_dependency_launch();
    const int c0 = chunk_begin(t, blockIdx.x), c1 = chunk_begin(t, blockIdx.x + 1);
    Sums a{0.f, 0.f, 0.f, 0.};
    each_tensor(t, c0, c1, [&](int i, int chunk, int count) {
        if (t.type[i] == STAGE_BF16) take_run<KIND>(Pieces<bf16>(t.src[i], t.size[i]), chunk, count, a);
        else take_run<KIND>(Pieces<float>(t.src[i], t.size[i]), chunk, count, a);
    });
    const Part v = block_join<KIND>(KIND == NORM_L2 ? Part{a.sum, a.lost, a.far} : Part{a.most, 0.f, 0.}, red);
    if (threadIdx.x == 0) parts[blockIdx.x] = v;
}

// The norm from all partials, the same in every block that asks: in fp32, and as |scale| root unit, unit a power of two,
// where fp32 does not hold it.
struct __align__(16) Norm {
    float value, root, unit;
};
template <int KIND> __device__ __forceinline__ Norm norm_of(const Part *parts, int count, float scale, Part *red) {
    Part v{0.f, 0.f, 0.};
#pragma unroll 4
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const Part x = parts[i];
        join<KIND>(v, x);
        if (KIND == NORM_L2 && x.far != 0.) v.far += x.far;
    }
    v = block_join<KIND>(v, red);
    if (KIND == NORM_L2 && v.far != 0.) {
        const double n = sqrt(v.far + ((double)v.sum + (double)v.lost));  // 2^-149 to 2^148
        const float value = (float)(fabs((double)scale) * n);
        return n >= 1. ? Norm{value, (float)(n * 0x1p-64), 0x1p64f} : Norm{value, (float)(n * 0x1p64), 0x1p-64f};
    }
    const float n = KIND == NORM_L2 ? sqrtf(v.sum + v.lost) : v.sum;
    return {fabsf(scale) * n, n, 1.f};
}

// What a value is multiplied by: two factors, the second one a power of two and 1 wherever fp32 holds their product.
struct Factor {
    float a, b;
    __device__ __forceinline__ float operator()(float v) const { return v * a * b; }
};
__device__ __forceinline__ Factor factor_of(const Norm &n, float scale, float max_norm) {
    constexpr float kLeast = 0x1p-126f;  // below, fp32 has fewer digits
    if (n.value <= max_norm) return {scale, 1.f};
    const float ratio = max_norm / n.value, f = scale * ratio;
    if (n.value != n.value || (n.value < INFINITY && n.value >= kLeast && ratio >= kLeast && fabsf(f) >= kLeast)) return {f, 1.f};
    const double x = copysign((double)max_norm, (double)scale) / ((double)n.root * (double)n.unit);
    return fabs(x) < 0x1p-100 ? Factor{(float)(x * 0x1p100), 0x1p-100f} : Factor{(float)x, 1.f};
}

template <int KIND>
__global__ void __launch_bounds__(kThreads) norm_join_kernel(const Part *parts, int count, float scale, float *norm, Norm *joined) {
    __shared__ Part red[kWarps];
    grid_dependency_wait();
    const Norm n = norm_of<KIND>(parts, count, scale, red);
    if (threadIdx.x) return;
    *norm = n.value;
    if (joined) *joined = n;
}

// Values of a piece to q, the place of its first one.
__device__ __forceinline__ void put_values(float *q, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(q) = make_float4(v[0], v[1], v[2], v[3]);
}
// 32 bytes as one store: two of 16 write each sector in halves (scaling one layer's bf16 gradients to fp32, the launch by
// itself: 62 us, 78 with two)
__device__ __forceinline__ void put_values(float *q, const float (&v)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
__device__ __forceinline__ void put_values(bf16 *q, const float (&v)[8]) { store8(q, v); }
__device__ __forceinline__ void put_values(bf16 *q, const float (&v)[4]) {
    *reinterpret_cast<uint2 *>(q) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

// A chunk that may be cut short, or whose values go to places that are not aligned.
template <typename TI, typename TO>
__device__ __forceinline__ void give_part(const Pieces<TI> &p, TO *q, int64_t first, Factor factor) {
    constexpr int V = Pieces<TI>::V;
    const Loaded x = load_part(p, first);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        float v[V];
        piece_values(x.u[k], v);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t at = (first + k * kThreads) * V + i;
            if (at >= p.head && at < p.end) q[at] = from_f<TO>(factor(v[i]));
        }
    }
}
template <typename TI, typename TO> __device__ __forceinline__ void give(const Loaded &x, TO *q, Factor factor) {
    constexpr int V = Pieces<TI>::V;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        float v[V];
        piece_values(x.u[k], v);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = factor(v[i]);
        put_values(q + k * kThreads * V, v);
    }
}
// Neighbouring chunks of one tensor, the whole ones in a loop that loads ahead.
template <typename TI, typename TO>
__device__ __forceinline__ void give_run(const Pieces<TI> &p, void *dst, int chunk, int count, Factor factor) {
    constexpr int V = Pieces<TI>::V, ALIGN = V * (int)sizeof(TO);  // of a piece's values
    TO *q = static_cast<TO *>(dst) - p.head;  // value `at` of the pieces goes to q[at]
    int lo, hi;
    p.whole_chunks(chunk, count, lo, hi);
    if (reinterpret_cast<uintptr_t>(q) & (ALIGN - 1)) lo = hi = 0;
    const int64_t first = (int64_t)chunk * kChunk + threadIdx.x;
    const auto part = [&](int from, int to) {
        for (int c = from; c < to; ++c) give_part(p, q, first + (int64_t)c * kChunk, factor);
    };
    part(0, lo);
    if (lo < hi) {
        const uint4 *from = reinterpret_cast<const uint4 *>(p.base) + first + (int64_t)lo * kChunk;
        TO *to = q + (first + (int64_t)lo * kChunk) * V;
        Loaded x = load_whole(from);
        for (int n = hi - lo - 1; n > 0; --n) {
            from += kChunk;
            const Loaded y = load_whole(from);
            give<TI>(x, to, factor);
            to += (int64_t)kChunk * V;
            x = y;
        }
        give<TI>(x, to, factor);
    }
    part(hi, count);
}

template <int CAP, int KIND>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) clip_kernel(const __grid_constant__ Table<CAP> t,
                                                                      const __grid_constant__ Outs<CAP> o, const Part *parts,
                                                                      int count, const Norm *joined, float scale,
                                                                      float max_norm, int in_place, float *norm) {
    __shared__ Part red[kWarps];
    const int c0 = chunk_begin(t, blockIdx.x), c1 = chunk_begin(t, blockIdx.x + 1);
    grid_dependency_wait();
    const Norm n = joined ? *joined : norm_of<KIND>(parts, count, scale, red);
    if (!joined && blockIdx.x == 0 && threadIdx.x == 0) *norm = n.value;
    const Factor factor = factor_of(n, scale, max_norm);
    if (in_place && factor.a == 1.f && factor.b == 1.f) return;
    each_tensor(t, c0, c1, [&](int i, int chunk, int count) {
        void *dst = o.dst[i];
        if (t.type[i] == STAGE_BF16) {
            const Pieces<bf16> p(t.src[i], t.size[i]);
            if (o.type[i] == STAGE_BF16) give_run<bf16, bf16>(p, dst, chunk, count, factor);
            else give_run<bf16, float>(p, dst, chunk, count, factor);
        } else {
            const Pieces<float> p(t.src[i], t.size[i]);
            if (o.type[i] == STAGE_BF16) give_run<float, bf16>(p, dst, chunk, count, factor);
            else give_run<float, float>(p, dst, chunk, count, factor);
        }
    });
}

struct Call {
    const void *const *grads;
    const int64_t *sizes;
    const int32_t *types;
    void *const *outs;  // null: the norm alone
    const int32_t *out_types;
    int32_t count;
    float scale, max_norm;
    int32_t kind;
    float *norm;
    void *workspace;
    int64_t workspace_bytes;
    cudaStream_t st;
};

// partials of the launches that form the norm
int64_t parts_of(int32_t count) {
    return std::max<int64_t>(1, ceil_div(count, kMany)) * num_sms() * kBlocksPerSm;
}
// and the norm itself, where more than one launch scales by it
int64_t workspace_of(int32_t count) {
    return parts_of(count) * (int64_t)sizeof(Part) + (count > kMany ? (int64_t)sizeof(Norm) : 0);
}

// No value is written twice, and none is read after another place's was written to it.
int check_outs(const Call &c, const std::string &what) {
    struct Range {
        uintptr_t from, to;
        int of;
    };
    std::vector<Range> outs;
    outs.reserve(c.count);
    for (int i = 0; i < c.count; ++i) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(c.outs[i]);
        if (c.sizes[i]) outs.push_back({p, p + c.sizes[i] * type_bytes(c.out_types[i]), i});
    }
    std::sort(outs.begin(), outs.end(), [](const Range &a, const Range &b) { return a.from < b.from; });
    for (size_t k = 1; k < outs.size(); ++k)
        if (outs[k].from < outs[k - 1].to)
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": two of the tensors that are written overlap");
    for (int i = 0; i < c.count; ++i) {
        if (!c.sizes[i]) continue;
        const uintptr_t p = reinterpret_cast<uintptr_t>(c.grads[i]), e = p + c.sizes[i] * type_bytes(c.types[i]);
        auto k = std::upper_bound(outs.begin(), outs.end(), p, [](uintptr_t a, const Range &r) { return a < r.to; });
        for (; k != outs.end() && k->from < e; ++k)
            if (k->of != i || k->from != p || c.types[i] != c.out_types[i])
                return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": a tensor that is written overlaps another one that is read");
    }
    return SPECOPTIM_OK;
}

int check_call(const Call &c, bool clip, const std::string &what) {
    if (c.count < 0 || c.count > 1 << 24) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": count outside [0, 2^24]");
    if (c.kind != NORM_L2 && c.kind != NORM_MAX)
        return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": kind must be NORM_L2 or NORM_MAX");
    if (!(c.scale - c.scale == 0.f)) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": scale must be finite");
    if (clip && !(c.max_norm >= 0.f)) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": max_norm must be >= 0");
    if (!c.norm || !c.workspace ||
        (c.count > 0 && (!c.grads || !c.sizes || !c.types || (clip && (!c.outs || !c.out_types)))))
        return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": null pointer");
    if (!aligned_to(c.norm, 4) || !aligned16(c.workspace))
        return fail(SPECOPTIM_ERR_MISALIGNED, what + ": norm must be aligned to 4 bytes, the workspace to 16");
    for (int i = 0; i < c.count; ++i) {
        if (!type_ok(c.types[i]) || (clip && !type_ok(c.out_types[i])))
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": types must be STAGE_BF16 or STAGE_FP32");
        if (c.sizes[i] < 0 || c.sizes[i] > (int64_t)1 << 40)
            return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": a tensor's size lies outside [0, 2^40]");
        if (c.sizes[i] == 0) continue;
        if (!c.grads[i] || (clip && !c.outs[i])) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": null pointer");
        if (!aligned_to(c.grads[i], type_bytes(c.types[i])) || (clip && !aligned_to(c.outs[i], type_bytes(c.out_types[i]))))
            return fail(SPECOPTIM_ERR_MISALIGNED, what + ": tensors must be aligned to their elements");
    }
    if (clip)
        if (int rc = check_outs(c, what)) return rc;
    return SPECOPTIM_OK;
}

// Fills a launch with tensors from `at` on; its chunks fit 31 bits.
template <int CAP> void fill(const Call &c, int &at, Table<CAP> *t, Outs<CAP> *o) {
    t->count = 0;
    t->first[0] = 0;
    for (; at < c.count && t->count < CAP; ++at) {
        if (c.sizes[at] == 0) continue;
        const int64_t b = (int64_t)type_bytes(c.types[at]), head = (int64_t)(reinterpret_cast<uintptr_t>(c.grads[at]) & 15);
        const int64_t chunks = t->first[t->count] + ceil_div(head + c.sizes[at] * b, kChunk * 16);
        if (chunks > INT32_MAX) break;  // one tensor has 2^28 at most
        const int k = t->count++;
        t->src[k] = c.grads[at];
        t->size[k] = c.sizes[at];
        t->type[k] = (uint8_t)c.types[at];
        t->first[k + 1] = (int)chunks;
        if (c.outs) {
            o->dst[k] = c.outs[at];
            o->type[k] = (uint8_t)c.out_types[at];
        }
    }
    t->blocks = (int)std::min<int64_t>(t->first[t->count], (int64_t)num_sms() * kBlocksPerSm);
}

template <int CAP, int KIND> int run(const Call &c) {
    Table<CAP> t;
    Outs<CAP> o;
    Part *parts = static_cast<Part *>(c.workspace);
    int total = 0, launches = 0;
    const int64_t room = parts_of(c.count);
    int in_place = c.outs != nullptr;
    for (int i = 0; in_place && i < c.count; ++i) in_place = c.sizes[i] == 0 || c.outs[i] == c.grads[i];
    for (int at = 0; at < c.count;) {
        fill(c, at, &t, &o);
        if (!t.count) break;
        if (total + t.blocks > room) return fail(SPECOPTIM_ERR_INVALID_ARG, "grad_norm: more values than a call takes");
        SPCO_LAUNCH("grad_norm", c.st, norm_parts_kernel<CAP, KIND><<<t.blocks, kThreads, 0, c.st>>>(t, parts + total));
        SPECOPTIM_LAUNCHED("norm_parts_kernel");
        total += t.blocks;
        ++launches;
    }
    cudaError_t e = cudaSuccess;
    const bool alone = !c.outs || !total;  // nothing to scale
    Norm *joined = !alone && launches > 1 ? reinterpret_cast<Norm *>(parts + room) : nullptr;
    if (alone || joined) {
        SPCO_LAUNCH("grad_norm_join", c.st,
                    e = launch_dependent(norm_join_kernel<KIND>, dim3(1), dim3(kThreads), 0, c.st, parts, total, c.scale,
                                         c.norm, joined));
        SPECOPTIM_CUDA(e);
    }
    if (alone) return SPECOPTIM_OK;
    for (int at = 0; at < c.count;) {
        if (launches > 1) fill(c, at, &t, &o);
        else at = c.count;  // the table of the norm's only launch
        if (!t.count) break;
        SPCO_LAUNCH("clip_grads", c.st,
                    e = launch_dependent(clip_kernel<CAP, KIND>, dim3(t.blocks), dim3(kThreads), 0, c.st, t, o, parts, total,
                                         joined, c.scale, c.max_norm, in_place, c.norm));
        SPECOPTIM_CUDA(e);
    }
    return SPECOPTIM_OK;
}

int run_call(const Call &c, bool clip, const char *what) {
    if (int rc = check_call(c, clip, what)) return rc;
    if (c.workspace_bytes < workspace_of(c.count))
        return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": the workspace is smaller than grad_norm_workspace() says");
    if (int rc = bind_device()) return rc;
    if (c.kind == NORM_L2) return c.count <= kFew ? run<kFew, NORM_L2>(c) : run<kMany, NORM_L2>(c);
    return c.count <= kFew ? run<kFew, NORM_MAX>(c) : run<kMany, NORM_MAX>(c);
}

}  // namespace
}  // namespace spco

using namespace spco;

extern "C" int64_t grad_norm_workspace(int32_t count) {
    int64_t bytes = -1;
    entry([&]() -> int {
        if (count < 0 || count > 1 << 24) return fail(SPECOPTIM_ERR_INVALID_ARG, "grad_norm: count outside [0, 2^24]");
        bytes = workspace_of(count);
        return SPECOPTIM_OK;
    });
    return bytes;
}

extern "C" int grad_norm(const void *const *grads, const int64_t *sizes, const int32_t *types, int32_t count, float scale,
                         int32_t kind, float *norm, void *workspace, int64_t workspace_bytes, void *stream) {
    return entry([&]() -> int {
        const Call c{grads, sizes, types, nullptr, nullptr, count, scale, 0.f, kind, norm, workspace, workspace_bytes,
                     static_cast<cudaStream_t>(stream)};
        return run_call(c, false, "grad_norm");
    });
}

extern "C" int clip_grads(const void *const *grads, const int64_t *sizes, const int32_t *types, void *const *outs,
                          const int32_t *out_types, int32_t count, float scale, float max_norm, int32_t kind, float *norm,
                          void *workspace, int64_t workspace_bytes, void *stream) {
    return entry([&]() -> int {
        const Call c{grads, sizes, types, outs, out_types, count, scale, max_norm, kind, norm, workspace, workspace_bytes,
                     static_cast<cudaStream_t>(stream)};
        return run_call(c, true, "clip_grads");
    });
}
