// The global norm of many tensors and clipping (include/finetune.h).
//
//   norm = sqrt(sum (scale g)^2) or max |scale g|,
//   out  = g scale (norm > max_norm ? max_norm / norm : 1)
//
// The tensors' addresses and sizes travel in the launch's parameters (no copy to
// the device that a captured graph would repeat), up to kMany tensors a launch.
// Their values are cut into chunks of kChunk; a block takes neighbouring chunks,
// whatever tensors they lie in, so many small tensors cost what one large one
// does.  Each block leaves one partial; a second launch adds the partials in
// their order, in every block that scales values by the result.
#include <algorithm>
#include <cstring>
#include <string>
#include <vector>

#include "../../include/finetune.h"
#include "rowvec.cuh"

namespace spco {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPieces = 4;                         // of 8 values, per thread and chunk
constexpr int kChunk = kThreads * kPieces * 8;
constexpr int kFew = 64, kMany = 1024;             // tensors of a launch
constexpr int kBlocksPerSm = 8;

// Tensors of one launch.  first[i]: chunks in front of tensor i.
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

// |b| or a, whichever is larger; NaN if one of them is
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
    return m;
}

// A block's chunks: [begin, end) of the launch's.
template <int CAP> __device__ __forceinline__ int chunk_begin(const Table<CAP> &t, int block) {
    return (int)((int64_t)t.first[t.count] * block / t.blocks);
}

__device__ __forceinline__ bool vec_aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Values i .. i + 7 of a tensor, zeros behind its end.
template <typename T> __device__ __forceinline__ void load_values(const T *p, int64_t i, int64_t size, bool vec, float (&v)[8]) {
    if (vec && i + 8 <= size) {
        load8(p + i, v);
    } else if (i < size) {
        load_any(Span<const T>(p, size), Span<const T>(p, size).lo + i, v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.f;
    }
}

// What is added up of one chunk by one thread: squares, or the largest magnitude.
// A square leaves fp32's range from 2^64 on and loses digits below 2^-50; where a
// thread's values reach there, it squares them in 64 bits.  Otherwise a chunk's 32
// squares are added in fp32 and the chunks in two floats: fp64 additions, 15 cycles for a
// warp's, would take an eighth of the time.
template <typename T, int KIND>
__device__ __forceinline__ void take_chunk(const T *p, int64_t from, int64_t size, float &sum, float &lost, double &far, float &most) {
    const bool vec = vec_aligned(p);
    float v[kPieces][8];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) load_values(p, from + (k * kThreads + (int)threadIdx.x) * 8, size, vec, v[k]);
    float top = 0.f, s = 0.f;
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            top = max_nan(top, v[k][i]);
            if (KIND == NORM_L2) s = fmaf(v[k][i], v[k][i], s);
        }
    most = max_nan(most, top);
    if (KIND == NORM_L2) {
        if (top < 0x1p50f && (top > 0x1p-50f || top == 0.f)) {
            // below 2^105 a chunk: 2^22 of them stay within fp32
            const float t = sum + s, u = t - sum;
            lost += (sum - (t - u)) + (s - u);
            sum = t;
        } else {
#pragma unroll 1
            for (int k = 0; k < kPieces; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) far = fma((double)v[k][i], (double)v[k][i], far);
        }
    }
}

// Sum (or largest) over the block, to thread 0.
template <int KIND> __device__ __forceinline__ double block_join(double v, double *red) {
    const auto join = [](double a, double b) { return KIND == NORM_L2 ? a + b : (double)max_nan((float)a, (float)b); };
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < kWarps; ++i) v = join(v, red[i]);
    return v;
}

template <int CAP, int KIND>
__global__ void __launch_bounds__(kThreads) norm_parts_kernel(const __grid_constant__ Table<CAP> t, double *__restrict__ parts) {
    __shared__ double red[kWarps];
    grid_dependency_launch();
    const int c0 = chunk_begin(t, blockIdx.x), c1 = chunk_begin(t, blockIdx.x + 1);
    float sum = 0.f, lost = 0.f, most = 0.f;
    double far = 0.;
    int i = c0 < c1 ? tensor_of(t, c0) : 0;
    for (int c = c0; c < c1; ++c) {
        while (c >= t.first[i + 1]) ++i;
        const int64_t from = (int64_t)(c - t.first[i]) * kChunk;
        if (t.type[i] == STAGE_BF16) take_chunk<bf16, KIND>(static_cast<const bf16 *>(t.src[i]), from, t.size[i], sum, lost, far, most);
        else take_chunk<float, KIND>(static_cast<const float *>(t.src[i]), from, t.size[i], sum, lost, far, most);
    }
    const double v = block_join<KIND>(KIND == NORM_L2 ? far + ((double)sum + (double)lost) : (double)most, red);
    if (threadIdx.x == 0) parts[blockIdx.x] = v;
}

// The norm from all partials, the same in every block that asks.  Twice: in fp32, and
// times 2^-64 for a norm that fp32 does not hold.
struct Norm {
    float value, small;
};
template <int KIND> __device__ __forceinline__ Norm norm_of(const double *parts, int count, float scale, double *red) {
    double v = 0.;
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const double x = parts[i];
        v = KIND == NORM_L2 ? v + x : (double)max_nan((float)v, (float)x);
    }
    v = block_join<KIND>(v, red);
    // fp64 arithmetic is slow: for what fp32 cannot do
    if (KIND == NORM_L2 && v > 0x1p-100 && v < 0x1p120) {
        const float n = fabsf(scale) * sqrtf((float)v);
        return {n, n * 0x1p-64f};
    }
    const double n = fabs((double)scale) * (KIND == NORM_L2 ? sqrt(v) : v);
    return {(float)n, (float)(n * 0x1p-64)};
}

template <int KIND>
__global__ void __launch_bounds__(kThreads) norm_join_kernel(const double *parts, int count, float scale, float *norm) {
    __shared__ double red[kWarps];
    grid_dependency_wait();
    const Norm n = norm_of<KIND>(parts, count, scale, red);
    if (threadIdx.x == 0) *norm = n.value;
}

template <typename TI, typename TO>
__device__ __forceinline__ void scale_chunk(const TI *p, TO *q, int64_t from, int64_t size, float factor) {
    const bool vec = vec_aligned(p), whole = vec_aligned(q);
    float v[kPieces][8];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) load_values(p, from + (k * kThreads + (int)threadIdx.x) * 8, size, vec, v[k]);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        const int64_t at = from + (k * kThreads + (int)threadIdx.x) * 8;
        if (at >= size) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] *= factor;
        if (whole && at + 8 <= size) {
            store8(q + at, v[k]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (at + i < size) q[at + i] = from_f<TO>(v[k][i]);
        }
    }
}

// The blocks go through their chunks from the back: what the norm's launch read last is in L2.
template <int CAP, int KIND>
__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ Table<CAP> t, const __grid_constant__ Outs<CAP> o,
                                                        const double *parts, int count, float scale, float max_norm,
                                                        float *norm) {
    __shared__ double red[kWarps];
    grid_dependency_wait();
    const Norm n = norm_of<KIND>(parts, count, scale, red);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n.value;
    float factor = scale;
    if (!(n.value <= max_norm)) factor *= n.value < INFINITY ? max_norm / n.value : max_norm * 0x1p-64f / n.small;
    const int c0 = chunk_begin(t, blockIdx.x), c1 = chunk_begin(t, blockIdx.x + 1);
    int i = c0 < c1 ? tensor_of(t, c1 - 1) : 0;
    for (int c = c1 - 1; c >= c0; --c) {
        while (c < t.first[i]) --i;
        if (factor == 1.f && o.dst[i] == t.src[i]) {  // in place and nothing to do: on to the tensor in front
            c = t.first[i];
            continue;
        }
        const int64_t from = (int64_t)(c - t.first[i]) * kChunk;
        const bool in16 = t.type[i] == STAGE_BF16, out16 = o.type[i] == STAGE_BF16;
        const bf16 *p16 = static_cast<const bf16 *>(t.src[i]);
        const float *p32 = static_cast<const float *>(t.src[i]);
        if (in16 && out16) scale_chunk(p16, static_cast<bf16 *>(o.dst[i]), from, t.size[i], factor);
        else if (in16) scale_chunk(p16, static_cast<float *>(o.dst[i]), from, t.size[i], factor);
        else if (out16) scale_chunk(p32, static_cast<bf16 *>(o.dst[i]), from, t.size[i], factor);
        else scale_chunk(p32, static_cast<float *>(o.dst[i]), from, t.size[i], factor);
    }
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

int64_t workspace_of(int32_t count) {
    const int64_t launches = std::max<int64_t>(1, ceil_div(count, kMany));
    return launches * num_sms() * kBlocksPerSm * 8;
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
        const int64_t chunks = t->first[t->count] + ceil_div(c.sizes[at], kChunk);
        if (chunks > INT32_MAX) break;  // one tensor has 2^27 at most
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
    double *parts = static_cast<double *>(c.workspace);
    int total = 0, launches = 0;
    const int64_t room = workspace_of(c.count) / 8;
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
    if (!c.outs || !total) {
        SPCO_LAUNCH("grad_norm_join", c.st,
                    e = launch_dependent(norm_join_kernel<KIND>, dim3(1), dim3(kThreads), 0, c.st, parts, total, c.scale,
                                         c.norm));
        SPECOPTIM_CUDA(e);
        return SPECOPTIM_OK;
    }
    for (int at = 0; at < c.count;) {
        if (launches > 1) fill(c, at, &t, &o);
        else at = c.count;  // the table of the norm's only launch
        if (!t.count) break;
        SPCO_LAUNCH("clip_grads", c.st,
                    e = launch_dependent(clip_kernel<CAP, KIND>, dim3(t.blocks), dim3(kThreads), 0, c.st, t, o, parts, total,
                                         c.scale, c.max_norm, c.norm));
        SPECOPTIM_CUDA(e);
    }
    return SPECOPTIM_OK;
}

int run_call(const Call &c, bool clip, const char *what) {
    if (int rc = check_call(c, clip, what)) return rc;
    if (int rc = bind_device()) return rc;
    if (c.workspace_bytes < workspace_of(c.count))
        return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": the workspace is smaller than grad_norm_workspace() says");
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
