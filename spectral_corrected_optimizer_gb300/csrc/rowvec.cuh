// Row vectors of the stage-end operators: 8 consecutive values of a row as
// floats; argument checks and the exception guard of their entries.
//
// Where rows are multiples of 16 bytes (VEC), a thread's 8 values are one or two
// 16-byte accesses.  Otherwise every row starts at another place between two
// 16-byte boundaries: the threads then take the 8-value pieces of memory that
// the row's output lies in (its first piece begins up to 7 values before the
// row), store whole pieces as vectors and only the row's two ends value by
// value, and read their inputs as the two pieces around them, shifted into
// place (Span::load).
#pragma once

#include <cuda_bf16.h>

#include <exception>

#include "../../include/stage_ends.h"
#include "common.cuh"

namespace spco {

using bf16 = __nv_bfloat16;

// What a kernel writes to the stage-end operators' device flag when it skips an
// id outside the vocabulary, or moves a sequence's offset into the tokens;
// read_stage_flag() and check_stage_flag() (embed.cu) read and clear it.
constexpr unsigned kSiteTokenId = 1, kSiteTarget = 2, kSiteOffset = 3;
unsigned *stage_flag_ptr();

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ bf16 from_f<bf16>(float x) { return __float2bfloat16_rn(x); }

// two bf16 values from the low and the high half of a word, and back (nearest even)
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Loads are plain ones, not read-only: callers read what the launch before them wrote while
// they were resident already, and pieces of which other threads write their own part (in-place
// calls, sums that are added to).  kLasting: nobody writes the tensor while the kernel is
// resident, so loads may be moved ahead of the kernel's stores (65536 rows of dy summed by id:
// 248 us with, 341 without).
constexpr bool kLasting = true;
template <bool LASTING, typename V> __device__ __forceinline__ V load_piece(const V *p) { return LASTING ? __ldg(p) : *p; }

// p[0..7] of a 16-byte aligned address
template <bool LASTING = false> __device__ __forceinline__ void load8(const bf16 *p, float (&v)[8]) {
    const uint4 u = load_piece<LASTING>(reinterpret_cast<const uint4 *>(p));
    v[0] = lo_f(u.x); v[1] = hi_f(u.x); v[2] = lo_f(u.y); v[3] = hi_f(u.y);
    v[4] = lo_f(u.z); v[5] = hi_f(u.z); v[6] = lo_f(u.w); v[7] = hi_f(u.w);
}
template <bool LASTING = false> __device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 *q = reinterpret_cast<const float4 *>(p);
    const float4 a = load_piece<LASTING>(q), b = load_piece<LASTING>(q + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(bf16 *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                               pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A tensor of `count` values as 16-byte pieces: `p` is its address rounded down to
// 16 bytes, its values have the indexes [lo, hi) from there.
template <typename T> struct Span {
    T *p;
    int64_t lo, hi;

    __host__ __device__ Span(T *q, int64_t count) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(q);
        p = reinterpret_cast<T *>(a & ~uintptr_t(15));
        lo = (int64_t)((a & 15) / sizeof(T));
        hi = lo + count;
    }
    __host__ __device__ Span(T *base, int64_t from, int64_t to) : p(base), lo(from), hi(to) {}
    __host__ __device__ Span<const T> read() const { return Span<const T>(p, lo, hi); }
};

// words o .. o + 3 (o < 4) of 8
__device__ __forceinline__ void pick_words(const uint32_t (&w)[8], int o, uint32_t (&r)[5]) {
    uint32_t t[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) t[i] = (o & 2) ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) r[i] = (o & 1) ? t[i + 1] : t[i];
}

// values i .. i + 7 of the span; 0 outside it
template <bool LASTING = false>
__device__ __forceinline__ void load_any(const Span<const bf16> &s, int64_t i, float (&v)[8]) {
    const int64_t a = i & ~(int64_t)7;
    const int sh = (int)(i & 7);
    if (a >= s.lo && a + (sh ? 16 : 8) <= s.hi) {
        const uint4 *q = reinterpret_cast<const uint4 *>(s.p + a);
        const uint4 x = load_piece<LASTING>(q);
        uint32_t r[5] = {x.x, x.y, x.z, x.w, 0};
        if (sh) {
            const uint4 y = load_piece<LASTING>(q + 1);
            const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            pick_words(w, sh >> 1, r);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t u = (sh & 1) ? __funnelshift_r(r[k], r[k + 1], 16) : r[k];
            v[2 * k] = lo_f(u);
            v[2 * k + 1] = hi_f(u);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = i + k >= s.lo && i + k < s.hi ? to_f(s.p[i + k]) : 0.f;
}
template <bool LASTING = false>
__device__ __forceinline__ void load_any(const Span<const float> &s, int64_t i, float (&v)[8]) {
    const int64_t a = i & ~(int64_t)3;
    const int sh = (int)(i & 3);
    if (a >= s.lo && a + (sh ? 12 : 8) <= s.hi) {
        const float4 *q = reinterpret_cast<const float4 *>(s.p + a);
        const float4 x = load_piece<LASTING>(q), y = load_piece<LASTING>(q + 1);
        float w[12] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, 0.f, 0.f, 0.f, 0.f};
        if (sh) {
            const float4 z = load_piece<LASTING>(q + 2);
            w[8] = z.x; w[9] = z.y; w[10] = z.z; w[11] = z.w;
        }
        float t[10];
#pragma unroll
        for (int k = 0; k < 10; ++k) t[k] = (sh & 2) ? w[k + 2] : w[k];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = (sh & 1) ? t[k + 1] : t[k];
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = i + k >= s.lo && i + k < s.hi ? s.p[i + k] : 0.f;
}
// 8 bytes, packed
__device__ __forceinline__ uint2 load_any8(const Span<const uint8_t> &s, int64_t i) {
    const int64_t a = i & ~(int64_t)7;
    const int sh = (int)(i & 7);
    if (a >= s.lo && a + (sh ? 16 : 8) <= s.hi) {
        const uint2 *q = reinterpret_cast<const uint2 *>(s.p + a);
        const uint2 x = q[0];
        if (!sh) return x;
        const uint2 y = q[1];
        const uint32_t w0 = (sh & 4) ? x.y : x.x, w1 = (sh & 4) ? y.x : x.y, w2 = (sh & 4) ? y.y : y.x;
        return make_uint2(__funnelshift_r(w0, w1, 8 * (sh & 3)), __funnelshift_r(w1, w2, 8 * (sh & 3)));
    }
    uint32_t u[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (i + k >= s.lo && i + k < s.hi) u[k / 4] |= (uint32_t)s.p[i + k] << (8 * (k & 3));
    return make_uint2(u[0], u[1]);
}

// v to i .. i + 7 of those that lie in [from, to); i is a multiple of 8
template <typename T>
__device__ __forceinline__ void store_any(const Span<T> &s, int64_t i, int64_t from, int64_t to, const float (&v)[8]) {
    if (i >= from && i + 8 <= to) {
        store8(s.p + i, v);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (i + k >= from && i + k < to) s.p[i + k] = from_f<T>(v[k]);
}

inline size_t type_bytes(int32_t type) { return type == STAGE_BF16 ? 2 : 4; }
inline bool type_ok(int32_t type) { return type == STAGE_BF16 || type == STAGE_FP32; }
inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline int64_t ceil_div(int64_t x, int64_t m) { return (x + m - 1) / m; }

// A launch that may begin while the one before it on the stream is finishing: its
// kernel waits (grid_dependency_wait) before it touches what that one wrote, and
// that one says early (grid_dependency_launch) that its successor may begin.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A &&...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Nothing is thrown across the C boundary: an exception (out of host memory in
// a message or a table) becomes a status.
template <typename F> int entry(F &&f) {
    try {
        clear_error();
        return f();
    } catch (const std::exception &) {
        return SPECOPTIM_ERR_CUDA;
    } catch (...) {
        return SPECOPTIM_ERR_CUDA;
    }
}

}  // namespace spco
