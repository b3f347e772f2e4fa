// Row vectors of the stage-end operators: 8 consecutive values of a row as
// floats, loaded and stored in 16-byte pieces where the tensor allows it, value
// by value otherwise; argument checks and the exception guard of their entries.
#pragma once

#include <cuda_bf16.h>

#include <exception>

#include "../../include/stage_ends.h"
#include "common.cuh"

namespace spco {

using bf16 = __nv_bfloat16;

// bit 31 marks a failed index check; these sites are ids outside the vocabulary
constexpr unsigned kSiteTokenId = 0x80000040u, kSiteTarget = 0x80000041u;

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

// v = p[0..7] (positions >= n are 0); VEC: p is 16-byte aligned and n >= 8
template <bool VEC> __device__ __forceinline__ void load8(const bf16 *p, int n, float (&v)[8]) {
    if (VEC) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
        v[0] = lo_f(u.x); v[1] = hi_f(u.x); v[2] = lo_f(u.y); v[3] = hi_f(u.y);
        v[4] = lo_f(u.z); v[5] = hi_f(u.z); v[6] = lo_f(u.w); v[7] = hi_f(u.w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f(p[i]) : 0.f;
    }
}
template <bool VEC> __device__ __forceinline__ void load8(const float *p, int n, float (&v)[8]) {
    if (VEC) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
    }
}
template <bool VEC> __device__ __forceinline__ void store8(bf16 *p, int n, const float (&v)[8]) {
    if (VEC) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                   pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = from_f<bf16>(v[i]);
    }
}
template <bool VEC> __device__ __forceinline__ void store8(float *p, int n, const float (&v)[8]) {
    if (VEC) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
}

inline size_t type_bytes(int32_t type) { return type == STAGE_BF16 ? 2 : 4; }
inline bool type_ok(int32_t type) { return type == STAGE_BF16 || type == STAGE_FP32; }
inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline int64_t ceil_div(int64_t x, int64_t m) { return (x + m - 1) / m; }

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
