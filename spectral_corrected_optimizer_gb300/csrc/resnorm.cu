// Residual sum + RMSNorm with an 8-bit checkpoint of the sum, and the backward
// pass from that checkpoint (include/stage_ends.h).
//
//   forward   s = x + r,  rstd = 1 / sqrt(mean s^2 + eps),  y = s rstd gamma,
//             per group of 128: scale = max(amax / 448, 2^-126), q = e4m3(s / scale)
//   backward  n = q scale rstd,  dx = ds + rstd (gamma dy - n mean(gamma dy n)),
//             dgamma = sum over rows of dy n,  y = n gamma
//
// All of it is one pass over the data: a block holds a row in registers (8
// values per thread and step), so the row is read once, its mean square and
// its groups' maxima are reduced by shuffles, and everything derived from it is
// written from the same registers.  A group of 128 values lies in 16
// neighbouring lanes.  What bounds both directions is the DRAM traffic.
//
// The norm statistics and every sum are fp32.  The checkpoint is the only
// tensor below 16 bits: e4m3 with a scale per 128 values keeps each value to
// 2^-4 of itself, or 2^-10 of the group's scale where that is more.
#include <cuda_fp8.h>

#include <algorithm>
#include <string>

#include "rowvec.cuh"

namespace spco {
namespace {

constexpr int kGroup = STAGE_CKPT_GROUP;
constexpr float kFp8Max = 448.f;
constexpr float kTinyScale = 1.17549435e-38f;  // 2^-126: its reciprocal is finite

// Sum over the block of one value per thread, to all threads, in a fixed order.
// `red` is one buffer of 32 floats per call site and parity of the loop, so one
// barrier is enough.
__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < warps; ++i) v += red[i];
    return v;
}

__device__ __forceinline__ uint32_t to_fp8x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ void from_fp8x4(uint32_t u, float *v) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> (16 * i)), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

template <bool VEC> __device__ __forceinline__ void load_q8(const uint8_t *p, int n, float (&v)[8]) {
    uint32_t u[2] = {0, 0};
    if (VEC) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
        u[0] = w.x;
        u[1] = w.y;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) u[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
    }
    from_fp8x4(u[0], v);
    from_fp8x4(u[1], v + 4);
}

template <bool VEC> __device__ __forceinline__ void store_q8(uint8_t *p, int n, uint32_t lo, uint32_t hi) {
    if (VEC) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
}

template <typename T, bool VEC, int NV>
__global__ void __launch_bounds__(512) resnorm_forward_kernel(
    const T *x, const T *r, const T *__restrict__ gamma, float eps, T *s_out, T *__restrict__ y,
    uint8_t *__restrict__ q, float *__restrict__ scale, float *__restrict__ rstd, int64_t rows, int dim) {
    __shared__ float red[2][32];
    const int groups = (dim + kGroup - 1) / kGroup;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, parity ^= 1) {
        const int64_t base = row * dim;
        float s[NV][8];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = (k * blockDim.x + threadIdx.x) * 8;
            if (col < dim) {
                load8<VEC>(x + base + col, dim - col, s[k]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) s[k][i] = 0.f;
            }
        }
        if (r) {
            float b[NV][8];
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * blockDim.x + threadIdx.x) * 8;
                if (col < dim) {
                    load8<VEC>(r + base + col, dim - col, b[k]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) b[k][i] = 0.f;
                }
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * blockDim.x + threadIdx.x) * 8;
                // the stream is held in T: norm and checkpoint are those of the rounded sum
#pragma unroll
                for (int i = 0; i < 8; ++i) s[k][i] = to_f(from_f<T>(s[k][i] + b[k][i]));
                if (col < dim) store8<VEC>(s_out + base + col, dim - col, s[k]);
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(s[k][i], s[k][i], ss);
        // the checkpoint needs no row sum: it is written while the sum is under way
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = (k * blockDim.x + threadIdx.x) * 8;
            float m = 0.f;
            bool bad = false;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m = fmaxf(m, fabsf(s[k][i]));
                bad |= s[k][i] != s[k][i];
            }
            if (bad) m = __int_as_float(0x7f800000);  // fmaxf drops NaN: an infinite scale marks the group
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float sc = fmaxf(m / kFp8Max, kTinyScale);
            const float inv = 1.f / sc;
            if (col < dim) {
                const uint32_t lo = to_fp8x4(s[k][0] * inv, s[k][1] * inv, s[k][2] * inv, s[k][3] * inv);
                const uint32_t hi = to_fp8x4(s[k][4] * inv, s[k][5] * inv, s[k][6] * inv, s[k][7] * inv);
                store_q8<VEC>(q + base + col, dim - col, lo, hi);
                if ((threadIdx.x & 15) == 0) scale[row * groups + col / kGroup] = sc;
            }
        }
        ss = block_sum(ss, red[parity]);
        const float rs = 1.f / sqrtf(ss / (float)dim + eps);
        if (threadIdx.x == 0) rstd[row] = rs;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = (k * blockDim.x + threadIdx.x) * 8;
            if (col >= dim) continue;
            float g[8];
            load8<VEC>(gamma + col, dim - col, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[k][i] = s[k][i] * rs * g[i];
            store8<VEC>(y + base + col, dim - col, s[k]);
        }
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) resnorm_recompute_kernel(const uint8_t *__restrict__ q,
                                                                const float *__restrict__ scale,
                                                                const float *__restrict__ rstd,
                                                                const T *__restrict__ gamma, T *__restrict__ y,
                                                                int64_t rows, int dim) {
    const int vecs = (dim + 7) / 8, groups = (dim + kGroup - 1) / kGroup;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const float rs = rstd[row];
        for (int v = threadIdx.x; v < vecs; v += blockDim.x) {
            const int col = v * 8;
            const float sc = scale[row * groups + col / kGroup];
            float n[8], g[8];
            load_q8<VEC>(q + row * dim + col, dim - col, n);
            load8<VEC>(gamma + col, dim - col, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] = n[i] * sc * rs * g[i];
            store8<VEC>(y + row * dim + col, dim - col, n);
        }
    }
}

// Each block keeps its columns' share of dgamma in registers over all its rows
// and writes it once, to partial[block][dim].
template <typename T, bool VEC, int NV>
__global__ void __launch_bounds__(512) resnorm_backward_kernel(
    const T *dy, const T *ds, const uint8_t *__restrict__ q, const float *__restrict__ scale,
    const float *__restrict__ rstd, const T *__restrict__ gamma, T *dx, T *__restrict__ y,
    float *__restrict__ partial, int64_t rows, int dim) {
    __shared__ float red[2][32];
    const int groups = (dim + kGroup - 1) / kGroup;
    float dg[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[k][i] = 0.f;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, parity ^= 1) {
        const int64_t base = row * dim;
        const float rs = rstd[row];
        float n[NV][8], d[NV][8];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = (k * blockDim.x + threadIdx.x) * 8;
            if (col < dim) {
                load8<VEC>(dy + base + col, dim - col, d[k]);
                load_q8<VEC>(q + base + col, dim - col, n[k]);
                const float sc = scale[row * groups + col / kGroup];
#pragma unroll
                for (int i = 0; i < 8; ++i) n[k][i] = n[k][i] * sc * rs;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) d[k][i] = n[k][i] = 0.f;
            }
        }
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = (k * blockDim.x + threadIdx.x) * 8;
            if (col >= dim) continue;
            float g[8];
            load8<VEC>(gamma + col, dim - col, g);  // stays in L1 over the rows
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dg[k][i] = fmaf(d[k][i], n[k][i], dg[k][i]);
                d[k][i] *= g[i];
                t = fmaf(d[k][i], n[k][i], t);
                g[i] *= n[k][i];
            }
            if (y) store8<VEC>(y + base + col, dim - col, g);
        }
        t = block_sum(t, red[parity]) / (float)dim;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = (k * blockDim.x + threadIdx.x) * 8;
            if (col >= dim) continue;
            float b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (ds) load8<VEC>(ds + base + col, dim - col, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = fmaf(rs, d[k][i] - n[k][i] * t, b[i]);
            store8<VEC>(dx + base + col, dim - col, b);
        }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int col = (k * blockDim.x + threadIdx.x) * 8;
        if (col < dim) store8<VEC>(partial + (int64_t)blockIdx.x * dim + col, dim - col, dg[k]);
    }
}

// dgamma[j] = sum over blocks of partial[block][j]: 32 columns per block, 8
// threads per column, joined in a fixed order.
__global__ void __launch_bounds__(256) dgamma_kernel(const float *__restrict__ partial, int blocks, int dim,
                                                     float *__restrict__ dgamma) {
    __shared__ float red[8][33];
    const int c = threadIdx.x & 31, w = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
    float a = 0.f;
    if (col < dim) {
#pragma unroll 8
        for (int b = w; b < blocks; b += 8) a += partial[(int64_t)b * dim + col];
    }
    red[w][c] = a;
    __syncthreads();
    if (w == 0 && col < dim) {
        for (int i = 1; i < 8; ++i) a += red[i][c];
        dgamma[col] = a;
    }
}

// Values per thread: 16 (NV = 2) up to a width of 8192, so that a row of 2048
// takes 4 warps and many rows are in flight on an SM; then 32 and 64.
struct Shape {
    int nv, threads;
};
constexpr int kMaxThreads = 512, kMaxDim = kMaxThreads * 8 * 8;
Shape shape_of(int dim) {
    const int64_t vecs = ceil_div(dim, 8);
    int nv = 1;
    while (nv < 8 && (vecs > kMaxThreads * nv || (nv < 2 && vecs > 32))) nv *= 2;
    return {nv, (int)round_up(ceil_div(vecs, nv), 32)};
}

template <typename F> int with_nv(int nv, F &&f) {
    switch (nv) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        default: return f(std::integral_constant<int, 8>{});
    }
}

constexpr int kBackwardBlocksPerSm = 8;

int backward_blocks(int64_t rows, const Shape &sh) {
    const int per_sm = std::max(1, std::min(kBackwardBlocksPerSm, 1024 / sh.threads));
    return (int)std::max<int64_t>(1, std::min<int64_t>(rows, (int64_t)num_sms() * per_sm));
}

int check_sizes(int64_t rows, int32_t dim, int32_t type, const char *what) {
    if (rows < 0 || rows > INT32_MAX)
        return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": rows outside [0, 2^31)");
    if (dim < 1 || dim > kMaxDim) return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": dim outside [1, 32768]");
    if (!type_ok(type))
        return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": type must be STAGE_BF16 or STAGE_FP32");
    return SPECOPTIM_OK;
}

template <typename T>
int run_forward(const Shape &sh, bool vec, const void *x, const void *r, const void *gamma, float eps, void *s, void *y,
                void *q, float *scale, float *rstd, int64_t rows, int dim, cudaStream_t st) {
    return with_nv(sh.nv, [&](auto nv) -> int {
        constexpr int NV = decltype(nv)::value;
        const int grid = (int)std::min<int64_t>(rows, (int64_t)num_sms() * 64);
        auto *k = vec ? &resnorm_forward_kernel<T, true, NV> : &resnorm_forward_kernel<T, false, NV>;
        SPCO_LAUNCH("resnorm_forward", st,
                    k<<<grid, sh.threads, 0, st>>>(static_cast<const T *>(x), static_cast<const T *>(r),
                                                   static_cast<const T *>(gamma), eps, static_cast<T *>(s),
                                                   static_cast<T *>(y), static_cast<uint8_t *>(q), scale, rstd, rows,
                                                   dim));
        SPECOPTIM_LAUNCHED("resnorm_forward_kernel");
        return SPECOPTIM_OK;
    });
}

template <typename T>
int run_backward(const Shape &sh, bool vec, int blocks, const void *dy, const void *ds, const void *q,
                 const float *scale, const float *rstd, const void *gamma, void *dx, float *dgamma, void *y,
                 int64_t rows, int dim, float *partial, cudaStream_t st) {
    return with_nv(sh.nv, [&](auto nv) -> int {
        constexpr int NV = decltype(nv)::value;
        auto *k = vec ? &resnorm_backward_kernel<T, true, NV> : &resnorm_backward_kernel<T, false, NV>;
        SPCO_LAUNCH("resnorm_backward", st,
                    k<<<blocks, sh.threads, 0, st>>>(static_cast<const T *>(dy), static_cast<const T *>(ds),
                                                     static_cast<const uint8_t *>(q), scale, rstd,
                                                     static_cast<const T *>(gamma), static_cast<T *>(dx),
                                                     static_cast<T *>(y), partial, rows, dim));
        SPECOPTIM_LAUNCHED("resnorm_backward_kernel");
        SPCO_LAUNCH("resnorm_dgamma", st,
                    dgamma_kernel<<<(unsigned)ceil_div(dim, 32), 256, 0, st>>>(partial, blocks, dim, dgamma));
        SPECOPTIM_LAUNCHED("dgamma_kernel");
        return SPECOPTIM_OK;
    });
}

}  // namespace
}  // namespace spco

using namespace spco;

extern "C" int resnorm_forward(const void *x, const void *r, const void *gamma, int32_t type, float eps, void *s,
                               void *y, void *q, float *scale, float *rstd, int64_t rows, int32_t dim, void *stream) {
    return entry([&]() -> int {
        if (int rc = check_sizes(rows, dim, type, "resnorm_forward")) return rc;
        if (!(eps >= 0.f)) return fail(SPECOPTIM_ERR_INVALID_ARG, "resnorm_forward: eps must be >= 0");
        if (rows == 0) return SPECOPTIM_OK;
        if (!x || !gamma || !y || !q || !scale || !rstd || (r && !s))
            return fail(SPECOPTIM_ERR_INVALID_ARG, "resnorm_forward: null pointer");
        const size_t b = type_bytes(type);
        if (!aligned_to(x, b) || !aligned_to(r, b) || !aligned_to(gamma, b) || !aligned_to(s, b) || !aligned_to(y, b) ||
            !aligned_to(scale, 4) || !aligned_to(rstd, 4))
            return fail(SPECOPTIM_ERR_MISALIGNED, "resnorm_forward: pointers must be aligned to their elements");
        if (int rc = bind_device()) return rc;
        const bool vec = dim % 8 == 0 && aligned16(x) && aligned16(r) && aligned16(gamma) && aligned16(y) &&
                         (!r || aligned16(s)) && aligned_to(q, 8);
        const Shape sh = shape_of(dim);
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        return type == STAGE_BF16 ? run_forward<bf16>(sh, vec, x, r, gamma, eps, s, y, q, scale, rstd, rows, dim, st)
                                  : run_forward<float>(sh, vec, x, r, gamma, eps, s, y, q, scale, rstd, rows, dim, st);
    });
}

extern "C" int resnorm_recompute(const void *q, const float *scale, const float *rstd, const void *gamma, int32_t type,
                                 void *y, int64_t rows, int32_t dim, void *stream) {
    return entry([&]() -> int {
        if (int rc = check_sizes(rows, dim, type, "resnorm_recompute")) return rc;
        if (rows == 0) return SPECOPTIM_OK;
        if (!q || !scale || !rstd || !gamma || !y)
            return fail(SPECOPTIM_ERR_INVALID_ARG, "resnorm_recompute: null pointer");
        const size_t b = type_bytes(type);
        if (!aligned_to(gamma, b) || !aligned_to(y, b) || !aligned_to(scale, 4) || !aligned_to(rstd, 4))
            return fail(SPECOPTIM_ERR_MISALIGNED, "resnorm_recompute: pointers must be aligned to their elements");
        if (int rc = bind_device()) return rc;
        const bool vec = dim % 8 == 0 && aligned16(gamma) && aligned16(y) && aligned_to(q, 8);
        const int threads = (int)std::min<int64_t>(256, round_up(ceil_div(dim, 8), 32));
        const int grid = (int)std::min<int64_t>(rows, (int64_t)num_sms() * 64);
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        auto go = [&](auto t) -> int {
            using T = decltype(t);
            auto *k = vec ? &resnorm_recompute_kernel<T, true> : &resnorm_recompute_kernel<T, false>;
            SPCO_LAUNCH("resnorm_recompute", st,
                        k<<<grid, threads, 0, st>>>(static_cast<const uint8_t *>(q), scale, rstd,
                                                    static_cast<const T *>(gamma), static_cast<T *>(y), rows, dim));
            SPECOPTIM_LAUNCHED("resnorm_recompute_kernel");
            return SPECOPTIM_OK;
        };
        return type == STAGE_BF16 ? go(bf16{}) : go(float{});
    });
}

extern "C" int64_t resnorm_backward_workspace(int64_t rows, int32_t dim) {
    int64_t bytes = -1;
    entry([&]() -> int {
        if (int rc = check_sizes(rows, dim, STAGE_BF16, "resnorm_backward")) return rc;
        bytes = (int64_t)backward_blocks(rows, shape_of(dim)) * dim * 4;
        return SPECOPTIM_OK;
    });
    return bytes;
}

extern "C" int resnorm_backward(const void *dy, const void *ds, const void *q, const float *scale, const float *rstd,
                                const void *gamma, int32_t type, void *dx, float *dgamma, void *y, int64_t rows,
                                int32_t dim, void *workspace, int64_t workspace_bytes, void *stream) {
    return entry([&]() -> int {
        if (int rc = check_sizes(rows, dim, type, "resnorm_backward")) return rc;
        if (!gamma || !dgamma || !workspace || (rows > 0 && (!dy || !q || !scale || !rstd || !dx)))
            return fail(SPECOPTIM_ERR_INVALID_ARG, "resnorm_backward: null pointer");
        const size_t b = type_bytes(type);
        if (!aligned_to(dy, b) || !aligned_to(ds, b) || !aligned_to(gamma, b) || !aligned_to(dx, b) ||
            !aligned_to(y, b) || !aligned_to(scale, 4) || !aligned_to(rstd, 4) || !aligned_to(dgamma, 4) ||
            !aligned16(workspace))
            return fail(SPECOPTIM_ERR_MISALIGNED, "resnorm_backward: pointers must be aligned to their elements, the workspace to 16 bytes");
        const Shape sh = shape_of(dim);
        const int blocks = backward_blocks(rows, sh);
        if (workspace_bytes < (int64_t)blocks * dim * 4)
            return fail(SPECOPTIM_ERR_INVALID_ARG, "resnorm_backward: the workspace is smaller than resnorm_backward_workspace() says");
        if (int rc = bind_device()) return rc;
        const bool vec = dim % 8 == 0 && aligned16(dy) && aligned16(ds) && aligned16(gamma) && aligned16(dx) &&
                         aligned16(y) && aligned_to(q, 8);
        float *partial = static_cast<float *>(workspace);
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        return type == STAGE_BF16
                   ? run_backward<bf16>(sh, vec, blocks, dy, ds, q, scale, rstd, gamma, dx, dgamma, y, rows, dim, partial, st)
                   : run_backward<float>(sh, vec, blocks, dy, ds, q, scale, rstd, gamma, dx, dgamma, y, rows, dim, partial, st);
    });
}
