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
// written from the same registers.  What bounds both directions is the DRAM
// traffic.  Where rows are multiples of 16 bytes a group of 128 values lies in 16
// neighbouring lanes; otherwise (rowvec.cuh) a thread's 8 values may belong to
// two groups, and the groups' maxima meet in shared memory.
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
constexpr int kMaxThreads = 512, kMaxDim = kMaxThreads * 8 * 8, kMaxGroups = kMaxDim / kGroup;
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

// Columns col .. col + 7 of the row that begins at `row`, as far as they lie in
// [0, dim): a vector where the piece lies in the row and on a boundary.
template <typename T>
__device__ __forceinline__ void store_span(const Span<T> &s, int64_t row, int col, int dim, const float (&v)[8]) {
    if (((row + col) & 7) == 0) {
        store_any(s, row + col, row, row + dim, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (col + i >= 0 && col + i < dim) s.p[row + col + i] = from_f<T>(v[i]);
}
__device__ __forceinline__ void store_q8(const Span<uint8_t> &s, int64_t row, int col, int dim, uint2 v) {
    if (col >= 0 && col + 8 <= dim && ((row + col) & 7) == 0) {
        *reinterpret_cast<uint2 *>(s.p + row + col) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (col + i >= 0 && col + i < dim) s.p[row + col + i] = (uint8_t)((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
}

// largest magnitude of v[from..to), infinite where one of them is a NaN (fmaxf
// drops it): the group's scale then marks the group
__device__ __forceinline__ float magnitude(const float (&v)[8], int from, int to) {
    float m = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i < from || i >= to) continue;
        m = fmaxf(m, fabsf(v[i]));
        bad |= v[i] != v[i];
    }
    return bad ? __int_as_float(0x7f800000) : m;
}
__device__ __forceinline__ float scale_of(float m) { return fmaxf(m / kFp8Max, kTinyScale); }

__device__ __forceinline__ void unpack_q8(uint2 u, float (&v)[8]) {
    from_fp8x4(u.x, v);
    from_fp8x4(u.y, v + 4);
}

// The tensors of one call as spans, and their width.  All of a type that are 16
// byte aligned begin each row at the same place between two boundaries.
template <typename T> struct Forward {
    Span<const T> x, r, gamma;
    Span<T> s, y;
    Span<uint8_t> q;
    float *scale, *rstd;
    int64_t rows;
    int dim;
    float eps;
};

// q of the 8 values and their group's (or two groups') scales
__device__ __forceinline__ uint2 quantise8(const float (&s)[8], float inv_lo, float inv_hi, int cut) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = s[i] * (i < cut ? inv_lo : inv_hi);
    return make_uint2(to_fp8x4(t[0], t[1], t[2], t[3]), to_fp8x4(t[4], t[5], t[6], t[7]));
}

template <typename T, bool VEC, int NV>
__global__ void __launch_bounds__(512) resnorm_forward_kernel(const Forward<T> a) {
    __shared__ float red[2][32];
    __shared__ int group_max[VEC ? 1 : 3][VEC ? 1 : kMaxGroups + 1];
    const int dim = a.dim, groups = (dim + kGroup - 1) / kGroup;
    if (!VEC) {
        for (int i = threadIdx.x; i < 3 * (kMaxGroups + 1); i += blockDim.x) (&group_max[0][0])[i] = 0;
        __syncthreads();
    }
    int parity = 0, turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1, turn = turn == 2 ? 0 : turn + 1) {
        const int64_t base = row * dim;
        const int first = VEC ? 0 : -(int)((a.y.lo + base) & 7);  // column where the row's first piece begins
        float s[NV][8];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = first + (int)(k * blockDim.x + threadIdx.x) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) s[k][i] = 0.f;
            if (col >= dim) continue;
            if (VEC) load8(a.x.p + base + col, s[k]);
            else load_any(a.x, a.x.lo + base + col, s[k]);
        }
        if (a.r.p) {
            float b[NV][8];
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = first + (int)(k * blockDim.x + threadIdx.x) * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) b[k][i] = 0.f;
                if (col >= dim) continue;
                if (VEC) load8(a.r.p + base + col, b[k]);
                else load_any(a.r, a.r.lo + base + col, b[k]);
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = first + (int)(k * blockDim.x + threadIdx.x) * 8;
                // the stream is held in T: norm and checkpoint are those of the rounded sum
#pragma unroll
                for (int i = 0; i < 8; ++i) s[k][i] = to_f(from_f<T>(s[k][i] + b[k][i]));
                if (col >= dim) continue;
                if (VEC) store8(a.s.p + base + col, s[k]);
                else store_span(a.s, a.s.lo + base, col, dim, s[k]);
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = first + (int)(k * blockDim.x + threadIdx.x) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!VEC && (col + i < 0 || col + i >= dim)) s[k][i] = 0.f;  // the neighbouring rows' values
                ss = fmaf(s[k][i], s[k][i], ss);
            }
        }
        if (VEC) {
            // the checkpoint needs no row sum: it is written while the sum is under way
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * blockDim.x + threadIdx.x) * 8;
                float m = magnitude(s[k], 0, 8);
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                const float sc = scale_of(m), inv = 1.f / sc;
                if (col >= dim) continue;
                *reinterpret_cast<uint2 *>(a.q.p + a.q.lo + base + col) = quantise8(s[k], inv, inv, 8);
                if ((threadIdx.x & 15) == 0) a.scale[row * groups + col / kGroup] = sc;
            }
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = first + (int)(k * blockDim.x + threadIdx.x) * 8;
                if (col >= dim) continue;
                const int g = max(col, 0) / kGroup, cut = min(8, (g + 1) * kGroup - col);
                atomicMax(&group_max[turn][g], __float_as_int(magnitude(s[k], 0, cut)));
                if (cut < 8) atomicMax(&group_max[turn][g + 1], __float_as_int(magnitude(s[k], cut, 8)));
            }
            __syncwarp();  // one warp: block_sum has no barrier
        }
        ss = block_sum(ss, red[parity]);
        const float rs = 1.f / sqrtf(ss / (float)dim + a.eps);
        if (threadIdx.x == 0) a.rstd[row] = rs;
        if (!VEC) {
            // the previous row's maxima have been read by all; they are used again the row after next
            int *stale = group_max[turn == 0 ? 2 : turn - 1];
            for (int i = threadIdx.x; i < groups; i += blockDim.x) {
                stale[i] = 0;
                a.scale[row * groups + i] = scale_of(__int_as_float(group_max[turn][i]));
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = first + (int)(k * blockDim.x + threadIdx.x) * 8;
                if (col >= dim) continue;
                const int g = max(col, 0) / kGroup, cut = min(8, (g + 1) * kGroup - col);
                const float lo = 1.f / scale_of(__int_as_float(group_max[turn][g]));
                const float hi = cut < 8 ? 1.f / scale_of(__int_as_float(group_max[turn][g + 1])) : lo;
                store_q8(a.q, a.q.lo + base, col, dim, quantise8(s[k], lo, hi, cut));
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = first + (int)(k * blockDim.x + threadIdx.x) * 8;
            if (col >= dim) continue;
            float g[8];
            if (VEC) load8(a.gamma.p + col, g);
            else load_any(a.gamma, a.gamma.lo + col, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[k][i] = s[k][i] * rs * g[i];
            if (VEC) store8(a.y.p + base + col, s[k]);
            else store_span(a.y, a.y.lo + base, col, dim, s[k]);
        }
    }
}

template <typename T> struct Backward {
    Span<const T> dy, ds, gamma;
    Span<const uint8_t> q;
    const float *scale, *rstd;
    Span<T> dx, y;
    float *partial;
    int64_t rows;
    int dim, pitch;
};

// n of 8 values: q times the scale of their group (or two groups) times rstd, 0
// outside the row
template <bool VEC>
__device__ __forceinline__ void load_n(const Span<const uint8_t> &q, const float *scale, int64_t row, int groups,
                                       int col, int dim, float rs, float (&n)[8]) {
    const int64_t at = q.lo + row * dim + col;
    unpack_q8(VEC ? __ldg(reinterpret_cast<const uint2 *>(q.p + at)) : load_any8(q, at), n);
    const int g = VEC ? col / kGroup : max(col, 0) / kGroup, cut = VEC ? 8 : min(8, (g + 1) * kGroup - col);
    const float lo = __ldg(scale + row * groups + g);
    const float hi = !VEC && cut < 8 && g + 1 < groups ? __ldg(scale + row * groups + g + 1) : lo;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        n[i] = n[i] * (i < cut ? lo : hi) * rs;
        if (!VEC && (col + i < 0 || col + i >= dim)) n[i] = 0.f;
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) resnorm_recompute_kernel(const Backward<T> a) {
    const int dim = a.dim, groups = (dim + kGroup - 1) / kGroup;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rs = a.rstd[row];
        const int first = VEC ? 0 : -(int)((a.y.lo + row * dim) & 7);
        for (int col = first + (int)threadIdx.x * 8; col < dim; col += blockDim.x * 8) {
            float n[8], g[8];
            load_n<VEC>(a.q, a.scale, row, groups, col, dim, rs, n);
            if (VEC) load8(a.gamma.p + col, g);
            else load_any(a.gamma, a.gamma.lo + col, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] *= g[i];
            if (VEC) store8(a.y.p + row * dim + col, n);
            else store_span(a.y, a.y.lo + row * dim, col, dim, n);
        }
    }
}

// Each block keeps its columns' share of dgamma in registers over all its rows
// and writes it once, to partial[block][pitch].  Where rows begin at different
// places, a block's rows lie a multiple of 8 rows apart and so begin alike.
template <typename T, bool VEC, int NV>
__global__ void __launch_bounds__(512) resnorm_backward_kernel(const Backward<T> a) {
    __shared__ float red[2][32];
    const int dim = a.dim, groups = (dim + kGroup - 1) / kGroup;
    const int first = VEC ? 0 : -(int)((a.dx.lo + (int64_t)blockIdx.x * dim) & 7);
    float dg[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[k][i] = 0.f;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
        const int64_t base = row * dim;
        const float rs = a.rstd[row];
        float n[NV][8], d[NV][8];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = first + (int)(k * blockDim.x + threadIdx.x) * 8;
            if (col < dim) {
                if (VEC) load8(a.dy.p + base + col, d[k]);
                else load_any(a.dy, a.dy.lo + base + col, d[k]);
                load_n<VEC>(a.q, a.scale, row, groups, col, dim, rs, n[k]);
                if (!VEC) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (col + i < 0 || col + i >= dim) d[k][i] = 0.f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) d[k][i] = n[k][i] = 0.f;
            }
        }
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = first + (int)(k * blockDim.x + threadIdx.x) * 8;
            if (col >= dim) continue;
            float g[8];
            if (VEC) load8(a.gamma.p + col, g);  // stays in L1 over the rows
            else load_any(a.gamma, a.gamma.lo + col, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dg[k][i] = fmaf(d[k][i], n[k][i], dg[k][i]);
                d[k][i] *= g[i];
                t = fmaf(d[k][i], n[k][i], t);
                g[i] *= n[k][i];
            }
            if (!a.y.p) continue;
            if (VEC) store8(a.y.p + base + col, g);
            else store_span(a.y, a.y.lo + base, col, dim, g);
        }
        t = block_sum(t, red[parity]) / (float)dim;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = first + (int)(k * blockDim.x + threadIdx.x) * 8;
            if (col >= dim) continue;
            float b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (a.ds.p) {
                if (VEC) load8(a.ds.p + base + col, b);
                else load_any(a.ds, a.ds.lo + base + col, b);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = fmaf(rs, d[k][i] - n[k][i] * t, b[i]);
            if (VEC) store8(a.dx.p + base + col, b);
            else store_span(a.dx, a.dx.lo + base, col, dim, b);
        }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int col = first + (int)(k * blockDim.x + threadIdx.x) * 8;
        if (col >= dim) continue;
        float *out = a.partial + (int64_t)blockIdx.x * a.pitch;
        if (VEC) {
            store8(out + col, dg[k]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i >= 0 && col + i < dim) out[col + i] = dg[k][i];
        }
    }
}

// dgamma[j] = sum over blocks of partial[block][j]: 32 columns per block, 8
// threads per column, joined in a fixed order.
__global__ void __launch_bounds__(256) dgamma_kernel(const float *__restrict__ partial, int blocks, int dim,
                                                     int pitch, float *__restrict__ dgamma) {
    __shared__ float red[8][33];
    const int c = threadIdx.x & 31, w = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
    float a = 0.f;
    if (col < dim) {
#pragma unroll 8
        for (int b = w; b < blocks; b += 8) a += partial[(int64_t)b * pitch + col];
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
Shape shape_of(int dim, bool vec) {
    const int64_t vecs = vec ? dim / 8 : (dim + 14) / 8;  // 8-value pieces that a row can touch
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

// A multiple of 8 where there are that many rows (see resnorm_backward_kernel)
int backward_blocks(int64_t rows, const Shape &sh) {
    const int per_sm = std::max(1, std::min(kBackwardBlocksPerSm, 1024 / sh.threads));
    return (int)std::max<int64_t>(1, std::min<int64_t>(rows, (int64_t)num_sms() * per_sm / 8 * 8));
}

int check_sizes(int64_t rows, int32_t dim, int32_t type, const char *what) {
    if (rows < 0 || rows > INT32_MAX)
        return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": rows outside [0, 2^31)");
    if (dim < 1 || dim > kMaxDim) return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": dim outside [1, 32768]");
    if (!type_ok(type))
        return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": type must be STAGE_BF16 or STAGE_FP32");
    return SPECOPTIM_OK;
}

template <typename T> int run_forward(const Shape &sh, bool vec, const Forward<T> &a, cudaStream_t st) {
    return with_nv(sh.nv, [&](auto nv) -> int {
        constexpr int NV = decltype(nv)::value;
        const int grid = (int)std::min<int64_t>(a.rows, (int64_t)num_sms() * 64);
        auto *k = vec ? &resnorm_forward_kernel<T, true, NV> : &resnorm_forward_kernel<T, false, NV>;
        SPCO_LAUNCH("resnorm_forward", st, k<<<grid, sh.threads, 0, st>>>(a));
        SPECOPTIM_LAUNCHED("resnorm_forward_kernel");
        return SPECOPTIM_OK;
    });
}

template <typename T>
int run_backward(const Shape &sh, bool vec, int blocks, const Backward<T> &a, float *dgamma, cudaStream_t st) {
    return with_nv(sh.nv, [&](auto nv) -> int {
        constexpr int NV = decltype(nv)::value;
        auto *k = vec ? &resnorm_backward_kernel<T, true, NV> : &resnorm_backward_kernel<T, false, NV>;
        SPCO_LAUNCH("resnorm_backward", st, k<<<blocks, sh.threads, 0, st>>>(a));
        SPECOPTIM_LAUNCHED("resnorm_backward_kernel");
        SPCO_LAUNCH("resnorm_dgamma", st,
                    dgamma_kernel<<<(unsigned)ceil_div(a.dim, 32), 256, 0, st>>>(a.partial, blocks, a.dim, a.pitch, dgamma));
        SPECOPTIM_LAUNCHED("dgamma_kernel");
        return SPECOPTIM_OK;
    });
}

// f(T{}) for the tensors' type
template <typename F> int with_type(int32_t type, F &&f) { return type == STAGE_BF16 ? f(bf16{}) : f(float{}); }

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
        const Shape sh = shape_of(dim, vec);
        const int64_t n = rows * dim;
        return with_type(type, [&](auto t) -> int {
            using T = decltype(t);
            const Forward<T> a{{static_cast<const T *>(x), n},
                               {static_cast<const T *>(r), n},
                               {static_cast<const T *>(gamma), dim},
                               {static_cast<T *>(s), n},
                               {static_cast<T *>(y), n},
                               {static_cast<uint8_t *>(q), n},
                               scale,
                               rstd,
                               rows,
                               dim,
                               eps};
            return run_forward<T>(sh, vec, a, static_cast<cudaStream_t>(stream));
        });
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
        const int threads = (int)std::min<int64_t>(256, round_up(ceil_div(dim + 7, 8), 32));
        const int grid = (int)std::min<int64_t>(rows, (int64_t)num_sms() * 64);
        const int64_t n = rows * dim;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        return with_type(type, [&](auto t) -> int {
            using T = decltype(t);
            const Backward<T> a{{nullptr, 0},
                                {nullptr, 0},
                                {static_cast<const T *>(gamma), dim},
                                {static_cast<const uint8_t *>(q), n},
                                scale,
                                rstd,
                                {nullptr, 0},
                                {static_cast<T *>(y), n},
                                nullptr,
                                rows,
                                dim,
                                dim};
            auto *k = vec ? &resnorm_recompute_kernel<T, true> : &resnorm_recompute_kernel<T, false>;
            SPCO_LAUNCH("resnorm_recompute", st, k<<<grid, threads, 0, st>>>(a));
            SPECOPTIM_LAUNCHED("resnorm_recompute_kernel");
            return SPECOPTIM_OK;
        });
    });
}

extern "C" int64_t resnorm_backward_workspace(int64_t rows, int32_t dim) {
    int64_t bytes = -1;
    entry([&]() -> int {
        if (int rc = check_sizes(rows, dim, STAGE_BF16, "resnorm_backward")) return rc;
        // of the two shapes the one with more blocks: the pointers' alignment is not known yet
        bytes = (int64_t)std::max(backward_blocks(rows, shape_of(dim, true)), backward_blocks(rows, shape_of(dim, false))) *
                round_up(dim, 8) * 4;
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
        const bool vec = dim % 8 == 0 && aligned16(dy) && aligned16(ds) && aligned16(gamma) && aligned16(dx) &&
                         aligned16(y) && aligned_to(q, 8);
        const Shape sh = shape_of(dim, vec);
        const int blocks = backward_blocks(rows, sh), pitch = (int)round_up(dim, 8);
        if (workspace_bytes < (int64_t)blocks * pitch * 4)
            return fail(SPECOPTIM_ERR_INVALID_ARG, "resnorm_backward: the workspace is smaller than resnorm_backward_workspace() says");
        if (int rc = bind_device()) return rc;
        const int64_t n = rows * dim;
        return with_type(type, [&](auto t) -> int {
            using T = decltype(t);
            const Backward<T> a{{static_cast<const T *>(dy), n},
                                {static_cast<const T *>(ds), n},
                                {static_cast<const T *>(gamma), dim},
                                {static_cast<const uint8_t *>(q), n},
                                scale,
                                rstd,
                                {static_cast<T *>(dx), n},
                                {static_cast<T *>(y), n},
                                static_cast<float *>(workspace),
                                rows,
                                dim,
                                pitch};
            return run_backward<T>(sh, vec, blocks, a, dgamma, static_cast<cudaStream_t>(stream));
        });
    });
}
