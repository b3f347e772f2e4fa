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
// written from the same registers.  The backward pass reads the next row while
// it works on one.  What bounds both directions is the DRAM traffic.
//
// Rows that are not multiples of 16 bytes (rowvec.cuh) are cut where memory is,
// not where the row is: a thread's 8 values are one 16-byte piece of the
// tensors (32 bytes in fp32), whose first `ph` values may belong to the row in
// front.  A block's rows lie a multiple of 8 rows apart, so ph is the same for
// all of them.  16 neighbouring threads then hold a group of 128 values, except
// that its last ph values are the first ph of the next 16 threads' first piece:
// those two maxima meet in shared memory.
//
// Measured on a GB300 (copy bandwidth 6.78 TB/s), bf16 [65536][2048] with a residual:
//   forward 182 us, 6.66 TB/s of x, r, s, y and the checkpoint (1.21 GB): 98 % of a copy;
//   backward with y 214 us, 5.65 TB/s (83 %): issue slots 55 % busy, 32 warps an SM; a
//     row's chain of shuffles, barrier and stores is what is waited for.  Two rows at a
//     time (112 registers, half the warps) took 231 us.  Without ds and y 170 us; y alone,
//     from the checkpoint, 74 us.
// Odd rows cost more instructions than bytes (440 per 256 values against 240): norm of
// 9749 x 6030 109 us (44 at the copy's rate), backward of 30001 x 3001 271 us (120).
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
constexpr int kMaxThreads = 512, kMaxDim = kMaxThreads * 8 * 8;
// Pieces of 8 values per thread.  A row that begins between two 16-byte boundaries touches
// one piece more than it has: from 32762 values on it needs a ninth per thread.
constexpr int kMaxPieces = 9;
constexpr int kMaxHeads = kMaxThreads * kMaxPieces / 16;  // 16 threads' pieces in a row
static_assert(kMaxThreads * kMaxPieces >= (kMaxDim + 14) / 8, "the widest row at any place");
constexpr float kFp8Max = 448.f;
constexpr float kTinyScale = 1.17549435e-38f;  // 2^-126: its reciprocal is finite

// Sum over the block of one value per thread, to all threads, in a fixed order.
// `red` holds one value per warp and zeros behind them (at most 16 warps), a
// buffer per parity of the loop, so one barrier is enough.
constexpr int kMaxWarps = kMaxThreads / 32;
struct BlockSum {
    float (*red)[kMaxWarps];
    int warps;

    __device__ __forceinline__ void init() const {
        for (int i = threadIdx.x; i < 2 * kMaxWarps; i += blockDim.x) (&red[0][0])[i] = 0.f;
        __syncthreads();
    }
    __device__ __forceinline__ float operator()(float v, int parity) const {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (warps == 1) return v;
        if ((threadIdx.x & 31) == 0) red[parity][threadIdx.x >> 5] = v;
        __syncthreads();
        const float4 *r = reinterpret_cast<const float4 *>(red[parity]);
        float4 a = r[0];
#pragma unroll
        for (int i = 1; i < kMaxWarps / 4; ++i) {
            if (warps <= 4 * i) break;
            const float4 b = r[i];
            a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
        }
        return (a.x + a.y) + (a.z + a.w);
    }
};

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

__device__ __forceinline__ void unpack_q8(uint2 u, float (&v)[8]) {
    from_fp8x4(u.x, v);
    from_fp8x4(u.y, v + 4);
}

// How the rows lie: multiples of 16 bytes from a 16-byte boundary; not multiples,
// but all tensors from a 16-byte boundary; anything else.
enum Rows : int { ROWS_VEC = 0, ROWS_ODD = 1, ROWS_ANY = 2 };

template <typename T> struct Raw8 {
    uint4 a[sizeof(T) / 2];
};
__device__ __forceinline__ void values(const Raw8<bf16> &r, float (&v)[8]) {
    const uint4 u = r.a[0];
    v[0] = lo_f(u.x); v[1] = hi_f(u.x); v[2] = lo_f(u.y); v[3] = hi_f(u.y);
    v[4] = lo_f(u.z); v[5] = hi_f(u.z); v[6] = lo_f(u.w); v[7] = hi_f(u.w);
}
__device__ __forceinline__ void values(const Raw8<float> &r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        v[4 * i] = __uint_as_float(r.a[i].x);
        v[4 * i + 1] = __uint_as_float(r.a[i].y);
        v[4 * i + 2] = __uint_as_float(r.a[i].z);
        v[4 * i + 3] = __uint_as_float(r.a[i].w);
    }
}
__device__ __forceinline__ void raw_of(const float (&v)[8], Raw8<bf16> &r) {
    r.a[0] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void raw_of(const float (&v)[8], Raw8<float> &r) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        r.a[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                            __float_as_uint(v[4 * i + 3]));
}

// values i .. i + 7 counted from the tensor's first one
template <int ROWS, typename T> __device__ __forceinline__ Raw8<T> load_raw(const Span<const T> &s, int64_t i) {
    Raw8<T> r;
    if (ROWS == ROWS_VEC || (ROWS == ROWS_ODD && i + 8 <= s.hi)) {
        const uint4 *q = reinterpret_cast<const uint4 *>(s.p + i);
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) r.a[k] = q[k];  // plain: the call may be writing in place
    } else {
        float v[8];
        if (ROWS == ROWS_ANY) {
            load_any(s, s.lo + i, v);
        } else {  // the tensor's last piece is cut short
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = i + k < s.hi ? to_f(s.p[i + k]) : 0.f;
        }
        raw_of(v, r);  // exact: the values are the tensor's own
    }
    return r;
}
template <int ROWS> __device__ __forceinline__ uint2 load_q(const Span<const uint8_t> &s, int64_t i) {
    if (ROWS == ROWS_VEC || (ROWS == ROWS_ODD && i + 8 <= s.hi)) return __ldg(reinterpret_cast<const uint2 *>(s.p + s.lo + i));
    if (ROWS == ROWS_ANY) return load_any8(s, s.lo + i);
    uint32_t u[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (i + k < s.hi) u[k / 4] |= (uint32_t)s.p[i + k] << (8 * (k & 3));
    return make_uint2(u[0], u[1]);
}

template <typename T> __device__ __forceinline__ bool aligned_piece(const T *p) {
    return (reinterpret_cast<uintptr_t>(p) & (sizeof(T) == 1 ? 7 : 15)) == 0;
}
// v to columns col .. col + 7 of the row that begins at value `row`, as far as they exist
template <int ROWS, typename T>
__device__ __forceinline__ void store_row(const Span<T> &s, int64_t row, int col, int dim, const float (&v)[8]) {
    T *p = s.p + s.lo + row + col;
    if (ROWS == ROWS_VEC || (col >= 0 && col + 8 <= dim && (ROWS == ROWS_ODD || aligned_piece(p)))) {
        store8(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i >= 0 && col + i < dim) p[i] = from_f<T>(v[i]);
    }
}
// the same for values that are packed already
template <int ROWS, typename T>
__device__ __forceinline__ void store_raw(const Span<T> &s, int64_t row, int col, int dim, const Raw8<T> &r) {
    T *p = s.p + s.lo + row + col;
    if (ROWS == ROWS_VEC || (col >= 0 && col + 8 <= dim && (ROWS == ROWS_ODD || aligned_piece(p)))) {
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) reinterpret_cast<uint4 *>(p)[k] = r.a[k];
    } else {
        float v[8];
        values(r, v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i >= 0 && col + i < dim) p[i] = from_f<T>(v[i]);
    }
}
template <int ROWS>
__device__ __forceinline__ void store_q(const Span<uint8_t> &s, int64_t row, int col, int dim, uint2 v) {
    uint8_t *p = s.p + s.lo + row + col;
    if (ROWS == ROWS_VEC || (col >= 0 && col + 8 <= dim && (ROWS == ROWS_ODD || aligned_piece(p)))) {
        *reinterpret_cast<uint2 *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i >= 0 && col + i < dim) p[i] = (uint8_t)((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
    }
}

// zeros for the values that belong to the rows in front and behind
template <int ROWS> __device__ __forceinline__ void mask_row(float (&v)[8], int col, int dim) {
    if (ROWS != ROWS_VEC && (col < 0 || col + 8 > dim)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < 0 || col + i >= dim) v[i] = 0.f;
    }
}

template <int ROWS, typename T>
__device__ __forceinline__ void load_gamma(const Span<const T> &gamma, int col, float (&g)[8]) {
    if (ROWS == ROWS_VEC) load8(gamma.p + col, g);
    else load_any(gamma, gamma.lo + col, g);
}

// largest of a and |b|, NaN if one of them is (fmaxf would drop it)
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
    return m;
}
// A group's scale from its largest magnitude: infinite where that is a NaN, which
// marks the group like an infinity does.
__device__ __forceinline__ float scale_of(float m) {
    return m == m ? fmaxf(m / kFp8Max, kTinyScale) : __int_as_float(0x7f800000);
}

// q of 8 values; the first ph of them are divided by another scale
__device__ __forceinline__ uint2 quantise8(const float (&s)[8], float inv_lo, float inv_hi, int ph) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = s[i] * (i < ph ? inv_lo : inv_hi);
    return make_uint2(to_fp8x4(t[0], t[1], t[2], t[3]), to_fp8x4(t[4], t[5], t[6], t[7]));
}

template <typename T> struct Forward {
    Span<const T> x, r, gamma;
    Span<T> s, y;
    Span<uint8_t> q;
    float *scale, *rstd;
    int64_t rows;
    int dim;
    float inv_dim, eps;
};

template <typename T, int ROWS, int NV>
__global__ void __launch_bounds__(kMaxThreads, NV * sizeof(T) <= 4 ? 2 : 1) resnorm_forward_kernel(const Forward<T> a) {
    __shared__ __align__(16) float red[2][kMaxWarps];
    // of each 16 threads' pieces: the maximum of their own group, and of the ph values in front of it
    __shared__ float group_max[2][ROWS == ROWS_VEC ? 1 : kMaxHeads + 1], head_max[2][ROWS == ROWS_VEC ? 1 : kMaxHeads + 1];
    const int dim = a.dim, groups = (dim + kGroup - 1) / kGroup;
    const int ph = ROWS == ROWS_VEC ? 0 : (int)((a.y.lo + (int64_t)blockIdx.x * dim) & 7);
    const int col0 = (int)threadIdx.x * 8 - ph, step = (int)blockDim.x * 8;
    const int hl = threadIdx.x & 15;
    if (ROWS != ROWS_VEC)
        for (int i = threadIdx.x; i < kMaxHeads + 1; i += blockDim.x) head_max[0][i] = head_max[1][i] = 0.f;
    const BlockSum block_sum{red, (int)blockDim.x >> 5};
    block_sum.init();
    float gm[NV <= 2 ? NV : 1][8];
    if (NV <= 2) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (col0 + k * step < dim) load_gamma<ROWS>(a.gamma, col0 + k * step, gm[k]);
    }
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
        const int64_t base = row * dim;
        float s[NV][8];
        {
            Raw8<T> x[NV], r[NV];
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (col0 + k * step < dim) x[k] = load_raw<ROWS>(a.x, base + col0 + k * step);
            if (a.r.p) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (col0 + k * step < dim) r[k] = load_raw<ROWS>(a.r, base + col0 + k * step);
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = col0 + k * step;
#pragma unroll
                for (int i = 0; i < 8; ++i) s[k][i] = 0.f;
                if (col >= dim) continue;
                values(x[k], s[k]);
                if (a.r.p) {
                    float b[8];
                    values(r[k], b);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[k][i] += b[i];
                    // the stream is held in T: norm and checkpoint are those of the rounded sum
                    raw_of(s[k], x[k]);
                    values(x[k], s[k]);
                    store_raw<ROWS>(a.s, base, col, dim, x[k]);
                }
                mask_row<ROWS>(s[k], col, dim);
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(s[k][i], s[k][i], ss);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = col0 + k * step;
            float m = 0.f, head = 0.f;  // head: of the first ph values, which may belong to the group in front
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (ROWS != ROWS_VEC && i < ph) head = max_nan(head, s[k][i]);
                else m = max_nan(m, s[k][i]);
            }
            if (ROWS != ROWS_VEC && hl != 0) m = max_nan(m, head);
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (ROWS == ROWS_VEC) {
                // the checkpoint needs no row sum: it is written while the sum is under way
                const float sc = scale_of(m), inv = 1.f / sc;
                if (col >= dim) continue;
                store_q<ROWS>(a.q, base, col, dim, quantise8(s[k], inv, inv, 0));
                if (hl == 0) a.scale[row * groups + col / kGroup] = sc;
            } else if (hl == 0) {
                const int h = (k * (int)blockDim.x + (int)threadIdx.x) / 16;
                group_max[parity][h] = m;
                head_max[parity][h] = head;
            }
        }
        if (ROWS != ROWS_VEC) __syncwarp();  // one warp: block_sum has no barrier
        const float rs = rsqrtf(fmaf(block_sum(ss, parity), a.inv_dim, a.eps));
        if (threadIdx.x == 0) a.rstd[row] = rs;
        if (ROWS != ROWS_VEC) {
            // a warp's pieces lie in two groups and end the one in front of them: lanes 0 to 2
            // form the three scales, the others repeat the last
            const int lane = threadIdx.x & 31;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = col0 + k * step;
                const int g = (k * (int)blockDim.x + (int)threadIdx.x - lane) / 16 + min(lane, 2) - 1;
                const float sc = scale_of(g >= 0 ? max_nan(group_max[parity][g], head_max[parity][g + 1]) : 0.f);
                const float inv = 1.f / sc;
                const float hi = __shfl_sync(0xffffffffu, inv, 1 + (lane >> 4));
                float lo = __shfl_sync(0xffffffffu, inv, lane >> 4);
                if (hl != 0) lo = hi;
                if ((lane == 1 || lane == 2) && g < groups) a.scale[row * groups + g] = sc;
                if (col < dim) store_q<ROWS>(a.q, base, col, dim, quantise8(s[k], lo, hi, ph));
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = col0 + k * step;
            if (col >= dim) continue;
            if (NV <= 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i) s[k][i] = s[k][i] * rs * gm[k < 2 ? k : 0][i];
            } else {
                float g[8];
                load_gamma<ROWS>(a.gamma, col, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[k][i] = s[k][i] * rs * g[i];
            }
            store_row<ROWS>(a.y, base, col, dim, s[k]);
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
    float inv_dim;
};

// The scales of the first ph values of a row's piece and of the others (piece
// h * 16 + 0 .. 15 of the row, the thread's place among 16 being hl).
struct Scales {
    float lo, hi;
};
template <int ROWS>
__device__ __forceinline__ Scales load_scales(const float *scale, int64_t row, int groups, int h, int hl) {
    const float *sc = scale + row * groups;
    Scales s;
    s.hi = __ldg(sc + (ROWS == ROWS_VEC ? h : min(h, groups - 1)));
    s.lo = ROWS != ROWS_VEC && hl == 0 && h > 0 ? __ldg(sc + h - 1) : s.hi;
    return s;
}
// n = q * scale * rstd, 0 outside the row
template <int ROWS>
__device__ __forceinline__ void normed(uint2 q, const Scales &s, float rs, int ph, int col, int dim, float (&n)[8]) {
    unpack_q8(q, n);
    const float lo = s.lo * rs, hi = s.hi * rs;
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] *= ROWS != ROWS_VEC && i < ph ? lo : hi;
    mask_row<ROWS>(n, col, dim);
}

template <typename T, int ROWS>
__global__ void __launch_bounds__(256) resnorm_recompute_kernel(const Backward<T> a) {
    const int dim = a.dim, groups = (dim + kGroup - 1) / kGroup;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rs = a.rstd[row];
        const int ph = ROWS == ROWS_VEC ? 0 : (int)((a.y.lo + row * dim) & 7);
        for (int j = threadIdx.x; j * 8 - ph < dim; j += blockDim.x) {
            const int col = j * 8 - ph;
            float n[8], g[8];
            normed<ROWS>(load_q<ROWS>(a.q, row * dim + col), load_scales<ROWS>(a.scale, row, groups, j / 16, j & 15), rs,
                         ph, col, dim, n);
            load_gamma<ROWS>(a.gamma, col, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] *= g[i];
            store_row<ROWS>(a.y, row * dim, col, dim, n);
        }
    }
}

__device__ __forceinline__ void copy_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async8(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Each block keeps its columns' share of dgamma in registers over all its rows
// and writes it once, to partial[block][pitch].
//
// RING > 0 (up to 16 values per thread and tensor): the rows ahead are copied to
// shared memory asynchronously, RING - 1 of them at a time, each piece by the
// thread that will use it, so no barrier is needed for them and the bytes in
// flight do not depend on registers (figures at ring_of).
template <typename T, int ROWS, int NV, int RING>
__global__ void __launch_bounds__(kMaxThreads, NV == 1 ? 2 : 1) resnorm_backward_kernel(const Backward<T> a) {
    __shared__ __align__(16) float red[2][kMaxWarps];
    extern __shared__ __align__(16) unsigned char ring[];
    constexpr int PIECES = (int)sizeof(T) / 2;  // 16-byte pieces of 8 values
    constexpr int STAGES = RING > 0 ? RING : 1;
    const int dim = a.dim, groups = (dim + kGroup - 1) / kGroup, threads = blockDim.x, tid = threadIdx.x;
    const int ph = ROWS == ROWS_VEC ? 0 : (int)((a.dx.lo + (int64_t)blockIdx.x * dim) & 7);
    const int col0 = tid * 8 - ph, step = threads * 8, hl = tid & 15;
    const BlockSum block_sum{red, threads >> 5};
    grid_dependency_launch();
    block_sum.init();
    float dg[NV][8], gm[RING ? NV : 1][8];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[k][i] = 0.f;
    if (RING) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (col0 + k * step < dim) load_gamma<ROWS>(a.gamma, col0 + k * step, gm[k]);
    }
    // ring: [stage][k][dy, ds][piece][thread] 16 bytes, then [stage][k][thread] 8 bytes of q
    uint4 *ring16 = reinterpret_cast<uint4 *>(ring);
    uint2 *ring8 = reinterpret_cast<uint2 *>(ring16 + STAGES * NV * 2 * PIECES * threads);
    auto slot16 = [&](int stage, int k, int which, int piece) {
        return ring16 + (((stage * NV + k) * 2 + which) * PIECES + piece) * threads + tid;
    };
    auto slot8 = [&](int stage, int k) { return ring8 + (stage * NV + k) * threads + tid; };
    auto copy_row = [&](int64_t row, int stage) {
        if (row < a.rows) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = col0 + k * step;
                if (col >= dim) continue;
                const int64_t at = row * dim + col;
                if (ROWS == ROWS_VEC || (ROWS == ROWS_ODD && at + 8 <= a.dy.hi)) {
#pragma unroll
                    for (int p = 0; p < PIECES; ++p) {
                        copy_async16(slot16(stage, k, 0, p), reinterpret_cast<const uint4 *>(a.dy.p + at) + p);
                        if (a.ds.p) copy_async16(slot16(stage, k, 1, p), reinterpret_cast<const uint4 *>(a.ds.p + at) + p);
                    }
                    copy_async8(slot8(stage, k), a.q.p + a.q.lo + at);
                } else {
                    const Raw8<T> x = load_raw<ROWS>(a.dy, at);
#pragma unroll
                    for (int p = 0; p < PIECES; ++p) *slot16(stage, k, 0, p) = x.a[p];
                    if (a.ds.p) {
                        const Raw8<T> y = load_raw<ROWS>(a.ds, at);
#pragma unroll
                        for (int p = 0; p < PIECES; ++p) *slot16(stage, k, 1, p) = y.a[p];
                    }
                    *slot8(stage, k) = load_q<ROWS>(a.q, at);
                }
            }
        }
        copy_async_commit();  // a group per row, empty ones too
    };
    Scales sc[NV];
    float rs = 0.f;
    auto fetch_scales = [&](int64_t row) {
        if (row >= a.rows) return;
        rs = __ldg(a.rstd + row);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (col0 + k * step < dim) sc[k] = load_scales<ROWS>(a.scale, row, groups, (k * threads + tid) / 16, hl);
    };
    const int64_t stride = gridDim.x;
    if (RING) {
#pragma unroll
        for (int i = 0; i < RING - 1; ++i) copy_row(blockIdx.x + i * stride, i);
        fetch_scales(blockIdx.x);
    }
    int parity = 0, stage = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += stride, parity ^= 1) {
        const int64_t base = row * dim;
        float n[NV][8], d[NV][8], t = 0.f;
        Raw8<T> add[NV];
        if (RING) {
            copy_async_wait<RING >= 2 ? RING - 2 : 0>();
        } else {
            fetch_scales(row);
        }
        const float r = rs;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = col0 + k * step;
            if (col >= dim) continue;
            Raw8<T> x;
            uint2 q;
            if (RING) {
#pragma unroll
                for (int p = 0; p < PIECES; ++p) {
                    x.a[p] = *slot16(stage, k, 0, p);
                    if (a.ds.p) add[k].a[p] = *slot16(stage, k, 1, p);
                }
                q = *slot8(stage, k);
            } else {
                x = load_raw<ROWS>(a.dy, base + col);
                q = load_q<ROWS>(a.q, base + col);
                if (a.ds.p) add[k] = load_raw<ROWS>(a.ds, base + col);
            }
            values(x, d[k]);
            mask_row<ROWS>(d[k], col, dim);
            normed<ROWS>(q, sc[k], r, ph, col, dim, n[k]);
        }
        if (RING) {  // into the slots that were read a row ago
            copy_row(row + (RING - 1) * stride, (stage + RING - 1) % STAGES);
            fetch_scales(row + stride);
            stage = (stage + 1) % STAGES;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = col0 + k * step;
            if (col >= dim) continue;
            float g[8];
            if (RING) {
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = gm[RING ? k : 0][i];
            } else {
                load_gamma<ROWS>(a.gamma, col, g);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dg[k][i] = fmaf(d[k][i], n[k][i], dg[k][i]);
                d[k][i] *= g[i];
                t = fmaf(d[k][i], n[k][i], t);
                g[i] *= n[k][i];
            }
            if (a.y.p) store_row<ROWS>(a.y, base, col, dim, g);
        }
        const float rt = r * (block_sum(t, parity) * a.inv_dim);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = col0 + k * step;
            if (col >= dim) continue;
            float b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (a.ds.p) values(add[k], b);
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = fmaf(-rt, n[k][i], fmaf(r, d[k][i], b[i]));
            store_row<ROWS>(a.dx, base, col, dim, b);
        }
    }
    if (RING) copy_async_wait<0>();
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int col = col0 + k * step;
        if (col >= dim) continue;
        float *out = a.partial + (int64_t)blockIdx.x * a.pitch;
        if (ROWS == ROWS_VEC) {
            store8(out + col, dg[k]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i >= 0 && col + i < dim) out[col + i] = dg[k][i];
        }
    }
}

// dgamma[j] = sum over blocks of partial[block][j]: 32 columns per block, 32
// threads per column, joined in a fixed order.
__global__ void __launch_bounds__(1024) dgamma_kernel(const float *partial, int blocks, int dim,
                                                      int pitch, float *__restrict__ dgamma) {
    __shared__ float red[32][33];
    grid_dependency_wait();
    const int c = threadIdx.x & 31, w = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
    float a = 0.f;
    if (col < dim) {
#pragma unroll 8
        for (int b = w; b < blocks; b += 32) a += partial[(int64_t)b * pitch + col];
    }
    red[w][c] = a;
    __syncthreads();
    a = red[c][w];  // warp w adds up column w of the block's 32
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (c == 0 && blockIdx.x * 32 + w < dim) dgamma[blockIdx.x * 32 + w] = a;
}

// Values per thread of the forward pass: 16 (NV = 2) up to a width of 8192, so
// that a row of 2048 takes 4 warps and many rows are in flight on an SM; then 32
// and 64 (72 for the widest rows off their boundaries).  fp32 and odd rows take 8 up to
// 4096.  Forward, 8 / 16 values per thread, cold: bf16 65536 x 512 57 / 55 us, x 1024 109 / 98, x 2048
// 215 / 184, 32768 x 4096 231 / 188; fp32 65536 x 1024 172 / 174, 16384 x 4096 184 / 191; odd 65536 x
// 1022 178 / 182.  The backward pass keeps four times as much per value and takes 8 up to
// 4096.  8 / 16, cold: bf16 65536 x 512 82 / 76 us, x 2048 219 / 191, 32768 x 4096 229 / 195, x 2046 201 /
// 160; fp32 65536 x 1024 250 / 260, 32768 x 2048 240 / 255, 16384 x 4096 270 / 240: for bf16 and from
// 4096 on 16 would be the better choice.
struct Shape {
    int nv, threads;
};
Shape shape_of(int dim, bool vec, bool one) {
    const int64_t vecs = vec ? dim / 8 : (dim + 14) / 8;  // 8-value pieces that a row can touch
    int nv = 1;
    while (nv < 8 && (vecs > kMaxThreads * nv || (!one && nv < 2 && vecs > 32))) nv *= 2;
    if (vecs > kMaxThreads * nv) nv = kMaxPieces;
    return {nv, (int)round_up(ceil_div(vecs, nv), 32)};
}

// Rows in the ring of the backward pass: four (three on their way while one is
// worked on), two where four do not fit, none for wide rows.  By this rule / with two rows /
// without a ring, cold: bf16 65536 x 2048 219 / 219 / 217 us, 32768 x 2046 201 / 217 / 208, 16384 x 8192
// 199 / 201 / 285; fp32 32768 x 2048 240 / 248 / 182, 16384 x 4096 270 / 231 / 178, 8192 x 8192 277 / 277 /
// 229: fp32 rows would do better without one.
constexpr int ring_of(int nv, int value_bytes) { return nv == 1 ? 4 : nv == 2 ? (value_bytes == 2 ? 4 : 2) : 0; }
constexpr int ring_bytes(const Shape &sh, int value_bytes) {
    return sh.threads * sh.nv * ring_of(sh.nv, value_bytes) * (2 * 8 * value_bytes + 8);
}

// Resident blocks: what registers and shared memory allow.  A multiple of 8
// where there are that many rows: a block's rows then begin alike.
int backward_blocks(int64_t rows, const Shape &sh, int value_bytes) {
    const int by_threads = (sh.nv == 1 ? 1024 : 512) / sh.threads;
    const int by_smem = 220 * 1024 / std::max(1, ring_bytes(sh, value_bytes) + 1024);
    const int per_sm = std::max(1, std::min({8, by_threads, by_smem}));
    return (int)std::max<int64_t>(1, std::min<int64_t>(rows, (int64_t)num_sms() * per_sm / 8 * 8));
}

template <typename F> int with_nv(int nv, F &&f) {
    switch (nv) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        case 8: return f(std::integral_constant<int, 8>{});
        default: return f(std::integral_constant<int, kMaxPieces>{});
    }
}
// the layout of vector rows, which never take the ninth piece
constexpr int vec_rows(int nv) { return nv == kMaxPieces ? ROWS_ODD : ROWS_VEC; }

int check_sizes(int64_t rows, int32_t dim, int32_t type, const char *what) {
    if (rows < 0 || rows > INT32_MAX)
        return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": rows outside [0, 2^31)");
    if (dim < 1 || dim > kMaxDim) return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": dim outside [1, 32768]");
    if (!type_ok(type))
        return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": type must be STAGE_BF16 or STAGE_FP32");
    return SPECOPTIM_OK;
}

template <typename T> int run_forward(const Shape &sh, int rows, const Forward<T> &a, cudaStream_t st) {
    return with_nv(sh.nv, [&](auto nv) -> int {
        constexpr int NV = decltype(nv)::value;
        // 64 blocks per SM; odd rows, whose blocks cost more to begin, as many as have 4096 threads
        // (9749 x 6030: 109 us with 8 of 384 threads, 138 with 64; 60000 x 300: 76 with 64 of 64, 105 with
        // 8).  Multiples of 8: a block's rows begin alike.
        const int per_sm = rows == ROWS_VEC ? 64 : std::max(8, 4096 / sh.threads / 8 * 8);
        const int grid = (int)std::min<int64_t>(a.rows, (int64_t)num_sms() * per_sm);
        auto *k = rows == ROWS_VEC   ? &resnorm_forward_kernel<T, vec_rows(NV), NV>
                  : rows == ROWS_ODD ? &resnorm_forward_kernel<T, ROWS_ODD, NV>
                                     : &resnorm_forward_kernel<T, ROWS_ANY, NV>;
        SPCO_LAUNCH("resnorm_forward", st, k<<<grid, sh.threads, 0, st>>>(a));
        SPECOPTIM_LAUNCHED("resnorm_forward_kernel");
        return SPECOPTIM_OK;
    });
}

template <typename T>
int run_backward(const Shape &sh, int rows, int blocks, const Backward<T> &a, float *dgamma, cudaStream_t st) {
    return with_nv(sh.nv, [&](auto nv) -> int {
        constexpr int NV = decltype(nv)::value;
        constexpr int RING = ring_of(NV, sizeof(T));
        auto *k = rows == ROWS_VEC   ? &resnorm_backward_kernel<T, vec_rows(NV), NV, RING>
                  : rows == ROWS_ODD ? &resnorm_backward_kernel<T, ROWS_ODD, NV, RING>
                                     : &resnorm_backward_kernel<T, ROWS_ANY, NV, RING>;
        const int smem = ring_bytes(sh, sizeof(T));
        if (smem > 48 * 1024)
            if (int rc = set_smem_limit(reinterpret_cast<const void *>(k), smem)) return rc;
        SPCO_LAUNCH("resnorm_backward", st, k<<<blocks, sh.threads, smem, st>>>(a));
        SPECOPTIM_LAUNCHED("resnorm_backward_kernel");
        cudaError_t e = cudaSuccess;
        SPCO_LAUNCH("resnorm_dgamma", st,
                    e = launch_dependent(dgamma_kernel, dim3((unsigned)ceil_div(a.dim, 32)), dim3(1024), 0, st, a.partial,
                                         blocks, a.dim, a.pitch, dgamma));
        SPECOPTIM_CUDA(e);
        return SPECOPTIM_OK;
    });
}

// how the rows of the given tensors lie
int rows_of(int dim, std::initializer_list<const void *> tensors) {
    for (const void *p : tensors)
        if (!aligned16(p)) return ROWS_ANY;
    return dim % 8 == 0 ? ROWS_VEC : ROWS_ODD;
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
        const int layout = rows_of(dim, {x, r, gamma, y, r ? s : nullptr, q});
        const Shape sh = shape_of(dim, layout == ROWS_VEC, layout != ROWS_VEC || type != STAGE_BF16);
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
                               1.f / (float)dim,
                               eps};
            return run_forward<T>(sh, layout, a, static_cast<cudaStream_t>(stream));
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
        const int layout = rows_of(dim, {gamma, y, q});
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
                                dim,
                                0.f};
            auto *k = layout == ROWS_VEC   ? &resnorm_recompute_kernel<T, ROWS_VEC>
                      : layout == ROWS_ODD ? &resnorm_recompute_kernel<T, ROWS_ODD>
                                           : &resnorm_recompute_kernel<T, ROWS_ANY>;
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
        // the most blocks of any type and layout: the call's are not known yet
        int blocks = 0;
        for (const bool vec : {true, false})
            for (const int value_bytes : {2, 4})
                blocks = std::max(blocks, backward_blocks(rows, shape_of(dim, vec, true), value_bytes));
        bytes = (int64_t)blocks * round_up(dim, 8) * 4;
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
        const int layout = rows_of(dim, {dy, ds, gamma, dx, y, q});
        const Shape sh = shape_of(dim, layout == ROWS_VEC, true);
        const int blocks = backward_blocks(rows, sh, (int)type_bytes(type)), pitch = (int)round_up(dim, 8);
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
                                pitch,
                                1.f / (float)dim};
            return run_backward<T>(sh, layout, blocks, a, dgamma, static_cast<cudaStream_t>(stream));
        });
    });
}
