// Residual sum + LayerNorm and its backward pass (include/finetune.h).
//
//   forward   s = x + r,  rstd = 1 / sqrt(mean (s - mean)^2 + eps),  y = (s - mean) rstd gamma + beta
//   backward  n = (s - mean) rstd,  g = gamma dy,
//             dx = ds + rstd (g - mean g - n mean(g n)),
//             dgamma = sum over rows of dy n,  dbeta = sum over rows of dy
//
// Forward: a row lies in the registers of a warp or of a block (8 values per
// thread and step) and is read once.  Each warp forms the mean of its values and
// the sum of squares about that mean; the warps' pairs join exactly (the squares
// about the common mean are those about the warp's plus count (difference)^2), so
// one barrier gives both statistics without the cancellation of mean(s^2) - mean^2.
//
// Backward: a group of threads holds the columns (8 values per thread and step)
// and walks over rows, R at a time, that arrive in shared memory by bulk
// copies some tiles ahead.  A tile goes from there to registers, one barrier forms its
// rows' sums, and its place is free for the tile some stages behind it.  The columns' shares of
// dgamma and dbeta stay in registers; each block leaves one partial, and a last launch adds the
// partials in their order.
//
// Rows that are not multiples of 16 bytes (ROWS_ODD) are cut where memory is: a
// thread's 8 values begin at a multiple of 8 of the tensor, the first ph of the
// row's first piece belong to the row in front.  The rows of a group lie a
// multiple of 8 rows apart, so ph is the same for all of them.
//
// Rows off a 16-byte boundary (ROWS_ANY) and rows of more than 1024 pieces take a backward pass of
// two kernels: one reads them twice, the other once more.  Those are rows above 8192 values, and odd
// ones from 8186 on, which may begin in the last value of a piece (16384 x 8190: 613 us, x 8192 181).
//
// All statistics and sums are fp32; s, y and dx are rounded once to their type.
//
// Measured on a GB300 (copy bandwidth 6.78 TB/s), cold, with a residual, bf16 65536 x 2048:
//   forward 162 us, 6.65 TB/s of x, r, s and y: 98 % of a copy; without the next row's loads 168,
//     values one by one instead of in pairs 170, unpacked vectors and all in registers 257;
//   backward 177 us, 6.08 TB/s (90 %): 240 instructions a warp and row, issue slots 55 % busy at
//     16 warps an SM, which the ring leaves; from registers instead of a second reading of shared
//     memory 177, with it 212 to 219.
// fp32 32768 x 2048 159 and 171 us.  Without ds the backward pass takes 164 (73 %), without r the
// forward pass 104 (77 %): a row's chain.  Odd rows cost instructions: 32768 x 2046 166 and 219 us
// (80 at the copy's rate).  Narrow rows too: 65536 x 64 21 and 31 (5).
// Bytes that spill, a thread: odd and unaligned bf16 rows of up to 2 pieces 96 to 132 forward (64
// registers, for two blocks an SM); fp32 forward 432 with 4 pieces and 848 to 1036 with 8 or 9; odd
// rows of 2 pieces backward 176 (bf16) and 280 (fp32); the other kernels 68 at most, but for the odd
// bf16 rows of 9 pieces (136).
#include <algorithm>
#include <string>

#include "../../include/finetune.h"
#include "f32x2.cuh"
#include "rowvec.cuh"

namespace spco {
namespace {

constexpr int kMaxDim = 32768;
constexpr int kMaxThreads = 512, kMaxWarps = kMaxThreads / 32;
// Pieces of 8 values of the widest row at any place between two boundaries: 4097, nine per thread.
constexpr int kMaxPieces = 9;
static_assert(kMaxThreads * kMaxPieces >= (kMaxDim + 14) / 8, "the widest row at any place");

// How the rows lie: multiples of 16 bytes from a 16-byte boundary; not multiples,
// but all tensors from a 16-byte boundary; anything else.
enum Rows : int { ROWS_VEC = 0, ROWS_ODD = 1, ROWS_ANY = 2 };

// 8 values as they lie in memory
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

__device__ __forceinline__ void values(const Raw8<bf16> &r, F2 (&v)[4]) {
    const uint4 u = r.a[0];
    v[0] = pair(lo_f(u.x), hi_f(u.x));
    v[1] = pair(lo_f(u.y), hi_f(u.y));
    v[2] = pair(lo_f(u.z), hi_f(u.z));
    v[3] = pair(lo_f(u.w), hi_f(u.w));
}
__device__ __forceinline__ void values(const Raw8<float> &r, F2 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        v[2 * i] = pair(__uint_as_float(r.a[i].x), __uint_as_float(r.a[i].y));
        v[2 * i + 1] = pair(__uint_as_float(r.a[i].z), __uint_as_float(r.a[i].w));
    }
}
template <typename T> __device__ __forceinline__ void raw_of(const F2 (&v)[4], Raw8<T> &r) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = both(v[i]);
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
    raw_of(f, r);
}

// values i .. i + 7 of the tensor
template <int ROWS, typename T> __device__ __forceinline__ Raw8<T> load_piece(const Span<const T> &s, int64_t i) {
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

// v to columns col .. col + 7 of the row that begins at value `row`, as far as they exist
template <int ROWS, typename T>
__device__ __forceinline__ void store_piece(const Span<T> &s, int64_t row, int col, int dim, const Raw8<T> &r) {
    T *p = s.p + s.lo + row + col;
    const bool whole = ROWS == ROWS_VEC || (col >= 0 && col + 8 <= dim &&
                                            (ROWS == ROWS_ODD || (reinterpret_cast<uintptr_t>(p) & 15) == 0));
    if (whole) {
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
template <int ROWS, typename T, typename V>
__device__ __forceinline__ void store_values(const Span<T> &s, int64_t row, int col, int dim, const V &v) {
    Raw8<T> r;
    raw_of(v, r);
    store_piece<ROWS>(s, row, col, dim, r);
}

// zeros for the values that belong to the rows in front and behind
template <int ROWS> __device__ __forceinline__ void mask_piece(float (&v)[8], int col, int dim) {
    if (ROWS != ROWS_VEC && (col < 0 || col + 8 > dim)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < 0 || col + i >= dim) v[i] = 0.f;
    }
}

// the same for values as they lie in memory: words that keep the row's
template <typename T> __device__ __forceinline__ Raw8<T> row_words(int col, int dim) {
    Raw8<T> m;
    uint32_t w[2 * sizeof(T)];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t in = col + i >= 0 && col + i < dim ? 0xffffffffu : 0u;
        if (sizeof(T) == 4) w[i] = in;
        else w[i / 2] = i & 1 ? w[i / 2] | (in & 0xffff0000u) : in & 0xffffu;
    }
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) m.a[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    return m;
}
template <int ROWS, typename T> __device__ __forceinline__ void keep_words(Raw8<T> &r, const Raw8<T> &m) {
    if (ROWS != ROWS_VEC)
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k)
            r.a[k] = make_uint4(r.a[k].x & m.a[k].x, r.a[k].y & m.a[k].y, r.a[k].z & m.a[k].z, r.a[k].w & m.a[k].w);
}
template <int ROWS> __device__ __forceinline__ void mask_piece(F2 (&v)[4], int col, int dim) {
    if (ROWS != ROWS_VEC && (col < 0 || col + 8 > dim)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = both(v[i]);
            const int c = col + 2 * i;
            v[i] = pair(c < 0 || c >= dim ? 0.f : f.x, c + 1 < 0 || c + 1 >= dim ? 0.f : f.y);
        }
    }
}

// a vector of dim values (gamma, beta), at any place
template <int ROWS, typename T> __device__ __forceinline__ Raw8<T> load_vector(const Span<const T> &s, int col) {
    if (ROWS == ROWS_VEC) return load_piece<ROWS_VEC>(s, col);
    float v[8];
    Raw8<T> r;
    load_any(s, s.lo + col, v);
    raw_of(v, r);
    return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---- forward -----------------------------------------------------------------------------

// Whether a row is loaded while the one in front is worked on.  Pays where the registers allow it: cold,
// with / without, bf16 65536 x 2048 163 / 168 us, 32768 x 4096 164 / 171, fp32 32768 x 2048 158 / 164; more
// pieces of fp32, or rows that are shifted into place, spill without it already, and more with it (fp32
// 16384 x 4096 with 4 pieces 202 / 176).
template <typename T> constexpr bool loads_ahead(int rows, int nv) {
    return rows == ROWS_VEC && nv * (int)sizeof(T) <= 8;
}

template <typename T> struct Forward {
    Span<const T> x, r, gamma, beta;  // r.p, beta.p null: none
    Span<T> s, y;
    float *mean, *rstd;
    int64_t rows;
    int dim;
    float inv_dim, eps;
};

// A row per block (WARP: per warp), NV pieces of 8 values per thread.
template <typename T, int ROWS, int NV, bool WARP>
__global__ void __launch_bounds__(kMaxThreads, ROWS != ROWS_VEC && NV * sizeof(T) <= 4 ? 2 : 1) layernorm_forward_kernel(const Forward<T> a) {
    // of each warp: the mean of its values, the squares about it, and how many they are; zeros behind the last
    __shared__ __align__(16) float red[2][2][kMaxWarps], count_of[kMaxWarps];
    constexpr bool AHEAD = loads_ahead<T>(ROWS, NV);
    const int dim = a.dim, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int threads = WARP ? 32 : blockDim.x, tid = WARP ? lane : threadIdx.x;
    const int64_t first = WARP ? (int64_t)blockIdx.x * warps + warp : blockIdx.x;
    const int64_t stride = WARP ? (int64_t)gridDim.x * warps : gridDim.x;
    const int ph = ROWS == ROWS_VEC ? 0 : (int)((a.y.lo + first * dim) & 7);
    const int col0 = tid * 8 - ph, step = threads * 8;
    float own = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) own += (float)max(0, min(col0 + k * step + 8, dim) - max(col0 + k * step, 0));
    own = warp_sum(own);
    const float inv_own = own > 0.f ? 1.f / own : 0.f;
    if (!WARP) {
        for (int i = threadIdx.x; i < 4 * kMaxWarps; i += blockDim.x) (&red[0][0][0])[i] = 0.f;
        if (threadIdx.x < kMaxWarps) count_of[threadIdx.x] = 0.f;
        __syncthreads();
        if (lane == 0) count_of[warp] = own;
        __syncthreads();
    }
    // the vectors stay in registers where a thread has few pieces
    Raw8<T> gm[NV <= 4 ? NV : 1], bt[NV <= 4 ? NV : 1];
    if (NV <= 4) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = col0 + k * step;
            bt[k < 4 ? k : 0] = Raw8<T>{};
            if (col >= dim) continue;
            gm[k < 4 ? k : 0] = load_vector<ROWS>(a.gamma, col);
            if (a.beta.p) bt[k < 4 ? k : 0] = load_vector<ROWS>(a.beta, col);
        }
    }
    int parity = 0;
    Raw8<T> x[NV], r[NV];
    auto fetch = [&](int64_t row) {
        if (row >= a.rows) return;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (col0 + k * step < dim) x[k] = load_piece<ROWS>(a.x, row * dim + col0 + k * step);
        if (a.r.p) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (col0 + k * step < dim) r[k] = load_piece<ROWS>(a.r, row * dim + col0 + k * step);
        }
    };
    if (AHEAD) fetch(first);
    for (int64_t row = first; row < a.rows; row += stride, parity ^= 1) {
        const int64_t base = row * dim;
        Raw8<T> s[NV];
        if (!AHEAD) fetch(row);
#pragma unroll
        for (int k = 0; k < NV; ++k) s[k] = x[k];
        if (a.r.p) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = col0 + k * step;
                if (col >= dim) continue;
                F2 v[4], b[4];
                values(s[k], v);
                values(r[k], b);
                // the stream is held in T: the norm is that of the rounded sum
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = v[i] + b[i];
                raw_of(v, s[k]);
                store_piece<ROWS>(a.s, base, col, dim, s[k]);
            }
        }
        if (AHEAD) fetch(row + stride);
        F2 sums = pair(0.f, 0.f), squares = sums;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (col0 + k * step >= dim) continue;
            F2 v[4];
            values(s[k], v);
            mask_piece<ROWS>(v, col0 + k * step, dim);
            sums = sums + ((v[0] + v[1]) + (v[2] + v[3]));
        }
        const float mid = warp_sum(sum2(sums)) * inv_own;
        const F2 minus_mid = pair(-mid, -mid);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = col0 + k * step;
            if (col >= dim) continue;
            F2 v[4];
            values(s[k], v);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = v[i] + minus_mid;
            mask_piece<ROWS>(v, col, dim);
#pragma unroll
            for (int i = 0; i < 4; ++i) squares = fma2(v[i], v[i], squares);
        }
        float sq = warp_sum(sum2(squares));
        float mean = mid;
        if (!WARP) {
            if (lane == 0) {
                red[parity][0][warp] = mid;
                red[parity][1][warp] = sq;
            }
            __syncthreads();
            const float4 *mids = reinterpret_cast<const float4 *>(red[parity][0]);
            const float4 *sqs = reinterpret_cast<const float4 *>(red[parity][1]);
            const float4 *counts = reinterpret_cast<const float4 *>(count_of);
            mean = 0.f;
#pragma unroll
            for (int i = 0; i < kMaxWarps / 4; ++i) {
                if (4 * i >= warps) break;
                const float4 m = mids[i], c = counts[i];
                mean += fmaf(c.x, m.x, c.y * m.y) + fmaf(c.z, m.z, c.w * m.w);
            }
            mean *= a.inv_dim;
            sq = 0.f;
#pragma unroll
            for (int i = 0; i < kMaxWarps / 4; ++i) {
                if (4 * i >= warps) break;
                const float4 m = mids[i], c = counts[i], q = sqs[i];
                const float dx = m.x - mean, dy = m.y - mean, dz = m.z - mean, dw = m.w - mean;
                sq += (fmaf(c.x * dx, dx, q.x) + fmaf(c.y * dy, dy, q.y)) + (fmaf(c.z * dz, dz, q.z) + fmaf(c.w * dw, dw, q.w));
            }
        }
        const float rs = rsqrtf(fmaf(sq, a.inv_dim, a.eps));
        const F2 minus_mean = pair(-mean, -mean), scale = pair(rs, rs);
        if (tid == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rs;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = col0 + k * step;
            if (col >= dim) continue;
            F2 v[4], g[4], b[4];
            values(s[k], v);
            if (NV <= 4) {
                values(gm[k < 4 ? k : 0], g);
                values(bt[k < 4 ? k : 0], b);
            } else {
                values(load_vector<ROWS>(a.gamma, col), g);
                values(a.beta.p ? load_vector<ROWS>(a.beta, col) : Raw8<T>{}, b);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fma2((v[i] + minus_mean) * scale, g[i], b[i]);
            store_values<ROWS>(a.y, base, col, dim, v);
        }
    }
}

// ---- backward ----------------------------------------------------------------------------

template <typename T> struct Backward {
    Span<const T> dy, ds, s, gamma;  // ds.p null: none
    const float *mean, *rstd;
    Span<T> dx;
    float *partial;  // [blocks][2][pitch]
    int64_t rows, stride;  // stride: groups of the launch
    int dim, pitch, threads;  // threads of a group
    int slot;    // bytes of one row of one tensor in a ring
    int stages;  // tiles in a ring
    float inv_dim;
};

// N values per thread summed over each warp: lane l ends with the sum of value
// l >> (5 - log2 N).  Every step halves the values that a lane still carries.
template <int N> __device__ __forceinline__ float warp_sums(float (&v)[N]) {
    const int lane = threadIdx.x & 31;
    int o = 16;
#pragma unroll
    for (int n = N / 2; n >= 1; n /= 2, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = up ? v[i] : v[n + i];
            const float keep = up ? v[n + i] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    float r = v[0];
    for (; o >= 1; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    return r;
}

// 8 values of a row in shared memory
template <typename T> __device__ __forceinline__ Raw8<T> load_shared(const T *p) {
    Raw8<T> r;
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) r.a[k] = reinterpret_cast<const uint4 *>(p)[k];
    return r;
}

// the sum of what the warps left
__device__ __forceinline__ float row_sum(const float *red, int warps) {
    const float4 *p = reinterpret_cast<const float4 *>(red);
    float4 v = p[0];
#pragma unroll
    for (int i = 1; i < kMaxWarps / 4; ++i) {
        if (4 * i >= warps) break;
        const float4 x = p[i];
        v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
    }
    return (v.x + v.y) + (v.z + v.w);
}

__device__ __forceinline__ void group_barrier(int group, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

constexpr int kMaxStages = 4, kMaxGroups = 8;
constexpr uint32_t kDrainLimit = 1u << 14;  // probes of up to 4 us, for what takes microseconds

// Dynamic shared memory: for each group a ring [stage][row][dy, s, ds][slot].
template <typename T, int ROWS, int NV, int R>
__global__ void __launch_bounds__(kMaxThreads, 1) layernorm_backward_kernel(const Backward<T> a, unsigned *flag) {
    extern __shared__ __align__(16) unsigned char ring_raw[];
    __shared__ uint64_t full_bars[kMaxGroups][kMaxStages];
    __shared__ __align__(16) float red_raw[kMaxGroups][2][2 * R][kMaxWarps];  // zeros behind the last warp
    const int threads = a.threads, group = threadIdx.x / threads, tid = threadIdx.x % threads, groups = blockDim.x / threads;
    const int lane = threadIdx.x & 31, warp = tid >> 5, warps = threads >> 5;
    const int dim = a.dim, tensors = a.ds.p ? 3 : 2;
    const int64_t first = (int64_t)blockIdx.x * groups + group;
    const int ph = ROWS == ROWS_VEC ? 0 : (int)((first * dim) & 7);
    const int pieces = (ph + dim + 7) / 8;
    uint64_t *full = full_bars[group];
    unsigned char *ring = ring_raw + (size_t)group * a.stages * R * tensors * a.slot;
    grid_dependency_launch();
    for (int i = threadIdx.x; i < kMaxGroups * 2 * 2 * R * kMaxWarps; i += blockDim.x) (&red_raw[0][0][0][0])[i] = 0.f;
    if (tid == 0) {
        for (int i = 0; i < a.stages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto slot_of = [&](int stage, int r, int which) {
        return reinterpret_cast<T *>(ring + ((size_t)(stage * R + r) * tensors + which) * a.slot);
    };
    // one thread of the group asks for a tile's rows
    auto fetch = [&](int64_t tile, int stage) {
        uint32_t bytes = 0, size[R];
        const int64_t row = first + tile * R * a.stride;
        int64_t from = row * dim - ph;
        const int64_t from0 = from, hop = a.stride * dim;
#pragma unroll
        for (int r = 0; r < R; ++r, from += hop) {
            size[r] = 0;
            if (row + r * a.stride >= a.rows) continue;
            if (ROWS == ROWS_VEC) {
                size[r] = (uint32_t)dim * sizeof(T);
            } else {
                const int64_t values = min((int64_t)pieces * 8, a.dy.hi - from);
                size[r] = (uint32_t)(values * sizeof(T)) & ~15u;
                for (int64_t i = size[r] / sizeof(T); i < values; ++i) {  // what the tensor's last 16 bytes lack
                    slot_of(stage, r, 0)[i] = a.dy.p[from + i];
                    slot_of(stage, r, 1)[i] = a.s.p[from + i];
                    if (tensors == 3) slot_of(stage, r, 2)[i] = a.ds.p[from + i];
                }
            }
            bytes += size[r] * tensors;
        }
        mbar_arrive_expect_tx(&full[stage], bytes);
        from = from0;
#pragma unroll
        for (int r = 0; r < R; ++r, from += hop) {
            if (!size[r]) continue;
            bulk_load(slot_of(stage, r, 0), a.dy.p + from, size[r], &full[stage]);
            bulk_load(slot_of(stage, r, 1), a.s.p + from, size[r], &full[stage]);
            if (tensors == 3) bulk_load(slot_of(stage, r, 2), a.ds.p + from, size[r], &full[stage]);
        }
    };
    // The copies under way end, again with a limit, before their place is written to or left: what asked for them waits
    // for either phase of each barrier, whichever is the one under way.
    auto give_up = [&] {
        if (tid == 0)
            for (int i = 0; i < 2 * a.stages; ++i) mbar_wait_limit(&full[i / 2], i & 1, nullptr, 0u, kDrainLimit);
        return false;
    };
    const int64_t own_rows = first < a.rows ? (a.rows - first + a.stride - 1) / a.stride : 0;
    const int64_t tiles = (own_rows + R - 1) / R;
    if (tid == 0)
        for (int i = 0; i < a.stages && i < tiles; ++i) fetch(i, i);
    const F2 zero = pair(0.f, 0.f);
    F2 dg[NV][4], db[NV][4], gm[NV][4];
    Raw8<T> own[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) dg[k][i] = db[k][i] = gm[k][i] = zero;
        const int j = tid + k * threads;
        if (j < pieces) values(load_vector<ROWS>(a.gamma, j * 8 - ph), gm[k]);
        own[k] = row_words<T>(j * 8 - ph, dim);
    }
    float mean[R], rstd[R];
    auto fetch_statistics = [&](int64_t tile) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = first + (tile * R + r) * a.stride;
            if (row < a.rows) {
                mean[r] = __ldg(a.mean + row);
                rstd[r] = __ldg(a.rstd + row);
            }
        }
    };
    fetch_statistics(0);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t tile = 0; tile < tiles; ++tile) {
        // a wait that gives up leaves its code in the flag; later ones do not wait again, and no further tile is asked for
        ok = ok && (mbar_wait_bounded(&full[stage], phase, flag, 0x701u) || give_up());
        float rs[R], sums[2 * R];
        F2 c[R][NV][4], g[R][NV][4];  // s - mean and rstd gamma dy
        Raw8<T> add[R][NV];
        const int64_t left = own_rows - tile * R;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            rs[r] = rstd[r];
            sums[2 * r] = sums[2 * r + 1] = 0.f;
            if (r >= left) continue;
            const F2 minus_mean = pair(-mean[r], -mean[r]), scale = pair(rs[r], rs[r]);
            F2 s1 = zero, s2 = zero;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int j = tid + k * threads;
                if (j >= pieces) continue;
                F2 d[4];
                Raw8<T> dy = load_shared(slot_of(stage, r, 0) + j * 8), x = load_shared(slot_of(stage, r, 1) + j * 8);
                if (tensors == 3) add[r][k] = load_shared(slot_of(stage, r, 2) + j * 8);
                // of the rows in front and behind: dy 0, s 0, so that their products are 0 whatever they hold
                keep_words<ROWS>(dy, own[k]);
                keep_words<ROWS>(x, own[k]);
                values(dy, d);
                values(x, c[r][k]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    c[r][k][i] = c[r][k][i] + minus_mean;
                    db[k][i] = db[k][i] + d[i];
                    d[i] = d[i] * scale;
                    dg[k][i] = fma2(d[i], c[r][k][i], dg[k][i]);
                    g[r][k][i] = d[i] * gm[k][i];
                    s1 = s1 + g[r][k][i];
                    s2 = fma2(g[r][k][i], c[r][k][i], s2);
                }
            }
            sums[2 * r] = sum2(s1);
            sums[2 * r + 1] = sum2(s2);
        }
        if (tile + 1 < tiles) fetch_statistics(tile + 1);
        float (*red)[kMaxWarps] = red_raw[group][tile & 1];
        {
            const float v = warp_sums(sums);
            constexpr int LANES = 32 / (2 * R);  // that hold the same value
            if (lane % LANES == 0) red[lane / LANES][warp] = v;
        }
        group_barrier(group, threads);
        // the tile is in registers: its place is for the one `stages` behind it
        if (tid == 0 && ok && tile + a.stages < tiles) fetch(tile + a.stages, stage);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= left) continue;
            // rstd mean g and rstd^2 mean(g n), negative
            const float m1 = -row_sum(red[2 * r], warps) * a.inv_dim;
            const float m2 = -row_sum(red[2 * r + 1], warps) * a.inv_dim * rs[r] * rs[r];
            const F2 m1s = pair(m1, m1), m2s = pair(m2, m2);
            const int64_t row = first + (tile * R + r) * a.stride;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int j = tid + k * threads;
                if (j >= pieces) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) g[r][k][i] = fma2(c[r][k][i], m2s, g[r][k][i] + m1s);
                if (tensors == 3) {
                    F2 b[4];
                    values(add[r][k], b);
#pragma unroll
                    for (int i = 0; i < 4; ++i) g[r][k][i] = g[r][k][i] + b[i];
                }
                store_values<ROWS>(a.dx, row * dim, j * 8 - ph, dim, g[r][k]);
            }
        }
        if (++stage == a.stages) {
            stage = 0;
            phase ^= 1;
        }
    }
    // the groups' shares of the vectors' gradients join in shared memory, in order
    float *out = a.partial + (int64_t)blockIdx.x * 2 * a.pitch;
    if (groups > 1) {
        __syncthreads();  // all rings have been read, no copy is under way
        float *share = reinterpret_cast<float *>(ring_raw);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = (tid + k * threads) * 8 - ph;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i >= 0 && col + i < dim) {
                    share[(size_t)group * 2 * a.pitch + col + i] = i & 1 ? both(dg[k][i / 2]).y : both(dg[k][i / 2]).x;
                    share[(size_t)group * 2 * a.pitch + a.pitch + col + i] = i & 1 ? both(db[k][i / 2]).y : both(db[k][i / 2]).x;
                }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * a.pitch; c += blockDim.x) {
            if (c % a.pitch >= dim) continue;
            float v = share[c];
            for (int g = 1; g < groups; ++g) v += share[(size_t)g * 2 * a.pitch + c];
            out[c] = v;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int col = (tid + k * threads) * 8 - ph;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i >= 0 && col + i < dim) {
                out[col + i] = i & 1 ? both(dg[k][i / 2]).y : both(dg[k][i / 2]).x;
                out[a.pitch + col + i] = i & 1 ? both(db[k][i / 2]).y : both(db[k][i / 2]).x;
            }
    }
}

// Any rows, any width: a block per row reads it twice.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) layernorm_dx_kernel(const Backward<T> a) {
    __shared__ float2 red[2][kMaxWarps];
    const int dim = a.dim, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
        const float mu = a.mean[row], rs = a.rstd[row];
        const int64_t base = row * dim;
        const int ph = (int)((a.dx.lo + base) & 7);
        float s1 = 0.f, s2 = 0.f;
        auto piece = [&](int col, float (&d)[8], float (&n)[8]) {
            float g[8];
            load_any(a.dy, a.dy.lo + base + col, d);
            load_any(a.s, a.s.lo + base + col, n);
            load_any(a.gamma, a.gamma.lo + col, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[i] *= g[i];
                n[i] = (n[i] - mu) * rs;
            }
            mask_piece<ROWS_ANY>(d, col, dim);
            mask_piece<ROWS_ANY>(n, col, dim);
        };
        for (int col = (int)threadIdx.x * 8 - ph; col < dim; col += blockDim.x * 8) {
            float d[8], n[8];
            piece(col, d, n);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s1 += d[i];
                s2 = fmaf(d[i], n[i], s2);
            }
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (lane == 0) red[parity][warp] = make_float2(s1, s2);
        __syncthreads();
        float m1 = 0.f, m2 = 0.f;
        for (int w = 0; w < warps; ++w) {
            m1 += red[parity][w].x;
            m2 += red[parity][w].y;
        }
        m1 *= a.inv_dim;
        m2 *= a.inv_dim;
        for (int col = (int)threadIdx.x * 8 - ph; col < dim; col += blockDim.x * 8) {
            float d[8], n[8], b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            piece(col, d, n);
            if (a.ds.p) load_any(a.ds, a.ds.lo + base + col, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = fmaf(rs, d[i] - m1 - n[i] * m2, b[i]);
            store_values<ROWS_ANY>(a.dx, base, col, dim, b);
        }
    }
}
// The vectors' gradients beside it: a warp's threads have 8 columns each, the block's 8
// warps and blockIdx.y shares of the rows.
template <typename T> __global__ void __launch_bounds__(256) layernorm_columns_kernel(const Backward<T> a) {
    __shared__ float red[8][2][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col0 = blockIdx.x * 256 + lane * 8;
    grid_dependency_launch();
    float dg[8], db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[i] = db[i] = 0.f;
    if (col0 < a.dim) {
#pragma unroll 2
        for (int64_t row = (int64_t)blockIdx.y * 8 + warp; row < a.rows; row += gridDim.y * 8) {
            const float mu = a.mean[row], rs = a.rstd[row];
            float d[8], n[8];
            load_any(a.dy, a.dy.lo + row * a.dim + col0, d);
            load_any(a.s, a.s.lo + row * a.dim + col0, n);
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // what lies behind the row reaches columns that nobody asks for
                dg[i] = fmaf(d[i], (n[i] - mu) * rs, dg[i]);
                db[i] += d[i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        red[warp][0][lane * 8 + i] = dg[i];
        red[warp][1][lane * 8 + i] = db[i];
    }
    __syncthreads();
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col >= a.dim) return;
    float *out = a.partial + (int64_t)blockIdx.y * 2 * a.pitch + col;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float v = red[0][k][threadIdx.x];
        for (int w = 1; w < 8; ++w) v += red[w][k][threadIdx.x];
        out[k * a.pitch] = v;
    }
}

// dgamma[j] (blockIdx.y 0) and dbeta[j] (1) from the blocks' partials: 32 columns
// per block, 32 threads per column, joined in a fixed order.
__global__ void __launch_bounds__(1024) layernorm_join_kernel(const float *partial, int blocks, int dim, int pitch,
                                                              float *dgamma, float *dbeta) {
    __shared__ float red[32][33];
    grid_dependency_wait();
    const int c = threadIdx.x & 31, w = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
    const float *from = partial + blockIdx.y * pitch + col;
    float v = 0.f;
    if (col < dim) {
#pragma unroll 8
        for (int b = w; b < blocks; b += 32) v += from[(int64_t)b * 2 * pitch];
    }
    red[w][c] = v;
    __syncthreads();
    v = warp_sum(red[c][w]);  // warp w adds up column w of the block's 32
    if (c == 0 && blockIdx.x * 32 + w < dim) (blockIdx.y ? dbeta : dgamma)[blockIdx.x * 32 + w] = v;
}

// ---- launches ----------------------------------------------------------------------------

// how the rows of the given tensors lie
int rows_of(int dim, std::initializer_list<const void *> tensors) {
    for (const void *p : tensors)
        if (!aligned16(p)) return ROWS_ANY;
    return dim % 8 == 0 ? ROWS_VEC : ROWS_ODD;
}

// Forward: pieces per thread and threads of a row.  A warp has a row to itself up to 256 or 512 values
// (bf16: 1024).  Then 2 pieces, or 4 of aligned bf16 (fewer warps wait at a row's barrier): cold, 2 / 4 pieces,
// bf16 65536 x 1024 91 / 89 us, x 2048 178 / 163, 16384 x 8192 205 / 185; fp32 16384 x 4096 172 / 176,
// 8192 x 8192 233 / 202; odd 32768 x 2046 153 / 162.  Rows above 8192 take as many as there are (bf16
// 4096 x 16384 with 8 pieces 92 us, 126 with 4 and twice the warps).
struct Shape {
    int nv, threads;
};
template <typename T> Shape forward_shape(int dim, int rows) {
    const int64_t pieces = rows == ROWS_VEC ? dim / 8 : (dim + 14) / 8;
    int nv = pieces <= 32 ? 1 : 2;
    if (rows == ROWS_VEC && pieces > (sizeof(T) == 2 ? 64 : kMaxThreads)) nv = 4;
    if (pieces > kMaxThreads * 2) nv = rows == ROWS_VEC ? 8 : kMaxPieces;
    return {nv, (int)round_up(ceil_div(pieces, nv), 32)};
}

template <typename T, int ROWS> int run_forward(const Forward<T> &a, cudaStream_t st) {
    const Shape sh = forward_shape<T>(a.dim, ROWS);
    constexpr bool VEC = ROWS == ROWS_VEC;
    const bool warp = sh.threads == 32;
    auto *k = sh.nv == 1   ? &layernorm_forward_kernel<T, ROWS, 1, true>
              : sh.nv == 2 ? (warp ? &layernorm_forward_kernel<T, ROWS, 2, true> : &layernorm_forward_kernel<T, ROWS, 2, false>)
              : sh.nv == 4 ? (warp ? &layernorm_forward_kernel<T, ROWS, VEC && sizeof(T) == 2 ? 4 : 1, true>
                                   : &layernorm_forward_kernel<T, ROWS, VEC ? 4 : 2, false>)
                           : &layernorm_forward_kernel<T, ROWS, VEC ? 8 : kMaxPieces, false>;
    // 8 rows per block, or multiples of 8 blocks: a thread's rows then begin alike
    const int64_t grid = warp ? std::min<int64_t>(ceil_div(a.rows, 8), (int64_t)num_sms() * 8)
                              : std::min<int64_t>(a.rows, (int64_t)num_sms() * 64);
    SPCO_LAUNCH("layernorm_forward", st, k<<<(unsigned)grid, warp ? 256 : sh.threads, 0, st>>>(a));
    SPECOPTIM_LAUNCHED("layernorm_forward_kernel");
    return SPECOPTIM_OK;
}

// Backward: how a launch is cut.
struct Plan {
    bool ring;         // rows through shared memory, else the two kernels that take any rows
    int nv, threads;   // of a group
    int groups, blocks;
    int tile, stages, slot, smem;
};
Plan backward_plan(int64_t rows, int dim, int layout, int value_bytes, int tensors) {
    Plan p{};
    const int pieces = layout == ROWS_VEC ? dim / 8 : (dim + 14) / 8;
    if (layout == ROWS_ANY || pieces > 2 * kMaxThreads) {
        // shares of the rows beside the columns' blocks, 8 rows at a time each
        p.blocks = (int)std::max<int64_t>(1, std::min<int64_t>(ceil_div(rows, 8), ceil_div(num_sms() * 8, ceil_div(dim, 256))));
        return p;
    }
    p.ring = true;
    p.nv = pieces <= kMaxThreads ? 1 : 2;
    p.threads = (int)round_up(ceil_div(pieces, p.nv), 32);
    p.groups = std::max(1, std::min(kMaxGroups, 256 / p.threads));
    p.slot = (int)round_up((int64_t)pieces * 8 * value_bytes, 16);
    // Two rows a tile: a barrier and its sums for two (bf16 65536 x 2048: 179 us, 206 with one; four spill).
    // 512 threads an SM: the ring's bytes are in flight all the same (163 against 171 us without ds).
    p.tile = p.nv == 1 ? 2 : 1;
    const int stage_bytes = p.groups * p.tile * p.slot * tensors, room = 220 * 1024;
    p.stages = std::max(1, std::min(3, room / stage_bytes));
    p.smem = std::max<int>(p.stages * stage_bytes, p.groups > 1 ? p.groups * 2 * (int)round_up(dim, 8) * 4 : 0);
    const int per_sm = std::max(1, std::min(room / (p.smem + 3 * 1024), 512 / (p.threads * p.groups)));
    p.blocks = (int)std::min<int64_t>(ceil_div(rows, p.groups), (int64_t)num_sms() * per_sm / 8 * 8);
    p.blocks = std::max(p.blocks, 1);
    return p;
}

template <typename T> int run_backward(Backward<T> a, const Plan &p, int layout, float *dgamma, float *dbeta, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (p.ring) {
        a.threads = p.threads;
        a.slot = p.slot;
        a.stages = p.stages;
        a.stride = (int64_t)p.blocks * p.groups;
        auto pick = [&](auto rows) {
            constexpr int ROWS = decltype(rows)::value;
            return p.nv == 2     ? &layernorm_backward_kernel<T, ROWS, 2, 1>
                                 : &layernorm_backward_kernel<T, ROWS, 1, 2>;
        };
        auto *k = layout == ROWS_VEC ? pick(std::integral_constant<int, ROWS_VEC>{}) : pick(std::integral_constant<int, ROWS_ODD>{});
        if (int rc = set_smem_limit(reinterpret_cast<const void *>(k), p.smem)) return rc;
        SPCO_LAUNCH("layernorm_backward", st,
                    k<<<p.blocks, p.threads * p.groups, p.smem, st>>>(a, device_flag_ptr()));
        SPECOPTIM_LAUNCHED("layernorm_backward_kernel");
    } else {
        // the columns first: dx may overwrite dy
        SPCO_LAUNCH("layernorm_columns", st,
                    layernorm_columns_kernel<T><<<dim3((unsigned)ceil_div(a.dim, 256), p.blocks), 256, 0, st>>>(a));
        SPECOPTIM_LAUNCHED("layernorm_columns_kernel");
        const int threads = (int)std::min<int64_t>(kMaxThreads, round_up(ceil_div(a.dim + 7, 8), 32));
        if (a.rows > 0)
            SPCO_LAUNCH("layernorm_dx", st,
                        layernorm_dx_kernel<T><<<(unsigned)std::min<int64_t>(a.rows, num_sms() * 16), threads, 0, st>>>(a));
        SPECOPTIM_LAUNCHED("layernorm_dx_kernel");
    }
    SPCO_LAUNCH("layernorm_join", st,
                e = launch_dependent(layernorm_join_kernel, dim3((unsigned)ceil_div(a.dim, 32), dbeta ? 2 : 1), dim3(1024), 0,
                                     st, a.partial, p.blocks, a.dim, a.pitch, dgamma, dbeta));
    SPECOPTIM_CUDA(e);
    return SPECOPTIM_OK;
}

int check_sizes(int64_t rows, int32_t dim, int32_t type, const std::string &what) {
    if (rows < 0 || rows > INT32_MAX) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": rows outside [0, 2^31)");
    if (dim < 1 || dim > kMaxDim) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": dim outside [1, 32768]");
    if (!type_ok(type)) return fail(SPECOPTIM_ERR_INVALID_ARG, what + ": type must be STAGE_BF16 or STAGE_FP32");
    return SPECOPTIM_OK;
}

// f(T{}) for the tensors' type
template <typename F> int with_type(int32_t type, F &&f) { return type == STAGE_BF16 ? f(bf16{}) : f(float{}); }

}  // namespace
}  // namespace spco

using namespace spco;

extern "C" int layernorm_forward(const void *x, const void *r, const void *gamma, const void *beta, int32_t type, float eps,
                                 void *s, void *y, float *mean, float *rstd, int64_t rows, int32_t dim, void *stream) {
    return entry([&]() -> int {
        if (int rc = check_sizes(rows, dim, type, "layernorm_forward")) return rc;
        if (!(eps >= 0.f)) return fail(SPECOPTIM_ERR_INVALID_ARG, "layernorm_forward: eps must be >= 0");
        if (rows == 0) return SPECOPTIM_OK;
        if (!x || !gamma || !y || !mean || !rstd || (r && !s))
            return fail(SPECOPTIM_ERR_INVALID_ARG, "layernorm_forward: null pointer");
        const size_t b = type_bytes(type);
        if (!aligned_to(x, b) || !aligned_to(r, b) || !aligned_to(gamma, b) || !aligned_to(beta, b) ||
            !aligned_to(y, b) || (r && !aligned_to(s, b)) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
            return fail(SPECOPTIM_ERR_MISALIGNED, "layernorm_forward: pointers must be aligned to their elements");
        if (int rc = bind_device()) return rc;
        const int layout = rows_of(dim, {x, r, gamma, beta, y, r ? s : nullptr});
        const int64_t n = rows * dim;
        return with_type(type, [&](auto t) -> int {
            using T = decltype(t);
            const Forward<T> a{{static_cast<const T *>(x), n},
                               {static_cast<const T *>(r), n},
                               {static_cast<const T *>(gamma), dim},
                               {static_cast<const T *>(beta), dim},
                               {static_cast<T *>(s), n},
                               {static_cast<T *>(y), n},
                               mean,
                               rstd,
                               rows,
                               dim,
                               1.f / (float)dim,
                               eps};
            cudaStream_t st = static_cast<cudaStream_t>(stream);
            return layout == ROWS_VEC   ? run_forward<T, ROWS_VEC>(a, st)
                   : layout == ROWS_ODD ? run_forward<T, ROWS_ODD>(a, st)
                                        : run_forward<T, ROWS_ANY>(a, st);
        });
    });
}

extern "C" int64_t layernorm_backward_workspace(int64_t rows, int32_t dim) {
    int64_t bytes = -1;
    entry([&]() -> int {
        if (int rc = check_sizes(rows, dim, STAGE_BF16, "layernorm_backward")) return rc;
        // the most blocks of any type and layout that such rows can have: the call's are not known yet
        int blocks = 1;
        for (const int layout : {dim % 8 == 0 ? ROWS_VEC : ROWS_ODD, ROWS_ANY})
            for (const int value_bytes : {2, 4})
                for (const int tensors : {2, 3})
                    blocks = std::max(blocks, backward_plan(rows, dim, layout, value_bytes, tensors).blocks);
        bytes = (int64_t)blocks * 2 * round_up(dim, 8) * 4;
        return SPECOPTIM_OK;
    });
    return bytes;
}

extern "C" int layernorm_backward(const void *dy, const void *ds, const void *s, const float *mean, const float *rstd,
                                  const void *gamma, int32_t type, void *dx, float *dgamma, float *dbeta, int64_t rows,
                                  int32_t dim, void *workspace, int64_t workspace_bytes, void *stream) {
    return entry([&]() -> int {
        if (int rc = check_sizes(rows, dim, type, "layernorm_backward")) return rc;
        if (!gamma || !dgamma || !workspace || (rows > 0 && (!dy || !s || !mean || !rstd || !dx)))
            return fail(SPECOPTIM_ERR_INVALID_ARG, "layernorm_backward: null pointer");
        const size_t b = type_bytes(type);
        if (!aligned_to(dy, b) || !aligned_to(ds, b) || !aligned_to(s, b) || !aligned_to(gamma, b) || !aligned_to(dx, b) ||
            !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(dgamma, 4) || !aligned_to(dbeta, 4) ||
            !aligned16(workspace))
            return fail(SPECOPTIM_ERR_MISALIGNED, "layernorm_backward: pointers must be aligned to their elements, the workspace to 16 bytes");
        const int layout = rows_of(dim, {dy, ds, s, gamma, dx});
        const Plan p = backward_plan(rows, dim, layout, (int)b, ds ? 3 : 2);
        const int pitch = (int)round_up(dim, 8);
        if (workspace_bytes < (int64_t)p.blocks * 2 * pitch * 4)
            return fail(SPECOPTIM_ERR_INVALID_ARG, "layernorm_backward: the workspace is smaller than layernorm_backward_workspace() says");
        if (int rc = bind_device()) return rc;
        const int64_t n = rows * dim;
        return with_type(type, [&](auto t) -> int {
            using T = decltype(t);
            Backward<T> a{{static_cast<const T *>(dy), n},
                          {static_cast<const T *>(ds), n},
                          {static_cast<const T *>(s), n},
                          {static_cast<const T *>(gamma), dim},
                          mean,
                          rstd,
                          {static_cast<T *>(dx), n},
                          static_cast<float *>(workspace),
                          rows,
                          1,
                          dim,
                          pitch,
                          0,
                          0,
                          0,
                          1.f / (float)dim};
            return run_backward<T>(a, p, layout, dgamma, dbeta, static_cast<cudaStream_t>(stream));
        });
    });
}
