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
// and walks over rows, R at a time, that arrive in shared memory by asynchronous
// copies some tiles ahead.  A tile is read twice from there, for the row sums and
// for dx, so that little has to stay in registers but the columns' shares of
// dgamma and dbeta, of which each block leaves one partial; a last launch adds the
// partials in their order.
//
// Rows that are not multiples of 16 bytes (ROWS_ODD) are cut where memory is: a
// thread's 8 values begin at a multiple of 8 of the tensor, the first ph of the
// row's first piece belong to the row in front.  The rows of a group lie a
// multiple of 8 rows apart, so ph is the same for all of them.
//
// All statistics and sums are fp32; s, y and dx are rounded once to their type.
#include <algorithm>
#include <string>

#include "../../include/finetune.h"
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

// values i .. i + 7 of the tensor
template <int ROWS, typename T> __device__ __forceinline__ void load_piece8(const Span<const T> &s, int64_t i, float (&v)[8]) {
    if (ROWS == ROWS_VEC || (ROWS == ROWS_ODD && i + 8 <= s.hi)) {
        load8(s.p + i, v);
    } else if (ROWS == ROWS_ANY) {
        load_any(s, s.lo + i, v);
    } else {  // the tensor's last piece is cut short
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = i + k < s.hi ? to_f(s.p[i + k]) : 0.f;
    }
}

// v to columns col .. col + 7 of the row that begins at value `row`, as far as they exist
template <int ROWS, typename T>
__device__ __forceinline__ void store_piece8(const Span<T> &s, int64_t row, int col, int dim, const float (&v)[8]) {
    T *p = s.p + s.lo + row + col;
    const bool whole = ROWS == ROWS_VEC || (col >= 0 && col + 8 <= dim &&
                                            (ROWS == ROWS_ODD || (reinterpret_cast<uintptr_t>(p) & 15) == 0));
    if (whole) {
        store8(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i >= 0 && col + i < dim) p[i] = from_f<T>(v[i]);
    }
}

// zeros for the values that belong to the rows in front and behind
template <int ROWS> __device__ __forceinline__ void mask_piece(float (&v)[8], int col, int dim) {
    if (ROWS != ROWS_VEC && (col < 0 || col + 8 > dim)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < 0 || col + i >= dim) v[i] = 0.f;
    }
}

// a vector of dim values (gamma, beta), at any place
template <int ROWS, typename T> __device__ __forceinline__ void load_vector(const Span<const T> &s, int col, float (&v)[8]) {
    if (ROWS == ROWS_VEC) load8(s.p + col, v);
    else load_any(s, s.lo + col, v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---- forward -----------------------------------------------------------------------------

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
__global__ void __launch_bounds__(kMaxThreads, NV * sizeof(T) <= 4 ? 2 : 1) layernorm_forward_kernel(const Forward<T> a) {
    __shared__ float2 red[2][kMaxWarps];   // each warp's mean and sum of squares about it
    __shared__ float count_of[kMaxWarps];  // its values
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
        if (lane == 0) count_of[warp] = own;
        __syncthreads();
    }
    // the vectors stay in registers where a thread has few pieces
    float gm[NV <= 2 ? NV : 1][8], bt[NV <= 2 ? NV : 1][8];
    if (NV <= 2) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = col0 + k * step;
#pragma unroll
            for (int i = 0; i < 8; ++i) bt[k < 2 ? k : 0][i] = 0.f;
            if (col >= dim) continue;
            load_vector<ROWS>(a.gamma, col, gm[k < 2 ? k : 0]);
            if (a.beta.p) load_vector<ROWS>(a.beta, col, bt[k < 2 ? k : 0]);
        }
    }
    int parity = 0;
    for (int64_t row = first; row < a.rows; row += stride, parity ^= 1) {
        const int64_t base = row * dim;
        float s[NV][8];
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (col0 + k * step < dim) load_piece8<ROWS>(a.x, base + col0 + k * step, s[k]);
        if (a.r.p) {
            float b[NV][8];
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (col0 + k * step < dim) load_piece8<ROWS>(a.r, base + col0 + k * step, b[k]);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = col0 + k * step;
                if (col >= dim) continue;
                // the stream is held in T: the norm is that of the rounded sum
#pragma unroll
                for (int i = 0; i < 8; ++i) s[k][i] = to_f(from_f<T>(s[k][i] + b[k][i]));
                store_piece8<ROWS>(a.s, base, col, dim, s[k]);
            }
        }
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (col0 + k * step >= dim) continue;
            mask_piece<ROWS>(s[k], col0 + k * step, dim);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += s[k][i];
        }
        const float mid = warp_sum(sum) * inv_own;
        float sq = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = col0 + k * step;
            if (col >= dim) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = s[k][i] - mid;
                if (ROWS == ROWS_VEC || (col + i >= 0 && col + i < dim)) sq = fmaf(d, d, sq);
            }
        }
        sq = warp_sum(sq);
        float mean = mid;
        if (!WARP) {
            if (lane == 0) red[parity][warp] = make_float2(mid, sq);
            __syncthreads();
            mean = 0.f;
            for (int w = 0; w < warps; ++w) mean = fmaf(count_of[w], red[parity][w].x, mean);
            mean *= a.inv_dim;
            sq = 0.f;
            for (int w = 0; w < warps; ++w) {
                const float2 p = red[parity][w];
                const float d = p.x - mean;
                sq += fmaf(count_of[w] * d, d, p.y);
            }
        }
        const float rs = rsqrtf(fmaf(sq, a.inv_dim, a.eps));
        if (tid == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rs;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int col = col0 + k * step;
            if (col >= dim) continue;
            if (NV <= 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i) s[k][i] = fmaf((s[k][i] - mean) * rs, gm[k < 2 ? k : 0][i], bt[k < 2 ? k : 0][i]);
            } else {
                float g[8], b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                load_vector<ROWS>(a.gamma, col, g);
                if (a.beta.p) load_vector<ROWS>(a.beta, col, b);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[k][i] = fmaf((s[k][i] - mean) * rs, g[i], b[i]);
            }
            store_piece8<ROWS>(a.y, base, col, dim, s[k]);
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

__device__ __forceinline__ void group_barrier(int group, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

constexpr int kMaxStages = 4, kMaxGroups = 8;

// Dynamic shared memory: for each group a ring [stage][row][dy, s, ds][slot].
template <typename T, int ROWS, int NV, int R>
__global__ void __launch_bounds__(kMaxThreads, 1) layernorm_backward_kernel(const Backward<T> a, unsigned *flag) {
    extern __shared__ __align__(16) unsigned char ring_raw[];
    __shared__ uint64_t full_bars[kMaxGroups][kMaxStages];
    __shared__ float red_raw[kMaxGroups][2][2 * R][kMaxWarps];
    const int threads = a.threads, group = threadIdx.x / threads, tid = threadIdx.x % threads, groups = blockDim.x / threads;
    const int lane = threadIdx.x & 31, warp = tid >> 5, warps = threads >> 5;
    const int dim = a.dim, tensors = a.ds.p ? 3 : 2;
    const int64_t first = (int64_t)blockIdx.x * groups + group;
    const int ph = ROWS == ROWS_VEC ? 0 : (int)((first * dim) & 7);
    const int pieces = (ph + dim + 7) / 8;
    uint64_t *full = full_bars[group];
    unsigned char *ring = ring_raw + (size_t)group * a.stages * R * tensors * a.slot;
    grid_dependency_launch();
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
        uint32_t bytes = 0;
        int64_t from[R];
        uint32_t size[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = first + (tile * R + r) * a.stride;
            size[r] = 0;
            if (row >= a.rows) continue;
            from[r] = row * dim - ph;
            const int64_t values = min((int64_t)pieces * 8, a.dy.hi - from[r]);
            size[r] = (uint32_t)(values * sizeof(T)) & ~15u;
            if (ROWS != ROWS_VEC) {  // what the tensor's last 16 bytes lack
                for (int64_t i = size[r] / sizeof(T); i < values; ++i) {
                    slot_of(stage, r, 0)[i] = a.dy.p[from[r] + i];
                    slot_of(stage, r, 1)[i] = a.s.p[from[r] + i];
                    if (tensors == 3) slot_of(stage, r, 2)[i] = a.ds.p[from[r] + i];
                }
            }
            bytes += size[r] * tensors;
        }
        mbar_arrive_expect_tx(&full[stage], bytes);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!size[r]) continue;
            bulk_load(slot_of(stage, r, 0), a.dy.p + from[r], size[r], &full[stage]);
            bulk_load(slot_of(stage, r, 1), a.s.p + from[r], size[r], &full[stage]);
            if (tensors == 3) bulk_load(slot_of(stage, r, 2), a.ds.p + from[r], size[r], &full[stage]);
        }
    };
    const int64_t own_rows = first < a.rows ? (a.rows - first + a.stride - 1) / a.stride : 0;
    const int64_t tiles = (own_rows + R - 1) / R;
    if (tid == 0)
        for (int i = 0; i < a.stages && i < tiles; ++i) fetch(i, i);
    float dg[NV][8], db[NV][8], gm[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[k][i] = db[k][i] = gm[k][i] = 0.f;
        const int j = tid + k * threads;
        if (j < pieces) load_vector<ROWS>(a.gamma, j * 8 - ph, gm[k]);
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
        // a wait that gives up leaves its code in the flag; later ones do not wait again
        ok = ok && mbar_wait_bounded(&full[stage], phase, flag, 0x701u);
        float mu[R], rs[R], sums[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mu[r] = mean[r];
            rs[r] = rstd[r];
            sums[2 * r] = sums[2 * r + 1] = 0.f;
        }
        const int64_t left = own_rows - tile * R;
        if (tile + 1 < tiles) fetch_statistics(tile + 1);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= left) continue;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int j = tid + k * threads;
                if (j >= pieces) continue;
                float d[8], n[8];
                load8(slot_of(stage, r, 0) + j * 8, d);
                load8(slot_of(stage, r, 1) + j * 8, n);
#pragma unroll
                for (int i = 0; i < 8; ++i) n[i] = (n[i] - mu[r]) * rs[r];
                mask_piece<ROWS>(d, j * 8 - ph, dim);
                mask_piece<ROWS>(n, j * 8 - ph, dim);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dg[k][i] = fmaf(d[i], n[i], dg[k][i]);
                    db[k][i] += d[i];
                    const float g = d[i] * gm[k][i];
                    sums[2 * r] += g;
                    sums[2 * r + 1] = fmaf(g, n[i], sums[2 * r + 1]);
                }
            }
        }
        float (*red)[kMaxWarps] = red_raw[group][tile & 1];
        {
            const float v = warp_sums(sums);
            constexpr int LANES = 32 / (2 * R);  // that hold the same value
            if (lane % LANES == 0) red[lane / LANES][warp] = v;
        }
        group_barrier(group, threads);
        // the tile in front is done with: its place is for the one `stages` behind it
        if (tid == 0 && tile > 0 && tile - 1 + a.stages < tiles)
            fetch(tile - 1 + a.stages, stage == 0 ? a.stages - 1 : stage - 1);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= left) continue;
            float m1 = 0.f, m2 = 0.f;
            for (int w = 0; w < warps; ++w) {
                m1 += red[2 * r][w];
                m2 += red[2 * r + 1][w];
            }
            m1 *= a.inv_dim;
            m2 *= a.inv_dim;
            const int64_t row = first + (tile * R + r) * a.stride;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int j = tid + k * threads;
                if (j >= pieces) continue;
                float d[8], n[8], b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                load8(slot_of(stage, r, 0) + j * 8, d);
                load8(slot_of(stage, r, 1) + j * 8, n);
                if (tensors == 3) load8(slot_of(stage, r, 2) + j * 8, b);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float t = fmaf(d[i], gm[k][i], -m1) - (n[i] - mu[r]) * rs[r] * m2;
                    b[i] = fmaf(rs[r], t, b[i]);
                }
                store_piece8<ROWS>(a.dx, row * dim, j * 8 - ph, dim, b);
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
                    share[(size_t)group * 2 * a.pitch + col + i] = dg[k][i];
                    share[(size_t)group * 2 * a.pitch + a.pitch + col + i] = db[k][i];
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
                out[col + i] = dg[k][i];
                out[a.pitch + col + i] = db[k][i];
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
            store_piece8<ROWS_ANY>(a.dx, base, col, dim, b);
        }
    }
}
// The vectors' gradients beside it: a thread per column, blockIdx.y a share of the rows.
template <typename T> __global__ void __launch_bounds__(256) layernorm_columns_kernel(const Backward<T> a) {
    const int col = blockIdx.x * 256 + threadIdx.x;
    grid_dependency_launch();
    if (col >= a.dim) return;
    const T *dy = a.dy.p + a.dy.lo + col, *s = a.s.p + a.s.lo + col;
    float dg = 0.f, db = 0.f;
#pragma unroll 4
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float d = to_f(dy[row * a.dim]);
        dg = fmaf(d, (to_f(s[row * a.dim]) - a.mean[row]) * a.rstd[row], dg);
        db += d;
    }
    float *out = a.partial + (int64_t)blockIdx.y * 2 * a.pitch + col;
    out[0] = dg;
    out[a.pitch] = db;
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

// Forward: pieces and threads of a row; a warp has a row to itself up to 2 pieces a lane.
struct Shape {
    int nv, threads;
};
Shape forward_shape(int dim, int rows) {
    const int64_t pieces = rows == ROWS_VEC ? dim / 8 : (dim + 14) / 8;
    int nv = pieces <= 32 ? 1 : 2;
    while (nv < 8 && pieces > kMaxThreads * nv) nv *= 2;
    if (pieces > kMaxThreads * nv) nv = kMaxPieces;
    return {nv, (int)round_up(ceil_div(pieces, nv), 32)};
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

template <typename T> int run_forward(const Forward<T> &a, int rows, cudaStream_t st) {
    const Shape sh = forward_shape(a.dim, rows);
    return with_nv(sh.nv, [&](auto nv) -> int {
        constexpr int NV = decltype(nv)::value;
        if (NV <= 2 && sh.threads == 32) {  // a warp per row, 8 rows per block
            const int64_t grid = std::min<int64_t>(ceil_div(a.rows, 8), (int64_t)num_sms() * 8);
            constexpr int N = NV <= 2 ? NV : 1;
            auto *k = rows == ROWS_VEC   ? &layernorm_forward_kernel<T, ROWS_VEC, N, true>
                      : rows == ROWS_ODD ? &layernorm_forward_kernel<T, ROWS_ODD, N, true>
                                         : &layernorm_forward_kernel<T, ROWS_ANY, N, true>;
            SPCO_LAUNCH("layernorm_forward", st, k<<<(unsigned)grid, 256, 0, st>>>(a));
        } else {
            // multiples of 8 blocks: a block's rows then begin alike
            const int64_t grid = std::min<int64_t>(a.rows, (int64_t)num_sms() * 64);
            auto *k = rows == ROWS_VEC   ? &layernorm_forward_kernel<T, vec_rows(NV), NV, false>
                      : rows == ROWS_ODD ? &layernorm_forward_kernel<T, ROWS_ODD, NV, false>
                                         : &layernorm_forward_kernel<T, ROWS_ANY, NV, false>;
            SPCO_LAUNCH("layernorm_forward", st, k<<<(unsigned)grid, sh.threads, 0, st>>>(a));
        }
        SPECOPTIM_LAUNCHED("layernorm_forward_kernel");
        return SPECOPTIM_OK;
    });
}

// Backward: how a launch is cut.
struct Plan {
    bool ring;         // rows through shared memory, else the two kernels that take any rows
    int nv, threads;   // of a group
    int groups, blocks;
    int tile, stages, slot, smem;
};
constexpr int kRingDim = 8192;

Plan backward_plan(int64_t rows, int dim, int layout, int value_bytes, int tensors) {
    Plan p{};
    if (layout == ROWS_ANY || dim > kRingDim) {
        p.blocks = (int)std::max<int64_t>(1, std::min<int64_t>({rows, num_sms() * 4, 512}));
        return p;
    }
    p.ring = true;
    const int pieces = layout == ROWS_VEC ? dim / 8 : (dim + 14) / 8;
    p.nv = pieces <= kMaxThreads ? 1 : pieces <= 2 * kMaxThreads ? 2 : 4;
    p.threads = (int)round_up(ceil_div(pieces, p.nv), 32);
    p.groups = std::max(1, std::min(kMaxGroups, 256 / p.threads));
    p.slot = (int)round_up((int64_t)pieces * 8 * value_bytes, 16);
    p.tile = 2;
    p.stages = 3;
    const int row_bytes = p.slot * tensors;
    const int room = 220 * 1024;
    while (p.stages > 2 && p.groups * p.stages * p.tile * row_bytes > room) --p.stages;
    if (p.groups * p.stages * p.tile * row_bytes > room) p.tile = 1;
    p.smem = std::max<int>(p.groups * p.stages * p.tile * row_bytes,
                           p.groups > 1 ? p.groups * 2 * (int)round_up(dim, 8) * 4 : 0);
    const int per_sm = std::max(1, std::min({room / (p.smem + 3072), 1024 / (p.threads * p.groups)}));
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
        auto pick = [&](auto nv) {
            constexpr int NV = decltype(nv)::value;
            return layout == ROWS_VEC ? (p.tile == 2 ? &layernorm_backward_kernel<T, ROWS_VEC, NV, 2>
                                                     : &layernorm_backward_kernel<T, ROWS_VEC, NV, 1>)
                                      : (p.tile == 2 ? &layernorm_backward_kernel<T, ROWS_ODD, NV, 2>
                                                     : &layernorm_backward_kernel<T, ROWS_ODD, NV, 1>);
        };
        auto *k = p.nv == 1   ? pick(std::integral_constant<int, 1>{})
                  : p.nv == 2 ? pick(std::integral_constant<int, 2>{})
                              : pick(std::integral_constant<int, 4>{});
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
            return run_forward<T>(a, layout, static_cast<cudaStream_t>(stream));
        });
    });
}

extern "C" int64_t layernorm_backward_workspace(int64_t rows, int32_t dim) {
    int64_t bytes = -1;
    entry([&]() -> int {
        if (int rc = check_sizes(rows, dim, STAGE_BF16, "layernorm_backward")) return rc;
        // the most blocks of any type and layout: the call's are not known yet
        int blocks = 1;
        for (const int layout : {ROWS_VEC, ROWS_ODD, ROWS_ANY})
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
