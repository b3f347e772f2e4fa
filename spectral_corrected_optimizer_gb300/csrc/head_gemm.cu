// tcgen05 products of the vocabulary head (include/stage_ends.h, head_loss*):
// bf16 operands (kind::f16), fp32 accumulation in TMEM.
//
//   l  = H W^T                 logits of a 128 x 256 tile, never stored: the
//                              epilogue reduces them to row statistics
//                              (HEAD_STATS) or turns them into a piece of
//                              softmax - onehot (HEAD_PROB)
//   dh = P W,  dw = P^T H      P a piece [rows][vocabulary rows of the piece]
//
// One persistent CTA per SM walks the tiles of up to three jobs (the next
// piece's probabilities beside the previous piece's two products, which do not
// depend on each other): warp 0 loads, one lane of warp 1 issues the MMAs, warps
// 2-9 run the epilogues from one of two TMEM accumulators while the other is
// being filled.  H, W and the pieces are read in 64 x 64 boxes with 128-byte
// swizzle; the same box serves an operand whose rows run along K (one row per M
// or N index) and one whose rows run along M or N (one row per k), so none of
// the four products needs a transposed copy.
//
// Every wait on an mbarrier is bounded, as in gemm_tc.cu.
#include <algorithm>
#include <cstring>

#include "head_gemm.cuh"

namespace spco {
namespace {

constexpr int BM = kHeadTileM, BN = kHeadTileN, BK = 64;
constexpr int STAGES = 4;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = (2 + EPI_WARPS) * 32;
constexpr uint32_t BOX_BYTES = 64 * 64 * 2;
constexpr uint32_t A_BYTES = BM * BK * 2;
constexpr uint32_t STAGE_BYTES = A_BYTES + BN * BK * 2;
constexpr uint32_t TMEM_COLS = 2 * BN;
constexpr size_t SMEM_BYTES = (size_t)STAGES * STAGE_BYTES + 1024 + 256;
static_assert(SMEM_BYTES <= 232448, "shared memory budget of one CTA");
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One tile of a job: where its operands start and how far k runs.
struct Tile {
    int kind, piece, job;
    int m, n;        // first row (M) and column (N) of the tile
    int k0, kb;      // first k, number of 64-k blocks
    int v0, width;   // vocabulary rows of the job's piece
    int split, add;
};

struct Walk {
    int rows, m_tiles, d_tiles;
    int tiles[kHeadJobs], total;
};

__device__ __forceinline__ Walk make_walk(const HeadGemm &g) {
    Walk w;
    w.rows = g.state->rows;
    w.m_tiles = (w.rows + BM - 1) / BM;
    w.d_tiles = (g.dim + BN - 1) / BN;
    w.total = 0;
#pragma unroll
    for (int j = 0; j < kHeadJobs; ++j) {
        int t = 0;
        if (j < g.jobs) {
            const HeadJob &q = g.job[j];
            if (q.kind <= HEAD_PROB) t = w.m_tiles * ((q.width + BN - 1) / BN);
            else if (q.kind == HEAD_DH) t = w.m_tiles * w.d_tiles * q.splits;
            else t = ((q.width + BM - 1) / BM) * w.d_tiles;
        }
        w.tiles[j] = t;
        w.total += t;
    }
    return w;
}

__device__ __forceinline__ Tile tile_at(const HeadGemm &g, const Walk &w, int t) {
    int j = 0;
    while (j + 1 < g.jobs && t >= w.tiles[j]) t -= w.tiles[j++];
    const HeadJob &q = g.job[j];
    Tile x;
    x.kind = q.kind;
    x.piece = q.piece;
    x.job = j;
    x.v0 = q.v0;
    x.width = q.width;
    x.split = 0;
    x.add = q.add;
    x.k0 = 0;
    if (q.kind <= HEAD_PROB) {         // M = rows (fastest: a W tile is read from DRAM once), N = vocabulary, K = dim
        x.m = (t % w.m_tiles) * BM;
        x.n = (t / w.m_tiles) * BN;
        x.kb = (g.dim + BK - 1) / BK;
    } else if (q.kind == HEAD_DH) {    // M = rows, N = dim, K = the piece's vocabulary rows, in `splits` parts
        const int per = w.m_tiles * w.d_tiles;
        x.split = t / per;
        t -= x.split * per;
        x.n = (t % w.d_tiles) * BN;
        x.m = (t / w.d_tiles) * BM;
        const int blocks = (q.width + BK - 1) / BK;
        const int b0 = (int)((int64_t)blocks * x.split / q.splits);
        const int b1 = (int)((int64_t)blocks * (x.split + 1) / q.splits);
        x.k0 = b0 * BK;
        x.kb = b1 - b0;
    } else {                           // M = the piece's vocabulary rows, N = dim, K = rows
        x.n = (t % w.d_tiles) * BN;
        x.m = (t / w.d_tiles) * BM;
        x.kb = (w.rows + BK - 1) / BK;
    }
    return x;
}

// ---- epilogues: thread = one row of the tile, 32 columns at a time -------------------

__device__ __forceinline__ void epilogue_stats(const HeadGemm &g, const Walk &w, const Tile &x, uint32_t acc, int q,
                                               int lane, int half) {
    const int row = x.m + q * 32 + lane;
    const int target = row < w.rows ? g.target[row] : -1;
    float m = -INFINITY, s = 0.f;
    for (int c = 0; c < BN / 2 / 32; ++c) {
        const int col0 = half * (BN / 2) + c * 32, v0 = x.n + col0;
        if (v0 >= g.vocab) break;
        float v[32];
        __syncwarp();
        tmem_ld32(acc + col0 + ((uint32_t)(q * 32) << 16), v);
        if (v0 + 32 > g.vocab) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (v0 + i >= g.vocab) v[i] = -INFINITY;
        }
        float top = v[0];
#pragma unroll
        for (int i = 1; i < 32; ++i) top = fmaxf(top, v[i]);
        if (top > m) {
            s *= ex2((m - top) * kLog2e);
            m = top;
        }
        if ((unsigned)(target - v0) < 32u) {  // the target's own term is added when the parts are joined
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (v0 + i == target) v[i] = -INFINITY;
        }
        // all -inf so far: any finite reference gives exp = 0 (and keeps a NaN visible)
        const float ref = m == -INFINITY ? 0.f : m;
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 32; ++i) part[i & 3] += ex2((v[i] - ref) * kLog2e);
        s += (part[0] + part[1]) + (part[2] + part[3]);
    }
    if (row < w.rows) g.stats[(int64_t)(x.n / (BN / 2) + half) * g.row_cap + row] = make_float2(m, s);
}

__device__ __forceinline__ void epilogue_prob(const HeadGemm &g, const Walk &w, const Tile &x, uint32_t acc, int q,
                                              int lane, int half) {
    const int row = x.m + q * 32 + lane;
    const bool in = row < w.rows;
    const int target = in ? g.target[row] - x.v0 : -1;  // column within the piece
    const float4 norm = in ? g.norm[row] : make_float4(0.f, 0.f, 0.f, 0.f);
    bf16 *out = g.piece[x.piece] + (int64_t)row * g.piece_ld + x.n;
    for (int c = 0; c < BN / 2 / 32; ++c) {
        const int col0 = half * (BN / 2) + c * 32, p0 = x.n + col0;
        float v[32];
        __syncwarp();
        tmem_ld32(acc + col0 + ((uint32_t)(q * 32) << 16), v);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            float p = ex2((v[i] - norm.x) * kLog2e) * norm.y;
            if (p0 + i == target) p = norm.z;
            v[i] = in && p0 + i < x.width ? p : 0.f;
        }
        uint4 *o = reinterpret_cast<uint4 *>(out + col0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                              pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
    }
}

__device__ __forceinline__ void epilogue_dh(const HeadGemm &g, const Walk &w, const Tile &x, uint32_t acc, int q,
                                            int lane, int half) {
    const int row = x.m + q * 32 + lane;
    float *out = g.dh + ((int64_t)x.split * g.row_cap + row) * g.dh_ld + x.n;
    for (int c = 0; c < BN / 2 / 32; ++c) {
        const int col0 = half * (BN / 2) + c * 32;
        if (x.n + col0 >= g.dim) break;
        float v[32];
        __syncwarp();
        tmem_ld32(acc + col0 + ((uint32_t)(q * 32) << 16), v);
        if (x.kb == 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8 && row < w.rows; ++i) {  // dh_ld is a multiple of 32
            float4 *o = reinterpret_cast<float4 *>(out + col0) + i;
            float4 f = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            if (x.add) {
                const float4 p = *o;
                f = make_float4(f.x + p.x, f.y + p.y, f.z + p.z, f.w + p.w);
            }
            *o = f;
        }
    }
}

__device__ __forceinline__ void epilogue_dw(const HeadGemm &g, const Tile &x, uint32_t acc, int q, int lane, int half,
                                            float factor) {
    const int local = x.m + q * 32 + lane;
    const int64_t row = x.v0 + local;
    for (int c = 0; c < BN / 2 / 32; ++c) {
        const int col0 = half * (BN / 2) + c * 32, col = x.n + col0;
        if (col >= g.dim) break;
        float v[32];
        __syncwarp();
        tmem_ld32(acc + col0 + ((uint32_t)(q * 32) << 16), v);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = x.kb == 0 ? 0.f : v[i] * factor;
        if (g.dw_vec) {  // dim % 8 == 0, 16-byte aligned: whole groups of 8
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (col + 8 * i >= g.dim || local >= x.width) break;
                float a[8];
                if (g.dw_bf16) {
                    uint4 *o = reinterpret_cast<uint4 *>(static_cast<bf16 *>(g.dw) + row * g.dim + col) + i;
                    if (g.dw_add) {
                        const uint4 u = *o;
                        a[0] = lo_f(u.x); a[1] = hi_f(u.x); a[2] = lo_f(u.y); a[3] = hi_f(u.y);
                        a[4] = lo_f(u.z); a[5] = hi_f(u.z); a[6] = lo_f(u.w); a[7] = hi_f(u.w);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[8 * i + j] += a[j];
                    }
                    *o = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                    pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
                } else {
                    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(g.dw) + row * g.dim + col) + 2 * i;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float4 f = make_float4(v[8 * i + 4 * h], v[8 * i + 4 * h + 1], v[8 * i + 4 * h + 2],
                                               v[8 * i + 4 * h + 3]);
                        if (g.dw_add) {
                            const float4 p = o[h];
                            f = make_float4(f.x + p.x, f.y + p.y, f.z + p.z, f.w + p.w);
                        }
                        o[h] = f;
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                if (col + i >= g.dim || local >= x.width) break;
                const int64_t o = row * g.dim + col + i;
                if (g.dw_bf16) {
                    bf16 *p = static_cast<bf16 *>(g.dw) + o;
                    *p = from_f<bf16>(g.dw_add ? to_f(*p) + v[i] : v[i]);
                } else {
                    float *p = static_cast<float *>(g.dw) + o;
                    *p = g.dw_add ? *p + v[i] : v[i];
                }
            }
        }
    }
}

// ---- the kernel ------------------------------------------------------------------------

__global__ void __launch_bounds__(THREADS, 1) head_gemm_kernel(const __grid_constant__ HeadGemm g, unsigned *flag) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + STAGES * STAGE_BYTES);
    uint64_t *empty = full + STAGES;
    uint64_t *tfull = empty + STAGES;
    uint64_t *tempty = tfull + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tempty + 2);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], EPI_WARPS * 32);
        }
        fence_mbar_init();
        prefetch_tmap(&g.tm_h);
        prefetch_tmap(&g.tm_w);
        prefetch_tmap(&g.tm_p[0]);
        prefetch_tmap(&g.tm_p[1]);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const Walk walk = make_walk(g);

    if (warp == 0 && lane == 0) {
        // ---------------- TMA producer
        uint32_t it = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < walk.total && ok; t += gridDim.x) {
            const Tile x = tile_at(g, walk, t);
            const CUtensorMap *ma = x.kind <= HEAD_PROB ? &g.tm_h : &g.tm_p[x.piece];
            const CUtensorMap *mb = x.kind == HEAD_DW ? &g.tm_h : &g.tm_w;
            for (int kb = 0; kb < x.kb; ++kb, ++it) {
                const int s = it % STAGES;
                const uint32_t ph = (it / STAGES) & 1u;
                if (!mbar_wait_bounded(&empty[s], ph ^ 1u, flag, 0x601u)) { ok = false; break; }
                unsigned char *sa = smem + s * STAGE_BYTES, *sb = sa + A_BYTES;
                const int k = x.k0 + kb * BK;
                mbar_arrive_expect_tx(&full[s], STAGE_BYTES);
#pragma unroll
                for (int i = 0; i < BM / 64; ++i) {
                    if (x.kind == HEAD_DW) tma_load_2d(sa + i * BOX_BYTES, ma, x.m + 64 * i, k, &full[s]);
                    else tma_load_2d(sa + i * BOX_BYTES, ma, k, x.m + 64 * i, &full[s]);
                }
#pragma unroll
                for (int i = 0; i < BN / 64; ++i) {
                    if (x.kind <= HEAD_PROB) tma_load_2d(sb + i * BOX_BYTES, mb, k, x.v0 + x.n + 64 * i, &full[s]);
                    else if (x.kind == HEAD_DH) tma_load_2d(sb + i * BOX_BYTES, mb, x.n + 64 * i, x.v0 + k, &full[s]);
                    else tma_load_2d(sb + i * BOX_BYTES, mb, x.n + 64 * i, k, &full[s]);
                }
            }
        }
    } else if (warp == 1 && lane == 0) {
        // ---------------- MMA issuer
        uint32_t it = 0, local = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < walk.total && ok; t += gridDim.x, ++local) {
            const Tile x = tile_at(g, walk, t);
            const bool a_mn = x.kind == HEAD_DW, b_mn = x.kind >= HEAD_DH;
            const uint32_t idesc = bf16_idesc(BM, BN, a_mn, b_mn);
            const uint32_t acc = local & 1u, aph = (local >> 1) & 1u;
            if (!mbar_wait_bounded(&tempty[acc], aph ^ 1u, flag, 0x602u)) break;
            tc_fence_after();
            const uint32_t d = tmem_base + acc * BN;
            for (int kb = 0; kb < x.kb; ++kb, ++it) {
                const int s = it % STAGES;
                const uint32_t ph = (it / STAGES) & 1u;
                if (!mbar_wait_bounded(&full[s], ph, flag, 0x603u)) { ok = false; break; }
                tc_fence_after();
                const uint32_t sa = smem_u32(smem + s * STAGE_BYTES), sb = sa + A_BYTES;
#pragma unroll
                for (int k = 0; k < BK / 16; ++k) {
                    // 16 k: 32 bytes along a K-major row, 16 rows of an MN-major block
                    const uint64_t da = a_mn ? smem_desc_mn_sw128(sa + k * 2048, BOX_BYTES) : smem_desc_sw128(sa + k * 32);
                    const uint64_t db = b_mn ? smem_desc_mn_sw128(sb + k * 2048, BOX_BYTES) : smem_desc_sw128(sb + k * 32);
                    mma_f16(d, da, db, idesc, (kb > 0 || k > 0) ? 1u : 0u);
                }
                mma_commit(&empty[s]);
            }
            mma_commit(&tfull[acc]);
        }
    } else if (warp >= 2) {
        // ---------------- epilogue
        const int q = warp % 4;           // TMEM lane quarter this warp may access
        const int half = (warp - 2) / 4;  // column half of the tile
        const float factor = g.grad_scale * g.state->inv_count;
        uint32_t local = 0;
        for (int t = blockIdx.x; t < walk.total; t += gridDim.x, ++local) {
            const Tile x = tile_at(g, walk, t);
            const uint32_t a = local & 1u, aph = (local >> 1) & 1u;
            if (!mbar_wait_bounded(&tfull[a], aph, flag, 0x604u)) break;
            tc_fence_after();
            const uint32_t acc = tmem_base + a * BN;
            if (x.kind == HEAD_STATS) epilogue_stats(g, walk, x, acc, q, lane, half);
            else if (x.kind == HEAD_PROB) epilogue_prob(g, walk, x, acc, q, lane, half);
            else if (x.kind == HEAD_DH) epilogue_dh(g, walk, x, acc, q, lane, half);
            else epilogue_dw(g, x, acc, q, lane, half, factor);
            tc_fence_before();
            mbar_arrive(&tempty[a]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

}  // namespace

int head_gemm(const HeadGemm &g, int max_tiles, const char *name, cudaStream_t st) {
    if (int rc = set_smem_limit(reinterpret_cast<const void *>(&head_gemm_kernel), SMEM_BYTES)) return rc;
    const int grid = std::max(1, std::min(max_tiles, num_sms()));
    SPCO_LAUNCH(name, st, head_gemm_kernel<<<grid, THREADS, SMEM_BYTES, st>>>(g, device_flag_ptr()));
    SPECOPTIM_LAUNCHED("head_gemm_kernel");
    return SPECOPTIM_OK;
}

}  // namespace spco
