// tcgen05 products of the vocabulary head (include/stage_ends.h, head_loss*):
// bf16 operands (kind::f16), fp32 accumulation in TMEM.
//
//   l  = H W^T                 logits of a 256 x 256 tile, never stored: the
//                              epilogue reduces them to row statistics
//                              (HEAD_STATS) or turns them into a piece of
//                              softmax - onehot (HEAD_PROB)
//   dh = P W,  dw = P^T H      P a piece [rows][vocabulary rows of the piece]
//
// Persistent pairs of CTAs (cta_group::2), one pair per two SMs, walk the tiles
// of up to three jobs (the next piece's probabilities beside the previous
// piece's two products, which do not depend on each other).  A pair owns a
// 256 x 256 tile: each CTA loads half of A's and half of B's rows (32 KB per 64
// k, where a CTA alone would load 48 KB for half the tile) and keeps half of the
// tile's rows in TMEM.  Warp 0 loads, one lane of rank 0's warp 1 issues the
// MMAs, warps 2-9 run the epilogues from one of two TMEM accumulators while the
// other is being filled.  H, W and the pieces are read in boxes 64 values wide with
// 128-byte swizzle: 128 rows high where an operand's rows run along K (one row
// per M or N index), 64 rows high where they run along M or N (one row per k),
// so none of the products needs a transposed copy.
//
// What bounds it: the power limit.  Measured on a GB300 (library bf16 product 1.88
// PFLOP/s, 1.66 to 1.76 once the card is at its power limit), H 2048 x 2048, W 128256 x
// 2048: statistics 560 us, 1.92 PFLOP/s, tensor pipe 89 % busy, before the limit, 610 us
// at it; a launch of gradients (a piece's probabilities beside the piece before's two
// products) keeps the tensor pipe 86 % busy.  Steps that led there, training step of
// 8192 tokens: one CTA per 128 x 256 tile 15.0 ms; pairs 12.3; one 128-row box per
// operand instead of two of 64 rows 10.35; tiles dealt out by load 10.2; column blocks,
// epilogues through tensor copies 9.8; two slabs handed over at a time 9.55; short
// tiles in turn among pairs of equal load 9.4; pieces of 256 MB instead of 128 9.25.
// A logits tile takes at least 2.2 us, its epilogue's time, and 0.6 us of its own beside
// 0.35 us per 64 k: narrow layers are bound by that (3974 x 112636 x 200: 212 us).
//
// Every wait on an mbarrier is bounded; where one gives up, a pair waits, again with a
// limit, for its loads and MMAs in flight before it frees TMEM and leaves.
#include <algorithm>
#include <cstring>
#include <mutex>
#include <string>

#include "head_gemm.cuh"

namespace spco {
namespace {

constexpr int BM = kHeadTileM, BN = kHeadTileN, BK = 64;  // of a pair of CTAs
constexpr int CM = BM / 2, CN = BN / 2;                    // one CTA's rows of A and of B
// 64-k slabs of a stage.  Two are handed over together: a hand-over (commit, wait)
// per slab with six stages costs 680 us against 610 us on 2048 x 128256 x 2048.
constexpr int SLABS = 2;
constexpr int STAGES = 3;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = (2 + EPI_WARPS) * 32;
constexpr uint32_t BOX_BYTES = 64 * 64 * 2;
constexpr uint32_t A_BYTES = CM * BK * 2;
constexpr uint32_t SLAB_BYTES = A_BYTES + CN * BK * 2, STAGE_BYTES = SLABS * SLAB_BYTES;
constexpr uint32_t TMEM_COLS = 2 * BN;
constexpr uint32_t OUT_BYTES = 32 * 128;  // one warp's block of 32 rows on its way out
constexpr size_t SMEM_BYTES = (size_t)STAGES * STAGE_BYTES + EPI_WARPS * OUT_BYTES + 1024 + 256;
static_assert(SMEM_BYTES <= 232448, "shared memory budget of one CTA");
constexpr uint32_t kDrainLimit = 1u << 14;  // probes of up to 4 us, for what takes microseconds
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One tile of a job: where its operands start and how far k runs.
struct Tile {
    int kind, piece;
    int m, n, bn;    // first row (M) and column (N) of the tile, its columns (256, or 128 at the end of dim)
    int k0, kb;      // first k, number of 64-k blocks
    int v0, width;   // vocabulary rows of the job's piece
    int split, add;
    int rank;        // of this CTA in its pair
};

// The tiles of one pair.  The two gradient products' tiles are few and long (a
// tile of dw runs over all rows, one of dh over the whole piece): they come
// first and are dealt out in turn.  The logits tiles are many and short; each
// pair takes as many as bring its load up to the others' (a load is counted in
// 64-k blocks and a tile's own cost as two of them).  With few rows dw's tiles are
// short too, less than half of one of dh, and are dealt out by load in front of
// the logits tiles (700 rows over 32001 x 4096: 520 us, in turn 560; 333 over 50001 x
// 1000: 126 and 139).  Pairs with the same load share a stretch of the short tiles
// in turn, so that neighbours work on the same rows of W or columns of a piece at
// the same time: 2048 rows over 128256 x 2048 take 2.59 ms, with a stretch of its
// own for each pair 2.84; 8192 9.3 and 9.55.
struct Walk {
    int rows, m_tiles, d_tiles;
    int long_dw, longs;                  // dw tiles dealt out in turn (in front of dh's); this pair's tiles in turn
    int line_dw;                         // dw tiles dealt out by load
    int first_short, step_short, shorts; // this pair's tiles of those and the logits
    int pair, pairs;
    int dw_job, dh_job, short_job;       // -1: none
};

// In 64-k blocks (0.35 us): what a tile costs beside its own, and what a tile of
// dw costs at least, its 256 KB (fp32) being written (one token over 128256 x 2048:
// 428 us with 4, 445 with 3; 333 over 50001 x 1000: 126 with 4, 129 with 6).
constexpr int kTileCost = 2;
constexpr int kDwCostFp32 = 4, kDwCostBf16 = 3;

__device__ __forceinline__ Walk make_walk(const HeadGemm &g, int pair, int pairs) {
    Walk w;
    w.pair = pair;
    w.pairs = pairs;
    w.rows = g.state->rows;
    w.m_tiles = (w.rows + BM - 1) / BM;
    w.d_tiles = (g.dim + BN - 1) / BN;
    w.dw_job = w.dh_job = w.short_job = -1;
    int n_short = 0, dw_tiles = 0, dh_tiles = 0, dw_cost = 1, dh_cost = 0;
#pragma unroll
    for (int j = 0; j < kHeadJobs; ++j) {
        if (j >= g.jobs) break;
        const HeadJob &q = g.job[j];
        if (q.kind <= HEAD_PROB) {
            w.short_job = j;
            n_short = w.m_tiles * ((q.width + BN - 1) / BN);
        } else if (q.kind == HEAD_DH) {
            w.dh_job = j;
            dh_tiles = w.m_tiles * w.d_tiles * q.splits;
            dh_cost = (q.width + BK - 1) / BK / q.splits + kTileCost;
        } else {
            w.dw_job = j;
            dw_tiles = ((q.width + BM - 1) / BM) * w.d_tiles;
            dw_cost = max((w.rows + BK - 1) / BK, g.dw_bf16 ? kDwCostBf16 : kDwCostFp32) + kTileCost;
        }
    }
    w.line_dw = 2 * dw_cost < dh_cost ? dw_tiles : 0;
    w.long_dw = dw_tiles - w.line_dw;
    const int long_tiles = w.long_dw + dh_tiles, line = w.line_dw + n_short;
    w.longs = pair < long_tiles ? (long_tiles - pair + pairs - 1) / pairs : 0;
    int first = 0, behind = line, p0 = 0, p1 = pairs;  // tiles [first, behind) of the line go to pairs [p0, p1) in turn
    if (long_tiles > 0) {
        // pairs below r1 have one dw tile more, pairs below r2 one long tile more:
        // three runs of pairs with equal loads
        const int r1 = w.long_dw % pairs, r2 = long_tiles % pairs;
        const int cost = (g.dim + BK - 1) / BK + kTileCost;
        const int64_t line_dw_cost = (int64_t)w.line_dw * dw_cost, line_cost = line_dw_cost + (int64_t)n_short * cost;
        const int64_t total = (int64_t)w.long_dw * dw_cost + (int64_t)dh_tiles * dh_cost + line_cost;
        const int edge[4] = {0, min(r1, r2), max(r1, r2), pairs};
        int64_t share[3], all = 0;  // `pairs` times what a pair of the run lacks to the mean load
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int n_dw = w.long_dw / pairs + (edge[k] < r1), n_long = long_tiles / pairs + (edge[k] < r2);
            const int64_t load = (int64_t)n_dw * dw_cost + (int64_t)(n_long - n_dw) * dh_cost;
            share[k] = max((int64_t)0, total - load * pairs);
            all += share[k] * (edge[k + 1] - edge[k]);
        }
        // integers throughout: a pair's last tile and the next one's first come from the same quotient
        const int shift = max(0, 33 - __clzll(all));  // sum < 2^31; line_cost < 2^31 as rows x width of a piece is bounded
        int64_t sum = 0;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            share[k] >>= shift;
            sum += share[k] * (edge[k + 1] - edge[k]);
        }
        // the first tile of the line (dw's, then the logits) that begins in or behind pair p's part of it
        auto first_of = [&](int p) -> int {
            if (p >= pairs || sum == 0) return p >= pairs ? line : 0;
            int64_t before = 0;
#pragma unroll
            for (int k = 0; k < 3; ++k) before += share[k] * (max(edge[k], min(edge[k + 1], p)) - edge[k]);
            const int64_t at = before * line_cost / sum;
            return at <= line_dw_cost ? (int)((at + dw_cost - 1) / dw_cost)
                                      : w.line_dw + (int)((at - line_dw_cost + cost - 1) / cost);
        };
        const int run = (pair >= edge[1]) + (pair >= edge[2]);
        p0 = edge[run];
        p1 = edge[run + 1];
        first = first_of(p0);
        behind = first_of(p1);
    }
    w.first_short = first + pair - p0;
    w.step_short = p1 - p0;
    w.shorts = max(0, (behind - w.first_short + w.step_short - 1) / w.step_short);
    return w;
}

__device__ __forceinline__ int tile_count(const Walk &w) { return w.longs + w.shorts; }

// the pair's i-th tile
__device__ __forceinline__ Tile tile_at(const HeadGemm &g, const Walk &w, int i, int rank) {
    int t, j;
    if (i < w.longs) {
        t = w.pair + i * w.pairs;
        j = t < w.long_dw ? w.dw_job : w.dh_job;
        if (t >= w.long_dw) t -= w.long_dw;
    } else {
        t = w.first_short + (i - w.longs) * w.step_short;
        j = t < w.line_dw ? w.dw_job : w.short_job;
        if (t >= w.line_dw) t -= w.line_dw;
    }
    const HeadJob &q = g.job[j];
    Tile x;
    x.kind = q.kind;
    x.piece = q.piece;
    x.rank = rank;
    x.v0 = q.v0;
    x.width = q.width;
    x.split = 0;
    x.add = q.add;
    x.k0 = 0;
    x.bn = BN;
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
    if (q.kind >= HEAD_DH && g.dim - x.n <= BN / 2) x.bn = BN / 2;
    return x;
}

// ---- epilogues: thread = one row of the tile, 32 columns at a time -------------------

// f(c, v) for the 32-column blocks c = 0 .. blocks - 1 of this warp's rows and
// columns; the next block is on its way from TMEM while f works on one.
template <typename F> __device__ __forceinline__ void for_columns(uint32_t taddr, int blocks, F &&f) {
    uint32_t next[32];
    __syncwarp();
    if (blocks > 0) tmem_ld32_begin(taddr, next);
    for (int c = 0; c < blocks; ++c) {
        float v[32];
        tmem_ld32_end(next);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(next[i]);
        __syncwarp();
        if (c + 1 < blocks) tmem_ld32_begin(taddr + (c + 1) * 32, next);
        f(c, v);
        __syncwarp();
    }
}

// how many of a warp's four 32-column blocks begin in front of `end`
__device__ __forceinline__ int blocks_before(int first, int end) { return min(4, max(0, (end - first + 31) / 32)); }

// What an epilogue needs of its row; loaded while the tile is still being formed.
struct RowOf {
    int row, target;
    bool in;
    HeadRow h;
    HeadNorm norm;  // HEAD_PROB
};
__device__ __forceinline__ RowOf row_of(const HeadGemm &g, const Walk &w, const Tile &x, int q, int lane) {
    RowOf o;
    o.row = x.m + x.rank * CM + q * 32 + lane;
    o.in = x.kind <= HEAD_PROB && o.row < w.rows;
    o.target = o.in ? g.target[o.row] : -1;
    o.h = HeadRow{0.f, 0.f};
    o.norm = HeadNorm{0.f, 0.f, 0.f};
    if (o.in) {
        o.h = g.rows[o.row];
        if (x.kind == HEAD_PROB) o.norm = g.norm[o.row];
    }
    return o;
}

// The part's sum is taken relative to 2^r, r a whole number: the exponent of each
// term is then one fused multiply-add, and parts are joined by exact powers of
// two.  r starts as the target's logit (in log2), which serves every row whose
// other logits are less than 2^100 / 128 times as likely -- so no pass for the
// maximum is needed; where a block of 32 terms reaches 2^100, r moves up to the
// block's maximum.
constexpr float kMuch = 1.2676506e30f;  // 2^100

__device__ __forceinline__ float sum_exp2(const float (&v)[32], float log2e, float r) {
    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; ++i) part[i & 3] += ex2(fmaf(v[i], log2e, -r));
    return (part[0] + part[1]) + (part[2] + part[3]);
}

__device__ __forceinline__ void epilogue_stats(const HeadGemm &g, const Tile &x, const RowOf &of, uint32_t acc, int q,
                                               int half) {
    const int target = of.target, first = x.n + half * (BN / 2);
    const float log2e = of.h.log2e;
    float r = rintf(of.h.target_logit * kLog2e), s = 0.f;
    // no reference in a target's logit that is not finite (an impossible target: -inf): the first block moves r up
    if (!(fabsf(r) < kMuch)) r = -kMuch;
    for_columns(acc + half * (BN / 2) + ((uint32_t)(q * 32) << 16), blocks_before(first, g.vocab), [&](int c, float (&v)[32]) {
        const int v0 = first + c * 32;
        if (v0 + 32 > g.vocab) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (v0 + i >= g.vocab) v[i] = -INFINITY;
        }
        if ((unsigned)(target - v0) < 32u) {  // the target's own term is added when the parts are joined
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (v0 + i == target) v[i] = -INFINITY;
        }
        float t = sum_exp2(v, log2e, r);
        if (!(t < kMuch)) {
            float top = v[0];
#pragma unroll
            for (int i = 1; i < 32; ++i) top = fmaxf(top, v[i]);
            const float most = rintf(top * log2e);
            if (most > r) {  // false where only NaN brought us here: it stays in the sum
                s *= ex2(r - most);
                r = most;
                t = sum_exp2(v, log2e, r);
            }
        }
        s += t;
    });
    if (of.in) g.stats[(int64_t)(x.n / (BN / 2) + half) * g.row_cap + of.row] = make_float2(r, s);
}

// A warp's way out: 32 rows of 128 bytes (64 bf16 or 32 fp32 columns) are laid
// out in shared memory with the 128-byte swizzle and stored, or added, by one
// tensor copy, which also clips what lies outside the tensor.  Each thread
// writes its own row; the swizzle spreads a warp's 16-byte pieces over the banks.
struct WayOut {
    unsigned char *buf;
    int lane;

    __device__ __forceinline__ void ready() const {  // the last copy has read the buffer
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
    }
    __device__ __forceinline__ void put(int piece16, uint4 v) const {
        *reinterpret_cast<uint4 *>(buf + lane * 128 + ((piece16 ^ (lane & 7)) << 4)) = v;
    }
    __device__ __forceinline__ void put_bf16(int first16, const float (&v)[32]) const {  // 4 pieces
#pragma unroll
        for (int i = 0; i < 4; ++i)
            put(first16 + i, make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                        pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7])));
    }
    __device__ __forceinline__ void put_fp32(const float (&v)[32]) const {  // 8 pieces
#pragma unroll
        for (int i = 0; i < 8; ++i)
            put(i, make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                              __float_as_uint(v[4 * i + 3])));
    }
    __device__ __forceinline__ void send(const CUtensorMap *map, int x, int y, bool add) const {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (add) tma_add_2d(map, buf, x, y);
            else tma_store_2d(map, buf, x, y);
            bulk_commit();
        }
    }
};

__device__ __forceinline__ void epilogue_prob(const HeadGemm &g, const Tile &x, const RowOf &of, uint32_t acc, int q,
                                              int half, const WayOut &out) {
    const int row0 = of.row - out.lane;
    const bool in = of.in;
    const int target = in ? of.target - x.v0 : -1;  // column within the piece
    const HeadNorm norm = of.norm;
    const float log2e = of.h.log2e;
    const int first = x.n + half * (BN / 2);
    for_columns(acc + half * (BN / 2) + ((uint32_t)(q * 32) << 16), 4, [&](int c, float (&v)[32]) {
        const int p0 = first + c * 32;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = ex2(fmaf(v[i], log2e, -norm.m)) * norm.inv;
        if ((unsigned)(target - p0) < 32u) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (p0 + i == target) v[i] = norm.target;
        }
        if (!in || p0 + 32 > x.width) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (!in || p0 + i >= x.width) v[i] = 0.f;
        }
        if ((c & 1) == 0) out.ready();
        out.put_bf16((c & 1) * 4, v);
        if (c & 1) out.send(&g.tm_p_st[x.piece], 0, (p0 / 64) * g.row_cap + row0, false);
    });
}

__device__ __forceinline__ void epilogue_dh(const HeadGemm &g, const Tile &x, uint32_t acc, int q,
                                            int half, const WayOut &out) {
    const int row0 = x.m + x.rank * CM + q * 32, first = x.n + half * (BN / 2);
    for_columns(acc + half * (BN / 2) + ((uint32_t)(q * 32) << 16), blocks_before(first, g.dim), [&](int c, float (&v)[32]) {
        if (x.kb == 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
        out.ready();
        out.put_fp32(v);
        // one addend per value and launch: the order of the sum is the order of the launches
        out.send(&g.tm_dh, first + c * 32, x.split * g.row_cap + row0, x.add != 0);
    });
}

// dw through shared memory and a tensor copy where its rows are multiples of 16
// bytes; otherwise, and for adding to a bf16 gradient (one rounding of the
// sum), value by value.
__device__ __forceinline__ void epilogue_dw(const HeadGemm &g, const Tile &x, uint32_t acc, int q, int half,
                                            float factor, const WayOut &out) {
    const int local0 = x.m + x.rank * CM + q * 32, local = local0 + out.lane;
    const int64_t row = (int64_t)x.v0 + local;
    const int first = x.n + half * (BN / 2), blocks = local0 < x.width ? blocks_before(first, g.dim) : 0;
    for_columns(acc + half * (BN / 2) + ((uint32_t)(q * 32) << 16), blocks, [&](int c, float (&v)[32]) {
        const int col = first + c * 32;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = x.kb == 0 ? 0.f : v[i] * factor;
        if (g.dw_tma && g.dw_bf16) {
            if ((c & 1) == 0) out.ready();
            out.put_bf16((c & 1) * 4, v);
            // the second half of the box may hold an earlier block where dim ends in the first: it is clipped
            if ((c & 1) || col + 32 >= g.dim) out.send(&g.tm_dw, col - (c & 1) * 32, x.v0 + local0, false);
        } else if (g.dw_tma) {
            out.ready();
            out.put_fp32(v);
            out.send(&g.tm_dw, col, x.v0 + local0, g.dw_add != 0);
        } else if (local < x.width) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                if (col + i >= g.dim) break;
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
    });
}

// ---- the kernel ------------------------------------------------------------------------

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
head_gemm_kernel(const __grid_constant__ HeadGemm g, unsigned *flag) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~uintptr_t(1023));
    unsigned char *way_out = smem + STAGES * STAGE_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(way_out + EPI_WARPS * OUT_BYTES);  // rank 0's: both CTAs' loads
    uint64_t *empty = full + STAGES;                                             // each CTA's own
    uint64_t *tfull = empty + STAGES;                                            // each CTA's own
    uint64_t *tempty = tfull + 2;                                                // rank 0's: both CTAs' epilogues
    uint64_t *drained = tempty + 2;                                              // all MMAs of the pair are done
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 1);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 2 * EPI_WARPS);
        }
        mbar_init(drained, 1);
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers exist and its TMEM is allocated
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_dependency_launch();
    grid_dependency_wait();  // up to here nothing of an earlier launch was touched
    const Walk walk = make_walk(g, blockIdx.x / 2, gridDim.x / 2);
    const int tiles = tile_count(walk);

    if (warp == 0 && lane == 0) {
        // ---------------- TMA producer: this CTA's half of A and of B
        // One thread issues everything, so a tile's coordinates are worked out once: each
        // operand has a first box, its step from one 64-k slab to the next, and, where its
        // rows run along M or N, a second box.
        struct Operand {
            const CUtensorMap *map;
            int x, y, dx, dy;   // first box, step per slab
            int x2, y2;         // second box relative to the first
            bool two;
        };
        uint32_t it = 0;
        bool ok = true;
        for (int t = 0; t < tiles && ok; ++t) {
            const Tile x = tile_at(g, walk, t, rank);
            const int m = x.m + rank * CM, n = x.n + rank * (x.bn / 2);
            const uint32_t bytes = 2 * (A_BYTES + (uint32_t)x.bn / 2 * BK * 2);
            Operand a, b;
            // h and the pieces lie in column blocks of 64: column c, row r at line c / 64 * row_cap + r
            if (x.kind == HEAD_DW) {
                a = {&g.tm_p[x.piece], 0, m / 64 * g.row_cap, 0, 64, 0, g.row_cap, true};
                b = {&g.tm_h, 0, n / 64 * g.row_cap, 0, 64, 0, g.row_cap, x.bn == BN};
            } else if (x.kind == HEAD_DH) {
                a = {&g.tm_p_k[x.piece], 0, x.k0 / 64 * g.row_cap + m, 0, g.row_cap, 0, 0, false};
                b = {&g.tm_w, n, x.v0 + x.k0, 0, 64, 64, 0, x.bn == BN};
            } else {
                a = {&g.tm_h_k, 0, m, 0, g.row_cap, 0, 0, false};
                b = {&g.tm_w_k, 0, x.v0 + n, 64, 0, 0, 0, false};
            }
            for (int kb = 0; kb < x.kb; kb += SLABS, ++it) {
                const int s = it % STAGES;
                const uint32_t ph = (it / STAGES) & 1u;
                if (!mbar_wait_bounded(&empty[s], ph ^ 1u, flag, 0x601u)) { ok = false; break; }
                const uint32_t bar = cluster_addr(&full[s], 0);
                const int slabs = min(SLABS, x.kb - kb);
                if (rank == 0) mbar_arrive_expect_tx(&full[s], slabs * bytes);
                unsigned char *sa = smem + s * STAGE_BYTES;
                for (int i = 0; i < slabs; ++i, sa += SLAB_BYTES) {
                    tma_load_2d_pair(sa, a.map, a.x, a.y, bar);
                    if (a.two) tma_load_2d_pair(sa + BOX_BYTES, a.map, a.x + a.x2, a.y + a.y2, bar);
                    tma_load_2d_pair(sa + A_BYTES, b.map, b.x, b.y, bar);
                    if (b.two) tma_load_2d_pair(sa + A_BYTES + BOX_BYTES, b.map, b.x + b.x2, b.y + b.y2, bar);
                    a.x += a.dx;
                    a.y += a.dy;
                    b.x += b.dx;
                    b.y += b.dy;
                }
            }
        }
        // Given up: the loads of the last stages may be on their way.  Rank 0's barriers count
        // both CTAs'; a stage that the other CTA filled alone never completes and the wait for it is
        // the time that its loads have to land.
        if (!ok && rank == 0)
            for (uint32_t j = it < (uint32_t)STAGES ? 0 : it - STAGES; j <= it; ++j)
                mbar_wait_limit(&full[j % STAGES], (j / STAGES) & 1u, nullptr, 0u, kDrainLimit);
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---------------- MMA issuer of the pair
        // The tensor core takes 128 cycles for an MMA of 16 k, so what this thread does per
        // MMA has to stay below that: descriptors are those of stage 0 plus an offset.
        const uint32_t sa0 = smem_u32(smem), sb0 = sa0 + A_BYTES;
        uint32_t it = 0, local = 0;
        bool ok = true;
        for (int t = 0; t < tiles && ok; ++t, ++local) {
            const Tile x = tile_at(g, walk, t, rank);
            const bool a_mn = x.kind == HEAD_DW, b_mn = x.kind >= HEAD_DH;
            const uint32_t idesc = bf16_idesc(BM, x.bn, a_mn, b_mn);
            const uint64_t da0 = a_mn ? smem_desc_mn_sw128(sa0, BOX_BYTES) : smem_desc_sw128(sa0);
            const uint64_t db0 = b_mn ? smem_desc_mn_sw128(sb0, BOX_BYTES) : smem_desc_sw128(sb0);
            // 16 k: 32 bytes along a K-major row, 16 rows of an MN-major block (in units of 16 bytes)
            const uint32_t da_step = a_mn ? 2048 / 16 : 32 / 16, db_step = b_mn ? 2048 / 16 : 32 / 16;
            const uint32_t acc = local & 1u, aph = (local >> 1) & 1u;
            if (!mbar_wait_bounded(&tempty[acc], aph ^ 1u, flag, 0x602u)) break;
            tc_fence_after();
            const uint32_t d = tmem_base + acc * BN;
            uint32_t accumulate = 0;
            for (int kb = 0; kb < x.kb; kb += SLABS, ++it) {
                const int s = it % STAGES;
                const uint32_t ph = (it / STAGES) & 1u;
                if (!mbar_wait_bounded(&full[s], ph, flag, 0x603u)) { ok = false; break; }
                tc_fence_after();
                const int slabs = min(SLABS, x.kb - kb);
                uint32_t at = s * (STAGE_BYTES / 16);
                for (int i = 0; i < slabs; ++i, at += SLAB_BYTES / 16) {
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k) {
                        mma_f16_pair(d, da0 + (at + k * da_step), db0 + (at + k * db_step), idesc, accumulate);
                        accumulate = 1;
                    }
                }
                mma_commit_pair(&empty[s]);
            }
            mma_commit_pair(&tfull[acc]);
        }
        // usually long done (the epilogues wait for the last tile)
        mma_commit_pair(drained);
        mbar_wait_limit(drained, 0, nullptr, 0u, kDrainLimit);
    } else if (warp >= 2) {
        // ---------------- epilogue of this CTA's rows
        const int q = warp % 4;           // TMEM lane quarter this warp may access
        const int half = (warp - 2) / 4;  // column half of the tile
        const float factor = g.grad_scale * g.state->inv_count;
        const WayOut out{way_out + (warp - 2) * OUT_BYTES, lane};
        uint32_t local = 0;
        for (int t = 0; t < tiles; ++t, ++local) {
            const Tile x = tile_at(g, walk, t, rank);
            const RowOf of = row_of(g, walk, x, q, lane);
            const uint32_t a = local & 1u, aph = (local >> 1) & 1u;
            // the lanes go on or give up together
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&tfull[a], aph, flag, 0x604u))) break;
            tc_fence_after();
            const uint32_t acc = tmem_base + a * BN;
            if (x.kind == HEAD_STATS) epilogue_stats(g, x, of, acc, q, half);
            else if (x.kind == HEAD_PROB) epilogue_prob(g, x, of, acc, q, half, out);
            else if (x.kind == HEAD_DH) epilogue_dh(g, x, acc, q, half, out);
            else epilogue_dw(g, x, acc, q, half, factor, out);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(cluster_addr(&tempty[a], 0));
        }
        if (lane == 0) bulk_wait_all();  // the copies out have been written
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no arrival is on its way to a CTA that has left
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

}  // namespace

int make_tmap_2d_bf16(CUtensorMap *map, const void *ptr, int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return fail(SPECOPTIM_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, box_rows}, steps[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, steps,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(SPECOPTIM_ERR_CUDA, "cuTensorMapEncodeTiled failed (" + std::to_string((int)r) + ")");
    return SPECOPTIM_OK;
}

int head_gemm(const HeadGemm &g, int max_tiles, const char *name, cudaStream_t st) {
    if (int rc = set_smem_limit(reinterpret_cast<const void *>(&head_gemm_kernel), SMEM_BYTES)) return rc;
    const int pairs = std::max(1, std::min(max_tiles, num_sms() / 2));
    cudaError_t e = cudaSuccess;
    SPCO_LAUNCH(name, st, e = launch_dependent(head_gemm_kernel, dim3(2 * pairs), dim3(THREADS), SMEM_BYTES, st, g, device_flag_ptr()));
    SPECOPTIM_CUDA(e);
    return SPECOPTIM_OK;
}

}  // namespace spco
