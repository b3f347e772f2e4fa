// Embedding lookup with scaling, and its gradient by sorted tokens
// (include/stage_ends.h): the first stage of the training pipeline.
//
//   out[t]  = scale * table[ids[t]]
//   grad[v] = scale * sum over t with ids[t] = v of dy[t]
//
// The gradient sorts (id, token) pairs with a stable radix sort (9 bits a
// pass), cuts the sorted list into chunks of equal length and gives each chunk
// to one block, whatever the ids' distribution: a block sums runs of equal ids
// in registers, in token order; a run that lies in one chunk goes straight to
// its row, one that crosses chunks leaves fp32 partial sums that a last kernel
// adds in chunk order.  So the sums cost the same whatever the ids are, and the
// result does not depend on timing.  Rows without a token are zero-filled by
// further blocks of the same launches.  The join of one id's chunks is the work of one
// block per 2048 columns, which shows where an id has a large part of the tokens: 65536
// tokens take 244 us with frequencies of 1 / rank, 266 with a tenth of them one id, 440
// with half, 655 with all.
//
// Measured on a GB300 (copy bandwidth 6.78 TB/s), 65536 tokens whose frequencies
// fall off as 1 / rank, vocabulary 128256, width 2048:
//   lookup, fp32 table to bf16: 84 us, 5.2 TB/s of the bytes that have to move (64 us
//     at the copy's rate).  The rows are read 3.3 times over from L2, 537 MB beside
//     432 MB of DRAM traffic.
//   gradient, bf16 to dense fp32: 244 us, 5.4 TB/s (195 us at the copy's rate).  The
//     sums move 5.7 TB/s with the zero rows beside them, the joins 4.7; the ids' count and
//     the sort's two passes (21 to 23 us each, an eighth of the zero rows beside each) are latency.
//     Added to what is there: 188 us (no zero rows); bf16 gradient 176; fp32 dy 279.
// Small calls are launch and latency bound: 777 tokens 24 us in three launches.
#include <algorithm>
#include <mutex>
#include <string>

#include "rowvec.cuh"

namespace spco {

static __device__ unsigned g_stage_flag;

unsigned *stage_flag_ptr() {
    static unsigned *ptr = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_stage_flag) == cudaSuccess) ptr = static_cast<unsigned *>(p);
    });
    return ptr;
}

// A page-locked word per thread that asks, so that copies into it do not hold the host up.
struct HostWord {
    unsigned *p = nullptr;
    HostWord() {
        void *q = nullptr;
        if (cudaMallocHost(&q, sizeof(unsigned)) == cudaSuccess) p = static_cast<unsigned *>(q);
    }
    ~HostWord() { cudaFreeHost(p); }
};
static unsigned *host_word() {
    static thread_local HostWord word;
    return word.p;
}

int read_stage_flag(cudaStream_t st) {
    unsigned *p = stage_flag_ptr(), *v = host_word();
    if (!p || !v) return fail(SPECOPTIM_ERR_CUDA, "no memory for the flag of token ids");
    SPECOPTIM_CUDA(cudaMemcpyAsync(v, p, sizeof(*v), cudaMemcpyDeviceToHost, st));
    return SPECOPTIM_OK;
}

int check_stage_flag(cudaStream_t st) {
    const unsigned v = *host_word();
    if (!v) return SPECOPTIM_OK;
    SPECOPTIM_CUDA(cudaMemsetAsync(stage_flag_ptr(), 0, sizeof(v), st));
    SPECOPTIM_CUDA(cudaStreamSynchronize(st));
    return fail(SPECOPTIM_ERR_BOUNDS, v == kSiteTokenId  ? "a token id lies outside the vocabulary"
                                      : v == kSiteTarget ? "a target lies outside the vocabulary"
                                                         : "offsets of sequences descend or lie outside the tokens");
}

namespace {

// ---- lookup ----------------------------------------------------------------------

// A block takes U tokens at a time: their ids first, then U independent row
// loads per thread, so a gather of 65536 rows keeps U x 16 or 32 bytes per
// thread in flight.
template <typename TI, typename TO, typename ID, bool VEC, int U>
__global__ void __launch_bounds__(256) lookup_kernel(const Span<const TI> table, const ID *__restrict__ ids,
                                                     int64_t tokens, int64_t vocab, int dim, float scale,
                                                     const Span<TO> out, unsigned *flag) {
    const int vecs = VEC ? dim / 8 : (dim + 14) / 8;
    for (int64_t t0 = (int64_t)blockIdx.x * U; t0 < tokens; t0 += (int64_t)gridDim.x * U) {
        int64_t id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            id[u] = t0 + u < tokens ? (int64_t)ids[t0 + u] : -1;
            if (t0 + u < tokens && (id[u] < 0 || id[u] >= vocab)) {
                if (threadIdx.x == 0) atomicExch(flag, kSiteTokenId);
                id[u] = -1;
            }
        }
        for (int v = threadIdx.x; v < vecs; v += blockDim.x) {
            float x[U][8];
            int col[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                col[u] = v * 8 - (VEC ? 0 : (int)((out.lo + (t0 + u) * dim) & 7));
#pragma unroll
                for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
                if (id[u] >= 0) {
                    if (VEC) load8(table.p + id[u] * dim + col[u], x[u]);
                    else load_any(table, table.lo + id[u] * dim + col[u], x[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t0 + u >= tokens) break;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[u][i] *= id[u] >= 0 ? scale : 0.f;
                const int64_t row = out.lo + (t0 + u) * dim;
                if (VEC) store8(out.p + row + col[u], x[u]);
                else store_any(out, row + col[u], row, row + dim, x[u]);
            }
        }
    }
}

template <typename TI, typename TO, typename ID>
void launch_lookup(const void *table, const void *ids, int64_t tokens, int64_t vocab, int dim, float scale,
                   void *out, cudaStream_t st) {
    const Span<const TI> tb(static_cast<const TI *>(table), vocab * dim);
    const Span<TO> o(static_cast<TO *>(out), tokens * dim);
    const ID *id = static_cast<const ID *>(ids);
    const int threads = (int)std::min<int64_t>(256, round_up(ceil_div(dim + 7, 8), 32));
    const bool vec = dim % 8 == 0 && aligned16(table) && aligned16(out);
    const int64_t resident = (int64_t)num_sms() * 8;
    // Few tokens: one per block, so that every row has an SM of its own.  Many: four at a
    // time in a grid that stays (65536 x 2048: 82 us; one at a time 117), but rows that are
    // not multiples of 16 bytes one at a time in many blocks (50000 x 1234: 47 us against
    // 69 with four: their shifts take the registers).
    const bool few = tokens <= resident;
    const int grid = (int)(few   ? tokens
                           : vec ? std::min<int64_t>(ceil_div(tokens, 4), resident)
                                 : std::min<int64_t>(tokens, resident * 8));
    auto *k = few ? (vec ? &lookup_kernel<TI, TO, ID, true, 1> : &lookup_kernel<TI, TO, ID, false, 1>)
                  : (vec ? &lookup_kernel<TI, TO, ID, true, 4> : &lookup_kernel<TI, TO, ID, false, 1>);
    k<<<grid, threads, 0, st>>>(tb, id, tokens, vocab, dim, scale, o, stage_flag_ptr());
}

template <typename TI, typename TO>
void launch_lookup(const void *table, const void *ids, int id_bytes, int64_t tokens, int64_t vocab, int dim,
                   float scale, void *out, cudaStream_t st) {
    if (id_bytes == 8) launch_lookup<TI, TO, int64_t>(table, ids, tokens, vocab, dim, scale, out, st);
    else launch_lookup<TI, TO, int32_t>(table, ids, tokens, vocab, dim, scale, out, st);
}

// ---- stable radix sort of (id, token) ---------------------------------------------

constexpr int kBits = 9, kBins = 1 << kBits;
constexpr int kSortThreads = 256, kSortItems = 8, kTile = kSortThreads * kSortItems;
constexpr int kSortWarps = kSortThreads / 32, kWarpItems = kTile / kSortWarps;

// The sort key of a token: its id, or `vocab` (behind every row) for a token
// that contributes nothing.
template <typename ID>
__device__ __forceinline__ uint32_t key_of(const ID *ids, int64_t t, int64_t vocab, int64_t padding, unsigned *flag) {
    const int64_t id = (int64_t)ids[t];
    if (id >= 0 && id < vocab) return id == padding ? (uint32_t)vocab : (uint32_t)id;
    if (flag) atomicExch(flag, kSiteTokenId);
    return (uint32_t)vocab;
}

// ---- zero rows ----------------------------------------------------------------------

// zeros to the bytes [from, to) of p
__device__ __forceinline__ void zero_bytes(char *p, int64_t from, int64_t to) {
    const int64_t lead = (16 - (reinterpret_cast<uintptr_t>(p + from) & 15)) & 15;
    const int64_t a = min(from + lead, to), b = a + (to - a) / 16 * 16;
    for (int64_t i = a + (int64_t)threadIdx.x * 16; i < b; i += (int64_t)blockDim.x * 16)
        *reinterpret_cast<uint4 *>(p + i) = make_uint4(0, 0, 0, 0);
    // up to 15 bytes on either side; values have 2 or 4 bytes
    const int64_t end = threadIdx.x < 8 ? from + 2 * threadIdx.x : b + 2 * ((int64_t)threadIdx.x - 8);
    if (threadIdx.x < 16 && end < (threadIdx.x < 8 ? a : to)) *reinterpret_cast<uint16_t *>(p + end) = 0;
}

// Zero-filling the rows without a token is most of the gradient's traffic and
// needs nothing but to know those rows, so it runs beside the sort and the joins
// (latency), a share of it in each of their launches: blocks behind a launch's
// own, kZeroRows rows each.
constexpr int kZeroRows = 64;
struct Fill {
    char *grad;
    int64_t row_bytes, vocab;
    int64_t first;  // this launch's first group of kZeroRows rows
};

__device__ __forceinline__ void fill_rows(const Fill &f, int64_t group, const bool *present) {
    const int64_t row0 = (f.first + group) * kZeroRows;
    const int rows = (int)min((int64_t)kZeroRows, f.vocab - row0);
    for (int i = 0; i < rows; ++i) {
        if (present[i]) continue;
        const int from = i;
        while (i + 1 < rows && !present[i + 1]) ++i;
        zero_bytes(f.grad, (row0 + from) * f.row_bytes, (row0 + i + 1) * f.row_bytes);
    }
}

// the rows that have a token by the map of them
__device__ __forceinline__ void fill_by_map(const Fill &f, int64_t group, const uint32_t *map) {
    __shared__ bool present[kZeroRows];
    const int64_t row0 = (f.first + group) * kZeroRows;
    for (int i = threadIdx.x; i < kZeroRows; i += blockDim.x)
        present[i] = row0 + i < f.vocab && (map[(row0 + i) >> 5] >> ((row0 + i) & 31)) & 1u;
    __syncthreads();
    fill_rows(f, group, present);
}

// the same from the ids themselves, where they are few
template <typename ID>
__device__ __forceinline__ void fill_by_ids(const Fill &f, int64_t group, const ID *__restrict__ ids, int64_t n,
                                            int64_t padding) {
    __shared__ bool present[kZeroRows];
    const int64_t row0 = (f.first + group) * kZeroRows;
    for (int i = threadIdx.x; i < kZeroRows; i += blockDim.x) present[i] = false;
    __syncthreads();
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < n; t += blockDim.x) {
        const int64_t id = (int64_t)ids[t];
        if (id >= row0 && id < row0 + kZeroRows && id != padding) present[id - row0] = true;
    }
    __syncthreads();
    fill_rows(f, group, present);
}

// Digits of one tile of kTile ids, counted into hist[block][bin], and the ids
// into the map of rows that have a token; the next pass's table is cleared on
// the way.
template <typename ID>
__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(const ID *__restrict__ ids, int64_t vocab,
                                                                 int64_t padding, int64_t n,
                                                                 uint32_t *__restrict__ hist,
                                                                 uint32_t *__restrict__ next_hist,
                                                                 uint32_t *__restrict__ map, unsigned *flag) {
    grid_dependency_launch();
    __shared__ uint32_t cnt[kBins];
    for (int b = threadIdx.x; b < kBins; b += kSortThreads) cnt[b] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * kTile;
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
        const int64_t t = base + i * kSortThreads + threadIdx.x;
        if (t >= n) break;
        const uint32_t k = key_of(ids, t, vocab, padding, flag);
        atomicAdd(&cnt[k & (kBins - 1)], 1u);
        if ((int64_t)k < vocab) atomicOr(&map[k >> 5], 1u << (k & 31));
    }
    __syncthreads();
    for (int b = threadIdx.x; b < kBins; b += kSortThreads) {
        hist[(int64_t)blockIdx.x * kBins + b] = cnt[b];
        next_hist[(int64_t)blockIdx.x * kBins + b] = 0;
    }
}

struct SortShared {
    uint32_t where[kSortWarps][kBins];
    uint32_t warp_total[kSortWarps];
};

// Moves one tile to its place in the order of this digit (bits shift ..
// shift + 8).  total and before are the counts of this thread's two bins over
// all tiles and over the tiles in front (ALONE: there is only this tile and
// they are counted here).  Within the tile each warp owns consecutive keys and
// ranks 32 of them at a time by matching digits, so equal digits keep their
// order.  next_hist (may be null) collects the next digit's counts by the tile
// that a key moves to; integer counts, so their order does not matter.
template <typename ID, bool FIRST, bool ALONE>
__device__ __forceinline__ void sort_tile(SortShared &sh, const ID *ids, int64_t vocab, int64_t padding,
                                          const uint32_t *keys, const uint32_t *vals, int64_t n, int64_t tile,
                                          int shift, uint32_t (&total)[2], const uint32_t (&before)[2],
                                          uint32_t *keys_out, uint32_t *vals_out, uint32_t *next_hist,
                                          unsigned *flag) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    for (int b = tid; b < kSortWarps * kBins; b += kSortThreads) (&sh.where[0][0])[b] = 0;
    __syncthreads();
    const int64_t base = tile * kTile + w * kWarpItems;
    uint32_t key[kWarpItems / 32], val[kWarpItems / 32];
#pragma unroll
    for (int i = 0; i < kWarpItems / 32; ++i) {
        const int64_t t = base + i * 32 + lane;
        key[i] = t < n ? (FIRST ? key_of(ids, t, vocab, padding, flag) : keys[t]) : 0u;
        val[i] = FIRST || t >= n ? (uint32_t)t : vals[t];
        if (t < n) atomicAdd(&sh.where[w][(key[i] >> shift) & (kBins - 1)], 1u);
    }
    __syncthreads();
    if (ALONE) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            total[j] = 0;
            for (int i = 0; i < kSortWarps; ++i) total[j] += sh.where[i][2 * tid + j];
        }
    }
    // exclusive sum of the bins' totals over the block: where each bin starts
    const uint32_t mine = total[0] + total[1];
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sh.warp_total[w] = incl;
    __syncthreads();
    uint32_t start = incl - mine;
    for (int i = 0; i < w; ++i) start += sh.warp_total[i];
    // where[w][bin] = first position of this warp's keys of the bin
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int b = 2 * tid + j;
        uint32_t at = start + (j ? total[0] : 0u) + before[j];
        for (int i = 0; i < kSortWarps; ++i) {
            const uint32_t c = sh.where[i][b];
            sh.where[i][b] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarpItems / 32; ++i) {
        const int64_t t = base + i * 32 + lane;
        const bool in = t < n;
        const uint32_t d = in ? (key[i] >> shift) & (kBins - 1) : kBins;  // kBins: no key
        const uint32_t peers = __match_any_sync(0xffffffffu, d);
        if (in) {
            const uint32_t to = sh.where[w][d] + __popc(peers & ((1u << lane) - 1u));
            keys_out[to] = key[i];
            vals_out[to] = val[i];
            if (next_hist)
                atomicAdd(&next_hist[(int64_t)(to / kTile) * kBins + ((key[i] >> (shift + kBits)) & (kBins - 1))], 1u);
        }
        __syncwarp();
        if (in && (peers >> lane) == 1u) sh.where[w][d] += __popc(peers);  // the last of the peers
        __syncwarp();
    }
}

// The table of counts turned into what stands in front of each tile, and each bin's
// total: 32 bins per block, the tiles in 32 stretches.
constexpr int kScanBins = 32, kScanStretches = 32;
__global__ void __launch_bounds__(kScanBins * kScanStretches) sort_scan_kernel(uint32_t *hist, int blocks,
                                                                               uint32_t *totals) {
    __shared__ uint32_t sums[kScanStretches][kScanBins];
    grid_dependency_launch();
    grid_dependency_wait();
    const int lane = threadIdx.x % kScanBins, w = threadIdx.x / kScanBins;
    const int from = (int)((int64_t)blocks * w / kScanStretches), to = (int)((int64_t)blocks * (w + 1) / kScanStretches);
    uint32_t *column = hist + blockIdx.x * kScanBins + lane, sum = 0;
#pragma unroll 8
    for (int b = from; b < to; ++b) sum += column[(int64_t)b * kBins];
    sums[w][lane] = sum;
    __syncthreads();
    uint32_t at = 0;
    for (int i = 0; i < w; ++i) at += sums[i][lane];
    if (w == kScanStretches - 1) totals[blockIdx.x * kScanBins + lane] = at + sum;
    for (int b0 = from; b0 < to; b0 += 8) {
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = b0 + i < to ? column[(int64_t)(b0 + i) * kBins] : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (b0 + i < to) column[(int64_t)(b0 + i) * kBins] = at;
            at += c[i];
        }
    }
}

// From so many tiles on the table is scanned by a launch of its own; below, each block
// adds all of it up itself, which grows with the square of the tiles but saves the launch
// (width 8, vocabulary 128256, added up / scanned: 64 tiles 98 / 100 us, 128 tiles 164 / 159,
// 512 tiles 499 / 463, 4096 tiles 6.04 / 3.57 ms).
constexpr int kScanTiles = 128;

// One pass over all tiles.  totals null: the table holds counts; otherwise what
// sort_scan_kernel made of them.
template <typename ID, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(
    const ID *ids, int64_t vocab, int64_t padding, const uint32_t *keys,
    const uint32_t *vals, int64_t n, int shift, const uint32_t *hist, const uint32_t *totals, int blocks,
    uint32_t *__restrict__ keys_out, uint32_t *__restrict__ vals_out, uint32_t *__restrict__ next_hist,
    uint32_t *__restrict__ clear_hist, const Fill fill, const uint32_t *map) {
    // beside a fill the successor's blocks would wait in slots that the fill can use (+6 us on 65536 x 2048)
    if ((int)gridDim.x == blocks) grid_dependency_launch();
    grid_dependency_wait();
    if ((int)blockIdx.x >= blocks) {
        fill_by_map(fill, (int)blockIdx.x - blocks, map);
        return;
    }
    __shared__ SortShared sh;
    uint32_t total[2] = {0, 0}, before[2] = {0, 0};  // of two neighbouring bins per thread
    const uint2 *h2 = reinterpret_cast<const uint2 *>(hist);
    if (totals) {
        const uint2 t = reinterpret_cast<const uint2 *>(totals)[threadIdx.x];
        const uint2 c = h2[(int64_t)blockIdx.x * (kBins / 2) + threadIdx.x];
        total[0] = t.x;
        total[1] = t.y;
        before[0] = c.x;
        before[1] = c.y;
    } else {
#pragma unroll 8
        for (int b = 0; b < blocks; ++b) {
            const uint2 c = h2[(int64_t)b * (kBins / 2) + threadIdx.x];
            total[0] += c.x;
            total[1] += c.y;
            if (b < (int)blockIdx.x) {
                before[0] += c.x;
                before[1] += c.y;
            }
        }
    }
    if (clear_hist) reinterpret_cast<uint2 *>(clear_hist)[(int64_t)blockIdx.x * (kBins / 2) + threadIdx.x] = make_uint2(0, 0);
    sort_tile<ID, FIRST, false>(sh, ids, vocab, padding, keys, vals, n, blockIdx.x, shift, total, before, keys_out,
                                vals_out, next_hist, nullptr);
}

// All passes of a list that fits one tile, in one block; zero rows in the others (cold,
// vocabulary 32001: 777 tokens of width 1000 38 us, with the launches of longer lists 47; 2048
// tokens of width 2048 63 and 82).
template <typename ID>
__global__ void __launch_bounds__(kSortThreads) sort_small_kernel(const ID *__restrict__ ids, int64_t vocab,
                                                                  int64_t padding, int64_t n, int passes, uint32_t *k0,
                                                                  uint32_t *v0, uint32_t *k1, uint32_t *v1,
                                                                  const Fill fill, unsigned *flag) {
    grid_dependency_launch();
    if (blockIdx.x > 0) {
        fill_by_ids(fill, (int)blockIdx.x - 1, ids, n, padding);
        return;
    }
    __shared__ SortShared sh;
    uint32_t total[2];
    const uint32_t before[2] = {0, 0};
    sort_tile<ID, true, true>(sh, ids, vocab, padding, nullptr, nullptr, n, 0, 0, total, before, k0, v0, nullptr, flag);
    for (int pass = 1; pass < passes; ++pass) {
        __syncthreads();  // the block's own writes of the last pass
        const bool odd = pass & 1;
        sort_tile<ID, false, true>(sh, nullptr, vocab, padding, odd ? k0 : k1, odd ? v0 : v1, n, 0, pass * kBits, total,
                                   before, odd ? k1 : k0, odd ? v1 : v0, nullptr, nullptr);
    }
}

// ---- segmented sums ----------------------------------------------------------------

struct Sorted {
    const uint32_t *keys, *vals;
    int64_t n;
    int chunk;
    int64_t chunks;
};

// What is left to do of the zero rows, and the map of the others.
struct Filling {
    Fill next;
    int64_t left;  // groups of rows
    const uint32_t *map;

    // the next share of them: this launch's blocks
    Fill take(int64_t groups) {
        const Fill f = next;
        next.first += groups;
        left -= groups;
        return f;
    }
};

// First column of a thread's 8 in row `row` of the gradient: rows that are not
// multiples of 16 bytes begin `phase` values into a 16-byte piece.
template <typename TG, bool VEC> __device__ __forceinline__ int phase(const Span<TG> &grad, int64_t row, int dim) {
    return VEC ? 0 : (int)((grad.lo + row * dim) & 7);
}

template <typename TG, bool VEC>
__device__ __forceinline__ void put_row(const Span<TG> &grad, int64_t row, int dim, int j, float scale,
                                        bool accumulate, float (&a)[8]) {
    const int64_t from = grad.lo + row * dim, at = from + j * 8 - phase<TG, VEC>(grad, row, dim);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] *= scale;
    if (accumulate) {
        float old[8];
        if (VEC) load8(static_cast<const TG *>(grad.p) + at, old);
        else load_any(grad.read(), at, old);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] += old[i];
    }
    if (VEC) store8(grad.p + at, a);
    else store_any(grad, at, from, from + dim, a);
}

constexpr int kMaxChunk = 64;

// One chunk of the sorted list per block and column block, 8 columns per
// thread.  partial: [chunks][2][pitch], slot 0 for a run that began before the
// chunk, slot 1 for one that begins in it and goes on; its columns are shifted
// as the run's row is.
template <typename TD, typename TG, bool VEC>
__global__ void __launch_bounds__(256) segment_sum_kernel(const Sorted s, const Span<const TD> dy, int64_t vocab,
                                                          int dim, int col_blocks, float scale, bool accumulate,
                                                          const Span<TG> grad, float *__restrict__ partial, int pitch,
                                                          const Fill fill, const uint32_t *map) {
    __shared__ uint32_t sk[kMaxChunk + 2], sv[kMaxChunk];
    if (s.chunks * col_blocks == (int64_t)gridDim.x) grid_dependency_launch();
    grid_dependency_wait();
    const int tid = threadIdx.x;
    // sums and zero rows are spread evenly over the blocks, so that both are under way at any time
    const int64_t sums = s.chunks * col_blocks, block = (int64_t)blockIdx.x * sums / gridDim.x;
    if (((int64_t)blockIdx.x + 1) * sums / gridDim.x == block) {
        fill_by_map(fill, (int64_t)blockIdx.x - block, map);
        return;
    }
    const int64_t c = block / col_blocks;
    const int j = (int)(block % col_blocks) * (int)blockDim.x + tid;
    const int64_t p0 = c * s.chunk;
    const int len = (int)(s.n - p0 < s.chunk ? s.n - p0 : s.chunk);
    // keys of the chunk and of its two neighbours (~0: none)
    for (int i = tid; i < len + 2; i += blockDim.x) {
        const int64_t p = p0 + i - 1;
        sk[i] = p >= 0 && p < s.n ? s.keys[p] : ~0u;
    }
    for (int i = tid; i < len; i += blockDim.x) sv[i] = s.vals[p0 + i];
    __syncthreads();
    if (j * 8 >= pitch) return;
    constexpr int kBatch = VEC ? 8 : 4;  // rows in flight per thread; shifting odd rows into place takes registers
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    bool began = sk[0] != sk[1];  // whether the current run begins in this chunk
    for (int i0 = 0; i0 < len; i0 += kBatch) {
        float x[kBatch][8];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (i0 + u >= len) continue;
            const int64_t at = dy.lo + (int64_t)sv[i0 + u] * dim + j * 8 - phase<TG, VEC>(grad, sk[i0 + u + 1], dim);
            if (VEC) load8<kLasting>(dy.p + at, x[u]);
            else load_any<kLasting>(dy, at, x[u]);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u;
            if (i >= len) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] += x[u][k];
            const uint32_t k = sk[i + 1], next = sk[i + 2];
            const bool run_ends = next != k;
            if (!run_ends && i + 1 < len) continue;
            if ((int64_t)k < vocab) {
                if (began && run_ends) put_row<TG, VEC>(grad, k, dim, j, scale, accumulate, acc);
                else store8(partial + (c * 2 + (began ? 1 : 0)) * pitch + j * 8, acc);
            }
#pragma unroll
            for (int l = 0; l < 8; ++l) acc[l] = 0.f;
            began = true;
        }
    }
}

// Blocks [0, chunks * col_blocks): if a run begins in the block's chunk and goes
// on, its partial sums are added in chunk order and written to its row.  Where
// rows are narrow, groups of `threads` threads add up one stretch of chunks each
// and their sums are added in order.  Blocks after them: zero rows.
template <typename TG, bool VEC>
__global__ void __launch_bounds__(256) segment_join_kernel(const Sorted s, int64_t vocab, int dim, int col_blocks,
                                                           int threads,
                                                           float scale, bool accumulate, const Span<TG> grad,
                                                           const float *partial, int pitch,
                                                           const Fill fill, const uint32_t *map) {
    grid_dependency_wait();
    const int64_t joins = s.chunks * col_blocks;
    if ((int64_t)blockIdx.x >= joins) {
        fill_by_map(fill, (int64_t)blockIdx.x - joins, map);
        return;
    }
    const int64_t c = (int64_t)blockIdx.x / col_blocks;
    const int64_t p0 = c * s.chunk, p1 = p0 + s.chunk;
    if (p1 >= s.n) return;
    const uint32_t k = s.keys[p1 - 1], next = s.keys[p1], head = s.keys[p0], prev = p0 > 0 ? s.keys[p0 - 1] : ~0u;
    if ((int64_t)k >= vocab || next != k) return;
    if (head == k && prev == k) return;  // the run began earlier
    // the chunks behind this one that begin with the run: all threads look at once
    int64_t more = 0;
    for (;;) {
        const int64_t q = (c + 1 + more + threadIdx.x) * s.chunk;
        const int here = __syncthreads_count(q < s.n && s.keys[q] == k);
        more += here;
        if (here < (int)blockDim.x) break;
    }
    const int groups = blockDim.x / threads, group = threadIdx.x / threads, at = threadIdx.x % threads;
    const int j = (int)((int64_t)blockIdx.x % col_blocks) * threads + at;
    const bool in = j * 8 < pitch;
    // partial 0 is the chunk's own (its second slot), partial i the first slot of the chunk i behind it
    const int64_t from = (more + 1) * group / groups, to = (more + 1) * (group + 1) / groups;
    const float *first = partial + (c * 2 + 1) * pitch + j * 8, *rest = partial + (c * 2) * pitch + j * 8;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in) {
#pragma unroll 16
        for (int64_t i = from; i < to; ++i) {
            float x[8];
            load8(i == 0 ? first : rest + i * 2 * pitch, x);
#pragma unroll
            for (int l = 0; l < 8; ++l) acc[l] += x[l];
        }
    }
    if (groups > 1) {
        __shared__ float sums[8][256];  // [value][thread]
#pragma unroll
        for (int l = 0; l < 8; ++l) sums[l][threadIdx.x] = acc[l];
        __syncthreads();
        if (group > 0) return;
        for (int g = 1; g < groups; ++g)
#pragma unroll
            for (int l = 0; l < 8; ++l) acc[l] += sums[l][g * threads + at];
    }
    if (in) put_row<TG, VEC>(grad, k, dim, j, scale, accumulate, acc);
}

// Tokens per chunk: as many blocks as give every SM 1024 threads, between 8 and 64
// tokens.  Cold, with chunks of 8 / by this rule / of 64: 777 x 1000 36 / 38 / 46 us, 2048 x
// 2048 63 / 63 / 77, 8192 x 2048 107 / 91 / 85, 65536 x 2048 457 / 246 / 247, 65536 x 128 71 / 65 / 58.
int chunk_len(int64_t tokens, int col_blocks, int threads) {
    const int64_t want = tokens * col_blocks / ((int64_t)num_sms() * (1024 / threads));
    int len = 8;
    while (len < kMaxChunk && len < want) len *= 2;
    return len;
}

struct GradPlan {
    int threads, col_blocks, chunk, passes, pitch;
    int64_t chunks, sort_blocks;
    int64_t off_map, off_totals, off_hist[3], off_k0, off_v0, off_k1, off_v1, off_partial, bytes;
};

GradPlan plan_grad(int64_t tokens, int64_t vocab, int32_t dim, bool vec) {
    GradPlan p{};
    p.pitch = vec ? dim : (int)round_up(dim + 7, 8);  // with the start of the piece it begins in
    p.threads = (int)std::min<int64_t>(256, round_up(p.pitch / 8, 32));
    p.col_blocks = (int)ceil_div(p.pitch, (int64_t)p.threads * 8);
    p.chunk = chunk_len(tokens, p.col_blocks, p.threads);
    p.chunks = ceil_div(tokens, p.chunk);
    p.sort_blocks = ceil_div(tokens, kTile);
    int bits = 1;
    while ((vocab >> bits) > 0) ++bits;  // keys run up to `vocab` itself
    p.passes = (bits + kBits - 1) / kBits;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += round_up(bytes, 256);
        return here;
    };
    p.off_map = take((vocab + 31) / 32 * 4);
    p.off_totals = take(kBins * 4);
    for (int64_t &off : p.off_hist) off = take(p.sort_blocks * kBins * 4);
    p.off_k0 = take(tokens * 4);
    p.off_v0 = take(tokens * 4);
    p.off_k1 = take(tokens * 4);
    p.off_v1 = take(tokens * 4);
    p.off_partial = take(p.chunks * 2 * p.pitch * 4);
    p.bytes = at;
    return p;
}

template <typename ID>
int sort_tokens(const GradPlan &p, const ID *ids, int64_t tokens, int64_t vocab, int64_t padding, char *ws,
                Filling *fill, cudaStream_t st, Sorted *out) {
    uint32_t *hist[3], *map = reinterpret_cast<uint32_t *>(ws + p.off_map);
    fill->map = map;
    for (int i = 0; i < 3; ++i) hist[i] = reinterpret_cast<uint32_t *>(ws + p.off_hist[i]);
    uint32_t *k[2] = {reinterpret_cast<uint32_t *>(ws + p.off_k0), reinterpret_cast<uint32_t *>(ws + p.off_k1)};
    uint32_t *v[2] = {reinterpret_cast<uint32_t *>(ws + p.off_v0), reinterpret_cast<uint32_t *>(ws + p.off_v1)};
    const int blocks = (int)p.sort_blocks, last = (p.passes - 1) & 1;
    if (blocks == 1) {
        const int64_t share = fill->left;
        const Fill f = fill->take(share);
        SPCO_LAUNCH("embed_sort_small", st,
                    sort_small_kernel<ID><<<(unsigned)(1 + share), kSortThreads, 0, st>>>(
                        ids, vocab, padding, tokens, p.passes, k[0], v[0], k[1], v[1], f, stage_flag_ptr()));
    } else {
        SPECOPTIM_CUDA(cudaMemsetAsync(map, 0, (size_t)((vocab + 31) / 32 * 4), st));
        SPCO_LAUNCH("embed_sort_hist", st, sort_hist_kernel<ID><<<blocks, kSortThreads, 0, st>>>(
                                               ids, vocab, padding, tokens, hist[0], hist[1], map, stage_flag_ptr()));
        const int64_t fills = fill->left;
        for (int pass = 0; pass < p.passes; ++pass) {
            // three tables in turn: pass i reads table i, counts for pass i + 1
            // into the next one and clears the one behind it
            const int to = pass & 1, from = to ^ 1;
            uint32_t *counts = hist[pass % 3];
            uint32_t *next = pass + 1 < p.passes ? hist[(pass + 1) % 3] : nullptr;
            uint32_t *clear = pass + 2 < p.passes ? hist[(pass + 2) % 3] : nullptr;
            uint32_t *totals = blocks >= kScanTiles ? reinterpret_cast<uint32_t *>(ws + p.off_totals) : nullptr;
            cudaError_t e = cudaSuccess;
            if (totals)
                SPCO_LAUNCH("embed_sort_scan", st,
                            e = launch_dependent(sort_scan_kernel, dim3(kBins / kScanBins),
                                                 dim3(kScanBins * kScanStretches), 0, st, counts, blocks, totals));
            SPECOPTIM_CUDA(e);
            const int64_t share = std::min(fill->left, fills / 8);
            const Fill f = fill->take(share);
            const unsigned grid = (unsigned)(blocks + share);
            auto *kernel = pass == 0 ? &sort_scatter_kernel<ID, true> : &sort_scatter_kernel<ID, false>;
            SPCO_LAUNCH("embed_sort_scatter", st,
                        e = launch_dependent(kernel, dim3(grid), dim3(kSortThreads), 0, st, ids, vocab, padding, k[from],
                                             v[from], tokens, pass * kBits, counts, totals, blocks, k[to], v[to], next, clear, f,
                                             map));
            SPECOPTIM_CUDA(e);
        }
    }
    out->keys = k[last];
    out->vals = v[last];
    SPECOPTIM_LAUNCHED("embed_grad sort");
    return SPECOPTIM_OK;
}

template <typename TD, typename TG, bool VEC>
int sum_segments(const GradPlan &p, const Sorted &s, Filling fill, const void *dy, int64_t vocab, int dim, float scale,
                 bool accumulate, void *grad, float *partial, cudaStream_t st) {
    const Span<const TD> in(static_cast<const TD *>(dy), s.n * dim);
    const Span<TG> out(static_cast<TG *>(grad), vocab * dim);
    const int64_t sums = s.chunks * p.col_blocks;
    const int64_t beside = fill.left - fill.left / 2;  // the rest beside the joins
    const Fill f = fill.take(beside);
    cudaError_t e = cudaSuccess;
    SPCO_LAUNCH("embed_segment_sum", st,
                e = launch_dependent(segment_sum_kernel<TD, TG, VEC>, dim3((unsigned)(sums + beside)), dim3(p.threads), 0,
                                     st, s, in, vocab, dim, p.col_blocks, scale, accumulate, out, partial, p.pitch, f,
                                     fill.map));
    SPECOPTIM_CUDA(e);
    if (s.chunks > 1 || fill.left > 0)
        SPCO_LAUNCH("embed_segment_join", st,
                    e = launch_dependent(segment_join_kernel<TG, VEC>, dim3((unsigned)(sums + fill.left)),
                                         dim3(256 / p.threads * p.threads), 0, st, s, vocab, dim, p.col_blocks, p.threads,
                                         scale, accumulate, out, partial, p.pitch, fill.next, fill.map));
    SPECOPTIM_CUDA(e);
    return SPECOPTIM_OK;
}

int check_sizes(int64_t tokens, int64_t vocab, int32_t dim, const char *what) {
    if (tokens < 0 || tokens > (int64_t)1 << 30)
        return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": tokens outside [0, 2^30]");
    if (vocab < 1 || vocab > (int64_t)1 << 30)
        return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": vocab outside [1, 2^30]");
    if (dim < 1 || dim > 1 << 20) return fail(SPECOPTIM_ERR_INVALID_ARG, std::string(what) + ": dim outside [1, 2^20]");
    return SPECOPTIM_OK;
}

}  // namespace
}  // namespace spco

using namespace spco;

extern "C" int embed_lookup(const void *table, int32_t table_type, const void *ids, int32_t id_bytes, int64_t tokens,
                            int64_t vocab, int32_t dim, float scale, void *out, int32_t out_type, void *stream) {
    return entry([&]() -> int {
        if (int rc = check_sizes(tokens, vocab, dim, "embed_lookup")) return rc;
        if (!type_ok(table_type) || !type_ok(out_type))
            return fail(SPECOPTIM_ERR_INVALID_ARG, "embed_lookup: types must be STAGE_BF16 or STAGE_FP32");
        if (id_bytes != 4 && id_bytes != 8)
            return fail(SPECOPTIM_ERR_INVALID_ARG, "embed_lookup: id_bytes must be 4 or 8");
        if (tokens == 0) return SPECOPTIM_OK;
        if (!table || !ids || !out) return fail(SPECOPTIM_ERR_INVALID_ARG, "embed_lookup: null pointer");
        if (!aligned_to(table, type_bytes(table_type)) || !aligned_to(out, type_bytes(out_type)) ||
            !aligned_to(ids, id_bytes))
            return fail(SPECOPTIM_ERR_MISALIGNED, "embed_lookup: pointers must be aligned to their elements");
        if (int rc = bind_device()) return rc;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        SPCO_LAUNCH("embed_lookup", st, {
            if (table_type == STAGE_BF16 && out_type == STAGE_BF16)
                launch_lookup<bf16, bf16>(table, ids, id_bytes, tokens, vocab, dim, scale, out, st);
            else if (table_type == STAGE_BF16)
                launch_lookup<bf16, float>(table, ids, id_bytes, tokens, vocab, dim, scale, out, st);
            else if (out_type == STAGE_BF16)
                launch_lookup<float, bf16>(table, ids, id_bytes, tokens, vocab, dim, scale, out, st);
            else
                launch_lookup<float, float>(table, ids, id_bytes, tokens, vocab, dim, scale, out, st);
        });
        SPECOPTIM_LAUNCHED("lookup_kernel");
        return SPECOPTIM_OK;
    });
}

extern "C" int64_t embed_grad_workspace(int64_t tokens, int64_t vocab, int32_t dim) {
    int64_t bytes = -1;
    entry([&]() -> int {
        if (int rc = check_sizes(tokens, vocab, dim, "embed_grad")) return rc;
        // Alignment is not known yet.  Neither plan is always the larger one: unaligned rows are wider, which
        // may make a second column block and with it longer chunks, so fewer partial sums.
        bytes = std::max(plan_grad(tokens, vocab, dim, true).bytes, plan_grad(tokens, vocab, dim, false).bytes);
        return SPECOPTIM_OK;
    });
    return bytes;
}

extern "C" int embed_grad(const void *ids, int32_t id_bytes, const void *dy, int32_t dy_type, int64_t tokens,
                          int64_t vocab, int32_t dim, int64_t padding_idx, float scale, void *grad,
                          int32_t grad_type, int32_t accumulate, void *workspace, int64_t workspace_bytes,
                          void *stream) {
    return entry([&]() -> int {
        if (int rc = check_sizes(tokens, vocab, dim, "embed_grad")) return rc;
        if (!type_ok(dy_type) || !type_ok(grad_type))
            return fail(SPECOPTIM_ERR_INVALID_ARG, "embed_grad: types must be STAGE_BF16 or STAGE_FP32");
        if (id_bytes != 4 && id_bytes != 8)
            return fail(SPECOPTIM_ERR_INVALID_ARG, "embed_grad: id_bytes must be 4 or 8");
        if (padding_idx < -1 || padding_idx >= vocab)
            return fail(SPECOPTIM_ERR_INVALID_ARG, "embed_grad: padding_idx outside [-1, vocab)");
        if (!grad || (tokens > 0 && (!ids || !dy)))
            return fail(SPECOPTIM_ERR_INVALID_ARG, "embed_grad: null pointer");
        if (!aligned_to(dy, type_bytes(dy_type)) || !aligned_to(grad, type_bytes(grad_type)) ||
            !aligned_to(ids, id_bytes) || !aligned16(workspace))
            return fail(SPECOPTIM_ERR_MISALIGNED, "embed_grad: pointers must be aligned to their elements, the workspace to 16 bytes");
        const bool vec = dim % 8 == 0 && aligned16(dy) && aligned16(grad);
        const GradPlan p = plan_grad(tokens, vocab, dim, vec);
        if (tokens > 0 && (!workspace || workspace_bytes < p.bytes))
            return fail(SPECOPTIM_ERR_INVALID_ARG, "embed_grad: the workspace is smaller than embed_grad_workspace() says");
        const int64_t fills = accumulate ? 0 : ceil_div(vocab, kZeroRows);
        if (p.chunks * p.col_blocks + p.sort_blocks + fills > INT32_MAX)
            return fail(SPECOPTIM_ERR_NOT_IMPLEMENTED, "embed_grad: tokens x dim too large for one launch");
        if (int rc = bind_device()) return rc;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        const int64_t row_bytes = dim * (int64_t)type_bytes(grad_type);
        if (tokens == 0) {
            if (!accumulate) SPECOPTIM_CUDA(cudaMemsetAsync(grad, 0, (size_t)(vocab * row_bytes), st));
            return SPECOPTIM_OK;
        }
        char *ws = static_cast<char *>(workspace);
        Sorted s{nullptr, nullptr, tokens, p.chunk, p.chunks};
        Filling fill{{static_cast<char *>(grad), row_bytes, vocab, 0}, fills, nullptr};
        const int rc = id_bytes == 8
                           ? sort_tokens(p, static_cast<const int64_t *>(ids), tokens, vocab, padding_idx, ws, &fill, st, &s)
                           : sort_tokens(p, static_cast<const int32_t *>(ids), tokens, vocab, padding_idx, ws, &fill, st, &s);
        if (rc) return rc;
        float *partial = reinterpret_cast<float *>(ws + p.off_partial);
        const bool acc = accumulate != 0;
        auto go = [&](auto td, auto tg) -> int {
            using TD = decltype(td);
            using TG = decltype(tg);
            return vec ? sum_segments<TD, TG, true>(p, s, fill, dy, vocab, dim, scale, acc, grad, partial, st)
                       : sum_segments<TD, TG, false>(p, s, fill, dy, vocab, dim, scale, acc, grad, partial, st);
        };
        if (dy_type == STAGE_BF16) return grad_type == STAGE_BF16 ? go(bf16{}, bf16{}) : go(bf16{}, float{});
        return grad_type == STAGE_BF16 ? go(float{}, bf16{}) : go(float{}, float{});
    });
}
