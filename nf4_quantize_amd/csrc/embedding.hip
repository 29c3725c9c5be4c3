// embedding.hip - the token embedding for gfx950: rows of a dense or an NF4
// table with a scale, and the gradient of the table by sorted tokens. The
// contracts are in nf4.h (nf4_embedding_forward, nf4_embedding_backward).
//
// The forward moves each looked-up row once in and once out. The backward
// sorts the tokens by their id (stable, so that a row's gradient is summed in
// the order of the tokens), sums runs of equal ids chunk by chunk and joins the
// runs that cross chunks; a dense gradient is cleared beside the sort. Few tokens
// take one launch without a sort. It is bound by reading dy and writing the table's
// gradient.
#include <type_traits>

#include "linear_common.h"
#include "training_internal.h"

namespace nf4 {
namespace {

constexpr int kThreads = 256;

// The row of token t, or `vocab` where it has none.
__device__ __forceinline__ uint32_t token_key(const void *ids, bool i64, int64_t t, int64_t vocab, int64_t skip) {
    const int64_t id = i64 ? static_cast<const int64_t *>(ids)[t] : (int64_t)static_cast<const int32_t *>(ids)[t];
    return id >= 0 && id < vocab && id != skip ? (uint32_t)id : (uint32_t)vocab;
}

// ---- forward ----

// A group of `lanes` lanes moves one row, kInFlight vectors of a lane at a time.
// The rows go out past the caches (16384 x 8192 bf16: 70 us instead of 80); the
// table's stay in them, as text asks for a few rows often (98 us without).
template <typename T, typename O, int kInFlight, typename C>
__global__ __launch_bounds__(kThreads) void lookup_kernel(const void *ids, bool i64, int64_t tokens, const T *table,
                                                          int64_t vocab, int32_t dim, float scale, O *out, int lanes) {
    const int each = kThreads / lanes, end = std::is_same_v<C, Fours> ? (dim + 511) / 512 * 512 : dim;
    for (int64_t t = (int64_t)blockIdx.x * each + threadIdx.x / lanes; t < tokens; t += (int64_t)gridDim.x * each) {
        const uint32_t row = token_key(ids, i64, t, vocab, -1);
        const T *src = table + (int64_t)row * dim;
        O *dst = out + t * dim;
        for (int c0 = (threadIdx.x & (lanes - 1)) * 8; c0 < end; c0 += lanes * 8 * kInFlight) {
            Raw8<T> raw[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u)
                if (row < vocab) raw[u] = load_cols(src, C(c0 + u * lanes * 8, dim));
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                const C c(c0 + u * lanes * 8, dim);
                float x[8];
                cols_values(raw[u], c, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = row < vocab ? x[j] * scale : 0.0f;
                stream_cols(dst, c, x);
            }
        }
    }
}

// Eight weights are four bytes of codes; eight lanes share a block's scale.
template <typename O>
__global__ __launch_bounds__(kThreads) void lookup_packed_kernel(const void *ids, bool i64, int64_t tokens, WView w,
                                                                 Levels lv, float scale, O *out, int lanes) {
    __shared__ float s_lv[16];
    if (threadIdx.x < 16) s_lv[threadIdx.x] = lv.q[threadIdx.x];
    __syncthreads();
    const int each = kThreads / lanes;
    const int64_t dim = w.k;
    for (int64_t t = (int64_t)blockIdx.x * each + threadIdx.x / lanes; t < tokens; t += (int64_t)gridDim.x * each) {
        const uint32_t row = token_key(ids, i64, t, w.n, -1);
        O *dst = out + t * dim;
        for (int64_t col = (threadIdx.x & (lanes - 1)) * 8; col < dim; col += lanes * 8) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.0f;
            if (row < w.n) {
                const int64_t i = (int64_t)row * dim + col;
                const uint32_t c = *reinterpret_cast<const uint32_t *>(w.codes + i / 2);
                const float s = wscale(w, i / kBlock);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = s_lv[(c >> (4 * j)) & 15u] * s * scale;
            }
            store8(dst + col, x);
        }
    }
}

int lanes_for(int64_t dim) {
    int lanes = 8;
    while (lanes < kThreads && (int64_t)lanes * 8 < dim) lanes *= 2;
    return lanes;
}

constexpr int64_t kMostWgs = int64_t(1) << 20;  // of a launch; more tokens go round

dim3 lookup_grid(int64_t tokens, int lanes) {
    const int64_t each = kThreads / lanes, need = (tokens + each - 1) / each;
    return dim3((uint32_t)(need < kMostWgs ? need : kMostWgs));
}

// ---- sorting the tokens ----

// Up to kOneTile each token counts its place among all, up to kRankTokens in its
// tile, and searches the others: a call with 7000 tokens takes 17.5 us the one way
// and 18.5 the other, with 9000 25.0 and 20.6. They cross between three tiles and
// four; the bound is three.
constexpr int kOneTile = 6144;
constexpr int kTile = 2048;
constexpr int kRankTokens = 32768;
constexpr int kTiles = 64;          // workgroups of a digit pass above
constexpr int kMaxBins = 1024;

// Lanes of the wave whose digit (of `width` bits) equals this lane's, among the
// live lanes.
__device__ __forceinline__ uint64_t same_digit(uint32_t d, int width, bool live) {
    uint64_t same = __ballot(live);
    for (int b = 0; b < width; ++b) {
        const bool bit = (d >> b) & 1u;
        const uint64_t set = __ballot(bit);
        same &= bit ? set : ~set;
    }
    return same;
}

// Exclusive sum over the workgroup's threads (1024), in the order of the threads.
__device__ __forceinline__ uint32_t scan1024(uint32_t x, uint32_t *s_wave) {
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    uint32_t scan = x;
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t up = __shfl_up(scan, o);
        scan += lane >= o ? up : 0u;
    }
    if (lane == 63) s_wave[wave] = scan;
    __syncthreads();
    uint32_t before = scan - x;
    for (int w = 0; w < wave; ++w) before += s_wave[w];
    return before;
}

// A dense gradient is cleared beside the sort's first launch, which hardly
// uses the memory.
template <typename G>
__device__ __forceinline__ void clear_share(G *grad, int64_t n, int64_t wg, int64_t wgs) {
    const float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    __builtin_amdgcn_s_setprio(3);  // few instructions, all of them stores: ahead of the sort's comparisons
    for (int64_t i = (wg * 1024 + threadIdx.x) * 8; i < n; i += wgs * 1024 * 8) store_upto8(grad + i, n - i, zero);
}

struct RankParams {
    const void *ids;
    bool i64;
    int32_t tokens, tile;
    int32_t wgs, each;  // workgroups that rank (those above clear the gradient), of `each` tokens: 16, 32 or 64
    int64_t vocab, skip;
    uint32_t *key_out, *idx_out;
    void *grad;
    int64_t n;
};

// Keys of s_key[0 .. 15] that are below `key`, or (kEqual) not above it.
template <bool kEqual>
__device__ __forceinline__ int count_below(const uint4 *s_key, uint32_t key) {
    int count = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 k = s_key[j];
        count += kEqual ? k.x <= key : k.x < key;
        count += kEqual ? k.y <= key : k.y < key;
        count += kEqual ? k.z <= key : k.z < key;
        count += kEqual ? k.w <= key : k.w < key;
    }
    return count;
}
// Those of a group that holds the key's own place: equal ones count up to there.
__device__ __forceinline__ int count_before(const uint4 *s_key, uint32_t key, int place) {
    int count = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 k = s_key[j];
        count += k.x < key || (k.x == key && 4 * j < place);
        count += k.y < key || (k.y == key && 4 * j + 1 < place);
        count += k.z < key || (k.z == key && 4 * j + 2 < place);
        count += k.w < key || (k.w == key && 4 * j + 3 < place);
    }
    return count;
}

// The place of each token in its tile's stable order, by counting the tokens
// before it: those with a smaller key, and earlier ones with its own. A
// workgroup takes `each` tokens; its 16 waves, and the 64 / each lanes of a token,
// compare with a share of the tile's keys in LDS, two instructions a pair. The
// work grows with the tile, but it is one launch on the whole chip.
template <typename G>
__global__ __launch_bounds__(1024) void rank_tokens_kernel(RankParams p) {
    __shared__ uint4 s_key4[kOneTile / 4];
    __shared__ int32_t s_count[16][64];
    if ((int)blockIdx.x >= p.wgs) {
        clear_share(static_cast<G *>(p.grad), p.n, blockIdx.x - p.wgs, gridDim.x - p.wgs);
        return;
    }
    uint32_t *s_key = reinterpret_cast<uint32_t *>(s_key4);
    const int first_token = blockIdx.x * p.each, tile0 = first_token / p.tile * p.tile;
    const int tokens = p.tokens - tile0 < p.tile ? p.tokens - tile0 : p.tile;
    const int padded = (tokens + 1023) / 1024 * 1024;  // at most kOneTile
    uint32_t k[kOneTile / 1024];
#pragma unroll
    for (int u = 0; u < kOneTile / 1024; ++u) {
        const int t = threadIdx.x + u * 1024;
        k[u] = token_key(p.ids, p.i64, tile0 + (t < tokens ? t : 0), p.vocab, p.skip);
    }
#pragma unroll
    for (int u = 0; u < kOneTile / 1024; ++u) {
        const int t = threadIdx.x + u * 1024;
        if (t < padded) s_key[t] = t < tokens ? k[u] : 0xFFFFFFFFu;
    }
    __syncthreads();
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int own = first_token - tile0, me = own + lane % p.each;
    const uint32_t key = s_key[me];
    // groups of 16 keys; the workgroup's own tokens are whole groups
    const int first = own / 16, last = first + p.each / 16, parts = 64 / p.each;
    const int shares = 16 * parts, share = wave * parts + lane / p.each;
    int count = 0;
    for (int t = share; t < padded / 16; t += shares) {
        if (t < first) count += count_below<true>(s_key4 + t * 4, key);
        else if (t >= last) count += count_below<false>(s_key4 + t * 4, key);
        else count += count_before(s_key4 + t * 4, key, me - t * 16);
    }
    for (int o = p.each; o < 64; o <<= 1) count += __shfl_xor(count, o);  // a token's lanes
    s_count[wave][lane] = count;
    __syncthreads();
    if ((int)threadIdx.x < p.each && me < tokens) {
        int r = tile0;
#pragma unroll
        for (int w = 0; w < 16; ++w) r += s_count[w][lane];
        p.key_out[r] = key;
        p.idx_out[r] = (uint32_t)(tile0 + me);
    }
}

// From sorted tiles to one order: a token's place is its place in its own tile
// and, in each other tile, the number of keys below its own (or equal, in
// earlier tiles). `lanes` lanes a token, one a tile, each with a binary search.
__global__ __launch_bounds__(kThreads) void merge_tiles_kernel(const uint32_t *key, const uint32_t *idx, int32_t tokens,
                                                               int32_t tile, int32_t lanes, uint32_t *key_out,
                                                               uint32_t *idx_out) {
    const int i = (int)((blockIdx.x * kThreads + threadIdx.x) / lanes), other = threadIdx.x & (lanes - 1);
    if (i >= tokens) return;
    const uint32_t k = key[i];
    const int mine = i / tile;
    int place = 0;
    if (other == mine) {
        place = i - mine * tile;
    } else if (other * tile < tokens) {
        const uint32_t *at = key + other * tile;
        const uint32_t bound = k + (other < mine ? 1u : 0u);
        int n = tokens - other * tile < tile ? tokens - other * tile : tile;
        while (n > 0) {  // place: so many are known to be below
            const int half = n / 2;
            const bool below = at[place + half] < bound;
            place += below ? half + 1 : 0;
            n = below ? n - half - 1 : half;
        }
    }
    for (int o = 1; o < lanes; o <<= 1) place += __shfl_xor(place, o);
    if (other == 0) {
        key_out[place] = k;
        idx_out[place] = idx[i];
    }
}

template <typename G>
__global__ __launch_bounds__(1024) void clear_kernel(G *grad, int64_t n) {
    clear_share(grad, n, blockIdx.x, gridDim.x);
}

struct DigitPass {
    const void *ids;        // first pass: the tokens
    const uint32_t *key, *idx;  // later passes: the last pass's output
    bool i64, first;
    int64_t tokens, tile, vocab, skip;
    int tiles, shift, width, bins;
    uint32_t *hist;         // [tiles][bins]
    uint32_t *key_out, *idx_out;
    void *grad;             // cleared beside the count, n elements (none: nullptr)
    int64_t n;
};

__device__ __forceinline__ uint32_t pass_key(const DigitPass &p, int64_t t) {
    return p.first ? token_key(p.ids, p.i64, t, p.vocab, p.skip) : p.key[t];
}

// The digits of each tile; the workgroups past the tiles clear the gradient.
template <typename G>
__global__ __launch_bounds__(1024) void digit_count_kernel(DigitPass p) {
    __shared__ uint32_t s_bin[kMaxBins];
    if ((int)blockIdx.x >= p.tiles) {
        clear_share(static_cast<G *>(p.grad), p.n, blockIdx.x - p.tiles, gridDim.x - p.tiles);
        return;
    }
    s_bin[threadIdx.x] = 0u;
    __syncthreads();
    const int64_t begin = blockIdx.x * p.tile, end = begin + p.tile < p.tokens ? begin + p.tile : p.tokens;
    for (int64_t t = begin + threadIdx.x; t < end; t += 1024)
        atomicAdd(&s_bin[(pass_key(p, t) >> p.shift) & (p.bins - 1)], 1u);
    __syncthreads();
    if ((int)threadIdx.x < p.bins) p.hist[(int64_t)blockIdx.x * p.bins + threadIdx.x] = s_bin[threadIdx.x];
}

// Stable scatter of one tile by one digit. Each of the 16 waves owns a run of
// the tile and a row of next places, which starts after all lower digits, all
// earlier tiles and the earlier waves; it takes 64 tokens at a time in order,
// and lanes with the same digit find each other by ballots over its bits.
__global__ __launch_bounds__(1024) void digit_scatter_kernel(DigitPass p) {
    __shared__ uint32_t s_next[16][kMaxBins];
    __shared__ uint32_t s_wave[16];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    for (int w = 0; w < 16; ++w) s_next[w][threadIdx.x] = 0u;
    __syncthreads();
    const int64_t run = p.tile / 16;
    const int64_t begin = blockIdx.x * p.tile + wave * run;
    const int64_t end = begin + run < p.tokens ? begin + run : p.tokens;
    for (int64_t t = begin + lane; t < end; t += 64)
        atomicAdd(&s_next[wave][(pass_key(p, t) >> p.shift) & (p.bins - 1)], 1u);
    uint32_t total = 0u, before = 0u;
    if ((int)threadIdx.x < p.bins)
        for (int t = 0; t < p.tiles; ++t) {
            const uint32_t c = p.hist[(int64_t)t * p.bins + threadIdx.x];
            before += t < (int)blockIdx.x ? c : 0u;
            total += c;
        }
    uint32_t place = scan1024(total, s_wave) + before;  // its barrier also ends the counting
    for (int w = 0; w < 16; ++w) {
        const uint32_t c = s_next[w][threadIdx.x];
        s_next[w][threadIdx.x] = place;
        place += c;
    }
    __syncthreads();
    volatile uint32_t *next = s_next[wave];
    for (int64_t t0 = begin; t0 < end; t0 += 64) {
        const int64_t t = t0 + lane;
        const bool live = t < end;
        const uint32_t key = live ? pass_key(p, t) : 0u;
        const uint32_t idx = !live || p.first ? (uint32_t)t : p.idx[t];
        const uint32_t d = (key >> p.shift) & (p.bins - 1);
        const uint64_t same = same_digit(d, p.width, live);
        const uint32_t rank = __popcll(same & ((1ull << lane) - 1ull));
        const uint32_t at = live ? next[d] + rank : 0u;
        __builtin_amdgcn_wave_barrier();
        if (live && rank == 0u) next[d] = at + (uint32_t)__popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (live) {
            p.key_out[at] = key;
            p.idx_out[at] = idx;
        }
    }
}

// ---- the gradient ----

constexpr int kFewTokens = 128;  // up to here one launch
constexpr int kMostChunk = 16;  // sorted places of a wave
constexpr int kCols = 512;  // columns of a wave
constexpr int kRows = 8;    // rows of dy, or shares of a run, in flight

struct GradParams {
    const uint32_t *key, *idx;  // sorted
    int64_t tokens, vocab, chunks;
    int32_t dim, slices, chunk;
    float scale;
    const void *dy;
    void *grad;
    float *partial;  // [chunks][2][dim]: the run that enters the chunk, the run that leaves it
    bool accumulate;
};

template <typename G>
__device__ __forceinline__ G *grad_row(const GradParams &p, uint32_t key) {
    return static_cast<G *>(p.grad) + (int64_t)key * p.dim;
}

// Each wave sums the runs of up to 16 sorted places in 512 columns. dy is read once, so
// where a wave's columns are whole cache lines (kStream) it is read past the
// caches: beside a gradient that the sort's launch has just cleared, 16384 x 4096
// bf16 into 32000 rows take 106 us in all instead of 117 (90 instead of 107 where
// every call writes the same gradient). With lines that two waves share it costs
// instead (5003 x 1601: 38 us for 36).
template <typename T, typename G, typename C, bool kStream, bool kAdd>
__global__ __launch_bounds__(kThreads) void run_sum_kernel(GradParams p) {
    const int lane = threadIdx.x % 64;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
    const int64_t c = unit / p.slices;
    if (c >= p.chunks) return;
    const C cols((int)(unit % p.slices) * kCols + lane * 8, p.dim);
    const int64_t start = c * p.chunk;
    const int len = (int)(p.tokens - start < p.chunk ? p.tokens - start : p.chunk);
    // lane j holds place start - 1 + j
    const int64_t place = start - 1 + lane;
    const bool there = lane < p.chunk + 2 && place >= 0 && place < p.tokens;
    const uint32_t vkey = there ? p.key[place] : 0xFFFFFFFFu, vidx = there ? p.idx[place] : 0u;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    bool entered = __builtin_amdgcn_readlane((int)vkey, 0) == __builtin_amdgcn_readlane((int)vkey, 1);
    for (int i0 = 0; i0 < len; i0 += kRows) {
        Raw8<T> raw[kRows];
        Raw8<G> old[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            // places past the tokens and keys that name no row load token 0 and are left below
            const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)vkey, i0 + u + 1);
            const uint32_t at = (uint32_t)__builtin_amdgcn_readlane((int)vidx, i0 + u + 1);
            const uint32_t idx = key < p.vocab ? at : 0u;
            const T *row = static_cast<const T *>(p.dy) + (int64_t)idx * p.dim;
            if constexpr (kStream) raw[u] = load_stream(row, cols);
            else raw[u] = load_cols(row, cols);
            // the row that a run ending here is added to; no other wave writes it
            const uint32_t after = (uint32_t)__builtin_amdgcn_readlane((int)vkey, i0 + u + 2);
            if (kAdd && after != key && key < p.vocab) old[u] = load_cols(grad_row<G>(p, key), cols);
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int i = i0 + u;
            const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)vkey, i + 1);
            const uint32_t after = (uint32_t)__builtin_amdgcn_readlane((int)vkey, i + 2);
            if (i >= len || key >= p.vocab) return;  // keys that name no row come last
            float x[8];
            cols_values(raw[u], cols, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += x[j];
            const bool leaves = after == key;
            if (leaves && i + 1 < len) continue;
            if (entered || leaves) {
                store_cols(p.partial + (c * 2 + (entered ? 0 : 1)) * p.dim, cols, acc);
            } else {
                if constexpr (kAdd) cols_values(old[u], cols, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = kAdd ? x[j] + acc[j] * p.scale : acc[j] * p.scale;
                store_cols(grad_row<G>(p, key), cols, x);
            }
            entered = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
        }
    }
}

// First place whose key is not below `key`: 64 probes a step.
__device__ __forceinline__ int64_t lower_bound(const uint32_t *keys, int64_t n, uint32_t key) {
    const int lane = threadIdx.x % 64;
    int64_t lo = 0, hi = n;  // the answer is in [lo, hi]
    while (hi > lo) {
        const int64_t step = (hi - lo + 63) / 64;
        const int64_t at = lo + lane * step;  // places before the answer are a prefix
        const uint64_t below = __ballot(at < hi && keys[at] < key);
        const int c = (int)__popcll(below);
        if (c == 0) return lo;
        const int64_t last = lo + (c - 1) * step;  // below
        hi = last + step < hi ? last + step : hi;
        lo = last + 1;
    }
    return lo;
}

// The runs that leave the chunk they begin in: their shares, chunk after chunk.
template <typename G, bool kNarrow>
__global__ __launch_bounds__(kThreads) void run_join_kernel(GradParams p) {
    const int lane = threadIdx.x % 64;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
    const int64_t c = unit / p.slices;
    if (c + 1 >= p.chunks) return;
    const Cols<kNarrow> cols((int)(unit % p.slices) * kCols + lane * 8, p.dim);
    const int64_t start = c * p.chunk, end = start + p.chunk;
    // One round of loads tells most of it: the chunks that the run enters are those
    // after this one that begin with its key.
    const int64_t ahead = end + lane * p.chunk;
    const uint32_t next = p.key[ahead < p.tokens ? ahead : p.tokens - 1];
    const uint32_t key = p.key[end - 1], begins = p.key[start], before = start > 0 ? p.key[start - 1] : 0xFFFFFFFFu;
    const uint64_t same = __ballot(ahead < p.tokens && next == key);
    if (!(same & 1) || key >= p.vocab) return;
    if (begins == key && before == key) return;  // begins before
    const int entered = (int)__popcll(same);
    const int64_t last = entered < 64 ? c + entered
                                      : (end + lower_bound(p.key + end, p.tokens - end, key + 1) - 1) / p.chunk;
    Raw8<G> old;
    if (p.accumulate) old = load_cols(grad_row<G>(p, key), cols);
    float acc[8];
    cols_values(load_cols(p.partial + (c * 2 + 1) * p.dim, cols), cols, acc);
    for (int64_t d = c + 1; d <= last; d += kRows) {
        Raw8<float> raw[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u)
            raw[u] = load_cols(p.partial + (d + u < last ? d + u : last) * 2 * p.dim, cols);
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if (d + u > last) break;
            float x[8];
            cols_values(raw[u], cols, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += x[j];
        }
    }
    float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (p.accumulate) cols_values(old, cols, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] += acc[j] * p.scale;
    store_cols(grad_row<G>(p, key), cols, x);
}

// The whole gradient of few tokens in one launch. A lane knows the ids of two
// tokens, so a wave finds all tokens of an id by ballots: the first one's wave adds
// their rows, in the order of the tokens, for 512 columns. Without kAdd the
// workgroups past those clear the rows that no token names. 128 tokens added to a
// gradient of 32000 x 4096 take 8.4 us a call instead of 13 with the sort, written
// 35 instead of 40; 128 times the same token 14.9 instead of 13, so no more than that.
struct FewParams {
    const void *ids;
    bool i64;
    int32_t tokens, dim, slices, wgs;
    int64_t vocab, skip;
    float scale;
    const void *dy;
    void *grad;
};
template <typename T, typename G, bool kNarrow, bool kAdd>
__global__ __launch_bounds__(kThreads) void few_tokens_kernel(FewParams p) {
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    uint32_t key[kFewTokens / 64];
#pragma unroll
    for (int k = 0; k < kFewTokens / 64; ++k) {
        const int t = lane + 64 * k;
        key[k] = token_key(p.ids, p.i64, t < p.tokens ? t : 0, p.vocab, p.skip);
        key[k] = t < p.tokens ? key[k] : 0xFFFFFFFFu;
    }
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if ((int)blockIdx.x >= p.wgs) {
        // a row is a wave's, or the workgroup's where it is longer than a wave's store
        const bool wide = p.dim > 512;
        constexpr int kEach = 16 / sizeof(G);
        const int each = wide ? 1 : kThreads / 64, step = (wide ? kThreads : 64) * kEach;
        const int64_t stride = (int64_t)(gridDim.x - p.wgs) * each;
        for (int64_t row = (int64_t)(blockIdx.x - p.wgs) * each + (wide ? 0 : wave); row < p.vocab; row += stride) {
            bool named = false;
#pragma unroll
            for (int k = 0; k < kFewTokens / 64; ++k) named |= key[k] == (uint32_t)row;
            if (__any(named)) continue;
            G *dst = static_cast<G *>(p.grad) + row * p.dim;
            for (int c = (wide ? (int)threadIdx.x : lane) * kEach; c < p.dim; c += step) {
                if (c + kEach <= p.dim) reinterpret_cast<u32x4_any2 *>(dst + c)->v = u32x4{0, 0, 0, 0};
                else
                    for (int j = c; j < p.dim; ++j) store1(dst + j, 0.0f);
            }
        }
        return;
    }
    const int unit = (int)blockIdx.x * (kThreads / 64) + wave, t = unit / p.slices;
    if (t >= p.tokens) return;
    uint32_t mine = 0;
#pragma unroll
    for (int k = 0; k < kFewTokens / 64; ++k)
        if (t / 64 == k) mine = (uint32_t)__builtin_amdgcn_readlane((int)key[k], t % 64);
    if (mine >= p.vocab) return;
    uint64_t same[kFewTokens / 64];
#pragma unroll
    for (int k = 0; k < kFewTokens / 64; ++k) {
        same[k] = __ballot(key[k] == mine);
        const uint64_t before = t / 64 > k ? ~uint64_t(0) : t / 64 == k ? (uint64_t(1) << (t % 64)) - 1 : 0;
        if (same[k] & before) return;  // not the first one
    }
    const Cols<kNarrow> cols((unit % p.slices) * kCols + lane * 8, p.dim);
    G *dst = static_cast<G *>(p.grad) + (int64_t)mine * p.dim;
    Raw8<G> old;
    if constexpr (kAdd) old = load_cols(dst, cols);
    int base = 0, left = 0;
#pragma unroll
    for (int k = 0; k < kFewTokens / 64; ++k) left += (int)__popcll(same[k]);
    for (; left > 0; left -= kRows) {
        Raw8<T> raw[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if (u >= left) break;  // a bit is left in some word as long as this does not hold
            while (same[0] == 0) {
#pragma unroll
                for (int k = 0; k + 1 < kFewTokens / 64; ++k) same[k] = same[k + 1];
                same[kFewTokens / 64 - 1] = 0;
                base += 64;
            }
            const int at = base + __builtin_ctzll(same[0]);
            same[0] &= same[0] - 1;
            raw[u] = load_cols(static_cast<const T *>(p.dy) + (int64_t)at * p.dim, cols);
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if (u >= left) break;
            float x[8];
            cols_values(raw[u], cols, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += x[j];
        }
    }
    float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (kAdd) cols_values(old, cols, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = kAdd ? x[j] + acc[j] * p.scale : acc[j] * p.scale;
    store_cols(dst, cols, x);
}

// ---- host side ----

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

struct Layout {
    size_t key, idx, key2, idx2, hist, partial, bytes;
    int64_t chunks;
    int32_t chunk, slices;
};
Layout layout_of(int64_t tokens, int64_t dim) {
    Layout l{};
    size_t at = 0;
    auto take = [&](size_t b) {
        const size_t was = at;
        at += up256(b);
        return was;
    };
    l.slices = (int32_t)((dim + kCols - 1) / kCols);
    // A wave's places are one after the other, so few tokens are cut finer: down to
    // 8 places as long as the chip is not full of waves.
    l.chunk = kMostChunk;
    while (l.chunk > 8 && tokens / l.chunk * l.slices < 8192) l.chunk /= 2;
    l.chunks = (tokens + l.chunk - 1) / l.chunk;
    l.key = take((size_t)tokens * 4), l.idx = take((size_t)tokens * 4);
    if (tokens > kOneTile) l.key2 = take((size_t)tokens * 4), l.idx2 = take((size_t)tokens * 4);
    if (tokens > kRankTokens) l.hist = take((size_t)kTiles * kMaxBins * 4);
    l.partial = take((size_t)(l.chunks * 2 * dim) * 4);
    l.bytes = at;
    return l;
}

constexpr int kClearWgs = 1024;  // of 1024 threads, four for each CU

// Workgroups that clear n elements.
uint32_t clear_wgs(int64_t n) {
    const int64_t need = (n + 8191) / 8192;
    return (uint32_t)(need < kClearWgs ? need : kClearWgs);
}

int bits_of(int64_t vocab) {  // the keys are 0 .. vocab
    int bits = 1;
    while ((vocab >> bits) != 0) ++bits;
    return bits;
}

struct Sort {
    const void *ids;
    bool i64;
    int64_t tokens, vocab, skip;
    uint32_t *key, *idx, *key2, *idx2, *hist;
    void *clear;  // a gradient of n elements to clear beside the sort, or nullptr
    int64_t n;
};

template <typename G>
hipError_t sort_tokens(const Sort &q, hipStream_t s) {
    const uint32_t clear = q.clear ? clear_wgs(q.n) : 0u;
    if (q.tokens == 0) {
        if (clear) clear_kernel<G><<<dim3(clear), dim3(1024), 0, s>>>(static_cast<G *>(q.clear), q.n);
        return hipGetLastError();
    }
    if (q.tokens <= kRankTokens) {
        const bool one = q.tokens <= kOneTile;
        RankParams p{};
        p.ids = q.ids, p.i64 = q.i64, p.tokens = (int32_t)q.tokens, p.vocab = q.vocab, p.skip = q.skip;
        p.tile = one ? kOneTile : kTile;
        // as many workgroups as there are CUs, where there are tokens for them
        p.each = p.tokens > 16384 ? 64 : p.tokens > 6144 ? 32 : 16;
        p.wgs = (p.tokens + p.each - 1) / p.each;
        p.key_out = one ? q.key : q.key2, p.idx_out = one ? q.idx : q.idx2, p.grad = q.clear, p.n = q.n;
        rank_tokens_kernel<G><<<dim3(p.wgs + clear), dim3(1024), 0, s>>>(p);
        if (!one) {
            int lanes = 2;
            while (lanes * kTile < p.tokens) lanes *= 2;
            merge_tiles_kernel<<<dim3((uint32_t)((q.tokens * lanes + kThreads - 1) / kThreads)), dim3(kThreads), 0, s>>>(
                q.key2, q.idx2, p.tokens, kTile, lanes, q.key, q.idx);
        }
        return hipGetLastError();
    }
    const int bits = bits_of(q.vocab), passes = (bits + 9) / 10;
    DigitPass p{};
    p.ids = q.ids, p.i64 = q.i64, p.tokens = q.tokens, p.vocab = q.vocab, p.skip = q.skip;
    p.tile = ((q.tokens + kTiles - 1) / kTiles + 1023) / 1024 * 1024;
    p.tiles = (int)((q.tokens + p.tile - 1) / p.tile);
    p.width = (bits + passes - 1) / passes, p.bins = 1 << p.width;
    p.hist = q.hist, p.grad = q.clear, p.n = q.n;
    hipError_t err = hipSuccess;
    for (int i = 0; i < passes; ++i) {
        const bool to_main = (passes - 1 - i) % 2 == 0;  // the last pass ends in (key, idx)
        p.first = i == 0, p.shift = i * p.width;
        p.key = to_main ? q.key2 : q.key, p.idx = to_main ? q.idx2 : q.idx;
        p.key_out = to_main ? q.key : q.key2, p.idx_out = to_main ? q.idx : q.idx2;
        digit_count_kernel<G><<<dim3(p.tiles + (i == 0 ? clear : 0u)), dim3(1024), 0, s>>>(p);
        digit_scatter_kernel<<<dim3(p.tiles), dim3(1024), 0, s>>>(p);
        const hipError_t r = hipGetLastError();
        if (err == hipSuccess) err = r;
    }
    return err;
}

template <typename T, typename G>
hipError_t gradient(const Sort &q, const GradParams &p, hipStream_t s) {
    hipError_t err = sort_tokens<G>(q, s);
    if (err != hipSuccess || p.tokens == 0) return err;
    const uint32_t wgs = (uint32_t)((p.chunks * p.slices + 3) / 4);
    const bool narrow = p.dim < 8, lines = p.dim * sizeof(T) % 128 == 0;
    const bool add = p.accumulate;
    typedef std::conditional_t<sizeof(T) == 2 && sizeof(G) == 2, Cols<false>, Fours> Lines;
    auto pick = [&](auto c, auto stream) {
        typedef typename decltype(c)::type C;
        return add ? run_sum_kernel<T, G, C, stream.value, true> : run_sum_kernel<T, G, C, stream.value, false>;
    };
    auto sum = narrow  ? pick(ColsTag<Cols<true>>{}, std::false_type{})
               : lines ? pick(ColsTag<Lines>{}, std::true_type{})
                       : pick(ColsTag<Cols<false>>{}, std::false_type{});
    sum<<<dim3(wgs), dim3(kThreads), 0, s>>>(p);
    if (p.chunks > 1) {
        auto join = narrow ? run_join_kernel<G, true> : run_join_kernel<G, false>;
        join<<<dim3(wgs), dim3(kThreads), 0, s>>>(p);
    }
    return hipGetLastError();
}

template <typename T, typename G>
hipError_t few_tokens(FewParams p, bool add, hipStream_t s) {
    p.wgs = (p.tokens * p.slices + 3) / 4;
    const int64_t rows = p.dim > 512 ? p.vocab : (p.vocab + 3) / 4;
    const int64_t clear = add ? 0 : rows < 2048 ? rows : 2048;  // eight for each CU
    auto kernel = p.dim < 8 ? (add ? few_tokens_kernel<T, G, true, true> : few_tokens_kernel<T, G, true, false>)
                            : (add ? few_tokens_kernel<T, G, false, true> : few_tokens_kernel<T, G, false, false>);
    kernel<<<dim3((uint32_t)(p.wgs + clear)), dim3(kThreads), 0, s>>>(p);
    return hipGetLastError();
}

template <typename T, typename O>
hipError_t lookup(const void *ids, bool i64, int64_t tokens, const void *table, int64_t vocab, int64_t dim,
                  float scale, void *out, hipStream_t s) {
    const int lanes = lanes_for(dim);
    // as many vectors in flight as a lane has, up to four: with more, a lane
    // works on columns past the row (16384 x 1000 bf16: 19 us instead of 12)
    const int64_t vecs = (dim + lanes * 8 - 1) / (lanes * 8);
    auto pick = [&](auto c) {
        typedef typename decltype(c)::type C;
        return vecs == 1 ? lookup_kernel<T, O, 1, C> : vecs == 2 ? lookup_kernel<T, O, 2, C> : lookup_kernel<T, O, 4, C>;
    };
    auto kernel = dim < 8 ? lookup_kernel<T, O, 1, Cols<true>> : pick(ColsTag<Cols<false>>{});
    if constexpr (sizeof(O) == 4)  // 16384 x 2048 bf16 to fp32: 30 us instead of 44
        if (dim % 8 == 0 && lanes >= 64) kernel = pick(ColsTag<Fours>{});
    kernel<<<lookup_grid(tokens, lanes), dim3(kThreads), 0, s>>>(
        ids, i64, tokens, static_cast<const T *>(table), vocab, (int32_t)dim, scale, static_cast<O *>(out), lanes);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_embedding_forward(const void *ids, bool i64, int64_t tokens, const void *table, nf4_dtype dt,
                                    int64_t vocab, int64_t dim, float scale, void *out, nf4_dtype ot, hipStream_t s) {
    if (dt == NF4_BF16)
        return ot == NF4_BF16 ? lookup<Bf16, Bf16>(ids, i64, tokens, table, vocab, dim, scale, out, s)
                              : lookup<Bf16, float>(ids, i64, tokens, table, vocab, dim, scale, out, s);
    return ot == NF4_BF16 ? lookup<float, Bf16>(ids, i64, tokens, table, vocab, dim, scale, out, s)
                          : lookup<float, float>(ids, i64, tokens, table, vocab, dim, scale, out, s);
}

hipError_t launch_embedding_packed(const void *ids, bool i64, int64_t tokens, const nf4_weight &w, float scale,
                                   void *out, nf4_dtype ot, hipStream_t s) {
    const int lanes = lanes_for(w.k_in);
    const dim3 grid = lookup_grid(tokens, lanes);
    if (ot == NF4_BF16)
        lookup_packed_kernel<Bf16><<<grid, dim3(kThreads), 0, s>>>(ids, i64, tokens, make_view(w), levels(), scale,
                                                                   static_cast<Bf16 *>(out), lanes);
    else
        lookup_packed_kernel<float><<<grid, dim3(kThreads), 0, s>>>(ids, i64, tokens, make_view(w), levels(), scale,
                                                                    static_cast<float *>(out), lanes);
    return hipGetLastError();
}

size_t embedding_backward_workspace(int64_t tokens, int64_t, int64_t dim) { return layout_of(tokens, dim).bytes; }

hipError_t launch_embedding_backward(const void *ids, bool i64, int64_t tokens, const void *dy, nf4_dtype dt,
                                     int64_t vocab, int64_t dim, float scale, int64_t padding_id, void *grad,
                                     nf4_dtype gt, bool accumulate, void *workspace, hipStream_t s) {
    const Layout l = layout_of(tokens, dim);
    if (tokens > 0 && tokens <= kFewTokens) {
        const FewParams p{ids, i64, (int32_t)tokens, (int32_t)dim, l.slices, 0, vocab, padding_id, scale, dy, grad};
        if (dt == NF4_BF16)
            return gt == NF4_BF16 ? few_tokens<Bf16, Bf16>(p, accumulate, s) : few_tokens<Bf16, float>(p, accumulate, s);
        return gt == NF4_BF16 ? few_tokens<float, Bf16>(p, accumulate, s) : few_tokens<float, float>(p, accumulate, s);
    }
    char *ws = static_cast<char *>(workspace);
    auto words = [ws](size_t at) { return reinterpret_cast<uint32_t *>(ws + at); };
    Sort q{};
    q.ids = ids, q.i64 = i64, q.tokens = tokens, q.vocab = vocab, q.skip = padding_id;
    q.key = words(l.key), q.idx = words(l.idx), q.key2 = words(l.key2), q.idx2 = words(l.idx2), q.hist = words(l.hist);
    q.clear = accumulate ? nullptr : grad, q.n = vocab * dim;
    GradParams p{};
    p.key = q.key, p.idx = q.idx;
    p.tokens = tokens, p.vocab = vocab, p.chunks = l.chunks;
    p.dim = (int32_t)dim, p.slices = l.slices, p.chunk = l.chunk;
    p.scale = scale, p.dy = dy, p.grad = grad;
    p.partial = reinterpret_cast<float *>(ws + l.partial), p.accumulate = accumulate;
    if (dt == NF4_BF16) return gt == NF4_BF16 ? gradient<Bf16, Bf16>(q, p, s) : gradient<Bf16, float>(q, p, s);
    return gt == NF4_BF16 ? gradient<float, Bf16>(q, p, s) : gradient<float, float>(q, p, s);
}

}  // namespace nf4
