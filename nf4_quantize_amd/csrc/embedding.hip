// embedding.hip - the token embedding for gfx950: rows of a dense or an NF4
// table with a scale, and the gradient of the table by sorted tokens. The
// contracts are in nf4.h (nf4_embedding_forward, nf4_embedding_backward).
//
// The forward moves each looked-up row once in and once out. The backward
// sorts the tokens by their id (stable, so that a row's gradient is summed in
// the order of the tokens), sums runs of equal ids chunk by chunk, joins the
// runs that cross chunks and, for a dense gradient, clears the rows that no
// token names. It is bound by reading dy and writing the table's gradient.
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

template <typename T, typename O>
__global__ __launch_bounds__(kThreads) void lookup_kernel(const void *ids, bool i64, int64_t tokens, const T *table,
                                                          int64_t vocab, int32_t dim, float scale, O *out, int lanes) {
    const int each = kThreads / lanes;
    for (int64_t t = (int64_t)blockIdx.x * each + threadIdx.x / lanes; t < tokens; t += (int64_t)gridDim.x * each) {
        const uint32_t row = token_key(ids, i64, t, vocab, -1);
        const T *src = table + (int64_t)row * dim;
        O *dst = out + t * dim;
        for (int col = (threadIdx.x & (lanes - 1)) * 8; col < dim; col += lanes * 8) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.0f;
            if (row < vocab) {
                load_upto8(src + col, dim - col, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= scale;
            }
            store_upto8(dst + col, dim - col, x);
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

constexpr int64_t kRankTokens = 8192;  // up to here ranks are counted, above the sort is by digits
constexpr int kTiles = 64;             // workgroups of a digit pass
constexpr int kMaxBins = 1024;

// Rank of each token by counting the tokens before it: id below its own, or
// equal and at an earlier place. 64 tokens a workgroup, each wave counts over a
// quarter of the others.
__global__ __launch_bounds__(kThreads) void rank_kernel(const void *ids, bool i64, int32_t tokens, int64_t vocab,
                                                        int64_t skip, uint32_t *skey, uint32_t *sidx) {
    __shared__ uint32_t s_key[kRankTokens];
    __shared__ int32_t s_count[4][64];
    const int padded = (tokens + 255) / 256 * 256;
    for (int t = threadIdx.x; t < padded; t += kThreads)
        s_key[t] = t < tokens ? token_key(ids, i64, t, vocab, skip) : 0xFFFFFFFFu;
    __syncthreads();
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int me = blockIdx.x * 64 + lane;  // < padded
    const uint32_t key = s_key[me];
    const int quarter = padded / 4, begin = wave * quarter;
    int count = 0;
    for (int j = begin; j < begin + quarter; ++j) {
        const uint32_t k = s_key[j];
        count += (k < key || (k == key && j < me)) ? 1 : 0;
    }
    s_count[wave][lane] = count;
    __syncthreads();
    if (wave == 0 && me < tokens) {
        const int r = s_count[0][lane] + s_count[1][lane] + s_count[2][lane] + s_count[3][lane];
        skey[r] = key;
        sidx[r] = (uint32_t)me;
    }
}

struct DigitPass {
    const void *ids;        // first pass: the tokens
    const uint32_t *key, *idx;  // later passes: the last pass's output
    bool i64, first;
    int64_t tokens, tile, vocab, skip;
    int shift, bins;
    uint32_t *hist;         // [tiles][bins]
    uint32_t *key_out, *idx_out;
};

__device__ __forceinline__ uint32_t pass_key(const DigitPass &p, int64_t t) {
    return p.first ? token_key(p.ids, p.i64, t, p.vocab, p.skip) : p.key[t];
}

__global__ __launch_bounds__(1024) void digit_count_kernel(DigitPass p) {
    __shared__ uint32_t s_bin[kMaxBins];
    s_bin[threadIdx.x] = 0u;
    __syncthreads();
    const int64_t begin = blockIdx.x * p.tile, end = begin + p.tile < p.tokens ? begin + p.tile : p.tokens;
    for (int64_t t = begin + threadIdx.x; t < end; t += 1024)
        atomicAdd(&s_bin[(pass_key(p, t) >> p.shift) & (p.bins - 1)], 1u);
    __syncthreads();
    if ((int)threadIdx.x < p.bins) p.hist[(int64_t)blockIdx.x * p.bins + threadIdx.x] = s_bin[threadIdx.x];
}

// Stable scatter of one tile by one digit. Each of the 16 waves owns a run of
// the tile and a row of next places, which starts at the digit's place after
// all lower digits, all earlier tiles and the earlier waves of this tile. A
// wave takes 64 keys at a time in order: lanes with the same digit find each
// other by ballots over its bits.
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
        for (uint32_t t = 0; t < gridDim.x; ++t) {
            const uint32_t c = p.hist[(int64_t)t * p.bins + threadIdx.x];
            before += t < blockIdx.x ? c : 0u;
            total += c;
        }
    uint32_t scan = total;  // inclusive over the wave's digits
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t up = __shfl_up(scan, o);
        scan += lane >= o ? up : 0u;
    }
    if (lane == 63) s_wave[wave] = scan;
    __syncthreads();
    uint32_t place = scan - total + before;
    for (int w = 0; w < wave; ++w) place += s_wave[w];
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
        uint64_t same = __ballot(live);
        for (int b = 1; b < p.bins; b <<= 1) {
            const uint64_t set = __ballot((d & b) != 0u);
            same &= (d & b) ? set : ~set;
        }
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

constexpr int kChunk = 16;  // sorted places of a wave
constexpr int kCols = 512;  // columns of a wave

struct GradParams {
    const uint32_t *key, *idx;  // sorted
    int64_t tokens, vocab, chunks;
    int32_t dim, slices;
    float scale;
    const void *dy;
    void *grad;
    float *partial;  // [chunks][2][dim]: the run that enters the chunk, the run that leaves it
    bool accumulate;
};

template <typename G>
__device__ __forceinline__ void write_row(const GradParams &p, uint32_t key, int col, float (&acc)[8]) {
    G *dst = static_cast<G *>(p.grad) + (int64_t)key * p.dim + col;
    const int live = p.dim - col;
    if (live <= 0) return;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    if (p.accumulate) load_upto8(dst, live, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] += acc[j] * p.scale;
    store_upto8(dst, live, x);
}

template <typename T, typename G>
__global__ __launch_bounds__(kThreads) void run_sum_kernel(GradParams p) {
    const int lane = threadIdx.x % 64;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
    const int64_t c = unit / p.slices;
    if (c >= p.chunks) return;
    const int col = (int)(unit % p.slices) * kCols + lane * 8;
    const int64_t start = c * kChunk;
    const int len = (int)(p.tokens - start < kChunk ? p.tokens - start : kChunk);
    // lane j holds place start - 1 + j
    const int64_t place = start - 1 + lane;
    const bool there = lane < kChunk + 2 && place >= 0 && place < p.tokens;
    const uint32_t vkey = there ? p.key[place] : 0xFFFFFFFFu, vidx = there ? p.idx[place] : 0u;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    bool entered = __builtin_amdgcn_readlane((int)vkey, 0) == __builtin_amdgcn_readlane((int)vkey, 1);
    for (int i = 0; i < len; ++i) {
        const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)vkey, i + 1);
        if (key >= p.vocab) return;
        const uint32_t idx = (uint32_t)__builtin_amdgcn_readlane((int)vidx, i + 1);
        const uint32_t after = (uint32_t)__builtin_amdgcn_readlane((int)vkey, i + 2);
        if (col < p.dim) {
            float x[8];
            load_upto8(static_cast<const T *>(p.dy) + (int64_t)idx * p.dim + col, p.dim - col, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += x[j];
        }
        const bool leaves = after == key;
        if (leaves && i + 1 < len) continue;
        if (entered || leaves) {
            float *dst = p.partial + (c * 2 + (entered ? 0 : 1)) * p.dim + col;
            if (col < p.dim) store_upto8(dst, p.dim - col, acc);
        } else {
            write_row<G>(p, key, col, acc);
        }
        entered = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
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
template <typename G>
__global__ __launch_bounds__(kThreads) void run_join_kernel(GradParams p) {
    const int lane = threadIdx.x % 64;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
    const int64_t c = unit / p.slices;
    if (c + 1 >= p.chunks) return;
    const int col = (int)(unit % p.slices) * kCols + lane * 8;
    const int64_t start = c * kChunk, end = start + kChunk;
    const uint32_t key = p.key[end - 1];
    if (p.key[end] != key || key >= p.vocab) return;
    if (p.key[start] == key && start > 0 && p.key[start - 1] == key) return;  // begins before
    const int64_t stop = end + lower_bound(p.key + end, p.tokens - end, key + 1);
    const int64_t last = (stop - 1) / kChunk;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    if (col < p.dim) {
        load_upto8(p.partial + (c * 2 + 1) * p.dim + col, p.dim - col, acc);
        for (int64_t d = c + 1; d <= last; ++d) {
            float x[8];
            load_upto8(p.partial + d * 2 * p.dim + col, p.dim - col, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += x[j];
        }
    }
    write_row<G>(p, key, col, acc);
}

constexpr int kClearRows = 64;

// Rows that no token names, 64 rows a workgroup.
template <typename G>
__global__ __launch_bounds__(kThreads) void clear_rows_kernel(GradParams p) {
    __shared__ uint32_t s_named[2];
    if (threadIdx.x < 2) s_named[threadIdx.x] = 0u;
    __syncthreads();
    const int64_t row0 = (int64_t)blockIdx.x * kClearRows;
    const int64_t rows = p.vocab - row0 < kClearRows ? p.vocab - row0 : kClearRows;
    if (threadIdx.x < 64) {
        const int64_t from = lower_bound(p.key, p.tokens, (uint32_t)row0);
        for (int64_t t0 = from; t0 < p.tokens; t0 += 64) {
            const int64_t t = t0 + threadIdx.x;
            const uint32_t off = t < p.tokens ? p.key[t] - (uint32_t)row0 : 0xFFFFFFFFu;
            if (off < rows) atomicOr(&s_named[off / 32], 1u << (off % 32));
            if (__ballot(off >= rows) != 0ull) break;
        }
    }
    __syncthreads();
    const uint64_t named = (uint64_t)s_named[0] | ((uint64_t)s_named[1] << 32);
    float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int r = 0; r < rows; ++r) {
        if ((named >> r) & 1ull) continue;
        G *dst = static_cast<G *>(p.grad) + (row0 + r) * p.dim;
        for (int col = threadIdx.x * 8; col < p.dim; col += kThreads * 8) store_upto8(dst + col, p.dim - col, zero);
    }
}

// ---- host side ----

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

struct Layout {
    size_t key, idx, key2, idx2, hist, partial, bytes;
    int64_t chunks;
};
Layout layout_of(int64_t tokens, int64_t dim) {
    Layout l{};
    size_t at = 0;
    auto take = [&](size_t b) {
        const size_t was = at;
        at += up256(b);
        return was;
    };
    l.chunks = (tokens + kChunk - 1) / kChunk;
    l.key = take((size_t)tokens * 4), l.idx = take((size_t)tokens * 4);
    if (tokens > kRankTokens) {
        l.key2 = take((size_t)tokens * 4), l.idx2 = take((size_t)tokens * 4);
        l.hist = take((size_t)kTiles * kMaxBins * 4);
    }
    l.partial = take((size_t)(l.chunks * 2 * dim) * 4);
    l.bytes = at;
    return l;
}

// Sorts by digits of equal width, at most 10 bits each; the keys are 0 .. vocab.
hipError_t sort_by_digits(const void *ids, bool i64, int64_t tokens, int64_t vocab, int64_t skip, uint32_t *key,
                          uint32_t *idx, uint32_t *key2, uint32_t *idx2, uint32_t *hist, hipStream_t s) {
    int bits = 1;
    while ((vocab >> bits) != 0) ++bits;
    const int passes = (bits + 9) / 10, width = (bits + passes - 1) / passes;
    DigitPass p{};
    p.ids = ids, p.i64 = i64, p.tokens = tokens, p.vocab = vocab, p.skip = skip;
    p.tile = ((tokens + kTiles - 1) / kTiles + 1023) / 1024 * 1024;
    p.bins = 1 << width, p.hist = hist;
    const uint32_t tiles = (uint32_t)((tokens + p.tile - 1) / p.tile);
    hipError_t err = hipSuccess;
    for (int i = 0; i < passes; ++i) {
        const bool to_main = (passes - 1 - i) % 2 == 0;  // the last pass ends in (key, idx)
        p.first = i == 0, p.shift = i * width;
        p.key = to_main ? key2 : key, p.idx = to_main ? idx2 : idx;
        p.key_out = to_main ? key : key2, p.idx_out = to_main ? idx : idx2;
        digit_count_kernel<<<dim3(tiles), dim3(1024), 0, s>>>(p);
        digit_scatter_kernel<<<dim3(tiles), dim3(1024), 0, s>>>(p);
        const hipError_t r = hipGetLastError();
        if (err == hipSuccess) err = r;
    }
    return err;
}

template <typename T, typename G>
hipError_t gradient(const GradParams &p, hipStream_t s) {
    hipError_t err = hipSuccess;
    if (p.tokens > 0) {
        const uint32_t wgs = (uint32_t)((p.chunks * p.slices + 3) / 4);
        run_sum_kernel<T, G><<<dim3(wgs), dim3(kThreads), 0, s>>>(p);
        err = hipGetLastError();
        if (p.chunks > 1) {
            run_join_kernel<G><<<dim3(wgs), dim3(kThreads), 0, s>>>(p);
            const hipError_t r = hipGetLastError();
            if (err == hipSuccess) err = r;
        }
    }
    if (!p.accumulate) {
        clear_rows_kernel<G><<<dim3((uint32_t)((p.vocab + kClearRows - 1) / kClearRows)), dim3(kThreads), 0, s>>>(p);
        const hipError_t r = hipGetLastError();
        if (err == hipSuccess) err = r;
    }
    return err;
}

template <typename T, typename O>
hipError_t lookup(const void *ids, bool i64, int64_t tokens, const void *table, int64_t vocab, int64_t dim,
                  float scale, void *out, hipStream_t s) {
    const int lanes = lanes_for(dim);
    lookup_kernel<T, O><<<lookup_grid(tokens, lanes), dim3(kThreads), 0, s>>>(
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
    char *ws = static_cast<char *>(workspace);
    uint32_t *key = reinterpret_cast<uint32_t *>(ws + l.key), *idx = reinterpret_cast<uint32_t *>(ws + l.idx);
    hipError_t err = hipSuccess;
    if (tokens > kRankTokens) {
        err = sort_by_digits(ids, i64, tokens, vocab, padding_id, key, idx, reinterpret_cast<uint32_t *>(ws + l.key2),
                             reinterpret_cast<uint32_t *>(ws + l.idx2), reinterpret_cast<uint32_t *>(ws + l.hist), s);
    } else if (tokens > 0) {
        rank_kernel<<<dim3((uint32_t)((tokens + 63) / 64)), dim3(kThreads), 0, s>>>(ids, i64, (int32_t)tokens, vocab,
                                                                                   padding_id, key, idx);
        err = hipGetLastError();
    }
    if (err != hipSuccess) return err;
    GradParams p{};
    p.key = key, p.idx = idx;
    p.tokens = tokens, p.vocab = vocab, p.chunks = l.chunks;
    p.dim = (int32_t)dim, p.slices = (int32_t)((dim + kCols - 1) / kCols);
    p.scale = scale, p.dy = dy, p.grad = grad;
    p.partial = reinterpret_cast<float *>(ws + l.partial), p.accumulate = accumulate;
    if (dt == NF4_BF16) return gt == NF4_BF16 ? gradient<Bf16, Bf16>(p, s) : gradient<Bf16, float>(p, s);
    return gt == NF4_BF16 ? gradient<float, Bf16>(p, s) : gradient<float, float>(p, s);
}

}  // namespace nf4
