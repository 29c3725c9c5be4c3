// muon.hip - the Muon step over a list of matrices and the orthogonalising alone, for
// gfx950. The formulas are in nf4.h (nf4_muon_step, nf4_orthogonalize).
//
// With X0 the update over its norm and S = X0^T X0 of the shorter side (s x s, s <=
// 256), every Newton-Schulz step multiplies X by the polynomial q(S_k) = a I + b S_k +
// c S_k^2 of its own Gram matrix S_k, and all of them commute: X_n = X0 P, P the product
// of the q(S_k), S_{k+1} = S_k q(S_k)^2. So the long matrices are read twice, once for
// S and once for the product with P, and the iteration runs on s x s matrices.
// What S has to hold: an eigenvalue far below the largest grows by a^2 = 11.9 a step, and
// so does its error, 2 10^4 times over the first four of five steps. S is therefore summed
// in fp32 over 32 rows and in fp64 beyond, and the s x s products run on the fp64 matrix
// instruction; the two passes over the long matrices split fp32 into bf16 parts.
#include <math.h>

#include <type_traits>

#include "training_internal.h"

namespace nf4 {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = 4;
constexpr int kSmall = 64;     // shorter sides up to here are iterated in one workgroup's LDS

// One matrix. `tall`: the longer side's index is the slow one (rows >= cols).
struct Item {
    const void *g;
    void *m;                 // NULL: no momentum
    void *w;                 // the weight, or the output
    float *master;
    int64_t length;          // of the longer side
    int64_t partial, mats;   // first element in the workspace's fp64 parts
    int32_t side;            // the shorter
    int32_t tall;
    float keep, step;        // w' = keep w - step O
    uint32_t gram_first, gram_chunk, gram_chunks, gram_pairs;
    uint32_t apply_first, apply_chunk;
    uint32_t p, pad;         // first element of P's parts, in units of 512
};
constexpr int kBatch = 34;
struct Batch {
    Item item[kBatch];
};
static_assert(sizeof(Batch) + 64 <= 4096, "kernel arguments");

struct List {
    const Item *item;
    const uint32_t *gram_first, *apply_first;
    int32_t count;
};
struct Scalars {
    float mu, one_mu;
    int32_t nesterov;
    double eps, a, b, c;
    int32_t iterations;
    bool step;               // the optimizer's step, or the orthogonalising alone
    bool w_bf16;
};
struct Space {
    double *partial, *mats, *norm;  // norm: of each matrix's update
    uint16_t *p;              // bf16 parts, see put_p
};

__global__ __launch_bounds__(kThreads) void muon_table_kernel(Batch b, int32_t count, Item *items, uint32_t *gram_first,
                                                              uint32_t *apply_first) {
    constexpr int kWords = sizeof(Item) / 4;
    const uint32_t *from = reinterpret_cast<const uint32_t *>(b.item);
    uint32_t *to = reinterpret_cast<uint32_t *>(items);
    for (int i = threadIdx.x; i < count * kWords; i += kThreads) to[i] = from[i];
    if ((int)threadIdx.x < count) {
        gram_first[threadIdx.x] = b.item[threadIdx.x].gram_first;
        apply_first[threadIdx.x] = b.item[threadIdx.x].apply_first;
    }
}

// The last entry whose first workgroup is not above `wg`: a wave's 64 questions at a time.
__device__ __forceinline__ int32_t find(const uint32_t *firsts, int32_t count, uint32_t wg) {
    int32_t n = 0;
    for (int32_t i = threadIdx.x % 64; i - (int32_t)(threadIdx.x % 64) < count; i += 64)
        n += __popcll(__ballot(i < count && firsts[i < count ? i : 0] <= wg));
    return __builtin_amdgcn_readfirstlane(n - 1);
}

// ---- elements of an update ----

struct None {};  // no momentum

// N consecutive elements (4 or 8) as they lie in memory, at any element's address. Of
// those, `live` (maybe none) are the matrix's; the others are zero.
template <typename T, int N> struct RawN;
template <> struct RawN<Bf16, 4> { u32x2 v; };
template <> struct RawN<float, 4> { f32x4 v; };
template <> struct RawN<Bf16, 8> { u32x4 v; };
template <> struct RawN<float, 8> { f32x4 v, w; };
template <int N> struct RawN<None, N> {};
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));

template <typename T, int N, bool kStream>
__device__ __forceinline__ RawN<T, N> load_n(const void *p, int64_t at, int live) {
    if constexpr (std::is_same_v<T, None>) return {};
    else {
        const T *q = static_cast<const T *>(p) + at;
        RawN<T, N> r{};
        if (live >= N) {
            if constexpr (sizeof(T) == 4) {
                const f32x4_at4 *f = reinterpret_cast<const f32x4_at4 *>(q);
                r.v = kStream ? __builtin_nontemporal_load(f) : *f;
                const f32x4_at4 *f1 = reinterpret_cast<const f32x4_at4 *>(q + 4);
                if constexpr (N == 8) r.w = kStream ? __builtin_nontemporal_load(f1) : *f1;
            } else if constexpr (N == 8) {
                const u32x4_at2 *f = reinterpret_cast<const u32x4_at2 *>(q);
                r.v = kStream ? __builtin_nontemporal_load(f) : *f;
            } else {
                const u32x2_at2 *f = reinterpret_cast<const u32x2_at2 *>(q);
                r.v = kStream ? __builtin_nontemporal_load(f) : *f;
            }
        } else if (live > 0) {
            float x[N];
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = j < live ? load1(q + j) : 0.0f;
            if constexpr (sizeof(T) == 4) {
                r.v = f32x4{x[0], x[1], x[2], x[3]};
                if constexpr (N == 8) r.w = f32x4{x[4], x[5], x[6], x[7]};
            } else {
#pragma unroll
                for (int j = 0; j < N / 2; ++j) r.v[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
            }
        }
        return r;
    }
}
template <int N>
__device__ __forceinline__ void values_n(const RawN<Bf16, N> &r, float *x) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) x[2 * j] = bf16_lo(r.v[j]), x[2 * j + 1] = bf16_hi(r.v[j]);
}
template <int N>
__device__ __forceinline__ void values_n(const RawN<float, N> &r, float *x) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = r.v[j];
    if constexpr (N == 8)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 + j] = r.w[j];
}
// Weights and momenta go past the caches: nothing here reads them again.
template <int N, typename T>
__device__ __forceinline__ void store_n(T *q, int live, const float *x) {
    if (live >= N) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < N; j += 4)
                __builtin_nontemporal_store(f32x4{x[j], x[j + 1], x[j + 2], x[j + 3]}, reinterpret_cast<f32x4_at4 *>(q + j));
        } else if constexpr (N == 8) {
            u32x4 r;
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
            __builtin_nontemporal_store(r, reinterpret_cast<u32x4_at2 *>(q));
        } else {
            __builtin_nontemporal_store(u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])},
                                        reinterpret_cast<u32x2_at2 *>(q));
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < live) store1(q + j, x[j]);
}

// Elements of the gradient and the momentum, as they lie in memory.
template <typename G, typename M, int N> struct Raw {
    RawN<G, N> g;
    RawN<M, N> m;
};
template <typename G, typename M, int N, bool kStream>
__device__ __forceinline__ Raw<G, M, N> load_update(const Item &e, int64_t at, int live) {
    return {load_n<G, N, kStream>(e.g, at, live), load_n<M, N, kStream>(e.m, at, live)};
}
// Their update, and the new momentum. Each is computed by the same operations in both
// passes, so both see the same bits.
template <typename G, typename M, int N>
__device__ __forceinline__ void update_of(const Raw<G, M, N> &r, const Scalars &c, float *u, float *m) {
    values_n<N>(r.g, u);
    if constexpr (!std::is_same_v<M, None>) {
        values_n<N>(r.m, m);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float g = c.one_mu * u[j];
            m[j] = fmaf(c.mu, m[j], g);
            u[j] = c.nesterov ? fmaf(c.mu, m[j], g) : m[j];
        }
    }
}

// ---- fp32 products on the bf16 matrix instruction ----
// An fp32 number is the sum of three bf16 numbers, the first two rounded, and products of
// bf16 are exact in the instruction's sums: with x = h + m + l the products hh, hm, mh,
// mm, hl, lh leave 2^-26 of |x| |y|. That is 6 instructions of 16 cycles for 32 rows of
// a 16 x 16 tile, 96 cycles; the fp32 instruction takes 8 of 32, 256 cycles. bf16 numbers
// (kParts 1) take one.
typedef short bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 bf16_operand;

template <int kParts> struct Operand {
    u32x4 part[kParts];
};
// Eight values: those of a lane's eight rows.
template <int kParts>
__device__ __forceinline__ Operand<kParts> operand_of(const float (&x)[8]) {
    Operand<kParts> r;
    float rest[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) rest[j] = x[j];
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = pack_bf16x2(rest[2 * j], rest[2 * j + 1]);
            r.part[p][j] = w;
            if (p + 1 < kParts) rest[2 * j] -= bf16_lo(w), rest[2 * j + 1] -= bf16_hi(w);
        }
    return r;
}
__device__ __forceinline__ f32x4 mfma_bf16(const u32x4 &a, const u32x4 &b, const f32x4 &c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16_operand, a), __builtin_bit_cast(bf16_operand, b), c, 0,
                                                   0, 0);
}
// c + a b over 32 rows, the small products first: their sum is rounded once with the large one.
template <int kParts>
__device__ __forceinline__ f32x4 mfma_f32(const Operand<kParts> &a, const Operand<kParts> &b, f32x4 c) {
#pragma unroll
    for (int sum = kParts - 1; sum > 0; --sum)
#pragma unroll
        for (int p = sum; p >= 0; --p) c = mfma_bf16(a.part[p], b.part[sum - p], c);
    return mfma_bf16(a.part[0], b.part[0], c);
}
template <typename G, typename M>
constexpr int kPartsOf = std::is_same_v<G, Bf16> && std::is_same_v<M, None> ? 1 : 3;

// ---- S: the Gram matrix ----

// A wave's share of S for the 16 NI columns from 64 bi on and the 16 NJ from 64 bj on, rows from
// `begin` to `end` of the longer side, 32 a step: a step's sums are rounded to fp32 once
// and added in fp64. In a tall matrix a lane loads NI consecutive columns of rows 4 r + k,
// so its column in operand i is NI n + i; in a wide one rows 8 k + r of column 16 i + n.
template <typename G, typename M, int NI, int NJ, bool kDiag>
__device__ __forceinline__ void gram_rows(const Item &e, const Scalars &c, int bi, int bj, int64_t begin, int64_t end,
                                          f64x4 *sums) {
    constexpr int kParts = kPartsOf<G, M>;
    constexpr int kTiles = kDiag ? NI * (NI + 1) / 2 : NI * NJ;
    const int lane = threadIdx.x % 64, n = lane % 16, k = lane / 16;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) sums[t] = f64x4{0.0, 0.0, 0.0, 0.0};
    auto load = [&](auto &ops, int block, int64_t row) {
        constexpr int N = sizeof(ops) / sizeof(ops[0]);
        if (e.tall) {
            const int col = 64 * block + N * n;
            const int64_t first = (row + k) * e.side + col, step = 4 * (int64_t)e.side;
            const int rows = (int)min(end - row - k, (int64_t)32);  // the lane's are every fourth of them
            float x[N][8];
            if constexpr (N == 4) {
                Raw<G, M, 4> raw[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) raw[r] = load_update<G, M, 4, false>(e, first + r * step, 4 * r < rows ? e.side - col : 0);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    float u[4], m[4];
                    update_of(raw[r], c, u, m);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j][r] = u[j];
                }
            } else {
                Raw<G, M, 4> raw[N][8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const int live = 4 * r < rows && col + j < e.side ? 1 : 0;
                        raw[j][r] = load_update<G, M, 4, false>(e, first + r * step + j, live);
                    }
#pragma unroll
                for (int r = 0; r < 8; ++r)
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        float u[4], m[4];
                        update_of(raw[j][r], c, u, m);
                        x[j][r] = u[0];
                    }
            }
#pragma unroll
            for (int j = 0; j < N; ++j) ops[j] = operand_of<kParts>(x[j]);
        } else {
            Raw<G, M, 8> raw[N];
            const int64_t l = row + 8 * k;
            const int rows = l < end ? (int)min(end - l, (int64_t)8) : 0;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int col = 64 * block + 16 * j + n;
                raw[j] = load_update<G, M, 8, false>(e, (int64_t)col * e.length + l, col < e.side ? rows : 0);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float u[8], m[8];
                update_of(raw[j], c, u, m);
                ops[j] = operand_of<kParts>(u);
            }
        }
    };
    for (int64_t row = begin; row < end; row += 32) {
        Operand<kParts> x[NI], y[kDiag ? 1 : NJ];
        load(x, bi, row);
        if constexpr (!kDiag) load(y, bj, row);
        int t = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = kDiag ? i : 0; j < NJ; ++j, ++t) {
                const f32x4 s = mfma_f32<kParts>(x[i], kDiag ? x[j] : y[j], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                for (int r = 0; r < 4; ++r) sums[t][r] += (double)s[r];
            }
    }
}

// Sums of the workgroup's waves, then out: [tile][register][lane].
template <typename G, typename M, int NI, int NJ, bool kDiag>
__device__ __forceinline__ void gram_part(const Item &e, const Scalars &c, int bi, int bj, int64_t begin, int64_t end,
                                          double *out, double (*part)[256]) {
    constexpr int kTiles = kDiag ? NI * (NI + 1) / 2 : NI * NJ;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t share = ((end - begin + kWaves - 1) / kWaves + 31) / 32 * 32;
    const int64_t b = min(begin + wave * share, end);
    f64x4 sums[kTiles];
    gram_rows<G, M, NI, NJ, kDiag>(e, c, bi, bj, b, min(b + share, end), sums);
    for (int v = 0; v < kWaves; ++v) {
        if (wave == v)
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    double &x = part[t][r * 64 + lane];
                    x = v == 0 ? sums[t][r] : x + sums[t][r];
                }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < kTiles * 256; i += kThreads) out[i] = part[i / 256][i % 256];
}

// Tiles of 256 sums that a workgroup leaves.
__host__ __device__ inline int gram_width(int side) { return side <= 16 ? 1 : side <= 32 ? 2 : 4; }
__host__ __device__ inline int gram_tiles(int side) {
    return side <= 16 ? 1 : side <= 32 ? 3 : side <= kSmall ? 10 : 16;
}
__device__ __forceinline__ void pair_of(int pair, int &bi, int &bj) {
    bj = 0;
    while ((bj + 1) * (bj + 2) / 2 <= pair) ++bj;
    bi = pair - bj * (bj + 1) / 2;
}

template <typename G, typename M, bool kLarge>
__global__ __launch_bounds__(kThreads, 2) void muon_gram_kernel(List list, Scalars c, Space ws) {
    __shared__ double part[kLarge ? 16 : 10][256];
    const uint32_t wg = blockIdx.x;
    const Item e = list.item[find(list.gram_first, list.count, wg)];
    if ((e.side > kSmall) != kLarge) return;
    const uint32_t own = wg - e.gram_first, chunk = own / e.gram_pairs, pair = own % e.gram_pairs;
    const int64_t begin = (int64_t)chunk * e.gram_chunk, end = min(begin + e.gram_chunk, e.length);
    double *out = ws.partial + e.partial + (int64_t)own * gram_tiles(e.side) * 256;
    if constexpr (kLarge) {
        int bi, bj;
        pair_of(pair, bi, bj);
        gram_part<G, M, 4, 4, false>(e, c, bi, bj, begin, end, out, part);
    } else {
        if (e.side <= 16) gram_part<G, M, 1, 1, true>(e, c, 0, 0, begin, end, out, part);
        else if (e.side <= 32) gram_part<G, M, 2, 2, true>(e, c, 0, 0, begin, end, out, part);
        else gram_part<G, M, 4, 4, true>(e, c, 0, 0, begin, end, out, part);
    }
}

// Where sum i of a pair of blocks lies in it; false for the half of a tile on the diagonal
// that its other half has too (rounded otherwise: one of the two is taken).
__device__ __forceinline__ bool place_of(const Item &e, int width, bool diag, int i, int &row, int &col) {
    int t = i / 256;
    const int reg = i / 64 % 4, lane = i % 64;
    int ti, tj;
    if (diag) {
        ti = 0;
        while (t >= width - ti) t -= width - ti, ++ti;
        tj = ti + t;
    } else {
        ti = t / width, tj = t % width;
    }
    const int r = 4 * (lane / 16) + reg, n = lane % 16;
    row = e.tall ? width * r + ti : 16 * ti + r;
    col = e.tall ? width * n + tj : 16 * tj + n;
    return ti != tj || r <= n;
}

// The sum of `count` partial sums, `stride` apart, in their order, eight loads in flight.
__device__ __forceinline__ double chunk_total(const double *from, int64_t stride, uint32_t count) {
    double x = 0.0;
    uint32_t k = 0;
    for (; k + 8 <= count; k += 8) {
        double y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = from[(k + j) * stride];
#pragma unroll
        for (int j = 0; j < 8; ++j) x += y[j];
    }
    for (; k < count; ++k) x += from[k * stride];
    return x;
}

__device__ __forceinline__ double block_total(double x, double *part) {
#pragma unroll
    for (int o = 32; o > 0; o /= 2) x += __shfl_xor(x, o, 64);
    const int waves = blockDim.x / 64;
    __syncthreads();
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = x;
    __syncthreads();
    x = 0.0;
    for (int v = 0; v < waves; ++v) x += part[v];
    return x;
}

// P as the product with U reads it: its element (row, col) in three bf16 parts. Lane
// 16 k + n of an operand holds eight columns of a row of P: columns 32 s + 8 k .. + 7 of
// operand s, and rows so permuted that lane (k, n) of the product finds those same
// columns of O in two operands' results: row 4 k + r of result i is row
// 32 (i / 2) + 8 k + 4 (i % 2) + r of P.
__host__ __device__ inline int p_blocks(int side) { return (side + 31) / 32; }  // operands of 32 columns
__host__ __device__ inline int64_t p_elements(int side) { return 3 * 2 * (int64_t)p_blocks(side) * p_blocks(side) * 512; }
__device__ __forceinline__ void put_p(uint16_t *p, int blocks, int row, int col, float x) {
    const int i = 2 * (row / 32) + row % 8 / 4, n = 4 * (row % 32 / 8) + row % 4;
    const int at = ((i * blocks + col / 32) * 64 + col % 32 / 8 * 16 + n) * 8 + col % 8;
#pragma unroll
    for (int part = 0; part < 3; ++part) {
        const uint32_t w = pack_bf16x2(x, 0.0f);
        p[(int64_t)part * 2 * blocks * blocks * 512 + at] = (uint16_t)w;
        x -= bf16_lo(w);
    }
}

// ---- the iteration, shorter sides up to 64: one workgroup a matrix ----

constexpr int kStride = kSmall + 2;  // doubles: 16 rows of two columns lie in different banks
typedef double SmallMat[kSmall][kStride];
constexpr int kSmallThreads = 1024;

// A wave takes tiles of the upper triangle (all matrices are symmetric) and writes
// both halves.
__global__ __launch_bounds__(kSmallThreads) void muon_small_kernel(List list, Scalars c, Space ws) {
    extern __shared__ double smem[];
    SmallMat &A = *reinterpret_cast<SmallMat *>(smem), &Q = (&A)[1], &P = (&A)[2];
    double *part = smem + 3 * kSmall * kStride;
    const Item e = list.item[blockIdx.x];
    if (e.side > kSmall) return;
    const int threads = blockDim.x, waves = threads / 64;
    const int tiles = gram_tiles(e.side), width = gram_width(e.side), edge = (e.side + 15) / 16;
    const double *from = ws.partial + e.partial;
    for (int i = threadIdx.x; i < tiles * 256; i += threads) {
        const double x = chunk_total(from + i, (int64_t)tiles * 256, e.gram_chunks);
        int row, col;
        if (place_of(e, width, true, i, row, col)) A[row][col] = x, A[col][row] = x;
    }
    __syncthreads();
    const double trace = block_total((int)threadIdx.x < e.side ? A[threadIdx.x][threadIdx.x] : 0.0, part);
    const double norm = sqrt(trace), inv = 1.0 / fmax(norm, c.eps);
    for (int i = threadIdx.x; i < 16 * edge * 16 * edge; i += threads) A[i / (16 * edge)][i % (16 * edge)] *= inv * inv;
    const int lane = threadIdx.x % 64, n = lane % 16, k4 = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int count = edge * (edge + 1) / 2;
    auto tile_of = [&](int t, int &ti, int &tj) { pair_of(t, ti, tj); };
    auto product = [&](const SmallMat &x, const SmallMat &y, int t) {
        int ti, tj;
        tile_of(t, ti, tj);
        f64x4 r = {0.0, 0.0, 0.0, 0.0};
        for (int k = 0; k < 16 * edge; k += 16)
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                r = __builtin_amdgcn_mfma_f64_16x16x4f64(x[16 * ti + n][k + j + k4], y[16 * tj + n][k + j + k4], r, 0, 0, 0);
        return r;
    };
    auto put = [&](SmallMat &x, const f64x4 &r, int t) {
        int ti, tj;
        tile_of(t, ti, tj);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 16 * ti + 4 * j + k4, col = 16 * tj + n;
            x[row][col] = r[j];
            if (ti != tj) x[col][row] = r[j];
        }
    };
    for (int it = 0; it < c.iterations; ++it) {
        const bool last = it + 1 == c.iterations;
        __syncthreads();
        for (int t = wave; t < count; t += waves) {
            f64x4 q = product(A, A, t);
            int ti, tj;
            tile_of(t, ti, tj);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = 16 * ti + 4 * j + k4, col = 16 * tj + n;
                q[j] = c.c * q[j] + c.b * A[row][col] + (row == col ? c.a : 0.0);
            }
            if (it == 0) put(P, q, t);
            put(Q, q, t);
        }
        __syncthreads();
        // A Q and P Q: at most two tiles a wave, held until all of them have been read
        f64x4 held[2];
        const int from_p = last ? 0 : count, all = from_p + (it > 0 ? count : 0);
        int mine = 0;
        for (int t = wave; t < all; t += waves, ++mine) {
            const f64x4 r = t < from_p ? product(A, Q, t) : product(P, Q, t - from_p);
            if (mine == 0) held[0] = r;
            else held[1] = r;
        }
        __syncthreads();
        mine = 0;
        for (int t = wave; t < all; t += waves, ++mine) {
            const f64x4 r = mine == 0 ? held[0] : held[1];
            if (t < from_p) put(A, r, t);
            else put(P, r, t - from_p);
        }
        if (last) break;
        __syncthreads();
        mine = 0;
        for (int t = wave; t < count; t += waves, ++mine) {
            const f64x4 r = product(A, Q, t);
            if (mine == 0) held[0] = r;
            else held[1] = r;
        }
        __syncthreads();
        mine = 0;
        for (int t = wave; t < count; t += waves, ++mine) put(A, mine == 0 ? held[0] : held[1], t);
    }
    __syncthreads();
    const int blocks = p_blocks(e.side), full = 32 * blocks;
    uint16_t *out = ws.p + (int64_t)e.p * 512;
    for (int i = threadIdx.x; i < full * full; i += threads) {
        const int row = i / full, col = i % full;
        put_p(out, blocks, row, col, row < e.side && col < e.side ? (float)(P[row][col] * inv) : 0.0f);
    }
    if (threadIdx.x == 0) ws.norm[blockIdx.x] = norm;
}

// ---- the iteration, shorter sides above 64: a launch a product ----

__host__ __device__ inline int blocks_of(int side) { return (side + 63) / 64; }
enum Mat { kA, kQ, kT, kP0, kP1, kMats };

__device__ __forceinline__ double *mat_of(const Item &e, const Space &ws, int which) {
    const int64_t edge = 64 * blocks_of(e.side);
    return ws.mats + e.mats + which * edge * edge;
}

// 64 x 64 sums of a pair of blocks are added up by kStartParts workgroups.
constexpr int kStartParts = 4;
__global__ __launch_bounds__(kThreads) void muon_start_kernel(List list, Scalars c, Space ws) {
    __shared__ double part[kWaves];
    const Item e = list.item[blockIdx.x];
    if (e.side <= kSmall || blockIdx.y >= e.gram_pairs) return;
    const double *from = ws.partial + e.partial;
    const int64_t stride = (int64_t)e.gram_pairs * 16 * 256;
    const int edge = 64 * blocks_of(e.side);
    // the trace, by every workgroup: thread s takes element (s, s), in the pair of its block with itself
    double x = 0.0;
    if ((int)threadIdx.x < e.side) {
        const int b = threadIdx.x / 64, d = threadIdx.x % 64, pair = b * (b + 1) / 2 + b;
        // its tile, row and column: (4 r + i) in a tall matrix, (16 i + r) in a wide one
        const int i = e.tall ? d % 4 : d / 16, r = e.tall ? d / 4 : d % 16;
        x = chunk_total(from + ((pair * 16) + i * 4 + i) * 256 + (r % 4) * 64 + (r / 4) * 16 + r, stride, e.gram_chunks);
    }
    const double trace = block_total(x, part);
    const double norm = sqrt(trace), inv = 1.0 / fmax(norm, c.eps);
    int bi, bj;
    pair_of(blockIdx.y, bi, bj);
    double *A = mat_of(e, ws, kA);
    constexpr int kEach = 16 * 256 / kStartParts;
    for (int i = blockIdx.z * kEach + threadIdx.x; i < ((int)blockIdx.z + 1) * kEach; i += kThreads) {
        const double sum = chunk_total(from + (int64_t)blockIdx.y * 16 * 256 + i, stride, e.gram_chunks) * inv * inv;
        int row, col;
        place_of(e, 4, false, i, row, col);
        row += 64 * bi, col += 64 * bj;
        // a block with itself holds both of each pair: the upper one is taken
        if (bi != bj || row <= col) A[(int64_t)row * edge + col] = sum, A[(int64_t)col * edge + row] = sum;
    }
    if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) ws.norm[blockIdx.x] = norm;
}

// out = x y, with q: c out + b x + a I (x = y), which also goes to `copy`; with fin: over
// the norm, in parts, to P. blockIdx.z chooses one of two products. All matrices are
// polynomials of one, so x y is symmetric: a workgroup takes 32 x 32 of the upper
// triangle, writes both halves, and reads a column of y as its row.
struct Product {
    int32_t x, y, out, copy;  // copy: -1 none
    bool q, fin;
};
struct Products {
    Product of[2];
};
constexpr int kEdge = 32, kSlab = 64;

__global__ __launch_bounds__(kThreads) void muon_product_kernel(List list, Scalars c, Space ws, Products products) {
    __shared__ double xs[kEdge][kSlab + 2], ys[kEdge][kSlab + 2];
    const Item e = list.item[blockIdx.x];
    const int edge = 64 * blocks_of(e.side), nb = edge / kEdge;
    if (e.side <= kSmall || (int)blockIdx.y >= nb * (nb + 1) / 2) return;
    const Product d = products.of[blockIdx.z];
    int bi, bj;
    pair_of(blockIdx.y, bi, bj);
    const double *x = mat_of(e, ws, d.x) + (int64_t)bi * kEdge * edge, *y = mat_of(e, ws, d.y) + (int64_t)bj * kEdge * edge;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, n = lane % 16, k4 = lane / 16;
    const int ti = wave / 2, tj = wave % 2;
    constexpr int kEach = kEdge * kSlab / 2 / kThreads;  // pairs of doubles of a thread and slab
    typedef double f64x2 __attribute__((ext_vector_type(2)));
    f64x2 rx[kEach], ry[kEach];
    auto load = [&](int k0) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = j * kThreads + threadIdx.x, row = i / (kSlab / 2), col = i % (kSlab / 2) * 2;
            rx[j] = *reinterpret_cast<const f64x2 *>(x + (int64_t)row * edge + k0 + col);
            ry[j] = *reinterpret_cast<const f64x2 *>(y + (int64_t)row * edge + k0 + col);
        }
    };
    load(0);
    f64x4 acc[2] = {{0.0, 0.0, 0.0, 0.0}, {0.0, 0.0, 0.0, 0.0}};
    for (int k0 = 0; k0 < edge; k0 += kSlab) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = j * kThreads + threadIdx.x, row = i / (kSlab / 2), col = i % (kSlab / 2) * 2;
            xs[row][col] = rx[j][0], xs[row][col + 1] = rx[j][1];
            ys[row][col] = ry[j][0], ys[row][col + 1] = ry[j][1];
        }
        __syncthreads();
        if (k0 + kSlab < edge) load(k0 + kSlab);
#pragma unroll
        for (int k = 0; k < kSlab; k += 8)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[j] = __builtin_amdgcn_mfma_f64_16x16x4f64(xs[16 * ti + n][k + 4 * j + k4], ys[16 * tj + n][k + 4 * j + k4],
                                                              acc[j], 0, 0, 0);
    }
    const double inv = 1.0 / fmax(ws.norm[blockIdx.x], c.eps);
    double *out = mat_of(e, ws, d.out), *copy = d.copy >= 0 ? mat_of(e, ws, d.copy) : nullptr;
    const double *whole = mat_of(e, ws, d.x);
    const int blocks = p_blocks(e.side);
    uint16_t *p = ws.p + (int64_t)e.p * 512;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = kEdge * bi + 16 * ti + 4 * r + k4, col = kEdge * bj + 16 * tj + n;
        const int64_t at = (int64_t)row * edge + col, mirror = (int64_t)col * edge + row;
        double v = acc[0][r] + acc[1][r];
        if (d.q) v = c.c * v + c.b * whole[at] + (row == col ? c.a : 0.0);
        if (d.fin) {
            if (row >= 32 * blocks || col >= 32 * blocks) continue;
            const float f = row < e.side && col < e.side ? (float)(v * inv) : 0.0f;
            put_p(p, blocks, row, col, f);
            if (bi != bj) put_p(p, blocks, col, row, f);
        } else {
            out[at] = v;
            if (bi != bj) out[mirror] = v;
            if (copy) copy[at] = v;
            if (copy && bi != bj) copy[mirror] = v;
        }
    }
}

// ---- O = U P and the step ----

// N consecutive weights before the step.
template <int N> struct Weight {
    RawN<Bf16, N> half;
    RawN<float, N> full;
};
template <int N>
__device__ __forceinline__ Weight<N> load_weight(const Item &e, const Scalars &c, int64_t at, int live) {
    Weight<N> r{};
    if (!c.step) return r;
    if (e.master) r.full = load_n<float, N, true>(e.master, at, live);
    else if (c.w_bf16) r.half = load_n<Bf16, N, true>(e.w, at, live);
    else r.full = load_n<float, N, true>(e.w, at, live);
    return r;
}
// Their step, or the output alone.
template <int N>
__device__ __forceinline__ void finish(const Item &e, const Scalars &c, const Weight<N> &before, int64_t at, int live, float *o) {
    if (c.step) {
        float w[N];
        if (!e.master && c.w_bf16) values_n<N>(before.half, w);
        else values_n<N>(before.full, w);
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = fmaf(-e.step, o[j], e.keep * w[j]);
        if (e.master) store_n<N>(e.master + at, live, o);
    }
    if (c.w_bf16) store_n<N>(static_cast<Bf16 *>(e.w) + at, live, o);
    else store_n<N>(static_cast<float *>(e.w) + at, live, o);
}
template <typename M, int N>
__device__ __forceinline__ void store_momentum(const Item &e, int64_t at, int live, const float *m) {
    if constexpr (!std::is_same_v<M, None>) store_n<N>(static_cast<M *>(e.m) + at, live, m);
}

// A part of P, `blocks` operands wide: result i, operand s.
__device__ __forceinline__ u32x4 p_part(const u32x4 *p, int blocks, int part, int i, int s) {
    return p[((part * 2 * blocks + i) * blocks + s) * 64 + threadIdx.x % 64];
}
// acc[i] += P's rows of result i times u, one operand s of 32 columns: six products of
// parts, or three where u is one part.
template <int kParts>
__device__ __forceinline__ Operand<3> p_operand(const u32x4 *p, int blocks, int i, int s) {
    Operand<3> r;
#pragma unroll
    for (int part = 0; part < 3; ++part) r.part[part] = p_part(p, blocks, part, i, s);
    return r;
}
template <int kParts>
__device__ __forceinline__ f32x4 mfma_p(const Operand<3> &p, const Operand<kParts> &u, f32x4 c) {
    if constexpr (kParts == 3) return mfma_f32<3>(p, u, c);
    else {
#pragma unroll
        for (int part = 2; part >= 0; --part) c = mfma_bf16(p.part[part], u.part[0], c);
        return c;
    }
}

// A matrix of up to 64 on its shorter side, P in LDS. In a tall matrix a wave takes 16
// rows, a lane columns 32 s + 8 k .. + 7 of row n, of U and of O; in a wide one 64 columns, a
// lane four of them (4 n .. + 3) in rows 32 s + 8 k .. + 7.
template <typename G, typename M, int kBlocks>
__device__ __forceinline__ void apply_small(const Item &e, const Scalars &c, const u32x4 *p, int64_t begin, int64_t end) {
    constexpr int kParts = kPartsOf<G, M>;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, n = lane % 16, k = lane / 16;
    if (e.tall) {
        for (int64_t row = begin + wave * 16; row < end; row += 16 * kWaves) {
            const int64_t l = row + n, at = l * e.side + 8 * k;
            const int live = l < end ? e.side - 8 * k : 0;
            Raw<G, M, 8> raw[kBlocks];
            Weight<8> before[kBlocks];
#pragma unroll
            for (int s = 0; s < kBlocks; ++s) raw[s] = load_update<G, M, 8, true>(e, at + 32 * s, live - 32 * s);
#pragma unroll
            for (int s = 0; s < kBlocks; ++s) before[s] = load_weight<8>(e, c, at + 32 * s, live - 32 * s);
            Operand<kParts> u[kBlocks];
#pragma unroll
            for (int s = 0; s < kBlocks; ++s) {
                float x[8], m[8];
                update_of(raw[s], c, x, m);
                store_momentum<M, 8>(e, at + 32 * s, live - 32 * s, m);
                u[s] = operand_of<kParts>(x);
            }
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                float o[8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < kBlocks; ++s) acc = mfma_p<kParts>(p_operand<kParts>(p, kBlocks, 2 * b + h, s), u[s], acc);
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[4 * h + r] = acc[r];
                }
                finish<8>(e, c, before[b], at + 32 * b, live - 32 * b, o);
            }
        }
    } else {
        for (int64_t col = begin + wave * 64; col < end; col += 64 * kWaves) {
            const int64_t l = col + 4 * n;
            const int live = l < end ? (int)min(end - l, (int64_t)4) : 0;
            f32x4 acc[2 * kBlocks][4];
#pragma unroll
            for (int i = 0; i < 2 * kBlocks; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < kBlocks; ++s) {
                Raw<G, M, 4> raw[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const int row = 32 * s + 8 * k + r;
                    raw[r] = load_update<G, M, 4, true>(e, (int64_t)row * e.length + l, row < e.side ? live : 0);
                }
                float x[4][8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const int row = 32 * s + 8 * k + r;
                    float u[4], m[4];
                    update_of(raw[r], c, u, m);
                    store_momentum<M, 4>(e, (int64_t)row * e.length + l, row < e.side ? live : 0, m);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j][r] = u[j];
                }
                Operand<kParts> u[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) u[j] = operand_of<kParts>(x[j]);
#pragma unroll
                for (int i = 0; i < 2 * kBlocks; ++i) {
                    const Operand<3> a = p_operand<kParts>(p, kBlocks, i, s);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = mfma_p<kParts>(a, u[j], acc[i][j]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2 * kBlocks; ++i) {
                Weight<4> before[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 32 * (i / 2) + 8 * k + 4 * (i % 2) + r;
                    before[r] = load_weight<4>(e, c, (int64_t)row * e.length + l, row < e.side ? live : 0);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 32 * (i / 2) + 8 * k + 4 * (i % 2) + r;
                    float o[4] = {acc[i][0][r], acc[i][1][r], acc[i][2][r], acc[i][3][r]};
                    finish<4>(e, c, before[r], (int64_t)row * e.length + l, row < e.side ? live : 0, o);
                }
            }
        }
    }
}

template <typename G, typename M>
__global__ __launch_bounds__(kThreads, 2) void muon_apply_kernel(List list, Scalars c, Space ws) {
    __shared__ u32x4 sp[3 * 2 * 2 * 2 * 64];
    const uint32_t wg = gridDim.x - 1 - blockIdx.x;  // the first pass's last reads may still be cached
    const int32_t index = find(list.apply_first, list.count, wg);
    const Item e = list.item[index];
    if (e.side > kSmall || (c.step && !isfinite(ws.norm[index]))) return;
    const int64_t begin = (int64_t)(wg - e.apply_first) * e.apply_chunk;
    const int64_t end = min(begin + e.apply_chunk, e.length);
    const u32x4 *p = reinterpret_cast<const u32x4 *>(ws.p + (int64_t)e.p * 512);
    for (int i = threadIdx.x; i < p_elements(e.side) / 8; i += kThreads) sp[i] = p[i];
    __syncthreads();
    if (e.side <= 32) apply_small<G, M, 1>(e, c, sp, begin, end);
    else apply_small<G, M, 2>(e, c, sp, begin, end);
}

// A matrix of up to 256 on its shorter side, 64 places of the longer at a time: the
// parts of U in LDS, read whole before anything is written; P from the caches; a wave
// takes pairs of results, eight columns of O a lane as above. Place of lane n in
// operand j: 16 j + n in a tall matrix, 4 n + j in a wide one.
constexpr int kLargeThreads = 512, kLargeWaves = kLargeThreads / 64;

template <typename G, typename M>
__global__ __launch_bounds__(kLargeThreads) void muon_apply_large_kernel(List list, Scalars c, Space ws) {
    extern __shared__ u32x4 us[];  // [part][place's operand j][operand s][lane]
    constexpr int kParts = kPartsOf<G, M>;
    const uint32_t wg = gridDim.x - 1 - blockIdx.x;
    const int32_t index = find(list.apply_first, list.count, wg);
    const Item e = list.item[index];
    if (e.side <= kSmall || (c.step && !isfinite(ws.norm[index]))) return;
    const int64_t begin = (int64_t)(wg - e.apply_first) * e.apply_chunk;
    const int64_t end = min(begin + e.apply_chunk, e.length);
    const u32x4 *p = reinterpret_cast<const u32x4 *>(ws.p + (int64_t)e.p * 512);
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, n = lane % 16, k = lane / 16;
    const int blocks = p_blocks(e.side);
    auto place = [&](int part, int j, int s) { return us + ((part * 4 + j) * blocks + s) * 64; };
    for (int64_t l0 = begin; l0 < end; l0 += 64) {
        const int rows = (int)min(end - l0, (int64_t)64);
        __syncthreads();
        if (e.tall) {
            for (int i = threadIdx.x; i < 64 * 4 * blocks; i += kLargeThreads) {
                const int row = i / (4 * blocks), col = i % (4 * blocks) * 8, live = row < rows ? e.side - col : 0;
                const int64_t at = (l0 + row) * e.side + col;
                float x[8], m[8];
                update_of(load_update<G, M, 8, true>(e, at, live), c, x, m);
                store_momentum<M, 8>(e, at, live, m);
                const Operand<kParts> u = operand_of<kParts>(x);
#pragma unroll
                for (int part = 0; part < kParts; ++part)
                    place(part, row / 16, col / 32)[col % 32 / 8 * 16 + row % 16] = u.part[part];
            }
        } else {
            for (int i = threadIdx.x; i < 16 * 4 * blocks; i += kLargeThreads) {
                const int first = i / 16 * 8, four = i % 16;
                const int64_t l = l0 + 4 * four;
                const int live = max(rows - 4 * four, 0);
                Raw<G, M, 4> raw[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    raw[r] = load_update<G, M, 4, true>(e, (int64_t)(first + r) * e.length + l, first + r < e.side ? live : 0);
                float x[4][8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    float u[4], m[4];
                    update_of(raw[r], c, u, m);
                    store_momentum<M, 4>(e, (int64_t)(first + r) * e.length + l, first + r < e.side ? live : 0, m);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j][r] = u[j];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Operand<kParts> u = operand_of<kParts>(x[j]);
#pragma unroll
                    for (int part = 0; part < kParts; ++part)
                        place(part, j, first / 32)[first % 32 / 8 * 16 + four] = u.part[part];
                }
            }
        }
        __syncthreads();
        for (int b = wave; b < blocks; b += kLargeWaves) {
            f32x4 acc[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[h][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            for (int s = 0; s < blocks; ++s) {
                const Operand<3> a[2] = {p_operand<kParts>(p, blocks, 2 * b, s), p_operand<kParts>(p, blocks, 2 * b + 1, s)};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    Operand<kParts> u;
#pragma unroll
                    for (int part = 0; part < kParts; ++part) u.part[part] = place(part, j, s)[lane];
#pragma unroll
                    for (int h = 0; h < 2; ++h) acc[h][j] = mfma_p<kParts>(a[h], u, acc[h][j]);
                }
            }
            const int first = 32 * b + 8 * k;
            if (e.tall) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = 16 * j + n, live = row < rows ? e.side - first : 0;
                    const int64_t at = (l0 + row) * e.side + first;
                    const Weight<8> before = load_weight<8>(e, c, at, live);
                    float o[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) o[r] = acc[r / 4][j][r % 4];
                    finish<8>(e, c, before, at, live, o);
                }
            } else {
                const int64_t l = l0 + 4 * n;
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const int live = first + r < e.side ? rows - 4 * n : 0;
                    const int64_t at = (int64_t)(first + r) * e.length + l;
                    const Weight<4> before = load_weight<4>(e, c, at, live);
                    float o[4] = {acc[r / 4][0][r % 4], acc[r / 4][1][r % 4], acc[r / 4][2][r % 4], acc[r / 4][3][r % 4]};
                    finish<4>(e, c, before, at, live, o);
                }
            }
        }
    }
}

// ---- host ----

size_t round_up(size_t x, size_t to) { return (x + to - 1) / to * to; }

// How a list is cut, and what lies where in the workspace. The longer sides are cut into
// about 2048 shares of each pass, so that the chip is full and few partial sums are left.
struct Plan {
    size_t items, gram_first, apply_first, norm, partial, mats, p, bytes;  // offsets
    uint32_t gram_wgs, apply_wgs;
    int32_t count, largest, smallest;  // matrices with elements; their largest and smallest shorter side
    bool fits;
};
constexpr int64_t kShares = 2048;

template <typename F>
Plan make_plan(const MuonMatrix *list, int32_t count, F &&each) {
    Plan p{};
    int64_t gram_rows = 0, apply_rows = 0;
    for (int32_t i = 0; i < count; ++i) {
        const int64_t side = list[i].rows < list[i].cols ? list[i].rows : list[i].cols;
        const int64_t length = list[i].rows < list[i].cols ? list[i].cols : list[i].rows;
        if (side == 0) continue;
        ++p.count;
        const int nb = blocks_of((int)side);
        gram_rows += length * (nb * (nb + 1) / 2);
        apply_rows += length;
        if (side > p.largest) p.largest = (int32_t)side;
        if (p.smallest == 0 || side < p.smallest) p.smallest = (int32_t)side;
    }
    // 64 rows a wave at least: the fp32 sums' length
    const int64_t gram_chunk = round_up(gram_rows / kShares < 128 ? 128 : gram_rows / kShares, 64);
    const int64_t apply_chunk = round_up(apply_rows / kShares < 64 ? 64 : apply_rows / kShares, 64);
    p.items = 0;
    p.gram_first = round_up(p.items + (size_t)p.count * sizeof(Item), 16);
    p.apply_first = round_up(p.gram_first + (size_t)p.count * 4, 16);
    p.norm = round_up(p.apply_first + (size_t)p.count * 4, 256);
    p.partial = round_up(p.norm + (size_t)p.count * 8, 256);
    int64_t partial = 0, mats = 0, wgs = 0, apply_wgs = 0, ps = 0;
    for (int32_t i = 0; i < count; ++i) {
        const MuonMatrix &x = list[i];
        Item e{};
        e.tall = x.rows >= x.cols;
        e.side = (int32_t)(e.tall ? x.cols : x.rows), e.length = e.tall ? x.rows : x.cols;
        if (e.side == 0) continue;
        const int nb = blocks_of(e.side);
        const int64_t edge = 64 * nb;
        e.gram_pairs = nb * (nb + 1) / 2;
        e.gram_chunk = (uint32_t)gram_chunk, e.gram_chunks = (uint32_t)((e.length + gram_chunk - 1) / gram_chunk);
        e.apply_chunk = (uint32_t)apply_chunk;
        e.gram_first = (uint32_t)wgs, e.apply_first = (uint32_t)apply_wgs;
        e.partial = partial, e.mats = mats, e.p = (uint32_t)ps;
        wgs += (int64_t)e.gram_chunks * e.gram_pairs;
        apply_wgs += (e.length + apply_chunk - 1) / apply_chunk;
        partial += (int64_t)e.gram_chunks * e.gram_pairs * gram_tiles(e.side) * 256;
        if (e.side > kSmall) mats += kMats * edge * edge;
        ps += p_elements(e.side) / 512;
        each(i, e);
    }
    p.mats = round_up(p.partial + (size_t)partial * 8, 256);
    p.p = round_up(p.mats + (size_t)mats * 8, 256);
    p.bytes = p.p + (size_t)ps * 1024;
    p.gram_wgs = (uint32_t)wgs, p.apply_wgs = (uint32_t)apply_wgs;
    // a grid holds 2^32 threads at most
    p.fits = wgs < (1 << 23) && apply_wgs < (1 << 23) && ps < (int64_t(1) << 32);
    return p;
}

// Dynamic LDS of more than 64 KB is asked for.
hipError_t allow_lds(const void *kernel, size_t bytes) {
    return bytes <= 65536 ? hipSuccess
                          : hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename G, typename M>
hipError_t run(const Plan &p, const List &list, const Scalars &c, const Space &ws, hipStream_t s) {
    hipError_t r = hipSuccess;
    auto note = [&] {
        const hipError_t x = hipGetLastError();
        if (r == hipSuccess) r = x;
        return r == hipSuccess;
    };
    const bool small = p.smallest <= kSmall, large = p.largest > kSmall;
    if (small) {
        muon_gram_kernel<G, M, false><<<dim3(p.gram_wgs), dim3(kThreads), 0, s>>>(list, c, ws);
        if (!note()) return r;
        constexpr size_t kSmallLds = (3 * kSmall * kStride + 16) * sizeof(double);
        if ((r = allow_lds(reinterpret_cast<const void *>(&muon_small_kernel), kSmallLds)) != hipSuccess) return r;
        // a tile a wave, up to ten; the few of short sides leave waves to add up the partial sums
        const int threads = p.largest <= 32 ? 256 : p.largest <= 48 ? 512 : kSmallThreads;
        muon_small_kernel<<<dim3(p.count), dim3(threads), kSmallLds, s>>>(list, c, ws);
        if (!note()) return r;
    }
    if (large) {
        muon_gram_kernel<G, M, true><<<dim3(p.gram_wgs), dim3(kThreads), 0, s>>>(list, c, ws);
        if (!note()) return r;
        const int nb = blocks_of(p.largest), pairs = 2 * nb * (2 * nb + 1) / 2;
        muon_start_kernel<<<dim3(p.count, nb * (nb + 1) / 2, kStartParts), dim3(kThreads), 0, s>>>(list, c, ws);
        if (!note()) return r;
        auto launch = [&](const Products &x, int z) {
            if (r != hipSuccess) return;
            muon_product_kernel<<<dim3(p.count, pairs, z), dim3(kThreads), 0, s>>>(list, c, ws, x);
            note();
        };
        int now = kP0;
        for (int it = 0; it < c.iterations; ++it) {
            const bool last = it + 1 == c.iterations;
            const int next = now == kP0 ? kP1 : kP0;
            launch({{{kA, kA, kQ, it == 0 ? now : -1, true, last && it == 0}, {}}}, 1);
            const Product step{kA, kQ, kT, -1, false, false}, grow{now, kQ, next, -1, false, last};
            if (it > 0 && last) launch({{grow, {}}}, 1);
            else if (it > 0) launch({{step, grow}}, 2);
            else if (!last) launch({{step, {}}}, 1);
            if (it > 0) now = next;
            if (!last) launch({{{kT, kQ, kA, -1, false, false}, {}}}, 1);
        }
        if (r != hipSuccess) return r;
    }
    if (small) {
        muon_apply_kernel<G, M><<<dim3(p.apply_wgs), dim3(kThreads), 0, s>>>(list, c, ws);
        if (!note()) return r;
    }
    if (large) {
        const size_t lds = (size_t)kPartsOf<G, M> * 4 * p_blocks(p.largest) * 1024;
        if ((r = allow_lds(reinterpret_cast<const void *>(&muon_apply_large_kernel<G, M>), lds)) != hipSuccess) return r;
        muon_apply_large_kernel<G, M><<<dim3(p.apply_wgs), dim3(kLargeThreads), lds, s>>>(list, c, ws);
        note();
    }
    return r;
}

}  // namespace

size_t muon_workspace(const MuonMatrix *list, int32_t count) {
    const Plan p = make_plan(list, count, [](int32_t, const Item &) {});
    return p.fits ? p.bytes : (size_t)-1;
}

hipError_t launch_muon(const MuonMatrix *list, int32_t count, const MuonCall &call, void *workspace, hipStream_t s) {
    // the table first, a batch a launch; offsets and sizes follow from the list alone
    const Plan sizes = make_plan(list, count, [](int32_t, const Item &) {});
    if (sizes.count == 0) return hipSuccess;
    char *base = static_cast<char *>(workspace);
    Item *items = reinterpret_cast<Item *>(base + sizes.items);
    uint32_t *gram_first = reinterpret_cast<uint32_t *>(base + sizes.gram_first);
    uint32_t *apply_first = reinterpret_cast<uint32_t *>(base + sizes.apply_first);
    Batch b{};
    int used = 0;
    int32_t done = 0;
    hipError_t err = hipSuccess;
    auto flush = [&] {
        if (used == 0 || err != hipSuccess) return;
        muon_table_kernel<<<dim3(1), dim3(kThreads), 0, s>>>(b, used, items + done, gram_first + done, apply_first + done);
        err = hipGetLastError();
        done += used, used = 0;
    };
    make_plan(list, count, [&](int32_t i, const Item &e) {
        if (used == kBatch) flush();
        Item &t = b.item[used++];
        t = e;
        const MuonMatrix &x = list[i];
        t.g = x.grad, t.m = x.m, t.w = x.w, t.master = x.master;
        t.keep = (float)(1.0 - (double)x.lr * (double)x.weight_decay);
        t.step = (float)((double)x.lr * (double)x.scale);
    });
    flush();
    if (err != hipSuccess) return err;
    Scalars c{};
    c.mu = (float)call.momentum, c.one_mu = (float)(1.0 - call.momentum), c.nesterov = call.nesterov;
    c.eps = call.eps, c.a = call.a, c.b = call.b, c.c = call.c, c.iterations = call.iterations;
    c.step = call.step, c.w_bf16 = call.w == NF4_BF16;
    const List l{items, gram_first, apply_first, sizes.count};
    const Space ws{reinterpret_cast<double *>(base + sizes.partial), reinterpret_cast<double *>(base + sizes.mats),
                   reinterpret_cast<double *>(base + sizes.norm), reinterpret_cast<uint16_t *>(base + sizes.p)};
    const bool g16 = call.grad == NF4_BF16, m16 = call.m == NF4_BF16;
    if (!call.step) return g16 ? run<Bf16, None>(sizes, l, c, ws, s) : run<float, None>(sizes, l, c, ws, s);
    if (g16) return m16 ? run<Bf16, Bf16>(sizes, l, c, ws, s) : run<Bf16, float>(sizes, l, c, ws, s);
    return m16 ? run<float, Bf16>(sizes, l, c, ws, s) : run<float, float>(sizes, l, c, ws, s);
}

}  // namespace nf4
