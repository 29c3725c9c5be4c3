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
// in fp32 over 64 rows at most and in fp64 beyond, and the s x s products run on the
// fp64 matrix instruction; the two passes over the long matrices use the fp32 one.
#include <math.h>

#include "training_internal.h"

namespace nf4 {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = 4;
constexpr int kSmall = 64;     // shorter sides up to here are iterated in one workgroup's LDS
constexpr int kFlush = 64;     // rows that a fp32 sum of S takes

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
    uint32_t p, pad;         // first element of P (fp32), in units of 256
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
    float *p;
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

template <typename T> struct Raw4;
template <> struct Raw4<Bf16> { u32x2 v; };
template <> struct Raw4<float> { f32x4 v; };
struct None {};
template <> struct Raw4<None> {};

template <typename T>
__device__ __forceinline__ Raw4<T> load4(const void *p, int64_t at, int live, bool vec) {
    if constexpr (sizeof(T) == 1) return {};  // None
    else {
        const T *q = static_cast<const T *>(p) + at;
        Raw4<T> r{};
        if (vec) {
            if (live > 0) r.v = *reinterpret_cast<const decltype(r.v) *>(q);
            return r;
        }
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = j < live ? load1(q + j) : 0.0f;
        if constexpr (sizeof(T) == 2) r.v = u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
        else r.v = f32x4{x[0], x[1], x[2], x[3]};
        return r;
    }
}
__device__ __forceinline__ void values4(const Raw4<Bf16> &r, float (&x)[4]) {
    x[0] = bf16_lo(r.v[0]), x[1] = bf16_hi(r.v[0]), x[2] = bf16_lo(r.v[1]), x[3] = bf16_hi(r.v[1]);
}
__device__ __forceinline__ void values4(const Raw4<float> &r, float (&x)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = r.v[j];
}
template <typename T>
__device__ __forceinline__ void store4(T *q, int live, bool vec, const float (&x)[4]) {
    if (vec) {
        if (live <= 0) return;
        if constexpr (sizeof(T) == 2) *reinterpret_cast<u32x2 *>(q) = u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
        else *reinterpret_cast<f32x4 *>(q) = f32x4{x[0], x[1], x[2], x[3]};
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < live) store1(q + j, x[j]);
}

// Four consecutive elements of the gradient and the momentum, as they lie in memory.
template <typename G, typename M> struct Raw {
    Raw4<G> g;
    Raw4<M> m;
};
template <typename G, typename M>
__device__ __forceinline__ Raw<G, M> load_update(const Item &e, int64_t at, int live, bool vec) {
    return {load4<G>(e.g, at, live, vec), load4<M>(e.m, at, live, vec)};
}
// The update of the four, and the new momentum. Each is computed by the same operations
// in both passes, so both see the same bits.
template <typename G, typename M>
__device__ __forceinline__ void update4(const Raw<G, M> &r, const Scalars &c, float (&u)[4], float (&m)[4]) {
    values4(r.g, u);
    if constexpr (sizeof(M) != 1) {
        values4(r.m, m);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float g = c.one_mu * u[j];
            m[j] = fmaf(c.mu, m[j], g);
            u[j] = c.nesterov ? fmaf(c.mu, m[j], g) : m[j];
        }
    }
}

// ---- S: the Gram matrix ----

// A wave's share of S for the 16 NI columns from 64 bi on and the 16 NJ from 64 bj on, rows from
// `begin` to `end` of the longer side. Operands of the matrix instruction hold four rows
// of 16 columns. In a tall matrix a lane loads NI consecutive columns, so its column in
// operand i is NI n + i; in a wide one four consecutive rows of column 16 i + n.
template <typename G, typename M, int NI, int NJ, bool kDiag>
__device__ __forceinline__ void gram_rows(const Item &e, const Scalars &c, int bi, int bj, int64_t begin, int64_t end,
                                          f64x4 *sums) {
    constexpr int kTiles = kDiag ? NI * (NI + 1) / 2 : NI * NJ;
    const int lane = threadIdx.x % 64, n = lane % 16, k = lane / 16;
    f32x4 acc[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f}, sums[t] = f64x4{0.0, 0.0, 0.0, 0.0};
    auto products = [&](const float (&x)[NI], const float (&y)[NJ]) {
        int t = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = kDiag ? i : 0; j < NJ; ++j, ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[j], acc[t], 0, 0, 0);
    };
    auto flush = [&] {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
#pragma unroll
            for (int r = 0; r < 4; ++r) sums[t][r] += (double)acc[t][r];
            acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    };
    // 16 rows of N columns each: rows 4 r + k of a tall matrix, 4 k + r of a wide one
    auto load = [&](auto &x, int block, int64_t row) {
        constexpr int N = sizeof(x[0]) / sizeof(float);
        if (e.tall) {
            const int col = 64 * block + N * n;
            const bool vec = e.side % N == 0;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t l = row + 4 * r + k;
                const int64_t at = l * e.side + col;
                const int live = l < end ? e.side - col : 0;
                if constexpr (N == 4) {
                    float m[4];
                    update4(load_update<G, M>(e, at, live, vec), c, x[r], m);
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        float u[4], m[4];
                        update4(load_update<G, M>(e, at + j, min(live - j, 1), false), c, u, m);
                        x[r][j] = u[0];
                    }
                }
            }
        } else {
            const bool vec = e.length % 4 == 0;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int col = 64 * block + 16 * j + n;
                const int64_t l = row + 4 * k;
                const int live = col < e.side && l < end ? (int)min(end - l, (int64_t)4) : 0;
                float u[4], m[4];
                update4(load_update<G, M>(e, (int64_t)col * e.length + l, live, vec), c, u, m);
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r][j] = u[r];
            }
        }
    };
    int since = 0;
    for (int64_t row = begin; row < end; row += 16) {
        float x[4][NI], y[4][NJ];
        load(x, bi, row);
        if constexpr (!kDiag) load(y, bj, row);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if constexpr (kDiag) products(x[r], x[r]);
            else products(x[r], y[r]);
        since += 16;
        if (since == kFlush) flush(), since = 0;
    }
    flush();
}

// Sums of the workgroup's waves, then out: [tile][register][lane].
template <typename G, typename M, int NI, int NJ, bool kDiag>
__device__ __forceinline__ void gram_part(const Item &e, const Scalars &c, int bi, int bj, int64_t begin, int64_t end,
                                          double *out, double (*part)[256]) {
    constexpr int kTiles = kDiag ? NI * (NI + 1) / 2 : NI * NJ;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t share = ((end - begin + kWaves - 1) / kWaves + 15) / 16 * 16;
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

template <typename G, typename M>
__global__ __launch_bounds__(kThreads) void muon_gram_kernel(List list, Scalars c, Space ws) {
    __shared__ double part[16][256];
    const Item e = list.item[find(list.gram_first, list.count, blockIdx.x)];
    const uint32_t own = blockIdx.x - e.gram_first, chunk = own / e.gram_pairs, pair = own % e.gram_pairs;
    const int64_t begin = (int64_t)chunk * e.gram_chunk, end = min(begin + e.gram_chunk, e.length);
    double *out = ws.partial + e.partial + (int64_t)own * gram_tiles(e.side) * 256;
    if (e.side <= 16) gram_part<G, M, 1, 1, true>(e, c, 0, 0, begin, end, out, part);
    else if (e.side <= 32) gram_part<G, M, 2, 2, true>(e, c, 0, 0, begin, end, out, part);
    else if (e.side <= kSmall) gram_part<G, M, 4, 4, true>(e, c, 0, 0, begin, end, out, part);
    else {
        int bi, bj;
        pair_of(pair, bi, bj);
        gram_part<G, M, 4, 4, false>(e, c, bi, bj, begin, end, out, part);
    }
}

// Where sum i of a pair of blocks of NI and NJ operands lies in it.
__device__ __forceinline__ void place_of(const Item &e, int width, bool diag, int i, int &row, int &col) {
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

// ---- the iteration, shorter sides up to 64: one workgroup a matrix ----

constexpr int kStride = kSmall + 2;  // doubles: 16 rows of two columns lie in different banks
typedef double SmallMat[kSmall][kStride];
constexpr int kSmallThreads = 1024;

__global__ __launch_bounds__(kSmallThreads) void muon_small_kernel(List list, Scalars c, Space ws) {
    extern __shared__ double smem[];
    SmallMat &A = *reinterpret_cast<SmallMat *>(smem), &Q = (&A)[1], &P = (&A)[2];
    double *part = smem + 3 * kSmall * kStride;
    const Item e = list.item[blockIdx.x];
    if (e.side > kSmall) return;
    const int tiles = gram_tiles(e.side), width = gram_width(e.side), edge = (e.side + 15) / 16;
    const double *from = ws.partial + e.partial;
    for (int i = threadIdx.x; i < tiles * 256; i += kSmallThreads) {
        double x = 0.0;
        for (uint32_t k = 0; k < e.gram_chunks; ++k) x += from[(int64_t)k * tiles * 256 + i];
        int row, col;
        place_of(e, width, true, i, row, col);
        A[row][col] = x, A[col][row] = x;
    }
    __syncthreads();
    const double trace = block_total((int)threadIdx.x < e.side ? A[threadIdx.x][threadIdx.x] : 0.0, part);
    const double norm = sqrt(trace), inv = 1.0 / fmax(norm, c.eps);
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * edge * 16 * edge; i += kSmallThreads) A[i / (16 * edge)][i % (16 * edge)] *= inv * inv;
    const int lane = threadIdx.x % 64, n = lane % 16, k4 = lane / 16;
    const int ti = threadIdx.x / 256, tj = threadIdx.x / 64 % 4;  // a wave's tile
    const bool live = ti < edge && tj < edge;
    auto product = [&](const SmallMat &x, const SmallMat &y) {
        f64x4 r = {0.0, 0.0, 0.0, 0.0};
        if (live)
            for (int k = 0; k < 16 * edge; k += 4)
                r = __builtin_amdgcn_mfma_f64_16x16x4f64(x[16 * ti + n][k + k4], y[16 * tj + n][k + k4], r, 0, 0, 0);
        return r;
    };
    auto put = [&](SmallMat &x, const f64x4 &r) {
        if (live)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[16 * ti + 4 * j + k4][16 * tj + n] = r[j];
    };
    for (int it = 0; it < c.iterations; ++it) {
        __syncthreads();
        f64x4 q = product(A, A);
        if (live)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = 16 * ti + 4 * j + k4, col = 16 * tj + n;
                q[j] = c.c * q[j] + c.b * A[row][col] + (row == col ? c.a : 0.0);
            }
        put(it == 0 ? P : Q, q);
        if (it == 0) put(Q, q);
        __syncthreads();
        f64x4 t, p;
        const bool last = it + 1 == c.iterations;
        if (!last) t = product(A, Q);
        if (it > 0) p = product(P, Q);
        __syncthreads();
        if (!last) put(A, t);
        if (it > 0) put(P, p);
        if (last) break;
        __syncthreads();
        t = product(A, Q);
        __syncthreads();
        put(A, t);
    }
    __syncthreads();
    float *out = ws.p + (int64_t)e.p * 256;
    for (int i = threadIdx.x; i < kSmall * kSmall; i += kSmallThreads) {
        const int row = i / kSmall, col = i % kSmall;
        out[i] = row < e.side && col < e.side ? (float)(P[row][col] * inv) : 0.0f;
    }
    if (threadIdx.x == 0) ws.norm[blockIdx.x] = norm;
}

// ---- the iteration, shorter sides above 64: a launch a product, 64 x 64 a workgroup ----

__host__ __device__ inline int blocks_of(int side) { return (side + 63) / 64; }
enum Mat { kA, kQ, kT, kP0, kP1, kMats };

__device__ __forceinline__ double *mat_of(const Item &e, const Space &ws, int which) {
    const int64_t edge = 64 * blocks_of(e.side);
    return ws.mats + e.mats + which * edge * edge;
}

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
        const int at = ((pair * 16) + i * 4 + i) * 256 + (r % 4) * 64 + (r / 4) * 16 + r;
        for (uint32_t k = 0; k < e.gram_chunks; ++k) x += from[k * stride + at];
    }
    const double trace = block_total(x, part);
    const double norm = sqrt(trace), inv = 1.0 / fmax(norm, c.eps);
    int bi, bj;
    pair_of(blockIdx.y, bi, bj);
    double *A = mat_of(e, ws, kA);
    for (int i = threadIdx.x; i < 16 * 256; i += kThreads) {
        double sum = 0.0;
        for (uint32_t k = 0; k < e.gram_chunks; ++k) sum += from[k * stride + (int64_t)blockIdx.y * 16 * 256 + i];
        int row, col;
        place_of(e, 4, false, i, row, col);
        sum *= inv * inv;
        row += 64 * bi, col += 64 * bj;
        // a block with itself holds both of each pair: the upper one is taken
        if (bi != bj || row <= col) A[(int64_t)row * edge + col] = sum, A[(int64_t)col * edge + row] = sum;
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) ws.norm[blockIdx.x] = norm;
}

// out = x y, with q: c out + b x + a I (x = y), which also goes to `copy`; with fin: over
// the norm, in fp32, to P. blockIdx.z chooses one of two products. All matrices are
// polynomials of one, so x y is symmetric and a column of y is read as its row.
struct Product {
    int32_t x, y, out, copy;  // copy: -1 none
    bool q, fin;
};
struct Products {
    Product of[2];
};
constexpr int kSlab = 32;

__global__ __launch_bounds__(kThreads) void muon_product_kernel(List list, Scalars c, Space ws, Products products) {
    __shared__ double xs[64][kSlab + 2], ys[64][kSlab + 2];
    const Item e = list.item[blockIdx.x];
    const int nb = blocks_of(e.side), edge = 64 * nb;
    if (e.side <= kSmall || (int)blockIdx.y >= nb * nb) return;
    const Product d = products.of[blockIdx.z];
    const int bi = blockIdx.y / nb, bj = blockIdx.y % nb;
    const double *x = mat_of(e, ws, d.x), *y = mat_of(e, ws, d.y);
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, n = lane % 16, k4 = lane / 16;
    f64x4 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f64x4{0.0, 0.0, 0.0, 0.0};
    for (int k0 = 0; k0 < edge; k0 += kSlab) {
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * kSlab; i += kThreads) {
            const int row = i / kSlab, col = i % kSlab;
            xs[row][col] = x[(int64_t)(64 * bi + row) * edge + k0 + col];
            ys[row][col] = y[(int64_t)(64 * bj + row) * edge + k0 + col];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSlab; k += 4)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[j] = __builtin_amdgcn_mfma_f64_16x16x4f64(xs[16 * wave + n][k + k4], ys[16 * j + n][k + k4], acc[j], 0, 0, 0);
    }
    const double inv = 1.0 / fmax(ws.norm[blockIdx.x], c.eps);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 64 * bi + 16 * wave + 4 * r + k4, col = 64 * bj + 16 * j + n;
            const int64_t at = (int64_t)row * edge + col;
            double v = acc[j][r];
            if (d.q) v = c.c * v + c.b * x[at] + (row == col ? c.a : 0.0);
            if (d.fin) {
                ws.p[(int64_t)e.p * 256 + at] = row < e.side && col < e.side ? (float)(v * inv) : 0.0f;
            } else {
                mat_of(e, ws, d.out)[at] = v;
                if (d.copy >= 0) mat_of(e, ws, d.copy)[at] = v;
            }
        }
}

// ---- O = U P and the step ----

// Four consecutive elements of O: the weight's step, or the output alone.
__device__ __forceinline__ void finish4(const Item &e, const Scalars &c, int64_t at, int live, bool vec, float (&o)[4]) {
    if (c.step) {
        float w[4];
        if (e.master) values4(load4<float>(e.master, at, live, vec), w);
        else if (c.w_bf16) values4(load4<Bf16>(e.w, at, live, vec), w);
        else values4(load4<float>(e.w, at, live, vec), w);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = fmaf(-e.step, o[j], e.keep * w[j]);
        if (e.master) store4(e.master + at, live, vec, o);
    }
    if (c.w_bf16) store4(static_cast<Bf16 *>(e.w) + at, live, vec, o);
    else store4(static_cast<float *>(e.w) + at, live, vec, o);
}

constexpr int kRowPad = 4;  // floats: the operands' rows start in different banks

// A matrix of up to 64 on its shorter side: P in LDS, a wave's U in registers in the
// places that O takes. In a tall matrix a wave takes 16 rows and a lane four columns of
// each 16; in a wide one 64 columns, a lane four of them in every row.
template <typename G, typename M>
__device__ __forceinline__ void apply_small(const Item &e, const Scalars &c, const float (*p)[kSmall + kRowPad], int64_t begin,
                                            int64_t end) {
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, n = lane % 16, k = lane / 16;
    const int edge = (e.side + 15) / 16;
    if (e.tall) {
        const bool vec = e.side % 4 == 0;
        for (int64_t row = begin + wave * 16; row < end; row += 16 * kWaves) {
            const int64_t l = row + n, at = l * e.side;
            float u[4][4];
            f32x4 acc[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int col = 16 * b + 4 * k, live = l < end ? e.side - col : 0;
                float m[4];
                update4(load_update<G, M>(e, at + col, live, vec), c, u[b], m);
                if constexpr (sizeof(M) != 1) store4(static_cast<M *>(e.m) + at + col, live, vec, m);
                acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (b >= edge) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i >= edge) break;
                    const f32x4 x = *reinterpret_cast<const f32x4 *>(&p[16 * i + n][16 * b + 4 * k]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[r], u[b][r], acc[i], 0, 0, 0);
                }
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int col = 16 * b + 4 * k, live = l < end ? e.side - col : 0;
                float o[4] = {acc[b][0], acc[b][1], acc[b][2], acc[b][3]};
                finish4(e, c, at + col, live, vec, o);
            }
        }
    } else {
        const bool vec = e.length % 4 == 0;
        for (int64_t col = begin + wave * 64; col < end; col += 64 * kWaves) {
            const int64_t l = col + 4 * n;
            const int live = l < end ? (int)min(end - l, (int64_t)4) : 0;
            f32x4 acc[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (b >= edge) break;
                float u[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * b + 4 * k + r, here = row < e.side ? live : 0;
                    float m[4];
                    update4(load_update<G, M>(e, (int64_t)row * e.length + l, here, vec), c, u[r], m);
                    if constexpr (sizeof(M) != 1)
                        store4(static_cast<M *>(e.m) + (int64_t)row * e.length + l, here, vec, m);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i >= edge) break;
                    const f32x4 x = *reinterpret_cast<const f32x4 *>(&p[16 * i + n][16 * b + 4 * k]);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[r], u[r][j], acc[i][j], 0, 0, 0);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * i + 4 * k + r, here = row < e.side ? live : 0;
                    float o[4] = {acc[i][0][r], acc[i][1][r], acc[i][2][r], acc[i][3][r]};
                    finish4(e, c, (int64_t)row * e.length + l, here, vec, o);
                }
        }
    }
}

// A matrix of up to 256 on its shorter side, 64 places of the longer: U in LDS, which a
// workgroup has read whole before it writes the momentum; a wave takes every fourth 16
// columns of O, and P from the caches.
template <typename G, typename M>
__device__ __forceinline__ void apply_large(const Item &e, const Scalars &c, const float *p, float *us, int64_t begin,
                                            int64_t end) {
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, n = lane % 16, k = lane / 16;
    const int nb = blocks_of(e.side), edge = 64 * nb, stride = edge + kRowPad, tiles = (e.side + 15) / 16;
    for (int64_t l0 = begin; l0 < end; l0 += 64) {
        const int rows = (int)min(end - l0, (int64_t)64);
        __syncthreads();
        if (e.tall) {
            const bool vec = e.side % 4 == 0;
            for (int i = threadIdx.x; i < 64 * edge / 4; i += kThreads) {
                const int row = i / (edge / 4), col = i % (edge / 4) * 4, live = row < rows ? e.side - col : 0;
                const int64_t at = (l0 + row) * e.side + col;
                float u[4], m[4];
                update4(load_update<G, M>(e, at, live, vec), c, u, m);
                if constexpr (sizeof(M) != 1) store4(static_cast<M *>(e.m) + at, live, vec, m);
                *reinterpret_cast<f32x4 *>(us + row * stride + col) = f32x4{u[0], u[1], u[2], u[3]};
            }
        } else {
            const bool vec = e.length % 4 == 0;
            for (int i = threadIdx.x; i < 16 * edge; i += kThreads) {
                const int row = i / 16, col = i % 16 * 4, live = row < e.side ? rows - col : 0;
                const int64_t at = (int64_t)row * e.length + l0 + col;
                float u[4], m[4];
                update4(load_update<G, M>(e, at, live, vec), c, u, m);
                if constexpr (sizeof(M) != 1) store4(static_cast<M *>(e.m) + at, live, vec, m);
#pragma unroll
                for (int j = 0; j < 4; ++j) us[(col + j) * stride + row] = u[j];
            }
        }
        __syncthreads();
        f32x4 acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int b = 0; b < tiles; ++b) {
            f32x4 u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = *reinterpret_cast<const f32x4 *>(us + (16 * j + n) * stride + 16 * b + 4 * k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tile = wave + 4 * i;
                if (tile >= tiles) break;
                const f32x4 x = *reinterpret_cast<const f32x4 *>(p + (int64_t)(16 * tile + n) * edge + 16 * b + 4 * k);
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[r], u[j][r], acc[i][j], 0, 0, 0);
            }
        }
        // O to LDS in U's place, so that both kinds leave whole lines
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tile = wave + 4 * i;
            if (tile >= tiles) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) *reinterpret_cast<f32x4 *>(us + (16 * j + n) * stride + 16 * tile + 4 * k) = acc[i][j];
        }
        __syncthreads();
        if (e.tall) {
            const bool vec = e.side % 4 == 0;
            for (int i = threadIdx.x; i < 64 * edge / 4; i += kThreads) {
                const int row = i / (edge / 4), col = i % (edge / 4) * 4, live = row < rows ? e.side - col : 0;
                const f32x4 x = *reinterpret_cast<const f32x4 *>(us + row * stride + col);
                float o[4] = {x[0], x[1], x[2], x[3]};
                finish4(e, c, (l0 + row) * e.side + col, live, vec, o);
            }
        } else {
            const bool vec = e.length % 4 == 0;
            for (int i = threadIdx.x; i < 16 * edge; i += kThreads) {
                const int row = i / 16, col = i % 16 * 4, live = row < e.side ? rows - col : 0;
                float o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = us[(col + j) * stride + row];
                finish4(e, c, (int64_t)row * e.length + l0 + col, live, vec, o);
            }
        }
    }
}

template <typename G, typename M>
__global__ __launch_bounds__(kThreads) void muon_apply_kernel(List list, Scalars c, Space ws) {
    extern __shared__ float sp[];
    const int32_t index = find(list.apply_first, list.count, blockIdx.x);
    const Item e = list.item[index];
    if (c.step && !isfinite(ws.norm[index])) return;
    const int64_t begin = (int64_t)(blockIdx.x - e.apply_first) * e.apply_chunk;
    const int64_t end = min(begin + e.apply_chunk, e.length);
    const float *p = ws.p + (int64_t)e.p * 256;
    if (e.side > kSmall) return apply_large<G, M>(e, c, p, sp, begin, end);
    float (*rows)[kSmall + kRowPad] = reinterpret_cast<float (*)[kSmall + kRowPad]>(sp);
    for (int i = threadIdx.x; i < kSmall * kSmall / 4; i += kThreads)
        *reinterpret_cast<f32x4 *>(&rows[i / 16][i % 16 * 4]) = *reinterpret_cast<const f32x4 *>(p + 4 * i);
    __syncthreads();
    apply_small<G, M>(e, c, rows, begin, end);
}

// ---- host ----

size_t round_up(size_t x, size_t to) { return (x + to - 1) / to * to; }

// How a list is cut, and what lies where in the workspace. The longer sides are cut into
// about 2048 shares of each pass, so that the chip is full and few partial sums are left.
struct Plan {
    size_t items, gram_first, apply_first, norm, partial, mats, p, bytes;  // offsets
    uint32_t gram_wgs, apply_wgs;
    int32_t count, largest;  // matrices with elements; the largest shorter side
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
        ps += edge * edge / 256;
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
    muon_gram_kernel<G, M><<<dim3(p.gram_wgs), dim3(kThreads), 0, s>>>(list, c, ws);
    hipError_t r = hipGetLastError();
    if (r != hipSuccess) return r;
    constexpr size_t kSmallLds = (3 * kSmall * kStride + 16) * sizeof(double);
    if ((r = allow_lds(reinterpret_cast<const void *>(&muon_small_kernel), kSmallLds)) != hipSuccess) return r;
    muon_small_kernel<<<dim3(p.count), dim3(kSmallThreads), kSmallLds, s>>>(list, c, ws);
    if ((r = hipGetLastError()) != hipSuccess) return r;
    if (p.largest > kSmall) {
        const int nb = blocks_of(p.largest);
        muon_start_kernel<<<dim3(p.count, nb * (nb + 1) / 2), dim3(kThreads), 0, s>>>(list, c, ws);
        if ((r = hipGetLastError()) != hipSuccess) return r;
        auto launch = [&](const Products &x, int z) {
            if (r != hipSuccess) return;
            muon_product_kernel<<<dim3(p.count, nb * nb, z), dim3(kThreads), 0, s>>>(list, c, ws, x);
            r = hipGetLastError();
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
    size_t lds = kSmall * (kSmall + kRowPad) * 4;
    if (p.largest > kSmall) lds = 64 * (64 * blocks_of(p.largest) + kRowPad) * 4;
    if ((r = allow_lds(reinterpret_cast<const void *>(&muon_apply_kernel<G, M>), lds)) != hipSuccess) return r;
    muon_apply_kernel<G, M><<<dim3(p.apply_wgs), dim3(kThreads), lds, s>>>(list, c, ws);
    return hipGetLastError();
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
                   reinterpret_cast<double *>(base + sizes.norm), reinterpret_cast<float *>(base + sizes.p)};
    const bool g16 = call.grad == NF4_BF16, m16 = call.m == NF4_BF16;
    if (!call.step) return g16 ? run<Bf16, None>(sizes, l, c, ws, s) : run<float, None>(sizes, l, c, ws, s);
    if (g16) return m16 ? run<Bf16, Bf16>(sizes, l, c, ws, s) : run<Bf16, float>(sizes, l, c, ws, s);
    return m16 ? run<float, Bf16>(sizes, l, c, ws, s) : run<float, float>(sizes, l, c, ws, s);
}

}  // namespace nf4
