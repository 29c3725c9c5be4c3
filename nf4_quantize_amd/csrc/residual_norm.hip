// residual_norm.hip - the residual step between two blocks for gfx950: the
// norm after a block, its gate and residual scale, the residual addition and
// the norm before the next block in one pass over each row, and the backward
// pass of all of them. The formulas are in nf4.h
// (nf4_residual_norm_forward, nf4_residual_norm_backward).
//
// Both are bound by HBM: the forward reads y and h and writes h' and x (8 bytes
// an element in bf16), the backward reads dx, dh', y and h' and writes dy and
// dh (12 bytes), and each element is moved once; the backward pass reads rows of more
// than 8192 columns twice. A row is held in registers by a group of lanes, eight
// consecutive elements a lane and vector.
#include <math.h>

#include <type_traits>

#include "training_internal.h"

namespace nf4 {
namespace {

struct ColumnOut {
    void *out[3];
};

struct NormParams {
    ResidualNormIn in;
    ResidualNormOut out;
    int64_t rows;
    int32_t dim;
    float inv_dim, eps, alpha, off;
    int32_t lanes;       // lanes of a row: 8 .. 64, a power of two, or the whole workgroup
    int32_t gate_kind;
    bool w_bf16;
    float *partial;      // backward: [workgroups][3][dim], unless there is one workgroup
    ColumnOut sums;      // the gradients summed over rows that are asked for
    float2 *means;       // backward, rows of several tiles: [rows]
};

// How a row lies in memory: fewer than eight elements; any number; or whole
// vectors (dim a multiple of 8), which are moved past the caches' usual order, as
// nothing here is read twice. The same rows as kRowAny take 67 us instead of 57
// forward and 96 instead of 83 backward (16384 x 2048 bf16). With an fp32 stream and
// more than 512 columns a lane takes two fours instead of an eight (kRowFours):
// 8192 x 8192 fp32 take 186 us instead of 203 forward and 286 instead of 366
// backward, bf16 blocks on an fp32 stream 137 (as before) and 217 instead of 259.
enum RowKind { kRowNarrow, kRowAny, kRowVecs, kRowFours };

template <RowKind kKind>
using ColsOf = std::conditional_t<kKind == kRowFours, Fours, Cols<kKind == kRowNarrow>>;

template <RowKind kKind, typename T>
__device__ __forceinline__ Raw8<T> load_row(const T *row, const ColsOf<kKind> &c) {
    if constexpr (kKind == kRowFours) return load_stream(row, c);
    else if constexpr (kKind == kRowVecs) return load_stream(row + (uint32_t)c.base);
    else return load_cols(row, c);
}
template <RowKind kKind, typename T>
__device__ __forceinline__ void row_values(const Raw8<T> &r, const ColsOf<kKind> &c, float (&x)[8]) {
    if constexpr (kKind == kRowVecs) {
        values(r, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = c.live > 0 ? x[j] : 0.0f;
    } else {
        cols_values(r, c, x);
    }
}
template <RowKind kKind, typename T>
__device__ __forceinline__ void store_row(T *row, const ColsOf<kKind> &c, const float (&x)[8]) {
    if constexpr (kKind == kRowVecs) {
        if (c.live > 0) store_stream(row + (uint32_t)c.col, x);
    } else {
        stream_cols(row, c, x);
    }
}

// Eight weights of the columns (fp32 or bf16).
template <typename C>
__device__ __forceinline__ void load_weight(const void *w, bool bf16, const C &c, float (&x)[8]) {
    if (bf16) cols_values(load_cols(static_cast<const Bf16 *>(w), c), c, x);
    else cols_values(load_cols(static_cast<const float *>(w), c), c, x);
}

// Sums of kK values over each row's lanes, the same bits in every lane. A row of
// more than a wave (kWide) is the whole workgroup's, and its waves meet in `part`; the
// caller alternates two buffers, so that one barrier a call is enough.
template <bool kWide, int kK>
__device__ __forceinline__ void row_sums(float (&x)[kK], int lanes, float (*part)[16]) {
#pragma unroll
    for (int k = 0; k < kK; ++k) x[k] = group_sum(x[k], kWide ? 64 : lanes);
    if constexpr (!kWide) return;
    const int lane = threadIdx.x % 64, waves = blockDim.x / 64;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < kK; ++k) part[k][threadIdx.x / 64] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kK; ++k) x[k] = group_sum(lane % 16 < waves ? part[k][lane % 16] : 0.0f, 16);
}

// The columns' weights: kept by workgroups of one vector a lane, which take many
// rows, and loaded for each row by the others.
template <typename C>
struct Weights {
    float pre[8], post[8], gate[8];
    __device__ __forceinline__ void load(const NormParams &p, bool channel, const C &c) {
        load_weight(p.in.w_pre, p.w_bf16, c, pre);
#pragma unroll
        for (int j = 0; j < 8; ++j) pre[j] += p.off, post[j] = 1.0f, gate[j] = 1.0f;
        if (p.in.w_post) {
            load_weight(p.in.w_post, p.w_bf16, c, post);
#pragma unroll
            for (int j = 0; j < 8; ++j) post[j] += p.off;
        }
        if (channel) load_weight(p.in.gate, p.w_bf16, c, gate);
    }
    // A lane's own weights in LDS.
    template <int kLanes>
    __device__ __forceinline__ void save(f32x4 (*s)[kLanes]) const {
        const float *const all[3] = {pre, post, gate};
#pragma unroll
        for (int k = 0; k < 6; ++k) {
            const float *x = all[k / 2] + k % 2 * 4;
            s[k][threadIdx.x] = f32x4{x[0], x[1], x[2], x[3]};
        }
    }
    template <bool kToken, int kLanes>
    __device__ __forceinline__ void restore(const f32x4 (*s)[kLanes]) {
        asm volatile("" ::: "memory");
        float *const all[3] = {pre, post, gate};
#pragma unroll
        for (int k = 0; k < (kToken ? 4 : 6); ++k) {
            const f32x4 x = s[k][threadIdx.x];
#pragma unroll
            for (int j = 0; j < 4; ++j) all[k / 2][k % 2 * 4 + j] = x[j];
        }
    }
};

// A workgroup takes every gridDim.x-th set of rows. With one vector a lane it
// loads the next set while it works on one.
template <typename T, typename R, int kVec, RowKind kKind, bool kWide>
__global__ __launch_bounds__(1024) void residual_norm_forward_kernel(NormParams p) {
    __shared__ float part[2][1][16];
    constexpr bool kOne = kVec == 1;
    typedef ColsOf<kKind> C;
    const int lanes = kWide ? blockDim.x : p.lanes;
    const int groups = kWide ? 1 : blockDim.x / lanes, group = kWide ? 0 : threadIdx.x / lanes;
    const int lane = kWide ? threadIdx.x : threadIdx.x % lanes;
    const T *y = static_cast<const T *>(p.in.y);
    const R *h_in = static_cast<const R *>(p.in.h);
    const bool post = p.in.w_post != nullptr, channel = y && p.gate_kind == NF4_GATE_CHANNEL;
    auto col = [&](int v) { return C((v * lanes + lane) * 8, p.dim); };
    Weights<C> w;
    Raw8<T> raw_y[kVec];
    Raw8<R> raw_h[kVec];
    auto load = [&](int64_t r0) {
        const int64_t row = r0 + group < p.rows ? r0 + group : p.rows - 1;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            raw_h[v] = load_row<kKind>(h_in + row * p.dim, col(v));
            if (y) raw_y[v] = load_row<kKind>(y + row * p.dim, col(v));
        }
    };
    const int64_t first = (int64_t)blockIdx.x * groups, stride = (int64_t)gridDim.x * groups;
    if constexpr (kOne) {
        load(first);
        w.load(p, channel, col(0));
    }
    int turn = 0;
    for (int64_t r0 = first; r0 < p.rows; r0 += stride) {
        const int64_t row = r0 + group, at = row * p.dim;
        const bool live_row = row < p.rows;
        if constexpr (!kOne) load(r0);
        float h[kVec][8], z[8];
        if constexpr (kOne) {
            row_values<kKind>(raw_h[0], col(0), h[0]);
            if (y) row_values<kKind>(raw_y[0], col(0), z);
            if (r0 + stride < p.rows) load(r0 + stride);
        }
        float r2 = 1.0f;
        if (post) {
            float s[1] = {0.0f};
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                if constexpr (!kOne) row_values<kKind>(raw_y[v], col(v), z);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[0] += z[j] * z[j];
            }
            row_sums<kWide>(s, lanes, part[turn]);
            turn ^= 1;
            r2 = 1.0f / sqrtf(s[0] * p.inv_dim + p.eps);
            if (live_row && lane == 0 && p.out.rstd_post) p.out.rstd_post[row] = r2;
        }
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            if constexpr (!kOne) row_values<kKind>(raw_h[v], col(v), h[v]);
            if (!y) continue;
            if constexpr (!kOne) {
                row_values<kKind>(raw_y[v], col(v), z);
                w.load(p, channel, col(v));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] *= r2 * w.post[j];
            if (p.gate_kind == NF4_GATE_TOKEN) {
                const int64_t there = (live_row ? row : p.rows - 1) * p.dim;
                float g[8];
                row_values<kKind>(load_row<kKind>(static_cast<const T *>(p.in.gate) + there, col(v)), col(v), g);
#pragma unroll
                for (int j = 0; j < 8; ++j) z[j] *= g[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) h[v][j] += p.alpha * (z[j] * w.gate[j]);
            if (live_row) store_row<kKind>(static_cast<R *>(p.out.h) + at, col(v), h[v]);
            if constexpr (!kOne) asm volatile("" ::: "memory");  // one vector's weights at a time
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += h[v][j] * h[v][j];
        row_sums<kWide>(s, lanes, part[turn]);
        turn ^= 1;
        const float r1 = 1.0f / sqrtf(s[0] * p.inv_dim + p.eps);
        if (live_row && lane == 0 && p.out.rstd_pre) p.out.rstd_pre[row] = r1;
        if (!live_row) continue;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            if constexpr (!kOne) w.load(p, false, col(v));
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = h[v][j] * (r1 * w.pre[j]);
            store_row<kKind>(static_cast<T *>(p.out.x) + at, col(v), x);
            if constexpr (!kOne) asm volatile("" ::: "memory");
        }
    }
}

// One vector of a row's inputs in the backward pass; kToken: the gate is one.
template <typename T, typename R, RowKind kKind, bool kToken>
struct BackwardRow {
    Raw8<T> dx, y, gate[kToken ? 1 : 0];
    Raw8<R> h, dh;
    typedef ColsOf<kKind> C;
    __device__ __forceinline__ void load(const NormParams &p, int64_t at, const C &c) {
        h = load_row<kKind>(static_cast<const R *>(p.in.h) + at, c);
        if (p.in.dx) dx = load_row<kKind>(static_cast<const T *>(p.in.dx) + at, c);
        if (p.in.dh_out) dh = load_row<kKind>(static_cast<const R *>(p.in.dh_out) + at, c);
        if (p.in.y) y = load_row<kKind>(static_cast<const T *>(p.in.y) + at, c);
        if constexpr (kToken) gate[0] = load_row<kKind>(static_cast<const T *>(p.in.gate) + at, c);
    }
};

// The values of one vector of a row in the backward pass.
template <typename T, typename R, RowKind kKind, bool kToken>
struct BackwardValues {
    typedef ColsOf<kKind> C;
    float dx[8], n1[8], n2[8], dh[8], g[8];  // g: the gate with alpha
    __device__ __forceinline__ void unpack(const NormParams &p, const BackwardRow<T, R, kKind, kToken> &raw,
                                           const Weights<ColsOf<kKind>> &w, const C &c, float r1, float r2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) dx[j] = dh[j] = n2[j] = 0.0f;
        row_values<kKind>(raw.h, c, n1);
        if (p.in.dx) row_values<kKind>(raw.dx, c, dx);
        if (p.in.dh_out) row_values<kKind>(raw.dh, c, dh);
        if (p.in.y) row_values<kKind>(raw.y, c, n2);
        if constexpr (kToken) row_values<kKind>(raw.gate[0], c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) n1[j] *= r1, n2[j] *= r2, g[j] = p.alpha * (kToken ? g[j] : w.gate[j]);
    }
    // One round of sums serves both norms: with e = alpha gate w_post' n2 the
    // inner product of the second, mean(dz w_post' n2), is mean(e dh), and dh is
    // known up to the first one's mean c1 = mean(dx w_pre' n1):
    //   sum e dh = sum e (dh_out + rstd_pre dx w_pre') - rstd_pre c1 sum e n1.
    __device__ __forceinline__ void add(const Weights<ColsOf<kKind>> &w, float r1, float (&s)[3]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q = dx[j] * w.pre[j], e = g[j] * w.post[j] * n2[j];
            s[0] += q * n1[j];
            s[1] += e * (dh[j] + r1 * q);
            s[2] += e * n1[j];
        }
    }
};
__device__ __forceinline__ void row_means(const float (&s)[3], float r1, float inv_dim, float &c1, float &c2) {
    c1 = s[0] * inv_dim;
    c2 = (s[1] - r1 * c1 * s[2]) * inv_dim;
}

// The two means of each row of more than 8192 columns: one workgroup a row, one
// vector after the other.
template <typename T, typename R, RowKind kKind, bool kToken>
__global__ __launch_bounds__(1024) void residual_norm_means_kernel(NormParams p) {
    __shared__ float part[2][3][16];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        const float r1 = p.in.rstd_pre[row], r2 = p.in.w_post ? p.in.rstd_post[row] : 1.0f;
        float s[3] = {0.0f, 0.0f, 0.0f};
        const int end = kKind == kRowFours ? (p.dim + 511) / 512 * 512 : p.dim;  // whole waves of fours
        for (int c0 = threadIdx.x * 8; c0 < end; c0 += 8192) {
            const ColsOf<kKind> c(c0, p.dim);
            BackwardRow<T, R, kKind, kToken> raw;
            Weights<ColsOf<kKind>> w;
            BackwardValues<T, R, kKind, kToken> x;
            raw.load(p, row * p.dim, c);
            w.load(p, p.in.y && p.gate_kind == NF4_GATE_CHANNEL, c);
            x.unpack(p, raw, w, c, r1, r2);
            x.add(w, r1, s);
        }
        row_sums<true>(s, 1024, part[turn]);
        float c1, c2;
        row_means(s, r1, p.inv_dim, c1, c2);
        if (threadIdx.x == 0) p.means[row] = make_float2(c1, c2);
    }
}

// As the forward: every gridDim.x-th set of rows, the next one's loads in
// flight. A workgroup keeps its columns' share of the weights' gradients in
// registers until its last row. A row of more than 8192 columns is cut into
// tiles (kTiled, blockIdx.y), whose means come from residual_norm_means_kernel:
// the row is read twice, but a lane's sums stay in registers (in one kernel, two
// vectors a lane spilled: 442 us for 2048 x 16384 bf16).
// kMost: threads of the workgroup at most. Up to 512 (4096 columns) a lane may have
// the 133 to 167 registers that it wants, on three waves a SIMD; with 128 on four
// it spills (4096 x 4096 with an fp32 stream and token gates: 74 us instead of 68;
// 16384 x 2304 bf16: 117 instead of 99).
template <typename T, typename R, RowKind kKind, bool kToken, bool kWide, bool kTiled, int kMost>
__global__ __launch_bounds__(kMost) void residual_norm_backward_kernel(NormParams p) {
    __shared__ float part[2][3][16];
    extern __shared__ float s_cols[];
    // Above 512 threads a CU holds one workgroup, and a lane's weights are in LDS: with
    // them in registers too it spilled more (8192 x 8192 bf16 162 us instead of 148, 8192
    // x 5120 124 instead of 96). What still spills there: fp32 rows 6 to 35 registers,
    // token gates 2 to 35, bf16 rows of odd width on an fp32 stream 6. Tiles of bf16
    // blocks on an fp32 stream spill 4 to 6 without LDS and are faster so (5461 x 12288:
    // 374 us with LDS, 355 without).
    constexpr bool kKeep = kMost <= 512 || (kTiled && sizeof(T) == 2 && kKind == kRowFours);
    __shared__ f32x4 s_w[kKeep ? 1 : 6][kKeep ? 1 : kMost];
    typedef ColsOf<kKind> C;
    const int lanes = kWide ? blockDim.x : p.lanes;
    const int groups = kWide ? 1 : blockDim.x / lanes, group = kWide ? 0 : threadIdx.x / lanes;
    const int lane = kWide ? threadIdx.x : threadIdx.x % lanes;
    const bool post = p.in.w_post != nullptr;
    const C c((lane + (kTiled ? blockIdx.y * lanes : 0)) * 8, p.dim);
    float acc[3][8];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[k][j] = 0.0f;
    auto row_at = [&](int64_t r0) { return r0 + group < p.rows ? r0 + group : p.rows - 1; };
    const int64_t first = (int64_t)blockIdx.x * groups, stride = (int64_t)gridDim.x * groups;
    BackwardRow<T, R, kKind, kToken> raw;
    Weights<C> w;
    float next_r1, next_r2 = 1.0f;
    float2 next_means = make_float2(0.0f, 0.0f);
    auto load = [&](int64_t row) {
        raw.load(p, row * p.dim, c);
        next_r1 = p.in.rstd_pre[row];
        if (post) next_r2 = p.in.rstd_post[row];
        if constexpr (kTiled) next_means = p.means[row];
    };
    load(row_at(first));
    w.load(p, p.in.y && p.gate_kind == NF4_GATE_CHANNEL, c);
    if constexpr (!kKeep) w.save(s_w);
    int turn = 0;
    for (int64_t r0 = first; r0 < p.rows; r0 += stride, turn ^= 1) {
        const int64_t at = row_at(r0) * p.dim;
        const bool live_row = r0 + group < p.rows;
        const float r1 = next_r1, r2 = next_r2;
        float c1 = next_means.x, c2 = next_means.y;
        if constexpr (!kKeep) w.template restore<kToken>(s_w);
        BackwardValues<T, R, kKind, kToken> x;
        x.unpack(p, raw, w, c, r1, r2);
        if (r0 + stride < p.rows) load(row_at(r0 + stride));
        if constexpr (!kTiled) {
            float s[3] = {0.0f, 0.0f, 0.0f};
            x.add(w, r1, s);
            row_sums<kWide>(s, lanes, part[turn]);
            row_means(s, r1, p.inv_dim, c1, c2);
        }
        if (!live_row) continue;
        float dg[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            acc[0][j] += x.dx[j] * x.n1[j];
            x.dh[j] += r1 * (x.dx[j] * w.pre[j] - x.n1[j] * c1);
            const float dz = x.g[j] * x.dh[j];
            dg[j] = p.alpha * x.dh[j] * (x.n2[j] * w.post[j]);
            acc[1][j] += dz * x.n2[j];
            acc[2][j] += dg[j];
            x.n2[j] = post ? r2 * (dz * w.post[j] - x.n2[j] * c2) : dz;  // dy
        }
        if (p.out.dh) store_row<kKind>(static_cast<R *>(p.out.dh) + at, c, x.dh);
        if (p.in.y && p.out.dy) store_row<kKind>(static_cast<T *>(p.out.dy) + at, c, x.n2);
        if (kToken && p.out.dgate) store_row<kKind>(static_cast<T *>(p.out.dgate) + at, c, dg);
    }
    const bool last = gridDim.x == 1;  // all rows are here
    float *mine = p.partial + (int64_t)blockIdx.x * 3 * p.dim;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (p.sums.out[k] == nullptr) continue;
        float *sums = last ? static_cast<float *>(p.sums.out[k]) : mine + k * p.dim;
        Bf16 *rounded = static_cast<Bf16 *>(p.sums.out[k]);
        if (groups > 1) {
            const int width = lanes * 8;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) s_cols[group * width + lane * 8 + j] = acc[k][j];
            __syncthreads();
            for (int i = threadIdx.x; i < p.dim; i += blockDim.x) {
                float t = 0.0f;
                for (int q = 0; q < groups; ++q) t += s_cols[q * width + i];
                if (last && p.w_bf16) store1(rounded + i, t);
                else sums[i] = t;
            }
        } else if (last && p.w_bf16) {
            store_cols(rounded, c, acc[k]);
        } else {
            store_cols(sums, c, acc[k]);
        }
    }
}

// Column sums over the workgroups' partial sums: 64 columns a workgroup, four a
// lane, and 64 shares of the rows; blockIdx.y is the gradient.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float *partial, int32_t parts, int32_t dim,
                                                          ColumnOut o, bool bf16) {
    __shared__ float s[64][65];
    const int k = blockIdx.y, c = threadIdx.x % 16 * 4, share = threadIdx.x / 16;
    const int col = blockIdx.x * 64 + c;
    if (o.out[k] == nullptr) return;
    float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const float *src = partial + (int64_t)k * dim + col;
    if (col + 4 <= dim) {
#pragma unroll 4
        for (int i = share; i < parts; i += 64) {
            const f32x4 x = reinterpret_cast<const f32x4_any4 *>(src + (int64_t)i * 3 * dim)->v;
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] += x[j];
        }
    } else {
        for (int i = share; i < parts; i += 64)
            for (int j = 0; j < 4; ++j) t[j] += col + j < dim ? src[(int64_t)i * 3 * dim + j] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) s[share][c + j] = t[j];
    __syncthreads();
    if (threadIdx.x < 64 && blockIdx.x * 64 + (int)threadIdx.x < dim) {
        const int out = blockIdx.x * 64 + threadIdx.x;
        float sum = 0.0f;
        for (int i = 0; i < 64; ++i) sum += s[i][threadIdx.x];
        if (bf16) store1(static_cast<Bf16 *>(o.out[k]) + out, sum);
        else static_cast<float *>(o.out[k])[out] = sum;
    }
}

// Lanes of a row, vectors of a lane, threads of a workgroup, and threads that a CU
// holds of the kernel: up to 512 columns a row is part of a wave and a workgroup takes
// several; above, a workgroup takes one row with as many waves as it needs, one vector a lane up to 8192 columns, two up
// to 16384 and four above, which spill 43 to 85 registers (1024 x 32768 bf16: 84 us,
// its bytes 41; 2048 x 16384 with two, the same bytes: 55).
struct Split {
    int lanes, vec, block, resident;
};
Split split_of(int64_t dim) {
    const int64_t vecs = (dim + 7) / 8;
    if (vecs <= 64) {
        int lanes = 8;
        while (lanes < vecs) lanes *= 2;
        return {lanes, 1, 256, 2048};
    }
    const int vec = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
    const int lanes = (int)((vecs + 64 * vec - 1) / (64 * vec)) * 64;
    return {lanes, vec, lanes, 2048};
}
// The backward pass needs many registers, so its workgroups of up to 512 threads
// have a power of two of waves that the four SIMDs can share evenly (8192 x 2304
// bf16: 53 us with eight waves, 57 with five); above, a CU holds one workgroup and
// idle waves only cost (8192 x 5120 with an fp32 stream: 268 us with sixteen, 230
// with ten). vec: tiles of a row here.
Split backward_split_of(int64_t dim) {
    Split sp = split_of(dim);
    if (sp.lanes > 64) {
        const int64_t vecs = (dim + 7) / 8;
        sp.vec = (int)((vecs + 1023) / 1024);
        sp.lanes = (int)((vecs + 64 * sp.vec - 1) / (64 * sp.vec)) * 64;
        if (sp.lanes < 512) sp.lanes = sp.lanes <= 128 ? 128 : sp.lanes <= 256 ? 256 : 512;
        sp.block = sp.lanes;
    }
    sp.resident = sp.block > 512 ? 1024 : 768;  // three waves a SIMD with up to 167 registers
    return sp;
}

// Workgroups that fill the chip's 256 CUs, as far as there are rows.
int64_t workgroups(int64_t rows, const Split &sp) {
    const int64_t groups = sp.block / sp.lanes, need = (rows + groups - 1) / groups;
    const int64_t most = 256 * (sp.resident / sp.block);
    return need < most ? need : most;
}
// Each workgroup of the backward pass leaves a row of partial sums, so beyond one
// for each CU none takes fewer than two sets of rows (1024 x 2048 bf16: 14 us
// instead of 18). A single one writes the sums itself, and there is no second launch
// (one row of 2048: 16.4 us a call instead of 18.6; with four rows in one workgroup
// a call alone takes longer, 4 x 8192 36 us instead of 31). Tiles of a row fill the
// chip together.
int64_t backward_workgroups(int64_t rows, const Split &sp) {
    const int64_t groups = sp.block / sp.lanes, pairs = (rows + 2 * groups - 1) / (2 * groups);
    const int64_t all = workgroups(rows, sp), one = all < 256 ? all : 256;
    if (sp.vec > 1) return all < 256 / sp.vec ? all : 256 / sp.vec;
    return all < pairs ? all : pairs < one ? one : pairs;
}

NormParams params_of(const nf4_residual_norm_shape &sh, const ResidualNormIn &in, const ResidualNormOut &out,
                     const Split &sp) {
    NormParams p{};
    p.in = in, p.out = out;
    p.rows = sh.rows, p.dim = (int32_t)sh.dim;
    p.inv_dim = 1.0f / (float)sh.dim, p.eps = sh.eps, p.alpha = sh.alpha, p.off = sh.w_offset;
    p.lanes = sp.lanes, p.gate_kind = sh.gate_kind, p.w_bf16 = sh.w_dtype == NF4_BF16;
    return p;
}

template <typename T, typename R, RowKind kKind>
hipError_t forward_kind(const NormParams &p, const Split &sp, hipStream_t s) {
    // What a kind comes with: fewer than eight columns are part of a wave, fours one
    // vector of a whole workgroup, fp32 vectors a part of a wave or several vectors.
    constexpr bool kMany = kKind == kRowAny || kKind == kRowVecs, kPart = kKind != kRowFours;
    constexpr bool kWhole = kKind == kRowFours || kKind == kRowAny || (kKind == kRowVecs && sizeof(R) == 2);
    auto kernel = sp.vec == 4   ? residual_norm_forward_kernel<T, R, kMany ? 4 : 1, kKind, !kPart || kMany>
                  : sp.vec == 2 ? residual_norm_forward_kernel<T, R, kMany ? 2 : 1, kKind, !kPart || kMany>
                  : sp.lanes > 64 ? residual_norm_forward_kernel<T, R, 1, kKind, kWhole>
                                  : residual_norm_forward_kernel<T, R, 1, kKind, !kPart>;
    kernel<<<dim3((uint32_t)workgroups(p.rows, sp)), dim3(sp.block), 0, s>>>(p);
    return hipGetLastError();
}
template <typename T, typename R, RowKind kKind, bool kToken>
hipError_t backward_kind(const NormParams &p, const Split &sp, hipStream_t s) {
    constexpr bool kPart = kKind != kRowFours;
    constexpr bool kWhole = kKind == kRowFours || kKind == kRowAny || (kKind == kRowVecs && sizeof(R) == 2);
    constexpr int kMost = kWhole ? 1024 : 512;
    auto kernel = sp.vec > 1       ? residual_norm_backward_kernel<T, R, kKind, kToken, kWhole, kWhole, kMost>
                  : sp.lanes > 512 ? residual_norm_backward_kernel<T, R, kKind, kToken, kWhole, false, kMost>
                  : sp.lanes > 64  ? residual_norm_backward_kernel<T, R, kKind, kToken, kWhole, false, 512>
                                   : residual_norm_backward_kernel<T, R, kKind, kToken, !kPart, false, 512>;
    if constexpr (kWhole)
        if (sp.vec > 1) {
            const int64_t wgs = p.rows < 512 ? p.rows : 512;
            residual_norm_means_kernel<T, R, kKind, kToken><<<dim3((uint32_t)wgs), dim3(1024), 0, s>>>(p);
        }
    const size_t lds = p.partial && sp.block > sp.lanes ? (size_t)sp.block * 8 * sizeof(float) : 0;
    const dim3 grid((uint32_t)backward_workgroups(p.rows, sp), sp.vec);
    kernel<<<grid, dim3(sp.block), lds, s>>>(p);
    return hipGetLastError();
}
template <typename T, typename R>
hipError_t forward_typed(const NormParams &p, const Split &sp, hipStream_t s) {
    if (p.dim < 8) return forward_kind<T, R, kRowNarrow>(p, sp, s);
    if (p.dim % 8) return forward_kind<T, R, kRowAny>(p, sp, s);
    // not with several vectors of a lane, which spill (1024 x 12288: 45 us instead of 36)
    if constexpr (sizeof(R) == 4)
        if (sp.lanes > 64 && sp.vec == 1) return forward_kind<T, R, kRowFours>(p, sp, s);
    return forward_kind<T, R, kRowVecs>(p, sp, s);
}
template <typename T, typename R, bool kToken>
hipError_t backward_gate(const NormParams &p, const Split &sp, hipStream_t s) {
    if (p.dim < 8) return backward_kind<T, R, kRowNarrow, kToken>(p, sp, s);
    if (p.dim % 8) return backward_kind<T, R, kRowAny, kToken>(p, sp, s);
    if constexpr (sizeof(R) == 4)
        if (sp.lanes > 64) return backward_kind<T, R, kRowFours, kToken>(p, sp, s);
    return backward_kind<T, R, kRowVecs, kToken>(p, sp, s);
}
template <typename T, typename R>
hipError_t backward_typed(const NormParams &p, const Split &sp, hipStream_t s) {
    return p.in.y && p.gate_kind == NF4_GATE_TOKEN ? backward_gate<T, R, true>(p, sp, s) : backward_gate<T, R, false>(p, sp, s);
}

}  // namespace

hipError_t launch_residual_norm_forward(const nf4_residual_norm_shape &sh, const ResidualNormIn &in,
                                        const ResidualNormOut &out, hipStream_t s) {
    const Split sp = split_of(sh.dim);
    const NormParams p = params_of(sh, in, out, sp);
    if (sh.dtype == NF4_F32) return forward_typed<float, float>(p, sp, s);
    if (sh.res_dtype == NF4_F32) return forward_typed<Bf16, float>(p, sp, s);
    return forward_typed<Bf16, Bf16>(p, sp, s);
}

// The means of rows of several tiles, then the partial sums.
size_t means_bytes(const nf4_residual_norm_shape &sh, const Split &sp) {
    return sp.vec > 1 ? ((size_t)sh.rows * sizeof(float2) + 255) / 256 * 256 : 0;
}
size_t residual_norm_workspace(const nf4_residual_norm_shape &sh, bool sums) {
    const Split sp = backward_split_of(sh.dim);
    const size_t partial = (size_t)(backward_workgroups(sh.rows, sp) * 3 * sh.dim) * sizeof(float);
    return means_bytes(sh, sp) + (sums ? partial : 0);
}

hipError_t launch_residual_norm_backward(const nf4_residual_norm_shape &sh, const ResidualNormIn &in,
                                         const ResidualNormOut &out, void *workspace, hipStream_t s) {
    const Split sp = backward_split_of(sh.dim);
    NormParams p = params_of(sh, in, out, sp);
    const int64_t wgs = backward_workgroups(sh.rows, sp);
    const ColumnOut cols{{out.dw_pre, out.dw_post, sh.gate_kind == NF4_GATE_CHANNEL ? out.dgate : nullptr}};
    const bool sums = cols.out[0] || cols.out[1] || cols.out[2];
    float *partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + means_bytes(sh, sp));
    p.partial = sums ? partial : nullptr;
    p.sums = cols;
    p.means = static_cast<float2 *>(workspace);
    if (wgs > 0) {
        hipError_t e;
        if (sh.dtype == NF4_F32) e = backward_typed<float, float>(p, sp, s);
        else if (sh.res_dtype == NF4_F32) e = backward_typed<Bf16, float>(p, sp, s);
        else e = backward_typed<Bf16, Bf16>(p, sp, s);
        if (e != hipSuccess) return e;
    }
    if (!sums || wgs == 1) return hipSuccess;
    column_sum_kernel<<<dim3((uint32_t)((sh.dim + 63) / 64), 3), dim3(1024), 0, s>>>(partial, (int32_t)wgs,
                                                                                     (int32_t)sh.dim, cols, p.w_bf16);
    return hipGetLastError();
}

}  // namespace nf4
