// residual_norm.hip - the residual step between two blocks for gfx950: the
// norm after a block, its gate and residual scale, the residual addition and
// the norm before the next block in one pass over each row, and the backward
// pass of all of them. The formulas are in nf4.h
// (nf4_residual_norm_forward, nf4_residual_norm_backward).
//
// Both are bound by HBM: the forward reads y and h and writes h' and x (8 bytes
// an element in bf16), the backward reads dx, dh', y and h' and writes dy and
// dh (12 bytes), and each element is moved once. A row is held in registers by
// a group of lanes, eight consecutive elements a lane and vector.
#include <math.h>

#include "training_internal.h"

namespace nf4 {
namespace {

struct NormParams {
    ResidualNormIn in;
    ResidualNormOut out;
    int64_t rows;
    int32_t dim;
    float inv_dim, eps, alpha, off;
    int32_t lanes;       // lanes of a row: a power of two, 8 .. 1024
    int32_t gate_kind;
    bool w_bf16;
    float *partial;      // backward: [workgroups][3][dim]
};

// Eight weights from column `col` (fp32 or bf16).
__device__ __forceinline__ void load_weight(const void *w, bool bf16, int col, int live, float (&x)[8]) {
    if (bf16) load_upto8(static_cast<const Bf16 *>(w) + col, live, x);
    else load_upto8(static_cast<const float *>(w) + col, live, x);
}

// Sums of kK values over each row's group of lanes, the same bits in every
// lane. Groups of more than a wave meet in `part`, one slot a wave; the caller
// alternates two buffers, so that one barrier a call is enough.
template <int kK>
__device__ __forceinline__ void row_sums(float (&x)[kK], int lanes, float (*part)[kK]) {
#pragma unroll
    for (int k = 0; k < kK; ++k) x[k] = group_sum(x[k], lanes < 64 ? lanes : 64);
    if (lanes <= 64) return;
    const int wave = threadIdx.x / 64, waves = lanes / 64, first = wave / waves * waves;
    if (threadIdx.x % 64 == 0)
#pragma unroll
        for (int k = 0; k < kK; ++k) part[wave][k] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kK; ++k) {
        float t = 0.0f;
        for (int j = 0; j < waves; ++j) t += part[first + j][k];
        x[k] = t;
    }
}

template <typename T, typename R, int kVec>
__global__ __launch_bounds__(1024) void residual_norm_forward_kernel(NormParams p) {
    __shared__ float part[2][16][1];
    const int lane = threadIdx.x & (p.lanes - 1), groups = blockDim.x / p.lanes;
    const T *y = static_cast<const T *>(p.in.y);
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < p.rows; r0 += (int64_t)gridDim.x * groups) {
        const int64_t row = r0 + threadIdx.x / p.lanes, at = row * p.dim;
        const bool live_row = row < p.rows;
        float h[kVec][8], z[kVec][8];
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const int col = (v * p.lanes + lane) * 8, live = live_row ? p.dim - col : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) h[v][j] = z[v][j] = 0.0f;
            if (live > 0) {
                load_upto8(static_cast<const R *>(p.in.h) + at + col, live, h[v]);
                if (y) load_upto8(y + at + col, live, z[v]);
            }
        }
        if (y) {
            float r2 = 1.0f;
            if (p.in.w_post) {
                float s[1] = {0.0f};
#pragma unroll
                for (int v = 0; v < kVec; ++v)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[0] += z[v][j] * z[v][j];
                row_sums<1>(s, p.lanes, part[turn]);
                turn ^= 1;
                r2 = 1.0f / sqrtf(s[0] * p.inv_dim + p.eps);
                if (live_row && lane == 0 && p.out.rstd_post) p.out.rstd_post[row] = r2;
            }
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                const int col = (v * p.lanes + lane) * 8, live = live_row ? p.dim - col : 0;
                if (live <= 0) continue;
                float w[8];
                if (p.in.w_post) {
                    load_weight(p.in.w_post, p.w_bf16, col, live, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[v][j] *= r2 * (w[j] + p.off);
                }
                if (p.gate_kind != NF4_GATE_NONE) {
                    if (p.gate_kind == NF4_GATE_CHANNEL) load_weight(p.in.gate, p.w_bf16, col, live, w);
                    else load_upto8(static_cast<const T *>(p.in.gate) + at + col, live, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[v][j] *= w[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) h[v][j] += p.alpha * z[v][j];
                store_upto8(static_cast<R *>(p.out.h) + at + col, live, h[v]);
            }
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += h[v][j] * h[v][j];
        row_sums<1>(s, p.lanes, part[turn]);
        turn ^= 1;
        const float r1 = 1.0f / sqrtf(s[0] * p.inv_dim + p.eps);
        if (live_row && lane == 0 && p.out.rstd_pre) p.out.rstd_pre[row] = r1;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const int col = (v * p.lanes + lane) * 8, live = live_row ? p.dim - col : 0;
            if (live <= 0) continue;
            float w[8];
            load_weight(p.in.w_pre, p.w_bf16, col, live, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = h[v][j] * (r1 * (w[j] + p.off));
            store_upto8(static_cast<T *>(p.out.x) + at + col, live, w);
        }
    }
}

// Each workgroup takes every gridDim.x-th set of rows and keeps its columns'
// share of the weights' gradients in registers until its last row.
//
// One round of sums serves both norms: with e = alpha gate w_post' n2 the inner
// product of the second, mean(dz w_post' n2), is mean(e dh), and dh is known up
// to the first one's mean c1 = mean(dx w_pre' n1):
//   sum e dh = sum e (dh_out + rstd_pre dx w_pre') - rstd_pre c1 sum e n1.
template <typename T, typename R, int kVec>
__global__ __launch_bounds__(1024) void residual_norm_backward_kernel(NormParams p) {
    __shared__ float part[2][16][3];
    extern __shared__ float s_cols[];
    const int lanes = p.lanes, groups = blockDim.x / lanes;
    const int lane = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes;
    const T *y = static_cast<const T *>(p.in.y);
    const T *dx = static_cast<const T *>(p.in.dx);
    const R *dho = static_cast<const R *>(p.in.dh_out);
    float acc[3][kVec][8];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[k][v][j] = 0.0f;

    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < p.rows; r0 += (int64_t)gridDim.x * groups, turn ^= 1) {
        const int64_t row = r0 + group, at = row * p.dim;
        const bool live_row = row < p.rows;
        const float r1 = live_row ? p.in.rstd_pre[row] : 0.0f;
        const float r2 = live_row && y && p.in.w_post ? p.in.rstd_post[row] : 1.0f;
        float vdx[kVec][8], vh[kVec][8], vdh[kVec][8], vy[kVec][8], w1[kVec][8], w2[kVec][8], g[kVec][8];
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const int col = (v * lanes + lane) * 8, live = live_row ? p.dim - col : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                vdx[v][j] = vh[v][j] = vdh[v][j] = vy[v][j] = w1[v][j] = w2[v][j] = g[v][j] = 0.0f;
            if (live > 0) {
                load_upto8(static_cast<const R *>(p.in.h) + at + col, live, vh[v]);
                if (dx) load_upto8(dx + at + col, live, vdx[v]);
                if (dho) load_upto8(dho + at + col, live, vdh[v]);
                load_weight(p.in.w_pre, p.w_bf16, col, live, w1[v]);
                if (y) {
                    load_upto8(y + at + col, live, vy[v]);
                    if (p.in.w_post) load_weight(p.in.w_post, p.w_bf16, col, live, w2[v]);
                    if (p.gate_kind == NF4_GATE_CHANNEL) load_weight(p.in.gate, p.w_bf16, col, live, g[v]);
                    if (p.gate_kind == NF4_GATE_TOKEN)
                        load_upto8(static_cast<const T *>(p.in.gate) + at + col, live, g[v]);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                w1[v][j] += p.off;
                w2[v][j] = p.in.w_post ? w2[v][j] + p.off : 1.0f;
                g[v][j] = p.gate_kind == NF4_GATE_NONE ? p.alpha : g[v][j] * p.alpha;
                vh[v][j] *= r1;   // n1
                vy[v][j] *= r2;   // n2
                const float q = vdx[v][j] * w1[v][j], e = g[v][j] * w2[v][j] * vy[v][j];
                s[0] += q * vh[v][j];
                s[1] += e * (vdh[v][j] + r1 * q);
                s[2] += e * vh[v][j];
            }
        }
        row_sums<3>(s, lanes, part[turn]);
        const float c1 = s[0] * p.inv_dim;
        const float c2 = (s[1] - r1 * c1 * s[2]) * p.inv_dim;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const int col = (v * lanes + lane) * 8, live = live_row ? p.dim - col : 0;
            if (live <= 0) continue;
            float dh[8], dy[8], dg[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dh[j] = vdh[v][j] + r1 * (vdx[v][j] * w1[v][j] - vh[v][j] * c1);
                const float dz = g[v][j] * dh[j];
                dy[j] = p.in.w_post ? r2 * (dz * w2[v][j] - vy[v][j] * c2) : dz;
                dg[j] = p.alpha * dh[j] * (vy[v][j] * w2[v][j]);
                acc[0][v][j] += vdx[v][j] * vh[v][j];
                acc[1][v][j] += dz * vy[v][j];
                acc[2][v][j] += dg[j];
            }
            if (p.out.dh) store_upto8(static_cast<R *>(p.out.dh) + at + col, live, dh);
            if (y) {
                if (p.out.dy) store_upto8(static_cast<T *>(p.out.dy) + at + col, live, dy);
                if (p.out.dgate && p.gate_kind == NF4_GATE_TOKEN)
                    store_upto8(static_cast<T *>(p.out.dgate) + at + col, live, dg);
            }
        }
    }
    if (p.partial == nullptr) return;
    float *mine = p.partial + (int64_t)blockIdx.x * 3 * p.dim;
    const int width = lanes * kVec * 8;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (groups > 1) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < kVec; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) s_cols[group * width + (v * lanes + lane) * 8 + j] = acc[k][v][j];
            __syncthreads();
            for (int c = threadIdx.x; c < p.dim; c += blockDim.x) {
                float t = 0.0f;
                for (int q = 0; q < groups; ++q) t += s_cols[q * width + c];
                mine[k * p.dim + c] = t;
            }
        } else {
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                const int col = (v * lanes + lane) * 8;
                if (p.dim - col > 0) store_upto8(mine + k * p.dim + col, p.dim - col, acc[k][v]);
            }
        }
    }
}

// Column sums over the workgroups' partial sums: 16 columns x 16 shares of the
// rows a workgroup; blockIdx.y is the gradient.
struct ColumnOut {
    void *out[3];
};
__global__ __launch_bounds__(256) void column_sum_kernel(const float *partial, int32_t parts, int32_t dim,
                                                         ColumnOut o, bool bf16) {
    __shared__ float s[16][16];
    const int k = blockIdx.y, c = threadIdx.x % 16, share = threadIdx.x / 16;
    const int col = blockIdx.x * 16 + c;
    if (o.out[k] == nullptr) return;
    float t = 0.0f;
    if (col < dim)
        for (int i = share; i < parts; i += 16) t += partial[((int64_t)i * 3 + k) * dim + col];
    s[share][c] = t;
    __syncthreads();
    if (share == 0 && col < dim) {
        t = 0.0f;
        for (int i = 0; i < 16; ++i) t += s[i][c];
        if (bf16) store1(static_cast<Bf16 *>(o.out[k]) + col, t);
        else static_cast<float *>(o.out[k])[col] = t;
    }
}

constexpr int64_t kMostWgs = int64_t(1) << 20;  // of a launch; more rows go round

// Lanes of a row and vectors of a lane.
struct Split {
    int lanes, vec;
};
Split split_of(int64_t dim) {
    const int64_t vecs = (dim + 7) / 8;
    int lanes = 8;
    while (lanes < 1024 && lanes < vecs) lanes *= 2;
    int vec = 1;
    while ((int64_t)lanes * vec < vecs) vec *= 2;
    return {lanes, vec};
}
int block_of(const Split &sp) { return sp.lanes < 256 ? 256 : sp.lanes; }

// Workgroups of the backward pass: as many as fill the chip's 256 CUs with
// 1024 threads each.
int64_t backward_workgroups(int64_t rows, const Split &sp) {
    const int64_t groups = block_of(sp) / sp.lanes, most = 256 * (1024 / block_of(sp));
    const int64_t need = (rows + groups - 1) / groups;
    return need < most ? need : most;
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

template <typename T, typename R>
hipError_t forward_typed(const NormParams &p, const Split &sp, hipStream_t s) {
    const int block = block_of(sp), groups = block / sp.lanes;
    const int64_t need = (p.rows + groups - 1) / groups;
    const dim3 grid((uint32_t)(need < kMostWgs ? need : kMostWgs));
    switch (sp.vec) {
        case 1: residual_norm_forward_kernel<T, R, 1><<<grid, dim3(block), 0, s>>>(p); break;
        case 2: residual_norm_forward_kernel<T, R, 2><<<grid, dim3(block), 0, s>>>(p); break;
        default: residual_norm_forward_kernel<T, R, 4><<<grid, dim3(block), 0, s>>>(p); break;
    }
    return hipGetLastError();
}

template <typename T, typename R>
hipError_t backward_typed(const NormParams &p, const Split &sp, int64_t wgs, hipStream_t s) {
    const int block = block_of(sp);
    const size_t lds = p.partial && block > sp.lanes ? (size_t)block * sp.vec * 8 * sizeof(float) : 0;
    const dim3 grid((uint32_t)wgs);
    switch (sp.vec) {
        case 1: residual_norm_backward_kernel<T, R, 1><<<grid, dim3(block), lds, s>>>(p); break;
        case 2: residual_norm_backward_kernel<T, R, 2><<<grid, dim3(block), lds, s>>>(p); break;
        default: residual_norm_backward_kernel<T, R, 4><<<grid, dim3(block), lds, s>>>(p); break;
    }
    return hipGetLastError();
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

size_t residual_norm_workspace(const nf4_residual_norm_shape &sh) {
    return (size_t)(backward_workgroups(sh.rows, split_of(sh.dim)) * 3 * sh.dim) * sizeof(float);
}

hipError_t launch_residual_norm_backward(const nf4_residual_norm_shape &sh, const ResidualNormIn &in,
                                         const ResidualNormOut &out, void *workspace, hipStream_t s) {
    const Split sp = split_of(sh.dim);
    NormParams p = params_of(sh, in, out, sp);
    const int64_t wgs = backward_workgroups(sh.rows, sp);
    const ColumnOut cols{{out.dw_pre, out.dw_post, sh.gate_kind == NF4_GATE_CHANNEL ? out.dgate : nullptr}};
    const bool sums = cols.out[0] || cols.out[1] || cols.out[2];
    p.partial = sums ? static_cast<float *>(workspace) : nullptr;
    if (wgs > 0) {
        hipError_t e;
        if (sh.dtype == NF4_F32) e = backward_typed<float, float>(p, sp, wgs, s);
        else if (sh.res_dtype == NF4_F32) e = backward_typed<Bf16, float>(p, sp, wgs, s);
        else e = backward_typed<Bf16, Bf16>(p, sp, wgs, s);
        if (e != hipSuccess) return e;
    }
    if (!sums) return hipSuccess;
    column_sum_kernel<<<dim3((uint32_t)((sh.dim + 15) / 16), 3), dim3(256), 0, s>>>(
        static_cast<const float *>(workspace), (int32_t)wgs, (int32_t)sh.dim, cols, p.w_bf16);
    return hipGetLastError();
}

}  // namespace nf4
