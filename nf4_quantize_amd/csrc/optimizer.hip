// optimizer.hip - AdamW over a list of tensors and the global norm of their
// gradients for gfx950. The step's formulas, the 8-bit storage of the moments
// and the random bits are defined in nf4.h (nf4_adamw_entry).
//
// Both are bound by HBM: a step reads and writes every weight and moment once
// and reads every gradient once, 10.06 bytes an element for bf16 weights and
// gradients with 8-bit moments, 30 with 32-bit moments, fp32 gradients and a
// master weight.
#pragma clang fp contract(off)

#include <math.h>

#include "training_internal.h"

namespace nf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kEach = 8;                   // elements of a thread in one pass
constexpr int kPass = kThreads * kEach;    // 2048 elements: 8 moment blocks
constexpr int kBatch = 48;                 // entries per launch: 3.9 KB of kernel arguments
constexpr float kScaleMin = 0x1p-126f;     // the smallest scale whose reciprocal is finite
constexpr float kE4m3Max = 448.0f;
constexpr float kE4m3Min = 0x1p-9f;

__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    x ^= x >> 16;
    return x;
}
constexpr uint32_t kWeyl = 0x9E3779B9u;

struct AdamwBatch {
    void *w[kBatch];
    float *master[kBatch];
    const void *g[kBatch];
    void *m[kBatch];
    void *v[kBatch];
    float *ms[kBatch];
    float *vs[kBatch];
    int64_t n[kBatch];
    float step[kBatch];   // lr / (1 - beta1^t)
    float keep[kBatch];   // 1 - lr weight_decay
    uint32_t key[kBatch];
    uint32_t first[kBatch];  // the entry's first workgroup in the launch
};
struct AdamwScalars {
    float beta1, one_beta1, beta2, one_beta2, eps, rbias2, max_norm;
    int32_t passes;  // passes of kPass elements of a workgroup
    const float *norm;
};
static_assert(sizeof(AdamwBatch) + sizeof(AdamwScalars) <= 4096, "kernel arguments");

// The entry of workgroup wg: the last one whose first workgroup is not above it.
template <int N>
__device__ __forceinline__ int find_entry(const uint32_t (&first)[N], uint32_t wg) {
    int k = 0;
#pragma unroll
    for (int j = 1; j < N; ++j) k = (wg >= first[j]) ? j : k;
    return k;
}


// Stochastic rounding of four values to packed E4M3 codes: gfx950's conversion
// adds the top 20 random bits below the kept mantissa bits and cuts (subnormal
// codes on their uniform grid).
__device__ __forceinline__ uint32_t pack_e4m3_sr(const float *t, const uint32_t *r) {
    int c = 0;
    c = __builtin_amdgcn_cvt_sr_fp8_f32(t[0], (int)r[0], c, 0);
    c = __builtin_amdgcn_cvt_sr_fp8_f32(t[1], (int)r[1], c, 1);
    c = __builtin_amdgcn_cvt_sr_fp8_f32(t[2], (int)r[2], c, 2);
    c = __builtin_amdgcn_cvt_sr_fp8_f32(t[3], (int)r[3], c, 3);
    return (uint32_t)c;
}
__device__ __forceinline__ void unpack_e4m3(uint32_t c, float scale, float *x) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    x[0] = lo[0] * scale, x[1] = lo[1] * scale, x[2] = hi[0] * scale, x[3] = hi[1] * scale;
}

// Scale of a block's storage and its reciprocal.
__device__ __forceinline__ float storage_scale(float amax, float *inv) {
    float s = amax * (1.0f / kE4m3Max);
    s = s < kScaleMin ? 0.0f : s;
    *inv = s > 0.0f ? 1.0f / s : 0.0f;
    return s;
}

// One workgroup: passes x 2048 consecutive elements of one entry. A half-wave
// holds one block of 256, eight elements a lane, so the block's maximum is a
// reduction over 32 lanes in registers and every byte is moved once.
template <typename W, typename G, bool kMaster, bool kEight>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwBatch b, AdamwScalars c) {
    float clip = 1.0f;
    if (c.norm != nullptr) {
        const float norm = *c.norm;
        if (!(fabsf(norm) < INFINITY)) return;
        if (c.max_norm > 0.0f && norm > c.max_norm) clip = c.max_norm * (1.0f / norm);
    }
    const int k = find_entry(b.first, blockIdx.x);
    const int64_t n = b.n[k];
    W *w = static_cast<W *>(b.w[k]);
    float *master = b.master[k];
    const G *g = static_cast<const G *>(b.g[k]);
    const float step = b.step[k], keep = b.keep[k];
    const uint32_t key = b.key[k];
    const int64_t begin = (int64_t)(blockIdx.x - b.first[k]) * c.passes * kPass;

    for (int p = 0; p < c.passes; ++p) {
        const int64_t base = begin + (int64_t)p * kPass;
        if (base >= n) return;
        const int64_t i = base + threadIdx.x * kEach;
        const int64_t live = n - i;  // may be <= 0: the lane still joins the reductions
        float x[8], gr[8], m[8], v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = gr[j] = m[j] = v[j] = 0.0f;
        if (live > 0) {
            if constexpr (kMaster) load_upto8(master + i, live, x);
            else load_upto8(w + i, live, x);
            load_upto8(g + i, live, gr);
            if constexpr (kEight) {
                const uint8_t *mq = static_cast<const uint8_t *>(b.m[k]) + i;
                const uint8_t *vq = static_cast<const uint8_t *>(b.v[k]) + i;
                const float ms = b.ms[k][i / kMomentBlock], vs = b.vs[k][i / kMomentBlock];
                uint32_t mw[2] = {0u, 0u}, vw[2] = {0u, 0u};
                if (live >= 8) {
                    const uint2 a = *reinterpret_cast<const uint2 *>(mq);
                    const uint2 d = *reinterpret_cast<const uint2 *>(vq);
                    mw[0] = a.x, mw[1] = a.y, vw[0] = d.x, vw[1] = d.y;
                } else {
                    for (int j = 0; j < (int)live; ++j) {
                        mw[j / 4] |= (uint32_t)mq[j] << (8 * (j % 4));
                        vw[j / 4] |= (uint32_t)vq[j] << (8 * (j % 4));
                    }
                }
                unpack_e4m3(mw[0], ms, m), unpack_e4m3(mw[1], ms, m + 4);
                unpack_e4m3(vw[0], vs, v), unpack_e4m3(vw[1], vs, v + 4);
            } else {
                load_upto8(static_cast<const float *>(b.m[k]) + i, live, m);
                load_upto8(static_cast<const float *>(b.v[k]) + i, live, v);
            }
        }
        float ma = 0.0f, va = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float gj = gr[j] * clip;
            // product by product, without contraction: the stored codes follow
            // from these fp32 values to the bit
            m[j] = c.beta1 * m[j] + c.one_beta1 * gj;
            v[j] = c.beta2 * v[j] + c.one_beta2 * (gj * gj);
            // the hardware's reciprocal and root are within 1 ulp: the step is
            // a small part of the weight it is added to
            const float d = __builtin_amdgcn_sqrtf(v[j] * c.rbias2) + c.eps;
            x[j] = fmaf(-step * m[j], __builtin_amdgcn_rcpf(d), x[j] * keep);
            ma = fmaxf(ma, fabsf(m[j])), va = fmaxf(va, v[j]);
        }
        if (live > 0) {
            if constexpr (kMaster) store_upto8(master + i, live, x);
            store_upto8(w + i, live, x);
        }
        if constexpr (kEight) {
            float rm, rv;
            const float ms = storage_scale(max32(ma), &rm);
            const float vs = storage_scale(max32(va), &rv);
            uint32_t rndm[8], rndv[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t r = mix((uint32_t)i * kWeyl + key + (uint32_t)j * kWeyl);
                rndm[j] = r & 0xFFFF0000u, rndv[j] = r << 16;
                m[j] = fminf(fmaxf(m[j] * rm, -kE4m3Max), kE4m3Max);
                v[j] = fminf(fmaxf(v[j] * rv, kE4m3Min), kE4m3Max);
            }
            if (live > 0) {
                uint8_t *mq = static_cast<uint8_t *>(b.m[k]) + i;
                uint8_t *vq = static_cast<uint8_t *>(b.v[k]) + i;
                const uint32_t mw[2] = {pack_e4m3_sr(m, rndm), pack_e4m3_sr(m + 4, rndm + 4)};
                const uint32_t vw[2] = {pack_e4m3_sr(v, rndv), pack_e4m3_sr(v + 4, rndv + 4)};
                if (live >= 8) {
                    *reinterpret_cast<uint2 *>(mq) = make_uint2(mw[0], mw[1]);
                    *reinterpret_cast<uint2 *>(vq) = make_uint2(vw[0], vw[1]);
                } else {
                    for (int j = 0; j < (int)live; ++j) {
                        mq[j] = (uint8_t)(mw[j / 4] >> (8 * (j % 4)));
                        vq[j] = (uint8_t)(vw[j / 4] >> (8 * (j % 4)));
                    }
                }
                if (threadIdx.x % 32 == 0) {
                    b.ms[k][i / kMomentBlock] = ms;
                    b.vs[k][i / kMomentBlock] = vs;
                }
            }
        } else if (live > 0) {
            store_upto8(static_cast<float *>(b.m[k]) + i, live, m);
            store_upto8(static_cast<float *>(b.v[k]) + i, live, v);
        }
    }
}

// ---- the gradients' norm ----

constexpr int kNormBatch = 128;
constexpr int64_t kNormChunk = 16384;  // elements of one partial sum

struct NormBatch {
    const void *g[kNormBatch];
    int64_t n[kNormBatch];
    uint32_t first[kNormBatch];
};
static_assert(sizeof(NormBatch) <= 4000, "kernel arguments");

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
    return x;
}

// Sum over the workgroup, in thread 0.
template <int kN>
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double part[kN / 64];
    x = wave_sum(x);
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = x;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int j = 0; j < kN / 64; ++j) t += part[j];
    return t;
}

// Squares of 16384 consecutive gradients, each exact in fp64.
template <typename G>
__global__ __launch_bounds__(kThreads) void grad_square_kernel(NormBatch b, double *partial) {
    const int k = find_entry(b.first, blockIdx.x);
    const int64_t n = b.n[k];
    const G *g = static_cast<const G *>(b.g[k]);
    const int64_t begin = (int64_t)(blockIdx.x - b.first[k]) * kNormChunk;
    const int64_t end = begin + kNormChunk < n ? begin + kNormChunk : n;
    double sum = 0.0;
    for (int64_t i = begin + threadIdx.x * kEach; i < end; i += kPass) {
        float x[8];
        load_upto8(g + i, end - i, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += (double)x[j] * (double)x[j];
    }
    sum = block_sum<kThreads>(sum);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__global__ __launch_bounds__(1024) void grad_norm_kernel(const double *partial, int64_t count, float *norm) {
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += 1024) sum += partial[i];
    sum = block_sum<1024>(sum);
    if (threadIdx.x == 0) *norm = (float)sqrt(sum);
}

int64_t norm_partials(const nf4_adamw_entry *e, int32_t count) {
    int64_t p = 0;
    for (int32_t i = 0; i < count; ++i) p += (e[i].n + kNormChunk - 1) / kNormChunk;
    return p;
}

template <typename W, typename G, bool kMaster, bool kEight>
hipError_t adamw_launches(const nf4_adamw_entry *e, int32_t count, const nf4_adamw_config &cfg,
                          const float *norm, hipStream_t s) {
    const double bias1 = 1.0 - pow(cfg.beta1, (double)cfg.step);
    const double bias2 = 1.0 - pow(cfg.beta2, (double)cfg.step);
    AdamwScalars c{};
    c.beta1 = (float)cfg.beta1, c.one_beta1 = (float)(1.0 - cfg.beta1);
    c.beta2 = (float)cfg.beta2, c.one_beta2 = (float)(1.0 - cfg.beta2);
    c.eps = cfg.eps, c.rbias2 = (float)(1.0 / bias2);
    c.max_norm = cfg.max_norm, c.norm = norm;
    int64_t total = 0;
    for (int32_t i = 0; i < count; ++i) total += (e[i].n + kPass - 1) / kPass;
    c.passes = 1;
    AdamwBatch b{};
    int used = 0;
    int64_t wgs = 0;
    hipError_t err = hipSuccess;
    auto flush = [&] {
        if (used == 0) return;
        for (int j = used; j < kBatch; ++j) b.first[j] = UINT32_MAX;
        adamw_kernel<W, G, kMaster, kEight><<<dim3((uint32_t)wgs), dim3(kThreads), 0, s>>>(b, c);
        const hipError_t r = hipGetLastError();
        if (err == hipSuccess) err = r;
        used = 0, wgs = 0;
    };
    constexpr int64_t kMaxWgs = (int64_t(1) << 31) / kThreads;
    for (int32_t i = 0; i < count; ++i) {
        if (e[i].n == 0) continue;
        if ((e[i].master != nullptr) != kMaster) continue;
        const int64_t need = (e[i].n + (int64_t)c.passes * kPass - 1) / ((int64_t)c.passes * kPass);
        if (used == kBatch || wgs + need > kMaxWgs) flush();
        b.w[used] = e[i].w, b.master[used] = e[i].master, b.g[used] = e[i].grad;
        b.m[used] = e[i].m, b.v[used] = e[i].v, b.ms[used] = e[i].m_scale, b.vs[used] = e[i].v_scale;
        b.n[used] = e[i].n;
        b.step[used] = (float)((double)e[i].lr / bias1);
        b.keep[used] = (float)(1.0 - (double)e[i].lr * (double)e[i].weight_decay);
        b.key[used] = mix(mix((uint32_t)i * kWeyl + (uint32_t)(cfg.seed >> 32)) + (uint32_t)cfg.seed);
        b.first[used] = (uint32_t)wgs;
        wgs += need;
        ++used;
    }
    flush();
    return err;
}

template <typename W, typename G>
hipError_t adamw_typed(const nf4_adamw_entry *e, int32_t count, bool eight, const nf4_adamw_config &c,
                       const float *norm, hipStream_t s) {
    hipError_t err = eight ? adamw_launches<W, G, false, true>(e, count, c, norm, s)
                           : adamw_launches<W, G, false, false>(e, count, c, norm, s);
    if constexpr (sizeof(W) == 2) {
        const hipError_t r = eight ? adamw_launches<W, G, true, true>(e, count, c, norm, s)
                                   : adamw_launches<W, G, true, false>(e, count, c, norm, s);
        if (err == hipSuccess) err = r;
    }
    return err;
}

}  // namespace

size_t grad_norm_workspace(const nf4_adamw_entry *e, int32_t count) {
    return (size_t)norm_partials(e, count) * sizeof(double);
}

hipError_t launch_grad_norm(const nf4_adamw_entry *e, int32_t count, nf4_dtype gt, float *norm,
                            void *workspace, hipStream_t s) {
    double *partial = static_cast<double *>(workspace);
    NormBatch b{};
    int used = 0;
    int64_t wgs = 0, done = 0;
    hipError_t err = hipSuccess;
    auto flush = [&] {
        if (used == 0) return;
        for (int j = used; j < kNormBatch; ++j) b.first[j] = UINT32_MAX;
        if (gt == NF4_BF16)
            grad_square_kernel<Bf16><<<dim3((uint32_t)wgs), dim3(kThreads), 0, s>>>(b, partial + done);
        else
            grad_square_kernel<float><<<dim3((uint32_t)wgs), dim3(kThreads), 0, s>>>(b, partial + done);
        const hipError_t r = hipGetLastError();
        if (err == hipSuccess) err = r;
        done += wgs, used = 0, wgs = 0;
    };
    constexpr int64_t kMaxWgs = (int64_t(1) << 31) / kThreads;
    for (int32_t i = 0; i < count; ++i) {
        if (e[i].n == 0) continue;
        const int64_t need = (e[i].n + kNormChunk - 1) / kNormChunk;
        if (used == kNormBatch || wgs + need > kMaxWgs) flush();
        b.g[used] = e[i].grad, b.n[used] = e[i].n, b.first[used] = (uint32_t)wgs;
        wgs += need;
        ++used;
    }
    flush();
    grad_norm_kernel<<<dim3(1), dim3(1024), 0, s>>>(partial, done, norm);
    const hipError_t r = hipGetLastError();
    return err == hipSuccess ? r : err;
}

hipError_t launch_adamw(const nf4_adamw_entry *e, int32_t count, nf4_dtype wt, nf4_dtype gt,
                        bool eight, const nf4_adamw_config &c, const float *norm, hipStream_t s) {
    if (wt == NF4_BF16)
        return gt == NF4_BF16 ? adamw_typed<Bf16, Bf16>(e, count, eight, c, norm, s)
                              : adamw_typed<Bf16, float>(e, count, eight, c, norm, s);
    return gt == NF4_BF16 ? adamw_typed<float, Bf16>(e, count, eight, c, norm, s)
                          : adamw_typed<float, float>(e, count, eight, c, norm, s);
}

}  // namespace nf4
