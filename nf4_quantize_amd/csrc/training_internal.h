// training_internal.h - internal declarations of the training-step operators
// (optimizer.hip, residual_norm.hip, embedding.hip); their contracts are in
// nf4.h. Shared by the library's own sources only.
#pragma once

#include "nf4_internal.h"

namespace nf4 {

constexpr int kMomentBlock = 256;  // elements per scale of the 8-bit moments

// Host-side launchers; each validates nothing.
size_t grad_norm_workspace(const nf4_adamw_entry *e, int32_t count);
hipError_t launch_grad_norm(const nf4_adamw_entry *e, int32_t count, nf4_dtype gt, float *norm,
                            void *workspace, hipStream_t s);
// own_norm: takes the gradients' norm first, into `norm`.
hipError_t launch_adamw(const nf4_adamw_entry *e, int32_t count, nf4_dtype wt, nf4_dtype gt,
                        bool eight, const nf4_adamw_config &c, float *norm, bool own_norm,
                        void *workspace, hipStream_t s);
size_t adamw_workspace(int32_t count);

struct ResidualNormIn {
    const void *dx, *dh_out;  // backward only
    const void *y, *h;        // h: the input (forward), the output (backward)
    const void *w_post, *gate, *w_pre;
    const float *rstd_post, *rstd_pre;  // backward only
};
struct ResidualNormOut {
    void *h, *x;                   // forward
    float *rstd_post, *rstd_pre;   // forward
    void *dy, *dh, *dgate, *dw_pre, *dw_post;  // backward
};
hipError_t launch_residual_norm_forward(const nf4_residual_norm_shape &sh, const ResidualNormIn &in,
                                        const ResidualNormOut &out, hipStream_t s);
// `sums`: whether a gradient that is summed over the rows is asked for.
size_t residual_norm_workspace(const nf4_residual_norm_shape &sh, bool sums);
hipError_t launch_residual_norm_backward(const nf4_residual_norm_shape &sh, const ResidualNormIn &in,
                                         const ResidualNormOut &out, void *workspace, hipStream_t s);

hipError_t launch_embedding_forward(const void *ids, bool i64, int64_t tokens, const void *table,
                                    nf4_dtype dt, int64_t vocab, int64_t dim, float scale, void *out,
                                    nf4_dtype ot, hipStream_t s);
hipError_t launch_embedding_packed(const void *ids, bool i64, int64_t tokens, const nf4_weight &w,
                                   float scale, void *out, nf4_dtype ot, hipStream_t s);
size_t embedding_backward_workspace(int64_t tokens, int64_t vocab, int64_t dim);
hipError_t launch_embedding_backward(const void *ids, bool i64, int64_t tokens, const void *dy,
                                     nf4_dtype dt, int64_t vocab, int64_t dim, float scale,
                                     int64_t padding_id, void *grad, nf4_dtype gt, bool accumulate,
                                     void *workspace, hipStream_t s);

// ---- device helpers ----

// Eight consecutive elements of a row that may start at any element: bf16 rows
// of odd width put 16-byte groups at 2-byte boundaries, which the global
// memory path of gfx950 takes in one instruction.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
struct __attribute__((packed, aligned(2))) u32x4_any2 { u32x4 v; };
struct __attribute__((packed, aligned(4))) f32x4_any4 { f32x4 v; };

struct Bf16 {
    uint16_t bits;
};

__device__ __forceinline__ void load8(const Bf16 *p, float (&x)[8]) {
    const u32x4 r = reinterpret_cast<const u32x4_any2 *>(p)->v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf16_lo(r[j]);
        x[2 * j + 1] = bf16_hi(r[j]);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const f32x4 a = reinterpret_cast<const f32x4_any4 *>(p)->v;
    const f32x4 b = reinterpret_cast<const f32x4_any4 *>(p + 4)->v;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = a[j], x[4 + j] = b[j];
}
__device__ __forceinline__ void store8(Bf16 *p, const float (&x)[8]) {
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
    reinterpret_cast<u32x4_any2 *>(p)->v = r;
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    reinterpret_cast<f32x4_any4 *>(p)->v = f32x4{x[0], x[1], x[2], x[3]};
    reinterpret_cast<f32x4_any4 *>(p + 4)->v = f32x4{x[4], x[5], x[6], x[7]};
}
__device__ __forceinline__ float load1(const Bf16 *p) { return bf16_lo(p->bits); }
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ void store1(Bf16 *p, float x) {
    p->bits = (uint16_t)(pack_bf16x2(x, 0.0f) & 0xFFFFu);
}
__device__ __forceinline__ void store1(float *p, float x) { *p = x; }

// The first `live` (1 .. 8) of the eight; the others are zero / not written.
template <typename T>
__device__ __forceinline__ void load_upto8(const T *p, int64_t live, float (&x)[8]) {
    if (live >= 8) return load8(p, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j < live ? load1(p + j) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void store_upto8(T *p, int64_t live, const float (&x)[8]) {
    if (live >= 8) return store8(p, x);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < live) store1(p + j, x[j]);
}

// Eight elements as they lie in memory, and their values. Loads are kept apart
// from the conversions so that several can be in flight.
template <typename T> struct Raw8;
template <> struct Raw8<Bf16> {
    u32x4 v;
};
template <> struct Raw8<float> {
    f32x4 a, b;
};
__device__ __forceinline__ Raw8<Bf16> load_raw(const Bf16 *p) {
    return {reinterpret_cast<const u32x4_any2 *>(p)->v};
}
__device__ __forceinline__ Raw8<float> load_raw(const float *p) {
    return {reinterpret_cast<const f32x4_any4 *>(p)->v, reinterpret_cast<const f32x4_any4 *>(p + 4)->v};
}
// The same past the caches' usual order: for data that is not read again soon.
// Loads are of 16-byte aligned addresses; stores take any element's.
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));
__device__ __forceinline__ Raw8<Bf16> load_stream(const Bf16 *p) {
    return {__builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p))};
}
__device__ __forceinline__ Raw8<float> load_stream(const float *p) {
    return {__builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p)),
            __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p + 4))};
}
__device__ __forceinline__ void store_stream(Bf16 *p, const float (&x)[8]) {
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
    __builtin_nontemporal_store(r, reinterpret_cast<u32x4_at2 *>(p));
}
__device__ __forceinline__ void store_stream(float *p, const float (&x)[8]) {
    __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4_at4 *>(p));
    __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, reinterpret_cast<f32x4_at4 *>(p + 4));
}
__device__ __forceinline__ void values(const Raw8<Bf16> &r, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf16_lo(r.v[j]);
        x[2 * j + 1] = bf16_hi(r.v[j]);
    }
}
__device__ __forceinline__ void values(const Raw8<float> &r, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = r.a[j], x[4 + j] = r.b[j];
}

// The eight columns from `col` of a row of `dim`. Where fewer are left, the
// load takes the row's last eight instead, and the values move down by `shift`
// with zeros above, so that no lane leaves the row and none waits in a branch
// of its own; lanes past the row load the same and get zeros. Rows of fewer
// than eight elements (kNarrow) are loaded one by one.
template <bool kNarrow> struct Cols {
    int dim, col, base, live;
    __device__ __forceinline__ Cols(int c, int d)
        : dim(d), col(c), base(kNarrow ? 0 : (c < d - 8 ? c : d - 8)), live(d - c) {}
};
__device__ __forceinline__ Raw8<Bf16> raw_of(const float (&x)[8], const Bf16 *) {
    Raw8<Bf16> r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
    return r;
}
__device__ __forceinline__ Raw8<float> raw_of(const float (&x)[8], const float *) {
    return {f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]}};
}
template <typename T, bool kNarrow>
__device__ __forceinline__ Raw8<T> load_cols(const T *row, const Cols<kNarrow> &c) {
    if constexpr (!kNarrow) {
        return load_raw(row + (uint32_t)c.base);
    } else {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = j < c.dim ? load1(row + j) : 0.0f;
        return raw_of(x, row);
    }
}
template <typename T, bool kNarrow>
__device__ __forceinline__ void cols_values(const Raw8<T> &r, const Cols<kNarrow> &c, float (&x)[8]) {
    values(r, x);
    if (c.live >= 8) return;  // all lanes of most waves
    const int shift = c.col - c.base;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (shift & o) ? (j + o < 8 ? x[j + o] : 0.0f) : x[j];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = shift >= 8 ? 0.0f : x[j];
}
template <typename T, bool kNarrow>
__device__ __forceinline__ void store_cols(T *row, const Cols<kNarrow> &c, const float (&x)[8]) {
    if (c.live >= 8) return store8(row + (uint32_t)c.col, x);
    if (c.live > 0) store_upto8(row + (uint32_t)c.col, c.live, x);
}

// load_cols and store_cols past the caches' usual order; the load is for rows of
// whole vectors.
template <typename T>
__device__ __forceinline__ Raw8<T> load_stream(const T *row, const Cols<false> &c) {
    return load_stream(row + (uint32_t)c.base);
}
template <typename T, bool kNarrow>
__device__ __forceinline__ void stream_cols(T *row, const Cols<kNarrow> &c, const float (&x)[8]) {
    if (c.live >= 8) return store_stream(row + (uint32_t)c.col, x);
    if (c.live > 0) store_upto8(row + (uint32_t)c.col, c.live, x);
}

// Another eight columns of a lane, for rows of whole vectors with fp32 among them:
// four, and four 256 further on, so that a wave's load covers whole cache lines.
// `c` counts as in Cols; a wave's 64 lanes cover the same 512 columns, so a row's
// last wave is whole.
template <typename C> struct ColsTag {
    typedef C type;
};
struct Fours {
    int lo, hi, from_lo, from_hi;
    bool live_lo, live_hi;
    __device__ __forceinline__ Fours(int c, int dim)
        : lo((c & ~511) + (c & 511) / 2), hi(lo + 256), from_lo(lo < dim ? lo : dim - 4),
          from_hi(hi < dim ? hi : dim - 4), live_lo(lo < dim), live_hi(hi < dim) {}
};
__device__ __forceinline__ Raw8<float> load_cols(const float *row, const Fours &c) {
    return {*reinterpret_cast<const f32x4 *>(row + (uint32_t)c.from_lo),
            *reinterpret_cast<const f32x4 *>(row + (uint32_t)c.from_hi)};
}
__device__ __forceinline__ Raw8<Bf16> load_cols(const Bf16 *row, const Fours &c) {
    const u32x2 a = *reinterpret_cast<const u32x2 *>(row + (uint32_t)c.from_lo);
    const u32x2 b = *reinterpret_cast<const u32x2 *>(row + (uint32_t)c.from_hi);
    return {u32x4{a[0], a[1], b[0], b[1]}};
}
__device__ __forceinline__ Raw8<float> load_stream(const float *row, const Fours &c) {
    return {__builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(row + (uint32_t)c.from_lo)),
            __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(row + (uint32_t)c.from_hi))};
}
__device__ __forceinline__ Raw8<Bf16> load_stream(const Bf16 *row, const Fours &c) {
    const u32x2 a = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(row + (uint32_t)c.from_lo));
    const u32x2 b = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(row + (uint32_t)c.from_hi));
    return {u32x4{a[0], a[1], b[0], b[1]}};
}
template <typename T>
__device__ __forceinline__ void cols_values(const Raw8<T> &r, const Fours &c, float (&x)[8]) {
    values(r, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = (j < 4 ? c.live_lo : c.live_hi) ? x[j] : 0.0f;
}
__device__ __forceinline__ void store_cols(float *row, const Fours &c, const float (&x)[8]) {
    if (c.live_lo) *reinterpret_cast<f32x4 *>(row + c.lo) = f32x4{x[0], x[1], x[2], x[3]};
    if (c.live_hi) *reinterpret_cast<f32x4 *>(row + c.hi) = f32x4{x[4], x[5], x[6], x[7]};
}
__device__ __forceinline__ void store_cols(Bf16 *row, const Fours &c, const float (&x)[8]) {
    const u32x2 a = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
    const u32x2 b = {pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
    if (c.live_lo) *reinterpret_cast<u32x2 *>(row + c.lo) = a;
    if (c.live_hi) *reinterpret_cast<u32x2 *>(row + c.hi) = b;
}
__device__ __forceinline__ void stream_cols(float *row, const Fours &c, const float (&x)[8]) {
    if (c.live_lo) __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4 *>(row + c.lo));
    if (c.live_hi) __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, reinterpret_cast<f32x4 *>(row + c.hi));
}
__device__ __forceinline__ void stream_cols(Bf16 *row, const Fours &c, const float (&x)[8]) {
    const u32x2 a = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
    const u32x2 b = {pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
    if (c.live_lo) __builtin_nontemporal_store(a, reinterpret_cast<u32x2 *>(row + c.lo));
    if (c.live_hi) __builtin_nontemporal_store(b, reinterpret_cast<u32x2 *>(row + c.hi));
}

// Sum and maximum over aligned groups of `lanes` lanes of a wave (a power of
// two, uniform; every lane active): every lane receives its group's result.
template <int kCtrl>
__device__ __forceinline__ float dpp(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), kCtrl, 0xF, 0xF, true));
}
// v_permlane16_swap / v_permlane32_swap of a register with itself: a holds the
// even 16-lane rows (the lower half) in both rows of each pair, b the odd ones.
__device__ __forceinline__ void rows16(float x, float &a, float &b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    a = __uint_as_float(r[0]), b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void rows32(float x, float &a, float &b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    a = __uint_as_float(r[0]), b = __uint_as_float(r[1]);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
__device__ __forceinline__ float group_sum(float x, int lanes) {
    float a, b;
    if (lanes > 1) x += dpp<kXor1>(x);
    if (lanes > 2) x += dpp<kXor2>(x);
    if (lanes > 4) x += dpp<kHalfMirror>(x);
    if (lanes > 8) x += dpp<kMirror>(x);
    if (lanes > 16) rows16(x, a, b), x = a + b;
    if (lanes > 32) rows32(x, a, b), x = a + b;
    return x;
}
// Maximum of non-negative values over aligned groups of 32 lanes, or the wave.
template <int kLanes>
__device__ __forceinline__ float group_max(float x) {
    static_assert(kLanes == 32 || kLanes == 64, "lanes");
    float a, b;
    x = fmaxf(x, dpp<kXor1>(x));
    x = fmaxf(x, dpp<kXor2>(x));
    x = fmaxf(x, dpp<kHalfMirror>(x));
    x = fmaxf(x, dpp<kMirror>(x));
    rows16(x, a, b);
    x = fmaxf(a, b);
    if constexpr (kLanes == 64) rows32(x, a, b), x = fmaxf(a, b);
    return x;
}

}  // namespace nf4
