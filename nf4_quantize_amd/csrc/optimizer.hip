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

#include <type_traits>

#include "training_internal.h"

namespace nf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kPass = 2048;                // elements of a workgroup: 8 moment blocks
constexpr int kEach = kPass / kThreads;    // the norm's elements of a thread in one pass
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

// One entry as the kernel reads it.
struct AdamwItem {
    void *w;
    float *master;
    const void *g;
    void *m, *v;
    float *ms, *vs;
    int64_t n;
    float step;      // lr / (1 - beta1^t)
    float keep;      // 1 - lr weight_decay
    uint32_t key;
    uint32_t first;  // the entry's first workgroup in the launch
};
static_assert(sizeof(AdamwItem) == 80, "packed without holes");
struct AdamwBatch {
    AdamwItem item[kBatch];
};
struct AdamwScalars {
    float beta1, one_beta1, beta2, one_beta2, eps, rbias2, max_norm;
    int32_t count;  // entries of the table, or of the list whose norm is taken here
    float *norm;
    const double *partial;    // sums of squares that the norm is still to be taken from
    int32_t parts;
    const AdamwItem *table;   // in the workspace, where there are more than kBatch entries
    const uint32_t *firsts;   // their `first`, one after the other
};
static_assert(sizeof(AdamwBatch) + sizeof(AdamwScalars) <= 4096, "kernel arguments");

// Copies a batch of entries from the kernel arguments into the table: 16 bytes a
// thread, as the arguments lie in host memory.
__global__ __launch_bounds__(kThreads) void adamw_table_kernel(AdamwBatch b, int32_t count, AdamwItem *table,
                                                               uint32_t *firsts) {
    constexpr int kParts = sizeof(AdamwItem) / 16;
    static_assert(kBatch * kParts <= kThreads, "one pass");
    const int i = threadIdx.x;
    if (i < count * kParts) reinterpret_cast<u32x4 *>(table)[i] = reinterpret_cast<const u32x4 *>(b.item)[i];
    if (i < count) firsts[i] = b.item[i].first;
}

// The entry of workgroup wg: the last one whose first workgroup is not above it.
// All of the wave's lanes probe; the result is uniform.
__device__ __forceinline__ int find_in_table(const uint32_t *firsts, int count, uint32_t wg) {
    int lo = 0, hi = count;  // firsts[lo] <= wg, and firsts[hi] is above it or past the end
    const int lane = threadIdx.x % 64;
    while (hi - lo > 1) {
        const int stride = (hi - lo + 63) / 64;
        const int at = lo + lane * stride;
        const uint64_t not_above = __ballot(at < hi && firsts[at] <= wg);  // a prefix that holds lane 0
        lo += ((int)__popcll(not_above) - 1) * stride;
        hi = lo + stride < hi ? lo + stride : hi;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}
template <typename B, int N>
__device__ __forceinline__ int find_in_batch(const B (&item)[N], uint32_t wg) {
    // eight at a time, then within the eight
    int k = 0;
#pragma unroll
    for (int j = 8; j < N; j += 8) k = (wg >= item[j].first) ? j : k;
    const B *eight = &item[k];
    int in = 0;
#pragma unroll
    for (int j = 1; j < 8; ++j) in = (wg >= eight[j].first) ? j : in;
    return k + in;
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

__device__ __forceinline__ float decode_e4m3(uint8_t c) { return __builtin_amdgcn_cvt_f32_fp8((int)c, 0); }

// Scale of a block's storage and its reciprocal. `least`: the scale of blocks that
// are too small for their own.
__device__ __forceinline__ float storage_scale(float amax, float least, float *inv) {
    float s = amax * (1.0f / kE4m3Max);
    s = s < kScaleMin ? least : s;
    *inv = s > 0.0f ? 1.0f / s : 0.0f;
    return s;
}

// v_sqrt_f32 takes subnormal numbers for zero, and second moments get there under
// gradients of 1e-18: those are scaled by 2^48, and their root by 2^-24, both exact.
// Such roots are below 2^-63, half of the last place of an eps from 2^-39 on, where
// kernels without the scaling run: 448 tensors take 280 us in them, 298 in those with
// it, and 289 where the kernel itself asks eps.
constexpr float kRootEps = 0x1p-39f;
__device__ __forceinline__ float root_of_any(float x) {
    const bool small = x < 0x1p-126f;
    return __builtin_amdgcn_sqrtf(x * (small ? 0x1p48f : 1.0f)) * (small ? 0x1p-24f : 1.0f);
}

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

// A thread's share of the squares of a list's gradients (up to kN / 8 entries): the
// waves take pieces of 512 elements in turn, each wave kVecs pieces in flight.
template <typename G, int kN, int kVecs, typename Item>
__device__ __forceinline__ double list_squares(const Item *item, int32_t count) {
    double sum = 0.0;
    // the elements past an entry's last eight, eight threads an entry
    const int at = threadIdx.x % 8;
    if ((int)threadIdx.x / 8 < count) {
        const Item &e = item[threadIdx.x / 8];
        if (at < (int)(e.n % 8)) {
            const double x = load1(static_cast<const G *>(e.g) + e.n / 8 * 8 + at);
            sum = fma(x, x, sum);
        }
    }
    const int lane = threadIdx.x % 64;
    int k = -1;  // the piece that is next, of entry k; uniform over the wave
    int32_t piece = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), eights = 0, pieces = 0;
    const G *g = nullptr;
    auto find = [&] {
        while (piece >= pieces && k < count) {
            piece -= pieces;
            if (++k == count) break;
            g = static_cast<const G *>(item[k].g);
            eights = (int32_t)(item[k].n / 8), pieces = (eights + 63) / 64;
        }
    };
    for (find(); k < count;) {
        Raw8<G> raw[kVecs];
        bool live[kVecs];
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            live[u] = k < count && piece * 64 + lane < eights;
            if (k < count) raw[u] = load_raw(g + (live[u] ? piece * 64 + lane : piece * 64) * 8);
            piece += kN / 64;
            find();
        }
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            float x[8];
            values(raw[u], x);
            if (live[u])
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = fma((double)x[j], (double)x[j], sum);
        }
    }
    return sum;
}

// A lane's four elements, as eight are loaded and stored by load_raw, load_stream
// and store_stream.
template <typename T> struct Raw4;
template <> struct Raw4<Bf16> { u32x2 v; };
template <> struct Raw4<float> { f32x4 v; };
__device__ __forceinline__ void values(const Raw4<Bf16> &r, float (&x)[4]) {
    x[0] = bf16_lo(r.v[0]), x[1] = bf16_hi(r.v[0]), x[2] = bf16_lo(r.v[1]), x[3] = bf16_hi(r.v[1]);
}
__device__ __forceinline__ void values(const Raw4<float> &r, float (&x)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = r.v[j];
}
template <int N, typename T>
__device__ __forceinline__ auto load_each(const T *p) {
    if constexpr (N == 8) return load_raw(p);
    else return *reinterpret_cast<const Raw4<T> *>(p);
}
template <int N, typename T>
__device__ __forceinline__ auto stream_each(const T *p) {
    if constexpr (N == 8) return load_stream(p);
    else return Raw4<T>{__builtin_nontemporal_load(&reinterpret_cast<const Raw4<T> *>(p)->v)};
}
__device__ __forceinline__ void store_stream(float *p, const float (&x)[4]) {
    __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4 *>(p));
}
__device__ __forceinline__ void store_stream(Bf16 *p, const float (&x)[4]) {
    __builtin_nontemporal_store(u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])}, reinterpret_cast<u32x2 *>(p));
}

template <typename T, int N>
__device__ __forceinline__ void store_upto(T *p, int64_t live, const float (&x)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < live) store1(p + j, x[j]);
}
template <typename Code, int N>
__device__ __forceinline__ void decode_each(Code q, float scale, float (&x)[N]) {
    unpack_e4m3((uint32_t)q, scale, x);
    if constexpr (N == 8) unpack_e4m3((uint32_t)(q >> 32), scale, x + 4);
}
template <typename Code, int N>
__device__ __forceinline__ Code encode_each(const float (&x)[N], const uint32_t (&r)[N]) {
    Code q = pack_e4m3_sr(x, r);
    if constexpr (N == 8) q |= (Code)pack_e4m3_sr(x + 4, r + 4) << 32;
    return q;
}

// One workgroup: 2048 consecutive elements of one entry, eight a lane, or four:
// then 16 bytes of an fp32 array, and a load covers whole cache lines. Four where
// weights are kept in fp32 or moments in 32 bits, eight where the bf16 weights and
// the codes are all there is: 60 million elements (8 | 4 a lane)
//   bf16 weights and gradients, 8-bit moments                    112 | 128 us
//   the same and a master weight                                 196 | 161
//   fp32 weights and gradients, 8-bit moments                    170 | 158
//   bf16 weights and gradients, 32-bit moments                   242 | 217
//   the same, fp32 gradients and a master weight                 370 | 306
// A block of 256 is 32 lanes or the wave, so the block's maximum is a reduction in
// registers and every byte is moved once. Weights and moments go past the caches'
// usual order (they are not read again before the next step), gradients do not,
// and the workgroups run from the end of the list: what the norm's pass read last
// is still in the memory-side cache. The 448 tensors take 362 us with both and 424
// without (with the norm's launches and the table's).
template <typename W, bool kMaster, bool kEight>
constexpr int kStepEach = (kEight && !kMaster && sizeof(W) == 2) ? 8 : 4;

// A pointer that was loaded from memory, as one to global memory; what the compiler
// cannot tell by itself it reads as flat memory (448 tensors: 291 us instead of 283).
template <typename T> __device__ __forceinline__ T *in_global(T *p) {
    return (T *)(__attribute__((address_space(1))) T *)reinterpret_cast<uintptr_t>(p);
}

// The step of workgroup wg's elements of its entry (kAnyRoot: see root_of_any).
template <typename W, typename G, bool kMaster, bool kEight, bool kAnyRoot, int N>
__device__ __forceinline__ void step_elements(const AdamwScalars &c, const AdamwItem &e, float clip, uint32_t wg) {
    constexpr int kBlockLanes = kMomentBlock / N;
    using Code = std::conditional_t<N == 8, uint64_t, uint32_t>;  // a lane's codes
    const int64_t i = (int64_t)(wg - e.first) * kPass + threadIdx.x * N;
    const int64_t live = e.n - i;  // may be <= 0: the lane still joins the reductions
    W *w = static_cast<W *>(e.w) + i;
    const G *g = static_cast<const G *>(e.g) + i;
    float x[N], gr[N], m[N], v[N];
    if (live >= N) {  // the loads first, all in flight, in this order (the weight before the codes: 4% more)
        const auto weight = [&] {
            if constexpr (kMaster) return stream_each<N>(e.master + i);
            else return stream_each<N>(w);
        };
        const auto rg = load_each<N>(g);
        if constexpr (kEight) {
            const uint8_t *pm = static_cast<const uint8_t *>(e.m) + i, *pv = static_cast<const uint8_t *>(e.v) + i;
            const Code mq = __builtin_nontemporal_load(reinterpret_cast<const Code *>(pm));
            const Code vq = __builtin_nontemporal_load(reinterpret_cast<const Code *>(pv));
            const float ms = e.ms[i / kMomentBlock], vs = e.vs[i / kMomentBlock];
            const auto rx = weight();
            __builtin_amdgcn_sched_barrier(0);
            values(rx, x);
            decode_each(mq, ms, m);
            decode_each(vq, vs, v);
        } else {
            const auto rm = stream_each<N>(static_cast<const float *>(e.m) + i);
            const auto rv = stream_each<N>(static_cast<const float *>(e.v) + i);
            const auto rx = weight();
            __builtin_amdgcn_sched_barrier(0);
            values(rx, x);
            values(rm, m), values(rv, v);
        }
        values(rg, gr);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            x[j] = gr[j] = m[j] = v[j] = 0.0f;
            if (j >= live) continue;
            x[j] = kMaster ? e.master[i + j] : load1(w + j);
            gr[j] = load1(g + j);
            if constexpr (kEight) {
                m[j] = decode_e4m3(static_cast<const uint8_t *>(e.m)[i + j]) * e.ms[i / kMomentBlock];
                v[j] = decode_e4m3(static_cast<const uint8_t *>(e.v)[i + j]) * e.vs[i / kMomentBlock];
            } else {
                m[j] = static_cast<const float *>(e.m)[i + j];
                v[j] = static_cast<const float *>(e.v)[i + j];
            }
        }
    }
    float ma = 0.0f, va = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float gj = gr[j] * clip;
        // product by product, without contraction: the stored codes follow
        // from these fp32 values to the bit
        m[j] = c.beta1 * m[j] + c.one_beta1 * gj;
        v[j] = c.beta2 * v[j] + c.one_beta2 * (gj * gj);
        // the hardware's reciprocal and root are within 1 ulp: the step is
        // a small part of the weight it is added to
        const float t = v[j] * c.rbias2, d = (kAnyRoot ? root_of_any(t) : __builtin_amdgcn_sqrtf(t)) + c.eps;
        // the reciprocal of a subnormal number is infinite there, so eps is scaled as well
        const float up = kAnyRoot && d < 0x1p-126f ? 0x1p24f : 1.0f;
        x[j] = fmaf(-(e.step * up) * m[j], __builtin_amdgcn_rcpf(d * up), x[j] * e.keep);
        ma = fmaxf(ma, fabsf(m[j])), va = fmaxf(va, v[j]);
    }
    if (live >= N) {
        if constexpr (kMaster) store_stream(e.master + i, x);
        store_stream(w, x);
    } else if (live > 0) {
        if constexpr (kMaster) store_upto(e.master + i, live, x);
        store_upto(w, live, x);
    }
    if constexpr (!kEight) {
        if (live >= N) {
            store_stream(static_cast<float *>(e.m) + i, m);
            store_stream(static_cast<float *>(e.v) + i, v);
        } else if (live > 0) {
            store_upto(static_cast<float *>(e.m) + i, live, m);
            store_upto(static_cast<float *>(e.v) + i, live, v);
        }
    } else {
        float rm, rv;
        const float ms = storage_scale(group_max<kBlockLanes>(ma), 0.0f, &rm);
        const float vs = storage_scale(group_max<kBlockLanes>(va), ms > 0.0f ? kScaleMin : 0.0f, &rv);
        uint32_t rndm[N], rndv[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint32_t r = mix((uint32_t)i * kWeyl + e.key + (uint32_t)j * kWeyl);
            rndm[j] = r & 0xFFFF0000u, rndv[j] = r << 16;
            m[j] = __builtin_amdgcn_fmed3f(m[j] * rm, -kE4m3Max, kE4m3Max);
            v[j] = __builtin_amdgcn_fmed3f(v[j] * rv, kE4m3Min, kE4m3Max);
        }
        if (live <= 0) return;
        uint8_t *mq = static_cast<uint8_t *>(e.m) + i, *vq = static_cast<uint8_t *>(e.v) + i;
        const Code mw = encode_each<Code>(m, rndm);
        const Code vw = encode_each<Code>(v, rndv);
        if (live >= N) {
            __builtin_nontemporal_store(mw, reinterpret_cast<Code *>(mq));
            __builtin_nontemporal_store(vw, reinterpret_cast<Code *>(vq));
        } else {
            for (int j = 0; j < (int)live; ++j) {
                mq[j] = (uint8_t)(mw >> (8 * j));
                vq[j] = (uint8_t)(vw >> (8 * j));
            }
        }
        if (threadIdx.x % kBlockLanes == 0) {
            e.ms[i / kMomentBlock] = ms;
            e.vs[i / kMomentBlock] = vs;
        }
    }
}

// Where a workgroup finds its entry, and the norm that the step clips by: the
// kernel arguments hold the list, or the workspace; or the arguments hold one of so
// few elements that every workgroup reads all gradients for the norm (kOwnNorm), or
// all of the norm's partial sums (kPartNorm).
enum ListKind { kInArgs, kInTable, kOwnNorm, kPartNorm };

template <typename W, typename G, bool kMaster, bool kEight, ListKind kList, int N = kStepEach<W, kMaster, kEight>,
          bool kAnyRoot = false>
__global__ __launch_bounds__(kPass / N) void adamw_kernel(AdamwBatch b, AdamwScalars c) {
    float clip = 1.0f;
    constexpr bool kTakesNorm = kList == kOwnNorm || kList == kPartNorm;
    if (kTakesNorm || c.norm != nullptr) {
        float norm;
        if constexpr (kTakesNorm) {
            __shared__ float s_norm;
            double sum = 0.0;
            if constexpr (kList == kOwnNorm) sum = list_squares<G, kPass / N, 8>(b.item, c.count);
            else
                for (int i = threadIdx.x; i < c.parts; i += kPass / N) sum += c.partial[i];
            sum = block_sum<kPass / N>(sum);
            if (threadIdx.x == 0) s_norm = (float)sqrt(sum);
            __syncthreads();
            norm = s_norm;
            if (blockIdx.x == 0 && threadIdx.x == 0) *c.norm = norm;
        } else {
            norm = *c.norm;
        }
        if (!(fabsf(norm) < INFINITY)) return;
        if (c.max_norm > 0.0f && norm > c.max_norm) clip = c.max_norm * (1.0f / norm);
    }
    const uint32_t wg = gridDim.x - 1 - blockIdx.x;
    AdamwItem e = kList == kInTable ? c.table[find_in_table(c.firsts, c.count, wg)] : b.item[find_in_batch(b.item, wg)];
    e.w = in_global(e.w), e.master = in_global(e.master), e.g = in_global(e.g);
    e.m = in_global(e.m), e.v = in_global(e.v), e.ms = in_global(e.ms), e.vs = in_global(e.vs);
    step_elements<W, G, kMaster, kEight, kAnyRoot, N>(c, e, clip, wg);
}

// ---- the gradients' norm ----

constexpr int kNormBatch = 160;
constexpr int64_t kSmallNorm = 1 << 17;  // elements, and
constexpr int64_t kMidNorm = 1 << 23;    // elements: the step takes the norm from the partial sums
constexpr int32_t kSmallEntries = 16;    // entries: lists whose norm a single workgroup takes
constexpr int kNormVecs = 8;                              // of a thread, in flight together
constexpr int64_t kNormChunk = (int64_t)kPass * kNormVecs;  // elements of one partial sum

struct NormItem {
    const void *g;
    int64_t n;
    uint32_t first, pad;
};
struct NormBatch {
    NormItem item[kNormBatch];
};
static_assert(sizeof(NormBatch) + 16 <= 4096, "kernel arguments");

// Squares of 16384 consecutive gradients, each exact in fp64.
template <typename G>
__global__ __launch_bounds__(kThreads) void grad_square_kernel(NormBatch b, double *partial) {
    const NormItem e = b.item[find_in_batch(b.item, blockIdx.x)];
    const int64_t begin = (int64_t)(blockIdx.x - e.first) * kNormChunk;
    const G *g = static_cast<const G *>(e.g) + begin;
    double sum = 0.0;
    if (e.n - begin >= kNormChunk) {
        Raw8<G> raw[kNormVecs];
#pragma unroll
        for (int u = 0; u < kNormVecs; ++u) raw[u] = load_raw(g + u * kPass + threadIdx.x * kEach);
#pragma unroll
        for (int u = 0; u < kNormVecs; ++u) {
            float x[8];
            values(raw[u], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fma((double)x[j], (double)x[j], sum);
        }
    } else {
        for (int64_t i = threadIdx.x * kEach; i < e.n - begin; i += kPass) {
            float x[8];
            load_upto8(g + i, e.n - begin - i, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fma((double)x[j], (double)x[j], sum);
        }
    }
    sum = block_sum<kThreads>(sum);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The whole norm in one workgroup, for lists of few elements: one launch instead
// of two.
template <typename G>
__global__ __launch_bounds__(1024) void grad_norm_small_kernel(NormBatch b, int32_t count, float *norm) {
    const double sum = block_sum<1024>(list_squares<G, 1024, 8>(b.item, count));
    if (threadIdx.x == 0) *norm = (float)sqrt(sum);
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

// Entries of one kind (with or without a master weight). Up to kBatch of them
// travel in the kernel arguments; more are first copied into a table in the
// workspace, 48 a launch, so that one launch runs over all of them: the 448
// adapters of a 32-layer stack took 10 launches of 17 million elements, each
// with its own ramp and drain.
template <typename W, typename G, bool kMaster, bool kEight>
hipError_t adamw_launches(const nf4_adamw_entry *e, int32_t count, const nf4_adamw_config &cfg,
                          float *norm, ListKind list, int64_t parts, void *workspace, hipStream_t s) {
    const double bias1 = 1.0 - pow(cfg.beta1, (double)cfg.step);
    const double bias2 = 1.0 - pow(cfg.beta2, (double)cfg.step);
    AdamwScalars c{};
    c.beta1 = (float)cfg.beta1, c.one_beta1 = (float)(1.0 - cfg.beta1);
    c.beta2 = (float)cfg.beta2, c.one_beta2 = (float)(1.0 - cfg.beta2);
    c.eps = cfg.eps, c.rbias2 = (float)(1.0 / bias2);
    c.max_norm = cfg.max_norm, c.norm = norm;
    c.partial = static_cast<const double *>(workspace), c.parts = (int32_t)parts;
    auto mine = [&](int32_t i) { return e[i].n > 0 && (e[i].master != nullptr) == kMaster; };
    int32_t total = 0;
    for (int32_t i = 0; i < count; ++i) total += mine(i) ? 1 : 0;
    if (total == 0) return hipSuccess;
    const bool table = total > kBatch;
    AdamwItem *items = static_cast<AdamwItem *>(workspace);
    uint32_t *firsts = reinterpret_cast<uint32_t *>(items + count);
    AdamwBatch b{};
    int used = 0;       // entries of the batch
    int32_t done = 0, from = 0;  // entries in the table; its first entry of the next launch
    int64_t wgs = 0;
    hipError_t err = hipSuccess;
    auto note = [&] {
        const hipError_t r = hipGetLastError();
        if (err == hipSuccess) err = r;
    };
    constexpr int kLaneElems = kStepEach<W, kMaster, kEight>;
    const dim3 threads(kPass / kLaneElems);
    const bool any_root = cfg.eps < kRootEps;
    auto copy = [&] {  // the batch into the table
        if (used == 0) return;
        adamw_table_kernel<<<dim3(1), dim3(kThreads), 0, s>>>(b, used, items + done, firsts + done);
        note();
        done += used, used = 0;
    };
    auto run = [&] {
        if (wgs == 0) return;
        if (table) {
            copy();
            c.table = items + from, c.firsts = firsts + from, c.count = done - from;
            if (any_root)
                adamw_kernel<W, G, kMaster, kEight, kInTable, kLaneElems, true>
                    <<<dim3((uint32_t)wgs), threads, 0, s>>>(b, c);
            else adamw_kernel<W, G, kMaster, kEight, kInTable><<<dim3((uint32_t)wgs), threads, 0, s>>>(b, c);
            from = done;
        } else {
            for (int j = used; j < kBatch; ++j) b.item[j].first = UINT32_MAX;
            c.count = used;
            if (list == kOwnNorm)
                adamw_kernel<W, G, kMaster, kEight, kOwnNorm, 4><<<dim3((uint32_t)wgs), dim3(kPass / 4), 0, s>>>(b, c);
            else if (list == kPartNorm)
                adamw_kernel<W, G, kMaster, kEight, kPartNorm><<<dim3((uint32_t)wgs), threads, 0, s>>>(b, c);
            else if (any_root)
                adamw_kernel<W, G, kMaster, kEight, kInArgs, kLaneElems, true>
                    <<<dim3((uint32_t)wgs), threads, 0, s>>>(b, c);
            else adamw_kernel<W, G, kMaster, kEight, kInArgs><<<dim3((uint32_t)wgs), threads, 0, s>>>(b, c);
            used = 0;
        }
        note();
        wgs = 0;
    };
    constexpr int64_t kMaxWgs = (int64_t(1) << 31) / (kPass / kLaneElems);  // threads of a grid
    for (int32_t i = 0; i < count; ++i) {
        if (!mine(i)) continue;
        const int64_t need = (e[i].n + kPass - 1) / kPass;
        if (wgs + need > kMaxWgs) run();
        if (used == kBatch) copy();  // only with a table: otherwise all entries fit
        AdamwItem &t = b.item[used++];
        t.w = e[i].w, t.master = e[i].master, t.g = e[i].grad, t.m = e[i].m, t.v = e[i].v;
        t.ms = e[i].m_scale, t.vs = e[i].v_scale, t.n = e[i].n;
        t.step = (float)((double)e[i].lr / bias1);
        t.keep = (float)(1.0 - (double)e[i].lr * (double)e[i].weight_decay);
        t.key = mix(mix((uint32_t)i * kWeyl + (uint32_t)(cfg.seed >> 32)) + (uint32_t)cfg.seed);
        t.first = (uint32_t)wgs;
        wgs += need;
    }
    run();
    return err;
}

template <typename W, typename G>
hipError_t adamw_typed(const nf4_adamw_entry *e, int32_t count, bool eight, const nf4_adamw_config &c,
                       float *norm, ListKind list, int64_t parts, void *ws, hipStream_t s) {
    hipError_t err = eight ? adamw_launches<W, G, false, true>(e, count, c, norm, list, parts, ws, s)
                           : adamw_launches<W, G, false, false>(e, count, c, norm, list, parts, ws, s);
    if constexpr (sizeof(W) == 2) {
        const hipError_t r = eight ? adamw_launches<W, G, true, true>(e, count, c, norm, list, parts, ws, s)
                                   : adamw_launches<W, G, true, false>(e, count, c, norm, list, parts, ws, s);
        if (err == hipSuccess) err = r;
    }
    return err;
}

// Elements and entries with any.
struct Extent {
    int64_t elements;
    int32_t live, masters;
};
Extent extent_of(const nf4_adamw_entry *e, int32_t count) {
    Extent x{};
    for (int32_t i = 0; i < count; ++i)
        if (e[i].n > 0) x.elements += e[i].n, ++x.live, x.masters += e[i].master ? 1 : 0;
    return x;
}

}  // namespace

size_t adamw_workspace(int32_t count) {
    return count > kBatch ? (size_t)count * (sizeof(AdamwItem) + sizeof(uint32_t)) : 0;
}

size_t grad_norm_workspace(const nf4_adamw_entry *e, int32_t count) {
    return (size_t)norm_partials(e, count) * sizeof(double);
}

// The sums of squares of chunks of the list; `done` of them.
hipError_t launch_squares(const nf4_adamw_entry *e, int32_t count, nf4_dtype gt, void *workspace, int64_t &done,
                          hipStream_t s) {
    double *partial = static_cast<double *>(workspace);
    NormBatch b{};
    int used = 0;
    int64_t wgs = 0;
    done = 0;
    hipError_t err = hipSuccess;
    auto flush = [&] {
        if (used == 0) return;
        for (int j = used; j < kNormBatch; ++j) b.item[j].first = UINT32_MAX;
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
        b.item[used] = NormItem{e[i].grad, e[i].n, (uint32_t)wgs, 0u};
        wgs += need;
        ++used;
    }
    flush();
    return err;
}

hipError_t launch_grad_norm(const nf4_adamw_entry *e, int32_t count, nf4_dtype gt, float *norm,
                            void *workspace, hipStream_t s) {
    // One launch less, but one workgroup's bandwidth: 4.8 us instead of 8.1 for two
    // tensors of 1000 elements (bf16), 7.0 and 7.1 for two of 65536, 11.2 and 7.0 for
    // two of 131072.
    const Extent x = extent_of(e, count);
    if (x.elements <= kSmallNorm && x.live <= kSmallEntries) {
        NormBatch b{};
        int used = 0;
        for (int32_t i = 0; i < count; ++i)
            if (e[i].n > 0) b.item[used++] = NormItem{e[i].grad, e[i].n, 0u, 0u};
        if (gt == NF4_BF16) grad_norm_small_kernel<Bf16><<<dim3(1), dim3(1024), 0, s>>>(b, used, norm);
        else grad_norm_small_kernel<float><<<dim3(1), dim3(1024), 0, s>>>(b, used, norm);
        return hipGetLastError();
    }
    int64_t parts;
    const hipError_t err = launch_squares(e, count, gt, workspace, parts, s);
    grad_norm_kernel<<<dim3(1), dim3(1024), 0, s>>>(static_cast<const double *>(workspace), parts, norm);
    const hipError_t r = hipGetLastError();
    return err == hipSuccess ? r : err;
}

hipError_t launch_adamw(const nf4_adamw_entry *e, int32_t count, nf4_dtype wt, nf4_dtype gt,
                        bool eight, const nf4_adamw_config &c, float *norm, bool own_norm, void *workspace,
                        hipStream_t s) {
    ListKind list = kInArgs;
    int64_t parts = 0;
    if (own_norm) {
        const Extent x = extent_of(e, count);
        const bool one_kind = x.masters == 0 || x.masters == x.live;
        if (c.eps < kRootEps) {
            // kernels with a root of any second moment take the norm as a number
        } else if (x.live > 0 && x.elements <= kSmallNorm && x.live <= kSmallEntries && one_kind) {
            // Every workgroup reads all gradients, but there is one launch: 7.4 us
            // instead of 10.8 for two tensors of 8192 elements (bf16, 8-bit moments),
            // 11.2 instead of 14.0 for 14 of them, 10.4 instead of 11.3 for two of
            // 65536; 16.5 against 13.6 for two of 131072.
            list = kOwnNorm;
        } else if (x.live > 0 && x.elements <= kMidNorm && x.live <= kBatch) {
            // One launch less, and a read of up to 560 partial sums in every workgroup:
            // 11.9 us instead of 15.2 for two tensors of 131072, 15.8 instead of 17.4 for
            // two of 2097152, 25.0 and 25.3 for two of 4194304; 50.3 against 48.4 for 40
            // of 524288.
            list = kPartNorm;
        }
        if (list != kOwnNorm) {
            const hipError_t r = list == kPartNorm ? launch_squares(e, count, gt, workspace, parts, s)
                                                   : launch_grad_norm(e, count, gt, norm, workspace, s);
            if (r != hipSuccess) return r;
        }
    }
    if (wt == NF4_BF16)
        return gt == NF4_BF16 ? adamw_typed<Bf16, Bf16>(e, count, eight, c, norm, list, parts, workspace, s)
                              : adamw_typed<Bf16, float>(e, count, eight, c, norm, list, parts, workspace, s);
    return gt == NF4_BF16 ? adamw_typed<float, Bf16>(e, count, eight, c, norm, list, parts, workspace, s)
                          : adamw_typed<float, float>(e, count, eight, c, norm, list, parts, workspace, s);
}

}  // namespace nf4
