// Drives the host side of the training step's entry points for the
// AddressSanitizer / UndefinedBehaviorSanitizer build of
// tests/test_sanitizers_training.py: argument validation and workspace sizes.
// Every call here is rejected, or is empty, before any HIP call, so no GPU is
// needed. The device pointers are never dereferenced.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <vector>

#include "nf4.h"

namespace {

int failures = 0;

#define EXPECT(expr, want)                                                                   \
    do {                                                                                     \
        const long long got_ = (long long)(expr);                                            \
        if (got_ != (long long)(want)) {                                                     \
            std::fprintf(stderr, "%s:%d: %s = %lld, want %lld\n", __FILE__, __LINE__, #expr, \
                         got_, (long long)(want));                                           \
            ++failures;                                                                      \
        }                                                                                    \
    } while (0)

template <typename T> T *at(uintptr_t off = 0) { return reinterpret_cast<T *>(uintptr_t(0x10000) + off); }

nf4_adamw_entry entry(int64_t n = 1000) {
    return {at<void>(), nullptr, at<const void>(), at<void>(), at<void>(), at<float>(), at<float>(), n, 1e-3f, 0.0f};
}

void adamw() {
    nf4_adamw_config c{0.9, 0.999, 1e-8f, 1.0f, 1, 0};
    auto step = [&](const std::vector<nf4_adamw_entry> &e, size_t bytes) {
        return nf4_adamw_step(e.data(), (int32_t)e.size(), NF4_BF16, NF4_BF16, NF4_MOMENTS_8, &c, at<float>(), at<void>(),
                              bytes, nullptr);
    };
    auto clip = [&](const std::vector<nf4_adamw_entry> &e, size_t bytes) {
        return nf4_adamw_clip_step(e.data(), (int32_t)e.size(), NF4_BF16, NF4_BF16, NF4_MOMENTS_8, &c, at<float>(),
                                   at<void>(), bytes, nullptr);
    };
    // the bad entry last, at sizes around a launch's and far beyond
    for (size_t count : {1u, 16u, 48u, 49u, 160u, 161u, 5000u}) {
        std::vector<nf4_adamw_entry> e(count, entry());
        e.back().v = nullptr;
        EXPECT(step(e, SIZE_MAX), NF4_ERR_NULL);
        EXPECT(clip(e, SIZE_MAX), NF4_ERR_NULL);
        e.back() = entry((int64_t(1) << 33) + 1);
        EXPECT(step(e, SIZE_MAX), NF4_ERR_SIZE);
        EXPECT(nf4_grad_norm_workspace_size(e.data(), (int32_t)count), (size_t)-1);
        e.back() = entry(int64_t(1) << 33);
        EXPECT(nf4_grad_norm_workspace_size(e.data(), (int32_t)count), 8 * (count - 1 + (int64_t(1) << 19)));
        EXPECT(clip(e, 7), NF4_ERR_WORKSPACE);
        EXPECT(nf4_grad_norm(e.data(), (int32_t)count, NF4_F32, at<float>(), at<void>(), 7, nullptr), NF4_ERR_WORKSPACE);
        for (auto &x : e) x.n = 0, x.grad = nullptr;
        EXPECT(nf4_grad_norm_workspace_size(e.data(), (int32_t)count), 0);
        const size_t need = nf4_adamw_workspace_size((int32_t)count);
        EXPECT(need > 0, count > 48);
        if (need == 0) EXPECT(step(e, 0), NF4_OK);
        else EXPECT(step(e, need - 1), NF4_ERR_WORKSPACE);
    }
    EXPECT(nf4_adamw_workspace_size(INT32_MIN), (size_t)-1);
    EXPECT(nf4_adamw_workspace_size(INT32_MAX), 84 * (long long)INT32_MAX);
    c.step = INT64_MIN;
    EXPECT(step({entry()}, SIZE_MAX), NF4_ERR_SIZE);
}

void norms() {
    nf4_residual_norm_shape s{4, 256, NF4_BF16, NF4_BF16, NF4_BF16, NF4_GATE_NONE, 1e-6f, 1.0f, 0.0f};
    auto forward = [&] {
        return nf4_residual_norm_forward(&s, at<void>(), at<void>(), nullptr, nullptr, at<void>(), at<void>(), nullptr,
                                         nullptr, nullptr, nullptr);
    };
    EXPECT(forward(), NF4_ERR_NULL);
    for (int64_t rows : {int64_t(-1), INT64_MIN, INT64_MAX}) {
        s.rows = rows;
        EXPECT(forward(), NF4_ERR_SIZE);
        EXPECT(nf4_residual_norm_backward_workspace_size(&s), (size_t)-1);
    }
    s.rows = 4;
    for (int64_t dim : {int64_t(0), int64_t(32769), INT64_MAX, INT64_MIN}) {
        s.dim = dim;
        EXPECT(forward(), NF4_ERR_SIZE);
        EXPECT(nf4_residual_norm_backward_workspace_size(&s), (size_t)-1);
    }
    for (int64_t dim : {1, 7, 512, 513, 4096, 4104, 8192, 8193, 32768}) {
        s.dim = dim, s.rows = (int64_t(1) << 37) / dim;
        EXPECT(nf4_residual_norm_backward_workspace_size(&s) != (size_t)-1, 1);
        EXPECT(nf4_residual_norm_backward(&s, nullptr, nullptr, nullptr, at<void>(), nullptr, nullptr, at<void>(), nullptr,
                                          at<float>(), nullptr, nullptr, nullptr, at<void>(), nullptr, at<void>(), 3,
                                          nullptr),
               NF4_ERR_WORKSPACE);
    }
    s.eps = NAN;
    EXPECT(forward(), NF4_ERR_SIZE);
}

void embedding() {
    for (int64_t tokens : {int64_t(-1), (int64_t(1) << 28) + 1, INT64_MAX, INT64_MIN}) {
        EXPECT(nf4_embedding_backward_workspace_size(tokens, 1000, 64), (size_t)-1);
        EXPECT(nf4_embedding_backward(at<void>(), NF4_I32, tokens, at<void>(), NF4_BF16, 1000, 64, 1.0f, -1, at<void>(),
                                      NF4_BF16, 0, at<void>(), SIZE_MAX, nullptr),
               NF4_ERR_SIZE);
    }
    for (int64_t tokens : {1, 16, 6144, 6145, 32768, 32769, 1 << 28})
        for (int64_t dim : {1, 512, 513, 4096}) {
            const size_t need = nf4_embedding_backward_workspace_size(tokens, 1000, dim);
            if (tokens * dim > int64_t(1) << 37) {  // more elements than any buffer may have
                EXPECT(need, (size_t)-1);
                continue;
            }
            EXPECT(need != (size_t)-1 && need >= 8 * (size_t)tokens, 1);
            EXPECT(nf4_embedding_backward(at<void>(), NF4_I64, tokens, at<void>(), NF4_F32, 1000, dim, 1.0f, -1, at<void>(),
                                          NF4_F32, 1, at<void>(), 8, nullptr),
                   NF4_ERR_WORKSPACE);
        }
    EXPECT(nf4_embedding_forward(at<void>(), NF4_I32, 4, nullptr, NF4_BF16, 10, 64, 1.0f, at<void>(), NF4_BF16, nullptr),
           NF4_ERR_NULL);
    EXPECT(nf4_embedding_forward(at<void>(), 7, 4, at<void>(), NF4_BF16, 10, 64, 1.0f, at<void>(), NF4_BF16, nullptr),
           NF4_ERR_UNSUPPORTED);
    EXPECT(nf4_embedding_forward_packed(at<void>(), NF4_I32, 4, nullptr, 1.0f, at<void>(), NF4_BF16, nullptr), NF4_ERR_NULL);
}

}  // namespace

int main() {
    adamw();
    norms();
    embedding();
    if (failures) return 1;
    std::puts("ok");
    return 0;
}
