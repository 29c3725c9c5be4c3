// Drives the host side of the rotation's and Muon's entry points for the
// AddressSanitizer / UndefinedBehaviorSanitizer build of
// tests/test_sanitizers_attention.py: argument validation and workspace sizes.
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

void rotation() {
    const nf4_rotary_shape good{2, 3, 4, 2, 64, 32, NF4_ROTARY_HALF, NF4_BF16, NF4_F32, 1e-6f, 0.0f, 1.0f};
    nf4_heads h{at<void>(), 3 * 4 * 64, 4 * 64, 64}, none{nullptr, 0, 0, 0};
    auto forward = [&](const nf4_rotary_shape *s, const nf4_heads *q, const nf4_heads *k, const nf4_heads *out) {
        return nf4_rotary_forward(s, at<uint64_t>(), nullptr, NF4_I64, 0, q, k, nullptr, nullptr, out, out, nullptr);
    };
    EXPECT(forward(nullptr, &h, &h, &h), NF4_ERR_NULL);
    EXPECT(forward(&good, &h, &none, &h), NF4_ERR_NULL);
    EXPECT(forward(&good, &h, nullptr, &h), NF4_ERR_NULL);
    EXPECT(forward(&good, &h, &h, nullptr), NF4_ERR_NULL);
    auto shaped = [&](auto change) {
        nf4_rotary_shape s = good;
        change(s);
        const size_t size = nf4_rotary_backward_workspace_size(&s);
        const nf4_status st = forward(&s, &h, &h, &h);
        EXPECT(size == (size_t)-1, st == NF4_ERR_SIZE || st == NF4_ERR_UNSUPPORTED);
        return st;
    };
    // products of sizes that pass 64 bits come as sizes, not as overflow
    EXPECT(shaped([](auto &s) { s.batch = INT64_MAX, s.tokens = INT64_MAX; }), NF4_ERR_SIZE);
    EXPECT(shaped([](auto &s) { s.batch = 1 << 15, s.tokens = (1 << 15) + 1; }), NF4_ERR_SIZE);
    EXPECT(shaped([](auto &s) { s.batch = INT64_MIN; }), NF4_ERR_SIZE);
    EXPECT(shaped([](auto &s) { s.heads_q = INT32_MAX; }), NF4_ERR_SIZE);
    EXPECT(shaped([](auto &s) { s.heads_k = -1; }), NF4_ERR_SIZE);
    EXPECT(shaped([](auto &s) { s.dim = 513; }), NF4_ERR_SIZE);
    EXPECT(shaped([](auto &s) { s.dim = INT32_MIN; }), NF4_ERR_SIZE);
    EXPECT(shaped([](auto &s) { s.rotated = 33; }), NF4_ERR_SIZE);
    EXPECT(shaped([](auto &s) { s.rotated = 66; }), NF4_ERR_SIZE);
    EXPECT(shaped([](auto &s) { s.rotated = 0; }), NF4_ERR_SIZE);
    EXPECT(shaped([](auto &s) { s.layout = 2; }), NF4_ERR_UNSUPPORTED);
    EXPECT(shaped([](auto &s) { s.dtype = 7; }), NF4_ERR_UNSUPPORTED);
    EXPECT(shaped([](auto &s) { s.eps = NAN; }), NF4_ERR_SIZE);
    EXPECT(shaped([](auto &s) { s.scale = INFINITY; }), NF4_ERR_SIZE);
    // nothing to do: nothing is read
    EXPECT(shaped([](auto &s) { s.tokens = 0; }), NF4_OK);
    EXPECT(shaped([](auto &s) { s.heads_q = s.heads_k = 0; }), NF4_OK);
    for (int64_t stride : {int64_t(-1), INT64_MIN, INT64_MAX, (int64_t(1) << 40) + 1}) {
        nf4_heads bad = h;
        bad.token_stride = stride;
        EXPECT(forward(&good, &bad, &h, &h), NF4_ERR_SIZE);
        EXPECT(nf4_rotary_forward(&good, at<uint64_t>(), at<void>(), NF4_I32, stride, &h, &h, nullptr, nullptr, &h, &h, nullptr),
               NF4_ERR_SIZE);
    }
    nf4_heads odd = h;
    odd.data = at<void>(1);
    EXPECT(forward(&good, &odd, &h, &h), NF4_ERR_ALIGN);
    EXPECT(nf4_rotary_forward(&good, at<uint64_t>(4), nullptr, NF4_I64, 0, &h, &h, nullptr, nullptr, &h, &h, nullptr), NF4_ERR_ALIGN);
    EXPECT(nf4_rotary_forward(&good, at<uint64_t>(), at<void>(4), NF4_I64, 0, &h, &h, nullptr, nullptr, &h, &h, nullptr),
           NF4_ERR_ALIGN);
    EXPECT(nf4_rotary_forward(&good, at<uint64_t>(), nullptr, 9, 0, &h, &h, nullptr, nullptr, &h, &h, nullptr), NF4_ERR_UNSUPPORTED);
    EXPECT(nf4_rotary_forward(&good, at<uint64_t>(), nullptr, NF4_I64, 0, &h, &h, at<void>(4), nullptr, &h, &h, nullptr),
           NF4_ERR_ALIGN);

    auto backward = [&](const nf4_heads *x, const void *w, void *dw, void *ws, size_t bytes) {
        return nf4_rotary_backward(&good, at<uint64_t>(), nullptr, NF4_I64, 0, &h, &h, x, x, w, nullptr, &h, &h, dw, nullptr, ws,
                                   bytes, nullptr);
    };
    const size_t need = nf4_rotary_backward_workspace_size(&good);
    EXPECT(backward(&h, nullptr, at<void>(), at<void>(), need), NF4_ERR_NULL);
    EXPECT(backward(nullptr, at<void>(), nullptr, nullptr, 0), NF4_ERR_NULL);
    EXPECT(backward(&h, at<void>(), at<void>(), at<void>(), need - 1), NF4_ERR_WORKSPACE);
    EXPECT(backward(&h, at<void>(), at<void>(2), at<void>(), need), NF4_ERR_ALIGN);
    EXPECT(nf4_rotary_backward_workspace_size(nullptr), (size_t)-1);
}

nf4_muon_entry entry(int64_t rows = 64, int64_t cols = 4096) {
    return {at<void>(), nullptr, at<const void>(), at<void>(), rows, cols, 1e-3f, 0.1f, 1.0f};
}

void muon() {
    nf4_muon_config c{0.95, 1e-7, 3.4445, -4.775, 2.0315, 1, 5};
    auto step = [&](const std::vector<nf4_muon_entry> &e, size_t bytes, int32_t w = NF4_BF16) {
        return nf4_muon_step(e.data(), (int32_t)e.size(), w, NF4_BF16, NF4_F32, &c, at<void>(), bytes, nullptr);
    };
    auto alone = [&](const std::vector<nf4_muon_entry> &e, size_t bytes) {
        return nf4_orthogonalize(e.data(), (int32_t)e.size(), NF4_F32, &c, at<void>(), bytes, nullptr);
    };
    auto size = [](const std::vector<nf4_muon_entry> &e) { return nf4_muon_workspace_size(e.data(), (int32_t)e.size()); };
    // the bad entry last, at lengths around a launch's and far beyond
    for (size_t count : {1u, 79u, 80u, 81u, 5000u}) {
        std::vector<nf4_muon_entry> e(count, entry());
        const size_t need = size(e);
        EXPECT(need > 0 && need != (size_t)-1, true);
        EXPECT(step(e, need - 1), NF4_ERR_WORKSPACE);
        EXPECT(alone(e, need - 1), NF4_ERR_WORKSPACE);
        e.back().m = nullptr;
        EXPECT(step(e, SIZE_MAX), NF4_ERR_NULL);
        e.back() = entry();
        e.back().w = at<void>(8);
        EXPECT(step(e, SIZE_MAX), NF4_ERR_ALIGN);
        EXPECT(alone(e, SIZE_MAX), NF4_ERR_ALIGN);
        for (const auto &[rows, cols] : {std::pair<int64_t, int64_t>{257, 257}, {-1, 4}, {INT64_MAX, INT64_MAX}, {256, INT64_MAX},
                                         {1, int64_t(1) << 30}, {INT64_MIN, 0}}) {
            e.back() = entry(rows, cols);
            EXPECT(size(e), (size_t)-1);
            EXPECT(step(e, SIZE_MAX), NF4_ERR_SIZE);
            EXPECT(alone(e, SIZE_MAX), NF4_ERR_SIZE);
        }
        e.back() = entry();
        e.back().lr = NAN;
        EXPECT(step(e, SIZE_MAX), NF4_ERR_SIZE);
        e.back() = entry();
        e.back().master = at<float>();
        EXPECT(step(e, SIZE_MAX, NF4_F32), NF4_ERR_UNSUPPORTED);
    }
    // the longest matrices of every side, and the largest of them together
    std::vector<nf4_muon_entry> all;
    for (int64_t side : {1, 15, 16, 17, 32, 33, 63, 64, 65, 128, 129, 255, 256}) {
        const int64_t length = ((int64_t(1) << 30) - 1) / side;
        EXPECT(size({entry(side, length)}) != (size_t)-1, true);
        EXPECT(step({entry(length, side)}, 7), NF4_ERR_WORKSPACE);
        all.push_back(entry(side, length));
    }
    EXPECT(size(all) != (size_t)-1, true);
    // empty ones need nothing
    EXPECT(size({}), 0);
    EXPECT(step({}, 0), NF4_OK);
    EXPECT(nf4_muon_workspace_size(nullptr, 1), (size_t)-1);
    EXPECT(nf4_muon_workspace_size(nullptr, -1), (size_t)-1);
    std::vector<nf4_muon_entry> none{entry(0, 64), entry(INT64_MAX, 0)};
    for (auto &x : none) x.w = x.m = nullptr, x.grad = nullptr;
    EXPECT(step(none, size(none)), NF4_OK);
    for (auto change : {+[](nf4_muon_config &x) { x.eps = 0.0; }, +[](nf4_muon_config &x) { x.eps = NAN; },
                        +[](nf4_muon_config &x) { x.iterations = 0; }, +[](nf4_muon_config &x) { x.iterations = INT32_MAX; },
                        +[](nf4_muon_config &x) { x.b = INFINITY; }}) {
        const nf4_muon_config kept = c;
        change(c);
        EXPECT(step({entry()}, SIZE_MAX), NF4_ERR_SIZE);
        EXPECT(alone({entry()}, SIZE_MAX), NF4_ERR_SIZE);
        c = kept;
    }
    c.momentum = 1.0;
    EXPECT(step({entry()}, SIZE_MAX), NF4_ERR_SIZE);
    c.momentum = 0.95, c.nesterov = 2;
    EXPECT(step({entry()}, SIZE_MAX), NF4_ERR_UNSUPPORTED);
}

}  // namespace

int main() {
    rotation();
    muon();
    if (failures) return 1;
    std::puts("ok");
    return 0;
}
