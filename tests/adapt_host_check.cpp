// Host-side checks of the entry points around an adapted layer, built with the
// host sanitizers (AddressSanitizer, UndefinedBehaviorSanitizer): argument
// validation of each with every class of invalid argument, and the workspace
// queries at the extreme accepted shapes. Every call made here is rejected
// before anything is enqueued; the calls with valid arguments (answered
// I8MM_EDEVICE) are made only when the runtime reports no device, so no
// pointer below is ever handed to a kernel.
#include "i8mm.h"

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>

namespace {

int g_fail = 0;
int g_checks = 0;

void expect(bool ok, const char* what, int line) {
    ++g_checks;
    if (!ok) {
        std::printf("FAILED line %d: %s\n", line, what);
        ++g_fail;
    }
}
#define EXPECT(c) expect((c), #c, __LINE__)
#define EXPECT_STATUS(call, want) expect((call) == (want), #call " == " #want, __LINE__)

constexpr int64_t kMaxI64 = std::numeric_limits<int64_t>::max();
constexpr int64_t kMinI64 = std::numeric_limits<int64_t>::min();
const int64_t kBad[] = {-1, kMinI64, kMaxI64, int64_t(1) << 62, int64_t(1) << 33};   // lengths, counts and strides

// Distinct, 256-byte-aligned addresses that are never dereferenced, and one
// that no element type is aligned at.
template <typename T>
T* fake(uintptr_t k) { return reinterpret_cast<T*>(uintptr_t(1) << 40 | k << 12); }
template <typename T>
T* misaligned(uintptr_t k) { return reinterpret_cast<T*>((uintptr_t(1) << 40 | k << 12) + 1); }

struct Norm {
    const void *X = fake<void>(1), *w = fake<void>(2), *b = fake<void>(3);
    void* Y = fake<void>(4);
    float *mean = fake<float>(5), *rstd = fake<float>(6), *dw = fake<float>(8), *db = fake<float>(9);
    const void* dY = fake<void>(7);
    void *dX = fake<void>(10), *ws = fake<void>(11);
    int32_t xt = I8MM_F16, wt = I8MM_F32;
    int64_t s = 4, h = 100, ldx = 100, ldy = 104, lddy = 128, lddx = 100;
    float eps = 1e-5f;
    i8mm_status forward() const { return i8mm_layer_norm(X, ldx, xt, s, h, w, b, wt, eps, Y, ldy, mean, rstd, nullptr); }
    i8mm_status backward() const {
        return i8mm_layer_norm_backward(dY, lddy, X, ldx, xt, s, h, w, wt, mean, rstd, dX, lddx, dw, db, ws, nullptr);
    }
};

// f changes a copy of a valid call, which then has to be refused.
#define REFUSED(Type, call, change)                          \
    do {                                                     \
        Type a;                                              \
        change;                                              \
        EXPECT_STATUS(a.call(), I8MM_EINVAL);                \
    } while (0)

void check_norm(bool no_device) {
    for (int64_t v : kBad) {
        REFUSED(Norm, forward, a.s = v);
        REFUSED(Norm, forward, a.h = v);
        REFUSED(Norm, forward, a.ldx = v);
        REFUSED(Norm, forward, a.ldy = v);
        REFUSED(Norm, backward, a.s = v);
        REFUSED(Norm, backward, a.h = v);
        REFUSED(Norm, backward, a.ldx = v);
        REFUSED(Norm, backward, a.lddy = v);
        REFUSED(Norm, backward, a.lddx = v);
    }
    REFUSED(Norm, forward, a.h = 0);
    REFUSED(Norm, forward, a.ldx = 99);
    for (int32_t t : {-1, 3, std::numeric_limits<int32_t>::min(), std::numeric_limits<int32_t>::max()}) {
        REFUSED(Norm, forward, a.xt = t);
        REFUSED(Norm, forward, a.wt = t);
        REFUSED(Norm, backward, a.xt = t);
        REFUSED(Norm, backward, a.wt = t);
    }
    REFUSED(Norm, forward, a.wt = I8MM_BF16);
    for (float e : {-1.0f, INFINITY, -INFINITY, NAN}) REFUSED(Norm, forward, a.eps = e);
    REFUSED(Norm, forward, a.X = nullptr);
    REFUSED(Norm, forward, a.Y = nullptr);
    REFUSED(Norm, forward, a.w = nullptr);
    REFUSED(Norm, forward, a.X = misaligned<void>(1));
    REFUSED(Norm, forward, a.w = misaligned<void>(1));
    REFUSED(Norm, forward, a.b = misaligned<void>(1));
    REFUSED(Norm, forward, a.Y = misaligned<void>(1));
    REFUSED(Norm, forward, a.mean = misaligned<float>(1));
    REFUSED(Norm, forward, a.rstd = misaligned<float>(1));
    REFUSED(Norm, forward, a.Y = const_cast<void*>(a.X));
    REFUSED(Norm, backward, a.dY = nullptr);
    REFUSED(Norm, backward, a.mean = nullptr);
    REFUSED(Norm, backward, a.rstd = nullptr);
    REFUSED(Norm, backward, a.dX = nullptr);
    REFUSED(Norm, backward, a.ws = nullptr);
    REFUSED(Norm, backward, a.ws = misaligned<void>(1));
    REFUSED(Norm, backward, a.dw = misaligned<float>(1));
    REFUSED(Norm, backward, a.dX = const_cast<void*>(a.dY));
    if (no_device) {
        EXPECT_STATUS(Norm().forward(), I8MM_EDEVICE);
        EXPECT_STATUS(Norm().backward(), I8MM_EDEVICE);
    }
    for (int64_t s : {int64_t(0), int64_t(1), int64_t(255), int64_t(256), int64_t(1) << 26, (int64_t(1) << 31) - 1})
        for (int64_t h : {int64_t(1), int64_t(64), int64_t(16385), int64_t(I8MM_NORM_MAX_H)}) {
            const size_t n = i8mm_layer_norm_backward_workspace_bytes(s, h);
            EXPECT(n >= size_t(8 * h) && n % 256 == 0);
        }
    for (int64_t v : kBad) {
        EXPECT(i8mm_layer_norm_backward_workspace_bytes(v, 64) == 0);
        EXPECT(i8mm_layer_norm_backward_workspace_bytes(4, v) == 0);
    }
}

struct Lora {
    const void *X = fake<void>(1), *dY = fake<void>(2), *A = fake<void>(3), *B = fake<void>(4), *base = fake<void>(5);
    const int32_t* ids = fake<int32_t>(6);
    const float* scale = fake<float>(7);
    void *Y = fake<void>(8), *dX = fake<void>(9), *ws = fake<void>(10);
    float *T = fake<float>(11), *dA = fake<float>(12), *dB = fake<float>(13);
    int32_t t = I8MM_BF16;
    int64_t s = 4, h = 128, o = 128, r = 5, G = 3, ldx = 128, ldy = 136, ldb = 128, lddy = 128, lddx = 128;
    i8mm_status forward() const {
        return i8mm_lora_forward(X, ldx, A, B, t, G, r, ids, scale, base, ldb, s, h, o, Y, ldy, T, ws, nullptr);
    }
    i8mm_status backward() const {
        return i8mm_lora_backward(dY, lddy, X, ldx, T, A, B, t, G, r, ids, scale, base, ldb, s, h, o, dX, lddx, dA, dB,
                                  ws, nullptr);
    }
};

#define REFUSED_BOTH(change)             \
    do {                                 \
        REFUSED(Lora, forward, change);  \
        REFUSED(Lora, backward, change); \
    } while (0)

void check_lora(bool no_device) {
    for (int64_t v : kBad) {
        REFUSED_BOTH(a.s = v);
        REFUSED_BOTH(a.h = v);
        REFUSED_BOTH(a.o = v);
        REFUSED_BOTH(a.r = v);
        REFUSED_BOTH(a.G = v);
        REFUSED_BOTH(a.ldx = v);
        REFUSED_BOTH(a.ldb = v);
        REFUSED(Lora, forward, a.ldy = v);
        REFUSED(Lora, backward, a.lddy = v);
        REFUSED(Lora, backward, a.lddx = v);
    }
    REFUSED_BOTH(a.s = I8MM_LORA_MAX_ROWS + 1);
    REFUSED_BOTH(a.r = I8MM_LORA_MAX_RANK + 1);
    REFUSED_BOTH(a.r = 0);
    REFUSED_BOTH(a.G = I8MM_LORA_MAX_ADAPTERS + 1);
    REFUSED_BOTH(a.G = 0);
    REFUSED_BOTH(a.h = 96);
    REFUSED_BOTH(a.o = 0);
    REFUSED_BOTH(a.t = I8MM_F32);
    REFUSED_BOTH(a.t = -1);
    REFUSED_BOTH(a.A = nullptr);
    REFUSED_BOTH(a.B = nullptr);
    REFUSED_BOTH(a.X = nullptr);
    REFUSED_BOTH(a.ids = nullptr);
    REFUSED_BOTH(a.scale = nullptr);
    REFUSED_BOTH(a.ws = nullptr);
    REFUSED_BOTH(a.A = misaligned<void>(1));
    REFUSED_BOTH(a.B = misaligned<void>(1));
    REFUSED_BOTH(a.X = misaligned<void>(1));
    REFUSED_BOTH(a.ids = misaligned<int32_t>(1));
    REFUSED_BOTH(a.scale = misaligned<float>(1));
    REFUSED_BOTH(a.base = misaligned<void>(1));
    REFUSED_BOTH(a.T = misaligned<float>(1));
    REFUSED_BOTH(a.ws = misaligned<void>(1));
    REFUSED(Lora, forward, a.Y = nullptr);
    REFUSED(Lora, forward, a.Y = const_cast<void*>(a.X));
    REFUSED(Lora, forward, a.Y = const_cast<void*>(a.base));     // another stride
    REFUSED(Lora, backward, a.dY = nullptr);
    REFUSED(Lora, backward, a.T = nullptr);
    REFUSED(Lora, backward, a.dA = nullptr);
    REFUSED(Lora, backward, a.dB = misaligned<float>(1));
    REFUSED(Lora, backward, a.dX = const_cast<void*>(a.dY));
    if (no_device) {
        EXPECT_STATUS(Lora().forward(), I8MM_EDEVICE);
        EXPECT_STATUS(Lora().backward(), I8MM_EDEVICE);
    }
    for (int64_t s : {int64_t(0), int64_t(1), int64_t(256), int64_t(257), int64_t(4097), int64_t(1) << 20,
                      int64_t(I8MM_LORA_MAX_ROWS)})
        for (int64_t h : {int64_t(64), int64_t(12288), int64_t(I8MM_MAX_H)})
            for (int64_t o : {int64_t(64), int64_t(I8MM_MAX_H)})
                for (int64_t r : {1, 33, I8MM_LORA_MAX_RANK}) {
                    EXPECT(i8mm_lora_forward_workspace_bytes(s, h, o, r) >= size_t(4 * s * r));
                    for (int64_t G : {1, 300, I8MM_LORA_MAX_ADAPTERS})
                        EXPECT(i8mm_lora_backward_workspace_bytes(s, h, o, r, G) >= size_t(8 * s * r));
                }
    for (int64_t v : kBad) {
        EXPECT(i8mm_lora_forward_workspace_bytes(v, 64, 64, 4) == 0);
        EXPECT(i8mm_lora_forward_workspace_bytes(4, v, 64, 4) == 0);
        EXPECT(i8mm_lora_forward_workspace_bytes(4, 64, v, 4) == 0);
        EXPECT(i8mm_lora_forward_workspace_bytes(4, 64, 64, v) == 0);
        EXPECT(i8mm_lora_backward_workspace_bytes(4, 64, 64, 4, v) == 0);
    }
}

struct Clip {
    const void* grads[4] = {fake<void>(1), fake<void>(2), nullptr, fake<void>(3)};
    void* outs[4] = {fake<void>(4), fake<void>(2), nullptr, fake<void>(5)};
    int64_t numels[4] = {5, 1 << 20, 0, int64_t(1) << 43};
    int32_t types[4] = {I8MM_F16, I8MM_F32, I8MM_BF16, I8MM_BF16};
    int64_t n = 4;
    float max_norm = 1.0f;
    void* ws = fake<void>(6);
    float* total = fake<float>(7);
    bool into = true;
    i8mm_status call() const {
        return i8mm_clip_grad_norm(grads, into ? outs : nullptr, numels, types, n, max_norm, ws, total, nullptr);
    }
};

void check_clip(bool no_device) {
    for (int64_t v : kBad) {
        REFUSED(Clip, call, a.n = v);
        EXPECT(i8mm_clip_grad_norm_workspace_bytes(nullptr, v) == 0);
    }
    for (int64_t v : {int64_t(-1), kMinI64, kMaxI64, (int64_t(1) << 44) - 3}) REFUSED(Clip, call, a.numels[0] = v);
    for (int32_t t : {-1, 3, std::numeric_limits<int32_t>::min()}) REFUSED(Clip, call, a.types[2] = t);
    for (float m : {-1.0f, -INFINITY, NAN}) REFUSED(Clip, call, a.max_norm = m);
    REFUSED(Clip, call, a.grads[1] = nullptr);
    REFUSED(Clip, call, a.grads[3] = misaligned<void>(1));
    REFUSED(Clip, call, a.outs[0] = nullptr);
    REFUSED(Clip, call, a.outs[0] = misaligned<void>(1));
    REFUSED(Clip, call, a.ws = nullptr);
    REFUSED(Clip, call, a.ws = misaligned<void>(1));
    REFUSED(Clip, call, a.total = nullptr);
    REFUSED(Clip, call, a.total = misaligned<float>(1));
    EXPECT_STATUS(i8mm_clip_grad_norm(nullptr, nullptr, nullptr, nullptr, 1, 1.0f, fake<void>(6), fake<float>(7), nullptr),
                  I8MM_EINVAL);
    const Clip c;
    for (int64_t n = 0; n <= 4; ++n) EXPECT(i8mm_clip_grad_norm_workspace_bytes(c.numels, n) >= 256);
    if (no_device) {
        for (bool into : {true, false}) {
            Clip a;
            a.into = into;
            EXPECT_STATUS(a.call(), I8MM_EDEVICE);
            a.n = 0;
            EXPECT_STATUS(a.call(), I8MM_EDEVICE);
        }
    }
}

}  // namespace

int main() {
    int devices = 0;
    const bool no_device = hipGetDeviceCount(&devices) != hipSuccess || devices == 0;
    check_norm(no_device);
    check_lora(no_device);
    check_clip(no_device);
    std::printf("%d checks, %d failed\n", g_checks, g_fail);
    return g_fail == 0 ? 0 : 1;
}
