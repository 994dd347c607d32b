// Host-side checks of the entry points of decoding (paged cache, its attention,
// beam selection), built with the host sanitizers (AddressSanitizer,
// UndefinedBehaviorSanitizer): every class of invalid argument, the workspace
// queries at the extreme accepted shapes, and host arrays of many pools. Calls
// with valid arguments (answered I8MM_EDEVICE) are made only when the runtime
// reports no device, so no pointer below is ever handed to a kernel.
#include "i8mm.h"

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>
#include <vector>

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

constexpr int64_t kMaxI64 = std::numeric_limits<int64_t>::max();
constexpr int64_t kMinI64 = std::numeric_limits<int64_t>::min();
const int64_t kBad[] = {-1, kMinI64, kMaxI64, int64_t(1) << 62, int64_t(1) << 41};

template <typename T>
T* fake(uintptr_t k) { return reinterpret_cast<T*>(uintptr_t(1) << 40 | k << 12); }

struct Cache {
    const void *K = fake<void>(1), *V = fake<void>(2), *Q = fake<void>(3);
    void *Kp = fake<void>(4), *Vp = fake<void>(5), *out = fake<void>(6), *ws = fake<void>(7);
    const int32_t *seq = fake<int32_t>(8), *pos = fake<int32_t>(9), *tables = fake<int32_t>(10), *lens = fake<int32_t>(11);
    const float* slopes = fake<float>(12);
    float* lse = fake<float>(13);
    int32_t type = I8MM_F16;
    int64_t s = 3, heads = 4, kv = 2, d = 80, ldk = 160, ldv = 168, ldq = 320, ldo = 328, n = 4, M = 40, ldt = 44, P = 9, page = 48,
            ks = 2 * 48 * 80, vs = 2 * 48 * 80 + 8, beams = 2;
    float scale = 0.1f;
    i8mm_status append() const {
        return i8mm_cache_append(K, ldk, V, ldv, type, s, kv, d, seq, pos, tables, ldt, n, M, Kp, ks, Vp, vs, P, page, nullptr);
    }
    i8mm_status attend() const {
        return i8mm_decode_attention(Q, ldq, type, n, heads, kv, d, Kp, ks, Vp, vs, P, page, tables, ldt, M, lens, beams, scale,
                                     slopes, out, ldo, lse, ws, nullptr);
    }
};

struct Books {
    const int32_t *tables = fake<int32_t>(1), *lens = fake<int32_t>(2), *refs = fake<int32_t>(3), *parents = fake<int32_t>(4),
                  *grow = fake<int32_t>(5);
    int32_t *to = fake<int32_t>(6), *lo = fake<int32_t>(7), *ro = fake<int32_t>(8), *state = fake<int32_t>(9),
            *moved = fake<int32_t>(10);
    void* ws = fake<void>(11);
    int64_t ldt = 7, ldto = 9, n = 3, M = 7, P = 100, page = 16, m = 5;
    std::vector<void*> at = std::vector<void*>(300, fake<void>(12));
    std::vector<int64_t> size = std::vector<int64_t>(300, 4096), step = std::vector<int64_t>(300, 8192);
    int64_t pools = 300;
    i8mm_status fork() const {
        return i8mm_cache_fork(tables, ldt, lens, refs, n, M, P, page, parents, grow, m, to, ldto, lo, ro, state, at.data(),
                               size.data(), step.data(), pools, ws, nullptr);
    }
    i8mm_status compact() const {
        return i8mm_cache_compact(tables, ldt, n, M, refs, P, to, ldto, ro, moved, state, at.data(), size.data(), step.data(), pools,
                                  ws, nullptr);
    }
};

struct Select {
    const void* x = fake<void>(1);
    const float* scores = fake<float>(2);
    float* so = fake<float>(3);
    int32_t *parents = fake<int32_t>(4), *tokens = fake<int32_t>(5), *ho = fake<int32_t>(7);
    const int32_t* h = fake<int32_t>(6);
    void* ws = fake<void>(8);
    int32_t type = I8MM_F32;
    int64_t ld = 100, n = 3, beams = 4, vocab = 99, k = 8, ldh = 7, T = 7, ldho = 8;
    i8mm_status select() const {
        return i8mm_beam_select(x, ld, type, n, beams, vocab, scores, k, so, parents, tokens, h, ldh, T, ho, ldho, ws, nullptr);
    }
};

// f changes a copy of a valid call, which then has to be refused.
#define REFUSED(Type, call, change)                                                             \
    do {                                                                                        \
        Type a;                                                                                 \
        change;                                                                                 \
        expect(a.call() == I8MM_EINVAL, #Type " " #call " refuses " #change, __LINE__);         \
    } while (0)
#define REFUSED_BAD(Type, call, field) \
    for (int64_t v : kBad) REFUSED(Type, call, a.field = v)

void check_cache() {
    REFUSED_BAD(Cache, append, s);
    REFUSED_BAD(Cache, append, kv);
    REFUSED_BAD(Cache, append, d);
    REFUSED_BAD(Cache, append, ldk);
    REFUSED_BAD(Cache, append, ldv);
    REFUSED_BAD(Cache, append, n);
    REFUSED_BAD(Cache, append, M);
    REFUSED_BAD(Cache, append, ldt);
    REFUSED_BAD(Cache, append, P);
    REFUSED_BAD(Cache, append, page);
    REFUSED_BAD(Cache, append, ks);
    REFUSED_BAD(Cache, append, vs);
    REFUSED_BAD(Cache, attend, heads);
    REFUSED_BAD(Cache, attend, kv);
    REFUSED_BAD(Cache, attend, d);
    REFUSED_BAD(Cache, attend, ldq);
    REFUSED_BAD(Cache, attend, ldo);
    REFUSED_BAD(Cache, attend, n);
    REFUSED_BAD(Cache, attend, M);
    REFUSED_BAD(Cache, attend, ldt);
    REFUSED_BAD(Cache, attend, P);
    REFUSED_BAD(Cache, attend, page);
    REFUSED_BAD(Cache, attend, ks);
    REFUSED_BAD(Cache, attend, vs);
    REFUSED_BAD(Cache, attend, beams);
    for (int32_t t : {-1, 2, 3, std::numeric_limits<int32_t>::min(), std::numeric_limits<int32_t>::max()}) {
        REFUSED(Cache, append, a.type = t);
        REFUSED(Cache, attend, a.type = t);
    }
    REFUSED(Cache, append, a.K = nullptr);
    REFUSED(Cache, append, a.Vp = nullptr);
    REFUSED(Cache, attend, a.ws = nullptr);
    REFUSED(Cache, attend, a.out = const_cast<void*>(a.Q));
    REFUSED(Cache, attend, a.scale = std::numeric_limits<float>::quiet_NaN());
    REFUSED(Cache, attend, a.scale = -std::numeric_limits<float>::infinity());
    for (int64_t n : {int64_t(0), int64_t(1), int64_t(I8MM_CACHE_MAX_SEQS)})
        for (int64_t h : {1, 7, 65535})
            for (int64_t d : {8, 80, I8MM_CACHE_MAX_HEAD}) EXPECT(i8mm_decode_attention_workspace_bytes(n, h, 1, d) > 0);
    for (int64_t v : kBad) {
        EXPECT(i8mm_decode_attention_workspace_bytes(v, 4, 4, 64) == 0);
        EXPECT(i8mm_decode_attention_workspace_bytes(4, v, 4, 64) == 0);
        EXPECT(i8mm_decode_attention_workspace_bytes(4, 4, v, 64) == 0);
        EXPECT(i8mm_decode_attention_workspace_bytes(4, 4, 4, v) == 0);
    }
}

void check_books() {
    REFUSED_BAD(Books, fork, n);
    REFUSED_BAD(Books, fork, m);
    REFUSED_BAD(Books, fork, M);
    REFUSED_BAD(Books, fork, P);
    REFUSED_BAD(Books, fork, page);
    REFUSED_BAD(Books, fork, ldt);
    REFUSED_BAD(Books, fork, ldto);
    REFUSED_BAD(Books, fork, pools);
    REFUSED_BAD(Books, compact, n);
    REFUSED_BAD(Books, compact, M);
    REFUSED_BAD(Books, compact, P);
    REFUSED_BAD(Books, compact, ldt);
    REFUSED_BAD(Books, compact, ldto);
    REFUSED_BAD(Books, compact, pools);
    for (int k : {0, 128, 299}) {                     // the last pool of a launch's batch, and of all
        REFUSED(Books, fork, a.at[k] = nullptr);
        REFUSED(Books, fork, a.size[k] = 24);
        REFUSED(Books, compact, a.step[k] = 4080);
        for (int64_t v : kBad) {
            REFUSED(Books, fork, a.size[k] = v);
            REFUSED(Books, compact, a.step[k] = v);
        }
    }
    REFUSED(Books, fork, a.to = const_cast<int32_t*>(a.tables));
    REFUSED(Books, fork, a.ro = const_cast<int32_t*>(a.refs));
    REFUSED(Books, compact, a.ro = const_cast<int32_t*>(a.refs));
    REFUSED(Books, compact, a.to = const_cast<int32_t*>(a.tables));       // with another stride
    for (int64_t v : kBad) {
        EXPECT(i8mm_cache_fork_workspace_bytes(v, 1, 1) == 0);
        EXPECT(i8mm_cache_fork_workspace_bytes(1, v, 1) == 0);
        EXPECT(i8mm_cache_fork_workspace_bytes(1, 1, v) == 0);
        EXPECT(i8mm_cache_compact_workspace_bytes(v) == 0);
    }
    EXPECT(i8mm_cache_fork_workspace_bytes(I8MM_CACHE_MAX_SEQS, I8MM_CACHE_MAX_SEQS, I8MM_CACHE_MAX_PAGES) > 0);
    EXPECT(i8mm_cache_compact_workspace_bytes(I8MM_CACHE_MAX_PAGES) > 0);
}

void check_select() {
    REFUSED_BAD(Select, select, ld);
    REFUSED_BAD(Select, select, n);
    REFUSED_BAD(Select, select, beams);
    REFUSED_BAD(Select, select, vocab);
    REFUSED_BAD(Select, select, k);
    REFUSED_BAD(Select, select, ldh);
    REFUSED_BAD(Select, select, T);
    REFUSED_BAD(Select, select, ldho);
    REFUSED(Select, select, a.h = nullptr);
    REFUSED(Select, select, a.so = const_cast<float*>(a.scores));
    REFUSED(Select, select, (a.beams = 1, a.vocab = 7));
    for (int64_t n : {int64_t(0), int64_t(1), int64_t(I8MM_CACHE_MAX_SEQS)})
        for (int64_t v : {1, 50257, I8MM_BEAM_MAX_VOCAB}) EXPECT(i8mm_beam_select_workspace_bytes(n, 64, v, 64) >= 256);
    for (int64_t v : kBad) {
        EXPECT(i8mm_beam_select_workspace_bytes(v, 1, 9, 1) == 0);
        EXPECT(i8mm_beam_select_workspace_bytes(1, v, 9, 1) == 0);
        EXPECT(i8mm_beam_select_workspace_bytes(1, 1, v, 1) == 0);
        EXPECT(i8mm_beam_select_workspace_bytes(1, 1, 9, v) == 0);
    }
}

}  // namespace

int main() {
    check_cache();
    check_books();
    check_select();
    int devices = 0;
    if (hipGetDeviceCount(&devices) != hipSuccess || devices == 0) {
        EXPECT(Cache().append() == I8MM_EDEVICE);
        EXPECT(Cache().attend() == I8MM_EDEVICE);
        EXPECT(Books().fork() == I8MM_EDEVICE);
        EXPECT(Books().compact() == I8MM_EDEVICE);
        EXPECT(Select().select() == I8MM_EDEVICE);
    }
    std::printf("%d checks, %d failed\n", g_checks, g_fail);
    return g_fail ? 1 : 0;
}
