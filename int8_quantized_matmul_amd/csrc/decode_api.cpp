// C-ABI layer of the entry points of decoding between int8 layers (paged
// cache, its attention, beam selection): host-side validation, the device
// check and the launch of each, as declared in include/i8mm.h.

#include "../../include/i8mm.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "host_checks.h"
#include "launch.h"

namespace {

using i8mm::aligned16;
using i8mm::aligned_to;
using i8mm::check_device;
using i8mm::Dtype;
using i8mm::launched;

// Between pages and rows, and from the first to the last of them: byte offsets stay below
// 2^63 (elements are 4 bytes at most).
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxSpan = int64_t(1) << 60;

bool aligned256(const void* p) { return aligned_to(p, 256); }
bool aligned4(const void* p) { return aligned_to(p, 4); }

bool between(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

bool valid_pages(int64_t n_pages, int64_t page, int64_t max_pages) {
    return between(n_pages, 1, I8MM_CACHE_MAX_PAGES) && between(page, 16, I8MM_CACHE_MAX_PAGE) && page % 16 == 0 &&
           between(max_pages, 1, I8MM_CACHE_MAX_ROW) && max_pages * page < (int64_t(1) << 31) - 4096;
}

bool valid_sequences(int64_t n) { return between(n, 0, I8MM_CACHE_MAX_SEQS); }

// `count` rows of `len`, ld apart
bool valid_row(int64_t ld, int64_t len, int64_t count) {
    return between(ld, len, kMaxStride) && (count <= 1 || ld <= kMaxSpan / count);
}

bool valid_heads(int64_t heads, int64_t d) {
    return between(heads, 1, 65535) && between(d, 8, I8MM_CACHE_MAX_HEAD) && d % 8 == 0;
}

// A 16-byte aligned matrix whose rows (or pages) are too.
bool valid_rows16(const void* p, int64_t ld, int64_t len, int64_t count) {
    return aligned16(p) && ld % 8 == 0 && valid_row(ld, len, count);
}

bool valid_half(int32_t t) { return t == I8MM_F16 || t == I8MM_BF16; }

bool valid_pools(void* const* pools, const int64_t* bytes, const int64_t* strides, int64_t n, int64_t n_pages) {
    if (!between(n, 0, 65536) || (n > 0 && (!pools || !bytes || !strides))) return false;
    for (int64_t i = 0; i < n; ++i) {
        if (!pools[i] || !aligned16(pools[i]) || !between(bytes[i], 16, int64_t(1) << 32) || bytes[i] % 16 != 0 ||
            strides[i] % 16 != 0 || !valid_row(strides[i], bytes[i], n_pages))
            return false;
    }
    return true;
}

bool valid_selection(int64_t n, int64_t beams, int64_t vocab, int64_t k) {
    return between(n, 0, I8MM_CACHE_MAX_SEQS) && between(beams, 1, I8MM_BEAM_MAX) && between(vocab, 1, I8MM_BEAM_MAX_VOCAB) &&
           between(k, 1, I8MM_BEAM_MAX) && k <= beams * vocab;
}

}  // namespace

extern "C" {

i8mm_status i8mm_cache_append(const void* K, int64_t ldk, const void* V, int64_t ldv, int32_t type, int64_t s,
                              int64_t kv_heads, int64_t d, const int32_t* seq, const int32_t* pos, const int32_t* tables,
                              int64_t ldt, int64_t n, int64_t max_pages, void* K_pages, int64_t k_stride, void* V_pages,
                              int64_t v_stride, int64_t n_pages, int64_t page, hipStream_t stream) {
    // seq may be null
    if (!valid_half(type) || !valid_heads(kv_heads, d) || !valid_pages(n_pages, page, max_pages) || !valid_sequences(n) ||
        !between(s, 0, I8MM_CACHE_MAX_APPEND))
        return I8MM_EINVAL;
    if (!K_pages || !V_pages || (s != 0 && (!K || !V || !pos)) || (n != 0 && !tables)) return I8MM_EINVAL;
    if (!valid_rows16(K, ldk, kv_heads * d, s) || !valid_rows16(V, ldv, kv_heads * d, s) ||
        !valid_rows16(K_pages, k_stride, kv_heads * page * d, n_pages) ||
        !valid_rows16(V_pages, v_stride, kv_heads * page * d, n_pages) || !valid_row(ldt, max_pages, n) || !aligned4(seq) ||
        !aligned4(pos) || !aligned4(tables))
        return I8MM_EINVAL;
    if (i8mm_status e = check_device()) return e;
    const i8mm::AppendArgs a{K, V, ldk, ldv, 2, s, static_cast<int>(kv_heads), static_cast<int>(d), seq, pos, tables, ldt, n,
                             static_cast<int>(max_pages), K_pages, V_pages, k_stride, v_stride, static_cast<int>(n_pages),
                             static_cast<int>(page)};
    return launched(i8mm::launch_cache_append(a, stream));
}

size_t i8mm_cache_fork_workspace_bytes(int64_t n, int64_t n_out, int64_t n_pages) {
    if (!valid_sequences(n) || !valid_sequences(n_out) || !between(n_pages, 1, I8MM_CACHE_MAX_PAGES)) return 0;
    return i8mm::cache_fork_scratch(n, n_out, n_pages);
}

i8mm_status i8mm_cache_fork(const int32_t* tables, int64_t ldt, const int32_t* lens, const int32_t* refs, int64_t n,
                            int64_t max_pages, int64_t n_pages, int64_t page, const int32_t* parents, const int32_t* grow,
                            int64_t n_out, int32_t* tables_out, int64_t ldto, int32_t* lens_out, int32_t* refs_out,
                            int32_t* state, void* const* pools, const int64_t* page_bytes, const int64_t* strides,
                            int64_t n_pools, void* workspace, hipStream_t stream) {
    // parents and grow may be null
    if (!valid_pages(n_pages, page, max_pages) || !valid_sequences(n) || !valid_sequences(n_out)) return I8MM_EINVAL;
    if (!refs || !refs_out || !state || !workspace || (n != 0 && (!tables || !lens)) ||
        (n_out != 0 && (!tables_out || !lens_out)))
        return I8MM_EINVAL;
    if (!valid_row(ldt, max_pages, n) || !valid_row(ldto, max_pages, n_out) || !aligned4(tables) || !aligned4(lens) ||
        !aligned4(refs) ||
        !aligned4(parents) || !aligned4(grow) || !aligned4(tables_out) || !aligned4(lens_out) || !aligned4(refs_out) ||
        !aligned4(state) || !aligned256(workspace))
        return I8MM_EINVAL;
    if (refs == refs_out || (n_out != 0 && (tables == tables_out || lens == lens_out))) return I8MM_EINVAL;
    if (!valid_pools(pools, page_bytes, strides, n_pools, n_pages)) return I8MM_EINVAL;
    if (i8mm_status e = check_device()) return e;
    const i8mm::ForkArgs a{tables, ldt, lens, refs, n, static_cast<int>(max_pages), static_cast<int>(n_pages),
                           static_cast<int>(page), parents, grow, n_out, tables_out, ldto, lens_out, refs_out, state};
    return launched(i8mm::launch_cache_fork(a, {pools, page_bytes, strides, n_pools}, workspace, stream));
}

size_t i8mm_cache_compact_workspace_bytes(int64_t n_pages) {
    if (!between(n_pages, 1, I8MM_CACHE_MAX_PAGES)) return 0;
    return i8mm::cache_compact_scratch(n_pages);
}

i8mm_status i8mm_cache_compact(const int32_t* tables, int64_t ldt, int64_t n, int64_t max_pages, const int32_t* refs,
                               int64_t n_pages, int32_t* tables_out, int64_t ldto, int32_t* refs_out, int32_t* moved,
                               int32_t* state, void* const* pools, const int64_t* page_bytes, const int64_t* strides,
                               int64_t n_pools, void* workspace, hipStream_t stream) {
    if (!valid_pages(n_pages, 16, max_pages) || !valid_sequences(n)) return I8MM_EINVAL;
    if (!refs || !refs_out || !moved || !state || !workspace || (n != 0 && (!tables || !tables_out))) return I8MM_EINVAL;
    if (!valid_row(ldt, max_pages, n) || !valid_row(ldto, max_pages, n) || !aligned4(tables) || !aligned4(refs) ||
        !aligned4(tables_out) || !aligned4(refs_out) || !aligned4(moved) || !aligned4(state) || !aligned256(workspace))
        return I8MM_EINVAL;
    if (refs == refs_out || (n > 1 && tables == tables_out && ldt != ldto)) return I8MM_EINVAL;
    if (!valid_pools(pools, page_bytes, strides, n_pools, n_pages)) return I8MM_EINVAL;
    if (i8mm_status e = check_device()) return e;
    const i8mm::CompactArgs a{tables, ldt, n, static_cast<int>(max_pages), refs, static_cast<int>(n_pages), tables_out, ldto,
                              refs_out, moved, state};
    return launched(i8mm::launch_cache_compact(a, {pools, page_bytes, strides, n_pools}, workspace, stream));
}

size_t i8mm_decode_attention_workspace_bytes(int64_t n, int64_t heads, int64_t kv_heads, int64_t d) {
    if (!valid_sequences(n) || !valid_heads(heads, d) || !between(kv_heads, 1, heads) || heads % kv_heads != 0) return 0;
    return i8mm::decode_attention_scratch(n, static_cast<int>(heads), static_cast<int>(kv_heads), static_cast<int>(d));
}

i8mm_status i8mm_decode_attention(const void* Q, int64_t ldq, int32_t type, int64_t n, int64_t heads, int64_t kv_heads,
                                  int64_t d, const void* K_pages, int64_t k_stride, const void* V_pages, int64_t v_stride,
                                  int64_t n_pages, int64_t page, const int32_t* tables, int64_t ldt, int64_t max_pages,
                                  const int32_t* lens, int64_t beams, float scale, const float* slopes, void* out,
                                  int64_t ldo, float* lse, void* workspace, hipStream_t stream) {
    // slopes and lse may be null
    if (!valid_half(type) || !valid_heads(heads, d) || !between(kv_heads, 1, heads) || heads % kv_heads != 0 ||
        !valid_pages(n_pages, page, max_pages) || !valid_sequences(n) || !between(beams, 1, I8MM_BEAM_MAX) || n % beams != 0 ||
        !std::isfinite(scale))
        return I8MM_EINVAL;
    if (!K_pages || !V_pages || (!workspace && !i8mm::attention_takes_whole(max_pages * page, beams)) ||
        (n != 0 && (!Q || !tables || !lens || !out)))
        return I8MM_EINVAL;
    if (!valid_rows16(Q, ldq, heads * d, n) || !valid_rows16(out, ldo, heads * d, n) ||
        !valid_rows16(K_pages, k_stride, kv_heads * page * d, n_pages) ||
        !valid_rows16(V_pages, v_stride, kv_heads * page * d, n_pages) || !valid_row(ldt, max_pages, n) || !aligned4(tables) ||
        !aligned4(lens) || !aligned4(slopes) || !aligned4(lse) ||
        !aligned256(workspace))
        return I8MM_EINVAL;
    if (n > 0 && out == Q) return I8MM_EINVAL;
    if (i8mm_status e = check_device()) return e;
    const i8mm::AttendArgs a{Q, ldq, static_cast<Dtype>(type), n, static_cast<int>(heads), static_cast<int>(kv_heads),
                             static_cast<int>(d), K_pages, V_pages, k_stride, v_stride, static_cast<int>(n_pages),
                             static_cast<int>(page), tables, ldt, static_cast<int>(max_pages), lens, static_cast<int>(beams),
                             scale, slopes, out, ldo, lse};
    return launched(i8mm::launch_decode_attention(a, workspace, stream));
}

size_t i8mm_beam_select_workspace_bytes(int64_t n, int64_t beams, int64_t vocab, int64_t k) {
    if (!valid_selection(n, beams, vocab, k)) return 0;
    const size_t bytes = i8mm::beam_select_scratch(n, static_cast<int>(beams), static_cast<int>(vocab), static_cast<int>(k));
    return bytes > 256 ? bytes : 256;
}

i8mm_status i8mm_beam_select(const void* logits, int64_t ld, int32_t type, int64_t n, int64_t beams, int64_t vocab,
                             const float* scores, int64_t k, float* scores_out, int32_t* parents, int32_t* tokens,
                             const int32_t* history, int64_t ldh, int64_t T, int32_t* history_out, int64_t ldho,
                             void* workspace, hipStream_t stream) {
    // history_out may be null, and history if T is 0
    if (!valid_half(type) && type != I8MM_F32) return I8MM_EINVAL;
    if (!valid_selection(n, beams, vocab, k)) return I8MM_EINVAL;
    if (!workspace || (n != 0 && (!logits || !scores || !scores_out || !parents || !tokens))) return I8MM_EINVAL;
    if (!valid_row(ld, vocab, n * beams) || !aligned_to(logits, type == I8MM_F32 ? 4 : 2) || !aligned4(scores) ||
        !aligned4(scores_out) ||
        !aligned4(parents) || !aligned4(tokens) || !aligned256(workspace))
        return I8MM_EINVAL;
    if (n > 0 && scores == scores_out) return I8MM_EINVAL;
    if (history_out) {
        if (!between(T, 0, (int64_t(1) << 31) - 2) || (T > 0 && n > 0 && !history) || !valid_row(ldh, T, n * beams) ||
            !valid_row(ldho, T + 1, n * k) || !aligned4(history) || !aligned4(history_out) || (n > 0 && history == history_out))
            return I8MM_EINVAL;
    }
    if (i8mm_status e = check_device()) return e;
    const i8mm::SelectArgs a{logits, ld, static_cast<Dtype>(type), n, static_cast<int>(beams), static_cast<int>(vocab), scores,
                             static_cast<int>(k), scores_out, parents, tokens, history, ldh, T, history_out, ldho};
    return launched(i8mm::launch_beam_select(a, workspace, stream));
}

}  // extern "C"
