// Host-side launchers of the gfx950 kernels. Arguments are validated by the
// C-ABI layer (api.cpp) before any of these is called; each launcher only
// picks a grid and enqueues work on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace i8mm {

// Threads that one dimension of a grid can have. What is beyond them does not
// run, and the launch reports no error.
constexpr int64_t kGridThreads = (int64_t(1) << 32) - 1;

// Rows of the int8 path's row kernels that one launch takes, at a block of 256
// threads a row or less; more go in runs.
constexpr int64_t kRowsAtOnce = int64_t(1) << 23;

// Calls f(first, n) for s rows in runs of at most `most`, until one fails.
template <typename F>
hipError_t for_row_runs(int64_t s, int64_t most, F&& f) {
    for (int64_t first = 0; first < s; first += most) {
        const hipError_t e = f(first, s - first < most ? s - first : most);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_detect(const uint16_t* X, int64_t s, int64_t h, float alpha,
                         uint32_t* mask, int32_t* idx, int32_t* n_out, hipStream_t stream);

// p[0 .. n) = v (one small kernel; also clears state inside captured graphs,
// where a memset node is avoided).
hipError_t launch_fill_u32(uint32_t* p, int64_t n, uint32_t v, hipStream_t stream);

hipError_t launch_quantize_rows(const uint16_t* X, int64_t s, int64_t h,
                                const uint32_t* mask, const int32_t* idx, const int32_t* n_out,
                                int8_t* Xq, float* c_x, uint16_t* X_O, int64_t ldo,
                                hipStream_t stream);

// Forward path: detection + index list + row quantisation in two launches,
// or in one for at most 8 rows and at most 24 KiB of X (no cross-block
// state; *clear_words is then 0). Cross-block state (the mask accumulator,
// or the row maxima for other inputs of at most 8 rows) goes to `acc`,
// which must be zero on entry;
// *clear_words is how many of its words the product launch must clear
// again (see launch_int8_gemm). For s > 8, Xq may be null: the codes are
// then not written (launch_int8_gemm_inline_quant makes them).
hipError_t launch_forward_prologue(const uint16_t* X, int64_t s, int64_t h, float alpha, uint32_t* acc,
                                   uint32_t* mask, int32_t* idx, int32_t* n_out, int8_t* Xq, float* c_x,
                                   uint16_t* X_O, int64_t ldo, hipStream_t stream, int* clear_words);

// The same for the tensor-wise (zeropoint = false; c_x receives the one
// constant in every entry) or zeropoint (c_x receives nd_x; zp_x and
// rowsum_x are written) row quantiser: detection into acc[0 .. h / 32),
// then the scheme's row quantiser, whose first block writes the mask, the
// index list and |O|.
hipError_t launch_forward_prologue_variant(bool zeropoint, const uint16_t* X, int64_t s, int64_t h, float alpha,
                                           uint32_t* acc, uint32_t* mask, int32_t* idx, int32_t* n_out, int8_t* Xq,
                                           float* c_x, int32_t* zp_x, int32_t* rowsum_x, uint16_t* X_O, int64_t ldo,
                                           hipStream_t stream, int* clear_words);

hipError_t launch_quantize_cols(const uint16_t* W, int64_t h, int64_t o,
                                int8_t* Wq, float* c_w, hipStream_t stream);

// Tensor-wise absmax: one constant for all of X's non-outlier part (written
// to every c_x[i]) or for all of W (every c_w[j]); same outputs otherwise.
// If idx is non-null, the first pass also writes the index list and |O|
// (and the mask to mask_out if that is non-null) from `mask`.
hipError_t launch_quantize_tensorwise(const uint16_t* X, int64_t s, int64_t h, const uint32_t* mask, int8_t* Xq,
                                      float* c_x, uint16_t* X_O, int64_t ldo, hipStream_t stream,
                                      uint32_t* mask_out = nullptr, int32_t* idx = nullptr,
                                      int32_t* n_out = nullptr);
hipError_t launch_quantize_weights_tensorwise(const uint16_t* W, int64_t h, int64_t o, int8_t* Wq, float* c_w,
                                              hipStream_t stream);

// Zeropoint quantisation: rows of X over the non-outlier columns (codes,
// nd_x, zp_x, code sums over the row, X_O gather) and columns of W at load
// time (panel codes, nd_w, zp_w, code sums over the column).
// (idx, n_out, mask_out: as for launch_quantize_tensorwise.)
hipError_t launch_quantize_rows_zp(const uint16_t* X, int64_t s, int64_t h, const uint32_t* mask, int8_t* Xq,
                                   float* nd_x, int32_t* zp_x, int32_t* rowsum_x, uint16_t* X_O, int64_t ldo,
                                   hipStream_t stream, uint32_t* mask_out = nullptr, int32_t* idx = nullptr,
                                   int32_t* n_out = nullptr);
hipError_t launch_quantize_cols_zp(const uint16_t* W, int64_t h, int64_t o, int8_t* Wq, float* nd_w, int32_t* zp_w,
                                   int32_t* colsum_w, hipStream_t stream);

// mode: product variant of the shared int8 main loop. W (Mixed only) may be
// null: outlier rows rebuilt from Wq / c_w. bias (Mixed only, optional):
// fp16 [o] added before the rounding. `clear` (optional): clear_words
// uint32 words that the first block zeroes (the forward path's
// accumulator, whose readers have finished by then).
// ZeroPoint: the product of zeropoint codes, C' = sum over k not in O of
// (Xq_ik + zp_x_i)(Wq_kj + zp_w_j), dequantised with 1 / (nd_x nd_w) (passed
// as c_x, c_w) plus the fp16 outlier product; ZpArgs carries the zero points
// and code sums (rowsum over the row's codes, colsum over all h codes of the
// column).
enum class GemmOut { Mixed = 0, Int32 = 1, Fp16Dense = 2, ZeroPoint = 3 };

struct ZpArgs {
    const int32_t* zp_x;
    const int32_t* rowsum_x;
    const int32_t* zp_w;
    const int32_t* colsum_w;
};

hipError_t launch_int8_gemm(GemmOut mode, const int8_t* Xq, const float* c_x,
                            const uint16_t* X_O, int64_t ldo,
                            const int32_t* idx, const int32_t* n_out,
                            const int8_t* Wq, const float* c_w, const uint16_t* W, const uint16_t* bias,
                            int64_t s, int64_t h, int64_t o, void* C, hipStream_t stream,
                            uint32_t* clear = nullptr, int clear_words = 0, ZpArgs zp = ZpArgs{});

// Dense fp16 product C = fp16(X W) with fp32 accumulation; Wp is W in the
// fp16 panel layout [h / 32][o][32] (see launch_pack_fp16_panels).
hipError_t launch_fp16_gemm(const uint16_t* X, const uint16_t* Wp, int64_t s, int64_t h, int64_t o, uint16_t* C,
                            hipStream_t stream);

// The LLM.int8() product with the int8 operand of X made inside the
// product kernel from the fp16 rows X, the final outlier mask and c_x
// (k_gemm_prefill<Mixed, QX>): no Xq. Any s (the tiled product); the other
// arguments as launch_int8_gemm's.
hipError_t launch_int8_gemm_inline_quant(const uint16_t* X, const uint32_t* mask, const float* c_x,
                                         const uint16_t* X_O, int64_t ldo, const int32_t* idx, const int32_t* n_out,
                                         const int8_t* Wq, const float* c_w, const uint16_t* W, const uint16_t* bias,
                                         int64_t s, int64_t h, int64_t o, uint16_t* C, hipStream_t stream,
                                         uint32_t* clear, int clear_words);

hipError_t launch_pack_fp16_panels(const uint16_t* W, int64_t h, int64_t o, uint16_t* Wp, hipStream_t stream);

// The whole forward in one launch for s <= 16 (k_decode_fused); the
// intermediates go to mask .. X_O (block 0 writes them).
hipError_t launch_decode_fused(const uint16_t* X, int64_t s, int64_t h, int64_t o, float alpha, const int8_t* Wq,
                               const float* c_w, const uint16_t* W, const uint16_t* bias, uint16_t* C, uint32_t* mask,
                               int32_t* idx, int32_t* n_out, int8_t* Xq, float* c_x, uint16_t* X_O, int64_t ldo,
                               hipStream_t stream);

hipError_t launch_outlier_matmul(const uint16_t* X_O, int64_t ldo,
                                 const int32_t* idx, const int32_t* n_out,
                                 const uint16_t* W, int64_t s, int64_t o,
                                 float* C_O, hipStream_t stream);

// Calibration stream of int8 MFMAs (k_calib_mfma_i8): `blocks` blocks of
// four wavefronts, 32 iters MFMAs per wavefront; codes holds 256 bytes per
// thread, out one int32 per thread.
hipError_t launch_calib_mfma_i8(const int8_t* codes, int64_t blocks, int64_t iters, int32_t* out,
                                hipStream_t stream);

// Element types of the kernels around an adapted layer (the values of
// i8mm_dtype).
enum class Dtype { F16 = 0, BF16 = 1, F32 = 2 };

// Layer norm of the rows of X and its gradients. Row strides in elements; wt
// is xt or F32; b, mean and rstd may be null, as may dw and db. `part` holds
// layer_norm_backward_parts(s) sums of 2 h floats (unused if dw and db are
// null).
hipError_t launch_layer_norm(const void* X, int64_t ldx, Dtype xt, int64_t s, int64_t h, const void* w, const void* b,
                             Dtype wt, float eps, void* Y, int64_t ldy, float* mean, float* rstd, hipStream_t stream);
int64_t layer_norm_backward_parts(int64_t s);
hipError_t launch_layer_norm_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, Dtype xt, int64_t s,
                                      int64_t h, const void* w, Dtype wt, const float* mean, const float* rstd,
                                      void* dX, int64_t lddx, float* dw, float* db, float* part, hipStream_t stream);

// What the adapter kernels share: the adapters A [G, r, h] and B [G, r, o]
// of `type` (F16 or BF16), the adapter of each of the s tokens, and a factor
// per adapter.
struct LoraArgs {
    const void* A;
    const void* B;
    Dtype type;
    int64_t G;
    int r;
    const int32_t* ids;
    const float* scale;
    int64_t s, h, o;
};

// Y = base + scale (X A^T) B with T = X A^T in fp32; base and T may be null.
size_t lora_forward_scratch(int64_t s, int64_t h, int64_t o, int64_t r);
hipError_t launch_lora_forward(const LoraArgs& a, const void* X, int64_t ldx, const void* base, int64_t ldb, void* Y,
                               int64_t ldy, float* T, void* workspace, hipStream_t stream);

// The gradients of Y for dY, given T; base and dX may be null.
size_t lora_backward_scratch(int64_t s, int64_t h, int64_t o, int64_t r, int64_t G);
hipError_t launch_lora_backward(const LoraArgs& a, const void* dY, int64_t lddy, const void* X, int64_t ldx,
                                const float* T, const void* base, int64_t ldb, void* dX, int64_t lddx, float* dA,
                                float* dB, void* workspace, hipStream_t stream);

// The norm over all n tensors to *total, and out = min(1, max_norm / norm)
// in (in place if out is null). `workspace`: clip_parts(n) doubles. The host
// arrays are read before the call returns.
int64_t clip_parts(int64_t n);
hipError_t launch_clip_grad_norm(const void* const* in, void* const* out, const int64_t* numel, const int32_t* types,
                                 int64_t n, float max_norm, void* workspace, float* total, hipStream_t stream);

// Decoding between int8 layers. A paged cache holds keys and values as
// [n_pages][kv_heads][page][d], with a stride between pages; a sequence's row of
// `tables` names its pages in order.

// Rows of K and V [s, kv_heads d] into the pages of the sequences seq[i] (or i)
// at the positions pos[i].
struct AppendArgs {
    const void *K, *V;
    int64_t ldk, ldv;
    int element_bytes;
    int64_t s;
    int kv_heads, d;
    const int32_t *seq, *pos;       // seq may be null
    const int32_t* tables;
    int64_t ldt;
    int64_t n;
    int max_pages;
    void *K_pages, *V_pages;
    int64_t k_stride, v_stride;
    int n_pages, page;
};
hipError_t launch_cache_append(const AppendArgs& a, hipStream_t stream);

// Page pools: n device pointers, a page's bytes and the bytes between pages
// (host arrays, read before the call returns).
struct Pools {
    void* const* at;
    const int64_t* bytes;
    const int64_t* strides;
    int64_t n;
};

struct ForkArgs {
    const int32_t* tables;
    int64_t ldt;
    const int32_t *lens, *refs;
    int64_t n;
    int max_pages, n_pages, page;
    const int32_t *parents, *grow;  // each may be null
    int64_t n_out;
    int32_t* tables_out;
    int64_t ldto;
    int32_t *lens_out, *refs_out, *state;
};
size_t cache_fork_scratch(int64_t n, int64_t n_out, int64_t n_pages);
hipError_t launch_cache_fork(const ForkArgs& a, const Pools& pools, void* workspace, hipStream_t stream);

struct CompactArgs {
    const int32_t* tables;
    int64_t ldt;
    int64_t n;
    int max_pages;
    const int32_t* refs;
    int n_pages;
    int32_t* tables_out;
    int64_t ldto;
    int32_t *refs_out, *moved, *state;
};
size_t cache_compact_scratch(int64_t n_pages);
hipError_t launch_cache_compact(const CompactArgs& a, const Pools& pools, void* workspace, hipStream_t stream);

// Attention of one query a sequence over its pages; slopes and lse may be null.
struct AttendArgs {
    const void* Q;
    int64_t ldq;
    Dtype type;
    int64_t n;
    int heads, kv_heads, d;
    const void *K, *V;
    int64_t k_stride, v_stride;
    int n_pages, page;
    const int32_t* tables;
    int64_t ldt;
    int max_pages;
    const int32_t* lens;
    int beams;
    float scale;
    const float* slopes;
    void* out;
    int64_t ldo;
    float* lse;
};
// Whether a block takes all keys of a sequence's head: one launch, no workspace.
bool attention_takes_whole(int64_t keys, int64_t beams);
size_t decode_attention_scratch(int64_t n, int heads, int kv_heads, int d);
hipError_t launch_decode_attention(const AttendArgs& a, void* workspace, hipStream_t stream);

// The k best of scores[b, i] + log_softmax(logits[b beams + i]) for each b;
// history and history_out may be null.
struct SelectArgs {
    const void* logits;
    int64_t ld;
    Dtype type;
    int64_t n;
    int beams;
    int vocab;
    const float* scores;
    int k;
    float* scores_out;
    int32_t *parents, *tokens;
    const int32_t* history;
    int64_t ldh;
    int64_t T;
    int32_t* history_out;
    int64_t ldho;
};
size_t beam_select_scratch(int64_t n, int beams, int vocab, int k);
hipError_t launch_beam_select(const SelectArgs& a, void* workspace, hipStream_t stream);

}  // namespace i8mm
