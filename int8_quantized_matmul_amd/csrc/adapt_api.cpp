// C-ABI layer of the entry points around an adapted layer (layer norm,
// low-rank adapters, gradient clipping): host-side validation, the device
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
using i8mm::round_up;

constexpr int64_t kMaxElements = int64_t(1) << 44;   // of all gradients of a call: chunk counts stay 32-bit

bool valid_type(int t) { return t == I8MM_F16 || t == I8MM_BF16 || t == I8MM_F32; }

uintptr_t element_bytes(int t) { return t == I8MM_F32 ? 4 : 2; }

bool valid_norm_shape(int64_t s, int64_t h) {
    return s >= 0 && s <= (int64_t(1) << 31) - 1 && h >= 1 && h <= I8MM_NORM_MAX_H;
}

bool valid_norm_types(int32_t x, int32_t w) {
    return valid_type(x) && valid_type(w) && (w == x || w == I8MM_F32);
}

bool valid_stride(int64_t ld, int64_t len) { return ld >= len && ld <= (int64_t(1) << 31); }

bool valid_lora_shape(int64_t s, int64_t h, int64_t o, int64_t r, int64_t G) {
    const auto len = [](int64_t v) { return v >= 64 && v % 64 == 0 && v <= I8MM_MAX_H; };
    return s >= 0 && s <= I8MM_LORA_MAX_ROWS && len(h) && len(o) && r >= 1 && r <= I8MM_LORA_MAX_RANK && G >= 1 &&
           G <= I8MM_LORA_MAX_ADAPTERS;
}

// A 16-byte aligned matrix whose rows are too.
bool valid_rows16(const void* p, int64_t ld, int64_t len) {
    return aligned16(p) && ld % 8 == 0 && valid_stride(ld, len);
}

bool aligned256(const void* p) { return aligned_to(p, 256); }

}  // namespace

extern "C" {

i8mm_status i8mm_layer_norm(const void* X, int64_t ldx, int32_t x_type, int64_t s, int64_t h, const void* weight,
                            const void* bias, int32_t w_type, float eps, void* Y, int64_t ldy, float* mean,
                            float* rstd, hipStream_t stream) {
    if (!weight || (s != 0 && (!X || !Y))) return I8MM_EINVAL;   // bias, mean and rstd may be null
    if (!valid_norm_shape(s, h) || !valid_norm_types(x_type, w_type)) return I8MM_EINVAL;
    if (!valid_stride(ldx, h) || !valid_stride(ldy, h)) return I8MM_EINVAL;
    if (!std::isfinite(eps) || eps < 0.0f) return I8MM_EINVAL;
    if (!aligned_to(X, element_bytes(x_type)) || !aligned_to(Y, element_bytes(x_type)) ||
        !aligned_to(weight, element_bytes(w_type)) || !aligned_to(bias, element_bytes(w_type)) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return I8MM_EINVAL;
    if (s > 1 && X == Y && ldx != ldy) return I8MM_EINVAL;
    if (i8mm_status d = check_device()) return d;
    return launched(i8mm::launch_layer_norm(X, ldx, static_cast<Dtype>(x_type), s, h, weight, bias,
                                            static_cast<Dtype>(w_type), eps, Y, ldy, mean, rstd, stream));
}

size_t i8mm_layer_norm_backward_workspace_bytes(int64_t s, int64_t h) {
    if (!valid_norm_shape(s, h)) return 0;
    const int64_t parts = i8mm::layer_norm_backward_parts(s);
    return static_cast<size_t>(round_up((parts > 0 ? parts : 1) * 2 * h * 4, 256));
}

i8mm_status i8mm_layer_norm_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, int32_t x_type,
                                     int64_t s, int64_t h, const void* weight, int32_t w_type, const float* mean,
                                     const float* rstd, void* dX, int64_t lddx, float* d_weight, float* d_bias,
                                     void* workspace, hipStream_t stream) {
    if (!weight || (s != 0 && (!dY || !X || !mean || !rstd || !dX))) return I8MM_EINVAL;
    if (!workspace && (d_weight || d_bias)) return I8MM_EINVAL;
    if (!valid_norm_shape(s, h) || !valid_norm_types(x_type, w_type)) return I8MM_EINVAL;
    if (!valid_stride(lddy, h) || !valid_stride(ldx, h) || !valid_stride(lddx, h)) return I8MM_EINVAL;
    const uintptr_t e = element_bytes(x_type);
    if (!aligned_to(dY, e) || !aligned_to(X, e) || !aligned_to(dX, e) ||
        !aligned_to(weight, element_bytes(w_type)) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
        !aligned_to(d_weight, 4) || !aligned_to(d_bias, 4) || !aligned256(workspace))
        return I8MM_EINVAL;
    if (s > 0 && (dX == X || dX == dY)) return I8MM_EINVAL;
    if (i8mm_status d = check_device()) return d;
    return launched(i8mm::launch_layer_norm_backward(dY, lddy, X, ldx, static_cast<Dtype>(x_type), s, h, weight,
                                                     static_cast<Dtype>(w_type), mean, rstd, dX, lddx, d_weight,
                                                     d_bias, static_cast<float*>(workspace), stream));
}

size_t i8mm_lora_forward_workspace_bytes(int64_t s, int64_t h, int64_t o, int64_t r) {
    if (!valid_lora_shape(s, h, o, r, 1)) return 0;
    return 256 + static_cast<size_t>(round_up(static_cast<int64_t>(i8mm::lora_forward_scratch(s, h, o, r)), 256));
}

i8mm_status i8mm_lora_forward(const void* X, int64_t ldx, const void* A, const void* B, int32_t type,
                              int64_t n_adapters, int64_t r, const int32_t* ids, const float* scale, const void* base,
                              int64_t ldb, int64_t s, int64_t h, int64_t o, void* Y, int64_t ldy, float* T,
                              void* workspace, hipStream_t stream) {
    // base and T may be null
    if (!A || !B || !scale || !workspace || (s != 0 && (!X || !ids || !Y))) return I8MM_EINVAL;
    if (type != I8MM_F16 && type != I8MM_BF16) return I8MM_EINVAL;
    if (!valid_lora_shape(s, h, o, r, n_adapters)) return I8MM_EINVAL;
    if (!valid_rows16(X, ldx, h) || !valid_rows16(Y, ldy, o) || (base && !valid_rows16(base, ldb, o)) ||
        !aligned16(A) || !aligned16(B) || !aligned_to(ids, 4) || !aligned_to(scale, 4) || !aligned_to(T, 4) ||
        !aligned256(workspace))
        return I8MM_EINVAL;
    if (s > 0 && (Y == X || (s > 1 && Y == base && ldy != ldb))) return I8MM_EINVAL;
    if (i8mm_status d = check_device()) return d;
    const i8mm::LoraArgs a{A, B, static_cast<Dtype>(type), n_adapters, static_cast<int>(r), ids, scale, s, h, o};
    return launched(i8mm::launch_lora_forward(a, X, ldx, base, ldb, Y, ldy, T, workspace, stream));
}

size_t i8mm_lora_backward_workspace_bytes(int64_t s, int64_t h, int64_t o, int64_t r, int64_t n_adapters) {
    if (!valid_lora_shape(s, h, o, r, n_adapters)) return 0;
    return 256 + static_cast<size_t>(
                     round_up(static_cast<int64_t>(i8mm::lora_backward_scratch(s, h, o, r, n_adapters)), 256));
}

i8mm_status i8mm_lora_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, const float* T,
                               const void* A, const void* B, int32_t type, int64_t n_adapters, int64_t r,
                               const int32_t* ids, const float* scale, const void* base, int64_t ldb, int64_t s,
                               int64_t h, int64_t o, void* dX, int64_t lddx, float* dA, float* dB, void* workspace,
                               hipStream_t stream) {
    // base and dX may be null
    if (!A || !B || !scale || !dA || !dB || !workspace || (s != 0 && (!dY || !X || !T || !ids))) return I8MM_EINVAL;
    if (type != I8MM_F16 && type != I8MM_BF16) return I8MM_EINVAL;
    if (!valid_lora_shape(s, h, o, r, n_adapters)) return I8MM_EINVAL;
    if (!valid_rows16(dY, lddy, o) || !valid_rows16(X, ldx, h) || (dX && !valid_rows16(dX, lddx, h)) ||
        (base && !valid_rows16(base, ldb, h)) || !aligned16(A) || !aligned16(B) || !aligned16(dA) ||
        !aligned16(dB) || !aligned_to(ids, 4) || !aligned_to(scale, 4) || !aligned_to(T, 4) ||
        !aligned256(workspace))
        return I8MM_EINVAL;
    if (s > 0 && dX && (dX == X || dX == dY || (s > 1 && dX == base && lddx != ldb))) return I8MM_EINVAL;
    if (i8mm_status d = check_device()) return d;
    const i8mm::LoraArgs a{A, B, static_cast<Dtype>(type), n_adapters, static_cast<int>(r), ids, scale, s, h, o};
    return launched(
        i8mm::launch_lora_backward(a, dY, lddy, X, ldx, T, base, ldb, dX, lddx, dA, dB, workspace, stream));
}

size_t i8mm_clip_grad_norm_workspace_bytes(const int64_t* numels, int64_t n) {
    if (n < 0 || n > (int64_t(1) << 24) || (n > 0 && !numels)) return 0;
    int64_t total = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (numels[i] < 0 || numels[i] > kMaxElements || (total += numels[i]) > kMaxElements) return 0;
    }
    return static_cast<size_t>(256 + round_up(8 * i8mm::clip_parts(n), 256));
}

i8mm_status i8mm_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* numels,
                                const int32_t* types, int64_t n, float max_norm, void* workspace, float* total_norm,
                                hipStream_t stream) {
    if (!workspace || !total_norm || !aligned256(workspace) || !aligned_to(total_norm, 4)) return I8MM_EINVAL;
    if (n > 0 && (!grads || !types)) return I8MM_EINVAL;   // outs may be null
    if (i8mm_clip_grad_norm_workspace_bytes(numels, n) == 0) return I8MM_EINVAL;
    if (std::isnan(max_norm) || max_norm < 0.0f) return I8MM_EINVAL;
    for (int64_t i = 0; i < n; ++i) {
        if (!valid_type(types[i])) return I8MM_EINVAL;
        if (numels[i] == 0) continue;
        if (!grads[i] || !aligned_to(grads[i], element_bytes(types[i]))) return I8MM_EINVAL;
        if (outs && (!outs[i] || !aligned_to(outs[i], element_bytes(types[i])))) return I8MM_EINVAL;
    }
    if (i8mm_status d = check_device()) return d;
    return launched(i8mm::launch_clip_grad_norm(grads, outs, numels, types, n, max_norm, workspace, total_norm,
                                                stream));
}

}  // extern "C"
