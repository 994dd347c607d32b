// Layer norm over the rows of X [s, h] and its gradients.
//
//   mean_i = sum_j x_ij / h,  var_i = sum_j (x_ij - mean_i)^2 / h,
//   rstd_i = 1 / sqrt(var_i + eps),  n_ij = (x_ij - mean_i) rstd_i,
//   y_ij = n_ij w_j + b_j.
// With g_ij = dy_ij w_j the gradients are
//   dx_ij = rstd_i (g_ij - mean_j(g_ij) - n_ij mean_j(g_ij n_ij)),
//   dw_j = sum_i dy_ij n_ij,  db_j = sum_i dy_ij.
// Sums and statistics are fp32 whatever the element type; y and dx are
// rounded once.

#include "launch.h"

#include "adapt_common.h"

namespace i8mm {
namespace {

constexpr int kNormThreads = 256;

template <typename T, typename W>
__global__ __launch_bounds__(kNormThreads) void k_layer_norm(const T* __restrict__ X, int64_t ldx, int h,
                                                             const W* __restrict__ w, const W* __restrict__ b,
                                                             float eps, T* __restrict__ Y, int64_t ldy,
                                                             float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float red[kNormThreads / 64];
    const int64_t row = blockIdx.x;
    const T* x = X + row * ldx;
    T* y = Y + row * ldy;
    float sum = 0.0f;
    for (int j = threadIdx.x; j < h; j += kNormThreads) sum += to_float(x[j]);
    const float m = block_sum<kNormThreads / 64>(sum, red) / static_cast<float>(h);
    float sq = 0.0f;
    for (int j = threadIdx.x; j < h; j += kNormThreads) {
        const float d = to_float(x[j]) - m;
        sq = fmaf(d, d, sq);
    }
    const float var = block_sum<kNormThreads / 64>(sq, red) / static_cast<float>(h);
    const float r = 1.0f / sqrtf(var + eps);
    for (int j = threadIdx.x; j < h; j += kNormThreads) {
        const float n = (to_float(x[j]) - m) * r;
        y[j] = from_float<T>(fmaf(n, to_float(w[j]), b ? to_float(b[j]) : 0.0f));
    }
    if (threadIdx.x == 0) {
        if (mean) mean[row] = m;
        if (rstd) rstd[row] = r;
    }
}

template <typename T, typename W>
__global__ __launch_bounds__(kNormThreads) void k_layer_norm_dx(const T* __restrict__ dY, int64_t lddy,
                                                                const T* __restrict__ X, int64_t ldx, int h,
                                                                const W* __restrict__ w,
                                                                const float* __restrict__ mean,
                                                                const float* __restrict__ rstd, T* __restrict__ dX,
                                                                int64_t lddx) {
    __shared__ float red[kNormThreads / 64];
    const int64_t row = blockIdx.x;
    const T* x = X + row * ldx;
    const T* dy = dY + row * lddy;
    T* dx = dX + row * lddx;
    const float m = mean[row], r = rstd[row];
    float sg = 0.0f, sgn = 0.0f;
    for (int j = threadIdx.x; j < h; j += kNormThreads) {
        const float g = to_float(dy[j]) * to_float(w[j]);
        sg += g;
        sgn = fmaf(g, (to_float(x[j]) - m) * r, sgn);
    }
    const float mg = block_sum<kNormThreads / 64>(sg, red) / static_cast<float>(h);
    const float mgn = block_sum<kNormThreads / 64>(sgn, red) / static_cast<float>(h);
    for (int j = threadIdx.x; j < h; j += kNormThreads) {
        const float g = to_float(dy[j]) * to_float(w[j]);
        const float n = (to_float(x[j]) - m) * r;
        dx[j] = from_float<T>(r * (g - mg - n * mgn));
    }
}

// Sums of dy n and dy over one block of rows for each column: part holds
// [blocks of rows][2][h].
template <typename T>
__global__ __launch_bounds__(kNormThreads) void k_layer_norm_dw_part(const T* __restrict__ dY, int64_t lddy,
                                                                     const T* __restrict__ X, int64_t ldx, int64_t s,
                                                                     int h, int64_t rows,
                                                                     const float* __restrict__ mean,
                                                                     const float* __restrict__ rstd,
                                                                     float* __restrict__ part) {
    const int j = blockIdx.x * kNormThreads + threadIdx.x;
    if (j >= h) return;
    const int64_t i0 = blockIdx.y * rows;
    const int64_t i1 = i0 + rows < s ? i0 + rows : s;
    float dw = 0.0f, db = 0.0f;
    for (int64_t i = i0; i < i1; ++i) {
        const float dy = to_float(dY[i * lddy + j]);
        db += dy;
        dw = fmaf(dy, (to_float(X[i * ldx + j]) - mean[i]) * rstd[i], dw);
    }
    float* p = part + static_cast<int64_t>(blockIdx.y) * 2 * h;
    p[j] = dw;
    p[h + j] = db;
}

__global__ __launch_bounds__(kNormThreads) void k_layer_norm_dw_sum(const float* __restrict__ part, int parts, int h,
                                                                    float* __restrict__ dw, float* __restrict__ db) {
    const int j = blockIdx.x * kNormThreads + threadIdx.x;
    if (j >= h) return;
    float a = 0.0f, b = 0.0f;
    for (int p = 0; p < parts; ++p) {
        a += part[static_cast<int64_t>(p) * 2 * h + j];
        b += part[static_cast<int64_t>(p) * 2 * h + h + j];
    }
    if (dw) dw[j] = a;
    if (db) db[j] = b;
}

// Calls f with a null pointer of each of the two element types.
template <typename F>
hipError_t with_types(Dtype x, Dtype w, F&& f) {
    if (x == Dtype::F16) return w == Dtype::F32 ? f((_Float16*)0, (float*)0) : f((_Float16*)0, (_Float16*)0);
    if (x == Dtype::BF16) return w == Dtype::F32 ? f((__bf16*)0, (float*)0) : f((__bf16*)0, (__bf16*)0);
    return f((float*)0, (float*)0);
}

}  // namespace

hipError_t launch_layer_norm(const void* X, int64_t ldx, Dtype xt, int64_t s, int64_t h, const void* w, const void* b,
                             Dtype wt, float eps, void* Y, int64_t ldy, float* mean, float* rstd,
                             hipStream_t stream) {
    if (s == 0) return hipSuccess;
    return with_types(xt, wt, [&](auto* tx, auto* tw) {
        using T = std::remove_pointer_t<decltype(tx)>;
        using W = std::remove_pointer_t<decltype(tw)>;
        k_layer_norm<T, W><<<static_cast<unsigned>(s), kNormThreads, 0, stream>>>(
            static_cast<const T*>(X), ldx, static_cast<int>(h), static_cast<const W*>(w), static_cast<const W*>(b),
            eps, static_cast<T*>(Y), ldy, mean, rstd);
        return hipGetLastError();
    });
}

int64_t layer_norm_backward_parts(int64_t s) { return s < 64 ? s : 64; }

hipError_t launch_layer_norm_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, Dtype xt, int64_t s,
                                      int64_t h, const void* w, Dtype wt, const float* mean, const float* rstd,
                                      void* dX, int64_t lddx, float* dw, float* db, float* part, hipStream_t stream) {
    const unsigned cols = static_cast<unsigned>((h + kNormThreads - 1) / kNormThreads);
    const int64_t parts = layer_norm_backward_parts(s);
    if (s > 0) {
        const int64_t rows = (s + parts - 1) / parts;
        const hipError_t e = with_types(xt, wt, [&](auto* tx, auto* tw) {
            using T = std::remove_pointer_t<decltype(tx)>;
            using W = std::remove_pointer_t<decltype(tw)>;
            k_layer_norm_dx<T, W><<<static_cast<unsigned>(s), kNormThreads, 0, stream>>>(
                static_cast<const T*>(dY), lddy, static_cast<const T*>(X), ldx, static_cast<int>(h),
                static_cast<const W*>(w), mean, rstd, static_cast<T*>(dX), lddx);
            if (dw || db)
                k_layer_norm_dw_part<T><<<dim3(cols, static_cast<unsigned>(parts)), kNormThreads, 0, stream>>>(
                    static_cast<const T*>(dY), lddy, static_cast<const T*>(X), ldx, s, static_cast<int>(h), rows, mean,
                    rstd, part);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    if (dw || db) {
        k_layer_norm_dw_sum<<<cols, kNormThreads, 0, stream>>>(part, static_cast<int>(parts), static_cast<int>(h), dw,
                                                               db);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace i8mm
