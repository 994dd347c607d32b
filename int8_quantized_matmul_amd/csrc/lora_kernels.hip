// Low-rank adapters of many requests beside one shared projection.
//
// Token i carries the adapter ids[i] = g of its request, or none (any value
// outside [0, G)). With A [G, r, h], B [G, r, o] and a factor per adapter:
//   T_i = X_i A_g^T,  Y_i = base_i + scale_g T_i B_g,
// and for gradients dY of Y:
//   dT_i = scale_g dY_i B_g^T,  dX_i = base_i + dT_i A_g,
//   dA_g = sum over the tokens of g of dT_i^T X_i,
//   dB_g = scale_g times the sum over the tokens of g of T_i^T dY_i.
// T and dT are held in fp32; products are summed in fp32; Y and dX are
// rounded once.

#include "launch.h"

#include "adapt_common.h"

namespace i8mm {
namespace {

constexpr int kLoraThreads = 256;

// One wavefront per (token, rank): P[i, k] = Z_i . M_g[k], times the
// adapter's factor if `scale` is given.
template <typename T>
__global__ __launch_bounds__(kLoraThreads) void k_lora_dot(const T* __restrict__ Z, int64_t ldz,
                                                           const T* __restrict__ M, int64_t G, int r, int64_t len,
                                                           const int32_t* __restrict__ ids,
                                                           const float* __restrict__ scale, int64_t s,
                                                           float* __restrict__ P) {
    const int64_t task = static_cast<int64_t>(blockIdx.x) * (kLoraThreads / 64) + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (task >= s * r) return;
    const int64_t i = task / r;
    const int k = static_cast<int>(task % r);
    const int64_t g = ids[i];
    float sum = 0.0f;
    if (g >= 0 && g < G) {
        const T* z = Z + i * ldz;
        const T* m = M + (g * r + k) * len;
        for (int64_t j = lane; j < len; j += 64) sum = fmaf(to_float(z[j]), to_float(m[j]), sum);
        sum = wave_sum(sum);
        if (scale) sum *= scale[g];
    }
    if (lane == 0) P[task] = sum;
}

// out_i = base_i + factor P_i M_g; base may be null, scale may be null.
template <typename T>
__global__ __launch_bounds__(kLoraThreads) void k_lora_add(const float* __restrict__ P, const T* __restrict__ M,
                                                           int64_t G, int r, int64_t len,
                                                           const int32_t* __restrict__ ids,
                                                           const float* __restrict__ scale, const T* base,
                                                           int64_t ldb, T* out, int64_t ldo) {
    const int64_t i = blockIdx.x;
    const int64_t g = ids[i];
    for (int64_t j = blockIdx.y * kLoraThreads + threadIdx.x; j < len; j += gridDim.y * kLoraThreads) {
        float v = 0.0f;
        if (g >= 0 && g < G) {
            for (int k = 0; k < r; ++k) v = fmaf(P[i * r + k], to_float(M[(g * r + k) * len + j]), v);
            if (scale) v *= scale[g];
        }
        out[i * ldo + j] = from_float<T>(base ? to_float(base[i * ldb + j]) + v : v);
    }
}

// out_g[k, j] = factor times the sum over the tokens of g of P[i, k] Z[i, j]
template <typename T>
__global__ __launch_bounds__(kLoraThreads) void k_lora_grad(const float* __restrict__ P, const T* __restrict__ Z,
                                                            int64_t ldz, int r, int64_t len, int64_t s,
                                                            const int32_t* __restrict__ ids,
                                                            const float* __restrict__ scale,
                                                            float* __restrict__ out) {
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kLoraThreads + threadIdx.x;
    const int k = blockIdx.y;
    const int64_t g = blockIdx.z;
    if (j >= len) return;
    float v = 0.0f;
    for (int64_t i = 0; i < s; ++i)
        if (ids[i] == g) v = fmaf(P[i * r + k], to_float(Z[i * ldz + j]), v);
    out[(g * r + k) * len + j] = scale ? v * scale[g] : v;
}

template <typename T>
hipError_t forward(const LoraArgs& a, const void* Xv, int64_t ldx, const void* basev, int64_t ldb, void* Yv,
                   int64_t ldy, float* P, hipStream_t stream) {
    const unsigned dots = static_cast<unsigned>((a.s * a.r + 3) / 4);
    k_lora_dot<T><<<dots, kLoraThreads, 0, stream>>>(static_cast<const T*>(Xv), ldx, static_cast<const T*>(a.A),
                                                     a.G, a.r, a.h, a.ids, nullptr, a.s, P);
    k_lora_add<T><<<dim3(static_cast<unsigned>(a.s), 8), kLoraThreads, 0, stream>>>(
        P, static_cast<const T*>(a.B), a.G, a.r, a.o, a.ids, a.scale, static_cast<const T*>(basev), ldb,
        static_cast<T*>(Yv), ldy);
    return hipGetLastError();
}

template <typename T>
hipError_t backward(const LoraArgs& a, const void* dYv, int64_t lddy, const void* Xv, int64_t ldx, const float* Tp,
                    const void* basev, int64_t ldb, void* dXv, int64_t lddx, float* dA, float* dB, float* P,
                    hipStream_t stream) {
    if (a.s > 0) {
        const unsigned dots = static_cast<unsigned>((a.s * a.r + 3) / 4);
        k_lora_dot<T><<<dots, kLoraThreads, 0, stream>>>(static_cast<const T*>(dYv), lddy,
                                                         static_cast<const T*>(a.B), a.G, a.r, a.o, a.ids, a.scale,
                                                         a.s, P);
        if (dXv)
            k_lora_add<T><<<dim3(static_cast<unsigned>(a.s), 8), kLoraThreads, 0, stream>>>(
                P, static_cast<const T*>(a.A), a.G, a.r, a.h, a.ids, nullptr, static_cast<const T*>(basev), ldb,
                static_cast<T*>(dXv), lddx);
    }
    const auto grid = [&](int64_t len) {
        return dim3(static_cast<unsigned>((len + kLoraThreads - 1) / kLoraThreads), static_cast<unsigned>(a.r),
                    static_cast<unsigned>(a.G));
    };
    k_lora_grad<T><<<grid(a.h), kLoraThreads, 0, stream>>>(P, static_cast<const T*>(Xv), ldx, a.r, a.h, a.s, a.ids,
                                                           nullptr, dA);
    k_lora_grad<T><<<grid(a.o), kLoraThreads, 0, stream>>>(Tp, static_cast<const T*>(dYv), lddy, a.r, a.o, a.s, a.ids,
                                                           a.scale, dB);
    return hipGetLastError();
}

}  // namespace

size_t lora_forward_scratch(int64_t s, int64_t, int64_t, int64_t r) { return 4 * static_cast<size_t>(s) * r; }

size_t lora_backward_scratch(int64_t s, int64_t, int64_t, int64_t r, int64_t) {
    return 4 * static_cast<size_t>(s) * r;
}

hipError_t launch_lora_forward(const LoraArgs& a, const void* X, int64_t ldx, const void* base, int64_t ldb, void* Y,
                               int64_t ldy, float* T, void* workspace, hipStream_t stream) {
    if (a.s == 0) return hipSuccess;
    float* P = T ? T : static_cast<float*>(workspace);
    return a.type == Dtype::F16 ? forward<_Float16>(a, X, ldx, base, ldb, Y, ldy, P, stream)
                                : forward<__bf16>(a, X, ldx, base, ldb, Y, ldy, P, stream);
}

hipError_t launch_lora_backward(const LoraArgs& a, const void* dY, int64_t lddy, const void* X, int64_t ldx,
                                const float* T, const void* base, int64_t ldb, void* dX, int64_t lddx, float* dA,
                                float* dB, void* workspace, hipStream_t stream) {
    float* P = static_cast<float*>(workspace);
    return a.type == Dtype::F16
               ? backward<_Float16>(a, dY, lddy, X, ldx, T, base, ldb, dX, lddx, dA, dB, P, stream)
               : backward<__bf16>(a, dY, lddy, X, ldx, T, base, ldb, dX, lddx, dA, dB, P, stream);
}

}  // namespace i8mm
