// Global gradient norm over many tensors, and clipping:
//   N = sqrt(sum over all tensors of the sum of squares),
//   c = min(1, max_norm / (N + 1e-6)),  out = c g.
// The squares are summed in fp64, so they neither overflow nor vanish for
// any fp32 gradient, and in an order that does not change from call to call.
//
// The tensors' addresses and sizes travel in the launch arguments, up to
// kBatch tensors a launch, so a call copies nothing to the device and keeps
// nothing.

#include "launch.h"

#include "adapt_common.h"

#include <cmath>

namespace i8mm {
namespace {

constexpr int kClipThreads = 256;
constexpr int kBatch = 96;
constexpr int64_t kChunk = 16384;    // elements per block

struct Batch {
    const void* in[kBatch];
    void* out[kBatch];
    int64_t numel[kBatch];
    uint32_t first[kBatch];          // the tensor's first chunk within the launch
    int32_t type[kBatch];
    int32_t n;
};

__device__ __forceinline__ float element(const void* p, int type, int64_t i) {
    if (type == static_cast<int>(Dtype::F16)) return to_float(static_cast<const _Float16*>(p)[i]);
    if (type == static_cast<int>(Dtype::BF16)) return to_float(static_cast<const __bf16*>(p)[i]);
    return static_cast<const float*>(p)[i];
}

// The tensor that chunk c of the launch belongs to.
__device__ __forceinline__ int tensor_of(const Batch& b, uint32_t c) {
    int lo = 0, hi = b.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (b.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ double block_sum_f64(double v, double* red) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kClipThreads / 64; ++w) t += red[w];
    return t;
}

__global__ __launch_bounds__(kClipThreads) void k_clip_squares(const Batch b, double* __restrict__ part) {
    __shared__ double red[kClipThreads / 64];
    const int t = tensor_of(b, blockIdx.x);
    const int64_t i0 = static_cast<int64_t>(blockIdx.x - b.first[t]) * kChunk;
    const int64_t i1 = i0 + kChunk < b.numel[t] ? i0 + kChunk : b.numel[t];
    double sum = 0.0;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kClipThreads) {
        const double v = element(b.in[t], b.type[t], i);
        sum = fma(v, v, sum);
    }
    sum = block_sum_f64(sum, red);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// One block: the norm and the factor, in slot[0] as fp32 pair.
__global__ __launch_bounds__(kClipThreads) void k_clip_total(const double* __restrict__ part, int64_t parts,
                                                             float max_norm, float* __restrict__ total,
                                                             float* __restrict__ factor) {
    __shared__ double red[kClipThreads / 64];
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < parts; i += kClipThreads) sum += part[i];
    sum = block_sum_f64(sum, red);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum);
        const double c = max_norm / (norm + 1e-6);
        total[0] = static_cast<float>(norm);
        factor[0] = c < 1.0 || c != c ? static_cast<float>(c) : 1.0f;   // a NaN norm reaches the gradients
    }
}

__global__ __launch_bounds__(kClipThreads) void k_clip_scale(const Batch b, const float* __restrict__ factor) {
    const int t = tensor_of(b, blockIdx.x);
    const int64_t i0 = static_cast<int64_t>(blockIdx.x - b.first[t]) * kChunk;
    const int64_t i1 = i0 + kChunk < b.numel[t] ? i0 + kChunk : b.numel[t];
    const float c = factor[0];
    if (c == 1.0f && b.in[t] == b.out[t]) return;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kClipThreads) {
        const float v = element(b.in[t], b.type[t], i) * c;
        if (b.type[t] == static_cast<int>(Dtype::F16)) static_cast<_Float16*>(b.out[t])[i] = from_float<_Float16>(v);
        else if (b.type[t] == static_cast<int>(Dtype::BF16)) static_cast<__bf16*>(b.out[t])[i] = from_float<__bf16>(v);
        else static_cast<float*>(b.out[t])[i] = v;
    }
}

int64_t chunks_of(int64_t numel) { return (numel + kChunk - 1) / kChunk; }

// Calls f(batch, chunks of the batch, chunks before it) for the tensors in
// groups that fit one launch; empty tensors are left out.
template <typename F>
hipError_t for_batches(const void* const* in, void* const* out, const int64_t* numel, const int32_t* types, int64_t n,
                       F&& f) {
    int64_t before = 0;
    for (int64_t i = 0; i < n;) {
        Batch b;
        b.n = 0;
        int64_t chunks = 0;
        for (; i < n && b.n < kBatch; ++i) {
            if (numel[i] == 0) continue;
            const int64_t c = chunks_of(numel[i]);
            if (b.n > 0 && chunks + c > 0x7fffffff) break;
            b.in[b.n] = in[i];
            b.out[b.n] = out ? out[i] : const_cast<void*>(in[i]);
            b.numel[b.n] = numel[i];
            b.first[b.n] = static_cast<uint32_t>(chunks);
            b.type[b.n] = types[i];
            ++b.n;
            chunks += c;
        }
        if (b.n == 0) break;
        const hipError_t e = f(b, chunks, before);
        if (e != hipSuccess) return e;
        before += chunks;
    }
    return hipSuccess;
}

}  // namespace

int64_t clip_parts(const int64_t* numel, int64_t n) {
    int64_t parts = 0;
    for (int64_t i = 0; i < n; ++i) parts += chunks_of(numel[i]);
    return parts;
}

hipError_t launch_clip_grad_norm(const void* const* in, void* const* out, const int64_t* numel, const int32_t* types,
                                 int64_t n, float max_norm, void* workspace, float* total, hipStream_t stream) {
    float* factor = static_cast<float*>(workspace);
    double* part = reinterpret_cast<double*>(static_cast<char*>(workspace) + 256);
    hipError_t e = for_batches(in, out, numel, types, n, [&](const Batch& b, int64_t chunks, int64_t before) {
        k_clip_squares<<<static_cast<unsigned>(chunks), kClipThreads, 0, stream>>>(b, part + before);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    k_clip_total<<<1, kClipThreads, 0, stream>>>(part, clip_parts(numel, n), max_norm, total, factor);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    return for_batches(in, out, numel, types, n, [&](const Batch& b, int64_t chunks, int64_t) {
        k_clip_scale<<<static_cast<unsigned>(chunks), kClipThreads, 0, stream>>>(b, factor);
        return hipGetLastError();
    });
}

}  // namespace i8mm
