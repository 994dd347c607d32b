// Global gradient norm over many tensors, and clipping:
//   N = sqrt(sum over all tensors of the sum of squares),
//   c = min(1, max_norm / (N + 1e-6)),  out = c g.
// The squares are summed in fp64, so they neither overflow nor vanish for
// any fp32 gradient, and in an order that does not change from call to call.
//
// The tensors' addresses and sizes travel in the launch arguments, up to
// kBatch tensors a launch, so a call copies nothing to the device and keeps
// nothing. Two launches a batch: the squares, one fp64 part a block; then the
// scaling, whose blocks each join all parts in the same order while their
// first loads are in flight.

#include "launch.h"

#include "adapt_common.h"

#include <type_traits>

namespace i8mm {
namespace {

constexpr int kThreads = 512;
constexpr int kBatch = 128;          // tensors a launch: 29 bytes each, within 4 KB of launch arguments
constexpr int kChunkBytes = kThreads * 128;

// Elements of a chunk, and the groups of eight that each thread has in flight.
__host__ __device__ constexpr int chunk_elements(int type) {
    return kChunkBytes / (type == static_cast<int>(Dtype::F32) ? 4 : 2);
}
template <typename T>
constexpr int kEights = kChunkBytes / (kThreads * 8 * static_cast<int>(sizeof(T)));

struct Batch {
    const void* in[kBatch];
    void* out[kBatch];
    int64_t numel[kBatch];
    uint32_t first[kBatch];          // the tensor's first chunk within the batch
    uint8_t type[kBatch];
    int32_t n;
    uint32_t chunks;
};

__device__ __forceinline__ int tensor_of(const Batch& b, uint32_t chunk) {
    int lo = 0, hi = b.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (b.first[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

struct Piece {                       // one chunk of one tensor
    int64_t first;                   // its first element
    int count;
};

__device__ __forceinline__ Piece piece_of(const Batch& b, int tensor, uint32_t chunk) {
    const int size = chunk_elements(b.type[tensor]);
    const int64_t first = static_cast<int64_t>(chunk - b.first[tensor]) * size;
    const int64_t left = b.numel[tensor] - first;
    return {first, left < size ? static_cast<int>(left) : size};
}

// The sum over the block, in every thread.
__device__ __forceinline__ double block_sum_f64(double v, double* red) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) t += red[w];
    return t;
}

template <typename T>
__device__ __forceinline__ void load_piece(Eight<T>(&v)[kEights<T>], const void* base, const Piece& p) {
    const T* x = static_cast<const T*>(base) + p.first;
#pragma unroll
    for (int c = 0; c < kEights<T>; ++c) {
        const int j = (c * kThreads + threadIdx.x) * 8;
        v[c].load(x + j, p.count - j);
    }
}

template <typename T>
__device__ __forceinline__ double squares(const void* base, const Piece& p) {
    Eight<T> v[kEights<T>];
    load_piece(v, base, p);
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < kEights<T>; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const double x = v[c].at(k);
            sum = fma(x, x, sum);
        }
    return sum;
}

// Calls f with a null pointer of the element type.
template <typename F>
__device__ __forceinline__ void with_type(int type, F&& f) {
    if (type == static_cast<int>(Dtype::F16)) f(static_cast<_Float16*>(nullptr));
    else if (type == static_cast<int>(Dtype::BF16)) f(static_cast<__bf16*>(nullptr));
    else f(static_cast<float*>(nullptr));
}

__global__ __launch_bounds__(kThreads) void k_clip_squares(const Batch b, double* __restrict__ part) {
    __shared__ double red[kThreads / 64];
    double sum = 0.0;
    for (uint32_t chunk = blockIdx.x; chunk < b.chunks; chunk += gridDim.x) {
        const int tensor = tensor_of(b, chunk);
        const Piece p = piece_of(b, tensor, chunk);
        with_type(b.type[tensor],
                  [&](auto* t) { sum += squares<std::remove_pointer_t<decltype(t)>>(b.in[tensor], p); });
    }
    sum = block_sum_f64(sum, red);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The chunks are taken from the last to the first: the ones that the squares
// read last are the ones that a cache still holds; the results go past the
// caches, so that they do not push those out. Both kernels are bound by
// memory. 403 M fp16 gradients (805 MB read twice, written once): 139 us for
// the squares (5.8 TB/s) and 290 us here (5.5 TB/s); with ordinary stores 171
// and 283, as the squares of the next call then wait for the write-back; with
// each block's chunks adjacent instead of a grid apart 172 and 300.
__global__ __launch_bounds__(kThreads) void k_clip_scale(const Batch b, const double* __restrict__ part, int parts,
                                                         float max_norm, float* total) {
    __shared__ double red[kThreads / 64];
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) sum += part[i];
    const double norm = sqrt(block_sum_f64(sum, red));
    if (total && blockIdx.x == 0 && threadIdx.x == 0) total[0] = static_cast<float>(norm);
    const double ratio = max_norm / (norm + 1e-6);
    // A ratio below fp32's normal numbers, which gradients near fp32's upper end
    // make of a small limit, is applied in two steps, the second a power of two.
    const bool tiny = ratio < 0x1p-126;
    const double up = tiny ? 0x1p126 : 1.0;
    const float down = tiny ? 0x1p-126f : 1.0f;
    // A NaN reaches the gradients; an infinite norm over an infinite limit, whose
    // ratio is NaN too, leaves them alone.
    const float c = norm != norm ? static_cast<float>(norm) : ratio < 1.0 ? static_cast<float>(ratio * up) : 1.0f;
    for (uint32_t k = blockIdx.x; k < b.chunks; k += gridDim.x) {
        const uint32_t chunk = b.chunks - 1 - k;
        const int tensor = tensor_of(b, chunk);
        const Piece p = piece_of(b, tensor, chunk);
        const void* in = b.in[tensor];
        void* out = b.out[tensor];
        if (c * down == 1.0f && in == out) continue;
        with_type(b.type[tensor], [&](auto* t) {
            using T = std::remove_pointer_t<decltype(t)>;
            Eight<T> v[kEights<T>];
            load_piece(v, in, p);
            T* y = static_cast<T*>(out) + p.first;
#pragma unroll
            for (int q = 0; q < kEights<T>; ++q) {
                const int j = (q * kThreads + threadIdx.x) * 8;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[q].set(e, v[q].at(e) * c * down);
                v[q].store_through(y + j, p.count - j);
            }
        });
    }
}

// Calls f(batch) for the tensors in groups that fit one launch; empty tensors
// are left out.
template <typename F>
hipError_t for_batches(const void* const* in, void* const* out, const int64_t* numel, const int32_t* types, int64_t n,
                       F&& f) {
    Batch b;
    for (int64_t i = 0; i < n;) {
        b.n = 0;
        int64_t chunks = 0;
        for (; i < n && b.n < kBatch; ++i) {
            if (numel[i] == 0) continue;
            b.in[b.n] = in[i];
            b.out[b.n] = out ? out[i] : const_cast<void*>(in[i]);
            b.numel[b.n] = numel[i];
            b.first[b.n] = static_cast<uint32_t>(chunks);
            b.type[b.n] = static_cast<uint8_t>(types[i]);
            ++b.n;
            chunks += (numel[i] + chunk_elements(types[i]) - 1) / chunk_elements(types[i]);
        }
        if (b.n == 0) break;
        b.chunks = static_cast<uint32_t>(chunks);
        const hipError_t e = f(b);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

int64_t launches_of(int64_t n) { return (n + kBatch - 1) / kBatch; }

// Blocks of a launch: enough to fill the chip several times over, fewer when
// there are many launches, since every scaling block joins all their parts.
int64_t most_blocks(int64_t n) { return launches_of(n) > 8 ? 256 : 2048 / (n > 0 ? launches_of(n) : 1); }

}  // namespace

int64_t clip_parts(int64_t n) { return launches_of(n) * most_blocks(n); }

hipError_t launch_clip_grad_norm(const void* const* in, void* const* out, const int64_t* numel, const int32_t* types,
                                 int64_t n, float max_norm, void* workspace, float* total, hipStream_t stream) {
    double* part = static_cast<double*>(workspace);
    const int64_t most = most_blocks(n);
    int parts = 0;
    const auto blocks_of = [most](const Batch& b) { return static_cast<unsigned>(b.chunks < most ? b.chunks : most); };
    hipError_t e = for_batches(in, out, numel, types, n, [&](const Batch& b) {
        const unsigned blocks = blocks_of(b);
        k_clip_squares<<<blocks, kThreads, 0, stream>>>(b, part + parts);
        parts += static_cast<int>(blocks);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    bool told = false;                   // the first scaling launch writes the norm
    e = for_batches(in, out, numel, types, n, [&](const Batch& b) {
        k_clip_scale<<<blocks_of(b), kThreads, 0, stream>>>(b, part, parts, max_norm, told ? nullptr : total);
        told = true;
        return hipGetLastError();
    });
    if (e != hipSuccess || told) return e;
    Batch none;
    none.n = 0;
    none.chunks = 0;
    k_clip_scale<<<1, kThreads, 0, stream>>>(none, part, 0, max_norm, total);
    return hipGetLastError();
}

}  // namespace i8mm
