// Beam search's selection: of all continuations (beam i, token v) of a request
// the k best by
//   t = score_i + x_iv - lse_i,  lse_i = log sum_v exp(x_iv),
// ties to the lowest (beam, token).
//
// The logits are read once. A wavefront takes a part of a row and holds, in
// each lane, a running maximum and sum of exponentials, and, one a lane, the
// part's k best so far in order (within a row the logits alone order the
// tokens). What is not above the last of them costs a comparison; what is, is
// put in its place by a shift of the lanes behind it. A second launch joins a
// request's parts: the sums in fp64, then the k best of the parts' candidates.

#include "launch.h"

#include "adapt_common.h"

namespace i8mm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kStep = kWave * 8;                 // tokens of a wavefront's step
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kNone = 0x7fffffff;                // an empty place of a list: behind every token

__device__ __forceinline__ float lane_float(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ double lane_double(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b), lane));
    const uint64_t hi = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane));
    return __builtin_bit_cast(double, hi << 32 | lo);
}
__device__ __forceinline__ float lane_value(float v, int lane) { return lane_float(v, lane); }
__device__ __forceinline__ double lane_value(double v, int lane) { return lane_double(v, lane); }

// -inf in fp64 from a register that the compiler does not look into: as a
// constant of a whole wavefront it would become a scalar move of a 64-bit
// literal, which this target has no encoding for and the compiler drops to 0.
__device__ __forceinline__ double minus_infinity() {
    float f = -INFINITY;
    asm("" : "+v"(f));
    return f;
}
template <typename V>
__device__ __forceinline__ V least() {
    if constexpr (sizeof(V) == 8) return minus_infinity();
    else return -INFINITY;
}

// The k <= 64 best (value, index) pairs seen by a wavefront, lane i the i-th.
template <typename V>
struct Best {
    V value = least<V>();
    int index = kNone;
    V last = least<V>();                         // the k-th
    int last_index = kNone;

    __device__ __forceinline__ bool wants(V v, int i) const { return v > last || (v == last && i < last_index); }
    __device__ __forceinline__ void insert(V v, int i, int k, int lane) {
        const uint64_t ahead = __ballot(value > v || (value == v && index < i));
        const int at = __builtin_popcountll(ahead);
        const V up = __shfl_up(value, 1, kWave);
        const int up_index = __shfl_up(index, 1, kWave);
        value = lane > at ? up : lane == at ? v : value;
        index = lane > at ? up_index : lane == at ? i : index;
        last = lane_value(value, k - 1);
        last_index = __builtin_amdgcn_readlane(index, k - 1);
    }
    // Each lane offers one pair.
    __device__ __forceinline__ void offer(V v, int i, bool real, int k, int lane) {
        uint64_t left = __ballot(real && wants(v, i));
        while (left) {
            const int from = __builtin_ctzll(left);
            insert(lane_value(v, from), __builtin_amdgcn_readlane(i, from), k, lane);
            left = __ballot(real && wants(v, i)) & left & (left - 1);
        }
    }
};

__device__ __forceinline__ float wave_max_f(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, kWave));
    return v;
}

struct SelectScratch {
    float* most;                                 // [rows][parts]
    float* sum;                                  // [rows][parts]
    float* value;                                // [rows][parts][k]
    int32_t* token;                              // [rows][parts][k]
};

// Part of a row: a running maximum and sum (of powers of 2 of the logits times
// log2 e), and the k largest logits.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_select_scan(const SelectArgs a, const SelectScratch w, int parts, int part_len) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t items = a.n * a.beams * parts;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWaves + wave; item < items;
         item += static_cast<int64_t>(gridDim.x) * kWaves) {
        const int64_t row = item / parts;
        const int part = static_cast<int>(item - row * parts);
        const T* x = static_cast<const T*>(a.logits) + row * a.ld;
        const int from = part * part_len, to = from + part_len < a.vocab ? from + part_len : a.vocab;
        Best<float> best;
        float m = -INFINITY, l = 0.0f;
        for (int v0 = from; v0 < to; v0 += kStep) {
            const int v = v0 + 8 * lane;
            float f[8];
            Eight<T> e;
            e.load(x + v, to - v);
            float most = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] = v + i < to ? e.at(i) : -INFINITY;
                most = fmaxf(most, f[i]);
            }
            const float up = fmaxf(m, most);
            const float off = up == -INFINITY ? 0.0f : up;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += __builtin_amdgcn_exp2f((f[i] - off) * kLog2e);
            l = __builtin_fmaf(l, m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - off) * kLog2e), s);
            m = up;
            if (__any(v < to && best.wants(most, v))) {
#pragma unroll
                for (int i = 0; i < 8; ++i) best.offer(f[i], v + i, v + i < to, a.k, lane);
            }
        }
        const float top = wave_max_f(m);
        l = wave_sum(m == -INFINITY ? l : l * __builtin_amdgcn_exp2f((m - top) * kLog2e));
        if (lane == 0) {
            w.most[item] = top;
            w.sum[item] = l;
        }
        if (lane < a.k) {
            w.value[item * a.k + lane] = best.value;
            w.token[item * a.k + lane] = best.index;
        }
    }
}

// A block a request.
__global__ __launch_bounds__(kThreads) void k_select_join(const SelectArgs a, const SelectScratch w, int parts) {
    __shared__ double s_value[kWaves][kWave];
    __shared__ int s_index[kWaves][kWave];
    __shared__ double s_lse[kWave];              // of each beam; NaN: the beam leaves nothing
    __shared__ int s_parent[kWave];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t b = blockIdx.x; b < a.n; b += gridDim.x) {
        const int64_t row0 = b * a.beams;
        for (int i = wave; i < a.beams; i += kWaves) {
            const float* most = w.most + (row0 + i) * parts;
            const float* sum = w.sum + (row0 + i) * parts;
            float top = -INFINITY;
            for (int p = lane; p < parts; p += kWave) top = fmaxf(top, most[p]);
            top = wave_max_f(top);
            double l = 0.0;
            for (int p = lane; p < parts; p += kWave) {
                const double by = most[p] == -INFINITY ? 0.0 : exp(static_cast<double>(most[p]) - top);
                l += sum[p] * by;
            }
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) l += __shfl_xor(l, off, kWave);
            const double score = a.scores[row0 + i];
            const double lse = top + log(l);
            if (lane == 0) s_lse[i] = (lse - lse) + (score - score) == 0.0 ? lse : NAN;
        }
        __syncthreads();
        Best<double> best;
        const int each = parts * a.k, all = a.beams * each;
        const float* value = w.value + row0 * each;
        const int32_t* token = w.token + row0 * each;
        // the parts' first candidates come first, so that few of the others are put in
        for (int c0 = wave * kWave; c0 < all; c0 += kThreads) {
            const int c = c0 + lane, rank = c / (a.beams * parts), list = c - rank * (a.beams * parts);
            const int beam = list / parts;
            const double none = minus_infinity();
            double t = none;
            int v = kNone;
            if (c < all) {
                const double lse = s_lse[beam];
                if (lse == lse) {
                    v = token[list * a.k + rank];
                    t = a.scores[row0 + beam] + (value[list * a.k + rank] - lse);
                } else if (list == beam * parts) {
                    v = rank < a.vocab ? rank : kNone;   // nothing to choose by: the lowest tokens, with no weight
                }
            }
            best.offer(t, v == kNone ? kNone : beam * a.vocab + v, v != kNone, a.k, lane);
        }
        s_value[wave][lane] = best.value;
        s_index[wave][lane] = best.index;
        __syncthreads();
        if (wave == 0) {
            for (int o = 1; o < kWaves; ++o)
                best.offer(s_value[o][lane], s_index[o][lane], lane < a.k && s_index[o][lane] != kNone, a.k, lane);
            if (lane < a.k) {
                const int beam = best.index / a.vocab, v = best.index - beam * a.vocab;
                a.scores_out[b * a.k + lane] = static_cast<float>(best.value);
                a.parents[b * a.k + lane] = static_cast<int>(row0 + beam);
                a.tokens[b * a.k + lane] = v;
                s_parent[lane] = beam;
                if (a.history_out) a.history_out[(b * a.k + lane) * a.ldho + a.T] = v;
            }
        }
        __syncthreads();
        if (a.history_out) {
            for (int i = wave; i < a.k; i += kWaves) {
                const int32_t* in = a.history + (row0 + s_parent[i]) * a.ldh;
                int32_t* out = a.history_out + (b * a.k + i) * a.ldho;
                for (int64_t t = lane; t < a.T; t += kWave) out[t] = in[t];
            }
        }
        __syncthreads();
    }
}

// Parts of a row: as many as fill the chip four wavefronts to a SIMD, each of
// four steps at least.
int parts_of(int64_t rows, int vocab) {
    const int64_t fill = 4096 / (rows < 1 ? 1 : rows < 4096 ? rows : 4096), most = (vocab + 4 * kStep - 1) / (4 * kStep);
    return static_cast<int>(fill < most ? fill : most);
}

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t beam_select_scratch(int64_t n, int beams, int vocab, int k) {
    const int64_t lists = n * beams * parts_of(n * beams, vocab);
    return static_cast<size_t>(2 * round256(4 * lists) + 2 * round256(4 * lists * k));
}

hipError_t launch_beam_select(const SelectArgs& a, void* workspace, hipStream_t stream) {
    if (a.n == 0) return hipSuccess;
    const int64_t rows = a.n * a.beams;
    const int parts = parts_of(rows, a.vocab);
    const int part_len = (a.vocab + parts * kStep - 1) / (parts * kStep) * kStep;
    const int64_t lists = rows * parts;
    char* at = static_cast<char*>(workspace);
    SelectScratch w;
    w.most = reinterpret_cast<float*>(at);
    w.sum = reinterpret_cast<float*>(at += round256(4 * lists));
    w.value = reinterpret_cast<float*>(at += round256(4 * lists));
    w.token = reinterpret_cast<int32_t*>(at + round256(4 * lists * a.k));
    const int64_t blocks = (lists + kWaves - 1) / kWaves;
    const unsigned grid = static_cast<unsigned>(blocks < 65536 ? blocks : 65536);
    if (a.type == Dtype::F16) k_select_scan<_Float16><<<grid, kThreads, 0, stream>>>(a, w, parts, part_len);
    else if (a.type == Dtype::BF16) k_select_scan<__bf16><<<grid, kThreads, 0, stream>>>(a, w, parts, part_len);
    else k_select_scan<float><<<grid, kThreads, 0, stream>>>(a, w, parts, part_len);
    k_select_join<<<static_cast<unsigned>(a.n < 65536 ? a.n : 65536), kThreads, 0, stream>>>(a, w, parts);
    return hipGetLastError();
}

}  // namespace i8mm
