// Attention of one new token of each sequence over a paged key-value cache:
//   s_j = scale q . k_j + slope (j - (len - 1)) for the keys j < len,
//   o = sum_j softmax(s)_j v_j,  lse = log sum_j exp(s_j),
// in one pass over the keys with a running maximum and sum.
//
// Both products run on matrix instructions straight from registers, without
// LDS between them. A wavefront takes 32 keys at a time, as two halves of 16
// that each lie within a page. K times the transposed queries gives the
// scores with a query in each column: lane l holds those of query l % 16 and
// of the keys 4 (l / 16) .. + 3 of each half. That is the layout which the
// second product, V transposed times the probabilities, takes its right
// operand in, if the instruction's 32 reduction slots are given to the keys in
// that same order. Its left operand wants eight keys of one feature in a lane:
// a lane loads some adjacent features of its eight keys and sorts the halves
// of the registers by byte permutes.
//
// The 16 columns hold the query heads that share a key-value head. One head
// alone fills one column of 16: the matrix units are idle nearly all the time
// even so (24 instructions of 16 cycles for 16 KB of cache), since the
// cache's bytes are what bounds the kernel.

#include "launch.h"

#include "adapt_common.h"

namespace i8mm {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kHalf = 16;                        // keys of one matrix instruction
constexpr int kStep = 2 * kHalf;                 // keys of a wavefront's step
constexpr int kTile = kWaves * kStep;            // keys of a block's step
constexpr int kCols = 16;                        // queries of one matrix instruction
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// The probabilities of the running maximum are 2^kShift, so that in fp16 those
// down to 2^-29 of the largest keep all digits. The sum has the same factor.
constexpr float kShift = 15.0f;

typedef unsigned v2u __attribute__((ext_vector_type(2)));

template <typename T>
struct Vec8;
template <>
struct Vec8<_Float16> { typedef v8h type; };
template <>
struct Vec8<__bf16> { typedef v8b type; };

__device__ __forceinline__ v4f mma(v8h a, v8h b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ v4f mma(v8b a, v8b b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

__device__ __forceinline__ unsigned bits_of(float v) { return __builtin_bit_cast(unsigned, v); }

// The largest and the sum over the four lanes that hold one column.
__device__ __forceinline__ float column_max(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(bits_of(v), bits_of(v), false, false);
    v = fmaxf(__builtin_bit_cast(float, static_cast<unsigned>(a[0])), __builtin_bit_cast(float, static_cast<unsigned>(a[1])));
    const auto b = __builtin_amdgcn_permlane32_swap(bits_of(v), bits_of(v), false, false);
    return fmaxf(__builtin_bit_cast(float, static_cast<unsigned>(b[0])), __builtin_bit_cast(float, static_cast<unsigned>(b[1])));
}
__device__ __forceinline__ float column_sum(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(bits_of(v), bits_of(v), false, false);
    v = __builtin_bit_cast(float, static_cast<unsigned>(a[0])) + __builtin_bit_cast(float, static_cast<unsigned>(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(bits_of(v), bits_of(v), false, false);
    return __builtin_bit_cast(float, static_cast<unsigned>(b[0])) + __builtin_bit_cast(float, static_cast<unsigned>(b[1]));
}

// One step's keys and values in registers. NC: 32-feature chunks of a key; EL:
// features of a value that a lane holds.
template <int NC, int EL>
struct Step {
    v4u k[2][NC];            // half, chunk: 8 features of key l % 16
    unsigned v[2][4][EL / 2];   // half, key 4 (l / 16) + r: features EL (l % 16) ..
    int id[2];               // the halves' pages, -1 where there is none
    int key;                 // the first half's first key
};

template <typename T, int NC, int EL>
struct Sums {
    v4f o[EL];               // feature EL (4 (l / 16) + r) + e of query l % 16
    float m, l;              // maximum (in powers of 2) of the query; sum of this lane's keys
};

template <typename T, int NC, int EL, bool Full>
__device__ __forceinline__ void load_step(Step<NC, EL>& s, const AttendArgs& a, int64_t head_at, int lane) {
    const int x = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int key = s.key + h * kHalf;
        const int64_t page = s.id[h] < 0 ? 0 : s.id[h];      // any page: what it holds is masked
        const int64_t at = head_at + static_cast<int64_t>(key % a.page) * a.d;
        const T* K = static_cast<const T*>(a.K) + page * a.k_stride + at;
        const T* V = static_cast<const T*>(a.V) + page * a.v_stride + at;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int f = 32 * c + 8 * g;
            if (Full || f < a.d) s.k[h][c] = *reinterpret_cast<const v4u*>(K + x * a.d + f);
            else s.k[h][c] = v4u{0, 0, 0, 0};
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const T* row = V + (4 * g + r) * a.d + EL * x;
            if constexpr (EL == 4) {
                const v2u w = Full || 4 * x < a.d ? *reinterpret_cast<const v2u*>(row) : v2u{0, 0};
                s.v[h][r][0] = w[0];
                s.v[h][r][1] = w[1];
            } else {
#pragma unroll
                for (int p = 0; p < EL / 8; ++p) {
                    const v4u w = Full || EL * x + 8 * p < a.d ? *reinterpret_cast<const v4u*>(row + 8 * p) : v4u{0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < 4; ++i) s.v[h][r][4 * p + i] = w[i];
                }
            }
        }
    }
}

// The step's part of the sums. bias: slope of this lane's query times log2(e);
// last: the sequence's last key.
template <typename T, int NC, int EL>
__device__ __forceinline__ void add_step(Sums<T, NC, EL>& sum, Step<NC, EL>& s, const v4u (&q)[NC], float scale, float bias,
                                         int last, int lane) {
    typedef typename Vec8<T>::type vec;
    const int g = lane >> 4;
    float p[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < NC; ++c) acc = mma(__builtin_bit_cast(vec, s.k[h][c]), __builtin_bit_cast(vec, q[c]), acc);
        const int from = s.key + h * kHalf + 4 * g - last;    // <= 0 for the sequence's keys
#pragma unroll
        for (int r = 0; r < 4; ++r) p[h][r] = __builtin_fmaf(bias, static_cast<float>(from + r), acc[r] * scale);
        if (s.id[h] < 0 || s.key + h * kHalf + kHalf - 1 > last) {
            // keys that are not there: no weight, and whatever their slots hold stays out of the sums
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool there = s.id[h] >= 0 && from + r <= 0;
                p[h][r] = there ? p[h][r] : -INFINITY;
#pragma unroll
                for (int i = 0; i < EL / 2; ++i) s.v[h][r][i] = there ? s.v[h][r][i] : 0u;
            }
        }
    }
    float most = fmaxf(fmaxf(fmaxf(p[0][0], p[0][1]), fmaxf(p[0][2], p[0][3])),
                       fmaxf(fmaxf(p[1][0], p[1][1]), fmaxf(p[1][2], p[1][3])));
    most = fmaxf(column_max(most), sum.m);
    if (__any(most > sum.m)) {
        const float f = sum.m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(sum.m - most);
        sum.m = most;
        sum.l *= f;
#pragma unroll
        for (int e = 0; e < EL; ++e) sum.o[e] *= f;
    }
    const float off = sum.m == -INFINITY ? 0.0f : sum.m - kShift;
    vec w;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float v = __builtin_amdgcn_exp2f(p[h][r] - off);
            sum.l += v;
            w[4 * h + r] = static_cast<T>(v);
        }
#pragma unroll
    for (int e = 0; e < EL; ++e) {
        const unsigned pick = e % 2 ? 0x07060302u : 0x05040100u;
        v4u t;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) t[2 * h + r] = __builtin_amdgcn_perm(s.v[h][2 * r + 1][e / 2], s.v[h][2 * r][e / 2], pick);
        sum.o[e] = mma(__builtin_bit_cast(vec, t), w, sum.o[e]);
    }
}

template <typename T, int NC, int EL, bool Full>
__global__ __launch_bounds__(kThreads) void k_attend(const AttendArgs a) {
    __shared__ float s_o[kWaves][kCols][16 * EL];
    __shared__ float s_m[kWaves][kCols], s_l[kWaves][kCols];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int x = lane & 15, g = lane >> 4;
    const int group = a.heads / a.kv_heads, parts = (group + kCols - 1) / kCols;
    const int64_t items = static_cast<int64_t>(a.n) * a.kv_heads * parts;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int part = static_cast<int>(item % parts);
        const int kv = static_cast<int>(item / parts % a.kv_heads);
        const int64_t i = item / parts / a.kv_heads;
        const int cols = group - part * kCols < kCols ? group - part * kCols : kCols;
        const int first = kv * group + part * kCols;            // the first column's head
        const int most = a.max_pages * a.page;
        const int len = a.lens[i] < most ? a.lens[i] : most;
        const int64_t head_at = static_cast<int64_t>(kv) * a.page * a.d;

        v4u q[NC];
        const T* row = static_cast<const T*>(a.Q) + i * a.ldq + static_cast<int64_t>(first + x) * a.d;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int f = 32 * c + 8 * g;
            q[c] = x < cols && f < a.d ? *reinterpret_cast<const v4u*>(row + f) : v4u{0, 0, 0, 0};
        }
        const float bias = a.slopes && x < cols ? a.slopes[first + x] * kLog2e : 0.0f;

        Sums<T, NC, EL> sum;
        sum.m = -INFINITY;
        sum.l = 0.0f;
#pragma unroll
        for (int e = 0; e < EL; ++e) sum.o[e] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int key = wave * kStep; key < len; key += kTile) {
            Step<NC, EL> s;
            s.key = key;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = key + h * kHalf;
                int id = at < len ? a.tables[i * a.ldt + at / a.page] : -1;
                if (id >= a.n_pages) id = -1;
                s.id[h] = __builtin_amdgcn_readfirstlane(id);
            }
            load_step<T, NC, EL, Full>(s, a, head_at, lane);
            add_step<T, NC, EL>(sum, s, q, a.scale * kLog2e, bias, len - 1, lane);
        }
        sum.l = column_sum(sum.l);

        if (x < cols) {
            if (g == 0) {
                s_m[wave][x] = sum.m;
                s_l[wave][x] = sum.l;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < EL; ++e) s_o[wave][x][EL * (4 * g + r) + e] = sum.o[e][r];
        }
        __syncthreads();
        T* out = static_cast<T*>(a.out) + i * a.ldo + static_cast<int64_t>(first) * a.d;
        for (int k = threadIdx.x; k < cols * a.d; k += kThreads) {
            const int c = k / a.d, f = k % a.d;
            float m = s_m[0][c];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) m = fmaxf(m, s_m[w][c]);
            float l = 0.0f, o = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float by = s_m[w][c] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(s_m[w][c] - m);
                l = __builtin_fmaf(by, s_l[w][c], l);
                o = __builtin_fmaf(by, s_o[w][c][f], o);
            }
            out[k] = static_cast<T>(l == 0.0f ? 0.0f : o / l);
            if (f == 0 && a.lse) a.lse[i * a.heads + first + c] = l == 0.0f ? -INFINITY : (m + __builtin_log2f(l) - kShift) * kLn2;
        }
        __syncthreads();
    }
}

template <typename T, int NC, int EL>
hipError_t attend(const AttendArgs& a, hipStream_t stream) {
    const int parts = (a.heads / a.kv_heads + kCols - 1) / kCols;
    const int64_t items = static_cast<int64_t>(a.n) * a.kv_heads * parts;
    const unsigned blocks = static_cast<unsigned>(items < 4096 ? items : 4096);
    if (a.d == 32 * NC && a.d == 16 * EL) k_attend<T, NC, EL, true><<<blocks, kThreads, 0, stream>>>(a);
    else k_attend<T, NC, EL, false><<<blocks, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t attend_type(const AttendArgs& a, hipStream_t stream) {
    if (a.d <= 64) return attend<T, 2, 4>(a, stream);
    if (a.d <= 96) return attend<T, 3, 8>(a, stream);
    if (a.d <= 128) return attend<T, 4, 8>(a, stream);
    return attend<T, 8, 16>(a, stream);
}

}  // namespace

size_t decode_attention_scratch(int64_t, int, int, int) { return 256; }

hipError_t launch_decode_attention(const AttendArgs& a, void*, hipStream_t stream) {
    if (a.n == 0) return hipSuccess;
    return a.type == Dtype::F16 ? attend_type<_Float16>(a, stream) : attend_type<__bf16>(a, stream);
}

}  // namespace i8mm
