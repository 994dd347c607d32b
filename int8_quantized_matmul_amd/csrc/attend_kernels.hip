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
// even so (16 instructions of 16 cycles for 16 KB of cache), since the cache's
// bytes are what bounds the kernel. The second product takes the probabilities in the
// cache's own type, in two parts: rounded, and what that rounding left, so that they are off
// by half a step of half a step (2^-16 in bf16, 2^-22 in fp16) and the values' sum is as
// good as the other sums, for 0.3 % of the time. (An infinite value times a second part that
// is 0 or negative is no number; such a column is computed again, see attend_again().)
//
// 64 sequences x 96 heads of 128 features, up to 2048 tokens each (3.2 GB): 528 us,
// 6.1 TB/s, and 10 us for joining. What it took: values loaded past the caches (51 us
// less than ordinary loads: a CU's L1 cache is smaller than what is in flight through
// it), and runs of about 24 tiles in the order of the rows, so that the heads of
// a page are read at about the same time (79 us less than one run a block, a twelfth
// of the heads apart). A step's loads before the last one's products, or three blocks
// a CU, change nothing: the wavefronts of a CU cover for one another.

#include "../../include/i8mm.h"
#include "launch.h"

#include "adapt_common.h"

#include <type_traits>

namespace i8mm {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kHalf = 16;                        // keys of one matrix instruction
constexpr int kStep = 2 * kHalf;                 // keys of a wavefront's step
constexpr int kTile = kWaves * kStep;            // keys of a block's step
constexpr int kCols = 16;                        // queries of one matrix instruction
constexpr int kRunTiles = 24;                    // tiles of a run, if there are enough for several runs a block
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
typedef unsigned v2u __attribute__((ext_vector_type(2)));

// kShift: the running maximum's probability is 2^kShift, and the sum has the same
// factor. In fp16 15: probabilities keep all digits down to 2^-29 of the largest, and
// sums of 2^31 values times 2^15 stay far below fp32's end. bf16 needs none.
template <typename T>
struct Vec8;
template <>
struct Vec8<_Float16> {
    typedef v8h type;
    static constexpr float kShift = 15.0f;
};
template <>
struct Vec8<__bf16> {
    typedef v8b type;
    static constexpr float kShift = 0.0f;
};

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
    v4u k[2][NC];               // half, chunk: 8 features of key l % 16
    unsigned v[2][4][EL / 2];   // half, key 4 (l / 16) + r: features EL (l % 16) ..
    int id[2];                  // the halves' pages, -1 where there is none
    int key;                    // the first half's first key
};

template <int EL>
struct Sums {
    v4f o[EL];               // feature EL (4 (l / 16) + r) + e of query l % 16
    float m, l;              // maximum (in powers of 2) of the query; sum of this lane's keys
};

// What a wavefront's columns ask for.
template <int NC>
struct Queries {
    v4u q[NC];               // 8 features of query l % 16
    float scale, bias;       // times log2 e
    int last;                // the query's own sequence's last key, which the biases count from
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
                const v2u w = Full || 4 * x < a.d ? __builtin_nontemporal_load(reinterpret_cast<const v2u*>(row)) : v2u{0, 0};
                s.v[h][r][0] = w[0];
                s.v[h][r][1] = w[1];
            } else {
#pragma unroll
                for (int p = 0; p < EL / 8; ++p) {
                    const v4u w = Full || EL * x + 8 * p < a.d ? __builtin_nontemporal_load(reinterpret_cast<const v4u*>(row + 8 * p))
                                                                : v4u{0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < 4; ++i) s.v[h][r][4 * p + i] = w[i];
                }
            }
        }
    }
}

// The step's part of the sums. last: the last key that may be seen. Alone: the
// step is that of some columns (`mine`), the others stay as they are.
template <typename T, int NC, int EL, bool Alone>
__device__ __forceinline__ void add_step(Sums<EL>& sum, Step<NC, EL>& s, const Queries<NC>& q, int last, bool mine, int lane) {
    typedef typename Vec8<T>::type vec;
    const int g = lane >> 4;
    float p[2][4];
    float least = INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < NC; ++c) acc = mma(__builtin_bit_cast(vec, s.k[h][c]), __builtin_bit_cast(vec, q.q[c]), acc);
        const int key = s.key + h * kHalf + 4 * g;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            p[h][r] = __builtin_fmaf(q.bias, static_cast<float>(key + r - q.last), acc[r] * q.scale);
        }
        float least_here = fminf(fminf(p[h][0], p[h][1]), fminf(p[h][2], p[h][3]));
        if (s.id[h] < 0 || s.key + h * kHalf + kHalf - 1 > last) {
            // keys that are not there: no weight, and whatever their slots hold stays out of the sums
            least_here = INFINITY;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool there = s.id[h] >= 0 && key + r <= last;
                least_here = there ? fminf(least_here, p[h][r]) : least_here;
                p[h][r] = there ? p[h][r] : -INFINITY;
#pragma unroll
                for (int i = 0; i < EL / 2; ++i) s.v[h][r][i] = there ? s.v[h][r][i] : 0u;
            }
        }
        least = fminf(least, least_here);
        if (Alone) {
#pragma unroll
            for (int r = 0; r < 4; ++r) p[h][r] = mine ? p[h][r] : -INFINITY;
        }
    }
    // A score of -inf is one that fp32 has no room for (or a sum that has left it on the way),
    // unless it is that of a key that is not there: its column is computed again.
    if (least == -INFINITY && (!Alone || mine)) sum.l = NAN;
    float most = fmaxf(fmaxf(fmaxf(p[0][0], p[0][1]), fmaxf(p[0][2], p[0][3])),
                       fmaxf(fmaxf(p[1][0], p[1][1]), fmaxf(p[1][2], p[1][3])));
    most = fmaxf(column_max(most), sum.m);
    if (__any(most > sum.m)) {
        const float f = sum.m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(sum.m - most);
        const float by = most == -INFINITY ? 1.0f : f;
        sum.m = most;
        sum.l *= by;
#pragma unroll
        for (int e = 0; e < EL; ++e) sum.o[e] *= by;
    }
    const float off = sum.m == -INFINITY ? 0.0f : sum.m - Vec8<T>::kShift;
    vec w, rest;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float v = __builtin_amdgcn_exp2f(p[h][r] - off);
            sum.l += v;
            w[4 * h + r] = static_cast<T>(v);
            rest[4 * h + r] = static_cast<T>(v - static_cast<float>(w[4 * h + r]));
        }
#pragma unroll
    for (int e = 0; e < EL; ++e) {
        const unsigned pick = e % 2 ? 0x07060302u : 0x05040100u;
        v4u t;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) t[2 * h + r] = __builtin_amdgcn_perm(s.v[h][2 * r + 1][e / 2], s.v[h][2 * r][e / 2], pick);
        const v4f o = mma(__builtin_bit_cast(vec, t), rest, mma(__builtin_bit_cast(vec, t), w, sum.o[e]));
        // a NaN among these values times a weight of 0 must not reach the other columns
        if (Alone) sum.o[e] = mine ? o : sum.o[e];
        else sum.o[e] = o;
    }
}

// ---------------------------------------------------------------- how the work is split
//
// Sequences are taken in groups: `beams` of them that may share pages, as many as
// their queries fill the 16 columns (one sequence if beams is 1). A group's tiles of
// 128 keys are first those that all its sequences share, read once for all, then each
// sequence's own. All groups, heads and tiles are one row of units, cut into equal
// runs: lengths may differ as they like, and a few long sequences fill the chip as
// well as many short ones. A run that covers all units of a (group, head) writes its
// result; the others leave partial sums (at most two a run: of the one it starts in,
// and of the one it ends in), which a second launch joins.

struct Split {
    int64_t groups;
    int gb, chunks;          // sequences of a group at most, groups of `beams` sequences
    int group, parts;        // heads that share a key-value head, in parts of 16
    const int32_t* shared;   // [groups]: tiles that a group's sequences share (null: groups of one)
    int cols;                // columns in use, at most
    int rounds;              // runs of a block, at most
    float* o;                // [runs][2][cols][d]: the partial sums
    float* ml;               // [runs][2][cols][2]: their maximum and sum
    struct Join {
        int64_t group;
        int head;            // key-value head and part
        int first;           // the run with the first partial sums, -1: nothing to join
        int64_t whole;       // the first (group, head) whose result the run writes itself
        int64_t beyond;      // and the last one that is not finite, -1: none
    }* joins;                // [runs]
};

__device__ __forceinline__ int clamped_len(const AttendArgs& a, int64_t seq) {
    const int len = a.lens[seq], most = a.max_pages * a.page;
    return len < 0 ? 0 : len < most ? len : most;
}

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

struct Group {
    int64_t first;           // its first sequence
    int n;                   // and how many they are
};
__device__ __forceinline__ Group group_at(const AttendArgs& a, const Split& w, int64_t gi) {
    if (w.chunks == 1) return {gi * a.beams, a.beams};
    const int64_t r = gi / w.chunks;
    const int c = static_cast<int>(gi - r * w.chunks) * w.gb;
    return {r * a.beams + c, a.beams - c < w.gb ? a.beams - c : w.gb};
}

// Units of a group for one head: at least one, which writes the result of empty sequences.
template <bool Beams>
__device__ __forceinline__ int64_t units_of(const AttendArgs& a, const Split& w, int64_t gi) {
    int64_t u = 0;
    if (Beams) {
        const Group g = group_at(a, w, gi);
        const int s = w.shared[gi];
        u = s;
        for (int b = 0; b < g.n; ++b) {
            const int t = tiles_of(clamped_len(a, g.first + b)) - s;
            u += t > 0 ? t : 0;
        }
    } else {
        u = tiles_of(clamped_len(a, gi));
    }
    return u > 0 ? u : 1;
}

// The tiles that all sequences of a group share: the same keys of the same pages. A wavefront a group.
__global__ __launch_bounds__(kThreads) void k_attend_shared(const AttendArgs a, const Split w, int32_t* shared) {
    const int lane = threadIdx.x & 63;
    for (int64_t gi = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6); gi < w.groups;
         gi += static_cast<int64_t>(gridDim.x) * kWaves) {
        const Group g = group_at(a, w, gi);
        int least = clamped_len(a, g.first), most = least;
        for (int b = 1; b < g.n; ++b) {
            const int len = clamped_len(a, g.first + b);
            least = len < least ? len : least;
            most = len > most ? len : most;
        }
        // where lengths differ, a tile is shared as far as it is full for all
        int keys = least == most ? tiles_of(most) * kTile : least / kTile * kTile;
        const int used = ((keys < most ? keys : most) + a.page - 1) / a.page;
        for (int c0 = 0; c0 < used; c0 += kWave) {
            const int c = c0 + lane;
            bool differ = false;
            if (c < used) {
                const int id = a.tables[g.first * a.ldt + c];
                for (int b = 1; b < g.n; ++b) differ |= a.tables[(g.first + b) * a.ldt + c] != id;
            }
            const uint64_t any = __ballot(differ);
            if (any) {
                keys = (c0 + __builtin_ctzll(any)) * a.page / kTile * kTile;
                break;
            }
        }
        if (lane == 0) shared[gi] = keys / kTile;
    }
}

// ---------------------------------------------------------------- beyond fp32
//
// A sum of values near fp32's end, a weighted mean that its weights' rounding takes past the
// type's largest number, or a score (or a part of its sum) beyond fp32 is infinite, while the
// result is not. A column whose result is not finite, or of which a key has a score of -inf
// (add_step() makes its sum a NaN then), is computed again by a block in fp64, which has room
// for all that finite inputs can give, from the definition: the keys' scores for the maximum,
// then once more for the weights, a key a thread, and the values with 8 features a thread, of
// 256 / (d / 8) groups that take the keys in turn. It is meant to be rare: one column of 2048
// keys of 128 features takes 110 us, of 100000 6.4 ms, all of 64 x 32 with 2048 1.4 ms on top
// of 0.4 (where the scores hold a NaN or infinity, which ends it after the maximum, 40 us,
// 2.4 and 0.6 ms). Smaller weights instead would lose the smallest values, so they would have
// to follow the values.

constexpr int kAgainAhead = 4;                   // loads of a thread on their way

struct Again {
    double value[kThreads];
    double part[kWaves];
    int64_t at[kThreads];    // a key's values, -1: there is no key
};

__device__ __forceinline__ bool finite(float v) { return v - v == 0.0f; }

// f(a, b) over all threads' values, in every thread.
template <typename F>
__device__ __forceinline__ double over_block(Again& s, double v, F&& f) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = f(v, __shfl_xor(v, off, kWave));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s.part[0];
    for (int k = 1; k < kWaves; ++k) v = f(v, s.part[k]);
    return v;
}

// Query head `head` of sequence `seq` over all its keys, out and lse (the block's earlier ones are written over).
template <typename T>
__device__ __forceinline__ void attend_again(const AttendArgs& a, Again& s, int64_t seq, int head) {
    typedef typename Vec8<T>::type vec;
    const int tid = static_cast<int>(threadIdx.x), len = clamped_len(a, seq), kv = head / (a.heads / a.kv_heads);
    const T* q = static_cast<const T*>(a.Q) + seq * a.ldq + static_cast<int64_t>(head) * a.d;
    T* out = static_cast<T*>(a.out) + seq * a.ldo + static_cast<int64_t>(head) * a.d;
    const auto wide = [](T v) { return static_cast<double>(static_cast<float>(v)); };
    const int eights = a.d / 8, sharers = kThreads / eights, by = tid / eights, i = 8 * (tid - by * eights);
    double most = minus_infinity(), l = 0.0, o[8] = {};
    const auto larger = [](double x, double y) { return y > x || y != y ? y : x; };   // (a NaN, if one of them is)
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int t0 = 0; t0 < len; t0 += kThreads) {
            const int t = t0 + tid, id = t < len ? a.tables[seq * a.ldt + t / a.page] : -1;
            const bool there = id >= 0 && id < a.n_pages;
            const int64_t page = there ? id : 0, within = (static_cast<int64_t>(kv) * a.page + t % a.page) * a.d;
            double x = minus_infinity();
            if (there) {
                const T* k = static_cast<const T*>(a.K) + page * a.k_stride + within;
                x = 0.0;
#pragma unroll 1
                for (int f0 = 0; f0 < a.d; f0 += 8 * kAgainAhead) {
                    vec u[kAgainAhead], v[kAgainAhead];
#pragma unroll
                    for (int b = 0; b < kAgainAhead; ++b) {
                        const int f = f0 + 8 * b < a.d ? f0 + 8 * b : 0;
                        u[b] = *reinterpret_cast<const vec*>(q + f);
                        v[b] = *reinterpret_cast<const vec*>(k + f);
                    }
#pragma unroll
                    for (int b = 0; b < kAgainAhead; ++b) {
                        if (f0 + 8 * b >= a.d) break;
#pragma unroll
                        for (int e = 0; e < 8; ++e) x = __builtin_fma(wide(u[b][e]), wide(v[b][e]), x);
                    }
                }
                x *= static_cast<double>(a.scale);
                if (a.slopes) x = __builtin_fma(static_cast<double>(a.slopes[head]), static_cast<double>(t - (len - 1)), x);
            }
            if (pass == 0) {
                most = larger(most, x);
                continue;
            }
            const double w = there ? exp(x - most) : 0.0;
            l += w;
            __syncthreads();
            s.value[tid] = w;
            s.at[tid] = there ? page * a.v_stride + within : -1;
            __syncthreads();
            const int count = by >= sharers ? 0 : len - t0 < kThreads ? len - t0 : kThreads;
#pragma unroll 1
            for (int k0 = by; k0 < count; k0 += kAgainAhead * sharers) {
                int64_t at[kAgainAhead];
                vec v[kAgainAhead];
#pragma unroll
                for (int b = 0; b < kAgainAhead; ++b) at[b] = k0 + b * sharers < count ? s.at[k0 + b * sharers] : -1;
#pragma unroll
                for (int b = 0; b < kAgainAhead; ++b)
                    v[b] = *reinterpret_cast<const vec*>(static_cast<const T*>(a.V) + (at[b] < 0 ? 0 : at[b]) + i);
#pragma unroll
                for (int b = 0; b < kAgainAhead; ++b) {
                    if (at[b] < 0) continue;
                    const double by_w = s.value[k0 + b * sharers];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = __builtin_fma(by_w, wide(v[b][e]), o[e]);
                }
            }
        }
        if (pass > 0) break;
        most = over_block(s, most, larger);
        if (most - most == 0.0) continue;
        // no number: it is the logarithm of the sum as well, and a weight is exp(inf - inf)
        if (by == 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) out[i + e] = static_cast<T>(NAN);
        }
        if (tid == 0 && a.lse) a.lse[seq * a.heads + head] = static_cast<float>(most);
        return;
    }
    l = over_block(s, l, [](double x, double y) { return x + y; });
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        s.value[tid] = o[e];
        __syncthreads();
        if (by == 0) {
            double sum = 0.0;
            for (int k = 0; k < sharers; ++k) sum += s.value[k * eights + tid];
            out[i + e] = static_cast<T>(static_cast<float>(sum / l));
        }
        __syncthreads();
    }
    if (tid == 0 && a.lse) a.lse[seq * a.heads + head] = static_cast<float>(most + log(l));
}

template <int NC, int EL>
struct Attend {
    static constexpr int kWide = 16 * EL;
    union {
        float o[kWaves][kCols][kWide];
        Again again;
    };
    float m[kWaves][kCols], l[kWaves][kCols];
    int64_t scan[kWaves];
    int64_t at_group, at_units;
    unsigned beyond;         // the columns whose result is not finite
};

// Joins the wavefronts' sums; f(column, feature, o, m, l) for each, o and l relative to the maximum m.
template <int NC, int EL, typename F>
__device__ __forceinline__ void join_waves(Attend<NC, EL>& s, const Sums<EL>& sum, int cols, int d, int wave, int lane, F&& f) {
    const int x = lane & 15, g = lane >> 4;
    const float l = column_sum(sum.l);
    if (x < cols) {
        if (g == 0) {
            s.m[wave][x] = sum.m;
            s.l[wave][x] = l;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < EL; ++e) s.o[wave][x][EL * (4 * g + r) + e] = sum.o[e][r];
    }
    __syncthreads();
    for (int k = threadIdx.x; k < cols * d; k += kThreads) {
        const int c = k / d, i = k - c * d;
        float m = s.m[0][c];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) m = fmaxf(m, s.m[w][c]);
        float all = 0.0f, o = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float by = s.m[w][c] == -INFINITY ? (s.l[w][c] == 0.0f ? 0.0f : 1.0f) : __builtin_amdgcn_exp2f(s.m[w][c] - m);
            all = __builtin_fmaf(by, s.l[w][c], all);
            o = __builtin_fmaf(by, s.o[w][c][i], o);
        }
        f(c, i, o, m, all);
    }
    __syncthreads();
}

template <typename T>
__device__ __forceinline__ float log_sum(float m, float l) {
    return l == 0.0f ? -INFINITY : (m + __builtin_log2f(l) - Vec8<T>::kShift) * kLn2;
}

// Column c of a group's head: its sequence and head.
struct Column {
    int64_t seq;
    int head;
};
__device__ __forceinline__ Column column_of(const Split& w, const Group& g, int kv, int part, int c) {
    if (w.parts > 1) return {g.first, kv * w.group + part * kCols + c};
    const int b = c / w.group;
    return {g.first + b, kv * w.group + c - b * w.group};
}

__device__ __forceinline__ int columns_of(const Split& w, const Group& g, int part) {
    if (w.parts > 1) return w.group - part * kCols < kCols ? w.group - part * kCols : kCols;
    return g.n * w.group;
}

// Feature i of a column's result; whether it is finite.
template <typename T>
__device__ __forceinline__ bool put(const AttendArgs& a, const Column& c, int i, float o, float m, float l) {
    const T v = static_cast<T>(l == 0.0f ? 0.0f : o / l);
    static_cast<T*>(a.out)[c.seq * a.ldo + static_cast<int64_t>(c.head) * a.d + i] = v;
    if (i == 0 && a.lse) a.lse[c.seq * a.heads + c.head] = log_sum<T>(m, l);
    return finite(static_cast<float>(v));
}

// Runs of the split kernel in multiples of the blocks that are resident at once; heads
// of up to 64 features take twice as many to have as much in flight.
template <int EL>
constexpr int kBlocks = EL == 16 ? 256 : EL == 8 ? 512 : 1024;

// Whole: each block takes whole (group, head)s, and nothing is left to join.
template <typename T, int NC, int EL, bool Full, bool Beams, bool Whole>
__global__ __launch_bounds__(kThreads, kBlocks<EL> / 256) void k_attend(const AttendArgs a, const Split w, int64_t run0) {
    __shared__ Attend<NC, EL> s;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int x = lane & 15, g = lane >> 4;
    const int heads = a.kv_heads * w.parts;
    const int64_t run = run0 + blockIdx.x;
    int64_t runs = 0, total = 0, before = 0, mine = 0, g0 = 0;
    if (!Whole) {
        // units of all groups: each thread sums some neighbours
        const int64_t per = (w.groups + kThreads - 1) / kThreads;
        g0 = threadIdx.x * per;
        const int64_t g1 = g0 + per < w.groups ? g0 + per : w.groups;
        for (int64_t k = g0; k < g1; ++k) mine += units_of<Beams>(a, w, k);
        int64_t upto = mine;
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
            const int64_t t = __shfl_up(upto, off, kWave);
            if (lane >= off) upto += t;
        }
        if (lane == 63) s.scan[wave] = upto;
        __syncthreads();
        for (int k = 0; k < kWaves; ++k) {
            if (k < wave) before += s.scan[k];
            total += s.scan[k];
        }
        before += upto - mine;
        total *= heads;
        const int64_t rounds = total / (static_cast<int64_t>(kBlocks<EL>) * kRunTiles);
        runs = kBlocks<EL> * (rounds < 1 ? 1 : rounds < w.rounds ? rounds : w.rounds);
        runs = total < runs ? total : runs;
        if (threadIdx.x == 0) {
            w.joins[run].first = -1;
            w.joins[run].beyond = -1;
        }
        if (run >= runs) return;
    }
    if (Whole && threadIdx.x == 0) s.beyond = 0;
    int64_t gi, u, end;                             // group; unit of the whole row, and where the run ends
    int64_t units, head, v;                         // the group's units for a head, the head, unit within it
    if (Whole) {
        gi = run / heads;
        head = run - gi * heads;
        units = units_of<Beams>(a, w, gi);
        v = 0;
        u = 0;
        end = units;
    } else {
        u = total * run / runs;
        end = total * (run + 1) / runs;
        const int64_t at = u / heads;
        if (at >= before && at < before + mine) {
            int64_t k = g0, from = before, n;
            while (k + 1 < w.groups && at >= from + (n = units_of<Beams>(a, w, k))) from += n, ++k;
            s.at_group = k;
            s.at_units = from;
        }
        __syncthreads();
        gi = s.at_group;
        units = units_of<Beams>(a, w, gi);
        const int64_t rest = u - s.at_units * heads;
        head = rest / units;
        v = rest - head * units;
        if (threadIdx.x == 0) w.joins[run].whole = gi * heads + head + (v > 0);
    }
    while (u < end) {
        const Group grp = Beams ? group_at(a, w, gi) : Group{gi, 1};
        const int kv = static_cast<int>(head / w.parts), part = static_cast<int>(head - static_cast<int64_t>(kv) * w.parts);
        const int cols = columns_of(w, grp, part);
        const int64_t head_at = static_cast<int64_t>(kv) * a.page * a.d;
        const Column col = column_of(w, grp, kv, part, x);

        Queries<NC> q;
        const T* row = static_cast<const T*>(a.Q) + col.seq * a.ldq + static_cast<int64_t>(col.head) * a.d;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int f = 32 * c + 8 * g;
            q.q[c] = x < cols && f < a.d ? *reinterpret_cast<const v4u*>(row + f) : v4u{0, 0, 0, 0};
        }
        q.scale = a.scale * kLog2e;
        q.bias = a.slopes && x < cols ? a.slopes[col.head] * kLog2e : 0.0f;
        q.last = (Beams && x >= cols ? 0 : clamped_len(a, Beams ? col.seq : gi)) - 1;

        Sums<EL> sum;
        sum.m = -INFINITY;
        sum.l = 0.0f;
#pragma unroll
        for (int e = 0; e < EL; ++e) sum.o[e] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

        // tiles t .. stop of sequence `seq`, for all columns or for those that are `mine`
        const auto pass = [&](auto alone, int64_t seq, int t, int stop, int len, bool mine) {
            constexpr bool kAlone = decltype(alone)::value;
            int ids = -1, base = t - kWave;
            const auto fetch = [&](Step<NC, EL>& st, int tile) {
                if (tile - base >= kWave / 2) {          // the next 32 tiles' pages, two a lane pair
                    base = tile;
                    const int key = ((tile + (lane >> 1)) * kWaves + wave) * kStep + (lane & 1) * kHalf;
                    ids = key < len && key >= 0 ? a.tables[seq * a.ldt + key / a.page] : -1;
                    if (ids >= a.n_pages) ids = -1;
                }
                st.key = (tile * kWaves + wave) * kStep;
#pragma unroll
                for (int h = 0; h < 2; ++h) st.id[h] = __builtin_amdgcn_readlane(ids, 2 * (tile - base) + h);
                load_step<T, NC, EL, Full>(st, a, head_at, lane);
            };
            for (; t < stop; ++t) {
                Step<NC, EL> st;
                fetch(st, t);
                add_step<T, NC, EL, kAlone>(sum, st, q, len - 1, mine, lane);
            }
        };
        const int64_t v1 = units - v < end - u ? units : v + (end - u);
        if (!Beams) {
            const int len = clamped_len(a, gi);
            const int tiles = tiles_of(len);
            pass(std::false_type{}, gi, static_cast<int>(v), static_cast<int>(v1 < tiles ? v1 : tiles), len, true);
        } else {
            const int shared = w.shared[gi];
            if (v < shared)
                pass(std::false_type{}, grp.first, static_cast<int>(v), static_cast<int>(v1 < shared ? v1 : shared),
                     clamped_len(a, grp.first), true);
            int64_t from = shared;
            for (int b = 0; b < grp.n; ++b) {
                const int len = clamped_len(a, grp.first + b);
                const int own = tiles_of(len) > shared ? tiles_of(len) - shared : 0;
                const int64_t lo = v > from ? v : from, hi = v1 < from + own ? v1 : from + own;
                if (lo < hi)
                    pass(std::true_type{}, grp.first + b, static_cast<int>(lo - from) + shared, static_cast<int>(hi - from) + shared,
                         len, col.seq == grp.first + b && x < cols);
                from += own;
            }
        }

        if (Whole || v1 - v == units) {
            join_waves<NC, EL>(s, sum, cols, a.d, wave, lane, [&](int c, int i, float o, float m, float l) {
                if (!put<T>(a, column_of(w, grp, kv, part, c), i, o, m, l)) {
                    if (Whole) atomicOr(&s.beyond, 1u << c);
                    else w.joins[run].beyond = gi * heads + head;
                }
            });
            if (Whole) {
                for (unsigned beyond = s.beyond; beyond; beyond &= beyond - 1) {
                    const Column c = column_of(w, grp, kv, part, __builtin_ctz(beyond));
                    attend_again<T>(a, s.again, c.seq, c.head);
                }
                return;
            }
        } else {
            const int64_t slot = (run * 2 + (v == 0)) * w.cols;
            join_waves<NC, EL>(s, sum, cols, a.d, wave, lane, [&](int c, int i, float o, float m, float l) {
                w.o[(slot + c) * a.d + i] = o;
                if (i == 0) {
                    w.ml[(slot + c) * 2] = m;
                    w.ml[(slot + c) * 2 + 1] = l;
                }
            });
            if (v > 0 && v1 == units && threadIdx.x == 0) {
                // the run with the first unit, u - v: the last one that starts at or before it
                w.joins[run].group = gi;
                w.joins[run].head = static_cast<int>(head);
                w.joins[run].first = static_cast<int>(((u - v + 1) * runs - 1) / total);
            }
        }
        u += v1 - v;
        v = 0;
        if (++head == heads) {
            head = 0;
            ++gi;
            if (u < end) units = units_of<Beams>(a, w, gi);
        }
    }
}

// The partial sums of one (group, head): the first run's second ones, and the others'
// first ones, kJoinCols columns a block. Every 16 bytes of the result are summed by one
// thread, or, where there are fewer of them than threads, by several that take the runs
// in turn, kJoinAhead of each on their way at once; the runs' weights lie in shared
// memory. One sequence of 12274 tokens, 64 heads on 4: 13.5 us, and 26 with a load after
// the other and the weights taken where they are used; 64 x 96 heads of two parts at most
// 10, and 1 less so. 16 on their way take 13 in each.
constexpr int kJoinCols = 4;
constexpr int kJoinAhead = 8;
constexpr int kJoinRuns = 512;

template <typename T>
__device__ __forceinline__ void join_runs(const AttendArgs& a, const Split& w, const Split::Join& j, unsigned* beyond) {
    __shared__ float s_m[kJoinCols], s_l[kJoinCols], s_f[kJoinCols][kJoinRuns];
    __shared__ v4f s_o[kThreads];
    const Group grp = group_at(a, w, j.group);
    const int kv = j.head / w.parts, part = j.head - kv * w.parts, cols = columns_of(w, grp, part);
    const int n = static_cast<int>(blockIdx.x) - j.first + 1;
    const int col0 = static_cast<int>(blockIdx.y) * kJoinCols, mine = cols - col0 < kJoinCols ? cols - col0 : kJoinCols;
    if (mine <= 0) return;
    const auto row = [&](int b, int c) { return (static_cast<int64_t>(j.first + b) * 2 + (b == 0)) * w.cols + col0 + c; };
    // of a run without a maximum: nothing if it has seen nothing, all (a NaN) otherwise
    const auto weight = [&](float m, float l, float most) {
        return m == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : __builtin_amdgcn_exp2f(m - most);
    };
    const int lane = threadIdx.x & 63;
    for (int c = threadIdx.x >> 6; c < mine; c += kWaves) {
        float m = -INFINITY, l = 0.0f;
        for (int b = lane; b < n; b += kWave) m = fmaxf(m, w.ml[row(b, c) * 2]);
        m = wave_max(m);
        for (int b = lane; b < n; b += kWave) {
            const float* p = w.ml + row(b, c) * 2;
            const float f = weight(p[0], p[1], m);
            l += p[1] * f;
            if (b < kJoinRuns) s_f[c][b] = f;
        }
        l = wave_sum(l);
        if (lane == 0) {
            s_m[c] = m;
            s_l[c] = l;
        }
    }
    __syncthreads();
    static_assert(kJoinCols * I8MM_CACHE_MAX_HEAD / 4 <= kThreads, "a thread for each 16 bytes of the result");
    const int quads = a.d / 4, all = mine * quads, sharers = kThreads / all;
    const int by = static_cast<int>(threadIdx.x) / all, k = static_cast<int>(threadIdx.x) - by * all;
    const int c = k / quads, i = 4 * (k - c * quads);
    v4f o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int b0 = 0; b0 < n; b0 += kJoinRuns) {
        const int count = n - b0 < kJoinRuns ? n - b0 : kJoinRuns;
        if (b0 > 0) {
            __syncthreads();
            for (int x = threadIdx.x; x < mine * kJoinRuns; x += kThreads) {
                const int xc = x / kJoinRuns, b = x - xc * kJoinRuns;
                if (b >= count) continue;
                const float* p = w.ml + row(b0 + b, xc) * 2;
                s_f[xc][b] = weight(p[0], p[1], s_m[xc]);
            }
            __syncthreads();
        }
        for (int b1 = by; by < sharers && b1 < count; b1 += kJoinAhead * sharers) {
            v4f part_o[kJoinAhead];
#pragma unroll
            for (int q = 0; q < kJoinAhead; ++q) {
                const int b = b1 + q * sharers;
                if (b < count) part_o[q] = *reinterpret_cast<const v4f*>(w.o + row(b0 + b, c) * a.d + i);
            }
#pragma unroll
            for (int q = 0; q < kJoinAhead; ++q)
                if (b1 + q * sharers < count) o += part_o[q] * s_f[c][b1 + q * sharers];
        }
    }
    if (sharers > 1) {
        s_o[threadIdx.x] = o;
        __syncthreads();
        if (by == 0)
            for (int b = 1; b < sharers; ++b) o += s_o[b * all + k];
    }
    if (by == 0) {
        const Column col = column_of(w, grp, kv, part, col0 + c);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (!put<T>(a, col, i + e, o[e], s_m[c], s_l[c])) atomicOr(beyond, 1u << (col0 + c));
    }
}

// And what is not finite is computed again: of the columns that the block joined, and (by
// the first block of a run) of the (group, head)s that the run wrote whole.
template <typename T>
__global__ __launch_bounds__(kThreads, 4) void k_attend_join(const AttendArgs a, const Split w) {
    __shared__ Again s_again;
    __shared__ unsigned s_beyond;
    const Split::Join j = w.joins[blockIdx.x];
    const int heads = a.kv_heads * w.parts;
    const int64_t last = blockIdx.y == 0 ? j.beyond : -1;
    int64_t next = last >= 0 ? j.whole : 0;
    if (j.first < 0 && last < 0) return;
    if (threadIdx.x == 0) s_beyond = 0;
    bool joined = j.first >= 0;
    if (joined) join_runs<T>(a, w, j, &s_beyond);
    __syncthreads();
    if (last < 0 && s_beyond == 0) return;           // as nearly always
#pragma unroll 1
    for (int64_t at = joined ? j.group * heads + j.head : next++; ; at = next++) {
        const int64_t gi = at / heads;
        const int head = static_cast<int>(at - gi * heads), kv = head / w.parts, part = head - kv * w.parts;
        const Group grp = group_at(a, w, gi);
        for (int k = threadIdx.x; !joined && k < columns_of(w, grp, part) * a.d; k += kThreads) {
            const int c = k / a.d;
            const Column col = column_of(w, grp, kv, part, c);
            const T v = static_cast<const T*>(a.out)[col.seq * a.ldo + static_cast<int64_t>(col.head) * a.d + (k - c * a.d)];
            if (!finite(static_cast<float>(v))) atomicOr(&s_beyond, 1u << c);
        }
        joined = false;
        __syncthreads();
        for (unsigned beyond = s_beyond; beyond; beyond &= beyond - 1) {
            const Column col = column_of(w, grp, kv, part, __builtin_ctz(beyond));
            attend_again<T>(a, s_again, col.seq, col.head);
        }
        if (next > last) return;
        __syncthreads();
        if (threadIdx.x == 0) s_beyond = 0;
        __syncthreads();
    }
}

// Rows of partial sums that the workspace holds: a run leaves two of each of its columns.
constexpr int kSumRows = 32768;

// Rounds of runs that a launch has blocks for: as many as the workspace holds the
// sums of, and as the tiles could ask for if every sequence filled its table.
int most_rounds(int cols, int blocks, int64_t tiles) {
    const int64_t room = kSumRows / (2 * cols * blocks), asked = tiles / (static_cast<int64_t>(blocks) * kRunTiles);
    const int64_t r = asked < room ? asked : room;
    return r < 1 ? 1 : r < 8 ? static_cast<int>(r) : 8;
}

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

template <typename T, int NC, int EL, bool Full>
hipError_t attend_with(const AttendArgs& a, Split w, void* workspace, hipStream_t stream) {
    w.group = a.heads / a.kv_heads;
    w.parts = (w.group + kCols - 1) / kCols;
    const int heads = a.kv_heads * w.parts;
    if (attention_takes_whole(static_cast<int64_t>(a.max_pages) * a.page, a.beams)) {
        w.groups = a.n;
        w.gb = w.chunks = 1;
        AttendArgs one = a;
        one.beams = 1;
        // in runs of blocks that one grid has threads for
        const int64_t items = a.n * heads;
        return for_row_runs(items, kGridThreads / kThreads, [&](int64_t first, int64_t count) {
            k_attend<T, NC, EL, Full, false, true><<<static_cast<unsigned>(count), kThreads, 0, stream>>>(one, w, first);
            return hipGetLastError();
        });
    }
    w.gb = w.parts > 1 ? 1 : kCols / w.group < a.beams ? kCols / w.group : a.beams;
    w.chunks = (a.beams + w.gb - 1) / w.gb;
    w.groups = a.n / a.beams * w.chunks;
    w.cols = w.parts > 1 ? kCols : w.gb * w.group;
    w.rounds = most_rounds(w.cols, kBlocks<EL>, a.n * heads * ((static_cast<int64_t>(a.max_pages) * a.page + kTile - 1) / kTile));
    char* at = static_cast<char*>(workspace);
    w.o = reinterpret_cast<float*>(at);
    w.ml = reinterpret_cast<float*>(at += round256(static_cast<int64_t>(kSumRows) * a.d * 4));
    w.joins = reinterpret_cast<Split::Join*>(at += round256(static_cast<int64_t>(kSumRows) * 2 * 4));
    at += round256(kSumRows / 2 * sizeof(Split::Join));
    if (w.gb > 1) {
        int32_t* shared = reinterpret_cast<int32_t*>(at);
        w.shared = shared;
        const int64_t blocks = (w.groups + kWaves - 1) / kWaves;
        k_attend_shared<<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), kThreads, 0, stream>>>(a, w, shared);
        k_attend<T, NC, EL, Full, true, false><<<kBlocks<EL> * w.rounds, kThreads, 0, stream>>>(a, w, 0);
    } else {
        k_attend<T, NC, EL, Full, false, false><<<kBlocks<EL> * w.rounds, kThreads, 0, stream>>>(a, w, 0);
    }
    k_attend_join<T><<<dim3(kBlocks<EL> * w.rounds, (w.cols + kJoinCols - 1) / kJoinCols), kThreads, 0, stream>>>(a, w);
    return hipGetLastError();
}

template <typename T, int NC, int EL>
hipError_t attend(const AttendArgs& a, void* workspace, hipStream_t stream) {
    return a.d == 32 * NC && a.d == 16 * EL ? attend_with<T, NC, EL, true>(a, {}, workspace, stream)
                                            : attend_with<T, NC, EL, false>(a, {}, workspace, stream);
}

template <typename T>
hipError_t attend_type(const AttendArgs& a, void* workspace, hipStream_t stream) {
    if (a.d <= 64) return attend<T, 2, 4>(a, workspace, stream);
    if (a.d <= 96) return attend<T, 3, 8>(a, workspace, stream);
    if (a.d <= 128) return attend<T, 4, 8>(a, workspace, stream);
    return attend<T, 8, 16>(a, workspace, stream);
}

}  // namespace

// Up to so many keys a block takes whole (group, head)s. At 1000 keys: 12 heads of 128
// sequences 123 us so and 130 split and joined, 32 heads of 16 43 and 48; 32, 12 or one
// head of one sequence 14 and 12 on the GPU, but a call 14 and 15 to 16, as it launches one
// kernel less. At 2048 96 heads of 64 993 and 982, and with lengths that differ 532 and 515.
// Beams that share pages gain by the split path's groups, so they take it earlier.
bool attention_takes_whole(int64_t keys, int64_t beams) { return keys * (beams > 1 ? 2 : 1) <= I8MM_ATTENTION_WHOLE_KEYS; }

size_t decode_attention_scratch(int64_t n, int, int, int d) {
    return static_cast<size_t>(round256(static_cast<int64_t>(kSumRows) * d * 4) + round256(static_cast<int64_t>(kSumRows) * 2 * 4) +
                               round256(kSumRows / 2 * sizeof(Split::Join)) + round256(4 * n) + 256);
}

hipError_t launch_decode_attention(const AttendArgs& a, void* workspace, hipStream_t stream) {
    if (a.n == 0) return hipSuccess;
    return a.type == Dtype::F16 ? attend_type<_Float16>(a, workspace, stream) : attend_type<__bf16>(a, workspace, stream);
}

}  // namespace i8mm
