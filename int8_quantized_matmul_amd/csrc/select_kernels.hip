// Beam search's selection: of all continuations (beam i, token v) of a request
// the k best by
//   t = score_i + x_iv - lse_i,  lse_i = log sum_v exp(x_iv),
// ties to the lowest (beam, token).
//
// The logits are read once. A wavefront takes a part of a row and holds, in
// each lane, a running maximum and sum of exponentials, and, one a lane, the
// part's k best so far in order (within a row the logits alone order the
// tokens). What is not above the last of them costs a comparison; what is, is
// kept until there is more of it, then sorted over the lanes and merged with
// them. A second launch joins a request's parts: the sums in fp64, then the k
// best of the parts' candidates. A few at a time are put in their places one
// after the other, by a shift of the lanes behind.

#include "../../include/i8mm.h"
#include "launch.h"

#include "adapt_common.h"

#include <type_traits>

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

template <typename V>
__device__ __forceinline__ V least() {
    if constexpr (sizeof(V) == 8) return minus_infinity();
    else return -INFINITY;
}

// The value of lane xor J: lane permutes within 16, swaps of rows beyond.
template <int J>
__device__ __forceinline__ unsigned other_bits(unsigned v, int lane) {
    if constexpr (J == 1) return __builtin_amdgcn_update_dpp(0, v, 0xb1, 0xf, 0xf, true);
    else if constexpr (J == 2) return __builtin_amdgcn_update_dpp(0, v, 0x4e, 0xf, 0xf, true);
    else if constexpr (J == 4)
        return __builtin_amdgcn_update_dpp(0, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, true), 0x1b, 0xf, 0xf, true);
    else if constexpr (J == 8) return __builtin_amdgcn_update_dpp(0, v, 0x128, 0xf, 0xf, true);
    else if constexpr (J == 16) {
        const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return lane & 16 ? p[0] : p[1];
    } else {
        const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return lane & 32 ? p[0] : p[1];
    }
}
template <int J>
__device__ __forceinline__ int other(int v, int lane) { return static_cast<int>(other_bits<J>(static_cast<unsigned>(v), lane)); }
template <int J>
__device__ __forceinline__ float other(float v, int lane) {
    return __builtin_bit_cast(float, other_bits<J>(__builtin_bit_cast(unsigned, v), lane));
}
template <int J>
__device__ __forceinline__ double other(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = other_bits<J>(static_cast<unsigned>(b), lane), hi = other_bits<J>(static_cast<unsigned>(b >> 32), lane);
    return __builtin_bit_cast(double, hi << 32 | lo);
}

// The value of the lane before (lane 0: its own).
__device__ __forceinline__ int previous(int v) { return __builtin_amdgcn_update_dpp(v, v, 0x138, 0xf, 0xf, false); }
__device__ __forceinline__ float previous(float v) { return __builtin_bit_cast(float, previous(__builtin_bit_cast(int, v))); }
__device__ __forceinline__ double previous(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = static_cast<uint32_t>(previous(static_cast<int>(b))), hi = static_cast<uint32_t>(previous(static_cast<int>(b >> 32)));
    return __builtin_bit_cast(double, hi << 32 | lo);
}

// One step of a bitonic sort: of lanes l and l xor J the better pair goes to the lower
// one, where `down`, else to the higher.
template <int J, typename V>
__device__ __forceinline__ void exchange(V& v, int& i, bool down, int lane) {
    const V ov = other<J>(v, lane);
    const int oi = other<J>(i, lane);
    const bool mine = (v > ov) | ((v == ov) & (i < oi)), low = (lane & J) == 0;
    if (mine != (low == down)) {
        v = ov;
        i = oi;
    }
}
template <int J, typename V>
__device__ __forceinline__ void bitonic_merge(V& v, int& i, bool down, int lane) {
    exchange<J>(v, i, down, lane);
    if constexpr (J > 1) bitonic_merge<J / 2>(v, i, down, lane);
}
// The wavefront's pairs in order, the best in lane 0.
template <int N = kWave, typename V>
__device__ __forceinline__ void sort_lanes(V& v, int& i, int lane) {
    if constexpr (N > 2) sort_lanes<N / 2>(v, i, lane);
    bitonic_merge<N / 2>(v, i, (lane & N) == 0, lane);
}

// The wavefront's values in order, the largest in lane 0.
template <int J>
__device__ __forceinline__ void value_merge(float& v, bool down, int lane) {
    const float o = other<J>(v, lane);
    v = ((lane & J) == 0) == down ? fmaxf(v, o) : fminf(v, o);
    if constexpr (J > 1) value_merge<J / 2>(v, down, lane);
}
template <int N = kWave>
__device__ __forceinline__ void sort_values(float& v, int lane) {
    if constexpr (N > 2) sort_values<N / 2>(v, lane);
    value_merge<N / 2>(v, (lane & N) == 0, lane);
}

// The k <= 64 best (value, index) pairs seen by a wavefront, lane i the i-th.
template <typename V>
struct Best {
    V value = least<V>();
    int index = kNone;
    V last = least<V>();                         // the k-th
    int last_index = kNone;

    __device__ __forceinline__ bool wants(V v, int i) const { return (v > last) | ((v == last) & (i < last_index)); }
    __device__ __forceinline__ void note_last(int k) {
        last = lane_value(value, k - 1);
        last_index = __builtin_amdgcn_readlane(index, k - 1);
    }
    // Behind the better ones; the others move up a lane. (note_last() is still to be called.)
    __device__ __forceinline__ void insert(V v, int i, int lane) {
        const int at = __builtin_popcountll(__ballot((value > v) | ((value == v) & (index < i))));
        const V up = previous(value);
        const int up_index = previous(index);
        value = lane > at ? up : lane == at ? v : value;
        index = lane > at ? up_index : lane == at ? i : index;
    }
    // A list in order, the i-th best in lane 63 - i: the better of each lane's two are
    // the 64 best, falling and rising, which a bitonic merge puts in order.
    __device__ __forceinline__ void merge_reversed(V v, int i, int k, int lane) {
        if ((v > value) | ((v == value) & (i < index))) {
            value = v;
            index = i;
        }
        bitonic_merge<kWave / 2>(value, index, true, lane);
        note_last(k);
    }
    // The lanes of `left` offer one pair each, which are put in one after the other.
    __device__ __forceinline__ void offer_few(V v, int i, uint64_t left, int k, int lane) {
        for (left &= __ballot(wants(v, i)); left; left &= left - 1) {
            const int from = __builtin_ctzll(left);
            insert(lane_value(v, from), __builtin_amdgcn_readlane(i, from), lane);
        }
        note_last(k);
    }
    // The same where they may be many: those are sorted and merged.
    __device__ __forceinline__ void offer(V v, int i, uint64_t left, int k, int lane) {
        if (__builtin_popcountll(left) > 8) {
            const bool real = left >> lane & 1;
            V sv = real ? v : least<V>();
            int si = real ? i : kNone;
            sort_lanes(sv, si, lane);
            merge_reversed(__shfl(sv, kWave - 1 - lane, kWave), __shfl(si, kWave - 1 - lane, kWave), k, lane);
        } else {
            offer_few(v, i, left, k, lane);
        }
    }
};

// The next fp32 number above v (v itself if there is none).
__device__ __forceinline__ float above(float v) {
    const int b = __builtin_bit_cast(int, v);
    const int up = v == 0.0f ? 1 : b < 0 ? b - 1 : b + (v < INFINITY);
    return __builtin_bit_cast(float, up);
}

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

constexpr int kHeld = 32;                        // tokens that wait before they are put in order
static_assert(kHeld <= kWave, "the room in k_select_scan");

// Part of a row, a quarter of it a wavefront: a running maximum and sum of
// exponentials, and the k largest logits. Tokens that are not below the bar wait in
// shared memory until there are kHeld of them, which are sorted over the lanes and
// merged with the k best; the first bar is the k-th of the lanes' largest of the first
// steps. A wavefront takes `Steps` steps of 512 tokens at once. 64 x 8 beams over 50272
// tokens in fp32 (103 MB): k = 16 in 29.5 us with two steps, 30.5 with one, 39 with
// three (of registers fewer wavefronts are left), 35 if each token is put in its place
// when it is met; k = 64 in 42 instead of 75 so, rows that rise 87 instead of 131. 19
// without the selection, which is what memory takes.
template <typename T, int Steps>
__global__ __launch_bounds__(kThreads) void k_select_scan(const SelectArgs a, const SelectScratch w, int parts, int quarter) {
    __shared__ float s_value[kWaves][kWave], s_m[kWaves], s_l[kWaves];
    __shared__ volatile float s_floor[kWaves];   // the k-th best of each wavefront so far: what lies below is not wanted
    __shared__ int s_index[kWaves][kWave];
    // wanted tokens of each wavefront, not yet put in: fewer than kWave from before, and a step's
    __shared__ float s_wanted[kWaves][kWave + Steps * kStep];
    __shared__ int s_token[kWaves][kWave + Steps * kStep];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t items = a.n * a.beams * parts;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t row = item / parts;
        const int part = static_cast<int>(item - row * parts);
        const T* x = static_cast<const T*>(a.logits) + row * a.ld;
        const int64_t first = (static_cast<int64_t>(part) * kWaves + wave) * quarter;
        const int from = static_cast<int>(first < a.vocab ? first : a.vocab);
        const int to = a.vocab - from < quarter ? a.vocab : from + quarter;
        if (lane == 0) s_floor[wave] = -INFINITY;
        __syncthreads();
        Best<float> best;
        int held = 0;
        float bar = -INFINITY;                   // what is below it is not wanted
        float m = -INFINITY, l = 0.0f;
        Eight<T> next[Steps];
#pragma unroll
        for (int q = 0; q < Steps; ++q) next[q].load(x + from + q * kStep + 8 * lane, to - from - q * kStep - 8 * lane);
        for (int v0 = from; v0 < to; v0 += Steps * kStep) {
            const int v = v0 + 8 * lane;
            float f[Steps][8];
            float most = -INFINITY;
#pragma unroll
            for (int q = 0; q < Steps; ++q)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    f[q][i] = v + q * kStep + i < to ? next[q].at(i) : -INFINITY;
                    most = fmaxf(most, f[q][i]);
                }
            const int v1 = v + Steps * kStep;
            if (v0 + Steps * kStep < to) {
#pragma unroll
                for (int q = 0; q < Steps; ++q) next[q].load(x + v1 + q * kStep, to - v1 - q * kStep);
            }
            const float up = fmaxf(m, most);
            const float off = up == -INFINITY ? 0.0f : up;
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < Steps; ++q)
#pragma unroll
                for (int i = 0; i < 8; ++i) s += __builtin_amdgcn_exp2f((f[q][i] - off) * kLog2e);
            l = __builtin_fmaf(l, m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - off) * kLog2e), s);
            m = up;
            if (v0 == from) {
                // at first, nothing below the k-th of the lanes' largest
                float sorted = most;
                sort_values(sorted, lane);
                bar = lane_float(sorted, a.k - 1);
                if (lane == 0) s_floor[wave] = bar;
            }
            bar = fmaxf(bar, fmaxf(fmaxf(s_floor[0], s_floor[1]), fmaxf(s_floor[2], s_floor[3])));
            if (__any(most >= bar)) {
#pragma unroll
                for (int q = 0; q < Steps; ++q)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const bool wanted = (f[q][i] >= bar) & (v + q * kStep + i < to);
                        const uint64_t left = __ballot(wanted);
                        if (left) {
                            const int at = held + __builtin_amdgcn_mbcnt_hi(left >> 32, __builtin_amdgcn_mbcnt_lo(left, 0));
                            if (wanted) {
                                s_wanted[wave][at] = f[q][i];
                                s_token[wave][at] = v + q * kStep + i;
                            }
                            held += __builtin_popcountll(left);
                        }
                    }
            }
            if (held >= kHeld || (v0 + Steps * kStep >= to && held > 0)) {
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                for (int c = 0; c < held; c += kWave) {
                    const bool real = c + lane < held;
                    const float fv = real ? s_wanted[wave][c + lane] : -INFINITY;
                    const int fi = real ? s_token[wave][c + lane] : kNone;
                    const uint64_t left = __ballot(real & best.wants(fv, fi));
                    if (left) best.offer(fv, fi, left, a.k, lane);
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                held = 0;
                // of what this one has k of, nothing up to the k-th (a later token loses a tie)
                if (best.last_index != kNone) {
                    bar = fmaxf(bar, above(best.last));
                    if (lane == 0) s_floor[wave] = best.last;
                }
            }
        }
        const float top = wave_max_f(m);
        l = wave_sum(m == -INFINITY ? l : l * __builtin_amdgcn_exp2f((m - top) * kLog2e));
        if (lane == 0) {
            s_m[wave] = top;
            s_l[wave] = l;
        }
        s_value[wave][lane] = best.value;
        s_index[wave][lane] = best.index;
        __syncthreads();
        if (wave == 0) {
            float all = s_m[0], sum = 0.0f;
#pragma unroll
            for (int o = 1; o < kWaves; ++o) {
                all = fmaxf(all, s_m[o]);
                best.merge_reversed(s_value[o][kWave - 1 - lane], s_index[o][kWave - 1 - lane], a.k, lane);
            }
#pragma unroll
            for (int o = 0; o < kWaves; ++o)
                sum += s_m[o] == -INFINITY ? s_l[o] : s_l[o] * __builtin_amdgcn_exp2f((s_m[o] - all) * kLog2e);
            if (lane == 0) {
                w.most[item] = all;
                w.sum[item] = sum;
            }
            if (lane < a.k) {
                w.value[item * a.k + lane] = best.value;
                w.token[item * a.k + lane] = best.index;
            }
        }
        __syncthreads();
    }
}

// A block a request: the sums of its rows, the candidates of all their parts, the chosen
// ones' histories. One wait after another bounds it: 12 us for 64 requests of 8 beams, k
// = 16 and histories of 700 tokens, 8 for one request of 4 beams in 25 parts each; 19 for
// one of 7872 candidates, k = 64 (22 if each is loaded when it is looked at).
__global__ __launch_bounds__(kThreads) void k_select_join(const SelectArgs a, const SelectScratch w, int parts) {
    __shared__ double s_value[kWaves][kWave];
    __shared__ int s_index[kWaves][kWave];
    static_assert(I8MM_BEAM_MAX * 4 <= kThreads && I8MM_BEAM_MAX <= kWave, "four lanes a beam, a lane a continuation");
    __shared__ double s_lse[kWave];              // of each beam; NaN: the beam leaves nothing
    __shared__ double s_score[kWave];
    __shared__ int s_parent[kWave];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t b = blockIdx.x; b < a.n; b += gridDim.x) {
        const int64_t row0 = b * a.beams;
        const int each = parts * a.k, all = a.beams * each, lists = a.beams * parts;
        const float* value = w.value + row0 * each;
        const int32_t* token = w.token + row0 * each;
        // a candidate's place: the lists' first ones come first, so that few of the others are put in
        const auto place = [&](int c) { return c % lists * a.k + c / lists; };
        float x = 0.0f;                          // a lane's candidate, on its way while the one before is looked at
        int v = kNone;
        const auto fetch = [&](int c) {
            x = c < all ? value[place(c)] : 0.0f;
            v = c < all ? token[place(c)] : kNone;
        };
        fetch(wave * kWave + lane);
        {
            // as many lanes a beam as there are, up to a wavefront
            const int lanes = a.beams <= 4 ? 64 : a.beams <= 8 ? 32 : a.beams <= 16 ? 16 : a.beams <= 32 ? 8 : 4;
            const int i = threadIdx.x / lanes, p0 = threadIdx.x & (lanes - 1);
            const bool there = i < a.beams;
            const float* most = w.most + (row0 + (there ? i : 0)) * parts;
            const float* sum = w.sum + (row0 + (there ? i : 0)) * parts;
            float top = -INFINITY;
            for (int p = p0; p < parts; p += lanes) top = fmaxf(top, most[p]);
            for (int off = lanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
            double l = 0.0;
            for (int p = p0; p < parts; p += lanes)
                l += sum[p] * (most[p] == -INFINITY ? 0.0 : exp(static_cast<double>(most[p]) - top));
            for (int off = lanes / 2; off > 0; off >>= 1) l += __shfl_xor(l, off, kWave);
            if (there && p0 == 0) {
                const double lse = top + log(l), score = a.scores[row0 + i];
                s_lse[i] = (lse - lse) + (score - score) == 0.0 ? lse : NAN;
                s_score[i] = score;
            }
        }
        __syncthreads();
        Best<double> best;
        for (int c0 = wave * kWave; c0 < all; c0 += kThreads) {
            const int c = c0 + lane, beam = c % lists / parts;
            const double none = minus_infinity();
            double t = none;
            int at = kNone;
            if (c < all) {
                const double lse = s_lse[beam];
                if (lse == lse) {
                    t = s_score[beam] + (x - lse);
                    at = v == kNone ? kNone : beam * a.vocab + v;
                } else if (c % lists == beam * parts && c / lists < a.vocab) {
                    // nothing to choose by: the lowest tokens, with no weight
                    at = beam * a.vocab + c / lists;
                }
            }
            if (c0 + kThreads < all) fetch(c + kThreads);
            const uint64_t left = __ballot((at != kNone) & best.wants(t, at));
            if (left) best.offer(t, at, left, a.k, lane);
        }
        s_value[wave][lane] = best.value;
        s_index[wave][lane] = best.index;
        __syncthreads();
        if (wave == 0) {
            for (int o = 1; o < kWaves; ++o)
                best.merge_reversed(s_value[o][kWave - 1 - lane], s_index[o][kWave - 1 - lane], a.k, lane);
            if (lane < a.k) {
                // (in range whatever the workspace holds, should calls that overlap share one)
                const unsigned rank = static_cast<unsigned>(best.index) / static_cast<unsigned>(a.vocab);
                const int beam = rank < static_cast<unsigned>(a.beams) ? static_cast<int>(rank) : a.beams - 1;
                const int v = best.index - beam * a.vocab;
                a.scores_out[b * a.k + lane] = static_cast<float>(best.value);
                a.parents[b * a.k + lane] = static_cast<int>(row0 + beam);
                a.tokens[b * a.k + lane] = v;
                s_parent[lane] = beam;
                if (a.history_out) a.history_out[(b * a.k + lane) * a.ldho + a.T] = v;
            }
        }
        __syncthreads();
        if (a.history_out) {
            // four tokens a thread and kEach times that in flight
            constexpr int kEach = 8;
            const int64_t quads = (a.T + 3) / 4, pieces = quads * a.k;
            for (int64_t p0 = threadIdx.x; p0 < pieces; p0 += kEach * kThreads) {
                v4i t[kEach];
                int32_t* to[kEach];
                int n[kEach];
#pragma unroll
                for (int q = 0; q < kEach; ++q) {
                    const int64_t p = p0 + q * kThreads;
                    n[q] = 0;
                    if (p >= pieces) continue;
                    const int i = static_cast<int>(p / quads);
                    const int64_t at = 4 * (p - i * quads);
                    const int32_t* in = a.history + (row0 + s_parent[i]) * a.ldh + at;
                    to[q] = a.history_out + (b * a.k + i) * a.ldho + at;
                    n[q] = a.T - at < 4 ? static_cast<int>(a.T - at) : 4;
                    if (n[q] == 4) {
                        __builtin_memcpy(&t[q], in, 16);
                    } else {
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            if (e < n[q]) t[q][e] = in[e];
                    }
                }
#pragma unroll
                for (int q = 0; q < kEach; ++q) {
                    if (n[q] == 4) {
                        __builtin_memcpy(to[q], &t[q], 16);
                    } else {
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            if (e < n[q]) to[q][e] = t[q][e];
                    }
                }
            }
        }
        __syncthreads();
    }
}

// Parts of a row: as many as fill the chip with four blocks a CU, of a step a wavefront
// at least.
int parts_of(int64_t rows, int vocab) {
    const int64_t fill = 1024 / (rows < 1 ? 1 : rows < 1024 ? rows : 1024), most = (vocab + kWaves * kStep - 1) / (kWaves * kStep);
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
    const int64_t steps = static_cast<int64_t>(parts) * kWaves * kStep;
    const int quarter = static_cast<int>((a.vocab + steps - 1) / steps * kStep);
    const int64_t lists = rows * parts;
    char* at = static_cast<char*>(workspace);
    SelectScratch w;
    w.most = reinterpret_cast<float*>(at);
    w.sum = reinterpret_cast<float*>(at += round256(4 * lists));
    w.value = reinterpret_cast<float*>(at += round256(4 * lists));
    w.token = reinterpret_cast<int32_t*>(at + round256(4 * lists * a.k));
    const unsigned grid = static_cast<unsigned>(lists < 65536 ? lists : 65536);
    // a wavefront with a step or two takes them one at a time
    const auto scan = [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        if (quarter <= 2 * kStep) k_select_scan<T, 1><<<grid, kThreads, 0, stream>>>(a, w, parts, quarter);
        else k_select_scan<T, 2><<<grid, kThreads, 0, stream>>>(a, w, parts, quarter);
    };
    if (a.type == Dtype::F16) scan(static_cast<_Float16*>(nullptr));
    else if (a.type == Dtype::BF16) scan(static_cast<__bf16*>(nullptr));
    else scan(static_cast<float*>(nullptr));
    k_select_join<<<static_cast<unsigned>(a.n < 65536 ? a.n : 65536), kThreads, 0, stream>>>(a, w, parts);
    return hipGetLastError();
}

}  // namespace i8mm
