// Low-rank adapters of many requests beside one shared projection.
//
// Token i carries the adapter ids[i] = g of its request, or none (any value
// outside [0, G)). With A [G, r, h], B [G, r, o] and a factor per adapter:
//   T_i = X_i A_g^T,  Y_i = base_i + scale_g T_i B_g,
// and for gradients dY of Y:
//   dT_i = scale_g dY_i B_g^T,  dX_i = base_i + dT_i A_g,
//   dA_g = sum over the tokens of g of dT_i^T X_i,
//   dB_g = scale_g times the sum over the tokens of g of T_i^T dY_i.
// With both adapters' ranks in rows, these are three products:
//   dot   P_i = Z_i M_g^T           (T; dT without its factor)
//   add   out_i = base_i + f_g P_i M_g   (Y; dX)
//   grad  out_g = sum_i (f_g P_i)^T Z_i  (dA; dB)
// and each streams one large operand once against a small one.
//
// Precision. P (T, dT) is summed and kept in fp32. Where it meets 16-bit
// values in a matrix instruction it is carried as a sum of 16-bit parts,
// multiplied one after another into the same fp32 sum. fp16: two parts of 11
// bits, after an exact power of two has brought the largest finite one of the
// values that share it near 2^14 (in Y and dX a token's ranks share it, in dA
// and dB the tokens of a chunk, each rank for itself); a value is then off by
// at most 2^-23 of itself or 2^-39 of that largest one, whichever is more.
// bf16, which has fp32's range: two parts of 8 bits towards a 16-bit result,
// three towards an fp32 one. Y and dX are rounded once.

#include "launch.h"

#include "adapt_common.h"
#include "../../include/i8mm.h"

#include <type_traits>

namespace i8mm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kCus = 256;

// One 16x16x32 matrix instruction: lane l holds, for row (a) or column (b)
// l % 16, the eight products' factors k = l / 16 * 8 ..+7; the sum c of
// column l % 16 holds rows l / 16 * 4 ..+3.
__device__ __forceinline__ v4f mma(v8h a, v8h b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ v4f mma(v8b a, v8b b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

template <typename T>
using Vec = typename Eight<T>::vec;

template <typename T>
constexpr bool kScaled = std::is_same_v<T, _Float16>;

template <typename T>
__device__ __forceinline__ Vec<T> load16(const T* p) { return *reinterpret_cast<const Vec<T>*>(p); }

// Memory serves four neighbouring lanes at a time, at full rate only if they
// read neighbouring bytes, while the matrix instruction wants neighbouring
// rows in neighbouring lanes. So a row's four 16-byte pieces are read by lanes
// 4 row ..+3 and handed on: lane 16 piece + row takes lane 4 row + piece's.
// (Read where they are wanted, 16 rows of 64 bytes went at 16 bytes a clock
// and CU, a quarter of the rate.)
template <typename T>
__device__ __forceinline__ Vec<T> hand_on(const Vec<T>& v) {
    const int from = ((threadIdx.x & 15) * 4 + (threadIdx.x >> 4 & 3)) * 4;
    v4u in = __builtin_bit_cast(v4u, v), out;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        out[k] = static_cast<unsigned>(__builtin_amdgcn_ds_bpermute(from, static_cast<int>(in[k])));
    return __builtin_bit_cast(Vec<T>, out);
}

// rows[i][j] -> columns[j][i] of an 8 x 8 block of 16-bit elements
template <typename T>
__device__ __forceinline__ void transpose8(const Vec<T>(&rows)[8], Vec<T>(&columns)[8]) {
    v4u in[8], out[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) in[i] = __builtin_bit_cast(v4u, rows[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // byte selectors: the low (high) halves of the two words, the first in the low half
            out[2 * j][k] = __builtin_amdgcn_perm(in[2 * k + 1][j], in[2 * k][j], 0x05040100u);
            out[2 * j + 1][k] = __builtin_amdgcn_perm(in[2 * k + 1][j], in[2 * k][j], 0x07060302u);
        }
#pragma unroll
    for (int j = 0; j < 8; ++j) columns[j] = __builtin_bit_cast(Vec<T>, out[j]);
}

// The power of two that takes finite values up to `most` in magnitude near
// 2^14, as its exponent; 0 if there are none.
template <typename T>
__device__ __forceinline__ int scale_exponent(float most) {
    if constexpr (!kScaled<T>) return 0;
    return most > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(most) : 0;
}

// What a value counts for in the largest of those that share a power of two:
// infinity and NaN, which no power of two changes, count for nothing, so that
// they cost the finite values beside them no digits.
__device__ __forceinline__ float finite_size(float v) {
    const float size = fabsf(v);
    return size < __builtin_inff() ? size : 0.0f;
}

// v 2^ex as a sum of N parts of type T. What is not finite is its own first
// part; what T rounds to 0 is a first part of T's smallest number less as much
// in the second, so that a first part is 0 for 0 alone.
template <typename T, int N>
__device__ __forceinline__ void split(float v, int ex, T(&part)[N]) {
    const float whole = v;
    if constexpr (kScaled<T>) v = ldexpf(v, ex);
    const bool finite = fabsf(v) < __builtin_inff();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        part[k] = from_float<T>(v);
        if (!kScaled<T> && k == 0 && finite)             // not rounded up to infinity
            part[0] = from_float<T>(fminf(fmaxf(v, -0x1.fep127f), 0x1.fep127f));
        if (k == 0 && to_float<T>(part[0]) == 0.0f && whole != 0.0f)
            part[0] = __builtin_bit_cast(T, static_cast<uint16_t>(whole < 0.0f ? 0x8001 : 1));
        v = finite ? v - to_float<T>(part[k]) : 0.0f;
    }
}

// An infinity times a factor's first part is what the definition gives. Its
// products with the other parts, of either sign or 0, are not: they would make
// NaN of it. Sums are formed without regard to that first; if there is a NaN
// among them, they are formed again, and there the other parts meet 0 in the
// place of what is not finite.
template <typename T>
__device__ __forceinline__ Vec<T> finite_only(const Vec<T>& v) {
    constexpr unsigned kExponent = kScaled<T> ? 0x7c00u : 0x7f80u;
    v4u w = __builtin_bit_cast(v4u, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if ((w[k] & kExponent) == kExponent) w[k] &= 0xffff0000u;
        if ((w[k] & kExponent << 16) == kExponent << 16) w[k] &= 0xffffu;
    }
    return __builtin_bit_cast(Vec<T>, w);
}

// Whether a lane of the wavefront may have a NaN among its sums (infinities of
// both signs count too).
template <int N>
__device__ __forceinline__ bool any_nan(const v4f (&sum)[N]) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) t += (sum[k][0] + sum[k][1]) + (sum[k][2] + sum[k][3]);
    return __ballot(t != t) != 0;
}

// Few tokens (at most kFew): a block takes one adapter and finds its tokens
// itself. `slots` = min(G, s) blocks stand for the adapters: adapter `slot` if
// there are no more adapters than tokens, else that of token `slot`, unless an
// earlier token has it too. One slot more stands for the tokens without one.
// tokens: their list; count: how many, 0 for a block without work.
constexpr int kFew = 256;

struct FewTokens {
    int64_t g;                       // the adapter, or -1 for tokens without one
    int count;

    __device__ __forceinline__ FewTokens(const int32_t* ids, int s, int64_t G, int slot, int slots,
                                         int (&tokens)[kFew], int (&counts)[kWaves]) {
        const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
        int id = i < s ? ids[i] : -2;
        if (i < s && (id < 0 || id >= G)) id = -1;
        g = slot == slots ? -1 : G <= s ? slot : ids[slot];
        if (g < 0 || g >= G) g = -1;
        const uint64_t vote = __ballot(id == g);
        if (lane == 0) counts[wave] = __popcll(vote);
        __syncthreads();
        int at = 0;
        count = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) at += counts[w];
            count += counts[w];
        }
        if (id == g) tokens[at + __popcll(vote & ((1ull << lane) - 1))] = i;
        __syncthreads();
        if (slot < slots && (g < 0 || (count > 0 && G > s && tokens[0] != slot))) count = 0;
    }
};

// The distinct adapters among the tokens of a tile, in the order of their
// first tokens; every lane of every wavefront walks them alike. id: the id of
// the tile's token lane % TOK, or -1 for none.
template <int TOK>
struct Adapters {
    uint64_t left;                   // tokens not yet walked (bit k: token k)
    int id;

    __device__ __forceinline__ Adapters(const int32_t* ids, int64_t first, int64_t s, int64_t G) {
        const int64_t i = first + (threadIdx.x & (TOK - 1));
        id = i < s ? ids[i] : -1;
        if (id < 0 || id >= G) id = -1;
        left = __ballot(id >= 0) & mask();
    }
    static __device__ __forceinline__ uint64_t mask() { return TOK == 64 ? ~0ull : (1ull << (TOK & 63)) - 1; }
    // the next adapter, and its tokens
    __device__ __forceinline__ int next(uint64_t& tokens) {
        const int g = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        tokens = __ballot(id == g) & mask();
        left &= ~tokens;
        return g;
    }
};

// ---------------------------------------------------------------------------
// dot: P[split][i, k] = sum over the split's part of len of Z[i, j] M_g[k, j].
//
// A block takes TOK = 16 MT tokens, all ranks (RT tiles of 16) and one of
// `splits` parts of len, of which each wavefront takes a quarter; the four
// sums are joined in LDS. The ranks are the rows of the matrix instruction
// and the tokens its columns; a token's sums depend on no other token, so
// rows past the end are read from the last row and their sums dropped. Of the
// tile's adapters the block takes every `slots`-th, and up to NA of them in
// one pass over Z: a tile where one request ends and the next begins costs no
// second pass. Where the registers hold one (NA = 1), slot 0 takes the tile's
// first adapter and the others the rest, in `late` parts instead of `splits`:
// they are few, and as long as slot 0's they would be what the launch waits
// for. Bound by memory up to 32 ranks (4096 x 12288, rank 16: 20 us by itself,
// 5.0 TB/s, 24-34 after an add, whose results are still being written back) and
// by the CU's loads beyond, where M's pieces are as many as Z's (4096 x 36864,
// rank 64, one adapter: 65-69 us by itself, 4.4 TB/s, 81 after an add). The next
// step's loads go before this one's sums (78 us by itself without).
__host__ __device__ constexpr int dot_tokens(int r) { return r > 64 ? 32 : 64; }

template <typename T, int MT, int RT, int NA>
__global__ __launch_bounds__(kThreads, 2) void k_lora_dot(const T* __restrict__ Z, int64_t ldz,
                                                          const T* __restrict__ M, int64_t G, int r, int len,
                                                          const int32_t* __restrict__ ids, int64_t s, int tiles,
                                                          int slots, int splits, int late,
                                                          float* __restrict__ P) {
    constexpr int TOK = 16 * MT;
    __shared__ v4f join[2][MT * RT * NA][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
    // Neighbouring blocks go to different XCDs, so a slot's blocks are neighbours,
    // most of the higher slots' having nothing to do, and a tile's parts are: those
    // of a tile with two adapters on one XCD took 107 us instead of 95.
    const int later = static_cast<int>(blockIdx.x) - tiles * splits;      // blocks past slot 0's
    const int slot = later < 0 ? 0 : 1 + later / (tiles * late), parts = slot == 0 ? splits : late;
    const int nth = slot == 0 ? static_cast<int>(blockIdx.x) : later % (tiles * late);
    const int part = nth % parts, tile = nth / parts;
    const int64_t first = static_cast<int64_t>(tile) * TOK;
    const int steps = len / 64, w = part * kWaves + wave, all = parts * kWaves;
    const int k0 = static_cast<int>(static_cast<int64_t>(steps) * w / all) * 64;
    const int k1 = static_cast<int>(static_cast<int64_t>(steps) * (w + 1) / all) * 64;
    P += static_cast<int64_t>(part) * s * r;

    const int lrow = lane >> 2, lpiece = (lane & 3) * 8;     // the row and elements of it that this lane reads
    const T* z[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t i = first + t * 16 + lrow;
        z[t] = Z + (i < s ? i : s - 1) * ldz + lpiece;
    }
    Adapters<TOK> adapters(ids, first, s, G);
    if (slot == 0 && wave == 0 && (~adapters.left & Adapters<TOK>::mask()) != 0) {   // rows without an adapter
        for (int t = 0; t < TOK; ++t) {
            const int64_t i = first + t;
            if ((adapters.left >> t & 1) == 0 && i < s)
                for (int k = lane; k < r; k += 64) P[i * r + k] = 0.0f;
        }
    }
    // one pass over Z for N adapters
    const auto pass = [&](auto count, const int64_t(&g)[NA], const uint64_t(&tokens)[NA]) {
        constexpr int N = decltype(count)::value, R = RT * N;
        const T* m[R];
#pragma unroll
        for (int t = 0; t < R; ++t) {
            const int k = t % RT * 16 + lrow;
            m[t] = M + (g[t / RT] * r + (k < r ? k : r - 1)) * len + lpiece;
        }
        v4f sum[MT][R];
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < R; ++b) sum[a][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        Vec<T> zn[2][MT], mn[2][R];      // the step on its way
        const auto fetch = [&](int k) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int t = 0; t < MT; ++t) zn[u][t] = load16(z[t] + k + u * 32);
#pragma unroll
                for (int t = 0; t < R; ++t) mn[u][t] = load16(m[t] + k + u * 32);
            }
        };
        if (k0 < k1) fetch(k0);
        for (int k = k0; k < k1; k += 64) {
            Vec<T> zv[2][MT], mv[2][R];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int t = 0; t < MT; ++t) zv[u][t] = hand_on<T>(zn[u][t]);
#pragma unroll
                for (int t = 0; t < R; ++t) mv[u][t] = hand_on<T>(mn[u][t]);
            }
            __builtin_amdgcn_sched_barrier(0);   // the next step's loads go before this one's sums
            fetch(k + 64 < k1 ? k + 64 : k);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b < R; ++b) sum[a][b] = mma(mv[u][b], zv[u][a], sum[a][b]);
        }
        // wavefronts 2 and 3 to 0 and 1, then 1 to 0
#pragma unroll
        for (int half = 2; half >= 1; half /= 2) {
            __syncthreads();
            if (wave >= half && wave < 2 * half) {
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b < R; ++b) join[wave - half][a * R + b][lane] = sum[a][b];
            }
            __syncthreads();
            if (wave < half) {
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b < R; ++b) sum[a][b] += join[wave][a * R + b][lane];
            }
        }
        if (wave != 0) return;
#pragma unroll
        for (int a = 0; a < MT; ++a) {
            float* p = P + (first + a * 16 + n) * r;
#pragma unroll
            for (int b = 0; b < R; ++b) {
                if ((tokens[b / RT] >> (a * 16 + n) & 1) == 0) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int k = b % RT * 16 + q * 4 + e;
                    if (k < r) p[k] = sum[a][b][e];
                }
            }
        }
    };
    int64_t g[NA];
    uint64_t tokens[NA];
    int held = 0;
    for (int turn = 0; adapters.left; ++turn) {
        uint64_t mine;
        const int64_t id = adapters.next(mine);
        if ((NA == 2 ? turn % slots : turn == 0 ? 0 : 1 + (turn - 1) % (slots - 1)) != slot) continue;
        if (NA == 2 && held == 0) {
            g[0] = id;
            tokens[0] = mine;
            held = 1;
        } else {
            g[NA - 1] = id;
            tokens[NA - 1] = mine;
            pass(std::integral_constant<int, NA>(), g, tokens);
            held = 0;
        }
    }
    if (NA == 2 && held == 1) pass(std::integral_constant<int, 1>(), g, tokens);
}

// dot for few tokens: a block takes one adapter's tokens, 16 at a time, every
// `spread`-th 16 of them, and one of `splits` parts of len; its wavefronts each
// a quarter of that. M, which is what has to be read, is read once for each 16.
template <typename T, int RT>
__global__ __launch_bounds__(kThreads, 2) void k_lora_dot_few(const T* __restrict__ Z, int64_t ldz,
                                                              const T* __restrict__ M, int64_t G, int r, int len,
                                                              const int32_t* __restrict__ ids, int s, int slots,
                                                              int spread, int splits, float* __restrict__ P) {
    __shared__ v4f join[2][RT][64];
    __shared__ int tokens[kFew], counts[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
    const int part = blockIdx.x % splits, group0 = blockIdx.x / splits % spread, slot = blockIdx.x / splits / spread;
    const FewTokens mine(ids, s, G, slot, slots, tokens, counts);
    P += static_cast<int64_t>(part) * s * r;
    if (mine.g < 0) {                    // tokens without an adapter
        for (int k = threadIdx.x; group0 == 0 && k < mine.count * r; k += kThreads)
            P[static_cast<int64_t>(tokens[k / r]) * r + k % r] = 0.0f;
        return;
    }
    const int steps = len / 64, w = part * kWaves + wave, all = splits * kWaves;
    const int k0 = static_cast<int>(static_cast<int64_t>(steps) * w / all) * 64;
    const int k1 = static_cast<int>(static_cast<int64_t>(steps) * (w + 1) / all) * 64;
    const int lrow = lane >> 2, lpiece = (lane & 3) * 8;
    const T* m[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int k = t * 16 + lrow;
        m[t] = M + (mine.g * r + (k < r ? k : r - 1)) * len + lpiece;
    }
    for (int first = group0 * 16; first < mine.count; first += spread * 16) {
        const int zi = tokens[first + lrow < mine.count ? first + lrow : mine.count - 1];
        const T* z = Z + zi * ldz + lpiece;
        v4f sum[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) sum[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        Vec<T> zn[2], mn[2][RT];         // the step on its way
        const auto fetch = [&](int k) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                zn[u] = load16(z + k + u * 32);
#pragma unroll
                for (int t = 0; t < RT; ++t) mn[u][t] = load16(m[t] + k + u * 32);
            }
        };
        if (k0 < k1) fetch(k0);
        for (int k = k0; k < k1; k += 64) {
            Vec<T> zv[2], mv[2][RT];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                zv[u] = hand_on<T>(zn[u]);
#pragma unroll
                for (int t = 0; t < RT; ++t) mv[u][t] = hand_on<T>(mn[u][t]);
            }
            __builtin_amdgcn_sched_barrier(0);
            fetch(k + 64 < k1 ? k + 64 : k);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int t = 0; t < RT; ++t) sum[t] = mma(mv[u][t], zv[u], sum[t]);
        }
#pragma unroll
        for (int half = 2; half >= 1; half /= 2) {
            __syncthreads();
            if (wave >= half && wave < 2 * half) {
#pragma unroll
                for (int t = 0; t < RT; ++t) join[wave - half][t][lane] = sum[t];
            }
            __syncthreads();
            if (wave < half) {
#pragma unroll
                for (int t = 0; t < RT; ++t) sum[t] += join[wave][t][lane];
            }
        }
        if (wave == 0 && first + n < mine.count) {
            float* p = P + static_cast<int64_t>(tokens[first + n]) * r;
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int k = t * 16 + q * 4 + e;
                    if (k < r) p[k] = sum[t][e];
                }
        }
    }
}

// ---------------------------------------------------------------------------
// add: out_i = base_i + f_g P_i M_g.
//
// P enters as two parts side by side, [16 ranks of the first, 16 of the
// second], so that one matrix instruction of 32 products takes 16 ranks whole.
// The tokens are its rows. A wavefront takes 128 columns: M's rows are read 16
// bytes a lane (eight columns of one rank) and turned in registers, so that
// eight instructions cover the columns and a lane ends with eight neighbouring
// columns of four tokens: base and out are moved 16 bytes a lane, 256 adjacent
// bytes of a token at a time.
constexpr int kAddColumns = kWaves * 128;

// M's rows [st 16, st 16 + 16) for eight operands of 16 ranks (both parts
// alike) x 16 columns; turned, operand j holds column mcol + j of each lane.
// Ranks past r are 0.
template <typename T>
__device__ __forceinline__ void load_rows(const T* Mg, int64_t len, int r, int st, int q, int mcol, Vec<T>(&rows)[8]) {
    const int k0 = st * 16 + (q & 1) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) rows[k] = load16(Mg + (k0 + k < r ? k0 + k : r - 1) * len + mcol);
    if (st * 16 + 16 > r) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k >= r) rows[k] = Vec<T>{};
    }
}

template <typename T>
__device__ __forceinline__ void load_ranks(const T* Mg, int64_t len, int r, int st, int q, int mcol,
                                           Vec<T>(&columns)[8]) {
    Vec<T> rows[8];
    load_rows<T>(Mg, len, r, st, q, mcol, rows);
    transpose8<T>(rows, columns);
}

// f_g 2^-ex, kept finite where f_g is (a sum of 0 has to stay 0).
__device__ __forceinline__ float factor_of(float f, int ex) {
    const float v = ldexpf(f, -ex);
    return fabsf(f) < __builtin_inff() ? fminf(fmaxf(v, -3.4028235e38f), 3.4028235e38f) : v;
}

// Where a lane's piece of its token e is.
template <typename T>
__device__ __forceinline__ T* piece_of(T* base, int64_t first, int q, int e, int64_t ld, int col) {
    return base + (first + q * 4 + e) * ld + col;
}

// The tokens of `tokens` (bit k: the tile's token k) among a lane's four.
template <typename T>
__device__ __forceinline__ void store_sums(T* out, int64_t first, int64_t ldo, int col, int q, uint64_t tokens,
                                           const Vec<T>(&b)[4], const v4f(&sum)[8], const float(&factor)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        Vec<T> y;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = from_float<T>(fmaf(sum[j][e], factor[e], to_float<T>(b[e][j])));
        if (tokens >> (q * 4 + e) & 1) *reinterpret_cast<Vec<T>*>(piece_of(out, first, q, e, ldo, col)) = y;
    }
}

// The sum of a value's splits, `stride` apart, in their order. Eight loads are
// on their way at once: one after another they cost a trip to L2 each (add for
// 64 decoded tokens, 8 splits: 27.6 us one after another, 21.9 at once).
__device__ __forceinline__ float join_splits(const float* p, int64_t stride, int splits) {
    float v = 0.0f;
    for (int u0 = 0; u0 < splits; u0 += 8) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = p[(u0 + e < splits ? u0 + e : splits - 1) * stride];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (u0 + e < splits) v += x[e];
    }
    return v;
}

// Few tokens: a block takes one adapter's tokens, 16 at a time, every
// `spread`-th 16 of them, and 512 columns. It joins the splits of its tokens'
// P itself, while M's first ranks and base are on their way, and its first
// columns' blocks also write them to T. Bound by the trips to memory that a
// block makes one after another (ids; P, M and base; out): 64 tokens with 24
// adapters of rank 16, 36864 columns: 16 us for 38 MB, 2.4 TB/s (18 us with a
// block for each 16 neighbouring tokens and adapter, which reads an adapter
// again for every 16). A second group of 512 columns a block, with its own
// loads on their way, took 22 us.
template <typename T>
__global__ __launch_bounds__(kThreads, 3) void k_lora_add_few(const float* __restrict__ P, int splits,
                                                              const T* __restrict__ M, int64_t G, int r, int len,
                                                              const int32_t* __restrict__ ids,
                                                              const float* __restrict__ scale, const T* base,
                                                              int64_t ldb, T* out, int64_t ldo, int s, int slots,
                                                              int spread, float* __restrict__ Tout) {
    constexpr int kSteps = I8MM_LORA_MAX_RANK / 16;
    __shared__ __align__(16) T parts[16 * kSteps * 32];
    __shared__ float values[16][kSteps * 16 + 1];
    __shared__ int exps[16], tokens[kFew], counts[kWaves];
    const int steps = (r + 15) / 16;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
    const int col_blocks = (len + kAddColumns - 1) / kAddColumns;
    const int cb = blockIdx.x % col_blocks, group0 = blockIdx.x / col_blocks % spread;
    const int slot = blockIdx.x / col_blocks / spread;
    const FewTokens mine(ids, s, G, slot, slots, tokens, counts);
    const int col = cb * kAddColumns + wave * 128 + n * 8;  // this lane's columns
    const bool inside = col < len;
    const int mcol = inside ? col : 0;
    const T* Mg = M + (mine.g < 0 ? 0 : mine.g) * r * len;
    const float f = mine.g < 0 ? 0.0f : scale[mine.g];
    for (int first = group0 * 16; first < mine.count; first += spread * 16) {
        Vec<T> rows[8], b[4];            // on their way until the parts are laid out
        int at[4];                       // this lane's tokens, or -1
        if (mine.g >= 0) load_rows<T>(Mg, len, r, 0, q, mcol, rows);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            at[e] = inside && first + q * 4 + e < mine.count ? tokens[first + q * 4 + e] : -1;
            b[e] = Vec<T>{};
            if (base && at[e] >= 0) b[e] = load16(base + static_cast<int64_t>(at[e]) * ldb + col);
        }
        const int t = threadIdx.x / 16, sub = threadIdx.x % 16;
        const int64_t it = first + t < mine.count ? tokens[first + t] : -1;
        if (mine.g < 0) {                // tokens without an adapter are base's
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (at[e] >= 0 && out != base) *reinterpret_cast<Vec<T>*>(out + static_cast<int64_t>(at[e]) * ldo + col) = b[e];
            for (int k = sub; Tout && cb == 0 && it >= 0 && k < r; k += 16) Tout[it * r + k] = 0.0f;
            continue;
        }
        float most = 0.0f;
#pragma unroll 1
        for (int st = 0; st < steps; ++st) {
            const int k = st * 16 + sub;
            const bool real = it >= 0 && k < r;
            const float sum = join_splits(P + (real ? it * r + k : 0), static_cast<int64_t>(s) * r, splits);
            if (real && Tout && cb == 0) Tout[it * r + k] = sum;
            values[t][k] = real ? sum : 0.0f;
            if (real) most = fmaxf(most, finite_size(sum));
        }
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) most = fmaxf(most, __shfl_xor(most, off, kWave));
        const int ex = scale_exponent<T>(most);
        __syncthreads();                 // the last 16 tokens' parts have been read
        if (sub == 0) exps[t] = ex;
#pragma unroll 1
        for (int st = 0; st < steps; ++st) {
            T part[2];
            split<T, 2>(values[t][st * 16 + sub], ex, part);      // the lane's own
            // [step][eight ranks][token]: the lanes of the matrix instruction in order
            T* to = parts + ((st * 4 + sub / 8) * 16 + t) * 8 + sub % 8;
            to[0] = part[0];
            to[2 * 16 * 8] = part[1];
        }
        __syncthreads();
        unsigned again = 0;
        v4f sum[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int st = 0; st < steps; ++st) {
            Vec<T> columns[8];
            if (st > 0) load_rows<T>(Mg, len, r, st, q, mcol, rows);
            transpose8<T>(rows, columns);
            const Vec<T> p = load16(parts + (st * 64 + lane) * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] = mma(p, columns[j], sum[j]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float factor = factor_of(f, exps[q * 4 + e]);
            Vec<T> y;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = fmaf(sum[j][e], factor, to_float<T>(b[e][j]));
                y[j] = from_float<T>(v[j]);
            }
            const float all = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
            const bool nan = all != all;             // or infinities of both signs
            if (at[e] >= 0 && !nan) *reinterpret_cast<Vec<T>*>(out + static_cast<int64_t>(at[e]) * ldo + col) = y;
            again |= (at[e] >= 0 && nan) << e;
        }
        // What has a NaN is formed again with care, without the matrix instruction:
        // kept apart from the sums above, it costs them no registers.
        while (again) {
            const int t = q * 4 + __builtin_ctz(again);
            again &= again - 1;
            v8f whole = {};
#pragma unroll 1
            for (int k = 0; k < r; ++k) {
                const T* part = parts + ((k / 16 * 4 + k / 8 % 2) * 16 + t) * 8 + k % 8;
                const float hi = to_float<T>(part[0]), lo = to_float<T>(part[2 * 16 * 8]);
                const Vec<T> m = load16(Mg + static_cast<int64_t>(k) * len + mcol), others = finite_only<T>(m);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    whole[j] = fmaf(lo, to_float<T>(others[j]), fmaf(hi, to_float<T>(m[j]), whole[j]));
            }
            const int64_t i = tokens[first + t];
            const Vec<T> old = base ? load16(base + i * ldb + col) : Vec<T>{};
            const float factor = factor_of(f, exps[t]);
            Vec<T> y;
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = from_float<T>(fmaf(whole[j], factor, to_float<T>(old[j])));
            *reinterpret_cast<Vec<T>*>(out + i * ldo + col) = y;
        }
    }
}

// Joins the splits of P for many tokens, 16 lanes a token: T (fp32) and, laid
// out as add takes them, the two parts: [tile of 16][step][eight ranks of a
// part][token][8], with the exponent of each token.
// A token whose adapter is not the first of its tile in dot has `late` splits.
__device__ __forceinline__ int splits_of(const int32_t* __restrict__ ids, int64_t G, int splits, int late, int r,
                                         int64_t s, int64_t i) {
    if (late == splits) return splits;
    const int tok = dot_tokens(r), lane = threadIdx.x & 63;
    const int64_t first = i / tok * tok, at = first + lane % tok;
    int id = at < s ? ids[at] : -1;
    if (id < 0 || id >= G) id = -1;
    const uint64_t some = __ballot(id >= 0);
    const int own = __shfl(id, static_cast<int>(i - first), kWave);
    return own >= 0 && own != __builtin_amdgcn_readlane(id, __builtin_ctzll(some)) ? late : splits;
}

template <typename T>
__device__ __forceinline__ void join_tile(const float* __restrict__ P, const int32_t* __restrict__ ids, int64_t G,
                                          int splits, int late, int r, int64_t s, int64_t tile,
                                          float* __restrict__ Tout, T* __restrict__ parts,
                                          int32_t* __restrict__ exps) {
    constexpr int kSteps = I8MM_LORA_MAX_RANK / 16;
    const int steps = (r + 15) / 16, t = threadIdx.x / 16 % 16, sub = threadIdx.x % 16;
    const int64_t i = tile * 16 + t;
    const int mine = splits_of(ids, G, splits, late, r, s, i);
    float v[kSteps], most = 0.0f;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
        v[st] = 0.0f;
        if (st >= steps) continue;
        const int k = st * 16 + sub;
        const bool real = i < s && k < r;
        const float sum = join_splits(P + (real ? i * r + k : 0), s * r, mine);
        if (real) {
            v[st] = sum;
            if (Tout) Tout[i * r + k] = sum;
        }
        most = fmaxf(most, finite_size(v[st]));
    }
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) most = fmaxf(most, __shfl_xor(most, off, kWave));
    const int ex = scale_exponent<T>(most);
    if (sub == 0) exps[i] = ex;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
        if (st >= steps) continue;
        T part[2];
        split<T, 2>(v[st], ex, part);
        T* to = parts + (((tile * steps + st) * 4 + sub / 8) * 16 + t) * 8 + sub % 8;
        to[0] = part[0];
        to[2 * 16 * 8] = part[1];
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_lora_join(const float* __restrict__ P, const int32_t* __restrict__ ids,
                                                        int64_t G, int splits, int late, int r, int64_t s,
                                                        float* __restrict__ Tout, T* __restrict__ parts,
                                                        int32_t* __restrict__ exps) {
    join_tile(P, ids, G, splits, late, r, s, blockIdx.x, Tout, parts, exps);
}

// Many tokens: a block takes 512 columns and `run` tiles of 16 tokens one
// after another, with the next tile's base, parts and ids on their way while
// this one's sums are formed. M's operands stay for as long as the adapter
// does not change: up to 32 ranks (ST steps of 16) in registers, up to 64 in
// LDS, each wavefront its own. Beyond (ST = 0) they are read again for each
// tile. Bound by memory: 4096 x 36864, rank 16: 107 us for 604 MB, 5.7 TB/s;
// 4096 x 12288, rank 64: 56 us for 303 MB, 5.4 TB/s (167 us with those operands
// in registers, which do not hold them). With the columns as the instruction's
// rows, where a wavefront's access is 16 rows of 64 bytes, rank 16 took 138 us.
template <typename T, int ST>
__global__ __launch_bounds__(kThreads, 2) void k_lora_add_many(const T* __restrict__ parts,
                                                               const int32_t* __restrict__ exps,
                                                               const T* __restrict__ M, int64_t G, int r, int len,
                                                               const int32_t* __restrict__ ids,
                                                               const float* __restrict__ scale, const T* base,
                                                               int64_t ldb, T* out, int64_t ldo, int64_t s, int tiles,
                                                               int run) {
    constexpr bool LDS = ST > 2;
    constexpr int KEEP = LDS || ST == 0 ? 1 : ST;
    __shared__ Vec<T> held[LDS ? kWaves * ST * 8 * 32 : 1];
    const int steps = ST > 0 ? ST : (r + 15) / 16;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
    const int col_blocks = (len + kAddColumns - 1) / kAddColumns;
    const int c0 = static_cast<int>(blockIdx.x % col_blocks) * kAddColumns + wave * 128;
    const int t0 = static_cast<int>(blockIdx.x / col_blocks) * run, t1 = t0 + run < tiles ? t0 + run : tiles;
    if (c0 >= len) return;
    const int col = c0 + n * 8;                             // this lane's columns
    const bool inside = col < len;
    const int mcol = inside ? col : c0;

    // operand j of step st: lanes of equal n and q % 2 hold the same ranks
    Vec<T>* const mine = held + (LDS ? wave * ST * 8 * 32 + (q & 1) * 16 + n : 0);
    struct Fetched {
        Vec<T> b[4], p[ST > 0 ? ST : 1];
        v4i ex;
        int id;
    };
    const auto fetch = [&](int tile, Fetched& f) {
        const int64_t first = static_cast<int64_t>(tile) * 16, i = first + n;
        f.id = i < s ? ids[i] : -1;
        if (f.id >= G) f.id = -1;
        f.ex = *reinterpret_cast<const v4i*>(exps + first + q * 4);
        if constexpr (ST > 0) {
#pragma unroll
            for (int st = 0; st < ST; ++st) f.p[st] = load16(parts + ((static_cast<int64_t>(tile) * ST + st) * 64 + lane) * 8);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f.b[e] = Vec<T>{};
            if (base) f.b[e] = load16(base + (first + q * 4 + e < s ? first + q * 4 + e : s - 1) * ldb + mcol);
        }
    };
    int64_t cur = -1;
    float f = 0.0f;
    Vec<T> columns[KEEP][8];
    Fetched next;
    fetch(t0, next);
    for (int tile = t0; tile < t1; ++tile) {
        const Fetched now = next;
        if (tile + 1 < t1) fetch(tile + 1, next);
        const int64_t first = static_cast<int64_t>(tile) * 16;
        uint64_t left = __ballot(now.id >= 0) & 0xffff;
        const uint64_t none = ~left & (s - first < 16 ? (1ull << (s - first)) - 1 : 0xffff);
        if (none && out != base && inside) {                 // rows without an adapter are base's
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (none >> (q * 4 + e) & 1)
                    *reinterpret_cast<Vec<T>*>(piece_of(out, first, q, e, ldo, col)) = now.b[e];
        }
        while (left) {
            const int64_t g = __builtin_amdgcn_readlane(now.id, __builtin_ctzll(left));
            const uint64_t tokens = __ballot(now.id == g) & left;
            left &= ~tokens;
            const T* Mg = M + g * r * len;
            if (g != cur) {
                cur = g;
                f = scale[g];
                if constexpr (LDS) {
                    for (int st = 0; st < ST; ++st) {
                        load_ranks<T>(Mg, len, r, st, q, mcol, columns[0]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) mine[(st * 8 + j) * 32] = columns[0][j];
                    }
                } else if constexpr (ST > 0) {
#pragma unroll
                    for (int st = 0; st < ST; ++st) load_ranks<T>(Mg, len, r, st, q, mcol, columns[st]);
                }
            }
            v4f sum[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (LDS) {
#pragma unroll
                for (int st = 0; st < ST; ++st)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] = mma(now.p[st], mine[(st * 8 + j) * 32], sum[j]);
            } else if constexpr (ST > 0) {
#pragma unroll
                for (int st = 0; st < ST; ++st)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] = mma(now.p[st], columns[st][j], sum[j]);
            } else {
                for (int st = 0; st < steps; ++st) {
                    const Vec<T> p = load16(parts + ((static_cast<int64_t>(tile) * steps + st) * 64 + lane) * 8);
                    load_ranks<T>(Mg, len, r, st, q, mcol, columns[0]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] = mma(p, columns[0][j], sum[j]);
                }
            }
            if (any_nan(sum)) {
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
                const auto careful = [&](const Vec<T>& p, auto&& column) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)          // lanes of q >= 2 hold what the second parts meet
                        sum[j] = mma(p, q >= 2 ? finite_only<T>(column(j)) : column(j), sum[j]);
                };
                if constexpr (ST > 0) {
#pragma unroll
                    for (int st = 0; st < ST; ++st)
                        careful(now.p[st], [&](int j) { return LDS ? mine[(st * 8 + j) * 32] : columns[LDS ? 0 : st][j]; });
                } else {
                    for (int st = 0; st < steps; ++st) {
                        const Vec<T> p = load16(parts + ((static_cast<int64_t>(tile) * steps + st) * 64 + lane) * 8);
                        load_ranks<T>(Mg, len, r, st, q, mcol, columns[0]);
                        careful(p, [&](int j) { return columns[0][j]; });
                    }
                }
            }
            float factor[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) factor[e] = factor_of(f, now.ex[e]);
            if (inside) store_sums<T>(out, first, ldo, col, q, tokens, now.b, sum, factor);
        }
    }
}

// ---------------------------------------------------------------------------
// grad: the tokens in the order of their adapters, in chunks of up to KC
// tokens of one adapter, each chunk in tiles of 32.

struct Chunk {
    int32_t g;                       // the adapter, or -1 for an unused entry
    int32_t first;                   // into the ordered tokens
    int32_t count;
    int32_t tile;                    // the chunk's first tile
    int32_t part;                    // partial sums of the chunk, or -1: the adapter's only one
};

struct Plan {
    int32_t* order;                  // [s + 32]: the tokens, by adapter and then by place
    int32_t* count;                  // [G]: tokens of each adapter
    int32_t* part;                   // [G]: its first partial sums
    int32_t* tile_chunk;             // [tiles]: the chunk of each tile, or -1
    Chunk* chunks;                   // [slots]
    float* most;                     // [2 rank tiles][tiles][16]: each rank's largest finite |factor|
    int32_t* exps;                   // [slots][2 rank tiles][16]: the power of two of each chunk and rank
    int slots, tiles, rank_tiles;
    unsigned first_block;            // of this launch among the blocks of grad
};

constexpr int kPlanThreads = 1024;

// One block an adapter: it counts the tokens of lower adapters (C), how many
// of those there are (D) and its own (n), then lists its own in order. Its
// chunks start at entry C / KC + D, its tiles at C / 32 rounded up plus D, its
// partial sums, if it has more than one chunk, at 2 C / KC: each leaves the
// adapters room whatever their counts, without one block knowing the others'.
// Unused entries up to the next adapter's are marked by this one.
__device__ __forceinline__ void plan_adapter(const int32_t* __restrict__ ids, int s, int G, int KC, const Plan& plan) {
    constexpr int W = kPlanThreads / 64;
    __shared__ int counts[4][W];
    __shared__ uint32_t seen[2048];
    const int g = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, words = (G + 31) / 32;
    for (int k = threadIdx.x; k < words; k += kPlanThreads) seen[k] = 0;
    __syncthreads();
    int lower = 0, own = 0, valid = 0;
    for (int i0 = 0; i0 < s; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x, id = i < s ? ids[i] : -1;
        const bool low = id >= 0 && id < g;
        valid += __popcll(__ballot(id >= 0 && id < G));
        own += __popcll(__ballot(id == g));
        lower += __popcll(__ballot(low));
        if (low && (seen[id >> 5] >> (id & 31) & 1) == 0) atomicOr(&seen[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
    int distinct = 0;
    for (int k0 = 0; k0 < words; k0 += kPlanThreads) {
        const int k = k0 + threadIdx.x;
        int d = k < words ? __popc(seen[k]) : 0;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) d += __shfl_xor(d, off, kWave);
        distinct += d;
    }
    if (lane == 0) {
        counts[0][wave] = lower;
        counts[1][wave] = own;
        counts[2][wave] = valid;
        counts[3][wave] = distinct;
    }
    __syncthreads();
    int total[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int w = 0; w < W; ++w) total[k] += counts[k][w];
    const int C = total[0], n = total[1], D = total[3];
    const bool last = C + n == total[2];
    const int used = (n + KC - 1) / KC, begin = C / KC + D, part = static_cast<int>(2 * static_cast<int64_t>(C) / KC);
    const int tile0 = (C + 31) / 32 + D;
    if (threadIdx.x == 0) {
        plan.count[g] = n;
        plan.part[g] = part;
    }
    if (n > 0 || (g == 0 && total[2] == 0)) {
        const int end = last ? plan.slots : (C + n) / KC + D + 1;
        for (int k = begin + threadIdx.x; k < end; k += kPlanThreads) {
            const int c = k - begin;
            Chunk e{-1, 0, 0, 0, -1};
            if (c < used)
                e = Chunk{g, C + c * KC, n - c * KC < KC ? n - c * KC : KC, tile0 + c * (KC / 32),
                          used > 1 ? part + c : -1};
            plan.chunks[k] = e;
        }
        const int tile_end = last ? plan.tiles : (C + n + 31) / 32 + D + 1;
        for (int k = tile0 + threadIdx.x; k < tile_end; k += kPlanThreads)
            plan.tile_chunk[k] = (k - tile0) * 32 < n ? begin + (k - tile0) * 32 / KC : -1;
    }
    if (n == 0) return;
    int before = C;
    for (int i0 = 0; i0 < s; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        const bool mine = i < s && ids[i] == g;
        const uint64_t vote = __ballot(mine);
        __syncthreads();
        if (lane == 0) counts[0][wave] = __popcll(vote);
        __syncthreads();
        int at = before, all = 0;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            if (k < wave) at += counts[0][k];
            all += counts[0][k];
        }
        if (mine) plan.order[at + __popcll(vote & ((1ull << lane) - 1))] = i;
        before += all;
    }
}

// The plan needs nothing of the dot product and the join nothing of the plan:
// one launch for both, the first G blocks for the plan (4096 tokens, rank 64,
// one adapter a tile: 9 us instead of 8 and 5; 15 where a tile has two, by the
// longer sums).
template <typename T>
__global__ __launch_bounds__(kPlanThreads) void k_lora_plan_join(const int32_t* __restrict__ ids, int s, int G, int KC,
                                                                 Plan plan, const float* __restrict__ P, int splits,
                                                                 int late, int r, float* __restrict__ dT, T* __restrict__ parts,
                                                                 int32_t* __restrict__ exps) {
    if (blockIdx.x < static_cast<unsigned>(G)) {
        plan_adapter(ids, s, G, KC, plan);
        return;
    }
    const int64_t tile = static_cast<int64_t>(blockIdx.x - G) * (kPlanThreads / 256) + threadIdx.x / 256;
    if (tile * 16 < s) join_tile(P, ids, G, splits, late, r, s, tile, dT, parts, exps);
}

// One of the two gradients: the streamed rows Z, the fp32 factors P [s, r] and
// what becomes of them.
struct Side {
    const void* Z;
    int64_t ldz;
    int len;
    const float* P;
    void* laid;                      // [tile][rank tile][parts][lane][8] of the element type
    float* out;                      // [G][r][len]
    float* part;                     // [.][r][len]
};

template <typename T>
constexpr int kParts = kScaled<T> ? 2 : 3;

// The factors f_g P of a tile of 32 ordered tokens: a lane's eight tokens of
// one rank. Tokens past the chunk's end and ranks past r are 0.
struct TileFactors {
    float f;
    int64_t at[8];                   // the tokens' rows in P, or -1

    __device__ __forceinline__ TileFactors(const Plan& plan, const Chunk& c, const float* scale, int r) {
        const int p0 = (static_cast<int>(blockIdx.x) - c.tile) * 32 + (threadIdx.x >> 4 & 3) * 8;
        f = scale[c.g];
#pragma unroll
        for (int e = 0; e < 8; ++e) at[e] = plan.order[c.first + p0 + e];   // 32 more than there are tokens
#pragma unroll
        for (int e = 0; e < 8; ++e) at[e] = p0 + e < c.count ? at[e] * r : -1;
    }
    __device__ __forceinline__ void load(const float* P, int k, int r, float(&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = P[(at[e] < 0 ? 0 : at[e]) + (k < r ? k : r - 1)];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = at[e] >= 0 && k < r ? f * v[e] : 0.0f;
    }
};

// The largest finite value in the four lanes of each rank, in all of them.
__device__ __forceinline__ float rank_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, kWave));
    return fmaxf(v, __shfl_xor(v, 32, kWave));
}

// The largest finite |f_g P| of each tile and rank, for both sides: a block
// takes one tile, a wavefront one task (16 ranks of one side).
__global__ __launch_bounds__(kThreads) void k_lora_most(Side x, Side y, const float* __restrict__ scale, int r,
                                                        Plan plan) {
    const int chunk = plan.tile_chunk[blockIdx.x], tasks = 2 * plan.rank_tiles;
    const int task = blockIdx.y * kWaves + (threadIdx.x >> 6);
    if (chunk < 0 || task >= tasks) return;
    const TileFactors t(plan, plan.chunks[chunk], scale, r);
    const int which = task >= plan.rank_tiles, rt = which ? task - plan.rank_tiles : task;
    float v[8], most = 0.0f;
    t.load(which ? y.P : x.P, rt * 16 + (threadIdx.x & 15), r, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) most = fmaxf(most, finite_size(v[e]));
    most = rank_max(most);
    if ((threadIdx.x & 63) < 16)
        plan.most[(static_cast<int64_t>(task) * plan.tiles + blockIdx.x) * 16 + threadIdx.x % 16] = most;
}

// The power of two of a chunk and rank task 16 + lane % 16, from all the
// chunk's tiles. Ranks do not share theirs: one that is far smaller than its
// neighbours, as a rank that has hardly been trained, keeps its digits.
template <typename T>
__device__ __forceinline__ int exponent_of(const Plan& plan, const Chunk& c, int task) {
    if constexpr (!kScaled<T>) return 0;
    const float* at = plan.most + (static_cast<int64_t>(task) * plan.tiles + c.tile) * 16;
    float most = 0.0f;
#pragma unroll 8
    for (int k = threadIdx.x & 63; k < (c.count + 31) / 32 * 16; k += 64) most = fmaxf(most, at[k]);
    return scale_exponent<T>(rank_max(most));
}

// Lays f_g P out as the matrix instruction takes it: a block takes one tile, a
// wavefront 16 ranks of one side at a time, a lane eight tokens of one rank.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_lora_lay(Side x, Side y, const float* __restrict__ scale, int r,
                                                       Plan plan) {
    const int chunk = plan.tile_chunk[blockIdx.x];
    const int task = blockIdx.y * kWaves + (threadIdx.x >> 6);
    if (chunk < 0 || task >= 2 * plan.rank_tiles) return;
    const Chunk c = plan.chunks[chunk];
    const TileFactors t(plan, c, scale, r);
    const int lane = threadIdx.x & 63, n = lane & 15;
    {
        const int which = task >= plan.rank_tiles, rt = which ? task - plan.rank_tiles : task;
        float v[8];
        t.load(which ? y.P : x.P, rt * 16 + n, r, v);
        const int ex = exponent_of<T>(plan, c, task);
        if (kScaled<T> && static_cast<int>(blockIdx.x) == c.tile && lane < 16)
            plan.exps[(static_cast<int64_t>(chunk) * 2 * plan.rank_tiles + task) * 16 + lane] = ex;
        Vec<T> out[kParts<T>];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            T part[kParts<T>];
            split<T, kParts<T>>(v[e], ex, part);
#pragma unroll
            for (int p = 0; p < kParts<T>; ++p) out[p][e] = part[p];
        }
        T* to = static_cast<T*>(which ? y.laid : x.laid) +
                (static_cast<int64_t>(blockIdx.x) * plan.rank_tiles + rt) * kParts<T> * 512;
#pragma unroll
        for (int p = 0; p < kParts<T>; ++p) *reinterpret_cast<Vec<T>*>(to + p * 512 + lane * 8) = out[p];
    }
}

// out_g[k, j] = sum over the chunk's tokens of f P[i, k] Z[i, j]: what the two
// kernels below share. A block takes one chunk and 128 columns of one side.
// Z's rows are read 16 bytes a lane (eight columns of one token) and turned in
// registers; the ranks are the rows of the matrix instruction, so a lane ends
// with eight neighbouring columns of four ranks. Tokens past the end have
// factors of 0 and rows of 0.
template <typename T>
struct GradBlock {
    typedef int v8i __attribute__((ext_vector_type(8)));
    Chunk c;
    const T* Z;
    const T* laid;
    const int32_t* order;
    float* out;
    int64_t ldz;
    int len, col, chunk, steps;
    bool second;

    __device__ __forceinline__ GradBlock(const Side& x, const Side& y, int r, const Plan& plan) {
        const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
        const int xblocks = (x.len + 127) / 128, blocks = xblocks + (y.len + 127) / 128;
        const unsigned block = plan.first_block + blockIdx.x;
        const int cb = blocks - 1 - static_cast<int>(block % blocks);
        chunk = block / blocks;
        c = plan.chunks[chunk];
        second = cb >= xblocks;
        len = second ? y.len : x.len;
        ldz = second ? y.ldz : x.ldz;
        col = (second ? cb - xblocks : cb) * 128 + n * 8;
        Z = static_cast<const T*>(second ? y.Z : x.Z) + (col < len ? col : 0);
        laid = static_cast<const T*>(second ? y.laid : x.laid) + lane * 8;
        order = plan.order + c.first + q * 8;
        out = c.part < 0 ? (second ? y.out : x.out) + static_cast<int64_t>(c.g) * r * len
                         : (second ? y.part : x.part) + static_cast<int64_t>(c.part) * r * len;
        steps = (c.count + 31) / 32;
    }
    // the lane's eight tokens of a tile: those past the end are not used
    __device__ __forceinline__ v8i tokens_of(int st) const {
        v8i t;
        __builtin_memcpy(&t, order + (st < steps ? st : steps - 1) * 32, sizeof(t));
        return t;
    }
    __device__ __forceinline__ void rows_of(int st, const v8i& t, Vec<T>(&rows)[8]) const {
        if (st * 32 + 32 <= c.count) {
#pragma unroll
            for (int e = 0; e < 8; ++e) rows[e] = load16(Z + static_cast<int64_t>(t[e]) * ldz);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                rows[e] = Vec<T>{};
                if (st * 32 + static_cast<int>(threadIdx.x >> 4 & 3) * 8 + e < c.count)
                    rows[e] = load16(Z + static_cast<int64_t>(t[e]) * ldz);
            }
        }
    }
    // the parts of a tile's factors for 16 ranks
    __device__ __forceinline__ void factors_of(const Plan& plan, int st, int rt, Vec<T>(&f)[kParts<T>]) const {
        const T* at = laid + (static_cast<int64_t>(c.tile + st) * plan.rank_tiles + rt) * kParts<T> * 512;
#pragma unroll
        for (int p = 0; p < kParts<T>; ++p) f[p] = load16(at + p * 512);
    }
    __device__ __forceinline__ void store(const Plan& plan, int rt, int r, const v4f(&sum)[8]) const {
        const int row = static_cast<int>(threadIdx.x >> 4 & 3) * 4;
        v4i exs{0, 0, 0, 0};
        if constexpr (kScaled<T>)
            exs = *reinterpret_cast<const v4i*>(
                plan.exps + (static_cast<int64_t>(chunk) * 2 * plan.rank_tiles + second * plan.rank_tiles + rt) * 16 + row);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = rt * 16 + row + e, ex = exs[e];
            if (k >= r || col >= len) continue;
            v4f lo, hi;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lo[j] = ldexpf(sum[j][e], -ex);
                hi[j] = ldexpf(sum[j + 4][e], -ex);
            }
            v4f* p = reinterpret_cast<v4f*>(out + static_cast<int64_t>(k) * len + col);
            p[0] = lo;
            p[1] = hi;
        }
    }
};

// The sums of RT tiles of ranks over the whole chunk by one wavefront, with
// care for infinities in Z: only for chunks that have made a NaN.
template <typename T, int RT>
__device__ __forceinline__ void careful_sums(const GradBlock<T>& b, const Plan& plan, int rt, v4f(&sum)[RT][8]) {
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[t][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int st = 0; st < b.steps; ++st) {
        Vec<T> rows[8], columns[8];
        b.rows_of(st, b.tokens_of(st), rows);
        transpose8<T>(rows, columns);
#pragma unroll
        for (int p = 0; p < kParts<T>; ++p) {
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                Vec<T> f[kParts<T>];
                b.factors_of(plan, st, rt + t < plan.rank_tiles ? rt + t : plan.rank_tiles - 1, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[t][j] = mma(f[p], columns[j], sum[t][j]);
            }
            if (p == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) columns[j] = finite_only<T>(columns[j]);
            }
        }
    }
}

// Blocks past those of the chunks, one for each adapter and 128 columns, write
// the zeros of adapters that no token carries. True for such a block.
__device__ __forceinline__ bool write_zeros(const Side& x, const Side& y, int r, const Plan& plan) {
    const int xblocks = (x.len + 127) / 128, blocks = xblocks + (y.len + 127) / 128;
    const unsigned block = plan.first_block + blockIdx.x;
    if (block < static_cast<unsigned>(plan.slots) * blocks) return false;
    const int at = block - plan.slots * blocks, g = at / blocks, cb = at % blocks;
    if (plan.count[g] > 0) return true;
    const bool second = cb >= xblocks;
    const int len = second ? y.len : x.len, col = (second ? cb - xblocks : cb) * 128 + (threadIdx.x & 31) * 4;
    float* out = (second ? y.out : x.out) + static_cast<int64_t>(g) * r * len;
    for (int k = threadIdx.x >> 5; k < r && col < len; k += kThreads / 32)
        *reinterpret_cast<v4f*>(out + static_cast<int64_t>(k) * len + col) = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    return true;
}

// Up to 32 ranks (RT tiles): every wavefront takes all ranks and every fourth
// tile, with the next one's rows, and the tokens of the one after, on their
// way while this one's sums are formed; the four sums are joined in LDS. Bound
// by memory: 4096 tokens x (12288 + 36864), 403 MB: rank 16 74-77 us (5.3 TB/s),
// rank 32 86-89 us.
template <typename T, int RT>
__global__ __launch_bounds__(kThreads, 2) void k_lora_grad(Side x, Side y, int r, Plan plan) {
    __shared__ v4f join[2][RT * 8][64];
    if (write_zeros(x, y, r, plan)) return;
    const GradBlock<T> b(x, y, r, plan);
    if (b.c.g < 0) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v4f sum[RT][8];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[t][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    Vec<T> rows[8];
    auto ahead = b.tokens_of(wave);
    if (wave < b.steps) b.rows_of(wave, ahead, rows);
    ahead = b.tokens_of(wave + kWaves);
    for (int st = wave; st < b.steps; st += kWaves) {
        Vec<T> f[RT][kParts<T>], columns[8];
#pragma unroll
        for (int t = 0; t < RT; ++t) b.factors_of(plan, st, t, f[t]);
        transpose8<T>(rows, columns);
        __builtin_amdgcn_sched_barrier(0);
        if (st + kWaves < b.steps) b.rows_of(st + kWaves, ahead, rows);
        ahead = b.tokens_of(st + 2 * kWaves);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int p = 0; p < kParts<T>; ++p)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[t][j] = mma(f[t][p], columns[j], sum[t][j]);
    }
#pragma unroll
    for (int half = 2; half >= 1; half /= 2) {
        __syncthreads();
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int j = 0; j < 8; ++j) join[wave - half][t * 8 + j][lane] = sum[t][j];
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[t][j] += join[wave][t * 8 + j][lane];
        }
    }
    if (wave != 0) return;
    bool nan = false;
#pragma unroll
    for (int t = 0; t < RT; ++t) nan |= any_nan(sum[t]);
    if (nan) careful_sums<T, RT>(b, plan, 0, sum);
#pragma unroll
    for (int t = 0; t < RT; ++t) b.store(plan, t, r, sum[t]);
}

// More ranks: the wavefronts divide the ranks (RW tiles of 16 each). Each
// reads and turns one tile of a round of four and leaves it in LDS for all, so
// that Z is read once and every wavefront has rows of its own on their way.
// 4096 tokens x (12288 + 36864), rank 64: 90-107 us for 403 MB and 50 MB of
// partial sums, up to 4.9 TB/s (with a wavefront's own rows 171 us, with pairs
// that read the same rows 148). It starts with the columns that the dot product
// before it read last, which a cache may still hold: 94 us instead of 107.
template <typename T, int RW>
__global__ __launch_bounds__(kThreads, 2) void k_lora_grad_shared(Side x, Side y, int r, Plan plan) {
    __shared__ Vec<T> turned[kWaves][8][64];
    if (write_zeros(x, y, r, plan)) return;
    const GradBlock<T> b(x, y, r, plan);
    if (b.c.g < 0) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v4f sum[RW][8];
#pragma unroll
    for (int t = 0; t < RW; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[t][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    Vec<T> rows[8];
    auto ahead = b.tokens_of(wave);
    if (wave < b.steps) b.rows_of(wave, ahead, rows);
    ahead = b.tokens_of(wave + kWaves);
    for (int st0 = 0; st0 < b.steps; st0 += kWaves) {
        const int st = st0 + wave;
        Vec<T> f[kWaves][RW][kParts<T>], columns[8];
#pragma unroll
        for (int u = 0; u < kWaves; ++u)
#pragma unroll
            for (int t = 0; t < RW; ++t) {
                const int rt = wave * RW + t;
                b.factors_of(plan, st0 + u < b.steps ? st0 + u : b.steps - 1,
                             rt < plan.rank_tiles ? rt : plan.rank_tiles - 1, f[u][t]);
            }
        transpose8<T>(rows, columns);
        // LDS alone is waited for: the factors stay on their way
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // the last round's reads have ended
#pragma unroll
        for (int j = 0; j < 8; ++j) turned[wave][j][lane] = columns[j];
        if (st + kWaves < b.steps) b.rows_of(st + kWaves, ahead, rows);
        ahead = b.tokens_of(st + 2 * kWaves);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int u = 0; u < kWaves; ++u) {
            if (st0 + u >= b.steps) break;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const Vec<T> z = turned[u][j][lane];
#pragma unroll
                for (int t = 0; t < RW; ++t)
#pragma unroll
                    for (int p = 0; p < kParts<T>; ++p) sum[t][j] = mma(f[u][t][p], z, sum[t][j]);
            }
        }
    }
    bool nan = false;
#pragma unroll
    for (int t = 0; t < RW; ++t) nan |= any_nan(sum[t]);
    if (nan) careful_sums<T, RW>(b, plan, wave * RW, sum);
#pragma unroll
    for (int t = 0; t < RW; ++t)
        if (wave * RW + t < plan.rank_tiles) b.store(plan, wave * RW + t, r, sum[t]);
}

// Adapters of several chunks: their partial sums in order. Adapters that no
// token carries: zeros.
__global__ __launch_bounds__(kThreads) void k_lora_grad_sum(Side x, Side y, int r, int KC, Plan plan) {
    const int g = blockIdx.y, n = plan.count[g];
    if (n > 0 && n <= KC) return;
    const int64_t xn = static_cast<int64_t>(r) * x.len / 4, yn = static_cast<int64_t>(r) * y.len / 4;
    int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (at >= xn + yn) return;
    const bool first = at < xn;
    const Side& side = first ? x : y;
    const int64_t size = first ? xn : yn;
    at -= first ? 0 : xn;
    const v4f* p = reinterpret_cast<const v4f*>(side.part) + plan.part[g] * size + at;
    v4f v{0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = 0; c < (n + KC - 1) / KC; ++c) v += p[c * size];
    reinterpret_cast<v4f*>(side.out)[g * size + at] = v;
}

// ---------------------------------------------------------------------------
// Host side.

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Few tokens, as in decoding, may each carry an adapter of their own: blocks
// for each adapter. With many, a block takes a tile of neighbours, most of
// which have one adapter; where a pass does not take two of them, the others
// have blocks of their own, which leave at once in all other tiles (4096 x
// 36864, rank 64, two adapters that meet inside a tile, in a backward pass: 145 us
// for the one block's two passes, 115 for two blocks, 90 with the second in
// smaller parts). Tokens of many adapters in turn cost their tiles a pass for
// each: 512 tokens of 64 adapters, 12288 -> 36864, rank 16: dot 50 and add 88 us,
// 19 and 35 for the same tokens in the adapters' order.
bool few(int64_t s) { return s <= kFew; }
int tile_slots(int64_t s, int64_t r) { return s <= 1024 ? 4 : r > 32 ? 2 : 1; }
int few_slots(int64_t s, int64_t G) { return static_cast<int>(G < s ? G : s); }
// blocks that share an adapter's tokens, in case they are all of one
int few_spread(int64_t s) { return static_cast<int>(up(s, 64)); }

// Parts that dot splits len into; each wavefront keeps at least two steps of
// 64. Few tokens: 8 to 16, so that one adapter alone has blocks enough. Many:
// about one block a CU (4096 x 36864, rank 64, by itself: 69 us at 256 blocks, 78
// at 512, 87 at 1024).
int dot_splits(int64_t s, int64_t len, int64_t r) {
    const int64_t most = len / 64 / 8;
    const int64_t want = few(s) ? (s <= 16 ? 16 : 8) : up(kCus, up(s, dot_tokens(static_cast<int>(r))));
    const int64_t n = want < most ? want : most;
    return static_cast<int>(n < 1 ? 1 : n);
}

// Parts for a tile's later adapters, where a pass takes one adapter. 4096 x
// 36864, rank 64, one tile with two adapters, in a backward pass: 115 us with as
// many parts as the first has, 95 with 16, 90 with 32, 83 without such a tile;
// rank 128, four such tiles, by itself: 223, 174, 162. Every token has room for as many sums, so they
// become fewer as the tiles become more: what the launch waits for at its end,
// a part of a later adapter, is then a smaller share of it anyway (rank 64, 12288
// columns, 131072 tokens: 749 us with 8 parts, 733 with 4; 262144: 1472 with 8,
// 1421 with 2; but 65536 tokens, 36864 columns: 1030 with 8, 1153 with 1), and the
// room beyond one sum a token stays below 135 MB.
int dot_late(int64_t s, int splits, int64_t r) {
    const int64_t room = 8192 / up(s > 0 ? s : 1, dot_tokens(static_cast<int>(r)));
    int n = 8 * splits < 32 ? 8 * splits : 32;
    if (room < n) n = static_cast<int>(room);
    return r <= 32 || splits > n ? splits : n;
}

template <typename T>
hipError_t dot(const LoraArgs& a, const void* Zv, int64_t ldz, const void* Mv, int64_t len, float* P,
               hipStream_t stream) {
    const T* Z = static_cast<const T*>(Zv);
    const T* M = static_cast<const T*>(Mv);
    const int splits = dot_splits(a.s, len, a.r), late = dot_late(a.s, splits, a.r), n = static_cast<int>(len);
    using std::integral_constant;
    const integral_constant<int, 1> one;
    const integral_constant<int, 2> two;
    const integral_constant<int, 4> four;
    const integral_constant<int, 8> eight;
    if (few(a.s)) {
        const int slots = few_slots(a.s, a.G), spread = few_spread(a.s);
        const auto go = [&](auto rt) {
            k_lora_dot_few<T, decltype(rt)::value>
                <<<static_cast<unsigned>((slots + 1) * spread * splits), kThreads, 0, stream>>>(
                    Z, ldz, M, a.G, a.r, n, a.ids, static_cast<int>(a.s), slots, spread, splits, P);
        };
        if (a.r <= 16) go(one);
        else if (a.r <= 32) go(two);
        else if (a.r <= 64) go(four);
        else go(eight);
    } else {                             // as many adapters a pass as the registers hold
        const auto go = [&](auto mt, auto rt, auto na) {
            constexpr int MT = decltype(mt)::value, RT = decltype(rt)::value, NA = decltype(na)::value;
            const int tiles = static_cast<int>(up(a.s, 16 * MT)), slots = tile_slots(a.s, a.r);
            k_lora_dot<T, MT, RT, NA>
                <<<static_cast<unsigned>(tiles * (splits + (slots - 1) * static_cast<int64_t>(late))), kThreads, 0,
                   stream>>>(Z, ldz, M, a.G, a.r, n, a.ids, a.s, tiles, slots, splits, late, P);
        };
        if (a.r <= 16) go(four, one, two);
        else if (a.r <= 32) go(four, two, two);
        else if (a.r <= 64) go(four, four, one);
        else go(two, eight, one);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t add_many(const LoraArgs& a, const void* parts, const int32_t* exps, const void* M, int64_t len,
                    const void* base, int64_t ldb, void* out, int64_t ldo, hipStream_t stream) {
    const int64_t col_blocks = up(len, kAddColumns), tiles = up(a.s, 16);
    const int64_t run = tiles * col_blocks / (6 * kCus) > 1 ? tiles * col_blocks / (6 * kCus) : 1;
    const auto go = [&](auto st) {
        k_lora_add_many<T, decltype(st)::value>
            <<<static_cast<unsigned>(up(tiles, run) * col_blocks), kThreads, 0, stream>>>(
                static_cast<const T*>(parts), exps, static_cast<const T*>(M), a.G, a.r, static_cast<int>(len), a.ids,
                a.scale, static_cast<const T*>(base), ldb, static_cast<T*>(out), ldo, a.s, static_cast<int>(tiles),
                static_cast<int>(run));
    };
    if (a.r <= 16) go(std::integral_constant<int, 1>());
    else if (a.r <= 32) go(std::integral_constant<int, 2>());
    else if (a.r <= 48) go(std::integral_constant<int, 3>());
    else if (a.r <= 64) go(std::integral_constant<int, 4>());
    else go(std::integral_constant<int, 0>());
    return hipGetLastError();
}

// Places in a workspace, each 256-byte aligned.
struct Places {
    size_t at = 0;
    size_t take(int64_t bytes) {
        const size_t p = at;
        at += static_cast<size_t>(up(bytes, 256) * 256);
        return p;
    }
};

// Workspace of a dot and what joins it.
struct DotPlaces {
    size_t P, parts, exps;
    DotPlaces(Places& w, int64_t s, int64_t len, int64_t r) {
        const int splits = dot_splits(s, len, r);
        P = w.take(4 * (few(s) ? splits : dot_late(s, splits, r)) * s * r);
        parts = w.take(up(s, 16) * up(r, 16) * 16 * 32 * 2);
        exps = w.take(4 * up(s, 16) * 16);
    }
};

template <typename T>
hipError_t join(const LoraArgs& a, int splits, const float* P, float* Tout, void* parts, int32_t* exps,
                hipStream_t stream) {
    k_lora_join<T><<<static_cast<unsigned>(up(a.s, 16)), kThreads, 0, stream>>>(
        P, a.ids, a.G, splits, dot_late(a.s, splits, a.r), a.r, a.s, Tout, static_cast<T*>(parts), exps);
    return hipGetLastError();
}

template <typename T>
hipError_t forward(const LoraArgs& a, const void* X, int64_t ldx, const void* base, int64_t ldb, void* Y, int64_t ldy,
                   float* Tp, void* workspace, hipStream_t stream) {
    Places w;
    const DotPlaces d(w, a.s, a.h, a.r);
    char* ws = static_cast<char*>(workspace);
    float* P = reinterpret_cast<float*>(ws + d.P);
    const int splits = dot_splits(a.s, a.h, a.r);
    hipError_t e = dot<T>(a, X, ldx, a.A, a.h, P, stream);
    if (e != hipSuccess) return e;
    if (few(a.s)) {
        const int slots = few_slots(a.s, a.G), spread = few_spread(a.s);
        k_lora_add_few<T>
            <<<static_cast<unsigned>((slots + 1) * spread * up(a.o, kAddColumns)), kThreads, 0, stream>>>(
                P, splits, static_cast<const T*>(a.B), a.G, a.r, static_cast<int>(a.o), a.ids, a.scale,
                static_cast<const T*>(base), ldb, static_cast<T*>(Y), ldy, static_cast<int>(a.s), slots, spread, Tp);
        return hipGetLastError();
    }
    int32_t* exps = reinterpret_cast<int32_t*>(ws + d.exps);
    if ((e = join<T>(a, splits, P, Tp, ws + d.parts, exps, stream)) != hipSuccess) return e;
    return add_many<T>(a, ws + d.parts, exps, a.B, a.o, base, ldb, Y, ldy, stream);
}

// The backward pass's workspace.
struct Layout {
    int KC, slots, tiles;
    size_t dT, order, count, part, tile_chunk, chunks, most, exps, laid[2], sums[2];
    Places w;
    DotPlaces d;

    Layout(int64_t s, int64_t h, int64_t o, int64_t r, int64_t G) : d(w, s, o, r) {
        // Chunks as long as still leave about 1024 blocks, up to 1024 tiles; for up
        // to 512 tokens no partial sums, whose launch costs more than the blocks
        // gain (301 tokens of three adapters, rank 8: 34.4 us with them, 30.0 without).
        const int64_t blocks = s <= 512 ? 4 * kCus : up(h, 128) + up(o, 128);
        int64_t kc = up(up(s > 0 ? s : 1, up(4 * kCus, blocks)), 128) * 128;
        kc = kc < 32768 ? kc : 32768;
        KC = static_cast<int>(kc);
        const int64_t groups = G < s ? G : s, rt = up(r, 16);
        slots = static_cast<int>(s / kc + groups + 1);
        tiles = static_cast<int>(up(s, 32) + groups + 1);
        const int64_t parts = kc < s ? 2 * s / kc + 1 : 0;
        dT = w.take(4 * s * r);
        order = w.take(4 * (s + 32));
        count = w.take(4 * G);
        part = w.take(4 * G);
        tile_chunk = w.take(4 * tiles);
        chunks = w.take(static_cast<int64_t>(sizeof(Chunk)) * slots);
        most = w.take(4 * 2 * rt * tiles * 16);
        exps = w.take(4 * 2 * rt * slots * 16);
        for (int k = 0; k < 2; ++k) {
            laid[k] = w.take(tiles * rt * 3 * 512 * 2);
            sums[k] = w.take(4 * parts * r * (k == 0 ? h : o));
        }
    }
};

template <typename T>
hipError_t backward(const LoraArgs& a, const void* dY, int64_t lddy, const void* X, int64_t ldx, const float* Tp,
                    const void* base, int64_t ldb, void* dX, int64_t lddx, float* dA, float* dB, void* workspace,
                    hipStream_t stream) {
    const Layout l(a.s, a.h, a.o, a.r, a.G);
    char* ws = static_cast<char*>(workspace);
    const auto ints = [ws](size_t at) { return reinterpret_cast<int32_t*>(ws + at); };
    const auto floats = [ws](size_t at) { return reinterpret_cast<float*>(ws + at); };
    const int rt = static_cast<int>(up(a.r, 16));
    Plan plan{ints(l.order), ints(l.count), ints(l.part), ints(l.tile_chunk),
              reinterpret_cast<Chunk*>(ws + l.chunks), floats(l.most), ints(l.exps), l.slots, l.tiles, rt, 0};
    float* dT = floats(l.dT);
    const Side x{X, ldx, static_cast<int>(a.h), dT, ws + l.laid[0], dA, floats(l.sums[0])};
    const Side y{dY, lddy, static_cast<int>(a.o), Tp, ws + l.laid[1], dB, floats(l.sums[1])};
    const int r = a.r;
    float* P = floats(l.d.P);
    const int splits = dot_splits(a.s, a.o, a.r), late = few(a.s) ? splits : dot_late(a.s, splits, a.r);
    const auto plan_join = [&] {
        k_lora_plan_join<T>
            <<<static_cast<unsigned>(a.G + up(a.s, kPlanThreads / 16)), kPlanThreads, 0, stream>>>(
                a.ids, static_cast<int>(a.s), static_cast<int>(a.G), l.KC, plan, P, splits, late, r, dT,
                reinterpret_cast<T*>(ws + l.d.parts), ints(l.d.exps));
        return hipGetLastError();
    };
    hipError_t e;
    if (a.s > 0) {
        if ((e = dot<T>(a, dY, lddy, a.B, a.o, P, stream)) != hipSuccess) return e;
        if ((e = plan_join()) != hipSuccess) return e;
        const dim3 per_tile(static_cast<unsigned>(l.tiles), static_cast<unsigned>(up(2 * rt, kWaves)));
        if constexpr (kScaled<T>)
            k_lora_most<<<per_tile, kThreads, 0, stream>>>(x, y, a.scale, r, plan);
        k_lora_lay<T><<<per_tile, kThreads, 0, stream>>>(x, y, a.scale, r, plan);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        // without partial sums the same launch also writes the zeros
        const int64_t all = (l.slots + (l.KC < a.s ? 0 : a.G)) * (up(a.h, 128) + up(a.o, 128));
        // tens of thousands of adapters on wide layers are more than one grid holds
        for (int64_t first = 0, most = kGridThreads / kThreads; first < all; first += most) {
            plan.first_block = static_cast<unsigned>(first);
            const unsigned blocks = static_cast<unsigned>(all - first < most ? all - first : most);
            if (rt == 1) k_lora_grad<T, 1><<<blocks, kThreads, 0, stream>>>(x, y, r, plan);
            else if (rt == 2) k_lora_grad<T, 2><<<blocks, kThreads, 0, stream>>>(x, y, r, plan);
            else if (rt <= 4) k_lora_grad_shared<T, 1><<<blocks, kThreads, 0, stream>>>(x, y, r, plan);
            else k_lora_grad_shared<T, 2><<<blocks, kThreads, 0, stream>>>(x, y, r, plan);
        }
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (dX && (e = add_many<T>(a, ws + l.d.parts, ints(l.d.exps), a.A, a.h, base, ldb, dX, lddx, stream)) !=
                      hipSuccess)
            return e;
    }
    if (a.s > 0 && l.KC >= a.s) return hipSuccess;
    if (a.s == 0 && (e = plan_join()) != hipSuccess) return e;
    const int64_t fours = static_cast<int64_t>(r) * (a.h + a.o) / 4;
    k_lora_grad_sum<<<dim3(static_cast<unsigned>(up(fours, kThreads)), static_cast<unsigned>(a.G)), kThreads, 0,
                      stream>>>(x, y, r, l.KC, plan);
    return hipGetLastError();
}

}  // namespace

size_t lora_forward_scratch(int64_t s, int64_t h, int64_t, int64_t r) {
    Places w;
    DotPlaces(w, s, h, r);
    return w.at;
}

size_t lora_backward_scratch(int64_t s, int64_t h, int64_t o, int64_t r, int64_t G) {
    return Layout(s, h, o, r, G).w.at;
}

hipError_t launch_lora_forward(const LoraArgs& a, const void* X, int64_t ldx, const void* base, int64_t ldb, void* Y,
                               int64_t ldy, float* T, void* workspace, hipStream_t stream) {
    if (a.s == 0) return hipSuccess;
    return a.type == Dtype::F16 ? forward<_Float16>(a, X, ldx, base, ldb, Y, ldy, T, workspace, stream)
                                : forward<__bf16>(a, X, ldx, base, ldb, Y, ldy, T, workspace, stream);
}

hipError_t launch_lora_backward(const LoraArgs& a, const void* dY, int64_t lddy, const void* X, int64_t ldx,
                                const float* T, const void* base, int64_t ldb, void* dX, int64_t lddx, float* dA,
                                float* dB, void* workspace, hipStream_t stream) {
    return a.type == Dtype::F16
               ? backward<_Float16>(a, dY, lddy, X, ldx, T, base, ldb, dX, lddx, dA, dB, workspace, stream)
               : backward<__bf16>(a, dY, lddy, X, ldx, T, base, ldb, dX, lddx, dA, dB, workspace, stream);
}

}  // namespace i8mm
