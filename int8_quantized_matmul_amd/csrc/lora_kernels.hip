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
// bits, after an exact power of two has brought the largest of the values
// that share it near 2^14, so that neither range nor subnormals cost digits;
// bf16, which has fp32's range: two parts of 8 bits towards a 16-bit result,
// three towards an fp32 one. Y and dX are rounded once.

#include "launch.h"

#include "adapt_common.h"

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

// The power of two that takes values up to `most` in magnitude near 2^14, as
// its exponent; 0 for none, for infinity and for NaN.
template <typename T>
__device__ __forceinline__ int scale_exponent(float most) {
    if constexpr (!kScaled<T>) return 0;
    return most > 0.0f && most < __builtin_inff() ? 15 - __builtin_amdgcn_frexp_expf(most) : 0;
}

// v 2^ex as a sum of N parts of type T. What is not finite is its own first
// part; a finite value that fp16 cannot hold (beside an infinity, which left
// ex at 0) stays finite.
template <typename T, int N>
__device__ __forceinline__ void split(float v, int ex, T(&part)[N]) {
    if constexpr (kScaled<T>) {
        v = ldexpf(v, ex);
        if (fabsf(v) < __builtin_inff()) v = fminf(fmaxf(v, -65504.0f), 65504.0f);
    }
    const bool finite = fabsf(v) < __builtin_inff();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        part[k] = from_float<T>(v);
        v = finite ? v - to_float<T>(part[k]) : 0.0f;
    }
}

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
// and the tokens its columns, both operands come from memory in the layout
// that the instruction wants, and a token's sums depend on no other token, so
// rows past the end are read from the last row and their sums dropped. Of the
// tile's adapters the block takes every `slots`-th.
template <typename T, int MT, int RT>
__global__ __launch_bounds__(kThreads) void k_lora_dot(const T* __restrict__ Z, int64_t ldz, const T* __restrict__ M,
                                                       int64_t G, int r, int len, const int32_t* __restrict__ ids,
                                                       int64_t s, int tiles, int slots, int splits,
                                                       float* __restrict__ P) {
    constexpr int TOK = 16 * MT;
    __shared__ v4f join[2][MT * RT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
    const int slot = blockIdx.x % slots, tile = blockIdx.x / slots % tiles, part = blockIdx.x / slots / tiles;
    const int64_t first = static_cast<int64_t>(tile) * TOK;
    const int steps = len / 64, w = part * kWaves + wave, all = splits * kWaves;
    const int k0 = static_cast<int>(static_cast<int64_t>(steps) * w / all) * 64;
    const int k1 = static_cast<int>(static_cast<int64_t>(steps) * (w + 1) / all) * 64;
    P += static_cast<int64_t>(part) * s * r;

    const T* z[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t i = first + t * 16 + n;
        z[t] = Z + (i < s ? i : s - 1) * ldz + q * 8;
    }
    Adapters<TOK> adapters(ids, first, s, G);
    if (slot == 0 && wave == 0) {        // rows without an adapter
        for (int t = 0; t < TOK; ++t) {
            const int64_t i = first + t;
            if ((adapters.left >> t & 1) == 0 && i < s)
                for (int k = lane; k < r; k += 64) P[i * r + k] = 0.0f;
        }
    }
    for (int turn = 0; adapters.left; ++turn) {
        uint64_t tokens;
        const int64_t g = adapters.next(tokens);
        if (turn % slots != slot) continue;
        const T* m[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int k = t * 16 + n < r ? t * 16 + n : r - 1;
            m[t] = M + (g * r + k) * len + q * 8;
        }
        v4f sum[MT][RT];
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < RT; ++b) sum[a][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = k0; k < k1; k += 64) {
            Vec<T> zv[2][MT], mv[2][RT];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int t = 0; t < MT; ++t) zv[u][t] = load16(z[t] + k + u * 32);
#pragma unroll
                for (int t = 0; t < RT; ++t) mv[u][t] = load16(m[t] + k + u * 32);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b < RT; ++b) sum[a][b] = mma(mv[u][b], zv[u][a], sum[a][b]);
        }
        // wavefronts 2 and 3 to 0 and 1, then 1 to 0
#pragma unroll
        for (int half = 2; half >= 1; half /= 2) {
            __syncthreads();
            if (wave >= half && wave < 2 * half) {
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b < RT; ++b) join[wave - half][a * RT + b][lane] = sum[a][b];
            }
            __syncthreads();
            if (wave < half) {
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b < RT; ++b) sum[a][b] += join[wave][a * RT + b][lane];
            }
        }
        if (wave == 0) {
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                if ((tokens >> (a * 16 + n) & 1) == 0) continue;
                float* p = P + (first + a * 16 + n) * r;
#pragma unroll
                for (int b = 0; b < RT; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int k = b * 16 + q * 4 + e;
                        if (k < r) p[k] = sum[a][b][e];
                    }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// add: out_i = base_i + f_g P_i M_g, with P the sum over the splits, which the
// blocks of the first columns also write to T.
//
// A block takes TOK = 16 MT tokens and 512 columns. It first joins the splits
// of its tokens' P and lays their two parts out in LDS, once for its four
// wavefronts: [token][16 ranks][first parts, second parts], so that one matrix
// instruction of 32 products takes 16 ranks with both parts. Each wavefront
// then takes 128 columns: M's rows are read 16 bytes a lane (eight columns of
// one rank) and turned in registers, so that the columns are the rows of the
// matrix instruction. The lane of row m reads the columns from
// (m % 4 * 4 + m / 4) * 8: a lane's four sums of one instruction then belong
// to four groups of eight columns 32 apart, and each group leaves as one
// 16-byte store beside its neighbours'.
constexpr int kAddColumns = kWaves * 128;

template <typename T, int MT>
__global__ __launch_bounds__(kThreads) void k_lora_add(const float* __restrict__ P, int splits,
                                                       const T* __restrict__ M, int64_t G, int r, int len,
                                                       const int32_t* __restrict__ ids,
                                                       const float* __restrict__ scale, const T* base, int64_t ldb,
                                                       T* out, int64_t ldo, int64_t s, int slots,
                                                       float* __restrict__ Tout) {
    constexpr int TOK = 16 * MT, PER = kThreads / TOK;      // PER threads a token lay out its parts
    extern __shared__ __align__(16) unsigned char lds[];
    const int steps = (r + 15) / 16, rp = steps * 16;
    T* parts = reinterpret_cast<T*>(lds);                               // [TOK][steps][32]
    float* values = reinterpret_cast<float*>(lds + TOK * rp * 4);       // [TOK][rp + 1]
    int* exps = reinterpret_cast<int*>(values + TOK * (rp + 1));        // [TOK]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
    const int col_blocks = (len + kAddColumns - 1) / kAddColumns;
    const int cb = blockIdx.x % col_blocks, slot = blockIdx.x / col_blocks % slots;
    const int64_t first = static_cast<int64_t>(blockIdx.x / col_blocks / slots) * TOK;
    Adapters<TOK> adapters(ids, first, s, G);
    {
        const int t = threadIdx.x / PER, sub = threadIdx.x % PER;
        const int64_t i = first + t;
        float most = 0.0f;
        for (int k = sub; k < rp; k += PER) {
            float v = 0.0f;
            if (k < r && i < s) {
                const float* p = P + i * r + k;
                for (int u = 0; u < splits; ++u) v += p[static_cast<int64_t>(u) * s * r];
                if (Tout && cb == 0 && slot == 0) Tout[i * r + k] = v;
            }
            values[t * (rp + 1) + k] = v;
            // NaN counts as infinity: no power of two for the row
            most = fmaxf(most, v == v ? fabsf(v) : __builtin_inff());
        }
#pragma unroll
        for (int off = 1; off < PER; off <<= 1) most = fmaxf(most, __shfl_xor(most, off, kWave));
        const int ex = scale_exponent<T>(most);
        if (sub == 0) exps[t] = ex;
        for (int k = sub; k < rp; k += PER) {
            T part[2];
            split<T, 2>(values[t * (rp + 1) + k], ex, part);
            T* to = parts + (t * steps + k / 16) * 32 + k % 16;
            to[0] = part[0];
            to[16] = part[1];
        }
    }
    __syncthreads();

    const int c0 = cb * kAddColumns + wave * 128;           // the wavefront's first column
    if (c0 >= len) return;
    const int mc = c0 + ((n & 3) * 4 + (n >> 2)) * 8;       // the columns that this lane reads of M
    const int mcol = mc < len ? mc : c0;
    const auto write = [&](int64_t i, const v4f(&sum)[8], float factor, int ex) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int col = c0 + e * 32 + q * 8;
            if (col >= len) continue;
            Vec<T> b{}, y;
            if (base) b = load16(base + i * ldb + col);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = from_float<T>(to_float<T>(b[j]) + ldexpf(sum[j][e], -ex) * factor);
            *reinterpret_cast<Vec<T>*>(out + i * ldo + col) = y;
        }
    };
    if (slot == 0 && out != base) {      // rows without an adapter are base's
#pragma unroll
        for (int a = 0; a < MT; ++a) {
            const int64_t i = first + a * 16 + n;
            if ((adapters.left >> (a * 16 + n) & 1) == 0 && i < s) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int col = c0 + e * 32 + q * 8;
                    if (col >= len) continue;
                    Vec<T> b{};
                    if (base) b = load16(base + i * ldb + col);
                    *reinterpret_cast<Vec<T>*>(out + i * ldo + col) = b;
                }
            }
        }
    }
    for (int turn = 0; adapters.left; ++turn) {
        uint64_t tokens;
        const int64_t g = adapters.next(tokens);
        if (turn % slots != slot) continue;
        v4f sum[MT][8];
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[a][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int st = 0; st < steps; ++st) {
            const int k0 = st * 16 + (q & 1) * 8;           // this lane's eight ranks, of both parts alike
            Vec<T> rows[8], columns[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                rows[k] = Vec<T>{};
                if (k0 + k < r) rows[k] = load16(M + (g * r + k0 + k) * len + mcol);
            }
            transpose8<T>(rows, columns);
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                const Vec<T> p = load16(parts + ((a * 16 + n) * steps + st) * 32 + q * 8);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[a][j] = mma(columns[j], p, sum[a][j]);
            }
        }
        const float factor = scale[g];
#pragma unroll
        for (int a = 0; a < MT; ++a)
            if (tokens >> (a * 16 + n) & 1) write(first + a * 16 + n, sum[a], factor, exps[a * 16 + n]);
    }
}

// ---------------------------------------------------------------------------
// grad: the tokens in the order of their adapters, in chunks of up to KC
// tokens of one adapter.

struct Chunk {
    int32_t g;                       // the adapter, or -1 for an unused entry
    int32_t first;                   // into the ordered tokens
    int32_t count;
    int32_t tile;                    // first tile of 32 positions in the laid-out factors
    int32_t part;                    // partial sums of the chunk, or -1: the adapter's only one
};

struct Plan {
    int32_t* order;                  // [s]: the tokens, by adapter and then by place
    int32_t* count;                  // [G]: tokens of each adapter
    int32_t* part;                   // [G]: its first partial sums
    Chunk* chunks;                   // [slots]
    int slots;
};

constexpr int kPlanThreads = 1024;

// One block an adapter: it counts the tokens of lower adapters (C), how many
// of those there are (D) and its own (n), then lists its own in order. Its
// chunks start at entry C / KC + D, its positions at the next multiple of 32
// from C plus 32 D, its partial sums, if it has more than one chunk, at
// 2 C / KC: each leaves the adapters room whatever their counts, without one
// block knowing the others'. Unused entries up to the next adapter's are
// marked by this one.
__global__ __launch_bounds__(kPlanThreads) void k_lora_plan(const int32_t* __restrict__ ids, int s, int G, int KC,
                                                            Plan plan) {
    __shared__ int wave_counts[kPlanThreads / 64];
    __shared__ uint32_t seen[2048];
    __shared__ int totals[4];
    const int g = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int k = threadIdx.x; k < (G + 31) / 32; k += kPlanThreads) seen[k] = 0;
    if (threadIdx.x < 4) totals[threadIdx.x] = 0;
    __syncthreads();
    int lower = 0, own = 0, valid = 0;
    for (int i = threadIdx.x; i < s; i += kPlanThreads) {
        const int id = ids[i];
        if (id < 0 || id >= G) continue;
        ++valid;
        own += id == g;
        if (id < g) {
            ++lower;
            if ((seen[id >> 5] >> (id & 31) & 1) == 0) atomicOr(&seen[id >> 5], 1u << (id & 31));
        }
    }
    __syncthreads();
    int distinct = 0;
    for (int k = threadIdx.x; k < (G + 31) / 32; k += kPlanThreads) distinct += __popc(seen[k]);
    atomicAdd(&totals[0], lower);        // integers: any order gives the same sum
    atomicAdd(&totals[1], own);
    atomicAdd(&totals[2], valid);
    atomicAdd(&totals[3], distinct);
    __syncthreads();
    const int C = totals[0], n = totals[1], D = totals[3];
    const bool last = C + n == totals[2];
    const int used = (n + KC - 1) / KC, begin = C / KC + D;
    const int end = last ? plan.slots : (C + n) / KC + D + 1;
    if (threadIdx.x == 0) {
        plan.count[g] = n;
        plan.part[g] = static_cast<int>(2 * static_cast<int64_t>(C) / KC);
    }
    if (n > 0 || (g == 0 && totals[2] == 0)) {
        for (int k = begin + threadIdx.x; k < end; k += kPlanThreads) {
            const int c = k - begin;
            Chunk e{-1, 0, 0, 0, -1};
            if (c < used)
                e = Chunk{g, C + c * KC, n - c * KC < KC ? n - c * KC : KC, (C + 31) / 32 + D + c * (KC / 32),
                          used > 1 ? static_cast<int32_t>(2 * static_cast<int64_t>(C) / KC) + c : -1};
            plan.chunks[k] = e;
        }
    }
    if (n == 0) return;
    int before = C;
    for (int i0 = 0; i0 < s; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        const bool mine = i < s && ids[i] == g;
        const uint64_t vote = __ballot(mine);
        if (lane == 0) wave_counts[wave] = __popcll(vote);
        __syncthreads();
        int at = before, all = 0;
        for (int k = 0; k < kPlanThreads / 64; ++k) {
            if (k < wave) at += wave_counts[k];
            all += wave_counts[k];
        }
        if (mine) plan.order[at + __popcll(vote & ((1ull << lane) - 1))] = i;
        before += all;
        __syncthreads();
    }
}

// One of the two gradients: the streamed rows Z, the factors P ([splits][s][r],
// joined here) and what becomes of them.
struct Side {
    const void* Z;
    int64_t ldz;
    int len;
    const float* P;
    int splits;
    void* laid;                      // [tile of 32][RT][parts][16 ranks][32] of the element type
    int32_t* exps;                   // [slots][RT]
    float* out;                      // [G][r][len]
    float* part;                     // [.][r][len]
};

template <typename T>
constexpr int kParts = kScaled<T> ? 2 : 3;

// Lays f_g P out as the matrix instruction takes it: a block takes one chunk,
// 16 ranks and one side; a wavefront takes 32 tokens at a time, a lane eight
// of them for one rank.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_lora_lay(Side x, Side y, const float* __restrict__ scale, int64_t s,
                                                       int r, Plan plan) {
    __shared__ float red[kWaves];
    const Chunk c = plan.chunks[blockIdx.x];
    if (c.g < 0) return;
    const Side& side = blockIdx.z == 0 ? x : y;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
    const int rt = blockIdx.y, tiles = (r + 15) / 16, k = rt * 16 + n;
    const int steps = (c.count + 31) / 32;
    const float f = scale[c.g];
    const auto value = [&](int p) {
        float v = 0.0f;
        if (p < c.count && k < r) {
            const float* at = side.P + static_cast<int64_t>(plan.order[c.first + p]) * r + k;
            for (int u = 0; u < side.splits; ++u) v += at[static_cast<int64_t>(u) * s * r];
            v *= f;
        }
        return v;
    };
    int ex = 0;
    if constexpr (kScaled<T>) {
        float most = 0.0f;
        for (int st = wave; st < steps; st += kWaves) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = value(st * 32 + q * 8 + e);
                most = fmaxf(most, v == v ? fabsf(v) : __builtin_inff());
            }
        }
        most = wave_max(most);
        if (lane == 0) red[wave] = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) most = fmaxf(most, red[w]);
        ex = scale_exponent<T>(most);
        if (threadIdx.x == 0) side.exps[static_cast<int64_t>(blockIdx.x) * tiles + rt] = ex;
    }
    for (int st = wave; st < steps; st += kWaves) {
        Vec<T> out[kParts<T>];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            T part[kParts<T>];
            split<T, kParts<T>>(value(st * 32 + q * 8 + e), ex, part);
#pragma unroll
            for (int p = 0; p < kParts<T>; ++p) out[p][e] = part[p];
        }
        T* to = static_cast<T*>(side.laid) + (static_cast<int64_t>(c.tile + st) * tiles + rt) * kParts<T> * 512;
#pragma unroll
        for (int p = 0; p < kParts<T>; ++p) *reinterpret_cast<Vec<T>*>(to + p * 512 + n * 32 + q * 8) = out[p];
    }
}

// out_g[k, j] = sum over the chunk's tokens of f P[i, k] Z[i, j]: a block
// takes one chunk, up to RT tiles of 16 ranks and 128 columns of one side, its
// wavefronts every fourth 32 tokens. Z's rows are read 16 bytes a lane (eight
// columns of one token) and turned in registers; the ranks are the rows of
// the matrix instruction, so a lane ends with eight neighbouring columns of
// four ranks. Tokens past the end have factors of 0 and rows of 0.
template <typename T, int RT>
__global__ __launch_bounds__(kThreads) void k_lora_grad(Side x, Side y, int r, Plan plan) {
    __shared__ v4f join[2][RT * 8][64];
    const int xblocks = (x.len + 127) / 128, yblocks = (y.len + 127) / 128;
    const int cb = blockIdx.x % (xblocks + yblocks);
    const Chunk c = plan.chunks[blockIdx.x / (xblocks + yblocks)];
    if (c.g < 0) return;
    const Side& side = cb < xblocks ? x : y;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
    const int col = (cb < xblocks ? cb : cb - xblocks) * 128 + n * 8;
    const int tiles = (r + 15) / 16, rt0 = blockIdx.y * RT;
    const T* Z = static_cast<const T*>(side.Z) + (col < side.len ? col : 0);
    const T* laid = static_cast<const T*>(side.laid) + n * 32 + q * 8;
    const int32_t* order = plan.order + c.first;
    v4f sum[RT][8];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[t][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int steps = (c.count + 31) / 32;
    for (int st = wave; st < steps; st += kWaves) {
        Vec<T> rows[8], columns[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int p = st * 32 + q * 8 + e;
            rows[e] = Vec<T>{};
            if (p < c.count) rows[e] = load16(Z + static_cast<int64_t>(order[p]) * side.ldz);
        }
        Vec<T> f[RT][kParts<T>];
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int p = 0; p < kParts<T>; ++p) {
                f[t][p] = Vec<T>{};
                if (rt0 + t < tiles)
                    f[t][p] = load16(laid + ((static_cast<int64_t>(c.tile + st) * tiles + rt0 + t) * kParts<T> + p) * 512);
            }
        transpose8<T>(rows, columns);
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
    if (wave != 0 || col >= side.len) return;
    float* out = c.part < 0 ? side.out + static_cast<int64_t>(c.g) * r * side.len
                            : side.part + static_cast<int64_t>(c.part) * r * side.len;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        if (rt0 + t >= tiles) continue;
        int ex = 0;
        if constexpr (kScaled<T>)
            ex = side.exps[static_cast<int64_t>(blockIdx.x / (xblocks + yblocks)) * tiles + rt0 + t];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = (rt0 + t) * 16 + q * 4 + e;
            if (k >= r) continue;
            v4f lo, hi;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lo[j] = ldexpf(sum[t][j][e], -ex);
                hi[j] = ldexpf(sum[t][j + 4][e], -ex);
            }
            v4f* p = reinterpret_cast<v4f*>(out + static_cast<int64_t>(k) * side.len + col);
            p[0] = lo;
            p[1] = hi;
        }
    }
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

// Tokens a tile of dot and add: few tokens most likely carry many adapters, so
// small tiles, and blocks for each of them.
bool few(int64_t s) { return s <= 256; }
int slots_for(int64_t s) { return s <= 256 ? 16 : s <= 1024 ? 4 : 1; }

// Parts that dot splits len into: enough blocks for the chip, while each
// wavefront keeps at least four steps of 64.
int dot_splits(int64_t s, int64_t len, int64_t r) {
    const int64_t tok = few(s) ? 16 : r > 64 ? 32 : 64;
    const int64_t want = up(2 * kCus, up(s > 0 ? s : 1, tok)), most = len / 64 / 16;
    const int64_t n = want < most ? want : most;
    return static_cast<int>(n < 1 ? 1 : n > 32 ? 32 : n);
}

template <typename T>
hipError_t dot(const LoraArgs& a, const void* Z, int64_t ldz, const void* M, int64_t len, float* P,
               hipStream_t stream) {
    const auto go = [&](auto mt, auto rt) {
        constexpr int MT = decltype(mt)::value, RT = decltype(rt)::value;
        const int tiles = static_cast<int>(up(a.s, 16 * MT)), slots = slots_for(a.s);
        const int splits = dot_splits(a.s, len, a.r);
        k_lora_dot<T, MT, RT><<<static_cast<unsigned>(static_cast<int64_t>(tiles) * slots * splits), kThreads, 0,
                               stream>>>(static_cast<const T*>(Z), ldz, static_cast<const T*>(M), a.G, a.r,
                                         static_cast<int>(len), a.ids, a.s, tiles, slots, splits, P);
    };
    using std::integral_constant;
    const auto ranks = [&](auto mt) {
        if (a.r <= 16) go(mt, integral_constant<int, 1>());
        else if (a.r <= 32) go(mt, integral_constant<int, 2>());
        else if (a.r <= 64) go(mt, integral_constant<int, 4>());
    };
    if (a.r > 64) {
        if (few(a.s)) go(integral_constant<int, 1>(), integral_constant<int, 8>());
        else go(integral_constant<int, 2>(), integral_constant<int, 8>());
    } else if (few(a.s)) {
        ranks(integral_constant<int, 1>());
    } else {
        ranks(integral_constant<int, 4>());
    }
    return hipGetLastError();
}

template <typename T>
hipError_t add(const LoraArgs& a, const float* P, int splits, const void* M, int64_t len, const void* base,
               int64_t ldb, void* out, int64_t ldo, float* Tout, hipStream_t stream) {
    const auto go = [&](auto mt) {
        constexpr int MT = decltype(mt)::value;
        const int64_t tiles = up(a.s, 16 * MT), rp = up(a.r, 16) * 16;
        const int slots = slots_for(a.s);
        const size_t lds = 16 * MT * (rp * 4 + (rp + 1) * 4 + 4);
        k_lora_add<T, MT><<<static_cast<unsigned>(tiles * slots * up(len, kAddColumns)), kThreads, lds, stream>>>(
            P, splits, static_cast<const T*>(M), a.G, a.r, static_cast<int>(len), a.ids, a.scale,
            static_cast<const T*>(base), ldb, static_cast<T*>(out), ldo, a.s, slots, Tout);
    };
    if (few(a.s)) go(std::integral_constant<int, 1>());
    else go(std::integral_constant<int, 2>());
    return hipGetLastError();
}

template <typename T>
hipError_t forward(const LoraArgs& a, const void* X, int64_t ldx, const void* base, int64_t ldb, void* Y, int64_t ldy,
                   float* Tp, void* workspace, hipStream_t stream) {
    const int splits = dot_splits(a.s, a.h, a.r);
    float* P = splits == 1 && Tp ? Tp : static_cast<float*>(workspace);
    const hipError_t e = dot<T>(a, X, ldx, a.A, a.h, P, stream);
    if (e != hipSuccess) return e;
    return add<T>(a, P, splits, a.B, a.o, base, ldb, Y, ldy, P == Tp ? nullptr : Tp, stream);
}

// The backward pass's workspace.
struct Layout {
    int KC, slots;
    int64_t tiles, parts;            // tiles of 32 positions; partial sums
    size_t P, order, count, part, chunks, laid[2], exps[2], sums[2], total;
};

Layout layout(int64_t s, int64_t h, int64_t o, int64_t r, int64_t G) {
    Layout l;
    // chunks as long as still leave about 1024 blocks
    const int64_t blocks = (up(h, 128) + up(o, 128)) * up(r, 64);
    const int64_t splits = up(4 * kCus, blocks);
    const int64_t kc = up(up(s > 0 ? s : 1, splits), 128) * 128;
    l.KC = static_cast<int>(kc);
    const int64_t groups = G < s ? G : s, rt = up(r, 16);
    l.slots = static_cast<int>(s / kc + groups + 1);
    l.tiles = up(s, 32) + groups + 1;
    l.parts = kc < s ? 2 * s / kc + 1 : 0;
    size_t at = 0;
    const auto take = [&](int64_t bytes) {
        const size_t p = at;
        at += static_cast<size_t>(up(bytes, 256) * 256);
        return p;
    };
    l.P = take(4 * dot_splits(s, o, r) * s * r);
    l.order = take(4 * s);
    l.count = take(4 * G);
    l.part = take(4 * G);
    l.chunks = take(static_cast<int64_t>(sizeof(Chunk)) * l.slots);
    for (int k = 0; k < 2; ++k) {
        l.laid[k] = take(l.tiles * rt * 3 * 512 * 2);
        l.exps[k] = take(4 * l.slots * rt);
        l.sums[k] = take(4 * l.parts * r * (k == 0 ? h : o));
    }
    l.total = at;
    return l;
}

template <typename T>
hipError_t backward(const LoraArgs& a, const void* dY, int64_t lddy, const void* X, int64_t ldx, const float* Tp,
                    const void* base, int64_t ldb, void* dX, int64_t lddx, float* dA, float* dB, void* workspace,
                    hipStream_t stream) {
    const Layout l = layout(a.s, a.h, a.o, a.r, a.G);
    char* ws = static_cast<char*>(workspace);
    const Plan plan{reinterpret_cast<int32_t*>(ws + l.order), reinterpret_cast<int32_t*>(ws + l.count),
                    reinterpret_cast<int32_t*>(ws + l.part), reinterpret_cast<Chunk*>(ws + l.chunks), l.slots};
    float* P = reinterpret_cast<float*>(ws + l.P);
    const int splits = dot_splits(a.s, a.o, a.r);
    const auto side = [&](int k, const void* Z, int64_t ldz, int64_t len, const float* p, int n, float* out) {
        return Side{Z, ldz, static_cast<int>(len), p, n, ws + l.laid[k], reinterpret_cast<int32_t*>(ws + l.exps[k]),
                    out, reinterpret_cast<float*>(ws + l.sums[k])};
    };
    const Side x = side(0, X, ldx, a.h, P, splits, dA), y = side(1, dY, lddy, a.o, Tp, 1, dB);
    const int r = a.r;
    k_lora_plan<<<static_cast<unsigned>(a.G), kPlanThreads, 0, stream>>>(a.ids, static_cast<int>(a.s),
                                                                        static_cast<int>(a.G), l.KC, plan);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.s > 0) {
        if ((e = dot<T>(a, dY, lddy, a.B, a.o, P, stream)) != hipSuccess) return e;
        if (dX && (e = add<T>(a, P, splits, a.A, a.h, base, ldb, dX, lddx, nullptr, stream)) != hipSuccess) return e;
        const unsigned rt = static_cast<unsigned>(up(r, 16)), slots = static_cast<unsigned>(l.slots);
        k_lora_lay<T><<<dim3(slots, rt, 2), kThreads, 0, stream>>>(x, y, a.scale, a.s, r, plan);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        const auto go = [&](auto n) {
            constexpr int RT = decltype(n)::value;
            const unsigned blocks = static_cast<unsigned>(up(a.h, 128) + up(a.o, 128));
            k_lora_grad<T, RT><<<dim3(slots * blocks, static_cast<unsigned>(up(rt, RT))), kThreads, 0, stream>>>(
                x, y, r, plan);
        };
        if (rt == 1) go(std::integral_constant<int, 1>());
        else if (rt == 2) go(std::integral_constant<int, 2>());
        else go(std::integral_constant<int, 4>());
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int64_t fours = static_cast<int64_t>(r) * (a.h + a.o) / 4;
    k_lora_grad_sum<<<dim3(static_cast<unsigned>(up(fours, kThreads)), static_cast<unsigned>(a.G)), kThreads, 0,
                      stream>>>(x, y, r, l.KC, plan);
    return hipGetLastError();
}

}  // namespace

size_t lora_forward_scratch(int64_t s, int64_t h, int64_t, int64_t r) {
    return 4 * static_cast<size_t>(dot_splits(s, h, r)) * s * r;
}

size_t lora_backward_scratch(int64_t s, int64_t h, int64_t o, int64_t r, int64_t G) {
    return layout(s, h, o, r, G).total;
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
