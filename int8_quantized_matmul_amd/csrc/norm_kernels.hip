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

#include <type_traits>

namespace i8mm {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kCus = 256;

// The sum of v over the TW threads of a row (whole wavefronts; a group of
// them for each row of the block), in each of them. red: one float for each
// wavefront of the block, not used again until every thread has passed
// another barrier. One wavefront needs neither LDS nor a barrier.
__device__ __forceinline__ float row_sum(float v, float* red, int waves) {
    v = wave_sum(v);
    if (waves == 1) return v;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    const int first = wave / waves * waves;
    float t = 0.0f;
    for (int k = 0; k < waves; ++k) t += red[first + k];
    return t;
}

// Two such sums with one barrier; red: two floats for each wavefront.
__device__ __forceinline__ void row_sum2(float& a, float& b, v2f* red, int waves) {
    a = wave_sum(a);
    b = wave_sum(b);
    if (waves == 1) return;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = v2f{a, b};
    __syncthreads();
    const int first = wave / waves * waves;
    a = b = 0.0f;
    for (int k = 0; k < waves; ++k) {
        const v2f t = red[first + k];
        a += t.x;
        b += t.y;
    }
}

// One row for each group of tw threads, held in registers between the single
// read of X and the single write of Y (NV groups of eight elements a thread).
// The variance is taken about the mean, from the registers. Bound by memory:
// 4096 x 12288 of fp16 takes 38-42 us, 4.8-5.2 TB/s of the bytes it has to
// move, where a large copy on this card reaches 4.9-5.1; 8 x 12288 takes 4.4-4.9
// us, two trips to memory and a launch.
template <typename T, typename W, int NV>
__global__ __launch_bounds__(kMaxThreads) void k_layer_norm(const T* X, int64_t ldx, int64_t s, int h, int tw,
                                                            const W* __restrict__ w, const W* __restrict__ b,
                                                            float eps, T* Y, int64_t ldy, float* __restrict__ mean,
                                                            float* __restrict__ rstd) {
    __shared__ float red[2][kMaxThreads / 64];
    const int t = threadIdx.x % tw, waves = tw / 64;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tw) + threadIdx.x / tw;
    const int left = row < s ? h : 0;              // a group past the last row only keeps the barriers
    const T* x = X + row * ldx;
    Eight<T> v[NV];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; ++c) v[c].load(x + (c * tw + t) * 8, left - (c * tw + t) * 8);
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += v[c].at(k);
    const float m = row_sum(sum, red[0], waves) / static_cast<float>(h);
    float sq = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int n = left - (c * tw + t) * 8;
        if (n >= 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) sq = fmaf(v[c].at(k) - m, v[c].at(k) - m, sq);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n) sq = fmaf(v[c].at(k) - m, v[c].at(k) - m, sq);
        }
    }
    const float r = 1.0f / sqrtf(row_sum(sq, red[1], waves) / static_cast<float>(h) + eps);
    if (left == 0) return;
    T* y = Y + row * ldy;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int j = (c * tw + t) * 8, n = h - j;
        if (n <= 0) break;
        Eight<W> wv, bv;
        wv.load(w + j, n);
        if (b) bv.load(b + j, n);
        Eight<T> out;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            out.set(k, fmaf((v[c].at(k) - m) * r, wv.at(k), b ? bv.at(k) : 0.0f));
        out.store(y + j, n);
    }
    if (t == 0) {
        if (mean) mean[row] = m;
        if (rstd) rstd[row] = r;
    }
}

// The same for rows that the registers of one block do not hold: three reads
// of the row, the later two mostly from cache.
template <typename T, typename W>
__global__ __launch_bounds__(kMaxThreads) void k_layer_norm_long(const T* X, int64_t ldx, int h,
                                                                 const W* __restrict__ w, const W* __restrict__ b,
                                                                 float eps, T* Y, int64_t ldy,
                                                                 float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float red[2][kMaxThreads / 64];
    const int64_t row = blockIdx.x;
    const T* x = X + row * ldx;
    T* y = Y + row * ldy;
    float sum = 0.0f;
    for (int j = threadIdx.x; j < h; j += kMaxThreads) sum += to_float(x[j]);
    const float m = row_sum(sum, red[0], kMaxThreads / 64) / static_cast<float>(h);
    float sq = 0.0f;
    for (int j = threadIdx.x; j < h; j += kMaxThreads) {
        const float d = to_float(x[j]) - m;
        sq = fmaf(d, d, sq);
    }
    const float r = 1.0f / sqrtf(row_sum(sq, red[1], kMaxThreads / 64) / static_cast<float>(h) + eps);
    for (int j = threadIdx.x; j < h; j += kMaxThreads) {
        const float n = (to_float(x[j]) - m) * r;
        y[j] = from_float<T>(fmaf(n, to_float(w[j]), b ? to_float(b[j]) : 0.0f));
    }
    if (threadIdx.x == 0) {
        if (mean) mean[row] = m;
        if (rstd) rstd[row] = r;
    }
}

// One pass over dY and X: dX, and this block's part of dw and db (part:
// [blocks][2][h]). A group of tw threads holds a row in registers (NV groups
// of eight elements a thread of each of dY and X), and each thread keeps the
// sums of its own columns over all the rows that its group meets; the block's
// groups join theirs in LDS at the end. A row's g and n stay in registers from
// its sums to its dX; the next row's loads are issued before the sums, so the
// barriers do not leave memory idle. One block a CU: every block more writes
// another 8 h bytes of sums. 4096 x 12288 of fp16: 62 us and 5 us for the sum
// over the blocks, 4.5 TB/s over both (two separate passes took 177 us; with
// two rows in flight 72 us; g and n computed twice instead of kept 81 us).
template <typename T, typename W, int NV, int MAXT, bool PARAMS>
__global__ __launch_bounds__(MAXT) void k_layer_norm_grad(const T* __restrict__ dY, int64_t lddy,
                                                          const T* __restrict__ X, int64_t ldx, int64_t s, int h,
                                                          int tw, const W* __restrict__ w,
                                                          const float* __restrict__ mean,
                                                          const float* __restrict__ rstd, T* __restrict__ dX,
                                                          int64_t lddx, float* __restrict__ part) {
    extern __shared__ float join[];                 // [h] if the block has more than one group
    __shared__ v2f red[2][kMaxThreads / 64];
    const int t = threadIdx.x % tw, waves = tw / 64, groups = blockDim.x / tw, group = threadIdx.x / tw;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    float dw[PARAMS ? NV : 1][8], db[PARAMS ? NV : 1][8];
#pragma unroll
    for (int c = 0; c < (PARAMS ? NV : 1); ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) dw[c][k] = db[c][k] = 0.0f;

    Eight<T> gy[NV], gx[NV];
    float m, r;
    const auto fetch = [&](int64_t row) {
        const int left = row < s ? h : 0;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int j = (c * tw + t) * 8;
            gy[c].load(dY + row * lddy + j, left - j);
            gx[c].load(X + row * ldx + j, left - j);
        }
        m = left ? mean[row] : 0.0f;
        r = left ? rstd[row] : 0.0f;
    };
    Eight<W> wv[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) wv[c].load(w + (c * tw + t) * 8, h - (c * tw + t) * 8);
    int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group;
    fetch(row);
    int turn = 0;
    // every group makes the same number of rounds, so that the barriers meet
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * groups; first < s; first += step, row += step) {
        float g[NV][8], n[NV][8], sg = 0.0f, sgn = 0.0f;
        const float m0 = m, r0 = r;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float dy = gy[c].at(k);
                g[c][k] = dy * wv[c].at(k);
                n[c][k] = (gx[c].at(k) - m0) * r0;
                if constexpr (PARAMS) {
                    dw[c][k] = fmaf(dy, n[c][k], dw[c][k]);
                    db[c][k] += dy;
                }
            }
        }
        fetch(row + step);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sg += g[c][k];
                sgn = fmaf(g[c][k], n[c][k], sgn);
            }
        }
        row_sum2(sg, sgn, red[turn], waves);
        turn ^= 1;                                  // this half is still being read during the next round
        if (row < s) {
            const float c0 = -r0 * (sg / static_cast<float>(h)), c1 = -r0 * (sgn / static_cast<float>(h));
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                const int j = (c * tw + t) * 8;
                if (j >= h) break;
                Eight<T> out;
#pragma unroll
                for (int k = 0; k < 8; ++k) out.set(k, fmaf(n[c][k], c1, fmaf(g[c][k], r0, c0)));
                out.store(dX + row * lddx + j, h - j);
            }
        }
    }
    if constexpr (PARAMS) {
        const auto join_groups = [&](float(&mine)[NV][8]) {
            for (int k = 1; k < groups; ++k) {      // groups 1, 2, ... add theirs to group 0's in this order
                __syncthreads();
#pragma unroll
                for (int c = 0; c < NV; ++c) {
                    const int j = (c * tw + t) * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (group == k && j + e < h) join[j + e] = mine[c][e];
                }
                __syncthreads();
#pragma unroll
                for (int c = 0; c < NV; ++c) {
                    const int j = (c * tw + t) * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (group == 0 && j + e < h) mine[c][e] += join[j + e];
                }
            }
        };
        join_groups(dw);
        join_groups(db);
        if (group == 0) {
            float* p = part + static_cast<int64_t>(blockIdx.x) * 2 * h;
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                const int j = (c * tw + t) * 8;
                Eight<float> a, b;
                for (int e = 0; e < 8; ++e) {
                    a.v[e] = dw[c][e];
                    b.v[e] = db[c][e];
                }
                a.store(p + j, h - j);
                b.store(p + h + j, h - j);
            }
        }
    }
}

// Rows that the registers do not hold: dX by one block a row, reading it
// twice, and the column sums by a second pass over both inputs. 4096 x 20480 of
// fp16: 179 and 106 us, where one pass at a copy's rate would take 101.
template <typename T, typename W>
__global__ __launch_bounds__(kMaxThreads) void k_layer_norm_dx_long(const T* __restrict__ dY, int64_t lddy,
                                                                    const T* __restrict__ X, int64_t ldx, int h,
                                                                    const W* __restrict__ w,
                                                                    const float* __restrict__ mean,
                                                                    const float* __restrict__ rstd,
                                                                    T* __restrict__ dX, int64_t lddx) {
    __shared__ float red[2][kMaxThreads / 64];
    const int64_t row = blockIdx.x;
    const T* x = X + row * ldx;
    const T* dy = dY + row * lddy;
    T* dx = dX + row * lddx;
    const float m = mean[row], r = rstd[row];
    float sg = 0.0f, sgn = 0.0f;
    for (int j = threadIdx.x; j < h; j += kMaxThreads) {
        const float g = to_float(dy[j]) * to_float(w[j]);
        sg += g;
        sgn = fmaf(g, (to_float(x[j]) - m) * r, sgn);
    }
    const float mg = row_sum(sg, red[0], kMaxThreads / 64) / static_cast<float>(h);
    const float mgn = row_sum(sgn, red[1], kMaxThreads / 64) / static_cast<float>(h);
    for (int j = threadIdx.x; j < h; j += kMaxThreads) {
        const float g = to_float(dy[j]) * to_float(w[j]);
        const float n = (to_float(x[j]) - m) * r;
        dx[j] = from_float<T>(r * (g - mg - n * mgn));
    }
}

constexpr int kColThreads = 256;

template <typename T>
__global__ __launch_bounds__(kColThreads) void k_layer_norm_dw_long(const T* __restrict__ dY, int64_t lddy,
                                                                    const T* __restrict__ X, int64_t ldx, int64_t s,
                                                                    int h, int64_t rows,
                                                                    const float* __restrict__ mean,
                                                                    const float* __restrict__ rstd,
                                                                    float* __restrict__ part) {
    const int j = blockIdx.x * kColThreads + threadIdx.x;
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

// dw and db from the parts: a block takes 64 columns of one of the two, each
// wavefront a quarter of the parts.
__global__ __launch_bounds__(kColThreads) void k_layer_norm_dw_sum(const float* __restrict__ part, int parts, int h,
                                                                   float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float red[3][64];
    float* out = blockIdx.y == 0 ? dw : db;
    if (!out) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int j = blockIdx.x * 64 + lane;
    const int p0 = parts * wave / 4, p1 = parts * (wave + 1) / 4;
    const float* p = part + static_cast<int64_t>(blockIdx.y) * h + j;
    float a = 0.0f;
    if (j < h) {
#pragma unroll 8
        for (int k = p0; k < p1; ++k) a += p[static_cast<int64_t>(k) * 2 * h];
    }
    if (wave > 0) red[wave - 1][lane] = a;
    __syncthreads();
    if (wave == 0 && j < h) out[j] = ((a + red[0][lane]) + red[1][lane]) + red[2][lane];
}

// Calls f with a null pointer of each of the two element types.
template <typename F>
hipError_t with_types(Dtype x, Dtype w, F&& f) {
    if (x == Dtype::F16) return w == Dtype::F32 ? f((_Float16*)0, (float*)0) : f((_Float16*)0, (_Float16*)0);
    if (x == Dtype::BF16) return w == Dtype::F32 ? f((__bf16*)0, (float*)0) : f((__bf16*)0, (__bf16*)0);
    return f((float*)0, (float*)0);
}

// Threads for a row of h elements at NV groups of eight each, in whole
// wavefronts.
int row_threads(int64_t h, int nv) {
    const int64_t eights = (h + 7) / 8;
    return static_cast<int>(((eights + nv - 1) / nv + 63) / 64 * 64);
}

// Calls f(first, n) for the s rows in runs of n whose grid, a block of
// `threads` for each `rows` of them, is one that can be launched.
template <typename F>
void for_rows(int64_t s, int rows, int threads, F&& f) {
    const int64_t most = kGridThreads / threads * rows;
    for (int64_t first = 0; first < s; first += most) f(first, s - first < most ? s - first : most);
}

}  // namespace

hipError_t launch_layer_norm(const void* X, int64_t ldx, Dtype xt, int64_t s, int64_t h, const void* w, const void* b,
                             Dtype wt, float eps, void* Y, int64_t ldy, float* mean, float* rstd,
                             hipStream_t stream) {
    if (s == 0) return hipSuccess;
    return with_types(xt, wt, [&](auto* tx, auto* tw) {
        using T = std::remove_pointer_t<decltype(tx)>;
        using W = std::remove_pointer_t<decltype(tw)>;
        const auto go = [&](auto nv) {
            constexpr int NV = decltype(nv)::value;
            const int threads = row_threads(h, NV);
            const int rows = threads >= 256 ? 1 : 256 / threads;      // rows of a block
            for_rows(s, rows, threads * rows, [&](int64_t first, int64_t n) {
                k_layer_norm<T, W, NV><<<static_cast<unsigned>((n + rows - 1) / rows), threads * rows, 0, stream>>>(
                    static_cast<const T*>(X) + first * ldx, ldx, n, static_cast<int>(h), threads,
                    static_cast<const W*>(w), static_cast<const W*>(b), eps, static_cast<T*>(Y) + first * ldy, ldy,
                    mean ? mean + first : nullptr, rstd ? rstd + first : nullptr);
            });
        };
        // Few rows (fewer than two a CU): as many threads as a row takes, for
        // latency. Otherwise 64 bytes a thread, so that short rows need one
        // wavefront and no barrier, and long ones keep several blocks a CU.
        // Measured, s x h of fp16: 8 x 12288 0.8 us more at 64 bytes a thread
        // than at 16 or 32; 4096 x 12288 42.4 at 32, 38.0 at 64, 40.2 at 128.
        int nv = s < 2 * kCus ? 1 : static_cast<int>(64 / (8 * sizeof(T)));
        while (nv <= 8 && row_threads(h, nv) > kMaxThreads) nv *= 2;
        if (nv == 1) go(std::integral_constant<int, 1>());
        else if (nv == 2) go(std::integral_constant<int, 2>());
        else if (nv == 4) go(std::integral_constant<int, 4>());
        else if (nv == 8) go(std::integral_constant<int, 8>());
        else
            for_rows(s, 1, kMaxThreads, [&](int64_t first, int64_t n) {
                k_layer_norm_long<T, W><<<static_cast<unsigned>(n), kMaxThreads, 0, stream>>>(
                    static_cast<const T*>(X) + first * ldx, ldx, static_cast<int>(h), static_cast<const W*>(w),
                    static_cast<const W*>(b), eps, static_cast<T*>(Y) + first * ldy, ldy,
                    mean ? mean + first : nullptr, rstd ? rstd + first : nullptr);
            });
        return hipGetLastError();
    });
}

int64_t layer_norm_backward_parts(int64_t s) { return s < kCus ? s : kCus; }

hipError_t launch_layer_norm_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, Dtype xt, int64_t s,
                                      int64_t h, const void* w, Dtype wt, const float* mean, const float* rstd,
                                      void* dX, int64_t lddx, float* dw, float* db, float* part, hipStream_t stream) {
    const bool params = dw || db;
    int64_t parts = layer_norm_backward_parts(s);
    if (s > 0) {
        const hipError_t e = with_types(xt, wt, [&](auto* tx, auto* tw) {
            using T = std::remove_pointer_t<decltype(tx)>;
            using W = std::remove_pointer_t<decltype(tw)>;
            const auto go = [&](auto nv, auto maxt, auto with) {
                constexpr int NV = decltype(nv)::value, MAXT = decltype(maxt)::value;
                constexpr bool PARAMS = decltype(with)::value;
                const int threads = row_threads(h, NV);
                int groups = MAXT / threads;
                while (groups > 1 && parts * (groups / 2) >= s) groups /= 2;
                const int64_t blocks = (s + groups - 1) / groups;
                parts = blocks < parts ? blocks : parts;
                const size_t lds = PARAMS && groups > 1 ? 4 * static_cast<size_t>(h) : 0;
                k_layer_norm_grad<T, W, NV, MAXT, PARAMS>
                    <<<static_cast<unsigned>(parts), threads * groups, lds, stream>>>(
                        static_cast<const T*>(dY), lddy, static_cast<const T*>(X), ldx, s, static_cast<int>(h),
                        threads, static_cast<const W*>(w), mean, rstd, static_cast<T*>(dX), lddx, part);
            };
            const auto pick = [&](auto nv, auto maxt) {
                if (params) go(nv, maxt, std::true_type());
                else go(nv, maxt, std::false_type());
            };
            using std::integral_constant;
            // The fewest columns a thread whose row fits a block; each NV with the most
            // threads whose registers hold its sums, g, n and the row in flight. fp32
            // rows beyond 12288 columns spill at that (4096 x 16384: 212 us for 805 MB,
            // 3.8 TB/s; fp16 83 us, 4.8 TB/s).
            if (row_threads(h, 1) <= 512) {
                pick(integral_constant<int, 1>(), integral_constant<int, 1024>());
            } else if (row_threads(h, 2) <= 768) {
                pick(integral_constant<int, 2>(), integral_constant<int, 768>());
            } else if (row_threads(h, 4) <= 512) {
                pick(integral_constant<int, 4>(), integral_constant<int, 512>());
            } else {
                for_rows(s, 1, kMaxThreads, [&](int64_t first, int64_t n) {
                    k_layer_norm_dx_long<T, W><<<static_cast<unsigned>(n), kMaxThreads, 0, stream>>>(
                        static_cast<const T*>(dY) + first * lddy, lddy, static_cast<const T*>(X) + first * ldx, ldx,
                        static_cast<int>(h), static_cast<const W*>(w), mean + first, rstd + first,
                        static_cast<T*>(dX) + first * lddx, lddx);
                });
                const int64_t rows = (s + parts - 1) / parts;
                if (params)
                    k_layer_norm_dw_long<T>
                        <<<dim3(static_cast<unsigned>((h + kColThreads - 1) / kColThreads),
                                static_cast<unsigned>(parts)),
                           kColThreads, 0, stream>>>(static_cast<const T*>(dY), lddy, static_cast<const T*>(X), ldx, s,
                                                     static_cast<int>(h), rows, mean, rstd, part);
            }
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    if (params) {
        k_layer_norm_dw_sum<<<dim3(static_cast<unsigned>((h + 63) / 64), 2), kColThreads, 0, stream>>>(
            part, static_cast<int>(parts), static_cast<int>(h), dw, db);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace i8mm
