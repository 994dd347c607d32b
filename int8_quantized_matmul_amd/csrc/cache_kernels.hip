// A paged key-value cache: rows appended to their pages, sequences forked,
// freed and grown, and the pages in use moved to the front of the pool.
//
// What is decided is integers alone: which pages a sequence holds, how many
// sequences hold a page, which page is taken next (the lowest free one, in the
// order of the sequences), so results do not depend on the order in which
// threads run. What takes time is memory: rows and whole pages are copied in
// 16-byte pieces.

#include "launch.h"

#include "device_common.h"

namespace i8mm {
namespace {

constexpr int kThreads = 256;
constexpr int kPlanThreads = 1024;

unsigned blocks_for(int64_t threads, int64_t most) {
    const int64_t b = (threads + kThreads - 1) / kThreads;
    return static_cast<unsigned>(b < 1 ? 1 : b < most ? b : most);
}

// ---------------------------------------------------------------- append

// Sixteen bytes of a row of K or V each; `pieces` of a row's two tensors.
__global__ __launch_bounds__(kThreads) void k_append(const AppendArgs a, int pieces, int per_head) {
    const int64_t total = a.s * 2 * pieces;
    const int64_t head_bytes = static_cast<int64_t>(a.page) * per_head * 16;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; t < total;
         t += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t i = t / (2 * pieces);
        int c = static_cast<int>(t - i * (2 * pieces));
        const bool value = c >= pieces;
        if (value) c -= pieces;
        const int64_t seq = a.seq ? a.seq[i] : i;
        const int pos = a.pos[i];
        if (seq < 0 || seq >= a.n || pos < 0 || pos / a.page >= a.max_pages) continue;
        const int id = a.tables[seq * a.ldt + pos / a.page];
        if (id < 0 || id >= a.n_pages) continue;
        const char* row = static_cast<const char*>(value ? a.V : a.K) + i * (value ? a.ldv : a.ldk) * a.element_bytes;
        char* page = static_cast<char*>(value ? a.V_pages : a.K_pages) +
                     id * (value ? a.v_stride : a.k_stride) * a.element_bytes;
        const int head = c / per_head, f = c - head * per_head;
        *reinterpret_cast<v4u*>(page + head * head_bytes + (static_cast<int64_t>(pos % a.page) * per_head + f) * 16) =
            *reinterpret_cast<const v4u*>(row + static_cast<int64_t>(c) * 16);
    }
}

// ---------------------------------------------------------------- copies of whole pages

constexpr int kBatch = 128;              // pools a launch: 24 bytes each, within 4 KB of launch arguments
constexpr int kPieceBytes = kThreads * 64;

struct PoolBatch {
    char* at[kBatch];
    int64_t stride[kBatch];
    int32_t pieces16[kBatch];            // 16-byte pieces of a page
    int32_t first[kBatch];               // the pool's first block-sized piece of a page
    int32_t n, pieces;                   // pools; block-sized pieces of a page over all of them
};

// Page src[k] to page dst[k] in every pool, for k < *count.
__global__ __launch_bounds__(kThreads) void k_copy_pages(const PoolBatch b, const int32_t* __restrict__ src,
                                                         const int32_t* __restrict__ dst,
                                                         const int32_t* __restrict__ count) {
    const int64_t items = static_cast<int64_t>(*count) * b.pieces;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t k = item / b.pieces;
        const int piece = static_cast<int>(item - k * b.pieces);
        int lo = 0, hi = b.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (b.first[mid] <= piece) lo = mid;
            else hi = mid - 1;
        }
        const int64_t from = src[k], to = dst[k];
        const int64_t first = static_cast<int64_t>(piece - b.first[lo]) * (kPieceBytes / 16);
        const v4u* x = reinterpret_cast<const v4u*>(b.at[lo] + from * b.stride[lo]) + first;
        v4u* y = reinterpret_cast<v4u*>(b.at[lo] + to * b.stride[lo]) + first;
        const int64_t left = b.pieces16[lo] - first;
        v4u v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int j = q * kThreads + threadIdx.x;
            if (j < left) v[q] = x[j];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int j = q * kThreads + threadIdx.x;
            if (j < left) y[j] = v[q];
        }
    }
}

hipError_t copy_pages(const Pools& pools, const int32_t* src, const int32_t* dst, const int32_t* count, int64_t most,
                      hipStream_t stream) {
    PoolBatch b;
    for (int64_t i = 0; i < pools.n && most > 0;) {
        int64_t pieces = 0;
        for (b.n = 0; i < pools.n && b.n < kBatch; ++i) {
            const int64_t more = (pools.bytes[i] + kPieceBytes - 1) / kPieceBytes;
            if (more == 0) continue;
            b.at[b.n] = static_cast<char*>(pools.at[i]);
            b.stride[b.n] = pools.strides[i];
            b.pieces16[b.n] = static_cast<int32_t>(pools.bytes[i] / 16);
            b.first[b.n] = static_cast<int32_t>(pieces);
            ++b.n;
            pieces += more;
        }
        if (b.n == 0) break;
        b.pieces = static_cast<int32_t>(pieces);
        k_copy_pages<<<static_cast<unsigned>(most * pieces < 2048 ? most * pieces : 2048), kThreads, 0, stream>>>(b, src, dst,
                                                                                                               count);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// ---------------------------------------------------------------- fork

struct ForkScratch {
    int32_t *children;                   // [n] new sequences of each old one
    int32_t *keeper, *growing;           // [n_pages] last sequence that writes on in a page, and how many do
    int32_t *base;                       // [n_out] a sequence's first fresh page, -1 if it does not grow
    int32_t *fresh;                      // [n_pages] the free pages taken
    int32_t *copied;                     // [n_out] the sequence takes a copy of its last page
    int32_t *src, *dst, *count;          // the copies
};

__device__ __forceinline__ int clamped_len(const ForkArgs& a, int64_t i) {
    const int len = a.lens[i], most = a.max_pages * a.page;
    return len < 0 ? 0 : len < most ? len : most;
}

// The old sequence that new sequence j goes on from, or -1.
__device__ __forceinline__ int64_t parent_of(const ForkArgs& a, int64_t j) {
    const int64_t p = a.parents ? a.parents[j] : j;
    return p >= 0 && p < a.n ? p : -1;
}

__device__ __forceinline__ int grown_by(const ForkArgs& a, int64_t j) {
    const int g = a.grow ? a.grow[j] : 0;
    return g > 0 ? g : 0;
}

// The page that new sequence j writes on in, or -1: its last one, if that is not full.
__device__ __forceinline__ int written_page(const ForkArgs& a, int64_t parent, int len, int grow) {
    if (parent < 0 || grow == 0 || len % a.page == 0) return -1;
    const int id = a.tables[parent * a.ldt + len / a.page];
    return id >= 0 && id < a.n_pages ? id : -1;
}

__global__ __launch_bounds__(kThreads) void k_fork_init(const ForkArgs a, const ForkScratch w) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads, t0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    for (int64_t p = t0; p < a.n_pages; p += step) {
        a.refs_out[p] = a.refs[p];
        w.keeper[p] = -1;
        w.growing[p] = 0;
    }
    for (int64_t i = t0; i < a.n; i += step) w.children[i] = 0;
}

__global__ __launch_bounds__(kThreads) void k_fork_children(const ForkArgs a, const ForkScratch w) {
    for (int64_t j = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; j < a.n_out;
         j += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t p = parent_of(a, j);
        if (p >= 0) atomicAdd(&w.children[p], 1);
        const int id = p < 0 ? -1 : written_page(a, p, clamped_len(a, p), grown_by(a, j));
        if (id >= 0) {
            atomicMax(&w.keeper[id], static_cast<int>(j));
            atomicAdd(&w.growing[id], 1);
        }
    }
}

// The pages of an old sequence are held once more by each child, once less by itself.
__global__ __launch_bounds__(kThreads) void k_fork_share(const ForkArgs a, const ForkScratch w) {
    for (int64_t i = blockIdx.x; i < a.n; i += gridDim.x) {
        const int more = w.children[i] - 1;
        if (more == 0) continue;
        const int used = (clamped_len(a, i) + a.page - 1) / a.page;
        for (int c = threadIdx.x; c < used; c += kThreads) {
            const int id = a.tables[i * a.ldt + c];
            if (id >= 0 && id < a.n_pages) atomicAdd(&a.refs_out[id], more);
        }
    }
}

// The sum of v over the threads before this one, and over all of them.
__device__ __forceinline__ int block_scan(int v, int* s_sum, int* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int upto = wave_inclusive_scan(v, lane);
    if (lane == 63) s_sum[wave] = upto;
    __syncthreads();
    int before = 0, all = 0;
    for (int k = 0; k < waves; ++k) {
        if (k < wave) before += s_sum[k];
        all += s_sum[k];
    }
    __syncthreads();
    *total = all;
    return before + upto - v;
}

// One block: what each sequence gets, which pages those are, and the copies.
__global__ __launch_bounds__(kPlanThreads) void k_fork_plan(const ForkArgs a, const ForkScratch w) {
    __shared__ int s_sum[kPlanThreads / 64];
    int free_pages = 0;
    for (int p0 = 0; p0 < a.n_pages; p0 += kPlanThreads) {
        const int64_t p = static_cast<int64_t>(p0) + threadIdx.x;
        int all;
        block_scan(p < a.n_pages && a.refs_out[p] <= 0, s_sum, &all);
        free_pages += all;
    }
    int64_t wanted = 0;
    int taken = 0, copies = 0, missed = 0;
    for (int64_t j0 = 0; j0 < a.n_out; j0 += kPlanThreads) {
        const int64_t j = j0 + threadIdx.x;
        int want = 0, len = 0, copy = 0, ok = 1, page = -1, grow = 0;
        if (j < a.n_out) {
            const int64_t parent = parent_of(a, j);
            len = parent < 0 ? 0 : clamped_len(a, parent);
            grow = grown_by(a, j);
            page = written_page(a, parent, len, grow);
            copy = page >= 0 && !(w.keeper[page] == j && w.growing[page] >= a.refs_out[page]);
            ok = grow <= a.max_pages * a.page - len;
            if (ok) want = (len + grow + a.page - 1) / a.page - (len + a.page - 1) / a.page + copy;
        }
        // sums stay below 2^31: 1024 sequences of at most 2^20 pages each are taken at a time
        int all;
        const int64_t before = wanted + block_scan(want, s_sum, &all);
        wanted += all;
        if (want > 0 && before + want > free_pages) ok = 0;
        copy = ok ? copy : 0;
        int n;
        const int at = copies + block_scan(copy, s_sum, &n);
        copies += n;
        block_scan(!ok, s_sum, &n);
        missed += n;
        block_scan(ok ? want : 0, s_sum, &n);
        taken += n;
        if (j < a.n_out) {
            w.base[j] = ok ? static_cast<int>(before < free_pages ? before : free_pages) : -1;
            w.copied[j] = copy;
            a.lens_out[j] = ok ? len + grow : len;
            if (copy) {
                w.src[at] = page;
                w.dst[at] = static_cast<int>(before);      // its place among the fresh pages, named below
            }
        }
    }
    // the first `taken` free pages
    for (int p0 = 0, found = 0; p0 < a.n_pages && found < taken; p0 += kPlanThreads) {
        const int64_t p = static_cast<int64_t>(p0) + threadIdx.x;
        const int is = p < a.n_pages && a.refs_out[p] <= 0;
        int all;
        const int at = found + block_scan(is, s_sum, &all);
        found += all;
        if (is && at < taken) {
            w.fresh[at] = static_cast<int>(p);
            a.refs_out[p] = 1;
        }
    }
    __threadfence_block();
    __syncthreads();
    for (int k = threadIdx.x; k < copies; k += kPlanThreads) {
        w.dst[k] = w.fresh[w.dst[k]];
        atomicSub(&a.refs_out[w.src[k]], 1);
    }
    if (threadIdx.x == 0) {
        *w.count = copies;
        a.state[0] = free_pages - taken;
        const int64_t less = wanted - free_pages;
        a.state[1] = less < 0 ? 0 : less > 0x7fffffff ? 0x7fffffff : static_cast<int>(less);
        a.state[2] = missed;
        a.state[3] = copies;
    }
}

__global__ __launch_bounds__(kThreads) void k_fork_tables(const ForkArgs a, const ForkScratch w) {
    for (int64_t j = blockIdx.x; j < a.n_out; j += gridDim.x) {
        const int64_t parent = parent_of(a, j);
        const int len = parent < 0 ? 0 : clamped_len(a, parent);
        const int used = (len + a.page - 1) / a.page, now = (a.lens_out[j] + a.page - 1) / a.page;
        const int base = w.base[j], copied = w.copied[j];
        for (int c = threadIdx.x; c < a.max_pages; c += kThreads) {
            int id = -1;
            if (c < used) id = copied && c == used - 1 ? w.fresh[base] : a.tables[parent * a.ldt + c];
            else if (c < now) id = w.fresh[base + copied + c - used];
            a.tables_out[j * a.ldto + c] = id;
        }
    }
}

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

// ---------------------------------------------------------------- compact

constexpr int kTilePages = 4096;

struct CompactScratch {
    int32_t *counts;                     // pages in use of each tile
    int32_t *rank;                       // [n_pages]: see k_compact_place
    int32_t *src, *dst, *count;          // the moves
};

__device__ __forceinline__ int block_sum(int v, int* s_sum) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = v;
    __syncthreads();
    int t = 0;
    for (int k = 0; k < kThreads / 64; ++k) t += s_sum[k];
    __syncthreads();
    return t;
}

__device__ __forceinline__ int live_between(const int32_t* refs, int64_t from, int64_t to, int* s_sum) {
    int n = 0;
    for (int64_t p = from + threadIdx.x; p < to; p += kThreads) n += refs[p] > 0;
    return block_sum(n, s_sum);
}

__global__ __launch_bounds__(kThreads) void k_compact_count(const CompactArgs a, const CompactScratch w) {
    __shared__ int s_sum[kThreads / 64];
    const int64_t from = static_cast<int64_t>(blockIdx.x) * kTilePages;
    const int64_t to = from + kTilePages < a.n_pages ? from + kTilePages : a.n_pages;
    const int n = live_between(a.refs, from, to, s_sum);
    if (threadIdx.x == 0) w.counts[blockIdx.x] = n;
}

// With n pages in use: page p in use stays if p < n (rank p); else it is the
// k-th to move (rank -2 - k), to the k-th free page below n. Free: rank -1.
__global__ __launch_bounds__(kThreads) void k_compact_place(const CompactArgs a, const CompactScratch w) {
    __shared__ int s_sum[kThreads / 64];
    const int tiles = gridDim.x, tile = blockIdx.x;
    int before = 0, all = 0;
    for (int t = threadIdx.x; t < tiles; t += kThreads) {
        all += w.counts[t];
        if (t < tile) before += w.counts[t];
    }
    before = block_sum(before, s_sum);
    const int n = block_sum(all, s_sum);
    const int edge = n / kTilePages;                 // the tile that n lies in (none if every page is in use)
    int below = 0;
    for (int t = threadIdx.x; t < tiles && t < edge; t += kThreads) below += w.counts[t];
    below = block_sum(below, s_sum);
    below += live_between(a.refs, static_cast<int64_t>(edge) * kTilePages, n, s_sum);
    if (tile == 0 && threadIdx.x == 0) {
        a.state[0] = n;
        a.state[1] = n - below;
        *w.count = n - below;
    }
    const int64_t from = static_cast<int64_t>(tile) * kTilePages;
    for (int64_t p0 = from; p0 < from + kTilePages && p0 < a.n_pages; p0 += kThreads) {
        const int64_t p = p0 + threadIdx.x;
        const int refs = p < a.n_pages ? a.refs[p] : 0, live = refs > 0;
        int m;
        const int at = before + block_scan(live, s_sum, &m);
        before += m;
        if (p >= a.n_pages) continue;
        int rank = -1;
        if (p < n) {
            if (live) {
                rank = static_cast<int>(p);
                a.refs_out[p] = refs;
            } else {
                w.dst[p - at] = static_cast<int>(p);
            }
        } else {
            if (live) {
                rank = -2 - (at - below);
                w.src[at - below] = static_cast<int>(p);
            }
            a.refs_out[p] = 0;
        }
        w.rank[p] = rank;
    }
}

__device__ __forceinline__ int new_place(const CompactScratch& w, int p) {
    const int r = w.rank[p];
    return r <= -2 ? w.dst[-2 - r] : r;
}

__global__ __launch_bounds__(kThreads) void k_compact_apply(const CompactArgs a, const CompactScratch w) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads, t0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    for (int64_t p = t0; p < a.n_pages; p += step) {
        const int to = new_place(w, static_cast<int>(p));
        a.moved[p] = to;
        if (to >= 0 && to != p) a.refs_out[to] = a.refs[p];
    }
    const int64_t entries = a.n * a.max_pages;
    for (int64_t t = t0; t < entries; t += step) {
        const int64_t i = t / a.max_pages, c = t - i * a.max_pages;
        const int id = a.tables[i * a.ldt + c];
        a.tables_out[i * a.ldto + c] = id >= 0 && id < a.n_pages ? new_place(w, id) : id;
    }
}

}  // namespace

hipError_t launch_cache_append(const AppendArgs& a, hipStream_t stream) {
    if (a.s == 0) return hipSuccess;
    const int per_head = a.d * a.element_bytes / 16, pieces = a.kv_heads * per_head;
    k_append<<<blocks_for(a.s * 2 * pieces, 8192), kThreads, 0, stream>>>(a, pieces, per_head);
    return hipGetLastError();
}

size_t cache_fork_scratch(int64_t n, int64_t n_out, int64_t n_pages) {
    return static_cast<size_t>(round256(4 * n) + 3 * round256(4 * n_pages) + 4 * round256(4 * n_out) + 256);
}

hipError_t launch_cache_fork(const ForkArgs& a, const Pools& pools, void* workspace, hipStream_t stream) {
    char* at = static_cast<char*>(workspace);
    const auto take = [&at](int64_t count) {
        int32_t* p = reinterpret_cast<int32_t*>(at);
        at += round256(4 * count);
        return p;
    };
    ForkScratch w;
    w.children = take(a.n);
    w.keeper = take(a.n_pages);
    w.growing = take(a.n_pages);
    w.fresh = take(a.n_pages);
    w.base = take(a.n_out);
    w.copied = take(a.n_out);
    w.src = take(a.n_out);
    w.dst = take(a.n_out);
    w.count = take(1);
    k_fork_init<<<blocks_for(a.n_pages > a.n ? a.n_pages : a.n, 1024), kThreads, 0, stream>>>(a, w);
    k_fork_children<<<blocks_for(a.n_out, 1024), kThreads, 0, stream>>>(a, w);
    k_fork_share<<<blocks_for(a.n * kThreads, 2048), kThreads, 0, stream>>>(a, w);
    k_fork_plan<<<1, kPlanThreads, 0, stream>>>(a, w);
    k_fork_tables<<<blocks_for(a.n_out * kThreads, 2048), kThreads, 0, stream>>>(a, w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return copy_pages(pools, w.src, w.dst, w.count, a.grow ? a.n_out : 0, stream);
}

size_t cache_compact_scratch(int64_t n_pages) {
    return static_cast<size_t>(round256(4 * ((n_pages + kTilePages - 1) / kTilePages)) + 3 * round256(4 * n_pages) + 256);
}

hipError_t launch_cache_compact(const CompactArgs& a, const Pools& pools, void* workspace, hipStream_t stream) {
    char* at = static_cast<char*>(workspace);
    const auto take = [&at](int64_t count) {
        int32_t* p = reinterpret_cast<int32_t*>(at);
        at += round256(4 * count);
        return p;
    };
    const int tiles = (a.n_pages + kTilePages - 1) / kTilePages;
    CompactScratch w;
    w.counts = take(tiles);
    w.rank = take(a.n_pages);
    w.src = take(a.n_pages);
    w.dst = take(a.n_pages);
    w.count = take(1);
    k_compact_count<<<tiles, kThreads, 0, stream>>>(a, w);
    k_compact_place<<<tiles, kThreads, 0, stream>>>(a, w);
    const int64_t entries = a.n * a.max_pages;
    k_compact_apply<<<blocks_for(entries > a.n_pages ? entries : a.n_pages, 2048), kThreads, 0, stream>>>(a, w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return copy_pages(pools, w.src, w.dst, w.count, a.n_pages / 2, stream);
}

}  // namespace i8mm
