// A paged key-value cache: rows appended to their pages, sequences forked,
// freed and grown, and the pages in use moved to the front of the pool.
//
// What is decided is integers alone: which pages a sequence holds, how many
// sequences hold a page, which page is taken next (the lowest free one, in the
// order of the sequences), so results do not depend on the order in which
// threads run. What takes time is memory: rows and whole pages are copied in
// 16-byte pieces.

#include "../../include/i8mm.h"
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

constexpr int kAppendEach = 4;           // pieces of 16 bytes that a thread has in flight

// A row's pieces are K's, then V's (`pieces` each), over all rows in one line. A block
// takes kThreads * kAppendEach neighbours: one division by the row's length for the
// block, 32-bit ones for its threads. Memory is the bound: five prompts with 10250 tokens
// of 32 heads (336 MB moved) 57 us on one cache, 66 on several in turn (5.1 TB/s); 82
// with one piece a thread, whose four loads depend on each other.
__global__ __launch_bounds__(kThreads) void k_append(const AppendArgs a, unsigned pieces, unsigned per_head) {
    const unsigned both = 2 * pieces;
    const int64_t total = a.s * both;
    const int64_t head_bytes = static_cast<int64_t>(a.page) * per_head * 16;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kThreads * kAppendEach; t0 < total;
         t0 += static_cast<int64_t>(gridDim.x) * kThreads * kAppendEach) {
        const int64_t row0 = t0 / both;
        const unsigned rest = static_cast<unsigned>(t0 - row0 * both);
        // each step for all of a thread's pieces before the next one, so that their loads are in flight together
        unsigned at[kAppendEach];
        int64_t row[kAppendEach], seq[kAppendEach];
        int pos[kAppendEach], id[kAppendEach];
        bool there[kAppendEach];
        v4u v[kAppendEach];
#pragma unroll
        for (int q = 0; q < kAppendEach; ++q) {
            const unsigned t = rest + q * kThreads + threadIdx.x;
            there[q] = t0 + (t - rest) < total;
            const unsigned down = t / both;
            row[q] = there[q] ? row0 + down : row0;
            at[q] = there[q] ? t - down * both : 0;
        }
#pragma unroll
        for (int q = 0; q < kAppendEach; ++q) {
            seq[q] = a.seq ? a.seq[row[q]] : row[q];
            pos[q] = a.pos[row[q]];
        }
#pragma unroll
        for (int q = 0; q < kAppendEach; ++q) {
            const unsigned c = at[q] < pieces ? at[q] : at[q] - pieces;
            const char* x = at[q] < pieces ? static_cast<const char*>(a.K) + row[q] * a.ldk * a.element_bytes
                                           : static_cast<const char*>(a.V) + row[q] * a.ldv * a.element_bytes;
            v[q] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(x) + c);
        }
#pragma unroll
        for (int q = 0; q < kAppendEach; ++q) {
            there[q] = there[q] && seq[q] >= 0 && seq[q] < a.n && pos[q] >= 0 && pos[q] / a.page < a.max_pages;
            id[q] = there[q] ? a.tables[seq[q] * a.ldt + pos[q] / a.page] : -1;
        }
#pragma unroll
        for (int q = 0; q < kAppendEach; ++q) {
            if (id[q] < 0 || id[q] >= a.n_pages) continue;
            const unsigned c = at[q] < pieces ? at[q] : at[q] - pieces;
            const unsigned head = c / per_head, f = c - head * per_head;
            char* page = at[q] < pieces ? static_cast<char*>(a.K_pages) + id[q] * a.k_stride * a.element_bytes
                                        : static_cast<char*>(a.V_pages) + id[q] * a.v_stride * a.element_bytes;
            *reinterpret_cast<v4u*>(page + head * head_bytes + (static_cast<int64_t>(pos[q] % a.page) * per_head + f) * 16) = v[q];
        }
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

// One block's piece of the copy of page `from` to page `to`. Through: past the caches, for
// what is not read again soon (a compaction that moves 370 MB takes 152 us so, 4.9 TB/s
// read and written, and 169 with ordinary accesses; a fork's few pages 7.5 us and 5.5).
template <bool Through>
__device__ __forceinline__ void copy_piece(const PoolBatch& b, int piece, int64_t from, int64_t to) {
    int lo = 0, hi = b.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (b.first[mid] <= piece) lo = mid;
        else hi = mid - 1;
    }
    const int64_t first = static_cast<int64_t>(piece - b.first[lo]) * (kPieceBytes / 16);
    const v4u* x = reinterpret_cast<const v4u*>(b.at[lo] + from * b.stride[lo]) + first;
    v4u* y = reinterpret_cast<v4u*>(b.at[lo] + to * b.stride[lo]) + first;
    const int64_t left = b.pieces16[lo] - first;
    v4u v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int j = q * kThreads + threadIdx.x;
        if (j < left) v[q] = Through ? __builtin_nontemporal_load(x + j) : x[j];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int j = q * kThreads + threadIdx.x;
        if (j >= left) continue;
        if (Through) __builtin_nontemporal_store(v[q], y + j);
        else y[j] = v[q];
    }
}

// Page src[k] to page dst[k] in every pool, for k < *count: a block's items from `item` (>= skip) on, the first copy being item `skip`.
template <bool Through>
__device__ __forceinline__ void copy_pages(const PoolBatch& b, const int32_t* src, const int32_t* dst, const int32_t* count,
                                           int64_t item, int64_t skip) {
    const int64_t items = static_cast<int64_t>(*count) * b.pieces;
    for (item -= skip; item < items; item += gridDim.x) {
        const int64_t k = item / b.pieces;
        copy_piece<Through>(b, static_cast<int>(item - k * b.pieces), src[k], dst[k]);
    }
}

// Calls f(batch) for the pools in groups that fit one launch, once at least.
template <typename F>
hipError_t for_pool_batches(const Pools& pools, F&& f) {
    PoolBatch b;
    int64_t i = 0;
    do {
        int64_t pieces = 0;
        for (b.n = 0; i < pools.n && b.n < kBatch; ++i) {
            b.at[b.n] = static_cast<char*>(pools.at[i]);
            b.stride[b.n] = pools.strides[i];
            b.pieces16[b.n] = static_cast<int32_t>(pools.bytes[i] / 16);
            b.first[b.n] = static_cast<int32_t>(pieces);
            ++b.n;
            pieces += (pools.bytes[i] + kPieceBytes - 1) / kPieceBytes;
        }
        b.pieces = static_cast<int32_t>(pieces);
        const hipError_t e = f(b);
        if (e != hipSuccess) return e;
    } while (i < pools.n);
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

// The page that new sequence j writes on in, or -1: its last one, if that is not full (and
// the table has room for what it asks for).
__device__ __forceinline__ int written_page(const ForkArgs& a, int64_t parent, int len, int grow) {
    if (parent < 0 || grow == 0 || len % a.page == 0 || grow > a.max_pages * a.page - len) return -1;
    const int id = a.tables[parent * a.ldt + len / a.page];
    return id >= 0 && id < a.n_pages ? id : -1;
}

// Threads that a phase is spread over: thread `at` of `of`.
struct Team {
    int64_t at, of;
};

// What atomics change is read past the L1 cache.
__device__ __forceinline__ int32_t fresh_load(const int32_t* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

__device__ __forceinline__ void fork_init(const ForkArgs& a, const ForkScratch& w, Team t) {
    for (int64_t p = t.at; p < a.n_pages; p += t.of) a.refs_out[p] = a.refs[p];
    for (int64_t i = t.at; i < a.n; i += t.of) w.children[i] = 0;
    for (int64_t j = t.at; j < a.n_out; j += t.of) {
        const int64_t p = parent_of(a, j);
        const int id = p < 0 ? -1 : written_page(a, p, clamped_len(a, p), grown_by(a, j));
        if (id >= 0) {
            w.keeper[id] = -1;
            w.growing[id] = 0;
        }
    }
}

__device__ __forceinline__ void fork_count(const ForkArgs& a, const ForkScratch& w, Team t) {
    for (int64_t j = t.at; j < a.n_out; j += t.of) {
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
// A wavefront a sequence.
__device__ __forceinline__ void fork_share(const ForkArgs& a, const ForkScratch& w, Team t) {
    const int lane = threadIdx.x & 63;
    for (int64_t i = t.at / kWave; i < a.n; i += t.of / kWave) {
        const int more = fresh_load(&w.children[i]) - 1;
        if (more == 0) continue;
        const int used = (clamped_len(a, i) + a.page - 1) / a.page;
#pragma unroll 4
        for (int c = lane; c < used; c += kWave) {
            const int id = a.tables[i * a.ldt + c];
            if (id >= 0 && id < a.n_pages) atomicAdd(&a.refs_out[id], more);
        }
    }
}

template <int CTRL, int ROWS>
__device__ __forceinline__ int shifted(int v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false); }

// The sum of v over the lanes up to this one, by lane permutes in the adder's operand path:
// shifts within 16 lanes, then the last lane of each 16 and 32 to the ones behind.
__device__ __forceinline__ int scan_lanes(int v) {
    v += shifted<0x111, 0xf>(v);
    v += shifted<0x112, 0xf>(v);
    v += shifted<0x114, 0xf>(v);
    v += shifted<0x118, 0xf>(v);
    v += shifted<0x142, 0xa>(v);
    v += shifted<0x143, 0xc>(v);
    return v;
}

// The sum of v over the threads before this one, and over all of them (of up to 16 wavefronts).
__device__ __forceinline__ int block_scan(int v, int* s_sum, int* total) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int upto = scan_lanes(v);
    if (lane == 63) s_sum[wave] = upto;
    __syncthreads();
    const int sums = scan_lanes(lane < waves ? s_sum[lane] : 0);
    __syncthreads();
    *total = __builtin_amdgcn_readlane(sums, 63);
    return (wave > 0 ? __builtin_amdgcn_readlane(sums, wave - 1) : 0) + upto - v;
}

// What new sequence j goes on from, and asks for.
struct Asked {
    int64_t parent;
    int len, grow, page;                 // page: the one that it writes on in, -1: none
};
__device__ __forceinline__ Asked asked_by(const ForkArgs& a, int64_t j) {
    Asked s = {-1, 0, 0, -1};
    if (j < a.n_out) {
        s.parent = parent_of(a, j);
        s.len = s.parent < 0 ? 0 : clamped_len(a, s.parent);
        s.grow = grown_by(a, j);
        s.page = written_page(a, s.parent, s.len, s.grow);
    }
    return s;
}

// Running totals over the sequences, in their order.
struct Plan {
    int free_pages;
    int64_t wanted;
    int taken, copies, missed;
};

// In a page's count of those that write on in it: one of them finds no page for its copy.
constexpr int kUncopied = 1 << 30;
static_assert(I8MM_CACHE_MAX_SEQS < kUncopied, "a bit above the count");

// What kPlanThreads sequences get, j this thread's. `held`: the count of the page it writes on in.
// The last one that writes on in a page keeps it, if the others that hold it all take copies;
// one that finds no page for its copy still holds it, and then the last one does not grow
// either. (It comes behind them, and a copy of its own would be short of a page as theirs are.)
__device__ __forceinline__ void plan_sequences(const ForkArgs& a, const ForkScratch& w, Plan& plan, int64_t j, const Asked& s,
                                               int held, int* s_sum) {
    const bool keep = s.page >= 0 && fresh_load(&w.keeper[s.page]) == j && (fresh_load(&w.growing[s.page]) & ~kUncopied) >= held;
    int copy = s.page >= 0 && !keep;
    int ok = s.grow <= a.max_pages * a.page - s.len;
    const int want = ok ? (s.len + s.grow + a.page - 1) / a.page - (s.len + a.page - 1) / a.page + copy : 0;
    // sums stay below 2^31: 1024 sequences of at most 2^20 pages each are taken at a time
    int all;
    const int64_t before = plan.wanted + block_scan(want, s_sum, &all);
    plan.wanted += all;
    if (want > 0 && before + want > plan.free_pages) ok = 0;
    if (plan.wanted > plan.free_pages) {             // (the same for all threads)
        if (copy && !ok) atomicOr(&w.growing[s.page], kUncopied);
        __syncthreads();
        if (keep && (fresh_load(&w.growing[s.page]) & kUncopied)) ok = 0;
    }
    copy = ok ? copy : 0;
    // copies and sequences that do not grow are at most 1024 each: one scan for both
    int both;
    const int at = plan.copies + (block_scan(copy + (ok ? 0 : 1 << 16), s_sum, &both) & 0xffff);
    plan.copies += both & 0xffff;
    plan.missed += both >> 16;
    block_scan(ok ? want : 0, s_sum, &all);
    plan.taken += all;
    if (j < a.n_out) {
        w.base[j] = ok ? static_cast<int>(before < plan.free_pages ? before : plan.free_pages) : -1;
        w.copied[j] = copy;
        a.lens_out[j] = ok ? s.len + s.grow : s.len;
        if (copy) {
            w.src[at] = s.page;
            w.dst[at] = static_cast<int>(before);      // its place among the fresh pages, named later
        }
    }
}

__device__ __forceinline__ void note_state(const ForkArgs& a, const ForkScratch& w, const Plan& plan) {
    *w.count = plan.copies;
    a.state[0] = plan.free_pages - plan.taken;
    const int64_t less = plan.wanted - plan.free_pages;
    a.state[1] = less < 0 ? 0 : less > 0x7fffffff ? 0x7fffffff : static_cast<int>(less);
    a.state[2] = plan.missed;
    a.state[3] = plan.copies;
}

// One block, after the counts.
__global__ __launch_bounds__(kPlanThreads) void k_fork_plan(const ForkArgs a, const ForkScratch w) {
    __shared__ int s_sum[kPlanThreads / 64];
    // each thread looks at some neighbouring pages
    const int64_t each = (a.n_pages + kPlanThreads - 1) / kPlanThreads;
    const int64_t p0 = threadIdx.x * each, p1 = p0 + each < a.n_pages ? p0 + each : a.n_pages;
    Plan plan = {};
    int mine = 0;
#pragma unroll 8
    for (int64_t p = p0; p < p1; ++p) mine += a.refs_out[p] <= 0;
    const int first_free = block_scan(mine, s_sum, &plan.free_pages);
    for (int64_t j0 = 0; j0 < a.n_out; j0 += kPlanThreads) {
        const int64_t j = j0 + threadIdx.x;
        const Asked s = asked_by(a, j);
        plan_sequences(a, w, plan, j, s, s.page >= 0 ? a.refs_out[s.page] : 0, s_sum);
    }
    __syncthreads();
    if (mine > 0 && first_free < plan.taken) {
        int at = first_free;
        for (int64_t p = p0; p < p1 && at < plan.taken; ++p) {
            if (a.refs_out[p] > 0) continue;
            w.fresh[at++] = static_cast<int>(p);
            a.refs_out[p] = 1;
        }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < plan.copies; k += kPlanThreads) {
        w.dst[k] = w.fresh[w.dst[k]];
        atomicSub(&a.refs_out[w.src[k]], 1);
    }
    if (threadIdx.x == 0) note_state(a, w, plan);
}

// Up to kAlonePages pages and kPlanThreads sequences: all of it in one launch of one block,
// which holds the counts in shared memory. With the launch that follows, 512 pages and 16
// sequences take 10 us instead of 19 in five launches, 17600 and 256 17 instead of 25, 32768
// and 1024 30 instead of 33, 32768 and 64 long ones 19 instead of 32.
constexpr int kAlonePages = 32768;

__global__ __launch_bounds__(kPlanThreads) void k_fork_alone(const ForkArgs a, const ForkScratch w) {
    __shared__ __attribute__((aligned(16))) int s_refs[kAlonePages];
    __shared__ int s_sum[kPlanThreads / 64], s_more[kPlanThreads], s_len[kPlanThreads];
    const int tid = static_cast<int>(threadIdx.x);
    // All that does not depend on anything first, and the tables' lines into the cache: memory
    // is waited for once here.
    int seen = 0;
    const int lines = (a.max_pages + 31) / 32, all_lines = static_cast<int>(a.n) * lines;
    if (all_lines <= 4 * kPlanThreads) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int l = tid + q * kPlanThreads, i = l / lines;
            if (l < all_lines) seen ^= a.tables[i * a.ldt + 32 * (l - i * lines)];
        }
    }
    Asked s = {-1, 0, 0, -1};
    if (tid < a.n_out) {
        s.parent = parent_of(a, tid);
        s.grow = grown_by(a, tid);
    }
    if (tid < a.n) s_len[tid] = clamped_len(a, tid);
    // counts by fours, all of a thread's in flight at once
    v4i four[kAlonePages / (4 * kPlanThreads)];
#pragma unroll
    for (int q = 0; q < kAlonePages / (4 * kPlanThreads); ++q) {
        const int p = 4 * (tid + q * kPlanThreads);
        if (p + 3 < a.n_pages) {
            __builtin_memcpy(&four[q], a.refs + p, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) four[q][e] = p + e < a.n_pages ? a.refs[p + e] : 0;
        }
    }
#pragma unroll
    for (int q = 0; q < kAlonePages / (4 * kPlanThreads); ++q)
        if (4 * (tid + q * kPlanThreads) < a.n_pages) *reinterpret_cast<v4i*>(s_refs + 4 * (tid + q * kPlanThreads)) = four[q];
    asm volatile("" ::"v"(seen));                // (not to be left out)
    s_more[tid] = -1;                            // children, less itself
    __syncthreads();
    if (s.parent >= 0) {
        s.len = s_len[s.parent];
        s.page = written_page(a, s.parent, s.len, s.grow);
        atomicAdd(&s_more[s.parent], 1);
    }
    if (s.page >= 0) {
        w.keeper[s.page] = -1;
        w.growing[s.page] = 0;
    }
    __syncthreads();
    if (s.page >= 0) {
        atomicMax(&w.keeper[s.page], tid);
        atomicAdd(&w.growing[s.page], 1);
    }
    // eight lanes an old sequence, 16 of a lane's entries in flight at once
    constexpr int kLanes = 8, kEntries = 16;
    for (int i = tid / kLanes; i < a.n; i += kPlanThreads / kLanes) {
        const int more = s_more[i], used = (s_len[i] + a.page - 1) / a.page;
        if (more == 0) continue;
        for (int c0 = tid % kLanes; c0 < used; c0 += kLanes * kEntries) {
            int id[kEntries];
#pragma unroll
            for (int q = 0; q < kEntries; ++q) {
                const int c = c0 + q * kLanes;
                id[q] = c < used ? a.tables[i * a.ldt + c] : -1;
            }
#pragma unroll
            for (int q = 0; q < kEntries; ++q)
                if (id[q] >= 0 && id[q] < a.n_pages) atomicAdd(&s_refs[id[q]], more);
        }
    }
    __syncthreads();
    // each thread looks at an odd number of neighbouring pages, so that a wavefront's reads fall into different banks
    const int each = (a.n_pages + kPlanThreads - 1) / kPlanThreads | 1;
    const int at0 = tid * each, p0 = at0 < a.n_pages ? at0 : a.n_pages, p1 = a.n_pages - p0 < each ? a.n_pages : p0 + each;
    Plan plan = {};
    int mine = 0;
    for (int p = p0; p < p1; ++p) mine += s_refs[p] <= 0;
    const int first_free = block_scan(mine, s_sum, &plan.free_pages);
    plan_sequences(a, w, plan, tid, s, s.page >= 0 ? s_refs[s.page] : 0, s_sum);
    __syncthreads();
    if (mine > 0 && first_free < plan.taken) {
        int at = first_free;
        for (int p = p0; p < p1 && at < plan.taken; ++p) {
            if (s_refs[p] > 0) continue;
            w.fresh[at++] = p;
            s_refs[p] = 1;
        }
    }
    __syncthreads();
    for (int k = tid; k < plan.copies; k += kPlanThreads) {
        w.dst[k] = w.fresh[w.dst[k]];
        atomicSub(&s_refs[w.src[k]], 1);
    }
    if (tid == 0) note_state(a, w, plan);
    __syncthreads();
    for (int p = 4 * tid; p < a.n_pages; p += 4 * kPlanThreads) {
        const v4i refs = *reinterpret_cast<const v4i*>(s_refs + p);
        if (p + 3 < a.n_pages) {
            __builtin_memcpy(a.refs_out + p, &refs, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (p + e < a.n_pages) a.refs_out[p + e] = refs[e];
        }
    }
}

__device__ __forceinline__ Team whole_grid() {
    return {static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, static_cast<int64_t>(gridDim.x) * blockDim.x};
}

__global__ __launch_bounds__(kThreads) void k_fork_init(const ForkArgs a, const ForkScratch w) { fork_init(a, w, whole_grid()); }
__global__ __launch_bounds__(kThreads) void k_fork_count(const ForkArgs a, const ForkScratch w) { fork_count(a, w, whole_grid()); }
__global__ __launch_bounds__(kThreads) void k_fork_share(const ForkArgs a, const ForkScratch w) { fork_share(a, w, whole_grid()); }

// The new tables' rows, then the copies.
__global__ __launch_bounds__(kThreads) void k_fork_apply(const ForkArgs a, const ForkScratch w, const PoolBatch b, bool rows) {
    const int64_t n = rows ? a.n_out : 0;
    int64_t j = blockIdx.x;
    for (; j < n; j += gridDim.x) {
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
    copy_pages<false>(b, w.src, w.dst, w.count, j, n);
}

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

// ---------------------------------------------------------------- compact

constexpr int kTilePages = 1024;

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
// `before` pages in use come before p, `below` are below n.
__device__ __forceinline__ void compact_place(const CompactArgs& a, const CompactScratch& w, int64_t p, int refs, int before,
                                              int n, int below) {
    const bool live = refs > 0;
    int rank = -1;
    if (p < n) {
        if (live) {
            rank = static_cast<int>(p);
            a.refs_out[p] = refs;
        } else {
            w.dst[p - before] = static_cast<int>(p);
        }
    } else {
        if (live) {
            rank = -2 - (before - below);
            w.src[before - below] = static_cast<int>(p);
        }
        a.refs_out[p] = 0;
    }
    w.rank[p] = rank;
}

__device__ __forceinline__ void compact_note(const CompactArgs& a, const CompactScratch& w, int n, int below) {
    a.state[0] = n;
    a.state[1] = n - below;
    *w.count = n - below;
}

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
    if (tile == 0 && threadIdx.x == 0) compact_note(a, w, n, below);
    const int64_t from = static_cast<int64_t>(tile) * kTilePages;
    for (int64_t p0 = from; p0 < from + kTilePages && p0 < a.n_pages; p0 += kThreads) {
        const int64_t p = p0 + threadIdx.x;
        const int refs = p < a.n_pages ? a.refs[p] : 0;
        int m;
        const int at = before + block_scan(refs > 0, s_sum, &m);
        before += m;
        if (p < a.n_pages) compact_place(a, w, p, refs, at, n, below);
    }
}

// The same in one block: a bit for each page in use, and the pages in use before each
// word of 64 (of which there may be as many as threads). 4096 pages 7.9 us with the
// launch that follows instead of 11.9 in three launches, 16384 12.3 in either (and a
// launch less for the host), and each further 16384 some 6 more here, 0.1 there.
constexpr int kPlanPages = 16384;
static_assert(kPlanPages <= 64 * kPlanThreads, "a thread a word");

__global__ __launch_bounds__(kPlanThreads) void k_compact_plan(const CompactArgs a, const CompactScratch w) {
    __shared__ int s_sum[kPlanThreads / 64], s_before[kPlanThreads];
    __shared__ uint64_t s_mask[kPlanThreads];
    const int words = (a.n_pages + 63) / 64, lane = threadIdx.x & 63;
    for (int p0 = threadIdx.x; p0 < words * 64; p0 += 4 * kPlanThreads) {
        int refs[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int p = p0 + q * kPlanThreads;
            refs[q] = p < a.n_pages ? a.refs[p] : 0;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint64_t mask = __ballot(refs[q] > 0);
            const int p = p0 + q * kPlanThreads;
            if (lane == 0 && p < words * 64) s_mask[p / 64] = mask;
        }
    }
    __syncthreads();
    const uint64_t mask = threadIdx.x < static_cast<unsigned>(words) ? s_mask[threadIdx.x] : 0;
    int n, below;
    s_before[threadIdx.x] = block_scan(__builtin_popcountll(mask), s_sum, &n);
    const int left = n - static_cast<int>(threadIdx.x) * 64;     // of this word's pages, those below n
    const uint64_t under = left <= 0 ? 0 : left >= 64 ? ~uint64_t(0) : (uint64_t(1) << left) - 1;
    block_scan(__builtin_popcountll(mask & under), s_sum, &below);
    if (threadIdx.x == 0) compact_note(a, w, n, below);
#pragma unroll 4
    for (int p = threadIdx.x; p < a.n_pages; p += kPlanThreads) {
        const int before = s_before[p / 64] + __builtin_popcountll(s_mask[p / 64] & ((uint64_t(1) << lane) - 1));
        compact_place(a, w, p, a.refs[p], before, n, below);
    }
}

__device__ __forceinline__ int new_place(const CompactScratch& w, int p) {
    const int r = w.rank[p];
    return r <= -2 ? w.dst[-2 - r] : r;
}

// The counts, the map and the tables, then the moves.
__global__ __launch_bounds__(kThreads) void k_compact_apply(const CompactArgs a, const CompactScratch w, const PoolBatch b,
                                                            bool tables) {
    if (tables) {
        const Team t = whole_grid();
        for (int64_t p = t.at; p < a.n_pages; p += t.of) {
            const int to = new_place(w, static_cast<int>(p));
            a.moved[p] = to;
            if (to >= 0 && to != p) a.refs_out[to] = a.refs[p];
        }
        const int64_t entries = a.n * a.max_pages;
        for (int64_t e = t.at; e < entries; e += t.of) {
            const int64_t i = e / a.max_pages, c = e - i * a.max_pages;
            const int id = a.tables[i * a.ldt + c];
            a.tables_out[i * a.ldto + c] = id >= 0 && id < a.n_pages ? new_place(w, id) : id;
        }
    }
    copy_pages<true>(b, w.src, w.dst, w.count, blockIdx.x, 0);
}

}  // namespace

hipError_t launch_cache_append(const AppendArgs& a, hipStream_t stream) {
    if (a.s == 0) return hipSuccess;
    const int per_head = a.d * a.element_bytes / 16, pieces = a.kv_heads * per_head;
    k_append<<<blocks_for((a.s * 2 * pieces + kAppendEach - 1) / kAppendEach, 8192), kThreads, 0, stream>>>(a, pieces, per_head);
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
    if (a.n_pages <= kAlonePages && a.n <= kPlanThreads && a.n_out <= kPlanThreads) {
        k_fork_alone<<<1, kPlanThreads, 0, stream>>>(a, w);
    } else {
        const int64_t most = a.n_pages > a.n ? a.n_pages : a.n;
        k_fork_init<<<blocks_for(most > a.n_out ? most : a.n_out, 1024), kThreads, 0, stream>>>(a, w);
        k_fork_count<<<blocks_for(a.n_out, 1024), kThreads, 0, stream>>>(a, w);
        k_fork_share<<<blocks_for(a.n * kWave, 2048), kThreads, 0, stream>>>(a, w);
        k_fork_plan<<<1, kPlanThreads, 0, stream>>>(a, w);
    }
    bool rows = true;
    return for_pool_batches(a.grow ? pools : Pools{nullptr, nullptr, nullptr, 0}, [&](const PoolBatch& b) {
        const int64_t items = a.n_out * (1 + static_cast<int64_t>(b.pieces));
        k_fork_apply<<<static_cast<unsigned>(items < 1 ? 1 : items < 2048 ? items : 2048), kThreads, 0, stream>>>(a, w, b, rows);
        rows = false;
        return hipGetLastError();
    });
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
    if (a.n_pages <= kPlanPages) {
        k_compact_plan<<<1, kPlanThreads, 0, stream>>>(a, w);
    } else {
        k_compact_count<<<tiles, kThreads, 0, stream>>>(a, w);
        k_compact_place<<<tiles, kThreads, 0, stream>>>(a, w);
    }
    bool tables = true;
    return for_pool_batches(pools, [&](const PoolBatch& b) {
        const int64_t entries = a.n * a.max_pages, most = entries > a.n_pages ? entries : a.n_pages;
        const int64_t items = a.n_pages / 2 * static_cast<int64_t>(b.pieces), blocks = blocks_for(most, 2048);
        const int64_t grid = items > blocks ? items : blocks;
        k_compact_apply<<<static_cast<unsigned>(grid < 2048 ? grid : 2048), kThreads, 0, stream>>>(a, w, b, tables);
        tables = false;
        return hipGetLastError();
    });
}

}  // namespace i8mm
