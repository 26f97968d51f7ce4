// The pool of a paged cache's pages: fork, reserve, free, compact.
//
// Everything is decided on the device, from tables and counts that are a few
// megabytes at most, so the decisions are bound by latency: a chain of dependent
// loads, scans and barriers.  Those that need an order (free pages from the lowest
// number up, requests by sequence and block) run in one CTA, or in one cluster of 8
// where there is more to look at, which scan 16 counts a thread at a time and
// exchange their sums through distributed shared memory.  The codes follow in
// a second kernel over the whole GPU, bound by the bytes of what moves (read and written once).
// Counts change by integer atomics only, whose order no result shows.
//
// In CUDA graphs: a fork of 3 sequences 2.5 us, of 224 with 72 entries each 4.3; pages given back 2.1 to 2.9 us; a
// reservation that lacks nothing 4.3 us, its moving kernel 1.0 of it; 48128 pages for 256 sequences in a pool of 314858
// 15.7; a compaction without a move 6.2. Each is a chain of four to ten trips to L2. Lists of sequences are searched for equal
// numbers by comparing each with all before it, which counts from some 10000 on: a fork of 4096 pairs 25 us, of 16384 98, of
// 65536 1110; 65536 rows given back 530 with a list, 210 without.

#include <climits>
#include <cooperative_groups.h>

#include "kv_pool.h"

namespace cg = cooperative_groups;

namespace pqk {
namespace {

constexpr int kMaxRanks = 8, kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kRowThreads = 256;           // of a block that works on one row of the table
constexpr int kLayersAtOnce = 64;          // layers of one launch of the moving kernel (its parameters)
constexpr int kMoveThreads = 256;

__device__ __forceinline__ void wait_for_inputs() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
}
__device__ __forceinline__ bool names(const PoolView &p, int page) { return (unsigned)page < (unsigned)p.n_pages; }
__device__ __forceinline__ int *row_of(const PoolView &p, int s) { return p.table + (size_t)s * p.table_ld; }
// Blocks that hold tokens of a sequence of m tokens.
__device__ __forceinline__ int blocks_of(const PoolView &p, int m) {
    return min((int)(((unsigned)m + (1u << p.shift) - 1) >> p.shift), p.table_ld);
}
// A barrier of the CTA, or of the cluster that the kernel is.
template <int RANKS> __device__ __forceinline__ void sync_all() {
    if constexpr (RANKS == 1) __syncthreads();
    else cg::this_cluster().sync();
}

// ---------------------------------------------------------------- fork

// Pair i, unless it names no sequence or an earlier one has its `to`. By the whole block.
__device__ __forceinline__ bool pair_counts(const PoolView &p, const int *from, const int *to, int i) {
    const int f = from[i], t = to[i];
    if ((unsigned)f >= (unsigned)p.n_seq || (unsigned)t >= (unsigned)p.n_seq) return false;
    bool taken = false;
    for (int j = threadIdx.x; j < i; j += blockDim.x) taken |= to[j] == t && (unsigned)from[j] < (unsigned)p.n_seq;
    return !__syncthreads_or(taken);
}

// The row that sequence t gets, as it is before any changes, and its pages' counts. By `threads` threads.
__device__ __forceinline__ void take_row(const PoolView &p, const PoolWs &w, int f, int t, int m, int thread, int threads) {
    const int *row = row_of(p, f);
    int *out = w.rows + (size_t)t * p.table_ld;
    for (int j = thread, end = blocks_of(p, m); j < end; j += threads) {
        const int page = row[j];
        out[j] = names(p, page) ? page : -1;
        if (names(p, page)) atomicAdd(p.refs + page, 1);
    }
}
// What the sequence of pair i held is given back, and the new row takes its place; the threads that took it.
__device__ __forceinline__ void put_row(const PoolView &p, const PoolWs &w, const int *from, const int *to, int i, int thread, int threads) {
    const int t = to[i];
    if ((unsigned)from[i] >= (unsigned)p.n_seq || (unsigned)t >= (unsigned)p.n_seq) return;
    const int2 pair = __ldcg(w.pair + t);
    if (pair.x != i) return;
    const int end = blocks_of(p, pair.y);
    int *row = row_of(p, t);
    const int *in = w.rows + (size_t)t * p.table_ld;
    for (int j = thread; j < p.table_ld; j += threads) {
        const int old = row[j];
        if (names(p, old)) atomicSub(p.refs + old, 1);
        row[j] = j < end ? in[j] : -1;
    }
    if (thread == 0) p.len[t] = pair.y;
}

// The rows that the sequences get.
__global__ void __launch_bounds__(kRowThreads) fork_take(PoolView p, const int *from, const int *to, const int *tokens, PoolWs w) {
    wait_for_inputs();
    const int i = blockIdx.x;
    if (!pair_counts(p, from, to, i)) return;
    const int f = from[i], t = to[i];
    int m = max(p.len[f], 0);
    if (tokens) m = min(m, max(tokens[i], 0));
    if (threadIdx.x == 0) w.pair[t] = make_int2(i, m);
    take_row(p, w, f, t, m, threadIdx.x, kRowThreads);
}

// What the sequences held is given back, and the new rows take its place.
__global__ void __launch_bounds__(kRowThreads) fork_put(PoolView p, const int *from, const int *to, PoolWs w) {
    wait_for_inputs();
    put_row(p, w, from, to, blockIdx.x, threadIdx.x, kRowThreads);
}

// Both by one CTA, a warp per pair: one launch less.
__global__ void __launch_bounds__(kPlanThreads) fork_few(PoolView p, int n, const int *from, const int *to, const int *tokens, PoolWs w) {
    wait_for_inputs();
    const int lane = threadIdx.x & 31, i = threadIdx.x >> 5;
    if (i < n) {
        const int f = from[i], t = to[i];
        bool out = (unsigned)f >= (unsigned)p.n_seq || (unsigned)t >= (unsigned)p.n_seq;
        if (lane < i) out |= to[lane] == t && (unsigned)from[lane] < (unsigned)p.n_seq;
        if (!__any_sync(0xffffffffu, out)) {
            int m = max(p.len[f], 0);
            if (tokens) m = min(m, max(tokens[i], 0));
            if (lane == 0) w.pair[t] = make_int2(i, m);
            take_row(p, w, f, t, m, lane, 32);
        }
    }
    __syncthreads();
    if (i < n) put_row(p, w, from, to, i, lane, 32);
}

// ---------------------------------------------------------------- free

__global__ void __launch_bounds__(kRowThreads) free_rows(PoolView p, const int *seq, const int *begin, const int *end) {
    wait_for_inputs();
    const int i = blockIdx.x, s = seq ? seq[i] : i;
    if ((unsigned)s >= (unsigned)p.n_seq) return;
    if (seq) {
        bool taken = false;
        for (int j = threadIdx.x; j < i; j += kRowThreads) taken |= seq[j] == s;
        if (__syncthreads_or(taken)) return;
    }
    const int size = 1 << p.shift, from = begin ? max(begin[i], 0) : 0, len = max(p.len[s], 0);
    int to = end ? end[i] : INT_MAX;
    if (to <= from) return;
    const bool rest = to >= len;
    const int first = (int)(((unsigned)from + size - 1) >> p.shift), last = rest ? p.table_ld : min(to >> p.shift, p.table_ld);
    int *row = row_of(p, s);
    __syncthreads();                       // all have read len
    if (threadIdx.x == 0 && rest && from < len) p.len[s] = from;
    constexpr int AT_ONCE = 4;
    for (int j0 = first + threadIdx.x; j0 < last; j0 += AT_ONCE * kRowThreads) {
        int page[AT_ONCE];
#pragma unroll
        for (int e = 0; e < AT_ONCE; ++e) page[e] = j0 + e * kRowThreads < last ? row[j0 + e * kRowThreads] : -1;
#pragma unroll
        for (int e = 0; e < AT_ONCE; ++e)
            if (j0 + e * kRowThreads < last) {
                if (names(p, page[e])) atomicSub(p.refs + page[e], 1);
                row[j0 + e * kRowThreads] = -1;
            }
    }
}

// ---------------------------------------------------------------- what plans: one CTA, or one cluster
//
// Most calls run this code once, so that its instructions come from far away: loops are kept rolled and sums short (with
// 8 requests a thread in registers and sums of two counts, ranking 4 requests took 5500 cycles).

// A value of every CTA, two at a time: the ones before may still be read while the next are written.
struct Board {
    unsigned v[2][kMaxRanks];
};

// This CTA's value to all, and a barrier of all: sums over the CTAs before this one, and over all.
struct Shares {
    unsigned before, all;
};
template <int RANKS> __device__ __forceinline__ Shares share(Board &board, int &turn, unsigned mine) {
    Shares s = {0, mine};
    if constexpr (RANKS > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        const int rank = (int)cluster.block_rank();
        if (threadIdx.x < RANKS) cluster.map_shared_rank(&board, threadIdx.x)->v[turn][rank] = mine;
        cluster.sync();
        s.all = 0;
        for (int r = 0; r < RANKS; ++r) {
            const unsigned x = board.v[turn][r];
            s.all += x;
            if (r < rank) s.before += x;
        }
        turn ^= 1;
    }
    return s;
}

// Sums over the warps before this one, and over all, of a number per warp. `sums` is shared memory, free when it returns.
__device__ __forceinline__ unsigned warps_before(unsigned of_warp, unsigned *sums, unsigned &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) sums[warp] = of_warp;
    __syncthreads();
    unsigned incl = sums[lane];            // every warp by itself: one barrier less
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    const unsigned before = __shfl_sync(0xffffffffu, incl, max(warp - 1, 0));
    __syncthreads();
    return warp ? before : 0;
}
// Exclusive sums over the block's threads, and their total.
__device__ __forceinline__ unsigned block_scan(unsigned x, unsigned *sums, unsigned &total) {
    const int lane = threadIdx.x & 31;
    unsigned incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    return incl - x + warps_before(__shfl_sync(0xffffffffu, incl, 31), sums, total);
}

constexpr int kPer = 16;                   // counts of a thread at a time, 32 apart
template <int RANKS> __host__ __device__ constexpr int sweep() { return RANKS * kPlanThreads * kPer; }

// The first of a thread's pages in the sweep from i0.
__device__ __forceinline__ int first_page(int i0, int tid) { return i0 + tid / 32 * 32 * kPer + (tid & 31); }
// Of kPer pages, 32 apart from `at`: bit i says that the i-th is in use.
__device__ __forceinline__ unsigned in_use(const PoolView &p, int at) {
    int held[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) held[i] = at + 32 * i < p.n_pages ? __ldcg(p.refs + at + 32 * i) : 0;
    unsigned used = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) used |= (held[i] > 0) << i;
    return used;
}
// Of the same, which there are.
__device__ __forceinline__ unsigned there_are(const PoolView &p, int at) {
    const int n = at < p.n_pages ? (p.n_pages - 1 - at) / 32 + 1 : 0;
    return n >= kPer ? (1u << kPer) - 1 : (1u << n) - 1;
}

// ---------------------------------------------------------------- reserve

constexpr int kCached = 8192;              // requests of a CTA that are looked up once

// Blocks that new tokens of this CTA's sequences go to, one behind the other.
struct Asks {
    int *start, *first, *len;              // per sequence, in shared memory: its blocks begin at start, with block `first` of its row; tokens
    int n, s0;                             // sequences, the first one
    int2 *seen;                            // in shared memory: what `look` found for the first kCached of them
};
constexpr unsigned kThere = 1u << 30, kShared = 1u << 31, kSeq = kThere - 1;

// The sequence of block i: the last one that starts there or before.
__device__ __noinline__ int seq_of(const Asks &a, int i) {
    int lo = 0, hi = a.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.start[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}
// Blocks i, i + kPlanThreads, .. as they are before anything changes: their pages, and their sequences with kThere if they have a
// page and kShared if others hold that too. N at a time, so that their loads overlap.
template <int N> __device__ __forceinline__ void look(const PoolView &p, const Asks &a, int i, int items, int2 (&x)[N]) {
    int held[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int at = i + e * kPlanThreads, s = at >= items ? 0 : at < kCached ? a.seen[at].y : seq_of(a, at);
        x[e] = make_int2(-1, s);
        if (at < items) x[e].x = row_of(p, a.s0 + s)[a.first[s] + at - a.start[s]];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) held[e] = names(p, x[e].x) ? p.refs[x[e].x] : -1;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (names(p, x[e].x)) x[e].y |= (int)kThere;
        if (held[e] > 1) x[e].y |= (int)kShared;
    }
}

// Two dependent trips to L2 look a request up, two more count the writers of shared pages, one finds free pages per
// sweep and one assigns them; 8 CTAs because one holds 8192 requests and scans 16384 pages at a time.
template <int RANKS> __global__ void __cluster_dims__(RANKS, 1, 1) __launch_bounds__(kPlanThreads)
    reserve_plan(PoolView p, const int *n_new, int *status, PoolWs w) {
    constexpr int NEAR = RANKS == 1 ? kPlanThreads : 1;      // free pages that go through shared memory
    extern __shared__ int2 asked[];
    __shared__ Board board;
    __shared__ unsigned sums[kPlanWarps], chunks[kCached / 32];
    __shared__ int near_free[NEAR];
    const int rank = blockIdx.x, tid = rank * kPlanThreads + threadIdx.x, lane = threadIdx.x & 31;
    const unsigned below = (1u << lane) - 1;
    const int per = (p.n_seq + RANKS - 1) / RANKS;
    Asks a;
    a.seen = asked;
    a.start = reinterpret_cast<int *>(asked + kCached);
    a.first = a.start + per + 1;
    a.len = a.first + per;
    a.s0 = min(rank * per, p.n_seq);
    a.n = min(per, p.n_seq - a.s0);
    int *count = w.list[1], *lowest = w.list[2], turn = 0;      // count: writers of a page less its holders; lowest: the lowest sequence that writes
    unsigned sum;
    if (RANKS > 1) sync_all<RANKS>();      // all CTAs run: their boards may be written
    wait_for_inputs();
    if (tid == 0) w.head[0] = 0;

    // the sequences' blocks, one behind the other
    int items = 0, narrow = 0;
    for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        int blocks = 0;
        bool short_row = false;
        if (i < a.n) {
            const int more = n_new[a.s0 + i], len = max(p.len[a.s0 + i], 0), first = len >> p.shift;
            if (more > 0) {
                const int last = (int)(((unsigned)len + (unsigned)more - 1u) >> p.shift);
                short_row = last >= p.table_ld;
                if (!short_row) blocks = last - first + 1;
            }
            a.first[i] = first;
            a.len[i] = len;
        }
        narrow += __syncthreads_count(short_row);
        const unsigned at = block_scan(blocks, sums, sum);
        if (i < a.n) a.start[i] = items + (int)at;
        items += (int)sum;
    }
    if (threadIdx.x == 0) a.start[a.n] = items;
    __syncthreads();

    // their sequences, a warp each; then which of them lack a page, and which have one that others hold too
    for (int s = threadIdx.x >> 5; s < a.n; s += kPlanWarps)
        for (int i = a.start[s] + lane; i < min(a.start[s + 1], kCached); i += 32) a.seen[i].y = s;
    __syncthreads();
    bool any = false;
    constexpr int N = 4;
    for (int i = threadIdx.x; i < items; i += N * kPlanThreads) {
        int2 x[N];
        look(p, a, i, items, x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (i + e * kPlanThreads < min(items, kCached)) a.seen[i + e * kPlanThreads] = x[e];
            if ((unsigned)x[e].y & kShared) {
                any = true;
                count[x[e].x] = -p.refs[x[e].x];     // the same from all who write here
                lowest[x[e].x] = INT_MAX;
            }
        }
    }
    any = __syncthreads_or(any);
    // in one sum: sequences whose row is too short (at most 2^16), CTAs that share pages, and those with requests to be looked up again
    const unsigned told = share<RANKS>(board, turn, (unsigned)narrow | (any ? 1u << 20 : 0u) | (items > kCached ? 1u << 24 : 0u)).all;
    narrow = (int)(told & 0xfffffu);
    const bool shared = (told >> 20) & 15u, later = told >> 24;
    auto seen = [&](int i) {
        int2 x[1];
        if (i < kCached) x[0] = a.seen[i];
        else look(p, a, i, items, x);
        return x[0];
    };
    if (shared) {
        for (int i = threadIdx.x; i < items; i += kPlanThreads) {
            const int2 x = seen(i);
            if ((unsigned)x.y & kShared) {
                atomicAdd(count + x.x, 1);
                atomicMin(lowest + x.x, a.s0 + (int)((unsigned)x.y & kSeq));
            }
        }
        sync_all<RANKS>();
    }
    // Whether a block's page stays with its other holders: unless the sequence keeps it, as the lowest of holders who all write.
    auto leaves = [&](const int2 &x) {
        return ((unsigned)x.y & kShared) && (__ldcg(count + x.x) != 0 || __ldcg(lowest + x.x) != a.s0 + (int)((unsigned)x.y & kSeq));
    };
    // How many of the kCached blocks from i0 need a page; `chunks` then says how many of them lie before each 32.
    auto rank_blocks = [&](int i0) {
        const int end = min(items - i0, kCached);
#pragma unroll 1
        for (int i = threadIdx.x; i - lane < end; i += kPlanThreads) {
            const int2 x = i < end ? seen(i0 + i) : make_int2(0, (int)kThere);
            const unsigned of = __ballot_sync(0xffffffffu, !((unsigned)x.y & kThere) || leaves(x));
            if (lane == 0) chunks[i / 32] = __popc(of);
        }
        __syncthreads();
        unsigned n;
        const unsigned before = block_scan(threadIdx.x * 32 < end ? chunks[threadIdx.x] : 0, sums, n);
        if (threadIdx.x * 32 < end) chunks[threadIdx.x] = before;
        __syncthreads();
        return n;
    };
    sum = 0;
    for (int i0 = 0; i0 < items; i0 += kCached) sum += rank_blocks(i0);
    const Shares needs = share<RANKS>(board, turn, sum);
    const int total = (int)needs.all;

    // the lowest free pages
    int found = 0;
    for (int i0 = 0; i0 < p.n_pages && found < total; i0 += sweep<RANKS>()) {
        const int at = first_page(i0, tid);
        const unsigned free = ~in_use(p, at) & there_are(p, at);
        const unsigned before = warps_before(__reduce_add_sync(0xffffffffu, __popc(free)), sums, sum);
        const Shares all = share<RANKS>(board, turn, sum);
        int k = found + (int)(all.before + before);
#pragma unroll 1
        for (int e = 0; e < kPer && k < total; ++e) {
            const unsigned of = __ballot_sync(0xffffffffu, (free >> e) & 1);
            const int to = k + __popc(of & below);
            if ((free >> e) & 1 && to < total) {
                if (RANKS == 1 && to < NEAR) near_free[to] = at + 32 * e;
                else w.list[0][to] = at + 32 * e;
            }
            k += __popc(of);
        }
        found += (int)all.all;
    }
    const bool done = found >= total && narrow == 0;
    if (tid == 0) {
        status[0] = max(total - found, 0);
        status[1] = narrow;
    }
    sync_all<RANKS>();
    if (done && total > 0) {
        int k = (int)needs.before;
        for (int i0 = 0; i0 < items; i0 += kCached) {
            unsigned n = 0;
            if (items > kCached) n = rank_blocks(i0);
#pragma unroll 2
            for (int i = i0 + threadIdx.x; i - lane < min(items, i0 + kCached); i += kPlanThreads) {
                int2 x = make_int2(0, (int)kThere);
                if (i < items) x = seen(i);
                const bool away = leaves(x), wants = away || !((unsigned)x.y & kThere);
                const unsigned of = __ballot_sync(0xffffffffu, wants);
                if (!wants) continue;
                const int at = k + (int)chunks[(i - i0) / 32] + __popc(of & below);
                const int seq = (int)((unsigned)x.y & kSeq), j = a.first[seq] + i - a.start[seq];
                const int to = RANKS == 1 && at < NEAR ? near_free[at] : __ldcg(w.list[0] + at);
                row_of(p, a.s0 + seq)[j] = to;
                p.refs[to] = 1;
                if (away) {                // the moves' order does not matter
                    w.moves[atomicAdd(w.head, 1)] = make_int4(x.x, to, min(max(a.len[seq] - (j << p.shift), 0), 1 << p.shift), 0);
                    if (!later) atomicSub(p.refs + x.x, 1);
                }
            }
            k += (int)n;
            if (items > kCached) __syncthreads();
        }
    }
    if (RANKS == 1 && !later) return;
    sync_all<RANKS>();                     // all have read the counts, and nobody's board is written any more
    if (later)
        for (int i = tid, n = __ldcg(w.head); i < n; i += RANKS * kPlanThreads) atomicSub(p.refs + __ldcg(w.moves + i).x, 1);
}

// ---------------------------------------------------------------- compact

// Two passes over the counts: how many are in use, then which are on the wrong side of that number; a pool of one sweep
// keeps them in registers between.
template <int RANKS> __global__ void __cluster_dims__(RANKS, 1, 1) __launch_bounds__(kPlanThreads)
    compact_plan(PoolView p, int *moved, int *n_used, PoolWs w) {
    __shared__ Board board;
    __shared__ unsigned sums[kPlanWarps];
    const int tid = blockIdx.x * kPlanThreads + threadIdx.x;
    int *holes = w.list[0], *live = w.list[1], *map = w.list[2], turn = 0;
    if (RANKS > 1) sync_all<RANKS>();      // all CTAs run: their boards may be written
    wait_for_inputs();
    unsigned sum, n = 0, used = 0;
    for (int i0 = 0; i0 < p.n_pages; i0 += sweep<RANKS>()) {
        used = in_use(p, first_page(i0, tid));
        n += __popc(used);
    }
    warps_before(__reduce_add_sync(0xffffffffu, n), sums, sum);
    const int total = (int)share<RANKS>(board, turn, sum).all;
    // the free pages below `total` and the pages in use from there on, in order: page x has x less the pages in use before it
    // free ones before it
    int before = 0;
    unsigned low = 0;                      // pages in use below `total`
    for (int i0 = 0; i0 < p.n_pages; i0 += sweep<RANKS>()) {
        const int at = first_page(i0, tid);
        if (p.n_pages > sweep<RANKS>()) used = in_use(p, at);
        const unsigned mine = warps_before(__reduce_add_sync(0xffffffffu, __popc(used)), sums, sum);
        const Shares all = share<RANKS>(board, turn, sum);
        int k = before + (int)(all.before + mine);
#pragma unroll 1
        for (int e = 0; e < kPer; ++e) {
            const int page = at + 32 * e;
            const bool in = (used >> e) & 1;
            const unsigned of = __ballot_sync(0xffffffffu, in);
            const int ahead = k + __popc(of & ((1u << (tid & 31)) - 1));      // pages in use before this one
            k += __popc(of);
            if (page >= p.n_pages) continue;
            if (page < total) {
                if (!in) holes[page - ahead] = page;
                low += in;
            } else {
                if (in) live[ahead] = page;
                map[page] = -1;
            }
            if (moved && !(in && page >= total)) moved[page] = in ? page : -1;
        }
        before += (int)all.all;
    }
    warps_before(__reduce_add_sync(0xffffffffu, low), sums, sum);
    const int keep = (int)share<RANKS>(board, turn, sum).all, n_high = total - keep;
    if (tid == 0) {
        *n_used = total;
        w.head[0] = n_high;
    }
    if (RANKS == 1) __syncthreads();
    for (int i = tid; i < n_high; i += RANKS * kPlanThreads) {
        const int from = __ldcg(live + keep + i), to = __ldcg(holes + i);
        p.refs[to] = p.refs[from];
        p.refs[from] = 0;
        map[from] = to;
        if (moved) moved[from] = to;
        w.moves[i] = make_int4(from, to, 1 << p.shift, 0);
    }
    if (RANKS > 1) sync_all<RANKS>();      // no CTA leaves while its board may be written
}

// Table entries from the first page that may have moved on.
__device__ __forceinline__ void rename(const PoolView &p, const int *map, const int *n_used, long long i, long long step) {
    const int used = *n_used;
    for (const long long n = (long long)p.n_seq * p.table_ld; i < n; i += step) {
        const int page = p.table[i];
        if (page >= used && page < p.n_pages) {
            const int to = map[page];
            if (to >= 0) p.table[i] = to;
        }
    }
}

// ---------------------------------------------------------------- codes and scales of the moves

struct MoveArgs {
    PoolView p;
    const int *head;
    const int4 *moves;
    const int *map, *n_used;               // of a compaction's first launch, else null
    int pieces, heads;                     // pieces of a page in all layers, kv heads of a piece
    FastDiv per_page, per_layer, per_half; // by the pieces of a page, of a layer's page, of its K or V
    PoolLayer layer[kLayersAtOnce];
};
// A warp at a time takes a piece: a move's tokens of one layer, K or V, and some kv heads. Loads in flight are few on
// purpose, 2 KB a warp and 32 warps an SM: 224 moves of 16 tokens, 32 layers of 8 kv heads of 128, a whole call with 4 KB
// 89 us and 64 warps 104, as it stands 60 (244 MB written, 35 read: 5.6 TB/s of the moving kernel); 156 pages of 64 tokens
// in all 32 layers 230, 251 and 215 (1.31 GB, 6.4 TB/s). One read of a page for all its copies: 69.
constexpr int kPieceBytes = 2048, kMoveCtas = 4;

__global__ void __launch_bounds__(kMoveThreads, kMoveCtas) move_pages(const __grid_constant__ MoveArgs a) {
    wait_for_inputs();
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * (kMoveThreads / 32), n = (long long)a.head[0] * a.pieces;
    for (long long i = (long long)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); i < n; i += warps) {
        const int move = i < 0x7fffffffll ? a.per_page.div((int)i) : (int)(i / a.per_page.d);
        const int part = (int)(i - (long long)move * a.per_page.d), l = a.per_layer.div(part), in_layer = part - l * a.per_layer.d;
        const int kv = in_layer >= a.per_half.d, h = (in_layer - kv * a.per_half.d) * a.heads;
        const PoolLayer &layer = a.layer[l];
        const int4 m = a.moves[move];
        const int heads = min(a.heads, layer.n_kv - h);
        if (heads <= 0 || m.z == 0) continue;
        const int row = (layer.d / 16) << a.p.shift;          // 16-byte units of a head in a page, and of its tokens
        const int units = m.z * (layer.d / 16), total = units * heads;
        const size_t from = (size_t)m.x * layer.n_kv + h, to = (size_t)m.y * layer.n_kv + h;
        int8_t *codes = kv ? layer.v : layer.k;
        float *scale = kv ? layer.v_scale : layer.k_scale;
        const uint4 *src = reinterpret_cast<const uint4 *>(codes) + from * row;
        uint4 *dst = reinterpret_cast<uint4 *>(codes) + to * row;
        // Unit f is number f - u * units of head u: the quotient by a reciprocal, which is off by less than the half that
        // keeps it from the next whole number (u below 2^5, units at most 2^11).
        const float inv = 1.f / (float)units;
        constexpr int AT_ONCE = 4;
        for (int f0 = lane; f0 < total; f0 += 32 * AT_ONCE) {
            uint4 x[AT_ONCE];
            int at[AT_ONCE];
#pragma unroll
            for (int e = 0; e < AT_ONCE; ++e) {
                const int f = f0 + 32 * e, u = (int)(((float)f + 0.5f) * inv);
                at[e] = f + u * (row - units);
                if (f < total) x[e] = __ldcs(src + at[e]);
            }
#pragma unroll
            for (int e = 0; e < AT_ONCE; ++e)
                if (f0 + 32 * e < total) __stcs(dst + at[e], x[e]);
        }
        for (int u = lane; u < heads; u += 32) scale[to + u] = scale[from + u];
    }
    if (a.map)
        rename(a.p, a.map, a.n_used, (long long)blockIdx.x * kMoveThreads + threadIdx.x, (long long)gridDim.x * kMoveThreads);
}

// A launch that may be scheduled while the kernel before it finishes.
template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), int grid, int threads, size_t smem, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// `tokens`: of a move, about.
cudaError_t launch_moves(const PoolView &p, const PoolLayer *layers, int n_layers, int tokens, const PoolWs &w, const int *n_used,
                         cudaStream_t s, const DeviceInfo &dev) {
    MoveArgs a;
    a.p = p;
    a.head = w.head;
    a.moves = w.moves;
    a.map = n_used ? w.list[2] : nullptr;
    a.n_used = n_used;
    int l = 0;
    do {
        const int here = n_layers - l < kLayersAtOnce ? n_layers - l : kLayersAtOnce;
        int heads = 1, bytes = 1;
        for (int i = 0; i < here; ++i) {
            a.layer[i] = layers[l + i];
            if (a.layer[i].n_kv > heads) heads = a.layer[i].n_kv;
            if (tokens * a.layer[i].d > bytes) bytes = tokens * a.layer[i].d;
        }
        a.heads = kPieceBytes / bytes < 1 ? 1 : kPieceBytes / bytes > 32 ? 32 : kPieceBytes / bytes;
        if (a.heads > heads) a.heads = heads;
        const int half = (heads + a.heads - 1) / a.heads;
        a.pieces = 2 * half * here;
        a.per_half = FastDiv(half);
        a.per_layer = FastDiv(2 * half);
        a.per_page = FastDiv(a.pieces > 0 ? a.pieces : 1);
        const cudaError_t e = launch(move_pages, dev.sm_count * kMoveCtas, kMoveThreads, 0, s, a);
        if (e != cudaSuccess) return e;
        a.map = a.n_used = nullptr;
        l += here;
    } while (l < n_layers);
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv_fork(const PoolView &p, int n, const int *from, const int *to, const int *tokens, const PoolWs &w,
                           cudaStream_t s) {
    // 4 pairs of 64 entries: 2.0 us less than as two launches; 224 pairs of 72 entries in a cluster of 8: 4 us more
    if (n <= kPlanWarps && p.table_ld <= 512) return launch(fork_few, 1, kPlanThreads, 0, s, p, n, from, to, tokens, w);
    const cudaError_t e = launch(fork_take, n, kRowThreads, 0, s, p, from, to, tokens, w);
    return e == cudaSuccess ? launch(fork_put, n, kRowThreads, 0, s, p, from, to, w) : e;
}

cudaError_t launch_kv_free(const PoolView &p, int n, const int *seq, const int *begin, const int *end, cudaStream_t s) {
    return launch(free_rows, n, kRowThreads, 0, s, p, seq, begin, end);
}

// Whether one CTA plans.
static bool small_pool(const PoolView &p) { return p.n_pages <= sweep<1>() && p.n_seq <= kPlanThreads; }

template <int RANKS> static cudaError_t launch_reserve_plan(const PoolView &p, const int *n_new, int *status, const PoolWs &w, cudaStream_t s) {
    auto bytes = [](int n_seq) { return kCached * sizeof(int2) + (size_t)(3 * ((n_seq + RANKS - 1) / RANKS) + 1) * sizeof(int); };
    static PerDeviceOnce once;
    const cudaError_t e = once.run([&] {
        return cudaFuncSetAttribute(reserve_plan<RANKS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)bytes(RANKS == 1 ? kPlanThreads : kPoolMaxSeq));
    });
    return e == cudaSuccess ? launch(reserve_plan<RANKS>, RANKS, kPlanThreads, bytes(p.n_seq), s, p, n_new, status, w) : e;
}

cudaError_t launch_kv_reserve(const PoolView &p, const PoolLayer *layers, int n_layers, const int *n_new, int *status,
                              const PoolWs &w, cudaStream_t s, const DeviceInfo &dev) {
    const cudaError_t e = small_pool(p) ? launch_reserve_plan<1>(p, n_new, status, w, s) : launch_reserve_plan<kMaxRanks>(p, n_new, status, w, s);
    return e == cudaSuccess && n_layers > 0 ? launch_moves(p, layers, n_layers, (1 << p.shift) / 2, w, nullptr, s, dev) : e;
}

cudaError_t launch_kv_compact(const PoolView &p, const PoolLayer *layers, int n_layers, int *moved, int *n_used,
                              const PoolWs &w, cudaStream_t s, const DeviceInfo &dev) {
    const cudaError_t e = small_pool(p) ? launch(compact_plan<1>, 1, kPlanThreads, 0, s, p, moved, n_used, w)
                                        : launch(compact_plan<kMaxRanks>, kMaxRanks, kPlanThreads, 0, s, p, moved, n_used, w);
    return e == cudaSuccess ? launch_moves(p, layers, n_layers, 1 << p.shift, w, n_used, s, dev) : e;
}

}  // namespace pqk
