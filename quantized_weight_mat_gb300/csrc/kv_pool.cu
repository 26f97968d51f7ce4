// The pool of a paged cache's pages: fork, reserve, free, compact.
//
// Everything is decided on the device, from tables and counts that are a few
// megabytes at most, so the decisions are bound by latency: a chain of dependent
// loads, scans and barriers.  Those that need an order (free pages from the lowest
// number up, requests by sequence and block) run in one cluster of 8 CTAs, which
// scans 32768 counts at a time and exchanges its sums through distributed shared
// memory; what is independent per sequence takes a block each.  The codes follow in
// a second kernel over the whole GPU, bound by the bytes of what moves (read and written once).
// Counts change by integer atomics only, whose order no result shows.

#include <climits>
#include <cooperative_groups.h>

#include "kv_pool.h"

namespace cg = cooperative_groups;

namespace pqk {
namespace {

constexpr int kRanks = 8, kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
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
__device__ __forceinline__ unsigned lanes_below() { return (1u << (threadIdx.x & 31)) - 1; }

// ---------------------------------------------------------------- fork

// Pair i, unless it names no sequence or an earlier one has its `to`. By the whole block.
__device__ __forceinline__ bool pair_counts(const PoolView &p, const int *from, const int *to, int i) {
    const int f = from[i], t = to[i];
    if ((unsigned)f >= (unsigned)p.n_seq || (unsigned)t >= (unsigned)p.n_seq) return false;
    bool taken = false;
    for (int j = threadIdx.x; j < i; j += blockDim.x) taken |= to[j] == t && (unsigned)from[j] < (unsigned)p.n_seq;
    return !__syncthreads_or(taken);
}

// The rows that the sequences get, as they are before any of them changes, and their pages' counts.
__global__ void __launch_bounds__(kRowThreads) fork_take(PoolView p, const int *from, const int *to, const int *tokens, PoolWs w) {
    wait_for_inputs();
    const int i = blockIdx.x;
    if (!pair_counts(p, from, to, i)) return;
    const int f = from[i], t = to[i];
    int m = max(p.len[f], 0);
    if (tokens) m = min(m, max(tokens[i], 0));
    if (threadIdx.x == 0) w.pair[t] = make_int2(i, m);
    const int *row = row_of(p, f);
    int *out = w.rows + (size_t)t * p.table_ld;
    for (int j = threadIdx.x, end = blocks_of(p, m); j < end; j += kRowThreads) {
        const int page = row[j];
        out[j] = names(p, page) ? page : -1;
        if (names(p, page)) atomicAdd(p.refs + page, 1);
    }
}

// What the sequences held is given back, and the new rows take its place.
__global__ void __launch_bounds__(kRowThreads) fork_put(PoolView p, const int *from, const int *to, PoolWs w) {
    wait_for_inputs();
    const int i = blockIdx.x, t = to[i];
    if ((unsigned)from[i] >= (unsigned)p.n_seq || (unsigned)t >= (unsigned)p.n_seq || w.pair[t].x != i) return;
    const int m = w.pair[t].y, end = blocks_of(p, m);
    int *row = row_of(p, t);
    const int *in = w.rows + (size_t)t * p.table_ld;
    for (int j = threadIdx.x; j < p.table_ld; j += kRowThreads) {
        const int old = row[j];
        if (names(p, old)) atomicSub(p.refs + old, 1);
        row[j] = j < end ? in[j] : -1;
    }
    if (threadIdx.x == 0) p.len[t] = m;
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
    for (int j = first + threadIdx.x; j < last; j += kRowThreads) {
        const int page = row[j];
        if (names(p, page)) atomicSub(p.refs + page, 1);
        row[j] = -1;
    }
}

// ---------------------------------------------------------------- the planning cluster

// A value of every CTA of the cluster, two at a time: the ones before may still be read while the next are written.
struct Board {
    unsigned long long v[2][kRanks];
};

__device__ __forceinline__ unsigned long long both(unsigned lo, unsigned hi) { return (unsigned long long)hi << 32 | lo; }

// This CTA's value to all, and a barrier of the cluster: sums over the CTAs before this one, and over all.
struct Shares {
    unsigned long long before, all;
};
__device__ __forceinline__ Shares share(cg::cluster_group &cluster, Board &board, int &turn, unsigned long long mine) {
    const int rank = (int)cluster.block_rank();
    if (threadIdx.x < kRanks) cluster.map_shared_rank(&board, threadIdx.x)->v[turn][rank] = mine;
    cluster.sync();
    Shares s = {0, 0};
#pragma unroll
    for (int r = 0; r < kRanks; ++r) {
        const unsigned long long x = board.v[turn][r];
        s.all += x;
        if (r < rank) s.before += x;
    }
    turn ^= 1;
    return s;
}

// Exclusive sums of two counts over the block's threads, and their totals. `sums` is shared memory, free when it returns.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long x, unsigned long long *sums, unsigned long long &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    unsigned long long of = sums[lane];    // every warp by itself: one barrier less
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long up = __shfl_up_sync(0xffffffffu, of, o);
        if (lane >= o) of += up;
    }
    total = __shfl_sync(0xffffffffu, of, 31);
    const unsigned long long before = __shfl_sync(0xffffffffu, of, max(warp - 1, 0));
    __syncthreads();
    return incl - x + (warp ? before : 0);
}

constexpr int kPer = 4, kSweep = kRanks * kPlanThreads * kPer;      // counts of a thread, and of the cluster, at a time

// Counts of 4 pages from `at`; 0 behind the last one if free ones are looked for, else 1 there stands for none.
__device__ __forceinline__ int4 load_refs(const PoolView &p, int at, int none) {
    if (at + kPer <= p.n_pages) return __ldcg(reinterpret_cast<const int4 *>(p.refs + at));
    int4 r = make_int4(none, none, none, none);
    if (at < p.n_pages) r.x = __ldcg(p.refs + at);
    if (at + 1 < p.n_pages) r.y = __ldcg(p.refs + at + 1);
    if (at + 2 < p.n_pages) r.z = __ldcg(p.refs + at + 2);
    return r;
}

// ---------------------------------------------------------------- reserve

// A sequence's blocks that new tokens go to.
struct Ask {
    int len, first, last;      // last < first: none
    bool narrow;               // behind its row's end
};
__device__ __forceinline__ Ask ask_of(const PoolView &p, const int *n_new, int s) {
    Ask a;
    const int more = n_new[s];
    a.len = max(p.len[s], 0);
    a.first = a.len >> p.shift;
    a.last = a.first - 1;
    a.narrow = false;
    if (more > 0) {
        const int last = (int)(((unsigned)a.len + (unsigned)more - 1u) >> p.shift);
        a.narrow = last >= p.table_ld;
        if (!a.narrow) a.last = last;
    }
    return a;
}

// count[page]: writers less holders; lowest[page]: lowest sequence that writes.
__global__ void __cluster_dims__(kRanks, 1, 1) __launch_bounds__(kPlanThreads)
    reserve_plan(PoolView p, const int *n_new, int *status, PoolWs w) {
    extern __shared__ int2 asks[];         // of this CTA's sequences: pages they need, and those among them that are copied
    __shared__ Board board;
    __shared__ unsigned long long sums[kPlanWarps];
    __shared__ int n_narrow, n_shared;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (p.n_seq + kRanks - 1) / kRanks, s0 = min(rank * per, p.n_seq), s1 = min(s0 + per, p.n_seq);
    int *count = w.list[1], *lowest = w.list[2], turn = 0;
    if (threadIdx.x == 0) n_narrow = n_shared = 0;
    __syncthreads();
    wait_for_inputs();

    // which blocks lack a page, and which have one that others hold too
    for (int s = s0 + warp; s < s1; s += kPlanWarps) {
        const Ask a = ask_of(p, n_new, s);
        const int *row = row_of(p, s);
        int need = 0, shared = 0;
        for (int j0 = a.first; j0 <= a.last; j0 += 32) {
            const bool in = j0 + lane <= a.last;
            const int page = in ? row[j0 + lane] : 0;
            const int held = in && names(p, page) ? p.refs[page] : 0;
            if (held > 1) {
                count[page] = -held;       // the same from all who write here
                lowest[page] = INT_MAX;
            }
            need += __popc(__ballot_sync(0xffffffffu, in && !names(p, page)));
            shared += __popc(__ballot_sync(0xffffffffu, held > 1));
        }
        if (lane == 0) {
            asks[s - s0] = make_int2(need, shared);
            if (a.narrow) atomicAdd(&n_narrow, 1);
            if (shared) atomicAdd(&n_shared, 1);
        }
    }
    __syncthreads();
    const Shares told = share(cluster, board, turn, both(n_narrow, n_shared));
    const int narrow = (int)(unsigned)told.all;
    if (told.all >> 32) {
        // f(sequence, block, page, lane's bits): the shared pages of this CTA's sequences, a warp at a time
        auto each_shared = [&](auto f) {
            for (int s = s0 + warp; s < s1; s += kPlanWarps) {
                if (!asks[s - s0].y) continue;
                const Ask a = ask_of(p, n_new, s);
                const int *row = row_of(p, s);
                int fresh = 0;
                for (int j0 = a.first; j0 <= a.last; j0 += 32) {
                    const bool in = j0 + lane <= a.last;
                    const int page = in ? row[j0 + lane] : -1;
                    const bool shared = names(p, page) && p.refs[page] > 1;
                    fresh += __popc(__ballot_sync(0xffffffffu, shared && f(s, page)));
                }
                __syncwarp();
                if (lane == 0) asks[s - s0] = make_int2(asks[s - s0].x, fresh);
                __syncwarp();
            }
        };
        each_shared([&](int s, int page) {
            atomicAdd(count + page, 1);
            atomicMin(lowest + page, s);
            return true;
        });
        cluster.sync();
        each_shared([&](int s, int page) { return __ldcg(count + page) != 0 || __ldcg(lowest + page) != s; });
        __syncthreads();
    }

    // places of the sequences among all that is needed
    unsigned long long run = 0;
    for (int i0 = 0; i0 < s1 - s0; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        const int2 a = i < s1 - s0 ? asks[i] : make_int2(0, 0);
        unsigned long long total;
        const unsigned long long at = run + block_scan(both(a.x + a.y, a.y), sums, total);
        if (i < s1 - s0) asks[i] = make_int2((int)(unsigned)at, (int)(at >> 32));
        run += total;
    }
    const Shares place = share(cluster, board, turn, run);
    const int total = (int)(unsigned)place.all, copies = (int)(place.all >> 32);
    const int my_copy = (int)(place.before >> 32), my_copies = (int)(run >> 32);

    // the lowest free pages
    int found = 0;
    for (int b = 0; b < p.n_pages && found < total; b += kSweep) {
        const int at = b + (rank * kPlanThreads + threadIdx.x) * kPer;
        const int4 r = load_refs(p, at, 1);
        unsigned long long sum;
        const unsigned free = (r.x <= 0) + (r.y <= 0) + (r.z <= 0) + (r.w <= 0);
        const unsigned long long mine = block_scan(free, sums, sum);
        const Shares all = share(cluster, board, turn, sum);
        int k = found + (int)(all.before + mine);
        auto put = [&](int page, int held) {
            if (held <= 0) {
                if (k < total) w.list[0][k] = page;
                ++k;
            }
        };
        put(at, r.x);
        put(at + 1, r.y);
        put(at + 2, r.z);
        put(at + 3, r.w);
        found += (int)all.all;
    }
    const bool done = found >= total && narrow == 0;
    if (rank == 0 && threadIdx.x == 0) {
        status[0] = max(total - found, 0);
        status[1] = narrow;
        w.head[0] = done ? copies : 0;
    }
    cluster.sync();
    if (done && total > 0) {
        for (int s = s0 + warp; s < s1; s += kPlanWarps) {
            const Ask a = ask_of(p, n_new, s);
            int *row = row_of(p, s);
            int k = (int)(unsigned)place.before + asks[s - s0].x, c = my_copy + asks[s - s0].y;
            for (int j0 = a.first; j0 <= a.last; j0 += 32) {
                const int j = j0 + lane;
                const bool in = j <= a.last;
                const int page = in ? row[j] : -1;
                const bool there = names(p, page);
                const bool moves = there && p.refs[page] > 1 && (__ldcg(count + page) != 0 || __ldcg(lowest + page) != s);
                const unsigned fresh = __ballot_sync(0xffffffffu, in && (!there || moves)), copy = __ballot_sync(0xffffffffu, moves);
                if (in && (!there || moves)) {
                    const int to = __ldcg(w.list[0] + k + __popc(fresh & lanes_below()));
                    row[j] = to;
                    p.refs[to] = 1;
                    if (moves)
                        w.moves[c + __popc(copy & lanes_below())] =
                            make_int4(page, to, min(max(a.len - (j << p.shift), 0), 1 << p.shift), 0);
                }
                k += __popc(fresh);
                c += __popc(copy);
            }
        }
    }
    cluster.sync();                        // all have read the counts, and nobody's board is written any more
    if (done)
        for (int i = threadIdx.x; i < my_copies; i += kPlanThreads) atomicSub(p.refs + w.moves[my_copy + i].x, 1);
}

// ---------------------------------------------------------------- compact

__global__ void __cluster_dims__(kRanks, 1, 1) __launch_bounds__(kPlanThreads)
    compact_plan(PoolView p, int *moved, int *n_used, PoolWs w) {
    __shared__ Board board;
    __shared__ unsigned long long sums[kPlanWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), tid = rank * kPlanThreads + threadIdx.x;
    int *holes = w.list[0], *high = w.list[1], *map = w.list[2], turn = 0;
    wait_for_inputs();
    auto live = [](const int4 &r) { return (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0); };
    unsigned long long sum, n = 0;
    for (int b = 0; b < p.n_pages; b += kSweep) n += live(load_refs(p, b + tid * kPer, 0));
    block_scan(n, sums, sum);
    const int used = (int)share(cluster, board, turn, sum).all;
    // the free pages below `used` and the pages in use from there on, in order
    int before = 0, n_high = 0;
    for (int b = 0; b < p.n_pages; b += kSweep) {
        const int at = b + tid * kPer;
        const int4 r = load_refs(p, at, 0);
        const int held[kPer] = {r.x, r.y, r.z, r.w};
        unsigned c[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (at + i < p.n_pages) c[at + i >= used] += held[i] > 0;
        const unsigned long long mine = block_scan(both(c[0], c[1]), sums, sum);
        const Shares all = share(cluster, board, turn, sum);
        int low = before + (int)(unsigned)(all.before + mine), up = n_high + (int)((all.before + mine) >> 32);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int page = at + i;
            if (page >= p.n_pages) continue;
            if (page < used) {
                if (held[i] <= 0) holes[page - low] = page;
                low += held[i] > 0;
                if (moved) moved[page] = held[i] > 0 ? page : -1;
            } else {
                if (held[i] > 0) high[up++] = page;
                map[page] = -1;
                if (moved && held[i] <= 0) moved[page] = -1;
            }
        }
        before += (int)(unsigned)all.all;
        n_high += (int)(all.all >> 32);
    }
    if (tid == 0) {
        *n_used = used;
        w.head[0] = n_high;
    }
    cluster.sync();
    for (int i = tid; i < n_high; i += kRanks * kPlanThreads) {
        const int from = __ldcg(high + i), to = __ldcg(holes + i);
        p.refs[to] = p.refs[from];
        p.refs[from] = 0;
        map[from] = to;
        if (moved) moved[from] = to;
        w.moves[i] = make_int4(from, to, 1 << p.shift, 0);
    }
    cluster.sync();                        // no CTA leaves while its board may be written
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
    int n_layers, heads;                   // heads: the most of a layer
    PoolLayer layer[kLayersAtOnce];
};

// A warp at a time takes a move's tokens of one layer, K or V, and kv head: up to 32 KB in one piece.
__global__ void __launch_bounds__(kMoveThreads) move_pages(const __grid_constant__ MoveArgs a) {
    wait_for_inputs();
    const int lane = threadIdx.x & 31, per_page = a.n_layers * 2 * a.heads;
    const long long warps = (long long)gridDim.x * (kMoveThreads / 32), n = (long long)a.head[0] * per_page;
    for (long long i = (long long)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); i < n; i += warps) {
        const int move = (int)(i / per_page), part = (int)(i - (long long)move * per_page);
        const int l = part / (2 * a.heads), kv = part / a.heads - 2 * l, h = part - (2 * l + kv) * a.heads;
        const PoolLayer &layer = a.layer[l];
        const int4 m = a.moves[move];
        if (h >= layer.n_kv || m.z == 0) continue;
        const size_t row = (size_t)layer.d << a.p.shift;      // bytes of a head in a page
        const size_t from = (size_t)m.x * layer.n_kv + h, to = (size_t)m.y * layer.n_kv + h;
        int8_t *codes = kv ? layer.v : layer.k;
        const uint4 *src = reinterpret_cast<const uint4 *>(codes + from * row);
        uint4 *dst = reinterpret_cast<uint4 *>(codes + to * row);
        const int units = m.z * (layer.d / 16);
        constexpr int AT_ONCE = 8;
        for (int u = lane; u < units; u += 32 * AT_ONCE) {
            uint4 x[AT_ONCE];
#pragma unroll
            for (int e = 0; e < AT_ONCE; ++e)
                if (u + 32 * e < units) x[e] = __ldcs(src + u + 32 * e);
#pragma unroll
            for (int e = 0; e < AT_ONCE; ++e)
                if (u + 32 * e < units) __stcs(dst + u + 32 * e, x[e]);
        }
        if (lane == 0) {
            float *scale = kv ? layer.v_scale : layer.k_scale;
            scale[to] = scale[from];
        }
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

cudaError_t launch_moves(const PoolView &p, const PoolLayer *layers, int n_layers, const PoolWs &w, const int *n_used,
                         cudaStream_t s, const DeviceInfo &dev) {
    MoveArgs a;
    a.p = p;
    a.head = w.head;
    a.moves = w.moves;
    a.map = n_used ? w.list[2] : nullptr;
    a.n_used = n_used;
    int l = 0;
    do {
        a.n_layers = n_layers - l < kLayersAtOnce ? n_layers - l : kLayersAtOnce;
        a.heads = 1;
        for (int i = 0; i < a.n_layers; ++i) {
            a.layer[i] = layers[l + i];
            if (a.layer[i].n_kv > a.heads) a.heads = a.layer[i].n_kv;
        }
        const cudaError_t e = launch(move_pages, dev.sm_count * 4, kMoveThreads, 0, s, a);
        if (e != cudaSuccess) return e;
        a.map = a.n_used = nullptr;
        l += a.n_layers;
    } while (l < n_layers);
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv_fork(const PoolView &p, int n, const int *from, const int *to, const int *tokens, const PoolWs &w,
                           cudaStream_t s) {
    const cudaError_t e = launch(fork_take, n, kRowThreads, 0, s, p, from, to, tokens, w);
    return e == cudaSuccess ? launch(fork_put, n, kRowThreads, 0, s, p, from, to, w) : e;
}

cudaError_t launch_kv_free(const PoolView &p, int n, const int *seq, const int *begin, const int *end, cudaStream_t s) {
    return launch(free_rows, n, kRowThreads, 0, s, p, seq, begin, end);
}

cudaError_t launch_kv_reserve(const PoolView &p, const PoolLayer *layers, int n_layers, const int *n_new, int *status,
                              const PoolWs &w, cudaStream_t s, const DeviceInfo &dev) {
    constexpr int most = kPoolMaxSeq / kRanks * (int)sizeof(int2);
    static PerDeviceOnce once;
    cudaError_t e = once.run([] { return cudaFuncSetAttribute(reserve_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, most); });
    if (e != cudaSuccess) return e;
    e = launch(reserve_plan, kRanks, kPlanThreads, (size_t)((p.n_seq + kRanks - 1) / kRanks) * sizeof(int2), s, p, n_new, status, w);
    return e == cudaSuccess && n_layers > 0 ? launch_moves(p, layers, n_layers, w, nullptr, s, dev) : e;
}

cudaError_t launch_kv_compact(const PoolView &p, const PoolLayer *layers, int n_layers, int *moved, int *n_used,
                              const PoolWs &w, cudaStream_t s, const DeviceInfo &dev) {
    const cudaError_t e = launch(compact_plan, kRanks, kPlanThreads, 0, s, p, moved, n_used, w);
    return e == cudaSuccess ? launch_moves(p, layers, n_layers, w, n_used, s, dev) : e;
}

}  // namespace pqk
