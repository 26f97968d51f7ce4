// How the attention kernels split their work over CTAs, decided on the device
// from the lengths there.
//
// The rows of one sequence and kv head (its tokens times the n_q / n_kv query
// heads of that kv head, token-major) are cut into row tiles of RT rows; the
// tokens that a row tile sees into tiles of KT tokens.  A unit is one token
// tile of one row tile and kv head; the units of an item (sequence, kv head,
// row tile) are consecutive.  All units, in the order sequence, kv head, row
// tile, token tile, are cut into one contiguous equal range per CTA, so that
// long and short sequences load every CTA alike; an item cut by a range's end
// is joined from its CTAs' parts, in CTA order, by whichever of them is the
// last to finish.
#pragma once

#include "kv_device.cuh"

namespace pqk {

constexpr int kAttnMaxGrid = 320;      // CTAs at most (parts and counters in the workspace)

// One row tile: its rows, the positions they cover, the token tiles they see.
struct RowTile {
    int rows;            // rows of the tile (the last one of a sequence may be short)
    int pos0, pos1;      // positions of the first and the last row's token
    int sinks, w0;       // unit y is token tile y below sinks, else w0 + (y - sinks)
    int units;           // at least 1, so that rows that see nothing are written
};

template <int RT, int KT>
__device__ __forceinline__ RowTile row_tile(const AttnArgs &p, int m, int len, int j, int group) {
    RowTile t;
    const int first = j * RT;
    t.rows = min(RT, m * group - first);
    t.pos0 = len - m + first / group;
    t.pos1 = len - m + (first + t.rows - 1) / group;
    const int cap = p.c.table_ld * p.c.page;
    const int end = t.pos1 < 0 ? 0 : min(t.pos1, cap - 1) / KT + 1;          // token tiles up to the last row's
    const int from = p.window > 0 ? max(0, t.pos0 - p.window + 1) / KT : 0;   // first tile of the first row's window
    t.w0 = min(from, end);
    t.sinks = min(p.n_sink / KT + (p.n_sink % KT != 0), t.w0);
    t.units = max(1, t.sinks + end - t.w0);
    return t;
}

// Where a CTA is in its range.  Every role of the CTA walks its own copy.
template <int RT, int KT> struct UnitWalk {
    int s, h, j, y;          // sequence, kv head, row tile, unit of the row tile
    int r0, m, len, tiles;   // of the sequence: first row, tokens, length, row tiles
    RowTile t;

    __device__ __forceinline__ void seq(const AttnArgs &p, int group) {
        seq_rows(p.c, s, r0, m);
        len = seq_len(p.c, s);
        tiles = (m * group + RT - 1) / RT;
    }
    // Enter sequence `seq_` at unit x of it, `per_head` units per kv head.
    __device__ __forceinline__ void start(const AttnArgs &p, int group, int seq_, long long x, long long per_head) {
        s = seq_;
        seq(p, group);
        h = (int)(x / per_head);
        long long left = x % per_head;
        for (j = 0;; ++j) {
            t = row_tile<RT, KT>(p, m, len, j, group);
            if (left < t.units) break;
            left -= t.units;
        }
        y = (int)left;
    }
    __device__ __forceinline__ int token0() const { return (y < t.sinks ? y : t.w0 + (y - t.sinks)) * KT; }
    // The next unit; returns whether it belongs to another item.
    __device__ __forceinline__ bool next(const AttnArgs &p, int group) {
        if (++y < t.units) return false;
        y = 0;
        if (++j == tiles) {
            j = 0;
            if (++h == p.c.n_kv) {
                h = 0;
                do {
                    if (++s >= p.c.n_seq) return true;      // past the end: no further unit is taken
                    seq(p, group);
                } while (m == 0);
            }
        }
        t = row_tile<RT, KT>(p, m, len, j, group);
        return true;
    }
};

// The CTA's range of units and where it starts.
struct UnitRange {
    long long total, first, last;     // units of the call; [first, last) is this CTA's
    long long offset, per_head;       // in sequence seq: first unit's index, units per kv head
    int grid;                         // CTAs that have units
    int seq;
};

__device__ __forceinline__ long long range_begin(long long c, long long total, int grid) { return c * total / grid; }
__device__ __forceinline__ int range_owner(long long u, long long total, int grid) { return (int)(((u + 1) * grid - 1) / total); }

// Units of one kv head of sequence s.
template <int RT, int KT> __device__ __forceinline__ long long seq_units(const AttnArgs &p, int s, int group) {
    int r0, m;
    seq_rows(p.c, s, r0, m);
    if (m == 0) return 0;
    const int len = seq_len(p.c, s), tiles = (m * group + RT - 1) / RT;
    long long n = 0;
    for (int j = 0; j < tiles; ++j) n += row_tile<RT, KT>(p, m, len, j, group).units;
    return n;
}

// Finds the range of CTA blockIdx.x, by all NT threads of the block; the
// answer lies in shared memory (`out`).  Ends with a barrier.
template <int RT, int KT, int NT> __device__ __forceinline__ void find_range(const AttnArgs &p, int group, UnitRange *out) {
    __shared__ long long warp_sum[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_seq = p.c.n_seq;
    long long total = 0, first = 0, before = 0;
    int grid = 1;
    // with more sequences than threads a first pass adds the units up
    for (int pass = n_seq > NT ? 0 : 1; pass < 2; ++pass) {
        before = 0;
        for (int s0 = 0; s0 < n_seq; s0 += NT) {
            const long long mine = s0 + tid < n_seq ? seq_units<RT, KT>(p, s0 + tid, group) : 0;
            long long incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            __syncthreads();
            if (lane == 31) warp_sum[warp] = incl;
            __syncthreads();
            long long add = before, all = 0;
#pragma unroll
            for (int w = 0; w < NT / 32; ++w) {
                if (w < warp) add += warp_sum[w];
                all += warp_sum[w];
            }
            incl += add;
            before += all;
            if (pass == 0) continue;
            if (n_seq <= NT) total = before * p.c.n_kv;
            grid = (int)min((long long)gridDim.x, max(total, 1ll));
            first = range_begin(blockIdx.x, total, grid);
            const long long lo = (incl - mine) * p.c.n_kv, hi = incl * p.c.n_kv;
            if ((int)blockIdx.x < grid && first >= lo && first < hi) {
                out->seq = s0 + tid;
                out->offset = first - lo;
                out->per_head = mine;
            }
        }
        if (pass == 0) total = before * p.c.n_kv;
    }
    if (tid == 0) {
        out->total = total;
        out->grid = grid;
        const bool any = total > 0 && (int)blockIdx.x < grid;
        out->first = any ? first : 0;
        out->last = any ? range_begin(blockIdx.x + 1, total, grid) : 0;
    }
    __syncthreads();
}

// Workspace: counters of the items that several CTAs share (item counter =
// index of its first CTA; zero between calls), then two parts per CTA (slot 2c:
// the item its range starts in, 2c + 1: the one it ends in).  A part is RT x D
// f32 sums, then RT maxima and RT weight sums.
__host__ __device__ constexpr size_t attn_counter_bytes() { return (size_t)kAttnMaxGrid * 4; }
__host__ __device__ constexpr size_t attn_part_floats(int rt, int d) { return (size_t)rt * (d + 2); }

}  // namespace pqk
