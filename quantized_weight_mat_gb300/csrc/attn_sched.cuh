// How the attention kernels split their work over CTAs, decided on the device
// from the lengths there.
//
// The rows of one sequence and kv head (its tokens times the n_q / n_kv query
// heads of that kv head, token-major) are cut into row tiles of RT rows; the
// tokens that a row tile sees into tiles of KT tokens.  A unit is one token
// tile of one row tile and kv head; the units of an item (sequence, kv head,
// row tile) are consecutive.  Places count 1 for every unit and COST for
// every item before its first one (what its rows' loads and the join cost, in units).  All
// places, in the order sequence, kv head, row tile, token tile, are cut into
// one contiguous equal range per CTA, so that long and short sequences load every CTA
// alike; an item cut by a range's end is joined from its CTAs' parts, in CTA
// order, by a second small kernel (one SM reading all parts of an item of a long
// sequence took 6 us of 52, and the last CTA's fence and counter 1 us of every split).
#pragma once

#include "kv_device.cuh"

namespace pqk {

constexpr int kAttnMaxGrid = 320;      // CTAs at most (parts in the workspace)

// A sequence's row tiles that one lane counts by itself; more may be spread over the lanes (4 sequences of 110, one
// by one: 14000 cycles before the first unit, spread 8000; 32 sequences of 9 the other way round: 20000 spread).
constexpr int kFewTiles = 4;

// One row tile: its rows, the positions they cover, the token tiles they see.
struct RowTile {
    int rows;            // rows of the tile (the last one of a sequence may be short)
    int pos0, pos1;      // positions of the first and the last row's token
    int sinks, w0;       // unit y is token tile y below sinks, else w0 + (y - sinks)
    int units;           // at least 1, so that rows that see nothing are written
};

template <int RT, int KT> __device__ __forceinline__ RowTile row_tile(const AttnArgs &p, int m, int len, int j) {
    RowTile t;
    const int first = j * RT;
    t.rows = min(RT, m * p.group.d - first);
    t.pos0 = len - m + p.group.div(first);
    t.pos1 = len - m + p.group.div(first + t.rows - 1);
    const int cap = p.c.table_ld * p.c.page;
    const int end = t.pos1 < 0 ? 0 : min(t.pos1, cap - 1) / KT + 1;          // token tiles up to the last row's
    const int from = p.window > 0 ? max(0, t.pos0 - p.window + 1) / KT : 0;   // first tile of the first row's window
    t.w0 = min(from, end);
    t.sinks = min(p.n_sink / KT + (p.n_sink % KT != 0), t.w0);
    t.units = max(1, t.sinks + end - t.w0);
    return t;
}

// 64-bit quotients are slow; nearly every call's numbers fit 32 bits.
__device__ __forceinline__ long long div_places(long long a, long long b) {
    return (((unsigned long long)a | (unsigned long long)b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// The cut of all places into ranges: the first `longer` ranges have size + 1
// places, the others size.
struct Cut {
    long long total, size, longer;
    int grid;                         // ranges: CTAs that have work

    // At most `most` ranges, of at least LEAST places. A range of an item's cost alone has no unit, and its CTA no work.
    template <int LEAST> static __device__ __forceinline__ Cut make(long long total, const FastDiv &most) {
        Cut c;
        c.total = total;
        if (total < 0x40000000ll && (int)total >= LEAST * most.d) {      // nearly every call: no division
            c.grid = most.d;
            c.size = most.div((int)total);
        } else {
            c.grid = (int)min((long long)most.d, max(div_places(total, LEAST), 1ll));
            c.size = div_places(total, c.grid);
        }
        c.longer = total - c.size * c.grid;
        return c;
    }
    __device__ __forceinline__ long long begin(int c) const { return c * size + min((long long)c, longer); }
    __device__ __forceinline__ int owner(long long w) const {
        const long long mid = longer * (size + 1);
        return (int)(w < mid ? div_places(w, size + 1) : longer + div_places(w - mid, size));
    }
};

// Where a CTA is in its range.
template <int RT, int KT, int COST> struct UnitWalk {
    long long w;             // place of the unit
    int s, h, j, y;          // sequence, kv head, row tile, unit of the row tile
    int r0, m, len, tiles;   // of the sequence: first row, tokens, length, row tiles
    RowTile t;

    __device__ __forceinline__ void seq(const AttnArgs &p) {
        seq_rows(p.c, s, r0, m);
        len = seq_len(p.c, s);
        tiles = (m * p.group.d + RT - 1) / RT;
    }
    // Places of one kv head of the sequence.
    __device__ __forceinline__ long long places(const AttnArgs &p) const {
        long long n = 0;
        for (int i = 0; i < tiles; ++i) n += tile_places(p, i);
        return n;
    }
    __device__ __forceinline__ int tile_places(const AttnArgs &p, int i) const { return row_tile<RT, KT>(p, m, len, i).units + COST; }
    // By one warp: the first unit at place `first` or after it, which lies `x` into the
    // sequence, of `per_head` places per kv head.
    __device__ __forceinline__ void start(const AttnArgs &p, long long first, long long x, long long per_head) {
        h = (int)div_places(x, per_head);
        long long left = x - h * per_head;
        j = 0;
        if (tiles > kFewTiles) {      // 32 row tiles at a time, one per lane
            const int lane = threadIdx.x & 31;
            for (;; j += 32) {
                const int n = j + lane < tiles ? row_tile<RT, KT>(p, m, len, j + lane).units + COST : 0;
                int incl = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += up;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, left < incl);
                const int at = hit ? __ffs((int)hit) - 1 : 31;
                left -= __shfl_sync(0xffffffffu, hit ? incl - n : incl, at);
                if (hit) {
                    j += at;
                    break;
                }
                if (j + 32 >= tiles) break;      // not reached: the places end in the sequence
            }
            t = row_tile<RT, KT>(p, m, len, j);
        } else {
            for (;; ++j) {
                t = row_tile<RT, KT>(p, m, len, j);
                if (left < t.units + COST) break;
                left -= t.units + COST;
            }
        }
        y = max(0, (int)left - COST);
        w = first + y + COST - left;
    }
    __device__ __forceinline__ int token0() const { return (y < t.sinks ? y : t.w0 + (y - t.sinks)) * KT; }
    // To the first unit of the next item.
    __device__ __forceinline__ void next_item(const AttnArgs &p) {
        w += t.units - y + COST;
        y = 0;
        if (++j == tiles) {
            j = 0;
            if (++h == p.c.n_kv) {
                h = 0;
                do {
                    if (++s >= p.c.n_seq) return;      // past the end: w is past every range
                    seq(p);
                } while (m == 0);
            }
        }
        t = row_tile<RT, KT>(p, m, len, j);
    }
};

// Places of the whole call, by one warp; lane 0's `walk` of every group of 32
// sequences is not kept.
template <class Walk> __device__ __forceinline__ long long warp_places(const AttnArgs &p, int s, Walk &walk, int lane) {
    walk.s = s + lane;
    walk.m = 0;
    if (walk.s < p.c.n_seq) walk.seq(p);
    const int tiles = walk.m > 0 ? walk.tiles : 0;
    // a few sequences of many row tiles one after the other, by all lanes: about 4 row tiles' time each, and one more
    // per 32 of them
    unsigned many = __ballot_sync(0xffffffffu, tiles > kFewTiles);
    if (many) {
        const int most = __reduce_max_sync(0xffffffffu, tiles);
        if (most <= __popc(many) * (4 + most / 32)) many = 0;
    }
    long long n = tiles > 0 && !((many >> lane) & 1) ? walk.places(p) : 0;
    for (; many; many &= many - 1) {
        const int src = __ffs((int)many) - 1, count = __shfl_sync(0xffffffffu, tiles, src);
        Walk of = walk;
        of.m = __shfl_sync(0xffffffffu, walk.m, src);
        of.len = __shfl_sync(0xffffffffu, walk.len, src);
        long long sum = 0;
        for (int i = lane; i < count; i += 32) sum += of.tile_places(p, i);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == src) n = sum;
    }
    return n;
}

// By one warp: the places of the call, cut into ranges of at least LEAST, and
// `walk` at the first unit of CTA blockIdx.x's range [first, last); first ==
// last when it has none.
template <class Walk, int LEAST>
__device__ __forceinline__ Cut find_range(const AttnArgs &p, Walk &walk, long long &first, long long &last) {
    const int lane = threadIdx.x & 31, n_seq = p.c.n_seq;
    long long total = 0, incl = 0, mine = 0;
    for (int s = 0; s < n_seq; s += 32) {
        mine = warp_places(p, s, walk, lane);
        incl = mine;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        incl += total;
        total = __shfl_sync(0xffffffffu, incl, 31);
    }
    const Cut cut = Cut::make<LEAST>(total * p.c.n_kv, p.grid);
    first = last = 0;
    if (total == 0 || (int)blockIdx.x >= cut.grid) return cut;
    first = cut.begin(blockIdx.x);
    last = cut.begin(blockIdx.x + 1);
    long long before = 0;
    for (int s = 0;; s += 32) {
        if (n_seq > 32) {      // else the first loop's one group is still there
            mine = warp_places(p, s, walk, lane);
            incl = mine;
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            incl += before;
        }
        const long long lo = (incl - mine) * p.c.n_kv;
        const unsigned hit = __ballot_sync(0xffffffffu, first >= lo && first < incl * p.c.n_kv);
        if (hit) {
            const int src = __ffs((int)hit) - 1;
            walk.s = __shfl_sync(0xffffffffu, walk.s, src);
            walk.r0 = __shfl_sync(0xffffffffu, walk.r0, src);
            walk.m = __shfl_sync(0xffffffffu, walk.m, src);
            walk.len = __shfl_sync(0xffffffffu, walk.len, src);
            walk.tiles = __shfl_sync(0xffffffffu, walk.tiles, src);
            walk.start(p, first, first - __shfl_sync(0xffffffffu, lo, src), __shfl_sync(0xffffffffu, mine, src));
            return cut;
        }
        before = __shfl_sync(0xffffffffu, incl, 31);
        if (s + 32 >= n_seq) break;
    }
    first = last = 0;
    return cut;
}

// One item of a CTA, as its walking warp hands it to the others.
struct Item {
    int r0, m, len, j, h;      // see UnitWalk
    int y0, n;                 // its units of this CTA: y0 .. y0 + n - 1; n == 0: no more items
    int rows, pos0, pos1, sinks, w0;
    int whole;                 // no other CTA has units of it
    int slot;                  // its part's place in the workspace
};

template <class Walk> __device__ __forceinline__ Item item_of(const Walk &at, long long first, long long last) {
    Item it;
    it.r0 = at.r0;
    it.m = at.m;
    it.len = at.len;
    it.j = at.j;
    it.h = at.h;
    it.y0 = at.y;
    it.rows = at.t.rows;
    it.pos0 = at.t.pos0;
    it.pos1 = at.t.pos1;
    it.sinks = at.t.sinks;
    it.w0 = at.t.w0;
    it.n = (int)min((long long)(at.t.units - at.y), last - at.w);
    const long long w0 = at.w - at.y, w1 = w0 + at.t.units - 1;      // places of its first and last unit
    it.whole = w0 >= first && w1 < last;
    it.slot = 2 * (int)blockIdx.x + (w0 < first ? 0 : 1);
    return it;
}

// Workspace: one Split per CTA, then two parts per CTA (slot 2c: an item that
// began in an earlier CTA, 2c + 1: one that begins here and goes on).  A part is
// RT x D f32 sums, then RT pairs of a maximum and a weight sum.  Nothing in it
// outlives the call.
struct Split {
    int c1, rows, r0, j, h;      // the item that begins here and goes on, to CTA c1 (-1: none does)
};
__host__ __device__ constexpr size_t attn_splits_bytes() { return (kAttnMaxGrid * sizeof(Split) + 15) / 16 * 16; }
__host__ __device__ constexpr size_t attn_part_floats(int rt, int d) { return (size_t)rt * (d + 2); }   // a multiple of 4 (rt is one of 8)
// The item at `at` if it begins in this CTA (range [first, last)) and goes on.
template <class Walk> __device__ __forceinline__ Split split_of(const Walk &at, const Cut &cut, long long first, long long last) {
    const long long w0 = at.w - at.y, w1 = w0 + at.t.units - 1;
    Split s;
    s.c1 = w0 >= first && w1 >= last ? cut.owner(w1) : -1;
    s.rows = at.t.rows;
    s.r0 = at.r0;
    s.j = at.j;
    s.h = at.h;
    return s;
}
__device__ __forceinline__ Split *splits_of(const AttnArgs &p) { return reinterpret_cast<Split *>(p.ws); }
__device__ __forceinline__ float *parts_of(const AttnArgs &p) { return reinterpret_cast<float *>(p.ws + attn_splits_bytes()); }

}  // namespace pqk
