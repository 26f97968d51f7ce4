// Attention over the paged 8-bit cache for few rows per sequence (decode steps,
// drafted tokens, short pieces), head sizes 64 and 128.
//
// Bound by the bytes of K and V: every code is read once per 8 or 16 rows, so
// the products go to the tensor cores and the loads to TMA.  Softmax in one
// pass (running maximum m and sum l of exp2(s - m)):
//     S = K q'      (16 tokens x 8 rows per mma.sync m16n8k16)
//     O += V^T P    (16 elements x 8 rows; f32 rows' tile by tile, see below: over 131072 tokens the products' own sums
//                    left O 2.5e-5 short, now 9e-7 off in all; 2048 rows over 10240 tokens 2077 us -> 2202)
// with K and V as the A operands, so that rows fill the narrow side (N = 8) and
// one token's code is loaded by exactly one thread.  Operands are exact where
// they can be: int8 codes become fp16 by a byte permute and one subtraction
// (0x6400 | (code + 128) is 1152 + code); q is scaled per row by a power of
// two, its largest element to 2^9..2^10 (16-bit rows as one fp16, exact but for bf16 elements 2^26 below
// the row's largest; f32 rows as a pair, 2^-21 of each element or 2^-34 of the largest).
// The softmax weights enter in fp16 for bf16 rows (their 11 bits lie far below
// the output's 8) and as an fp16 pair for f16 and f32 rows (one fp16 would add half
// as much again to f16's own rounding, and the loads hide the second product), already times
// their page's V scale, over a power of two R that follows the largest product of
// a weight and its page's scale: not the largest scale, since a page that weighs
// nothing may have one far above the page that holds the weight.  fp16 holds
// 2^15 of R down to 2^-24 of it (kLift), so a weight is off by 2^-12 of itself (2^-23 as
// a pair) or by 2^-32 of the row's largest product.  The sum l is of the weights before,
// over their own running maximum.  Both references are whole powers of two (no
// rounding when they move) and move rarely, when a new value passes them by
// 2^8: rescaling O costs a warp half a tile's time.
//
// ldmatrix gives a thread four codes of one token (K) or, transposed in 2-byte
// units, two elements of two tokens (V): the byte permutes of the conversion
// sort them, so the transposition of V costs nothing.
//
// 64 sequences of 2560 tokens (32 heads over 8 of 128, bf16) take 61.6 us, 5.4 TB/s
// of K and V where the same loads without the arithmetic take 59; one sequence of 131072
// 54, of 4096 (f32) 12.0, of which 4.5 pass before the first tile is there (lengths,
// table, TMA) and 2.5 in the second kernel.  More warps of 16 tokens each: 78 us against 64.
//
// Pipeline: warp 4 walks the CTA's units (the other warps get each item from it
// through a small ring) and brings 128-token tiles of K and V through a ring of
// stages (one TMA box per page, swizzled; page numbers read for four tiles at a
// time; page scales by 4-byte asynchronous copies onto the same barrier); warp 5
// turns the next item's rows of q into fp16 operands in shared memory while
// the present item runs; warps 0-3 take 32 tokens of a tile each, as two independent
// groups of 16, with a running maximum of their own, and join at the end of
// an item.

#include <type_traits>

#include "attn_common.cuh"

namespace pqk {
namespace {

constexpr int kConsumers = 4;                // warps, 32 tokens of a tile each
constexpr int kThreads = 32 * (kConsumers + 2);
constexpr int kItemCost = 2;                 // places of an item beside its units (64 ragged sequences: 1: 70.7 us, 2: 65.6, 3: 67.4)
constexpr int kLeast = 2;                    // places of a CTA (one f32 row over 4096 tokens, before its sums were added up by tiles: 1: 12.7 us, 2: 11.7, 3: 12.7; over 512: 8.6, 9.3, 10.0)
constexpr int kItems = 8;                    // items that the walking warp may be ahead (more than the tiles it looks up at a time)

template <int D> __host__ __device__ constexpr int tile_bytes() { return KT * D; }
template <int D> __host__ __device__ constexpr int stages() { return D == 128 ? 3 : 6; }
// q as fp16: row pitch in elements (8 words past a multiple of 32 banks)
template <int D> __host__ __device__ constexpr int q_pitch() { return D + 16; }
template <int D> __host__ __device__ constexpr int red_pitch() { return D + 8; }
// One buffer for q (hi rows, for f32 lo rows) while an item runs, and for the
// join of 4 rows of each warp at its end.
template <int D, int NT, bool PAIR> __host__ __device__ constexpr int shared_bytes() {
    const int q = 8 * NT * (PAIR ? 2 : 1) * q_pitch<D>() * 2, red = kConsumers * 4 * red_pitch<D>() * 4;
    return q > red ? q : red;
}
template <int D, int NT, bool PAIR> __host__ __device__ constexpr int smem_bytes() {
    return 1024 + stages<D>() * 2 * tile_bytes<D>() + shared_bytes<D, NT, PAIR>();
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// n + add for a small whole number n, without the conversion instruction (a quarter of the rate of additions, and the
// exponentials' unit: 2048 f32 rows over 10240 tokens 31 us more with it).
__device__ __forceinline__ float small_float(int n, float add) { return __int_as_float(0x4b400000 + n) - (12582912.f - add); }
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <class T, int D, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    attn_mma(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, AttnArgs p) {
    constexpr int RT = 8 * NT, NS = stages<D>(), CH = D / 16;
    constexpr bool PAIR = sizeof(T) == 4;            // q as fp16 pairs
    constexpr bool WPAIR = !std::is_same<T, __nv_bfloat16>::value;      // the weights as fp16 pairs
    constexpr int kLift = 7;                         // weights are at most 2^kSlack R: this far up, fp16 holds them and as many small ones as it can
    constexpr int RLD = red_pitch<D>(), QP = q_pitch<D>();
    constexpr int AHEAD_C = NT == 1 ? CH / 2 : 1;    // K chunk pairs loaded ahead of their use
    using Walk = UnitWalk<RT, KT, kItemCost>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[NS], empty[NS], i_full[kItems], i_empty[kItems], q_full, q_empty;
    __shared__ __align__(16) TileMeta meta[NS];
    __shared__ Item items[kItems];
    __shared__ long long q_out[RT];
    __shared__ float red_m[kConsumers][RT], red_l[kConsumers][RT], q_fac[RT];
    __shared__ int q_pos[RT];
    __shared__ volatile int stop;

    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *shared = ring + NS * 2 * tile_bytes<D>();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        stop = 0;
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1 + kGroups);
            mbar_init(&empty[i], kConsumers);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&i_full[i], 1);
            mbar_init(&i_empty[i], 2);
        }
        mbar_init(&q_full, 1);
        mbar_init(&q_empty, 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 32 * kConsumers) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
    }
    __syncthreads();
    // what the preceding kernels on the stream wrote (lengths, table, codes, q)
    // is complete after this; the next kernel may then be scheduled beside this one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    if (warp == kConsumers + 1) {
        // ---------------- rows of q ----------------
        constexpr int LPR = D / 4, RPP = 32 / LPR, NP = RT / RPP;      // lanes per row, rows per pass, passes
        const int sub = lane / LPR, col = lane % LPR;
        for (uint32_t k = 0;; ++k) {
            if (!mbar_wait(&i_full[k % kItems], (k / kItems) & 1u)) return;
            const Item it = items[k % kItems];
            __syncwarp();
            if (lane == 0) mbar_arrive(&i_empty[k % kItems]);
            if (it.n == 0) return;
            float v[NP][4];
            int tok[NP], head[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int r = i * RPP + sub, rr = it.j * RT + r;
                tok[i] = p.group.div(rr);
                head[i] = it.h * p.group.d + rr - tok[i] * p.group.d;
                if (r < it.rows)
                    load4(static_cast<const T *>(p.q) + (it.r0 + tok[i]) * p.ldq + (long long)head[i] * D + 4 * col, v[i]);
                else v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
            }
            if (!mbar_wait(&q_empty, (k + 1) & 1u)) return;
            __half *q = reinterpret_cast<__half *>(shared);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int r = i * RPP + sub;
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(v[i][e]) & 0x7fffffffu);
#pragma unroll
                for (int w = LPR / 2; w > 0; w >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, w));
                const int ex = tc_scale_exponent(top);
                const float up = __uint_as_float((uint32_t)(127 + ex) << 23), down = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] *= up;
                const uint32_t h[2] = {pack2(v[i][0], v[i][1]), pack2(v[i][2], v[i][3])};
                *reinterpret_cast<uint2 *>(q + r * QP + 4 * col) = make_uint2(h[0], h[1]);
                if constexpr (PAIR) {
                    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&h[0]));
                    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&h[1]));
                    *reinterpret_cast<uint2 *>(q + (RT + r) * QP + 4 * col) =
                        make_uint2(pack2(v[i][0] - a.x, v[i][1] - a.y), pack2(v[i][2] - b.x, v[i][3] - b.y));
                }
                if (col == 0) {
                    q_fac[r] = down * (p.scale * kLog2e);
                    q_pos[r] = r < it.rows ? it.len - it.m + tok[i] : -1;
                    q_out[r] = (it.r0 + tok[i]) * p.ldo + (long long)head[i] * D;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full);
        }
        return;
    }

    if (warp == kConsumers) {
        // ---------------- producer ----------------
        constexpr int BATCH = 32 / kGroups;                    // tiles looked up at a time
        const int g = lane % kGroups, sub = lane / kGroups;
        Walk at;
        long long first, last;
        const Cut cut = find_range<Walk, kLeast>(p, at, first, last);
        Split split;                       // of the last item: only that can go on in another CTA
        split.c1 = -1;
        if (lane == 0) splits_of(p)[blockIdx.x].c1 = -1;      // should a wait below run out
        int slot = 0;
        uint32_t phase = 1, k = 0;
        bool fresh = true;
        at.w = first == last ? last : at.w;
        while (at.w < last) {
            // lane kGroups * i + g looks up group g of the i-th unit from here
            int tok = 0, seq = 0, head = 0, n = 0;
            for (; n < BATCH && at.w < last; ++n) {
                if (fresh) {
                    fresh = false;
                    if (!mbar_wait(&i_empty[k % kItems], (k / kItems + 1) & 1u)) return;
                    if (lane == 0) {
                        items[k % kItems] = item_of(at, first, last);
                        mbar_arrive(&i_full[k % kItems]);
                    }
                    ++k;
                }
                if (sub == n) {
                    tok = at.token0() + 16 * g;
                    seq = at.s;
                    head = at.h;
                }
                if (at.w + 1 == last) split = split_of(at, cut, first, last);
                if (at.y + 1 < at.t.units) {
                    ++at.y;
                    ++at.w;
                } else {
                    at.next_item(p);
                    fresh = true;
                }
            }
            const int pg = sub < n ? page_of(p.c, seq, tok / p.c.page) : -1;
            for (int i = 0; i < n; ++i) {
                if (!mbar_wait(&empty[slot], phase)) return;
                if (sub == i) meta[slot].have[g] = pg >= 0;
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(&full[slot], 2 * tile_bytes<D>());
                __syncwarp();
                if (sub == i) {
                    if (16 * g % p.c.page == 0) {
                        // no page: a box outside the tensor, which reads as zeros
                        const int row = head * p.c.page + tok % p.c.page, z = pg >= 0 ? pg : p.c.n_pages;
                        const uint32_t dst = smem_u32(ring + slot * 2 * tile_bytes<D>()) + 16 * g * D;
                        tma_load_3d(dst, &kmap, 0, row, z, &full[slot]);
                        tma_load_3d(dst + tile_bytes<D>(), &vmap, 0, row, z, &full[slot]);
                    }
                    const long long si = pg >= 0 ? (long long)pg * p.c.n_kv + head : 0;
                    copy4(&meta[slot].ks[g], p.c.k_scale + si, pg >= 0);
                    copy4(&meta[slot].vs[g], p.c.v_scale + si, pg >= 0);
                    copies_arrive(&full[slot]);
                }
                if (++slot == NS) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        if (lane == 0) splits_of(p)[blockIdx.x] = split;
        if (!mbar_wait(&i_empty[k % kItems], (k / kItems + 1) & 1u)) return;
        if (lane == 0) {
            items[k % kItems].n = 0;
            mbar_arrive(&i_full[k % kItems]);
        }
        return;
    }

    // ---------------- consumers ----------------
    const int g = lane >> 2, t = lane & 3;
    // ldmatrix: this lane gives the address of row lr of 16-byte chunk 2c + lc
    const int lr = (lane & 7) + 8 * ((lane >> 3) & 1), lc = lane >> 4;
    const uint32_t lrow = (uint32_t)((32 * warp + lr) * D);
    const uint32_t lswz = D == 128 ? (uint32_t)(lr & 7) : (uint32_t)((lr >> 1) & 3);
    const uint32_t lofs = ((uint32_t)lc ^ lswz) << 4;      // chunk c of the row lies at lrow + ((16 c) ^ lofs)
    float *red = reinterpret_cast<float *>(shared);
    const __half *qrow = reinterpret_cast<const __half *>(shared) + g * QP + 4 * t;

    // one block of 8 rows: q stays in registers; two: it is read where it is used
    uint32_t qh[CH][2], ql[PAIR ? CH : 1][2];
    float fac[NT][2];                                // of rows 2t, 2t+1: undoes q's scale, times scale * log2 e
    int pos[NT][2];                                  // their positions, -1 for none
    float m[NT][2], l[NT][2], o[NT][CH][4];          // m is a whole number
    int vexp[NT][2];                                 // O is in units of R = 2^(m + vexp): V scales are taken over 2^vexp
    int least = kLeastExp;                           // the smallest of them, or less
    bool dead = false;
    int slot = 0;
    uint32_t phase = 0;
    for (uint32_t k = 0;; ++k) {
        if (!mbar_wait(&i_full[k % kItems], (k / kItems) & 1u)) stop = 1;
        named_sync(1, 32 * kConsumers);              // every warp leaves here, or none
        const Item &it = items[k % kItems];
        if (stop || it.n == 0) return;
        const int y0 = it.y0, n = it.n, pos0 = it.pos0, pos1 = it.pos1, sinks = it.sinks, w0 = it.w0;
        if (!dead && !mbar_wait(&q_full, k & 1u)) dead = true;
        {
            if constexpr (NT == 1) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint2 h = *reinterpret_cast<const uint2 *>(qrow + 16 * c);
                    qh[c][0] = h.x;
                    qh[c][1] = h.y;
                    if constexpr (PAIR) {
                        const uint2 lo = *reinterpret_cast<const uint2 *>(qrow + RT * QP + 16 * c);
                        ql[c][0] = lo.x;
                        ql[c][1] = lo.y;
                    }
                }
            }
            least = kLeastExp;
#pragma unroll
            for (int x = 0; x < NT; ++x) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    fac[x][e] = q_fac[8 * x + 2 * t + e];
                    pos[x][e] = q_pos[8 * x + 2 * t + e];
                    m[x][e] = pos[x][e] < 0 ? kNever : -INFINITY;      // a row without tokens has nothing to follow
                    l[x][e] = 0.f;
                    vexp[x][e] = pos[x][e] < 0 ? 0 : kLeastExp;
                }
#pragma unroll
                for (int c = 0; c < CH; ++c) o[x][c][0] = o[x][c][1] = o[x][c][2] = o[x][c][3] = 0.f;
            }
        }
        for (int y = y0; y < y0 + n; ++y) {
        if (!dead && !mbar_wait(&full[slot], phase)) dead = true;
        const int t0 = (y < sinks ? y : w0 + (y - sinks)) * KT + 32 * warp;
        const TileMeta &mt = meta[slot];
        // both groups: a page, and every row sees every token
        const bool have0 = mt.have[2 * warp], have1 = mt.have[2 * warp + 1];
        const float ks[2] = {mt.ks[2 * warp], mt.ks[2 * warp + 1]}, vs[2] = {mt.vs[2 * warp], mt.vs[2 * warp + 1]};
        // nothing to see: no page, after the last row's token, or between the sinks and the first row's window
        const bool skip = !(have0 || have1) || t0 > pos1 ||
                          (p.window > 0 && t0 >= p.n_sink && t0 + 31 <= pos0 - p.window);
        if (!skip) {
            const uint32_t kt = smem_u32(ring + slot * 2 * tile_bytes<D>()) + lrow, vt = kt + tile_bytes<D>();
            // s[i][x][0..1]: token g of group i, rows 2t and 2t+1 of block x; s[i][x][2..3]: token g + 8.
            // Two sums (even and odd chunks) halve the chain of dependent products.
            float s[2][NT][4], s2[2][NT][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][x][e] = s2[i][x][e] = 0.f;
            uint32_t w[CH / 2][2][4];
#pragma unroll
            for (int cb = 0; cb < CH / 2; cb += AHEAD_C) {
#pragma unroll
                for (int c2 = cb; c2 < cb + AHEAD_C; ++c2)
#pragma unroll
                    for (int i = 0; i < 2; ++i) ldsm4(kt + 16 * i * D + ((uint32_t)(32 * c2) ^ lofs), w[c2][i]);
#pragma unroll
                for (int c2 = cb; c2 < cb + AHEAD_C; ++c2) {
                    uint2 b[NT][2][PAIR ? 2 : 1];
#pragma unroll
                    for (int x = 0; x < NT; ++x)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int z = 0; z < (PAIR ? 2 : 1); ++z) {
                                const int c = 2 * c2 + e;
                                if constexpr (NT > 1)
                                    b[x][e][z] = *reinterpret_cast<const uint2 *>(qrow + (z * RT + 8 * x) * QP + 16 * c);
                                else
                                    b[x][e][z] = z == 0 ? make_uint2(qh[c][0], qh[c][1]) : make_uint2(ql[PAIR ? c : 0][0], ql[PAIR ? c : 0][1]);
                            }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[c2][i][e] ^= 0x80808080u;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t lo = w[c2][i][2 * e], hi = w[c2][i][2 * e + 1];
                            const uint32_t a[4] = {codes2<0x4140>(lo), codes2<0x4140>(hi), codes2<0x4342>(lo), codes2<0x4342>(hi)};
#pragma unroll
                            for (int x = 0; x < NT; ++x)
#pragma unroll
                                for (int z = 0; z < (PAIR ? 2 : 1); ++z) mma(e ? s2[i][x] : s[i][x], a, b[x][e][z].x, b[x][e][z].y);
                        }
                    }
                }
            }
            // V's codes on their way while the weights are formed
            if constexpr (NT == 1) {
#pragma unroll
                for (int c2 = 0; c2 < CH / 2; ++c2)
#pragma unroll
                    for (int i = 0; i < 2; ++i) ldsm4t(vt + 16 * i * D + ((uint32_t)(32 * c2) ^ lofs), w[c2][i]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][x][e] = (s[i][x][e] + s2[i][x][e]) * (ks[i] * fac[x][e & 1]);
            const bool all = have0 && have1 && t0 + 31 <= pos0 &&
                             (p.window == 0 || t0 > pos1 - p.window || t0 + 31 < p.n_sink);
            uint32_t hidden = 0;                     // bit 4 (2x + i) + e: s[i][x][e] is not seen
            if (!all) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int x = 0; x < NT; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int tok = t0 + 16 * i + g + 8 * (e >> 1), ps = pos[x][e & 1];
                            if (tok > ps || (p.window > 0 && ps - tok >= p.window && tok >= p.n_sink) || !(i ? have1 : have0)) {
                                hidden |= 1u << (4 * (2 * x + i) + e);
                                s[i][x][e] = -INFINITY;
                            }
                        }
            }
            // exponents e of the V scales, |scale| < 2^e; scales below 2^-126 count as 0, and those whose codes
            // overflow f32, infinities and NaNs make NaN of every weight
            int ve[2];
            float vu[2];
            bool raise = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int be = (int)(__float_as_uint(vs[i]) >> 23) & 255;
                ve[i] = be == 0 || be > 127 + kMaxExp - 4 ? kMinExp : be - 126;
                vu[i] = be == 0 ? 0.f : be > 127 + kMaxExp - 4 ? __int_as_float(0x7fc00000) : vs[i];
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // the lower of the two references, as a score of this group
                        const float most = m[x][e] + small_float(min(0, vexp[x][e] - ve[i]), kSlack);
                        raise |= s[i][x][e] > most || s[i][x][e + 2] > most;
                    }
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top[2];                // of each group
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            top[i] = fmaxf(s[i][x][e], s[i][x][e + 2]);
#pragma unroll
                            for (int w = 4; w < 32; w <<= 1) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], w));
                        }
                        const float mn = fmaxf(m[x][e], ceilf(fmaxf(top[0], top[1])));
                        const int up = m[x][e] == -INFINITY ? kFarExp : (int)fminf(mn - m[x][e], (float)kFarExp);
                        // R stays while m moves, as far as vexp can follow, unless the group's products are above it
                        int vn = max(vexp[x][e] - up, kLeastExp);
#pragma unroll
                        for (int i = 0; i < 2; ++i) vn = max(vn, (int)ceilf(fmaxf(top[i] - mn, -(float)kFarExp)) + ve[i]);
                        const float a = pow2(vexp[x][e] - up - vn);
                        least = x + e == 0 ? vn : min(least, vn);
                        l[x][e] *= pow2(-up);
                        m[x][e] = mn;
                        vexp[x][e] = vn;
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            o[x][c][e] *= a;
                            o[x][c][e + 2] *= a;
                        }
                    }
            }
            float vrel[2][NT][2];                    // the V scales over R / 2^m
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float inv = pow2(kLift - vexp[x][e]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) vrel[i][x][e] = vu[i] * inv;
                }
            // a scale that far above R belongs to weights near 2^-126: they must not become 0 times infinity
            if (max(ve[0], ve[1]) + kLift - least > 126) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int x = 0; x < NT; ++x)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (fabsf(vrel[i][x][e]) == INFINITY) vrel[i][x][e] = copysignf(pow2(126), vu[i]);
            }
            uint32_t ph[2][NT][2], pl[2][WPAIR ? NT : 1][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    float w[4];
                    if (all) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            w[e] = ex2(s[i][x][e] - m[x][e & 1]);
                            l[x][e & 1] += w[e];
                            w[e] *= vrel[i][x][e & 1];
                        }
                    } else {
                        // zeros before the sum (a row without tokens has inf - inf here) and after the scale (a
                        // page that is not seen may have a NaN there)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool see = !(hidden & (1u << (4 * (2 * x + i) + e)));
                            w[e] = see ? ex2(s[i][x][e] - m[x][e & 1]) : 0.f;
                            l[x][e & 1] += w[e];
                            w[e] = see ? w[e] * vrel[i][x][e & 1] : 0.f;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t hi = pack2(w[2 * e], w[2 * e + 1]);
                        ph[i][x][e] = transpose8x8(hi);
                        if constexpr (WPAIR) {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                            pl[i][x][e] = transpose8x8(pack2(w[2 * e] - f.x, w[2 * e + 1] - f.y));
                        }
                    }
                }
#pragma unroll
            for (int c2 = 0; c2 < CH / 2; ++c2) {
                if constexpr (NT > 1) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) ldsm4t(vt + 16 * i * D + ((uint32_t)(32 * c2) ^ lofs), w[c2][i]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[c2][i][e] ^= 0x80808080u;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // Products cut their sums off instead of rounding them: about 2^-25 of O each, always towards zero. f32 rows'
                    // start from zero in every tile and are added to O with a rounding.
                    float part[NT][4];
#pragma unroll
                    for (int x = 0; x < NT; ++x)
#pragma unroll
                        for (int r = 0; r < 4; ++r) part[x][r] = 0.f;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // row g of the fragment is element 2g of the chunk, row g + 8 element 2g + 1
                        const uint32_t lo = w[c2][i][2 * e], hi = w[c2][i][2 * e + 1];
                        const uint32_t a[4] = {codes2<0x4240>(lo), codes2<0x4341>(lo), codes2<0x4240>(hi), codes2<0x4341>(hi)};
#pragma unroll
                        for (int x = 0; x < NT; ++x) {
                            float(&to)[4] = PAIR ? part[x] : o[x][2 * c2 + e];
                            mma(to, a, ph[i][x][0], ph[i][x][1]);
                            if constexpr (WPAIR) mma(to, a, pl[i][x][0], pl[i][x][1]);
                        }
                    }
                    if constexpr (PAIR) {
#pragma unroll
                        for (int x = 0; x < NT; ++x) {
                            add2(o[x][2 * c2 + e][0], o[x][2 * c2 + e][1], part[x][0], part[x][1]);
                            add2(o[x][2 * c2 + e][2], o[x][2 * c2 + e][3], part[x][2], part[x][3]);
                        }
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        if (++slot == NS) {
            slot = 0;
            phase ^= 1u;
        }
        }

        // ---------------- the item's end: join the four warps ----------------
        {
            const bool whole = it.whole;
            const int tid = threadIdx.x, rows = it.rows;
            constexpr int COLS = D / 4;                      // groups of 4 elements
            const int col = tid % COLS, line = tid / COLS;
            float *parts = parts_of(p);
            constexpr size_t PF = attn_part_floats(RT, D);
            float *part = parts + (size_t)it.slot * PF;
            // 4 elements of a row of the item
            auto put = [&](int row, float4 v, float sum) {
                const float inv = sum != 0.f ? 1.f / sum : 0.f;      // no visible token: zeros
                store4(static_cast<T *>(p.out) + q_out[row] + 4 * col, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
            };
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float sum = l[x][e];
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                    if (g == 0) {
                        red_m[warp][8 * x + 2 * t + e] = m[x][e];
                        red_l[warp][8 * x + 2 * t + e] = sum;
                    }
                }
            named_sync(1, 32 * kConsumers);                  // every warp is done with q, which the buffer held
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int first = 8 * x + 4 * hf;        // rows first .. first + 3
                    if (first >= rows) continue;
                    if ((t >> 1) == hf) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float back = pow2(vexp[x][e] - kLift);
                            float *mine = red + (warp * 4 + 2 * (t & 1) + e) * RLD + 2 * g;
#pragma unroll
                            for (int c = 0; c < CH; ++c)
                                *reinterpret_cast<float2 *>(mine + 16 * c) =
                                    make_float2(o[x][c][e] * back, o[x][c][e + 2] * back);
                        }
                    }
                    named_sync(1, 32 * kConsumers);
                    const int row = first + line;
                    if (line < 4 && row < rows) {
                        float top = red_m[0][row];
#pragma unroll
                        for (int w = 1; w < kConsumers; ++w) top = fmaxf(top, red_m[w][row]);
                        float sum = 0.f;
                        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int w = 0; w < kConsumers; ++w) {
                            const float a = red_m[w][row] == -INFINITY ? 0.f : ex2(red_m[w][row] - top);
                            const float4 v = *reinterpret_cast<const float4 *>(red + (w * 4 + line) * RLD + 4 * col);
                            sum += red_l[w][row] * a;
                            acc.x += v.x * a;
                            acc.y += v.y * a;
                            acc.z += v.z * a;
                            acc.w += v.w * a;
                        }
                        if (whole) {
                            put(row, acc, sum);
                        } else {
                            *reinterpret_cast<float4 *>(part + row * D + 4 * col) = acc;
                            if (col == 0) {
                                *reinterpret_cast<float2 *>(part + RT * D + 2 * row) = make_float2(top, sum);
                            }
                        }
                    }
                    named_sync(1, 32 * kConsumers);
                }
            named_sync(1, 32 * kConsumers);                  // the item and the buffer are free
            if (tid == 0) {
                mbar_arrive(&q_empty);
                mbar_arrive(&i_empty[k % kItems]);
            }
        }
    }
}

template <class T, int D, int NT> cudaError_t launch(const AttnArgs &a, cudaStream_t s, const DeviceInfo &dev) {
    constexpr int smem = smem_bytes<D, NT, sizeof(T) == 4>();
    static PerDeviceOnce once;
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(attn_mma<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    CUtensorMap km, vm;
    if (!make_map(&km, a.c.k, a.c) || !make_map(&vm, a.c.v, a.c)) return cudaErrorInvalidValue;
    // two CTAs per SM, and no more than there can be units
    const long long tiles = ((long long)a.c.table_ld * a.c.page + KT - 1) / KT;
    const long long row_tiles = ((long long)a.c.n_rows * (a.n_q / a.c.n_kv) + 8 * NT - 1) / (8 * NT) + a.c.n_seq;
    long long grid = 2 * dev.sm_count;
    if (grid > kAttnMaxGrid) grid = kAttnMaxGrid;
    if (row_tiles < grid && tiles * row_tiles * a.c.n_kv < grid) grid = tiles * row_tiles * a.c.n_kv;
    return launch_with_join<T, D, 8 * NT>(attn_mma<T, D, NT>, (int)grid, kThreads, smem, km, vm, a, s);
}

template <class T> cudaError_t launch_t(const AttnArgs &a, int rows, cudaStream_t s, const DeviceInfo &dev) {
    // Rows on the narrow side of a product: 8, or 16 where a sequence brings more than 8 per kv head (16 rows, 64
    // sequences of 2048 tokens, 32 heads over 8: 70.5 us, as two times 8 rows 92.7; 16 sequences 30.2 and 29.1).
    if (a.c.d == 128) return rows <= 8 ? launch<T, 128, 1>(a, s, dev) : launch<T, 128, 2>(a, s, dev);
    return rows <= 8 ? launch<T, 64, 1>(a, s, dev) : launch<T, 64, 2>(a, s, dev);
}

}  // namespace

unsigned attn_mma_wait_timeouts(bool reset) {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof(v)) != cudaSuccess) return 0;
    if (reset) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_wait_timeouts, &z, sizeof(z));
    }
    return v;
}

size_t attn_mma_ws_bytes(int d) { return attn_splits_bytes() + 2 * kAttnMaxGrid * attn_part_floats(16, d) * 4; }

cudaError_t launch_attn_mma(int dt, const AttnArgs &a, int rows, cudaStream_t s, const DeviceInfo &dev) {
    if (dt == PQ_F32) return launch_t<float>(a, rows, s, dev);
    if (dt == PQ_F16) return launch_t<__half>(a, rows, s, dev);
    return launch_t<__nv_bfloat16>(a, rows, s, dev);
}

}  // namespace pqk
