// Attention over the paged 8-bit cache for few rows per sequence (decode steps,
// drafted tokens, short pieces), head sizes 64 and 128.
//
// Bound by the bytes of K and V: every code is read once per 8 or 16 rows, so
// the products go to the tensor cores and the loads to TMA.  Softmax in one
// pass (running maximum m and sum l of exp2(s - m)):
//     S = K q'      (16 tokens x 8 rows per mma.sync m16n8k16)
//     O += V^T P    (16 elements x 8 rows)
// with K and V as the A operands, so that rows fill the narrow side (N = 8) and
// one token's code is loaded by exactly one thread.  Operands are exact where
// they can be: int8 codes become fp16 by a byte permute and one subtraction
// (0x6400 | (code + 128) is 1152 + code); q is scaled per row by a power of
// two into fp16's range (one fp16 for 16-bit rows, an fp16 pair for f32 rows).
// The softmax weights enter in fp16 (f32 rows: an fp16 pair), already times
// their page's V scale over the largest one seen so far: weights and ratios
// are at most 1 times the 2^8 that the running maximum may lag behind, so fp16
// holds them whatever the scales.
//
// ldmatrix gives a thread four codes of one token (K) or, transposed in 2-byte
// units, two elements of two tokens (V): the byte permutes of the conversion
// sort them, so the transposition of V costs nothing.
//
// Pipeline: warp 4 brings 64-token tiles of K and V through a ring of stages (TMA boxes
// of one page or half a page, swizzled; page numbers read for eight tiles at a
// time; page scales by 4-byte asynchronous copies onto the same barrier); warps
// 0-3 take 16 tokens of a tile each, with a running maximum of their own,
// and join at the end of an item.

#include <cuda.h>

#include "attn_sched.cuh"
#include "pq_device.cuh"
#include "pq_ptx.cuh"

namespace pqk {
namespace {

constexpr int KT = 64;                       // tokens per tile
constexpr int kConsumers = 4;                // warps, 16 tokens of a tile each
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;                // the running maximum may lag by this many powers of two

template <int D> __host__ __device__ constexpr int tile_bytes() { return KT * D; }
template <int D> __host__ __device__ constexpr int stages() { return D == 128 ? 5 : 10; }
// join buffer: 8 rows of each consumer warp at a time
template <int D> __host__ __device__ constexpr int red_bytes() { return kConsumers * 8 * (D + 8) * 4; }
template <int D> __host__ __device__ constexpr int smem_bytes() {
    return 1024 + stages<D>() * 2 * tile_bytes<D>() + red_bytes<D>();
}

struct TileMeta {
    float ks[4], vs[4];      // scales of the tile's four groups of 16 tokens
    int have[4];             // whether the group has a page
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Two biased codes (code + 128) of w, chosen by the permutation SEL, as exact fp16.
template <uint32_t SEL> __device__ __forceinline__ uint32_t codes2(uint32_t w) {
    const uint32_t v = __byte_perm(w, 0x64646464u, SEL), bias = 0x64806480u;      // 1152
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&bias));
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
// 4 bytes (or zeros when !have) to shared memory, asynchronously.
__device__ __forceinline__ void copy4(void *dst, const void *src, bool have) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(have ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Four consecutive elements as f32.
__device__ __forceinline__ void load4(const float *p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
template <class T> __device__ __forceinline__ void load4(const T *p, float (&x)[4]) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    const T *e = reinterpret_cast<const T *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = to_f32(e[i]);
}

template <class T, int D, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    attn_mma(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, AttnArgs p) {
    constexpr int RT = 8 * NT, NS = stages<D>(), CH = D / 16;
    constexpr bool PAIR = sizeof(T) == 4;            // q and the weights as fp16 pairs
    constexpr float kLift = PAIR ? 128.f : 1.f;      // keeps the low halves of small weights above fp16's last bit
    constexpr int RLD = D + 8;                       // row pitch of the join buffer
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[NS], empty[NS];
    __shared__ __align__(16) TileMeta meta[NS];
    __shared__ UnitRange range;
    __shared__ float red_m[kConsumers][RT], red_l[kConsumers][RT];
    __shared__ int last_part;

    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = p.n_q / p.c.n_kv;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1 + 4);
            mbar_init(&empty[i], kConsumers);
        }
        fence_mbar_init();
    }
    find_range<RT, KT, kThreads>(p, group, &range);
    const int count = (int)(range.last - range.first);
    if (count == 0) return;

    UnitWalk<RT, KT> at;
    at.start(p, group, range.seq, range.offset, range.per_head);

    if (warp == kConsumers) {
        // ---------------- producer ----------------
        const int box = min(p.c.page, KT);                     // tokens per TMA box
        const int g = lane & 3, sub = lane >> 2;
        for (int n0 = 0; n0 < count; n0 += 8) {
            // lane 4i + g looks up group g of unit n0 + i
            int tok = 0, seq = 0, head = 0;
            for (int i = 0; i < 8 && n0 + i < count; ++i) {
                if (sub == i) {
                    tok = at.token0() + 16 * g;
                    seq = at.s;
                    head = at.h;
                }
                at.next(p, group);
            }
            const int pg = n0 + sub < count ? page_of(p.c, seq, tok / p.c.page) : -1;
            for (int i = 0; i < 8 && n0 + i < count; ++i) {
                const int n = n0 + i, slot = n % NS;
                if (!mbar_wait(&empty[slot], (uint32_t)(n / NS + 1) & 1u)) return;
                if (sub == i) meta[slot].have[g] = pg >= 0;
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(&full[slot], 2 * tile_bytes<D>());
                __syncwarp();
                if (sub == i) {
                    if (16 * g % box == 0) {
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
            }
        }
        return;
    }

    // ---------------- consumers ----------------
    const int g = lane >> 2, t = lane & 3;
    // ldmatrix: this lane gives the address of row lr of 16-byte chunk 2c + lc
    const int lr = (lane & 7) + 8 * ((lane >> 3) & 1), lc = lane >> 4;
    const uint32_t lrow = (uint32_t)((16 * warp + lr) * D);
    const uint32_t lswz = D == 128 ? (uint32_t)(lr & 7) : (uint32_t)((lr >> 1) & 3);
    float *red = reinterpret_cast<float *>(ring + NS * 2 * tile_bytes<D>());

    uint32_t qh[NT][CH][2], ql[PAIR ? NT : 1][PAIR ? CH : 1][2];
    float fac[NT][2];                                // of rows 2t, 2t+1: undoes q's scale, times scale * log2 e
    int pos[NT][2];                                  // their positions, -1 for none
    float m[NT][2], l[NT][2], vref[NT][2], o[NT][CH][4];
    float vinv[NT][2];                               // kLift / vref
    bool fresh = true, dead = false;
    for (int n = 0; n < count; ++n) {
        if (fresh) {
            fresh = false;
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                // row g of this block of 8: query head and token
                const int r = at.j * RT + 8 * x + g;
                const bool have = 8 * x + g < at.t.rows;
                const T *src = static_cast<const T *>(p.q) + (long long)(at.r0 + r / group) * p.ldq +
                               (long long)(at.h * group + r % group) * D + 4 * t;
                float v[CH][4];
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    if (have) load4(src + 16 * c, v[c]);
                    else v[c][0] = v[c][1] = v[c][2] = v[c][3] = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(v[c][e]) & 0x7fffffffu);
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int ex = tc_scale_exponent(top);
                const float up = __uint_as_float((uint32_t)(127 + ex) << 23), down = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float a = v[c][2 * e] * up, b = v[c][2 * e + 1] * up;
                        qh[x][c][e] = pack2(a, b);
                        if constexpr (PAIR) {
                            const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&qh[x][c][e]));
                            ql[x][c][e] = pack2(a - hi.x, b - hi.y);
                        }
                    }
                const float f = down * (p.scale * kLog2e);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    fac[x][e] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + e));
                    const int rr = 8 * x + 2 * t + e;
                    pos[x][e] = rr < at.t.rows ? at.len - at.m + (at.j * RT + rr) / group : -1;
                    m[x][e] = -INFINITY;
                    l[x][e] = vref[x][e] = vinv[x][e] = 0.f;
                }
#pragma unroll
                for (int c = 0; c < CH; ++c) o[x][c][0] = o[x][c][1] = o[x][c][2] = o[x][c][3] = 0.f;
            }
        }
        const int slot = n % NS;
        if (!dead && !mbar_wait(&full[slot], (uint32_t)(n / NS) & 1u)) dead = true;
        const int t0 = at.token0() + 16 * warp;
        const float ks = meta[slot].ks[warp], vs = meta[slot].vs[warp];
        // nothing to see: no page, after the last row's token, or between the sinks and the first row's window
        const bool skip = !meta[slot].have[warp] || t0 > at.t.pos1 ||
                          (p.window > 0 && t0 >= p.n_sink && t0 + 15 <= at.t.pos0 - p.window);
        if (!skip) {
            const uint32_t kt = smem_u32(ring + slot * 2 * tile_bytes<D>()) + lrow, vt = kt + tile_bytes<D>();
            float s[NT][4];
#pragma unroll
            for (int x = 0; x < NT; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
#pragma unroll
            for (int c = 0; c < CH; c += 2) {
                uint32_t w[4];
                ldsm4(kt + (((uint32_t)(c + lc) ^ lswz) << 4), w);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] ^= 0x80808080u;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t a[4] = {codes2<0x4140>(w[2 * i]), codes2<0x4140>(w[2 * i + 1]), codes2<0x4342>(w[2 * i]),
                                           codes2<0x4342>(w[2 * i + 1])};
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        mma(s[x], a, qh[x][c + i][0], qh[x][c + i][1]);
                        if constexpr (PAIR) mma(s[x], a, ql[x][c + i][0], ql[x][c + i][1]);
                    }
                }
            }
            // s[x][0..1]: token g, rows 2t and 2t+1; s[x][2..3]: token g + 8
            const bool all = t0 + 15 <= at.t.pos0 && (p.window == 0 || t0 > at.t.pos1 - p.window || t0 + 15 < p.n_sink);
            const float av = fabsf(vs);
            const bool usable = av >= 1.17549435e-38f && av < INFINITY;     // else 0, or NaN in every weight
            bool hide[NT][4];
            bool raise = false;
#pragma unroll
            for (int x = 0; x < NT; ++x) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[x][e] *= ks * fac[x][e & 1];
                    hide[x][e] = false;
                    if (!all) {
                        const int tok = t0 + g + 8 * (e >> 1), ps = pos[x][e & 1];
                        hide[x][e] = tok > ps || (p.window > 0 && ps - tok >= p.window && tok >= p.n_sink);
                        if (hide[x][e]) s[x][e] = -INFINITY;
                    }
                    raise |= s[x][e] > m[x][e & 1] + kSlack;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) raise |= usable && av > vref[x][e];
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(s[x][e], s[x][e + 2]);
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                        const float mn = fmaxf(m[x][e], top);
                        float a = m[x][e] == -INFINITY ? 0.f : ex2(m[x][e] - mn);
                        m[x][e] = mn;
                        l[x][e] *= a;
                        // a row takes the page's V scale only if it sees a token of the page
                        const int ps = pos[x][e];
                        const bool sees = t0 <= ps && !(p.window > 0 && t0 >= p.n_sink && t0 + 15 <= ps - p.window);
                        if (sees && usable && av > vref[x][e]) {
                            a *= vref[x][e] / av;
                            vref[x][e] = av;
                            vinv[x][e] = kLift / av;
                        }
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            o[x][c][e] *= a;
                            o[x][c][e + 2] *= a;
                        }
                    }
            }
            const float vu = usable ? vs : (av < INFINITY ? 0.f : __int_as_float(0x7fc00000));
            uint32_t ph[NT][2], pl[PAIR ? NT : 1][2];
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float pr = hide[x][e] ? 0.f : ex2(s[x][e] - m[x][e & 1]);
                    l[x][e & 1] += pr;
                    w[e] = hide[x][e] ? 0.f : pr * (vu * vinv[x][e & 1]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t hi = pack2(w[2 * e], w[2 * e + 1]);
                    ph[x][e] = transpose8x8(hi);
                    if constexpr (PAIR) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                        pl[x][e] = transpose8x8(pack2(w[2 * e] - f.x, w[2 * e + 1] - f.y));
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < CH; c += 2) {
                uint32_t w[4];
                ldsm4t(vt + (((uint32_t)(c + lc) ^ lswz) << 4), w);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] ^= 0x80808080u;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // row g of the fragment is element 2g of the chunk, row g + 8 element 2g + 1
                    const uint32_t a[4] = {codes2<0x4240>(w[2 * i]), codes2<0x4341>(w[2 * i]), codes2<0x4240>(w[2 * i + 1]),
                                           codes2<0x4341>(w[2 * i + 1])};
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        mma(o[x][c + i], a, ph[x][0], ph[x][1]);
                        if constexpr (PAIR) mma(o[x][c + i], a, pl[x][0], pl[x][1]);
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);

        const long long u = range.first + n, item0 = u - at.y, item1 = item0 + at.t.units;
        const bool end = u + 1 == item1;
        if (end || n + 1 == count) {
            // ---------------- join the four warps ----------------
            const bool whole = item0 >= range.first && item1 <= range.last;
            const int tid = threadIdx.x;
            const int side = item0 <= range.first ? 0 : 1;
            float *part = reinterpret_cast<float *>(p.ws + attn_counter_bytes()) +
                          (size_t)(2 * blockIdx.x + side) * attn_part_floats(RT, D);
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
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                // 8 rows at a time through the join buffer
                const float back[2] = {vref[x][0] * (1.f / kLift), vref[x][1] * (1.f / kLift)};
                float *mine = red + (size_t)(warp * 8) * RLD;
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float2 *>(mine + (2 * t + e) * RLD + 16 * c + 2 * g) =
                            make_float2(o[x][c][e] * back[e], o[x][c][e + 2] * back[e]);
                named_sync(1, 32 * kConsumers);
                for (int i = tid; i < 8 * D; i += 32 * kConsumers) {
                    const int r = i / D, d = i % D, row = 8 * x + r;
                    if (row >= at.t.rows) continue;
                    float top = red_m[0][row];
#pragma unroll
                    for (int w = 1; w < kConsumers; ++w) top = fmaxf(top, red_m[w][row]);
                    float sum = 0.f, acc = 0.f;
#pragma unroll
                    for (int w = 0; w < kConsumers; ++w) {
                        const float a = red_m[w][row] == -INFINITY ? 0.f : ex2(red_m[w][row] - top);
                        sum += red_l[w][row] * a;
                        acc += red[(size_t)(w * 8 + r) * RLD + d] * a;
                    }
                    if (whole) {
                        const int rr = at.j * RT + row;
                        T *dst = static_cast<T *>(p.out) + (long long)(at.r0 + rr / group) * p.ldo +
                                 (long long)(at.h * group + rr % group) * D;
                        from_f32(dst[d], sum != 0.f ? acc / sum : 0.f);
                    } else {
                        part[(size_t)row * D + d] = acc;
                        if (d == 0) {
                            part[(size_t)RT * D + row] = top;
                            part[(size_t)RT * D + RT + row] = sum;
                        }
                    }
                }
                named_sync(1, 32 * kConsumers);
            }
            if (!whole) {
                // ---------------- join the CTAs' parts ----------------
                const int c0 = range_owner(item0, range.total, range.grid), c1 = range_owner(item1 - 1, range.total, range.grid);
                unsigned *counter = reinterpret_cast<unsigned *>(p.ws) + c0;
                __threadfence();
                named_sync(1, 32 * kConsumers);
                if (tid == 0) {
                    const bool is_last = atomicAdd(counter, 1u) == (unsigned)(c1 - c0);
                    if (is_last) *counter = 0u;          // ready for the next call
                    last_part = is_last;
                }
                named_sync(1, 32 * kConsumers);
                if (last_part) {
                    __threadfence();
                    const float *parts = reinterpret_cast<const float *>(p.ws + attn_counter_bytes());
                    const size_t pf = attn_part_floats(RT, D);
                    // only the first CTA's part can be the item its range ends in
                    const int side0 = item0 <= range_begin(c0, range.total, range.grid) ? 0 : 1;
                    const int rows = at.t.rows;
                    for (int i = tid; i < rows * D; i += 32 * kConsumers) {
                        const int row = i / D, d = i % D;
                        float top = -INFINITY, sum = 0.f, acc = 0.f;
                        for (int c = c0; c <= c1; ++c) {
                            const float *pp = parts + (size_t)(2 * c + (c == c0 ? side0 : 0)) * pf;
                            const float pm = __ldcg(pp + (size_t)RT * D + row);
                            const float plv = __ldcg(pp + (size_t)RT * D + RT + row);
                            const float pa = __ldcg(pp + (size_t)row * D + d);
                            const float mn = fmaxf(top, pm);
                            const float a = top == -INFINITY ? 0.f : ex2(top - mn), b = pm == -INFINITY ? 0.f : ex2(pm - mn);
                            sum = sum * a + plv * b;
                            acc = acc * a + pa * b;
                            top = mn;
                        }
                        const int rr = at.j * RT + row;
                        T *dst = static_cast<T *>(p.out) + (long long)(at.r0 + rr / group) * p.ldo +
                                 (long long)(at.h * group + rr % group) * D;
                        from_f32(dst[d], sum != 0.f ? acc / sum : 0.f);
                    }
                }
                named_sync(1, 32 * kConsumers);
            }
            fresh = true;
        }
        at.next(p, group);
    }
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
    static EncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(ptr);
    });
    return fn;
}

// The codes as a tensor of (element, kv head and token of the page, page).
bool make_map(CUtensorMap *map, const int8_t *codes, const KvView &c) {
    EncodeTiled enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t rows = (cuuint64_t)c.n_kv * c.page;
    const cuuint64_t dims[3] = {(cuuint64_t)c.d, rows, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[2] = {(cuuint64_t)c.d, rows * c.d};
    const cuuint32_t box[3] = {(cuuint32_t)c.d, (cuuint32_t)(c.page < KT ? c.page : KT), 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t *>(codes), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, c.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int D, int NT> cudaError_t launch(const AttnArgs &a, cudaStream_t s, const DeviceInfo &dev) {
    constexpr int smem = smem_bytes<D>();
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
    attn_mma<T, D, NT><<<(unsigned)grid, kThreads, smem, s>>>(km, vm, a);
    return cudaGetLastError();
}

template <class T> cudaError_t launch_t(const AttnArgs &a, int rows, cudaStream_t s, const DeviceInfo &dev) {
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

size_t attn_mma_ws_bytes(int d) { return attn_counter_bytes() + 2 * kAttnMaxGrid * attn_part_floats(16, d) * 4; }

cudaError_t launch_attn_mma(int dt, const AttnArgs &a, int rows, cudaStream_t s, const DeviceInfo &dev) {
    if (dt == PQ_F32) return launch_t<float>(a, rows, s, dev);
    if (dt == PQ_F16) return launch_t<__half>(a, rows, s, dev);
    return launch_t<__nv_bfloat16>(a, rows, s, dev);
}

}  // namespace pqk
