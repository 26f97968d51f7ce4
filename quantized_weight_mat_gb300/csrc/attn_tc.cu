// Attention over the paged 8-bit cache for prompts (many rows per sequence) on
// the 5th-generation tensor cores: 16-bit rows, head sizes 64 and 128.
//
// The same one-pass softmax as the decode kernel, with the rows on the wide
// side: 128 rows by 128 tokens per product,
//     S = q' K^T     A = q' (fp16, shared memory), B = K's codes (fp16, K-major)
//     O += P V       A = P (fp16, tensor memory, over S), B = V's codes (MN-major)
// q' is q scaled per row by a power of two (exact for bf16 and f16), codes are
// exact in fp16.  A CTA takes 256 rows of one sequence and kv head, as two
// halves whose products and softmaxes alternate, so that both share one
// conversion of each K and V tile from 8 bits.
//
// Bound by the tensor cores (4 x 512 cycles a tile for 256 rows at head size
// 128) and, close to it, by shared memory (operands of four products, 64 KB of
// converted codes) and the exponentials (256 x 128 a tile).
//
//   warps 0-7    softmax, thread = row (tensor-memory lane), warps 0-3 the
//                first half: maximum of S, exponentials, P back to tensor memory; at an item's
//                start the row of q, at its end the row of the output
//   warps 8-11   codes -> fp16 into the operand image (rows of 8 x 16 bytes: the
//                same image serves as K-major K and as MN-major V)
//   warp 12      walks the units, TMA of K and V tiles, page numbers and scales
//   warp 13      one thread issues the products
// Shared memory: q 64 KB, converted K and V 32 KB each, three raw tiles 96 KB.
//
// Per page the weights are formed as exp2(S * f + c), f = q's and K's scales,
// c = log2(V's scale over a power of two above the largest seen) - maximum:
// the V scale costs nothing per element; the weight sum undoes it once a page.
// The running maximum and the power of two lag as in the decode kernel, so O
// is rescaled (by its own row's thread) only now and then.

#include "attn_common.cuh"
#include "pq_tcgen05.cuh"

namespace pqk {
namespace {

constexpr int RT = 256, HALF = 128;          // rows of an item, and of each half
constexpr int kSoftmaxWarps = 8, kConvertWarps = 4;
constexpr int kWalkWarp = kSoftmaxWarps + kConvertWarps, kMmaWarp = kWalkWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kRaw = 3, kMeta = 4, kItems = 8, kItemCost = 2;
constexpr int kTcGrid = 160;                 // CTAs at most: one per SM
constexpr int kTmemCols = 512;
using Walk = UnitWalk<RT, KT, kItemCost>;

template <int D> __host__ __device__ constexpr int smem_bytes() {
    return 1024 + RT * D * 2 + 2 * KT * D * 2 + kRaw * 2 * KT * D;
}
static_assert(smem_bytes<128>() <= 226 * 1024, "shared memory per CTA, beside the static part");

// Operand image of n rows of D fp16: 8 x 16-byte core matrices, the next 8
// elements of a row 128 bytes on, the next 8 rows 16 * D bytes on.
template <int D> __device__ __forceinline__ uint32_t image_at(int row, int chunk) {
    return (uint32_t)(row >> 3) * (16 * D) + chunk * 128 + (row & 7) * 16;
}

__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One tile of codes (128 tokens, swizzled as TMA left it) to its fp16 image, by the four converting warps.
template <int D> __device__ __forceinline__ void convert_tile(uint32_t raw, uint32_t image, int warp, int lane) {
    constexpr int CHUNKS = D / 16, PER = CHUNKS / 4;            // 16-code chunks of a row; a warp takes 8 rows x 4 chunks
#pragma unroll
    for (int i = 0; i < 16 * PER / kConvertWarps; ++i) {
        const int unit = i * kConvertWarps + warp, row = unit / PER * 8 + (lane & 7), c = unit % PER * 4 + (lane >> 3);
        const int sw = D == 128 ? row & 7 : (row >> 1) & 3;
        uint4 w = lds128(raw + row * D + ((c ^ sw) << 4));
        w.x ^= 0x80808080u;
        w.y ^= 0x80808080u;
        w.z ^= 0x80808080u;
        w.w ^= 0x80808080u;
        const uint32_t to = image + image_at<D>(row, 2 * c);
        sts128(to, make_uint4(codes2<0x4140>(w.x), codes2<0x4342>(w.x), codes2<0x4140>(w.y), codes2<0x4342>(w.y)));
        sts128(to + 128, make_uint4(codes2<0x4140>(w.z), codes2<0x4342>(w.z), codes2<0x4140>(w.w), codes2<0x4342>(w.w)));
    }
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, AttnArgs p) {
    constexpr uint32_t ID_S = instr_desc(HALF, KT), ID_O = instr_desc(HALF, D) | (1u << 16);      // bit 16: B is MN-major
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t raw_full[kRaw], raw_empty[kRaw], meta_full[kMeta], meta_empty[kMeta], i_full[kItems],
        i_empty[kItems], k_ready, k_free, v_ready, v_free, s_full[2], p_ready[2], pv_done[2], q_ready;
    __shared__ __align__(16) TileMeta meta[kMeta];
    __shared__ Item items[kItems];
    __shared__ uint32_t tmem_base;
    __shared__ int last_part;
    __shared__ volatile int stop, stop_convert;

    // converted V and K, q, raw tiles, from a 1024-byte boundary
    const uint32_t v0 = (smem_u32(smem_raw) + 1023u) & ~1023u, k0 = v0 + KT * D * 2, q0 = k0 + KT * D * 2, raw0 = q0 + RT * D * 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        stop = stop_convert = 0;
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], kConvertWarps);
        }
        for (int i = 0; i < kMeta; ++i) {
            mbar_init(&meta_full[i], 1 + kGroups);
            mbar_init(&meta_empty[i], kSoftmaxWarps);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&i_full[i], 1);
            mbar_init(&i_empty[i], 3);
        }
        mbar_init(&k_ready, kConvertWarps);
        mbar_init(&k_free, 1);
        mbar_init(&v_ready, kConvertWarps);
        mbar_init(&v_free, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(&q_ready, kSoftmaxWarps);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;         // columns: S (and P) of each half at 0 and 128, O at 256 and 384
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    if (warp == kWalkWarp) {
        // ---------------- walk and loads ----------------
        constexpr int BATCH = 32 / kGroups;
        const int g = lane % kGroups, sub = lane / kGroups;
        Walk at;
        long long first, last;
        const Cut cut = find_range<Walk, kItemCost>(p, at, first, last);
        uint32_t k = 0, n_unit = 0;
        bool fresh = true, dead = false;
        at.w = first == last ? last : at.w;
        while (at.w < last && !dead) {
            // lane kGroups * i + g looks up group g of the i-th unit from here
            int tok = 0, seq = 0, head = 0, n = 0;
            for (; n < BATCH && at.w < last && !dead; ++n) {
                if (fresh) {
                    fresh = false;
                    if (!mbar_wait(&i_empty[k % kItems], (k / kItems + 1) & 1u)) dead = true;
                    if (lane == 0 && !dead) {
                        items[k % kItems] = item_of(at, cut, first, last);
                        mbar_arrive(&i_full[k % kItems]);
                    }
                    ++k;
                }
                if (sub == n) {
                    tok = at.token0() + 16 * g;
                    seq = at.s;
                    head = at.h;
                }
                if (at.y + 1 < at.t.units) {
                    ++at.y;
                    ++at.w;
                } else {
                    at.next_item(p);
                    fresh = true;
                }
            }
            const int pg = sub < n ? page_of(p.c, seq, tok / p.c.page) : -1;
            for (int i = 0; i < n && !dead; ++i, ++n_unit) {
                const int slot = n_unit % kRaw, ms = n_unit % kMeta;
                if (!mbar_wait(&meta_empty[ms], (n_unit / kMeta + 1) & 1u) || !mbar_wait(&raw_empty[slot], (n_unit / kRaw + 1) & 1u)) {
                    dead = true;
                    break;
                }
                if (sub == i) meta[ms].have[g] = pg >= 0;
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&meta_full[ms]);
                    mbar_arrive_expect_tx(&raw_full[slot], 2 * KT * D);
                }
                __syncwarp();
                if (sub == i) {
                    if (16 * g % p.c.page == 0) {
                        // no page: a box outside the tensor, which reads as zeros
                        const int row = head * p.c.page + tok % p.c.page, z = pg >= 0 ? pg : p.c.n_pages;
                        const uint32_t dst = raw0 + slot * 2 * KT * D + 16 * g * D;
                        tma_load_3d(dst, &kmap, 0, row, z, &raw_full[slot]);
                        tma_load_3d(dst + KT * D, &vmap, 0, row, z, &raw_full[slot]);
                    }
                    const long long si = pg >= 0 ? (long long)pg * p.c.n_kv + head : 0;
                    copy4(&meta[ms].ks[g], p.c.k_scale + si, pg >= 0);
                    copy4(&meta[ms].vs[g], p.c.v_scale + si, pg >= 0);
                    copies_arrive(&meta_full[ms]);
                }
            }
        }
        if (!dead && !mbar_wait(&i_empty[k % kItems], (k / kItems + 1) & 1u)) dead = true;
        if (lane == 0 && !dead) {
            items[k % kItems].n = 0;
            mbar_arrive(&i_full[k % kItems]);
        }
    } else if (warp == kMmaWarp) {
        // ---------------- products ----------------
        if (lane == 0) {
            uint32_t units = 0, parity[2] = {0u, 0u};
            const uint64_t kd = smem_desc(k0, 128u, 16u * D), vd = smem_desc(v0, 16u * D, 128u);
            uint64_t qd[2];
            for (int h = 0; h < 2; ++h) qd[h] = smem_desc(q0 + h * HALF * D * 2, 128u, 16u * D);
            auto scores = [&](int h) {
#pragma unroll
                for (int c = 0; c < D / 16; ++c) mma_f16(tmem + 128u * h, qd[h] + 16u * c, kd + 16u * c, ID_S, c > 0);
                mma_commit(&s_full[h]);
            };
            auto outputs = [&](int h, bool add) {
#pragma unroll
                for (int c = 0; c < KT / 16; ++c)
                    mma_f16_ta(tmem + 256u + 128u * h, tmem + 128u * h + 8u * c, vd + (uint64_t)(2 * D * c), ID_O, add || c > 0);
                mma_commit(&pv_done[h]);
            };
            bool dead = false;
            for (uint32_t k = 0; !dead; ++k) {
                if (!mbar_wait(&i_full[k % kItems], (k / kItems) & 1u)) break;
                const int n = items[k % kItems].n, halves = items[k % kItems].rows > HALF ? 2 : 1;
                if (n == 0) break;
                mbar_arrive(&i_empty[k % kItems]);
                if (!mbar_wait(&q_ready, k & 1u) || !mbar_wait(&k_ready, units & 1u)) break;
                tc_fence_after();
                for (int h = 0; h < halves; ++h) scores(h);
                mma_commit(&k_free);
                for (int i = 0; i < n && !dead; ++i, ++units) {
                    for (int h = 0; h < halves; ++h) {
                        // P V of this tile, then S of the next one over the same columns
                        if ((h == 0 && !mbar_wait(&v_ready, units & 1u)) || !mbar_wait(&p_ready[h], parity[h])) {
                            dead = true;
                            break;
                        }
                        parity[h] ^= 1u;
                        tc_fence_after();
                        outputs(h, i > 0);
                        if (h == halves - 1) mma_commit(&v_free);
                        if (i + 1 < n) {
                            if (h == 0) {
                                if (!mbar_wait(&k_ready, (units + 1) & 1u)) {
                                    dead = true;
                                    break;
                                }
                                tc_fence_after();
                            }
                            scores(h);
                            if (h == halves - 1) mma_commit(&k_free);
                        }
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp >= kSoftmaxWarps) {
        // ---------------- codes to fp16 ----------------
        const int cw = warp - kSoftmaxWarps;
        uint32_t unit = 0;
        bool dead = false;
        for (uint32_t k = 0;; ++k) {
            if (!mbar_wait(&i_full[k % kItems], (k / kItems) & 1u)) stop_convert = 1;
            named_sync(2, 32 * kConvertWarps);
            const int n = items[k % kItems].n;
            if (stop_convert || n == 0) break;
            named_sync(2, 32 * kConvertWarps);
            if (cw == 0 && lane == 0) mbar_arrive(&i_empty[k % kItems]);
            for (int i = 0; i < n; ++i, ++unit) {
                const int slot = unit % kRaw;
                const uint32_t raw = raw0 + slot * 2 * KT * D;
                if (!dead && (!mbar_wait(&raw_full[slot], (unit / kRaw) & 1u) || !mbar_wait(&k_free, (unit + 1) & 1u))) dead = true;
                convert_tile<D>(raw, k0, cw, lane);
                proxy_fence();
                __syncwarp();
                if (lane == 0) mbar_arrive(&k_ready);
                if (!dead && !mbar_wait(&v_free, (unit + 1) & 1u)) dead = true;
                convert_tile<D>(raw + KT * D, v0, cw, lane);
                proxy_fence();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&v_ready);
                    mbar_arrive(&raw_empty[slot]);
                }
            }
        }
    } else {
        // ---------------- softmax ----------------
        const int half = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + 128u * half + lanes, to = tmem + 256u + 128u * half + lanes;
        uint32_t unit = 0, tiles = 0;                     // units of the CTA, and those with this half
        bool dead = false;
        for (uint32_t k = 0;; ++k) {
            if (!mbar_wait(&i_full[k % kItems], (k / kItems) & 1u)) stop = 1;
            named_sync(1, 32 * kSoftmaxWarps);            // every warp leaves here, or none
            const Item it = items[k % kItems];
            if (stop || it.n == 0) break;
            const bool act = it.rows > HALF * half;
            const int r = HALF * half + 32 * (warp & 3) + lane;
            const bool have = r < it.rows;
            const int tok = p.group.div(it.j * RT + r), head = it.h * p.group.d + it.j * RT + r - tok * p.group.d;
            const int pos = have ? it.len - it.m + tok : -1;
            float fac = 0.f;
            if (act) {
                // the row of q: power-of-two scale, fp16, operand image
                const T *src = static_cast<const T *>(p.q) + (it.r0 + tok) * p.ldq + (long long)head * D;
                uint4 raw[D / 8];
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) raw[c] = have ? *reinterpret_cast<const uint4 *>(src + 8 * c) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    float x[8];
                    load8(reinterpret_cast<const T *>(&raw[c]), x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
                }
                const int ex = tc_scale_exponent(top);
                const float up = pow2(ex);
                fac = pow2(-ex) * (p.scale * kLog2e);
                const uint32_t dst = q0 + half * HALF * D * 2;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    float x[8];
                    load8(reinterpret_cast<const T *>(&raw[c]), x);
                    sts128(dst + image_at<D>(r - HALF * half, c),
                           make_uint4(pack2(x[0] * up, x[1] * up), pack2(x[2] * up, x[3] * up), pack2(x[4] * up, x[5] * up),
                                      pack2(x[6] * up, x[7] * up)));
                }
                proxy_fence();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_ready);

            float m = -INFINITY, l = 0.f;
            int vexp = kMinExp;
            for (int y = it.y0; y < it.y0 + it.n; ++y, ++unit) {
                const TileMeta &mt = meta[unit % kMeta];
                if (!dead && !mbar_wait(&meta_full[unit % kMeta], (unit / kMeta) & 1u)) dead = true;
                if (act) {
                    if (!dead && !mbar_wait(&s_full[half], tiles & 1u)) dead = true;
                    tc_fence_after();
                    const int t0 = (y < it.sinks ? y : it.w0 + (y - it.sinks)) * KT;
                    bool pages = true;
#pragma unroll
                    for (int i = 0; i < kGroups; ++i) pages &= mt.have[i] != 0;
                    // every row of the warp sees every token (rows that are not there may)
                    const bool all = __all_sync(0xffffffffu, pages && (!have || (t0 + KT - 1 <= pos && (p.window == 0 || t0 > pos - p.window ||
                                                                                                       t0 + KT - 1 < p.n_sink))));
                    auto hides = [&](int t, int g) {
                        return t > pos || (p.window > 0 && pos - t >= p.window && t >= p.n_sink) || !mt.have[g];
                    };
                    // ---- the row's largest score, and the V scales that it sees
                    float top = -INFINITY;
                    int big = kMinExp;
#pragma unroll
                    for (int c = 0; c < KT / 32; ++c) {
                        uint32_t s[32];
                        tmem_ld32(ts + 32 * c, s);
                        tmem_ld_wait(s);
#pragma unroll
                        for (int gi = 0; gi < 2; ++gi) {
                            const int g = 2 * c + gi;
                            const float f = mt.ks[g] * fac;
                            bool sees = have;
                            if (!all) {
                                sees = false;
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const bool h = hides(t0 + 16 * g + e, g);
                                    sees |= !h;
                                    if (!h) top = fmaxf(top, __uint_as_float(s[16 * gi + e]) * f);
                                }
                            } else if (f >= 0.f) {
                                float x = __uint_as_float(s[16 * gi]);
#pragma unroll
                                for (int e = 1; e < 16; ++e) x = fmaxf(x, __uint_as_float(s[16 * gi + e]));
                                top = fmaxf(top, x * f);
                            } else {
#pragma unroll
                                for (int e = 0; e < 16; ++e) top = fmaxf(top, __uint_as_float(s[16 * gi + e]) * f);
                            }
                            const int be = (int)(__float_as_uint(mt.vs[g]) >> 23) & 255;
                            if (sees && be != 0 && be <= 127 + kMaxExp - 4) big = max(big, be - 126);
                        }
                    }
                    // ---- move the references, rarely
                    const bool raise = top > m + kSlack || big > vexp;
                    if (__any_sync(0xffffffffu, raise)) {
                        float a = 1.f;
                        const float mn = fmaxf(m, top);
                        a = m == -INFINITY ? 0.f : ex2(m - mn);
                        m = mn;
                        l *= a;
                        if (big > vexp) {
                            big += 2;                 // room to grow
                            a = vexp == kMinExp ? 0.f : a * pow2(vexp - big);
                            vexp = big;
                        }
                        if (y > it.y0) {
                            if (!dead && !mbar_wait(&pv_done[half], (tiles + 1) & 1u)) dead = true;
                            tc_fence_after();
#pragma unroll
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld32(to + 32 * c, o);
                                tmem_ld_wait(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                                tmem_st32(to + 32 * c, o);
                            }
                            tmem_st_wait();
                        }
                    }
                    // ---- weights
                    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
                    for (int c2 = 0; c2 < KT / 64; ++c2) {
                        uint32_t out[32];
#pragma unroll
                        for (int cc = 0; cc < 2; ++cc) {
                            uint32_t s[32];
                            tmem_ld32(ts + 64 * c2 + 32 * cc, s);
                            tmem_ld_wait(s);
#pragma unroll
                            for (int gi = 0; gi < 2; ++gi) {
                                const int g = 4 * c2 + 2 * cc + gi;
                                const float f = mt.ks[g] * fac, vs = mt.vs[g];
                                const int be = (int)(__float_as_uint(vs) >> 23);      // with the sign: a negative scale is not plain
                                const float lr = lg2(vs) - (float)vexp;
                                // the V scale goes into the exponent where it is an ordinary number
                                const bool plain = __all_sync(0xffffffffu, be != 0 && be <= 127 + kMaxExp - 4 && (lr > -60.f || !have));
                                float w[16], sum = 0.f;
                                const float add = plain ? lr - base : -base;
#pragma unroll
                                for (int e = 0; e < 16; ++e) w[e] = ex2(fmaf(__uint_as_float(s[16 * gi + e]), f, add));
                                if (!all) {
#pragma unroll
                                    for (int e = 0; e < 16; ++e)
                                        if (hides(t0 + 16 * g + e, g)) w[e] = 0.f;
                                }
#pragma unroll
                                for (int e = 0; e < 16; ++e) sum += w[e];
                                if (plain) {
                                    l = fmaf(sum, ex2(-lr), l);
                                } else {
                                    l += sum;
                                    const int bu = be & 255;
                                    const float ratio = bu == 0 ? 0.f : bu > 127 + kMaxExp - 4 ? __int_as_float(0x7fc00000) : vs * pow2(-vexp);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) w[e] = !all && hides(t0 + 16 * g + e, g) ? 0.f : w[e] * ratio;
                                }
#pragma unroll
                                for (int e = 0; e < 8; ++e) out[16 * cc + 8 * gi + e] = pack2(w[2 * e], w[2 * e + 1]);
                            }
                        }
                        tmem_st32(ts + 32 * c2, out);      // over columns of S that have been read
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_ready[half]);
                    ++tiles;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&meta_empty[unit % kMeta]);
            }

            // ---------------- the item's end ----------------
            const bool whole = it.c0 == it.c1;
            float *parts = reinterpret_cast<float *>(p.ws + attn_counter_bytes());
            constexpr size_t PF = attn_part_floats(RT, D);
            T *out = static_cast<T *>(p.out) + (it.r0 + tok) * p.ldo + (long long)head * D;
            if (act) {
                if (!dead && !mbar_wait(&pv_done[half], (tiles + 1) & 1u)) dead = true;
                tc_fence_after();
                float back = vexp == kMinExp ? 0.f : pow2(vexp);
                if (whole) back = l != 0.f ? back / l : 0.f;      // no visible token: zeros
                float *part = parts + (size_t)it.slot * PF + (size_t)r * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(to + 32 * c, o);
                    tmem_ld_wait(o);
                    if (!have) continue;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float x[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(o[e + i]) * back;
                        if (whole) store8(out + 32 * c + e, x);
                        else store8(part + 32 * c + e, x);
                    }
                }
                if (!whole && have) *reinterpret_cast<float2 *>(parts + (size_t)it.slot * PF + (size_t)RT * D + 2 * r) = make_float2(m, l);
                tc_fence_before();
            }
            if (!whole) {
                unsigned *counter = reinterpret_cast<unsigned *>(p.ws) + it.c0;
                __threadfence();
                named_sync(1, 32 * kSoftmaxWarps);
                if (threadIdx.x == 0) {
                    const bool is_last = atomicAdd(counter, 1u) == (unsigned)(it.c1 - it.c0);
                    if (is_last) *counter = 0u;          // ready for the next call
                    last_part = is_last;
                }
                named_sync(1, 32 * kSoftmaxWarps);
                if (last_part) {
                    __threadfence();
                    auto part_of = [&](int c) { return parts + (size_t)(2 * c + (c == it.c0 ? 1 : 0)) * PF; };
                    // a line of threads per row, 4 elements a thread
                    constexpr int COLS = D / 4, LINES = 32 * kSoftmaxWarps / COLS, AHEAD = 8;
                    const int col = threadIdx.x % COLS, line = threadIdx.x / COLS;
                    for (int row = line; row < it.rows; row += LINES) {
                        float pm = -INFINITY, sum = 0.f;
                        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                        for (int c = it.c0; c <= it.c1; c += AHEAD) {
                            float2 ml[AHEAD];
                            float4 v[AHEAD];
#pragma unroll
                            for (int i = 0; i < AHEAD; ++i) {
                                if (c + i > it.c1) continue;
                                const float *pp = part_of(c + i);
                                ml[i] = __ldcg(reinterpret_cast<const float2 *>(pp + (size_t)RT * D) + row);
                                v[i] = __ldcg(reinterpret_cast<const float4 *>(pp + (size_t)row * D) + col);
                            }
#pragma unroll
                            for (int i = 0; i < AHEAD; ++i) {
                                if (c + i > it.c1) continue;
                                const float mn = fmaxf(pm, ml[i].x);
                                const float a = pm == -INFINITY ? 0.f : ex2(pm - mn), b = ml[i].x == -INFINITY ? 0.f : ex2(ml[i].x - mn);
                                pm = mn;
                                sum = sum * a + ml[i].y * b;
                                acc.x = acc.x * a + v[i].x * b;
                                acc.y = acc.y * a + v[i].y * b;
                                acc.z = acc.z * a + v[i].z * b;
                                acc.w = acc.w * a + v[i].w * b;
                            }
                        }
                        const float inv = sum != 0.f ? 1.f / sum : 0.f;
                        const int tk = p.group.div(it.j * RT + row), hd = it.h * p.group.d + it.j * RT + row - tk * p.group.d;
                        store4(static_cast<T *>(p.out) + (it.r0 + tk) * p.ldo + (long long)hd * D + 4 * col,
                               make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
                    }
                }
            }
            named_sync(1, 32 * kSoftmaxWarps);
            if (threadIdx.x == 0) mbar_arrive(&i_empty[k % kItems]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
}

template <class T, int D> cudaError_t launch(const AttnArgs &a, cudaStream_t s, const DeviceInfo &dev) {
    constexpr int smem = smem_bytes<D>();
    static PerDeviceOnce once;
    cudaError_t e = once.run([] { return cudaFuncSetAttribute(attn_tc<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    CUtensorMap km, vm;
    if (!make_map(&km, a.c.k, a.c) || !make_map(&vm, a.c.v, a.c)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(dev.sm_count < kTcGrid ? dev.sm_count : kTcGrid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_tc<T, D>, km, vm, a);
}

}  // namespace

unsigned attn_tc_wait_timeouts(bool reset) {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof(v)) != cudaSuccess) return 0;
    if (reset) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_wait_timeouts, &z, sizeof(z));
    }
    return v;
}

size_t attn_tc_ws_bytes(int d) { return attn_counter_bytes() + 2 * kTcGrid * attn_part_floats(RT, d) * 4; }

cudaError_t launch_attn_tc(int dt, const AttnArgs &a, cudaStream_t s, const DeviceInfo &dev) {
    if (dt == PQ_F16) return a.c.d == 128 ? launch<__half, 128>(a, s, dev) : launch<__half, 64>(a, s, dev);
    return a.c.d == 128 ? launch<__nv_bfloat16, 128>(a, s, dev) : launch<__nv_bfloat16, 64>(a, s, dev);
}

}  // namespace pqk
