// Attention over the paged 8-bit cache for prompts (many rows per sequence) on
// the 5th-generation tensor cores: 16-bit rows, head sizes 64 and 128.
//
// The same one-pass softmax as the decode kernel, with the rows on the wide
// side: 128 rows by 128 tokens per product,
//     S = q' K^T     A = q' (fp16, shared memory), B = K's codes (fp16, K-major)
//     O += P V       A = P (fp16, tensor memory, over S), B = V's codes (MN-major)
// q' is q scaled per row by a power of two, its largest element to 2^9..2^10 (exact, but for bf16 elements 2^26 below
// the row's largest, which lose last bits), codes are exact in fp16.  A CTA takes 256 rows of one sequence and kv head, as two
// halves whose products and softmaxes alternate, so that both share one
// conversion of each K and V tile from 8 bits.  P lies over the S it came from.
//
// Each half's chain is softmax -> P V -> S of the next tile, and the two
// halves' chains share the tensor cores: of a tile's 3400 cycles at head size
// 128 the products take 2048.  A row's thread needs about 1900 for its 128
// weights (fma, exponential, sum, packing: 2.5 instructions each, and the
// reads of tensor memory), the products after it 512 + 512, the hand-overs
// 400.  2048 rows of 32 heads over 10240 tokens (8 kv heads of 128) take
// 248 us, 1.2 PFLOP/s of the 1.93 that a large bf16 product reaches; 4 prompts of
// 1000 to 4096 tokens with a window of 1024 (14 heads of 64 over 2) 83 us, where
// the items' starts and ends and the masked tiles cost as much as the rest.
// Measured and not taken: halves of a tile's tokens as products of their own
// (S: 305 us, P V: 285), with 128 weights held before any is stored 282.
//
//   warps 0-7    softmax, thread = row (tensor-memory lane), warps 0-3 the
//                first half: weights of S back to tensor memory; at an item's
//                start the rows of q, at its end the rows of the output
//   warps 8-11   codes -> fp16 into operand images (rows of 8 x 16 bytes: the
//                same image serves as K-major K and as MN-major V)
//   warp 12      walks the units, TMA of K and V tiles, page numbers and scales
//   warp 13      issues the products: the whole warp together, one elected lane
//                (from a single thread's branch 8 products took 900 cycles to issue, so 400)
//   warp 14      what the softmax needs of a tile's page scales
// Shared memory at head size 128: q 64 KB, a ring of three converted tiles
// (K and V in turn: with one of each, a conversion waited for the products of the
// tile before, 341 -> 312 us) 96 KB, four raw ones 64 KB.
//
// Per page the weights are formed as exp2(S * f + c), f = q's and K's scales,
// c = log2(V's scale) - log2 R, R a power of two that follows the largest product of
// a weight and its page's V scale, as in the decode kernel: the V scale costs
// nothing per element; the weight sum undoes it once a page.
// The running maximum and R lag as in the decode kernel, so O
// is rescaled (by its own row's thread) only now and then: when a
// row's weights of 64 tokens, with or without the scales, sum to more than 2^15, which keeps each inside
// fp16 and needs no maximum per element.  P is rounded to fp16: 11 bits, below
// 2^-14 of R an absolute 2^-25 of it; the sum l is taken of the weights before.
// bf16 rows, which have 8 bits, do not see it (1.66e-3 of the output off against 64 bits, 1.65e-3
// by the output's own rounding).  f16 rows do (2.9e-4 against 2.1e-4): as pairs of fp16, as the
// decode kernel takes them, they are at 2.1e-4, but the second P V and the packing cost
// 2048 rows over 10240 tokens 317 us instead of 248 and the windowed prompts 97 instead of 83.
// The products cut their sums off towards zero: O ends up to 6e-5 short over 131072 tokens, a third of an f16 rounding.
// pq_attn_mod (MOD): 32 columns at a time (a cap over 64: 445 us where 32 took 433: code fetch), those that
// nobody sees passed over, biased items from the row's own token back. Capped scores cost 14 cycles a pair in the
// multipliers and 14 in the exponentials' unit, see kNearCap: the same 2048 rows 430 us; two halves' weights, which run side by
// side, take 3500 cycles of a tile's 6400. Packed documents (2 x 4096 rows, about 700 tokens each) 169 us, a third of it the starts
// and ends of items of 4 tiles.
// Tiles at an edge of some row's view take the same step with a mask; tiles
// with missing pages, with scales that are no ordinary positive numbers, or
// with maxima past 2^20 (where the V scale would be lost beside it) a slower one.

#include <type_traits>

#include "attn_common.cuh"
#include "pq_tcgen05.cuh"

namespace pqk {
namespace {

constexpr int RT = 256, HALF = 128;          // rows of an item, and of each half
constexpr int kSoftmaxWarps = 8, kConvertWarps = 4;
constexpr int kWalkWarp = kSoftmaxWarps + kConvertWarps, kMmaWarp = kWalkWarp + 1, kScaleWarp = kWalkWarp + 2;
constexpr int kThreads = 32 * (kScaleWarp + 1);
constexpr int kImages = 3, kMeta = 4, kItems = 8;
// An item's rows in and out, its masked tiles and its empty pipeline, in units (2: a prompt of 8192 tokens, 32 heads
// over 8, 585 us, windowed prompts 94; 6: 470 and 88; 10: 478 and 89).
constexpr int kItemCost = 6;
constexpr int kModItemCost = 4;              // with pq_attn_mod's dearer tiles (packed documents: 2: 181 us, 4: 176, 6: 185)
constexpr int kLeast = 3;                    // places of a CTA (64 rows over 4096 tokens: 8: 32.6 us, 4: 25.0, 3: 24.2, 2: 24.6)
constexpr int kTcGrid = 160;                 // CTAs at most: one per SM
constexpr int kTmemCols = 512;
constexpr float kMost = 32768.f;             // the running maximum moves when a row's weights of one step sum to more: fp16 holds each
constexpr float kFar = 1048576.f;            // maxima up to here leave room for the V scales beside them

// raw tiles, K and V in turn
template <int D> __host__ __device__ constexpr int raw_tiles() { return D == 128 ? 4 : 8; }
template <int D> __host__ __device__ constexpr int smem_bytes() {
    return 1024 + RT * D * 2 + kImages * KT * D * 2 + raw_tiles<D>() * KT * D;
}
static_assert(smem_bytes<128>() <= 226 * 1024, "shared memory per CTA, beside the static part");

// Operand image of n rows of D fp16: 8 x 16-byte core matrices, the next 8
// elements of a row 128 bytes on, the next 8 rows 16 * D bytes on.
template <int D> __device__ __forceinline__ uint32_t image_at(int row, int chunk) {
    return (uint32_t)(row >> 3) * (16 * D) + chunk * 128 + (row & 7) * 16;
}

// 16 bytes (or zeros when !have) to shared memory, asynchronously and past the L1 cache; and the wait for a thread's own.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (x, y) * f + a.
__device__ __forceinline__ void fma2(uint32_t &x, uint32_t &y, float f, float a) {
    asm("{\n .reg .b64 p, q, r;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %2};\n mov.b64 r, {%3, %3};\n"
        " fma.rn.f32x2 p, p, q, r;\n mov.b64 {%0, %1}, p;\n}"
        : "+r"(x), "+r"(y)
        : "f"(f), "f"(a));
}

// (x, y) * (u, v) + a.
__device__ __forceinline__ void fma2(uint32_t &x, uint32_t &y, float u, float v, float a) {
    asm("{\n .reg .b64 p, q, r;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n mov.b64 r, {%4, %4};\n"
        " fma.rn.f32x2 p, p, q, r;\n mov.b64 {%0, %1}, p;\n}"
        : "+r"(x), "+r"(y)
        : "f"(u), "f"(v), "f"(a));
}
__device__ __forceinline__ void fma2(float &x, float &y, float u, float v, float a) {
    asm("{\n .reg .b64 p, q, r;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n mov.b64 r, {%4, %4};\n"
        " fma.rn.f32x2 p, p, q, r;\n mov.b64 {%0, %1}, p;\n}"
        : "+f"(x), "+f"(y)
        : "f"(u), "f"(v), "f"(a));
}
// (x, y) squared.
__device__ __forceinline__ void square2(float &x, float &y) {
    asm("{\n .reg .b64 p;\n mov.b64 p, {%0, %1};\n mul.rn.f32x2 p, p, p;\n mov.b64 {%0, %1}, p;\n}" : "+f"(x), "+f"(y));
}
// (x, y) * f.
__device__ __forceinline__ void mul2(uint32_t &x, uint32_t &y, float f) {
    asm("{\n .reg .b64 p, q;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %2};\n mul.rn.f32x2 p, p, q;\n mov.b64 {%0, %1}, p;\n}"
        : "+r"(x), "+r"(y)
        : "f"(f));
}

// Bits of the f32 with the value of a positive 16-bit pattern (both order as their bits do).
template <class T> __device__ __forceinline__ uint32_t magnitude(uint32_t bits) {
    if (std::is_same<T, __nv_bfloat16>::value) return bits << 16;
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)bits)));
}

// A tile's page scales as the softmax takes them.
struct TileScales {
    float ks[kGroups], vs[kGroups], lv[kGroups];      // lv = log2(vs)
    float lv_min;                                     // of the plain ones
    int ve[kGroups];                                  // |vs| < 2^ve; kMinExp for those that take no part
    int ve_max;
    int have;                                         // bit g: group g has a page
    int plain;                                        // bit g: it does, with ordinary positive scales
    int t0;                                           // its first token
    bool quick;                                       // all groups plain, the V scales within 2^58 of each other
};

// One tile of codes (128 tokens, swizzled as TMA left it) to its fp16 image, by the four converting warps.
template <int D> __device__ __forceinline__ void convert_tile(uint32_t raw, uint32_t image, int warp, int lane) {
    constexpr int CHUNKS = D / 16, PER = CHUNKS / 4;            // 16-code chunks of a row; a warp takes 8 rows x 4 chunks
#pragma unroll
    for (int i0 = 0; i0 < 16 * PER / kConvertWarps; i0 += 4) {
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int unit = (i0 + i) * kConvertWarps + warp, row = unit / PER * 8 + (lane & 7), c = unit % PER * 4 + (lane >> 3);
            const int sw = D == 128 ? row & 7 : (row >> 1) & 3;
            w[i] = lds128(raw + row * D + ((c ^ sw) << 4));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int unit = (i0 + i) * kConvertWarps + warp, row = unit / PER * 8 + (lane & 7), c = unit % PER * 4 + (lane >> 3);
            const uint32_t x = w[i].x ^ 0x80808080u, y = w[i].y ^ 0x80808080u, z = w[i].z ^ 0x80808080u, v = w[i].w ^ 0x80808080u;
            const uint32_t to = image + image_at<D>(row, 2 * c);
            sts128(to, make_uint4(codes2<0x4140>(x), codes2<0x4342>(x), codes2<0x4140>(y), codes2<0x4342>(y)));
            sts128(to + 128, make_uint4(codes2<0x4140>(z), codes2<0x4342>(z), codes2<0x4140>(v), codes2<0x4342>(v)));
        }
    }
}

// MOD: 0 for pq_attn, else kViews and what else of pq_attn_mod.
template <class T, int D, int MOD>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, AttnArgs p) {
    constexpr uint32_t ID_S = instr_desc(HALF, KT), ID_O = instr_desc(HALF, D) | (1u << 16);      // bit 16: B is MN-major
    constexpr int kRaw = raw_tiles<D>();
    constexpr bool EXACT = MOD == kExact;
    using Walk = UnitWalk<RT, KT, MOD ? kModItemCost : kItemCost, MOD != 0>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t raw_full[kRaw], raw_empty[kRaw], meta_full[kMeta], meta_empty[kMeta], scales_full[kMeta], i_full[kItems],
        i_empty[kItems], image_full[kImages], image_empty[kImages], s_full[2], p_ready[2], pv_done[2], q_ready;
    __shared__ __align__(16) TileMeta meta[kMeta];
    __shared__ __align__(16) TileScales scales[kMeta];
    __shared__ Item items[kItems];
    __shared__ uint32_t tmem_base;
    __shared__ volatile int stop, stop_convert;

    // converted tiles, q, raw tiles, from a 1024-byte boundary; of both kinds of tile, K of unit u is number 2 u and V 2 u + 1
    const uint32_t image0 = (smem_u32(smem_raw) + 1023u) & ~1023u, q0 = image0 + kImages * KT * D * 2, raw0 = q0 + RT * D * 2;
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
            mbar_init(&scales_full[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&i_full[i], 1);
            mbar_init(&i_empty[i], 4);
        }
        for (int i = 0; i < kImages; ++i) {
            mbar_init(&image_full[i], kConvertWarps);
            mbar_init(&image_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(&q_ready, kSoftmaxWarps);
        fence_mbar_init();
    }
    if (threadIdx.x == 32 * kWalkWarp) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
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

    if (warp >= kWalkWarp) {
        if (warp == kWalkWarp) {
        // ---------------- walk and loads ----------------
        constexpr int BATCH = 32 / kGroups;
        const int g = lane % kGroups, sub = lane / kGroups;
        Walk at;
        long long first, last;
        const Cut cut = find_range<Walk, kLeast>(p, at, first, last);
        Split split;                       // of the last item: only that can go on in another CTA
        split.c1 = -1;
        if (lane == 0) splits_of(p)[blockIdx.x].c1 = -1;      // should a wait below run out
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
                        items[k % kItems] = item_of(at, first, last);
                        mbar_arrive(&i_full[k % kItems]);
                    }
                    ++k;
                }
                if (sub == n) {
                    tok = at.token0((MOD & kBias) != 0) + 16 * g;
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
            for (int i = 0; i < n && !dead; ++i, ++n_unit) {
                const int ms = n_unit % kMeta;
                if (!mbar_wait(&meta_empty[ms], (n_unit / kMeta + 1) & 1u)) {
                    dead = true;
                    break;
                }
                if (sub == i) meta[ms].have[g] = pg >= 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&meta_full[ms]);
                __syncwarp();
                if (sub == i) {
                    const long long si = pg >= 0 ? (long long)pg * p.c.n_kv + head : 0;
                    copy4(&meta[ms].ks[g], p.c.k_scale + si, pg >= 0);
                    copy4(&meta[ms].vs[g], p.c.v_scale + si, pg >= 0);
                    copies_arrive(&meta_full[ms]);
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t j = 2 * n_unit + kv, slot = j % kRaw;
                    if (dead || !mbar_wait(&raw_empty[slot], (j / kRaw + 1) & 1u)) {
                        dead = true;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&raw_full[slot], KT * D);
                    __syncwarp();
                    if (sub == i && 16 * g % p.c.page == 0) {
                        // no page: a box outside the tensor, which reads as zeros
                        const int row = head * p.c.page + tok % p.c.page, z = pg >= 0 ? pg : p.c.n_pages;
                        tma_load_3d(raw0 + slot * KT * D + 16 * g * D, kv ? &vmap : &kmap, 0, row, z, &raw_full[slot]);
                    }
                }
            }
        }
        if (lane == 0) splits_of(p)[blockIdx.x] = split;
        if (!dead && !mbar_wait(&i_empty[k % kItems], (k / kItems + 1) & 1u)) dead = true;
        if (lane == 0 && !dead) {
            items[k % kItems].n = 0;
            mbar_arrive(&i_full[k % kItems]);
        }
        } else if (warp == kMmaWarp) {
        // ---------------- products (the whole warp, one lane issuing) ----------------
            const uint32_t one = elect_one(), tm = __reduce_max_sync(0xffffffffu, tmem);
            uint32_t units = 0, parity[2] = {0u, 0u};
            const uint64_t kd = smem_desc(image0, 128u, 16u * D), vd = smem_desc(image0, 16u * D, 128u), qd = smem_desc(q0, 128u, 16u * D);
            auto wait = [](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0; };
            auto image = [](uint32_t j) { return (uint64_t)(j % kImages * (KT * D * 2 / 16)); };
            auto filled = [&](uint32_t j) { return wait(&image_full[j % kImages], (j / kImages) & 1u); };
            auto scores = [&](int h, uint32_t u) {
                const uint64_t a = qd + (uint64_t)(h * (HALF * D * 2 / 16)), b = kd + image(2 * u);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) mma_f16_one(one, tm + 128u * h, a + 16u * c, b + 16u * c, ID_S, c > 0);
                mma_commit_one(one, &s_full[h]);
            };
            auto outputs = [&](int h, uint32_t u, bool add) {
                const uint64_t b = vd + image(2 * u + 1);
#pragma unroll
                for (int c = 0; c < KT / 16; ++c)
                    mma_f16_ta_one(one, tm + 256u + 128u * h, tm + 128u * h + 8u * c, b + (uint64_t)(2 * D * c), ID_O, add || c > 0);
                mma_commit_one(one, &pv_done[h]);
            };
            bool dead = false;
            for (uint32_t k = 0; !dead; ++k) {
                if (!wait(&i_full[k % kItems], (k / kItems) & 1u)) break;
                const int n = (int)__reduce_max_sync(0xffffffffu, (unsigned)items[k % kItems].n);
                const int halves = __any_sync(0xffffffffu, items[k % kItems].rows > HALF) ? 2 : 1;
                if (n == 0) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(&i_empty[k % kItems]);
                if (!wait(&q_ready, k & 1u) || !filled(2 * units)) break;
                tc_fence_after();
                scores(0, units);
                if (halves == 2) scores(1, units);
                mma_commit_one(one, &image_empty[2 * units % kImages]);
                for (int i = 0; i < n && !dead; ++i, ++units) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (dead || h == halves) break;
                        // P V of this tile, then S of the next one over the same columns
                        if ((h == 0 && !filled(2 * units + 1)) || !wait(&p_ready[h], parity[h])) {
                            dead = true;
                            break;
                        }
                        parity[h] ^= 1u;
                        tc_fence_after();
                        outputs(h, units, i > 0);
                        if (h == halves - 1) mma_commit_one(one, &image_empty[(2 * units + 1) % kImages]);
                        if (i + 1 < n) {
                            if (h == 0) {
                                if (!filled(2 * units + 2)) {
                                    dead = true;
                                    break;
                                }
                                tc_fence_after();
                            }
                            scores(h, units + 1);
                            if (h == halves - 1) mma_commit_one(one, &image_empty[(2 * units + 2) % kImages]);
                        }
                    }
                }
            }
        } else if (warp == kScaleWarp) {
        // ---------------- a tile's scales, as the softmax takes them ----------------
            const int g = lane % kGroups;
            uint32_t unit = 0;
            bool dead = false;
            for (uint32_t k = 0; !dead; ++k) {
                if (!mbar_wait(&i_full[k % kItems], (k / kItems) & 1u)) break;
                const int n = items[k % kItems].n, y0 = items[k % kItems].y0, sinks = items[k % kItems].sinks, w0 = items[k % kItems].w0;
                const int s0 = MOD ? items[k % kItems].s0 : 0, last = (MOD & kBias) ? items[k % kItems].units - 1 : 0;
                __syncwarp();
                if (n == 0) break;
                if (lane == 0) mbar_arrive(&i_empty[k % kItems]);
                for (int i = 0; i < n && !dead; ++i, ++unit) {
                    const int ms = unit % kMeta;
                    if (!mbar_wait(&meta_full[ms], (unit / kMeta) & 1u)) dead = true;
                    const float ks = meta[ms].ks[g], vs = meta[ms].vs[g];
                    const bool have = meta[ms].have[g] != 0;
                    const int be = (int)(__float_as_uint(vs) >> 23), bu = be & 255;      // be: with the sign
                    const bool usable = bu != 0 && bu <= 127 + kMaxExp - 4;
                    const bool plain = have && usable && be < 256 && ks >= 0.f && ks < INFINITY;
                    const float lv = lg2(vs);
                    float lv_min = plain ? lv : INFINITY;
                    const int ve = usable ? bu - 126 : kMinExp;
                    int ve_max = ve;
#pragma unroll
                    for (int w = 1; w < kGroups; w <<= 1) {
                        lv_min = fminf(lv_min, __shfl_xor_sync(0xffffffffu, lv_min, w));
                        ve_max = max(ve_max, __shfl_xor_sync(0xffffffffu, ve_max, w));
                    }
                    const unsigned haves = __ballot_sync(0xffffffffu, have), plains = __ballot_sync(0xffffffffu, plain);
                    TileScales &ts = scales[ms];
                    if (lane < kGroups) {
                        ts.ks[g] = ks;
                        ts.vs[g] = vs;
                        ts.lv[g] = lv;
                        ts.ve[g] = ve;
                    }
                    if (lane == 0) {
                        ts.lv_min = lv_min;
                        ts.ve_max = ve_max;
                        ts.have = (int)(haves & 0xffu);
                        ts.plain = (int)(plains & 0xffu);
                        // scores with a bias by distance rise towards the row's own token: from there back, the references hardly move
                        const int u = (MOD & kBias) ? last - (y0 + i) : y0 + i;
                        ts.t0 = (u < sinks ? s0 + u : w0 + (u - sinks)) * KT;
                        ts.quick = p.scale >= 0.f && (plains & 0xffu) == 0xffu && lv_min - (float)ve_max > -58.f;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&scales_full[ms]);
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
#pragma unroll 1
                for (uint32_t j = 2 * unit; j < 2 * unit + 2; ++j) {
                    const uint32_t slot = j % kRaw, im = j % kImages;
                    if (!dead && (!mbar_wait(&raw_full[slot], (j / kRaw) & 1u) || !mbar_wait(&image_empty[im], (j / kImages + 1) & 1u))) dead = true;
                    convert_tile<D>(raw0 + slot * KT * D, image0 + im * KT * D * 2, cw, lane);
                    proxy_fence();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&image_full[im]);
                        mbar_arrive(&raw_empty[slot]);
                    }
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
        // rows of the output leave through the 32 rows' part of the q image, 16 bytes a lane, CH lanes a row, so that
        // global memory sees whole rows
        constexpr int CH = D / 8, ROWS = 32 / CH;
        const int sub = lane / CH, ch = lane % CH, row0 = HALF * half + 32 * (warp & 3);
        const uint32_t stage = q0 + row0 * D * 2;
        for (uint32_t k = 0;; ++k) {
            if (!mbar_wait(&i_full[k % kItems], (k / kItems) & 1u)) stop = 1;
            named_sync(1, 32 * kSoftmaxWarps);            // every warp leaves here, or none
            const Item &it = items[k % kItems];           // this group's until it says so below
            if (stop || it.n == 0) break;
            const bool act = it.rows > HALF * half;
            const int r = row0 + lane;
            const bool have = r < it.rows;
            const int tok = p.group.div(it.j * RT + r), head = it.h * p.group.d + it.j * RT + r - tok * p.group.d;
            const int pos = have ? it.len - it.m + tok : -1;
            float fac = 0.f;
            RowView row_sees = {0, 0};
            float slope = 0.f;
            if (MOD && pos >= 0) row_sees = row_view(p, it.r0 + tok, it.len);
            if ((MOD & kBias) && have) slope = slope_of<MOD == kExact>(p, head);
            if (act) {
                // the row of q: power-of-two scale, fp16, operand image
                const T *mine = static_cast<const T *>(p.q) + (it.r0 + tok) * p.ldq + (long long)head * D;
                // through the rows' own part of the operand image, whole rows a load and no two lanes on one bank either way: loads to
                // registers, 8 rows by 64 bytes each for the sake of the banks, took 4200 cycles to issue
                constexpr int PER = D / 32;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int src = i * ROWS + sub;
                    const unsigned long long row = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), src);
                    copy16(stage + src * D * 2 + ((ch ^ (src & 7)) << 4), reinterpret_cast<const uint4 *>(row) + ch, row0 + src < it.rows);
                }
                copies_wait();
                __syncwarp();
                uint4 w[4][PER];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < PER; ++j)
                        w[i][j] = lds128(stage + (8 * i + (lane & 7)) * D * 2 + (((4 * j + (lane >> 3)) ^ (lane & 7)) << 4));
                __syncwarp();
                uint32_t top[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    top[i] = 0;
#pragma unroll
                    for (int j = 0; j < PER; ++j)
                        top[i] = __vmaxu2(top[i], __vmaxu2(__vmaxu2(w[i][j].x & 0x7fff7fffu, w[i][j].y & 0x7fff7fffu),
                                                           __vmaxu2(w[i][j].z & 0x7fff7fffu, w[i][j].w & 0x7fff7fffu)));
                    top[i] = magnitude<T>(max(top[i] & 0xffffu, top[i] >> 16));
                }
#pragma unroll
                for (int o = 8; o < 32; o <<= 1)
#pragma unroll
                    for (int i = 0; i < 4; ++i) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
                uint32_t of_mine = top[0];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (lane >> 3 == i) of_mine = top[i];
                    const float up = pow2(tc_scale_exponent(top[i]));
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        float x[8];
                        load8(reinterpret_cast<const T *>(&w[i][j]), x);
                        sts128(stage + image_at<D>(8 * i + (lane & 7), 4 * j + (lane >> 3)),
                               make_uint4(pack2(x[0] * up, x[1] * up), pack2(x[2] * up, x[3] * up), pack2(x[4] * up, x[5] * up),
                                          pack2(x[6] * up, x[7] * up)));
                    }
                }
                const int ex = tc_scale_exponent(of_mine);
                fac = pow2(-ex) * (p.scale * kLog2e);
                proxy_fence();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_ready);

            float m = -INFINITY, l = 0.f;
            int vexp = kLeastExp;                         // O is in units of 2^(m + vexp), m a whole number
            const int n = it.n;
            for (int i = 0; i < n; ++i, ++unit) {
                const TileScales &sc = scales[unit % kMeta];
                if (!dead && !mbar_wait(&scales_full[unit % kMeta], (unit / kMeta) & 1u)) dead = true;
                if (act) {
                    // the row sees the tile's tokens e with e <= last and (e >= first or e < sink): all of them,
                    auto whole_view = [&] {
                        const int last = pos - sc.t0, first = p.window > 0 ? last - p.window + 1 : 0, sink = p.n_sink - sc.t0;
                        if (MOD) {
                            const bool ahead = row_sees.prefix - sc.t0 >= KT;
                            return row_sees.first <= sc.t0 && (last >= KT - 1 ? first <= 0 || sink >= KT || ahead : ahead && !(MOD & kBias));
                        }
                        return last >= KT - 1 && (first <= 0 || sink >= KT);
                    };
                    // and which of 32 c .. 32 c + 31
                    auto view = [&](int c) {
                        auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };
                        const int last = pos - sc.t0, first = p.window > 0 ? last - p.window + 1 : 0, sink = p.n_sink - sc.t0;
                        const uint32_t pages = ((sc.have >> (2 * c)) & 1 ? 0xffffu : 0u) | ((sc.have >> (2 * c + 1)) & 1 ? 0xffff0000u : 0u);
                        const uint32_t behind = below(last + 1 - 32 * c) & (~below(first - 32 * c) | below(sink - 32 * c));
                        if (MOD) return pages & (behind | below(row_sees.prefix - sc.t0 - 32 * c)) & ~below(row_sees.first - sc.t0 - 32 * c);
                        return pages & behind;
                    };
                    // O of the tiles before this one, times the row's a
                    auto rescale = [&](float a) {
                        if (i == 0) return;
                        if (!dead && !mbar_wait(&pv_done[half], (tiles + 1) & 1u)) dead = true;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(to + 16 * c, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                            tmem_st16(to + 16 * c, o);
                        }
                        tmem_st_wait();
                    };
                    // a score times log2 e of a token `away` before the row's own, capped and biased; of the tile's token e
                    auto modified = [&](float x, float away) {
                        if (MOD & kCap) x = capped<EXACT>(x, p.mod);
                        if (MOD & kBias) x = fmaf(-slope, fabsf(away), x);
                        return x;
                    };
                    auto before = [&](int e) { return (MOD & kBias) ? (float)(pos - sc.t0 - e) : 0.f; };
                    // ---- mostly all rows see the whole tile. V scales in the exponent: at most 2^60 below the reference, which
                    // may move to ve_max, and beside a maximum whose last bit does not swallow them
                    bool near = true, all = true;
                    const bool quick = __all_sync(0xffffffffu, sc.quick && (!have || (whole_view() && fabsf(m) < kFar && sc.lv_min - (float)vexp > -60.f)));
                    if (__builtin_expect(!quick, 0)) {
                        near = p.scale >= 0.f && __all_sync(0xffffffffu, !have || (m == -INFINITY ? sc.lv_min - (float)(sc.ve_max + 2) > -60.f
                                                                                                   : fabsf(m) < kFar && sc.lv_min - (float)max(vexp, sc.ve_max + 2) > -60.f));
                        all = near && sc.plain == (1 << kGroups) - 1;
                    }
                    if (!dead && !mbar_wait(&s_full[half], tiles & 1u)) dead = true;
                    tc_fence_after();
                    // The row's references move, if they are smaller, to the largest score that it sees (bits) of the n steps
                    // from c, and to the largest one times its page's V scale; the weights of the steps before are in place.
                    // Both are whole numbers: a power of two takes the stored fp16 weights along without another rounding, but
                    // for those that become smaller than 2^-14 of the new largest, which keep an absolute 2^-25 of it.
                    auto raise = [&](int c, int n, unsigned long long bits) {
                        float top = -INFINITY, tv = -INFINITY;      // tv: the largest score plus V exponent, less top
                        tmem_st_wait();
#pragma unroll 1
                        for (int g = 2 * c; g < 2 * (c + n); ++g, bits >>= 16) {
                            uint32_t x[16];
                            tmem_ld16(ts + 16 * g, x);
                            tmem_ld_wait(x);
                            const float f = sc.ks[g] * fac, away = before(16 * g);
                            float most = -INFINITY;
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if ((bits >> e) & 1) most = fmaxf(most, modified(__fmul_rn(__uint_as_float(x[e]), f), away - (float)e));
                            if (most > -INFINITY) {
                                const float t = fmaxf(top, most);
                                tv = fmaxf(tv + (top - t), (float)sc.ve[g] + (most - t));
                                top = t;
                            }
                        }
                        float a = 1.f;
                        bool turn = false;      // whether something is stored in the old units: not of a row that saw nothing before
                        if (top > -INFINITY) {
                            const float mn = fmaxf(m, ceilf(top));
                            const int up = m == -INFINITY ? kFarExp : (int)fminf(mn - m, (float)kFarExp);
                            // O's unit 2^(m + vexp) stays while m moves, as far as vexp can follow
                            const int vn = max(max(vexp - up, kLeastExp), (int)ceilf(fmaxf(tv + (top - mn), -(float)kFarExp)));
                            a = pow2(vexp - up - vn);
                            turn = m > -INFINITY && a != 1.f;
                            l *= pow2(-up);
                            m = mn;
                            vexp = vn;
                        }
                        if (!__any_sync(0xffffffffu, turn)) return;
                        rescale(a);
#pragma unroll 1
                        for (int i = 0; i < c; ++i) {
                            uint32_t w[16];
                            tmem_ld16(ts + 16 * i, w);
                            tmem_ld_wait(w);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
                                w[e] = pack2(f.x * a, f.y * a);
                            }
                            tmem_st16(ts + 16 * i, w);
                        }
                    };
                    int done = 0;                             // steps of 32 columns
                    // weights of the 32 STEPS tokens from step done, of those in b0 and b1 if MASK: fp16 pairs times their V scales, the
                    // sum without the scales, and with them (sw)
                    constexpr int STEPS = MOD ? 1 : 2;
                    uint32_t out[16 * STEPS];
                    auto store_weights = [&] {      // over columns of S that have been read
                        if constexpr (STEPS == 2) tmem_st32(ts + 16 * done, out);
                        else tmem_st16(ts + 16 * done, out);
                    };
                    float sw;
                    // NEAR: capped scores of the first three pairs in four by a polynomial, which holds for squares over the cap up
                    // to kNearCap (`beyond`: the largest), of the fourth as in capped(): the exponentials' unit would take 16
                    // cycles for each the second way, the multipliers 8 the first way, so both take 7
                    // EXACT: all by the polynomial, and where that does not hold by capped<true>() in the last of the loops below (2048
                    // rows over 10240 tokens 520 us, all by the last loop 1479)
                    constexpr float kNearCap = EXACT ? 0.36f : 0.64f, kLargest = 3.4e38f;
                    float beyond = 0.f;
                    auto weights_by = [&](auto mask, auto near_cap, uint32_t b0, uint32_t b1) {
                        constexpr bool MASK = decltype(mask)::value, NEAR = EXACT || decltype(near_cap)::value;
                        uint32_t x[2][16];
                        float add = 0.f;
                        sw = 0.f;
                        tmem_ld16(ts + 32 * done, x[0]);
#pragma unroll
                        for (int g = 0; g < 2 * STEPS; ++g) {
                            float f = sc.ks[2 * done + g] * fac;
                            const float lr = sc.lv[2 * done + g] - (float)vexp, undo = ex2(-lr);
                            float c = have ? lr - m : -INFINITY;
                            const float away = before(32 * done + 16 * g);      // of the group's first token
                            if (MOD & kCap) f = fminf(f * p.mod.to_unit, kLargest);      // a score of 0 stays 0
                            // where all is seen nothing lies ahead of the row, and the distances fall by 1 a token
                            if ((MOD & kBias) && !MASK) c = fmaf(-slope, away, c);
                            const float f2 = fminf(f * (2.f * kLog2e), kLargest), c2 = c + p.mod.top;
                            uint32_t(&s)[16] = x[g & 1];
                            tmem_ld_wait(s);
                            if (g + 1 < 2 * STEPS) tmem_ld16(ts + 32 * done + 16 * (g + 1), x[(g + 1) & 1]);
                            float sx = 0.f, sy = 0.f;
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                if ((MOD & kCap) && NEAR && (EXACT || e % 8 != 6)) {
                                    mul2(s[e], s[e + 1], f);
                                    float zx = __uint_as_float(s[e]), zy = __uint_as_float(s[e + 1]);
                                    square2(zx, zy);
                                    beyond = fmaxf(fmaxf(beyond, zx), zy);
                                    float px = p.mod.near[4], py = px;
#pragma unroll
                                    for (int k = 3; k >= 0; --k) fma2(px, py, zx, zy, p.mod.near[k]);
                                    fma2(s[e], s[e + 1], px, py, c);
                                } else if (MOD & kCap) {      // as in capped()
                                    mul2(s[e], s[e + 1], f2);
                                    float ux = ex2(__uint_as_float(s[e])), uy = ex2(__uint_as_float(s[e + 1]));
                                    add2(ux, uy, 1.f, 1.f);
                                    s[e] = __float_as_uint(rcp(ux));
                                    s[e + 1] = __float_as_uint(rcp(uy));
                                    fma2(s[e], s[e + 1], -2.f * p.mod.top, c2);
                                } else {
                                    fma2(s[e], s[e + 1], f, c);
                                }
                                if (MOD & kBias) {
                                    s[e] = __float_as_uint(fmaf(MASK ? -slope : slope, MASK ? fabsf(away - e) : (float)e, __uint_as_float(s[e])));
                                    s[e + 1] = __float_as_uint(fmaf(MASK ? -slope : slope, MASK ? fabsf(away - (e + 1)) : (float)(e + 1), __uint_as_float(s[e + 1])));
                                }
                                if (MASK) {
                                    const uint32_t b = (g < 2 ? b0 : b1) >> (16 * (g & 1) + e);
                                    if (!(b & 1)) s[e] = 0xff800000u;
                                    if (!(b & 2)) s[e + 1] = 0xff800000u;
                                }
                                const float wx = ex2(__uint_as_float(s[e])), wy = ex2(__uint_as_float(s[e + 1]));
                                add2(sx, sy, wx, wy);
                                out[8 * g + e / 2] = pack2(wx, wy);
                            }
                            sx += sy;
                            sw += sx;
                            add = fmaf(sx, undo, add);
                        }
                        return add;
                    };
                    auto weights = [&](auto mask, uint32_t b0, uint32_t b1) { return weights_by(mask, std::false_type(), b0, b1); };
                    bool go = quick || (MOD && all);
                    if constexpr (MOD != 0) {
#pragma unroll 1
                        while (go && done < 4) {
                            const uint32_t b = quick ? ~0u : view(done);
                            if (!quick && !__any_sync(0xffffffffu, b != 0)) {      // nothing of it is seen
#pragma unroll
                                for (int e = 0; e < 16; ++e) out[e] = 0u;
                                store_weights();
                                ++done;
                                continue;
                            }
                            float add = 0.f;
                            bool fits = quick || __all_sync(0xffffffffu, !have || (b == ~0u && fabsf(m) < kFar && (!(MOD & kBias) || pos - sc.t0 >= 32 * done + 31)));
                            if (fits) {
                                beyond = 0.f;
                                add = weights_by(std::false_type(), std::true_type(), 0u, 0u);
                                fits = !__any_sync(0xffffffffu, have && (fmaxf(add, sw) > kMost || beyond > kNearCap));
                                go = !EXACT || !__any_sync(0xffffffffu, have && beyond > kNearCap);
                                if (!go) break;
                            }
                            if (!fits) {
                                const uint32_t seen = have ? b : 0u;
                                bool move = __any_sync(0xffffffffu, seen != 0 && m == -INFINITY), moved = false;
#pragma unroll 1
                                do {
                                    if (move) {
                                        raise(done, 1, seen);
                                        moved = true;
                                        go = __all_sync(0xffffffffu, seen == 0 || fabsf(m) < kFar);
                                        if (!go) break;
                                    }
                                    beyond = 0.f;
                                    add = weights(std::true_type(), seen, 0u);
                                    go = !EXACT || !__any_sync(0xffffffffu, seen != 0 && beyond > kNearCap);
                                    if (!go) break;
                                    move = !moved && __any_sync(0xffffffffu, fmaxf(add, sw) > kMost);      // at the true maximum no weight is above 1
                                } while (move);
                            }
                            if (!go) break;
                            l += add;
                            store_weights();
                            ++done;
                        }
                    } else {
#pragma unroll 1
                    for (; go && done < 4; done += go ? 2 : 0) {
                        const float add = weights(std::false_type(), 0u, 0u);
                        if (__any_sync(0xffffffffu, have && fmaxf(add, sw) > kMost)) break;      // a reference has to move
                        l += add;
                        store_weights();
                    }
                    go = all;
#pragma unroll 1
                    while (go && done < 4) {
                        const uint32_t b0 = view(done), b1 = view(done + 1);
                        float add = 0.f;
                        bool move = __any_sync(0xffffffffu, (b0 | b1) != 0 && m == -INFINITY), moved = false;
#pragma unroll 1
                        do {
                            if (move) {
                                raise(done, 2, b0 | (unsigned long long)b1 << 32);
                                moved = true;
                                go = __all_sync(0xffffffffu, (b0 | b1) == 0 || fabsf(m) < kFar);
                                if (!go) break;
                            }
                            add = weights(std::true_type(), b0, b1);
                            move = !moved && __any_sync(0xffffffffu, fmaxf(add, sw) > kMost);      // at the true maximum no weight is above 1
                        } while (move);
                        if (!go) break;
                        l += add;
                        store_weights();
                        done += 2;
                    }
                    }
                    // the same with other scales, or far from zero
                    const unsigned plain = near ? (unsigned)sc.plain : 0u;
#pragma unroll 1
                    for (; done < 4; ++done) {
                        uint32_t out16[16];
                        const uint32_t bits = view(done);
                        float add = 0.f;
                        bool move = __any_sync(0xffffffffu, bits != 0 && m == -INFINITY), moved = false;
#pragma unroll 1
                        do {
                            if (move) {
                                raise(done, 1, bits);
                                moved = true;
                            }
                            uint32_t x[32];
                            tmem_ld32(ts + 32 * done, x);
                            tmem_ld_wait(x);
                            const float base = m == -INFINITY ? 0.f : m;
                            add = sw = 0.f;
#pragma unroll
                            for (int gi = 0; gi < 2; ++gi) {
                                const int g = 2 * done + gi;
                                const bool in = (plain >> g) & 1;      // the V scale is in the exponent
                                const float f = sc.ks[g] * fac, lr = in ? sc.lv[g] - (float)vexp : 0.f, away = before(16 * g);
                                float w[16], sx = 0.f, sy = 0.f;
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const bool see = (bits >> (16 * gi + e)) & 1;
                                    w[e] = ex2(see ? modified(__fmul_rn(__uint_as_float(x[16 * gi + e]), f), away - (float)e) - base + lr : -INFINITY);
                                }
#pragma unroll
                                for (int e = 0; e < 16; e += 2) add2(sx, sy, w[e], w[e + 1]);
                                add = fmaf(sx + sy, ex2(-lr), add);
                                if (!in) {
                                    const float vs = sc.vs[g];
                                    const int bu = (int)(__float_as_uint(vs) >> 23) & 255;
                                    float ratio = bu == 0 ? 0.f : bu > 127 + kMaxExp - 4 ? __int_as_float(0x7fc00000) : vs * pow2(-vexp);
                                    // a scale that far above belongs to weights near 2^-126: not 0 times infinity
                                    if (fabsf(ratio) == INFINITY) ratio = copysignf(pow2(126), vs);
                                    sx = sy = 0.f;
#pragma unroll
                                    for (int e = 0; e < 16; ++e) w[e] = (bits >> (16 * gi + e)) & 1 ? w[e] * ratio : 0.f;      // the ratio may be NaN
#pragma unroll
                                    for (int e = 0; e < 16; e += 2) add2(sx, sy, fabsf(w[e]), fabsf(w[e + 1]));
                                }
                                sw += sx + sy;
#pragma unroll
                                for (int e = 0; e < 8; ++e) out16[8 * gi + e] = pack2(w[2 * e], w[2 * e + 1]);
                            }
                            move = !moved && __any_sync(0xffffffffu, fmaxf(add, sw) > kMost);
                        } while (move);
                        l += add;
                        tmem_st16(ts + 16 * done, out16);
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
            const bool whole = it.whole;
            float *parts = parts_of(p);
            constexpr size_t PF = attn_part_floats(RT, D);
            T *out = static_cast<T *>(p.out) + (it.r0 + tok) * p.ldo + (long long)head * D;
            if (act) {
                if (!dead && !mbar_wait(&pv_done[half], (tiles + 1) & 1u)) dead = true;
                tc_fence_after();
                // in two factors where 2^vexp over the sum would not be a normal number
                const bool tiny = __any_sync(0xffffffffu, vexp < -60);
                const float rest = vexp < -60 ? pow2(-60) : 1.f;
                float back = pow2(vexp < -60 ? vexp + 60 : vexp);
                if (whole) back = l != 0.f ? back / l : 0.f;      // no visible token: zeros
                const auto mine = reinterpret_cast<unsigned long long>(whole ? static_cast<void *>(out)
                                                                             : static_cast<void *>(parts + (size_t)it.slot * PF + (size_t)r * D));
                auto leave = [&](unsigned at) {                   // bytes at .. at + 2 D - 1 of the rows
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        const int src = i * ROWS + sub;
                        const unsigned long long row = __shfl_sync(0xffffffffu, mine, src) + at;
                        if (row0 + src < it.rows) *(reinterpret_cast<uint4 *>(row) + ch) = lds128(stage + src * D * 2 + ((ch ^ (src & 7)) << 4));
                    }
                    __syncwarp();
                };
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(to + 32 * c, o);
                    tmem_ld_wait(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * back);
                    if (tiny) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * rest);
                    }
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            float x[8];
                            uint4 w;
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(o[e + i]);
                            store8(reinterpret_cast<T *>(&w), x);
                            sts128(stage + lane * D * 2 + (((4 * c + e / 8) ^ (lane & 7)) << 4), w);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            sts128(stage + lane * D * 2 + (((8 * c % CH + e / 4) ^ (lane & 7)) << 4), make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
                        if (8 * (c + 1) % CH == 0) leave(32 * c / (D / 2) * D * 2);
                    }
                }
                if (whole) leave(0);
                if (!whole && have) *reinterpret_cast<float2 *>(parts + (size_t)it.slot * PF + (size_t)RT * D + 2 * r) = make_float2(m, l);
                tc_fence_before();
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

template <class T, int D, int MOD> cudaError_t launch(const AttnArgs &a, cudaStream_t s, const DeviceInfo &dev) {
    constexpr int smem = smem_bytes<D>();
    static PerDeviceOnce once;
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(attn_tc<T, D, MOD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    CUtensorMap km, vm;
    if (!make_map(&km, a.c.k, a.c) || !make_map(&vm, a.c.v, a.c)) return cudaErrorInvalidValue;
    if (MOD && (e = launch_bounds<RT, kModItemCost>(a, s)) != cudaSuccess) return e;
    return launch_with_join<T, D, RT>(attn_tc<T, D, MOD>, dev.sm_count < kTcGrid ? dev.sm_count : kTcGrid, kThreads, smem, km, vm, a, s);
}

template <int MOD> cudaError_t launch_dt(int dt, const AttnArgs &a, cudaStream_t s, const DeviceInfo &dev) {
    if (dt == PQ_F16) return a.c.d == 128 ? launch<__half, 128, MOD>(a, s, dev) : launch<__half, 64, MOD>(a, s, dev);
    return a.c.d == 128 ? launch<__nv_bfloat16, 128, MOD>(a, s, dev) : launch<__nv_bfloat16, 64, MOD>(a, s, dev);
}

}  // namespace

#ifndef PQ_ATTN_MOD      // attn_tc_*.cu have the instances for pq_attn_mod

unsigned attn_tc_wait_timeouts(bool reset) {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof(v)) != cudaSuccess) return 0;
    if (reset) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_wait_timeouts, &z, sizeof(z));
    }
    return v;
}

size_t attn_tc_ws_bytes(int d) { return attn_splits_bytes() + 2 * kTcGrid * attn_part_floats(RT, d) * 4; }

cudaError_t launch_attn_tc(int dt, const AttnArgs &a, cudaStream_t s, const DeviceInfo &dev) { return launch_dt<0>(dt, a, s, dev); }

#endif

}  // namespace pqk
