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
// conversion of each K and V tile from 8 bits.  P lies over the S it came from.
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
//   warp 14      what the softmax needs of a tile's page scales
// Shared memory: q 64 KB, converted K and V 32 KB each, three raw tiles 96 KB.
//
// Per page the weights are formed as exp2(S * f + c), f = q's and K's scales,
// c = log2(V's scale over a power of two above the largest seen) - maximum:
// the V scale costs nothing per element; the weight sum undoes it once a page.
// The running maximum and the power of two lag as in the decode kernel, so O
// is rescaled (by its own row's thread) only now and then.  A row goes through
// tensor memory once, 64 columns at a time; columns that pass the maximum by
// more than its lag are found beside their weights: the thread then moves the
// maximum (O, the sum and the row's earlier weights of the tile are rescaled)
// and takes those columns again.  Tiles at an edge of some row's view, or with
// page scales that are no ordinary positive numbers, take a masking variant.

#include "attn_common.cuh"
#include "pq_tcgen05.cuh"

namespace pqk {
namespace {

constexpr int RT = 256, HALF = 128;          // rows of an item, and of each half
constexpr int kSoftmaxWarps = 8, kConvertWarps = 4;
constexpr int kWalkWarp = kSoftmaxWarps + kConvertWarps, kMmaWarp = kWalkWarp + 1, kScaleWarp = kWalkWarp + 2;
constexpr int kThreads = 32 * (kScaleWarp + 1);
constexpr int kRaw = 3, kMeta = 4, kItems = 8, kItemCost = 2;
constexpr int kLeast = 4;                    // places of a CTA
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

// (x, y) * f + a, and sums of pairs.
__device__ __forceinline__ void fma2(uint32_t &x, uint32_t &y, float f, float a) {
    asm("{\n .reg .b64 p, q, r;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %2};\n mov.b64 r, {%3, %3};\n"
        " fma.rn.f32x2 p, p, q, r;\n mov.b64 {%0, %1}, p;\n}"
        : "+r"(x), "+r"(y)
        : "f"(f), "f"(a));
}
__device__ __forceinline__ void add2(float &sx, float &sy, float x, float y) {
    asm("{\n .reg .b64 p, q;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n add.rn.f32x2 p, p, q;\n mov.b64 {%0, %1}, p;\n}"
        : "+f"(sx), "+f"(sy)
        : "f"(x), "f"(y));
}

__device__ __forceinline__ float max3(uint32_t x, uint32_t y, uint32_t z) {
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(__uint_as_float(x)), "f"(__uint_as_float(y)), "f"(__uint_as_float(z)));
    return m;
}

// A tile's page scales as the softmax takes them.
struct TileScales {
    float ks[kGroups], vs[kGroups], lv[kGroups];      // lv = log2(vs)
    float lv_min;                                     // of the plain ones
    int ve[kGroups];                                  // |vs| < 2^ve; kMinExp for those that take no part
    int ve_max;
    int have;                                         // bit g: group g has a page
    int plain;                                        // bit g: it does, with ordinary positive scales
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

template <class T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, AttnArgs p) {
    constexpr uint32_t ID_S = instr_desc(HALF, KT), ID_O = instr_desc(HALF, D) | (1u << 16);      // bit 16: B is MN-major
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t raw_full[kRaw], raw_empty[kRaw], meta_full[kMeta], meta_empty[kMeta], scales_full[kMeta], i_full[kItems],
        i_empty[kItems], k_ready, k_free, v_ready, v_free, s_full[2], p_ready[2], pv_done[2], q_ready;
    __shared__ __align__(16) TileMeta meta[kMeta];
    __shared__ __align__(16) TileScales scales[kMeta];
    __shared__ Item items[kItems];
    __shared__ uint32_t tmem_base;
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
            mbar_init(&scales_full[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&i_full[i], 1);
            mbar_init(&i_empty[i], 4);
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
        if (lane == 0) splits_of(p)[blockIdx.x] = split;
        if (!dead && !mbar_wait(&i_empty[k % kItems], (k / kItems + 1) & 1u)) dead = true;
        if (lane == 0 && !dead) {
            items[k % kItems].n = 0;
            mbar_arrive(&i_full[k % kItems]);
        }
        } else if (warp == kMmaWarp && lane == 0) {
        // ---------------- products ----------------
            uint32_t units = 0, parity[2] = {0u, 0u};
            const uint64_t kd = smem_desc(k0, 128u, 16u * D), vd = smem_desc(v0, 16u * D, 128u);
            uint64_t qd[2];
#pragma unroll
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
                scores(0);
                if (halves == 2) scores(1);
                mma_commit(&k_free);
                for (int i = 0; i < n && !dead; ++i, ++units) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (dead || h == halves) break;
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
        } else if (warp == kScaleWarp) {
        // ---------------- a tile's scales, as the softmax takes them ----------------
            const int g = lane % kGroups;
            uint32_t unit = 0;
            bool dead = false;
            for (uint32_t k = 0; !dead; ++k) {
                if (!mbar_wait(&i_full[k % kItems], (k / kItems) & 1u)) break;
                const int n = items[k % kItems].n;
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
            const Item &it = items[k % kItems];           // this group's until it says so below
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
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    float x[8];
                    if (have) load8(src + 8 * c, x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = max(top, have ? __float_as_uint(x[e]) & 0x7fffffffu : 0u);
                }
                const int ex = tc_scale_exponent(top);
                const float up = pow2(ex);
                fac = pow2(-ex) * (p.scale * kLog2e);
                const uint32_t dst = q0 + half * HALF * D * 2;
                // (read again: the row would not fit beside what the loop below keeps)
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    if (have) load8(src + 8 * c, x);
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
                const TileScales &sc = scales[unit % kMeta];
                if (!dead && !mbar_wait(&scales_full[unit % kMeta], (unit / kMeta) & 1u)) dead = true;
                if (act) {
                    const int t0 = (y < it.sinks ? y : it.w0 + (y - it.sinks)) * KT;
                    // the row sees the tile's tokens e with e <= to_pos and (e > to_window or e < to_sink)
                    const int to_pos = pos - t0, to_window = p.window > 0 ? pos - p.window - t0 : -1, to_sink = p.n_sink - t0;
                    const bool whole_view = !have || (to_pos >= KT - 1 && (to_window < 0 || to_sink >= KT));
                    // V scales in the exponent: at most 2^60 below the reference, which may move to ve_max + 2
                    const bool near = p.scale >= 0.f && __all_sync(0xffffffffu, !have || sc.lv_min - (float)max(vexp, sc.ve_max + 2) > -60.f);
                    const bool all = near && __all_sync(0xffffffffu, whole_view) && sc.plain == (1 << kGroups) - 1;
                    // which of the tokens 32c .. 32c + 31 the row sees
                    auto view = [&](int c) {
                        auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };
                        const uint32_t pages = ((sc.have >> (2 * c)) & 1 ? 0xffffu : 0u) | ((sc.have >> (2 * c + 1)) & 1 ? 0xffff0000u : 0u);
                        return pages & below(to_pos + 1 - 32 * c) & (~below(to_window + 1 - 32 * c) | below(to_sink - 32 * c));
                    };
                    // O of the tiles before this one, times the row's a
                    auto rescale = [&](float a) {
                        if (y == it.y0) return;
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
                    // ---- the V scales' reference
                    int big = kMinExp;
                    if (all) {
                        if (have) big = sc.ve_max;
                    } else if (__any_sync(0xffffffffu, sc.ve_max > vexp)) {
#pragma unroll 1
                        for (int g = 0; g < kGroups; ++g)
                            if (((sc.have >> g) & 1) && 16 * g <= to_pos && (min(16 * g + 15, to_pos) > to_window || 16 * g < to_sink))
                                big = max(big, sc.ve[g]);
                    }
                    if (__any_sync(0xffffffffu, big > vexp)) {
                        float a = 1.f;
                        if (big > vexp) {
                            big += 2;                 // room to grow
                            a = vexp == kMinExp ? 0.f : pow2(vexp - big);
                            vexp = big;
                        }
                        rescale(a);
                    }
                    if (!dead && !mbar_wait(&s_full[half], tiles & 1u)) dead = true;
                    tc_fence_after();
                    // the row's maximum moves to `top` if that is larger, with c times 16 columns of P in place
                    auto raise = [&](int c, float top) {
                        float a = 1.f;
                        if (top > m) {
                            a = m == -INFINITY ? 0.f : ex2(m - top);
                            m = top;
                        }
                        l *= a;
                        rescale(a);
                        const uint32_t a2 = pack2(a, a);
#pragma unroll 1
                        for (int i = 0; i < c; ++i) {
                            uint32_t w[16];
                            tmem_st_wait();
                            tmem_ld16(ts + 16 * i, w);
                            tmem_ld_wait(w);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&w[e]), *reinterpret_cast<const __half2 *>(&a2));
                                w[e] = *reinterpret_cast<const uint32_t *>(&h);
                            }
                            tmem_st16(ts + 16 * i, w);
                        }
                    };
                    if (all) {
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            uint32_t out[32];
                            float add;
                            for (;;) {
                                uint32_t s[2][32];
                                tmem_ld32(ts + 64 * c, s[0]);
                                tmem_ld32(ts + 64 * c + 32, s[1]);
                                tmem_ld_wait(s[0]);
                                tmem_ld_wait(s[1]);
                                const float base = m == -INFINITY ? 0.f : m;
                                float top = -INFINITY;
                                add = 0.f;
#pragma unroll
                                for (int gi = 0; gi < 4; ++gi) {
                                    const float f = sc.ks[4 * c + gi] * fac, lr = sc.lv[4 * c + gi] - (float)vexp;
                                    uint32_t *x = &s[gi >> 1][16 * (gi & 1)];
#pragma unroll
                                    for (int e = 0; e < 16; e += 2) fma2(x[e], x[e + 1], f, lr - base);
                                    float a = max3(x[0], x[1], x[2]), b = max3(x[3], x[4], x[5]);
#pragma unroll
                                    for (int e = 6; e < 14; e += 4) {
                                        a = max3(__float_as_uint(a), x[e], x[e + 1]);
                                        b = max3(__float_as_uint(b), x[e + 2], x[e + 3]);
                                    }
                                    a = max3(__float_as_uint(a), x[14], x[15]);
                                    top = fmaxf(top, fmaxf(a, b) - lr);
                                    float sx = 0.f, sy = 0.f;
#pragma unroll
                                    for (int e = 0; e < 16; e += 2) {
                                        const float wx = ex2(__uint_as_float(x[e])), wy = ex2(__uint_as_float(x[e + 1]));
                                        add2(sx, sy, wx, wy);
                                        out[8 * gi + e / 2] = pack2(wx, wy);
                                    }
                                    add = fmaf(sx + sy, ex2(-lr), add);
                                }
                                // the maximum is passed by more than its lag, or there is none yet: move it, and again
                                if (!__any_sync(0xffffffffu, top > kSlack || (m == -INFINITY && top > -INFINITY))) break;
                                raise(2 * c, top + base);
                            }
                            l += add;
                            tmem_st32(ts + 32 * c, out);      // over columns of S that have been read
                        }
                    } else {
                        // the same at an edge of some row's view, or with other scales
                        const unsigned plain = near ? (unsigned)sc.plain : 0u;
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t out[16];
                            const uint32_t bits = view(c);
                            float add;
                            for (;;) {
                                uint32_t x[32];
                                tmem_ld32(ts + 32 * c, x);
                                tmem_ld_wait(x);
                                const float base = m == -INFINITY ? 0.f : m;
                                float top = -INFINITY;
                                add = 0.f;
#pragma unroll
                                for (int gi = 0; gi < 2; ++gi) {
                                    const int g = 2 * c + gi;
                                    const bool in = (plain >> g) & 1;      // the V scale is in the exponent
                                    const float f = sc.ks[g] * fac, lr = in ? sc.lv[g] - (float)vexp : 0.f;
                                    float gm = -INFINITY, w[16], sx = 0.f, sy = 0.f;
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        const bool see = (bits >> (16 * gi + e)) & 1;
                                        const float y = see ? fmaf(__uint_as_float(x[16 * gi + e]), f, lr - base) : -INFINITY;
                                        gm = fmaxf(gm, y);
                                        w[e] = ex2(y);
                                    }
                                    top = fmaxf(top, gm - lr);
#pragma unroll
                                    for (int e = 0; e < 16; e += 2) add2(sx, sy, w[e], w[e + 1]);
                                    add = fmaf(sx + sy, ex2(-lr), add);
                                    if (!in) {
                                        const float vs = sc.vs[g];
                                        const int bu = (int)(__float_as_uint(vs) >> 23) & 255;
                                        const float ratio = bu == 0 ? 0.f : bu > 127 + kMaxExp - 4 ? __int_as_float(0x7fc00000) : vs * pow2(-vexp);
#pragma unroll
                                        for (int e = 0; e < 16; ++e) w[e] = (bits >> (16 * gi + e)) & 1 ? w[e] * ratio : 0.f;      // the ratio may be NaN
                                    }
#pragma unroll
                                    for (int e = 0; e < 8; ++e) out[8 * gi + e] = pack2(w[2 * e], w[2 * e + 1]);
                                }
                                if (!__any_sync(0xffffffffu, top > kSlack || (m == -INFINITY && top > -INFINITY))) break;
                                raise(c, top + base);
                            }
                            l += add;
                            tmem_st16(ts + 16 * c, out);
                        }
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
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(attn_tc<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    CUtensorMap km, vm;
    if (!make_map(&km, a.c.k, a.c) || !make_map(&vm, a.c.v, a.c)) return cudaErrorInvalidValue;
    return launch_with_join<T, D, RT>(attn_tc<T, D>, dev.sm_count < kTcGrid ? dev.sm_count : kTcGrid, kThreads, smem, km, vm, a, s);
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

size_t attn_tc_ws_bytes(int d) { return attn_splits_bytes() + 2 * kTcGrid * attn_part_floats(RT, d) * 4; }

cudaError_t launch_attn_tc(int dt, const AttnArgs &a, cudaStream_t s, const DeviceInfo &dev) {
    if (dt == PQ_F16) return a.c.d == 128 ? launch<__half, 128>(a, s, dev) : launch<__half, 64>(a, s, dev);
    return a.c.d == 128 ? launch<__nv_bfloat16, 128>(a, s, dev) : launch<__nv_bfloat16, 64>(a, s, dev);
}

}  // namespace pqk
