// Shared by the attention kernels that bring tiles of K and V by TMA.
#pragma once

#include <climits>
#include <cuda.h>

#include "attn_sched.cuh"
#include "pq_device.cuh"
#include "pq_ptx.cuh"

namespace pqk {
namespace {

// Of pq_attn_mod: first tokens and prefixes (with the others too), capped, biased scores; kExact: caps that 16-bit rows need
// relative errors for, biased or not.
enum : int { kViews = 1, kCap = 2, kBias = 4, kExact = 8 | kViews | kCap | kBias };
constexpr int KT = 128;                      // tokens per tile
constexpr int kGroups = KT / 16;             // groups of 16 tokens: always within one page
constexpr int kMinExp = -200, kMaxExp = 125;   // of V scales: one that takes no part, and the largest
constexpr int kLeastExp = -118;              // of a row's reference for V scales: 2^-(kLeastExp - 7) is a normal number, the smallest scale 2^-8 of it
constexpr int kFarExp = 400;                 // differences of exponents beyond which nothing is left
constexpr float kNever = 1e30f;              // a maximum that no score passes
constexpr float kSlack = 8.f;                // the running maximum may lag by this many powers of two

struct TileMeta {
    float ks[kGroups], vs[kGroups];      // scales of the tile's groups of 16 tokens
    int have[kGroups];                   // whether the group has a page
};

// 2^e, 0 below the smallest normal number, 2^127 above it.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(min(max(e, -127), 127) + 127) << 23); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// (sx, sy) += (x, y), each rounded to nearest.
__device__ __forceinline__ void add2(float &sx, float &sy, float x, float y) {
    asm("{\n .reg .b64 p, q;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n add.rn.f32x2 p, p, q;\n mov.b64 {%0, %1}, p;\n}"
        : "+f"(sx), "+f"(sy)
        : "f"(x), "f"(y));
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

__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
template <class T> __device__ __forceinline__ void store4(T *p, float4 v) {
    T e[4];
    from_f32(e[0], v.x);
    from_f32(e[1], v.y);
    from_f32(e[2], v.z);
    from_f32(e[3], v.w);
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(e);
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
    const cuuint32_t box[3] = {(cuuint32_t)c.d, (cuuint32_t)c.page, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t *>(codes), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, c.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Joins the parts of the item that CTA blockIdx.x of an attention kernel began,
// up to 32 rows a block: a line of threads per row, 4 elements a thread, the
// parts in CTA order.
template <class T, int D, int RT> __global__ void __launch_bounds__(256) attn_join(AttnArgs p) {
    constexpr int COLS = D / 4, LINES = 256 / COLS, BLOCK = RT < 32 ? RT : 32;
    constexpr int ROWS = BLOCK > LINES ? BLOCK / LINES : 1, AHEAD = ROWS > 2 ? 4 : 8;
    constexpr size_t PF = attn_part_floats(RT, D);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int c0 = blockIdx.x;
    const Split it = splits_of(p)[c0];
    const int col = threadIdx.x % COLS, line = threadIdx.x / COLS, row0 = BLOCK * blockIdx.y + line;
    if (it.c1 < 0 || line >= BLOCK || row0 >= it.rows) return;
    const float *parts = parts_of(p);
    float m[ROWS], sum[ROWS];
    float4 acc[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        m[r] = -INFINITY;
        sum[r] = 0.f;
        acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int c = c0; c <= it.c1; c += AHEAD) {
        float2 ml[AHEAD][ROWS];
        float4 v[AHEAD][ROWS];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int row = row0 + r * LINES;
                ml[i][r] = make_float2(-INFINITY, 0.f);
                if (c + i > it.c1 || row >= it.rows) continue;
                // the first CTA's part is the item its range ends in, the others' the one theirs starts in
                const float *pp = parts + (size_t)(2 * (c + i) + (c + i == c0 ? 1 : 0)) * PF;
                ml[i][r] = __ldcg(reinterpret_cast<const float2 *>(pp + (size_t)RT * D) + row);
                v[i][r] = __ldcg(reinterpret_cast<const float4 *>(pp + (size_t)row * D) + col);
            }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const float mn = fmaxf(m[r], ml[i][r].x);
                if (ml[i][r].x == -INFINITY) {
                    sum[r] += ml[i][r].y;      // nothing, or NaN
                    continue;
                }
                const float a = m[r] == -INFINITY ? 0.f : ex2(m[r] - mn), b = ex2(ml[i][r].x - mn);
                m[r] = mn;
                sum[r] = sum[r] * a + ml[i][r].y * b;
                acc[r].x = acc[r].x * a + v[i][r].x * b;
                acc[r].y = acc[r].y * a + v[i][r].y * b;
                acc[r].z = acc[r].z * a + v[i][r].z * b;
                acc[r].w = acc[r].w * a + v[i][r].w * b;
            }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int row = row0 + r * LINES;
        if (row >= it.rows) break;
        const float inv = sum[r] != 0.f ? 1.f / sum[r] : 0.f;
        const int tk = p.group.div(it.j * RT + row), hd = it.h * p.group.d + it.j * RT + row - tk * p.group.d;
        store4(static_cast<T *>(p.out) + (it.r0 + tk) * p.ldo + (long long)hd * D + 4 * col,
               make_float4(acc[r].x * inv, acc[r].y * inv, acc[r].z * inv, acc[r].w * inv));
    }
}

// What the rows of each row tile see at most, the first token of any and the end of any's prefix, and the places of a kv head
// of each sequence (pq_attn_mod calls of several rows per sequence: else every CTA would look them up for all row tiles
// before its first unit). A warp per row tile; sequences in blockIdx.x, every kBoundsSplit * kBoundsWarps row tiles in blockIdx.y.
constexpr int kBoundsWarps = 8;
template <int RT, int COST> __global__ void __launch_bounds__(32 * kBoundsWarps) attn_bounds(AttnArgs p) {
    __shared__ long long sums[kBoundsWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, s = blockIdx.x;
    int r0, m;
    seq_rows(p.c, s, r0, m);
    const int len = seq_len(p.c, s), rows = m * p.group.d;
    long long places = 0;
    for (int j = blockIdx.y * kBoundsWarps + warp; j * RT < rows; j += kBoundsSplit * kBoundsWarps) {
        const int end = p.group.div(min((j + 1) * RT, rows) - 1);
        int first = INT_MAX, prefix = 0;
        for (int tok = p.group.div(j * RT) + lane; tok <= end; tok += 32)
            if (len - m + tok >= 0) {
                const RowView v = row_view(p, r0 + tok, len);
                first = min(first, v.first);
                prefix = max(prefix, v.prefix);
            }
        first = __reduce_min_sync(0xffffffffu, first);
        prefix = __reduce_max_sync(0xffffffffu, prefix);
        if (lane == 0) {
            p.mod.bounds[bounds_at<RT>(p, s, r0, j)] = make_int2(first, prefix);
            places += row_tile<RT, KT, true>(p, s, r0, m, len, j).units + COST;
        }
    }
    if (lane == 0) sums[warp] = places;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kBoundsWarps; ++i) places += sums[i];
        p.mod.places[(size_t)s * kBoundsSplit + blockIdx.y] = places;
    }
}
template <int RT, int COST> cudaError_t launch_bounds(const AttnArgs &a, cudaStream_t s) {
    if (!a.c.row_start || !(a.mod.first || a.mod.prefix)) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.c.n_seq, kBoundsSplit);
    cfg.blockDim = dim3(32 * kBoundsWarps);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_bounds<RT, COST>, a);
}

// Launches an attention kernel and the join of its parts, each so that it may be
// scheduled while the kernel before it finishes.
template <class T, int D, int RT, class K>
cudaError_t launch_with_join(K kernel, int grid, int threads, int smem, const CUtensorMap &km, const CUtensorMap &vm,
                             AttnArgs a, cudaStream_t s) {
    a.grid = FastDiv(grid);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, km, vm, a);
    if (e != cudaSuccess) return e;
    cfg.gridDim.y = RT > 32 ? RT / 32 : 1;
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attn_join<T, D, RT>, a);
}

}  // namespace
}  // namespace pqk
