// Attention over the paged 8-bit cache on CUDA cores, any head size.
//
// One block per (row, query head); its warps take 32 tokens at a time in turn:
// lane t forms the score of token t (q in shared memory, f32), the warp keeps
// the running maximum m and the sum l of exp2(s - m) of a softmax, and every
// lane the weighted sum of its own elements of v; the warps' parts are joined
// in order at the end.  For head sizes that the tensor-core kernels do not
// take (80, 96, 256): bound by its arithmetic, one conversion and one
// multiply-add per code on every query head.  With a warp per (row, query head) and
// the tokens of V one after the other, 16 sequences of 2048 tokens (20 query heads over
// 4 of 80 elements) took 589 us, as it stands 85; 256 rows of one sequence took 1162 us and take 729.

#include "kv_device.cuh"

namespace pqk {
namespace {

constexpr int kWarps = 8, kMaxD = 256, kStride = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;

template <class T> __global__ void __launch_bounds__(32 * kWarps) attn_generic(AttnArgs p) {
    __shared__ float qs[kMaxD], part[kWarps][kMaxD], part_m[kWarps], part_l[kWarps];
    __shared__ int sh;
    const KvView &c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.x / p.n_q, h = blockIdx.x - r * p.n_q;
    const int s = find_seq(c, r, &sh);
    int pos = -1;
    if (s >= 0) {
        int r0, n;
        seq_rows(c, s, r0, n);
        pos = seq_len(c, s) - n + (r - r0);
    }
    const T *q = static_cast<const T *>(p.q) + (long long)r * p.ldq + h * c.d;
    for (int i = threadIdx.x; i < c.d; i += kStride) qs[i] = to_f32(q[i]) * (p.scale * kLog2e);
    __syncthreads();
    const int kvh = h / (p.n_q / c.n_kv);
    const int units = c.d / 16;
    float m = -INFINITY, l = 0.f, acc[kMaxD / 32];
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i) acc[i] = 0.f;
    const int end = (int)min((long long)pos + 1, (long long)c.table_ld * c.page);
    const int from = p.window > 0 ? max(0, pos - p.window + 1) : 0;      // first token of the window
    for (int t0 = 32 * warp; t0 < end; t0 += kStride) {
        if (t0 >= p.n_sink && t0 + 32 <= from) {                          // nothing visible: on to the window
            t0 += (from / 32 * 32 - t0 + kStride - 1) / kStride * kStride - kStride;
            continue;
        }
        const int t = t0 + lane;
        const int pg = t < end ? page_of(c, s, t / c.page) : -1;
        const bool see = pg >= 0 && (t >= from || t < p.n_sink);
        float x = -INFINITY, vs = 0.f;
        long long vrow = 0;
        if (see) {
            const size_t at = page_base(c, pg, kvh) + (size_t)(t % c.page) * c.d;
            const uint4 *kr = reinterpret_cast<const uint4 *>(c.k + at);
            float dot = 0.f;
#pragma unroll 4
            for (int u = 0; u < units; ++u) {
                const uint4 w = kr[u];
                const uint32_t b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    dot = fmaf(qs[16 * u + e], (float)(int8_t)(b[e >> 2] >> (8 * (e & 3))), dot);
            }
            const long long si = (long long)pg * c.n_kv + kvh;
            x = dot * c.k_scale[si];
            vs = c.v_scale[si];
            vrow = (long long)at;
        }
        const unsigned any = __ballot_sync(0xffffffffu, see);
        if (!any) continue;
        float top = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float mn = fmaxf(m, top);
        const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn);
        const float w = see ? exp2f(x - mn) : 0.f;
        l = l * alpha + w;
        const float wv = see ? w * vs : 0.f;
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i) acc[i] *= alpha;
        // tokens out of view count for nothing, whatever row they read
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
            const float wk = __shfl_sync(0xffffffffu, wv, k);
            const int8_t *vr = c.v + __shfl_sync(0xffffffffu, vrow, k);
#pragma unroll
            for (int i = 0; i < kMaxD / 32; ++i)
                if (32 * i + lane < c.d) acc[i] = fmaf(wk, (float)vr[32 * i + lane], acc[i]);
        }
        m = mn;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i)
        if (32 * i + lane < c.d) part[warp][32 * i + lane] = acc[i];
    if (lane == 0) {
        part_m[warp] = m;
        part_l[warp] = l;
    }
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w]);
    T *o = static_cast<T *>(p.out) + (long long)r * p.ldo + h * c.d;
    for (int i = threadIdx.x; i < c.d; i += kStride) {      // once: head sizes are at most the block's threads
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = part_m[w] == -INFINITY ? 1.f : exp2f(part_m[w] - top);      // nothing, or NaN, in the first case
            sum += part_l[w] * f;
            x += part[w][i] * f;
        }
        const float inv = sum != 0.f ? 1.f / sum : 0.f;      // no visible token: zeros
        from_f32(o[i], x * inv);
    }
}

}  // namespace

cudaError_t launch_attn_generic(int dt, const AttnArgs &a, cudaStream_t s) {
    const long long grid = (long long)a.c.n_rows * a.n_q;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    if (dt == PQ_F32) attn_generic<float><<<(unsigned)grid, 32 * kWarps, 0, s>>>(a);
    else if (dt == PQ_F16) attn_generic<__half><<<(unsigned)grid, 32 * kWarps, 0, s>>>(a);
    else attn_generic<__nv_bfloat16><<<(unsigned)grid, 32 * kWarps, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace pqk
