// Writing and reading the paged 8-bit cache (grouped-query attention's keys
// and values: PESTI README, "Conformance").

#include "kv_device.cuh"

namespace pqk {
namespace {

constexpr int kAppendThreads = 128;

// A unit is 16 elements of one head in two groups of 8 (offsets ia and ib):
// below rot/16 the two groups of a rotation, after that a plain copy.
struct Unit {
    int ia, ib;
    bool turned;
};
__device__ __forceinline__ Unit unit_of(int u, int rot, int pair) {
    Unit t;
    t.turned = u < rot / 16;
    if (t.turned && !pair) {
        t.ia = 8 * u;
        t.ib = rot / 2 + 8 * u;
    } else {
        t.ia = 16 * u;
        t.ib = 16 * u + 8;
    }
    return t;
}

// Loads and rotates unit u of a head.  Every product, difference and sum is
// rounded to f32 by itself, so that the result does not depend on how a
// compiler contracts them.
template <class T>
__device__ __forceinline__ void load_unit(const T *head, const Unit &t, int u, const KvAppendArgs &p, int pos,
                                          float (&a)[8], float (&b)[8]) {
    load8(head + t.ia, a);
    load8(head + t.ib, b);
    if (!t.turned) return;
    float c[8], s[8];
    if (pos < p.n_pos) {
        const size_t o = (size_t)max(pos, 0) * (p.rot / 2) + 8 * u;
        load8(p.cos + o, c);
        load8(p.sin + o, s);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = s[i] = __int_as_float(0x7fc00000);
    }
    if (!p.pair) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i];
            a[i] = __fsub_rn(__fmul_rn(x, c[i]), __fmul_rn(y, s[i]));
            b[i] = __fadd_rn(__fmul_rn(x, s[i]), __fmul_rn(y, c[i]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
            a[2 * i] = __fsub_rn(__fmul_rn(x, c[i]), __fmul_rn(y, s[i]));
            a[2 * i + 1] = __fadd_rn(__fmul_rn(x, s[i]), __fmul_rn(y, c[i]));
            b[2 * i] = __fsub_rn(__fmul_rn(z, c[4 + i]), __fmul_rn(w, s[4 + i]));
            b[2 * i + 1] = __fadd_rn(__fmul_rn(z, s[4 + i]), __fmul_rn(w, c[4 + i]));
        }
    }
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t unit_max(const float (&a)[8], const float (&b)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, max(abs_bits(a[i]), abs_bits(b[i])));
    return m;
}
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int q = min(127, max(-127, __float2int_rn(x[i] * inv)));
        w[i >> 2] |= (uint32_t)(q & 255) << (8 * (i & 3));
    }
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ uint32_t requant4(uint32_t w, float ratio) {
    uint32_t y = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int q = __float2int_rn((float)(int8_t)(w >> (8 * i)) * ratio);
        y |= (uint32_t)(q & 255) << (8 * i);
    }
    return y;
}

// Grid: first the (block item, kv head) pairs, an item being one page that a
// sequence's rows reach, then one block per row of q.  In a block the first
// half of the threads handles K, the second half V; one block sees every new
// token of its page and head, so the page's scale needs no other block.
template <class T>
__global__ void __launch_bounds__(kAppendThreads) kv_append(KvAppendArgs p, int items) {
    constexpr int HALF = kAppendThreads / 2;
    __shared__ int sh[4];
    __shared__ uint32_t shmax[kAppendThreads / 32];
    const KvView &c = p.c;
    const int units = c.d / 16;
    if ((int)blockIdx.x >= items * c.n_kv) {
        const int r = blockIdx.x - items * c.n_kv;
        const int s = find_seq(c, r, sh);
        int pos = 0;
        if (s >= 0) {
            int r0, n;
            seq_rows(c, s, r0, n);
            pos = seq_len(c, s) - n + (r - r0);
        }
        const T *q = static_cast<const T *>(p.q) + (long long)r * p.ldq;
        T *o = static_cast<T *>(p.q_out) + (long long)r * p.ldqo;
        for (int i = threadIdx.x; i < p.n_q * units; i += kAppendThreads) {
            const int h = i / units, u = i % units;
            const Unit t = unit_of(u, p.rot, p.pair);
            float a[8], b[8];
            load_unit(q + h * c.d, t, u, p, pos, a, b);
            store8(o + h * c.d + t.ia, a);
            store8(o + h * c.d + t.ib, b);
        }
        return;
    }

    // which sequence and which of its pages this item is
    const int item = blockIdx.x / c.n_kv, head = blockIdx.x % c.n_kv;
    int s = -1, j = 0;
    if (!c.row_start) {
        s = item;
    } else {
        // running count of the pages that the sequences' rows reach
        __shared__ int warp_sum[kAppendThreads / 32];
        if (threadIdx.x == 0) sh[0] = -1;
        int before = 0;
        for (int s0 = 0; s0 < c.n_seq; s0 += kAppendThreads) {
            const int t = s0 + threadIdx.x;
            int cnt = 0;
            if (t < c.n_seq) {
                int r0, n;
                seq_rows(c, t, r0, n);
                const int len = seq_len(c, t), first = max(len - n, 0);
                if (n > 0 && len > 0) cnt = (len - 1) / c.page - first / c.page + 1;
            }
            int incl = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl, o);
                if ((threadIdx.x & 31) >= o) incl += up;
            }
            if ((threadIdx.x & 31) == 31) warp_sum[threadIdx.x >> 5] = incl;
            __syncthreads();
            int add = before;
            for (int w = 0; w < kAppendThreads / 32; ++w) {
                if (w < (int)(threadIdx.x >> 5)) add += warp_sum[w];
                before += warp_sum[w];
            }
            incl += add;
            if (item >= incl - cnt && item < incl) {
                sh[0] = t;
                sh[1] = item - (incl - cnt);
            }
            __syncthreads();
            if (before > item) break;
        }
        s = sh[0];
        j = sh[1];
    }
    if (s < 0) return;
    int r0, n;
    seq_rows(c, s, r0, n);
    const int len = seq_len(c, s), start = len - n;
    if (n == 0 || len == 0) return;
    const int block = max(start, 0) / c.page + j;
    const int pg = page_of(c, s, block);
    if (pg < 0) return;
    const int lo = max(max(start, 0), block * c.page), hi = min(len, (block + 1) * c.page);   // positions written here
    const int keep = lo - block * c.page;                                                      // older tokens of the page

    const int side = threadIdx.x / HALF, ht = threadIdx.x % HALF;
    const T *src = static_cast<const T *>(side ? p.v : p.k);
    const long long ld = side ? p.ldv : p.ldk;
    int8_t *dst = (side ? c.v : c.k) + page_base(c, pg, head);
    float *scale = (side ? c.v_scale : c.k_scale) + (long long)pg * c.n_kv + head;
    const int rot = side ? 0 : p.rot;
    const int count = (hi - lo) * units;
    uint32_t m = 0;
    for (int i = ht; i < count; i += HALF) {
        const int pos = lo + i / units, u = i % units;
        const T *x = src + (long long)(r0 + pos - start) * ld + head * c.d;
        const Unit t = unit_of(u, rot, p.pair);
        float a[8], b[8];
        load_unit(x, t, u, p, pos, a, b);
        m = max(m, unit_max(a, b));
    }
    const float old = keep > 0 ? *scale : 0.f;
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) shmax[threadIdx.x >> 5] = m;
    __syncthreads();      // every thread has read the old scale by now
#pragma unroll
    for (int w = 0; w < HALF / 32; ++w) m = max(m, shmax[side * (HALF / 32) + w]);
    float now = __fdiv_rn(__uint_as_float(m), 127.f);
    if (now < 1.17549435e-38f) now = 0.f;
    if (m >= 0x7f800000u || !(old == old)) now = __int_as_float(0x7fc00000);
    else if (old > now) now = old;
    const float inv = now > 0.f ? __fdiv_rn(1.f, now) : 0.f;
    if (ht == 0) *scale = now;
    if (keep > 0 && now > old) {
        const float ratio = __fdiv_rn(old, now);
        uint4 *w = reinterpret_cast<uint4 *>(dst);
        for (int i = ht; i < keep * units; i += HALF) {
            uint4 x = w[i];
            x.x = requant4(x.x, ratio);
            x.y = requant4(x.y, ratio);
            x.z = requant4(x.z, ratio);
            x.w = requant4(x.w, ratio);
            w[i] = x;
        }
    }
    for (int i = ht; i < count; i += HALF) {
        const int pos = lo + i / units, u = i % units;
        const T *x = src + (long long)(r0 + pos - start) * ld + head * c.d;
        const Unit t = unit_of(u, rot, p.pair);
        float a[8], b[8];
        load_unit(x, t, u, p, pos, a, b);
        int8_t *y = dst + (pos - block * c.page) * c.d;
        *reinterpret_cast<uint2 *>(y + t.ia) = codes8(a, inv);
        *reinterpret_cast<uint2 *>(y + t.ib) = codes8(b, inv);
    }
}

// One block per row; a thread takes 16 codes at a time.
template <class T>
__global__ void __launch_bounds__(128) kv_gather(KvView c, T *k_out, long long ldk, T *v_out, long long ldv) {
    __shared__ int sh;
    const int r = blockIdx.x;
    const int s = find_seq(c, r, &sh);
    int pg = -1, slot = 0;
    if (s >= 0) {
        int r0, n;
        seq_rows(c, s, r0, n);
        const int pos = seq_len(c, s) - n + (r - r0);
        if (pos >= 0) {
            pg = page_of(c, s, pos / c.page);
            slot = pos % c.page;
        }
    }
    const int units = c.d / 16, per = c.n_kv * units;
    for (int i = threadIdx.x; i < 2 * per; i += blockDim.x) {
        const int side = i / per, h = i % per / units, u = i % units;
        float a[8], b[8];
        if (pg >= 0) {
            const float sc = (side ? c.v_scale : c.k_scale)[(long long)pg * c.n_kv + h];
            const int8_t *src = (side ? c.v : c.k) + page_base(c, pg, h) + slot * c.d + 16 * u;
            const uint4 w = *reinterpret_cast<const uint4 *>(src);
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                a[e] = sc * (float)(int8_t)(x[e >> 2] >> (8 * (e & 3)));
                b[e] = sc * (float)(int8_t)(x[2 + (e >> 2)] >> (8 * (e & 3)));
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = b[e] = 0.f;
        }
        T *o = (side ? v_out + (long long)r * ldv : k_out + (long long)r * ldk) + h * c.d + 16 * u;
        store8(o, a);
        store8(o + 8, b);
    }
}

}  // namespace

template <class T> static cudaError_t append_t(const KvAppendArgs &a, cudaStream_t s) {
    // pages that the rows can reach: one per sequence, and for several rows
    // one more wherever a page boundary can lie
    const long long items = a.c.row_start
                                ? (long long)a.c.n_rows / a.c.page + 2ll * (a.c.n_seq < a.c.n_rows ? a.c.n_seq : a.c.n_rows)
                                : a.c.n_seq;
    const long long grid = items * a.c.n_kv + (a.q ? a.c.n_rows : 0);
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    kv_append<T><<<(unsigned)grid, kAppendThreads, 0, s>>>(a, (int)items);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(int dt, const KvAppendArgs &a, cudaStream_t s) {
    return dt == PQ_F32 ? append_t<float>(a, s) : dt == PQ_F16 ? append_t<__half>(a, s) : append_t<__nv_bfloat16>(a, s);
}

cudaError_t launch_kv_gather(int dt, const KvView &c, void *k_out, long long ldk, void *v_out, long long ldv,
                             cudaStream_t s) {
    const unsigned grid = (unsigned)c.n_rows;
    if (dt == PQ_F32)
        kv_gather<float><<<grid, 128, 0, s>>>(c, static_cast<float *>(k_out), ldk, static_cast<float *>(v_out), ldv);
    else if (dt == PQ_F16)
        kv_gather<__half><<<grid, 128, 0, s>>>(c, static_cast<__half *>(k_out), ldk, static_cast<__half *>(v_out), ldv);
    else
        kv_gather<__nv_bfloat16><<<grid, 128, 0, s>>>(c, static_cast<__nv_bfloat16 *>(k_out), ldk,
                                                      static_cast<__nv_bfloat16 *>(v_out), ldv);
    return cudaGetLastError();
}

}  // namespace pqk
