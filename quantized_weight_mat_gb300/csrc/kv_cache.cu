// Writing and reading the paged 8-bit cache (grouped-query attention's keys
// and values: PESTI README, "Conformance").

#include "kv_device.cuh"

namespace pqk {
namespace {

constexpr int kGatherRows = 2;      // of a block (8192 rows of 8 heads of 128: one 13.0 us, two 12.0; 7 ragged prompts, 2 of 64: 4.8 and 3.2)

// What the preceding kernels on the stream wrote is complete after this; the
// next kernel may then be scheduled beside this one.
__device__ __forceinline__ void after_predecessors() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
}

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

// The angles of unit u at a position.
struct Angle {
    float c[8], s[8];
};
__device__ __forceinline__ void load_angle(Angle &g, int u, const KvAppendArgs &p, int pos) {
    if (pos < p.n_pos) {
        const size_t o = (size_t)max(pos, 0) * (p.rot / 2) + 8 * u;
        load8(p.cos + o, g.c);
        load8(p.sin + o, g.s);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) g.c[i] = g.s[i] = __int_as_float(0x7fc00000);
    }
}
// Rotates a unit.  Every product, difference and sum is rounded to f32 by
// itself, so that the result does not depend on how a compiler contracts them.
__device__ __forceinline__ void turn(const Angle &g, const KvAppendArgs &p, float (&a)[8], float (&b)[8]) {
    const float(&c)[8] = g.c, (&s)[8] = g.s;
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
template <class T>
__device__ __forceinline__ void load_unit(const T *head, const Unit &t, int u, const KvAppendArgs &p, int pos,
                                          float (&a)[8], float (&b)[8]) {
    load8_once(head + t.ia, a);
    load8_once(head + t.ib, b);
    if (!t.turned) return;
    Angle g;
    load_angle(g, u, p, pos);
    turn(g, p, a, b);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t unit_max(const float (&a)[8], const float (&b)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, max(abs_bits(a[i]), abs_bits(b[i])));
    return m;
}
// rint(x * inv) of eight values, |x * inv| < 127.5: adding 1.5 * 2^23 leaves the
// integer in the low bits (the conversion instruction has a quarter of the rate).
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(__fadd_rn(__fmul_rn(x[i], inv), 12582912.f));
    return make_uint2(__byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040), 0x5410));
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

constexpr int kQueryRows = 4;      // of a block, prompts

// Block b of the query rows.  One row per sequence: 64 units of one warp,
// through all rows; prompts: four rows, whose sequences and positions are looked
// up together while the first units are on their way.
template <bool SINGLE, class T>
__device__ __forceinline__ void rotate_queries(const KvAppendArgs &p, int b, int *place, const T *q, T *o) {
    constexpr int NT = SINGLE ? 32 : 128, AHEAD = SINGLE ? 2 : 1;
    const KvView &c = p.c;
    const int units = c.d / 16, per = p.n_q * units, tid = threadIdx.x;
    const int row0 = SINGLE ? 0 : b * kQueryRows;
    const int from = SINGLE ? b * 64 : 0, to = SINGLE ? min(from + 64, c.n_rows * per) : min(kQueryRows, c.n_rows - row0) * per;
    Angle g;
    int have_u = -1, have_pos = 0;
    for (int i0 = from; i0 < to; i0 += AHEAD * NT) {
        float x[AHEAD][8], y[AHEAD][8];
        int row[AHEAD], u[AHEAD];
        long long at[AHEAD];
        Unit t[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int i = i0 + k * NT + tid;
            row[k] = i < to ? p.per_row.div(i) : -1;
            const int j = i - row[k] * per, h = p.units.div(j);
            u[k] = j - h * units;
            t[k] = unit_of(u[k], p.rot, p.pair);
            at[k] = (long long)h * c.d;
            if (row[k] < 0) continue;
            const T *src = q + (row0 + row[k]) * p.ldq + at[k];
            load8_once(src + t[k].ia, x[k]);
            load8_once(src + t[k].ib, y[k]);
        }
        if (!SINGLE && i0 == 0) {
            if (tid < kQueryRows) place[tid] = 0;
            __syncthreads();
            for (int s = tid; s < c.n_seq; s += NT) {
                int r0, n;
                seq_rows(c, s, r0, n);
                if (r0 + n <= row0 || r0 >= row0 + kQueryRows) continue;
                const int first = seq_len(c, s) - n - r0;      // position of row r: first + r
                for (int r = max(r0, row0); r < min(r0 + n, row0 + kQueryRows); ++r) place[r - row0] = first + r;
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (row[k] < 0) continue;
            if (t[k].turned) {
                const int pos = SINGLE ? seq_len(c, row[k]) - 1 : place[row[k]];
                if (u[k] != have_u || pos != have_pos) load_angle(g, u[k], p, pos);      // mostly the same for another head
                have_u = u[k];
                have_pos = pos;
                turn(g, p, x[k], y[k]);
            }
            T *dst = o + (row0 + row[k]) * p.ldqo + at[k];
            store8(dst + t[k].ia, x[k]);
            store8(dst + t[k].ib, y[k]);
        }
    }
}

// Grid: first the (block item, kv head, K or V) triples, an item being one page
// that a sequence's rows reach, then the blocks of the query rows.  A block sees every new token of its page and head, so the page's
// scale needs no other block.  The values are read and rotated once: between the
// maximum and the codes they wait in registers (SINGLE: one row per sequence,
// one unit a thread, one warp a block) or as f32 in shared memory.
// 8192 new tokens of 8 kv heads of 128 with the 32 query heads' rotation take
// 49.2 us (bf16; 20.4 without q), where the bytes alone need 27: a block's phases
// (load, maximum, codes) hide each other's latency only across the 6 blocks of an SM.
// Single tokens are bound by the chain of dependent loads (length, page, scale):
// 2.5 us for one sequence, 3.8 for 128.
template <class T, bool SINGLE>
__global__ void __launch_bounds__(SINGLE ? 32 : 128) kv_append(KvAppendArgs p, int items) {
    constexpr int NT = SINGLE ? 32 : 128;
    extern __shared__ float4 held[];              // unit i's k-th float4 at k * page * units + i
    __shared__ int sh[4];
    __shared__ uint32_t shmax[NT / 32];
    after_predecessors();
    const KvView &c = p.c;
    const int units = c.d / 16;
    if ((int)blockIdx.x >= 2 * items * c.n_kv) {
        rotate_queries<SINGLE>(p, blockIdx.x - 2 * items * c.n_kv, sh, static_cast<const T *>(p.q), static_cast<T *>(p.q_out));
        return;
    }

    // which sequence and which of its pages this item is
    const int side = blockIdx.x & 1, pair = blockIdx.x >> 1, item = pair / c.n_kv, head = pair - item * c.n_kv;      // side 1: V
    int s = -1, j = 0;
    if (SINGLE || !c.row_start) {
        s = item;
    } else {
        // running count of the pages that the sequences' rows reach
        __shared__ int warp_sum[NT / 32];
        if (threadIdx.x == 0) sh[0] = -1;
        int before = 0;
        for (int s0 = 0; s0 < c.n_seq; s0 += NT) {
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
            for (int w = 0; w < NT / 32; ++w) {
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
    const int lo = max(max(start, 0), block * c.page), hi = min(len, (block + 1) * c.page);   // positions written here
    const int keep = lo - block * c.page;                                                      // older tokens of the page

    const T *src = static_cast<const T *>(side ? p.v : p.k);
    const long long ld = side ? p.ldv : p.ldk;
    const int rot = side ? 0 : p.rot, tid = threadIdx.x;
    const int count = (hi - lo) * units, cap = c.page * units;
    const T *rows = src + (long long)(r0 + lo - start) * ld + head * c.d;
    float a[8], b[8];
    uint32_t m = 0;
    if constexpr (SINGLE) {
        if (tid < count) {
            load_unit(rows, unit_of(tid, rot, p.pair), tid, p, lo, a, b);
            m = unit_max(a, b);
        }
    } else {
#pragma unroll 2
        for (int i = tid; i < count; i += NT) {
            const int row = p.units.div(i), u = i - row * units;
            load_unit(rows + row * ld, unit_of(u, rot, p.pair), u, p, lo + row, a, b);
            m = max(m, unit_max(a, b));
            held[i] = make_float4(a[0], a[1], a[2], a[3]);
            held[cap + i] = make_float4(a[4], a[5], a[6], a[7]);
            held[2 * cap + i] = make_float4(b[0], b[1], b[2], b[3]);
            held[3 * cap + i] = make_float4(b[4], b[5], b[6], b[7]);
        }
    }
    if (pg < 0) return;      // looked at only here: the rows' loads need not wait for the table's
    int8_t *dst = (side ? c.v : c.k) + page_base(c, pg, head);
    float *scale = (side ? c.v_scale : c.k_scale) + (long long)pg * c.n_kv + head;
    const float old = keep > 0 ? *scale : 0.f;
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (!SINGLE) {
        if ((tid & 31) == 0) shmax[tid >> 5] = m;
        __syncthreads();      // every thread has read the old scale by now
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) m = max(m, shmax[w]);
    }
    float now = __fdiv_rn(__uint_as_float(m), 127.f);
    if (now < 1.17549435e-38f) now = 0.f;
    if (m >= 0x7f800000u || !(old == old)) now = __int_as_float(0x7fc00000);
    else if (old > now) now = old;
    const float inv = now > 0.f ? __fdiv_rn(1.f, now) : 0.f;
    if (tid == 0) *scale = now;
    if (keep > 0 && now > old) {
        const float ratio = __fdiv_rn(old, now);
        uint4 *w = reinterpret_cast<uint4 *>(dst);
#pragma unroll 4
        for (int i = tid; i < keep * units; i += NT) {
            uint4 x = w[i];
            x.x = requant4(x.x, ratio);
            x.y = requant4(x.y, ratio);
            x.z = requant4(x.z, ratio);
            x.w = requant4(x.w, ratio);
            w[i] = x;
        }
    }
    const bool zero = !(now > 0.f);      // nothing but zeros, or a page that reads as NaN
    for (int i = tid; i < count; i += NT) {
        if constexpr (!SINGLE) {
            const float4 f[4] = {held[i], held[cap + i], held[2 * cap + i], held[3 * cap + i]};      // this thread's own
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float4 x = f[e >> 2], y = f[2 + (e >> 2)];
                a[e] = (e & 3) == 0 ? x.x : (e & 3) == 1 ? x.y : (e & 3) == 2 ? x.z : x.w;
                b[e] = (e & 3) == 0 ? y.x : (e & 3) == 1 ? y.y : (e & 3) == 2 ? y.z : y.w;
            }
        }
        const int row = p.units.div(i), u = i - row * units;
        const Unit t = unit_of(u, rot, p.pair);
        int8_t *y = dst + (keep + row) * c.d;
        *reinterpret_cast<uint2 *>(y + t.ia) = zero ? make_uint2(0u, 0u) : codes8(a, inv);
        *reinterpret_cast<uint2 *>(y + t.ib) = zero ? make_uint2(0u, 0u) : codes8(b, inv);
    }
}

// A block takes two rows, a thread 16 codes at a time: the rows' places are
// looked up together, so that the chain of dependent loads (sequence, page,
// codes) is paid once for both.
template <class T>
__global__ void __launch_bounds__(128) kv_gather(KvView c, T *k_out, long long ldk, T *v_out, long long ldv) {
    __shared__ int seq[kGatherRows], page[kGatherRows], slot[kGatherRows];
    after_predecessors();
    const int tid = threadIdx.x;
    const int first = blockIdx.x * kGatherRows;
    if (tid < kGatherRows) seq[tid] = c.row_start ? -1 : first + tid;
    __syncthreads();
    if (c.row_start) {
        for (int s = tid; s < c.n_seq; s += blockDim.x) {
            int r0, n;
            seq_rows(c, s, r0, n);
            for (int r = max(r0, first); r < min(r0 + n, first + kGatherRows); ++r) seq[r - first] = s;
        }
        __syncthreads();
    }
    const int rows = min(kGatherRows, c.n_rows - first);
    if (tid < rows) {
        const int s = seq[tid];
        int pg = -1, at = 0;
        if (s >= 0) {
            int r0, n;
            seq_rows(c, s, r0, n);
            const int pos = seq_len(c, s) - n + (first + tid - r0);
            if (pos >= 0) {
                pg = page_of(c, s, pos / c.page);
                at = pos % c.page;
            }
        }
        page[tid] = pg;
        slot[tid] = at;
    }
    __syncthreads();
    const int units = c.d / 16, per = c.n_kv * units;
    for (int i = tid; i < 2 * per; i += blockDim.x) {
        const int side = i >= per, j = i - (side ? per : 0), h = j / units, u = j - h * units;
        const float *scale = (side ? c.v_scale : c.k_scale) + h;
        const int8_t *codes = (side ? c.v : c.k) + page_base(c, 0, h) + 16 * u;
        T *out = (side ? v_out + (long long)first * ldv : k_out + (long long)first * ldk) + h * c.d + 16 * u;
        const long long ld = side ? ldv : ldk;
        uint4 w[kGatherRows];
        float sc[kGatherRows];
#pragma unroll
        for (int r = 0; r < kGatherRows; ++r) {
            const int pg = r < rows ? page[r] : -1;
            w[r] = make_uint4(0u, 0u, 0u, 0u);
            sc[r] = 0.f;
            if (pg >= 0) {
                w[r] = *reinterpret_cast<const uint4 *>(codes + page_base(c, pg, 0) + slot[r] * c.d);
                sc[r] = scale[(long long)pg * c.n_kv];
            }
        }
#pragma unroll
        for (int r = 0; r < kGatherRows; ++r) {
            if (r >= rows) break;
            const uint32_t x[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
            float a[8], b[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                a[e] = sc[r] * (float)(int8_t)(x[e >> 2] >> (8 * (e & 3)));
                b[e] = sc[r] * (float)(int8_t)(x[2 + (e >> 2)] >> (8 * (e & 3)));
            }
            store8(out + r * ld, a);
            store8(out + r * ld + 8, b);
        }
    }
}

// Launched so that it may be scheduled while the kernel before it finishes.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, int threads, int smem, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace

template <class T> static cudaError_t append_t(const KvAppendArgs &a, cudaStream_t s) {
    // pages that the rows can reach: one per sequence, and for several rows
    // one more wherever a page boundary can lie
    const long long items = a.c.row_start
                                ? (long long)a.c.n_rows / a.c.page + 2ll * (a.c.n_seq < a.c.n_rows ? a.c.n_seq : a.c.n_rows)
                                : a.c.n_seq;
    const long long per = (long long)a.n_q * a.c.d / 16;
    const long long blocks = 2 * items * a.c.n_kv;
    const long long q_grid = !a.q ? 0 : a.c.row_start ? (a.c.n_rows + kQueryRows - 1) / kQueryRows : (a.c.n_rows * per + 63) / 64;
    if (blocks + q_grid > 0x7fffffffll || a.c.n_rows * per > 0x40000000ll) return cudaErrorInvalidValue;
    if (!a.c.row_start) return launch_after(kv_append<T, true>, (unsigned)(blocks + q_grid), 32, 0, s, a, (int)items);
    static PerDeviceOnce once;
    const cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(kv_append<T, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 256 * 4);
    });
    if (e != cudaSuccess) return e;
    return launch_after(kv_append<T, false>, (unsigned)(blocks + q_grid), 128, a.c.page * a.c.d * 4, s, a, (int)items);
}

cudaError_t launch_kv_append(int dt, const KvAppendArgs &a, cudaStream_t s) {
    return dt == PQ_F32 ? append_t<float>(a, s) : dt == PQ_F16 ? append_t<__half>(a, s) : append_t<__nv_bfloat16>(a, s);
}

cudaError_t launch_kv_gather(int dt, const KvView &c, void *k_out, long long ldk, void *v_out, long long ldv,
                             cudaStream_t s) {
    const unsigned grid = (unsigned)((c.n_rows + kGatherRows - 1) / kGatherRows);
    if (dt == PQ_F32)
        return launch_after(kv_gather<float>, grid, 128, 0, s, c, static_cast<float *>(k_out), ldk, static_cast<float *>(v_out), ldv);
    if (dt == PQ_F16)
        return launch_after(kv_gather<__half>, grid, 128, 0, s, c, static_cast<__half *>(k_out), ldk, static_cast<__half *>(v_out), ldv);
    return launch_after(kv_gather<__nv_bfloat16>, grid, 128, 0, s, c, static_cast<__nv_bfloat16 *>(k_out), ldk,
                        static_cast<__nv_bfloat16 *>(v_out), ldv);
}

}  // namespace pqk
