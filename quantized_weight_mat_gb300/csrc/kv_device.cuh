// Device helpers shared by the paged-cache kernels: element types, row
// places, page lookup.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_internal.h"

namespace pqk {

// 8 consecutive elements (16-byte aligned) as f32, and back (rounded to nearest).
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __half *p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
// The same of values that are read once: they do not displace others in the L1 cache.
__device__ __forceinline__ void load8_once(const float *p, float (&x)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <class T> __device__ __forceinline__ void load8_once(const T *p, float (&x)[8]) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
    load8(reinterpret_cast<const T *>(&u), x);
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__half *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float &y, float x) { y = x; }
__device__ __forceinline__ void from_f32(__half &y, float x) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_f32(__nv_bfloat16 &y, float x) { y = __float2bfloat16_rn(x); }

// The rows of sequence s: first row and count, kept inside [0, n_rows].
__device__ __forceinline__ void seq_rows(const KvView &c, int s, int &r0, int &n) {
    if (!c.row_start) {
        r0 = s;
        n = 1;
        return;
    }
    const int a = c.row_start[s], b = c.row_start[s + 1];
    r0 = min(max(a, 0), c.n_rows);
    n = max(min(b, c.n_rows) - r0, 0);
}

// Tokens of sequence s that can lie in pages of its table.
__device__ __forceinline__ int seq_len(const KvView &c, int s) { return max(c.len[s], 0); }

// Page of block j of sequence s, or -1.
__device__ __forceinline__ int page_of(const KvView &c, int s, int j) {
    if (j < 0 || j >= c.table_ld) return -1;
    const int p = c.table[(long long)s * c.table_ld + j];
    return (unsigned)p < (unsigned)c.n_pages ? p : -1;
}

// Sequence of row r, by the whole block (`found` is shared memory): -1 when no
// sequence has it.  Ends with a barrier.
__device__ __forceinline__ int find_seq(const KvView &c, int r, int *found) {
    if (!c.row_start) return r;
    if (threadIdx.x == 0) *found = -1;
    __syncthreads();
    for (int s = threadIdx.x; s < c.n_seq; s += blockDim.x) {
        int r0, n;
        seq_rows(c, s, r0, n);
        if (r >= r0 && r < r0 + n) *found = s;
    }
    __syncthreads();
    return *found;
}

// First element of page p, kv head h.
__device__ __forceinline__ size_t page_base(const KvView &c, int p, int h) {
    return ((size_t)p * c.n_kv + h) * (size_t)c.page * (size_t)c.d;
}

}  // namespace pqk
