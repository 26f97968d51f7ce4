// Internal interface of the paged 8-bit cache: validated arguments of the
// append, gather and attention kernels, and their launchers.
#pragma once

#include <vector_types.h>

#include "pq_internal.h"

namespace pqk {

// Where a call's rows lie in the sequences (see pq.h, "Rows").
struct KvView {
    int8_t *k, *v;
    float *k_scale, *v_scale;
    const int *table;
    const int *len;
    const int *row_start;      // null: one row per sequence
    int n_pages, n_kv, page, d, n_seq, table_ld;
    int n_rows;
};

// Quotients by a divisor known on the host, exact for 0 <= n < 2^31:
// n / d = (mulhi(n, magic) + n) >> shift with shift = ceil(log2 d) and magic =
// floor(2^32 (2^shift - d) / d) + 1 (Granlund and Montgomery, 1994).
struct FastDiv {
    unsigned magic, shift;
    int d;
    explicit FastDiv(int divisor = 1) : shift(0), d(divisor) {
        while ((1u << shift) < (unsigned)d) ++shift;
        magic = (unsigned)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int div(int n) const { return (int)((__umulhi((unsigned)n, magic) + (unsigned)n) >> shift); }
#endif
};

struct KvAppendArgs {
    KvView c;
    const void *k, *v, *q;
    void *q_out;
    long long ldk, ldv, ldq, ldqo;
    const float *cos, *sin;
    int n_q, n_pos, rot, pair;   // pair: rotate (2i, 2i+1) instead of (i, i + rot/2)
    FastDiv units, per_row;      // d / 16, and n_q times that
};

constexpr int kBoundsSplit = 8;
// What pq_attn_mod does to scores and views; all empty in pq_attn.
struct AttnMod {
    float to_unit, top;        // a score times log2 e -> the cap's unit, and the cap times log2 e; 0: no cap
    bool large;                // a cap of which 16-bit rows would see 2^-20
    float near[5];             // of the polynomial that stands for the cap's curve up to 0.8 caps (large: 0.6), times `top`
    const float *slope;        // [n_q] or null
    const int *first, *prefix; // [n_rows] or null
    // of sequences of several rows, what attn_bounds leaves behind the workspace of pq_attn: their row tiles' bounds, and the
    // places of one kv head (see attn_sched.cuh) in kBoundsSplit parts
    int2 *bounds;
    long long *places;
    bool any() const { return top > 0.f || slope || first || prefix; }
};

struct AttnArgs {
    KvView c;
    AttnMod mod;
    FastDiv group;             // query heads per kv head
    FastDiv grid;              // CTAs of the launch (set by the launcher)
    const void *q;
    void *out;
    long long ldq, ldo;
    float scale;
    int n_q, window, n_sink;
    uint8_t *ws;
};

// dt: a pq_dtype value
cudaError_t launch_kv_append(int dt, const KvAppendArgs &a, cudaStream_t s);
cudaError_t launch_kv_gather(int dt, const KvView &c, void *k_out, long long ldk, void *v_out, long long ldv,
                             cudaStream_t s);
// Attention for head sizes 64 and 128, `rows` (tokens times query heads per kv
// head) of a typical sequence deciding between row tiles of 8 and 16 rows.
cudaError_t launch_attn_mma(int dt, const AttnArgs &a, int rows, cudaStream_t s, const DeviceInfo &dev);
cudaError_t launch_attn_mma_mod(int dt, const AttnArgs &a, int rows, cudaStream_t s, const DeviceInfo &dev);      // no cap
cudaError_t launch_attn_mma_cap(int dt, const AttnArgs &a, int rows, cudaStream_t s, const DeviceInfo &dev);
size_t attn_mma_ws_bytes(int d);
unsigned attn_mma_wait_timeouts(bool reset);
unsigned attn_mma_mod_wait_timeouts(bool reset);
unsigned attn_mma_cap_wait_timeouts(bool reset);
// The same for prompts: 16-bit rows, tensor-core products of 128 rows.
cudaError_t launch_attn_tc(int dt, const AttnArgs &a, cudaStream_t s, const DeviceInfo &dev);
cudaError_t launch_attn_tc_mod(int dt, const AttnArgs &a, cudaStream_t s, const DeviceInfo &dev);      // no cap
cudaError_t launch_attn_tc_cap(int dt, const AttnArgs &a, cudaStream_t s, const DeviceInfo &dev);
size_t attn_tc_ws_bytes(int d);
unsigned attn_tc_wait_timeouts(bool reset);
unsigned attn_tc_mod_wait_timeouts(bool reset);
unsigned attn_tc_cap_wait_timeouts(bool reset);
// Any head size, CUDA cores.
cudaError_t launch_attn_generic(int dt, const AttnArgs &a, cudaStream_t s);

}  // namespace pqk
