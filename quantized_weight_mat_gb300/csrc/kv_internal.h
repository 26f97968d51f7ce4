// Internal interface of the paged 8-bit cache: validated arguments of the
// append, gather and attention kernels, and their launchers.
#pragma once

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

struct KvAppendArgs {
    KvView c;
    const void *k, *v, *q;
    void *q_out;
    long long ldk, ldv, ldq, ldqo;
    const float *cos, *sin;
    int n_q, n_pos, rot, pair;   // pair: rotate (2i, 2i+1) instead of (i, i + rot/2)
};

struct AttnArgs {
    KvView c;
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
size_t attn_mma_ws_bytes(int d);
unsigned attn_mma_wait_timeouts(bool reset);
// Any head size, CUDA cores.
cudaError_t launch_attn_generic(int dt, const AttnArgs &a, cudaStream_t s);

}  // namespace pqk
