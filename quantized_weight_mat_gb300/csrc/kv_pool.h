// Internal interface of the page pool: validated arguments of its kernels, and their launchers.
#pragma once

#include "kv_internal.h"

namespace pqk {

struct PoolView {
    int *refs, *table, *len;
    int n_pages, shift, n_seq, table_ld;      // pages of 1 << shift tokens
};

// One layer's codes and scales.
struct PoolLayer {
    int8_t *k, *v;
    float *k_scale, *v_scale;
    int n_kv, d;
};

// Workspace of a call that plans moves: their count, the moves (page, new page, tokens), three lists of a number per
// page. Of a fork: a pair and a length per sequence, then the rows that the sequences get.
struct PoolWs {
    int *head;
    int4 *moves;
    int *list[3];
    int2 *pair;
    int *rows;
};
constexpr int kPoolMaxSeq = 65536;
inline size_t pool_ws_bytes(const PoolView &p) {
    const size_t plan = 64 + (16 + 3 * 4) * (size_t)p.n_pages, fork = (size_t)p.n_seq * (8 + 4 * (size_t)p.table_ld);
    return ((plan > fork ? plan : fork) + 15) / 16 * 16;
}
inline PoolWs pool_ws(const PoolView &p, void *ws) {
    PoolWs w;
    char *at = static_cast<char *>(ws);
    w.head = reinterpret_cast<int *>(at);
    w.moves = reinterpret_cast<int4 *>(at + 64);
    for (int i = 0; i < 3; ++i) w.list[i] = reinterpret_cast<int *>(w.moves + p.n_pages) + (size_t)i * p.n_pages;
    w.pair = reinterpret_cast<int2 *>(at);
    w.rows = reinterpret_cast<int *>(w.pair + p.n_seq);
    return w;
}

cudaError_t launch_kv_fork(const PoolView &p, int n, const int *from, const int *to, const int *tokens, const PoolWs &w,
                           cudaStream_t s);
cudaError_t launch_kv_free(const PoolView &p, int n, const int *seq, const int *begin, const int *end, cudaStream_t s);
cudaError_t launch_kv_reserve(const PoolView &p, const PoolLayer *layers, int n_layers, const int *n_new, int *status,
                              const PoolWs &w, cudaStream_t s, const DeviceInfo &dev);
cudaError_t launch_kv_compact(const PoolView &p, const PoolLayer *layers, int n_layers, int *moved, int *n_used,
                              const PoolWs &w, cudaStream_t s, const DeviceInfo &dev);

}  // namespace pqk
