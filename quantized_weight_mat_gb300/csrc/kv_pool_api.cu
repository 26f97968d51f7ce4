// C ABI of the page pool: argument checks, all on the host before any launch.

#include <algorithm>
#include <cstdint>

#include "kv_checks.h"
#include "kv_pool.h"

using namespace pqk;

namespace {

struct Span {
    const void *p;
    int64_t n;
};

constexpr int kMaxLayers = 1024;

int check_pool(const pq_kv_pool *p) {
    if (!p || !p->refs || !p->table || !p->len) return PQ_ERR_ARG;
    if (p->n_pages <= 0 || p->n_seq <= 0 || p->table_ld <= 0) return PQ_ERR_ARG;
    if (!page_ok(p->page)) return PQ_ERR_LAYOUT;
    // positions are 32-bit on the device
    if ((int64_t)p->table_ld * p->page > (INT64_C(1) << 30) || p->n_seq > kPoolMaxSeq || p->n_pages > (1 << 28) ||
        (int64_t)p->n_seq * p->table_ld > (INT64_C(1) << 28))
        return PQ_ERR_SIZE;
    if ((uintptr_t)p->refs % 16 || (uintptr_t)p->table % 4 || (uintptr_t)p->len % 4) return PQ_ERR_ALIGN;
    return PQ_OK;
}

PoolView view_of(const pq_kv_pool &p) {
    PoolView v;
    v.refs = p.refs;
    v.table = p.table;
    v.len = p.len;
    v.n_pages = p.n_pages;
    v.shift = 0;
    while (1 << v.shift < p.page) ++v.shift;
    v.n_seq = p.n_seq;
    v.table_ld = p.table_ld;
    return v;
}

// What a call writes, then what it only reads; null ones are left out.
struct Buffers {
    Span of[12];
    int n = 0, written = 0;
    void writes(const void *p, int64_t bytes) {
        reads(p, bytes);
        written = n;
    }
    void reads(const void *p, int64_t bytes) {
        if (p && bytes > 0) of[n++] = {p, bytes};
    }
    bool clash() const {
        for (int i = 0; i < written; ++i)
            for (int j = i + 1; j < n; ++j)
                if (span_overlaps(of[i].p, of[i].n, of[j].p, of[j].n)) return true;
        return false;
    }
    bool touches(const void *p, int64_t bytes) const {
        for (int i = 0; i < n; ++i)
            if (span_overlaps(of[i].p, of[i].n, p, bytes)) return true;
        return false;
    }
};

Buffers pool_buffers(const pq_kv_pool &p) {
    Buffers b;
    b.writes(p.refs, 4 * (int64_t)p.n_pages);
    b.writes(p.table, 4 * (int64_t)p.n_seq * p.table_ld);
    b.writes(p.len, 4 * (int64_t)p.n_seq);
    return b;
}

int check_list(const int *list, bool needed) {
    if (!list && needed) return PQ_ERR_ARG;
    return (uintptr_t)list % 4 ? PQ_ERR_ALIGN : PQ_OK;
}

int check_ws(const pq_kv_pool &p, const void *ws, size_t ws_bytes) {
    if (!ws) return PQ_ERR_ARG;
    if ((uintptr_t)ws % 16) return PQ_ERR_ALIGN;
    return ws_bytes < pool_ws_bytes(view_of(p)) ? PQ_ERR_WS : PQ_OK;
}

// The caches of all layers, against the pool, the call's other buffers and each other.
int check_layers(const pq_kv_pool &p, const pq_kv_cache *caches, int n, const Buffers &others, PoolLayer *out) {
    if (n < 0 || (n > 0 && !caches)) return PQ_ERR_ARG;
    if (n > kMaxLayers) return PQ_ERR_SIZE;
    Span all[4 * kMaxLayers];
    for (int i = 0; i < n; ++i) {
        const pq_kv_cache &c = caches[i];
        const int st = check_values(c);
        if (st) return st;
        if (c.n_pages != p.n_pages || c.page != p.page) return PQ_ERR_ARG;
        const Span own[4] = {{c.k, cache_bytes(c)}, {c.v, cache_bytes(c)}, {c.k_scale, scale_bytes(c)}, {c.v_scale, scale_bytes(c)}};
        for (int j = 0; j < 4; ++j) {
            if (others.touches(own[j].p, own[j].n)) return PQ_ERR_ARG;
            all[j * n + i] = own[j];      // a layer's buffers of one kind mostly lie one behind the other
        }
        out[i] = {reinterpret_cast<int8_t *>(c.k), reinterpret_cast<int8_t *>(c.v), c.k_scale, c.v_scale, c.n_kv, c.d};
    }
    const auto below = [](const Span &a, const Span &b) { return (uintptr_t)a.p < (uintptr_t)b.p; };
    for (int j = 0; j < 4; ++j)
        if (!std::is_sorted(all + j * n, all + (j + 1) * n, below)) std::sort(all + j * n, all + (j + 1) * n, below);
    // the four sorted runs, always the lowest next
    int at[4] = {0, 0, 0, 0};
    uintptr_t end = 0;
    for (int k = 0; k < 4 * n; ++k) {
        int low = -1;
        for (int j = 0; j < 4; ++j)
            if (at[j] < n && (low < 0 || below(all[j * n + at[j]], all[low * n + at[low]]))) low = j;
        const Span &x = all[low * n + at[low]++];
        if ((uintptr_t)x.p < end) return PQ_ERR_ARG;
        end = (uintptr_t)x.p + (uintptr_t)x.n;
    }
    return PQ_OK;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? PQ_OK : PQ_ERR_LAUNCH; }

}  // namespace

extern "C" {

size_t pq_kv_pool_ws_bytes(const pq_kv_pool *pool) { return check_pool(pool) ? 0 : pool_ws_bytes(view_of(*pool)); }

int pq_kv_fork(const pq_kv_pool *pool, int n, const int *from, const int *to, const int *tokens, void *ws, size_t ws_bytes,
               struct CUstream_st *stream) {
    int st = check_pool(pool);
    if (st) return st;
    if (n < 0) return PQ_ERR_ARG;
    if (n > pool->n_seq) return PQ_ERR_SIZE;
    if ((st = check_list(from, n > 0)) || (st = check_list(to, n > 0)) || (st = check_list(tokens, false)) ||
        (st = check_ws(*pool, ws, ws_bytes)))
        return st;
    Buffers b = pool_buffers(*pool);
    b.writes(ws, (int64_t)ws_bytes);
    b.reads(from, 4 * (int64_t)n);
    b.reads(to, 4 * (int64_t)n);
    b.reads(tokens, 4 * (int64_t)n);
    if (b.clash()) return PQ_ERR_ARG;
    if ((st = check_gb300())) return st;
    if (n == 0) return PQ_OK;
    const PoolView p = view_of(*pool);
    return status_of(launch_kv_fork(p, n, from, to, tokens, pool_ws(p, ws), stream));
}

int pq_kv_reserve(const pq_kv_pool *pool, const pq_kv_cache *caches, int n_caches, const int *n_new, int *status, void *ws,
                  size_t ws_bytes, struct CUstream_st *stream) {
    int st = check_pool(pool);
    if (st) return st;
    if ((st = check_list(n_new, true)) || (st = check_list(status, true)) || (st = check_ws(*pool, ws, ws_bytes))) return st;
    Buffers b = pool_buffers(*pool);
    b.writes(ws, (int64_t)ws_bytes);
    b.writes(status, 8);
    b.reads(n_new, 4 * (int64_t)pool->n_seq);
    if (b.clash()) return PQ_ERR_ARG;
    PoolLayer layers[kMaxLayers];
    if ((st = check_layers(*pool, caches, n_caches, b, layers))) return st;
    const DeviceInfo *dev = nullptr;
    if ((st = check_gb300(&dev))) return st;
    const PoolView p = view_of(*pool);
    return status_of(launch_kv_reserve(p, layers, n_caches, n_new, status, pool_ws(p, ws), stream, *dev));
}

int pq_kv_free(const pq_kv_pool *pool, int n, const int *seq, const int *begin, const int *end, struct CUstream_st *stream) {
    int st = check_pool(pool);
    if (st) return st;
    if (n < 0) return PQ_ERR_ARG;
    if (n > pool->n_seq) return PQ_ERR_SIZE;
    if ((st = check_list(seq, false)) || (st = check_list(begin, false)) || (st = check_list(end, false))) return st;
    Buffers b = pool_buffers(*pool);
    b.reads(seq, 4 * (int64_t)n);
    b.reads(begin, 4 * (int64_t)n);
    b.reads(end, 4 * (int64_t)n);
    if (b.clash()) return PQ_ERR_ARG;
    if ((st = check_gb300())) return st;
    if (n == 0) return PQ_OK;
    return status_of(launch_kv_free(view_of(*pool), n, seq, begin, end, stream));
}

int pq_kv_compact(const pq_kv_pool *pool, const pq_kv_cache *caches, int n_caches, int *moved, int *n_used, void *ws,
                  size_t ws_bytes, struct CUstream_st *stream) {
    int st = check_pool(pool);
    if (st) return st;
    if ((st = check_list(moved, false)) || (st = check_list(n_used, true)) || (st = check_ws(*pool, ws, ws_bytes))) return st;
    Buffers b = pool_buffers(*pool);
    b.writes(ws, (int64_t)ws_bytes);
    b.writes(moved, 4 * (int64_t)pool->n_pages);
    b.writes(n_used, 4);
    if (b.clash()) return PQ_ERR_ARG;
    PoolLayer layers[kMaxLayers];
    if ((st = check_layers(*pool, caches, n_caches, b, layers))) return st;
    const DeviceInfo *dev = nullptr;
    if ((st = check_gb300(&dev))) return st;
    const PoolView p = view_of(*pool);
    return status_of(launch_kv_compact(p, layers, n_caches, moved, n_used, pool_ws(p, ws), stream, *dev));
}

}  // extern "C"
