// C ABI of the paged 8-bit cache and the attention over it: argument checks,
// all on the host before any launch, kernel choice, launches.

#include <cmath>
#include <cstdint>

#include "kv_internal.h"

using namespace pqk;

namespace {

bool span_overlaps(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t pa = (uintptr_t)a, pb = (uintptr_t)b;
    return na > 0 && nb > 0 && pa < pb + (uintptr_t)nb && pb < pa + (uintptr_t)na;
}

int check_gb300(const DeviceInfo **out = nullptr) {
    const DeviceInfo *dev = device_info();
    if (!dev || dev->major != 10 || dev->minor != 3) return PQ_ERR_DEVICE;
    if (out) *out = dev;
    return PQ_OK;
}

constexpr int64_t kMost = INT64_C(1) << 40;

int elem_bytes(int dt) { return dt == PQ_F32 ? 4 : dt == PQ_F16 || dt == PQ_BF16 ? 2 : 0; }

bool head_size_ok(int d) { return d >= 16 && d <= 256 && d % 16 == 0; }

int64_t cache_bytes(const pq_kv_cache &c) { return (int64_t)c.n_pages * c.n_kv * c.page * c.d; }

// The cache and the rows' places.
int check_cache(const pq_kv_cache *c, const int *row_start, int n_rows) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->table || !c->len) return PQ_ERR_ARG;
    if (c->n_pages <= 0 || c->n_kv <= 0 || c->n_seq <= 0 || c->table_ld <= 0 || n_rows < 0) return PQ_ERR_ARG;
    if (!row_start && n_rows != c->n_seq) return PQ_ERR_ARG;
    if (!head_size_ok(c->d) || (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)) return PQ_ERR_LAYOUT;
    // positions are 32-bit on the device
    if ((int64_t)c->table_ld * c->page > (INT64_C(1) << 30)) return PQ_ERR_SIZE;
    if ((int64_t)c->n_kv * c->d > (INT64_C(1) << 24) || (int64_t)c->n_pages * c->n_kv > kMost / (c->page * c->d))
        return PQ_ERR_SIZE;
    if ((uintptr_t)c->k % 16 || (uintptr_t)c->v % 16 || (uintptr_t)c->k_scale % 4 || (uintptr_t)c->v_scale % 4 ||
        (uintptr_t)c->table % 4 || (uintptr_t)c->len % 4 || (uintptr_t)row_start % 4)
        return PQ_ERR_ALIGN;
    return PQ_OK;
}

// Rows of `width` elements, `ld` apart; without rows no address either.
int check_rows(const void *p, int64_t ld, int64_t width, int n_rows, int eb) {
    if ((!p && n_rows > 0) || ld < width) return PQ_ERR_ARG;
    if (width > (INT64_C(1) << 24) || ld > kMost / (n_rows > 0 ? n_rows : 1)) return PQ_ERR_SIZE;
    if ((uintptr_t)p % 16 || ld * eb % 16) return PQ_ERR_ALIGN;
    return PQ_OK;
}

int64_t rows_bytes(int64_t ld, int64_t width, int n_rows, int eb) {
    return n_rows > 0 ? ((int64_t)(n_rows - 1) * ld + width) * eb : 0;
}

// n_rows rows of `width` elements of `eb` bytes, `ld` apart (checked by check_rows).
struct Rows {
    const void *p;
    int64_t ld, width;
    int n_rows, eb;
    int64_t bytes() const { return rows_bytes(ld, width, n_rows, eb); }
};

// Whether two sets of rows share a byte: with one stride by the columns (row i of a against row i + k of b),
// else by the whole spans, gaps between the rows included.
bool rows_overlap(const Rows &a, const Rows &b) {
    if (a.n_rows == 0 || b.n_rows == 0) return false;
    if (a.ld * a.eb != b.ld * b.eb) return span_overlaps(a.p, a.bytes(), b.p, b.bytes());
    const int64_t ld = a.ld * a.eb, wa = a.width * a.eb, wb = b.width * b.eb;
    const int64_t delta = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p);
    // the first k with b's row ending behind the start of a's: delta + k * ld > -wb
    const int64_t from = -wb - delta;
    int64_t k = (from >= 0 ? from / ld : -((-from + ld - 1) / ld)) + 1;
    if (k < 1 - a.n_rows) k = 1 - a.n_rows;
    return k < b.n_rows && delta + k * ld < wa && delta + k * ld > -wb;
}

int64_t scale_bytes(const pq_kv_cache &c) { return 4 * (int64_t)c.n_pages * c.n_kv; }

// What every entry reads of the places: table, lengths, row_start.
bool touches_places(const void *p, int64_t bytes, const pq_kv_cache &c, const int *row_start) {
    return span_overlaps(p, bytes, c.table, 4 * (int64_t)c.n_seq * c.table_ld) ||
           span_overlaps(p, bytes, c.len, 4 * (int64_t)c.n_seq) ||
           (row_start && span_overlaps(p, bytes, row_start, 4 * ((int64_t)c.n_seq + 1)));
}

// Codes and scales, which an append writes.
bool touches_values(const void *p, int64_t bytes, const pq_kv_cache &c) {
    const int64_t cb = cache_bytes(c), sb = scale_bytes(c);
    return span_overlaps(p, bytes, c.k, cb) || span_overlaps(p, bytes, c.v, cb) ||
           span_overlaps(p, bytes, c.k_scale, sb) || span_overlaps(p, bytes, c.v_scale, sb);
}

bool touches_cache(const void *p, int64_t bytes, const pq_kv_cache &c, const int *row_start) {
    return touches_values(p, bytes, c) || touches_places(p, bytes, c, row_start);
}

// Whether the buffers that an append writes overlap each other, or the places that it reads.
bool cache_overlaps_itself(const pq_kv_cache &c, const int *row_start) {
    const void *p[4] = {c.k, c.v, c.k_scale, c.v_scale};
    const int64_t n[4] = {cache_bytes(c), cache_bytes(c), scale_bytes(c), scale_bytes(c)};
    for (int i = 0; i < 4; ++i) {
        if (touches_places(p[i], n[i], c, row_start)) return true;
        for (int j = 0; j < i; ++j)
            if (span_overlaps(p[i], n[i], p[j], n[j])) return true;
    }
    return false;
}

KvView view_of(const pq_kv_cache &c, const int *row_start, int n_rows) {
    KvView v;
    v.k = reinterpret_cast<int8_t *>(c.k);
    v.v = reinterpret_cast<int8_t *>(c.v);
    v.k_scale = c.k_scale;
    v.v_scale = c.v_scale;
    v.table = c.table;
    v.len = c.len;
    v.row_start = row_start;
    v.n_pages = c.n_pages;
    v.n_kv = c.n_kv;
    v.page = c.page;
    v.d = c.d;
    v.n_seq = c.n_seq;
    v.table_ld = c.table_ld;
    v.n_rows = n_rows;
    return v;
}

}  // namespace

extern "C" {

int pq_kv_append(const pq_kv_cache *cache, const int *row_start, int n_rows, pq_dtype dt, const void *k,
                 long long ldk, const void *v, long long ldv, const void *q, long long ldq, int n_q, void *q_out,
                 long long ldqo, const float *rope_cos, const float *rope_sin, int n_pos, int rot, int rope_mode,
                 struct CUstream_st *stream) {
    int st = check_cache(cache, row_start, n_rows);
    if (st) return st;
    const int eb = elem_bytes((int)dt);
    if (!eb) return PQ_ERR_DTYPE;
    const pq_kv_cache &c = *cache;
    const int64_t kw = (int64_t)c.n_kv * c.d;
    if ((st = check_rows(k, ldk, kw, n_rows, eb)) || (st = check_rows(v, ldv, kw, n_rows, eb))) return st;
    if (rot < 0 || rot > c.d || rot % 16) return PQ_ERR_LAYOUT;
    if (rope_mode != PQ_ROPE_HALF && rope_mode != PQ_ROPE_PAIR) return PQ_ERR_ARG;
    if (rot > 0) {
        if (!rope_cos || !rope_sin || n_pos <= 0) return PQ_ERR_ARG;
        if ((uintptr_t)rope_cos % 16 || (uintptr_t)rope_sin % 16) return PQ_ERR_ALIGN;
    }
    if (cache_overlaps_itself(c, row_start) || touches_values(k, rows_bytes(ldk, kw, n_rows, eb), c) ||
        touches_values(v, rows_bytes(ldv, kw, n_rows, eb), c))
        return PQ_ERR_ARG;
    const int64_t rope_bytes = 4 * (int64_t)n_pos * (rot / 2);
    if (rot > 0 && (touches_values(rope_cos, rope_bytes, c) || touches_values(rope_sin, rope_bytes, c))) return PQ_ERR_ARG;
    if (!q != !q_out) return PQ_ERR_ARG;
    if (q) {
        if (n_q <= 0) return PQ_ERR_ARG;
        if (n_q % c.n_kv) return PQ_ERR_LAYOUT;
        const int64_t qw = (int64_t)n_q * c.d;
        if (n_rows * (qw / 16) > (INT64_C(1) << 30)) return PQ_ERR_SIZE;
        if ((st = check_rows(q, ldq, qw, n_rows, eb)) || (st = check_rows(q_out, ldqo, qw, n_rows, eb))) return st;
        const int64_t ob = rows_bytes(ldqo, qw, n_rows, eb);
        const bool in_place = q_out == q && ldqo == ldq;
        const Rows to{q_out, ldqo, qw, n_rows, eb};
        // q, k and v are read while q_out is written
        if ((!in_place && rows_overlap(to, {q, ldq, qw, n_rows, eb})) || rows_overlap(to, {k, ldk, kw, n_rows, eb}) ||
            rows_overlap(to, {v, ldv, kw, n_rows, eb}))
            return PQ_ERR_ARG;
        if (touches_cache(q_out, ob, c, row_start) || touches_values(q, rows_bytes(ldq, qw, n_rows, eb), c)) return PQ_ERR_ARG;
        if (rot > 0 && (span_overlaps(q_out, ob, rope_cos, rope_bytes) || span_overlaps(q_out, ob, rope_sin, rope_bytes)))
            return PQ_ERR_ARG;
    }
    if ((st = check_gb300())) return st;
    if (n_rows == 0) return PQ_OK;
    KvAppendArgs a;
    a.c = view_of(c, row_start, n_rows);
    a.k = k;
    a.v = v;
    a.q = q;
    a.q_out = q_out;
    a.ldk = ldk;
    a.ldv = ldv;
    a.ldq = ldq;
    a.ldqo = ldqo;
    a.cos = rope_cos;
    a.sin = rope_sin;
    a.n_q = q ? n_q : 0;
    a.n_pos = n_pos;
    a.rot = rot;
    a.pair = rope_mode == PQ_ROPE_PAIR;
    a.units = FastDiv(c.d / 16);
    a.per_row = FastDiv(q ? n_q * (c.d / 16) : 1);
    return launch_kv_append((int)dt, a, stream) == cudaSuccess ? PQ_OK : PQ_ERR_LAUNCH;
}

int pq_kv_gather(const pq_kv_cache *cache, const int *row_start, int n_rows, pq_dtype dt, void *k_out, long long ldk,
                 void *v_out, long long ldv, struct CUstream_st *stream) {
    int st = check_cache(cache, row_start, n_rows);
    if (st) return st;
    const int eb = elem_bytes((int)dt);
    if (!eb) return PQ_ERR_DTYPE;
    const pq_kv_cache &c = *cache;
    const int64_t w = (int64_t)c.n_kv * c.d;
    if ((st = check_rows(k_out, ldk, w, n_rows, eb)) || (st = check_rows(v_out, ldv, w, n_rows, eb))) return st;
    if (touches_cache(k_out, rows_bytes(ldk, w, n_rows, eb), c, row_start) ||
        touches_cache(v_out, rows_bytes(ldv, w, n_rows, eb), c, row_start) ||
        rows_overlap({k_out, ldk, w, n_rows, eb}, {v_out, ldv, w, n_rows, eb}))
        return PQ_ERR_ARG;
    if ((st = check_gb300())) return st;
    if (n_rows == 0) return PQ_OK;
    return launch_kv_gather((int)dt, view_of(c, row_start, n_rows), k_out, ldk, v_out, ldv, stream) == cudaSuccess
               ? PQ_OK
               : PQ_ERR_LAUNCH;
}

size_t pq_attn_ws_bytes(int n_q, int n_kv, int d) {
    if (n_q <= 0 || n_kv <= 0 || n_q % n_kv || !head_size_ok(d)) return 0;
    if (d != 64 && d != 128) return 16;
    const size_t a = attn_mma_ws_bytes(d), b = attn_tc_ws_bytes(d);
    return a > b ? a : b;
}

int pq_attn(const pq_kv_cache *cache, const int *row_start, int n_rows, pq_dtype dt, const void *q, long long ldq,
            int n_q, float scale, int window, int n_sink, void *out, long long ldo, void *ws, size_t ws_bytes,
            struct CUstream_st *stream) {
    int st = check_cache(cache, row_start, n_rows);
    if (st) return st;
    const int eb = elem_bytes((int)dt);
    if (!eb) return PQ_ERR_DTYPE;
    const pq_kv_cache &c = *cache;
    if (n_q <= 0 || window < 0 || n_sink < 0 || !std::isfinite(scale) || !ws) return PQ_ERR_ARG;
    if (n_q % c.n_kv) return PQ_ERR_LAYOUT;
    const int64_t w = (int64_t)n_q * c.d;
    if ((int64_t)n_rows * n_q > (INT64_C(1) << 30)) return PQ_ERR_SIZE;
    if ((st = check_rows(q, ldq, w, n_rows, eb)) || (st = check_rows(out, ldo, w, n_rows, eb))) return st;
    if ((uintptr_t)ws % 16) return PQ_ERR_ALIGN;
    if (ws_bytes < pq_attn_ws_bytes(n_q, c.n_kv, c.d)) return PQ_ERR_WS;
    const int64_t ob = rows_bytes(ldo, w, n_rows, eb), qb = rows_bytes(ldq, w, n_rows, eb);
    if (rows_overlap({out, ldo, w, n_rows, eb}, {q, ldq, w, n_rows, eb}) || touches_cache(out, ob, c, row_start) || span_overlaps(ws, (int64_t)ws_bytes, out, ob) ||
        span_overlaps(ws, (int64_t)ws_bytes, q, qb) || touches_cache(ws, (int64_t)ws_bytes, c, row_start))
        return PQ_ERR_ARG;
    const DeviceInfo *dev = nullptr;
    if ((st = check_gb300(&dev))) return st;
    if (n_rows == 0) return PQ_OK;
    AttnArgs a;
    a.c = view_of(c, row_start, n_rows);
    a.group = FastDiv(n_q / c.n_kv);
    a.q = q;
    a.out = out;
    a.ldq = ldq;
    a.ldo = ldo;
    a.scale = scale;
    a.n_q = n_q;
    // positions stay below 2^30 (check_cache), so larger values change nothing
    a.window = window < (1 << 30) ? window : 1 << 30;
    a.n_sink = n_sink < (1 << 30) ? n_sink : 1 << 30;
    a.ws = static_cast<uint8_t *>(ws);
    const int group = a.group.d;
    const int rows = row_start ? (int)(((int64_t)n_rows + c.n_seq - 1) / c.n_seq) * group : group;
    cudaError_t e;
    // 16-bit rows: the wide kernel (256 rows at a time) from more than 32 rows per sequence and kv head. 16 sequences
    // of 2048 tokens, bf16, head size 128: 16 rows 30.1 us (narrow) against 41.9 (wide), 32 rows 43.3 against 42.4, 64 rows
    // 69.7 against 43.9; head size 64: 28 rows 13.7 against 18.1, 56 rows 18.8 against 18.3. f32 rows keep the pair of fp16
    // for q and for the weights that only the narrow one has.
    if (c.d != 64 && c.d != 128) e = launch_attn_generic((int)dt, a, stream);
    else if (dt != PQ_F32 && rows > 32) e = launch_attn_tc((int)dt, a, stream, *dev);
    else e = launch_attn_mma((int)dt, a, rows, stream, *dev);
    return e == cudaSuccess ? PQ_OK : PQ_ERR_LAUNCH;
}

}  // extern "C"
