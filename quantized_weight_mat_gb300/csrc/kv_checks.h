// Argument checks shared by the entries of the paged cache and of its pool.
#pragma once

#include <cstdint>

#include "kv_internal.h"

namespace pqk {

inline bool span_overlaps(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t pa = (uintptr_t)a, pb = (uintptr_t)b;
    return na > 0 && nb > 0 && pa < pb + (uintptr_t)nb && pb < pa + (uintptr_t)na;
}

inline int check_gb300(const DeviceInfo **out = nullptr) {
    const DeviceInfo *dev = device_info();
    if (!dev || dev->major != 10 || dev->minor != 3) return PQ_ERR_DEVICE;
    if (out) *out = dev;
    return PQ_OK;
}

constexpr int64_t kMost = INT64_C(1) << 40;

inline bool head_size_ok(int d) { return d >= 16 && d <= 256 && d % 16 == 0; }
inline bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

inline int64_t cache_bytes(const pq_kv_cache &c) { return (int64_t)c.n_pages * c.n_kv * c.page * c.d; }
inline int64_t scale_bytes(const pq_kv_cache &c) { return 4 * (int64_t)c.n_pages * c.n_kv; }

// The codes and scales of a cache.
inline int check_values(const pq_kv_cache &c) {
    if (!c.k || !c.v || !c.k_scale || !c.v_scale || c.n_pages <= 0 || c.n_kv <= 0) return PQ_ERR_ARG;
    if (!head_size_ok(c.d) || !page_ok(c.page)) return PQ_ERR_LAYOUT;
    if ((int64_t)c.n_kv * c.d > (INT64_C(1) << 24) || (int64_t)c.n_pages * c.n_kv > kMost / (c.page * c.d)) return PQ_ERR_SIZE;
    if ((uintptr_t)c.k % 16 || (uintptr_t)c.v % 16 || (uintptr_t)c.k_scale % 4 || (uintptr_t)c.v_scale % 4) return PQ_ERR_ALIGN;
    return PQ_OK;
}

}  // namespace pqk
