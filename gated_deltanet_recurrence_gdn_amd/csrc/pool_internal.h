// pool_internal.h -- what the row-pool calls share: the host checks of pools and
// the kernels' check of a caller's pair of rows.
#pragma once

#include "gdn_internal.h"

namespace gdn {

// Whether pair i may be copied: rows in range, and its destination neither
// another pair's destination nor, within one pool, another pair's source.  The
// whole workgroup, of THREADS threads, asks together.
template <int THREADS, typename Args>
__device__ bool pair_stands(const Args& a, int i, int s, int d) {
    bool bad = s < -1 || s >= a.src_slots || d >= a.dst_slots || d < -1;
    if (!bad && d >= 0)
        for (int j = threadIdx.x; j < a.n; j += THREADS)
            if (j != i && (a.dst_row[j] == d || (a.same && a.src_row[j] == d))) bad = true;
    return __syncthreads_or(bad) == 0;
}

// One past the last byte of a pool.
inline const unsigned char* pool_end(const gdn_pool& p) {
    return static_cast<const unsigned char*>(p.data) + (int64_t)(p.n_layers - 1) * p.layer_bytes + (int64_t)p.n_slots * p.row_bytes;
}

// Whether two pools share a byte.  A layer's rows are one range, and a pool's layers
// may lie between another's: for each layer of the pool with fewer of them, only the
// other's last layer that starts before its end can reach into it.
inline bool overlap(const gdn_pool& x, const gdn_pool& y) {
    if (x.n_layers == 0 || y.n_layers == 0 || x.data >= pool_end(y) || y.data >= pool_end(x)) return false;
    const gdn_pool &a = x.n_layers <= y.n_layers ? x : y, &b = x.n_layers <= y.n_layers ? y : x;
    const int64_t size = a.n_slots * a.row_bytes, b_size = b.n_slots * b.row_bytes;
    // a's layer from b's first byte
    int64_t at = static_cast<const unsigned char*>(a.data) - static_cast<const unsigned char*>(b.data);
    for (int32_t l = 0; l < a.n_layers; ++l, at += a.layer_bytes) {
        if (at + size <= 0) continue;
        int64_t m = b.n_layers > 1 ? (at + size - 1) / b.layer_bytes : 0;
        if (m >= b.n_layers) m = b.n_layers - 1;
        if (m * b.layer_bytes + b_size > at) return true;
    }
    return false;
}

inline int check_pools(const gdn_pool* pools, int32_t n_pools) {
    if (n_pools < 1 || n_pools > GDN_MAX_POOLS) return GDN_ERR_SHAPE;
    if (pools == nullptr) return GDN_ERR_NULL;
    for (int i = 0; i < n_pools; ++i) {
        const gdn_pool& p = pools[i];
        if (p.n_layers < 0 || p.n_slots < 1 || p.n_slots != pools[0].n_slots) return GDN_ERR_SHAPE;
        if (p.row_bytes < 16 || p.row_bytes % 16 != 0 || p.row_bytes > (int64_t{1} << 40)) return GDN_ERR_SHAPE;
        if (p.layer_bytes % 16 != 0 || p.layer_bytes > (int64_t{1} << 46)) return GDN_ERR_SHAPE;
        if (p.n_layers > 1 && p.layer_bytes / p.row_bytes < p.n_slots) return GDN_ERR_SHAPE;
        // more than any memory: the sums below stay inside 64 bits
        if ((double)p.n_layers * (double)p.layer_bytes + (double)p.n_slots * (double)p.row_bytes > 0x1p60) return GDN_ERR_SHAPE;
        if (p.n_layers == 0) continue;
        if (p.data == nullptr) return GDN_ERR_NULL;
        if (!aligned(p.data, 16)) return GDN_ERR_ALIGN;
    }
    return GDN_OK;
}

}  // namespace gdn
