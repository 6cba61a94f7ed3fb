// pool.hip -- rows of the state pool: copies, forks, release and compaction (gfx950).
//
// Page "LightSeek's TokenSpeed Hits 580 Tokens per Second on Qwen3.5's 400B
// Model", section "How they actually got there": sequences own rows of a state
// pool through an index table, cached prefixes are states kept in rows, and a
// row is copied when a second sequence continues from it.  A row is one
// sequence's memory in one layer (its recurrent state, or its convolution
// history), so one row index names n_layers rows in each of several pools.
//
// A fork or a compaction is two launches.  The plan kernel, one workgroup,
// turns the index table into a bitmap of the rows in use (LDS), ranks the free
// rows, or the rows that have to move, by prefix sums over the bitmap's words,
// writes the (source, destination) pairs to the workspace and the new table.
// The copy kernel moves the rows of every pair.  Both are integer moves and
// byte copies: results do not depend on the order of anything.
//
// The copies are bound by HBM: every row is read once and written once (8 rows of
// 48 layers, 2.46 GB: 490 us, 5.0 TB/s, a plain copy's rate; one plan kernel 4 to 7
// us).  One
// workgroup moves tiles of 32 KiB, eight 16-byte loads in flight in each
// thread before the first store; a grid that walks the tiles (rather than one
// workgroup per tile) lets a compaction, whose number of moves only the device
// knows, launch without idle workgroups.
#include <cstring>

#include "gdn_device.h"
#include "pool_internal.h"

namespace gdn {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyDeep = 8;                                // 16-byte pieces per thread and tile
constexpr int kTileBytes = kCopyThreads * kCopyDeep * 16;   // 32 KiB
constexpr int kCopyGrid = 4096;                             // workgroups that walk the tiles
constexpr int kPlanThreads = 1024;
constexpr int kMaxWords = GDN_POOL_MAX_ROWS / 32;

struct PoolPart {
    const unsigned char* src;
    unsigned char* dst;
    int64_t src_layer, dst_layer, row;  // bytes
    int32_t tiles;                      // tiles of a row
    int32_t items;                      // layers * tiles
};

struct CopyRowsArgs {
    PoolPart part[GDN_MAX_POOLS];
    const int32_t* src_row;
    const int32_t* dst_row;
    const int32_t* n_dev;  // number of pairs, where only the device knows it
    int32_t* status;
    int32_t n_parts, n, per_pair;
    int32_t src_slots, dst_slots;
    int32_t check;  // 1: the pairs are the caller's and are checked here
    int32_t same;   // 1: sources and destinations are rows of the same pools
};

__global__ __launch_bounds__(kCopyThreads) void pool_copy_kernel(const CopyRowsArgs a) {
    const int n = a.n_dev != nullptr ? *a.n_dev : a.n;
    const uint32_t total = (uint32_t)n * (uint32_t)a.per_pair;
    int at = -1, s = -1, d = -1;
    bool go = false;
    for (uint32_t it = blockIdx.x; it < total; it += gridDim.x) {
        const int pair = it / (uint32_t)a.per_pair;
        int item = it % (uint32_t)a.per_pair;
        if (pair != at) {
            at = pair;
            s = a.src_row[pair];
            d = a.dst_row[pair];
            go = true;
            if (a.check) {
                go = pair_stands<kCopyThreads>(a, pair, s, d);
                if (!go && threadIdx.x == 0 && a.status != nullptr) a.status[0] = GDN_ERR_SLOT;
            }
            if (d < 0 || (a.same && s == d)) go = false;
        }
        if (!go) continue;
        int p = 0;
        while (p + 1 < a.n_parts && item >= a.part[p].items) item -= a.part[p++].items;
        const PoolPart& q = a.part[p];
        const int layer = item / q.tiles;
        const int64_t begin = (int64_t)(item % q.tiles) * kTileBytes;
        const int64_t left = q.row - begin;
        const unsigned char* src = q.src + layer * q.src_layer + (int64_t)s * q.row + begin;
        unsigned char* dst = q.dst + layer * q.dst_layer + (int64_t)d * q.row + begin;
        u32x4 v[kCopyDeep];
#pragma unroll
        for (int k = 0; k < kCopyDeep; ++k) {
            const int o = (k * kCopyThreads + (int)threadIdx.x) * 16;
            v[k] = u32x4{0, 0, 0, 0};
            if (s >= 0 && o < left) v[k] = *reinterpret_cast<const u32x4*>(src + o);
        }
#pragma unroll
        for (int k = 0; k < kCopyDeep; ++k) {
            const int o = (k * kCopyThreads + (int)threadIdx.x) * 16;
            if (o < left) *reinterpret_cast<u32x4*>(dst + o) = v[k];
        }
    }
}

struct PlanArgs {
    const int32_t* table;
    const int32_t* released;
    const int32_t* parent;
    const int32_t* child;
    int32_t* table_out;
    int32_t* count;   // nullable
    int32_t* n_pairs; // workspace: number of moves (compaction)
    int32_t* src;     // workspace: the pairs
    int32_t* dst;
    int32_t* status;
    int32_t n_seqs, n_rows, n_slots, n_released, n_children;
};

__device__ __forceinline__ void slot_error(const PlanArgs& a) {
    if (a.status != nullptr) a.status[0] = GDN_ERR_SLOT;
}

// Exclusive prefix sum over the workgroup of one value per thread; *sum is the total.
__device__ int block_prefix(int x, int* sum) {
    __shared__ int wave_sum[kPlanThreads / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();  // the sums of an earlier call have been read
    if (lane == 63) wave_sum[wave] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 64; ++w) {
        const int v = wave_sum[w];
        if (w < wave) before += v;
        all += v;
    }
    *sum = all;
    return before + inc - x;
}

// The rows in use and the released sequences, as bitmaps.  Rows of released
// sequences count as used where keep_released is set.
__device__ void mark_rows(const PlanArgs& a, uint32_t* used, uint32_t* gone, bool keep_released) {
    for (int w = threadIdx.x; w < kMaxWords; w += kPlanThreads) used[w] = 0;
    for (int w = threadIdx.x; w < GDN_POOL_MAX_SEQS / 32; w += kPlanThreads) gone[w] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.n_released; i += kPlanThreads) {
        const int s = a.released[i];
        if (s < 0 || s >= a.n_seqs) slot_error(a);
        else atomicOr(&gone[s >> 5], 1u << (s & 31));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.n_seqs; i += kPlanThreads) {
        const int r = a.table[i];
        if (r < -1 || r >= a.n_slots) slot_error(a);
        const bool counts = keep_released || !((gone[i >> 5] >> (i & 31)) & 1);
        if (counts && r >= 0 && r < a.n_rows) atomicOr(&used[r >> 5], 1u << (r & 31));
    }
    __syncthreads();
}

// Bits of word w that are rows.
__device__ __forceinline__ uint32_t row_bits(const PlanArgs& a, int w) {
    const int left = a.n_rows - 32 * w;
    return left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1;
}

constexpr int kWordsPerThread = kMaxWords / kPlanThreads;

__global__ __launch_bounds__(kPlanThreads) void pool_fork_plan_kernel(const PlanArgs a) {
    __shared__ uint32_t used[kMaxWords], gone[GDN_POOL_MAX_SEQS / 32];
    __shared__ int first[GDN_POOL_MAX_SEQS];  // the first child that names a sequence
    for (int i = threadIdx.x; i < a.n_seqs; i += kPlanThreads) first[i] = 0x7fffffff;
    // the rows of sequences released by this call are not handed out by it: a
    // child may have a released parent
    mark_rows(a, used, gone, true);
    for (int i = threadIdx.x; i < a.n_children; i += kPlanThreads) {
        const int c = a.child[i];
        if (c >= 0 && c < a.n_seqs) atomicMin(&first[c], i);
    }
    uint32_t open[kWordsPerThread];
    int n_open = 0;
#pragma unroll
    for (int k = 0; k < kWordsPerThread; ++k) {
        const int w = threadIdx.x * kWordsPerThread + k;
        open[k] = ~used[w] & row_bits(a, w);
        n_open += __popc(open[k]);
    }
    int total;
    int rank = block_prefix(n_open, &total);
#pragma unroll
    for (int k = 0; k < kWordsPerThread; ++k)
        for (uint32_t m = open[k]; m != 0 && rank < a.n_children; m &= m - 1)
            a.dst[rank++] = 32 * (int)(threadIdx.x * kWordsPerThread + k) + __ffs(m) - 1;
    __syncthreads();
    // pair i: the parent's row -> the i-th lowest free row
    for (int i = threadIdx.x; i < a.n_children; i += kPlanThreads) {
        const int c = a.child[i], p = a.parent[i];
        bool ok = i < total && c >= 0 && c < a.n_seqs && p >= -1 && p < a.n_seqs;
        if (ok) ok = first[c] == i && (a.table[c] == -1 || ((gone[c >> 5] >> (c & 31)) & 1));
        int row = -1;
        if (ok && p >= 0) {
            row = a.table[p];
            ok = row >= 0 && row < a.n_slots;
        }
        a.src[i] = row;
        if (!ok) {
            a.dst[i] = -1;
            slot_error(a);
        }
    }
    __syncthreads();  // every read of the table is done: table_out may be the table
    for (int i = threadIdx.x; i < a.n_seqs; i += kPlanThreads)
        a.table_out[i] = ((gone[i >> 5] >> (i & 31)) & 1) ? -1 : a.table[i];
    __syncthreads();
    for (int i = threadIdx.x; i < a.n_children; i += kPlanThreads) {
        const int d = a.dst[i];
        if (d >= 0) a.table_out[a.child[i]] = d;
    }
}

__global__ __launch_bounds__(kPlanThreads) void pool_compact_plan_kernel(const PlanArgs a) {
    __shared__ uint32_t used[kMaxWords], gone[GDN_POOL_MAX_SEQS / 32];
    __shared__ int before[kMaxWords];  // used rows below each word
    mark_rows(a, used, gone, false);
    int n_used = 0;
#pragma unroll
    for (int k = 0; k < kWordsPerThread; ++k) n_used += __popc(used[threadIdx.x * kWordsPerThread + k]);
    int live;
    int rank = block_prefix(n_used, &live);
#pragma unroll
    for (int k = 0; k < kWordsPerThread; ++k) {
        const int w = threadIdx.x * kWordsPerThread + k;
        before[w] = rank;
        rank += __popc(used[w]);
    }
    __syncthreads();
    // The live rows fill [0, live): the m-th used row at or above `live` moves to
    // the m-th free row below it, so no row is both a source and a destination.
    const int kept = live < a.n_rows ? before[live >> 5] + __popc(used[live >> 5] & ((1u << (live & 31)) - 1)) : live;
#pragma unroll
    for (int k = 0; k < kWordsPerThread; ++k) {
        const int w = threadIdx.x * kWordsPerThread + k;
        int m = before[w];
        for (uint32_t u = used[w]; u != 0; u &= u - 1, ++m)
            if (m >= kept) a.src[m - kept] = 32 * w + __ffs(u) - 1;
        int hole = 32 * w - before[w];
        for (uint32_t f = ~used[w]; f != 0; f &= f - 1, ++hole) {
            const int r = 32 * w + __ffs(f) - 1;
            if (r >= live) break;
            a.dst[hole] = r;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.n_seqs; i += kPlanThreads) {
        int r = a.table[i];
        if ((gone[i >> 5] >> (i & 31)) & 1) r = -1;
        else if (r >= live && r < a.n_rows)
            r = a.dst[before[r >> 5] + __popc(used[r >> 5] & ((1u << (r & 31)) - 1)) - kept];
        a.table_out[i] = r;
    }
    if (threadIdx.x == 0) {
        *a.n_pairs = live - kept;
        if (a.count != nullptr) *a.count = live;
    }
}

// Fills the copy's pool parts; per_pair * n has to fit the kernel's 32-bit tile count.
int plan_parts(const gdn_pool* dst, const gdn_pool* src, int32_t n_pools, int64_t n, CopyRowsArgs* a) {
    int64_t per_pair = 0;
    a->n_parts = 0;
    for (int i = 0; i < n_pools; ++i) {
        if (dst[i].n_layers == 0) continue;
        PoolPart& p = a->part[a->n_parts++];
        p.src = static_cast<const unsigned char*>(src[i].data);
        p.dst = static_cast<unsigned char*>(dst[i].data);
        p.src_layer = src[i].layer_bytes;
        p.dst_layer = dst[i].layer_bytes;
        p.row = dst[i].row_bytes;
        const int64_t tiles = (p.row + kTileBytes - 1) / kTileBytes;
        if (tiles * dst[i].n_layers > 0x7fffffffLL) return GDN_ERR_SHAPE;
        p.tiles = (int32_t)tiles;
        p.items = (int32_t)(tiles * dst[i].n_layers);
        per_pair += p.items;
    }
    if (per_pair * n > 0x7fffffffLL) return GDN_ERR_SHAPE;
    a->per_pair = (int32_t)per_pair;
    return GDN_OK;
}

hipError_t launch_copy(const CopyRowsArgs& a, int64_t n, hipStream_t stream) {
    const int64_t items = n * a.per_pair;
    if (items == 0) return hipSuccess;
    hipLaunchKernelGGL(pool_copy_kernel, dim3((unsigned)(items < kCopyGrid ? items : kCopyGrid)), dim3(kCopyThreads), 0, stream, a);
    return hipGetLastError();
}

int check_table(const gdn_pool* pools, int32_t n_pools, const int32_t* table, int32_t n_seqs, int32_t n_rows,
                const int32_t* released, int32_t n_released, const int32_t* table_out) {
    const int rc = check_pools(pools, n_pools);
    if (rc != GDN_OK) return rc;
    if (n_seqs < 0 || n_seqs > GDN_POOL_MAX_SEQS || n_rows < 1 || n_rows > GDN_POOL_MAX_ROWS || n_rows > pools[0].n_slots ||
        n_released < 0)
        return GDN_ERR_SHAPE;
    for (int i = 0; i < n_pools; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(pools[i], pools[j])) return GDN_ERR_SHAPE;
    if (n_seqs > 0 && (table == nullptr || table_out == nullptr)) return GDN_ERR_NULL;
    if (n_released > 0 && released == nullptr) return GDN_ERR_NULL;
    if (!aligned(table, 4) || !aligned(table_out, 4) || !aligned(released, 4)) return GDN_ERR_ALIGN;
    if (table != table_out && table < table_out + n_seqs && table_out < table + n_seqs) return GDN_ERR_SHAPE;
    return GDN_OK;
}

int check_workspace(const void* workspace, size_t have, size_t need) {
    if (workspace == nullptr || have < need) return GDN_ERR_WORKSPACE;
    return aligned(workspace, 16) ? GDN_OK : GDN_ERR_ALIGN;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_pool_copy(const gdn_pool* dst, const gdn_pool* src, int32_t n_pools, const int32_t* src_row, const int32_t* dst_row,
                  int32_t n, int32_t* status, void* stream) {
    int rc = check_pools(dst, n_pools);
    if (rc != GDN_OK) return rc;
    if (src != nullptr && (rc = check_pools(src, n_pools)) != GDN_OK) return rc;
    if (n < 0) return GDN_ERR_SHAPE;
    CopyRowsArgs a;
    std::memset(&a, 0, sizeof(a));
    a.same = src == nullptr;
    for (int i = 0; i < n_pools; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(dst[i], dst[j])) return GDN_ERR_SHAPE;
        if (src == nullptr) continue;
        if (src[i].row_bytes != dst[i].row_bytes || src[i].n_layers != dst[i].n_layers) return GDN_ERR_SHAPE;
        for (int j = 0; j < n_pools; ++j)
            if (overlap(dst[i], src[j])) return GDN_ERR_SHAPE;
    }
    if (n == 0) return GDN_OK;
    if (src_row == nullptr || dst_row == nullptr) return GDN_ERR_NULL;
    if (!aligned(src_row, 4) || !aligned(dst_row, 4) || !aligned(status, 4)) return GDN_ERR_ALIGN;
    if ((rc = plan_parts(dst, src != nullptr ? src : dst, n_pools, n, &a)) != GDN_OK) return rc;
    a.src_row = src_row;
    a.dst_row = dst_row;
    a.status = status;
    a.n = n;
    a.src_slots = (src != nullptr ? src : dst)[0].n_slots;
    a.dst_slots = dst[0].n_slots;
    a.check = 1;
    return launch_copy(a, n, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

size_t gdn_pool_fork_workspace_bytes(int32_t n_children) { return n_children > 0 ? 8 * (size_t)n_children : 0; }

int gdn_pool_fork(const gdn_pool* pools, int32_t n_pools, const int32_t* table, int32_t n_seqs, int32_t n_rows,
                  const int32_t* released, int32_t n_released, const int32_t* parent, const int32_t* child,
                  int32_t n_children, int32_t* table_out, void* workspace, size_t workspace_bytes, int32_t* status,
                  void* stream) {
    int rc = check_table(pools, n_pools, table, n_seqs, n_rows, released, n_released, table_out);
    if (rc != GDN_OK) return rc;
    if (n_children < 0 || n_children > GDN_POOL_MAX_SEQS) return GDN_ERR_SHAPE;
    if (n_children > 0 && (parent == nullptr || child == nullptr)) return GDN_ERR_NULL;
    if (!aligned(parent, 4) || !aligned(child, 4) || !aligned(status, 4)) return GDN_ERR_ALIGN;
    if (n_children > 0 && (rc = check_workspace(workspace, workspace_bytes, gdn_pool_fork_workspace_bytes(n_children))) != GDN_OK)
        return rc;
    CopyRowsArgs c;
    std::memset(&c, 0, sizeof(c));
    if ((rc = plan_parts(pools, pools, n_pools, n_children, &c)) != GDN_OK) return rc;
    if (n_seqs == 0 && n_children == 0 && n_released == 0) return GDN_OK;
    PlanArgs a;
    std::memset(&a, 0, sizeof(a));
    a.table = table; a.released = released; a.parent = parent; a.child = child; a.table_out = table_out;
    a.src = static_cast<int32_t*>(workspace);
    a.dst = a.src + n_children;
    a.status = status; a.n_seqs = n_seqs; a.n_rows = n_rows; a.n_slots = pools[0].n_slots;
    a.n_released = n_released; a.n_children = n_children;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipLaunchKernelGGL(pool_fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, a);
    if (hipGetLastError() != hipSuccess) return GDN_ERR_HIP;
    c.src_row = a.src;
    c.dst_row = a.dst;
    c.n = n_children;
    c.same = 1;
    return launch_copy(c, n_children, st) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

size_t gdn_pool_compact_workspace_bytes(int32_t n_rows) { return n_rows > 0 ? 16 + 8 * (size_t)n_rows : 0; }

int gdn_pool_compact(const gdn_pool* pools, int32_t n_pools, const int32_t* table, int32_t n_seqs, int32_t n_rows,
                     const int32_t* released, int32_t n_released, int32_t* table_out, int32_t* count, void* workspace,
                     size_t workspace_bytes, int32_t* status, void* stream) {
    int rc = check_table(pools, n_pools, table, n_seqs, n_rows, released, n_released, table_out);
    if (rc != GDN_OK) return rc;
    if (!aligned(count, 4) || !aligned(status, 4)) return GDN_ERR_ALIGN;
    if ((rc = check_workspace(workspace, workspace_bytes, gdn_pool_compact_workspace_bytes(n_rows))) != GDN_OK) return rc;
    // a row that moves leaves a free row below it behind: at most half of the rows move
    const int64_t most = n_seqs < n_rows / 2 ? n_seqs : n_rows / 2;
    CopyRowsArgs c;
    std::memset(&c, 0, sizeof(c));
    if ((rc = plan_parts(pools, pools, n_pools, most, &c)) != GDN_OK) return rc;
    PlanArgs a;
    std::memset(&a, 0, sizeof(a));
    a.table = table; a.released = released; a.table_out = table_out; a.count = count;
    a.n_pairs = static_cast<int32_t*>(workspace);
    a.src = a.n_pairs + 4;
    a.dst = a.src + n_rows;
    a.status = status; a.n_seqs = n_seqs; a.n_rows = n_rows; a.n_slots = pools[0].n_slots; a.n_released = n_released;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipLaunchKernelGGL(pool_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, a);
    if (hipGetLastError() != hipSuccess) return GDN_ERR_HIP;
    c.src_row = a.src;
    c.dst_row = a.dst;
    c.n_dev = a.n_pairs;
    c.same = 1;
    return launch_copy(c, most, st) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // extern "C"
