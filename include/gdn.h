/*
 * gdn.h -- C ABI of the Gated DeltaNet recurrent-state library for MI355X
 * (gfx950): speculative-draft verify over a chain or a tree, commit of the
 * accepted node, chunked prefill, the training scan, the rows of the state
 * pool (also in 8 bits), and what stands around the rule in a layer: the input
 * norm, the gated norm of its outputs, both to 8 bits and with gradients, and
 * projections in 8 bits.
 *
 * The recurrence, per (sequence, value head), with S the d_v x d_k state:
 *     S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *     o_t = scale * S_t q_t                     (read after the update)
 * This is the gated delta rule of a Gated DeltaNet layer, the layer of the
 * page "LightSeek's TokenSpeed Hits 580 Tokens per Second on Qwen3.5's 400B
 * Model", section "Why Qwen3.5 is hard to serve fast": a fixed state of
 * head-dimension-squared size per layer, updated per token, with the output
 * read from the current state.  The page states it in words; the formula
 * above is this library's definition of it.
 *
 * Conventions for every entry point
 *  - All tensors are dense, C-contiguous, in device memory, with these
 *    layouts (B = shape.batch, N = shape.n_nodes):
 *        q, k         [B][N][h_qk][d_k]      qkv_dtype (F32 or BF16)
 *        v            [B][N][h_v][d_v]       qkv_dtype
 *        alpha, beta  [B][N][h_v]            fp32
 *        state        [n_slots][h_v][d_v][d_k] fp32   (row j = value channel j)
 *        state_slot   [B] int32, nullable: sequence b uses state[state_slot[b]];
 *                     NULL means sequence b uses state[b]
 *        out          [B][N][h_v][d_v]       out_dtype (F32, F16 or BF16)
 *        persist      [B][N][h_v][d_v][d_k]  persist_dtype (F16 or F32)
 *        final_state  [B][h_v][d_v][d_k]     fp32
 *    Value head h reads q/k head h / (h_v / h_qk).
 *  - q, k, v, state, persist and final_state must be 16-byte aligned; the
 *    other pointers 4-byte aligned.
 *  - The caller owns every buffer.  The library allocates no memory and is
 *    safe to call from several host threads.  Its only host-side state is
 *    set once per device and never changes afterwards: the compute-unit count
 *    it reads, and the attribute that lets a kernel use all of a compute
 *    unit's LDS (both behind atomics).
 *  - `stream` is a hipStream_t (NULL = the default stream).  Calls only
 *    enqueue work on it and return; they never synchronise the host.
 *  - Errors found on the host (null or misaligned pointers, bad shapes or
 *    dtypes, bad parent arrays, small workspace) return a negative
 *    gdn_status before anything is enqueued; no buffer is touched.
 *    Errors only the device can see (an out-of-range accepted node or state
 *    slot) skip that sequence, leave its buffers untouched and store the
 *    code into *status when `status` is not NULL.  The caller zeroes
 *    *status beforehand; concurrent errors leave one of their codes.
 *  - A failed kernel launch returns GDN_ERR_HIP.
 *  - The library built with -DGDN_DEBUG (libgdn_debug.so) checks the indices
 *    its kernels form into the caller's arrays and the workspace: one past
 *    its array's end stores GDN_ERR_INTERNAL into *status and is clamped into
 *    the array.  The release build carries no such checks.  The kernels of
 *    gdn_scan_*, gdn_pool_*, gdn_norm_*, gdn_gated_norm_* and gdn_project have
 *    none in either build: their indices follow from the shape, the offsets and
 *    the row numbers, which every build checks.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_MAX_NODES 32      /* draft nodes per verify call (a 22-node tree plus margin) */
#define GDN_MAX_TREE_DEPTH 16 /* nodes on a root-to-leaf path, root included */
#define GDN_PREFILL_CHUNK 64  /* tokens per chunk of gdn_prefill_chunked */
#define GDN_MAX_CONV_WIDTH 8  /* taps of the causal convolution whose history gdn_conv_commit keeps */
#define GDN_MAX_POOLS 8       /* pools of one gdn_pool_copy, gdn_pool_fork or gdn_pool_compact call */
#define GDN_POOL_MAX_ROWS 65536 /* rows gdn_pool_fork hands out and gdn_pool_compact moves */
#define GDN_POOL_MAX_SEQS 8192  /* entries of their index table */

typedef enum gdn_status {
    GDN_OK = 0,
    GDN_ERR_NULL = -1,        /* a required pointer is NULL */
    GDN_ERR_SHAPE = -2,       /* a size is out of range or inconsistent */
    GDN_ERR_DTYPE = -3,       /* a dtype code is not allowed where it was given */
    GDN_ERR_ALIGN = -4,       /* a pointer is not aligned as required */
    GDN_ERR_PARENT = -5,      /* the parent array is not a valid tree */
    GDN_ERR_NODE = -6,        /* device: accepted node outside [0, N) */
    GDN_ERR_WORKSPACE = -7,   /* workspace missing or too small */
    GDN_ERR_UNSUPPORTED = -8, /* valid request this library does not implement */
    GDN_ERR_HIP = -9,         /* the HIP runtime refused the launch */
    GDN_ERR_SLOT = -10,       /* device: state slot outside [0, n_slots) */
    GDN_ERR_RANGE = -11,      /* device: a prefill value left the f16 range of the matrix-core operands */
    GDN_ERR_INTERNAL = -12    /* device, debug build only: an index check inside a kernel failed */
} gdn_status;

typedef enum gdn_dtype { GDN_F32 = 0, GDN_BF16 = 1, GDN_F16 = 2 } gdn_dtype;

typedef struct gdn_shape {
    int32_t batch;         /* independent sequences (or sequence x layer units), >= 0 */
    int32_t n_nodes;       /* draft nodes per sequence; tokens per sequence for prefill */
    int32_t h_qk;          /* q/k heads, >= 1 */
    int32_t h_v;           /* value heads, a multiple of h_qk; verify and commit by replay need
                              h_v * d_v * d_k * GDN_MAX_NODES < 2^32 */
    int32_t d_k;           /* key channels: 32, 64 or 128 */
    int32_t d_v;           /* value channels: a multiple of 16, at most 256 */
    int32_t n_slots;       /* rows of `state` when state_slot is given (ignored otherwise) */
    int32_t qkv_dtype;     /* GDN_F32 or GDN_BF16 */
    int32_t out_dtype;     /* GDN_F32, GDN_F16 or GDN_BF16 */
    int32_t persist_dtype; /* GDN_F16 or GDN_F32 */
    float scale;           /* output scale; 1 for the plain rule */
} gdn_shape;

/*
 * Verify a causal chain of N draft nodes per sequence.
 * Page "400 tok/s with Qwen3.5", sections "Speculative verification in a
 * megakernel" and "Handling recurrent state": the target checks a block of
 * draft tokens in one causal pass, keeping the recurrent working state on
 * chip across the block.
 *
 * Node n of sequence b starts from node n-1 (node 0 from the cached state
 * state[slot(b)], which is only read).  For every node the output goes to
 * out (nullable) and the state after the node to persist (nullable), stored
 * in persist_dtype with round-to-nearest-even: page "We got 207 tok/s with
 * Qwen3.5-27B on an RTX 3090", section "Key wins" (an f16 per-node cache,
 * written by the recurrence kernel itself).  The fp32 state after node N-1
 * goes to final_state (nullable), exactly as computed.  final_state may be
 * `state` itself (in-place advance) when state_slot is NULL.
 */
int gdn_verify_chain(const gdn_shape* shape, const void* q, const void* k, const void* v,
                     const float* alpha, const float* beta, const float* state,
                     const int32_t* state_slot, void* out, void* persist, float* final_state,
                     int32_t* status, void* stream);

/*
 * One launch for a decode step: commit the previous step's accepted node, then
 * verify the next chain from the committed state.  Equivalent to
 *     gdn_commit(shape, accepted_prev, persist_prev, final_prev, state, state_slot, status)
 *     gdn_verify_chain(shape, q, k, v, alpha, beta, state, state_slot, out, persist,
 *                      final_state, status)
 * with the commit fused into the verify's state load, so the committed state is
 * read once (as the f16 node copy, or final_prev on full acceptance), written to
 * state[slot(b)] and used directly.  Page "400 tok/s with Qwen3.5", section
 * "Handling recurrent state" (state set to the accepted boundary before the next
 * verification).
 *
 * persist_prev and final_prev (nullable) are the previous step's persist and
 * final_state: same layout, n_nodes and persist_dtype as this call's outputs.
 * They may be the very buffers this call writes (each value is read before it
 * is overwritten).  accepted_prev is a device array [B]; a node outside [0, N)
 * skips the sequence entirely (state and outputs untouched) and sets *status to
 * GDN_ERR_NODE.  Other arguments and errors as gdn_verify_chain; final_state
 * may not be `state` here.
 */
int gdn_commit_verify_chain(const gdn_shape* shape, const int32_t* accepted_prev, const void* persist_prev,
                            const float* final_prev, const void* q, const void* k, const void* v,
                            const float* alpha, const float* beta, float* state, const int32_t* state_slot,
                            void* out, void* persist, float* final_state, int32_t* status, void* stream);

/*
 * Verify a tree of N draft nodes per sequence.
 * Page "Qwen3.6 27B: From 20 t/s to 184 t/s", section "Diffusion applied to
 * text": a best-first tree of up to 22 nodes is verified in one target pass.
 *
 * `parent` is a HOST array of n_trees x N int32, n_trees = 1 (one tree for
 * every sequence) or batch (one per sequence).  parent[0] = -1 (node 0, the
 * root, starts from the cached state); for n >= 1, 0 <= parent[n] < n; no
 * root-to-leaf path holds more than GDN_MAX_TREE_DEPTH nodes.  Node n starts
 * from the exact fp32 state of node parent[n]; outputs and persisted states
 * are indexed by node.  The array is read during the call only.
 */
int gdn_verify_tree(const gdn_shape* shape, const int32_t* parent, int32_t n_trees, const void* q,
                    const void* k, const void* v, const float* alpha, const float* beta,
                    const float* state, const int32_t* state_slot, void* out, void* persist,
                    int32_t* status, void* stream);

/*
 * One launch for a tree decode step: commit the previous step's accepted node,
 * then verify the next tree from the committed state.  Equivalent to
 *     gdn_commit(shape, accepted_prev, persist_prev, NULL, state, state_slot, status)
 *     gdn_verify_tree(shape, parent, n_trees, q, k, v, alpha, beta, state, state_slot,
 *                     out, persist, status)
 * with the commit fused into the verify's state load: the accepted node's
 * persisted copy is read once, widened to fp32, written to state[slot(b)] and
 * used directly as the root's starting state.  Page "400 tok/s with Qwen3.5",
 * section "Handling recurrent state" (state set to the accepted boundary before
 * the next verification); page "Qwen3.6 27B: From 20 t/s to 184 t/s", section
 * "Diffusion applied to text" (the tree verified in one pass).
 *
 * persist_prev is the previous step's persist: same layout, n_nodes and
 * persist_dtype as this call's; it may be the very buffer this call writes
 * (each value is read before it is overwritten).  accepted_prev is a device
 * array [B] of node indices of the previous step (the last node of its accepted
 * path); a node outside [0, N) skips the sequence entirely (state and outputs
 * untouched) and sets *status to GDN_ERR_NODE.  parent, n_trees and the other
 * arguments and errors as gdn_verify_tree.
 */
int gdn_commit_verify_tree(const gdn_shape* shape, const int32_t* accepted_prev, const void* persist_prev,
                           const int32_t* parent, int32_t n_trees, const void* q, const void* k, const void* v,
                           const float* alpha, const float* beta, float* state, const int32_t* state_slot,
                           void* out, void* persist, int32_t* status, void* stream);

/*
 * Commit the accepted node of every sequence into the state cache.
 * Page "400 tok/s with Qwen3.5", section "Handling recurrent state": after a
 * rejection the state is set to the accepted boundary; a fully accepted
 * block uses the verified state directly.
 *
 * accepted_node is a DEVICE array [B] of node indices (node L-1 for an
 * accepted chain prefix of length L; the last node of the accepted path in a
 * tree).  state[slot(b)] <- persist[b][a] widened to fp32, or final_state[b]
 * when final_state is not NULL and a = N-1.  Only shape.batch, n_nodes, h_v,
 * d_k, d_v, n_slots and persist_dtype are read.  An accepted node outside
 * [0, N) or a slot outside [0, n_slots) skips the sequence and sets *status.
 */
int gdn_commit(const gdn_shape* shape, const int32_t* accepted_node, const void* persist,
               const float* final_state, float* state, const int32_t* state_slot,
               int32_t* status, void* stream);

/*
 * Commit by replay: set the cached state to the accepted node's state by
 * running the recurrence again over the accepted nodes, from the state the
 * block was verified from, with the block's retained inputs.  Page "400 tok/s
 * with Qwen3.5", section "Handling recurrent state" (checkpoint-and-replay: the
 * state from before the draft block is kept with the projected inputs, and a
 * replay kernel advances it through the accepted positions only).  With this
 * commit a verify needs to persist no node states (persist = NULL).
 *
 * On entry state[slot(b)] is the state the block was verified from (the
 * checkpoint); on return it is the fp32 state after node accepted_node[b]
 * (device array [B]).  The nodes replayed are the node's root path: nodes
 * 0 .. a of a chain (parent == NULL), or the ancestors of a, root first, of a
 * tree (parent: HOST array as in gdn_verify_tree, n_trees x N with n_trees = 1
 * or batch).  The arithmetic per node is the verify's, so the result equals
 * bit for bit the fp32 node state that gdn_verify_chain / gdn_verify_tree
 * persist with persist_dtype F32 for the same inputs.  q, k, v, alpha, beta are
 * the block's inputs, laid out as for verify.  No outputs are written;
 * shape.out_dtype, persist_dtype and scale are not used.  A node outside
 * [0, N) or a slot outside [0, n_slots) skips the sequence (its state is left
 * as it was) and sets *status.
 */
int gdn_commit_replay(const gdn_shape* shape, const int32_t* parent, int32_t n_trees,
                      const int32_t* accepted_node, const void* q, const void* k, const void* v,
                      const float* alpha, const float* beta, float* state, const int32_t* state_slot,
                      int32_t* status, void* stream);

/*
 * One launch for a decode step with commit by replay: replay the previous chain
 * block's accepted nodes (as gdn_commit_replay with parent = NULL, inputs
 * q_prev .. beta_prev and accepted_prev), write the result to state[slot(b)],
 * then verify the next chain (q .. beta) from it, as gdn_verify_chain would
 * from the updated cache.  Page "400 tok/s with Qwen3.5", section "Handling
 * recurrent state".  The replayed state never leaves registers between the
 * two.  persist is usually NULL in this scheme (nothing to persist: the next
 * step replays); out and final_state are as in gdn_verify_chain, and
 * final_state may not be `state`.  The previous block has this call's shape.
 * An accepted node outside [0, N) skips the sequence entirely (state and
 * outputs untouched) and sets *status to GDN_ERR_NODE.
 */
int gdn_replay_verify_chain(const gdn_shape* shape, const int32_t* accepted_prev, const void* q_prev,
                            const void* k_prev, const void* v_prev, const float* alpha_prev,
                            const float* beta_prev, const void* q, const void* k, const void* v,
                            const float* alpha, const float* beta, float* state, const int32_t* state_slot,
                            void* out, void* persist, float* final_state, int32_t* status, void* stream);

/*
 * Index-table commit: commit the accepted node by pointing the sequence's
 * index-table entry at the row that already holds its state, instead of
 * copying the state.  Page "LightSeek's TokenSpeed Hits 580 Tokens per Second
 * on Qwen3.5's 400B Model", section "How they actually got there" (move
 * pointers, not data: the state buffer gains a draft region, and an index
 * table records which row holds each sequence's state).
 *
 * Protocol.  `state` is a pool [n_slots][h_v][d_v][d_k] fp32 whose rows
 * draft_row0 .. draft_row0 + B N - 1 form the draft region; state_slot [B] is
 * the index table.  gdn_verify_chain / gdn_verify_tree are called with this
 * state_slot and with persist = the pool's row draft_row0 (persist_dtype F32),
 * so node n of sequence b is persisted, exactly, in row draft_row0 + b N + n.
 * A verify may persist over the row it reads its state from: every element is
 * read before it is written.  gdn_commit_index then sets, on the device,
 *     state_slot[b] <- draft_row0 + b N + accepted_node[b]
 * and the next verify reads the accepted node's exact fp32 state from there.
 * accepted_node and state_slot are DEVICE arrays [B]; draft_row0 + B N must
 * not exceed n_slots.  An accepted node outside [0, n_nodes) leaves the entry
 * as it was and sets *status to GDN_ERR_NODE.
 */
int gdn_commit_index(const int32_t* accepted_node, int32_t* state_slot, int32_t batch, int32_t n_nodes,
                     int32_t draft_row0, int32_t n_slots, int32_t* status, void* stream);

/*
 * Rows of a state pool.  A sequence of a hybrid model owns one row: its
 * recurrent state in every layer, and its convolution history.  Page
 * "LightSeek's TokenSpeed Hits 580 Tokens per Second on Qwen3.5's 400B Model",
 * section "How they actually got there": states live in the rows of a buffer,
 * an index table records which row holds each sequence's state, and cached
 * prefixes are states that other sequences continue from.
 *
 * A gdn_pool is one array of rows for several layers: row r of layer l starts
 * at data + l layer_bytes + r row_bytes.  The pools of one call have the same
 * n_slots, share no byte (the layers of one may lie between another's), and row
 * r means row r of every layer of each of them.  Rows hold anything (bytes are
 * moved).
 */
typedef struct gdn_pool {
    void* data;          /* 16-byte aligned (not read where n_layers is 0) */
    int64_t row_bytes;   /* bytes of a row, a multiple of 16, at least 16 */
    int64_t layer_bytes; /* from one layer to the next, a multiple of 16, at least n_slots * row_bytes */
    int32_t n_layers;    /* >= 0 */
    int32_t n_slots;     /* rows of a layer, >= 1 */
} gdn_pool;

/*
 * Copy rows: row dst_row[i] of every dst pool <- row src_row[i] of the src pool
 * of the same place, for i < n (restoring a cached prefix into a sequence's
 * row, keeping a row as a checkpoint).  src NULL copies within dst; otherwise
 * src[p] has dst[p]'s row_bytes and n_layers, rows of its own number, and shares
 * no byte with any dst pool.  src_row and dst_row are DEVICE arrays [n].  A
 * source row of -1 zero-fills the destination row (a fresh sequence); a pair
 * whose destination row is -1 is passed over.  One source may be named by any
 * number of pairs.  A pair with a row outside the pools, and every pair whose
 * destination is also another pair's destination or (within dst) another
 * pair's source, is not copied and sets *status to GDN_ERR_SLOT; rows that no
 * copied pair names are left as they were.
 */
int gdn_pool_copy(const gdn_pool* dst, const gdn_pool* src, int32_t n_pools, const int32_t* src_row,
                  const int32_t* dst_row, int32_t n, int32_t* status, void* stream);

/*
 * Release sequences and fork others.  `table` (DEVICE, [n_seqs]) is the index
 * table: the row of each sequence, -1 where it has none.  The rows this call
 * may hand out are rows 0 .. n_rows - 1 (n_rows <= n_slots: the rest, such as
 * the draft region of gdn_commit_index, is not touched) that no entry of
 * `table` names.  In this order:
 *   - child i (i < n_children) gets the i-th lowest free row; the row of
 *     sequence parent[i] is copied there in all pools (a parent of -1: zeroed);
 *   - table_out is `table` with -1 for the sequences in released[n_released],
 *     then the new row for each sequence child[i].
 * A parent may be released by the same call (its row is not handed out by it),
 * and a child may be a released sequence, but no child may hold a row that is
 * not released.  A child that does, one outside [0, n_seqs), one that an
 * earlier child names too, one whose parent is outside [-1, n_seqs) or holds
 * no row, and one for which no free row is left gets nothing and sets *status
 * to GDN_ERR_SLOT, as do a released sequence outside [0, n_seqs) and a table
 * entry outside [-1, n_slots) (both are otherwise passed over).
 * released, parent and child are DEVICE arrays; table_out is `table` itself or
 * does not overlap it.  With n_children = 0 the call only releases.
 * `workspace`: device memory of gdn_pool_fork_workspace_bytes(n_children)
 * bytes, 16-byte aligned; calls that share one are ordered on one stream.
 */
size_t gdn_pool_fork_workspace_bytes(int32_t n_children);
int gdn_pool_fork(const gdn_pool* pools, int32_t n_pools, const int32_t* table, int32_t n_seqs, int32_t n_rows,
                  const int32_t* released, int32_t n_released, const int32_t* parent, const int32_t* child,
                  int32_t n_children, int32_t* table_out, void* workspace, size_t workspace_bytes, int32_t* status,
                  void* stream);

/*
 * Release sequences and move the rows still in use together.  With L the
 * number of rows below n_rows that the entries of `table` name once the
 * sequences in released[n_released] have none, the rows in use end up in rows
 * 0 .. L - 1: the m-th row in use at or above L (in row order) moves to the
 * m-th free row below L, all others stay.  table_out is the table with the
 * moved rows' new places and -1 for the released sequences; sequences that
 * share a row still share it.  Entries at or above n_rows stay as they are.
 * *count (nullable, DEVICE) receives L.  Vacated rows keep their contents.
 * Other arguments and device errors as gdn_pool_fork; `workspace` holds
 * gdn_pool_compact_workspace_bytes(n_rows) bytes.
 */
size_t gdn_pool_compact_workspace_bytes(int32_t n_rows);
int gdn_pool_compact(const gdn_pool* pools, int32_t n_pools, const int32_t* table, int32_t n_seqs, int32_t n_rows,
                     const int32_t* released, int32_t n_released, int32_t* table_out, int32_t* count, void* workspace,
                     size_t workspace_bytes, int32_t* status, void* stream);

/*
 * State rows in 8 bits: cached prefixes in 26 % of the room (d_k = 128).  A row
 * of a state pool holds n = row_bytes / (element size * d_k) value channels of
 * d_k states each (n = h_v d_v); channel c of a packed row is
 *     scale[c] = max(max_k |S[c][k]| / 127, 2^-126)       fp32, rounded to nearest
 *                (down where 127 of it would be infinite: a channel of FLT_MAX)
 *     code[c][k] = S[c][k] / scale[c] to the nearest integer, ties to even  int8
 * and stands for code * scale.  Uniform steps: a value is off by at most half a
 * scale, amax / 254.  A channel that holds a NaN or an infinity is packed as
 * scale NaN and codes 0: all of it reads back as NaN, other channels do not see
 * it.
 *
 * `states` is a pool of fp32, f16 or bf16 states (the persisted node states of a
 * verify are one too: one layer, a row per node), `codes` and `scales` are pools
 * of int8 rows [n][d_k] and of fp32 rows [n]: row_bytes n d_k and 4 n, the same
 * n_layers, and n_slots of their own, the same in both.  d_k is 32, 64 or 128, n a
 * multiple of 4.  No two of the three share a byte.
 *
 * gdn_pool_pack writes packed row dst_row[i] from state row src_row[i] in every
 * layer, gdn_pool_unpack state row dst_row[i] from packed row src_row[i], i < n.
 * src_row, dst_row, their order, the row numbers -1 (a source of -1: a row of
 * zeros) and device errors are those of gdn_pool_copy with a src.
 */
int gdn_pool_pack(const gdn_pool* states, const gdn_pool* codes, const gdn_pool* scales, int32_t d_k, int32_t dtype,
                  const int32_t* src_row, const int32_t* dst_row, int32_t n, int32_t* status, void* stream);
int gdn_pool_unpack(const gdn_pool* codes, const gdn_pool* scales, const gdn_pool* states, int32_t d_k, int32_t dtype,
                    const int32_t* src_row, const int32_t* dst_row, int32_t n, int32_t* status, void* stream);

/* Shape of a causal-convolution history commit. */
typedef struct gdn_conv_shape {
    int32_t batch;    /* sequences, >= 0 */
    int32_t n_nodes;  /* draft nodes per sequence, 1 .. GDN_MAX_NODES */
    int32_t channels; /* C, input channels of the convolution; C * element size a multiple of 16 bytes */
    int32_t width;    /* W, taps of the convolution, 2 .. GDN_MAX_CONV_WIDTH; the history keeps W - 1 rows */
    int32_t n_slots;  /* rows of conv_state when state_slot is given (ignored otherwise) */
    int32_t dtype;    /* element type of x and conv_state: GDN_F32, GDN_BF16 or GDN_F16 (bytes are copied) */
} gdn_conv_shape;

/*
 * Commit the causal-convolution input history to the accepted boundary.
 * Page "400 tok/s with Qwen3.5", section "Handling recurrent state": the
 * convolution history is committed to the same boundary as the recurrent
 * state.  A causal convolution of width W reads the current input row and the
 * W - 1 before it, so each sequence keeps its last W - 1 input rows:
 *     conv_state [n_slots][W-1][C]   oldest row first (16-byte aligned)
 *     x          [B][N][C]           the draft block's convolution inputs
 * On return conv_state[slot(b)] holds the last W - 1 rows of the accepted
 * stream: the previous history rows followed by the inputs of the nodes on
 * accepted_node[b]'s root path, root first (nodes 0 .. a of a chain when
 * parent == NULL; parent as in gdn_verify_tree otherwise, n_trees = 1 or
 * batch).  Rows are copied bit for bit.  accepted_node is a DEVICE array [B];
 * a node outside [0, N) or a slot outside [0, n_slots) skips the sequence and
 * sets *status.
 */
int gdn_conv_commit(const gdn_conv_shape* shape, const int32_t* parent, int32_t n_trees,
                    const int32_t* accepted_node, const void* x, void* conv_state,
                    const int32_t* state_slot, int32_t* status, void* stream);

/*
 * Chunked prefill of a prompt: the same recurrence over shape.n_nodes = T
 * tokens per sequence, evaluated GDN_PREFILL_CHUNK tokens at a time in the
 * WY / UT form.  Page "We got 207 tok/s with Qwen3.5-27B on an RTX 3090",
 * section "Prefill" (prompts are processed in micro-batches of tokens); the
 * chunk algebra is derived from the rule (see the kernel source).
 *
 * q, k [B][T][h_qk][d_k], v [B][T][h_v][d_v] (qkv_dtype F32 or BF16; values
 * are converted to f16 for the matrix cores, so they must lie inside the f16
 * range, |x| <= 65504, and magnitudes below 2^-14 keep an absolute precision
 * of 2^-25).  A q or k element outside that range, or a value of the
 * recurrence that leaves it on the way (from v, the state or the initial
 * state, which then leaves the final state non-finite), sets *status to
 * GDN_ERR_RANGE when status is not NULL; the outputs and the state of that
 * call are then not meaningful;
 * alpha, beta [B][T][h_v] fp32; out [B][T][h_v][d_v] in out_dtype (F32, F16
 * or BF16), 16-byte aligned.  state[slot(b)] holds the initial state on entry and the state
 * after token T-1 on return (updated in place).  A zero alpha resets the state
 * up to a factor e^-80 (the log-gate is clamped at -80).  d_k must be 32, 64 or
 * 128, d_v a multiple of 32 and h_v / h_qk at most 128 (else GDN_ERR_UNSUPPORTED).
 * persist_dtype is ignored.  T = 0 or batch = 0
 * is a no-op.
 *
 * `workspace` is caller-owned device memory of at least
 * gdn_prefill_workspace_bytes(shape) bytes (16-byte aligned), used during the
 * call for the per-chunk operands that do not depend on the state (the UT
 * transform and masked Q K^T per chunk and value head in f16, the gate factors,
 * K and Q in f16 per chunk and q/k head); about 1.3 MB per 64 tokens at 48 value
 * heads, 16 q/k heads and d_k = 128.  Its contents on entry are ignored.  A missing or short workspace
 * returns GDN_ERR_WORKSPACE.  Calls sharing one workspace must be ordered on
 * one stream.
 */
size_t gdn_prefill_workspace_bytes(const gdn_shape* shape);
int gdn_prefill_chunked(const gdn_shape* shape, const void* q, const void* k, const void* v,
                        const float* alpha, const float* beta, float* state,
                        const int32_t* state_slot, void* out, void* workspace,
                        size_t workspace_bytes, int32_t* status, void* stream);

/*
 * gdn_prefill_chunked for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation): no workspace argument.  The per-chunk operands go to a static
 * array of this library, GDN_PREFILL_SCRATCH_BYTES per GPU, which each GPU the
 * library runs on holds until the process ends.  A prompt whose workspace
 * (gdn_prefill_workspace_bytes) exceeds the array is processed in segments of
 * whole 64-token chunks, each a launch pair that reuses it; the results are
 * bit for bit those of gdn_prefill_chunked.  Heads so large that one 64-token
 * chunk does not fit return GDN_ERR_WORKSPACE before anything is enqueued.
 * Every call on one GPU uses the same array: calls that may overlap on one GPU
 * (on different streams, or from several host threads without ordering) race
 * and must not be issued.  The call allocates nothing: no hipMalloc, hipFree
 * or allocating library routine.  Other arguments, limits and errors as
 * gdn_prefill_chunked.
 */
#define GDN_PREFILL_SCRATCH_BYTES (32u << 20)
int gdn_prefill_chunked_noalloc(const gdn_shape* shape, const void* q, const void* k, const void* v,
                                const float* alpha, const float* beta, float* state, const int32_t* state_slot,
                                void* out, int32_t* status, void* stream);

/*
 * Varlen batched prefill with chunk-boundary states.  The same recurrence
 * and chunked evaluation as gdn_prefill_chunked, for `batch` sequences of
 * different lengths packed one after another along the token dimension, in
 * one call.  Page "LightSeek's TokenSpeed Hits 580 Tokens per Second on
 * Qwen3.5's 400B Model", section "How they actually got there" (hybrid prefix
 * caching needs the recurrent state at the exact prefix boundary): the call
 * can also emit the state at every state_interval-th chunk boundary.
 *
 * cu_seqlens is a HOST array [batch + 1]: 0 = cu[0] <= cu[1] <= ... <=
 * cu[batch] = shape.n_nodes (the total token count); sequence b holds tokens
 * cu[b] .. cu[b+1]-1 of
 *     q, k [total][h_qk][d_k],  v [total][h_v][d_v],  alpha, beta [total][h_v],
 *     out [total][h_v][d_v] (out_dtype, 16-byte aligned),
 * and state[slot(b)] (initial state in, final state out, in place; an empty
 * sequence keeps its state).  chunk_states (nullable, fp32, [n][h_v][d_v][d_k])
 * receives, sequence after sequence, the state after token
 * 64 state_interval m - 1 of the sequence for m = 1, 2, ... while that token
 * exists: n = gdn_prefill_boundary_states(cu_seqlens, batch, state_interval)
 * states in all.  state_interval >= 1 when chunk_states is set.  Sequences
 * are processed in launches of up to 64; the workspace (at least
 * gdn_prefill_varlen_workspace_bytes(shape, cu_seqlens) bytes) is reused by
 * each.  Other arguments, limits and errors as gdn_prefill_chunked; an
 * invalid cu_seqlens returns GDN_ERR_SHAPE (GDN_ERR_NULL if missing).
 */
size_t gdn_prefill_varlen_workspace_bytes(const gdn_shape* shape, const int32_t* cu_seqlens);
int64_t gdn_prefill_boundary_states(const int32_t* cu_seqlens, int32_t batch, int32_t state_interval);
int gdn_prefill_varlen(const gdn_shape* shape, const int32_t* cu_seqlens, const void* q, const void* k,
                       const void* v, const float* alpha, const float* beta, float* state,
                       const int32_t* state_slot, void* out, float* chunk_states, int32_t state_interval,
                       void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/*
 * The training scan: the recurrence over packed sequences at fp32 accuracy,
 * with its gradients.  gdn_prefill_varlen evaluates the same rule for serving,
 * with f16 matrix operands; here every product has fp32's accuracy (sums are
 * rounded to fp32, what is left out of a product is below 2^-23 of it and of
 * either sign), so the gradients, those of the gates included, are accurate to
 * fp32.  That holds for magnitudes from 2^-109 to 3.39e38: of smaller values what
 * lies below 2^-126 is lost, and 2^128 - 2^119 and above count as infinite.
 *
 * cu_seqlens is a HOST array [batch + 1] as for gdn_prefill_varlen (batch
 * equal sequences [B][T] are the offsets 0, T, 2 T, ...), and q, k [total]
 * [h_qk][d_k], v, out [total][h_v][d_v], alpha, beta [total][h_v] are packed
 * alike (total = shape.n_nodes).  q, k, v are F32 or BF16, out F32, F16 or
 * BF16; d_k is 32, 64 or 128, d_v a multiple of 16 up to 256.  alpha is at
 * least 0; a gate of 0 forgets the state before it, of any finite size, and has
 * its gradient all the same.  (In the gradient of a gate below 2^-60, another one
 * below 2^-60 in its chunk counts as 0.)
 *
 * gdn_scan_forward starts sequence b from state[slot(b)] (only read), or from
 * zeros where `state` is NULL, and writes `out` and the fp32 state after the
 * last token to final_state[b] (nullable; may be `state` itself when state_slot
 * is NULL).  A sequence without tokens has its initial state as its final one.
 * A slot outside [0, n_slots) skips the sequence (its outputs are left as they
 * were, and so are its gradients in the backward pass) and sets *status.
 *
 * `tape` (gdn_scan_tape_bytes bytes) receives what the backward pass needs
 * besides the inputs: the state before every 64-token chunk, the delta rule's
 * errors, the chunks' triangular inverses and the gates, about 5.6 MB per 64
 * tokens at 48 value heads and d_k = d_v = 128.  Without one (NULL) the
 * workspace holds it during the call.
 *
 * gdn_scan_backward takes the same shape, cu_seqlens and inputs, the tape as
 * gdn_scan_forward left it, the gradients dout (out_dtype) of the outputs and
 * dfinal (nullable: zeros) of the final states, and writes the gradients dq,
 * dk, dv (qkv_dtype; those of a q/k head are summed over its value heads in
 * fp32), dalpha, dbeta (fp32) and dstate [B][h_v][d_v][d_k] (nullable) of the
 * inputs and the initial states.  The tape is only read: a second backward pass
 * over it gives the same result.  Nothing is accumulated with atomics; results
 * repeat bit for bit.
 *
 * Apart from final_state = state, and dstate = dfinal, no output overlaps an
 * input or another output.  A NaN or an infinity in q, k, v, alpha, beta, dout,
 * dfinal or a state leaves nothing finite of what the rule computes from it, and
 * may reach other results of its sequence and heads: outputs from the start of
 * its 64-token chunk on, gradients of the whole sequence (one in dout: up to the
 * end of its chunk).  Other sequences and heads do not see it.
 *
 * tape, workspaces, out, dout, dv, dfinal and dstate are 16-byte aligned, the
 * other outputs 4-byte.  The workspaces' contents on entry are ignored; calls that
 * share one are ordered on one stream.
 */
size_t gdn_scan_tape_bytes(const gdn_shape* shape, const int32_t* cu_seqlens);
size_t gdn_scan_forward_workspace_bytes(const gdn_shape* shape, const int32_t* cu_seqlens, int32_t with_tape);
int gdn_scan_forward(const gdn_shape* shape, const int32_t* cu_seqlens, const void* q, const void* k, const void* v,
                     const float* alpha, const float* beta, const float* state, const int32_t* state_slot, void* out,
                     float* final_state, void* tape, size_t tape_bytes, void* workspace, size_t workspace_bytes,
                     int32_t* status, void* stream);
size_t gdn_scan_backward_workspace_bytes(const gdn_shape* shape, const int32_t* cu_seqlens);
int gdn_scan_backward(const gdn_shape* shape, const int32_t* cu_seqlens, const void* q, const void* k, const void* v,
                      const float* alpha, const float* beta, const void* tape, size_t tape_bytes, const void* dout,
                      const float* dfinal, void* dq, void* dk, void* dv, float* dalpha, float* dbeta, float* dstate,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * Around the rule in a layer: the input norm, the projections to q, k, v and the
 * output gate, the gated norm of the rule's outputs, the output projection.
 * Serving keeps the operands of the projections in 8 bits:
 *   activations  e4m3 codes [rows][width] and a scale byte for each GDN_GROUP
 *                channels of a row (the last group may be shorter), a power of
 *                two: byte b stands for 2^(b - 127), 255 for NaN (e8m0).  Scales
 *                are [rows][scale_stride] bytes, scale_stride a multiple of 4 and
 *                at least the number of groups; the bytes behind the last group
 *                are neither written nor used.
 *   weights      e4m3 codes [columns][inner] and a scale for each block of
 *                GDN_GROUP columns x GDN_GROUP inner channels (the last ones may
 *                be shorter), fp32 (GDN_F32) or a power of two as above (GDN_E8M0).
 * e4m3 is the OCP format: values up to 448, steps of 2^-3 of the power of two below
 * a value, 2^-9 at the least.  The codes a norm writes are y 2^-e to the nearest, ties to even, with the
 * smallest e from -126 on that leaves no |y| 2^-e of the group above 448.  A group
 * with a NaN or an infinity has scale byte 255 and codes NaN.  Codes and scales are those of
 * y in 64 bits, but where a product of y's first factors (the normed value, in the gated norm
 * with the weight) is below 2^-126 or overflows in fp32 and the next factor makes up for it.
 */
#define GDN_GROUP 128       /* channels that share a scale */
#define GDN_MAX_PARTS 8     /* outputs of one gdn_project call */
#define GDN_MAX_WIDTH 16384 /* channels of gdn_norm_forward and gdn_norm_backward */
#define GDN_E8M0 3          /* scale type of gdn_project: a power of two in a byte */

typedef struct gdn_norm_shape {
    int64_t rows;          /* tokens, 0 .. 2^31 - 1 */
    int64_t x_stride;      /* elements from one row of x (backward: of r) to the next, a multiple of 8, width .. 2^31 */
    int32_t width;         /* channels, a multiple of 8 up to GDN_MAX_WIDTH */
    int32_t dtype;         /* of x, out and dout: GDN_F32, GDN_BF16 or GDN_F16 */
    int32_t residual_dtype;/* of residual, residual_out, r, dresidual and dx */
    int32_t weight_dtype;
    int32_t scale_stride;  /* bytes from one row's scales to the next (ignored without codes) */
    float eps;             /* at least 0 */
    float weight_offset;   /* w0: 1 where weights are stored as differences from 1 */
} gdn_norm_shape;

/*
 * Root mean square norm with the residual's addition:
 *     r = x + residual, rounded to residual_dtype;  residual_out = r
 *     y = r / sqrt(mean_k r_k^2 + eps) * (w + w0)
 * The norm is of r as stored, so the backward pass needs nothing but r.  Without a
 * residual (NULL; residual_out is NULL then) r is x.  y goes to `out` (nullable, dtype)
 * and, or, to `codes` and `scales` (nullable, both or none).  Sums and products of `out`
 * are fp32.
 * residual, residual_out, out and codes are dense [rows][width]; residual_out may be
 * residual, and out may be a dense x (no other output overlaps an input).  x, residual,
 * residual_out, out and weight are 16-byte aligned, codes 8-byte, scales 4-byte.  A row
 * of zeros with eps = 0 is NaN; a NaN or an infinity in a row leaves nothing finite of
 * the channels that hold one and may reach its whole row, but no other.  Other rows may be
 * of any magnitude, subnormal ones with eps = 0 included: one whose squares leave fp32's
 * range is summed again, scaled.
 *
 * gdn_norm_backward: from dout [rows][width] (dtype) and r (residual_dtype; x itself, in
 * residual_dtype = dtype, where there was no residual)
 *     g = dout (w + w0),  s = 1 / sqrt(mean r^2 + eps)
 *     dx = dresidual + s g - r s^3 mean_k g_k r_k,   dweight = sum_rows dout r s
 * dx (residual_dtype; the gradient of x and of residual alike) may be dresidual
 * (nullable: zeros).  Sums and products are fp32; a sum of g r that leaves its range is formed
 * again, scaled.  dweight is fp32 [width]; its sums are taken in a fixed order
 * and repeat bit for bit.  With no rows it is zero.  dx and dweight are nullable.
 * `workspace`: gdn_norm_backward_workspace_bytes(shape) bytes, 16-byte aligned;
 * calls that share one are ordered on one stream.
 */
int gdn_norm_forward(const gdn_norm_shape* shape, const void* x, const void* residual, const void* weight,
                     void* residual_out, void* out, void* codes, void* scales, void* stream);
size_t gdn_norm_backward_workspace_bytes(const gdn_norm_shape* shape);
int gdn_norm_backward(const gdn_norm_shape* shape, const void* dout, const void* r, const void* weight,
                      const void* dresidual, void* dx, float* dweight, void* workspace, size_t workspace_bytes,
                      void* stream);

typedef struct gdn_gated_norm_shape {
    int64_t rows;          /* tokens, 0 .. 2^31 - 1; rows * ceil(h_v d_v / lcm(d_v, 128)) below 2^32 */
    int64_t x_stride;      /* elements from one row of x to the next, a multiple of 8, h_v d_v .. 2^31 */
    int64_t z_stride;      /* of z, likewise */
    int32_t h_v;           /* value heads, >= 1, at most 2^20 */
    int32_t d_v;           /* value channels: a multiple of 16 up to 256 */
    int32_t x_dtype;       /* of x and dx: GDN_F32, GDN_BF16 or GDN_F16 */
    int32_t z_dtype;       /* of z, out, dout and dz */
    int32_t weight_dtype;
    int32_t scale_stride;  /* bytes from one row's scales to the next (ignored without codes) */
    float eps;             /* at least 0 */
} gdn_gated_norm_shape;

/*
 * Gated norm of the rule's outputs, head by head:
 *     n = x / sqrt(mean_j x_j^2 + eps)  over the d_v channels of a head
 *     y = n w silu(z),   silu(z) = z / (1 + e^-z)
 * x is `out` of a verify, prefill or scan ([rows][h_v][d_v]), z the gate's projection,
 * weight [d_v].  y goes to `out` (nullable, z_dtype) and, or, to `codes` and `scales`
 * (nullable, both or none), [rows][h_v d_v] as the output projection reads them.  out
 * may be a dense z, or a dense x of its type.  A NaN or an infinity in x or z may reach its whole head,
 * and makes its group's scale NaN, but no other head's `out`.  Heads and gates may be of any
 * finite magnitude, as the norm's rows.
 *
 * gdn_gated_norm_backward: with s = 1 / sqrt(mean x^2 + eps), a = 1 / (1 + e^-z) and
 * g = dout w silu(z)
 *     dx = s g - x s^3 mean_j g_j x_j,   dz = dout n w a (1 + z (1 - a)),
 *     dweight = sum over rows and heads of dout n silu(z)   (fp32 [d_v])
 * dx, dz and dweight are nullable.  Alignment, the sums and the workspace are
 * those of gdn_norm_backward; dz may be dout or z, dx may be x (the same rows, dense).
 */
int gdn_gated_norm_forward(const gdn_gated_norm_shape* shape, const void* x, const void* z, const void* weight,
                           void* out, void* codes, void* scales, void* stream);
size_t gdn_gated_norm_backward_workspace_bytes(const gdn_gated_norm_shape* shape);
int gdn_gated_norm_backward(const gdn_gated_norm_shape* shape, const void* dout, const void* x, const void* z,
                            const void* weight, void* dx, void* dz, float* dweight, void* workspace,
                            size_t workspace_bytes, void* stream);

/* One output of gdn_project: columns [tokens][columns], rows `stride` elements apart. */
typedef struct gdn_project_part {
    void* data;       /* aligned to its element size; 16 bytes for the widest stores */
    int64_t stride;   /* at least columns */
    int32_t columns;  /* >= 1; of all parts together N, at most 2^27 */
    int32_t reserved; /* 0 */
} gdn_project_part;

typedef struct gdn_project_shape {
    int64_t tokens;       /* M >= 0, below 2^31; ceil(M / 256) * ceil(N / 256) at most 2^21 */
    int64_t a_stride;     /* bytes from one row of a to the next, a multiple of 16, inner .. 2^22 */
    int64_t w_stride;     /* of w, likewise */
    int32_t inner;        /* K, a multiple of 16, at least 16 */
    int32_t a_scale_stride; /* bytes from one row of a_scales to the next, a multiple of 4, ceil(K / 128) .. 2^22 */
    int32_t w_scale_stride; /* GDN_E8M0: likewise; GDN_F32: elements, at least ceil(K / 128) */
    int32_t w_scale_dtype;  /* GDN_F32 or GDN_E8M0 */
    int32_t out_dtype;      /* GDN_BF16 or GDN_F16 */
} gdn_project_shape;

/*
 * Projections of 8-bit activations by 8-bit weights,
 *     y[m][n] = sum_g 2^(a_scales[m][g] - 127) w_scale[n / 128][g] sum_{k in group g} a[m][k] w[n][k],
 * the columns n = 0 .. N - 1 (N = the parts' columns together) cut into parts[0],
 * parts[1], ...: one call writes q, k, v, the gate z and the rest in the layouts the
 * verify, the prefill and the gated norm take.  a [M][K] and w [N][K] are e4m3 codes
 * with the scales above (a: codes and scales of gdn_norm_forward or
 * gdn_gated_norm_forward), 16-byte aligned; a_scales and GDN_E8M0 scales are
 * 4-byte aligned.  No output overlaps an input or another output.
 *
 * Groups are summed in fp32, in an order that depends on the shape alone, so results
 * repeat bit for bit; the matrix instruction adds the products within a group with
 * about 17 bits below the largest (1.5e-5 of the 2-norm of y for normal operands, 2.3e-5
 * for a layer's), which is why y is bf16 or f16 and not fp32.  f16 outputs above 65504 become infinite.  A
 * scale of NaN, or a NaN code, makes NaN every y that it has part in.  Scales may be of
 * any magnitude: a group's sum is formed with both, so it overflows where y does.
 */
int gdn_project(const gdn_project_shape* shape, const void* a, const void* a_scales, const void* w,
                const void* w_scales, const gdn_project_part* parts, int32_t n_parts, void* stream);

/*
 * Plan (and validate) the walk gdn_verify_tree takes through one tree.
 * Host-only; enqueues nothing.  Writes n_nodes steps to `walk` (host,
 * uint16 each): bits 0-4 the node, bit 5 "restore the parent's state from
 * fork slot bits 6-9 first", bit 10 "save the state to fork slot bits 11-14
 * after the node".  Nodes are visited depth first, children in index order;
 * a step without bit 5 continues from the previous step's state (node 0 from
 * the cached state).  *fork_slots receives the number of slots the walk
 * needs (at most GDN_MAX_TREE_DEPTH - 1).  Returns GDN_ERR_PARENT for an
 * invalid tree, with the rules of gdn_verify_tree.
 */
int gdn_tree_walk(const int32_t* parent, int32_t n_nodes, uint16_t* walk, int32_t* fork_slots);

/* Human-readable name of a gdn_status code (static storage). */
const char* gdn_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
