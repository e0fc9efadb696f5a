/*
 * hyb_spec.h -- speculative decoding on the hybrid_v2 cache: attention for a
 * tree of drafted tokens, and the block tables and slot maps of a batch built
 * on the GPU from request lengths.
 *
 * The cache, its layouts and the conventions of every call are those of
 * hyb_kv.h (device pointers are the caller's, work is enqueued on `stream`,
 * host errors are returned and enqueue nothing, device errors go to the sticky
 * status word).  Same library (libhybkv.so).  The web page that hyb_kv.h cites
 * has no counterpart of these calls: its decode step has one query per
 * sequence, and it takes the block table as given.
 *
 * One verification step of a batch:
 *   1. hyb_pool_resize   blocks for the lengths the step may reach;
 *   2. hyb_tree_attn     every drafted node's query over the cache and the
 *                        node's ancestors (the cache is not changed);
 *   3. hyb_kv_append     the K and V of the accepted path.
 * hyb_slot_map tells where the tokens of any packed selection live, for code
 * that moves or inspects cached tokens itself.
 */
#ifndef HYB_SPEC_H
#define HYB_SPEC_H

#include <stddef.h>
#include <stdint.h>

#include "hyb_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* device status codes of these calls, beside those of hyb_kv.h */
#define HYB_STATUS_POOL 7     /* hyb_pool_resize: the pool has too few free blocks (that sequence left
                                 unchanged), or its counts contradict each other (nothing changed) */
#define HYB_STATUS_BAD_TREE 8 /* hyb_tree_attn: n_tree[b] < 0 or > max_tree; b skipped */

/* Most nodes of one sequence's tree (a mask is one 64-bit word). */
#define HYB_MAX_TREE 64

/*
 * Attention for a tree of drafted tokens.  Node t of sequence b (t <
 * n_tree[b]) has a query of its own; it attends every token of the sequence's
 * cache and the drafted nodes its mask names:
 *   S(b,t) = cached positions 0..seq_lens[b]-1, and the nodes j < n_tree[b]
 *            with bit j of tree_mask[b][t] set,
 *   out[b][t][h] = sum_j softmax_j(z) V_j over S(b,t),
 *   z_j = softmax_scale * (q[b][t][h] . K_j),
 * K_j, V_j of kv head h / (Hq/Hkv) as in hyb_decode_attn for cached positions,
 * the rows of k_tree / v_tree for nodes.  A node attends itself only if its
 * own bit is set.  An empty S gives out = 0 and lse = -inf.  A value of a node
 * that a query does not attend never reaches it, whatever it is (infinities
 * and NaN included).
 *   q        device FP16 [batch][max_tree][Hq][D], 16-byte aligned.
 *   k_tree, v_tree  device FP16 [batch][max_tree][Hkv][D] (the layout of
 *            hyb_kv_append's k_new / v_new), 16-byte aligned.
 *   tree_mask  device uint64 [batch][max_tree], 8-byte aligned, or NULL: the
 *            drafted tokens are a chain (node t attends nodes 0..t).  Bits at
 *            and above n_tree[b] are ignored.
 *   n_tree   device int32 [batch], each in [0, max_tree], or NULL: max_tree
 *            nodes for every sequence.
 *   max_tree 1..HYB_MAX_TREE.
 *   softmax_scale  finite.
 *   workspace  at least hyb_tree_workspace_bytes() bytes, 16-byte aligned; its
 *            contents need no preparation.  Calls that share it must not
 *            overlap on the GPU.
 *   out      device FP16 [batch][max_tree][Hq][D] (round to nearest even),
 *            16-byte aligned.  Rows t >= n_tree[b] are left as they were.  It may
 *            be q itself; otherwise out and lse_out overlap no input.
 *   lse_out  device FP32 [batch][max_tree][Hq], natural log, or NULL; likewise.
 * The cache is only read.  Nothing is sized by the lengths: a captured call
 * may be replayed after the sequences grew.
 * Device errors: HYB_STATUS_BAD_TREE (that sequence's rows left as they were),
 * HYB_STATUS_SEQ_LEN (seq_lens[b] < 0 or beyond the block table: its rows
 * become 0 and -inf), HYB_STATUS_BAD_BLOCK (that block's tokens are not
 * attended), HYB_STATUS_TIMEOUT (a bounded wait ran out: rows in work at that
 * time are undefined).
 * Returns HYB_OK, HYB_ERR_INVALID_VALUE (descriptor, null or misaligned
 * pointer, max_tree < 1, softmax_scale not finite), HYB_ERR_UNSUPPORTED
 * (max_tree > HYB_MAX_TREE, or hyb_check_desc's cases), HYB_ERR_WORKSPACE or
 * HYB_ERR_CUDA.
 */
int hyb_tree_attn(const hyb_cache_desc *desc, const void *q, const void *k_tree, const void *v_tree,
                  const uint64_t *tree_mask, const int32_t *n_tree, int32_t max_tree, float softmax_scale,
                  void *workspace, size_t workspace_bytes, void *out, float *lse_out, hyb_stream_t stream);

/* Bytes of workspace hyb_tree_attn needs (0 with invalid arguments; never 0
 * otherwise).  It depends on the GPU's SM count, not on the lengths. */
size_t hyb_tree_workspace_bytes(const hyb_cache_desc *desc, int32_t max_tree);

/*
 * A pool of physical blocks and the block tables of a batch (host struct; the
 * pointers inside are device memory).  The free blocks are a ring: entry i of
 * the free list (i < count) is ring[(head + i) % num_phys_blocks], state =
 * {head, count}.  Sequence b holds n_blocks[b] blocks, named by the first
 * n_blocks[b] entries of its table row; the other entries mean nothing.  A
 * block is either in the ring or held once, so count + sum n_blocks <=
 * num_phys_blocks.
 */
typedef struct hyb_pool_desc {
  int32_t batch;              /* sequences, >= 1 */
  int32_t max_blocks_per_seq; /* columns of block_table, >= 1 */
  int32_t num_phys_blocks;    /* >= 1 */
  int32_t hot_tokens;         /* 16, 32, 64 or 128: these tokens need no block */
  int32_t block_size;         /* 32, 64 or 128 */
  int32_t reserved;           /* set to 0 */
  int32_t *ring;              /* device int32 [num_phys_blocks] */
  int32_t *state;             /* device int32 [2]: head, count */
  int32_t *n_blocks;          /* device int32 [batch] */
  int32_t *block_table;       /* device int32 [batch][max_blocks_per_seq] */
  int32_t *status;            /* device int32, 0 = ok */
} hyb_pool_desc;

/* Host-only check of a pool descriptor: HYB_OK, HYB_ERR_INVALID_VALUE or
 * HYB_ERR_UNSUPPORTED, by the rules of hyb_check_desc. */
int hyb_check_pool(const hyb_pool_desc *pool);

/*
 * Give every sequence the blocks that lens[b] tokens need: want_b =
 * ceil(max(0, lens[b] - hot_tokens) / block_size).  lens[b] is any length the
 * caller wants room for (0: the sequence ended); it need not be seq_lens.
 *   - Sequences that need more take blocks from the head of the free ring, in
 *     the order of b, then of the table column.  Sequence b gets its blocks if
 *     the free blocks cover its need and that of every sequence before it;
 *     otherwise it is left unchanged and HYB_STATUS_POOL is recorded.
 *   - Sequences that need fewer give their last blocks back at the tail of the
 *     ring, in the same order.  A block given back is free for the next call,
 *     not for this one.
 * The result is written to `to`: table rows (entries from want_b on are -1),
 * counts and ring state.  `to` is the pool itself (NULL or the same pointers:
 * in place), or a successor: a pool of the same sizes and the same ring whose
 * state, n_blocks and block_table are other memory, so that the next step's
 * tables can be built while this step still reads `from` (a call may mix: each
 * of the three is either the same pointer or memory that overlaps none of
 * from's).  Only one line of successors is valid: a later call on `from`
 * hands out the same ring entries again.
 *   lens       device int32 [batch].
 *   workspace  at least hyb_pool_workspace_bytes() bytes, 16-byte aligned,
 *              zero-filled before its first use and left ready for the next
 *              call; calls that share it must not overlap on the GPU.
 * Device errors, recorded in to's status word: HYB_STATUS_SEQ_LEN (lens[b] <
 * 0), HYB_STATUS_CAPACITY (more blocks than columns, or n_blocks[b] outside
 * [0, columns]): that sequence is left unchanged; HYB_STATUS_POOL;
 * HYB_STATUS_BAD_BLOCK (an entry given back, or taken from the ring, is not a
 * block number; the pool is then damaged and must be rebuilt).
 * The result does not depend on the launch.  Returns HYB_OK,
 * HYB_ERR_INVALID_VALUE, HYB_ERR_UNSUPPORTED, HYB_ERR_WORKSPACE or
 * HYB_ERR_CUDA.
 */
int hyb_pool_resize(const hyb_pool_desc *from, const hyb_pool_desc *to, const int32_t *lens,
                    void *workspace, size_t workspace_bytes, hyb_stream_t stream);

/* Bytes of workspace hyb_pool_resize needs (0 with an invalid descriptor). */
size_t hyb_pool_workspace_bytes(const hyb_pool_desc *pool);

/* what hyb_slot_map writes for a token outside its sequence */
#define HYB_SLOT_NONE (-1)

/*
 * Where packed tokens live.  n_tok[b] tokens of each sequence, positions
 * first[b] .. first[b] + n_tok[b] - 1, are packed one sequence after the other
 * (cu[b] = sum of n_tok before b).  For the token at position p of sequence b,
 * a sequence of lens[b] tokens, slots[] receives
 *   block_table[b][p / BLK] * BLK + p % BLK   cold: p < lens[b] - HOT,
 *   -2 - (b * HOT + p % HOT)                  in the hot ring,
 *   HYB_SLOT_NONE                             p < 0 or p >= lens[b], or the
 *                                             block has no valid table entry.
 *   lens, n_tok  device int32 [batch]; first  device int32 [batch] or NULL
 *              (all 0).  A negative lens[b] is an empty sequence.
 *   max_total  entries of slots; tokens beyond it are dropped
 *              (HYB_STATUS_CAPACITY) and cu stops there.
 *   cu         device int32 [batch + 1] or NULL.
 *   slots      device int64 [max_total], 8-byte aligned (NULL only with
 *              max_total 0).  Entries at and behind cu[batch] are left as they
 *              were.
 * Reads the pool's block_table and geometry only (its ring, state and n_blocks
 * may be NULL).  Device errors: HYB_STATUS_BAD_N_NEW (n_tok[b] < 0, taken as
 * 0), HYB_STATUS_CAPACITY, HYB_STATUS_BAD_BLOCK (a table entry out of range, or
 * a position beyond the table).  Returns as hyb_pool_resize.
 */
int hyb_slot_map(const hyb_pool_desc *pool, const int32_t *lens, const int32_t *first, const int32_t *n_tok,
                 int32_t max_total, int32_t *cu, int64_t *slots, hyb_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* HYB_SPEC_H */
