/*
 * moe_paged.h -- C ABI of a key/value cache in pages, beside the attention half
 * of moe_attention.h, for MI355X (gfx950).
 *
 * The keys and values of a sequence lie in pages of page_size tokens, anywhere
 * in one pool; a row of the page table names them in order.  Three operators:
 *
 *   moe_paged_append     new keys, normed and rotated on the way, and values
 *                        into their pages; the queries of the same tokens
 *                        normed and rotated too; per page and head the smallest
 *                        and largest key element of every column
 *   moe_paged_attention  causal softmax attention over the pages; groups of
 *                        sequences may share a prefix, which is then read once
 *                        for all their rows; or, with a list of blocks per token
 *                        and key head, attention over those pages alone
 *   moe_select_blocks    that list: the pages whose bounds promise the largest
 *                        products with the token's queries
 *
 * The conventions of moe_attention.h hold (device pointers, caller-owned
 * buffers, host-side refusals, deterministic results, bf16 as uint16_t, no
 * backward pass).
 */
#ifndef MOE_PAGED_H
#define MOE_PAGED_H

#include "moe_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A bf16 tensor [n_pages, page_size, kv_heads, head_dim] with unit stride inside a
 * head: slot s of head h in page p starts at base + p * page_stride + s *
 * row_stride + h * head_stride (elements).  The strides are positive multiples of
 * 8, row_stride at most 2^22, base is 16-byte aligned. */
typedef struct moe_pages {
  uint16_t* base;
  int64_t page_stride;
  int64_t row_stride;
  int64_t head_stride;
} moe_pages;

/* The sequences of a call, packed along the rows of q (and of k and v), and
 * their pages.  Sequence b owns rows cu_q[b] .. cu_q[b + 1] - 1 (Lq of them)
 * and holds Lk = kv_len[b] tokens, these rows' included: row i of it is at
 * position i + Lk - Lq.  The token at position p is in slot p % page_size of page
 * page_table[b, p / page_size].
 *
 * cu_q int32 [n_seqs + 1], kv_len int32 [n_seqs], page_table int32 [n_seqs,
 * table_pages] with rows table_stride elements apart: device arrays, read by the
 * kernels.  Row ranges are cut to the q_rows rows there are; positions below 0 or
 * past the table, and entries of the table outside 0 .. n_pages - 1, name no page:
 * nothing is stored to them and no row sees them.  So no value in these arrays
 * reads or writes outside the tensors. */
typedef struct moe_paged {
  uint32_t abi_version; /* MOE_ABI_VERSION */
  int32_t head_dim;     /* 64, 128 or 256 */
  int32_t q_heads;      /* a positive multiple of kv_heads, at most 1024 (moe_paged_append: or 0) */
  int32_t kv_heads;
  int32_t n_seqs;       /* at most 65536 */
  int32_t q_rows;       /* at most MOE_MAX_TOKENS */
  int32_t n_pages;      /* of the cache */
  int32_t page_size;    /* 16, 32, 64 or 128 */
  int32_t table_pages;  /* of a row of the table; table_pages * page_size < 2^30 */
  int32_t reserved;     /* 0 */
  int64_t table_stride; /* at least table_pages */
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* page_table;
} moe_paged;

/* ------------------------------------------------------------------ append
 *
 * For every row t of a sequence, at position p:
 *   k_pages(p) = rotate(norm(k[t], k_weight), pos(t)),  v_pages(p) = v[t],
 *   q_out[t] = rotate(norm(q[t], q_weight), pos(t))
 * with norm and rotation as in moe_qk_norm_rope (norm = 0: none), pos(t) =
 * positions[t], or p where positions is NULL; a position outside [0, n_positions)
 * gives NaN in the rotated elements.  q is done for every row of a sequence, also
 * where its page is none.  Rows of no sequence are left as they are.
 *
 * bounds, bf16 [n_pages, 2, kv_heads, head_dim] contiguous, or NULL: after the
 * call, [page, 0] and [page, 1] are the smallest and largest of what they were
 * and of the stored keys that the call brought to the page, in each column; what
 * they were does not count where the call stored to slot 0.  NaN does not count;
 * a column with nothing that counts is +infinity, -infinity.  So the bounds hold
 * for every key in a page that was filled from slot 0 on.
 *
 * Two rows that name the same slot, or sequences that bring tokens to one page
 * in the same call, race: the caller gives every sequence pages of its own to
 * write to.  q_out may be q itself; the outputs must not otherwise overlap the inputs.
 */
typedef struct moe_append {
  moe_paged p;
  int32_t norm; /* 0 or 1 */
  float eps;    /* >= 0 */
  int32_t n_positions;
  int32_t rot_dim;     /* a multiple of 16 (0: no rotation) */
  int32_t rot_offset;  /* a multiple of 8; rot_offset + rot_dim <= head_dim */
  int32_t interleaved; /* 0 or 1 */
  moe_heads q, q_out;  /* [q_rows, q_heads, head_dim]; q_heads = 0 leaves q out */
  moe_heads k, v;      /* [q_rows, kv_heads, head_dim] */
  moe_pages k_pages, v_pages;
  uint16_t* bounds;
  const float* q_weight; /* float32 [head_dim], 16-byte aligned, or NULL; NULL without norm */
  const float* k_weight;
  const int32_t* positions; /* int32 [q_rows], or NULL */
  const float* cos_sin;     /* float32 [n_positions, rot_dim], 16-byte aligned; may be NULL when rot_dim = 0 */
} moe_append;

/* At most 2^24 - 1 blocks of threads (MOE_ESHAPE otherwise): kv_heads * min(q_rows, q_rows /
 * page_size + 2 * min(n_seqs, q_rows)) + q_rows * q_heads * head_dim / 2048. */
int moe_paged_append(const moe_append* a, void* stream);

/* ------------------------------------------------------------------ attention
 *
 * Row i of a sequence sees its keys j <= i + Lk - Lq:
 *   out[i] = sum_j softmax_j(scale * q[i] . k[j]) v[j],  lse[i] = log sum_j exp(scale * q[i] . k[j])
 * with everything else (grouped heads, rounding, rows that see nothing, hidden
 * values) as in moe_attention.
 *
 * Shared prefixes.  cu_group int32 [n_groups + 1] (device) cuts the sequences into
 * groups of consecutive ones; the first prefix_len[g] keys of all sequences of
 * group g are the same, and in the same pages where they fill pages, so these are
 * read through the table row of the group's first sequence, once for all rows: that row names
 * all of them, also where the sequence itself is shorter.  (A
 * sequence shorter than prefix_len holds the first of these pages, the last in part.)
 * n_groups = 0 (cu_group and prefix_len may then be NULL), or sequences outside
 * every group: no shared prefix.  The result does not depend on the grouping but
 * for the order of its sums.
 *
 * Blocks.  blocks int32 [q_rows, kv_heads, n_blocks] (device), n_blocks > 0: row i sees a key j of key
 * head h only if j / page_size is among blocks[i, h, :].  Entries below 0, or past the row's
 * last page, name no block; a block named twice counts once.  n_blocks = 0: every block.  Not
 * together with groups.
 *
 * max_q bounds Lq; max_prefix bounds prefix_len; max_kv bounds the keys of a
 * sequence behind its prefix (all of them without groups): host values that
 * choose kernels, grids and splits.  Rows past max_q get no output, a prefix is cut to max_prefix,
 * keys from prefix + max_kv on are not seen; none of them moves the causal diagonal.
 */
typedef struct moe_paged_attn {
  moe_paged p;
  int32_t max_q;      /* 0 .. q_rows */
  int32_t max_kv;     /* 0 .. table_pages * page_size */
  int32_t n_groups;   /* 0 .. n_seqs */
  int32_t max_prefix; /* 0 .. table_pages * page_size */
  int32_t n_blocks;   /* 0 .. 1024; max_kv / page_size at most 32768 where it is not 0 */
  float scale;        /* > 0, at most 2^127 */
  moe_heads q, out;   /* out must not overlap the inputs */
  moe_pages k, v;
  const int32_t* cu_group;
  const int32_t* prefix_len;
  const int32_t* blocks;
  float* lse; /* float32 [q_rows, q_heads] out, or NULL */
} moe_paged_attn;

/* Depends on the shape fields only (heads, head_dim, n_seqs, q_rows, page_size, max_*,
 * n_groups, n_blocks); 0 for a shape that needs none or is not supported.  Not supported (MOE_ESHAPE), besides
 * what the fields say: q_rows * q_heads of 2^30 or more, and launches of 2^24 blocks of threads or more (one per
 * row tile, key head and piece of the keys; where keys come in pieces, one per 1024 / head_dim rows for their
 * join, one per row where the pieces are more than 16). */
size_t moe_paged_attention_workspace_size(const moe_paged_attn* a);

/* ws: at least that many bytes, 256-byte aligned (may be NULL when that is 0). */
int moe_paged_attention(const moe_paged_attn* a, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ selection
 *
 * For row i of a sequence and key head h, over the blocks (pages in the order of
 * the table) 0 .. n - 1 that hold a key the row sees:
 *   score(b) = sum over the columns d of Q+[d] * high[d] + Q-[d] * low[d],
 *   Q+ and Q- the sums over the query heads g of h of max(q[i, g], 0) and min(q[i, g], 0)
 * with low and high the bounds of b's page; this is at least the sum over g of
 * q[i, g] . k for every key k in the page.  Summed in float64; a score that is not
 * finite counts as the largest, that of a page that is none as the smallest.  The
 * first `first` and the last `last` blocks are taken, then those of the highest
 * scores, the lower block first where scores are equal, until there are n_blocks
 * or no more.  blocks[i, h, :] are their numbers, ascending, then -1.  Rows of no
 * sequence are left as they are.
 *
 * Every key of a block below the row's own last one is one that the row sees; last >= 1
 * takes that last one, so the choice never hangs on a later key.
 */
typedef struct moe_select {
  moe_paged p;
  int32_t max_q;
  int32_t max_kv;   /* a bound on Lk: keys from max_kv on are not seen; at most 32768 pages */
  int32_t n_blocks; /* 1 .. 1024 */
  int32_t first;    /* >= 0 */
  int32_t last;     /* >= 1; first + last <= n_blocks */
  int32_t reserved; /* 0 */
  moe_heads q;
  const uint16_t* bounds; /* as moe_paged_append keeps them, 16-byte aligned */
  int32_t* blocks;        /* out */
} moe_select;

/* Depends on the shape fields only (kv_heads, n_seqs, q_rows, page_size, max_q, max_kv); 0 for a shape
 * that needs none or is not supported. */
size_t moe_select_blocks_workspace_size(const moe_select* a);

/* ws: at least that many bytes, 256-byte aligned (may be NULL when that is 0).  q_rows * kv_heads < 2^23
 * (MOE_ESHAPE otherwise). */
int moe_select_blocks(const moe_select* a, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_PAGED_H */
