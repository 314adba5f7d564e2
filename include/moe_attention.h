/*
 * moe_attention.h -- C ABI of the attention half of a decoder block, beside
 * the MoE layer of moe.h, for MI355X (gfx950).
 *
 * Three operators that run in this order on one HIP stream, for prompts and
 * for single tokens:
 *
 *   moe_fp8_linear     projections with E4M3 weights, one scale per 128 x 128
 *                      block ("DeepSeek-V4-Flash" dense weights: FP8 128 x 128
 *                      blocks)
 *   moe_qk_norm_rope   RMS norm and rotary position of every query and key head
 *   moe_attention      packed causal softmax attention with grouped heads
 *
 * The conventions of moe.h hold: device pointers unless a comment says host,
 * the caller owns every buffer, calls only enqueue kernels on `stream` and
 * never allocate, synchronise, print or abort; arguments are validated on the
 * host before anything is enqueued; status codes are moe_status; bf16 tensors
 * are uint16_t bit patterns; results are deterministic (no floating-point
 * atomics, every reduction in a fixed order).  The operators are inference
 * operators, like the layer: there is no backward pass.
 */
#ifndef MOE_ATTENTION_H
#define MOE_ATTENTION_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ fp8 linear
 *
 * y[t, n] = bf16( sum_b  sx[t, b] * sw[n / 128, b] * sum_{k in block b} cx[t, k] * w[n, k] )
 *
 * over the blocks b of 128 consecutive columns k of K (the last one partial
 * when 128 does not divide K).  w is E4M3 (OCP FP8 without infinities: bias 7,
 * largest value 448, codes 0x7f and 0xff NaN), row-major [N, K], with one
 * scale per 128 x 128 block, row-major [ceil(N / 128), ceil(K / 128)]:
 *   MOE_SCALE_E8M0  uint8, value 2^(e - 127) (e = 255 NaN), as everywhere in moe.h
 *   MOE_SCALE_F32   float32
 * x is bf16 and is quantised by the call, per token and block, in the same
 * kind of scale.  With a = max(2^-100, max |x| over the block):
 *   MOE_SCALE_E8M0  sx = the least power of two with a / sx <= 448; cx = e4m3(x / sx)
 *   MOE_SCALE_F32   sx = a / 448; cx = e4m3(x * (448 / a)), each float32 operation rounded once
 * where e4m3 rounds to nearest even.  A token that holds an infinity or a NaN
 * gives NaN in all of its outputs.  Products are summed in float32 on the fp8
 * matrix cores, which align each eight neighbouring products (columns 8 j .. 8 j +
 * 7) to the largest of them and drop what lies below 2^-13 of its power of two
 * before they add them up (measured on gfx950; half a code of E4M3 is 2^-4 of
 * a value); y is rounded once.
 *
 * x         bf16 [T, K], rows x_stride elements apart (a multiple of 8, at least K), 16-byte aligned
 * w         E4M3 bytes [N, K], contiguous, 16-byte aligned
 * w_scale   as above (float32: 4-byte aligned)
 * y         bf16 [T, N] out, rows y_stride elements apart (at least N), 2-byte aligned;
 *           must not overlap x, w, w_scale or ws
 * ws        at least moe_fp8_linear_workspace_size(T, N, K) bytes, 256-byte aligned
 * Requirements: T <= MOE_MAX_TOKENS; N, K <= MOE_MAX_DIM, both positive, K a
 * multiple of 16 (MOE_ESHAPE otherwise).
 */
#define MOE_SCALE_E8M0 0
#define MOE_SCALE_F32 1

size_t moe_fp8_linear_workspace_size(int32_t T, int32_t N, int32_t K);
int moe_fp8_linear(const uint16_t* x, int64_t x_stride, int32_t T, int32_t K, const uint8_t* w, const void* w_scale,
                   int32_t scale_type, int32_t N, uint16_t* y, int64_t y_stride, void* ws, size_t ws_bytes,
                   void* stream);

/* ------------------------------------------------------------------ heads
 * A bf16 tensor [rows, heads, head_dim] with unit stride inside a head: row r
 * of head h starts at base + r * row_stride + h * head_stride (elements).  Both
 * strides are positive multiples of 8, base is 16-byte aligned.  So the three parts
 * of a fused q|k|v projection, or a cache in either order of heads and rows,
 * are used where they are.
 */
typedef struct moe_heads {
  uint16_t* base;
  int64_t row_stride;
  int64_t head_stride;
} moe_heads;

/* ------------------------------------------------------------------ norm and rotation
 *
 * For every row t and head of q (and of k):
 *   n = x * w / sqrt(mean(x^2) + eps)            (w = 1 where the weight is NULL)
 *   the pairs (a, b) of n[rot_offset .. rot_offset + rot_dim) are rotated by
 *   the angle of row t:  a' = a c - b s,  b' = b c + a s
 * and the rest of n is passed through; float32 throughout, rounded once.  Pair
 * j is (n[rot_offset + j], n[rot_offset + rot_dim / 2 + j]), or, interleaved,
 * (n[rot_offset + 2 j], n[rot_offset + 2 j + 1]).  Its cosine and sine are
 * cos_sin[p, j] and cos_sin[p, rot_dim / 2 + j] with p = positions[t]; a
 * position outside [0, n_positions) gives NaN in the rotated elements.
 *
 * q, k          [T, q_heads | k_heads, head_dim]; k_heads = 0 leaves k out
 * q_weight, k_weight  float32 [head_dim], 16-byte aligned, or NULL
 * positions     int32 [T]; cos_sin float32 [n_positions, rot_dim], 16-byte aligned
 *               (both may be NULL when rot_dim = 0)
 * q_out, k_out  out; may be q and k themselves (in place) but must not otherwise overlap them
 * Requirements: head_dim a multiple of 8 up to 512; rot_dim a multiple of 16
 * (0 = no rotation), rot_offset a multiple of 8, rot_offset + rot_dim <=
 * head_dim; 1 <= q_heads, 0 <= k_heads, q_heads + k_heads <= 1024, T * (q_heads +
 * k_heads) < 2^28, for a head_dim above 256 with the heads rounded up to a multiple of
 * four (MOE_ESHAPE otherwise); eps >= 0 (MOE_EINVAL).
 */
int moe_qk_norm_rope(const moe_heads* q, int32_t q_heads, const moe_heads* k, int32_t k_heads, int32_t T,
                     int32_t head_dim, const float* q_weight, const float* k_weight, float eps,
                     const int32_t* positions, const float* cos_sin, int32_t n_positions, int32_t rot_dim,
                     int32_t rot_offset, int32_t interleaved, const moe_heads* q_out, const moe_heads* k_out,
                     void* stream);

/* ------------------------------------------------------------------ attention
 *
 * B sequences are packed along the rows of q: sequence b owns rows cu_q[b] ..
 * cu_q[b + 1] - 1 (Lq of them) and attends to rows kv_start[b] .. kv_start[b] +
 * kv_len[b] - 1 (Lk of them) of k and v.  Query i of a sequence sees its keys j
 * <= i + Lk - Lq (causal != 0: the last query sees every key) or all of them:
 *   out[i] = sum_j softmax_j(scale * q[i] . k[j]) v[j]
 *   lse[i] = log sum_j exp(scale * q[i] . k[j])             (natural logarithm)
 * Query head h reads key head h / (q_heads / kv_heads).  Scores, softmax and
 * sums are float32; the weights are rounded to bf16 for the matrix cores, out
 * is rounded once.  A row that sees no key (Lk = 0, or Lq > Lk and i < Lq - Lk)
 * gives zeros and lse = -infinity, and so does one whose every score is -infinity.
 * Keys and values that a row does not see never reach it, infinities and NaN included.
 *
 * A prompt: kv_start = kv_len = NULL (the keys and values of a sequence are the
 * rows cu_q names).  A chunk of a prompt, or a single token, over a cache:
 * kv_start[b] is the cache row where b begins and kv_len[b] its length,
 * the new rows included.
 *
 * cu_q int32 [n_seqs + 1], kv_start and kv_len int32 [n_seqs]: device arrays,
 * read by the kernels.  Ranges are cut to q's q_rows and k's kv_rows rows, so
 * no value in them reads or writes outside the tensors; rows of out and lse that belong to no
 * sequence are left as they are.  max_q and max_kv are the caller's bounds on
 * Lq and Lk (host values; they choose kernels, grids and splits): rows of a
 * sequence past max_q get no output, keys past max_kv are not seen.  Bounds and cuts
 * of the keys take keys away and move nothing: Lk above is kv_len[b] (Lq) as given,
 * Lq the length that cu_q gives inside q's rows.
 *
 * The struct is a host object, read during the call.
 */
typedef struct moe_attn {
  uint32_t abi_version;   /* MOE_ABI_VERSION */
  int32_t head_dim;       /* 64, 128 or 256 */
  int32_t q_heads;        /* a positive multiple of kv_heads, at most 1024 */
  int32_t kv_heads;
  int32_t n_seqs;         /* B, at most 65536 */
  int32_t q_rows;         /* rows of q and out, at most MOE_MAX_TOKENS */
  int32_t kv_rows;        /* rows of k and v */
  int32_t max_q;          /* 0 .. q_rows */
  int32_t max_kv;         /* 0 .. kv_rows */
  int32_t causal;         /* 0 or 1 */
  float scale;            /* > 0, at most 2^127 */
  int32_t reserved;       /* 0 */
  moe_heads q, k, v, out; /* out: must not overlap the others; row_stride of k and v at most 2^23 */
  const int32_t* cu_q;
  const int32_t* kv_start; /* NULL: cu_q[b] */
  const int32_t* kv_len;   /* NULL: Lq (both or neither) */
  float* lse;              /* float32 [q_rows, q_heads] out, or NULL */
} moe_attn;

/* Fill a descriptor for contiguous q, k, v, out of the given shape
 * ([rows, heads, head_dim]), causal, scale 1 / sqrt(head_dim), max_q = q_rows,
 * max_kv = kv_rows, no kv_start, kv_len and lse.  MOE_EINVAL for a NULL
 * pointer; the values themselves are checked by moe_attention. */
int moe_attn_init(moe_attn* a, const uint16_t* q, const uint16_t* k, const uint16_t* v, uint16_t* out,
                  const int32_t* cu_q, int32_t n_seqs, int32_t q_rows, int32_t kv_rows, int32_t q_heads,
                  int32_t kv_heads, int32_t head_dim);

/* Workspace of a call: depends on the shape fields only (q_rows, max_q,
 * max_kv, n_seqs, heads, head_dim); 0 for a shape that needs none or is not supported. */
size_t moe_attention_workspace_size(const moe_attn* a);

/* ws: at least moe_attention_workspace_size(a) bytes, 256-byte aligned (may be
 * NULL when that is 0). */
int moe_attention(const moe_attn* a, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTENTION_H */
