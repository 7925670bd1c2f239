/*
 * pi_attn.h -- C ABI of libpi, the attention side of a decode layer: rotary
 * positions, an 8-bit key/value cache with the attention that reads
 * it, and eviction from it.  These calls follow the conventions at the top
 * of pi.h, which includes this file (device pointers, streams, host checks before any
 * launch, bitwise reproducible results) with these additions:
 *  - Token rows [n_tok][n_heads][head_dim] are given as a pointer and two
 *    strides in ELEMENTS (between tokens, between heads), so a part of a
 *    fused projection needs no copy; a head's elements are contiguous, and
 *    every head starts on a 16-byte boundary.
 *  - The tokens of a call belong to sequences: those of sequence s are rows
 *    q_start[s] .. q_start[s + 1) (q_start: [n_seqs + 1] int32 on the device;
 *    NULL: every sequence has max_new (max_q) rows, one after the other).
 *    lens[s] (device int32) counts the tokens that sequence s holds, those of
 *    the call among them.
 *  - Values in device memory cannot be checked on the host.  The kernels
 *    check them before they use them: a sequence whose rows are not inside
 *    [0, n_tok], number more than max_new (max_q), or whose lens is negative
 *    or more than its table row (or max_len) holds is INVALID, and a page
 *    number outside [0, n_pages) is a BAD PAGE.  Each call says what becomes
 *    of them; nothing is read or written out of range.
 *  - PI_E_SHAPE also for sizes of which a launch could not hold the threads
 *    (2^32 - 1), before the first launch of the call.
 *
 * The cache.  A block is PI_KV_BLOCK tokens of one kv head of one sequence
 * and is stored as one page of 2 * PI_KV_BLOCK * head_dim bytes, the keys' half, then
 * the values' half, with an fp32 scale for each half.  A stored value is
 * scale * (code - 128), with scale = amax / 127 and code = 128 +
 * rint(127 x / amax) (ties to even, decided exactly), amax being the largest
 * magnitude of the block's half.  A half that holds an infinity or a NaN has the
 * scale NaN and reads as NaN throughout.  Order of the bytes in a half (t: the token
 * in the block, e: the element of the head), made so that 16 bytes of a lane
 * are a matrix-core operand and 64 lanes read 1 KB in a row:
 *   keys:   (((t / 16) * (head_dim / 64) + e / 64) * 4 + e / 16 % 4) * 256
 *             + t % 16 * 16 + e % 16
 *   values: (e / 32 * 4 + t % 16 / 4) * 256 + e % 16 * 16 + e / 16 % 2 * 8
 *             + t / 16 * 4 + t % 4
 * Slots of the last, partly filled block past its tokens hold code 128 (zero).
 * The rows of that block are also kept as they came (open), because its
 * amax, and so all of its codes, may change with every appended token.  */
#ifndef PI_ATTN_H_
#define PI_ATTN_H_

#include "pi.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens of a block.  */
#define PI_KV_BLOCK 32

typedef enum pi_rope_layout {
  PI_ROPE_HALF = 0,        /* pairs (i, i + rot / 2)                        */
  PI_ROPE_INTERLEAVED = 1  /* pairs (2 i, 2 i + 1)                          */
} pi_rope_layout;

/* Rotation of queries and keys, with an optional RMS norm of each head.  */
typedef struct pi_rope {
  int32_t head_dim;     /* multiple of 8, at most 256                       */
  int32_t rot;          /* rotated elements at the head's start; even, in [2, head_dim] */
  int32_t layout;       /* pi_rope_layout                                   */
  float scale;          /* the rotated elements are multiplied by it (1 for plain rotation) */
  float eps;            /* of the norms; >= 0                               */
  const double* freqs;  /* [rot / 2] turns per position (radians / 2 pi)    */
  const float* q_norm;  /* [head_dim] weight of the queries' norm; NULL: none */
  const float* k_norm;  /* [head_dim] weight of the keys' norm; NULL: none  */
} pi_rope;

/* y = x * w / sqrt(mean(x^2) + eps) where a norm weight is given, then each
 * pair (a, b) of the first rot elements becomes scale * (a cos - b sin,
 * b cos + a sin) at the angle 2 pi pos f.  The angle is reduced in 64 bits
 * (a far position times the fastest frequency leaves no fraction in 32), the
 * rest is in fp32 with one rounding at the end.
 *   q, k:  [n_tok][n_heads][head_dim], [n_tok][n_kv_heads][head_dim], dtype
 *          PI_F16 or PI_F32; either may be NULL with its head count 0
 *   pos:   [n_tok] device int32, any value
 *   q_out, k_out: may be the inputs themselves with the same strides, else
 *          must not overlap them
 * Errors: PI_E_NULL, PI_E_SHAPE (sizes, strides shorter than a head or not a
 * multiple of 16 bytes), PI_E_DTYPE (dtype, layout), PI_E_ALIGN, PI_E_RANGE
 * (scale or eps not finite, eps < 0, partial overlap), PI_E_HIP.  */
pi_status pi_qk_rope(const pi_rope* rope, const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                     int32_t n_heads, const void* k, int64_t k_tok_stride, int64_t k_head_stride,
                     int32_t n_kv_heads, const int32_t* pos, int32_t n_tok, int32_t dtype,
                     void* q_out, int64_t qo_tok_stride, int64_t qo_head_stride,
                     void* k_out, int64_t ko_tok_stride, int64_t ko_head_stride, void* stream);

typedef struct pi_kv_cache {
  int32_t n_seqs;
  int32_t n_kv_heads;
  int32_t head_dim;      /* 64 or 128                                       */
  int32_t max_blocks;    /* blocks that a table row names                   */
  int32_t n_pages;
  int32_t dtype;         /* of open and of every row: PI_F16 or PI_F32      */
  uint8_t* pages;        /* [n_pages][2][PI_KV_BLOCK * head_dim]            */
  float* scales;         /* [n_pages][2]; >= 0 (a negative one reads as NaN) */
  void* open;            /* [n_seqs][n_kv_heads][2][PI_KV_BLOCK][head_dim]; read and written by
                            pi_kv_append alone                             */
  const int32_t* table;  /* [n_seqs][n_kv_heads][max_blocks] page numbers   */
  float* score;          /* [n_seqs][n_kv_heads][max_blocks] accumulated attention weight; NULL: none */
} pi_kv_cache;

/* Append the rows of a call to the cache: the blocks from token lens - new on
 * are quantised anew (the first of them from its open rows and the new ones),
 * and the rows of the block that stays partly filled are kept in open.  Pages
 * written in one call must be distinct.  An invalid sequence (or one whose
 * lens is less than its rows) is left as it was; a bad page is not written.
 *   k, v: [n_tok][n_kv_heads][head_dim]
 * Errors: PI_E_NULL, PI_E_SHAPE, PI_E_DTYPE, PI_E_ALIGN, PI_E_HIP.  */
pi_status pi_kv_append(const pi_kv_cache* cache, const void* k, int64_t k_tok_stride, int64_t k_head_stride,
                       const void* v, int64_t v_tok_stride, int64_t v_head_stride, int32_t n_tok,
                       const int32_t* lens, const int32_t* q_start, int32_t max_new, void* stream);

/* Read back the values that the cache holds for the last rows of each
 * sequence (tokens lens - new .. lens), scale * (code - 128) in fp32, rounded
 * once.  Rows of an invalid sequence and values of a bad page are NaN.  k_out and
 * v_out must not overlap.
 * Errors: as pi_kv_append, and PI_E_RANGE (overlap).  */
pi_status pi_kv_read(const pi_kv_cache* cache, const int32_t* lens, const int32_t* q_start, int32_t max_new,
                     void* k_out, int64_t k_tok_stride, int64_t k_head_stride,
                     void* v_out, int64_t v_tok_stride, int64_t v_head_stride, int32_t n_tok, void* stream);

/* Bytes of workspace that pi_attend needs for these bounds; 0 for invalid
 * arguments.  add_score asks for 4 bytes per row, kv head and block more:
 * n_seqs * max_q * n_heads * ceil(max_len / PI_KV_BLOCK) * 4.  (A long prompt
 * with scores is better appended and attended in chunks.)  */
size_t pi_attend_workspace_bytes(const pi_kv_cache* cache, int32_t n_heads, int32_t max_q, int32_t max_len,
                                 int32_t add_score);

/* Attention over the cache: out = softmax(scale * q k^T) v over the tokens
 * that a row sees, for query head j with kv head j / (n_heads / n_kv_heads).
 * Row i of a sequence's new rows sees tokens 0 .. lens - new + i (itself the
 * last); a row that sees none gives zeros.  Logits, the softmax's statistics
 * and all sums are fp32.  Queries and codes enter the products unrounded (fp32
 * queries as two fp16 parts, 22 significant bits).  Weights enter as two fp16 parts,
 * too, except those of fp16 rows that see more than 512 tokens in a sequence with more than 32
 * rows to a kv head (new tokens times n_heads / n_kv_heads): they may enter as one, 11
 * bits, over the sum of the rounded weights.  A weight holds to
 * half a step of its logit in fp32, as any fp32 softmax's.  Value scales of a
 * sequence's kv head may count as 0 below 2^-74 of the largest of them.
 *   q, out:    [n_tok][n_heads][head_dim]; out must not overlap q
 *   max_q:     host bound on the new rows of a sequence (1: decode)
 *   max_len:   host bound on lens, in [1, max_blocks * PI_KV_BLOCK]
 *   scale:     of the logits, e.g. 1 / sqrt(head_dim); finite, not negative
 *   add_score: nonzero adds to score[s][h][b] the weights that the call's
 *              rows of kv head h's query heads gave to the tokens of block b
 *   ws:        workspace, zero-filled when new (its header collects flags)
 * Rows of an invalid sequence are NaN (its score stays), and so are rows that
 * see a token of a bad page; both raise PI_FLAG_KV_RANGE in ws.
 * Errors: PI_E_NULL (also add_score without a score), PI_E_SHAPE, PI_E_DTYPE, PI_E_ALIGN,
 * PI_E_RANGE (max_len, scale, overlap), PI_E_WORKSPACE, PI_E_HIP.  */
pi_status pi_attend(const pi_kv_cache* cache, const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                    int32_t n_heads, int32_t n_tok, const int32_t* lens, const int32_t* q_start, int32_t max_q,
                    int32_t max_len, float scale, int32_t add_score, void* out, int64_t o_tok_stride,
                    int64_t o_head_stride, void* ws, size_t ws_bytes, void* stream);

/* Evict blocks by accumulated weight: each (sequence, kv head) that holds
 * more than keep blocks keeps its last `recent` ones and, of the older ones,
 * the keep - recent with the largest score (ties: the lower slot; a NaN is
 * the largest), in their order.  The pages of the blocks that leave follow
 * them in the table, in their order, with score 0; slots past the held
 * blocks stay.  lens_out = lens - PI_KV_BLOCK * (blocks that left).
 *   table, score: [n_seqs][n_kv_heads][max_blocks]
 *   table_out, score_out: the same shape; may be table and score themselves
 *          (both) when max_blocks <= PI_KV_EVICT_IN_PLACE, else must not overlap them
 *   lens:  [n_seqs]; less than 0 counts as 0, more than the table as the table
 *   keep, recent: 1 <= recent <= keep (the last block may be partly filled,
 *          so it always stays)
 *   lens_out: [n_seqs], not lens
 * Errors: PI_E_NULL, PI_E_SHAPE, PI_E_ALIGN, PI_E_RANGE (keep, recent, overlap), PI_E_HIP.  */
#define PI_KV_EVICT_IN_PLACE 16384
pi_status pi_kv_evict(const int32_t* table, const float* score, const int32_t* lens, int32_t n_seqs,
                      int32_t n_kv_heads, int32_t max_blocks, int32_t keep, int32_t recent,
                      int32_t* table_out, float* score_out, int32_t* lens_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PI_ATTN_H_ */
