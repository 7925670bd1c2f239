// Arguments and launches of the attention side's kernels (pi_attn.h says what each
// computes).  Apart from pi_internal.h, so that the FFN's sources are not touched
// where the attention side changes.
#pragma once

#include "pi_internal.h"

namespace pi {

// A launch holds fewer than 2^32 threads.
constexpr int64_t kMaxThreads = 0xffffffffll;

// Rows [n_tok][n_heads][head_dim] of a call; strides in elements.
struct HeadRows {
  void* p;
  int64_t ts, hs;           // between tokens, between heads
  int32_t n;                // heads
};

struct RopeArgs {
  int d, rot, layout, dtype, n_tok;
  float scale, eps;
  const double* freqs;
  const float* w[2];        // norm weights of queries and keys; NULL: none
  HeadRows in[2], out[2];   // queries, keys
  const int32_t* pos;
};
int64_t qk_rope_threads(const RopeArgs& a);
hipError_t launch_qk_rope(const RopeArgs& a, hipStream_t s);

struct CacheArgs {
  int n_seqs, hk, d, max_blocks, n_pages, dtype;
  uint8_t* pages;
  float* scales;
  void* open;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* q_start;   // nullable
  int max_new, n_tok;
  HeadRows kv[2];           // rows in (append) or out (read)
};
int64_t kv_cache_threads(const CacheArgs& a);      // of an append or a read
hipError_t launch_kv_append(const CacheArgs& a, hipStream_t s);
hipError_t launch_kv_read(const CacheArgs& a, hipStream_t s);

// How a pi_attend call is cut up (by sizes and types alone).
struct AttendPlan {
  int nb;                   // 16-row tiles per wave
  bool many;                // each wave has rows of its own; else the waves of a workgroup share rows and split the blocks
  bool two;                 // many: all fp16 rows' weights as two parts (else by what they see)
  int waves;                // that have rows of their own, in a workgroup (many; the others take other blocks)
  int tiles;                // workgroups over the rows of a (sequence, kv head)
  int splits;               // workgroups over the blocks (with slots: on average)
  int slots;                // workgroups that the sequences share by their lengths; 0: splits each
  int splits_max;           // of a (sequence, kv head)
  float share_even, share_safe; // blocks to a workgroup per block of all sequences: evenly, and always enough
  int r_max;                // rows of a (sequence, kv head): max_q * group
  int max_nb;               // blocks of max_len
  int64_t row_groups, score_groups; // workgroups of the join (0: none)
  int64_t threads;          // of the larger launch
  size_t part, ml, lse, count;  // offsets in the workspace (after its header)
  size_t total;             // bytes, the header among them
};
AttendPlan attend_plan(int n_seqs, int hk, int group, int d, int dtype, int max_q, int max_len, bool score);

struct AttendArgs {
  const void* q;
  int64_t q_ts, q_hs;
  void* out;
  int64_t o_ts, o_hs;
  const int32_t* lens;
  const int32_t* q_start;   // nullable
  const uint8_t* pages;
  const float* scales;
  const int32_t* table;
  float* score;             // nullable: no score
  int n_seqs, hk, group, n_tok, max_q, max_len, max_blocks, n_pages;
  float scale;              // of the logits, times log2(e)
  int r_max, max_nb, tiles, splits, slots, splits_max;
  float* part;              // [splits_max][n_seqs * hk][r_max][d] means of a split's values by their weights
  float share_even, share_safe;
  float2* ml;               // [splits_max][n_seqs * hk][r_max] reference exponent and sum of the weights
  float* lse;               // [n_seqs * hk][max_nb][r_max] log2 of a block's weights
  int* count;               // [n_seqs * hk] splits (where slots > 0)
  unsigned* flags;
};
hipError_t launch_attend(const AttendArgs& a, const AttendPlan& p, int d, int dtype, hipStream_t s);

struct EvictArgs {
  const int32_t* table;
  const float* score;
  const int32_t* lens;
  int n_seqs, hk, max_blocks, keep, recent;
  int32_t* table_out;
  float* score_out;
  int32_t* lens_out;
};
int64_t kv_evict_threads(const EvictArgs& a);
hipError_t launch_kv_evict(const EvictArgs& a, hipStream_t s);

}  // namespace pi
