// Host-side description of a decode kernel variant, shared by the
// CUDA-core kernel (pa_decode.cu) and the tensor-core kernel
// (pa_decode_tc.cu).
#pragma once

#include <cuda_runtime.h>

#include "pa_decode_common.cuh"

namespace pa {

struct Variant;
using LaunchFn = cudaError_t (*)(const Variant& v, const DecodeParams& prm, int ctas, cudaStream_t stream);

struct Variant {
  const void* kernel;  // for occupancy queries and attributes
  int threads;
  int smem_bytes;
  int part_stride;  // floats per partial slot: query rows per unit * (D + 2)
  LaunchFn launch;
  int unit_cost;    // partition cost of finishing a unit (DecodeParams::unit_cost)
  bool fuses_update = false;  // tensor-core decode family: takes new tokens (DecodeParams::upd_*) into its launch and writes log normalisers (DecodeParams::lse)
  int ctas_per_sm = 0;  // of a default launch; 0: as many as the card holds of this kernel
};

// Tensor-core variants (pa_attn_tc.cuh), if one exists for this pool and
// shape.  `group` is the number of query heads per kv head.
// Plain decode (pa_decode_tc.cu): groups of 1, 2, 4 and 8, blocks of 8, 16
// or 32 tokens.
bool select_tc_variant(const pa_pool_desc& pool, int group, Variant& v);
// The plain decode's instances at blocks of 8 and 32 tokens
// (pa_decode_tc_blocks.cu).
bool select_tc_decode_other_block(int block_size, bool bf16, int group, Variant& v);
// Multi-query decode with q_len >= 2 positions (pa_attn_tc_multi.cu); tiles
// = units (row tiles) per sequence.
bool select_tc_multi_variant(const pa_pool_desc& pool, int group, int q_len, Variant& v, int& tiles);
// Its instances at blocks of 8 and 32 tokens (pa_attn_tc_multi_b8.cu,
// pa_attn_tc_multi_b32.cu): rg row groups a unit, tiled = several units a
// sequence.
bool select_tc_multi_b8(bool bf16, int group, int rg, bool tiled, Variant& v);
bool select_tc_multi_b32(bool bf16, int group, int rg, bool tiled, Variant& v);
// Query-major tiles of 128 rows (pa_attn_tc_prefill.cu) when a sequence's
// G x q_len rows fill at least one (blocks of 8, 16 or 32): tiles = units
// per sequence and kv head.  Its instances at blocks of 8 and 32 tokens:
// pa_attn_tc_prefill_b8.cu, pa_attn_tc_prefill_b32.cu.
bool select_tc_prefill_variant(const pa_pool_desc& pool, int group, int q_len, Variant& v, int& tiles);
bool select_tc_prefill_b8(bool bf16, int group, Variant& v);
bool select_tc_prefill_b32(bool bf16, int group, Variant& v);
// Shared-prefix decode over groups of up to max_members sequences
// (pa_attn_tc_group.cu).
bool select_tc_group_variant(const pa_pool_desc& pool, int group, int max_members, Variant& v);
// Its instances at blocks of 8 and 32 tokens (pa_attn_tc_group_b8.cu,
// pa_attn_tc_group_b32.cu), rg row groups (members) a unit.
bool select_tc_group_b8(bool bf16, int group, int rg, Variant& v);
bool select_tc_group_b32(bool bf16, int group, int rg, Variant& v);

// ---- host pieces shared by the decode entry points (pa_decode.cu) ---------

// Argument checks; PA_OK for an empty batch before its pointers are looked at.
pa_status check_decode_args(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
                            int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs,
                            int32_t num_q_heads, float scale, const void* out, const pa_pool_desc* pool);
DecodeParams make_params(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
                         int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads,
                         float scale, void* out, void* scratch, int ctas, int part_stride, int32_t* dev_status,
                         const pa_pool_desc* pool, int flags);
bool group_of(const pa_pool_desc& pool, int num_q_heads, int& G);
// CTA counts of a launch (0 on failure) and of a workspace-size query.
int resolve_ctas(const Variant& v, const pa_decode_opts* opts);
bool query_ctas(const Variant& v, const pa_decode_opts* opts, int& ctas);
size_t workspace_bytes_for(int num_seqs, int num_kv_heads, int ctas, int part_stride);

// ---- accumulated attention weights (pa_weights.cu) --------------------------
// Behind the decode's own workspace: the rows' log2 normalisers
// [num_seqs][num_q_heads], then the log2-domain scores
// [num_seqs][num_kv_heads][score_tokens_of(...)][G].
long long score_tokens_of(int max_blocks_per_seq, int block_size);
size_t scores_bytes(int num_seqs, int num_q_heads, int max_blocks_per_seq, int block_size);
void split_scores(char* base, int num_seqs, int num_q_heads, float** norm2, float** scores);
bool token_weights_ok(const pa_token_weights* w, int max_blocks_per_seq, int num_seqs, const pa_pool_desc* pool);
// Adds 2^(score - normaliser) over each kv head's query heads to the rows; to
// none of them if *failed (or null), and not to those of a sequence with a bad
// entry in its table.
pa_status accumulate_weights(const float* scores, const float* norm2, const pa_token_weights& w,
                             const int32_t* block_tables, const int32_t* seq_lens, int num_seqs, int num_q_heads,
                             int max_blocks_per_seq, const int32_t* failed, int32_t* dev_status,
                             const pa_pool_desc* pool, cudaStream_t stream);

// Tensor-core decode instances that also write scores and normalisers
// (pa_decode_tc_scores.cu and its instance files), if one exists.
bool select_tc_scores(const pa_pool_desc& pool, int group, Variant& v);
// The same at head_dim 64 (pa_weights_d64.cu).
bool select_scores_d64(const pa_pool_desc& pool, int group, Variant& v);
bool select_tc_scores_b8(bool bf16, int group, Variant& v);
bool select_tc_scores_b32(bool bf16, int group, Variant& v);

}  // namespace pa
