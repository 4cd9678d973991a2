// latent.h -- host-side declarations of the latent cache's attention launches.
#pragma once

#include "pa_internal.h"

namespace pa {

// Absorbed form over the paged latent cache (latent_decode.cu).
struct LatentArgs {
  void *out;    // [Tq][H][latent_dim]
  float *lse;   // [Tq][H], nullable
  const void *q;  // [Tq][H][latent_dim + rope_dim]
  const void *cache;
  const int32_t *block_tables;
  const int32_t *context_lens;
  const int32_t *query_start_loc;  // nullable: one row per sequence
  int num_seqs, num_q_tokens, max_query_len, num_heads;
  int latent_dim, rope_dim, block_size, num_blocks, max_blocks_per_seq, max_context_len;
  float scale_log2;  // scale * log2(e)
  void *ws;
  unsigned int *err;
};
size_t latent_decode_ws(int num_seqs, int max_query_len, int num_heads, int latent_dim, int sm_count);
// Whether the kernels' 32-bit counts hold the batch.
bool latent_decode_fits(int num_seqs, int max_query_len, int num_heads, int latent_dim, int max_context_len);
cudaError_t launch_latent_decode(const LatentArgs &a, int dtype, int sm_count, cudaStream_t stream);

// Expanded form over ragged contiguous keys and values (latent_prefill.cu).
struct LatentPrefillArgs {
  void *out;    // [Tq][H][v_dim]
  float *lse;   // [Tq][H], nullable
  const void *q;  // [Tq][H][nope_dim + 64]
  const void *k, *k_rope, *v;
  int64_t k_token_stride, k_head_stride, k_rope_stride, v_token_stride, v_head_stride;  // elements
  const int32_t *query_start_loc, *context_start_loc;
  int num_seqs, num_q_tokens, num_k_tokens, max_query_len, num_heads, nope_dim, causal;
  float scale_log2;
  void *ws;
  unsigned int *err;
};
size_t latent_prefill_ws(int num_seqs, int num_q_tokens, int num_k_tokens, int num_heads, int nope_dim, int sm_count);
cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, int dtype, int sm_count, cudaStream_t stream);

}  // namespace pa
