// latent.h -- host-side declarations of the latent cache's attention launches.
#pragma once

#include "pa_internal.h"

namespace pa {

// Ragged batches laid out in places: sequence s, whose rows begin at `start[s]`
// (times `mul`), has the places first_place(s) and following, one for every
// per = 2^shift of its rows.  n rows need ceil(n / per) places, and
// ceil(n / per) <= (begin + n) / per - begin / per + 1, so sequences never share
// one, all places lie below rows / per + num_seqs, and whose a place is follows
// from the offsets alone, without a sum over the sequences.
__device__ __forceinline__ int64_t first_place(const int32_t *start, int s, int mul, int shift) {
  return ((int64_t)start[s] * mul >> shift) + s;
}
// The last sequence whose places begin at or before `place`; a whole warp asks,
// 32 sequences at a time.  (Offsets that go back give some sequence: callers
// compare the place with the sequence's own.)
__device__ __forceinline__ int seq_of_place(const int32_t *start, int num_seqs, int mul, int shift, int64_t place) {
  int lo = 0, n = num_seqs;
  while (n > 1) {
    const int step = (n + 31) / 32, i = (int)(threadIdx.x & 31) * step;
    const bool at = i < n && first_place(start, lo + i, mul, shift) <= place;
    const int before = __popc(__ballot_sync(0xffffffffu, at));
    const int skip = before > 0 ? (before - 1) * step : 0;
    lo += skip;
    n = n - skip < step ? n - skip : step;
  }
  return lo;
}

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
