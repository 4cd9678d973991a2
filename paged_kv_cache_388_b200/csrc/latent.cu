// latent.cu -- the latent cache's entry points (argument checks) and the
// scatter of new rows into their slots.
#include <float.h>
#include <math.h>

#include "latent.h"
#include "pa_device.cuh"

namespace pa {
namespace {

// One thread per 16-byte vector of a token's row: the first `lv` vectors come
// from the latent part, the rest from the rope part.  Reads and writes are
// coalesced within a row of 640 or 1152 bytes.  I: the type that counts vectors
// (64-bit divisions make 16411 rows of 1152 bytes 8.4 us instead of 6.6).  Bound: memory traffic
// and, for a decode step's few tokens, the latency of one dependent load (the
// slot).
template <typename I>
__global__ void __launch_bounds__(256) latent_write_kernel(
    const uint4 *__restrict__ latent, const uint4 *__restrict__ rope, uint4 *__restrict__ cache,
    const int64_t *__restrict__ slots, int num_tokens, int64_t latent_stride, int64_t rope_stride,
    int lv, int rv, int64_t num_slots, unsigned int *err) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const I row = (I)(lv + rv), total = (I)num_tokens * row;
  for (I i = (I)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (I)gridDim.x * blockDim.x) {
    const int64_t t = i / row;
    const int v = (int)(i - (I)t * row);
    const uint4 x = __ldcs(v < lv ? latent + t * latent_stride + v : rope + t * rope_stride + (v - lv));
    const int64_t slot = slots[t];
    if (slot < 0) continue;  // padding token
    if (slot >= num_slots) {
      if (v == 0) raise_error(err, PA_DEVERR_SLOT);
      continue;
    }
    cache[slot * (lv + rv) + v] = x;
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dtype16(int dtype) { return dtype == PA_F16 || dtype == PA_BF16; }
bool scale_ok(float s) { return isfinite(s) && s >= 0.f; }

// scale * log2(e); never 0, so that a masked -infinity stays one (a scale this
// small leaves every finite logit at 0)
float scale_log2(float scale) { return fmaxf(scale * 1.4426950408889634f, FLT_MIN); }

// Checks shared by the entry points that take a latent cache.
int latent_shape(int latent_dim, int rope_dim, int block_size, int dtype) {
  if (!dtype16(dtype)) return PA_ERR_UNSUPPORTED;
  if ((latent_dim != 256 && latent_dim != 512) || rope_dim != 64) return PA_ERR_UNSUPPORTED;
  if (block_size != 16 && block_size != 32 && block_size != 64) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int pa_latent_write(const void *latent, const void *rope, void *latent_cache,
                    const int64_t *slot_mapping, int num_tokens, int64_t latent_stride,
                    int64_t rope_stride, int latent_dim, int rope_dim, int block_size, int num_blocks,
                    int dtype, struct CUstream_st *stream) {
  if (num_tokens < 0 || num_blocks <= 0) return PA_ERR_INVALID_ARG;
  const int rc = latent_shape(latent_dim, rope_dim, block_size, dtype);
  if (rc != PA_OK) return rc;
  if (num_tokens == 0) return PA_OK;
  if (!latent || !rope || !latent_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
  if (!aligned16(latent) || !aligned16(rope) || !aligned16(latent_cache)) return PA_ERR_INVALID_ARG;
  if (latent_stride < 0 || rope_stride < 0 || latent_stride % 8 || rope_stride % 8)
    return PA_ERR_INVALID_ARG;
  DevInfo dev;
  if (device_info(&dev) != cudaSuccess) return PA_ERR_CUDA;
  const int lv = latent_dim / 8, rv = rope_dim / 8;
  int64_t blocks = ((int64_t)num_tokens * (lv + rv) + 255) / 256;
  if (blocks > (int64_t)dev.sm_count * 16) blocks = (int64_t)dev.sm_count * 16;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // below 2^31 vectors the loop's last step stays below 2^32 too
  const bool narrow = (int64_t)num_tokens * (lv + rv) < (int64_t)1 << 31;
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, narrow ? latent_write_kernel<uint32_t> : latent_write_kernel<uint64_t>,
      static_cast<const uint4 *>(latent), static_cast<const uint4 *>(rope),
      static_cast<uint4 *>(latent_cache), slot_mapping, num_tokens, latent_stride / 8, rope_stride / 8,
      lv, rv, (int64_t)num_blocks * block_size, dev.err);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_latent_decode_workspace_size(int num_seqs, int max_query_len, int num_heads, int latent_dim) {
  if (num_seqs <= 0 || max_query_len <= 0 || num_heads <= 0 || latent_dim <= 0) return 0;
  DevInfo dev;
  if (device_info(&dev) != cudaSuccess) return 0;
  return latent_decode_ws(num_seqs, max_query_len, num_heads, latent_dim, dev.sm_count);
}

int pa_latent_decode(void *out, float *lse, const void *q, const void *latent_cache,
                     const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                     const int32_t *query_start_loc, int num_seqs, int num_q_tokens, int max_query_len,
                     int num_heads, int latent_dim, int rope_dim, int block_size, int num_blocks,
                     float scale, int max_context_len, int dtype, void *workspace,
                     size_t workspace_bytes, struct CUstream_st *stream) {
  if (num_seqs < 0 || num_q_tokens < 0 || num_heads <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0 || !scale_ok(scale))
    return PA_ERR_INVALID_ARG;
  const int rc = latent_shape(latent_dim, rope_dim, block_size, dtype);
  if (rc != PA_OK) return rc;
  if (!query_start_loc) {
    if (num_q_tokens != num_seqs) return PA_ERR_INVALID_ARG;
    max_query_len = 1;
  } else if (max_query_len < 1) {
    return PA_ERR_INVALID_ARG;
  }
  if (num_seqs == 0 || num_q_tokens == 0) return PA_OK;
  if (!out || !q || !latent_cache || !block_tables || !context_lens) return PA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(latent_cache)) return PA_ERR_INVALID_ARG;
  if (out == q) return PA_ERR_INVALID_ARG;
  if ((int64_t)max_blocks_per_seq * block_size > (int64_t)1 << 30) return PA_ERR_UNSUPPORTED;
  if ((int64_t)num_q_tokens * num_heads > (int64_t)1 << 30) return PA_ERR_UNSUPPORTED;
  if ((int64_t)num_blocks * block_size > (int64_t)1 << 31) return PA_ERR_UNSUPPORTED;
  if (max_query_len > num_q_tokens) max_query_len = num_q_tokens;
  const int cap = max_blocks_per_seq * block_size;
  if (max_context_len <= 0 || max_context_len > cap) max_context_len = cap;
  if (!latent_decode_fits(num_seqs, max_query_len, num_heads, latent_dim, max_context_len))
    return PA_ERR_UNSUPPORTED;
  DevInfo dev;
  if (device_info(&dev) != cudaSuccess) return PA_ERR_CUDA;
  const size_t need = latent_decode_ws(num_seqs, max_query_len, num_heads, latent_dim, dev.sm_count);
  if (need && (!workspace || workspace_bytes < need || !aligned16(workspace))) return PA_ERR_WORKSPACE;
  LatentArgs a{};
  a.out = out;
  a.lse = lse;
  a.q = q;
  a.cache = latent_cache;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.query_start_loc = query_start_loc;
  a.num_seqs = num_seqs;
  a.num_q_tokens = num_q_tokens;
  a.max_query_len = max_query_len;
  a.num_heads = num_heads;
  a.latent_dim = latent_dim;
  a.rope_dim = rope_dim;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_context_len = max_context_len;
  a.scale_log2 = scale_log2(scale);
  a.ws = workspace;
  a.err = dev.err;
  const cudaError_t e = launch_latent_decode(a, dtype, dev.sm_count, (cudaStream_t)stream);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_latent_prefill_workspace_size(int num_seqs, int num_q_tokens, int num_k_tokens, int num_heads,
                                        int nope_dim) {
  if (num_seqs <= 0 || num_q_tokens <= 0 || num_k_tokens <= 0 || num_heads <= 0 || nope_dim <= 0) return 0;
  DevInfo dev;
  if (device_info(&dev) != cudaSuccess) return 0;
  return latent_prefill_ws(num_seqs, num_q_tokens, num_k_tokens, num_heads, nope_dim, dev.sm_count);
}

int pa_latent_prefill(void *out, float *lse, const void *q, const void *k, const void *k_rope,
                      const void *v, int64_t k_token_stride, int64_t k_head_stride,
                      int64_t k_rope_stride, int64_t v_token_stride, int64_t v_head_stride,
                      const int32_t *query_start_loc, const int32_t *context_start_loc, int num_seqs,
                      int num_q_tokens, int num_k_tokens, int max_query_len, int num_heads,
                      int nope_dim, int rope_dim, int v_dim, float scale, int causal, int dtype,
                      void *workspace, size_t workspace_bytes, struct CUstream_st *stream) {
  if (num_seqs < 0 || num_q_tokens < 0 || num_k_tokens < 0 || num_heads <= 0 || max_query_len < 1 ||
      !scale_ok(scale))
    return PA_ERR_INVALID_ARG;
  if (!dtype16(dtype) || rope_dim != 64 || nope_dim != v_dim || (nope_dim != 64 && nope_dim != 128))
    return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || num_q_tokens == 0) return PA_OK;
  if (!out || !q || !query_start_loc || !context_start_loc) return PA_ERR_INVALID_ARG;
  if (num_k_tokens > 0 && (!k || !k_rope || !v)) return PA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k) || !aligned16(k_rope) || !aligned16(v))
    return PA_ERR_INVALID_ARG;
  const int64_t strides[5] = {k_token_stride, k_head_stride, k_rope_stride, v_token_stride, v_head_stride};
  for (int i = 0; i < 5; ++i)
    if (strides[i] <= 0 || strides[i] % 8 || strides[i] >= (int64_t)1 << 38) return PA_ERR_INVALID_ARG;
  if (out == q) return PA_ERR_INVALID_ARG;
  if ((int64_t)num_q_tokens * num_heads > (int64_t)1 << 30 || (int64_t)num_seqs * num_heads > (int64_t)1 << 30)
    return PA_ERR_UNSUPPORTED;
  if (max_query_len > num_q_tokens) max_query_len = num_q_tokens;
  DevInfo dev;
  if (device_info(&dev) != cudaSuccess) return PA_ERR_CUDA;
  const size_t need = latent_prefill_ws(num_seqs, num_q_tokens, num_k_tokens, num_heads, nope_dim, dev.sm_count);
  if (need && (!workspace || workspace_bytes < need || !aligned16(workspace))) return PA_ERR_WORKSPACE;
  LatentPrefillArgs a{};
  a.ws = workspace;
  a.out = out;
  a.lse = lse;
  a.q = q;
  a.k = k;
  a.k_rope = k_rope;
  a.v = v;
  a.k_token_stride = k_token_stride;
  a.k_head_stride = k_head_stride;
  a.k_rope_stride = k_rope_stride;
  a.v_token_stride = v_token_stride;
  a.v_head_stride = v_head_stride;
  a.query_start_loc = query_start_loc;
  a.context_start_loc = context_start_loc;
  a.num_seqs = num_seqs;
  a.num_q_tokens = num_q_tokens;
  a.num_k_tokens = num_k_tokens;
  a.max_query_len = max_query_len;
  a.num_heads = num_heads;
  a.nope_dim = nope_dim;
  a.causal = causal != 0;
  a.scale_log2 = scale_log2(scale);
  a.err = dev.err;
  const cudaError_t e = launch_latent_prefill(a, dtype, dev.sm_count, (cudaStream_t)stream);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
