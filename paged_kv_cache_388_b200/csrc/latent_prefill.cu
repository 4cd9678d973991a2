// latent_prefill.cu -- attention of new tokens in the expanded form.
//
// The plain kernel: one CTA per (query row, head), its warps take keys in
// turn with an online softmax each and are joined through shared memory.
#include "latent.h"
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;

template <typename T, int DN>
__global__ void __launch_bounds__(32 * kWarps) latent_prefill_kernel(const LatentPrefillArgs a) {
  constexpr int PN = DN / 32, PL = PN + 2;
  __shared__ float so[kWarps][DN];
  __shared__ float sm[kWarps], sl[kWarps];
  const int H = a.num_heads, h = blockIdx.x % H;
  const int t = (int)((blockIdx.x / H) % a.max_query_len), seq = (int)(blockIdx.x / H / a.max_query_len);
  const int q0 = a.query_start_loc[seq], Q = a.query_start_loc[seq + 1] - q0;
  const int k0 = a.context_start_loc[seq], L = a.context_start_loc[seq + 1] - k0;
  if (q0 < 0 || Q < 0 || q0 > a.num_q_tokens - Q || k0 < 0 || L < 0 || k0 > a.num_k_tokens - L) {
    raise_error(a.err, PA_DEVERR_QUERY_LEN);
    return;
  }
  if (Q > a.max_query_len && threadIdx.x == 0) raise_error(a.err, PA_DEVERR_QUERY_LEN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int row = t; row < Q; row += a.max_query_len) {
    const int64_t r = (int64_t)(q0 + row) * H + h;
    const int n = Q > a.max_query_len ? 0 : a.causal ? max(0, L - Q + row + 1) : L;
    float q[PL], o[PN], m = -INFINITY, l = 0.f;
    for (int i = 0; i < PL; ++i) q[i] = Elem<T>::to_f(static_cast<const T *>(a.q)[r * (DN + 64) + i * 32 + lane]);
    for (int i = 0; i < PN; ++i) o[i] = 0.f;
    for (int j = warp; j < n; j += kWarps) {
      const T *k = static_cast<const T *>(a.k) + (k0 + j) * a.k_token_stride + h * a.k_head_stride;
      const T *kr = static_cast<const T *>(a.k_rope) + (k0 + j) * a.k_rope_stride;
      const T *v = static_cast<const T *>(a.v) + (k0 + j) * a.v_token_stride + h * a.v_head_stride;
      float s = 0.f;
      for (int i = 0; i < PN; ++i) s += q[i] * Elem<T>::to_f(k[i * 32 + lane]);
      for (int i = 0; i < 2; ++i) s += q[PN + i] * Elem<T>::to_f(kr[i * 32 + lane]);
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      s *= a.scale_log2;
      const float mn = fmaxf(m, s);
      const float f = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(s - mn);
      l = l * f + p;
      for (int i = 0; i < PN; ++i) o[i] = o[i] * f + p * Elem<T>::to_f(v[i * 32 + lane]);
      m = mn;
    }
    for (int i = 0; i < PN; ++i) so[warp][i * 32 + lane] = o[i];
    if (lane == 0) sm[warp] = m, sl[warp] = l;
    __syncthreads();
    float M = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
    for (int w = 0; w < kWarps; ++w) sum += sm[w] == -INFINITY ? 0.f : sl[w] * exp2f(sm[w] - M);
    const bool none = M == -INFINITY;
    for (int d = threadIdx.x; d < DN; d += 32 * kWarps) {
      float x = 0.f;
      for (int w = 0; w < kWarps; ++w)
        if (sm[w] != -INFINITY) x += so[w][d] * exp2f(sm[w] - M);
      static_cast<T *>(a.out)[r * DN + d] = Elem<T>::from_f(none ? 0.f : x / sum);
    }
    if (a.lse && threadIdx.x == 0) a.lse[r] = none ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
    __syncthreads();
  }
}

template <typename T>
cudaError_t launch_t(const LatentPrefillArgs &a, cudaStream_t s) {
  const int64_t grid = (int64_t)a.num_seqs * a.max_query_len * a.num_heads;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  if (a.nope_dim == 128) latent_prefill_kernel<T, 128><<<(unsigned)grid, 32 * kWarps, 0, s>>>(a);
  else latent_prefill_kernel<T, 64><<<(unsigned)grid, 32 * kWarps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, int dtype, int, cudaStream_t stream) {
  return dtype == PA_BF16 ? launch_t<__nv_bfloat16>(a, stream) : launch_t<__half>(a, stream);
}

}  // namespace pa
