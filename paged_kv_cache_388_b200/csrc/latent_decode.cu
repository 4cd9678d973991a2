// latent_decode.cu -- attention over the latent cache in the absorbed form.
//
// The plain kernel: one CTA per (query row, head), its warps take keys in
// turn with an online softmax each (running max m, sum l, weighted sum o in
// registers) and are joined through shared memory.
#include "latent.h"
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr int kWarps = 8;

template <typename T, int R>
__global__ void __launch_bounds__(32 * kWarps) latent_decode_kernel(const LatentArgs a) {
  constexpr int D = R + 64, PL = D / 32, PO = R / 32;
  __shared__ float so[kWarps][R];
  __shared__ float sm[kWarps], sl[kWarps];
  __shared__ int bad;
  const int H = a.num_heads, h = blockIdx.x % H;
  const int t = (int)((blockIdx.x / H) % a.max_query_len), seq = (int)(blockIdx.x / H / a.max_query_len);
  int q0 = seq, Q = 1;
  if (a.query_start_loc) {
    q0 = a.query_start_loc[seq];
    Q = a.query_start_loc[seq + 1] - q0;
    if (q0 < 0 || Q < 0 || q0 > a.num_q_tokens - Q) {
      raise_error(a.err, PA_DEVERR_QUERY_LEN);
      return;
    }
  }
  const int L = a.context_lens[seq];
  const bool wrong = L < 0 || L > a.max_context_len || Q > a.max_query_len;
  if (wrong && threadIdx.x == 0)
    raise_error(a.err, Q > a.max_query_len ? PA_DEVERR_QUERY_LEN : PA_DEVERR_CONTEXT_LEN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  for (int row = t; row < Q; row += a.max_query_len) {
    const int64_t r = (int64_t)(q0 + row) * H + h;
    const int n = wrong ? 0 : max(0, L - Q + row + 1);
    float q[PL], o[PO], m = -INFINITY, l = 0.f;
    for (int i = 0; i < PL; ++i) q[i] = Elem<T>::to_f(static_cast<const T *>(a.q)[r * D + i * 32 + lane]);
    for (int i = 0; i < PO; ++i) o[i] = 0.f;
    for (int j = warp; j < n; j += kWarps) {
      const int b = a.block_tables[(int64_t)seq * a.max_blocks_per_seq + j / a.block_size];
      if (b < 0 || b >= a.num_blocks) {
        raise_error(a.err, PA_DEVERR_BLOCK_ID);
        bad = 1;
        break;
      }
      const T *c = static_cast<const T *>(a.cache) + ((int64_t)b * a.block_size + j % a.block_size) * D;
      float x[PL], s = 0.f;
      for (int i = 0; i < PL; ++i) {
        x[i] = Elem<T>::to_f(c[i * 32 + lane]);
        s += q[i] * x[i];
      }
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      s *= a.scale_log2;
      const float mn = fmaxf(m, s);
      const float f = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(s - mn);
      l = l * f + p;
      for (int i = 0; i < PO; ++i) o[i] = o[i] * f + p * x[i];
      m = mn;
    }
    for (int i = 0; i < PO; ++i) so[warp][i * 32 + lane] = o[i];
    if (lane == 0) sm[warp] = m, sl[warp] = l;
    __syncthreads();
    float M = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
    for (int w = 0; w < kWarps; ++w) sum += sm[w] == -INFINITY ? 0.f : sl[w] * exp2f(sm[w] - M);
    const bool none = M == -INFINITY || bad;
    for (int d = threadIdx.x; d < R; d += 32 * kWarps) {
      float x = 0.f;
      for (int w = 0; w < kWarps; ++w)
        if (sm[w] != -INFINITY) x += so[w][d] * exp2f(sm[w] - M);
      static_cast<T *>(a.out)[r * R + d] = Elem<T>::from_f(none ? 0.f : x / sum);
    }
    if (a.lse && threadIdx.x == 0)
      a.lse[r] = none ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
    __syncthreads();
  }
}

template <typename T>
cudaError_t launch_t(const LatentArgs &a, cudaStream_t s) {
  const int64_t grid = (int64_t)a.num_seqs * a.max_query_len * a.num_heads;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  if (a.latent_dim == 512) latent_decode_kernel<T, 512><<<(unsigned)grid, 32 * kWarps, 0, s>>>(a);
  else latent_decode_kernel<T, 256><<<(unsigned)grid, 32 * kWarps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t latent_decode_ws(int, int, int, int, int) { return 0; }

cudaError_t launch_latent_decode(const LatentArgs &a, int dtype, int, cudaStream_t stream) {
  return dtype == PA_BF16 ? launch_t<__nv_bfloat16>(a, stream) : launch_t<__half>(a, stream);
}

}  // namespace pa
