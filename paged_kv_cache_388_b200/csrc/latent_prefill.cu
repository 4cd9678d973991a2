// latent_prefill.cu -- attention of new tokens in the expanded form on the
// 5th-generation tensor cores.
//
// Head h of a token has a key [k_nope (DN) | k_rope (64, shared by the heads)]
// and a value of DN; row t of a sequence with Q rows and L keys sees the keys
// j <= L-Q+t (causal) or all of them.  With S = scale * Q K^T (base 2 below),
// a running maximum m and sum l per row, O = sum_j 2^(s_j - m) v_j:
//     out = O / l,  lse = (m + log2 l) ln 2.
//
// CTA = (sequence, head, 256 query rows held as two Q tiles of 128).  Per
// 128-key tile j and Q tile t the tensor cores compute S_t = Q_t K_j^T (K =
// DN + 64) and O_t += P_t V_j, fp32 accumulators in tensor memory (128 columns
// each: all 512 are used); P_t (16 bits, two keys a word) overwrites S_t and
// is the A operand of P V from there.  The chains P V_t(j), S_t(j+1), softmax of
// the two Q tiles run side by side, so that the softmax of one lies under the
// products of the other.
//
// K and V arrive by TMA in chunks of 128 keys x 64 columns (16 KB, the
// 128-byte-swizzle layout the products read), K's chunks and V's through one
// ring in the order they are consumed: with Q's 96 KB there is no room for two
// whole K/V tiles, but eight chunks keep V(j+1) and the head of K(j+2) in
// flight while tile j is worked on.
//
// Warps: 8 softmax (4 per Q tile; thread = row = TMEM lane), 1 TMA producer,
// 2 MMA issuers (one per Q tile; the first also owns the tensor memory).
#include "latent.h"
#include "pa_device.cuh"
#include "tc_common.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;  // rows per Q tile (MMA M)
constexpr int kKeys = 128;  // keys per tile
constexpr int kQTiles = 2;
constexpr int kChunk = 128 * 64 * 2;       // bytes of 128 rows x 64 columns
constexpr float kRescaleThreshold = 8.0f;  // log2 units: P stays <= 2^8 between rescales
constexpr int kSoftmaxWarps = 4 * kQTiles;
constexpr int kProducerWarp = kSoftmaxWarps, kMmaWarp = kSoftmaxWarps + 1;
constexpr int kThreads = 32 * (kSoftmaxWarps + 1 + kQTiles);

// Barriers of K and V are kept by tile parity: the ring holds two
// tiles at most, so that a tile's chunks are asked for only after the products of the
// tile two before have let theirs go.
enum {
  kQFull = 0,
  kKFull = 1,                   // [2] K of the tile landed
  kVFull = kKFull + 2,          // [2] V of the tile landed
  kKEmpty = kVFull + 2,         // [2] both Q tiles' S done
  kVEmpty = kKEmpty + 2,        // [2] both Q tiles' P V done
  kSFull = kVEmpty + 2,         // [Q tile] S in tensor memory
  kPFull = kSFull + kQTiles,    // [Q tile][half] 64 keys of P written over S (4 warps)
  kPvDone = kPFull + 2 * kQTiles,  // [Q tile] P V complete
  kTurn = kPvDone + kQTiles,    // S_1 of the tile is being issued
  kDone = kTurn + 1,            // [Q tile]
  kNumBars = kDone + kQTiles
};

template <int DN>
struct Shape {
  static constexpr int kKC = DN / 64 + 1;  // chunks of K a tile
  static constexpr int kVC = DN / 64;      // chunks of V a tile
  static constexpr int kTC = kKC + kVC;
  // chunks in flight: two tiles at most (see the barriers)
  static constexpr int kRing = 2 * kTC < 8 ? 2 * kTC : 8;
  static constexpr int kQBytes = kKC * kChunk;  // one Q tile
  static constexpr int kOffRing = kQTiles * kQBytes;
  static constexpr int kOffBar = kOffRing + kRing * kChunk;
  static constexpr int kSmem = kOffBar + 8 * kNumBars + 64 + 1024;  // + TMEM slot, flag, alignment
};
static_assert(Shape<128>::kSmem <= 227 * 1024, "shared memory per CTA");

__device__ __forceinline__ uint32_t tmem_s_col(int t) { return (uint32_t)t * 256u; }
__device__ __forceinline__ uint32_t tmem_o_col(int t) { return (uint32_t)t * 256u + 128u; }

// Scores of keys past the last visible one (`last`, counted from the first of
// these 64 columns) become -infinity.
__device__ __forceinline__ void mask_keys(uint32_t (&s)[2][32], int last) {
#pragma unroll
  for (int i = 0; i < 64; ++i)
    if (i > last) s[i >> 5][i & 31] = __float_as_uint(-INFINITY);
}

template <typename T, int DN>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const LatentPrefillArgs a, const __grid_constant__ CUtensorMap tmq,
                          const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmr,
                          const __grid_constant__ CUtensorMap tmv, int tiles) {
  using TT = TcType<T>;
  using SH = Shape<DN>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SH::kOffBar);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + SH::kOffBar + 8 * kNumBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const uint32_t sbase = smem_addr(smem);
  const uint32_t ring = sbase + SH::kOffRing;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- the CTA's rows; tiles with the most keys first ----------------------
  const int H = a.num_heads;
  const int per_tile = a.num_seqs * H;
  const int tile = tiles - 1 - (int)(blockIdx.x / per_tile);
  const int rest = blockIdx.x % per_tile;
  const int seq = rest / H, h = rest % H;
  const int q0 = a.query_start_loc[seq], Q = a.query_start_loc[seq + 1] - q0;
  const int k0 = a.context_start_loc[seq], L = a.context_start_loc[seq + 1] - k0;
  // CTA-uniform exits, before any barrier
  if (q0 < 0 || Q < 0 || q0 > a.num_q_tokens - Q || k0 < 0 || L < 0 || k0 > a.num_k_tokens - L) {
    if (tid == 0) raise_error(a.err, PA_DEVERR_QUERY_LEN);
    return;
  }
  const bool over = Q > a.max_query_len;
  if (over && tid == 0) raise_error(a.err, PA_DEVERR_QUERY_LEN);
  const int t0 = tile * kQTiles * kRows;
  if (t0 >= Q) return;
  const int ntok = min(kQTiles * kRows, Q - t0);
  const int kend = a.causal ? min(L, L - Q + t0 + ntok) : L;  // keys [0, kend) are visible to some row
  if (over || kend <= 0) {  // zeros; a sequence with too many rows has more of them than the grid's tiles
    for (int t = t0; t < Q; t += over ? tiles * kQTiles * kRows : Q)
      for (int i = tid; i < min(kQTiles * kRows, Q - t) * DN; i += kThreads) {
        const int64_t r = (int64_t)(q0 + t + i / DN) * H + h;
        static_cast<T *>(a.out)[r * DN + i % DN] = Elem<T>::from_f(0.f);
        if (a.lse && i % DN == 0) a.lse[r] = -INFINITY;
      }
    return;
  }
  const int nq = ntok > kRows ? 2 : 1;
  const int ntiles = (kend + kKeys - 1) / kKeys;
  // tiles of Q tile 0 (rows t0 .. t0+127); Q tile nq-1 takes all of them
  const int kend0 = a.causal ? min(L, L - Q + t0 + min(ntok, kRows)) : L;
  const int nt0 = max(0, (kend0 + kKeys - 1) / kKeys);

  // ---- set-up: barriers, tensor memory -------------------------------------
  if (tid == 0) {
    mbar_init(&bars[kQFull], 1);
    mbar_init(&bars[kTurn], 1);
    for (int p = 0; p < 2; ++p) {
      mbar_init(&bars[kKFull + p], 1);
      mbar_init(&bars[kVFull + p], 1);
      mbar_init(&bars[kKEmpty + p], nq);
      mbar_init(&bars[kVEmpty + p], nq);
    }
    for (int t = 0; t < kQTiles; ++t) {
      mbar_init(&bars[kSFull + t], 1);
      mbar_init(&bars[kPFull + 2 * t], 4);
      mbar_init(&bars[kPFull + 2 * t + 1], 4);
      mbar_init(&bars[kPvDone + t], 1);
      mbar_init(&bars[kDone + t], 1);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto fail = [&](void) {
    if (!*abort_flag) raise_error(a.err, PA_DEVERR_TIMEOUT);
    *abort_flag = 1;
  };

  const uint32_t bar0 = smem_addr(bars);
  auto warp_wait = [&](int bar, uint32_t parity) -> bool {
    return mbar_warp_wait(bar0 + 8 * bar, parity, abort_flag, a.err);
  };

  if (warp == kProducerWarp) {
    // ======================= producer =======================================
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars[kQFull], nq * SH::kQBytes);
      for (int t = 0; t < nq; ++t)
        for (int c = 0; c < SH::kKC; ++c)
          tma_load_3d(sbase + t * SH::kQBytes + c * kChunk, &tmq, c * 64, h, q0 + t0 + t * kRows,
                      &bars[kQFull]);
    }
    __syncwarp();
    uint32_t x = 0;              // chunk
    int last_k = -1, last_v = -1;  // last tile whose K (V) was announced
    bool ok = true;
    for (int j = 0; j < ntiles && ok; ++j) {
      const int row = k0 + j * kKeys, p = j & 1;
#pragma unroll
      for (int c = 0; c < SH::kTC; ++c, ++x) {
        if (x >= SH::kRing) {  // the chunk SH::kRing before has been let go with its tile's K or V
          const uint32_t tj = (x - SH::kRing) / SH::kTC, tc = (x - SH::kRing) % SH::kTC;
          ok = warp_wait((tc < SH::kKC ? kKEmpty : kVEmpty) + (tj & 1), (tj >> 1) & 1);
          if (!ok) break;
        }
        if (lane == 0) {
          const uint32_t dst = ring + (x % SH::kRing) * kChunk;
          uint64_t *bar = &bars[(c < SH::kKC ? kKFull : kVFull) + p];
          if (c == 0) mbar_arrive_expect_tx(bar, SH::kKC * kChunk);
          if (c == SH::kKC) mbar_arrive_expect_tx(bar, SH::kVC * kChunk);
          if (c < SH::kKC - 1) tma_load_3d(dst, &tmk, c * 64, h, row, bar);
          else if (c == SH::kKC - 1) tma_load_2d(dst, &tmr, 0, row, bar);
          else tma_load_3d(dst, &tmv, (c - SH::kKC) * 64, h, row, bar);
        }
        __syncwarp();
        if (c == SH::kKC - 1) last_k = j;
        if (c == SH::kTC - 1) last_v = j;
      }
    }
    // Every copy has landed before the CTA can exit.  After a failure part of a
    // tile's chunks may be on their way under a barrier that waits for the
    // others too: what is missing is taken off it.
    if (!ok && lane == 0) {
      const int j = (int)(x / SH::kTC), c = (int)(x % SH::kTC);
      if (c > 0 && c < SH::kKC) mbar_complete_tx(&bars[kKFull + (j & 1)], (SH::kKC - c) * kChunk), last_k = j;
      if (c > SH::kKC) mbar_complete_tx(&bars[kVFull + (j & 1)], (SH::kTC - c) * kChunk), last_v = j;
    }
    if (lane == 0) {
      bool landed = mbar_wait(&bars[kQFull], 0);
      for (int j = last_k; j >= 0 && j > last_k - 2; --j) landed = mbar_wait(&bars[kKFull + (j & 1)], (j >> 1) & 1) && landed;
      for (int j = last_v; j >= 0 && j > last_v - 2; --j) landed = mbar_wait(&bars[kVFull + (j & 1)], (j >> 1) & 1) && landed;
      if (!landed) fail();
    }
  } else if (warp >= kMmaWarp) {
    // ======================= MMA issue ======================================
    // One warp per Q tile: a thread that has issued products goes on only when
    // they have started, so one warp for both would hold P_0 V back behind S_1.
    constexpr uint32_t idesc_s = umma_idesc(TT::kFmt, 0, 0, kRows, kKeys);
    constexpr uint32_t idesc_pv = umma_idesc(TT::kFmt, 0, 1, kRows, 64);
    constexpr uint32_t kHi = umma_desc_hi(1024);
    const int t = warp - kMmaWarp;
    const int nt = t == nq - 1 ? ntiles : t < nq ? nt0 : 0;
    const uint32_t a_lo = umma_desc_lo(sbase + t * SH::kQBytes, 16);
    const uint32_t k_lo = umma_desc_lo(ring, 16), v_lo = umma_desc_lo(ring, kChunk);
    // S_t(j) = Q_t K_j^T: both K-major, 8-row groups 1 KB apart
    auto issue_s = [&](int j) {
      const uint32_t x0 = (uint32_t)j * SH::kTC;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t d = tmem + tmem_s_col(t);
        if (t == 1) mbar_arrive(&bars[kTurn]);
#pragma unroll
        for (int c = 0; c < SH::kKC; ++c) {
          const uint32_t b_lo = k_lo + ((x0 + c) % SH::kRing) * (kChunk >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_lo(d, a_lo + ((c * kChunk + kk * 32) >> 4), kHi, b_lo + ((kk * 32) >> 4), kHi, idesc_s,
                    (c | kk) ? 1u : 0u);
        }
        umma_commit(&bars[kSFull + t]);
        umma_commit(&bars[kKEmpty + (j & 1)]);
      }
      __syncwarp();
    };
    // O_t += P_t(j) V_j: A = P from tensor memory (16 keys in 8 columns), B =
    // V with columns contiguous, 64 of them a product, 8-key groups 1 KB apart
    auto issue_pv = [&](int j, int half) {
      const uint32_t x0 = (uint32_t)j * SH::kTC + SH::kKC;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t keep = (j | half) ? 1u : 0u;
        const uint32_t pcol = tmem + tmem_s_col(t) + half * 32;
#pragma unroll
        for (int c = 0; c < SH::kVC; ++c) {
          const uint32_t b_lo = v_lo + ((x0 + c) % SH::kRing) * (kChunk >> 4) + half * (8192 >> 4);
#pragma unroll
          for (int ks = 0; ks < kKeys / 32; ++ks)
            umma_ts_lo(tmem + tmem_o_col(t) + c * 64, pcol + ks * 8, b_lo + ((ks * 2048) >> 4), kHi, idesc_pv,
                       ks > 0 ? 1u : keep);
        }
        if (half) {
          umma_commit(&bars[kPvDone + t]);
          umma_commit(&bars[kVEmpty + (j & 1)]);
        }
      }
      __syncwarp();
    };
    // The two chains are kept half a step apart: S_1(j) is issued when half of
    // P_0(j) is there, S_0(j+1) when S_1(j) has been issued.  In step they would meet at
    // the exponentials (16 a cycle and SM: 1024 cycles for a tile of 128 x 128),
    // then leave those units idle together.
    // The waits that are usually over go before those that are not.
    const bool pair = nq == 2;
    auto k_ready = [&](int j) { return warp_wait(kKFull + (j & 1), (j >> 1) & 1); };
    auto turn = [&](int j) {
      if (pair && t == 1 && j < nt0) return warp_wait(kPFull, j & 1);
      if (pair && t == 0 && j > 0) return warp_wait(kTurn, (j - 1) & 1);
      return true;
    };
    bool ok = t < nq && warp_wait(kQFull, 0);
    if (ok && nt > 0) {
      ok = k_ready(0) && turn(0);
      if (ok) issue_s(0);
    }
    for (int j = 0; j < nt && ok; ++j) {
      const bool more = j + 1 < nt;
      ok = warp_wait(kVFull + (j & 1), (j >> 1) & 1) && warp_wait(kPFull + 2 * t, j & 1);
      if (ok) issue_pv(j, 0);
      if (more) ok = ok && k_ready(j + 1) && (t == 1 || turn(j + 1));
      ok = ok && warp_wait(kPFull + 2 * t + 1, j & 1);
      if (!ok) break;
      issue_pv(j, 1);
      if (!more) break;
      // S(j+1) overwrites P(j): its P V must be complete
      ok = warp_wait(kPvDone + t, j & 1) && (t == 0 || turn(j + 1));
      if (ok) issue_s(j + 1);
    }
    // tiles that only the other Q tile takes are let go as they land
    if (t < nq)
      for (int j = nt; j < ntiles && ok; ++j) {
        ok = warp_wait(kKFull + (j & 1), (j >> 1) & 1);
        if (ok && lane == 0) mbar_arrive(&bars[kKEmpty + (j & 1)]);
        ok = ok && warp_wait(kVFull + (j & 1), (j >> 1) & 1);
        if (ok && lane == 0) mbar_arrive(&bars[kVEmpty + (j & 1)]);
      }
    if (elect_one()) {
      umma_commit(&bars[kDone + t]);  // completes when every MMA above has finished
      if (!mbar_wait(&bars[kDone + t], 0)) fail();
    }
    __syncwarp();
  } else {
    // ======================= softmax warps ==================================
    const int qt = warp >> 2, qd = warp & 3;
    const int r = qd * 32 + lane;  // row of the Q tile = TMEM lane
    const int nt = qt == nq - 1 ? ntiles : nt0;
    if (qt < nq) {
      const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
      const uint32_t ts = tmem + tmem_s_col(qt) + lane_off;
      const uint32_t to = tmem + tmem_o_col(qt) + lane_off;
      const int row = qt * kRows + r;  // among the CTA's rows
      const int limit = a.causal ? min(L - Q + t0 + row, L - 1) : L - 1;  // last key this row sees
      const int limit_lo = a.causal ? min(L - Q + t0 + qt * kRows, L - 1) : L - 1;
      const float sl2 = a.scale_log2;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < nt; ++j) {
        ok = warp_wait(kSFull + qt, (uint32_t)(j & 1));
        if (!ok) break;
        tc_fence_after();
        // Two passes over S, 64 columns at a time.  The first ends with the columns
        // that the second begins with; the others are read again under its work.
        // (All 128 kept in registers spill at the 168 that 11 warps leave.)
        const int kt = j * kKeys;
        const bool masked = kt + kKeys - 1 > limit_lo;  // warp-uniform
        float m2[2] = {-INFINITY, -INFINITY};
        uint32_t s0[2][32], s1[2][32];
        tmem_ld32(ts + 64, s1[0]);
        tmem_ld32(ts + 96, s1[1]);
        tmem_wait_ld();
        tmem_ld32(ts, s0[0]);
        tmem_ld32(ts + 32, s0[1]);
        if (masked) mask_keys(s1, limit - kt - 64);
#pragma unroll
        for (int i = 0; i < 32; i += 2)
#pragma unroll
          for (int c = 0; c < 2; ++c) m2[c] = fmax3(m2[c], __uint_as_float(s1[c][i]), __uint_as_float(s1[c][i + 1]));
        tmem_wait_ld();
        if (masked) mask_keys(s0, limit - kt);
#pragma unroll
        for (int i = 0; i < 32; i += 2)
#pragma unroll
          for (int c = 0; c < 2; ++c) m2[c] = fmax3(m2[c], __uint_as_float(s0[c][i]), __uint_as_float(s0[c][i + 1]));
        const float mx = fmaxf(m2[0], m2[1]) * sl2;
        // lazy rescale: move the reference only when the tile's maximum exceeds
        // it by more than 2^8 (first tile with a visible key: always).  O_t is
        // at rest here: S_t(j) was issued after P V of tile j-1 completed.
        const bool need = mx > m + kRescaleThreshold;
        float alpha = 1.f;
        if (need) {
          alpha = m == -INFINITY ? 0.f : fast_exp2(m - mx);
          m = mx;
          l *= alpha;
        }
        if (j > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
          for (int c = 0; c < DN / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(to + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st16(to + 16 * c, o);
          }
        }
        // keys past the last one, in the sequence's last tile: zero their V rows
        // (P is 0 there, but 0 * NaN is not).  The warps of the first Q tile that
        // takes the tile do it before its P V.
        if ((j + 1) * kKeys > L && (qt == 0 || j >= nt0) && warp_wait(kVFull + (j & 1), (j >> 1) & 1)) {
          for (int c = 0; c < SH::kVC; ++c) {
            const uint32_t x = (uint32_t)j * SH::kTC + SH::kKC + c;
            const uint32_t vst = ring + (x % SH::kRing) * kChunk;
            for (int i = (L - j * kKeys) * 8 + r; i < kKeys * 8; i += kRows) st_shared_v4(vst + i * 16, 0, 0, 0, 0);
          }
          fence_proxy_async_smem();  // generic-proxy writes -> tensor-core reads
        }
        // P = 2^(s * scale * log2 e - m), key pairs in packed arithmetic; the sum
        // takes the unrounded weights (lse keeps fp32 accuracy), the product P
        // rounded to 16 bits: an error of half a step a weight, of the size of
        // the result's own rounding
        const float ref = m == -INFINITY ? 0.f : m;
        const float2 sl2x2 = make_float2(sl2, sl2), negx2 = make_float2(-ref, -ref);
        float2 psum = make_float2(0.f, 0.f);
        auto weigh = [&](uint32_t (&s)[2][32], int hf) {
          uint32_t w[2][16];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 x = make_float2(__uint_as_float(s[i >> 4][2 * (i & 15)]),
                                         __uint_as_float(s[i >> 4][2 * (i & 15) + 1]));
            const float2 e = __ffma2_rn(x, sl2x2, negx2);
            const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));
            psum = __fadd2_rn(psum, p);
            w[i >> 4][i & 15] = TT::pack(p.x, p.y);
          }
          // over columns already read: keys 64 hf .. go to columns 32 hf ..
          tmem_st16(ts + 32 * hf, w[0]);
          tmem_st16(ts + 32 * hf + 16, w[1]);
          tmem_wait_st();
          tc_fence_before();  // the stores of P (and O) -> the MMA thread
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kPFull + 2 * qt + hf]);  // half of P for the product
        };
        tmem_ld32(ts + 64, s1[0]);
        tmem_ld32(ts + 96, s1[1]);
        weigh(s0, 0);
        tmem_wait_ld();
        if (masked) mask_keys(s1, limit - kt - 64);
        weigh(s1, 1);
        l += psum.x + psum.y;
      }
      // ---- epilogue: O / l -> out ----
      const bool fin = ok && !*abort_flag && (nt == 0 || warp_wait(kPvDone + qt, (uint32_t)((nt - 1) & 1)));
      tc_fence_after();
      const float inv = fin && l > 0.f ? 1.f / l : (l != l ? l : 0.f);
      const bool write = row < ntok;
      const int64_t orow = (int64_t)(q0 + t0 + row) * H + h;
      T *dst = static_cast<T *>(a.out) + orow * DN;
#pragma unroll 1
      for (int c = 0; c < DN / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(to + 32 * c, o);
        tmem_wait_ld();
        if (write) {
          const bool none = inv == 0.f;  // no visible key: O may never have been written
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint4 v;
            v.x = TT::pack(__uint_as_float(o[i + 0]) * inv, __uint_as_float(o[i + 1]) * inv);
            v.y = TT::pack(__uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
            v.z = TT::pack(__uint_as_float(o[i + 4]) * inv, __uint_as_float(o[i + 5]) * inv);
            v.w = TT::pack(__uint_as_float(o[i + 6]) * inv, __uint_as_float(o[i + 7]) * inv);
            if (none) v = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(dst + 32 * c + i) = v;
          }
        }
      }
      if (write && a.lse) a.lse[orow] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : (l != l ? l : -INFINITY);
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// [tokens][heads][width] with token and head strides in elements; box = 128
// tokens of one head x 64 columns.  Tokens past the last read as zero.
template <typename T>
bool make_map3(CUtensorMap *m, const void *p, int width, int heads, int tokens, int64_t head_stride,
               int64_t token_stride) {
  cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)token_stride * 2};
  cuuint32_t box[3] = {64, 1, 128};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn_tc()(m, TcType<T>::kTma, 3, const_cast<void *>(p), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DN>
cudaError_t launch_t(const LatentPrefillArgs &a, cudaStream_t stream) {
  if (!encode_fn_tc()) return cudaErrorNotSupported;
  CUtensorMap tmq, tmk, tmr, tmv;
  // without keys every row is zeros and the K and V maps are never used: they
  // then describe q, so that they are valid
  const bool any = a.num_k_tokens > 0;
  const int64_t qs = DN + 64;
  const void *k = any ? a.k : a.q, *v = any ? a.v : a.q, *kr = any ? a.k_rope : a.q;
  const int heads = any ? a.num_heads : 1, tk = any ? a.num_k_tokens : 1;
  bool ok = make_map3<T>(&tmq, a.q, DN + 64, a.num_heads, a.num_q_tokens, qs, qs * a.num_heads) &&
            make_map3<T>(&tmk, k, DN, heads, tk, any ? a.k_head_stride : qs, any ? a.k_token_stride : qs) &&
            make_map3<T>(&tmv, v, DN, heads, tk, any ? a.v_head_stride : qs, any ? a.v_token_stride : qs);
  if (ok) {
    cuuint64_t dims[2] = {64, (cuuint64_t)tk};
    cuuint64_t strides[1] = {(cuuint64_t)(any ? a.k_rope_stride : qs) * 2};
    cuuint32_t box[2] = {64, 128};
    cuuint32_t estr[2] = {1, 1};
    ok = encode_fn_tc()(&tmr, TcType<T>::kTma, 2, const_cast<void *>(kr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  if (!ok) {
    debug_log("latent_prefill: tensor map refused");
    return cudaErrorInvalidValue;
  }
  auto kern = latent_prefill_kernel<T, DN>;
  constexpr int kSmem = Shape<DN>::kSmem;
  const cudaError_t e = set_smem_limit_once(reinterpret_cast<const void *>(kern), kSmem, true);
  if (e != cudaSuccess) return e;
  const int tiles = (a.max_query_len + kQTiles * kRows - 1) / (kQTiles * kRows);
  const int64_t grid = (int64_t)tiles * a.num_seqs * a.num_heads;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  kern<<<(unsigned)grid, kThreads, kSmem, stream>>>(a, tmq, tmk, tmr, tmv, tiles);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, int dtype, int, cudaStream_t stream) {
  if (dtype == PA_BF16)
    return a.nope_dim == 128 ? launch_t<__nv_bfloat16, 128>(a, stream) : launch_t<__nv_bfloat16, 64>(a, stream);
  return a.nope_dim == 128 ? launch_t<__half, 128>(a, stream) : launch_t<__half, 64>(a, stream);
}

}  // namespace pa
