// latent_prefill.cu -- attention of new tokens in the expanded form on the
// 5th-generation tensor cores.
//
// Head h of a token has a key [k_nope (DN) | k_rope (64, shared by the heads)]
// and a value of DN; row t of a sequence with Q rows and L keys sees the keys
// j <= L-Q+t (causal) or all of them.  With S = scale * Q K^T (base 2 below),
// a running reference m (the maximum, less a headroom) and sum l per row, O =
// sum_j 2^(s_j - m) v_j:
//     out = O / l,  lse = (m + log2 l) ln 2.
//
// An item is (sequence, head, 256 query rows held as two Q tiles of 128).  Per
// 128-key tile j and Q tile t the tensor cores compute S_t = Q_t K_j^T (K =
// DN + 64) and O_t += P_t V_j, fp32 accumulators in tensor memory (128 columns
// each: all 512 are used); P_t (16 bits, two keys a word) overwrites S_t and
// is the A operand of P V from there.  The chains P V_t(j), S_t(j+1), softmax of
// the two Q tiles run side by side, half a step apart, so that the softmax of
// one lies under the products of the other.
//
// Work split.  Where there are items enough to fill the machine a CTA takes one
// item, those with the most keys first (see kMostEmpty).  Few rows over a long prefix would keep
// a few SMs busy: there the key tiles of all items form one line (with one unit
// more an item, for its queries and its epilogue) that is cut into equal ranges,
// one a CTA; an item that lies in one range is written at once, a cut one leaves
// a record (sums, maximum, total) per range, which a second kernel joins in the
// order of the ranges.  For many items the line was slower (256 equal items of
// 130 tiles, which take two rounds on 148 SMs where 1.73 suffice: 640 us against
// 590 at 1965 MHz, 660 in a long run, whose clock the power limit holds at 1750; a
// batch of nine prompts: 141 against 106): cut items cost their records,
// and K and V are read at different places at a time.
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
constexpr float kRescaleThreshold = 8.0f;  // log2 units: P stays <= 2^(8 + headroom) between rescales
constexpr int kSoftmaxWarps = 4 * kQTiles;
constexpr int kProducerWarp = kSoftmaxWarps, kMmaWarp = kSoftmaxWarps + 1;
constexpr int kThreads = 32 * (kSoftmaxWarps + 1 + kQTiles);

// Barriers of K and V are kept by tile parity: the ring holds two
// tiles at most, so that a tile's chunks are asked for only after the products of the
// tile two before have let theirs go.
enum {
  kQFull = 0,
  kQEmpty = 1,                  // both Q tiles' last S of the item done
  kKFull = 2,                   // [2] K of the tile landed
  kVFull = kKFull + 2,          // [2] V of the tile landed
  kKEmpty = kVFull + 2,         // [2] both Q tiles' S done
  kVEmpty = kKEmpty + 2,        // [2] both Q tiles' P V done
  kSFull = kVEmpty + 2,         // [Q tile] S in tensor memory
  kPFull = kSFull + kQTiles,    // [Q tile][half] 64 keys of P written over S (4 warps)
  kPvDone = kPFull + 2 * kQTiles,  // [Q tile] P V complete
  kOFree = kPvDone + kQTiles,   // [Q tile] O of the item has been read out (4 warps)
  kTurn0 = kOFree + kQTiles,    // half of P_0 of the tile is there, for Q tile 1 (4 warps)
  kTurn1 = kTurn0 + 1,          // [4] S_1 is being issued, by its number
  kDone = kTurn1 + 4,           // [Q tile]
  kNumBars = kDone + kQTiles
};

__device__ __forceinline__ uint32_t tmem_s_col(int t) { return (uint32_t)t * 256u; }
__device__ __forceinline__ uint32_t tmem_o_col(int t) { return (uint32_t)t * 256u + 128u; }

// Scores of keys past the last visible one (`last`, counted from the first of
// these 64 columns) become -infinity.
__device__ __forceinline__ void mask_keys(uint32_t (&s)[2][32], int last) {
#pragma unroll
  for (int i = 0; i < 64; ++i)
    if (i > last) s[i >> 5][i & 31] = __float_as_uint(-INFINITY);
}

constexpr int kExtra = 1;       // units an item has beside its tiles
// Units a worker is worth: 1 row of 16 heads over 1024 keys took 20.5 / 22.6 / 26.6
// us at 2 / 3 / 6, 200 rows over 2048 keys 53 / 49 / 51.
constexpr int kMinUnits = 3;
constexpr int kPairRows = kQTiles * kRows, kPairShift = 8;
static_assert(kPairRows == 1 << kPairShift, "rows of an item");
// CTAs of the grid of pairs for each of the grid of places, at most.  A CTA
// without an item holds an SM's shared memory for a microsecond, and there is one
// for every pair that the longest sequence has and another has not: a prompt of
// 8192 rows among 255 single rows, 128 heads, took 10.9 ms by pairs and takes 4.1
// by places, nine prompts of 1000 rows announced as 9000 133 and 108 us.  Where few
// are empty pairs are as fast or faster, the longest items of all sequences being
// first (64 prompts of 128 rows 79 against 82 us, nine of 1000 104 against 109; 32
// of 1 to 2048, nearly half of the CTAs empty, 414 against 398).
constexpr int kMostEmpty = 2;
// Keys of all sequences together from which items are cut: records and joining
// cost about 10 us where a sequence has few rows, 25 to 30 where it has hundreds.
// Cut / whole, us, 16 heads: 1 row over 512 keys 20.5 / 16.4, 1024 22.5 / 24.6,
// 2048 24.6 / 38.9, 16384 53 / 256; 200 rows over 1024 37 / 31, 2048 49 / 49, 8192
// 74 / 168; two sequences of 512 rows over 512 41 / 22.5, 2048 61 / 53, 8192 123 /
// 174.  The host knows the sum of the keys alone, and a long sequence left whole
// costs more than short ones cut.
constexpr int kSplitTokens = 1024, kSplitTokensManyRows = 2048;
constexpr int kManyRows = 128;  // rows a sequence, on average: more than one Q tile

// A cut item's piece, as its worker leaves it for the joining kernel.
struct Piece {
  int valid, last;       // last: the piece ends the item
  int64_t row0;          // the item's first row of out, as token * heads + head
  int nrow;
};

struct Seq {
  int Q, q0, L, k0, pairs;
  bool over;  // more rows than announced: all are zeros
};

__device__ __forceinline__ Seq seq_of(const LatentPrefillArgs &a, int s, unsigned int *err) {
  Seq x;
  x.q0 = a.query_start_loc[s];
  x.Q = a.query_start_loc[s + 1] - x.q0;
  x.k0 = a.context_start_loc[s];
  x.L = a.context_start_loc[s + 1] - x.k0;
  const bool bad = x.q0 < 0 || x.Q < 0 || x.q0 > a.num_q_tokens - x.Q || x.k0 < 0 || x.L < 0 ||
                   x.k0 > a.num_k_tokens - x.L;
  if (bad) x.Q = 0;
  x.over = x.Q > a.max_query_len;
  if (bad || x.over) raise_error(err, PA_DEVERR_QUERY_LEN);
  x.pairs = (x.Q + kPairRows - 1) / kPairRows;
  return x;
}
// Keys that the rows [0, row1) of a sequence see, at most.
__device__ __forceinline__ int keys_of(const LatentPrefillArgs &a, const Seq &x, int row1) {
  return x.over ? 0 : a.causal ? min(x.L, x.L - x.Q + row1) : x.L;
}
__device__ __forceinline__ int tiles_of(const LatentPrefillArgs &a, const Seq &x, int row1) {
  return max(0, (keys_of(a, x, row1) + kKeys - 1) / kKeys);
}
__device__ __forceinline__ int64_t head_units(const LatentPrefillArgs &a, const Seq &x) {
  int64_t n = 0;
  for (int p = 0; p < x.pairs; ++p) n += tiles_of(a, x, min(x.Q, (p + 1) * kPairRows)) + kExtra;
  return n;
}

struct Item {
  Seq x;
  int head, t0, ntok, nq;
  int ntiles, nt0;  // key tiles of the item, of Q tile 0 (Q tile nq-1 takes all of them)
  int j0, j1;       // the worker's piece of them
  __device__ __forceinline__ void set(const LatentPrefillArgs &a, const Seq &s, int h, int pair) {
    x = s;
    head = h;
    t0 = pair * kPairRows;
    ntok = min(kPairRows, s.Q - t0);
    nq = ntok > kRows ? 2 : 1;
    ntiles = tiles_of(a, s, t0 + ntok);
    nt0 = tiles_of(a, s, t0 + min(ntok, kRows));
    j0 = 0;
    j1 = ntiles;
  }
  __device__ __forceinline__ int tiles(int t) const { return t == nq - 1 ? ntiles : t < nq ? nt0 : 0; }
  // Q tile t's tiles within the piece: [j0, end(t))
  __device__ __forceinline__ int end(int t) const { return max(j0, min(j1, tiles(t))); }
};

// The walk over a worker's range.  Every role walks for itself.
struct Walk {
  Seq x;
  int seq, head, pair, off, left;
  __device__ __forceinline__ void start(const LatentPrefillArgs &a, int s, int64_t o, int n) {
    seq = s;
    left = n;
    x = seq_of(a, s, nullptr);
    const int64_t per = head_units(a, x);
    head = (int)(o / per);
    o -= head * per;
    for (pair = 0;; ++pair) {
      const int u = tiles_of(a, x, min(x.Q, (pair + 1) * kPairRows)) + kExtra;
      if (o < u) break;
      o -= u;
    }
    off = (int)o;
  }
  __device__ __forceinline__ bool next(const LatentPrefillArgs &a, Item &it) {
    while (left > 0) {
      if (pair >= x.pairs) {
        pair = 0;
        if (++head >= a.num_heads || x.pairs == 0) {
          head = 0;
          if (++seq >= a.num_seqs) return false;
          x = seq_of(a, seq, nullptr);
        }
        continue;
      }
      it.set(a, x, head, pair);
      const int per = it.ntiles + kExtra, at = off, take = min(left, per - at);
      left -= take;
      off += take;
      if (off == per) {
        off = 0;
        ++pair;
      }
      it.j0 = max(0, at - kExtra);
      it.j1 = max(0, at + take - kExtra);
      if (it.j1 > it.j0 || (it.ntiles == 0 && at == 0)) return true;  // (without keys: zeros)
    }
    return false;
  }
};

struct WalkState {
  Walk walk;
  Item item;
  int more;
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
  static constexpr int kOffWalk = kOffBar + 8 * (kNumBars + 20);  // after the barriers and words
  static constexpr int kSmem = kOffWalk + kSoftmaxWarps * (int)sizeof(WalkState) + 1024;  // + alignment
};
static_assert(Shape<128>::kSmem <= 227 * 1024, "shared memory per CTA");

template <typename T, int DN, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const LatentPrefillArgs a, const __grid_constant__ CUtensorMap tmq,
                          const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmr,
                          const __grid_constant__ CUtensorMap tmv, float *rec, float2 *rec_ml, Piece *pieces,
                          int pairs /* not SPLIT: items of a sequence and head, at most; 0: CTAs by places */) {
  using TT = TcType<T>;
  using SH = Shape<DN>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SH::kOffBar);
  volatile int64_t *scan = reinterpret_cast<volatile int64_t *>(bars + kNumBars);  // [16]
  volatile int64_t *start_off = scan + 16;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kNumBars + 17);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *start_seq = abort_flag + 1;
  const uint32_t sbase = smem_addr(smem);
  const uint32_t ring = sbase + SH::kOffRing;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.num_heads, worker = blockIdx.x;

  if (tid == 0) {
    mbar_init(&bars[kQFull], 1);
    mbar_init(&bars[kQEmpty], 2);
    for (int p = 0; p < 2; ++p) {
      mbar_init(&bars[kKFull + p], 1);
      mbar_init(&bars[kVFull + p], 1);
      mbar_init(&bars[kKEmpty + p], 2);
      mbar_init(&bars[kVEmpty + p], 2);
    }
    for (int t = 0; t < kQTiles; ++t) {
      mbar_init(&bars[kSFull + t], 1);
      mbar_init(&bars[kPFull + 2 * t], 4);
      mbar_init(&bars[kPFull + 2 * t + 1], 4);
      mbar_init(&bars[kPvDone + t], 1);
      mbar_init(&bars[kOFree + t], 4);
      mbar_init(&bars[kDone + t], 1);
    }
    mbar_init(&bars[kTurn0], 4);
    for (int i = 0; i < 4; ++i) mbar_init(&bars[kTurn1 + i], 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  int64_t lo = 0, hi = 0;
  Item it;  // the CTA's one item, or the item that a role's walk has come to
  if constexpr (!SPLIT) {
    // ---- the CTA's item; those with the most keys come first (by places: first
    // within their sequence) ---------------------------------------------------
    int seq, pair, step;
    if (pairs) {
      const int per_pair = a.num_seqs * H;
      seq = worker % per_pair / H;
      pair = pairs - 1 - worker / per_pair;
      step = pairs;
    } else {
      const int place = worker / H;
      seq = seq_of_place(a.query_start_loc, a.num_seqs, 1, kPairShift, place);
      pair = (int)(place - first_place(a.query_start_loc, seq, 1, kPairShift));
      step = 0x7fffffff;
      // there are at least as many CTAs as sequences: each looks one over
      if (tid == 0 && worker < a.num_seqs) seq_of(a, worker, a.err);
    }
    const Seq x = seq_of(a, seq, pairs && tid == 0 ? a.err : nullptr);
    if (pair < 0 || pair >= x.pairs) return;  // CTA-uniform, before tensor memory is taken
    if (!pairs) pair = x.pairs - 1 - pair;
    it.set(a, x, worker % H, pair);
    if (it.ntiles == 0) {
      // zeros; a sequence with more rows than announced has more items than a grid of pairs
      for (int64_t p = pair; p < x.pairs; p += step)
        for (int i = tid; i < min(kPairRows, x.Q - (int)p * kPairRows) * DN; i += kThreads) {
          const int64_t orow = (x.q0 + p * kPairRows + i / DN) * H + it.head;
          static_cast<T *>(a.out)[orow * DN + i % DN] = Elem<T>::from_f(0.f);
          if (a.lse && i % DN == 0) a.lse[orow] = -INFINITY;
        }
      return;
    }
  } else {
    // ---- the worker's range of units ----------------------------------------
    if (tid < 2) pieces[worker * 2 + tid].valid = 0;
    unsigned int *err0 = worker == 0 ? a.err : nullptr;
    int64_t sum = 0, first_units = 0;
    for (int s = tid; s < a.num_seqs; s += kThreads) {
      const int64_t n = head_units(a, seq_of(a, s, err0)) * H;
      if (s == tid) first_units = n;
      sum += n;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) scan[warp] = sum;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < kThreads / 32; ++w) total += scan[w];
    const int64_t worth = (total + kMinUnits - 1) / kMinUnits;
    const int workers = (int)min((int64_t)gridDim.x, worth);
    lo = worker < workers ? total * worker / workers : 0;
    hi = worker < workers ? total * (worker + 1) / workers : 0;
    if (lo >= hi) return;  // CTA-uniform, before tensor memory is taken
    int64_t base = 0;
    for (int s0 = 0; s0 < a.num_seqs && base <= lo; s0 += kThreads) {  // CTA-uniform
      const int s = s0 + tid;
      const int64_t n = s0 == 0 ? first_units : s < a.num_seqs ? head_units(a, seq_of(a, s, nullptr)) * H : 0;
      int64_t x = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      __syncthreads();  // the previous use of scan[] is over
      if (lane == 31) scan[warp] = x;
      __syncthreads();
      int64_t before = base;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += scan[w];
        base += scan[w];
      }
      before += x - n;
      if (before <= lo && lo < before + n) {
        *start_seq = s;
        *start_off = lo - before;
      }
    }
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

  Walk walk;
  if (SPLIT && warp >= kSoftmaxWarps) walk.start(a, *start_seq, *start_off, (int)(hi - lo));

  if (warp == kProducerWarp) {
    // ======================= producer =======================================
    uint32_t x = 0;                // chunk
    uint32_t g = 0, items = 0;     // tile, item
    int last_k = -1, last_v = -1;  // last tile whose K (V) was announced in full
    bool ok = true;
    for (bool more = !SPLIT || walk.next(a, it); ok && more; more = SPLIT && walk.next(a, it)) {
      if (it.j1 == it.j0) continue;
      ok = warp_wait(kQEmpty, (items & 1) ^ 1);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[kQFull], it.nq * SH::kQBytes);
        for (int t = 0; t < it.nq; ++t)
          for (int c = 0; c < SH::kKC; ++c)
            tma_load_3d(sbase + t * SH::kQBytes + c * kChunk, &tmq, c * 64, it.head,
                        it.x.q0 + it.t0 + t * kRows, &bars[kQFull]);
      }
      __syncwarp();
      ++items;
      for (int j = it.j0; j < it.j1 && ok; ++j, ++g) {
        const int row = it.x.k0 + j * kKeys, p = g & 1;
#pragma unroll
        for (int c = 0; c < SH::kTC; ++c, ++x) {
          if (x >= SH::kRing) {  // the chunk kRing before has been let go with its tile's K or V
            const uint32_t tj = (x - SH::kRing) / SH::kTC, tc = (x - SH::kRing) % SH::kTC;
            ok = warp_wait((tc < SH::kKC ? kKEmpty : kVEmpty) + (tj & 1), (tj >> 1) & 1);
            if (!ok) break;
          }
          if (lane == 0) {
            const uint32_t dst = ring + (x % SH::kRing) * kChunk;
            uint64_t *bar = &bars[(c < SH::kKC ? kKFull : kVFull) + p];
            if (c == 0) mbar_arrive_expect_tx(bar, SH::kKC * kChunk);
            if (c == SH::kKC) mbar_arrive_expect_tx(bar, SH::kVC * kChunk);
#ifdef PA_TEST_LOST_COPY
            // test build only: the first chunk of tile PA_TEST_LOST_COPY of CTA 0
            // is announced but never copied, so that the waits for it expire
            if (worker == 0 && x == (uint32_t)(PA_TEST_LOST_COPY * SH::kTC)) {
            } else
#endif
            if (c < SH::kKC - 1) tma_load_3d(dst, &tmk, c * 64, it.head, row, bar);
            else if (c == SH::kKC - 1) tma_load_2d(dst, &tmr, 0, row, bar);
            else tma_load_3d(dst, &tmv, (c - SH::kKC) * 64, it.head, row, bar);
          }
          __syncwarp();
          if (c == SH::kKC - 1) last_k = (int)g;
          if (c == SH::kTC - 1) last_v = (int)g;
        }
        if (!ok) break;
      }
    }
    // Every copy has landed before the CTA can exit.  After a failure part of a
    // tile's chunks may be on their way under a barrier that waits for the
    // others too: what is missing is taken off it.
    if (lane == 0) {
      if (!ok) {
        const int j = (int)(x / SH::kTC), c = (int)(x % SH::kTC);
        if (c > 0 && c < SH::kKC) mbar_complete_tx(&bars[kKFull + (j & 1)], (SH::kKC - c) * kChunk), last_k = j;
        if (c > SH::kKC) mbar_complete_tx(&bars[kVFull + (j & 1)], (SH::kTC - c) * kChunk), last_v = j;
      }
      bool landed = items == 0 || mbar_wait(&bars[kQFull], (items - 1) & 1);
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
    const uint32_t a_lo = umma_desc_lo(sbase + t * SH::kQBytes, 16);
    const uint32_t k_lo = umma_desc_lo(ring, 16), v_lo = umma_desc_lo(ring, kChunk);
    uint32_t sn = 0;  // S products issued
    // S_t = Q_t K^T of tile g: both K-major, 8-row groups 1 KB apart
    auto issue_s = [&](uint32_t g, bool last) {
      const uint32_t x0 = g * SH::kTC;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t d = tmem + tmem_s_col(t);
        if (t == 1) mbar_arrive(&bars[kTurn1 + (sn & 3)]);
#pragma unroll
        for (int c = 0; c < SH::kKC; ++c) {
          const uint32_t b_lo = k_lo + ((x0 + c) % SH::kRing) * (kChunk >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_lo(d, a_lo + ((c * kChunk + kk * 32) >> 4), kHi, b_lo + ((kk * 32) >> 4), kHi, idesc_s,
                    (c | kk) ? 1u : 0u);
        }
        umma_commit(&bars[kSFull + t]);
        umma_commit(&bars[kKEmpty + (g & 1)]);
        if (last) umma_commit(&bars[kQEmpty]);
      }
      __syncwarp();
      ++sn;
    };
    // O_t += P_t V: A = P from tensor memory (16 keys in 8 columns), B = V with
    // columns contiguous, 64 of them a product, 8-key groups 1 KB apart
    auto issue_pv = [&](uint32_t g, int half, bool first) {
      const uint32_t x0 = g * SH::kTC + SH::kKC;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t keep = first ? 0u : 1u;
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
          umma_commit(&bars[kVEmpty + (g & 1)]);
        }
      }
      __syncwarp();
    };
    // The two chains are kept half a step apart: S_1(j) is issued when half of
    // P_0(j) is there, S_0(j+1) when S_1(j) has been issued.  In step they would
    // meet at the exponentials (16 a cycle and SM: 1024 cycles for a tile of 128
    // x 128), then leave those units idle together.  Both signals are counted
    // and waited for one by one, so that no phase of theirs is skipped, and
    // neither side can overtake a wait: P_0's signal is never more than one
    // ahead, S_1's never more than three (two tiles of an item that Q tile 0 has
    // done with, one of the next), for which it has four barriers.
    uint32_t g0 = 0;             // tile number of the item's first
    uint32_t n = 0;              // tiles of this Q tile so far
    uint32_t items = 0, mine = 0;  // items, those with tiles of this Q tile
    uint32_t turns = 0;          // signals of the other waited for
    uint32_t ones = 0;           // t == 0: S_1 products that come before the next S_0
    bool ok = true;
    for (bool go = !SPLIT || walk.next(a, it); ok && go; go = SPLIT && walk.next(a, it)) {
      const int j0 = it.j0, j1 = it.j1, nt = it.end(t), nt0 = it.end(0), nt1 = it.nq == 2 ? it.end(1) : j0;
      if (j1 == j0) continue;
      auto tile = [&](int j) { return g0 + (uint32_t)(j - j0); };
      auto k_ready = [&](int j) { return warp_wait(kKFull + (tile(j) & 1), (tile(j) >> 1) & 1); };
      auto turn = [&](int j) {  // before S_t(j)
        bool go = true;
        if (t == 1 && j < nt0) go = warp_wait(kTurn0, turns++ & 1);
        if (t == 0)
          for (const uint32_t want = ones + (uint32_t)min(j - j0, nt1 - j0); go && turns < want; ++turns)
            go = warp_wait(kTurn1 + (turns & 3), (turns >> 2) & 1);
        return go;
      };
      ok = warp_wait(kQFull, items & 1);
      if (ok && nt > j0) {
        ok = k_ready(j0) && turn(j0);
        if (ok) issue_s(tile(j0), nt == j0 + 1);
      } else if (ok && lane == 0) {
        mbar_arrive(&bars[kQEmpty]);
      }
      for (int j = j0; j < nt && ok; ++j, ++n) {
        const uint32_t g = tile(j);
        const bool more = j + 1 < nt;
        ok = warp_wait(kVFull + (g & 1), (g >> 1) & 1);
        if (j == j0) ok = ok && warp_wait(kOFree + t, (mine & 1) ^ 1);  // O of the item before has been read out
        ok = ok && warp_wait(kPFull + 2 * t, n & 1);
        if (!ok) break;
        issue_pv(g, 0, j == j0);
        if (more) ok = k_ready(j + 1) && (t == 1 || turn(j + 1));
        ok = ok && warp_wait(kPFull + 2 * t + 1, n & 1);
        if (!ok) break;
        issue_pv(g, 1, false);
        // S(j+1), of the next item too, overwrites P(j): its P V must be complete
        ok = warp_wait(kPvDone + t, n & 1);
        if (more) {
          ok = ok && (t == 0 || turn(j + 1));
          if (ok) issue_s(tile(j + 1), j + 2 == nt);
        }
      }
      // tiles that only the other Q tile takes are let go as they land
      for (int j = nt; j < j1 && ok; ++j) {
        ok = k_ready(j);
        if (ok && lane == 0) mbar_arrive(&bars[kKEmpty + (tile(j) & 1)]);
        ok = ok && warp_wait(kVFull + (tile(j) & 1), (tile(j) >> 1) & 1);
        if (ok && lane == 0) mbar_arrive(&bars[kVEmpty + (tile(j) & 1)]);
      }
      if (ok && t == 0) ok = turn(j1);  // all of the item's
      mine += nt > j0;
      ones += (uint32_t)(nt1 - j0);
      ++items;
      g0 += (uint32_t)(j1 - j0);
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
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    const uint32_t ts = tmem + tmem_s_col(qt) + lane_off;
    const uint32_t to = tmem + tmem_o_col(qt) + lane_off;
    const float sl2 = a.scale_log2;
    uint32_t g0 = 0, n = 0;  // tile number of the item's first; tiles of this Q tile so far
    bool ok = true;
    // These warps have no registers to spare across the tile loop: their walk
    // lies in shared memory and lane 0 takes its steps.
    WalkState &state = reinterpret_cast<WalkState *>(smem + SH::kOffWalk)[warp];
    if (SPLIT && lane == 0) state.walk.start(a, *start_seq, *start_off, (int)(hi - lo));
    for (bool go = true; go; go = SPLIT) {
      if constexpr (SPLIT) {
        __syncwarp();
        if (lane == 0) state.more = state.walk.next(a, state.item);
        __syncwarp();
        if (!state.more) break;
        it = state.item;
      }
      const int L = it.x.L, j0 = it.j0, nt = it.end(qt);
      // last key the tile's first row sees, and this one
      const int limit_lo = a.causal ? min(L - it.x.Q + it.t0 + qt * kRows, L - 1) : L - 1;
      const int limit = a.causal ? min(limit_lo + r, L - 1) : L - 1;
      float m = -INFINITY, l = 0.f;
      for (int j = j0; j < nt && ok; ++j, ++n) {
        const uint32_t g = g0 + (uint32_t)(j - j0);
        ok = warp_wait(kSFull + qt, n & 1);
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
        const float mx = fmaxf(m2[0], m2[1]) * sl2 - TT::kHeadroom;
        // lazy rescale: move the reference only when the tile's maximum, kHeadroom
        // below it, exceeds it by more than 2^8 (first tile with a visible key:
        // always).  O_t is at rest here: S_t(j) was issued after P V of tile j-1
        // completed.
        const bool need = mx > m + kRescaleThreshold;
        float alpha = 1.f;
        if (need) {
          alpha = m == -INFINITY ? 0.f : fast_exp2(m - mx);
          m = mx;
          l *= alpha;
        }
        if (j > j0 && __any_sync(0xffffffffu, need)) {
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
        if ((j + 1) * kKeys > L && (qt == 0 || j >= it.end(0)) && warp_wait(kVFull + (g & 1), (g >> 1) & 1)) {
          for (int c = 0; c < SH::kVC; ++c) {
            const uint32_t x = g * SH::kTC + SH::kKC + c;
            const uint32_t vst = ring + (x % SH::kRing) * kChunk;
            for (int i = (L - j * kKeys) * 8 + r; i < kKeys * 8; i += kRows) st_shared_v4(vst + i * 16, 0, 0, 0, 0);
          }
          fence_proxy_async_smem();  // generic-proxy writes -> tensor-core reads
        }
        // P = 2^(s * scale * log2 e - m), key pairs in packed arithmetic; the sum
        // takes the unrounded weights (lse keeps fp32 accuracy), the product P
        // rounded to 16 bits: an error of half a step a weight, of the size of
        // the result's own rounding.  f16 weights that fall below its normal range
        // lose at most 2^-25 each, 2^-32 of the largest with the headroom.
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
            w[i >> 4][i & 15] = TT::weights(p.x, p.y);
          }
          // over columns already read: keys 64 hf .. go to columns 32 hf ..
          tmem_st16(ts + 32 * hf, w[0]);
          tmem_st16(ts + 32 * hf + 16, w[1]);
          tmem_wait_st();
          tc_fence_before();  // the stores of P (and O) -> the MMA thread
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars[kPFull + 2 * qt + hf]);  // half of P for the product
            if (hf == 0 && qt == 0 && it.nq == 2) mbar_arrive(&bars[kTurn0]);
          }
        };
        tmem_ld32(ts + 64, s1[0]);
        tmem_ld32(ts + 96, s1[1]);
        weigh(s0, 0);
        tmem_wait_ld();
        if (masked) mask_keys(s1, limit - kt - 64);
        weigh(s1, 1);
        l += psum.x + psum.y;
      }
      // ---- epilogue: O / l -> out, or a record ----
      const bool some = nt > j0;  // else O holds nothing of this item
      if (some && ok) ok = warp_wait(kPvDone + qt, (n - 1) & 1);
      const bool fin = ok && !*abort_flag;
      tc_fence_after();
      if constexpr (SPLIT) it = state.item;
      const int row = qt * kRows + r;  // among the item's rows
      const int64_t orow = (int64_t)(it.x.q0 + it.t0 + row) * H + it.head;
      T *dst = static_cast<T *>(a.out) + orow * DN;
      const bool write = row < it.ntok, whole = j0 == 0 && it.j1 == it.ntiles;
      const int64_t slot = (int64_t)worker * 2 + (j0 == 0 ? 1 : 0);
      // an item whose waits ran out has no sum: zeros, and -infinity as lse
      const float inv = !fin ? 0.f : l > 0.f ? 1.f / l : (l != l ? l : 0.f);
      const bool none = !some || inv == 0.f;  // no visible key
      if (whole || it.ntiles == 0) {
#pragma unroll 1
        for (int c = 0; c < DN / 32; ++c) {
          uint32_t o[32];
          if (some) {
            tmem_ld32(to + 32 * c, o);
            tmem_wait_ld();
          }
          if (!write) continue;
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
        if (write && a.lse)
          a.lse[orow] = !fin ? -INFINITY : l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : (l != l ? l : -INFINITY);
      } else if constexpr (SPLIT) {
        const int64_t rrow = slot * kPairRows + row;
        if (write) rec_ml[rrow] = make_float2(m, fin ? l : -1.f);  // a negative sum marks a failure
#pragma unroll 1
        for (int c = 0; c < DN / 32 && some; ++c) {
          uint32_t o[32];
          tmem_ld32(to + 32 * c, o);
          tmem_wait_ld();
          if (!write) continue;
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4 *>(rec + rrow * DN + 32 * c + i) =
                make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]),
                            __uint_as_float(o[i + 3]));
        }
        if (tid == 0) {
          Piece &p = pieces[slot];
          p.last = it.j1 == it.ntiles;
          p.row0 = (int64_t)(it.x.q0 + it.t0) * H + it.head;
          p.nrow = it.ntok;
          p.valid = 1;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (some && lane == 0) mbar_arrive(&bars[kOFree + qt]);
      g0 += (uint32_t)(it.j1 - it.j0);
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// Joins the pieces of a cut item: CTA (w, c) takes rows c, c + gridDim.y, ... of
// the item that worker w began and did not end, a warp a row.
constexpr int kJoinWarps = 8;
template <typename T, int DN>
__global__ void __launch_bounds__(32 * kJoinWarps)
    latent_prefill_join_kernel(const LatentPrefillArgs a, const float *rec, const float2 *rec_ml, const Piece *pieces) {
  constexpr int V = DN / 64;  // float2 a lane: values lane * 2 + 64 v
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int w = blockIdx.x;
  const Piece head = pieces[w * 2 + 1];
  if (!head.valid) return;
  const int lane = threadIdx.x & 31;
  for (int row = (int)blockIdx.y * kJoinWarps + (int)(threadIdx.x >> 5); row < head.nrow;
       row += (int)gridDim.y * kJoinWarps) {
    float2 o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = make_float2(0.f, 0.f);
    float M = -INFINITY, l = 0.f;
    bool bad = false, more = true;
    // the pieces after the first are the next workers' first ones
    for (int64_t slot = (int64_t)w * 2 + 1; more; slot = slot == (int64_t)w * 2 + 1 ? slot + 1 : slot + 2) {
      const int64_t k = slot * kPairRows + row;
      const float2 ml = rec_ml[k];
      float2 p[V];
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] = __ldcs(reinterpret_cast<const float2 *>(rec + k * DN + v * 64 + lane * 2));
      more = !pieces[slot].last;
      bad = bad || ml.y < 0.f;
      // a piece without a visible key has no sums (a NaN total is not one)
      if (ml.x == -INFINITY && ml.y <= 0.f) continue;
      const float top = fmaxf(M, ml.x);
      const float f0 = M == -INFINITY ? 0.f : exp2f(M - top), f = exp2f(ml.x - top);
      M = top;
      l = l * f0 + f * ml.y;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        o[v].x = o[v].x * f0 + f * p[v].x;
        o[v].y = o[v].y * f0 + f * p[v].y;
      }
    }
    const int64_t orow = head.row0 + (int64_t)row * a.num_heads;
    const bool none = bad || l == 0.f;
    const float inv = 1.f / l;
#pragma unroll
    for (int v = 0; v < V; ++v)
      *reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + orow * DN + v * 64 + lane * 2) =
          none ? 0u : TcType<T>::pack(o[v].x * inv, o[v].y * inv);
    if (a.lse && lane == 0) a.lse[orow] = none ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
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

// Items are cut where, counted from above, they do not fill the machine and a
// sequence can be long enough to be worth it.
bool splits(int num_seqs, int num_q_tokens, int num_k_tokens, int num_heads, int sm_count) {
  const int64_t most = (int64_t)num_heads * ((int64_t)num_q_tokens / kPairRows + num_seqs);
  const bool many = num_q_tokens > (int64_t)kManyRows * num_seqs;
  return most < sm_count && num_k_tokens >= (many ? kSplitTokensManyRows : kSplitTokens);
}

struct PrefillWs {
  size_t pieces, ml, rec, total;
};
PrefillWs prefill_ws(int nope_dim, int sm_count) {
  PrefillWs w;
  const size_t rows = (size_t)sm_count * 2 * kPairRows;
  w.pieces = 0;
  w.ml = ((size_t)sm_count * 2 * sizeof(Piece) + 255) / 256 * 256;
  w.rec = w.ml + rows * sizeof(float2);
  w.total = w.rec + rows * nope_dim * sizeof(float);
  return w;
}

template <typename T, int DN>
cudaError_t launch_t(const LatentPrefillArgs &a, int sm_count, cudaStream_t stream) {
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
  const bool split = splits(a.num_seqs, a.num_q_tokens, a.num_k_tokens, a.num_heads, sm_count);
  auto kern = split ? latent_prefill_kernel<T, DN, true> : latent_prefill_kernel<T, DN, false>;
  constexpr int kSmem = Shape<DN>::kSmem;
  const cudaError_t e = set_smem_limit_once(reinterpret_cast<const void *>(kern), kSmem, true);
  if (e != cudaSuccess) return e;
  const PrefillWs w = prefill_ws(DN, sm_count);
  char *ws = static_cast<char *>(a.ws);
  float *rec = reinterpret_cast<float *>(ws + w.rec);
  float2 *ml = reinterpret_cast<float2 *>(ws + w.ml);
  Piece *pieces = reinterpret_cast<Piece *>(ws + w.pieces);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  // One CTA a (pair of Q tiles, sequence, head), or one a (place, head) where that
  // leaves many CTAs without an item.  The latter fit a grid: the entry point holds
  // rows * heads and sequences * heads to 2^30 each.
  const int64_t places = (int64_t)a.num_q_tokens / kPairRows + a.num_seqs;
  int pairs = (a.max_query_len + kPairRows - 1) / kPairRows;
  int64_t grid = (int64_t)pairs * a.num_seqs * a.num_heads;
  if (split || grid > kMostEmpty * places * a.num_heads || grid > 0x7fffffff) {
    pairs = 0;
    grid = split ? sm_count : places * a.num_heads;
  }
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  const cudaError_t e2 = cudaLaunchKernelEx(&cfg, kern, a, tmq, tmk, tmr, tmv, rec, ml, pieces, pairs);
  if (e2 != cudaSuccess || !split) return e2;
  cfg.gridDim = dim3((unsigned)sm_count, 4);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, latent_prefill_join_kernel<T, DN>, a, (const float *)rec, (const float2 *)ml,
                            (const Piece *)pieces);
}

}  // namespace

size_t latent_prefill_ws(int num_seqs, int num_q_tokens, int num_k_tokens, int num_heads, int nope_dim, int sm_count) {
  return splits(num_seqs, num_q_tokens, num_k_tokens, num_heads, sm_count) ? prefill_ws(nope_dim, sm_count).total : 0;
}

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, int dtype, int sm_count, cudaStream_t stream) {
  if (dtype == PA_BF16)
    return a.nope_dim == 128 ? launch_t<__nv_bfloat16, 128>(a, sm_count, stream)
                             : launch_t<__nv_bfloat16, 64>(a, sm_count, stream);
  return a.nope_dim == 128 ? launch_t<__half, 128>(a, sm_count, stream) : launch_t<__half, 64>(a, sm_count, stream);
}

}  // namespace pa
