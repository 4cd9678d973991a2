// latent_decode.cu -- attention over the paged latent cache in the absorbed
// form, on the 5th-generation tensor cores.
//
// Row r of a sequence is (token t, head h), r = t * H + h; its query q_r has R
// latent and 64 rope values, as every cache row c_j does, and it sees the keys
// j <= L-Q+t:
//     s_rj = scale * q_r . c_j,  out_r = sum_j softmax(s_r)_j c_j[0..R)
// The cache row is key and value at once, so a tile of keys is read once from
// memory and used by two products.
//
// A CTA holds NR query rows (16, 32 or 64) in shared memory and streams tiles
// of KT keys (32 for R = 512, 64 for 256).  What shapes the products is tensor
// memory: 128 rows of R = 512 fp32 sums would fill all of its 512 columns and
// leave none for S, so the second product is turned round:
//     S   [rows x keys] = Q C^T           M 64, N KT, K R+64
//     O^T [values x rows] += C^T P^T      M 128 (R/128 times), N NR, K KT
// O^T takes NR columns per 128 values (256 columns at NR 64, R 512) beside two
// buffers of S.  A row of S lies in four threads of a warp (its quarter holds 16
// rows, read as 16 lanes x KT columns so that all 32 threads have work), so the
// softmax needs two shuffles and, for the rare rescaling of O^T, whose rows lie
// across all threads, one vote.  P goes to shared memory in the K-major layout
// that the B operand wants.  C is read from shared memory as it lies: K-major
// for S, values-contiguous as the A operand of O^T.
//
// Keys arrive by TMA through the block table, one box a block: a 4-D view of
// the cache splits rows into groups of 8 and each row into 64-value pieces, so
// that a box lands as [8-key group][piece][8 keys][128 B] with one stride
// between groups across the blocks of a tile.
//
// Work split: the tiles of all sequences form one line that is cut into equal
// ranges (see Line).  A sequence that lies in one range is written at once; a
// cut one leaves a record (sums, maximum, total) per range, and the merge kernel
// joins them in the order of the ranges.
//
// Bound: memory (each row of the cache once) up to about 32 rows a sequence: 256
// ragged sequences of 16 heads and 512 values, 320 MB, take 70 us (4.6 TB/s with
// the merge, tiles arriving at 7 TB/s in between); beyond that the issue of S (36
// products a tile, 28 cycles each): 64 sequences of 2048 to 8192 keys and 128
// heads take 143 us (670 TFLOP/s) at 1965 MHz, 163 (590) in a long run of them,
// whose clock sinks to about 1800.  With 256 values a tile's softmax is the
// longest step (1800 cycles for 64 rows x 64 keys).
#include <limits.h>

#include "latent.h"
#include "pa_device.cuh"
#include "tc_common.cuh"

namespace pa {
namespace {

constexpr float kRescaleThreshold = 8.0f;  // log2 units: P stays <= 2^(8 + headroom) between rescales
constexpr int kProducerWarp = 4, kSWarp = 5, kPvWarp = 6;
constexpr int kThreads = 224;
constexpr int kMaxSmem = 227 * 1024;
constexpr int kBadSlots = 16;  // more than the items the producer can be ahead by
constexpr int kMaxStages = 6;

// KT keys a tile
template <int R, int NR, int KT>
struct Shape {
  static constexpr int kD = R + 64;
  static constexpr int kPieces = kD / 64;         // 64-value pieces of a row
  static constexpr int kGroup = kPieces * 1024;   // bytes of 8 keys
  static constexpr int kStage = KT / 8 * kGroup;
  static constexpr int kQPiece = NR * 128;        // one piece of the Q rows
  static constexpr int kQBytes = kPieces * kQPiece;
  // two buffers of P: 128-byte rows of 64 keys each, or of the two halves of one
  static constexpr int kPBytes = (KT == 64 ? 2 : 1) * NR * 128;
  static constexpr int kPNext = KT == 64 ? NR * 128 : 64;
  static constexpr int kFixed = 1024 /* alignment */ + kPBytes + 2048 /* barriers, row state */;
  // two Q buffers where enough stages still fit
  static constexpr int kWant = KT == 64 ? 3 : 4;
  static constexpr int kQBufs = kFixed + 2 * kQBytes + kWant * kStage <= kMaxSmem ? 2 : 1;
  static constexpr int kRoom = (kMaxSmem - kFixed - kQBufs * kQBytes) / kStage;
  static constexpr int kStages = kRoom < kMaxStages ? kRoom : kMaxStages;
  static constexpr int kOffQ = 0;
  static constexpr int kOffStage = kQBufs * kQBytes;
  static constexpr int kOffP = kOffStage + kStages * kStage;
  static constexpr int kOffBar = kOffP + kPBytes;
  static constexpr int kSmem = kOffBar + 2048 + 1024;
  static constexpr int kMTiles = R / 128;
  static_assert(kStages >= 2 && kSmem <= kMaxSmem, "two stages");
  // the S product reads 64 rows from each Q piece: with fewer it runs into what
  // follows (never past the allocation), and those rows of S are not used
  static_assert(kOffQ + kQBufs * kQBytes + 64 * 128 <= kSmem, "Q reads stay inside");
};

enum {
  kQFull = 0,                      // [2]
  kQEmpty = 2,                     // [2]
  kFull = 4,                       // [kMaxStages]
  kEmpty = kFull + kMaxStages,     // [kMaxStages]
  kSFull = kEmpty + kMaxStages,    // [2]
  kSEmpty = kSFull + 2,            // [2]
  kPFull = kSEmpty + 2,            // [2]
  kPvDone = kPFull + 2,            // [2]
  kOFree = kPvDone + 2,
  kDone = kOFree + 1,              // [2]
  kNumBars = kDone + 2
};
// words after the barriers
constexpr int kWSlot = 2 * kNumBars;             // TMEM address
constexpr int kWAbort = kWSlot + 1;
constexpr int kWBad = kWAbort + 1;               // [kBadSlots]
constexpr int kWStart = kWBad + kBadSlots;       // [2] first sequence, its first unit
constexpr int kWScan = kWStart + 2;              // [8] block scan
constexpr int kWAlpha = kWScan + 8;              // [2][64] rescale factors, by tile parity
constexpr int kWInv = kWAlpha + 128;             // [2][64] 1 over the sums, by item parity
static_assert((kWInv + 128) * 4 <= 2048, "row state");

constexpr uint32_t kTmemO = 128;  // S: columns 0..127

struct Seq {
  int tiles, L, q0, Q;
};

// How the work is laid out in a line of units: an item (a sequence's tiles for
// one row tile) has one unit a tile and `extra` for what it costs beside them.
// Lockstep: a sequence is one item and each worker is `lanes` CTAs, one per row
// tile, that read the same keys at the same time (one of them from memory).  Flat
// (lanes 1): a sequence is an item per row tile it really has, and a worker is
// one CTA; for batches whose sequences differ in rows.
struct Line {
  int workers, lanes, flat, nr, kt, extra;
  __device__ __forceinline__ int row_tiles(const Seq &x, int heads) const {
    return flat ? (x.Q * heads + nr - 1) / nr : 1;
  }
  __device__ __forceinline__ int units(const Seq &x, int heads) const {
    return x.tiles ? (x.tiles + extra) * row_tiles(x, heads) : 0;
  }
};

// Sequence s as the kernels take it: no tiles if it has no keys, no rows, or
// anything about it is out of range.
__device__ __forceinline__ Seq seq_of(const LatentArgs &a, const Line &ln, int s, unsigned int *err) {
  Seq x;
  x.q0 = s;
  x.Q = 1;
  x.L = a.context_lens[s];
  if (a.query_start_loc) {
    x.q0 = a.query_start_loc[s];
    x.Q = a.query_start_loc[s + 1] - x.q0;
  }
  unsigned int bad = 0;
  if (x.q0 < 0 || x.Q < 0 || x.q0 > a.num_q_tokens - x.Q) {
    bad = PA_DEVERR_QUERY_LEN;
    x.Q = 0;
  } else if (x.Q > a.max_query_len) {
    bad = PA_DEVERR_QUERY_LEN;
  }
  if (x.L < 0 || x.L > a.max_context_len) bad |= PA_DEVERR_CONTEXT_LEN;
  if (bad) raise_error(err, bad);
  x.tiles = bad || x.Q == 0 ? 0 : (x.L + ln.kt - 1) / ln.kt;
  return x;
}

// A warp's walk over its worker's range: items (sequence, row tile, tiles [t0,
// t1)).  32 sequences are read at once, one a lane.
struct Walk {
  const LatentArgs &a;
  const Line &ln;
  int base;
  Seq mine;
  int seq, off, left, lane_rt;
  // the item
  Seq x;
  int first_row, t0, t1;
  __device__ __forceinline__ Walk(const LatentArgs &args, const Line &line, int s, int o, int n, int rt)
      : a(args), ln(line), seq(s), off(o), left(n), lane_rt(rt) {
    load(s);
    t0 = t1 = first_row = 0;
    x = Seq{0, 0, 0, 0};
  }
  __device__ __forceinline__ void load(int s) {
    base = s;
    const int i = s + (int)(threadIdx.x & 31);
    mine = Seq{0, 0, 0, 0};
    if (i < a.num_seqs) mine = seq_of(a, ln, i, nullptr);
  }
  __device__ __forceinline__ bool next() {
    while (left > 0 && seq < a.num_seqs) {
      if (seq >= base + 32) load(seq);
      x.tiles = __shfl_sync(0xffffffffu, mine.tiles, seq - base);
      x.L = __shfl_sync(0xffffffffu, mine.L, seq - base);
      x.q0 = __shfl_sync(0xffffffffu, mine.q0, seq - base);
      x.Q = __shfl_sync(0xffffffffu, mine.Q, seq - base);
      if (off >= ln.units(x, a.num_heads)) {
        ++seq;
        off = 0;
        continue;
      }
      const int per = x.tiles + ln.extra;
      const int rt = ln.flat ? off / per : 0;
      const int at = off - rt * per;
      const int take = min(left, per - at);
      off += take;
      left -= take;
      t0 = max(0, at - ln.extra);
      t1 = max(0, at + take - ln.extra);
      first_row = (rt + lane_rt) * ln.nr;
      if (t1 > t0 && first_row < x.Q * a.num_heads) return true;
    }
    return false;
  }
};

__device__ __forceinline__ void tmem_ld_s(uint32_t addr, uint32_t (&r)[32]) { tmem_ld16x64(addr, r); }
__device__ __forceinline__ void tmem_ld_s(uint32_t addr, uint32_t (&r)[16]) { tmem_ld16x32(addr, r); }

// any thread's pred over the 128 softmax threads
__device__ __forceinline__ bool vote_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred)
      : "memory");
  return r != 0;
}

template <typename T, int R, int NR, int KT, int BS>
__global__ void __launch_bounds__(kThreads, 1)
    latent_decode_kernel(const LatentArgs a, const __grid_constant__ CUtensorMap tmq,
                         const __grid_constant__ CUtensorMap tmc, float *rec, float *rec_ml, int *pref,
                         const Line line) {
  using TT = TcType<T>;
  using SH = Shape<R, NR, KT>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SH::kOffBar);
  volatile int *words = reinterpret_cast<volatile int *>(bars);
  volatile float *row_alpha = reinterpret_cast<volatile float *>(words + kWAlpha);
  volatile float *row_inv = reinterpret_cast<volatile float *>(words + kWInv);
  volatile int *abort_flag = words + kWAbort;
  const uint32_t sbase = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.num_heads;
  const int worker = blockIdx.x / line.lanes, rt = blockIdx.x % line.lanes;

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(&bars[i], (i >= kSEmpty && i < kPvDone) || i == kOFree ? 4 : 1);
    *abort_flag = 0;
    for (int i = 0; i < kBadSlots; ++i) words[kWBad + i] = 0;
    mbar_init_fence();
  }
  if (tid == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmq)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmc)) : "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the worker's range of units -----------------------------------------
  volatile int *scan = words + kWScan;
  unsigned int *err0 = blockIdx.x == 0 ? a.err : nullptr;
  const int n_first = tid < a.num_seqs ? line.units(seq_of(a, line, tid, err0), H) : 0;
  int sum = n_first;
  for (int s = tid + kThreads; s < a.num_seqs; s += kThreads) sum += line.units(seq_of(a, line, s, err0), H);
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) scan[warp] = sum;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) total += scan[w];
  // no more workers than units, so that every worker between a cut sequence's
  // first and last has a piece of it
  const int workers = min(line.workers, total);
  const int lo = worker < workers ? (int)((int64_t)total * worker / workers) : 0;
  const int hi = worker < workers ? (int)((int64_t)total * (worker + 1) / workers) : 0;
  if (lo >= hi && blockIdx.x != 0) return;  // CTA-uniform, before tensor memory is taken
  int base = 0;
  for (int s0 = 0; s0 < a.num_seqs; s0 += kThreads) {
    const int s = s0 + tid;
    const int n = s0 == 0 ? n_first : s < a.num_seqs ? line.units(seq_of(a, line, s, nullptr), H) : 0;
    int x = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    __syncthreads();  // the previous use of scan[] is over
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int before = base, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += scan[w];
      all += scan[w];
    }
    before += x - n;
    if (n > 0 && before <= lo && lo < before + n) {
      words[kWStart] = s;
      words[kWStart + 1] = lo - before;
    }
    if (blockIdx.x == 0 && s < a.num_seqs) pref[s] = before;
    base += all;
    if (blockIdx.x != 0 && base > lo) break;  // CTA-uniform
  }
  if (blockIdx.x == 0 && tid == 0) pref[a.num_seqs] = total;
  if (lo >= hi) return;

  if (warp == kSWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     sbase + SH::kOffBar + 4 * kWSlot),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)words[kWSlot];

  auto fail = [&](void) {
    if (!*abort_flag) raise_error(a.err, PA_DEVERR_TIMEOUT);
    *abort_flag = 1;
  };
  const uint32_t bar0 = smem_addr(bars);
  auto warp_wait = [&](int bar, uint32_t parity) -> bool {
    return mbar_warp_wait(bar0 + 8 * bar, parity, abort_flag, a.err);
  };

  Walk walk(a, line, words[kWStart], words[kWStart + 1], hi - lo, rt);

  if (warp == kProducerWarp) {
    // ======================= producer =======================================
    constexpr int kBox = BS < KT ? BS : KT;  // keys a box
    constexpr int kBpt = KT / kBox;
    uint32_t g = 0, item = 0;
    bool ok = true;
    while (ok && walk.next()) {
      const int32_t *table = a.block_tables + (int64_t)walk.seq * a.max_blocks_per_seq;
      const int nblk = (walk.x.L + BS - 1) / BS;
      // 32 ids at a time, the next 32 on their way
      int grp = walk.t0 * KT / BS;
      int ids = grp + lane < nblk ? table[grp + lane] : 0;
      int ids_next = grp + 32 + lane < nblk ? table[grp + 32 + lane] : 0;
      const uint32_t qb = item % SH::kQBufs;
      ok = warp_wait(kQEmpty + qb, ((item / SH::kQBufs) & 1) ^ 1);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[kQFull + qb], SH::kQBytes);
        for (int c = 0; c < SH::kPieces; ++c)
          tma_load_2d(sbase + SH::kOffQ + qb * SH::kQBytes + c * SH::kQPiece, &tmq, c * 64,
                      walk.x.q0 * H + walk.first_row, &bars[kQFull + qb]);
      }
      for (int j = walk.t0; j < walk.t1; ++j, ++g) {
        const uint32_t st = g % SH::kStages;
        const int key = j * KT + lane * kBox, blk = key / BS;  // this lane's box
        if (j * KT / BS >= grp + 32) {
          grp += 32;
          ids = ids_next;
          ids_next = grp + 32 + lane < nblk ? table[grp + 32 + lane] : 0;
        }
        const int nb = min(kBpt, (walk.x.L - j * KT + kBox - 1) / kBox);
        ok = warp_wait(kEmpty + st, ((g / SH::kStages) & 1) ^ 1);
        if (!ok) break;
        const int id = __shfl_sync(0xffffffffu, ids, (blk - grp) & 31);
        const bool wrong = lane < nb && (id < 0 || id >= a.num_blocks);
        if (wrong) {
          raise_error(a.err, PA_DEVERR_BLOCK_ID);
          words[kWBad + item % kBadSlots] = (int)item + 1;  // its rows are written as zeros
        }
        if (lane == 0) mbar_arrive_expect_tx(&bars[kFull + st], nb * kBox * SH::kD * 2);
        __syncwarp();
#ifdef PA_TEST_LOST_COPY
        // test build only: tile PA_TEST_LOST_COPY of CTA 0 is announced on its
        // barrier but never copied, so that the waits for it expire
        if (blockIdx.x == 0 && g == (uint32_t)PA_TEST_LOST_COPY) continue;
#endif
        if (lane < nb)  // a bad id is replaced by a valid block
          tma_load_4d(sbase + SH::kOffStage + st * SH::kStage + lane * (kBox / 8) * SH::kGroup, &tmc, 0, 0, 0,
                      (wrong ? 0 : id) * (BS / 8) + (key % BS) / 8, &bars[kFull + st]);
        __syncwarp();
      }
      ++item;
    }
    // every copy has landed before the CTA can exit
    if (lane == 0) {
      const bool keys = drain_ring(&bars[kFull], SH::kStages, g), queries = drain_ring(&bars[kQFull], SH::kQBufs, item);
      if (!keys || !queries) fail();
    }
  } else if (warp == kSWarp) {
    // ======================= S = Q C^T ======================================
    // The two products are issued by warps of their own: S(j+1) then runs under
    // the softmax of tile j, and where its keys are still on the way the product
    // of P(j) goes ahead and frees its stage.
    constexpr uint32_t idesc = umma_idesc(TT::kFmt, 0, 0, 64, KT);
    constexpr uint32_t kHiQ = umma_desc_hi(1024), kHiC = umma_desc_hi(SH::kGroup);
    const uint32_t q_lo = umma_desc_lo(sbase + SH::kOffQ, 16), c_lo = umma_desc_lo(sbase + SH::kOffStage, 16);
    uint32_t g = 0, item = 0;
    bool ok = true;
    for (; ok && walk.next(); ++item) {
      const uint32_t qb = item % SH::kQBufs;
      ok = warp_wait(kQFull + qb, (item / SH::kQBufs) & 1);
      for (int j = walk.t0; ok && j < walk.t1; ++j, ++g) {
        const uint32_t st = g % SH::kStages;
        ok = warp_wait(kFull + st, (g / SH::kStages) & 1) && warp_wait(kSEmpty + (g & 1), ((g >> 1) & 1) ^ 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t b_lo = c_lo + st * (SH::kStage >> 4), a_lo = q_lo + qb * (SH::kQBytes >> 4);
          const uint32_t d = tmem + (g & 1) * KT;
#pragma unroll
          for (int c = 0; c < SH::kPieces; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_lo(d, a_lo + ((c * SH::kQPiece + kk * 32) >> 4), kHiQ, b_lo + ((c * 1024 + kk * 32) >> 4), kHiC,
                      idesc, (c | kk) ? 1u : 0u);
          umma_commit(&bars[kSFull + (g & 1)]);
          if (j == walk.t1 - 1) umma_commit(&bars[kQEmpty + qb]);
        }
        __syncwarp();
      }
    }
    // every product has finished before tensor memory is given back
    if (elect_one()) {
      umma_commit(&bars[kDone]);
      if (!mbar_wait(&bars[kDone], 0)) fail();
    }
  } else if (warp == kPvWarp) {
    // ======================= O^T += C^T P^T =================================
    constexpr uint32_t idesc = umma_idesc(TT::kFmt, 1, 0, 128, NR);
    constexpr uint32_t kHiP = umma_desc_hi(1024), kHiC = umma_desc_hi(SH::kGroup);
    const uint32_t p_lo = umma_desc_lo(sbase + SH::kOffP, 16), v_lo = umma_desc_lo(sbase + SH::kOffStage, 1024);
    uint32_t g = 0, item = 0;
    bool ok = true;
    for (; ok && walk.next(); ++item) {
      ok = warp_wait(kOFree, (item & 1) ^ 1);  // the sums of the item before have been read out
      for (int j = walk.t0; ok && j < walk.t1; ++j, ++g) {
        const uint32_t st = g % SH::kStages;
        ok = warp_wait(kPFull + (g & 1), (g >> 1) & 1);  // P is written; the keys landed before S was computed
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t a_lo = v_lo + st * (SH::kStage >> 4), b_lo = p_lo + (g & 1) * (SH::kPNext >> 4);
          const uint32_t keep = j == walk.t0 ? 0u : 1u;
#pragma unroll
          for (int mt = 0; mt < SH::kMTiles; ++mt)
#pragma unroll
            for (int ks = 0; ks < KT / 16; ++ks)
              umma_lo(tmem + kTmemO + mt * NR, a_lo + ((mt * 2048 + ks * 2 * SH::kGroup) >> 4), kHiC,
                      b_lo + ((ks * 32) >> 4), kHiP, idesc, ks > 0 ? 1u : keep);
          umma_commit(&bars[kEmpty + st]);
          umma_commit(&bars[kPvDone + (g & 1)]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) {
      umma_commit(&bars[kDone + 1]);
      if (!mbar_wait(&bars[kDone + 1], 0)) fail();
    }
  } else {
    // ======================= softmax warps ==================================
    // A warp's quarter holds 16 rows; the thread has two of them, 8 apart, and
    // KT / 4 keys of each: two neighbours in every group of 8.
    constexpr int kG = KT / 8;
    const int r0 = warp * 16 + (lane >> 2);
    const bool has_rows = warp * 16 < NR;  // warp-uniform
    const uint32_t ts = tmem + ((uint32_t)(warp * 32) << 16);
    const float sl2 = a.scale_log2;
    // where this lane's 16-byte row of P goes in a store of four 8x8 pieces
    const int pr = warp * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
    const uint32_t prow = (pr >> 3) * 1024 + (pr & 7) * 128;
    uint32_t g = 0, item = 0;
    bool ok = true;
    while (walk.next()) {
      const Seq x = walk.x;
      const int first_row = walk.first_row;
      const int nrow = min(NR, x.Q * H - first_row);
      bool valid[2];
      int limit[2];  // last key the row sees
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        valid[i] = r0 + 8 * i < nrow;
        limit[i] = valid[i] ? min(x.L - x.Q + (first_row + r0 + 8 * i) / H, x.L - 1) : -1;
      }
      const int limit_lo = min(x.L - x.Q + first_row / H, x.L - 1);  // the tile's least
      for (int j = walk.t0; j < walk.t1; ++j, ++g) {
        // after a failed wait the loop runs on without waiting, so that the
        // four warps keep meeting at their barrier
        ok = ok && warp_wait(kSFull + (g & 1), (g >> 1) & 1);
        tc_fence_after();
        float alpha[2] = {1.f, 1.f};
        bool need = false;
        uint32_t s[4 * kG], w[2 * kG];
        if (has_rows) {
          tmem_ld_s(ts + (g & 1) * KT, s);
          tmem_wait_ld();
        }
        tc_fence_before();  // S has been read
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kSEmpty + (g & 1)]);
        if (has_rows) {
          const int kt = j * KT;
          if (kt + KT - 1 > limit_lo) {
            const int k0 = kt + 2 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 4 * kG; ++i)
              if (k0 + 8 * (i >> 2) + (i & 1) > limit[(i >> 1) & 1]) s[i] = __float_as_uint(-INFINITY);
          }
          // the two rows side by side, so that their chains overlap
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < kG; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              mx[i] = fmax3(mx[i], __uint_as_float(s[4 * k + 2 * i]), __uint_as_float(s[4 * k + 2 * i + 1]));
#pragma unroll
          for (int d = 1; d < 4; d <<= 1)
#pragma unroll
            for (int i = 0; i < 2; ++i) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], d));
          float2 psum[2], negx2[2];
          const float2 sl2x2 = make_float2(sl2, sl2);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // lazy rescale: the reference moves when the tile's maximum, kHeadroom
            // below it, exceeds it by more than 2^8 (first tile with a visible
            // key: always)
            const float top = mx[i] * sl2 - TT::kHeadroom;
            const bool up = valid[i] && top > m[i] + kRescaleThreshold;
            need = need || up;
            alpha[i] = up ? (m[i] == -INFINITY ? 0.f : fast_exp2(m[i] - top)) : 1.f;
            m[i] = up ? top : m[i];
            const float ref = m[i] == -INFINITY ? 0.f : m[i];
            negx2[i] = make_float2(-ref, -ref);
            psum[i] = make_float2(0.f, 0.f);
          }
          // The sum takes the unrounded weights, the product P rounded to 16
          // bits: half a step a weight, of the size of the result's own rounding.
          // f16 weights that fall below its normal range lose at most 2^-25 each,
          // 2^-32 of the largest with the headroom (a million keys: 2^-12).
#pragma unroll
          for (int k = 0; k < kG; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 v = make_float2(__uint_as_float(s[4 * k + 2 * i]), __uint_as_float(s[4 * k + 2 * i + 1]));
              const float2 e = __ffma2_rn(v, sl2x2, negx2[i]);
              const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));
              psum[i] = __fadd2_rn(psum[i], p);
              w[2 * k + i] = TT::weights(p.x, p.y);
            }
#pragma unroll
          for (int i = 0; i < 2; ++i) l[i] = l[i] * alpha[i] + (psum[i].x + psum[i].y);
        }
        const bool rest = j > walk.t0;
        if (rest && has_rows && (lane & 3) == 0) {
          row_alpha[(g & 1) * 64 + r0] = alpha[0];
          row_alpha[(g & 1) * 64 + r0 + 8] = alpha[1];
        }
        const bool any = vote_any(need) && rest;
        ok = ok && warp_wait(kPvDone + (g & 1), ((g >> 1) & 1) ^ 1);  // tile g-2 has read this buffer of P
        if (any) {
          ok = ok && warp_wait(kPvDone + ((g - 1) & 1), ((g - 1) >> 1) & 1);  // O is at rest
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < SH::kMTiles * NR / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(ts + kTmemO + c * 16, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * row_alpha[(g & 1) * 64 + (c * 16 + i) % NR]);
            tmem_st16(ts + kTmemO + c * 16, o);
          }
          tmem_wait_st();
        }
        if (has_rows) {
          const uint32_t pdst = sbase + SH::kOffP + prow + (KT == 64 ? (g & 1) * SH::kPNext : 0);
          const int c0 = KT == 64 ? 0 : (g & 1) * 4 /* the row's half */;
#pragma unroll
          for (int k = 0; k < kG; k += 2)  // pieces: rows 0-7 and 8-15 of keys 8k.., then of keys 8(k+1)..
            stsm_x4(pdst + (((c0 + k + (lane >> 4)) ^ (pr & 7)) << 4), w[2 * k], w[2 * k + 1], w[2 * k + 2],
                    w[2 * k + 3]);
        }
        // slots past the last key: zero their values (P is 0 there, but 0 * NaN is not)
        if ((j + 1) * KT > x.L) {
          const uint32_t cst = sbase + SH::kOffStage + (g % SH::kStages) * SH::kStage;
          const int z0 = x.L - j * KT;
          for (int i = z0 * (R / 8) + tid; i < KT * (R / 8); i += 128) {
            const int key = i / (R / 8), v = i % (R / 8);
            st_shared_v4(cst + (key >> 3) * SH::kGroup + (v >> 3) * 1024 + (key & 7) * 128 + (v & 7) * 16, 0, 0,
                         0, 0);
          }
        }
        fence_proxy_async_smem();  // generic-proxy writes -> tensor-core reads
        tc_fence_before();         // stores to O -> the issuing thread
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kPFull + (g & 1)]);
      }
      // ---- epilogue ----
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      }
      ok = ok && warp_wait(kPvDone + ((g - 1) & 1), ((g - 1) >> 1) & 1);
      tc_fence_after();
      const bool whole = walk.t0 == 0 && walk.t1 == x.tiles;
      const bool bad = words[kWBad + item % kBadSlots] == (int)item + 1 || !ok;
      const int64_t row0 = (int64_t)x.q0 * H + first_row;
      const int64_t slot = ((int64_t)worker * 2 + (walk.t0 == 0 ? 1 : 0)) * line.lanes + rt;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + 8 * i;
        if (!valid[i] || (lane & 3)) continue;
        if (whole) {
          row_inv[(item & 1) * 64 + r] = l[i] > 0.f ? 1.f / l[i] : (l[i] != l[i] ? l[i] : 0.f);
          if (a.lse)
            a.lse[row0 + r] = bad ? -INFINITY : l[i] > 0.f ? (m[i] + log2f(l[i])) * 0.6931471805599453f
                                              : (l[i] != l[i] ? l[i] : -INFINITY);
        } else {
          rec_ml[(slot * NR + r) * 2] = m[i];
          rec_ml[(slot * NR + r) * 2 + 1] = bad ? -1.f : l[i];  // a negative sum marks a bad sequence
        }
      }
      named_sync(1, 128);
      const volatile float *inv = row_inv + (item & 1) * 64;
      constexpr int kC = SH::kMTiles * NR;  // columns of O^T: 128 values a row, tile after tile
      constexpr int kW = 32;  // read at once
#pragma unroll 1
      for (int c0 = 0; c0 < kC; c0 += kW) {
        uint32_t o[kW / 16][16];
#pragma unroll
        for (int c = 0; c < kW / 16; ++c) tmem_ld16(ts + kTmemO + c0 + c * 16, o[c]);
        tmem_wait_ld();
        if (c0 + kW == kC) {  // O may be written again
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kOFree]);
        }
#pragma unroll
        for (int c = 0; c < kW / 16; ++c) {
          const int n0 = (c0 + c * 16) % NR;
          const int dim = (c0 + c * 16) / NR * 128 + warp * 32 + lane;
          if (n0 >= nrow) continue;  // warp-uniform
          if (whole) {
            // neighbouring lanes exchange, so that each stores two values of a row
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float f0 = inv[n0 + i], f1 = inv[n0 + i + 1];
              const float v0 = bad || f0 == 0.f ? 0.f : __uint_as_float(o[c][i]) * f0;
              const float v1 = bad || f1 == 0.f ? 0.f : __uint_as_float(o[c][i + 1]) * f1;
              const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v0 : v1, 1);
              const int n = n0 + i + (lane & 1);
              const uint32_t two = (lane & 1) ? TT::pack(other, v1) : TT::pack(v0, other);
              if (n < nrow)
                *reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + (row0 + n) * R + (dim & ~1)) = two;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (n0 + i < nrow) rec[(slot * NR + n0 + i) * R + dim] = __uint_as_float(o[c][i]);
          }
        }
      }
      ++item;
    }
  }
  __syncthreads();
  if (warp == kSWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// Joins the records of the sequences that were cut, writes zeros where there
// is no key to see.  One CTA of 8 warps per (sequence, rows_per_cta rows): a
// warp a row when there are rows enough to fill the machine, else 2, 4 or 8
// warps that share a row's pieces and join through shared memory (one long
// sequence is cut into as many pieces as there are workers).  per_seq: CTAs a
// sequence, or 0, a CTA a place (see first_place) where most of those would find no
// row: 256 single rows announced as 256 each, 16 heads, took 595 us by sequence and
// take 101 by places (96 announced as they are), 2000 rows beside 255 single ones at
// 128 heads 28.3 and 2.0 ms.
constexpr int kMergeWarps = 8;
constexpr int kMostEmpty = 2;  // CTAs by sequence for each by places, at most
template <typename T, int R>
__global__ void __launch_bounds__(32 * kMergeWarps)
    latent_merge_kernel(const LatentArgs a, const float *rec, const float *rec_ml, const int *pref,
                        const Line line, int rows_per_cta, int per_seq) {
  constexpr int V = R / 128;  // float4 a lane: values lane * 4 + 128 v
  __shared__ float4 so[kMergeWarps][R / 4];
  __shared__ float sm[kMergeWarps], sl[kMergeWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int s;
  int64_t first, step;  // the CTA's rows: first, first + step, ... and rows_per_cta from each
  if (per_seq) {
    s = blockIdx.x / per_seq;
    first = (int64_t)(blockIdx.x % per_seq) * rows_per_cta;
    step = (int64_t)per_seq * rows_per_cta;
  } else {
    const int shift = 31 - __clz(rows_per_cta);
    s = seq_of_place(a.query_start_loc, a.num_seqs, a.num_heads, shift, blockIdx.x);
    first = (int64_t)blockIdx.x - first_place(a.query_start_loc, s, a.num_heads, shift);
    if (first < 0) return;
    first <<= shift;
    step = (int64_t)1 << 31;  // past every row
  }
  const int total = pref[a.num_seqs], p0 = pref[s];
  const Seq x = seq_of(a, line, s, nullptr);
  const int rows = x.Q * a.num_heads, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int workers = min(line.workers, total);
  // the worker of unit u: the last w with total * w / workers <= u
  const bool narrow = (uint64_t)total * (uint64_t)workers <= 0xffffffffu;
  auto owner = [&](int u) -> int {
    return narrow ? (int)((((uint32_t)u + 1) * (uint32_t)workers - 1) / (uint32_t)total)
                  : (int)((((int64_t)u + 1) * workers - 1) / total);
  };
  if (x.tiles && owner(p0) == owner(p0 + line.units(x, a.num_heads) - 1)) return;  // written by its worker
  const int share = kMergeWarps / rows_per_cta, group = warp / share, part = warp % share;
  for (int64_t base = first; base < rows; base += step) {
    const int row = (int)base + group;  // the same for all warps that meet at the barrier below
    if (row >= rows) break;
    const int rt = row / line.nr, r = row % line.nr;
    // units of the row's tiles, and the workers that hold them
    const int u0 = p0 + line.extra + (line.flat ? rt * (x.tiles + line.extra) : 0);
    const int w0 = x.tiles ? owner(u0) : 0, w1 = x.tiles ? owner(u0 + x.tiles - 1) : 0;
    const int np = x.tiles ? w1 - w0 + 1 : 0;
    if (np == 1) continue;  // written by its worker
    // record of the i-th piece: the first starts the sequence, the others continue it
    auto at = [&](int i) {
      return (((int64_t)(w0 + i) * 2 + (i == 0 ? 1 : 0)) * line.lanes + (line.flat ? 0 : rt)) * line.nr + r;
    };
    // four pieces at a time, joined as they come: maxima and sums are read together
    float4 o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, l = 0.f;
    bool bad = false;
    for (int i0 = part; i0 < np; i0 += 4 * share) {
      float2 ml[4];
      float4 p[4][V];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * share;
        ml[u] = make_float2(-INFINITY, 0.f);
        if (i >= np) continue;
        const int64_t k = at(i);
        ml[u] = *reinterpret_cast<const float2 *>(rec_ml + k * 2);
#pragma unroll
        for (int v = 0; v < V; ++v) p[u][v] = __ldcs(reinterpret_cast<const float4 *>(rec + k * R + v * 128 + lane * 4));
      }
      const float top = fmaxf(fmaxf(fmaxf(M, ml[0].x), fmaxf(ml[1].x, ml[2].x)), ml[3].x);
      const float f0 = M == -INFINITY ? 0.f : exp2f(M - top);
      M = top;
      l *= f0;
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = make_float4(o[v].x * f0, o[v].y * f0, o[v].z * f0, o[v].w * f0);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        bad = bad || ml[u].y < 0.f;
        // a piece without a visible key has no sums (a NaN total is not one)
        if (ml[u].x == -INFINITY && ml[u].y <= 0.f) continue;
        const float f = exp2f(ml[u].x - M);
        l += f * ml[u].y;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          o[v].x += f * p[u][v].x;
          o[v].y += f * p[u][v].y;
          o[v].z += f * p[u][v].z;
          o[v].w += f * p[u][v].w;
        }
      }
    }
    if (share > 1) {
      named_sync(1 + group, 32 * share);  // an earlier row has been joined
#pragma unroll
      for (int v = 0; v < V; ++v) so[warp][v * 32 + lane] = o[v];
      if (lane == 0) {
        sm[warp] = M;
        sl[warp] = bad ? -1.f : l;
      }
      named_sync(1 + group, 32 * share);
      if (part) continue;
      for (int w = warp; w < warp + share; ++w) M = fmaxf(M, sm[w]);
      l = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = warp; w < warp + share; ++w) {
        bad = bad || sl[w] < 0.f;
        if (sm[w] == -INFINITY && sl[w] <= 0.f) continue;
        const float f = exp2f(sm[w] - M);
        l += f * sl[w];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float4 y = so[w][v * 32 + lane];
          o[v].x += f * y.x;
          o[v].y += f * y.y;
          o[v].z += f * y.z;
          o[v].w += f * y.w;
        }
      }
    }
    const int64_t orow = (int64_t)x.q0 * a.num_heads + row;
    const bool none = bad || l == 0.f;
    const float inv = 1.f / l;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      uint2 y = make_uint2(0, 0);
      if (!none) {
        y.x = TcType<T>::pack(o[v].x * inv, o[v].y * inv);
        y.y = TcType<T>::pack(o[v].z * inv, o[v].w * inv);
      }
      *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + orow * R + v * 128 + lane * 4) = y;
    }
    if (a.lse && lane == 0) a.lse[orow] = none ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
  }
}

struct Plan {
  Line line;
  int row_tiles;
  size_t pref, ml, rec, total;  // workspace offsets
};

// Keys a tile: 32 where a row is long (512 values), so that four or five tiles
// fit and the next ones are on their way while one is worked on; 64 halve the
// waits per key where four of those fit.
constexpr int key_tile(int latent_dim) { return latent_dim == 512 ? 32 : 64; }

Plan plan_of(int num_seqs, int max_query_len, int num_heads, int latent_dim, int ragged, int sm_count) {
  Plan p;
  const int64_t rows = (int64_t)max_query_len * num_heads;
  // rows a CTA holds: fewer cost less in the second product (its N) and leave
  // shared memory for the keys
  p.line.nr = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  p.line.kt = key_tile(latent_dim);
  p.row_tiles = (int)((rows + p.line.nr - 1) / p.line.nr);
  // An item's queries and epilogue, in tiles: CTAs with one item and with four
  // or five of 256 ragged sequences then end within a few microseconds (2.6 us
  // an item at 16 rows, 8 at 64 of 512 values, beside 0.8 a tile).
  p.line.extra = 3 + p.line.nr * latent_dim / 8192;
  p.line.flat = ragged && p.row_tiles > 1;
  p.line.lanes = p.line.flat ? 1 : p.row_tiles;
  p.line.workers = sm_count / p.line.lanes;
  if (p.line.workers < 1) p.line.workers = 1;
  const size_t recs = p.line.workers > 1 ? (size_t)p.line.workers * 2 * p.line.lanes * p.line.nr : 0;
  p.pref = 0;
  p.ml = ((size_t)(num_seqs + 1) * 4 + 255) / 256 * 256;
  p.rec = p.ml + (recs * 8 + 255) / 256 * 256;
  p.total = p.rec + recs * latent_dim * 4;
  return p;
}

template <typename T, int R, int NR, int KT, int BS>
cudaError_t launch_t(const LatentArgs &a, const Plan &p, cudaStream_t stream) {
  using SH = Shape<R, NR, KT>;
  auto fn = encode_fn_tc();
  if (!fn) return cudaErrorNotSupported;
  CUtensorMap tmq, tmc;
  constexpr int D = R + 64;
  CUresult r;
  {
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)a.num_q_tokens * a.num_heads};
    cuuint64_t strides[1] = {(cuuint64_t)D * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)NR};
    cuuint32_t estr[2] = {1, 1};
    r = fn(&tmq, TcType<T>::kTma, 2, const_cast<void *>(a.q), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (r == CUDA_SUCCESS) {
    // [8-key group][piece][8 keys][64 values], innermost first below
    cuuint64_t dims[4] = {64, 8, (cuuint64_t)SH::kPieces, (cuuint64_t)a.num_blocks * (BS / 8)};
    cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 16};
    cuuint32_t box[4] = {64, 8, (cuuint32_t)SH::kPieces, (cuuint32_t)((BS < KT ? BS : KT) / 8)};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    r = fn(&tmc, TcType<T>::kTma, 4, const_cast<void *>(a.cache), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (r != CUDA_SUCCESS) {
    debug_log("latent_decode: tensor map refused (CUresult %d)", (int)r);
    return cudaErrorInvalidValue;
  }
  auto kern = latent_decode_kernel<T, R, NR, KT, BS>;
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void *>(kern), SH::kSmem, true);
  if (e != cudaSuccess) return e;
  char *ws = static_cast<char *>(a.ws);
  int *pref = reinterpret_cast<int *>(ws + p.pref);
  float *ml = reinterpret_cast<float *>(ws + p.ml), *rec = reinterpret_cast<float *>(ws + p.rec);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3((unsigned)(p.line.workers * p.line.lanes));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = SH::kSmem;
  e = cudaLaunchKernelEx(&cfg, kern, a, tmq, tmc, rec, ml, pref, p.line);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)a.max_query_len * a.num_heads;
  int rows_per_cta = 1;  // 512 CTAs at most, if a warp a row allows it
  while (rows_per_cta < kMergeWarps && a.num_seqs * rows > 512 * (int64_t)rows_per_cta) rows_per_cta *= 2;
  int per_seq = (int)((rows + rows_per_cta - 1) / rows_per_cta);
  int64_t grid = (int64_t)a.num_seqs * per_seq;
  const int64_t all = (int64_t)a.num_q_tokens * a.num_heads;
  if (a.query_start_loc && grid > kMostEmpty * (all / rows_per_cta + a.num_seqs)) {
    per_seq = 0;
    for (rows_per_cta = 1; rows_per_cta < kMergeWarps && all > 512 * (int64_t)rows_per_cta;) rows_per_cta *= 2;
    grid = all / rows_per_cta + a.num_seqs;
  }
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, latent_merge_kernel<T, R>, a, (const float *)rec, (const float *)ml,
                            (const int *)pref, p.line, rows_per_cta, per_seq);
}

template <typename T, int R, int NR>
cudaError_t launch_bs(const LatentArgs &a, const Plan &p, cudaStream_t s) {
  if (a.block_size == 16) return launch_t<T, R, NR, key_tile(R), 16>(a, p, s);
  if (a.block_size == 32) return launch_t<T, R, NR, key_tile(R), 32>(a, p, s);
  return launch_t<T, R, NR, key_tile(R), 64>(a, p, s);
}

template <typename T, int R>
cudaError_t launch_nr(const LatentArgs &a, const Plan &p, cudaStream_t s) {
  if (p.line.nr == 16) return launch_bs<T, R, 16>(a, p, s);
  if (p.line.nr == 32) return launch_bs<T, R, 32>(a, p, s);
  return launch_bs<T, R, 64>(a, p, s);
}

}  // namespace

size_t latent_decode_ws(int num_seqs, int max_query_len, int num_heads, int latent_dim, int sm_count) {
  const size_t even = plan_of(num_seqs, max_query_len, num_heads, latent_dim, 0, sm_count).total;
  const size_t ragged = plan_of(num_seqs, max_query_len, num_heads, latent_dim, 1, sm_count).total;
  return even > ragged ? even : ragged;
}

bool latent_decode_fits(int num_seqs, int max_query_len, int num_heads, int latent_dim, int max_context_len) {
  const Plan p = plan_of(num_seqs, max_query_len, num_heads, latent_dim, 1, 1);
  const int64_t per = (int64_t)(max_context_len / p.line.kt + 1 + p.line.extra) * p.row_tiles;
  return per <= INT_MAX / num_seqs && (int64_t)num_seqs * max_query_len * num_heads <= INT_MAX;
}

cudaError_t launch_latent_decode(const LatentArgs &a, int dtype, int sm_count, cudaStream_t stream) {
  const Plan p = plan_of(a.num_seqs, a.max_query_len, a.num_heads, a.latent_dim, a.query_start_loc != nullptr,
                         sm_count);
  if (dtype == PA_BF16)
    return a.latent_dim == 512 ? launch_nr<__nv_bfloat16, 512>(a, p, stream)
                               : launch_nr<__nv_bfloat16, 256>(a, p, stream);
  return a.latent_dim == 512 ? launch_nr<__half, 512>(a, p, stream) : launch_nr<__half, 256>(a, p, stream);
}

}  // namespace pa
