// tables.cu -- block tables, lengths and reference counts held on the device:
// one scheduling step (release, fork, grow with copy-on-write) and compaction
// of the pool ("核心概念", sections 按需分配 and 内存共享; "理解 vLLM
// PagedAttention", sections 四 and 六: blocks are taken on demand, shared by
// reference count and copied before a shared one is written).
//
// Both are prefix sums over the pool and over the rows with scattered integer
// writes around them.  Order decides every result (lowest free id first, rows
// in order) and no result depends on the order of atomics: reference counts
// are integer sums.
//
// Each is one cooperative kernel whose phases are parted by grid barriers: the
// work of a phase is a few microseconds at most, so that launches would cost
// more than it: as six dependent launches a step of 256 rows took 13 us more of
// the host's time.  On the device alone the six took 15 us and this kernel takes
// 18, so that in a captured loop, where the host's time is nil, the barriers cost
// what the launches save elsewhere (a replay of the six was not measured).  What
// one CTA can sum up in less than a barrier takes -- the counts of the pool's
// chunks, the needs of the rows -- every CTA sums up for itself.
#include <cooperative_groups.h>
#include <limits.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kPerThread = 4;
constexpr int kChunk = kThreads * kPerThread;  // pool blocks counted at a time
constexpr int kRowThreads = 128;               // threads that share a row
constexpr int kRowGroups = kThreads / kRowThreads;
constexpr int kMaxRows = 4096;
constexpr int kPoolsPerLaunch = 64;

// Workspace arrays (offsets in bytes, all 256-byte aligned).
struct TableWs {
  size_t len, writes, info, base, chunk, list, rows, total;
};

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

TableWs table_ws(int num_seqs, int width, int num_blocks) {
  TableWs w;
  const size_t chunks = ((size_t)num_blocks + kChunk - 1) / kChunk;
  size_t off = 0;
  w.len = off;  // [num_seqs] length after release and fork
  off += align_up((size_t)num_seqs * 4);
  w.writes = off;  // [num_seqs] block that the row's next token is written into, -1: none held
  off += align_up((size_t)num_seqs * 4);
  w.info = off;  // [num_seqs] blocks needed, and whether one is for a copy-on-write
  off += align_up((size_t)num_seqs * 4);
  w.base = off;  // [num_seqs] first fresh block, -1: not grown
  off += align_up((size_t)num_seqs * 4);
  w.chunk = off;  // [chunks] counts
  off += align_up(chunks * 4);
  w.list = off;  // step: [num_blocks] fresh ids; compact: remap
  off += align_up((size_t)num_blocks * 4);
  w.rows = off;  // step: [num_seqs][width] forked rows; compact: holes and sources, num_blocks / 2 each
  const size_t forked = align_up((size_t)num_seqs * width * 4), lists = align_up((size_t)num_blocks * 4);
  off += forked > lists ? forked : lists;
  w.total = off;
  return w;
}

struct Pools {
  uint4 *p[kPoolsPerLaunch];
  int64_t vecs[kPoolsPerLaunch];  // 16-byte vectors per block
  int n;
};

struct StepArgs {
  int32_t *tables, *lens, *refs;
  const int32_t *release, *fork_src, *append;
  int64_t *slots, *pairs;
  int32_t *qsl;
  int S, W, NB, bs, max_new, chunks;
  int *wlen, *writes, *info, *base, *chunk, *fresh, *wrows;
  unsigned int *err;
};

__device__ __forceinline__ int row_len(const int32_t *lens, int i, int cap, unsigned int *err) {
  const int n = lens[i];
  if (n >= 0 && n <= cap) return n;
  raise_error(err, PA_DEVERR_CONTEXT_LEN);
  return 0;
}

// Exclusive prefix of v over the block; *total gets the sum.  s: kThreads / 32 + 1 entries.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *s, T *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // s may still be read from an earlier scan
  if (lane == 31) s[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const T w = lane < kThreads / 32 ? s[lane] : 0;
    T y = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const T z = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) y += z;
    }
    if (lane < kThreads / 32) s[lane] = y - w;
    if (lane == 31) s[kThreads / 32] = y;
  }
  __syncthreads();
  *total = s[kThreads / 32];
  return x - v + s[warp];
}

// A CTA's contiguous share of n chunks.
__device__ __forceinline__ void chunk_range(int n, int *c0, int *c1) {
  const int per = (n + (int)gridDim.x - 1) / (int)gridDim.x;
  *c0 = min(n, (int)blockIdx.x * per);
  *c1 = min(n, *c0 + per);
}

// Sums of the chunk counts: all of them, and those before c0.
__device__ __forceinline__ void sum_chunks(const int *chunk, int n, int c0, int *s, int *all, int *before) {
  int x = 0, y = 0;
  for (int c = threadIdx.x; c < n; c += kThreads) {
    const int v = chunk[c];
    x += v;
    if (c < c0) y += v;
  }
  block_scan(x, s, all);
  block_scan(y, s, before);
}

// Copies whole blocks (src, dst) in every pool of the list: pieces of 4 KB, one
// a warp, eight 16-byte loads in flight a thread.  Pairs of -1 are skipped.
// Bound: memory traffic.
constexpr int kMoveVecs = 8 * 32;
__device__ __forceinline__ void move_blocks(const Pools &pools, const int64_t *pairs, int n) {
  const int lane = threadIdx.x & 31;
  for (int k = 0; k < pools.n; ++k) {
    const int64_t vecs = pools.vecs[k];
    const int64_t pieces = (vecs + kMoveVecs - 1) / kMoveVecs;
    for (int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < n * pieces;
         w += (int64_t)gridDim.x * (kThreads / 32)) {
      const int64_t pair = w / pieces, v0 = (w - pair * pieces) * kMoveVecs + lane;
      const int64_t src = pairs[2 * pair], dst = pairs[2 * pair + 1];
      if (src < 0 || dst < 0) continue;
      const uint4 *from = pools.p[k] + src * vecs + v0;
      uint4 *to = pools.p[k] + dst * vecs + v0;
      const int left = (int)min(vecs - v0, (int64_t)kMoveVecs);
      uint4 r[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (u * 32 < left) r[u] = __ldcs(from + u * 32);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (u * 32 < left) to[u * 32] = r[u];
    }
  }
}

// The same as a launch of its own, for the pools past the first kPoolsPerLaunch
// and for moves that a pass of the cooperative grid does not cover: with eight
// small CTAs a SM and 16 KB pieces it reaches 5.6 TB/s where the cooperative
// grid's two large ones reach 5.1 (65536 blocks of 32 KB, half of them used).
constexpr int kMoverThreads = 256, kMoverVecs = 4 * kMoverThreads;
__global__ void __launch_bounds__(kMoverThreads) move_blocks_kernel(const Pools pools, const int64_t *pairs,
                                                                    int num_pairs) {
  for (int k = 0; k < pools.n; ++k) {
    const int64_t vecs = pools.vecs[k];
    const int64_t pieces = (vecs + kMoverVecs - 1) / kMoverVecs;
    for (int64_t w = blockIdx.x; w < num_pairs * pieces; w += gridDim.x) {
      const int64_t pair = w / pieces, v0 = (w - pair * pieces) * kMoverVecs + threadIdx.x;
      const int64_t src = pairs[2 * pair], dst = pairs[2 * pair + 1];
      if (src < 0 || dst < 0) continue;
      const uint4 *from = pools.p[k] + src * vecs;
      uint4 *to = pools.p[k] + dst * vecs;
      uint4 r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (v0 + u * kMoverThreads < vecs) r[u] = __ldcs(from + v0 + u * kMoverThreads);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (v0 + u * kMoverThreads < vecs) to[v0 + u * kMoverThreads] = r[u];
    }
  }
}

// ---- pa_table_step ------------------------------------------------------------

__global__ void __launch_bounds__(kThreads, 2) step_kernel(const StepArgs a, const Pools pools) {
  __shared__ int s[kThreads / 32 + 1];
  __shared__ int64_t s64[kThreads / 32 + 1];  // sums over rows may pass 32 bits
  __shared__ int s_group[kRowGroups];
  cg::grid_group grid = cg::this_grid();
  const int cap = a.W * a.bs;
  const int group = threadIdx.x / kRowThreads, gt = threadIdx.x % kRowThreads;
  const int row0 = blockIdx.x * kRowGroups + group, row_step = gridDim.x * kRowGroups;

  // 1. Rows give up and take over blocks (integer atomics on the counts).  The
  // blocks of a fork's source are put aside, since its row may itself change.
  for (int i = row0; i < a.S; i += row_step) {
    int src = a.fork_src ? a.fork_src[i] : -1;
    if (src >= a.S) {
      if (gt == 0) raise_error(a.err, PA_DEVERR_TABLE);
      src = -1;
    }
    const bool forked = src >= 0;
    const bool drop = forked || (a.release && a.release[i] != 0);
    const int len = row_len(a.lens, i, cap, gt == 0 ? a.err : nullptr);
    const int add = a.append[i];
    const int32_t *own = a.tables + (int64_t)i * a.W, *from = own;
    int now = drop ? 0 : len;
    if (drop) {
      const int n = (len + a.bs - 1) / a.bs;
      for (int j = gt; j < n; j += kRowThreads) {
        const int b = own[j];
        if (b >= 0 && b < a.NB) atomicSub(a.refs + b, 1);
        else raise_error(a.err, PA_DEVERR_BLOCK_ID);
      }
    }
    if (forked) {
      now = row_len(a.lens, src, cap, nullptr);
      from = a.tables + (int64_t)src * a.W;
      int *keep = a.wrows + (int64_t)i * a.W;
      const int n = (now + a.bs - 1) / a.bs;
      for (int j = gt; j < n; j += kRowThreads) {
        const int b = from[j];
        keep[j] = b;
        if (b >= 0 && b < a.NB) atomicAdd(a.refs + b, 1);
        else raise_error(a.err, PA_DEVERR_BLOCK_ID);
      }
    }
    if (gt == 0) {
      a.wlen[i] = now;
      int b = -1;
      if (add > 0 && now % a.bs != 0 && (int64_t)now + add <= cap) {
        b = from[now / a.bs];
        if (b < 0 || b >= a.NB) b = -1;
      }
      a.writes[i] = b;
    }
  }
  grid.sync();

  // 2. Free blocks a chunk; forked rows' entries into the tables; the rows'
  // needs.  Of the rows that write into one shared block, in row order, all copy
  // it but the last of its holders: the k-th writer of a block with r holders
  // copies while r - k > 1.
  for (int c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const int id = c * kChunk + threadIdx.x * kPerThread;
    int n = 0, total;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k)
      if (id + k < a.NB) n += a.refs[id + k] == 0;
    block_scan(n, s, &total);
    if (threadIdx.x == 0) a.chunk[c] = total;
  }
  for (int i = row0; i < a.S; i += row_step) {
    const int now = a.wlen[i], add = a.append[i];
    const int held = (now + a.bs - 1) / a.bs;
    const int src = a.fork_src ? a.fork_src[i] : -1;
    if (src >= 0 && src < a.S) {
      const int *keep = a.wrows + (int64_t)i * a.W;
      int32_t *t = a.tables + (int64_t)i * a.W;
      for (int j = gt; j < held; j += kRowThreads) t[j] = keep[j];
    }
    const bool bad = add < 0 || (int64_t)now + add > cap;
    const int last = a.writes[i];
    const int holders = last >= 0 ? a.refs[last] : 0;
    int before = 0;
    if (holders > 1) {  // uniform over the row's threads
      if (gt == 0) s_group[group] = 0;
      for (int r = gt; r < i; r += kRowThreads) before += a.writes[r] == last;
      before = __reduce_add_sync(0xffffffffu, before);
      named_sync(1 + group, kRowThreads);
      if ((gt & 31) == 0 && before) atomicAdd(&s_group[group], before);
      named_sync(1 + group, kRowThreads);
      before = s_group[group];
      named_sync(1 + group, kRowThreads);  // read before the next row clears it
    }
    if (gt == 0) {
      const int cow = holders - before > 1;
      const int more = bad || add == 0 ? 0 : (int)(((int64_t)now + add + a.bs - 1) / a.bs) - held;
      if (bad) raise_error(a.err, PA_DEVERR_CONTEXT_LEN);
      a.info[i] = (more + cow) << 1 | cow;
    }
  }
  grid.sync();

  // 3. Every CTA: which rows fit (need is never negative, so they are a leading
  // run) and how many blocks those take; then the free blocks of lowest id, in
  // order, into the list of fresh ones.
  int c0, c1, avail, rank;
  chunk_range(a.chunks, &c0, &c1);
  sum_chunks(a.chunk, a.chunks, c0, s, &avail, &rank);
  int64_t taken = 0, tokens = 0;
  int take = 0;
  for (int r0 = 0; r0 < a.S; r0 += kThreads) {
    const int i = r0 + threadIdx.x;
    const int add = i < a.S ? a.append[i] : 0;
    const int need = i < a.S ? a.info[i] >> 1 : 0;
    int64_t t_need, t_add;
    const int64_t first = taken + block_scan<int64_t>(need, s64, &t_need);
    const int64_t tok = tokens + block_scan<int64_t>(max(add, 0), s64, &t_add);
    const bool fits = first + need <= avail;
    if (i < a.S) {
      if (fits) take = max(take, (int)first + need);
      if (blockIdx.x == 0) {
        const bool ok = fits && add >= 0 && (int64_t)a.wlen[i] + add <= cap;
        if (!fits && add > 0) raise_error(a.err, PA_DEVERR_POOL);
        a.base[i] = ok ? (int)first : -1;
        a.qsl[i] = (int)min(tok, (int64_t)INT_MAX);
      }
    }
    taken += t_need;
    tokens += t_add;
  }
  take = __reduce_max_sync(0xffffffffu, take);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = take;
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) take = max(take, s[w]);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.qsl[a.S] = (int)min(tokens, (int64_t)INT_MAX);
    if (tokens > a.max_new) raise_error(a.err, PA_DEVERR_SLOT);
  }
  for (int c = c0; c < c1 && rank < take; ++c) {  // CTA-uniform
    const int id = c * kChunk + threadIdx.x * kPerThread;
    bool free_[kPerThread];
    int n = 0, total;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      free_[k] = id + k < a.NB && a.refs[id + k] == 0;
      n += free_[k];
    }
    int x = rank + block_scan(n, s, &total);
#pragma unroll
    for (int k = 0; k < kPerThread; ++k)
      if (free_[k]) {
        if (x < take) {
          a.fresh[x] = id + k;
          a.refs[id + k] = 1;
        }
        ++x;
      }
    rank += total;
  }
  grid.sync();

  // 4. The rows' fresh blocks, slots and lengths; -1 behind the last slot.
  for (int64_t x = (int64_t)a.qsl[a.S] + blockIdx.x * kThreads + threadIdx.x; x < a.max_new;
       x += (int64_t)gridDim.x * kThreads)
    a.slots[x] = -1;
  for (int i = row0; i < a.S; i += row_step) {
    const int now = a.wlen[i], add = max(a.append[i], 0), base = a.base[i];
    const int info = a.info[i], cow = info & 1, more = (info >> 1) - cow;
    const int held = (now + a.bs - 1) / a.bs;
    const int64_t p0 = a.qsl[i];
    const bool grown = base >= 0;
    int32_t *row = a.tables + (int64_t)i * a.W;
    const int copy = grown && cow ? a.fresh[base] : -1;
    if (gt == 0) {
      const int last = a.writes[i];
      if (copy >= 0) {
        row[held - 1] = copy;
        atomicSub(a.refs + last, 1);
      }
      a.pairs[2 * i] = copy >= 0 ? last : -1;
      a.pairs[2 * i + 1] = copy;
      a.lens[i] = grown ? now + add : now;
    }
    if (grown)
      for (int k = gt; k < more; k += kRowThreads) row[held + k] = a.fresh[base + cow + k];
    const int n = (int)min((int64_t)add, max((int64_t)0, a.max_new - p0));
    for (int t = gt; t < n; t += kRowThreads) {
      const int pos = now + t, j = pos / a.bs;
      int64_t slot = -1;
      if (grown) {
        const int b = j >= held ? a.fresh[base + cow + j - held] : copy >= 0 ? copy : row[j];
        if (b >= 0 && b < a.NB) slot = (int64_t)b * a.bs + pos % a.bs;
      }
      a.slots[p0 + t] = slot;
    }
  }
  if (pools.n == 0) return;  // uniform over the grid
  grid.sync();

  // 5. Copy-on-write copies in all pools.
  move_blocks(pools, a.pairs, a.S);
}

// ---- pa_table_compact ------------------------------------------------------------

struct CompactArgs {
  int32_t *tables, *refs, *live;
  const int32_t *lens;
  int64_t *moves;
  int S, W, NB, bs, chunks, max_moves;
  int *chunk, *remap, *holes, *sources;
  unsigned int *err;
};

__global__ void __launch_bounds__(kThreads, 2) compact_kernel(const CompactArgs a, const Pools pools) {
  __shared__ int s[kThreads / 32 + 1];
  cg::grid_group grid = cg::this_grid();

  // 1. used blocks a chunk
  for (int c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const int id = c * kChunk + threadIdx.x * kPerThread;
    int n = 0, total;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k)
      if (id + k < a.NB) n += a.refs[id + k] > 0;
    block_scan(n, s, &total);
    if (threadIdx.x == 0) a.chunk[c] = total;
  }
  grid.sync();

  // 2. k-th free id below the border `live` and k-th used id at or past it
  int c0, c1, live, before, total;
  chunk_range(a.chunks, &c0, &c1);
  sum_chunks(a.chunk, a.chunks, c0, s, &live, &before);
  int below = 0;  // used blocks below the border
  {
    const int border = live / kChunk;
    int x = 0;
    for (int c = threadIdx.x; c < min(border, a.chunks); c += kThreads) x += a.chunk[c];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      const int id = border * kChunk + threadIdx.x * kPerThread + k;
      if (id < live) x += a.refs[id] > 0;
    }
    block_scan(x, s, &below);
  }
  const int moves = live - below;
  for (int c = c0; c < c1; ++c) {
    const int id = c * kChunk + threadIdx.x * kPerThread;
    bool used[kPerThread];
    int n = 0;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      used[k] = id + k < a.NB && a.refs[id + k] > 0;
      n += used[k];
    }
    int x = before + block_scan(n, s, &total);
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      const int b = id + k;
      if (b < live && !used[k]) a.holes[b - x] = b;
      if (b >= live && b < a.NB) {
        if (used[k]) a.sources[x - below] = b;
        else a.remap[b] = b;  // a held block without a count stays where it is
      }
      x += used[k];
    }
    before += total;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.live = live;
  grid.sync();

  // 3. the moves
  for (int k = blockIdx.x * kThreads + threadIdx.x; k < a.max_moves; k += gridDim.x * kThreads) {
    int src = -1, dst = -1;
    if (k < moves) {
      src = a.sources[k];
      dst = a.holes[k];
      a.remap[src] = dst;
      a.refs[dst] = a.refs[src];
      a.refs[src] = 0;
    }
    a.moves[2 * (int64_t)k] = src;
    a.moves[2 * (int64_t)k + 1] = dst;
  }
  grid.sync();

  // 4. tables, and the blocks of all pools
  const int group = threadIdx.x / kRowThreads, gt = threadIdx.x % kRowThreads;
  for (int i = blockIdx.x * kRowGroups + group; i < a.S; i += gridDim.x * kRowGroups) {
    const int len = row_len(a.lens, i, a.W * a.bs, gt == 0 ? a.err : nullptr);
    int32_t *t = a.tables + (int64_t)i * a.W;
    const int n = (len + a.bs - 1) / a.bs;
    for (int j = gt; j < n; j += kRowThreads) {
      const int b = t[j];
      if (b < 0 || b >= a.NB) raise_error(a.err, PA_DEVERR_BLOCK_ID);
      else if (b >= live) t[j] = a.remap[b];
    }
  }
  move_blocks(pools, a.moves, moves);
}

// ---- host ---------------------------------------------------------------------------

// Cooperative launch: the grid's CTAs are resident together (two a SM at most).
template <typename... Args>
cudaError_t launch_coop(void (*kernel)(Args...), int grid, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The pools [p0, p0 + kPoolsPerLaunch) of the list, and the CTAs' shares of 16
// pieces in copying `pairs` blocks of theirs.
Pools pool_list(void *const *pools, const int64_t *bytes, int n, int p0, int64_t pairs, int64_t *pieces) {
  Pools list;
  list.n = n - p0 < kPoolsPerLaunch ? n - p0 : kPoolsPerLaunch;
  if (list.n < 0) list.n = 0;
  *pieces = 0;
  for (int k = 0; k < list.n; ++k) {
    list.p[k] = static_cast<uint4 *>(pools[p0 + k]);
    list.vecs[k] = bytes[p0 + k] / 16;
    const int64_t x = ((list.vecs[k] + kMoveVecs - 1) / kMoveVecs * pairs + kThreads / 32 - 1) / (kThreads / 32);
    if (x > *pieces) *pieces = x;
  }
  return list;
}

// CTAs: what the largest phase can use, two a SM at most.
int coop_grid(int64_t want, int sm_count) {
  const int64_t most = (int64_t)sm_count * 2;
  return (int)(want < 1 ? 1 : want > most ? most : want);
}

// Moves in the pools from p0 on, in launches of their own.
cudaError_t launch_moves(void *const *pools, const int64_t *bytes, int n, int p0, const int64_t *pairs,
                         int num_pairs, int sm_count, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  for (; p0 < n && e == cudaSuccess; p0 += kPoolsPerLaunch) {
    int64_t pieces;
    const Pools list = pool_list(pools, bytes, n, p0, num_pairs, &pieces);
    const int64_t want = pieces * 4, most = (int64_t)sm_count * 8;  // 16 KB a CTA and pass
    move_blocks_kernel<<<(unsigned)(want < most ? want : most), kMoverThreads, 0, s>>>(list, pairs, num_pairs);
    e = cudaGetLastError();
  }
  return e;
}

bool pools_ok(void *const *pools, const int64_t *bytes, int n) {
  if (n < 0 || n > 1024 || (n > 0 && (!pools || !bytes))) return false;
  for (int i = 0; i < n; ++i)
    if (!pools[i] || (reinterpret_cast<uintptr_t>(pools[i]) & 15u) || bytes[i] <= 0 || bytes[i] % 16) return false;
  return true;
}

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_table_workspace_size(int num_seqs, int max_blocks_per_seq, int num_blocks) {
  if (num_seqs <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0) return 0;
  return table_ws(num_seqs, max_blocks_per_seq, num_blocks).total;
}

int pa_table_step(int32_t *block_tables, int max_blocks_per_seq, int32_t *context_lens,
                  int32_t *ref_counts, const int32_t *release, const int32_t *fork_src,
                  const int32_t *append, int num_seqs, int num_blocks, int block_size,
                  int64_t *slot_mapping, int max_new_tokens, int32_t *query_start_loc,
                  int64_t *copy_pairs, void *const *pools, const int64_t *pool_block_bytes,
                  int num_pools, void *workspace, size_t workspace_bytes, struct CUstream_st *stream) {
  if (num_seqs <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || block_size <= 0 ||
      max_new_tokens < 0 || !pools_ok(pools, pool_block_bytes, num_pools))
    return PA_ERR_INVALID_ARG;
  if (num_seqs > kMaxRows) return PA_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * block_size > (int64_t)1 << 29) return PA_ERR_UNSUPPORTED;
  if (num_blocks > 1 << 30) return PA_ERR_UNSUPPORTED;
  if (!block_tables || !context_lens || !ref_counts || !append || !query_start_loc || !copy_pairs ||
      (max_new_tokens > 0 && !slot_mapping))
    return PA_ERR_INVALID_ARG;
  const TableWs w = table_ws(num_seqs, max_blocks_per_seq, num_blocks);
  if (!workspace || workspace_bytes < w.total || !aligned(workspace, 16)) return PA_ERR_WORKSPACE;
  DevInfo dev;
  if (device_info(&dev) != cudaSuccess) return PA_ERR_CUDA;
  char *ws = static_cast<char *>(workspace);
  StepArgs a;
  a.tables = block_tables;
  a.lens = context_lens;
  a.refs = ref_counts;
  a.release = release;
  a.fork_src = fork_src;
  a.append = append;
  a.slots = slot_mapping;
  a.pairs = copy_pairs;
  a.qsl = query_start_loc;
  a.S = num_seqs;
  a.W = max_blocks_per_seq;
  a.NB = num_blocks;
  a.bs = block_size;
  a.max_new = max_new_tokens;
  a.chunks = (num_blocks + kChunk - 1) / kChunk;
  a.wlen = reinterpret_cast<int *>(ws + w.len);
  a.writes = reinterpret_cast<int *>(ws + w.writes);
  a.info = reinterpret_cast<int *>(ws + w.info);
  a.base = reinterpret_cast<int *>(ws + w.base);
  a.chunk = reinterpret_cast<int *>(ws + w.chunk);
  a.fresh = reinterpret_cast<int *>(ws + w.list);
  a.wrows = reinterpret_cast<int *>(ws + w.rows);
  a.err = dev.err;
  cudaStream_t s = (cudaStream_t)stream;
  int64_t pieces;
  const Pools list = pool_list(pools, pool_block_bytes, num_pools, 0, num_seqs, &pieces);
  int64_t want = (num_seqs + kRowGroups - 1) / kRowGroups;
  if (a.chunks > want) want = a.chunks;
  if (pieces > want) want = pieces;
  cudaError_t e = launch_coop(step_kernel, coop_grid(want, dev.sm_count), s, (const StepArgs)a, (const Pools)list);
  if (e == cudaSuccess)
    e = launch_moves(pools, pool_block_bytes, num_pools, kPoolsPerLaunch, copy_pairs, num_seqs, dev.sm_count, s);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_table_compact(int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                     int32_t *ref_counts, int num_seqs, int num_blocks, int block_size,
                     int32_t *num_live, int64_t *block_moves, void *const *pools,
                     const int64_t *pool_block_bytes, int num_pools, void *workspace,
                     size_t workspace_bytes, struct CUstream_st *stream) {
  if (num_seqs <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || block_size <= 0 ||
      !pools_ok(pools, pool_block_bytes, num_pools))
    return PA_ERR_INVALID_ARG;
  if ((int64_t)max_blocks_per_seq * block_size > (int64_t)1 << 29) return PA_ERR_UNSUPPORTED;
  if (num_blocks > 1 << 30) return PA_ERR_UNSUPPORTED;
  if (!block_tables || !context_lens || !ref_counts || !num_live || !block_moves) return PA_ERR_INVALID_ARG;
  const TableWs w = table_ws(num_seqs, max_blocks_per_seq, num_blocks);
  if (!workspace || workspace_bytes < w.total || !aligned(workspace, 16)) return PA_ERR_WORKSPACE;
  DevInfo dev;
  if (device_info(&dev) != cudaSuccess) return PA_ERR_CUDA;
  char *ws = static_cast<char *>(workspace);
  CompactArgs a;
  a.tables = block_tables;
  a.refs = ref_counts;
  a.live = num_live;
  a.lens = context_lens;
  a.moves = block_moves;
  a.S = num_seqs;
  a.W = max_blocks_per_seq;
  a.NB = num_blocks;
  a.bs = block_size;
  a.chunks = (num_blocks + kChunk - 1) / kChunk;
  a.max_moves = num_blocks / 2 > 1 ? num_blocks / 2 : 1;
  a.chunk = reinterpret_cast<int *>(ws + w.chunk);
  a.remap = reinterpret_cast<int *>(ws + w.list);
  // at most num_blocks / 2 holes are filled, but up to `live` are listed from
  // the front; sources and holes are equally many, so both halves suffice
  a.holes = reinterpret_cast<int *>(ws + w.rows);
  a.sources = a.holes + num_blocks / 2;
  a.err = dev.err;
  cudaStream_t s = (cudaStream_t)stream;
  int64_t pieces;
  Pools list = pool_list(pools, pool_block_bytes, num_pools, 0, a.max_moves, &pieces);
  const bool apart = pieces > dev.sm_count * 2;  // more than a pass of the cooperative grid
  if (apart) list.n = 0;
  int64_t want = (num_seqs + kRowGroups - 1) / kRowGroups;
  if (a.chunks > want) want = a.chunks;
  if (!apart && pieces > want) want = pieces;
  cudaError_t e =
      launch_coop(compact_kernel, coop_grid(want, dev.sm_count), s, (const CompactArgs)a, (const Pools)list);
  if (e == cudaSuccess)
    e = launch_moves(pools, pool_block_bytes, num_pools, apart ? 0 : kPoolsPerLaunch, block_moves, a.max_moves,
                     dev.sm_count, s);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
