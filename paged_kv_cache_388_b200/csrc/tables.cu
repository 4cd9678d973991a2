// tables.cu -- block tables, lengths and reference counts held on the device:
// one scheduling step (release, fork, grow with copy-on-write) and compaction
// of the pool ("核心概念", sections 按需分配 and 内存共享; "理解 vLLM
// PagedAttention", sections 四 and 六: blocks are taken on demand, shared by
// reference count and copied before a shared one is written).
//
// Both are prefix sums over the pool and over the rows with scattered integer
// writes around them.  Order decides every result (lowest free id first, rows
// in order) and no result depends on the order of atomics: reference counts
// are integer sums.  The kernels of a call are chained with programmatic
// dependent launches; each waits for its predecessor's writes before it reads
// anything, so the chain costs little more than its dependent memory trips.
#include <limits.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kChunk = 1024;      // pool blocks per counting CTA (4 a thread)
constexpr int kThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kMaxRows = 4096;    // rows the one-CTA plan scans, 4 a thread
constexpr int kPoolsPerLaunch = 64;

// Workspace arrays (offsets in bytes, all 256-byte aligned).
struct TableWs {
  size_t scal, len, info, base, chunk, list, rows, total;
};

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

TableWs table_ws(int num_seqs, int width, int num_blocks) {
  TableWs w;
  const size_t chunks = ((size_t)num_blocks + kChunk - 1) / kChunk;
  size_t off = 0;
  w.scal = off;  // [8] ints: total taken, live, moves
  off += 256;
  w.len = off;  // [num_seqs] length after release and fork
  off += align_up((size_t)num_seqs * 4);
  w.info = off;  // [num_seqs][2] blocks needed | copy-on-write flag, last block
  off += align_up((size_t)num_seqs * 8);
  w.base = off;  // [num_seqs] first fresh block, -1: not grown
  off += align_up((size_t)num_seqs * 4);
  w.chunk = off;  // [chunks] counts, then their exclusive prefix
  off += align_up(chunks * 4);
  w.list = off;  // step: [num_blocks] fresh ids; compact: remap
  off += align_up((size_t)num_blocks * 4);
  w.rows = off;  // step: [num_seqs][width] forked rows; compact: [num_blocks] holes and sources
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
  int *scal, *wlen, *info, *base, *chunk, *fresh, *wrows;
  unsigned int *err;
};

__device__ __forceinline__ void pdl_begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ int row_len(const int32_t *lens, int i, int cap, unsigned int *err) {
  const int n = lens[i];
  if (n >= 0 && n <= cap) return n;
  raise_error(err, PA_DEVERR_CONTEXT_LEN);
  return 0;
}

// Exclusive prefix of v over a block of NT threads; *total gets the sum.  s: NT / 32 + 1 entries.
template <int NT, typename T>
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
    const T w = lane < NT / 32 ? s[lane] : 0;
    T y = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const T z = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) y += z;
    }
    if (lane < NT / 32) s[lane] = y - w;
    if (lane == 31) s[NT / 32] = y;
  }
  __syncthreads();
  *total = s[NT / 32];
  return x - v + s[warp];
}

// ---- pa_table_step ------------------------------------------------------------

// 1 and 2 of the step: one CTA per row.  Counts change by integer atomics; the
// blocks of a fork's source are put aside, since its row may itself change.
__global__ void __launch_bounds__(kThreads) step_release_kernel(const StepArgs a) {
  pdl_begin();
  const int i = blockIdx.x, cap = a.W * a.bs;
  int src = a.fork_src ? a.fork_src[i] : -1;
  if (src >= a.S) {
    if (threadIdx.x == 0) raise_error(a.err, PA_DEVERR_TABLE);
    src = -1;
  }
  const bool forked = src >= 0;
  const bool drop = forked || (a.release && a.release[i] != 0);
  const int len = row_len(a.lens, i, cap, threadIdx.x == 0 ? a.err : nullptr);
  int now = drop ? 0 : len;
  if (drop) {
    const int32_t *t = a.tables + (int64_t)i * a.W;
    const int n = (len + a.bs - 1) / a.bs;
    for (int j = threadIdx.x; j < n; j += kThreads) {
      const int b = t[j];
      if (b >= 0 && b < a.NB) atomicSub(a.refs + b, 1);
      else raise_error(a.err, PA_DEVERR_BLOCK_ID);
    }
  }
  if (forked) {
    now = row_len(a.lens, src, cap, nullptr);
    const int32_t *t = a.tables + (int64_t)src * a.W;
    int *keep = a.wrows + (int64_t)i * a.W;
    const int n = (now + a.bs - 1) / a.bs;
    for (int j = threadIdx.x; j < n; j += kThreads) {
      const int b = t[j];
      keep[j] = b;
      if (b >= 0 && b < a.NB) atomicAdd(a.refs + b, 1);
      else raise_error(a.err, PA_DEVERR_BLOCK_ID);
    }
  }
  if (threadIdx.x == 0) a.wlen[i] = now;
}

// The block that row r's next token is written into when its last block is
// partly filled, else -1.
__device__ __forceinline__ int write_block(const StepArgs &a, int r) {
  const int add = a.append[r], now = a.wlen[r];
  if (add <= 0 || now % a.bs == 0 || (int64_t)now + add > (int64_t)a.W * a.bs) return -1;
  const int src = a.fork_src ? a.fork_src[r] : -1;
  const int *t = src >= 0 && src < a.S ? a.wrows + (int64_t)r * a.W : a.tables + (int64_t)r * a.W;
  const int b = t[now / a.bs];
  return b >= 0 && b < a.NB ? b : -1;
}

// The first `chunks` CTAs count the pool's free blocks; the others take a row
// each: the forked rows' entries go into the tables and the row's need is
// worked out.  Of the rows that write into one shared block, in row order, all
// copy it but the last of its holders: the k-th writer of a block with r
// holders copies while r - k > 1.
__global__ void __launch_bounds__(kThreads) step_count_kernel(const StepArgs a) {
  __shared__ int s[kThreads / 32 + 1];
  pdl_begin();
  int total;
  if ((int)blockIdx.x < a.chunks) {
    const int id = blockIdx.x * kChunk + threadIdx.x * 4;
    int n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (id + k < a.NB) n += a.refs[id + k] == 0;
    block_scan<kThreads>(n, s, &total);
    if (threadIdx.x == 0) a.chunk[blockIdx.x] = total;
    return;
  }
  const int i = blockIdx.x - a.chunks;
  const int now = a.wlen[i], add = a.append[i];
  const int held = (now + a.bs - 1) / a.bs;
  const int src = a.fork_src ? a.fork_src[i] : -1;
  if (src >= 0 && src < a.S) {
    const int *keep = a.wrows + (int64_t)i * a.W;
    int32_t *t = a.tables + (int64_t)i * a.W;
    for (int j = threadIdx.x; j < held; j += kThreads) t[j] = keep[j];
  }
  const bool bad = add < 0 || (int64_t)now + add > (int64_t)a.W * a.bs;
  const int last = write_block(a, i);
  const int holders = last >= 0 ? a.refs[last] : 0;
  int before = 0;
  if (holders > 1)
    for (int r = threadIdx.x; r < i; r += kThreads) before += write_block(a, r) == last;
  block_scan<kThreads>(before, s, &total);
  if (threadIdx.x == 0) {
    const int cow = holders - total > 1;
    const int more = bad || add == 0 ? 0 : (int)(((int64_t)now + add + a.bs - 1) / a.bs) - held;
    if (bad) raise_error(a.err, PA_DEVERR_CONTEXT_LEN);
    a.info[2 * i] = (more + cow) << 1 | cow;
    a.info[2 * i + 1] = last;
  }
}

// One CTA: prefix sums of the free counts, of the rows' needs and of their
// tokens; the first row that does not fit ends the growing.
__global__ void __launch_bounds__(kPlanThreads) step_plan_kernel(const StepArgs a) {
  __shared__ int s[kPlanThreads / 32 + 1];
  __shared__ int64_t s64[kPlanThreads / 32 + 1];  // sums over rows may pass 32 bits
  pdl_begin();
  int avail = 0;
  for (int c0 = 0; c0 < a.chunks; c0 += kPlanThreads) {
    const int c = c0 + threadIdx.x;
    int total;
    const int n = c < a.chunks ? a.chunk[c] : 0;
    const int off = block_scan<kPlanThreads>(n, s, &total);
    if (c < a.chunks) a.chunk[c] = avail + off;
    avail += total;
  }
  int64_t taken = 0, tokens = 0;
  int best = 0;  // blocks taken by the leading run of rows that fit
  for (int r0 = 0; r0 < a.S; r0 += kPlanThreads) {
    const int i = r0 + threadIdx.x;
    const int add = i < a.S ? max(a.append[i], 0) : 0;
    const int need = i < a.S ? a.info[2 * i] >> 1 : 0;
    int64_t t_need, t_add;
    const int64_t first = taken + block_scan<kPlanThreads, int64_t>(need, s64, &t_need);
    const int64_t tok = tokens + block_scan<kPlanThreads, int64_t>(add, s64, &t_add);
    if (i < a.S) {
      // need is never negative, so the rows that fit are a leading run
      const bool fits = first + need <= avail;
      const bool ok = fits && a.append[i] >= 0 && (int64_t)a.wlen[i] + add <= (int64_t)a.W * a.bs;
      if (!fits && add > 0) raise_error(a.err, PA_DEVERR_POOL);
      a.base[i] = ok ? (int)first : -1;
      a.qsl[i] = (int)min(tok, (int64_t)INT_MAX);
      if (ok) best = max(best, (int)first + need);
    }
    taken += t_need;
    tokens += t_add;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = best;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kPlanThreads / 32; ++w) best = max(best, s[w]);
    a.scal[0] = best;
    a.qsl[a.S] = (int)min(tokens, (int64_t)INT_MAX);
    if (tokens > a.max_new) raise_error(a.err, PA_DEVERR_SLOT);
  }
}

// The free blocks of lowest id, in order, into the list of fresh ones.
__global__ void __launch_bounds__(kThreads) step_take_kernel(const StepArgs a) {
  __shared__ int s[kThreads / 32 + 1];
  pdl_begin();
  const int take = a.scal[0];
  int rank = a.chunk[blockIdx.x];
  if (rank >= take) return;
  const int id = blockIdx.x * kChunk + threadIdx.x * 4;
  bool free_[4];
  int n = 0, total;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    free_[k] = id + k < a.NB && a.refs[id + k] == 0;
    n += free_[k];
  }
  rank += block_scan<kThreads>(n, s, &total);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (free_[k]) {
      if (rank < take) {
        a.fresh[rank] = id + k;
        a.refs[id + k] = 1;
      }
      ++rank;
    }
}

// One CTA per row: its fresh blocks, slots, length; the CTAs after them fill
// the rest of slot_mapping.
__global__ void __launch_bounds__(kThreads) step_apply_kernel(const StepArgs a) {
  pdl_begin();
  const int i = blockIdx.x;
  if (i >= a.S) {
    const int64_t p = (int64_t)a.qsl[a.S] + (int64_t)(i - a.S) * kThreads + threadIdx.x;
    for (int64_t x = p; x < a.max_new; x += (int64_t)(gridDim.x - a.S) * kThreads) a.slots[x] = -1;
    return;
  }
  const int now = a.wlen[i], add = max(a.append[i], 0), base = a.base[i];
  const int info = a.info[2 * i], cow = info & 1, more = (info >> 1) - cow;
  const int held = (now + a.bs - 1) / a.bs;
  const int64_t p0 = a.qsl[i];
  if (base < 0) {
    if (threadIdx.x == 0) {
      a.lens[i] = now;
      a.pairs[2 * i] = a.pairs[2 * i + 1] = -1;
    }
    for (int t = threadIdx.x; t < add; t += kThreads)
      if (p0 + t < a.max_new) a.slots[p0 + t] = -1;
    return;
  }
  int32_t *row = a.tables + (int64_t)i * a.W;
  for (int k = threadIdx.x; k < more; k += kThreads) row[held + k] = a.fresh[base + cow + k];
  if (threadIdx.x == 0) {
    const int last = a.info[2 * i + 1];
    const int dst = cow ? a.fresh[base] : -1;
    if (cow) {
      row[held - 1] = dst;
      atomicSub(a.refs + last, 1);
    }
    a.pairs[2 * i] = cow ? last : -1;
    a.pairs[2 * i + 1] = dst;
    a.lens[i] = now + add;
  }
  __syncthreads();
  for (int t = threadIdx.x; t < add; t += kThreads) {
    if (p0 + t >= a.max_new) break;
    const int pos = now + t, b = row[pos / a.bs];
    a.slots[p0 + t] = b >= 0 && b < a.NB ? (int64_t)b * a.bs + pos % a.bs : -1;
  }
}

// ---- block moves -----------------------------------------------------------------

// Copies whole blocks (src, dst) in every pool of the list: one 8 KB piece per
// CTA iteration, four 16-byte loads in flight per thread.  `count`: pairs, on
// the device; pairs of -1 are skipped.  Bound: memory traffic.
constexpr int kMoveVecs = 4 * kThreads;
__global__ void __launch_bounds__(kThreads) move_blocks_kernel(const Pools pools, const int64_t *pairs,
                                                               const int *count, int max_pairs) {
  pdl_begin();
  const int n = count ? min(*count, max_pairs) : max_pairs;
  for (int k = 0; k < pools.n; ++k) {
    const int64_t vecs = pools.vecs[k];
    const int64_t pieces = (vecs + kMoveVecs - 1) / kMoveVecs;
    for (int64_t w = blockIdx.x; w < n * pieces; w += gridDim.x) {
      const int64_t pair = w / pieces, v0 = (w - pair * pieces) * kMoveVecs + threadIdx.x;
      const int64_t src = pairs[2 * pair], dst = pairs[2 * pair + 1];
      if (src < 0 || dst < 0) continue;
      const uint4 *from = pools.p[k] + src * vecs;
      uint4 *to = pools.p[k] + dst * vecs;
      uint4 r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (v0 + u * kThreads < vecs) r[u] = __ldcs(from + v0 + u * kThreads);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (v0 + u * kThreads < vecs) to[v0 + u * kThreads] = r[u];
    }
  }
}

// ---- pa_table_compact ------------------------------------------------------------

struct CompactArgs {
  int32_t *tables, *refs, *live;
  const int32_t *lens;
  int64_t *moves;
  int S, W, NB, bs, chunks, max_moves;
  int *scal, *chunk, *remap, *holes, *sources;
  unsigned int *err;
};

__global__ void __launch_bounds__(kThreads) compact_count_kernel(const CompactArgs a) {
  __shared__ int s[kThreads / 32 + 1];
  pdl_begin();
  const int id = blockIdx.x * kChunk + threadIdx.x * 4;
  int n = 0, total;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (id + k < a.NB) n += a.refs[id + k] > 0;
  block_scan<kThreads>(n, s, &total);
  if (threadIdx.x == 0) a.chunk[blockIdx.x] = total;
}

// One CTA: used blocks before each chunk, the live count, and the used blocks
// that already lie below it.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactArgs a) {
  __shared__ int s[kPlanThreads / 32 + 1];
  pdl_begin();
  int live = 0, total;
  for (int c0 = 0; c0 < a.chunks; c0 += kPlanThreads) {
    const int c = c0 + threadIdx.x;
    const int n = c < a.chunks ? a.chunk[c] : 0;
    const int off = block_scan<kPlanThreads>(n, s, &total);
    if (c < a.chunks) a.chunk[c] = live + off;
    live += total;
  }
  __syncthreads();
  const int c = live / kChunk;  // the chunk that the border falls into
  int below = live;
  if (c < a.chunks) {
    const int id = c * kChunk + threadIdx.x;
    block_scan<kPlanThreads, int>(id < live && a.refs[id] > 0, s, &total);
    below = a.chunk[c] + total;
  }
  if (threadIdx.x == 0) {
    a.scal[0] = live - below;  // moves
    a.scal[1] = live;
    a.scal[2] = below;
    *a.live = live;
  }
}

// k-th free id below the border and k-th used id at or past it.
__global__ void __launch_bounds__(kThreads) compact_list_kernel(const CompactArgs a) {
  __shared__ int s[kThreads / 32 + 1];
  pdl_begin();
  const int live = a.scal[1], below = a.scal[2];
  const int id = blockIdx.x * kChunk + threadIdx.x * 4;
  bool used[4];
  int n = 0, total;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    used[k] = id + k < a.NB && a.refs[id + k] > 0;
    n += used[k];
  }
  int before = a.chunk[blockIdx.x] + block_scan<kThreads>(n, s, &total);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int b = id + k;
    if (b < live && !used[k]) a.holes[b - before] = b;
    if (b >= live && b < a.NB) a.remap[b] = b;  // a held block without a count stays where it is
    if (b >= live && used[k]) a.sources[before - below] = b;
    before += used[k];
  }
}

__global__ void __launch_bounds__(kThreads) compact_move_kernel(const CompactArgs a) {
  pdl_begin();
  const int n = a.scal[0];
  const int k = blockIdx.x * kThreads + threadIdx.x;
  if (k < n) {
    const int src = a.sources[k], dst = a.holes[k];
    a.remap[src] = dst;
    a.refs[dst] = a.refs[src];
    a.refs[src] = 0;
    a.moves[2 * (int64_t)k] = src;
    a.moves[2 * (int64_t)k + 1] = dst;
  } else if (k < a.max_moves) {
    a.moves[2 * (int64_t)k] = a.moves[2 * (int64_t)k + 1] = -1;
  }
}

__global__ void __launch_bounds__(kThreads) compact_tables_kernel(const CompactArgs a) {
  pdl_begin();
  const int i = blockIdx.x, live = a.scal[1];
  const int len = row_len(a.lens, i, a.W * a.bs, threadIdx.x == 0 ? a.err : nullptr);
  int32_t *t = a.tables + (int64_t)i * a.W;
  const int n = (len + a.bs - 1) / a.bs;
  for (int j = threadIdx.x; j < n; j += kThreads) {
    const int b = t[j];
    if (b < 0 || b >= a.NB) raise_error(a.err, PA_DEVERR_BLOCK_ID);
    else if (b >= live) t[j] = a.remap[b];
  }
}

// ---- host ---------------------------------------------------------------------------

template <typename... Args>
cudaError_t launch_dep(void (*kernel)(Args...), int grid, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool pools_ok(void *const *pools, const int64_t *bytes, int n) {
  if (n < 0 || n > 1024 || (n > 0 && (!pools || !bytes))) return false;
  for (int i = 0; i < n; ++i)
    if (!pools[i] || (reinterpret_cast<uintptr_t>(pools[i]) & 15u) || bytes[i] <= 0 || bytes[i] % 16) return false;
  return true;
}

cudaError_t launch_moves(void *const *pools, const int64_t *bytes, int n, const int64_t *pairs,
                         const int *count, int max_pairs, int sm_count, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  for (int p0 = 0; p0 < n && max_pairs > 0 && e == cudaSuccess; p0 += kPoolsPerLaunch) {
    Pools list;
    list.n = n - p0 < kPoolsPerLaunch ? n - p0 : kPoolsPerLaunch;
    int64_t pieces = 0;
    for (int k = 0; k < list.n; ++k) {
      list.p[k] = static_cast<uint4 *>(pools[p0 + k]);
      list.vecs[k] = bytes[p0 + k] / 16;
      const int64_t x = (list.vecs[k] + kMoveVecs - 1) / kMoveVecs;
      if (x > pieces) pieces = x;
    }
    int64_t grid = pieces * max_pairs;
    if (grid > (int64_t)sm_count * 8) grid = (int64_t)sm_count * 8;
    e = launch_dep(move_blocks_kernel, (int)grid, kThreads, s, list, pairs, count, max_pairs);
  }
  return e;
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
  a.scal = reinterpret_cast<int *>(ws + w.scal);
  a.wlen = reinterpret_cast<int *>(ws + w.len);
  a.info = reinterpret_cast<int *>(ws + w.info);
  a.base = reinterpret_cast<int *>(ws + w.base);
  a.chunk = reinterpret_cast<int *>(ws + w.chunk);
  a.fresh = reinterpret_cast<int *>(ws + w.list);
  a.wrows = reinterpret_cast<int *>(ws + w.rows);
  a.err = dev.err;
  cudaStream_t s = (cudaStream_t)stream;
  int tail = (max_new_tokens + kThreads - 1) / kThreads;
  if (tail > 64) tail = 64;
  cudaError_t e = launch_dep(step_release_kernel, num_seqs, kThreads, s, (const StepArgs)a);
  if (e == cudaSuccess) e = launch_dep(step_count_kernel, a.chunks + num_seqs, kThreads, s, (const StepArgs)a);
  if (e == cudaSuccess) e = launch_dep(step_plan_kernel, 1, kPlanThreads, s, (const StepArgs)a);
  if (e == cudaSuccess) e = launch_dep(step_take_kernel, a.chunks, kThreads, s, (const StepArgs)a);
  if (e == cudaSuccess) e = launch_dep(step_apply_kernel, num_seqs + tail, kThreads, s, (const StepArgs)a);
  if (e == cudaSuccess)
    e = launch_moves(pools, pool_block_bytes, num_pools, copy_pairs, nullptr, num_seqs, dev.sm_count, s);
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
  a.scal = reinterpret_cast<int *>(ws + w.scal);
  a.chunk = reinterpret_cast<int *>(ws + w.chunk);
  a.remap = reinterpret_cast<int *>(ws + w.list);
  // at most num_blocks / 2 holes are filled, but up to `live` are listed from
  // the front; sources and holes are equally many, so both halves suffice
  a.holes = reinterpret_cast<int *>(ws + w.rows);
  a.sources = a.holes + num_blocks / 2;
  a.err = dev.err;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = launch_dep(compact_count_kernel, a.chunks, kThreads, s, (const CompactArgs)a);
  if (e == cudaSuccess) e = launch_dep(compact_plan_kernel, 1, kPlanThreads, s, (const CompactArgs)a);
  if (e == cudaSuccess) e = launch_dep(compact_list_kernel, a.chunks, kThreads, s, (const CompactArgs)a);
  if (e == cudaSuccess)
    e = launch_dep(compact_move_kernel, (a.max_moves + kThreads - 1) / kThreads, kThreads, s, (const CompactArgs)a);
  if (e == cudaSuccess) e = launch_dep(compact_tables_kernel, num_seqs, kThreads, s, (const CompactArgs)a);
  if (e == cudaSuccess)
    e = launch_moves(pools, pool_block_bytes, num_pools, block_moves, a.scal, a.max_moves, dev.sm_count, s);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
