// The paged caches' bookkeeping: block tables and reference counts, and the rows that move with
// them, on the device. free, grow, fork, copy, compact as include/v4a.h states them.
//
// Every choice of a page goes by rank: the k-th block that needs one takes the k-th free page, the
// k-th used page behind the front moves to the k-th free one in it. Ranks are prefix sums, taken in
// two steps: counts by chunks of 4096 pages in a first kernel, ranks inside the chunks in a second.
// A kernel that changes counts reads those of its own pages only, so nothing depends on the order in
// which blocks run.
//
// Bound: launches and dependent lookups for free and grow (a table of 64 x 512 blocks and 16,384
// pages: 1.9 and 8.4 us); HBM for the rows that fork, copy and compact move (1,500 pages of six pools,
// 0.85 GB moved: 132 us, 6.4 TB/s, 96 % of a plain copy's; 45 forks of eight pools 14 us).
#include <cstdint>

#include "kernels.h"
#include "latent.h"

using namespace v4a;

namespace v4a {
namespace {

constexpr int kChunk = 4096;         // pages that a block counts or ranks
constexpr int kCountThreads = 256, kRankThreads = 1024;
constexpr int kPart = 16384;         // bytes of a page that a block moves at a time
constexpr int kCopyThreads = 256;

struct Pools {
  int32_t n;
  int32_t parts[V4A_MAX_POOLS + 1];  // parts of a page before each pool's
  v4a_pool pool[V4A_MAX_POOLS];
};

__device__ __forceinline__ bool is_page(int32_t v, int64_t n_pages) { return v >= 0 && v < n_pages; }
// The page of a table entry, or -1.
__device__ __forceinline__ int32_t page_of(int32_t v, int64_t n_pages, int32_t* err) {
  if (is_page(v, n_pages)) return v;
  if (v != -1) raise_err(err, V4A_DEV_BAD_PAGE);
  return -1;
}

// Exclusive prefix sum of v over the block (kThreads threads); *total its sum. tot: 32 words.
template <int kThreads>
__device__ __forceinline__ int block_scan(int v, int32_t* tot, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                   // the previous use of tot
  if (lane == 31) tot[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    const int t = tot[i];
    if (i < warp) before += t;
    all += t;
  }
  *total = all;
  return before + x - v;
}

// Which of the four pages p .. p + 3 are free (bit i), counting none outside the pool.
__device__ __forceinline__ int free4(const int32_t* refs, int64_t p, int64_t n_pages) {
  int4 r = make_int4(1, 1, 1, 1);
  if (p + 3 < n_pages) {
    r = *reinterpret_cast<const int4*>(refs + p);
  } else {
    if (p < n_pages) r.x = refs[p];
    if (p + 1 < n_pages) r.y = refs[p + 1];
    if (p + 2 < n_pages) r.z = refs[p + 2];
  }
  return (r.x <= 0) | (r.y <= 0) << 1 | (r.z <= 0) << 2 | (r.w <= 0) << 3;
}

// Free pages of a chunk, by the whole block (kCountThreads threads).
__device__ __forceinline__ void count_chunk(const int32_t* refs, int64_t n_pages, int chunk, int32_t* free_cnt) {
  __shared__ int32_t sum;
  if (threadIdx.x == 0) sum = 0;
  __syncthreads();
  int c = 0;
#pragma unroll
  for (int i = 0; i < kChunk / 4 / kCountThreads; ++i)
    c += __popc(free4(refs, (int64_t)chunk * kChunk + 4 * (threadIdx.x + i * kCountThreads), n_pages));
  c = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0 && c) atomicAdd(&sum, c);
  __syncthreads();
  if (threadIdx.x == 0) free_cnt[chunk] = sum;
}

// Free pages in the chunks before `chunk` and in all of them, by the whole block.
template <int kThreads>
__device__ __forceinline__ int chunks_before(const int32_t* free_cnt, int n_chunks, int chunk, int32_t* tot, int* all) {
  int a = 0, b = 0;
  for (int i = threadIdx.x; i < n_chunks; i += kThreads) {
    const int c = free_cnt[i];
    b += c;
    if (i < chunk) a += c;
  }
  int before;
  block_scan<kThreads>(a, tot, &before);
  block_scan<kThreads>(b, tot, all);
  return before;
}

// ------------------------------------------------------------------------------- free
__global__ void __launch_bounds__(256) pages_free_kernel(const v4a_page_table t, const int32_t* first,
                                                         const int32_t* last, int32_t* err) {
  pdl_wait();
  const int b = blockIdx.y;
  const int a = max(0, __ldg(first + b)), e = min(t.max_blocks, __ldg(last + b));
  for (int64_t k = a + (int64_t)blockIdx.x * 256 + threadIdx.x; k < e; k += (int64_t)gridDim.x * 256) {
    int32_t* at = t.block_table + (int64_t)b * t.max_blocks + k;
    const int32_t v = *at;
    if (v == -1) continue;
    *at = -1;
    const int32_t page = page_of(v, t.n_pages, err);
    if (page >= 0 && atomicSub(t.refs + page, 1) <= 0) {
      atomicAdd(t.refs + page, 1);
      raise_err(err, V4A_DEV_BAD_PAGE);
    }
  }
}

// ------------------------------------------------------------------------------- grow
struct GrowParams {
  v4a_page_table t;
  const int32_t* first;
  const int32_t* last;
  int32_t* free_cnt;   // [n_chunks]
  int32_t* need;       // [n_seq] blocks without a page
  int32_t* cell;       // [n_seq][max_blocks] which
  int32_t* err;
  int32_t n_chunks;
};

// Blocks 0 .. n_chunks - 1 count free pages, the others list the blocks of a row that need one.
__global__ void __launch_bounds__(kCountThreads) pages_need_kernel(const GrowParams p) {
  __shared__ int32_t tot[32];
  pdl_wait();
  if ((int)blockIdx.x < p.n_chunks) return count_chunk(p.t.refs, p.t.n_pages, blockIdx.x, p.free_cnt);
  const int b = blockIdx.x - p.n_chunks;
  const int a = max(0, __ldg(p.first + b)), e = min(p.t.max_blocks, __ldg(p.last + b));
  const int32_t* row = p.t.block_table + (int64_t)b * p.t.max_blocks;
  int32_t* cell = p.cell + (int64_t)b * p.t.max_blocks;
  int n = 0;
  for (int k0 = a; k0 < e; k0 += kCountThreads) {
    const int k = k0 + threadIdx.x;
    const bool takes = k < e && page_of(row[k], p.t.n_pages, p.err) < 0;
    int all;
    const int r = block_scan<kCountThreads>(takes, tot, &all);
    if (takes) cell[n + r] = k;
    n += all;
  }
  if (threadIdx.x == 0) p.need[b] = n;
}

__global__ void __launch_bounds__(kRankThreads) pages_give_kernel(const GrowParams p) {
  __shared__ int32_t pre[V4A_MAX_SEQ + 1];
  __shared__ int32_t tot[32];
  pdl_wait();
  seq_prefix(p.t.n_seq, pre, tot, [&](int b) { return p.need[b]; });
  const int needed = pre[p.t.n_seq];
  int all, here;
  int rank = chunks_before<kRankThreads>(p.free_cnt, p.n_chunks, blockIdx.x, tot, &all);
  if (blockIdx.x == 0 && threadIdx.x == 0 && needed > all) raise_err(p.err, V4A_DEV_NO_PAGE);
  if (rank >= needed) return;
  const int64_t page = (int64_t)blockIdx.x * kChunk + 4 * threadIdx.x;
  const int is_free = free4(p.t.refs, page, p.t.n_pages);
  rank += block_scan<kRankThreads>(__popc(is_free), tot, &here);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!(is_free >> i & 1) || rank >= needed) continue;
    const int b = latent_seq_at(pre, p.t.n_seq, rank);
    const int64_t row = (int64_t)b * p.t.max_blocks;
    p.t.block_table[row + p.cell[row + rank - pre[b]]] = (int32_t)(page + i);
    p.t.refs[page + i] = 1;
    ++rank;
  }
}

// ------------------------------------------------------------------------- moving rows
// Bytes [part * kPart, ..) of a page, up to `bytes` of it, by the whole block, 64 bytes a thread
// in flight.
__device__ __forceinline__ void copy_part(const v4a_pool& pool, int64_t from, int64_t to, int part, int64_t bytes,
                                          int rows) {
  const int64_t page = pool.row_bytes * pool.rows_per_block, at = (int64_t)part * kPart;
  const uint4* a = reinterpret_cast<const uint4*>(static_cast<const char*>(pool.data) + from * page + at);
  uint4* b = reinterpret_cast<uint4*>(static_cast<char*>(pool.data) + to * page + at);
  const int n = (int)max((int64_t)0, min((int64_t)kPart, bytes - at)) / 16;
  uint4 v[kPart / 16 / kCopyThreads];
#pragma unroll
  for (int i = 0; i < kPart / 16 / kCopyThreads; ++i) {
    const int k = threadIdx.x + i * kCopyThreads;
    if (k < n) v[i] = __ldcs(a + k);
  }
#pragma unroll
  for (int i = 0; i < kPart / 16 / kCopyThreads; ++i) {
    const int k = threadIdx.x + i * kCopyThreads;
    if (k < n) __stcs(b + k, v[i]);
  }
  if (part == 0 && pool.scale && (int)threadIdx.x < rows)      // at most 256 rows
    pool.scale[to * pool.rows_per_block + threadIdx.x] = pool.scale[from * pool.rows_per_block + threadIdx.x];
}

// The pool of part r of a page (all pools' parts in one line); r becomes the part in its pool.
__device__ __forceinline__ int pool_of(const Pools& pools, int& r) {
  int y = 0;
  while (y + 1 < pools.n && r >= pools.parts[y + 1]) ++y;
  r -= pools.parts[y];
  return y;
}

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ Pools pools, int64_t n_pages,
                                                                  const int32_t* src, const int32_t* dst,
                                                                  int32_t* err) {
  pdl_wait();
  const int i = blockIdx.y;
  int part = blockIdx.x;
  const int32_t a = __ldg(src + i), b = __ldg(dst + i);
  if (!is_page(a, n_pages) || !is_page(b, n_pages)) {
    if (part == 0 && threadIdx.x == 0) raise_err(err, V4A_DEV_BAD_PAGE);
    return;
  }
  if (a == b) return;
  const v4a_pool& pool = pools.pool[pool_of(pools, part)];
  copy_part(pool, a, b, part, pool.row_bytes * pool.rows_per_block, pool.rows_per_block);
}

// ------------------------------------------------------------------------------- fork
// An entry is to be carried out; its cut block, and the last whole block before it, need pages.
constexpr int32_t kForkOk = 1, kForkCut = 2, kForkLate = 4;
struct ForkParams {
  v4a_page_table t;
  const int32_t* src;
  const int32_t* dst;
  const int64_t* length;
  int32_t* free_cnt;   // [n_chunks]
  int32_t* state;      // [n] kFork* bits
  int32_t* page;       // [2][n] new pages of cut blocks, and of last whole blocks, or -1
  int32_t* err;
  int32_t n, n_chunks;
  int32_t late;        // the most of the pools': tokens behind a block that still write into it
};

// Blocks 0 .. n_chunks - 1 count free pages, the others look an entry over.
__global__ void __launch_bounds__(kCountThreads) pages_fork_check_kernel(const ForkParams p) {
  pdl_wait();
  if ((int)blockIdx.x < p.n_chunks) return count_chunk(p.t.refs, p.t.n_pages, blockIdx.x, p.free_cnt);
  const int i = blockIdx.x - p.n_chunks;
  const int s = __ldg(p.src + i), d = __ldg(p.dst + i);
  const int64_t len = __ldg(p.length + i);
  bool bad = s < 0 || s >= p.t.n_seq || d < 0 || d >= p.t.n_seq || s == d || len < 0 ||
             len > (int64_t)p.t.max_blocks * kBlock;
  if (!bad) {
    for (int j = threadIdx.x; j < p.n; j += kCountThreads)
      if (j != i) bad |= __ldg(p.dst + j) == d || __ldg(p.src + j) == d;
    for (int k = threadIdx.x; k < p.t.max_blocks; k += kCountThreads)
      bad |= page_of(p.t.block_table[(int64_t)d * p.t.max_blocks + k], p.t.n_pages, p.err) >= 0;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x != 0) return;
  int state = 0;
  if (bad) {
    raise_err(p.err, V4A_DEV_BAD_INDEX);
  } else {
    state = kForkOk;
    const int32_t* at = p.t.block_table + (int64_t)s * p.t.max_blocks + len / kBlock;
    if (len % kBlock && page_of(at[0], p.t.n_pages, p.err) >= 0) state |= kForkCut;
    if (len >= kBlock && len % kBlock < p.late && page_of(at[-1], p.t.n_pages, p.err) >= 0) state |= kForkLate;
  }
  p.state[i] = state;
}

// Their free pages: the k-th for the k-th block that needs one. Block (entry, 0): of the cut block,
// (entry, 1): of the one before it.
__global__ void __launch_bounds__(kCountThreads) pages_fork_find_kernel(const ForkParams p) {
  __shared__ int32_t tot[32];
  __shared__ int32_t found, left;
  pdl_wait();
  const int i = blockIdx.x, state = p.state[i];
  if (!(state & (blockIdx.y ? kForkLate : kForkCut))) return;
  int32_t* const page_at = p.page + (int64_t)blockIdx.y * p.n + i;
  int k = 0, rank, all;
  for (int j = threadIdx.x; j < i; j += kCountThreads) k += __popc(p.state[j] & (kForkCut | kForkLate));
  block_scan<kCountThreads>(k, tot, &rank);
  if (blockIdx.y == 0 && (state & kForkLate)) ++rank;
  if (threadIdx.x == 0) found = -1;
  for (int c0 = 0; c0 < p.n_chunks; c0 += kCountThreads) {      // the chunk that holds it
    const int c = c0 + threadIdx.x, n = c < p.n_chunks ? p.free_cnt[c] : 0;
    const int before = block_scan<kCountThreads>(n, tot, &all);
    if (before <= rank && rank < before + n) {
      found = c;
      left = rank - before;
    }
    __syncthreads();
    if (found >= 0) break;
    rank -= all;
  }
  const int chunk = found;
  rank = left;
  if (chunk < 0) {
    if (threadIdx.x == 0) {
      *page_at = -1;
      raise_err(p.err, V4A_DEV_NO_PAGE);
    }
    return;
  }
  constexpr int kSteps = kChunk / 4 / kCountThreads;
  for (int q = 0; q < kSteps; ++q) {
    const int64_t page = (int64_t)chunk * kChunk + 4 * (q * kCountThreads + threadIdx.x);
    int is_free = free4(p.t.refs, page, p.t.n_pages);
    const int before = block_scan<kCountThreads>(__popc(is_free), tot, &all);
    if (before <= rank && rank < before + __popc(is_free)) {
      for (int drop = rank - before; drop > 0; --drop) is_free &= is_free - 1;
      *page_at = (int32_t)(page + __ffs(is_free) - 1);
    }
    rank -= all;
  }
}

// Block (part, entry, 0): its part of the cut block's rows; the first also writes table and counts.
// Block (part, entry, 1): the same part of the whole block before it, where that one is copied.
__global__ void __launch_bounds__(kCopyThreads) pages_fork_move_kernel(const ForkParams p,
                                                                       const __grid_constant__ Pools pools) {
  pdl_wait();
  const int i = blockIdx.y;
  const int state = p.state[i];
  if (!(state & kForkOk)) return;
  const int64_t len = __ldg(p.length + i);
  const int whole = (int)(len / kBlock), cut = (int)(len % kBlock);
  const int32_t* from = p.t.block_table + (int64_t)__ldg(p.src + i) * p.t.max_blocks;
  const bool before = blockIdx.z;
  const int32_t cut_page = state & kForkCut ? p.page[i] : -1, late_page = state & kForkLate ? p.page[p.n + i] : -1;
  if (blockIdx.x == 0 && !before) {
    int32_t* to = p.t.block_table + (int64_t)__ldg(p.dst + i) * p.t.max_blocks;
    for (int k = threadIdx.x; k < (state & kForkLate ? whole - 1 : whole); k += kCopyThreads) {
      const int32_t v = page_of(from[k], p.t.n_pages, p.err);
      if (v < 0) continue;
      to[k] = v;
      atomicAdd(p.t.refs + v, 1);
    }
    if (threadIdx.x == 0 && cut_page >= 0) {
      to[whole] = cut_page;
      p.t.refs[cut_page] = 1;
    }
    if (threadIdx.x == 0 && late_page >= 0) {
      to[whole - 1] = late_page;
      p.t.refs[late_page] = 1;
    }
  }
  const int32_t page = before ? late_page : cut_page;
  if (page < 0 || pools.n == 0) return;
  int part = blockIdx.x;
  const v4a_pool& pool = pools.pool[pool_of(pools, part)];
  const int rows = before ? pool.rows_per_block : (pool.rows_per_block * cut + kBlock - 1) / kBlock;
  copy_part(pool, from[before ? whole - 1 : whole], page, part, rows * pool.row_bytes, rows);
}

// ---------------------------------------------------------------------------- compact
struct CompactParams {
  v4a_page_table t;
  int32_t* free_cnt;   // [n_chunks]
  int32_t* n_moves;
  int32_t* from;       // [n_pages] used pages behind the front, in order
  int32_t* to;         // [n_pages] free pages in it
  int32_t* rank;       // [n_pages] a page's place in `from`, or -1
  int32_t* n_used;
  int32_t* moved;
  int32_t* err;
  int32_t n_chunks;
};

__global__ void __launch_bounds__(kCountThreads) pages_count_kernel(const int32_t* refs, int64_t n_pages,
                                                                    int32_t* free_cnt) {
  pdl_wait();
  count_chunk(refs, n_pages, blockIdx.x, free_cnt);
}

__global__ void __launch_bounds__(kRankThreads) pages_rank_kernel(const CompactParams p) {
  __shared__ int32_t tot[32];
  pdl_wait();
  int all, inside, here;
  const int free_before = chunks_before<kRankThreads>(p.free_cnt, p.n_chunks, blockIdx.x, tot, &all);
  const int used = (int)p.t.n_pages - all;
  // free pages below the front's end
  const int edge = used / kChunk;
  int front = chunks_before<kRankThreads>(p.free_cnt, p.n_chunks, edge, tot, &all);
  {
    const int64_t page = (int64_t)edge * kChunk + 4 * threadIdx.x;
    int f = free4(p.t.refs, page, p.t.n_pages);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (page + i >= used) f &= ~(1 << i);
    block_scan<kRankThreads>(__popc(f), tot, &inside);
    front += inside;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *p.n_used = used;
    *p.n_moves = front;
  }
  const int64_t page = (int64_t)blockIdx.x * kChunk + 4 * threadIdx.x;
  const int is_free = free4(p.t.refs, page, p.t.n_pages);
  int fr = free_before + block_scan<kRankThreads>(__popc(is_free), tot, &here);   // free pages before
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t q = page + i;
    if (q >= p.t.n_pages) break;
    const bool f = is_free >> i & 1;
    int m = -1;
    if (f && q < used) p.to[fr] = (int32_t)q;
    if (!f && q >= used) {
      m = (int)(q - fr) - (used - front);          // used pages before it, less those in the front
      p.from[m] = (int32_t)q;
    }
    p.rank[q] = m;
    if (p.moved && m < 0) p.moved[q] = f ? -1 : (int32_t)q;
    fr += f;
  }
}

__global__ void __launch_bounds__(kCopyThreads) pages_move_kernel(const CompactParams p,
                                                                  const __grid_constant__ Pools pools) {
  pdl_wait();
  const int moves = *p.n_moves;
  const int64_t threads = (int64_t)gridDim.x * kCopyThreads, tid = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
  // the table (the counts, which change here, are not read for it)
  const int64_t cells = (int64_t)p.t.n_seq * p.t.max_blocks;
  for (int64_t c = tid; c < cells; c += threads) {
    const int32_t v = page_of(p.t.block_table[c], p.t.n_pages, p.err);
    const int32_t m = v >= 0 ? p.rank[v] : -1;
    if (m >= 0) p.t.block_table[c] = p.to[m];
  }
  for (int64_t m = tid; m < moves; m += threads) {
    const int32_t a = p.from[m], b = p.to[m];
    p.t.refs[b] = p.t.refs[a];
    p.t.refs[a] = 0;
    if (p.moved) p.moved[a] = b;
  }
  if (pools.n == 0) return;
  const int per = pools.parts[pools.n];
  const int64_t items = (int64_t)moves * per;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int m = (int)(it / per);
    int part = (int)(it - (int64_t)m * per);
    const v4a_pool& pool = pools.pool[pool_of(pools, part)];
    copy_part(pool, p.from[m], p.to[m], part, pool.row_bytes * pool.rows_per_block, pool.rows_per_block);
  }
}

// ------------------------------------------------------------------------------- host
constexpr int64_t kMaxPages = (int64_t)1 << 23;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int chunks_of(const v4a_page_table* t) { return (int)((t->n_pages + kChunk - 1) / kChunk); }

int check_table(const v4a_page_table* t) {
  if (!t || t->n_seq < 0 || t->max_blocks < 0 || t->n_pages < 0) return V4A_ERR_ARG;
  if (t->n_seq > V4A_MAX_SEQ || t->n_pages > kMaxPages || t->max_blocks > (1 << 20)) return V4A_ERR_UNSUPPORTED;
  if (t->n_seq > 0 && t->max_blocks > 0 && (!t->block_table || !aligned(t->block_table, 4))) return V4A_ERR_ARG;
  if (t->n_pages > 0 && (!t->refs || !aligned(t->refs, 16))) return V4A_ERR_ARG;
  return V4A_OK;
}

int check_pools(const v4a_pool* pools, int32_t n, Pools* out) {
  if (n < 0 || (n > 0 && !pools)) return V4A_ERR_ARG;
  if (n > V4A_MAX_POOLS) return V4A_ERR_UNSUPPORTED;
  out->n = n;
  out->parts[0] = 0;
  for (int i = 0; i < n; ++i) {
    const v4a_pool& p = pools[i];
    if (!p.data || !aligned(p.data, 16) || !aligned(p.scale, 4) || p.reserved != 0) return V4A_ERR_ARG;
    if (p.rows_per_block < 1 || p.rows_per_block > kBlock) return V4A_ERR_ARG;
    if (p.row_bytes <= 0 || p.row_bytes % 16) return V4A_ERR_ARG;
    if (p.late < 0 || p.late >= kBlock) return V4A_ERR_ARG;
    if (p.row_bytes > (1 << 20)) return V4A_ERR_UNSUPPORTED;
    const int64_t parts = (p.row_bytes * p.rows_per_block + kPart - 1) / kPart;
    out->pool[i] = p;
    out->parts[i + 1] = out->parts[i] + (int32_t)parts;
  }
  return V4A_OK;
}

// Words of the workspace: chunk counts, then what the calls keep (n_seq words and the table's size,
// three lists of forks, three of the pool's size and one word).
size_t words(const v4a_page_table* t) {
  size_t most = (size_t)t->n_seq * t->max_blocks + t->n_seq;
  if (most < 3 * (size_t)V4A_MAX_SEQ) most = 3 * V4A_MAX_SEQ;
  if (most < 3 * (size_t)t->n_pages + 1) most = 3 * (size_t)t->n_pages + 1;
  return (size_t)chunks_of(t) + most;
}

bool has_workspace(const v4a_page_table* t, const void* ws, size_t bytes) {
  return ws && aligned(ws, 256) && bytes >= v4a_pages_workspace_size(t);
}

int done(cudaError_t e) { return e == cudaSuccess ? V4A_OK : V4A_ERR_CUDA; }

}  // namespace
}  // namespace v4a

extern "C" {

size_t v4a_pages_workspace_size(const v4a_page_table* table) {
  if (check_table(table)) return 0;
  return (words(table) * sizeof(int32_t) + 255) / 256 * 256;
}

int v4a_pages_free(const v4a_page_table* table, const int32_t* first, const int32_t* last, int32_t* dev_err,
                   v4a_stream_t stream) {
  const int rc = check_table(table);
  if (rc) return rc;
  if (table->n_seq == 0 || table->max_blocks == 0) return V4A_OK;
  if (!first || !last) return V4A_ERR_ARG;
  const int64_t want = ((int64_t)table->max_blocks + 255) / 256;
  const dim3 grid((unsigned)(want < 64 ? want : 64), (unsigned)table->n_seq);
  return done(launch_pdl(pages_free_kernel, grid, dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), *table, first,
                         last, dev_err));
}

int v4a_pages_grow(const v4a_page_table* table, const int32_t* first, const int32_t* last, void* workspace,
                   size_t workspace_bytes, int32_t* dev_err, v4a_stream_t stream) {
  const int rc = check_table(table);
  if (rc) return rc;
  if (table->n_seq == 0 || table->max_blocks == 0) return V4A_OK;
  if (!first || !last || !has_workspace(table, workspace, workspace_bytes)) return V4A_ERR_ARG;
  GrowParams p{};
  p.t = *table;
  p.first = first;
  p.last = last;
  p.n_chunks = chunks_of(table);
  p.free_cnt = static_cast<int32_t*>(workspace);
  p.need = p.free_cnt + p.n_chunks;
  p.cell = p.need + table->n_seq;
  p.err = dev_err;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pdl(pages_need_kernel, dim3((unsigned)(p.n_chunks + table->n_seq)), dim3(kCountThreads), 0,
                             st, p);
  // (one block at least, which says that an empty pool has no page)
  if (e == cudaSuccess)
    e = launch_pdl(pages_give_kernel, dim3((unsigned)(p.n_chunks > 0 ? p.n_chunks : 1)), dim3(kRankThreads), 0, st, p);
  return done(e);
}

int v4a_pages_fork(const v4a_page_table* table, const v4a_pool* pools, int32_t n_pools, int32_t n, const int32_t* src,
                   const int32_t* dst, const int64_t* length, void* workspace, size_t workspace_bytes,
                   int32_t* dev_err, v4a_stream_t stream) {
  int rc = check_table(table);
  if (rc) return rc;
  Pools pl;
  if ((rc = check_pools(pools, n_pools, &pl))) return rc;
  if (n < 0) return V4A_ERR_ARG;
  if (n > V4A_MAX_SEQ) return V4A_ERR_UNSUPPORTED;
  if (n == 0) return V4A_OK;
  if (!src || !dst || !length || !has_workspace(table, workspace, workspace_bytes)) return V4A_ERR_ARG;
  ForkParams p{};
  p.t = *table;
  p.src = src;
  p.dst = dst;
  p.length = length;
  p.n = n;
  p.n_chunks = chunks_of(table);
  p.free_cnt = static_cast<int32_t*>(workspace);
  p.state = p.free_cnt + p.n_chunks;
  p.page = p.state + n;
  p.err = dev_err;
  for (int i = 0; i < pl.n; ++i) p.late = p.late > pl.pool[i].late ? p.late : pl.pool[i].late;
  const unsigned places = p.late > 0 ? 2 : 1;     // (no blocks for what no pool asks for)
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pdl(pages_fork_check_kernel, dim3((unsigned)(p.n_chunks + n)), dim3(kCountThreads), 0, st, p);
  if (e == cudaSuccess) e = launch_pdl(pages_fork_find_kernel, dim3((unsigned)n, places), dim3(kCountThreads), 0, st, p);
  const int parts = pl.parts[pl.n] > 0 ? pl.parts[pl.n] : 1;
  if (e == cudaSuccess)
    e = launch_pdl(pages_fork_move_kernel, dim3((unsigned)parts, (unsigned)n, places), dim3(kCopyThreads), 0, st, p, pl);
  return done(e);
}

int v4a_pages_copy(const v4a_page_table* table, const v4a_pool* pools, int32_t n_pools, int32_t n, const int32_t* src,
                   const int32_t* dst, int32_t* dev_err, v4a_stream_t stream) {
  int rc = check_table(table);
  if (rc) return rc;
  Pools pl;
  if ((rc = check_pools(pools, n_pools, &pl))) return rc;
  if (n < 0) return V4A_ERR_ARG;
  if (n > (1 << 20)) return V4A_ERR_UNSUPPORTED;
  if (n == 0 || pl.n == 0) return V4A_OK;
  if (!src || !dst) return V4A_ERR_ARG;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  for (int i = 0; i < n; i += 65535) {
    const int m = n - i < 65535 ? n - i : 65535;
    const cudaError_t e = launch_pdl(pages_copy_kernel, dim3((unsigned)pl.parts[pl.n], (unsigned)m),
                                     dim3(kCopyThreads), 0, st, pl, table->n_pages, src + i, dst + i, dev_err);
    if (e != cudaSuccess) return done(e);
  }
  return V4A_OK;
}

int v4a_pages_compact(const v4a_page_table* table, const v4a_pool* pools, int32_t n_pools, int32_t* n_used,
                      int32_t* moved, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                      v4a_stream_t stream) {
  int rc = check_table(table);
  if (rc) return rc;
  Pools pl;
  if ((rc = check_pools(pools, n_pools, &pl))) return rc;
  if (!n_used || !has_workspace(table, workspace, workspace_bytes)) return V4A_ERR_ARG;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (table->n_pages == 0) return done(cudaMemsetAsync(n_used, 0, sizeof(int32_t), st));
  CompactParams p{};
  p.t = *table;
  p.n_chunks = chunks_of(table);
  p.free_cnt = static_cast<int32_t*>(workspace);
  p.n_moves = p.free_cnt + p.n_chunks;
  p.from = p.n_moves + 1;
  p.to = p.from + table->n_pages;
  p.rank = p.to + table->n_pages;
  p.n_used = n_used;
  p.moved = moved;
  p.err = dev_err;
  const int32_t* refs = table->refs;
  cudaError_t e = launch_pdl(pages_count_kernel, dim3((unsigned)p.n_chunks), dim3(kCountThreads), 0, st, refs,
                             table->n_pages, p.free_cnt);
  if (e == cudaSuccess) e = launch_pdl(pages_rank_kernel, dim3((unsigned)p.n_chunks), dim3(kRankThreads), 0, st, p);
  if (e == cudaSuccess)
    e = launch_pdl(pages_move_kernel, dim3((unsigned)(8 * sm_count())), dim3(kCopyThreads), 0, st, p, pl);
  return done(e);
}

}  // extern "C"
