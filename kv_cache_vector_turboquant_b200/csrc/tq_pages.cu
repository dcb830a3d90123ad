// Pages of a paged packed cache: fork (a child sequence shares its parent's
// full pages and gets a copy of the partly filled last one), trim (pages that
// no later query sees, or whose sequence has ended, are given back) and
// compact (the used pages move to the front of the pools).
//
// State, all on the device: block_tables [n_rows, max_blocks] (page of
// positions [16 j, 16 j + 16) of a row, negative = none), lens [n_rows],
// refs [num_blocks] (rows holding the page; <= 0 = free) and the pools (any
// number of arrays of num_blocks pages of block_bytes each: the codes and
// norms of every layer). Each call reads one set of tables and writes
// another, which may be the same arrays.
//
// A call is one planning kernel, which reads only what the call's last kernel
// does not write (so that in-place calls need no copy), and one grid-wide
// kernel that writes tables and counts and moves pages. Results do not depend
// on the order of threads: page choices follow page numbers, counts are
// integer sums.
//
// Bound: the pages that move, read and written once (a warp moves 2 KB at a
// time, 64 B per lane in flight), and the tables and counts, read and written
// once; small calls are bound by their two launches. Measured: fork of 256
// rows, each with a partly filled page in 32 layers' pools (205 MB moved), plan
// 6.3 us and apply 36.7 us, 5.6 TB/s; compaction of 8192 pages, 60 % used, of
// 16 layers (837 MB), plan 9.4 us and apply 140 us, 6.0 TB/s; trim of 512 rows
// of 2048 table entries, copy 4.3 us and trim 10 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "tq_common.cuh"

namespace tq {

constexpr int PG_THREADS = 256;
constexpr int PG_PLAN_THREADS = 1024;
constexpr int PG_SEG = 4 * PG_PLAN_THREADS;   // pages counted per step of a planning CTA
constexpr int PG_SEG_PAGES = 2 * PG_SEG;      // pages of one planning CTA of compact
constexpr int PG_UNIT = 2048;                 // bytes moved by a warp at a time
constexpr int PG_TOKENS = 16;                 // positions of a page

// The pools, in the kernel parameters: base and size of a page, and the units
// of a page over all pools in order (prefix sums).
struct PgPools {
  uint8_t* base[TQ_MAX_PAGE_POOLS];
  uint32_t bytes[TQ_MAX_PAGE_POOLS];
  uint32_t unit0[TQ_MAX_PAGE_POOLS + 1];
  int n;
};

// Shared copy of the pools' table (every thread of the CTA; ends with a barrier).
struct PgShared {
  uint8_t* base[TQ_MAX_PAGE_POOLS];
  uint32_t bytes[TQ_MAX_PAGE_POOLS];
  uint32_t unit0[TQ_MAX_PAGE_POOLS + 1];
};
TQ_DEV void pg_load_pools(PgShared& s, const PgPools& p) {
  for (int i = threadIdx.x; i < p.n; i += blockDim.x) {
    s.base[i] = p.base[i];
    s.bytes[i] = p.bytes[i];
    s.unit0[i] = p.unit0[i];
  }
  if (threadIdx.x == 0) s.unit0[p.n] = p.unit0[p.n];
  __syncthreads();
}

// Copy unit u of page src to page dst (one warp).
TQ_DEV void pg_move_unit(const PgShared& s, int n_pools, uint32_t u, int64_t src, int64_t dst, uint32_t lane) {
  int lo = 0, hi = n_pools - 1;  // the pool with unit0[pool] <= u < unit0[pool + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.unit0[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  const uint32_t bytes = s.bytes[lo], off = (u - s.unit0[lo]) * PG_UNIT;
  const uint8_t* from = s.base[lo] + src * (int64_t)bytes + off;
  uint8_t* to = s.base[lo] + dst * (int64_t)bytes + off;
  const uint32_t left = bytes - off;
  uint4 v[PG_UNIT / 512];
#pragma unroll
  for (int i = 0; i < PG_UNIT / 512; ++i)
    if (lane * 16u + i * 512u < left) v[i] = *reinterpret_cast<const uint4*>(from + lane * 16u + i * 512u);
#pragma unroll
  for (int i = 0; i < PG_UNIT / 512; ++i)
    if (lane * 16u + i * 512u < left) *reinterpret_cast<uint4*>(to + lane * 16u + i * 512u) = v[i];
}

// Exclusive prefix sum of v over the CTA's threads and its total (two
// barriers; `buf` holds one int per warp and one more).
TQ_DEV int pg_scan(int v, int* buf, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += o;
  }
  __syncthreads();  // the previous call's readers are done with buf
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int w = lane < nw ? buf[lane] : 0;
    int y = w;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, y, m);
      if (lane >= m) y += o;
    }
    if (lane < nw) buf[lane] = y - w;
    if (lane == 31) buf[32] = y;
  }
  __syncthreads();
  total = buf[32];
  return buf[warp] + x - v;
}

// Grid-stride copy of n ints (skipped when in place).
TQ_DEV void pg_copy_ints(int32_t* to, const int32_t* from, int64_t n, int64_t t, int64_t step) {
  if (to == from) return;
  if (((reinterpret_cast<uintptr_t>(to) | reinterpret_cast<uintptr_t>(from)) & 15) == 0) {
    for (int64_t i = t; i < n / 4; i += step)
      reinterpret_cast<int4*>(to)[i] = reinterpret_cast<const int4*>(from)[i];
    for (int64_t i = (n & ~(int64_t)3) + t; i < n; i += step) to[i] = from[i];
  } else {
    for (int64_t i = t; i < n; i += step) to[i] = from[i];
  }
}

// ------------------------------------------------------------------ fork

struct PgFork {
  const int32_t *tables, *lens, *refs, *parents, *children;
  int32_t *tables_out, *lens_out, *refs_out;
  // plan of fork i: state[i] (0 skipped, 1 taken, 2 child left empty), the
  // pages copied, src[i] -> dst[i] (-1: none)
  int32_t *state, *src, *dst;
  int32_t* fresh;  // the lowest free pages, in order
  int64_t num_blocks;
  int n_rows, max_blocks, n;
  uint32_t* err;
};

TQ_DEV int64_t pg_length(const PgFork& a, int row) {
  const int64_t most = (int64_t)a.max_blocks * PG_TOKENS, len = a.lens[row];
  return len < 0 ? 0 : (len > most ? most : len);
}

// CTA 0 plans; the others copy the tables and counts of out-of-place calls.
// A child named twice, or that is a parent too, and rows outside the table are
// skipped and flagged; the free pages are given out in order of page number
// to the forks in list order.
__global__ void __launch_bounds__(PG_PLAN_THREADS) fork_plan_kernel(const __grid_constant__ PgFork a) {
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    const int64_t t = (int64_t)(blockIdx.x - 1) * blockDim.x + tid, step = (int64_t)(gridDim.x - 1) * blockDim.x;
    pg_copy_ints(a.tables_out, a.tables, (int64_t)a.n_rows * a.max_blocks, t, step);
    pg_copy_ints(a.lens_out, a.lens, a.n_rows, t, step);
    pg_copy_ints(a.refs_out, a.refs, a.num_blocks, t, step);
    return;
  }
  extern __shared__ uint32_t marks[];  // per row: named as a child, as one twice, as a parent
  __shared__ int buf[33];
  const int words = (a.n_rows + 31) / 32;
  uint32_t *child = marks, *twice = marks + words, *parent = marks + 2 * words;
  for (int i = tid; i < 3 * words; i += blockDim.x) marks[i] = 0;
  __syncthreads();
  for (int i = tid; i < a.n; i += blockDim.x) {
    const int c = a.children[i], p = a.parents[i];
    if (c >= 0 && c < a.n_rows) {
      const uint32_t bit = 1u << (c & 31);
      if (atomicOr(&child[c >> 5], bit) & bit) atomicOr(&twice[c >> 5], bit);
    }
    if (p >= 0 && p < a.n_rows) atomicOr(&parent[p >> 5], 1u << (p & 31));
  }
  __syncthreads();
  int want = 0;  // pages given out so far
  for (int i0 = 0; i0 < a.n; i0 += blockDim.x) {
    const int i = i0 + tid;
    int state = 0, src = -1;
    if (i < a.n) {
      const int c = a.children[i], p = a.parents[i];
      const bool ok = c >= 0 && c < a.n_rows && p >= 0 && p < a.n_rows &&
                      !((twice[c >> 5] | parent[c >> 5]) >> (c & 31) & 1u);
      if (ok) {
        state = 1;
        if (a.lens[p] > (int64_t)a.max_blocks * PG_TOKENS) record_error(a.err, TQ_DEVERR_POS_RANGE);
        const int64_t len = pg_length(a, p);
        if (len % PG_TOKENS) {
          src = a.tables[(int64_t)p * a.max_blocks + len / PG_TOKENS];
          if (src >= a.num_blocks) {
            record_error(a.err, TQ_DEVERR_BLOCK_RANGE);
            src = -1;
          }
          src = src < 0 ? -1 : src;
        }
      } else {
        record_error(a.err, TQ_DEVERR_ROW_RANGE);
      }
    }
    int total;
    const int rank = pg_scan(src >= 0, buf, total);
    if (i < a.n) {
      a.state[i] = state;
      a.src[i] = src;
      a.dst[i] = src >= 0 ? want + rank : -1;  // its place among the free pages
    }
    want += total;
  }
  int found = 0;
  for (int64_t b0 = 0; b0 < a.num_blocks && found < want; b0 += PG_SEG) {
    bool free_[4];
    int mine = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t b = b0 + 4 * tid + k;
      free_[k] = b < a.num_blocks && a.refs[b] <= 0;
      mine += free_[k];
    }
    int total, at = pg_scan(mine, buf, total);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (free_[k]) {
        if (found + at < want) a.fresh[found + at] = (int32_t)(b0 + 4 * tid + k);
        ++at;
      }
    }
    found += total;
  }
  __syncthreads();
  for (int i = tid; i < a.n; i += blockDim.x) {
    const int place = a.dst[i];
    if (place < 0) continue;
    if (place < found) {
      a.dst[i] = a.fresh[place];
    } else {
      record_error(a.err, TQ_DEVERR_POOL_FULL);
      a.state[i] = 2;
      a.src[i] = a.dst[i] = -1;
    }
  }
}

__global__ void __launch_bounds__(PG_THREADS) fork_apply_kernel(const __grid_constant__ PgFork a,
                                                               const __grid_constant__ PgPools pools) {
  __shared__ PgShared s;
  pg_load_pools(s, pools);
  grid_dep_wait();
  // rows: parents' rows are never written (a child that is a parent is skipped)
  for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
    const int state = a.state[i];
    if (state == 0) continue;
    const int c = a.children[i], p = a.parents[i];
    const int64_t len = state == 1 ? pg_length(a, p) : 0;
    const int whole = (int)(len / PG_TOKENS), fresh = a.dst[i];
    const int32_t* from = a.tables + (int64_t)p * a.max_blocks;
    int32_t* to = a.tables_out + (int64_t)c * a.max_blocks;
    for (int j = threadIdx.x; j < a.max_blocks; j += blockDim.x) {
      int e = -1;
      if (j < whole) {
        e = from[j];
        if (e >= a.num_blocks) record_error(a.err, TQ_DEVERR_BLOCK_RANGE);
        if (e < 0 || e >= a.num_blocks) e = -1;
        else atomicAdd(a.refs_out + e, 1);
      } else if (j == whole && fresh >= 0) {
        e = fresh;
        a.refs_out[e] = 1;
      }
      to[j] = e;
    }
    if (threadIdx.x == 0) a.lens_out[c] = (int32_t)len;
  }
  const uint32_t units = s.unit0[pools.n];
  const int64_t all = (int64_t)units * a.n, step = (int64_t)gridDim.x * (PG_THREADS / 32);
  for (int64_t w = (int64_t)blockIdx.x * (PG_THREADS / 32) + (threadIdx.x >> 5); w < all; w += step) {
    const int i = (int)(w / units);
    const int dst = a.dst[i];
    if (dst >= 0) pg_move_unit(s, pools.n, (uint32_t)(w - (int64_t)i * units), a.src[i], dst, threadIdx.x & 31);
  }
}

// ------------------------------------------------------------------ trim

struct PgTrim {
  const int32_t *tables, *lens, *refs;
  int32_t *tables_out, *lens_out, *refs_out;
  const uint8_t* release;
  int64_t num_blocks, window, sinks;  // window < 0: none
  int n_rows, max_blocks;
  uint32_t* err;
};

__global__ void __launch_bounds__(PG_THREADS) trim_copy_kernel(const __grid_constant__ PgTrim a) {
  grid_dep_launch();
  const int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
  pg_copy_ints(a.refs_out, a.refs, a.num_blocks, t, step);
}

// Page j of a row of length L is given back when its row is released, or when
// it holds no sink position and ends at or before L - window: the query at
// position p sees t > p - window, and every query from the row's last token
// on has p >= L - 1.
__global__ void __launch_bounds__(PG_THREADS) trim_kernel(const __grid_constant__ PgTrim a) {
  const int64_t n = (int64_t)a.n_rows * a.max_blocks, most = (int64_t)a.max_blocks * PG_TOKENS;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  bool waited = false;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
    const int row = (int)(i / a.max_blocks), j = (int)(i - (int64_t)row * a.max_blocks);
    const int32_t e = a.tables[i];
    int64_t len = a.lens[row];
    const bool released = a.release != nullptr && a.release[row] != 0;
    // (in place, only a released row's length changes, and its pages go
    // whatever its length: the row's other threads need not have read it)
    if (j == 0) {
      if (len > most) record_error(a.err, TQ_DEVERR_POS_RANGE);
      if (released) a.lens_out[row] = 0;
      else if (a.lens_out != a.lens) a.lens_out[row] = (int32_t)len;
    }
    len = min64(len, most);
    const int64_t first = (int64_t)j * PG_TOKENS;
    const bool gone = released || (a.window >= 0 && first >= a.sinks && first + PG_TOKENS <= len - a.window);
    if (!waited) grid_dep_wait();
    waited = true;
    int32_t out = e;
    if (gone && e >= 0) {
      if (e < a.num_blocks) atomicSub(a.refs_out + e, 1);
      else record_error(a.err, TQ_DEVERR_BLOCK_RANGE);
      out = -1;
    }
    a.tables_out[i] = out;
  }
  if (!waited) grid_dep_wait();
}

// ------------------------------------------------------------------ compact

struct PgCompact {
  const int32_t *tables, *refs;
  int32_t *tables_out, *refs_out, *remap, *used;
  // workspace: head[0] = used pages U, head[1] = free pages below U (= moves)
  int32_t *head, *seg_used;
  int32_t* rank;  // used page: pages used before it; free page: -1 - that count
  int32_t* src;   // by rank: the used pages at or above U
  int32_t* dst;   // the free pages below U, in order
  int64_t num_blocks;
  int n_rows, max_blocks, segs;
  uint32_t* err;
};

__global__ void __launch_bounds__(PG_PLAN_THREADS) compact_count_kernel(const __grid_constant__ PgCompact a) {
  __shared__ int buf[33];
  const int64_t b0 = (int64_t)blockIdx.x * PG_SEG_PAGES, b1 = min64(b0 + PG_SEG_PAGES, a.num_blocks);
  int mine = 0;
  for (int64_t b = b0 + threadIdx.x; b < b1; b += blockDim.x) mine += a.refs[b] > 0;
  int total;
  pg_scan(mine, buf, total);
  if (threadIdx.x == 0) a.seg_used[blockIdx.x] = total;
}

__global__ void __launch_bounds__(PG_PLAN_THREADS) compact_plan_kernel(const __grid_constant__ PgCompact a) {
  __shared__ int buf[33];
  const int tid = threadIdx.x;
  // used pages in all, and in the segments before this CTA's (a single CTA
  // counts them itself)
  int before_ = 0, all_ = 0;
  if (a.segs == 1) {
    for (int64_t b = tid; b < a.num_blocks; b += blockDim.x) all_ += a.refs[b] > 0;
  } else {
    for (int s = tid; s < a.segs; s += blockDim.x) {
      const int v = a.seg_used[s];
      all_ += v;
      before_ += s < (int)blockIdx.x ? v : 0;
    }
  }
  int used, before;
  pg_scan(all_, buf, used);
  pg_scan(before_, buf, before);
  if (blockIdx.x == 0 && tid == 0) {
    a.head[0] = used;
    *a.used = used;
    if (used == a.num_blocks) a.head[1] = 0;
  }
  const int64_t b0 = (int64_t)blockIdx.x * PG_SEG_PAGES, b1 = min64(b0 + PG_SEG_PAGES, a.num_blocks);
  for (int64_t c0 = b0; c0 < b1; c0 += PG_SEG) {
    bool u[4];
    int mine = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t b = c0 + 4 * tid + k;
      u[k] = b < b1 && a.refs[b] > 0;
      mine += u[k];
    }
    int total, r = before + pg_scan(mine, buf, total);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t b = c0 + 4 * tid + k;
      if (b >= b1) break;
      a.rank[b] = u[k] ? r : -1 - r;
      if (b == used) a.head[1] = used - r;  // free pages below U: U less the used ones
      if (u[k] && b >= used) a.src[r] = (int32_t)b;
      if (!u[k] && b < used) a.dst[b - r] = (int32_t)b;
      r += u[k];
    }
    before += total;
  }
}

// New page of a page with rank r: itself below U, else the free page paired
// with it (the k-th used page from U on takes the k-th free page below U).
TQ_DEV int32_t pg_new_page(const PgCompact& a, int32_t e, int32_t r, int32_t used, int32_t moves) {
  if (r < 0) return -1;
  return e < used ? e : a.dst[r - (used - moves)];
}

__global__ void __launch_bounds__(PG_THREADS) compact_apply_kernel(const __grid_constant__ PgCompact a,
                                                                  const __grid_constant__ PgPools pools) {
  __shared__ PgShared s;
  pg_load_pools(s, pools);
  grid_dep_wait();
  const int32_t used = a.head[0], moves = a.head[1];
  const uint32_t units = s.unit0[pools.n];
  const int64_t all = (int64_t)units * moves, wstep = (int64_t)gridDim.x * (PG_THREADS / 32);
  for (int64_t w = (int64_t)blockIdx.x * (PG_THREADS / 32) + (threadIdx.x >> 5); w < all; w += wstep) {
    const int k = (int)(w / units);
    pg_move_unit(s, pools.n, (uint32_t)(w - (int64_t)k * units), a.src[used - moves + k], a.dst[k],
                 threadIdx.x & 31);
  }
  const int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t b = t; b < a.num_blocks; b += step) {
    const int32_t r = a.rank[b];
    a.remap[b] = pg_new_page(a, (int32_t)b, r, used, moves);
    // a free page below U takes its partner's count; the partner's is cleared
    // by the same thread, so calls in place need no second copy
    if (r >= 0) {
      if (b < used && a.refs_out != a.refs) a.refs_out[b] = a.refs[b];
    } else if (b < used) {
      const int32_t from = a.src[used - moves + (b - (-1 - r))];
      a.refs_out[b] = a.refs[from];
      a.refs_out[from] = 0;
    } else {
      a.refs_out[b] = 0;
    }
  }
  const int64_t n = (int64_t)a.n_rows * a.max_blocks;
  for (int64_t i = t; i < n; i += step) {
    const int32_t e = a.tables[i];
    int32_t out = -1;
    if (e >= a.num_blocks) record_error(a.err, TQ_DEVERR_BLOCK_RANGE);
    else if (e >= 0) out = pg_new_page(a, e, a.rank[e], used, moves);
    a.tables_out[i] = out;
  }
}

// Pools into the kernel parameters.
static PgPools make_pools(const tq_page_pool* pools, int n) {
  PgPools p{};
  p.n = n;
  for (int i = 0; i < n; ++i) {
    p.base[i] = static_cast<uint8_t*>(pools[i].base);
    p.bytes[i] = (uint32_t)pools[i].block_bytes;
    p.unit0[i + 1] = p.unit0[i] + (uint32_t)((pools[i].block_bytes + PG_UNIT - 1) / PG_UNIT);
  }
  return p;
}

inline size_t pg_align(size_t x) { return (x + 15) & ~(size_t)15; }

static int copy_ctas(int64_t ints, int sms) {
  return (int)std::min<int64_t>(4 * sms, (ints / 4 + PG_THREADS - 1) / PG_THREADS + 1);
}

}  // namespace tq

using namespace tq;

size_t tq_pages_fork_workspace_impl(int n) { return 4 * pg_align((size_t)n * 4); }

size_t tq_pages_compact_workspace_impl(int64_t num_blocks) {
  const size_t segs = (size_t)((num_blocks + PG_SEG_PAGES - 1) / PG_SEG_PAGES);
  return 16 + pg_align(segs * 4) + 3 * pg_align((size_t)num_blocks * 4);
}

tq_status tq_launch_pages_fork(const tq_page_pool* pools, int n_pools, int64_t num_blocks, const int32_t* tables,
                               int32_t* tables_out, const int32_t* lens, int32_t* lens_out, const int32_t* refs,
                               int32_t* refs_out, int n_rows, int max_blocks, const int32_t* parents,
                               const int32_t* children, int n, void* workspace, void* stream) {
  PgFork a{};
  a.tables = tables;
  a.tables_out = tables_out;
  a.lens = lens;
  a.lens_out = lens_out;
  a.refs = refs;
  a.refs_out = refs_out;
  a.parents = parents;
  a.children = children;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t part = pg_align((size_t)n * 4);
  a.state = reinterpret_cast<int32_t*>(ws);
  a.src = reinterpret_cast<int32_t*>(ws + part);
  a.dst = reinterpret_cast<int32_t*>(ws + 2 * part);
  a.fresh = reinterpret_cast<int32_t*>(ws + 3 * part);
  a.num_blocks = num_blocks;
  a.n_rows = n_rows;
  a.max_blocks = max_blocks;
  a.n = n;
  a.err = tq_error_word();
  int dev = 0;
  if (!a.err || cudaGetDevice(&dev) != cudaSuccess) return TQ_ERR_CUDA;
  const int sms = tq_sm_count(dev);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool copies = tables_out != tables || lens_out != lens || refs_out != refs;
  if (n == 0 && !copies) return TQ_OK;
  const int64_t ints = (int64_t)n_rows * max_blocks + num_blocks;
  const int plan_grid = 1 + (copies ? (int)std::min<int64_t>(sms, ints / PG_SEG + 1) : 0);
  const size_t smem = (size_t)((n_rows + 31) / 32) * 12;
  // (from 130 700 rows on, with the kernel's static part, above the 48 KB that need no leave)
  if (smem > 47 * 1024 && cudaFuncSetAttribute(fork_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               TQ_MAX_PAGE_ROWS / 32 * 12) != cudaSuccess)
    return TQ_ERR_CUDA;
  fork_plan_kernel<<<plan_grid, PG_PLAN_THREADS, smem, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return TQ_ERR_CUDA;
  if (n == 0) return TQ_OK;
  const PgPools p = make_pools(pools, n_pools);
  const int64_t warps = (int64_t)p.unit0[n_pools] * n;
  const int grid = (int)std::min<int64_t>(6 * sms, std::max<int64_t>(n, (warps + 7) / 8));
  if (tq_launch_pdl(fork_apply_kernel, dim3(grid), dim3(PG_THREADS), 0, st, a, p) != cudaSuccess)
    return TQ_ERR_CUDA;
  return TQ_OK;
}

tq_status tq_launch_pages_trim(const int32_t* tables, int32_t* tables_out, const int32_t* lens, int32_t* lens_out,
                               const int32_t* refs, int32_t* refs_out, int n_rows, int max_blocks,
                               int64_t num_blocks, int64_t window, int64_t sinks, const uint8_t* release,
                               void* stream) {
  PgTrim a{};
  a.tables = tables;
  a.tables_out = tables_out;
  a.lens = lens;
  a.lens_out = lens_out;
  a.refs = refs;
  a.refs_out = refs_out;
  a.release = release;
  a.num_blocks = num_blocks;
  a.window = window;
  a.sinks = sinks;
  a.n_rows = n_rows;
  a.max_blocks = max_blocks;
  a.err = tq_error_word();
  int dev = 0;
  if (!a.err || cudaGetDevice(&dev) != cudaSuccess) return TQ_ERR_CUDA;
  const int sms = tq_sm_count(dev);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (refs_out != refs) {
    trim_copy_kernel<<<copy_ctas(num_blocks, sms), PG_THREADS, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return TQ_ERR_CUDA;
  }
  const int64_t n = (int64_t)n_rows * max_blocks;
  const int grid = (int)std::min<int64_t>(8 * sms, (n + PG_THREADS - 1) / PG_THREADS);
  if (refs_out != refs) {
    if (tq_launch_pdl(trim_kernel, dim3(grid), dim3(PG_THREADS), 0, st, a) != cudaSuccess) return TQ_ERR_CUDA;
  } else {
    trim_kernel<<<grid, PG_THREADS, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return TQ_ERR_CUDA;
  }
  return TQ_OK;
}

tq_status tq_launch_pages_compact(const tq_page_pool* pools, int n_pools, int64_t num_blocks, const int32_t* tables,
                                  int32_t* tables_out, const int32_t* refs, int32_t* refs_out, int n_rows,
                                  int max_blocks, int32_t* remap, int32_t* used, void* workspace, void* stream) {
  PgCompact a{};
  a.tables = tables;
  a.tables_out = tables_out;
  a.refs = refs;
  a.refs_out = refs_out;
  a.remap = remap;
  a.used = used;
  a.num_blocks = num_blocks;
  a.n_rows = n_rows;
  a.max_blocks = max_blocks;
  a.segs = (int)((num_blocks + PG_SEG_PAGES - 1) / PG_SEG_PAGES);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t part = pg_align((size_t)num_blocks * 4);
  a.head = reinterpret_cast<int32_t*>(ws);
  a.seg_used = reinterpret_cast<int32_t*>(ws + 16);
  a.rank = reinterpret_cast<int32_t*>(ws + 16 + pg_align((size_t)a.segs * 4));
  a.src = a.rank + part / 4;
  a.dst = a.src + part / 4;
  a.err = tq_error_word();
  int dev = 0;
  if (!a.err || cudaGetDevice(&dev) != cudaSuccess) return TQ_ERR_CUDA;
  const int sms = tq_sm_count(dev);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.segs > 1) {
    compact_count_kernel<<<a.segs, PG_PLAN_THREADS, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return TQ_ERR_CUDA;
  }
  compact_plan_kernel<<<a.segs, PG_PLAN_THREADS, 0, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return TQ_ERR_CUDA;
  const PgPools p = make_pools(pools, n_pools);
  const int64_t most = (int64_t)p.unit0[n_pools] * (num_blocks / 2) / (PG_THREADS / 32);
  const int64_t ints = ((int64_t)n_rows * max_blocks + num_blocks) / PG_THREADS;
  const int grid = (int)std::min<int64_t>(6 * sms, std::max(most, ints) + 1);
  if (tq_launch_pdl(compact_apply_kernel, dim3(grid), dim3(PG_THREADS), 0, st, a, p) != cudaSuccess)
    return TQ_ERR_CUDA;
  return TQ_OK;
}
