// Pages of a cache: given out, taken back, shared between requests and moved up
// (moe_pages_resize, moe_pages_fork, moe_pages_compact).
//
// State: refs[p], how many page-table entries hold page p (0: free), the page
// table and the requests' lengths, all on the device.  The r-th page that a call
// takes is the r-th free page from the lowest number, and requests are served in
// order, so the outcome is a function of the state alone: what runs in any order
// are additions to refs, and a release before the search makes pages free whatever
// the order.
//
// A call's bookkeeping is one CTA: a prefix sum over the requests' needs, then a
// walk over refs from page 0 until as many free pages are found as are needed.  It
// is bound by latency (a few dependent reads of the tables).  The pages to copy
// (each is rare in a resize, one a child in a fork) go to a list that the rest of the
// CTA's cluster works off, or a second launch over all SMs, bound by the bytes: its grid is
// fixed, as the list's length is known on the device only.
#include <limits.h>
#include <string.h>

#include "epilogue.cuh"
#include "kv4.cuh"
#include "moe.h"

namespace moe {
namespace {

constexpr int kBookThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyChunk = kCopyThreads * 8 * 16;  // bytes a CTA copies at a time
constexpr int kCompactThreads = 128;
constexpr int kCopyCluster = 8;
constexpr long long kFewBytes = 4ll << 20;

struct BookParams {
  int32_t* refs;
  int n_pages;
  int32_t* table;
  int B, width, page, page_log2;
  int32_t* len;
  const int32_t* new_len;      // resize
  const int32_t *src, *dst;    // fork
  int n;                       // fork: pairs
  int32_t* status;
  // workspace
  int32_t* count;              // copies
  int2* copies;                // (from, to)
  int4* state;                 // of a request: (first new page's rank, what it does, old and new length);
                               // of a pair: (rank, length)
  int32_t* claim;              // fork: the lowest pair that names a request as its child
  int32_t* list;               // free pages in order
};

struct PoolArg {
  uint8_t* data;
  long long page_bytes;
  int format, heads, head_dim;
  int row_chunks;              // rows: 16-byte chunks of a slot
};
struct CopyParams {
  PoolArg pool[MOE_MAX_POOLS];
  int chunk0[MOE_MAX_POOLS + 1];  // first chunk of a page's copy in each pool
  int n_pools;
  const int32_t* count;
  const int2* copies;
};
struct CompactParams {
  PoolArg pool[MOE_MAX_POOLS];
  int n_pools, n_pages, B, n, width, page, page_log2;
  const int32_t *table, *base, *keep;
  int32_t* new_len;
  int32_t* status;
};

__device__ __forceinline__ void record_pool(int32_t* status) {
  if (atomicCAS(status, 0, kStatusPool) == 0) atomicExch(status + 1, kInfoPool);
}

// What requests need can pass 32 bits in all (65536 of them, 2^25 pages each); how many there
// are cannot (n_pages < 2^28).  Sums stop at a number above that: a request at or past it is
// refused, whatever it would be.
constexpr int kManyPages = 1 << 29;
__device__ __forceinline__ int add_pages(int a, int b) { return min(a + b, kManyPages); }

// Exclusive prefix sum over the CTA; `total` gets the sum of all.
__device__ int block_scan(int v, int& total) {
  __shared__ int sums[kBookThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc = add_pages(inc, u);
  }
  if (lane == 31) sums[warp] = inc;
  const int left = __shfl_up_sync(0xffffffffu, inc, 1);
  __syncthreads();
  if (warp == 0) {
    int s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s = add_pages(s, u);
    }
    sums[lane] = s;
  }
  __syncthreads();
  const int before = warp > 0 ? sums[warp - 1] : 0;
  total = sums[kBookThreads / 32 - 1];
  __syncthreads();
  return add_pages(before, lane > 0 ? left : 0);
}

// The lowest `need` free pages in order, to p.list; -> how many there are of them.
__device__ int find_free(const BookParams& p, int need) {
  int found = 0;
  for (int base = 0; base < p.n_pages && found < need; base += 4 * kBookThreads) {
    const int at = base + 4 * threadIdx.x;
    int v[4];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = at + i < p.n_pages ? __ldcg(p.refs + at + i) : 1;
      mine += v[i] == 0;
    }
    int total;
    int rank = found + block_scan(mine, total);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (v[i] == 0) {
        if (rank < need) p.list[rank] = at + i;
        ++rank;
      }
    found += total;
  }
  __syncthreads();
  return min(found, need);
}

// Threads that share a request: all of the CTA for one, a warp each for 32 or more.
__device__ __forceinline__ int threads_each(int items) {
  int t = kBookThreads;
  while (t > 32 && kBookThreads / t < items) t >>= 1;
  return t;
}

enum : int { kSkip = -1, kPlain = 0, kSplit = 1 };

__device__ void resize_book(const BookParams& p) {
  __shared__ int n_copies;
  const int tid = threadIdx.x, each = threads_each(p.B), sub = tid % each, groups = kBookThreads / each;
  const int cap = p.width << p.page_log2;
  if (tid == 0) n_copies = 0;
  // pages past the new length go back
  for (int b = tid / each; b < p.B; b += groups) {
    const int old = p.len[b], now = p.new_len[b];
    if (old < 0 || old > cap || now < 0 || now > cap) {
      if (sub == 0) record_index(p.status, kInfoLength);
      continue;
    }
    const int has = (old + p.page - 1) >> p.page_log2, want = (now + p.page - 1) >> p.page_log2;
    int32_t* row = p.table + static_cast<long long>(b) * p.width;
    for (int c = want + sub; c < has; c += each) {
      const int pg = row[c];
      row[c] = -1;
      if (static_cast<uint32_t>(pg) >= static_cast<uint32_t>(p.n_pages)) {
        record_index(p.status, kInfoPage);
      } else if (atomicSub(p.refs + pg, 1) <= 0) {  // held by no one: left so
        atomicAdd(p.refs + pg, 1);
        record_index(p.status, kInfoPage);
      }
    }
  }
  __syncthreads();
  // what each request needs: pages past its old length, and one in the place of a
  // page that goes on being written while another request holds it too
  int need = 0;
  for (int b0 = 0; b0 < p.B; b0 += kBookThreads) {
    const int b = b0 + tid;
    int mine = 0, what = kSkip, old = 0, now = 0;
    if (b < p.B) {
      old = p.len[b];
      now = p.new_len[b];
      if (old >= 0 && old <= cap && now >= 0 && now <= cap) {
        const int has = (old + p.page - 1) >> p.page_log2, want = (now + p.page - 1) >> p.page_log2;
        const int stay = min(old, now);
        what = kPlain;
        mine = max(0, want - has);
        if (stay & (p.page - 1)) {
          const int last = p.table[static_cast<long long>(b) * p.width + (stay >> p.page_log2)];
          if (static_cast<uint32_t>(last) >= static_cast<uint32_t>(p.n_pages)) {
            record_index(p.status, kInfoPage);
          } else if (__ldcg(p.refs + last) > 1) {
            what = kSplit;
            ++mine;
          }
        }
      }
    }
    int total;
    const int first = need + block_scan(mine, total);
    if (b < p.B) p.state[b] = make_int4(first, what, old, now);
    need = add_pages(need, total);
  }
  __syncthreads();
  const int found = need > 0 ? find_free(p, need) : 0;
  for (int b = tid / each; b < p.B; b += groups) {
    const int4 s = p.state[b];
    if (s.y == kSkip) continue;
    const int old = s.z, now = s.w, stay = min(old, now);
    const int has = (old + p.page - 1) >> p.page_log2, want = (now + p.page - 1) >> p.page_log2;
    const int more = max(0, want - has), split = s.y == kSplit, takes = more + split;
    const bool ok = takes == 0 || s.x + takes <= found;
    int32_t* row = p.table + static_cast<long long>(b) * p.width;
    if (ok && takes > 0) {
      for (int i = sub; i < more; i += each) {
        const int pg = p.list[s.x + split + i];
        p.refs[pg] = 1;
        row[has + i] = pg;
      }
      if (split && sub == 0) {
        const int at = stay >> p.page_log2, last = row[at], pg = p.list[s.x];
        p.refs[pg] = 1;
        row[at] = pg;
        atomicSub(p.refs + last, 1);
        p.copies[atomicAdd(&n_copies, 1)] = make_int2(last, pg);
      }
    }
    if (sub == 0) {
      if (!ok) record_pool(p.status);
      p.len[b] = ok ? now : stay;
    }
  }
  __syncthreads();
  if (tid == 0) *p.count = n_copies;
}

__device__ void fork_book(const BookParams& p) {
  __shared__ int n_copies;
  const int tid = threadIdx.x, each = threads_each(p.n), sub = tid % each, groups = kBookThreads / each;
  const int cap = p.width << p.page_log2;
  if (tid == 0) n_copies = 0;
  // a request that several pairs name as their child is the first one's
  for (int i = tid; i < p.n; i += kBookThreads)
    if (static_cast<uint32_t>(p.dst[i]) < static_cast<uint32_t>(p.B)) p.claim[p.dst[i]] = INT_MAX;
  __syncthreads();
  for (int i = tid; i < p.n; i += kBookThreads)
    if (p.src[i] >= 0 && static_cast<uint32_t>(p.dst[i]) < static_cast<uint32_t>(p.B)) atomicMin(p.claim + p.dst[i], i);
  __syncthreads();
  int need = 0;
  for (int i0 = 0; i0 < p.n; i0 += kBookThreads) {
    const int i = i0 + tid;
    int mine = 0, length = -1;  // -1: not made
    if (i < p.n && p.src[i] >= 0 && p.dst[i] >= 0) {
      const int from = p.src[i], to = p.dst[i];
      if (from < p.B && to < p.B && __ldcg(p.claim + to) == i && p.len[to] == 0) {
        length = p.len[from];
        if (length < 0 || length > cap) {
          record_index(p.status, kInfoLength);
          length = -1;
        }
      } else {
        record_index(p.status, kInfoFork);
      }
      mine = length > 0 && (length & (p.page - 1)) ? 1 : 0;
    }
    int total;
    const int first = need + block_scan(mine, total);
    if (i < p.n) p.state[i] = make_int4(first, length, 0, 0);
    need += total;
  }
  __syncthreads();
  const int found = need > 0 ? find_free(p, need) : 0;
  for (int i = tid / each; i < p.n; i += groups) {
    const int4 s = p.state[i];
    if (s.y < 0) continue;
    const int whole = s.y >> p.page_log2;
    const bool tail = (s.y & (p.page - 1)) != 0, ok = !tail || s.x < found;
    if (!ok) {
      if (sub == 0) record_pool(p.status);
      continue;
    }
    const int32_t* from = p.table + static_cast<long long>(p.src[i]) * p.width;
    int32_t* to = p.table + static_cast<long long>(p.dst[i]) * p.width;
    for (int c = sub; c < whole; c += each) {
      const int pg = from[c];
      to[c] = pg;
      if (static_cast<uint32_t>(pg) < static_cast<uint32_t>(p.n_pages)) atomicAdd(p.refs + pg, 1);
      else record_index(p.status, kInfoPage);
    }
    if (sub == 0) {
      if (tail) {
        const int last = from[whole], pg = p.list[s.x];
        p.refs[pg] = 1;
        to[whole] = pg;
        if (static_cast<uint32_t>(last) < static_cast<uint32_t>(p.n_pages))
          p.copies[atomicAdd(&n_copies, 1)] = make_int2(last, pg);
        else
          record_index(p.status, kInfoPage);
      }
      p.len[p.dst[i]] = s.y;
    }
  }
  __syncthreads();
  if (tid == 0) *p.count = n_copies;
}

// The listed pages' bytes in every pool: chunks first, first + step, .. by kCopyThreads
// threads, of which this is the tid-th.
__device__ __forceinline__ void copy_pages(const CopyParams& p, int first, int step, int tid) {
  const int per = p.chunk0[p.n_pools];
  const long long units = static_cast<long long>(__ldcg(p.count)) * per;
  for (long long u = first; u < units; u += step) {
    const int2 c = __ldcg(p.copies + u / per);
    const int chunk = static_cast<int>(u % per);
    int k = 0;
    while (chunk >= p.chunk0[k + 1]) ++k;
    const long long bytes = p.pool[k].page_bytes, at = static_cast<long long>(chunk - p.chunk0[k]) * kCopyChunk;
    const uint8_t* src = p.pool[k].data + c.x * bytes + at;
    uint8_t* dst = p.pool[k].data + c.y * bytes + at;
    const int left = static_cast<int>(min(static_cast<long long>(kCopyChunk), bytes - at));
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int o = (i * kCopyThreads + tid) * 16;
      if (o < left) v[i] = __ldcs(reinterpret_cast<const uint4*>(src + o));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int o = (i * kCopyThreads + tid) * 16;
      if (o < left) __stcs(reinterpret_cast<uint4*>(dst + o), v[i]);
    }
  }
}
// Over all SMs.  128 requests forked (330 MB read and written): 68.5 us with the bookkeeping,
// 4.8 TB/s; with four loads a thread under way instead of eight 4 us more, without the
// streaming hints one.
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ CopyParams p) {
  griddep_wait();
  copy_pages(p, blockIdx.x, gridDim.x, threadIdx.x);
}

// The bookkeeping alone (a CTA), or with its copies (a cluster, which does them once its
// first CTA has listed them: one launch in place of two, but the copies on 8 SMs).  A
// resize copies only what goes on being written while another request shares it, mostly
// nothing: 8 requests in 5 pools take 4.1 us like this and 5.4 with two launches; if all of
// them copy a page (2.8 MB), 13.6 and 7.2.  So it is taken where no more than kFewBytes can
// have to be copied; a fork, which always copies, has two launches.  By the bytes that a call
// may have to copy (one launch with none of them copied and with all; two launches): 0.7 MB
// 3.8 and 7.4 to 8.7 us, 5.4 and 6.6; 5.6 MB 3.8 and 21, 5.5 and 7.3; 11 MB 4.1 and 34, 5.4 and
// 8.6; 45 MB 4.6 and 120, 5.9 and 17.  At the line a call that copies everything loses what
// some six that copy nothing win.
template <bool kFork, bool kCopies>
__global__ void __launch_bounds__(kBookThreads) pages_book_kernel(const __grid_constant__ BookParams b, const __grid_constant__ CopyParams c) {
  griddep_wait();
  if (!kCopies || cluster_rank() == 0) {
    if (kFork) fork_book(b);
    else resize_book(b);
  }
  if (kCopies) {
    constexpr int kTeams = kBookThreads / kCopyThreads;
    cluster_sync();
    copy_pages(c, static_cast<int>(cluster_rank()) * kTeams + threadIdx.x / kCopyThreads, kCopyCluster * kTeams,
               threadIdx.x % kCopyThreads);
  }
}

// Moves rows from[j] -> to[j], j < count, in order: `size` bytes at the same place
// of each.  The lists' offsets grow and from[j] lies behind to[j], so no row is
// written before it is read: four are under way at a time.
template <typename T, typename Place>
__device__ __forceinline__ void move_rows(const int2* rows, int count, const Place& place) {
  for (int j0 = 0; j0 < count; j0 += 4) {
    T v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j0 + i < count && rows[j0 + i].x != rows[j0 + i].y) v[i] = *reinterpret_cast<const T*>(place(rows[j0 + i].x));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j0 + i < count && rows[j0 + i].x != rows[j0 + i].y) *reinterpret_cast<T*>(place(rows[j0 + i].y)) = v[i];
  }
}

// A CTA: one request in one pool.
__global__ void __launch_bounds__(kCompactThreads) pages_compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ int2 rows[MOE_MAX_BLOCK];  // (from, to) slots
  __shared__ int count;
  griddep_wait();
  const int b = blockIdx.x, k = blockIdx.y, tid = threadIdx.x;
  const int base = p.base[b], cap = p.width << p.page_log2;
  const int32_t* keep = p.keep + static_cast<long long>(b) * p.n;
  const int32_t* row = p.table + static_cast<long long>(b) * p.width;
  const bool placed = base >= 0 && base <= cap;
  if (tid == 0) {
    count = placed ? p.n : 0;
    if (!placed) record_index(p.status, kInfoLength);
  }
  __syncthreads();
  if (placed)
    for (int j = tid; j < p.n; j += kCompactThreads)
      if (keep[j] < 0) atomicMin(&count, j);
  __syncthreads();
  const int listed = count;
  __syncthreads();
  for (int j = tid; j < listed; j += kCompactThreads) {
    const int o = keep[j], before = j > 0 ? keep[j - 1] : -1;
    // offsets grow and lie in the table, as do the rows that they go to: an entry behind one
    // out of order is looked at too, and with o >= j (true of every list that grows) its
    // place base + j <= base + o lies in the table as well
    bool bad = o <= before || o < j || o >= cap - base;
    if (!bad) {
      const int from = row[(base + o) >> p.page_log2], to = row[(base + j) >> p.page_log2];
      bad = static_cast<uint32_t>(from) >= static_cast<uint32_t>(p.n_pages) ||
            static_cast<uint32_t>(to) >= static_cast<uint32_t>(p.n_pages);
      if (!bad)
        rows[j] = make_int2((from << p.page_log2) + ((base + o) & (p.page - 1)),
                            (to << p.page_log2) + ((base + j) & (p.page - 1)));
    }
    if (bad) {
      record_index(p.status, kInfoKeep);
      atomicMin(&count, j);
    }
  }
  __syncthreads();
  const int n = count;
  if (k == 0 && tid == 0 && p.new_len) p.new_len[b] = max(0, min(base, cap)) + n;
  if (p.n_pools == 0) return;
  const PoolArg& pool = p.pool[k];
  const int mask = p.page - 1, log2 = p.page_log2;
  if (pool.format == MOE_POOL_ROWS) {
    for (int c = tid; c < pool.row_chunks; c += kCompactThreads)
      move_rows<uint4>(rows, n, [&](int slot) {
        return pool.data + (static_cast<long long>(slot) * pool.row_chunks + c) * 16;
      });
  } else {
    const int D = pool.head_dim, groups = D / 32, codes = 2 * groups * pool.heads;
    const int block = p.page * kv4_slot_bytes(D);
    for (int c = tid; c < codes; c += kCompactThreads)
      move_rows<uint4>(rows, n, [&](int slot) {
        return pool.data + (static_cast<long long>(slot >> log2) * pool.heads + c / (2 * groups)) * block +
               (c % (2 * groups)) * p.page * 16 + (slot & mask) * 16;
      });
    for (int c = tid; c < 2 * pool.heads; c += kCompactThreads) {
      const auto place = [&](int slot) {
        return pool.data + (static_cast<long long>(slot >> log2) * pool.heads + c / 2) * block +
               kv4_scales_at(D, p.page, c % 2) + (slot & mask) * groups;
      };
      if (groups == 4) move_rows<uint32_t>(rows, n, place);
      else move_rows<uint16_t>(rows, n, place);
    }
  }
}

struct PagesLayout {
  size_t o_copies, o_state, o_claim, o_list, total;
};
PagesLayout pages_layout(int B, int n_pages) {
  PagesLayout L;
  size_t o = kWsHeaderBytes + kWsAlign;  // the count of copies comes first
  L.o_copies = o; o += ws_align_up(8 * static_cast<size_t>(B));
  L.o_state = o; o += ws_align_up(16 * static_cast<size_t>(B));
  L.o_claim = o; o += ws_align_up(4 * static_cast<size_t>(B));
  L.o_list = o; o += ws_align_up(4 * static_cast<size_t>(n_pages));
  L.total = o;
  return L;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

moe_status check_sizes(int n_pages, int B, int width, int page) {
  if (n_pages < 0 || B < 0 || width < 0 || page < 1) return MOE_ERR_INVALID_ARG;
  if (page < 8 || page > 1024 || (page & (page - 1)) != 0 || B > MOE_MAX_REQUESTS ||
      static_cast<long long>(width) * page > MOE_MAX_KEYS || static_cast<long long>(n_pages) * page > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The pools as the kernels take them; each shares no byte with another or with
// what else the call reads and writes.
moe_status check_pools(const moe_page_pool* pools, int n_pools, int n_pages, int page, PoolArg* out,
                       const RowSet* others, int n_others) {
  if (n_pools < 0 || (n_pools > 0 && !pools)) return MOE_ERR_INVALID_ARG;
  if (n_pools > MOE_MAX_POOLS) return MOE_ERR_UNSUPPORTED;
  RowSet sets[MOE_MAX_POOLS];
  for (int i = 0; i < n_pools; ++i) {
    const moe_page_pool& a = pools[i];
    PoolArg& o = out[i];
    o.data = static_cast<uint8_t*>(a.data);
    o.format = a.format;
    o.heads = a.heads;
    o.head_dim = a.head_dim;
    o.row_chunks = 0;
    if (a.format == MOE_POOL_ROWS) {
      if (a.row_bytes < 1) return MOE_ERR_INVALID_ARG;
      if (a.row_bytes % 16 || a.row_bytes > (1 << 24)) return MOE_ERR_UNSUPPORTED;
      o.row_chunks = static_cast<int>(a.row_bytes / 16);
      o.page_bytes = a.row_bytes * page;
    } else if (a.format == MOE_POOL_KV4) {
      if (a.heads < 1) return MOE_ERR_INVALID_ARG;
      if ((a.head_dim != 64 && a.head_dim != 128) || a.heads > 1024) return MOE_ERR_UNSUPPORTED;
      o.page_bytes = static_cast<long long>(a.heads) * page * kv4_slot_bytes(a.head_dim);
    } else {
      return MOE_ERR_INVALID_ARG;
    }
    if (n_pages > 0 && !a.data) return MOE_ERR_INVALID_ARG;
    if (!aligned16(a.data)) return MOE_ERR_INVALID_ARG;
    sets[i] = {a.data, 1, o.page_bytes * n_pages, 0};
    for (int j = 0; j < i; ++j)
      if (rows_meet(sets[i], sets[j])) return MOE_ERR_INVALID_ARG;
    for (int j = 0; j < n_others; ++j)
      if (rows_meet(sets[i], others[j])) return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

template <typename... P>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, int cluster, cudaStream_t s, const P&... p) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p...);
}

// One kind of bookkeeping and the copies that it lists.
template <bool kFork>
moe_status run_book(BookParams& b, const moe_page_pool* pools, int n_pools,
                    const RowSet* sets, int n_sets, void* ws, size_t ws_bytes, cudaStream_t stream) {
  for (int i = 0; i < n_sets; ++i)
    for (int j = 0; j < i; ++j)
      if (rows_meet(sets[i], sets[j])) return MOE_ERR_INVALID_ARG;
  CopyParams c;
  memset(&c, 0, sizeof(c));
  const moe_status st = check_pools(pools, n_pools, b.n_pages, b.page, c.pool, sets, n_sets);
  if (st != MOE_OK) return st;
  const PagesLayout L = pages_layout(b.B, b.n_pages);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kWsAlign) != 0 || ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  while ((1 << b.page_log2) < b.page) ++b.page_log2;
  char* w = static_cast<char*>(ws);
  b.status = reinterpret_cast<int32_t*>(w);
  b.count = reinterpret_cast<int32_t*>(w + kWsHeaderBytes);
  b.copies = reinterpret_cast<int2*>(w + L.o_copies);
  b.state = reinterpret_cast<int4*>(w + L.o_state);
  b.claim = reinterpret_cast<int32_t*>(w + L.o_claim);
  b.list = reinterpret_cast<int32_t*>(w + L.o_list);
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  c.n_pools = n_pools;
  long long most = 0;  // bytes that a resize may have to copy
  for (int i = 0; i < n_pools; ++i) {
    const long long chunks = (c.pool[i].page_bytes + kCopyChunk - 1) / kCopyChunk;
    c.chunk0[i + 1] = c.chunk0[i] + static_cast<int>(chunks);
    most += c.pool[i].page_bytes * b.B;
  }
  c.count = b.count;
  c.copies = b.copies;
  if (!kFork && n_pools > 0 && most <= kFewBytes)
    return launch(pages_book_kernel<false, true>, dim3(kCopyCluster), kBookThreads, kCopyCluster, stream, b, c) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  if (launch(pages_book_kernel<kFork, false>, dim3(1), kBookThreads, 1, stream, b, c) != cudaSuccess) return MOE_ERR_CUDA;
  if (n_pools == 0) return MOE_OK;
  return launch(pages_copy_kernel, dim3(8 * sms), kCopyThreads, 1, stream, c) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_pages_workspace_bytes(int B, int n_pages) {
  using namespace moe;
  if (B < 0 || n_pages < 0 || B > MOE_MAX_REQUESTS) return 0;
  return pages_layout(B, n_pages).total;
}

moe_status moe_pages_resize(int32_t* refs, int n_pages, int32_t* page_table, int B, int table_width, int page_size,
                            int32_t* own_len, const int32_t* new_len, const moe_page_pool* pools, int n_pools,
                            void* ws, size_t ws_bytes, cudaStream_t stream) {
  using namespace moe;
  const moe_status st = check_sizes(n_pages, B, table_width, page_size);
  if (st != MOE_OK) return st;
  if (B == 0) return MOE_OK;
  if (!own_len || !new_len || (n_pages > 0 && !refs) || (table_width > 0 && !page_table)) return MOE_ERR_INVALID_ARG;
  BookParams b;
  memset(&b, 0, sizeof(b));
  b.refs = refs; b.n_pages = n_pages; b.table = page_table; b.B = B; b.width = table_width; b.page = page_size;
  b.len = own_len; b.new_len = new_len;
  const RowSet sets[] = {{refs, 1, 4ll * n_pages, 0}, {page_table, 1, 4ll * B * table_width, 0},
                         {own_len, 1, 4ll * B, 0}, {new_len, 1, 4ll * B, 0}};
  return run_book<false>(b, pools, n_pools, sets, 4, ws, ws_bytes, stream);
}

moe_status moe_pages_fork(int32_t* refs, int n_pages, int32_t* page_table, int B, int table_width, int page_size,
                          int32_t* own_len, const int32_t* src, const int32_t* dst, int n, const moe_page_pool* pools,
                          int n_pools, void* ws, size_t ws_bytes, cudaStream_t stream) {
  using namespace moe;
  if (n < 0) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_sizes(n_pages, B, table_width, page_size);
  if (st != MOE_OK) return st;
  if (n > B) return MOE_ERR_INVALID_ARG;  // children are distinct
  if (n == 0) return MOE_OK;
  if (!own_len || !src || !dst || (n_pages > 0 && !refs) || (table_width > 0 && !page_table))
    return MOE_ERR_INVALID_ARG;
  BookParams b;
  memset(&b, 0, sizeof(b));
  b.refs = refs; b.n_pages = n_pages; b.table = page_table; b.B = B; b.width = table_width; b.page = page_size;
  b.len = own_len; b.src = src; b.dst = dst; b.n = n;
  const RowSet sets[] = {{refs, 1, 4ll * n_pages, 0}, {page_table, 1, 4ll * B * table_width, 0},
                         {own_len, 1, 4ll * B, 0}, {src, 1, 4ll * n, 0}, {dst, 1, 4ll * n, 0}};
  return run_book<true>(b, pools, n_pools, sets, 5, ws, ws_bytes, stream);
}

moe_status moe_pages_compact(const int32_t* page_table, int n_pages, int B, int table_width, int page_size,
                             const int32_t* base, const int32_t* keep, int n, const moe_page_pool* pools, int n_pools,
                             int32_t* new_len, void* ws, size_t ws_bytes, cudaStream_t stream) {
  using namespace moe;
  if (n < 0) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_sizes(n_pages, B, table_width, page_size);
  if (st != MOE_OK) return st;
  if (n > MOE_MAX_BLOCK) return MOE_ERR_UNSUPPORTED;
  if (B == 0) return MOE_OK;
  if (!base || (n > 0 && !keep) || (table_width > 0 && !page_table)) return MOE_ERR_INVALID_ARG;
  CompactParams p;
  memset(&p, 0, sizeof(p));
  const RowSet sets[] = {{page_table, 1, 4ll * B * table_width, 0}, {base, 1, 4ll * B, 0}, {keep, 1, 4ll * B * n, 0},
                         {new_len, 1, 4ll * B, 0}};
  for (int i = 0; i < 3; ++i)
    if (rows_meet(sets[i], sets[3])) return MOE_ERR_INVALID_ARG;
  const moe_status pst = check_pools(pools, n_pools, n_pages, page_size, p.pool, sets, 4);
  if (pst != MOE_OK) return pst;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kWsAlign) != 0 || ws_bytes < MOE_STATUS_BYTES)
    return MOE_ERR_WORKSPACE;
  p.n_pools = n_pools; p.n_pages = n_pages; p.B = B; p.n = n; p.width = table_width; p.page = page_size;
  while ((1 << p.page_log2) < page_size) ++p.page_log2;
  p.table = page_table; p.base = base; p.keep = keep; p.new_len = new_len;
  p.status = static_cast<int32_t*>(ws);
  const dim3 grid(B, n_pools > 0 ? n_pools : 1);
  return launch(pages_compact_kernel, grid, kCompactThreads, 1, stream, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
