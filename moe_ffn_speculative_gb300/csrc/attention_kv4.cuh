// The attention over a 4-bit cache: what its kernels share.  The list of work, its cut
// into the CTAs' shares, the walk through a share, and the parts that it leaves.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include "kv4.cuh"
#include "moe_internal.cuh"

namespace moe {

constexpr int kTile = 128;       // keys of a unit of work
constexpr int kRows = 64;        // most rows of a row tile
// An item's fixed cost in units: queries, the first reference, its parts.  (8 blocks of 9 over
// 4096 keys and their own: 41.6 us with 0, 35.0 with 2, 32.4 with 4, 35.3 with 8; 16 single
// tokens over as many: 34.9, 32.8, 28.8 and 28.2.)
constexpr int kItemCost = 4;
// What the row's maximum counts when the reference is set, and how far a later score may
// pass that (powers of two): the largest power is 2^14, a key is held to within 2^-32 of
// the row's largest.
constexpr float kLift = 7.f, kRescaleAt = 7.f;

struct Kv4Attn {
  int T, B, Hq, Hkv, G, tpt;     // tpt: tokens of a row tile
  int n_pages, page, page_log2;
  const uint16_t* q;
  long long q_stride;
  const uint8_t* cache;
  const int32_t *q_start, *prefix_pages, *prefix_len, *page_table, *own_len;
  int prefix_cap, table_width, causal;
  float scale_log2;
  int ctas;
  uint16_t* out;
  float* lse;
  // workspace
  int32_t* status;
  struct Plan* plan;
  struct RequestPlan* requests;  // [T] of every token
  float2* ml;                    // (reference, sum) of every part row
  float* o;                      // its fp32 elements
};

// A list of units cut into equal shares: share w holds [start(w), start(w + 1)), the
// first `rest` shares one more than the others.  (Counted in 32 bits: the entry point
// refuses work that could exceed them.)
struct Shares {
  uint32_t each, rest;
  __device__ uint32_t start(uint32_t w) const { return w * each + (w < rest ? w : rest); }
  __device__ uint32_t of(uint32_t u) const {
    const uint32_t v = rest * (each + 1);
    return u < v ? u / (each + 1) : rest + (u - v) / each;
  }
};
struct Plan {
  uint32_t per_head;  // units of one head's list
  int prefix_tiles;
  Shares s;
};
// A token's request as kv4_merge_kernel reads it.
struct __align__(16) RequestPlan {
  int a, n, len;        // first token, tokens, own keys
  uint32_t first_unit;  // units of a head's list before it
};

__host__ __device__ inline int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }
__host__ __device__ inline int units_of(int tiles) { return tiles > 0 ? tiles + kItemCost : 0; }

// A length read on the device, held within its page table.
__device__ __forceinline__ int held(int len, int pages, int page, int32_t* status) {
  if (len >= 0 && len <= pages * page) return len;
  record_index(status, kInfoLength);
  return len < 0 ? 0 : pages * page;
}

struct Request {
  int a, n, len;  // first token, tokens, own keys
  bool ok;        // its starts are in order
  // keys seen by the last token of row tile rt
  __device__ int seen(const Kv4Attn& p, int rt) const {
    if (!p.causal) return len;
    return max(0, min(len, len - n + min(n, (rt + 1) * p.tpt)));
  }
  __device__ int row_tiles(const Kv4Attn& p) const { return (n + p.tpt - 1) / p.tpt; }
  __device__ uint32_t units(const Kv4Attn& p) const {
    const int k = row_tiles(p);
    if (!p.causal) return static_cast<uint32_t>(k) * units_of(tiles_of(len));
    uint32_t u = 0;
    for (int rt = 0; rt < k; ++rt) u += units_of(tiles_of(seen(p, rt)));
    return u;
  }
};
static __device__ __noinline__ Request read_request(const Kv4Attn& p, int b) {
  Request r;
  r.a = __ldg(p.q_start + b);
  const int z = __ldg(p.q_start + b + 1);
  r.n = z - r.a;
  r.len = p.table_width > 0 ? held(__ldg(p.own_len + b), p.table_width, p.page, p.status) : 0;
  r.ok = r.a >= 0 && z >= r.a && z <= p.T;
  if (!r.ok) {
    record_index(p.status, kInfoStarts);
    r.a = r.n = 0;
  }
  return r;
}

// One share's run through one item: a row tile against key tiles [j0, j1).
struct Segment {
  int live;             // 0: the list has ended
  int h, tok0, toks;    // key head; tokens of the row tile
  int keys;             // keys that any of its rows sees
  int own, lim0;        // causal own keys: token t sees min(keys, max(0, lim0 + t)) of them
  int least;            // keys that every row sees
  int j0, j1;
  const int32_t* pages;
  long long part_row;   // part row of token tok0, head h * G
};

// Part rows: every head's prefix rows, then its own rows, and a row tile more for every
// share before: two parts never meet, as a share's last and the next one's first may
// belong to one item, which has no more rows than that.
__device__ __forceinline__ long long part_row(const Kv4Attn& p, int h, int t, bool own, int share) {
  return (static_cast<long long>(h) * 2 * p.T + (own ? p.T : 0) + t) * p.G + static_cast<long long>(kRows) * share;
}

// Where a CTA's share begins, as find_share leaves it in shared memory.
struct Start {
  uint32_t sums[32];
  unsigned long long claimed;
  uint32_t units;
  int head, request, skip, batch;
};

// The share's segments in order.
struct Walker {
  int share;
  uint32_t left;  // units still to walk
  int off;        // units of the current item before the share
  int h, i, rt;   // i: request, or -1 for the prefix; rt: row tile
  int batch, prefix_len, prefix_items;
  Request rq;

  __device__ __forceinline__ void begin(const Kv4Attn& p, const Start& c, int plen) {
    share = blockIdx.x;
    left = c.units;
    h = c.head;
    i = c.request;
    batch = c.batch;
    prefix_len = plen;
    prefix_items = plen > 0 ? (p.T + p.tpt - 1) / p.tpt : 0;
    rt = 0;
    off = c.skip;
    if (left > 0 && i >= 0) rq = read_request(p, i);
    // of the prefix's row tiles, all alike, those before the share
    if (left > 0 && i < 0 && plen > 0) {
      const int per = units_of(tiles_of(plen));
      rt = min(off / per, prefix_items);
      off -= rt * per;
    }
  }

  __device__ void next_request(const Kv4Attn& p) {
    rt = 0;
    if (++i >= batch) { i = -1; ++h; }
    if (i >= 0) rq = read_request(p, i);
  }
  __device__ bool next(const Kv4Attn& p, Segment& s) {
    while (left > 0 && h < p.Hkv) {
      const bool prefix = i < 0;
      if (rt >= (prefix ? prefix_items : rq.row_tiles(p))) { next_request(p); continue; }
      const int keys = prefix ? prefix_len : rq.seen(p, rt), units = units_of(tiles_of(keys)), room = units - off;
      if (room > 0) {
        const int take = left < static_cast<uint32_t>(room) ? static_cast<int>(left) : room;
        s.live = 1;
        s.h = h;
        s.j0 = max(off - kItemCost, 0);
        s.j1 = off + take - kItemCost;
        s.keys = keys;
        if (prefix) {
          s.tok0 = rt * p.tpt;
          s.toks = min(p.tpt, p.T - s.tok0);
          s.own = 0; s.lim0 = 0; s.least = keys;
          s.pages = p.prefix_pages;
        } else {
          s.tok0 = rq.a + rt * p.tpt;
          s.toks = min(p.tpt, rq.a + rq.n - s.tok0);
          s.own = p.causal; s.lim0 = rq.len - rq.n - rq.a + 1;
          s.least = p.causal ? max(0, min(keys, s.lim0 + s.tok0)) : keys;
          s.pages = p.page_table + static_cast<long long>(i) * p.table_width;
        }
        s.part_row = part_row(p, h, s.tok0, !prefix, share);
        left -= take;
        off += take;
      }
      if (off >= units) {
        off -= units;
        ++rt;
      }
      if (room > 0 && s.j1 > s.j0) return true;
    }
    return false;
  }
};

// Where the CTA's share begins in its head's list: a scan over the requests' units.
// What kv4_merge_kernel needs of it goes to the workspace.  Starts out of order may
// leave blocks that overlap: where they claim more than the T tokens that the entry
// point counted units for, no request is served.
// -> the prefix's length.
template <int kThreads>
__device__ __forceinline__ int find_share(const Kv4Attn& p, Start& c) {
  const int prefix = p.prefix_cap > 0 ? __ldg(p.prefix_len) : 0;  // (looked at when the requests are under way)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
  // the tokens' requests, for kv4_merge_kernel: every CTA writes those of its remainder (none
  // yet)
  for (int t = static_cast<int>(blockIdx.x) + tid * p.ctas; t < p.T; t += kThreads * p.ctas)
    p.requests[t] = RequestPlan{0, 0, 0, 0};
  uint32_t mine = 0, cost0 = 0;
  long long tokens = 0;
  bool ok = true;
  for (int b = tid; b < p.B; b += kThreads) {
    const Request rq = read_request(p, b);
    const uint32_t u = rq.units(p);
    if (b == tid) cost0 = u;
    mine += u;
    tokens += rq.n;
    ok &= rq.ok;
  }
  const int plen = held(prefix, p.prefix_cap, p.page, p.status);
  const uint32_t lead = plen > 0 ? static_cast<uint32_t>((p.T + p.tpt - 1) / p.tpt) * units_of(tiles_of(plen)) : 0;
  uint32_t all = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) c.sums[warp] = all;
  int batch = p.B;
  if (!__syncthreads_and(ok)) {
    if (tid == 0) c.claimed = 0;
    __syncthreads();
    atomicAdd(&c.claimed, static_cast<unsigned long long>(tokens));
    __syncthreads();
    if (c.claimed > static_cast<unsigned long long>(p.T)) batch = 0;
  }
  all = 0;
  if (batch > 0)
    for (int w = 0; w < kWarps; ++w) all += c.sums[w];
  __syncthreads();
  const uint32_t per_head = lead + all, units = per_head * p.Hkv;
  const Shares s = {units / p.ctas, units % p.ctas};
  if (blockIdx.x == 0 && tid == 0) *p.plan = Plan{per_head, tiles_of(plen), s};
  const uint32_t u0 = s.start(blockIdx.x), n = s.start(blockIdx.x + 1) - u0, head = n > 0 ? u0 / per_head : 0;
  const uint32_t at = n > 0 ? u0 - head * per_head : 0xffffffffu;
  if (tid == 0) {
    c.units = n;
    c.head = static_cast<int>(head);
    c.request = -1;
    c.skip = static_cast<int>(at);
    c.batch = batch;
  }
  uint32_t base = lead;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + tid;
    uint32_t own = b < batch ? cost0 : 0;
    if (b0 > 0) own = b < batch ? read_request(p, b).units(p) : 0;
    uint32_t inc = own;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    uint32_t first = base + inc - own;
    if (lane == 31) c.sums[warp] = inc;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) first += c.sums[w];
      base += c.sums[w];
    }
    __syncthreads();
    if (at >= first && at - first < own) {
      c.request = b;
      c.skip = static_cast<int>(at - first);
    }
    if (b < batch) {
      const Request rq = read_request(p, b);
      const int i0 = (static_cast<int>(blockIdx.x) - rq.a % p.ctas + p.ctas) % p.ctas;
      for (int i = i0; i < rq.n; i += p.ctas) p.requests[rq.a + i] = RequestPlan{rq.a, rq.n, rq.len, first};
    }
  }
  return plen;
}

// The same for up to 32 requests, by the warp that walks the list alone, a lane a request: the
// other warps have nothing to wait for but its first segment.  (Single tokens over 640 keys:
// 11.9 us with the whole CTA's scan, 11.3 like this; 8 blocks of 9 over 4096 31.3 and 29.4.)
constexpr int kWarpRequests = 32;
__device__ __forceinline__ int find_share_by_warp(const Kv4Attn& p, Start& c) {
  const int prefix = p.prefix_cap > 0 ? __ldg(p.prefix_len) : 0;  // (looked at when the requests are under way)
  const int lane = threadIdx.x & 31;
  Request rq = {0, 0, 0, true};
  if (lane < p.B) rq = read_request(p, lane);
  for (int t = static_cast<int>(blockIdx.x) + lane * p.ctas; t < p.T; t += 32 * p.ctas)
    p.requests[t] = RequestPlan{0, 0, 0, 0};
  const int plen = held(prefix, p.prefix_cap, p.page, p.status);
  int batch = p.B;
  if (!__all_sync(0xffffffffu, rq.ok)) {
    long long claimed = rq.n;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) claimed += __shfl_xor_sync(0xffffffffu, claimed, o);
    if (claimed > p.T) batch = 0;
  }
  const uint32_t lead = plen > 0 ? static_cast<uint32_t>((p.T + p.tpt - 1) / p.tpt) * units_of(tiles_of(plen)) : 0;
  const uint32_t own = lane < batch ? rq.units(p) : 0;
  uint32_t inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  const uint32_t first = lead + inc - own, per_head = lead + __shfl_sync(0xffffffffu, inc, 31), units = per_head * p.Hkv;
  const Shares s = {units / p.ctas, units % p.ctas};
  const uint32_t u0 = s.start(blockIdx.x), n = s.start(blockIdx.x + 1) - u0, head = n > 0 ? u0 / per_head : 0;
  const uint32_t at = n > 0 ? u0 - head * per_head : 0xffffffffu;
  const uint32_t here = __ballot_sync(0xffffffffu, at >= first && at - first < own);
  const uint32_t skip = at - __shfl_sync(0xffffffffu, first, here ? __ffs(here) - 1 : 0);
  if (lane == 0) {
    if (blockIdx.x == 0) *p.plan = Plan{per_head, tiles_of(plen), s};
    c.units = n;
    c.head = static_cast<int>(head);
    c.request = here ? __ffs(here) - 1 : -1;
    c.skip = static_cast<int>(here ? skip : at);
    c.batch = batch;
  }
  __syncwarp();
  if (lane < batch) {
    const int i0 = (static_cast<int>(blockIdx.x) - rq.a % p.ctas + p.ctas) % p.ctas;
    for (int i = i0; i < rq.n; i += p.ctas) p.requests[rq.a + i] = RequestPlan{rq.a, rq.n, rq.len, first};
  }
  return plen;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}

// ---------------------------------------------------------------- copies of keys
// Those of the kKeys keys from `first` (a multiple of kKeys) that a segment needs go into
// shared memory, as blocks of min(page, kKeys) slots, by one warp: a lane a page, or, of a
// longer page, a lane a run of it.
// A segment's page numbers, 32 at a time a lane each and the next 32 on their way: the
// copies are issued faster than a page table answers (850 clocks a stage where each
// waited for its own number).
template <int kKeys>
struct Pages {
  const int32_t* at;
  int count, chunk, now, next;
  __device__ __forceinline__ int read(int c, int lane) const { return 32 * c + lane < count ? __ldg(at + 32 * c + lane) : 0; }
  __device__ __forceinline__ void begin(const Kv4Attn& p, const Segment& s, int lane) {
    at = s.pages;
    count = (min(s.j1 * kTile, s.keys) + p.page - 1) >> p.page_log2;
    chunk = (s.j0 * kTile / kKeys * kKeys >> p.page_log2) >> 5;
    now = read(chunk, lane);
    next = read(chunk + 1, lane);
  }
  // The lane's page of those from key `first` on (a stage's are among one 32).
  __device__ __forceinline__ int of(const Kv4Attn& p, int first, int lane) {
    const int i = first >> p.page_log2;
    if (i >> 5 != chunk) {
      chunk = i >> 5;
      now = next;
      next = read(chunk + 1, lane);
    }
    return __shfl_sync(0xffffffffu, now, (i + lane) & 31);
  }
};
// (Pages outside the cache are recorded and read as zeros.)
template <int D, int kKeys>
__device__ __forceinline__ void copy_keys(const Kv4Attn& p, const Segment& s, int first, int page, uint8_t* dst,
                                          uint64_t* bar, int lane) {
  constexpr int kGroups = D / 32, kWhole = kKeys * kv4_slot_bytes(D);
  const int block = p.page * kv4_slot_bytes(D), at = first + (lane << p.page_log2);
  const bool runs = p.page > kKeys;
  if (runs) page = __shfl_sync(0xffffffffu, page, 0);
  const bool need = runs || (lane << p.page_log2 < kKeys && at < min(s.j1 * kTile, s.keys) && at + p.page > s.j0 * kTile);
  const bool bad = need && static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.n_pages);
  const uint32_t bads = __ballot_sync(0xffffffffu, bad), goods = __ballot_sync(0xffffffffu, need && !bad);
  if (bads) {
    if (bad) record_index(p.status, kInfoPage);
    const int bytes = runs ? kWhole : block;
    for (int i = 0; i < (runs ? 1 : 32); ++i)
      if ((bads >> i) & 1u)
        for (int o = lane * 16; o < bytes; o += 512)
          *reinterpret_cast<uint4*>(dst + i * bytes + o) = make_uint4(0, 0, 0, 0);
    fence_proxy_async();
    __syncwarp();
  }
  const uint8_t* src = p.cache + (static_cast<long long>(bad ? 0 : page) * p.Hkv + s.h) * block;
  if (!runs) {
    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(goods) * block);
    __syncwarp();
    if (need && !bad) bulk_load(dst + lane * block, src, block, bar);
  } else {
    if (lane == 0) mbar_arrive_expect_tx(bar, bads ? 0 : kWhole);
    __syncwarp();
    const int slot = first & (p.page - 1);
    if (!bads && lane < 2 * kGroups) {
      bulk_load(dst + lane * kKeys * 16, src + (lane * p.page + slot) * 16, kKeys * 16, bar);
    } else if (!bads && lane < 2 * kGroups + 2) {
      const int w = lane - 2 * kGroups;
      bulk_load(dst + kv4_scales_at(D, kKeys, w), src + kv4_scales_at(D, p.page, w) + slot * kGroups, kKeys * kGroups, bar);
    }
  }
}

// Few rows against many keys (attention_kv4_few.cu): whether a call takes it, the most
// rows of its row tiles, and its launch.
int kv4_few_rows(int T, int B, int G, int page, int prefix_cap, int table_width);
cudaError_t launch_kv4_few(const Kv4Attn& p, int rows, int D, bool bf16, cudaStream_t s);

}  // namespace moe
