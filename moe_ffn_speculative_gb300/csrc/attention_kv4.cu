// Attention of a batch of requests over a shared prefix and pages of their own, keys
// and values held in 4 bits (moe_prefix_attention_kv4).  Cache: kv4.cuh.
//
// For the query of token t (the i-th of its request's n) and head h, over the prefix
// keys and the first `seen` of the request's own keys:
//   o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = scale log2(e) q . k_j.
//
// What bounds it is the expansion of the codes, beside the bytes: a key head's key
// and value are 272 bytes in 16 bits and 272/2 here, but 256 numbers either way, and a
// few queries read them.  So both products run transposed, with the keys' 128 lanes in
// the MMA's M dimension and the query rows (heads of a group x tokens of a block, up to
// 64) in N, whose width follows the rows:
//   S^T [keys x rows]     = K Q^T    K expanded into tensor memory, a key a thread
//   O^T [channels x rows] += V^T P^T  V expanded into shared memory, a key a thread
// A thread that holds a key has its scales as scalars, and K never passes through
// shared memory again.  The softmax's thread holds one key and all rows: its sums stay
// in its registers until a segment ends, and the only thing that has to cross threads
// is the reference m.  That moves when a tile's score passes it by more than 2^7 (as in
// the 16-bit kernel), which one vote a tile finds out; only then are the rows' maxima
// taken.
//
// Both products are f16.  A code times its scale (2^-23 .. 2^13) is exact in f16, an
// f16 query is taken as it is, and a bf16 one after its row is scaled by the power of
// two that brings its largest element to [2^14, 2^15): exact down to 2^-31 of that,
// with an error of at most 2^-40 of it below.  Powers enter the second product with
// the row's maximum counting 2^7 (at most 2^14 before m moves), so that a key is held
// to within 2^-32 of the row's largest; their sum stays fp32, unrounded.
//
// Work.  A key head's list holds the prefix against every row tile of the batch, then
// every request's row tiles against its own keys, in tiles of 128 keys; an item counts
// kItemCost tiles more than it has.  The lists of all heads, one after the other, are
// cut into equal contiguous shares, one a CTA.  Every (item, share) leaves its rows'
// references, sums and fp32 outputs in the workspace, and kv4_merge_kernel joins a row's
// parts in a fixed order: results do not depend on timing.
//
// A CTA (one per SM): warp 0 copies tiles (a page of a head is one run of bytes), warp
// 1 issues the MMAs, warp 2 walks the list, warp 3 loads queries; warps 4..7 expand
// keys, 8..11 are the softmax, 12..15 expand values.
//
// Keys past a length are never read as numbers: their codes are replaced by zeros, and
// their scores before the maximum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include <initializer_list>

#include "kv4.cuh"
#include "moe.h"

namespace moe {
namespace {

constexpr int kTile = 128;       // keys of a tile
constexpr int kRows = 64;        // most rows of a row tile
constexpr int kThreads = 512;
constexpr int kItemCost = 2;     // an item's fixed cost, in key tiles
constexpr float kLift = 7.f, kRescaleAt = 7.f;
constexpr int kSmem = 232448;    // 227 KB
constexpr int kMaxStages = 12;
constexpr int kSegments = 4;
constexpr int kReaders = 15;     // of a segment: producer, issuer, query loader, 12 warps
// Registers a thread, moved between the warpgroups: 128 x (88 + 104 + 216 + 104) = 512 x 128
constexpr int kRegsFew = 88, kRegsExpand = 104, kRegsSoftmax = 216;

struct Params {
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
  struct RequestPlan* requests;  // [B]
  int32_t* request_of;           // [T] the request of a token
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
// A request as kv4_merge_kernel reads it.
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
  __device__ int seen(const Params& p, int rt) const {
    if (!p.causal) return len;
    return max(0, min(len, len - n + min(n, (rt + 1) * p.tpt)));
  }
  __device__ int row_tiles(const Params& p) const { return (n + p.tpt - 1) / p.tpt; }
  __device__ uint32_t units(const Params& p) const {
    const int k = row_tiles(p);
    if (!p.causal) return static_cast<uint32_t>(k) * units_of(tiles_of(len));
    uint32_t u = 0;
    for (int rt = 0; rt < k; ++rt) u += units_of(tiles_of(seen(p, rt)));
    return u;
  }
};
__device__ __noinline__ Request read_request(const Params& p, int b) {
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
__device__ __forceinline__ long long part_row(const Params& p, int h, int t, bool own, int share) {
  return (static_cast<long long>(h) * 2 * p.T + (own ? p.T : 0) + t) * p.G + static_cast<long long>(kRows) * share;
}

struct Walker {
  int share;
  uint32_t left;  // units still to walk
  int off;        // units of the current item before the share
  int h, i, rt;   // i: request, or -1 for the prefix; rt: row tile
  int batch, prefix_len, prefix_items;
  Request rq;

  __device__ void next_request(const Params& p) {
    rt = 0;
    if (++i >= batch) { i = -1; ++h; }
    if (i >= 0) rq = read_request(p, i);
  }
  __device__ bool next(const Params& p, Segment& s) {
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

// ---------------------------------------------------------------- tensor memory, MMA
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// A from tensor memory: its rows lanes, two 16-bit values a column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\ttcgen05.mma.cta_group::1."
      "kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Lower descriptor word of an operand whose M or N dimension is contiguous: 64 elements
// of one key in 128 bytes, 128-byte swizzle, 8-key groups 1024 bytes apart, blocks of 64
// elements kTile * 128 bytes apart.
constexpr uint32_t kDescLoN = static_cast<uint32_t>((kTile * 128) >> 4) << 16;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ unsigned long long pair(float a, float b) {
  unsigned long long v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpair(unsigned long long v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
// The four softmax warps: do any of their threads say yes?
__device__ __forceinline__ bool softmax_any(bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 2, 128, p;\n\tselp.u32 %0, 1, 0, "
      "q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(mine))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 2, 128;" ::: "memory"); }

// ---------------------------------------------------------------- shared memory
template <int D>
struct Geometry {
  static constexpr int kGroups = D / 32;
  static constexpr int kStageBytes = kTile * kv4_slot_bytes(D);
  static constexpr int kValueBytes = kTile * D * 2, kProbBytes = kTile * kRows * 2, kQueryBytes = kRows * D * 2;
  static constexpr int kValuesAt = 0, kProbsAt = 2 * kValueBytes, kQueriesAt = kProbsAt + 2 * kProbBytes;
  static constexpr int kRingAt = kQueriesAt + 2 * kQueryBytes;
  static constexpr int kFit = (kSmem - 4096 - 1024 - kRingAt) / kStageBytes;  // 4 KB for the control words
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kDynamic = 1024 + kRingAt + kStages * kStageBytes;
  // tensor memory: two expanded key tiles, two score tiles, two output tiles
  static constexpr uint32_t kKeysCol = 0, kScoresCol = D, kOutCol = D + 2 * kRows;
};

struct Control {
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
  uint64_t k_full[2], k_empty[2], s_full[2], s_empty[2], v_full[2], v_empty[2], p_full[2], p_empty[2];
  uint64_t q_full[2], q_empty[2], o_full[2], o_empty[2], drain;
  uint64_t seg_full[kSegments], seg_empty[kSegments];
  Segment seg[kSegments];
  uint32_t tmem;
  int abort_flag;
  // of a segment's rows: score scale and keys seen, with the queries
  float row_scale[2][kRows];
  int row_limit[2][kRows];
  // of the softmax: the reference, its negative (0 for none), the factor of a move, the warps' maxima
  float m[kRows], neg[kRows], factor[kRows];
  float top[4][kRows];
  uint32_t sums[kThreads / 32];
  unsigned long long claimed;
  Shares s;
  uint32_t per_head, units;
  int head, request, skip, batch;
};

__device__ __forceinline__ bool warp_wait(Control& c, uint64_t* bar, uint32_t parity, int32_t* status, int32_t info) {
  const bool ok = mbar_wait(bar, parity, &c.abort_flag);
  if (__all_sync(0xffffffffu, ok)) return true;
  if ((threadIdx.x & 31) == 0) record_failure(status, &c.abort_flag, info);
  return false;
}
// The n-th segment of the CTA.
__device__ __forceinline__ bool take(Control& c, int& n, Segment& s, int32_t* status) {
  const int e = n % kSegments;
  if (!warp_wait(c, &c.seg_full[e], (n / kSegments) & 1, status, kInfoAttnList)) return false;
  s = c.seg[e];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&c.seg_empty[e]);
  ++n;
  return true;
}
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ---------------------------------------------------------------- producer (warp 0)
// A lane a page (or, of a page longer than a tile, a lane a run): the tile lies in
// shared memory as the blocks of pages of min(page, 128) slots.
template <int D>
struct Producer {
  using Geo = Geometry<D>;
  const Params& p;
  Control& c;
  uint8_t* ring_mem;
  Ring ring;
  int filled;
  int lane;

  __device__ __forceinline__ int pages_in(const Segment& s, int j) const {
    const int valid = min(kTile, s.keys - j * kTile);
    return p.page >= kTile ? 1 : (valid + p.page - 1) >> p.page_log2;
  }
  __device__ __forceinline__ int page_at(const Segment& s, int j) const {
    return lane < pages_in(s, j) ? __ldg(s.pages + ((j * kTile) >> p.page_log2) + lane) : 0;
  }
  __device__ __forceinline__ bool load(const Segment& s, int j, int page) {
    if (!warp_wait(c, &c.kv_empty[ring.stage], ring.phase ^ 1u, p.status, kInfoAttnStage)) return false;
    const int n = pages_in(s, j);
    uint64_t* bar = &c.kv_full[ring.stage];
    uint8_t* dst = ring_mem + ring.stage * Geo::kStageBytes;
    const int block = p.page * kv4_slot_bytes(D);
    if (p.page > kTile) page = __shfl_sync(0xffffffffu, page, 0);
    const bool some = p.page > kTile || lane < n;
    const bool bad = some && static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.n_pages);
    const uint32_t bads = __ballot_sync(0xffffffffu, bad);
    if (bads) {  // read as zeros
      if (bad) record_index(p.status, kInfoPage);
      const int bytes = p.page > kTile ? Geo::kStageBytes : block;
      for (int i = 0; i < n; ++i)
        if (p.page > kTile || ((bads >> i) & 1u))
          for (int o = lane * 16; o < bytes; o += 512)
            *reinterpret_cast<uint4*>(dst + i * bytes + o) = make_uint4(0, 0, 0, 0);
      fence_proxy_async();
      __syncwarp();
    }
    const uint8_t* src = p.cache + (static_cast<long long>(bad ? 0 : page) * p.Hkv + s.h) * block;
    if (p.page <= kTile) {
      if (lane == 0) mbar_arrive_expect_tx(bar, (n - __popc(bads)) * block);
      __syncwarp();
      if (lane < n && !bad) bulk_load(dst + lane * block, src, block, bar);
    } else {
      if (lane == 0) mbar_arrive_expect_tx(bar, bads ? 0 : Geo::kStageBytes);
      __syncwarp();
      const int at = (j * kTile) & (p.page - 1);
      if (!bads && lane < 2 * Geo::kGroups)
        bulk_load(dst + lane * kTile * 16, src + (lane * p.page + at) * 16, kTile * 16, bar);
      else if (!bads && lane < 2 * Geo::kGroups + 2) {
        const int w = lane - 2 * Geo::kGroups;
        bulk_load(dst + kv4_scales_at(D, kTile, w), src + kv4_scales_at(D, p.page, w) + at * Geo::kGroups,
                  kTile * Geo::kGroups, bar);
      }
    }
    ++filled;
    ring.next(Geo::kStages);
    return true;
  }
  __device__ void run() {
    Segment s;
    int n = 0;
    while (take(c, n, s, p.status) && s.live) {
      int page = page_at(s, s.j0);
      for (int j = s.j0; j < s.j1; ++j) {
        const int next = j + 1 < s.j1 ? page_at(s, j + 1) : 0;
        if (!load(s, j, page)) return;
        page = next;
      }
    }
  }
  // Every copy that was issued has landed (also after a failure).
  __device__ void drain() {
    for (int e = 0; e < Geo::kStages; ++e) {
      const int fills = filled / Geo::kStages + (e < filled % Geo::kStages ? 1 : 0);
      if (fills > 0 && !mbar_wait(&c.kv_full[e], (fills - 1) & 1, nullptr))
        record_failure(p.status, &c.abort_flag, kInfoAttnDrain);
    }
  }
};

// ---------------------------------------------------------------- expansion (warps 4..7 and 12..15)
// A thread a key: its codes of one kind, as f16.
template <int D, bool kValues>
__device__ __forceinline__ void expand(const Params& p, Control& c, uint8_t* ring_mem, uint8_t* v_mem, uint32_t tmem) {
  using Geo = Geometry<D>;
  const int key = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3;
  const int local = min(p.page, kTile), log2 = min(p.page_log2, 7), at = key & (local - 1);
  // places of the key's codes and scales in a stage
  const int base = (key >> log2) * local * kv4_slot_bytes(D);
  const int codes_at = base + kv4_codes_at(D, local, kValues) + at * 16;
  const int scales_at = base + kv4_scales_at(D, local, kValues) + at * Geo::kGroups;
  Segment s;
  Ring ring;
  int n = 0, i = 0;
  while (take(c, n, s, p.status) && s.live) {
    for (int j = s.j0; j < s.j1; ++j, ++i) {
      const int buf = i & 1;
      if (!warp_wait(c, &c.kv_full[ring.stage], ring.phase, p.status, kInfoAttnStage)) return;
      const uint8_t* st = ring_mem + ring.stage * Geo::kStageBytes;
      uint4 w[Geo::kGroups];
      uint32_t scales;
#pragma unroll
      for (int g = 0; g < Geo::kGroups; ++g) w[g] = *reinterpret_cast<const uint4*>(st + codes_at + g * local * 16);
      if (Geo::kGroups == 4) scales = *reinterpret_cast<const uint32_t*>(st + scales_at);
      else scales = *reinterpret_cast<const uint16_t*>(st + scales_at);
      arrive_warp(&c.kv_empty[ring.stage]);
      ring.next(Geo::kStages);
      const bool past = j * kTile + key >= s.keys;
      if (!warp_wait(c, kValues ? &c.v_empty[buf] : &c.k_empty[buf], ((i >> 1) & 1) ^ 1u, p.status, kInfoAttnProbs))
        return;
      if (!kValues) tc_fence_after();
#pragma unroll
      for (int g = 0; g < Geo::kGroups; ++g) {
        const uint32_t f = past ? 0u : kv4_scale_h2((scales >> (8 * g)) & 255u);
        const uint32_t x[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
        uint32_t y[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          kv4_expand(x[k], *reinterpret_cast<uint32_t(*)[4]>(y + 4 * k));
#pragma unroll
          for (int b = 0; b < 4; ++b) y[4 * k + b] = kv4_mul2(y[4 * k + b], f);
        }
        if (kValues) {
          uint8_t* row = v_mem + buf * Geo::kValueBytes + (g / 2) * (kTile * 128) + key * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(row + (((g % 2) * 4 + k) ^ (key & 7)) * 16) =
                make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
        } else {
          tmem_st16(tmem + Geo::kKeysCol + buf * (D / 2) + g * 16 + (static_cast<uint32_t>(warp * 32) << 16), y);
        }
      }
      if (kValues) {
        fence_proxy_async();
        arrive_warp(&c.v_full[buf]);
      } else {
        tmem_st_wait();
        tc_fence_before();
        arrive_warp(&c.k_full[buf]);
      }
    }
  }
}

// ---------------------------------------------------------------- queries (warp 3)
// Rows into the K-major, 128-byte-swizzled tile of the first product, in f16, with
// their scales and limits.  A lane group of D / 8 lanes takes a row.
template <bool kBf16, int D>
__device__ __forceinline__ void load_queries(const Params& p, Control& c, uint8_t* q_mem) {
  using Geo = Geometry<D>;
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
  const int lane = threadIdx.x & 31, ch = lane % kLanes, sub = lane / kLanes;
  Segment s;
  int n = 0;
  while (true) {
    const int seg = n, buf = seg & 1;
    if (!take(c, n, s, p.status) || !s.live) return;
    if (!warp_wait(c, &c.q_empty[buf], ((seg >> 1) & 1) ^ 1u, p.status, kInfoAttnQuery)) return;
    const int rows = s.toks * p.G, width = (rows + 15) / 16 * 16;
    uint8_t* dst = q_mem + buf * Geo::kQueryBytes;
    for (int r0 = 0; r0 < width; r0 += 8 * kAtOnce) {
      uint4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = r0 + k * kAtOnce + sub;
        x[k] = make_uint4(0, 0, 0, 0);
        if (r < rows)
          x[k] = __ldg(reinterpret_cast<const uint4*>(p.q + (s.tok0 + r / p.G) * p.q_stride + (s.h * p.G + r % p.G) * D +
                                                      ch * 8));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = r0 + k * kAtOnce + sub;
        float scale = p.scale_log2;
        if (kBf16) {
          uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, top = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
          top = max(top & 0xffffu, top >> 16);
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          // the largest element goes to [2^14, 2^15); rows of zeros, infinities or NaN stay
          int e = static_cast<int>(top >> 7) - 127 - 14;
          if (top == 0 || top >= 0x7f80u) e = 0;
          e = max(e, -126);
          const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          scale *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = pack_h2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
          x[k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (r < width) {
          *reinterpret_cast<uint4*>(dst + (ch / 8) * (kRows * 128) + r * 128 + ((ch % 8) ^ (r & 7)) * 16) = x[k];
          if (ch == 0) {
            c.row_scale[buf][r] = scale;
            // rows past the tile's see every key, so that they ask for no mask
            c.row_limit[buf][r] =
                r < rows ? (s.own ? max(0, min(s.keys, s.lim0 + s.tok0 + r / p.G)) : s.keys) : 0x7fffffff;
          }
        }
      }
    }
    fence_proxy_async();
    arrive_warp(&c.q_full[buf]);
  }
}

// ---------------------------------------------------------------- MMA issuer (warp 1)
// In the order S(0), S(1), O(0), S(2), O(1), ... over the tiles of all segments: the
// scores of a tile are there when the softmax is done with the one before.
template <int D>
struct Issuer {
  using Geo = Geometry<D>;
  const Params& p;
  Control& c;
  uint32_t v_lo, p_lo, q_lo;
  uint32_t tmem;

  struct Step {
    int i, seg;      // tile and segment of the CTA
    int width;       // rows, a multiple of 16
    bool first, last;
  };
  __device__ __forceinline__ bool scores(const Step& t) {
    const int buf = t.i & 1, qb = t.seg & 1;
    if (t.first && !warp_wait(c, &c.q_full[qb], (t.seg >> 1) & 1, p.status, kInfoAttnQuery)) return false;
    if (!warp_wait(c, &c.k_full[buf], (t.i >> 1) & 1, p.status, kInfoAttnStage) ||
        !warp_wait(c, &c.s_empty[buf], ((t.i >> 1) & 1) ^ 1u, p.status, kInfoAttnScores))
      return false;
    tc_fence_after();
    if (elect()) {
      const uint32_t id = idesc_f16(kTile, t.width), b = kDescLoK + q_lo + qb * (Geo::kQueryBytes / 16);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        mma_ts(tmem + Geo::kScoresCol + buf * kRows, tmem + Geo::kKeysCol + buf * (D / 2) + ks * 8,
               b + (ks / 4) * (kRows * 128 / 16) + (ks % 4) * 2, kDescHi, id, ks > 0 ? 1u : 0u);
      mma_commit(&c.s_full[buf]);
      mma_commit(&c.k_empty[buf]);
      if (t.last) mma_commit(&c.q_empty[qb]);
    }
    __syncwarp();
    return true;
  }
  __device__ __forceinline__ bool outputs(const Step& t) {
    const int buf = t.i & 1, ob = t.seg & 1;
    if (t.first && !warp_wait(c, &c.o_empty[ob], ((t.seg >> 1) & 1) ^ 1u, p.status, kInfoAttnOut)) return false;
    if (!warp_wait(c, &c.v_full[buf], (t.i >> 1) & 1, p.status, kInfoAttnStage) ||
        !warp_wait(c, &c.p_full[buf], (t.i >> 1) & 1, p.status, kInfoAttnProbs))
      return false;
    tc_fence_after();
    if (elect()) {
      const uint32_t id = idesc_f16(kTile, t.width) | (3u << 15);  // A: M-major, B: N-major
      const uint32_t a = kDescLoN + v_lo + buf * (Geo::kValueBytes / 16);
      const uint32_t b = kDescLoN + p_lo + buf * (Geo::kProbBytes / 16);
#pragma unroll
      for (int ks = 0; ks < kTile / 16; ++ks)
        mma_ss(tmem + Geo::kOutCol + ob * kRows, a + ks * (2048 / 16), kDescHi, b + ks * (2048 / 16), kDescHi, id,
               ks > 0 || !t.first ? 1u : 0u);
      mma_commit(&c.v_empty[buf]);
      mma_commit(&c.p_empty[buf]);
      if (t.last) mma_commit(&c.o_full[ob]);
    }
    __syncwarp();
    return true;
  }
  __device__ void run() {
    Segment s;
    Step cur, before;
    bool have = false;
    int n = 0, i = 0;
    while (true) {
      const int seg = n;
      if (!take(c, n, s, p.status)) return;
      if (!s.live) break;
      const int width = (s.toks * p.G + 15) / 16 * 16;
      for (int j = s.j0; j < s.j1; ++j, ++i) {
        cur = Step{i, seg, width, j == s.j0, j + 1 == s.j1};
        if (!scores(cur)) return;
        if (have && !outputs(before)) return;
        before = cur;
        have = true;
      }
    }
    if (have) outputs(before);
  }
};

// ---------------------------------------------------------------- softmax (warps 8..11)
// The four warps agree on every turn: what one of them alone finds out (a wait that ran
// out) goes through a vote before any leaves.
// Moves the reference of the rows whose scores pass it (all of them at a segment's first
// tile, i of the CTA), and what was added up under the old one: the outputs here, the
// callers' sums by c.factor.  (Not inlined: it is rare, and its code would push the
// softmax's out of the instruction cache.)
template <int D>
__device__ __noinline__ bool move_reference(Control& c, int32_t* status, uint32_t tmem, uint32_t lanes, int key, int i,
                                            int seg, int width, int at, bool masked, bool first, bool failed) {
  using Geo = Geometry<D>;
  if (softmax_any(failed)) return false;
  const int buf = i & 1, qb = seg & 1, lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  const uint32_t t = tmem + Geo::kScoresCol + buf * kRows + lanes;
  for (int r0 = 0; r0 < width; r0 += 16) {
    uint32_t x[16];
    tmem_ld16(t + r0, x);
    tmem_ld_wait();
    float mine = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (masked && at >= c.row_limit[qb][r0 + k]) x[k] = 0xff800000u;  // -infinity
      // in the order of their bits
      int v = static_cast<int>(x[k]);
      v ^= (v >> 31) & 0x7fffffff;
      v = __reduce_max_sync(0xffffffffu, v);
      v ^= (v >> 31) & 0x7fffffff;
      if (lane == k) mine = __int_as_float(v);
    }
    if (lane < 16) c.top[warp][r0 + lane] = mine;
  }
  softmax_sync();
  if (key < width) {
    float top = -INFINITY;
    for (int w = 0; w < 4; ++w) {
      const float v = c.top[w][key];
      top = isnan(v) || isnan(top) ? NAN : fmaxf(top, v);
    }
    if (top != -INFINITY) top *= c.row_scale[qb][key];
    const float old = first ? -INFINITY : c.m[key];
    // (not: top > ..., so that NaN moves too)
    const bool moves = !(top <= old + (kLift + kRescaleAt)) && top != -INFINITY;
    const float now = moves ? top - kLift : old;
    c.m[key] = now;
    c.neg[key] = now == -INFINITY ? 0.f : -now;
    c.factor[key] = old == -INFINITY ? 0.f : (moves ? ex2(old - now) : 1.f);
  }
  softmax_sync();
  if (first) return true;
  // the products so far are complete
  const bool ok = warp_wait(c, &c.p_empty[(i - 1) & 1], ((i - 1) >> 1) & 1, status, kInfoAttnProbs);
  if (softmax_any(!ok)) return false;
  tc_fence_after();
  const uint32_t o = tmem + Geo::kOutCol + (seg & 1) * kRows + lanes;
  for (int r0 = 0; r0 < width; r0 += 16) {
    uint32_t y[16];
    tmem_ld16(o + r0, y);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * c.factor[r0 + k]);
    tmem_st16(o + r0, y);
  }
  tmem_st_wait();
  return true;
}

template <int D>
struct Softmax {
  using Geo = Geometry<D>;
  const Params& p;
  Control& c;
  uint8_t* p_mem;
  uint32_t tmem;
  int key;             // of the tile: the thread's tensor memory lane
  uint32_t lanes;

  __device__ __forceinline__ void load_scores(uint32_t (&x)[kRows], int buf, int width) {
    const uint32_t t = tmem + Geo::kScoresCol + buf * kRows + lanes;
#pragma unroll
    for (int r = 0; r < kRows; r += 16)
      if (r < width) tmem_ld16(t + r, *reinterpret_cast<uint32_t(*)[16]>(x + r));
    tmem_ld_wait();
  }
  // Logits of keys that a row does not see: -infinity.
  __device__ __forceinline__ void mask(uint32_t (&x)[kRows], int qb, int width, int at) {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (r < width && at >= c.row_limit[qb][r]) x[r] = 0xff800000u;
  }
  // Scores to logits relative to the reference; -> their largest.
  __device__ __forceinline__ float logits(uint32_t (&x)[kRows], int qb, int width, int at, bool masked) {
    const float *scale = c.row_scale[qb], *neg = c.neg;
#pragma unroll
    for (int r = 0; r < kRows; r += 4)
      if (r < width) {
        const float4 a = *reinterpret_cast<const float4*>(scale + r), b = *reinterpret_cast<const float4*>(neg + r);
        float t[4];
        unpair(fma2(pair(__uint_as_float(x[r]), __uint_as_float(x[r + 1])), pair(a.x, a.y), pair(b.x, b.y)), t[0], t[1]);
        unpair(fma2(pair(__uint_as_float(x[r + 2]), __uint_as_float(x[r + 3])), pair(a.z, a.w), pair(b.z, b.w)), t[2],
               t[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[r + k] = __float_as_uint(t[k]);
      }
    if (masked) mask(x, qb, width, at);
    float top = -INFINITY;
#pragma unroll
    for (int r = 0; r < kRows; r += 2)
      if (r < width) top = max3(top, __uint_as_float(x[r]), __uint_as_float(x[r + 1]));
    return top;
  }

  __device__ __forceinline__ bool segment(const Segment& s, int seg, int& i) {
    const int qb = seg & 1, rows = s.toks * p.G, width = (rows + 15) / 16 * 16;
    float l[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) l[r] = 0.f;
    bool ok = warp_wait(c, &c.q_full[qb], (seg >> 1) & 1, p.status, kInfoAttnQuery);
    for (int j = s.j0; j < s.j1; ++j, ++i) {
      const int buf = i & 1, at = j * kTile + key;
      const bool first = j == s.j0, masked = (j + 1) * kTile > s.least;
      ok = ok && warp_wait(c, &c.s_full[buf], (i >> 1) & 1, p.status, kInfoAttnScores);
      tc_fence_after();
      if (first && !move_reference<D>(c, p.status, tmem, lanes, key, i, seg, width, at, masked, true, !ok)) return false;
      uint32_t x[kRows];
      load_scores(x, buf, width);
      const float top = logits(x, qb, width, at, masked);
      if (!first && softmax_any(!ok || top > kLift + kRescaleAt)) {
        if (!move_reference<D>(c, p.status, tmem, lanes, key, i, seg, width, at, masked, false, !ok)) return false;
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          if (r < width) l[r] *= c.factor[r];
        load_scores(x, buf, width);
        logits(x, qb, width, at, masked);
      }
      tc_fence_before();
      arrive_warp(&c.s_empty[buf]);
      ok = warp_wait(c, &c.p_empty[buf], ((i >> 1) & 1) ^ 1u, p.status, kInfoAttnProbs);
      uint8_t* row = p_mem + buf * Geo::kProbBytes + key * 128;
#pragma unroll
      for (int r = 0; r < kRows; r += 8)
        if (r < width) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float e0 = ex2(__uint_as_float(x[r + 2 * k])), e1 = ex2(__uint_as_float(x[r + 2 * k + 1]));
            l[r + 2 * k] += e0;
            l[r + 2 * k + 1] += e1;
            w[k] = pack_h2(e0, e1);
          }
          *reinterpret_cast<uint4*>(row + ((r / 8) ^ (key & 7)) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      fence_proxy_async();
      tc_fence_before();
      arrive_warp(&c.p_full[buf]);
    }
    ok = ok && warp_wait(c, &c.o_full[qb], (seg >> 1) & 1, p.status, kInfoAttnOut);
    if (softmax_any(!ok)) return false;
    tc_fence_after();
    // channels are lanes: a row is written 128 bytes a warp
    const uint32_t o = tmem + Geo::kOutCol + qb * kRows + lanes;
    float* dst = p.o + s.part_row * D + key;
    for (int r0 = 0; r0 < width; r0 += 16) {
      uint32_t y[16];
      tmem_ld16(o + r0, y);
      tmem_ld_wait();
      if (key < D) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (r0 + k < rows) dst[static_cast<long long>(r0 + k) * D] = __uint_as_float(y[k]);
      }
    }
    tc_fence_before();
    arrive_warp(&c.o_empty[qb]);
    // the threads' sums meet over the probabilities, which all products have read
    float* sums = reinterpret_cast<float*>(p_mem);
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (r < width) sums[r * kTile + key] = l[r];
    softmax_sync();
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
    for (int r = warp; r < rows; r += 4) {
      const float4 v = *reinterpret_cast<const float4*>(sums + r * kTile + lane * 4);
      float t = (v.x + v.y) + (v.z + v.w);
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) t += __shfl_xor_sync(0xffffffffu, t, k);
      if (lane == 0) p.ml[s.part_row + r] = make_float2(c.m[r], t);
    }
    arrive_warp(&c.q_empty[qb]);
    softmax_sync();
    return true;
  }
  __device__ void run() {
    Segment s;
    int n = 0, i = 0;
    while (true) {
      const int seg = n;
      const bool got = take(c, n, s, p.status);
      if (softmax_any(!got)) return;
      if (!s.live) return;
      if (!segment(s, seg, i)) return;
    }
  }
};

// ---------------------------------------------------------------- list (all warps, then warp 2)
// Where the CTA's share begins in its head's list: a scan over the requests' units.
// What kv4_merge_kernel needs of it goes to the workspace.  Starts out of order may
// leave blocks that overlap: where they claim more than the T tokens that the entry
// point counted units for, no request is served.
__device__ __forceinline__ void find_share(const Params& p, Control& c, int plen) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
  const uint32_t lead = plen > 0 ? static_cast<uint32_t>((p.T + p.tpt - 1) / p.tpt) * units_of(tiles_of(plen)) : 0;
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
    c.s = s;
    c.per_head = per_head;
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
    if (b < p.B && b % p.ctas == static_cast<int>(blockIdx.x)) {
      const Request rq = read_request(p, b);
      p.requests[b] = RequestPlan{rq.a, b < batch ? rq.n : 0, rq.len, first};
    }
  }
}

// Hands the segments over, one whenever its readers have made room.
__device__ __forceinline__ void hand_list(const Params& p, Control& c, int plen) {
  Walker w;
  w.share = blockIdx.x;
  w.left = c.units;
  w.h = c.head;
  w.i = c.request;
  w.batch = c.batch;
  w.prefix_len = plen;
  w.prefix_items = plen > 0 ? (p.T + p.tpt - 1) / p.tpt : 0;
  w.rt = 0;
  w.off = c.skip;
  if (w.left > 0 && w.i >= 0) w.rq = read_request(p, w.i);
  // of the prefix's row tiles, all alike, those before the share
  if (w.left > 0 && w.i < 0 && plen > 0) {
    const int per = units_of(tiles_of(plen));
    w.rt = min(w.off / per, w.prefix_items);
    w.off -= w.rt * per;
  }
  for (int n = 0;; ++n) {
    Segment s;
    if (!w.next(p, s)) s.live = 0;
    const int e = n % kSegments;
    if (!mbar_wait(&c.seg_empty[e], ((n / kSegments) & 1) ^ 1u, &c.abort_flag)) {
      record_failure(p.status, &c.abort_flag, kInfoAttnList);
      return;
    }
    c.seg[e] = s;
    mbar_arrive(&c.seg_full[e]);
    if (!s.live) return;
  }
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kThreads, 1) prefix_attention_kv4_kernel(const __grid_constant__ Params p) {
  using Geo = Geometry<D>;
  extern __shared__ uint8_t dynamic[];
  __shared__ Control c;
  uint8_t* mem = dynamic + ((1024u - (smem_u32(dynamic) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    c.abort_flag = 0;
    for (int s = 0; s < Geo::kStages; ++s) { mbar_init(&c.kv_full[s], 1); mbar_init(&c.kv_empty[s], 8); }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&c.k_full[b], 4); mbar_init(&c.k_empty[b], 1);
      mbar_init(&c.s_full[b], 1); mbar_init(&c.s_empty[b], 4);
      mbar_init(&c.v_full[b], 4); mbar_init(&c.v_empty[b], 1);
      mbar_init(&c.p_full[b], 4); mbar_init(&c.p_empty[b], 1);
      mbar_init(&c.q_full[b], 1); mbar_init(&c.q_empty[b], 5);
      mbar_init(&c.o_full[b], 1); mbar_init(&c.o_empty[b], 4);
    }
    for (int s = 0; s < kSegments; ++s) { mbar_init(&c.seg_full[s], 1); mbar_init(&c.seg_empty[s], kReaders); }
    mbar_init(&c.drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  }
  griddep_launch_dependents();  // kv4_merge_kernel's blocks wait for all of this grid
  griddep_wait();               // what the previous kernel on the stream wrote is visible
  const int plen = p.prefix_cap > 0 ? held(__ldg(p.prefix_len), p.prefix_cap, p.page, p.status) : 0;
  find_share(p, c, plen);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp == 0) {
      Producer<D> r{p, c, mem + Geo::kRingAt, Ring(), 0, lane};
      r.run();
      __syncwarp();
      r.drain();
    } else if (warp == 1) {
      Issuer<D> r{p, c, smem_u32(mem + Geo::kValuesAt) >> 4, smem_u32(mem + Geo::kProbsAt) >> 4,
                  smem_u32(mem + Geo::kQueriesAt) >> 4, tmem};
      r.run();
      __syncwarp();
      if (elect()) {  // every MMA issued above has completed once `drain` flips
        mma_commit(&c.drain);
        if (!mbar_wait(&c.drain, 0, nullptr)) record_failure(p.status, &c.abort_flag, kInfoAttnDrain);
      }
    } else if (warp == 2) {
      if (lane == 0) hand_list(p, c, plen);
      __syncwarp();
      // the tokens' requests, for kv4_merge_kernel: every CTA writes some
      for (int b = blockIdx.x; b < c.batch; b += p.ctas) {
        const Request rq = read_request(p, b);
        for (int t = lane; t < rq.n; t += 32) p.request_of[rq.a + t] = b;
      }
    } else {
      load_queries<kBf16, D>(p, c, mem + Geo::kQueriesAt);
    }
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsExpand));
    expand<D, false>(p, c, mem + Geo::kRingAt, nullptr, tmem);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    Softmax<D> r{p, c, mem + Geo::kProbsAt, tmem, tid & 127, static_cast<uint32_t>((warp & 3) * 32) << 16};
    r.run();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsExpand));
    expand<D, true>(p, c, mem + Geo::kRingAt, mem + Geo::kValuesAt, tmem);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- joining a row's parts
// A warp a row (token, query head).  Its parts are the shares that hold tiles of its
// items: consecutive ones of the prefix item, consecutive ones of the request's.
constexpr int kMergeThreads = 128;

template <bool kBf16, int D>
__global__ void __launch_bounds__(kMergeThreads) kv4_merge_kernel(const __grid_constant__ Params p) {
  constexpr int kEach = D / 32;  // elements of a lane
  const int lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * (kMergeThreads / 32) + (threadIdx.x >> 5);
  if (unit >= static_cast<long long>(p.T) * p.Hq) return;
  const int t = static_cast<int>(unit / p.Hq), hq = static_cast<int>(unit % p.Hq), h = hq / p.G, g = hq % p.G;
  griddep_wait();
  const Plan plan = *p.plan;
  const int b = p.B > 0 ? p.request_of[t] : -1;
  RequestPlan rp = {0, 0, 0, 0};
  // (a token outside every request reads what an earlier call left: checked)
  if (b >= 0 && b < p.B) rp = p.requests[b];
  const bool owned = t >= rp.a && t < rp.a + rp.n;
  const Request rq = {rp.a, rp.n, rp.len, true};
  float m = -INFINITY, l = 0.f, acc[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    int tiles = 0;
    uint32_t u = h * plan.per_head + kItemCost;
    if (owned && k == 0) {
      tiles = plan.prefix_tiles;
      u += (t / p.tpt) * units_of(tiles);
    } else if (owned) {
      const int rt = (t - rq.a) / p.tpt;
      tiles = tiles_of(rq.seen(p, rt));
      u += rp.first_unit;
      if (!p.causal) u += rt * units_of(tiles);
      else
        for (int i = 0; i < rt; ++i) u += units_of(tiles_of(rq.seen(p, i)));
    }
    if (tiles == 0) continue;
    const int first = plan.s.of(u), count = plan.s.of(u + tiles - 1) - first + 1;
    const long long row = part_row(p, h, t, k == 1, first) + g;
#pragma unroll 1
    for (int i0 = 0; i0 < count; i0 += 32) {
      // lane i: the i-th part of the chunk
      float2 ml = make_float2(-INFINITY, 0.f);
      if (i0 + lane < count) ml = __ldcg(p.ml + row + static_cast<long long>(kRows) * (i0 + lane));
      float top = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float v = __shfl_xor_sync(0xffffffffu, top, o);
        top = isnan(top) || isnan(v) ? NAN : fmaxf(top, v);
      }
      const float m1 = isnan(top) || isnan(m) ? NAN : fmaxf(m, top), base = m1 == -INFINITY ? 0.f : m1;
      const float old = m == -INFINITY ? 0.f : ex2(m - base), mine = ml.x == -INFINITY ? 0.f : ex2(ml.x - base);
      m = m1;
      float sum = mine * ml.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l = l * old + sum;
#pragma unroll
      for (int i = 0; i < kEach; ++i) acc[i] *= old;
      const int n = min(32, count - i0);
#pragma unroll 4
      for (int x = 0; x < n; ++x) {
        const float a = __shfl_sync(0xffffffffu, mine, x);
        const float* o = p.o + (row + static_cast<long long>(kRows) * (i0 + x)) * D + lane * kEach;
        if (kEach == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(o));
          acc[0] += a * v.x; acc[1] += a * v.y; acc[kEach - 2] += a * v.z; acc[kEach - 1] += a * v.w;
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(o));
          acc[0] += a * v.x; acc[1] += a * v.y;
        }
      }
    }
  }
  const float f = l == 0.f ? 0.f : 1.f / l;  // l is 0 where no key was seen
  uint16_t* out = p.out + unit * D + lane * kEach;
  uint32_t w[kEach / 2];
#pragma unroll
  for (int i = 0; i < kEach / 2; ++i) {
    const float a = l == 0.f ? 0.f : acc[2 * i] * f, z = l == 0.f ? 0.f : acc[2 * i + 1] * f;
    if (kBf16) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(a, z);
      memcpy(&w[i], &v, 4);
    } else {
      w[i] = pack_h2(a, z);
    }
  }
  if (kEach == 4) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[kEach / 2 - 1]);
  else *reinterpret_cast<uint32_t*>(out) = w[0];
  if (lane == 0 && p.lse) p.lse[unit] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// MOE_OK where a batch of this shape is within the kernels' limits.
moe_status shape_status(int T, int B, int Hq, int Hkv, int D) {
  if (T < 0 || B < 0 || Hq < 1 || Hkv < 1 || D < 1) return MOE_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return MOE_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || Hq / Hkv > kRows || Hq > 1024 || T > MOE_MAX_ATTN_TOKENS || B > MOE_MAX_REQUESTS)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Workspace after the fixed header.  Monotone in T and B: a size serves every smaller
// call of the same heads.
struct Layout {
  size_t o_plan, o_req, o_of, o_ml, o_o, total;
};
Layout layout(int T, int B, int Hq, int D, int ctas) {
  Layout L;
  const size_t rows = 2 * static_cast<size_t>(T) * Hq + static_cast<size_t>(kRows) * (ctas + 1);
  size_t o = kWsHeaderBytes;
  L.o_plan = o; o += kWsAlign;
  L.o_req = o; o += ws_align_up(sizeof(RequestPlan) * static_cast<size_t>(B));
  L.o_of = o; o += ws_align_up(4 * static_cast<size_t>(T));
  L.o_ml = o; o += ws_align_up(8 * rows);
  L.o_o = o; o += ws_align_up(4 * rows * D);
  L.total = o;
  return L;
}

template <typename K>
cudaError_t launch_one(K* kernel, const Params& p, unsigned grid, int threads, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}
template <bool kBf16, int D>
cudaError_t launch(const Params& p, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(prefix_attention_kv4_kernel<kBf16, D>, Geometry<D>::kDynamic, done);
  if (e != cudaSuccess) return e;
  e = launch_one(prefix_attention_kv4_kernel<kBf16, D>, p, static_cast<unsigned>(p.ctas), kThreads,
                 Geometry<D>::kDynamic, s);
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(p.T) * p.Hq, each = kMergeThreads / 32;
  return launch_one(kv4_merge_kernel<kBf16, D>, p, static_cast<unsigned>((rows + each - 1) / each), kMergeThreads, 0, s);
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_prefix_attention_kv4_workspace_bytes(int T, int B, int Hq, int Hkv, int D) {
  using namespace moe;
  if (shape_status(T, B, Hq, Hkv, D) != MOE_OK) return 0;
  const int sms = device_sms();
  return sms > 0 ? layout(T, B, Hq, D, sms).total : 0;
}

moe_status moe_prefix_attention_kv4(const void* q, long long q_stride, int T, int B, const int32_t* q_start, int Hq,
                                    int Hkv, int D, int dtype, const void* cache, int n_pages, int page_size,
                                    const int32_t* prefix_pages, int prefix_cap, const int32_t* prefix_len,
                                    const int32_t* page_table, int table_width, const int32_t* own_len, int causal,
                                    float scale, void* out, float* lse, void* ws, size_t ws_bytes,
                                    cudaStream_t stream) {
  using namespace moe;
  const moe_status st = shape_status(T, B, Hq, Hkv, D);
  if (st != MOE_OK) return st;
  if (n_pages < 0 || page_size < 1 || prefix_cap < 0 || table_width < 0) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return MOE_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale < INFINITY)) return MOE_ERR_INVALID_ARG;
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(prefix_cap) * page_size > MOE_MAX_KEYS ||
      static_cast<long long>(table_width) * page_size > MOE_MAX_KEYS ||
      static_cast<long long>(n_pages) * page_size > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  // units of the lists, at most, in 31 bits
  {
    const long long tpt = kRows / (Hq / Hkv), row_tiles = (T + tpt - 1) / tpt;
    const long long pt = tiles_of(prefix_cap * page_size) + kItemCost, ot = tiles_of(table_width * page_size) + kItemCost;
    if ((row_tiles * pt + (row_tiles + B) * ot) * Hkv >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
  }
  if (!q || !out || (T > 1 && q_stride < static_cast<long long>(Hq) * D)) return MOE_ERR_INVALID_ARG;
  if (B > 0 && !q_start) return MOE_ERR_INVALID_ARG;
  if (prefix_cap > 0 && (!prefix_pages || !prefix_len)) return MOE_ERR_INVALID_ARG;
  if (B > 0 && table_width > 0 && (!page_table || !own_len)) return MOE_ERR_INVALID_ARG;
  if (prefix_cap + table_width > 0 && (n_pages < 1 || !cache)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(cache) || !aligned16(out) || q == out) return MOE_ERR_INVALID_ARG;
  if (q_stride % 8) return MOE_ERR_UNSUPPORTED;
  const long long row = 2ll * Hq * D;
  const long long pool = static_cast<long long>(n_pages) * page_size * Hkv * kv4_slot_bytes(D);
  const RowSet o = {out, 1, row * T, 0}, z = {lse, 1, 4ll * T * Hq, 0};
  for (const RowSet& read : {RowSet{q, T, row, 2 * q_stride}, RowSet{cache, 1, pool, 0}})
    if (rows_meet(o, read) || rows_meet(z, read)) return MOE_ERR_INVALID_ARG;
  if (rows_meet(o, z)) return MOE_ERR_INVALID_ARG;
  // a workspace that cannot even hold the fixed header is refused before any device query
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kWsAlign) != 0 || ws_bytes < kWsHeaderBytes) return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  const Layout L = layout(T, B, Hq, D, sms);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  Params p;
  memset(&p, 0, sizeof(p));
  p.T = T; p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.tpt = kRows / p.G;
  p.n_pages = n_pages; p.page = page_size;
  while ((1 << p.page_log2) < page_size) ++p.page_log2;
  p.q = static_cast<const uint16_t*>(q); p.q_stride = q_stride;
  p.cache = static_cast<const uint8_t*>(cache);
  p.q_start = q_start; p.prefix_pages = prefix_pages; p.prefix_len = prefix_len; p.page_table = page_table;
  p.own_len = own_len;
  p.prefix_cap = prefix_cap; p.table_width = table_width; p.causal = causal;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.ctas = sms;
  p.out = static_cast<uint16_t*>(out); p.lse = lse;
  char* w = static_cast<char*>(ws);
  p.status = reinterpret_cast<int32_t*>(w);
  p.plan = reinterpret_cast<Plan*>(w + L.o_plan);
  p.requests = reinterpret_cast<RequestPlan*>(w + L.o_req);
  p.request_of = reinterpret_cast<int32_t*>(w + L.o_of);
  p.ml = reinterpret_cast<float2*>(w + L.o_ml);
  p.o = reinterpret_cast<float*>(w + L.o_o);
  const cudaError_t e = dtype == MOE_DTYPE_BF16 ? (D == 64 ? launch<true, 64>(p, stream) : launch<true, 128>(p, stream))
                                                : (D == 64 ? launch<false, 64>(p, stream) : launch<false, 128>(p, stream));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
