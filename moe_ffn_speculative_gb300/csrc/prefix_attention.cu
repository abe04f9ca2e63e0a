// Attention of a batch of requests whose cached context begins with one
// prefix that all of them share, followed by pages of their own
// (moe_prefix_attention).
//
// For the query of token t (the i-th of its request's n) and head h, over the
// prefix keys and the first `seen` of the request's own keys:
//   o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = scale log2(e) q . k_j,
// computed over tiles of 128 keys with a running reference m and running sums
// (fp32).  m is the row's maximum when it was last moved; it moves only when
// a tile's maximum exceeds it by more than 8, so that the accumulator is
// rarely rescaled and no power exceeds 2^8 (the ratio is exact whatever m is).
//
// Work.  The G = Hq / Hkv heads of a token that read one key head are rows of
// one product, so a row tile is floor(128 / G) tokens x G heads.
//   Phase 1: the prefix against pairs of row tiles of the whole batch: each key
//     tile is loaded once for 256 rows.
//   Phase 2: row tiles of one request's block against its own keys, and the
//     last row tile of the batch against the prefix when their number is odd.
// Each phase's list of (row tiles, key tile) steps, heads outermost, is cut
// into equal contiguous shares: one per CTA in phase 1, one per slot in phase
// 2 (a CTA has two slots, each with its own accumulator), an item counting
// kItemCost steps more than it has tiles.  So a long context is split over the
// SMs and short ones are packed.  Every (item, share) leaves its row sums,
// references and unnormalised fp32 output rows in the workspace, and
// merge_kernel joins a row's parts in a fixed order: results do not depend on
// timing.
//
// A CTA (one per SM): warp 0 loads query, key and value tiles by TMA (a page
// is a box of its rows) into a ring of stages; warp 1 issues the MMAs, S = Q K^T
// with both from shared memory, then O += P V with P from tensor memory; warps
// 4..7 and 8..11 are the two slots' softmax, one row a thread.  While one
// slot's softmax runs, the tensor cores work for the other.  Tensor memory is
// full: two S tiles (P overwrites its own S) and two O tiles.
//
// Keys past a length are never read as numbers: their logits are replaced
// before the maximum, the second product's reduction ends at the next
// multiple of 16 keys, and the value rows up to there are zeroed in shared
// memory, so that slots no length covers may hold NaN.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include "moe.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kTile = 128;           // keys of a tile, rows of a row tile
constexpr int kAttnThreads = 384;    // 12 warps
constexpr int kItemCost = 1;         // an item's fixed cost, in key tiles
constexpr float kRescaleAt = 8.f;    // how far a tile's maximum may pass the reference (powers of two)
constexpr int kAttnSmem = 232448;    // 227 KB

struct AttnParams {
  int T, B, Hq, Hkv, G, tpt;         // tpt: tokens of a row tile
  int n_pages, page, page_log2;
  const int32_t *q_start, *prefix_pages, *prefix_len, *page_table, *own_len;
  int prefix_cap, table_width, causal;
  float scale_log2;
  int ctas;
  int pairs, left;                   // row tile pairs of phase 1; 1: the last row tile joins phase 2
  uint16_t* out;
  float* lse;
  // workspace
  int32_t* status;
  struct Plan* plan;
  long long* first_unit;             // [B+1] units of a head's list before each request's
  float2 *ml1, *ml2;                 // (reference, sum) of every part row, phases 1 and 2
  float *o1, *o2;                    // their fp32 rows
};

struct Plan {
  long long per_head;                // phase 2 units of one head
  int prefix_tiles;
};

// ---------------------------------------------------------------- geometry
__host__ __device__ inline int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }
__host__ __device__ inline int units_of(int tiles) { return tiles > 0 ? tiles + kItemCost : 0; }

// The share [start(w), start(w + 1)) of `shares` that holds unit u.
__device__ __forceinline__ long long share_start(long long w, long long total, int shares) {
  return w * total / shares;
}
__device__ __forceinline__ int share_of(long long u, long long total, int shares) {
  return static_cast<int>(((u + 1) * shares - 1) / total);
}

// A length read on the device, held within its page table.
__device__ __forceinline__ int held(int len, int pages, int page, int32_t* status) {
  if (len >= 0 && len <= pages * page) return len;
  record_index(status, kInfoLength);
  return len < 0 ? 0 : pages * page;
}

struct Request {
  int a, n, len;  // first token, tokens, own keys
  // keys seen by the last token of row tile rt
  __device__ int seen(const AttnParams& p, int rt) const {
    if (!p.causal) return len;
    const int last = min(n, (rt + 1) * p.tpt);
    return max(0, min(len, len - n + last));
  }
  __device__ int row_tiles(const AttnParams& p) const { return (n + p.tpt - 1) / p.tpt; }
  __device__ long long units(const AttnParams& p) const {
    long long u = 0;
    const int k = row_tiles(p);
    if (!p.causal) return static_cast<long long>(k) * units_of(tiles_of(len));
    for (int rt = 0; rt < k; ++rt) u += units_of(tiles_of(seen(p, rt)));
    return u;
  }
};

__device__ __forceinline__ Request read_request(const AttnParams& p, int b) {
  Request r;
  r.a = __ldg(p.q_start + b);
  const int z = __ldg(p.q_start + b + 1);
  r.n = z - r.a;
  r.len = p.table_width > 0 ? held(__ldg(p.own_len + b), p.table_width, p.page, p.status) : 0;
  if (r.a < 0 || z < r.a || z > p.T) {
    record_index(p.status, kInfoStarts);
    r.a = r.n = 0;
  }
  return r;
}

// One share's run through one item: row tile(s) against key tiles [j0, j1).
struct Segment {
  int h, tok0, tok_end;      // key head, first token of the (first) row tile, end of valid tokens
  int keys;                  // keys that any of its rows sees
  int own, lim0;             // own keys: token t sees min(keys, max(0, lim0 + t)) of them (causal)
  const int32_t* pages;
  int j0, j1;
  long long part_row;        // part row of token tok0, head h * G
};

// Walks a share's segments; every role of a CTA runs its own copy.
struct Walker {
  int phase, share;
  long long left;  // units still to walk
  int off;         // units of the current item before the share
  int h, i, rt;    // phase 1: h, pair i; phase 2: h, request i (-1: the prefix item), row tile rt
  Request rq;
  int prefix_len, prefix_tiles;

  // Phase 1, share c of p.ctas.
  __device__ void begin1(const AttnParams& p, int plen, int c) {
    phase = 1; share = c; prefix_len = plen; prefix_tiles = tiles_of(plen);
    const long long per = units_of(prefix_tiles), total = per * p.pairs * p.Hkv;
    const long long u0 = share_start(c, total, p.ctas);
    left = share_start(c + 1, total, p.ctas) - u0;
    off = 0; h = i = rt = 0;
    if (left > 0) {
      const long long item = u0 / per;
      off = static_cast<int>(u0 - item * per);
      h = static_cast<int>(item / p.pairs);
      i = static_cast<int>(item % p.pairs);
    }
  }
  // Phase 2, share w of 2 * p.ctas; the list position of its first unit was
  // found by the scan of the requests.
  __device__ void begin2(const AttnParams& p, int plen, int w, long long units, int head, int request, int skip) {
    phase = 2; share = w; prefix_len = plen; prefix_tiles = tiles_of(plen);
    left = units; h = head; i = request; rt = 0; off = skip;
    if (left > 0 && i >= 0) rq = read_request(p, i);
  }
  __device__ void next_request(const AttnParams& p) {
    rt = 0;
    if (++i >= p.B) { i = -1; ++h; }
    if (i >= 0) rq = read_request(p, i);
  }
  __device__ bool next(const AttnParams& p, Segment& s) {
    while (left > 0 && h < p.Hkv) {
      int tiles;
      const bool prefix = phase == 1 || i < 0;
      if (prefix) {
        tiles = (phase == 1 || p.left) ? prefix_tiles : 0;
      } else {
        if (rt >= rq.row_tiles(p)) { next_request(p); continue; }
        tiles = tiles_of(rq.seen(p, rt));
      }
      const int units = units_of(tiles);
      const long long room = units - off;
      if (room > 0) {
        const long long take = left < room ? left : room;
        s.h = h;
        s.j0 = max(off - kItemCost, 0);
        s.j1 = static_cast<int>(off + take) - kItemCost;
        if (prefix) {
          s.tok0 = (phase == 1 ? 2 * i : 2 * p.pairs) * p.tpt;
          s.tok_end = p.T;
          s.keys = prefix_len; s.own = 0; s.lim0 = 0;
          s.pages = p.prefix_pages;
        } else {
          s.tok0 = rq.a + rt * p.tpt;
          s.tok_end = rq.a + rq.n;
          s.keys = rq.seen(p, rt); s.own = p.causal; s.lim0 = rq.len - rq.n - rq.a + 1;
          s.pages = p.page_table + static_cast<long long>(i) * p.table_width;
        }
        s.part_row = part_row(p, phase, h, s.tok0, !prefix, share);
        left -= take;
        off += static_cast<int>(take);
      }
      if (off >= units) {  // on to the next item (unless the share ends inside this one)
        off -= units;
        if (phase == 1) { if (++i >= p.pairs) { i = 0; ++h; } }
        else if (i < 0) next_request(p);
        else ++rt;
      }
      if (room > 0 && s.j1 > s.j0) return true;
    }
    return false;
  }
  // Part rows: an item's rows in list order, plus a row tile (or pair) for
  // every share before it; two parts never meet, as a share's last and the
  // next share's first part may belong to one item.
  __device__ static long long part_row(const AttnParams& p, int phase, int h, int t, bool own, int share) {
    if (phase == 1) return (static_cast<long long>(h) * p.T + t) * p.G + 2ll * kTile * share;
    const int l0 = p.left ? p.T - 2 * p.pairs * p.tpt : 0;  // tokens of the prefix item
    const long long row = static_cast<long long>(h) * (p.T + l0) + (own ? l0 + t : t - 2 * p.pairs * p.tpt);
    return row * p.G + static_cast<long long>(kTile) * share;
  }
};

// ---------------------------------------------------------------- tensor memory, MMA
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem]: A's rows are lanes, two 16-bit values a column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, "
      "p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of a B operand whose N dimension is contiguous (value rows:
// 64 columns of one key in 128 bytes, 128-byte swizzle): 8-key groups 1024
// bytes apart, 64-column blocks kTile * 128 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((kTile * 128) >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t u;
  if (kBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    memcpy(&u, &h, 4);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    memcpy(&u, &h, 4);
  }
  return u;
}

// ---------------------------------------------------------------- shared memory
template <int D>
struct Geometry {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQBufs = D == 64 ? 2 : 1;  // query tiles a slot
  static constexpr int kStages = (kAttnSmem - 1024 - 2 * kQBufs * kTileBytes) / kTileBytes;
  static constexpr int kDynamic = 1024 + (2 * kQBufs + kStages) * kTileBytes;
};

struct Control {
  uint64_t q_full[2][2], q_empty[2][2];
  uint64_t kv_full[16], kv_empty[16];
  uint64_t s_full[2], p_full[2], o_full[2], drain;
  uint32_t tmem;
  int abort_flag;
  long long sums[kAttnThreads / 32];
  long long units[2];  // phase 2 shares of the two slots
  int head[2], request[2], skip[2];
  int prefix_len;
};

// A slot's place in its list of tiles.
struct Cursor {
  Walker w;
  Segment s;
  int j;
  bool live;
  __device__ void start(const AttnParams& p) {
    live = w.next(p, s);
    j = s.j0;
  }
  __device__ bool last() const { return j + 1 == s.j1; }
  __device__ void step(const AttnParams& p) {
    if (++j == s.j1) start(p);
  }
  __device__ int valid() const { return min(kTile, s.keys - j * kTile); }  // keys of the tile that some row sees
};

struct StageRing {
  int stage = 0;
  uint32_t phase = 0;
};

__device__ __forceinline__ bool warp_wait(Control& c, uint64_t* bar, uint32_t parity, int32_t* status, int32_t info) {
  const bool ok = mbar_wait(bar, parity, &c.abort_flag);
  if (__all_sync(0xffffffffu, ok)) return true;
  if ((threadIdx.x & 31) == 0) record_failure(status, &c.abort_flag, info);
  return false;
}

// ---------------------------------------------------------------- TMA producer (warp 0)
template <int D>
struct Producer {
  using Geo = Geometry<D>;
  const AttnParams& p;
  Control& c;
  uint8_t* q_mem;
  uint8_t* kv_mem;
  const CUtensorMap *tm_q, *tm_k, *tm_v;
  StageRing ring;
  int lane;
  int q_fills[2];       // query tiles loaded so far, per slot
  int kv_fills;         // stages filled so far

  // Page of this lane's box of tile j: boxes of min(page, 128) rows, a lane
  // for each (box, 64-column half).
  __device__ int page_id(const Segment& s, int j) {
    const int box_rows = min(p.page, kTile);
    const int box = lane / (D / 64);
    const int key = j * kTile + box * box_rows;
    if (box * box_rows >= kTile || key >= s.keys) return -1;
    int pg = __ldg(s.pages + (key >> p.page_log2));
    if (pg < 0 || pg >= p.n_pages) {
      record_index(p.status, kInfoPage);
      pg = p.n_pages;  // out of range: the copy fills zeros
    }
    return pg;
  }
  __device__ bool load_kv(const CUtensorMap* tm, const Segment& s, int j, int pg) {
    if (!warp_wait(c, &c.kv_empty[ring.stage], ring.phase ^ 1u, p.status, kInfoAttnStage)) return false;
    const int box_rows = min(p.page, kTile);
    const int valid = min(kTile, s.keys - j * kTile);
    uint64_t* bar = &c.kv_full[ring.stage];
    uint8_t* dst = kv_mem + ring.stage * Geo::kTileBytes;
    if (lane == 0) mbar_arrive_expect_tx(bar, ((valid + box_rows - 1) / box_rows) * box_rows * D * 2);
    __syncwarp();
    if (pg >= 0) {
      const int box = lane / (D / 64), half = lane % (D / 64);
      const int row = box * box_rows;
      tma_load_4d(dst + half * (kTile * 128) + row * 128, tm, bar, half * 64, s.h, (j * kTile + row) & (p.page - 1),
                  pg);
    }
    ++kv_fills;
    if (++ring.stage == Geo::kStages) { ring.stage = 0; ring.phase ^= 1u; }
    return true;
  }
  // The query tile of a segment for `slot`: row tile `which` from its first.
  __device__ bool load_q(const Segment& s, int slot, int which) {
    const int n = q_fills[slot]++, buf = n % Geo::kQBufs;
    if (!warp_wait(c, &c.q_empty[slot][buf], ((n / Geo::kQBufs) & 1) ^ 1u, p.status, kInfoAttnQuery)) return false;
    if (lane == 0) {
      uint64_t* bar = &c.q_full[slot][buf];
      uint8_t* dst = q_mem + (slot * Geo::kQBufs + buf) * Geo::kTileBytes;
      mbar_arrive_expect_tx(bar, p.G * p.tpt * D * 2);
      for (int half = 0; half < D / 64; ++half)
        tma_load_4d(dst + half * (kTile * 128), tm_q, bar, half * 64, 0, s.h, s.tok0 + which * p.tpt);
    }
    __syncwarp();
    return true;
  }

  __device__ bool phase1() {
    Cursor u;
    u.w.begin1(p, c.prefix_len, blockIdx.x);
    u.start(p);
    if (!u.live) return true;
    int pg = page_id(u.s, u.j);
    if (!load_q(u.s, 0, 0) || !load_q(u.s, 1, 1) || !load_kv(tm_k, u.s, u.j, pg)) return false;
    while (u.live) {
      const Segment cur = u.s;
      const int j = u.j, pg_cur = pg;
      const bool fresh = u.last();
      u.step(p);
      if (u.live) pg = page_id(u.s, u.j);
      if (!load_kv(tm_v, cur, j, pg_cur)) return false;
      if (u.live) {
        if (fresh && (!load_q(u.s, 0, 0) || !load_q(u.s, 1, 1))) return false;
        if (!load_kv(tm_k, u.s, u.j, pg)) return false;
      }
    }
    return true;
  }
  __device__ bool phase2() {
    Cursor u[2];
    int pg[2] = {-1, -1};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      u[x].w.begin2(p, c.prefix_len, 2 * blockIdx.x + x, c.units[x], c.head[x], c.request[x], c.skip[x]);
      u[x].start(p);
      if (u[x].live) {
        pg[x] = page_id(u[x].s, u[x].j);
        if (!load_q(u[x].s, x, 0) || !load_kv(tm_k, u[x].s, u[x].j, pg[x])) return false;
      }
    }
    while (u[0].live || u[1].live) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!u[x].live) continue;
        const Segment cur = u[x].s;
        const int j = u[x].j, pg_cur = pg[x];
        const bool fresh = u[x].last();
        u[x].step(p);
        if (u[x].live) pg[x] = page_id(u[x].s, u[x].j);
        if (!load_kv(tm_v, cur, j, pg_cur)) return false;
        if (u[x].live) {
          if (fresh && !load_q(u[x].s, x, 0)) return false;
          if (!load_kv(tm_k, u[x].s, u[x].j, pg[x])) return false;
        }
      }
    }
    return true;
  }
  // Every copy that was issued has landed (also after a failure).
  __device__ void drain() {
    bool ok = true;
    for (int st = 0; st < Geo::kStages; ++st) {
      const int fills = kv_fills / Geo::kStages + (st < kv_fills % Geo::kStages ? 1 : 0);
      if (fills > 0) ok &= mbar_wait(&c.kv_full[st], (fills - 1) & 1, nullptr);
    }
    for (int slot = 0; slot < 2; ++slot)
      for (int b = 0; b < Geo::kQBufs; ++b) {
        const int fills = q_fills[slot] / Geo::kQBufs + (b < q_fills[slot] % Geo::kQBufs ? 1 : 0);
        if (fills > 0) ok &= mbar_wait(&c.q_full[slot][b], (fills - 1) & 1, nullptr);
      }
    if (!ok) record_failure(p.status, &c.abort_flag, kInfoAttnDrain);
  }
};

// ---------------------------------------------------------------- MMA issuer (warp 1)
template <bool kBf16, int D>
struct Issuer {
  using Geo = Geometry<D>;
  const AttnParams& p;
  Control& c;
  uint8_t* q_mem;
  uint8_t* kv_mem;
  uint32_t tmem;
  StageRing ring;
  int lane;
  int q_uses[2];         // query tiles taken so far, per slot
  int q_buf[2];          // buffer of the slot's current query tile
  uint32_t p_phase[2];   // parity of the slot's next P

  __device__ uint32_t idesc(int n) const { return kBf16 ? idesc_bf16(kTile, n) : idesc_f16(kTile, n); }

  __device__ bool wait_q(int slot) {
    const int n = q_uses[slot]++;
    q_buf[slot] = n % Geo::kQBufs;
    if (!warp_wait(c, &c.q_full[slot][q_buf[slot]], (n / Geo::kQBufs) & 1, p.status, kInfoAttnQuery)) return false;
    return true;
  }
  __device__ bool wait_stage(StageRing& at) {
    at = ring;
    if (++ring.stage == Geo::kStages) { ring.stage = 0; ring.phase ^= 1u; }
    if (!warp_wait(c, &c.kv_full[at.stage], at.phase, p.status, kInfoAttnStage)) return false;
    return true;
  }
  // S = Q K^T over the tile's keys (up to the next multiple of 16).
  __device__ void scores(int slot, int stage, int valid, bool release_q) {
    tc_fence_after();
    if (lane == 0) {
      const uint32_t id = idesc(((valid + 15) / 16) * 16);
      const uint32_t a = smem_u32(q_mem + (slot * Geo::kQBufs + q_buf[slot]) * Geo::kTileBytes);
      const uint32_t b = smem_u32(kv_mem + stage * Geo::kTileBytes);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t o = (ks / 4) * (kTile * 128) + (ks % 4) * 32;
        mma_bf16(tmem + slot * kTile, sw128_desc(a + o), sw128_desc(b + o), id, ks > 0 ? 1u : 0u);
      }
      mma_commit(&c.s_full[slot]);
      if (release_q) mma_commit(&c.q_empty[slot][q_buf[slot]]);
    }
    __syncwarp();
  }
  // Value rows from the last key to the next multiple of 16: zeros.
  __device__ void zero_tail(int stage, int valid) {
    const int end = ((valid + 15) / 16) * 16;
    uint8_t* v = kv_mem + stage * Geo::kTileBytes;
    for (int i = lane; i < (end - valid) * (D / 8); i += 32) {
      const int row = valid + i / (D / 8), ch = i % (D / 8);
      *reinterpret_cast<uint4*>(v + (ch / 8) * (kTile * 128) + row * 128 + (ch % 8) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async();
    __syncwarp();
  }
  // O (+)= P V.
  __device__ bool outputs(int slot, int stage, int valid, bool first, bool last) {
    if (!warp_wait(c, &c.p_full[slot], p_phase[slot], p.status, kInfoAttnProbs)) return false;
    p_phase[slot] ^= 1u;
    tc_fence_after();
    if (lane == 0) {
      const uint32_t id = idesc(D) | (1u << 16);  // B: N-major
      const uint32_t b = smem_u32(kv_mem + stage * Geo::kTileBytes);
      const int steps = (valid + 15) / 16;
      for (int ks = 0; ks < steps; ++ks)
        mma_ts(tmem + 2 * kTile + slot * kTile, tmem + slot * kTile + ks * 8, sw128_desc_mn(b + ks * 2048), id,
               (!first || ks > 0) ? 1u : 0u);
      if (last) mma_commit(&c.o_full[slot]);
    }
    __syncwarp();
    return true;
  }
  __device__ void release(int stage) {
    if (lane == 0) mma_commit(&c.kv_empty[stage]);
    __syncwarp();
  }

  __device__ bool phase1() {
    Cursor u;
    u.w.begin1(p, c.prefix_len, blockIdx.x);
    u.start(p);
    if (!u.live) return true;
    StageRing k, v;
    if (!wait_stage(k)) return false;
    for (int x = 0; x < 2; ++x) {
      if (!wait_q(x)) return false;
      scores(x, k.stage, u.valid(), u.last());
    }
    release(k.stage);
    while (u.live) {
      const bool first = u.j == u.s.j0, last = u.last();
      const int valid = u.valid();
      u.step(p);
      if (!wait_stage(v)) return false;
      if (valid % 16) zero_tail(v.stage, valid);
      if (!outputs(0, v.stage, valid, first, last)) return false;
      if (u.live) {
        if (last && !wait_q(0)) return false;
        if (!wait_stage(k)) return false;
        scores(0, k.stage, u.valid(), u.last());
      }
      if (!outputs(1, v.stage, valid, first, last)) return false;
      release(v.stage);
      if (u.live) {
        if (last && !wait_q(1)) return false;
        scores(1, k.stage, u.valid(), u.last());
        release(k.stage);
      }
    }
    return true;
  }
  __device__ bool phase2() {
    Cursor u[2];
    StageRing at;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      u[x].w.begin2(p, c.prefix_len, 2 * blockIdx.x + x, c.units[x], c.head[x], c.request[x], c.skip[x]);
      u[x].start(p);
      if (u[x].live) {
        if (!wait_q(x) || !wait_stage(at)) return false;
        scores(x, at.stage, u[x].valid(), u[x].last());
        release(at.stage);
      }
    }
    while (u[0].live || u[1].live) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!u[x].live) continue;
        const bool first = u[x].j == u[x].s.j0, last = u[x].last();
        const int valid = u[x].valid();
        u[x].step(p);
        if (!wait_stage(at)) return false;
        if (valid % 16) zero_tail(at.stage, valid);
        if (!outputs(x, at.stage, valid, first, last)) return false;
        release(at.stage);
        if (u[x].live) {
          if (last && !wait_q(x)) return false;
          if (!wait_stage(at)) return false;
          scores(x, at.stage, u[x].valid(), u[x].last());
          release(at.stage);
        }
      }
    }
    return true;
  }
};

// ---------------------------------------------------------------- softmax (one slot's 4 warps)
template <bool kBf16, int D>
struct Softmax {
  const AttnParams& p;
  Control& c;
  int slot, row;              // row of the tile: its tensor memory lane
  uint32_t s_tmem, o_tmem;    // this warp's lanes of the slot's S (and P) and O
  uint32_t s_phase, o_phase;

  __device__ bool wait(uint64_t* bar, uint32_t parity, int32_t info) {
    return warp_wait(c, bar, parity, p.status, info);
  }
  // One segment: rows of row tile `which` from the segment's first.
  __device__ bool run(const Segment& s, int which, float2* ml, float* o) {
    const int tok = s.tok0 + which * p.tpt + row / p.G;
    const bool valid_row = row < p.tpt * p.G && tok < s.tok_end;
    const int limit = s.own ? max(0, min(s.keys, s.lim0 + tok)) : s.keys;
    float m = -INFINITY, l = 0.f;
    for (int j = s.j0; j < s.j1; ++j) {
      if (!wait(&c.s_full[slot], s_phase, kInfoAttnScores)) return false;
      s_phase ^= 1u;
      tc_fence_after();
      uint32_t x[kTile];
#pragma unroll
      for (int i = 0; i < kTile / 32; ++i) tmem_ld32(s_tmem + 32 * i, x + 32 * i);
      tmem_ld_wait();
      const int seen = limit - j * kTile;
      if (__any_sync(0xffffffffu, seen < kTile)) {
#pragma unroll
        for (int i = 0; i < kTile; ++i)
          if (i >= seen) x[i] = 0xff800000u;  // -infinity
      }
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < kTile; ++i) top[i % 4] = fmaxf(top[i % 4], __uint_as_float(x[i]));
      const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2;
      const bool move = mt > m + kRescaleAt;  // also from -infinity
      if (__any_sync(0xffffffffu, move)) {
        const float m1 = move ? mt : m;
        const float a = move ? ex2(m - m1) : 1.f;
        m = m1;
        l *= a;
        if (j > s.j0) {
          // the slot's earlier products are complete: the same commit that
          // announced this S followed them
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t y[32];
            tmem_ld32(o_tmem + 32 * i, y);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * a);
            tmem_st32(o_tmem + 32 * i, y);
          }
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kTile / 2; ++i) {
        const float e0 = ex2(fmaf(__uint_as_float(x[2 * i]), p.scale_log2, -base));
        const float e1 = ex2(fmaf(__uint_as_float(x[2 * i + 1]), p.scale_log2, -base));
        sum[i % 2] += e0;
        sum[2 + i % 2] += e1;
        x[i] = pack2<kBf16>(e0, e1);
        if (i % 32 == 31) tmem_st32(s_tmem + (i - 31), x + (i - 31));
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&c.p_full[slot]);
    }
    if (!wait(&c.o_full[slot], o_phase, kInfoAttnOut)) return false;
    o_phase ^= 1u;
    tc_fence_after();
    const long long r = s.part_row + static_cast<long long>(which) * p.tpt * p.G + row;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t y[32];
      tmem_ld32(o_tmem + 32 * i, y);
      tmem_ld_wait();
      if (valid_row) {
        float4* dst = reinterpret_cast<float4*>(o + r * D + 32 * i);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          dst[k] = make_float4(__uint_as_float(y[4 * k]), __uint_as_float(y[4 * k + 1]), __uint_as_float(y[4 * k + 2]),
                               __uint_as_float(y[4 * k + 3]));
      }
    }
    if (valid_row) ml[r] = make_float2(m, l);
    return true;
  }
};

// The list position of both slots' phase 2 shares: a scan over the requests'
// units.  CTA 0 also leaves the scan for merge_kernel.
__device__ void find_shares(const AttnParams& p, Control& c, int plen) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kAttnThreads / 32;
  long long mine = 0, cost0 = 0;
  for (int b = tid; b < p.B; b += kAttnThreads) {
    const long long u = read_request(p, b).units(p);
    if (b == tid) cost0 = u;
    mine += u;
  }
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) c.sums[warp] = mine;
  __syncthreads();
  long long per_head = p.left ? units_of(tiles_of(plen)) : 0;
  const long long lead = per_head;
  for (int w = 0; w < kWarps; ++w) per_head += c.sums[w];
  __syncthreads();
  const long long total = per_head * p.Hkv;
  long long rem[2];
  for (int x = 0; x < 2; ++x) {
    const long long u0 = share_start(2 * blockIdx.x + x, total, 2 * p.ctas);
    const long long units = share_start(2 * blockIdx.x + x + 1, total, 2 * p.ctas) - u0;
    const int head = per_head > 0 ? static_cast<int>(u0 / per_head) : 0;
    rem[x] = units > 0 ? u0 - head * per_head - lead : -1;
    if (tid == 0) {
      c.units[x] = units;
      c.head[x] = head;
      if (rem[x] < 0) { c.request[x] = -1; c.skip[x] = units > 0 ? static_cast<int>(rem[x] + lead) : 0; }
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.plan->per_head = per_head;
    p.plan->prefix_tiles = tiles_of(plen);
  }
  long long base = 0;
  for (int b0 = 0; b0 < p.B; b0 += kAttnThreads) {
    const int b = b0 + tid;
    const long long u = b < p.B ? (b0 == 0 ? cost0 : read_request(p, b).units(p)) : 0;
    long long inc = u;
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) c.sums[warp] = inc;
    __syncthreads();
    long long before = base, all = base;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += c.sums[w];
      all += c.sums[w];
    }
    const long long first = before + inc - u;
    for (int x = 0; x < 2; ++x)
      if (b < p.B && rem[x] >= first && rem[x] < first + u) {
        c.request[x] = b;
        c.skip[x] = static_cast<int>(rem[x] - first);
      }
    if (blockIdx.x == 0 && b < p.B) p.first_unit[b] = first;
    base = all;
    __syncthreads();
  }
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
    prefix_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ AttnParams p) {
  using Geo = Geometry<D>;
  extern __shared__ uint8_t dynamic[];
  __shared__ Control c;
  uint8_t* q_mem = dynamic + ((1024u - (smem_u32(dynamic) & 1023u)) & 1023u);
  uint8_t* kv_mem = q_mem + 2 * Geo::kQBufs * Geo::kTileBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    c.abort_flag = 0;
    for (int s = 0; s < 2; ++s) {
      for (int b = 0; b < 2; ++b) { mbar_init(&c.q_full[s][b], 1); mbar_init(&c.q_empty[s][b], 1); }
      mbar_init(&c.s_full[s], 1);
      mbar_init(&c.p_full[s], kTile);
      mbar_init(&c.o_full[s], 1);
    }
    for (int s = 0; s < Geo::kStages; ++s) { mbar_init(&c.kv_full[s], 1); mbar_init(&c.kv_empty[s], 1); }
    mbar_init(&c.drain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  }
  griddep_wait();  // what the previous kernel on the stream wrote is visible
  const int plen = p.prefix_cap > 0 ? held(__ldg(p.prefix_len), p.prefix_cap, p.page, p.status) : 0;
  if (tid == 0) c.prefix_len = plen;
  find_shares(p, c, plen);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;

  if (warp == 0) {
    Producer<D> r{p, c, q_mem, kv_mem, &tm_q, &tm_k, &tm_v, StageRing(), lane, {0, 0}, 0};
    if (r.phase1()) r.phase2();
    if (lane == 0) r.drain();
  } else if (warp == 1) {
    Issuer<kBf16, D> r{p, c, q_mem, kv_mem, tmem, StageRing(), lane, {0, 0}, {0, 0}, {0, 0}};
    if (r.phase1()) r.phase2();
    // every MMA issued above has completed once `drain` flips
    if (lane == 0) {
      mma_commit(&c.drain);
      if (!mbar_wait(&c.drain, 0, nullptr)) record_failure(p.status, &c.abort_flag, kInfoAttnDrain);
    }
  } else if (warp >= 4) {
    const int slot = (warp - 4) / 4;
    const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
    Softmax<kBf16, D> r{p, c, slot, (warp % 4) * 32 + lane, tmem + slot * kTile + lanes,
                        tmem + 2 * kTile + slot * kTile + lanes, 0, 0};
    Walker w;
    Segment s;
    bool ok = true;
    w.begin1(p, plen, blockIdx.x);
    while (ok && w.next(p, s)) ok = r.run(s, slot, p.ml1, p.o1);
    w.begin2(p, plen, 2 * blockIdx.x + slot, c.units[slot], c.head[slot], c.request[slot], c.skip[slot]);
    while (ok && w.next(p, s)) ok = r.run(s, 0, p.ml2, p.o2);
  }
  griddep_launch_dependents();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- joining a row's parts
// One warp per (token, head).  A row's parts are the shares that hold tiles of
// its items: consecutive shares, those without units left out.
template <bool kBf16, int D>
__global__ void __launch_bounds__(128) merge_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kPer = D / 32;
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long row = blockIdx.x * 4ll + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(p.T) * p.Hq) return;
  const int t = static_cast<int>(row / p.Hq), hq = static_cast<int>(row % p.Hq), h = hq / p.G, g = hq % p.G;
  const long long per_head = p.plan->per_head, total2 = per_head * p.Hkv;
  const int ptiles = p.plan->prefix_tiles;

  // up to two runs of parts: the prefix item's, the request's
  const float2* ml[2] = {nullptr, nullptr};
  const float* o[2] = {nullptr, nullptr};
  long long first_row[2] = {0, 0}, total[2] = {1, 1};
  int first[2] = {0, 0}, last[2] = {-1, -1}, shares[2] = {1, 1}, stride[2] = {0, 0};
  // the request of token t: the last b with q_start[b] <= t
  int lo = 0, hi = p.B;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (__ldg(p.q_start + mid) <= t) lo = mid + 1; else hi = mid;
  }
  const int b = lo - 1;
  Request rq;
  rq.n = 0;
  if (b >= 0) rq = read_request(p, b);
  const bool owned = b >= 0 && t >= rq.a && t < rq.a + rq.n;
  if (owned && ptiles > 0) {
    const int rt = t / p.tpt;
    const long long per = units_of(ptiles);
    if (rt < 2 * p.pairs) {
      total[0] = per * p.pairs * p.Hkv; shares[0] = p.ctas; stride[0] = 2 * kTile;
      const long long u = (static_cast<long long>(h) * p.pairs + rt / 2) * per + kItemCost;
      first[0] = share_of(u, total[0], shares[0]);
      last[0] = share_of(u + ptiles - 1, total[0], shares[0]);
      first_row[0] = Walker::part_row(p, 1, h, t, false, 0) + g;
      ml[0] = p.ml1; o[0] = p.o1;
    } else {
      total[0] = total2; shares[0] = 2 * p.ctas; stride[0] = kTile;
      const long long u = h * per_head + kItemCost;
      first[0] = share_of(u, total2, shares[0]);
      last[0] = share_of(u + ptiles - 1, total2, shares[0]);
      first_row[0] = Walker::part_row(p, 2, h, t, false, 0) + g;
      ml[0] = p.ml2; o[0] = p.o2;
    }
  }
  if (owned) {
    const int rt = (t - rq.a) / p.tpt;
    const int tiles = tiles_of(rq.seen(p, rt));
    if (tiles > 0) {
      long long u = h * per_head + (p.left ? units_of(ptiles) : 0) + p.first_unit[b] + kItemCost;
      for (int i = 0; i < rt; ++i) u += units_of(tiles_of(rq.seen(p, i)));
      total[1] = total2; shares[1] = 2 * p.ctas; stride[1] = kTile;
      first[1] = share_of(u, total2, shares[1]);
      last[1] = share_of(u + tiles - 1, total2, shares[1]);
      first_row[1] = Walker::part_row(p, 2, h, t, true, 0) + g;
      ml[1] = p.ml2; o[1] = p.o2;
    }
  }
  float m = -INFINITY;
  for (int k = 0; k < 2; ++k)
    for (int w = first[k] + lane; w <= last[k]; w += 32)
      if (share_start(w + 1, total[k], shares[k]) > share_start(w, total[k], shares[k]))
        m = fmaxf(m, ml[k][first_row[k] + static_cast<long long>(stride[k]) * w].x);
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[kPer];
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
  for (int k = 0; k < 2; ++k)
    for (int w = first[k]; w <= last[k]; ++w) {
      if (share_start(w + 1, total[k], shares[k]) <= share_start(w, total[k], shares[k])) continue;
      const long long r = first_row[k] + static_cast<long long>(stride[k]) * w;
      const float2 part = ml[k][r];
      const float a = ex2(part.x - base);
      l += part.y * a;
      const float* src = o[k] + r * D + lane * kPer;
      for (int i = 0; i < kPer; ++i) acc[i] += a * src[i];
    }
  const float r = l > 0.f ? 1.f / l : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + row * D + lane * kPer);
  for (int i = 0; i < kPer / 2; ++i)
    dst[i] = l == 0.f ? 0u : pack2<kBf16>(acc[2 * i] * r, acc[2 * i + 1] * r);
  if (lane == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (base + log2f(l)) * 0.6931471805599453f;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// MOE_OK where a batch of this shape is within the kernels' limits.
moe_status shape_status(int T, int B, int Hq, int Hkv, int D) {
  if (T < 0 || B < 0 || Hq < 1 || Hkv < 1 || D < 1) return MOE_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return MOE_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || Hq / Hkv > kTile || Hq > 1024 || T > MOE_MAX_ATTN_TOKENS || B > MOE_MAX_REQUESTS)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Workspace after the fixed header: the plan, the requests' first units, the
// parts' (reference, sum) pairs and rows.
struct AttnLayout {
  int tpt, pairs, left;
  size_t o_plan, o_first, o_ml1, o_ml2, o_o1, o_o2, total;
};
AttnLayout attn_layout(int T, int B, int Hq, int Hkv, int D, int ctas) {
  AttnLayout L;
  L.tpt = kTile / (Hq / Hkv);
  const int row_tiles = ceil_div(T, L.tpt);
  L.pairs = row_tiles / 2;
  L.left = row_tiles % 2;
  const int l0 = L.left ? T - 2 * L.pairs * L.tpt : 0;
  const size_t rows1 = L.pairs ? static_cast<size_t>(T) * Hq + 2ull * kTile * ctas : 0;
  const size_t rows2 = (static_cast<size_t>(T) + l0) * Hq + 2ull * kTile * ctas;
  size_t o = kWsHeaderBytes;
  L.o_plan = o; o += kWsAlign;
  L.o_first = o; o += ws_align_up(8 * (static_cast<size_t>(B) + 1));
  L.o_ml1 = o; o += ws_align_up(8 * rows1);
  L.o_ml2 = o; o += ws_align_up(8 * rows2);
  L.o_o1 = o; o += ws_align_up(4 * rows1 * D);
  L.o_o2 = o; o += ws_align_up(4 * rows2 * D);
  L.total = o;
  return L;
}

cudaError_t launch_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, unsigned grid, int threads, size_t smem,
                          cudaStream_t s) {
  memset(cfg, 0, sizeof(*cfg));
  cfg->gridDim = dim3(grid);
  cfg->blockDim = dim3(threads);
  cfg->dynamicSmemBytes = smem;
  cfg->stream = s;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
  return cudaSuccess;
}

template <bool kBf16, int D>
cudaError_t launch(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnParams& p,
                   cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(prefix_attention_kernel<kBf16, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Geometry<D>::kDynamic);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  launch_config(&cfg, &attr, static_cast<unsigned>(p.ctas), kAttnThreads, Geometry<D>::kDynamic, s);
  e = cudaLaunchKernelEx(&cfg, prefix_attention_kernel<kBf16, D>, tm_q, tm_k, tm_v, p);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.T) * p.Hq + 3) / 4);
  launch_config(&cfg, &attr, grid, 128, 0, s);
  return cudaLaunchKernelEx(&cfg, merge_kernel<kBf16, D>, p);
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_prefix_attention_workspace_bytes(int T, int B, int Hq, int Hkv, int D) {
  using namespace moe;
  if (shape_status(T, B, Hq, Hkv, D) != MOE_OK) return 0;
  const int sms = device_sms();
  return sms > 0 ? attn_layout(T, B, Hq, Hkv, D, sms).total : 0;
}

moe_status moe_prefix_attention(const void* q, long long q_stride, int T, int B, const int32_t* q_start, int Hq,
                                int Hkv, int D, int dtype, const void* k_cache, const void* v_cache, int n_pages,
                                int page_size, const int32_t* prefix_pages, int prefix_cap, const int32_t* prefix_len,
                                const int32_t* page_table, int table_width, const int32_t* own_len, int causal,
                                float scale, void* out, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  using namespace moe;
  const moe_status st = shape_status(T, B, Hq, Hkv, D);
  if (st != MOE_OK) return st;
  if (n_pages < 0 || page_size < 1 || prefix_cap < 0 || table_width < 0) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return MOE_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale < INFINITY)) return MOE_ERR_INVALID_ARG;
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(prefix_cap) * page_size > MOE_MAX_KEYS ||
      static_cast<long long>(table_width) * page_size > MOE_MAX_KEYS)
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!q || !out || (T > 1 && q_stride < static_cast<long long>(Hq) * D)) return MOE_ERR_INVALID_ARG;
  if (B > 0 && !q_start) return MOE_ERR_INVALID_ARG;
  if (prefix_cap > 0 && (!prefix_pages || !prefix_len)) return MOE_ERR_INVALID_ARG;
  if (B > 0 && table_width > 0 && (!page_table || !own_len)) return MOE_ERR_INVALID_ARG;
  if (prefix_cap + table_width > 0 && (n_pages < 1 || !k_cache || !v_cache)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || q == out)
    return MOE_ERR_INVALID_ARG;
  if (q_stride % 8) return MOE_ERR_UNSUPPORTED;
  // a workspace that cannot even hold the fixed header is refused before any device query
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kWsAlign) != 0 || ws_bytes < kWsHeaderBytes) return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  const AttnLayout L = attn_layout(T, B, Hq, Hkv, D, sms);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  AttnParams p;
  memset(&p, 0, sizeof(p));
  p.T = T; p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.tpt = L.tpt;
  p.n_pages = n_pages; p.page = page_size;
  while ((1 << p.page_log2) < page_size) ++p.page_log2;
  p.q_start = q_start; p.prefix_pages = prefix_pages; p.prefix_len = prefix_len; p.page_table = page_table;
  p.own_len = own_len;
  p.prefix_cap = prefix_cap; p.table_width = table_width; p.causal = causal;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.ctas = sms; p.pairs = L.pairs; p.left = L.left;
  p.out = static_cast<uint16_t*>(out); p.lse = lse;
  char* w = static_cast<char*>(ws);
  p.status = reinterpret_cast<int32_t*>(w);
  p.plan = reinterpret_cast<Plan*>(w + L.o_plan);
  p.first_unit = reinterpret_cast<long long*>(w + L.o_first);
  p.ml1 = reinterpret_cast<float2*>(w + L.o_ml1); p.ml2 = reinterpret_cast<float2*>(w + L.o_ml2);
  p.o1 = reinterpret_cast<float*>(w + L.o_o1); p.o2 = reinterpret_cast<float*>(w + L.o_o2);
  // q as [T][key head][group][D], boxes of 64 columns x G heads x tpt tokens;
  // the caches as [page][slot][key head][D], boxes of 64 columns x one head x
  // up to 128 slots (without any page nothing is loaded: q stands in)
  const bool f16 = dtype == MOE_DTYPE_F16;
  CUtensorMap tm_q, tm_k, tm_v;
  const uint64_t hd = static_cast<uint64_t>(D);
  const uint64_t qd[4] = {hd, static_cast<uint64_t>(p.G), static_cast<uint64_t>(Hkv), static_cast<uint64_t>(T)};
  const uint64_t qs[3] = {hd * 2, hd * 2 * p.G, static_cast<uint64_t>(T > 1 ? q_stride : Hq * D) * 2};
  const uint32_t qb[4] = {64, static_cast<uint32_t>(p.G), 1, static_cast<uint32_t>(p.tpt)};
  const bool pages = prefix_cap + table_width > 0;
  const uint64_t kd[4] = {hd, static_cast<uint64_t>(Hkv), static_cast<uint64_t>(page_size),
                          static_cast<uint64_t>(pages ? n_pages : 1)};
  const uint64_t ks[3] = {hd * 2, hd * 2 * Hkv, hd * 2 * Hkv * page_size};
  const uint32_t kb[4] = {64, 1, static_cast<uint32_t>(page_size < kTile ? page_size : kTile), 1};
  if (!encode_map_16(&tm_q, f16, q, 4, qd, qs, qb) || !encode_map_16(&tm_k, f16, pages ? k_cache : q, 4, kd, ks, kb) ||
      !encode_map_16(&tm_v, f16, pages ? v_cache : q, 4, kd, ks, kb))
    return MOE_ERR_CUDA;
  const cudaError_t e = f16 ? (D == 64 ? launch<false, 64>(tm_q, tm_k, tm_v, p, stream)
                                       : launch<false, 128>(tm_q, tm_k, tm_v, p, stream))
                            : (D == 64 ? launch<true, 64>(tm_q, tm_k, tm_v, p, stream)
                                       : launch<true, 128>(tm_q, tm_k, tm_v, p, stream));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
