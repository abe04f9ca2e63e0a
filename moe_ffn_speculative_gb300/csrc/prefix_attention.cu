// Attention of a batch of requests whose cached context begins with one
// prefix that all of them share, followed by pages of their own
// (moe_prefix_attention).
//
// For the query of token t (the i-th of its request's n) and head h, over the
// prefix keys and the first `seen` of the request's own keys:
//   o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = scale log2(e) q . k_j,
// computed over tiles of 128 keys with a running reference m and running sums
// (fp32).  m is the row's maximum when it was last moved, less kLift; it moves
// only when a tile's maximum exceeds that maximum by more than 8 (f16: 7), so that
// the accumulator is rarely rescaled (the ratio is exact whatever m is).
//
// The powers enter the second product in the inputs' 16-bit type, as the MMA
// takes both operands in one type: one rounding of at most e/2 each, independent
// from key to key, beside the output's own (their sums l stay fp32, unrounded).
// Held in two halves they would lose nothing, at half as much tensor time again.
// bf16 has fp32's exponents.  f16 ends at 2^-24 and 65504, so there the maximum
// counts 2^7 (kLift) and no power passes 2^14 (two more bits are left for the
// rounding of logits past 2^24): a key is held to within 2^-32 of the row's
// largest, however many there are.  (With the maximum at 1, the bound was 2^-25:
// 131072 keys 17.4 nats below one lost all of their weight together, 0.36 %.)
//
// Work.  The G = Hq / Hkv heads of a token that read one key head are rows of
// one product, so a row tile is floor(128 / G) tokens x G heads (in phase 2
// floor(64 / G) where the blocks are that short: the query tiles then leave
// room for another stage of keys, and half of the MMA's rows are idle).
//   Phase 1: the prefix against pairs of row tiles of the whole batch: each key
//     tile is loaded once for 256 rows.
//   Phase 2: row tiles of one request's block against its own keys, and the
//     last row tile of the batch against the prefix when their number is odd.
// Each phase's list of (row tiles, key tile) steps, heads outermost, is cut
// into equal contiguous shares, an item counting kItemCost steps more than it
// has tiles.  The CTAs are divided between the phases by their work: a CTA of
// phase 1 takes one share, a CTA of phase 2 two, one for each of its slots (each
// with its own accumulator).  So a long context is split over the SMs, short
// ones are packed, and the arithmetic of the one phase runs beside the
// bandwidth of the other.  (When every CTA took a share of both, there were
// twice the parts to write and join: the 72-token verify step took 40 us.)
// Every (item, share) leaves its row sums, references and unnormalised fp32
// output rows in the workspace, and merge_kernel joins a row's parts in a fixed
// order: results do not depend on timing.
//
// A CTA (one per SM): warp 0 loads query, key and value tiles by TMA (a page
// is a box of its rows) into a ring of stages; warps 1 and 2 issue the two
// slots' MMAs, S = Q K^T with both from shared memory, then O += P V with P from
// tensor memory; warps 4..7 and 8..11 are the slots' softmax, one row a thread.  While one
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

#include <initializer_list>

#include "moe.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kTile = 128;           // keys of a tile, rows of a row tile
constexpr int kAttnThreads = 384;    // 12 warps
constexpr int kItemCost = 1;         // an item's fixed cost, in key tiles
// What the row's maximum counts when the reference is set, and how far a later
// tile's maximum may pass that (powers of two).
template <bool kBf16> constexpr float kLift = kBf16 ? 0.f : 7.f;
template <bool kBf16> constexpr float kRescaleAt = kBf16 ? 8.f : 7.f;
constexpr int kAttnSmem = 232448;    // 227 KB
// Registers a thread: 384 x 168 at launch, moved from warps 0..3 to the
// softmax warps, which hold a row's 128 scores (128 x (104 + 2 x 200) = 384 x 168)
constexpr int kRegsFew = 104, kRegsMany = 200;

struct AttnParams {
  int T, B, Hq, Hkv, G;
  int tpt, tpt2;                     // tokens of a row tile of phase 1, of phase 2
  int compact;                       // 1: phase 2's row tiles have at most 64 rows
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
  struct RequestPlan* requests;      // [B]
  int32_t* request_of;               // [T] the request of a token, or -1
  float2 *ml1, *ml2;                 // (reference, sum) of every part row, phases 1 and 2
  float4 *o1, *o2;                   // their fp32 rows (part_chunk)
};

// A list of units cut into equal shares: share w holds the units [start(w),
// start(w + 1)), the first `rest` shares one more than the others.  (Units are
// counted in 32 bits: the entry point refuses work that could exceed them.)
struct Shares {
  uint32_t each, rest;
  __host__ __device__ uint32_t start(uint32_t w) const { return w * each + (w < rest ? w : rest); }
  __host__ __device__ uint32_t of(uint32_t u) const {  // the share that holds unit u
    const uint32_t v = rest * (each + 1);
    return u < v ? u / (each + 1) : rest + (u - v) / each;
  }
};
__host__ __device__ inline Shares cut(uint32_t units, uint32_t shares) {
  return Shares{units / shares, units % shares};
}

struct Plan {
  uint32_t per_head;                 // phase 2 units of one head
  int prefix_tiles;
  Shares s1, s2;
};
// CTAs of phase 1.  A unit of it keeps a CTA busy for about 2500 clocks, one of
// phase 2 (two slots at a time) for 0.75 as long and 0.028 more for every box
// that a tile is copied in.  (64 requests over 16384 shared keys, pages of 64,
// 0.75 + 0.028 x 2 boxes: 153.7 us, 0.82 + 0.014 x: 155.4, 0.6 and 1 alone, before
// the loads got faster: 182, 170.  Draft blocks over 30011, pages of 16: 64.6,
// 65.7.)
__device__ __forceinline__ int ctas_of_phase1(uint32_t units1, uint32_t units2, int ctas, int page) {
  if (units1 == 0) return 0;
  if (units2 == 0) return ctas;
  const float cost = 0.75f + 0.028f * static_cast<float>(page < kTile ? kTile / page : 1);
  const float u1 = static_cast<float>(units1), u2 = cost * static_cast<float>(units2);
  const int c = __float2int_rn(static_cast<float>(ctas) * u1 / (u1 + u2));
  return max(1, min(ctas - 1, c));
}
// A request as merge_kernel reads it.
struct __align__(16) RequestPlan {
  int a, n, len;         // first token, tokens, own keys
  uint32_t first_unit;   // units of a head's list before it
};

// ---------------------------------------------------------------- geometry
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
  __device__ int seen(const AttnParams& p, int rt) const {
    if (!p.causal) return len;
    const int last = min(n, (rt + 1) * p.tpt2);
    return max(0, min(len, len - n + last));
  }
  __device__ int row_tiles(const AttnParams& p) const { return (n + p.tpt2 - 1) / p.tpt2; }
  __device__ uint32_t units(const AttnParams& p) const {
    uint32_t u = 0;
    const int k = row_tiles(p);
    if (!p.causal) return static_cast<uint32_t>(k) * units_of(tiles_of(len));
    for (int rt = 0; rt < k; ++rt) u += units_of(tiles_of(seen(p, rt)));
    return u;
  }
};

// (Not inlined, as what runs once a launch is bound by fetching its code.)
__device__ __noinline__ Request read_request(const AttnParams& p, int b) {
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

// One share's run through one item: a slot's row tile against key tiles
// [j0, j1).
struct Segment {
  int phase;                 // 0: the list has ended
  int h, tok0, tok_end;      // key head, first token of the row tile, end of valid tokens
  int keys;                  // keys that any of its rows sees
  int own, lim0;             // own keys: token t sees min(keys, max(0, lim0 + t)) of them (causal)
  int j0, j1;
  const int32_t* pages;
  long long part_row;        // part row of token tok0, head h * G
};

// Walks a share's segments.
struct Walker {
  int phase, share;
  uint32_t left;   // units still to walk
  int off;         // units of the current item before the share
  int h, i, rt;    // phase 1: h, pair i; phase 2: h, request i (-1: the prefix item), row tile rt
  int batch;       // requests that are served
  Request rq;
  int prefix_len, prefix_tiles;

  // Phase 1, share c.
  __device__ void begin1(const AttnParams& p, int plen, const Shares& sh, int c) {
    phase = 1; share = c; prefix_len = plen; prefix_tiles = tiles_of(plen);
    const uint32_t u0 = sh.start(c);
    left = sh.start(c + 1) - u0;
    const uint32_t per = units_of(prefix_tiles), item = u0 / per;
    off = static_cast<int>(u0 - item * per);
    h = static_cast<int>(item / p.pairs);
    i = static_cast<int>(item) - h * p.pairs;
    rt = 0;
  }
  // Phase 2, share w; the list position of its first unit was found by the
  // scan of the requests.
  __device__ void begin2(const AttnParams& p, int plen, int w, uint32_t units, int head, int request, int skip,
                         int served) {
    phase = 2; share = w; batch = served; prefix_len = plen; prefix_tiles = tiles_of(plen);
    left = units; h = head; i = request; rt = 0; off = skip;
    if (left > 0 && i >= 0) rq = read_request(p, i);
  }
  __device__ void next_request(const AttnParams& p) {
    rt = 0;
    if (++i >= batch) { i = -1; ++h; }
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
      const int room = units - off;
      if (room > 0) {
        const int take = left < static_cast<uint32_t>(room) ? static_cast<int>(left) : room;
        s.phase = phase;
        s.h = h;
        s.j0 = max(off - kItemCost, 0);
        s.j1 = off + take - kItemCost;
        if (prefix) {
          s.tok0 = (phase == 1 ? 2 * i : 2 * p.pairs) * p.tpt;
          s.tok_end = p.T;
          s.keys = prefix_len; s.own = 0; s.lim0 = 0;
          s.pages = p.prefix_pages;
        } else {
          s.tok0 = rq.a + rt * p.tpt2;
          s.tok_end = rq.a + rq.n;
          s.keys = rq.seen(p, rt); s.own = p.causal; s.lim0 = rq.len - rq.n - rq.a + 1;
          s.pages = p.page_table + static_cast<long long>(i) * p.table_width;
        }
        s.part_row = part_row(p, phase, h, s.tok0, !prefix, share);
        left -= take;
        off += take;
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

// Part rows lie in blocks of 32, four elements of every row together, so that a
// warp whose lanes are rows writes 512 bytes at a time: place of elements
// [4 c, 4 c + 4) of part row r, in float4s.
template <int D>
__device__ __forceinline__ long long part_chunk(long long r, int c) {
  return ((r >> 5) * (D / 4) + c) * 32 + (r & 31);
}

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
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The same with A from tensor memory: its rows lanes, two 16-bit values a column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\ttcgen05.mma.cta_group::1."
      "kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of a B operand whose N dimension is contiguous (value rows:
// 64 columns of one key in 128 bytes, 128-byte swizzle): 8-key groups 1024
// bytes apart, 64-column blocks kTile * 128 bytes apart.
constexpr uint32_t kDescLoN = static_cast<uint32_t>((kTile * 128) >> 4) << 16;  // lower word (kDescHi the upper)
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
// The larger of three, and two fp32 operations in one instruction.
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
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
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
  // 2 KB for the control words, 1 KB to align the tiles
  static constexpr int kSpace = (kAttnSmem - 2048 - 1024) / kTileBytes * kTileBytes;
  static constexpr int kDynamic = 1024 + kSpace;
};
// Shared memory of a CTA: the query tiles (whole, or 64 rows each), then as many
// stages of keys and values as fit.
template <int D>
struct Room {
  int q_bytes, q_half;  // of a query tile, and of its 64-column half
  int stages;
  __device__ explicit Room(bool compact) {
    using Geo = Geometry<D>;
    q_bytes = compact ? Geo::kTileBytes / 2 : Geo::kTileBytes;
    q_half = q_bytes / (D / 64);
    stages = (Geo::kSpace - 2 * Geo::kQBufs * q_bytes) / Geo::kTileBytes;
  }
};

// Key and value tiles land in a ring of stages in the order that the producer
// chose; a slot's issuer finds its n-th tile through these.  At most 16 stages
// are in use, so an entry is free again by the time it is written.
constexpr int kSequence = 16;
// A slot's segments pass from the planner to its 6 readers (producer, issuer,
// four softmax warps) through a window of this many.
constexpr int kSegments = 4;
constexpr int kReaders = 6;
constexpr int kPagesAtOnce = 8;  // pages whose copies are issued together

struct Control {
  uint64_t q_full[2][2], q_empty[2][2];
  uint64_t kv_full[2][kSequence];  // per slot: its n-th tile has landed
  uint64_t kv_empty[16];
  uint64_t s_full[2], p_full[2], o_full[2], drain[2];
  uint64_t turn[2];                // the slot may issue
  int ended[2];                    // the slot's issuer takes no more turns
  uint64_t seg_full[2][kSegments], seg_empty[2][kSegments];
  Segment seg[2][kSegments];
  int stage_of[2][kSequence];      // where the slot's n-th tile is
  uint32_t tmem;
  int abort_flag;
  uint32_t sums[kAttnThreads / 32];
  // the CTA's phase and (first) share; of phase 2, each slot's units and place
  int phase, share;
  Shares s1;
  uint32_t units[2];
  int head[2], request[2], skip[2];
  int batch;                       // requests that are served
  unsigned long long claimed;      // tokens, where some starts are out of order
};

__device__ __forceinline__ bool warp_wait(Control& c, uint64_t* bar, uint32_t parity, int32_t* status, int32_t info) {
  const bool ok = mbar_wait(bar, parity, &c.abort_flag);
  if (__all_sync(0xffffffffu, ok)) return true;
  if ((threadIdx.x & 31) == 0) record_failure(status, &c.abort_flag, info);
  return false;
}
// The slot's n-th segment.
__device__ __forceinline__ bool take(Control& c, int slot, int& n, Segment& s, int32_t* status) {
  const int e = n % kSegments;
  if (!warp_wait(c, &c.seg_full[slot][e], (n / kSegments) & 1, status, kInfoAttnList)) return false;
  s = c.seg[slot][e];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&c.seg_empty[slot][e]);
  ++n;
  return true;
}
// Keys of tile j that some row of the segment sees.
__device__ __forceinline__ int valid_keys(const Segment& s, int j) { return min(kTile, s.keys - j * kTile); }

// ---------------------------------------------------------------- TMA producer (warp 0)
// The lanes wait and walk together; one of them issues.  A tile's pages are read
// a lane each while the tile before is loaded, and go to the issuing lane by
// shuffle, kPagesAtOnce before its copies.  (Draft blocks over pages of 16: 78.5,
// 73.2, 67.2, 64.6 us with 1, 2, 4, 8; a single thread that read pages in pairs
// ahead of their copies took 76.5.)
// One copy of the load serves both slots, keys and values: a slot's state is
// selected, not unrolled, since this warp is bound by fetching its code (with
// six inlined copies a load took it 1300 clocks, and the own keys' bandwidth
// was that).
template <int D>
struct Producer {
  using Geo = Geometry<D>;
  const AttnParams& p;
  Control& c;
  uint8_t* q_mem;
  uint8_t* kv_mem;
  const CUtensorMap *tm_q, *tm_k, *tm_v;
  Room<D> room;
  int box_rows;     // rows of a box: a page's, up to a tile's
  int q_tokens;     // tokens of a query tile
  Ring ring;
  int q_fills0, q_fills1;    // query tiles loaded so far, per slot
  int kv_fills0, kv_fills1;  // tiles announced so far, per slot
  int lane;
  bool bad;                  // this lane saw a page outside the cache

  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int32_t info) {
    return warp_wait(c, bar, parity, p.status, info);
  }
  // The slot's n-th segment, read where it lies until it is released.
  __device__ __forceinline__ const Segment* take(int slot, int n) {
    if (!wait(&c.seg_full[slot][n % kSegments], (n / kSegments) & 1, kInfoAttnList)) return nullptr;
    return &c.seg[slot][n % kSegments];
  }
  __device__ __forceinline__ void release(int slot, int n) {
    __syncwarp();
    if (elect()) mbar_arrive(&c.seg_empty[slot][n % kSegments]);
  }
  // Pages outside the cache become the first one past it: the copy fills zeros.
  __device__ __forceinline__ int page_at(const int32_t* pages, int i) {
    const uint32_t pg = static_cast<uint32_t>(__ldg(pages + i)), n = static_cast<uint32_t>(p.n_pages);
    bad |= pg >= n;
    return static_cast<int>(min(pg, n));
  }
  __device__ __forceinline__ int boxes(int keys, int j) const {
    return (min(kTile, keys - j * kTile) + box_rows - 1) / box_rows;
  }
  // The pages of tile j, a lane each (pages have 8 keys or more: 16 at most).
  __device__ __forceinline__ int pages_of(const Segment* s, int j) {
    return lane < boxes(s->keys, j) ? page_at(s->pages + ((j * kTile) >> p.page_log2), lane) : 0;
  }
  // The next tile of `slot` (in phase 1, of both: announced to slot 0): a box
  // for each page and 64-column half.
  __device__ __forceinline__ bool load_kv(const CUtensorMap* tm, const Segment* s, int j, int slot, int pages) {
    if (!wait(&c.kv_empty[ring.stage], ring.phase ^ 1u, kInfoAttnStage)) return false;
    const int n = boxes(s->keys, j), h = s->h, fills = slot ? kv_fills1++ : kv_fills0++, entry = fills % kSequence;
    uint64_t* bar = &c.kv_full[slot][entry];
    uint8_t* dst = kv_mem + ring.stage * Geo::kTileBytes;
    if (elect()) {
      c.stage_of[slot][entry] = ring.stage;
      mbar_arrive_expect_tx(bar, n * box_rows * D * 2);
    }
    const int row = (j * kTile) & (p.page - 1), step = box_rows * 128;
#pragma unroll 1
    for (int i = 0; i < n; i += kPagesAtOnce) {
      int page[kPagesAtOnce];
#pragma unroll
      for (int k = 0; k < kPagesAtOnce; ++k) page[k] = __shfl_sync(0xffffffffu, pages, i + k);
      if (elect()) {
#pragma unroll
        for (int k = 0; k < kPagesAtOnce; ++k) {
          if (i + k >= n) break;
#pragma unroll
          for (int half = 0; half < D / 64; ++half)
            tma_load_4d(dst + half * (kTile * 128) + k * step, tm, bar, half * 64, h, row, page[k]);
        }
      }
      dst += kPagesAtOnce * step;
    }
    ring.next(room.stages);
    return true;
  }
  __device__ __forceinline__ bool load_q(const Segment* s, int slot) {
    const int n = slot ? q_fills1++ : q_fills0++, buf = n % Geo::kQBufs;
    if (!wait(&c.q_empty[slot][buf], ((n / Geo::kQBufs) & 1) ^ 1u, kInfoAttnQuery)) return false;
    uint64_t* bar = &c.q_full[slot][buf];
    uint8_t* dst = q_mem + (slot * Geo::kQBufs + buf) * room.q_bytes;
    if (elect()) {
      mbar_arrive_expect_tx(bar, p.G * q_tokens * D * 2);
#pragma unroll
      for (int half = 0; half < D / 64; ++half)
        tma_load_4d(dst + half * room.q_half, tm_q, bar, half * 64, 0, s->h, s->tok0);
    }
    return true;
  }

  // In turn, each slot's values of tile j and keys of tile j + 1 (the first
  // time, only the keys of its first).  In phase 1 slot 0's tiles serve both,
  // whose segments differ in their row tile only.
  __device__ __forceinline__ bool run(bool phase2) {
    int n0 = 0, n1 = 0, j0 = -1, j1 = -1;      // segment and tile of each slot (-1: none yet)
    int pages0 = 0, pages1 = 0;                // the tile's pages
    bool live0 = true, live1 = phase2;
#pragma unroll 1
    for (int x = 0; live0 || live1; x = phase2 ? x ^ 1 : 0) {
      if (!(x ? live1 : live0)) continue;
      int n = x ? n1 : n0, j = x ? j1 : j0;
      const Segment* s = &c.seg[x][n % kSegments];
      bool fresh = j < 0;
      int next = 0;  // the next tile's pages, under way during this one's values
      if (!fresh) {
        const bool more = j + 1 < s->j1;
        if (more) next = pages_of(s, j + 1);
        if (!load_kv(tm_v, s, j, x, x ? pages1 : pages0)) return false;
        ++j;
        if (!more) {
          release(x, n);
          if (!phase2) release(1, n);
          ++n;
          fresh = true;
        }
      }
      bool ended = false;
      if (fresh) {
        if ((s = take(x, n)) == nullptr) return false;
        const Segment* other = s;
        if (!phase2 && (other = take(1, n)) == nullptr) return false;
        ended = s->phase == 0;
        if (!ended) {
          j = s->j0;
          next = pages_of(s, j);
          if (!load_q(s, x) || (!phase2 && !load_q(other, 1))) return false;
        }
      }
      if (!ended && !load_kv(tm_k, s, j, x, next)) return false;
      if (bad) {
        bad = false;
        record_index(p.status, kInfoPage);
      }
      if (x) { n1 = n; j1 = j; pages1 = next; live1 = !ended; }
      else { n0 = n; j0 = j; pages0 = next; live0 = !ended; }
    }
    return true;
  }
  // Every copy that was issued has landed (also after a failure).
  __device__ void drain() {
    bool ok = true;
#pragma unroll 1
    for (int slot = 0; slot < 2; ++slot) {
      const int kv = slot ? kv_fills1 : kv_fills0, q = slot ? q_fills1 : q_fills0;
#pragma unroll 1
      for (int e = 0; e < kSequence; ++e) {
        const int fills = kv / kSequence + (e < kv % kSequence ? 1 : 0);
        if (fills > 0) ok &= mbar_wait(&c.kv_full[slot][e], (fills - 1) & 1, nullptr);
      }
#pragma unroll 1
      for (int b = 0; b < Geo::kQBufs; ++b) {
        const int fills = q / Geo::kQBufs + (b < q % Geo::kQBufs ? 1 : 0);
        if (fills > 0) ok &= mbar_wait(&c.q_full[slot][b], (fills - 1) & 1, nullptr);
      }
    }
    if (!ok) record_failure(p.status, &c.abort_flag, kInfoAttnDrain);
  }
};

// ---------------------------------------------------------------- MMA issuers (warps 1 and 2, one a slot)
// A slot's MMAs in the order S(0), O(0), S(1), O(1), ...: S(j + 1) overwrites
// P(j), which O(j), issued just before by the same thread, has read.  The
// slots take turns of O(j), S(j + 1): left to themselves their MMAs mix, both
// slots' scores come at the same time, and the tensor cores idle while both
// compute their probabilities.
template <bool kBf16, int D>
struct Issuer {
  using Geo = Geometry<D>;
  const AttnParams& p;
  Control& c;
  uint32_t q_lo, kv_lo;  // lower descriptor words of the slot's first query tile and of stage 0
  uint32_t q_tile, q_half;  // from one query tile to the next, from one half of it to the other
  uint32_t s_tmem;       // the slot's S (and P); O lies 2 tiles further
  int slot;
  int q_uses, seen;      // query tiles and key/value tiles taken so far
  uint32_t p_phase;      // parity of the slot's next P
  uint32_t turn_phase;   // parity of the slot's next turn
  bool mine;             // the first turn is slot 0's without a wait
  bool alone;            // the other slot has ended

  __device__ __forceinline__ uint32_t idesc(int n) const { return kBf16 ? idesc_bf16(kTile, n) : idesc_f16(kTile, n); }

  // The next tile announced to `sequence`: its stage, or -1.
  __device__ __forceinline__ int wait_stage(int sequence) {
    const int e = seen % kSequence;
    if (!warp_wait(c, &c.kv_full[sequence][e], (seen / kSequence) & 1, p.status, kInfoAttnStage)) return -1;
    ++seen;
    return *reinterpret_cast<volatile int*>(&c.stage_of[sequence][e]);
  }
  __device__ __forceinline__ bool begin_turn() {
    if (alone) return true;
    if (!mine) {
      if (!warp_wait(c, &c.turn[slot], turn_phase, p.status, kInfoAttnTurn)) return false;
      turn_phase ^= 1u;
    }
    mine = false;
    alone = *static_cast<volatile int*>(&c.ended[slot ^ 1]) != 0;
    return true;
  }
  // kv_empty counts two users: both slots in phase 1, one (an arrival at once,
  // the other with its last MMA) in phase 2.
  __device__ __forceinline__ void release(int stage, bool both) {
    if (!both) mbar_arrive(&c.kv_empty[stage]);
    mma_commit(&c.kv_empty[stage]);
  }
  // Value rows from the last key to the next multiple of 16: zeros.  (In
  // phase 1 both slots' issuers write the same zeros.)
  __device__ void zero_tail(uint8_t* v, int valid) {
    const int end = ((valid + 15) / 16) * 16;
    for (int i = threadIdx.x & 31; i < (end - valid) * (D / 8); i += 32) {
      const int row = valid + i / (D / 8), ch = i % (D / 8);
      *reinterpret_cast<uint4*>(v + (ch / 8) * (kTile * 128) + row * 128 + (ch % 8) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async();
    __syncwarp();
  }
  // One tile's operands of S, all waited for: its query buffer and stage.
  struct Keys {
    int q_buf, stage, valid;
    bool both, last;  // both slots' stage; the segment's last tile
  };
  __device__ __forceinline__ bool wait_keys(Keys& k, const Segment& s, int j) {
    k.both = s.phase == 1;  // phase 1's tiles are announced to slot 0
    k.valid = valid_keys(s, j);
    k.last = j + 1 == s.j1;
    if (j == s.j0) {
      if (!warp_wait(c, &c.q_full[slot][q_uses % Geo::kQBufs], (q_uses / Geo::kQBufs) & 1, p.status, kInfoAttnQuery))
        return false;
      ++q_uses;
    }
    k.q_buf = (q_uses - 1) % Geo::kQBufs;
    k.stage = wait_stage(k.both ? 0 : slot);
    return k.stage >= 0;
  }
  // S = Q K^T over the tile's keys (up to the next multiple of 16), by one
  // thread.  The turn ends while the last products are still queued: the other
  // slot's follow them without a gap.
  __device__ __forceinline__ void scores(const Keys& k) {
    const uint32_t id = idesc(((k.valid + 15) / 16) * 16);
    const uint32_t a = kDescLoK + q_lo + k.q_buf * q_tile;
    const uint32_t b = kDescLoK + kv_lo + k.stage * (Geo::kTileBytes / 16);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      mma_ss(s_tmem, a + (ks / 4) * q_half + (ks % 4) * 2, kDescHi,
             b + (ks / 4) * (kTile * 128 / 16) + (ks % 4) * 2, kDescHi, id, ks > 0 ? 1u : 0u);
      if (ks == D / 16 - 4 && !alone) mbar_arrive(&c.turn[slot ^ 1]);
    }
    mma_commit(&c.s_full[slot]);
    release(k.stage, k.both);
    if (k.last) mma_commit(&c.q_empty[slot][k.q_buf]);
  }
  // O (+)= P V, by one thread.
  __device__ __forceinline__ void outputs(const Keys& k, int stage, bool first) {
    const uint32_t id = idesc(D) | (1u << 16);  // B: N-major
    const uint32_t b = kDescLoN + kv_lo + stage * (Geo::kTileBytes / 16);
    const uint32_t d = s_tmem + 2 * kTile;
    const int steps = (k.valid + 15) / 16;
    if (steps == kTile / 16) {
#pragma unroll
      for (int ks = 0; ks < kTile / 16; ++ks)
        mma_ts(d, s_tmem + ks * 8, b + ks * (2048 / 16), kDescHi, id, ks > 0 ? 1u : first ? 0u : 1u);
    } else {
      for (int ks = 0; ks < steps; ++ks)
        mma_ts(d, s_tmem + ks * 8, b + ks * (2048 / 16), kDescHi, id, ks > 0 || !first ? 1u : 0u);
    }
    if (k.last) mma_commit(&c.o_full[slot]);
    release(stage, k.both);
  }

  __device__ __forceinline__ bool walk(uint8_t* kv_mem) {
    Segment u;
    Keys cur, next;
    int n = 0;
    if (!take(c, slot, n, u, p.status)) return false;
    if (u.phase == 0) return true;
    int j = u.j0;
    if (!wait_keys(cur, u, j) || !begin_turn()) return false;
    tc_fence_after();
    if (elect()) scores(cur);
    __syncwarp();
    while (true) {
      // all of the turn's operands are there before it begins
      const int stage = wait_stage(cur.both ? 0 : slot);
      if (stage < 0) return false;
      const bool first = j == u.j0;
      if (cur.valid % 16) zero_tail(kv_mem + stage * Geo::kTileBytes, cur.valid);
      ++j;
      if (cur.last) {
        if (!take(c, slot, n, u, p.status)) return false;
        j = u.j0;
      }
      const bool more = u.phase != 0;
      if (more && !wait_keys(next, u, j)) return false;
      // the turn first: it usually comes while the probabilities are computed
      if (!begin_turn()) return false;
      if (!warp_wait(c, &c.p_full[slot], p_phase, p.status, kInfoAttnProbs)) return false;
      p_phase ^= 1u;
      tc_fence_after();
      if (elect()) {
        outputs(cur, stage, first);
        if (more) scores(next);
      }
      __syncwarp();
      if (!more) return true;
      cur = next;
    }
  }
  __device__ __forceinline__ void run(uint8_t* kv_mem) {
    walk(kv_mem);
    // the turn, if it is this slot's or comes to it, is the other's from here on
    if (elect()) {
      *static_cast<volatile int*>(&c.ended[slot]) = 1;
      mbar_arrive(&c.turn[slot ^ 1]);
    }
    __syncwarp();
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
  __device__ __forceinline__ bool segment(const Segment& s) {
    const int tok = s.tok0 + row / p.G;
    const bool valid_row = row < (s.phase == 1 ? p.tpt : p.tpt2) * p.G && tok < s.tok_end;
    const int limit = s.own ? max(0, min(s.keys, s.lim0 + tok)) : s.keys;
    // a warp without a valid row (a block of few tokens) only keeps step
    const bool idle = !__any_sync(0xffffffffu, valid_row);
    float m = -INFINITY, l = 0.f;
    for (int j = s.j0; j < s.j1; ++j) {
      if (!wait(&c.s_full[slot], s_phase, kInfoAttnScores)) return false;
      s_phase ^= 1u;
      if (idle) {
        mbar_arrive(&c.p_full[slot]);
        continue;
      }
      tc_fence_after();
      uint32_t x[kTile];
#pragma unroll
      for (int i = 0; i < kTile / 32; ++i) tmem_ld32(s_tmem + 32 * i, x + 32 * i);
      tmem_ld_wait();
      const int seen = limit - j * kTile;
      if (__any_sync(0xffffffffu, seen < kTile)) {
#pragma unroll
        for (int i = 0; i < kTile; i += 32)
          if (__any_sync(0xffffffffu, seen < i + 32)) {
#pragma unroll
            for (int k = i; k < i + 32; ++k)
              if (k >= seen) x[k] = 0xff800000u;  // -infinity
          }
      }
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < kTile; i += 2)
        top[(i / 2) % 4] = max3(top[(i / 2) % 4], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
      const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2;
      const bool move = mt > m + (kLift<kBf16> + kRescaleAt<kBf16>);  // also from -infinity
      if (__any_sync(0xffffffffu, move)) {
        const float m1 = move ? mt - kLift<kBf16> : m;
        const float a = move ? ex2(m - m1) : 1.f;
        m = m1;
        l *= a;
        if (j > s.j0) {
          // the slot's earlier products are complete: the same commit that
          // announced this S followed them
#pragma unroll 1
          for (int i = 0; i < D / 16; ++i) {
            uint32_t y[16];
            tmem_ld16(o_tmem + 16 * i, y);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * a);
            tmem_st16(o_tmem + 16 * i, y);
          }
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      const unsigned long long scale2 = pair(p.scale_log2, p.scale_log2), base2 = pair(-base, -base);
      unsigned long long sum[2] = {0ull, 0ull};  // two zeros each
#pragma unroll
      for (int i = 0; i < kTile / 2; ++i) {
        float e0, e1;
        unpair(fma2(pair(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), scale2, base2), e0, e1);
        e0 = ex2(e0);
        e1 = ex2(e1);
        sum[i % 2] = add2(sum[i % 2], pair(e0, e1));
        x[i] = pack2<kBf16>(e0, e1);
        if (i % 16 == 15) tmem_st16(s_tmem + (i - 15), x + (i - 15));
      }
      float s0, s1;
      unpair(add2(sum[0], sum[1]), s0, s1);
      l += s0 + s1;
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&c.p_full[slot]);
    }
    if (!wait(&c.o_full[slot], o_phase, kInfoAttnOut)) return false;
    o_phase ^= 1u;
    tc_fence_after();
    const long long r = s.part_row + row;
    float4* dst = (s.phase == 1 ? p.o1 : p.o2) + part_chunk<D>(r, 0);
#pragma unroll 1  // what runs once a segment is bound by fetching its code
    for (int i = 0; i < D / 32; ++i) {
      uint32_t y[32];
      tmem_ld32(o_tmem + 32 * i, y);
      tmem_ld_wait();
      if (valid_row) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          dst[32 * (8 * i + k)] = make_float4(__uint_as_float(y[4 * k]), __uint_as_float(y[4 * k + 1]),
                                       __uint_as_float(y[4 * k + 2]), __uint_as_float(y[4 * k + 3]));
      }
    }
    if (valid_row) (s.phase == 1 ? p.ml1 : p.ml2)[r] = make_float2(m, l);
    return true;
  }
  __device__ __forceinline__ void run() {
    Segment s;
    int n = 0;
    while (take(c, slot, n, s, p.status) && s.phase != 0)
      if (!segment(s)) return;
  }
};

// ---------------------------------------------------------------- planner (warp 3)
// Both slots' places in the phase 2 list: a scan over the requests' units by
// the whole CTA (a warp alone takes longer even over 8 requests).  What
// merge_kernel needs of it goes to the workspace.  Starts out of order anywhere
// may leave blocks that overlap: where they claim more than the T tokens that the
// entry point counted units for, no request is served.
__device__ __forceinline__ void find_shares(const AttnParams& p, Control& c, int plen) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kAttnThreads / 32;
  const uint32_t lead = p.left ? units_of(tiles_of(plen)) : 0;  // the prefix item comes first
  uint32_t mine = 0, cost0 = 0;
  int tokens = 0;  // (T of each of 65536 / 384 requests, at most)
  bool ok = true;
  for (int b = tid; b < p.B; b += kAttnThreads) {
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
  const uint32_t per_head = lead + all, units1 = units_of(tiles_of(plen)) * p.pairs * p.Hkv;
  const int c1 = ctas_of_phase1(units1, per_head * p.Hkv, p.ctas, p.page);
  const Shares s1 = cut(units1, max(c1, 1)), s2 = cut(per_head * p.Hkv, max(2 * (p.ctas - c1), 1));
  if (blockIdx.x == 0 && tid == 0) *p.plan = Plan{per_head, tiles_of(plen), s1, s2};
  // where each slot's phase 2 share begins in its head's list; below `lead`:
  // inside the prefix item
  const int w0 = 2 * (static_cast<int>(blockIdx.x) - c1);
  uint32_t at[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const uint32_t u0 = w0 >= 0 ? s2.start(w0 + x) : 0, units = w0 >= 0 ? s2.start(w0 + x + 1) - u0 : 0;
    const uint32_t head = units > 0 ? u0 / per_head : 0;
    at[x] = units > 0 ? u0 - head * per_head : 0xffffffffu;
    if (tid == 0) {
      c.units[x] = units;
      c.head[x] = static_cast<int>(head);
      c.request[x] = -1;
      c.skip[x] = static_cast<int>(at[x]);
    }
  }
  if (tid == 0) {
    c.s1 = s1;
    c.share = w0 < 0 ? static_cast<int>(blockIdx.x) : w0;
    c.phase = w0 < 0 ? 1 : 2;
    c.batch = batch;
  }
  uint32_t base = lead;
  for (int b0 = 0; b0 < p.B; b0 += kAttnThreads) {
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
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (at[x] >= first && at[x] - first < own) {
        c.request[x] = b;
        c.skip[x] = static_cast<int>(at[x] - first);
      }
    if (b < p.B && b % p.ctas == static_cast<int>(blockIdx.x)) {
      const Request rq = read_request(p, b);
      p.requests[b] = RequestPlan{rq.a, b < batch ? rq.n : 0, rq.len, first};
    }
  }
}

// Hands a slot's list over, a segment whenever its readers have made room.
// (Lane x is slot x: neither slot waits for the other.)
__device__ __forceinline__ void hand_list(const AttnParams& p, Control& c, int slot, int plen) {
  Walker w;
  Segment s;
  int n = 0;
  bool have = false;
  if (c.phase == 1) w.begin1(p, plen, c.s1, c.share);
  else w.begin2(p, plen, c.share + slot, c.units[slot], c.head[slot], c.request[slot], c.skip[slot],
               c.batch);
  long long t0 = clock64();
  while (true) {
    if (!have) {
      if (!w.next(p, s)) s.phase = 0;
      if (s.phase == 1 && slot == 1) {  // the pair's second row tile
        s.tok0 += p.tpt;
        s.part_row += static_cast<long long>(p.tpt) * p.G;
      }
      have = true;
    }
    const int e = n % kSegments;
    if (mbar_test_wait(&c.seg_empty[slot][e], ((n / kSegments) & 1) ^ 1u)) {
      c.seg[slot][e] = s;
      mbar_arrive(&c.seg_full[slot][e]);
      if (s.phase == 0) return;
      ++n;
      have = false;
      t0 = clock64();
    } else {
      if (*static_cast<volatile int*>(&c.abort_flag)) return;
      if (clock64() - t0 > kWaitLimitCycles) {
        record_failure(p.status, &c.abort_flag, kInfoAttnList);
        return;
      }
      __nanosleep(64);
    }
  }
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
    prefix_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q2,
                            const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const __grid_constant__ AttnParams p) {
  using Geo = Geometry<D>;
  extern __shared__ uint8_t dynamic[];
  __shared__ Control c;
  uint8_t* q_mem = dynamic + ((1024u - (smem_u32(dynamic) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    c.abort_flag = 0;
    for (int s = 0; s < 2; ++s) {
      for (int b = 0; b < 2; ++b) { mbar_init(&c.q_full[s][b], 1); mbar_init(&c.q_empty[s][b], 1); }
      mbar_init(&c.s_full[s], 1);
      mbar_init(&c.p_full[s], kTile);
      mbar_init(&c.o_full[s], 1);
      mbar_init(&c.turn[s], 1);
      c.ended[s] = 0;
    }
    for (int s = 0; s < 2 * kSegments; ++s) {
      mbar_init(&c.seg_full[s / kSegments][s % kSegments], 1);
      mbar_init(&c.seg_empty[s / kSegments][s % kSegments], kReaders);
    }
    for (int s = 0; s < kSequence; ++s) { mbar_init(&c.kv_full[0][s], 1); mbar_init(&c.kv_full[1][s], 1); }
    for (int s = 0; s < kSequence; ++s) mbar_init(&c.kv_empty[s], 2);
    mbar_init(&c.drain[0], 1);
    mbar_init(&c.drain[1], 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_q2);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  }
  // merge_kernel's blocks may be placed as this grid's leave (they wait for all
  // of it)
  griddep_launch_dependents();
  griddep_wait();  // what the previous kernel on the stream wrote is visible
  const int plen = p.prefix_cap > 0 ? held(__ldg(p.prefix_len), p.prefix_cap, p.page, p.status) : 0;
  find_shares(p, c, plen);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  const bool phase2 = c.phase == 2;
  const Room<D> room(phase2 && p.compact);
  uint8_t* kv_mem = q_mem + 2 * Geo::kQBufs * room.q_bytes;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp == 0) {
      Producer<D> r{p,    c,    q_mem, kv_mem, phase2 ? &tm_q2 : &tm_q, &tm_k, &tm_v, room, min(p.page, kTile),
                    phase2 ? p.tpt2 : p.tpt, Ring(), 0, 0, 0, 0, lane, false};
      r.run(phase2);
      r.drain();
    } else if (warp <= 2) {
      const int slot = warp - 1;
      Issuer<kBf16, D> r{p, c, smem_u32(q_mem + slot * Geo::kQBufs * room.q_bytes) >> 4, smem_u32(kv_mem) >> 4,
                         static_cast<uint32_t>(room.q_bytes) >> 4, static_cast<uint32_t>(room.q_half) >> 4,
                         tmem + slot * kTile, slot, 0, 0, 0, 0u, slot == 0, false};
      r.run(kv_mem);
      // every MMA issued above has completed once `drain` flips
      if (elect()) {
        mma_commit(&c.drain[slot]);
        if (!mbar_wait(&c.drain[slot], 0, nullptr)) record_failure(p.status, &c.abort_flag, kInfoAttnDrain);
      }
    } else if (warp == 3) {
      if (lane < 2) hand_list(p, c, lane, plen);
      __syncwarp();
      // the tokens' requests, for merge_kernel: every CTA writes some
#pragma unroll 1
      for (int b = blockIdx.x; b < c.batch; b += p.ctas) {
        const Request rq = read_request(p, b);
        for (int t = lane; t < rq.n; t += 32) p.request_of[rq.a + t] = b;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
    const int slot = (warp - 4) / 4;
    const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
    Softmax<kBf16, D> r{p, c, slot, (warp % 4) * 32 + lane, tmem + slot * kTile + lanes,
                        tmem + 2 * kTile + slot * kTile + lanes, 0, 0};
    r.run();
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
// kWarps warps per token and two of a key head's rows, which lie next to each
// other in every part: lane l takes row l % 2 and the row's elements from 4 (l /
// 2), so that it reads whole sectors.  A row's parts are the shares that hold
// tiles of its items: consecutive shares.  They are independent loads, so a part
// costs little more than its bytes; the fewer rows a call has, the more parts
// each has, and the more warps take it.
struct Parts {
  const float2* ml;
  const float4* o;
  long long row;  // part row of share 0
  int first, count, stride;
  __device__ long long at(int i) const { return row + static_cast<long long>(stride) * (first + i); }
};

constexpr int merge_threads(int warps) { return warps > 4 ? 32 * warps : 128; }

template <bool kBf16, int D, int kWarps>
__global__ void __launch_bounds__(merge_threads(kWarps)) merge_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kChunks = D / 64;  // of four elements, a lane
  constexpr int kUnits = merge_threads(kWarps) / 32 / kWarps;  // of a block
  __shared__ float2 ml_all[kWarps][2];
  __shared__ float4 acc_all[kWarps][kChunks][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part_warp = warp % kWarps, sub = lane & 1;
  const int pairs = (p.G + 1) / 2;
  const long long unit = static_cast<long long>(blockIdx.x) * kUnits + warp / kWarps;
  if (unit >= static_cast<long long>(p.T) * p.Hkv * pairs) return;  // whole blocks where kWarps > 1
  const int t = static_cast<int>(unit / (p.Hkv * pairs)), hp = static_cast<int>(unit % (p.Hkv * pairs));
  const int h = hp / pairs, g = 2 * (hp % pairs);
  const bool two = g + 1 < p.G;
  griddep_wait();
  const uint32_t per_head = p.plan->per_head;
  const int ptiles = p.plan->prefix_tiles;
  const Shares s1 = p.plan->s1, s2 = p.plan->s2;
  const int b = p.B > 0 ? p.request_of[t] : -1;
  RequestPlan rp = {0, 0, 0, 0};
  // (a token outside every request reads what an earlier call left: checked)
  if (b >= 0 && b < p.B) rp = p.requests[b];
  const bool owned = t >= rp.a && t < rp.a + rp.n;
  const Request rq = {rp.a, rp.n, rp.len, true};
  Parts run[2];  // the prefix item's parts, the request's
  run[0].count = run[1].count = 0;
  if (owned && ptiles > 0) {
    const int rt = t / p.tpt;
    const bool paired = rt < 2 * p.pairs;
    Parts& r = run[0];
    r.ml = paired ? p.ml1 : p.ml2;
    r.o = paired ? p.o1 : p.o2;
    r.stride = paired ? 2 * kTile : kTile;
    const Shares sh = paired ? s1 : s2;
    const uint32_t u = (paired ? (h * p.pairs + rt / 2) * units_of(ptiles) : h * per_head) + kItemCost;
    r.first = sh.of(u);
    r.count = sh.of(u + ptiles - 1) - r.first + 1;
    r.row = Walker::part_row(p, paired ? 1 : 2, h, t, false, 0) + g;
  }
  if (owned) {
    const int rt = (t - rq.a) / p.tpt2;
    const int tiles = tiles_of(rq.seen(p, rt));
    if (tiles > 0) {
      uint32_t u = h * per_head + rp.first_unit + kItemCost;
      for (int i = 0; i < rt; ++i) u += units_of(tiles_of(rq.seen(p, i)));
      Parts& r = run[1];
      r.ml = p.ml2; r.o = p.o2; r.stride = kTile;
      r.first = s2.of(u);
      r.count = s2.of(u + tiles - 1) - r.first + 1;
      r.row = Walker::part_row(p, 2, h, t, true, 0) + g;
    }
  }
  // of both rows: reference and sum; of this lane's: its elements
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float4 acc[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const Parts r = run[k];
#pragma unroll 1
    for (int i0 = 0; i0 < r.count; i0 += 32 * kWarps) {
      // lane i: this warp's i-th part of the chunk
      const int i = i0 + lane * kWarps + part_warp;
      const long long at = i < r.count ? r.at(i) : -1;
      float mine[2], old[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float2 ml = at >= 0 && (x == 0 || two) ? r.ml[at + x] : make_float2(-INFINITY, 0.f);
        float top = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float m1 = fmaxf(m[x], top), base = m1 == -INFINITY ? 0.f : m1;
        old[x] = ex2(m[x] - base);
        mine[x] = ex2(ml.x - base);
        m[x] = m1;
        float sum = mine[x] * ml.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[x] = l[x] * old[x] + sum;
      }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const float f = sub ? old[1] : old[0];
        acc[c].x *= f; acc[c].y *= f; acc[c].z *= f; acc[c].w *= f;
      }
      const int count = min(32, (r.count - i0 - part_warp + kWarps - 1) / kWarps);
#pragma unroll 8
      for (int x = 0; x < count; ++x) {
        const long long row = __shfl_sync(0xffffffffu, at, x) + (two ? sub : 0);
        const float a0 = __shfl_sync(0xffffffffu, mine[0], x), a1 = __shfl_sync(0xffffffffu, mine[1], x);
        const float a = sub ? a1 : a0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const float4 v = __ldcg(r.o + part_chunk<D>(row, lane / 2 + 16 * c));
          acc[c].x += a * v.x; acc[c].y += a * v.y; acc[c].z += a * v.z; acc[c].w += a * v.w;
        }
      }
    }
  }
  if (kWarps > 1) {
    if (lane < 2) ml_all[warp][lane] = make_float2(m[lane], l[lane]);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) acc_all[warp][c][lane] = acc[c];
    __syncthreads();
    if (warp != 0) return;
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml_all[w][sub].x);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < kWarps; ++w) {
      const float a = ex2(ml_all[w][sub].x - base);
      sum += a * ml_all[w][sub].y;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const float4 v = acc_all[w][c][lane];
        acc[c].x += a * v.x; acc[c].y += a * v.y; acc[c].z += a * v.z; acc[c].w += a * v.w;
      }
    }
    m[0] = m[1] = top;
    l[0] = l[1] = sum;
  }
  if (sub && !two) return;
  const float top = sub ? m[1] : m[0], sum = sub ? l[1] : l[0];
  const float base = top == -INFINITY ? 0.f : top;
  const float f = sum > 0.f ? 1.f / sum : 0.f;
  const long long row = static_cast<long long>(t) * p.Hq + h * p.G + g + sub;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const float4 v = acc[c];
    const uint2 out = sum == 0.f ? make_uint2(0u, 0u)
                                 : make_uint2(pack2<kBf16>(v.x * f, v.y * f), pack2<kBf16>(v.z * f, v.w * f));
    *reinterpret_cast<uint2*>(p.out + row * D + 4 * (lane / 2 + 16 * c)) = out;
  }
  if (lane < 2 && p.lse) p.lse[row] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
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

// Workspace after the fixed header: the plan, the requests, the tokens' requests, the
// parts' (reference, sum) pairs and rows.
struct AttnLayout {
  int tpt, tpt2, compact, pairs, left;
  size_t o_plan, o_req, o_of, o_ml1, o_ml2, o_o1, o_o2, total;
};
AttnLayout attn_layout(int T, int B, int Hq, int Hkv, int D, int ctas) {
  AttnLayout L;
  const int G = Hq / Hkv;
  L.tpt = kTile / G;
  // phase 2 in tiles of 64 rows (and another stage for keys) where the requests'
  // blocks have that many on average: longer ones would read their keys twice as
  // often.  us in tiles of 64 / 128: 64 x 9 tokens, 2000 own keys, G = 4: 113.0 /
  // 114.4; 16 x 20: 54.0 / 47.7; 4 x 256: 89.7 / 64.9
  L.compact = G <= kTile / 2 && static_cast<long long>(T) * G <= kTile / 2 * static_cast<long long>(B) ? 1 : 0;
  L.tpt2 = L.compact ? kTile / 2 / G : L.tpt;
  const int row_tiles = ceil_div(T, L.tpt);
  L.pairs = row_tiles / 2;
  L.left = row_tiles % 2;
  if (L.left && T - 2 * L.pairs * L.tpt > L.tpt2) {  // too long for phase 2: a pair with an empty second tile
    ++L.pairs;
    L.left = 0;
  }
  const int l0 = L.left ? T - 2 * L.pairs * L.tpt : 0;
  const size_t rows1 = L.pairs ? static_cast<size_t>(T) * Hq + 2ull * kTile * ctas : 0;
  const size_t rows2 = (static_cast<size_t>(T) + l0) * Hq + 2ull * kTile * ctas;
  size_t o = kWsHeaderBytes;
  L.o_plan = o; o += kWsAlign;
  L.o_req = o; o += ws_align_up(sizeof(RequestPlan) * static_cast<size_t>(B));
  L.o_of = o; o += ws_align_up(4 * static_cast<size_t>(T));
  L.o_ml1 = o; o += ws_align_up(8 * rows1);
  L.o_ml2 = o; o += ws_align_up(8 * rows2);
  L.o_o1 = o; o += ws_align_up(4 * ((rows1 + 31) / 32 * 32) * D);
  L.o_o2 = o; o += ws_align_up(4 * ((rows2 + 31) / 32 * 32) * D);
  L.total = o;
  return L;
}

// Bytes that serve every call of at most T tokens and B requests of these heads:
// attn_layout with the terms that T, B and their ratio move either way (the pairs,
// the last row tile's tokens) at their largest.
size_t attn_bytes_upto(int T, int B, int Hq, int Hkv, int D, int ctas) {
  const int tpt = kTile / (Hq / Hkv);
  const size_t spare = 2ull * kTile * ctas;
  const size_t rows1 = static_cast<size_t>(T) * Hq + spare;
  const size_t rows2 = (static_cast<size_t>(T) + (T < tpt ? T : tpt)) * Hq + spare;
  size_t o = kWsHeaderBytes + kWsAlign + ws_align_up(sizeof(RequestPlan) * static_cast<size_t>(B)) +
             ws_align_up(4 * static_cast<size_t>(T));
  for (const size_t rows : {rows1, rows2}) o += ws_align_up(8 * rows) + ws_align_up(4 * ((rows + 31) / 32 * 32) * D);
  return o;
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
cudaError_t launch(const CUtensorMap& tm_q, const CUtensorMap& tm_q2, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                   const AttnParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(prefix_attention_kernel<kBf16, D>, Geometry<D>::kDynamic, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  launch_config(&cfg, &attr, static_cast<unsigned>(p.ctas), kAttnThreads, Geometry<D>::kDynamic, s);
  e = cudaLaunchKernelEx(&cfg, prefix_attention_kernel<kBf16, D>, tm_q, tm_q2, tm_k, tm_v, p);
  if (e != cudaSuccess) return e;
  // warps a unit of two rows: more while the units leave the SMs room for them.
  // us of both launches with 1, 4, 8 warps: 9 tokens over 4096 keys (144 units)
  // 53.0, 27.0, 21.0; 8 x 9 tokens (1152 units) 40.7, 31.0, 36.9; 64 x 9 (9216)
  // 155, 177, 233
  const long long units = static_cast<long long>(p.T) * p.Hkv * ((p.G + 1) / 2);
  if (units <= 4ll * p.ctas) {
    launch_config(&cfg, &attr, static_cast<unsigned>(units), merge_threads(8), 0, s);
    return cudaLaunchKernelEx(&cfg, merge_kernel<kBf16, D, 8>, p);
  }
  if (units <= 16ll * p.ctas) {
    launch_config(&cfg, &attr, static_cast<unsigned>(units), merge_threads(4), 0, s);
    return cudaLaunchKernelEx(&cfg, merge_kernel<kBf16, D, 4>, p);
  }
  launch_config(&cfg, &attr, static_cast<unsigned>((units + 3) / 4), merge_threads(1), 0, s);
  return cudaLaunchKernelEx(&cfg, merge_kernel<kBf16, D, 1>, p);
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_prefix_attention_workspace_bytes(int T, int B, int Hq, int Hkv, int D) {
  using namespace moe;
  if (shape_status(T, B, Hq, Hkv, D) != MOE_OK) return 0;
  const int sms = device_sms();
  return sms > 0 ? attn_bytes_upto(T, B, Hq, Hkv, D, sms) : 0;
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
  // units of both phases' lists, at most, in 31 bits
  {
    const long long tpt = kTile / (Hq / Hkv), row_tiles = 2 * ((T + tpt - 1) / tpt) + 2;
    const long long pt = tiles_of(prefix_cap * page_size) + kItemCost, ot = tiles_of(table_width * page_size) + kItemCost;
    if ((row_tiles * pt + (row_tiles + B) * ot) * Hkv >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
  }
  if (!q || !out || (T > 1 && q_stride < static_cast<long long>(Hq) * D)) return MOE_ERR_INVALID_ARG;
  if (B > 0 && !q_start) return MOE_ERR_INVALID_ARG;
  if (prefix_cap > 0 && (!prefix_pages || !prefix_len)) return MOE_ERR_INVALID_ARG;
  if (B > 0 && table_width > 0 && (!page_table || !own_len)) return MOE_ERR_INVALID_ARG;
  if (prefix_cap + table_width > 0 && (n_pages < 1 || !k_cache || !v_cache)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || q == out)
    return MOE_ERR_INVALID_ARG;
  if (q_stride % 8) return MOE_ERR_UNSUPPORTED;
  const long long row = 2ll * Hq * D, pool = prefix_cap + table_width > 0 ? 2ll * n_pages * page_size * Hkv * D : 0;
  const RowSet o = {out, 1, row * T, 0}, z = {lse, 1, 4ll * T * Hq, 0};
  for (const RowSet& read : {RowSet{q, T, row, 2 * q_stride}, RowSet{k_cache, 1, pool, 0}, RowSet{v_cache, 1, pool, 0}})
    if (rows_meet(o, read) || rows_meet(z, read)) return MOE_ERR_INVALID_ARG;
  if (rows_meet(o, z)) return MOE_ERR_INVALID_ARG;
  // a workspace that cannot even hold the fixed header is refused before any device query
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kWsAlign) != 0 || ws_bytes < kWsHeaderBytes) return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  const AttnLayout L = attn_layout(T, B, Hq, Hkv, D, sms);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  AttnParams p;
  memset(&p, 0, sizeof(p));
  p.T = T; p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv;
  p.tpt = L.tpt; p.tpt2 = L.tpt2; p.compact = L.compact;
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
  p.requests = reinterpret_cast<RequestPlan*>(w + L.o_req);
  p.request_of = reinterpret_cast<int32_t*>(w + L.o_of);
  p.ml1 = reinterpret_cast<float2*>(w + L.o_ml1); p.ml2 = reinterpret_cast<float2*>(w + L.o_ml2);
  p.o1 = reinterpret_cast<float4*>(w + L.o_o1); p.o2 = reinterpret_cast<float4*>(w + L.o_o2);
  // q as [T][key head][group][D], boxes of 64 columns x G heads x tpt tokens;
  // the caches as [page][slot][key head][D], boxes of 64 columns x one head x
  // up to 128 slots (without any page nothing is loaded: q stands in)
  const bool f16 = dtype == MOE_DTYPE_F16;
  CUtensorMap tm_q, tm_q2, tm_k, tm_v;
  const uint64_t hd = static_cast<uint64_t>(D);
  const uint64_t qd[4] = {hd, static_cast<uint64_t>(p.G), static_cast<uint64_t>(Hkv), static_cast<uint64_t>(T)};
  const uint64_t qs[3] = {hd * 2, hd * 2 * p.G, static_cast<uint64_t>(T > 1 ? q_stride : Hq * D) * 2};
  const uint32_t qb[4] = {64, static_cast<uint32_t>(p.G), 1, static_cast<uint32_t>(p.tpt)};
  const uint32_t qb2[4] = {64, static_cast<uint32_t>(p.G), 1, static_cast<uint32_t>(p.tpt2)};
  const bool pages = prefix_cap + table_width > 0;
  const uint64_t kd[4] = {hd, static_cast<uint64_t>(Hkv), static_cast<uint64_t>(page_size),
                          static_cast<uint64_t>(pages ? n_pages : 1)};
  const uint64_t ks[3] = {hd * 2, hd * 2 * Hkv, hd * 2 * Hkv * page_size};
  const uint32_t kb[4] = {64, 1, static_cast<uint32_t>(page_size < kTile ? page_size : kTile), 1};
  if (!encode_map_16(&tm_q, f16, q, 4, qd, qs, qb) || !encode_map_16(&tm_q2, f16, q, 4, qd, qs, qb2) ||
      !encode_map_16(&tm_k, f16, pages ? k_cache : q, 4, kd, ks, kb) ||
      !encode_map_16(&tm_v, f16, pages ? v_cache : q, 4, kd, ks, kb))
    return MOE_ERR_CUDA;
  const cudaError_t e = f16 ? (D == 64 ? launch<false, 64>(tm_q, tm_q2, tm_k, tm_v, p, stream)
                                       : launch<false, 128>(tm_q, tm_q2, tm_k, tm_v, p, stream))
                            : (D == 64 ? launch<true, 64>(tm_q, tm_q2, tm_k, tm_v, p, stream)
                                       : launch<true, 128>(tm_q, tm_q2, tm_k, tm_v, p, stream));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
