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
// A CTA (one per SM): warp 0 copies tiles (a page of a head is one run of bytes), warps
// 1 and 2 issue the first and the second products' MMAs, warp 3 walks the list; warps 4..7
// expand keys, 8..23 are the softmax, 24..27 expand values.  Every role's code is a short
// loop: with few warps of a role on a scheduler, what is unrolled runs at the rate at which
// it is fetched (a tile took 1.7 times as long with the four groups of the expansion
// unrolled).
//
// Measured: 8 blocks of 9 tokens over 4096 shared keys and up to 900 own ones 29.0 us (2 more
// when it signalled its joining launch early); 13 blocks of 8 over 30011, D = 64, 78 us; 64
// blocks of 9 over 16384 and up to 2000, 347 us, 2250 clocks a tile of 64 rows.  Of those,
// without the expansion of keys 316, without that of values 307, without the second product
// 331, without exponentials 343; without any of them 255: what is left is one role waiting
// for another, at some ten clocks an instruction.  A second warpgroup for the values'
// expansion (338), one for the keys' (360) or issue by whole warps were no faster throughout.
//
// Keys past a length are never read as numbers: their codes are replaced by zeros, and
// their scores before the maximum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include <initializer_list>

#include "attention_kv4.cuh"
#include "issue.cuh"
#include "kv4.cuh"
#include "moe.h"

namespace moe {
namespace {

constexpr int kThreads = 896;
constexpr int kSoftGroups = 4;   // of the softmax, four warps each
constexpr int kSmem = 232448;    // 227 KB
constexpr int kMaxStages = 12;
constexpr int kSegments = 4;
constexpr int kReaders = kThreads / 32 - 1;  // of a segment: every warp but the one that walks
// Registers a thread, moved between the warpgroups: 3 x 56 + 4 x 80 <= 7 x 72
constexpr int kRegsFew = 56, kRegsSoftmax = 80;

// ---------------------------------------------------------------- tensor memory, MMA
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
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
// The four warps of a softmax group: do any of their threads say yes?
__device__ __forceinline__ bool softmax_any(int group, bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, "
      "q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(mine)), "r"(2 + group)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void softmax_sync(int group) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(2 + group) : "memory");
}

// ---------------------------------------------------------------- shared memory
template <int D>
struct Geometry {
  static constexpr int kGroups = D / 32;
  static constexpr int kStageBytes = kTile * kv4_slot_bytes(D);
  static constexpr int kValueBytes = kTile * D * 2, kProbBytes = kTile * kRows * 2, kQueryBytes = kRows * D * 2;
  static constexpr int kValuesAt = 0, kProbsAt = 2 * kValueBytes, kQueriesAt = kProbsAt + 2 * kProbBytes;
  static constexpr int kRingAt = kQueriesAt + kQueryBytes;
  static constexpr int kFit = (kSmem - 4096 - 1024 - kRingAt) / kStageBytes;  // 4 KB for the control words
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kDynamic = 1024 + kRingAt + kStages * kStageBytes;
  // tensor memory: two expanded key tiles, two score tiles, two output tiles
  static constexpr uint32_t kKeysCol = 0, kScoresCol = D, kOutCol = D + 2 * kRows;
};

struct Control {
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
  uint64_t k_full[2], k_empty[2], s_full[2], s_empty[2], v_full[2], v_empty[2], p_full[2], p_empty[2];
  uint64_t q_full, o_full[2], o_empty[2], drain[2];
  uint64_t seg_full[kSegments], seg_empty[kSegments];
  Segment seg[kSegments];
  uint32_t tmem;
  int abort_flag;
  // of a segment's rows: score scale and keys seen, with the queries
  alignas(16) float row_scale[2][kRows];
  alignas(16) int row_limit[2][kRows];
  // of the softmax: the reference, its negative (0 for none), the factor of a move, the warps'
  // maxima (and sums, at a segment's end)
  alignas(16) float neg[kRows];
  float m[kRows], factor[kRows];
  float top[4][kRows];
  Start start;
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
template <int D>
struct Producer {
  using Geo = Geometry<D>;
  const Kv4Attn& p;
  Control& c;
  uint8_t* ring_mem;
  Ring ring;
  int filled;
  int lane;

  __device__ __forceinline__ bool load(const Segment& s, int j, int page) {
    if (!warp_wait(c, &c.kv_empty[ring.stage], ring.phase ^ 1u, p.status, kInfoAttnStage)) return false;
    copy_keys<D, kTile>(p, s, j * kTile, page, ring_mem + ring.stage * Geo::kStageBytes, &c.kv_full[ring.stage], lane);
    ++filled;
    ring.next(Geo::kStages);
    return true;
  }
  __device__ void run() {
    Segment s;
    int n = 0;
    while (take(c, n, s, p.status) && s.live) {
      Pages<kTile> pages;
      pages.begin(p, s, lane);
      for (int j = s.j0; j < s.j1; ++j)
        if (!load(s, j, pages.of(p, j * kTile, lane))) return;
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

// ---------------------------------------------------------------- expansion (warps 4..7 and 24..27)
// A thread a key: its codes of one kind, as f16.
template <int D, bool kValues>
__device__ __forceinline__ void expand(const Kv4Attn& p, Control& c, const uint8_t* ring_mem, uint8_t* v_mem, uint32_t tmem) {
  using Geo = Geometry<D>;
  const int key = threadIdx.x & 127;
  const int local = min(p.page, kTile), log2 = min(p.page_log2, 7), at = key & (local - 1);
  // places of the key's codes and scales in a stage
  const int base = (key >> log2) * local * kv4_slot_bytes(D);
  const uint8_t* codes_at = ring_mem + base + kv4_codes_at(D, local, kValues) + at * 16;
  const uint8_t* scales_at = ring_mem + base + kv4_scales_at(D, local, kValues) + at * Geo::kGroups;
  // where its f16 go: shared memory (a key a row of 128 bytes, swizzled), or columns of its lane
  uint8_t* row0 = kValues ? v_mem + key * 128 : nullptr;
  const uint32_t cols0 = tmem + Geo::kKeysCol + (static_cast<uint32_t>(((threadIdx.x >> 5) & 3) * 32) << 16);
  Segment s;
  Ring ring;
  int n = 0, i = 0;
  while (take(c, n, s, p.status) && s.live) {
    for (int j = s.j0; j < s.j1; ++j, ++i, ring.next(Geo::kStages)) {
      const int buf = i & 1;
      uint64_t *full = kValues ? &c.v_full[buf] : &c.k_full[buf], *empty = kValues ? &c.v_empty[buf] : &c.k_empty[buf];
      uint8_t* row = row0 + buf * Geo::kValueBytes;
      const uint32_t cols = cols0 + buf * (D / 2);
      if (!warp_wait(c, &c.kv_full[ring.stage], ring.phase, p.status, kInfoAttnStage)) return;
      const uint8_t* codes = codes_at + ring.stage * Geo::kStageBytes;
      const uint8_t* st = scales_at + ring.stage * Geo::kStageBytes;
      uint32_t scales;
      if (Geo::kGroups == 4) scales = *reinterpret_cast<const uint32_t*>(st);
      else scales = *reinterpret_cast<const uint16_t*>(st);
      uint4 w = *reinterpret_cast<const uint4*>(codes);
      const bool past = j * kTile + key >= s.keys;
      if (!warp_wait(c, empty, ((i >> 1) & 1) ^ 1u, p.status, kInfoAttnProbs)) return;
      if (!kValues) tc_fence_after();
#pragma unroll 1
      for (int g = 0; g < Geo::kGroups; ++g) {
        const uint32_t f = past ? 0u : kv4_scale_h2(scales & 255u);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
        if (g + 1 < Geo::kGroups) w = *reinterpret_cast<const uint4*>(codes + (g + 1) * local * 16);
        scales >>= 8;
        uint32_t y[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          kv4_expand(x[k], *reinterpret_cast<uint32_t(*)[4]>(y + 4 * k));
#pragma unroll
          for (int b = 0; b < 4; ++b) y[4 * k + b] = kv4_mul2(y[4 * k + b], f);
        }
        if (kValues) {
          uint8_t* dst = row + (g / 2) * (kTile * 128);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(dst + (((g % 2) * 4 + k) ^ (key & 7)) * 16) =
                make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
        } else {
          tmem_st16(cols + g * 16, y);
        }
      }
      arrive_warp(&c.kv_empty[ring.stage]);
      if (kValues) {
        fence_proxy_async();
      } else {
        tmem_st_wait();
        tc_fence_before();
      }
      arrive_warp(full);
    }
  }
}

// ---------------------------------------------------------------- MMA issuers (warps 1 and 2)
// S = K Q^T of the tiles in order.
template <int D>
__device__ __forceinline__ void issue_scores(const Kv4Attn& p, Control& c, uint32_t q_lo, uint32_t tmem) {
  using Geo = Geometry<D>;
  Segment s;
  int n = 0, i = 0;
  while (true) {
    const uint32_t q_phase = n & 1;
    if (!take(c, n, s, p.status) || !s.live) return;
    const uint32_t id = idesc_f16(kTile, (s.toks * p.G + 15) / 16 * 16), b = kDescLoK + q_lo;
    if (!warp_wait(c, &c.q_full, q_phase, p.status, kInfoAttnQuery)) return;
    for (int j = s.j0; j < s.j1; ++j, ++i) {
      const int buf = i & 1;
      const uint32_t phase = (i >> 1) & 1;
      if (!warp_wait(c, &c.s_empty[buf], phase ^ 1u, p.status, kInfoAttnScores) ||
          !warp_wait(c, &c.k_full[buf], phase, p.status, kInfoAttnStage))
        return;
      tc_fence_after();
      if (elect()) {
        const uint32_t d = tmem + Geo::kScoresCol + buf * kRows, a = tmem + Geo::kKeysCol + buf * (D / 2);
#pragma unroll 4
        for (int ks = 0; ks < D / 16; ++ks)
          mma_ts(d, a + ks * 8, b + (ks / 4) * (kRows * 128 / 16) + (ks % 4) * 2, kDescHi, id, ks > 0 ? 1u : 0u);
        mma_commit(&c.s_full[buf]);
        mma_commit(&c.k_empty[buf]);
      }
      __syncwarp();
    }
  }
}
// O (+)= V^T P^T of the tiles in order.
template <int D>
__device__ __forceinline__ void issue_outputs(const Kv4Attn& p, Control& c, uint32_t v_lo, uint32_t p_lo, uint32_t tmem) {
  using Geo = Geometry<D>;
  Segment s;
  int n = 0, i = 0;
  while (true) {
    const int ob = n & 1;
    const uint32_t o_phase = (n >> 1) & 1;
    if (!take(c, n, s, p.status) || !s.live) return;
    const uint32_t id = idesc_f16(kTile, (s.toks * p.G + 15) / 16 * 16) | (3u << 15);  // A: M-major, B: N-major
    const uint32_t d = tmem + Geo::kOutCol + ob * kRows;
    if (!warp_wait(c, &c.o_empty[ob], o_phase ^ 1u, p.status, kInfoAttnOut)) return;
    for (int j = s.j0; j < s.j1; ++j, ++i) {
      const int buf = i & 1;
      const uint32_t phase = (i >> 1) & 1;
      if (!warp_wait(c, &c.v_full[buf], phase, p.status, kInfoAttnStage) ||
          !warp_wait(c, &c.p_full[buf], phase, p.status, kInfoAttnProbs))
        return;
      tc_fence_after();
      if (elect()) {
        const uint32_t a = kDescLoN + v_lo + buf * (Geo::kValueBytes / 16), b = kDescLoN + p_lo + buf * (Geo::kProbBytes / 16);
#pragma unroll 4
        for (int ks = 0; ks < kTile / 16; ++ks)
          mma_ss(d, a + ks * (2048 / 16), kDescHi, b + ks * (2048 / 16), kDescHi, id, ks > 0 || j > s.j0 ? 1u : 0u);
        mma_commit(&c.v_empty[buf]);
        mma_commit(&c.p_empty[buf]);
        if (j + 1 == s.j1) mma_commit(&c.o_full[ob]);
      }
      __syncwarp();
    }
  }
}
// Every MMA that this thread issued has completed once its barrier flips.
__device__ __forceinline__ void drain_mma(const Kv4Attn& p, Control& c, int which) {
  if (elect()) {
    mma_commit(&c.drain[which]);
    if (!mbar_wait(&c.drain[which], 0, nullptr)) record_failure(p.status, &c.abort_flag, kInfoAttnDrain);
  }
  __syncwarp();
}

// ---------------------------------------------------------------- softmax (warps 8..23)
// Four groups of four warps, 8 or 16 of the rows each, which have nothing to do with one
// another.  A step's waits, votes and loads take longer than the arithmetic of so few rows:
// two tiles share them.  (64 blocks of 9 tokens: 347 us, with two groups of up to 32 rows,
// a tile a step, 374; 13 draft blocks 81 and 92.)  A group's warps agree on every turn: what
// one of them alone finds out (a wait that ran out) goes through a vote before any leaves.

// A segment's queries, by all softmax warps: rows into the K-major, 128-byte-swizzled tile
// of the first product, in f16, with their scales and limits.  D / 8 lanes take a row; all
// loads of a warp are under way together.  (The products of the segment before, which read
// this tile, are complete: their scores have been seen.  One warp that loaded ahead took 12
// us for 64 rows.)
template <bool kBf16, int D>
__device__ __forceinline__ void load_queries(const Kv4Attn& p, Control& c, uint8_t* q_mem, const Segment& s, int seg) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kWarps = 4 * kSoftGroups, kPasses = kRows / (kWarps * kAtOnce);
  const int lane = threadIdx.x & 31, ch = lane % kLanes, buf = seg & 1, rows = s.toks * p.G;
  const int r0 = ((threadIdx.x >> 5) - 8) * kAtOnce + lane / kLanes;
  uint4 x[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int r = r0 + k * kWarps * kAtOnce;
    x[k] = make_uint4(0, 0, 0, 0);
    if (r < rows)
      x[k] = __ldg(reinterpret_cast<const uint4*>(p.q + (s.tok0 + r / p.G) * p.q_stride + (s.h * p.G + r % p.G) * D + ch * 8));
  }
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int r = r0 + k * kWarps * kAtOnce;
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
    *reinterpret_cast<uint4*>(q_mem + (ch / 8) * (kRows * 128) + r * 128 + ((ch % 8) ^ (r & 7)) * 16) = x[k];
    if (ch == 0) {
      c.row_scale[buf][r] = scale;
      // rows past the tile's see every key, so that they ask for no mask
      c.row_limit[buf][r] =
          r < rows ? (s.own ? max(0, min(s.keys, s.lim0 + s.tok0 + r / p.G)) : s.keys) : 0x7fffffff;
    }
  }
  fence_proxy_async();
  arrive_warp(&c.q_full);
}

template <bool kBf16, int D>
struct Softmax {
  using Geo = Geometry<D>;
  const Kv4Attn& p;
  Control& c;
  uint8_t *p_mem, *q_mem;
  uint32_t tmem;
  int key;             // of the tile: the thread's tensor memory lane
  int group;
  uint32_t lanes;

  // kMine rows of the group (a multiple of 8), the first of them row0.
  template <int kMine, int kTiles>
  __device__ __forceinline__ void load_scores(uint32_t (&x)[kTiles][kMine], int i, int row0) {
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const uint32_t t = tmem + Geo::kScoresCol + ((i + n) & 1) * kRows + lanes + row0;
#pragma unroll
      for (int r = 0; r < kMine; r += 8) tmem_ld8(t + r, *reinterpret_cast<uint32_t(*)[8]>(x[n] + r));
    }
    tmem_ld_wait();
  }
  // Scores to logits relative to the reference, -infinity for keys that a row does not
  // see; -> their largest.
  template <int kMine, int kTiles>
  __device__ __forceinline__ float logits(uint32_t (&x)[kTiles][kMine], int qb, int row0, int at, bool masked) {
    const float *scale = c.row_scale[qb] + row0, *neg = c.neg + row0;
#pragma unroll
    for (int r = 0; r < kMine; r += 4) {
      const float4 a = *reinterpret_cast<const float4*>(scale + r), b = *reinterpret_cast<const float4*>(neg + r);
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        float t[4];
        unpair(fma2(pair(__uint_as_float(x[n][r]), __uint_as_float(x[n][r + 1])), pair(a.x, a.y), pair(b.x, b.y)), t[0],
               t[1]);
        unpair(fma2(pair(__uint_as_float(x[n][r + 2]), __uint_as_float(x[n][r + 3])), pair(a.z, a.w), pair(b.z, b.w)),
               t[2], t[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[n][r + k] = __float_as_uint(t[k]);
      }
    }
    if (masked) {
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int r = 0; r < kMine; ++r)
          if (at + n * kTile >= c.row_limit[qb][row0 + r]) x[n][r] = 0xff800000u;
    }
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int r = 0; r < kMine; r += 2)
        top[(r / 2) % 4] = max3(top[(r / 2) % 4], __uint_as_float(x[n][r]), __uint_as_float(x[n][r + 1]));
    return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  }

  // Rows' values z over the lanes of a warp: every exchange halves the rows that a lane goes
  // on with, until lane r has row r's (of up to 32).
  template <int kMine, typename Op>
  __device__ __forceinline__ float over_lanes(const float (&z)[kMine], float none, const Op& op) {
    const int lane = threadIdx.x & 31;
    float y[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) y[r] = r < kMine ? z[r < kMine ? r : 0] : none;
#pragma unroll
    for (int h = 16; h > 0; h >>= 1)
#pragma unroll
      for (int r = 0; r < h; ++r) {
        const bool up = lane & h;
        const float give = up ? y[r] : y[r + h], keep = up ? y[r + h] : y[r];
        y[r] = op(keep, __shfl_xor_sync(0xffffffffu, give, h));
      }
    return y[0];
  }

  // Moves the references of the group's rows whose logits pass them (of all rows at a
  // segment's first tile, where they are relative to 0), and the outputs under the old
  // ones; l is the callers' by c.factor.
  template <int kMine, int kTiles>
  __device__ __forceinline__ bool move(const uint32_t (&x)[kTiles][kMine], int i, int seg, int row0, bool first, bool failed) {
    if (softmax_any(group, failed)) return false;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
    float z[kMine];
#pragma unroll
    for (int r = 0; r < kMine; ++r)
      z[r] = kTiles == 1 ? __uint_as_float(x[0][r]) : fmaxf(__uint_as_float(x[0][r]), __uint_as_float(x[kTiles - 1][r]));
    const float high = over_lanes<kMine>(z, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
    if (lane < kMine) c.top[warp][row0 + lane] = high;
    softmax_sync(group);
    if (key < kMine) {
      const int r = row0 + key;
      const float top = fmaxf(fmaxf(c.top[0][r], c.top[1][r]), fmaxf(c.top[2][r], c.top[3][r]));
      const float old = c.m[r];
      const bool none = old == -INFINITY, moves = top != -INFINITY && (none || top > kLift + kRescaleAt);
      const float now = moves ? (none ? top : old + top) - kLift : old;
      c.m[r] = now;
      c.neg[r] = now == -INFINITY ? 0.f : -now;
      c.factor[r] = none ? 0.f : (moves ? ex2(old - now) : 1.f);
    }
    softmax_sync(group);
    if (first) return true;
    // the products so far are complete
    const bool ok = warp_wait(c, &c.p_empty[(i - 1) & 1], ((i - 1) >> 1) & 1, p.status, kInfoAttnProbs);
    if (softmax_any(group, !ok)) return false;
    tc_fence_after();
    const uint32_t o = tmem + Geo::kOutCol + (seg & 1) * kRows + lanes;
#pragma unroll 1
    for (int r0 = row0; r0 < row0 + kMine; r0 += 8) {
      uint32_t y[8];
      tmem_ld8(o + r0, y);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * c.factor[r0 + k]);
      tmem_st8(o + r0, y);
    }
    tmem_st_wait();
    return true;
  }

  // kTiles tiles from j, the i-th of the CTA.
  template <int kMine, int kTiles>
  __device__ __forceinline__ bool step(const Segment& s, int seg, int i, int j, float (&l)[kMine], bool& ok) {
    const int qb = seg & 1, row0 = group * kMine, at = j * kTile + key;
    const bool first = j == s.j0, masked = (j + kTiles) * kTile > s.least;
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
      ok = ok && warp_wait(c, &c.s_full[(i + n) & 1], ((i + n) >> 1) & 1, p.status, kInfoAttnScores);
    tc_fence_after();
    uint32_t x[kTiles][kMine];
    load_scores<kMine, kTiles>(x, i, row0);
    const float top = logits<kMine, kTiles>(x, qb, row0, at, masked);
    if (first || softmax_any(group, !ok || top > kLift + kRescaleAt)) {
      if (!move<kMine, kTiles>(x, i, seg, row0, first, !ok)) return false;
#pragma unroll
      for (int r = 0; r < kMine; ++r) l[r] *= c.factor[row0 + r];
      load_scores<kMine, kTiles>(x, i, row0);
      logits<kMine, kTiles>(x, qb, row0, at, masked);
    }
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
      for (int n = 0; n < kTiles; ++n) mbar_arrive(&c.s_empty[(i + n) & 1]);
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const int buf = (i + n) & 1;
      ok = ok && warp_wait(c, &c.p_empty[buf], (((i + n) >> 1) & 1) ^ 1u, p.status, kInfoAttnProbs);
      uint8_t* row = p_mem + buf * Geo::kProbBytes + key * 128;
#pragma unroll
      for (int r = 0; r < kMine; r += 8) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float e0 = ex2(__uint_as_float(x[n][r + 2 * k])), e1 = ex2(__uint_as_float(x[n][r + 2 * k + 1]));
          l[r + 2 * k] += e0;
          l[r + 2 * k + 1] += e1;
          w[k] = pack_h2(e0, e1);
        }
        *reinterpret_cast<uint4*>(row + (((row0 + r) / 8) ^ (key & 7)) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_proxy_async();
      tc_fence_before();
      arrive_warp(&c.p_full[buf]);
    }
    return true;
  }

  // The group's rows of a segment: their number is fixed in the code, as a branch a row
  // costs more than the row.
  template <int kMine>
  __device__ __forceinline__ bool segment(const Segment& s, int seg, int& i) {
    const int qb = seg & 1, rows = s.toks * p.G, row0 = group * kMine;
    float l[kMine];
#pragma unroll
    for (int r = 0; r < kMine; ++r) l[r] = 0.f;
    // (the rows may have been another group's in the segment before, which it is done with once
    // all warps have brought their queries)
    bool ok = warp_wait(c, &c.q_full, seg & 1, p.status, kInfoAttnQuery);
    if (key < kMine) {
      c.m[row0 + key] = -INFINITY;
      c.neg[row0 + key] = 0.f;
    }
    softmax_sync(group);
    int j = s.j0;
    for (; j + 1 < s.j1; j += 2, i += 2)
      if (!step<kMine, 2>(s, seg, i, j, l, ok)) return false;
    for (; j < s.j1; ++j, ++i)
      if (!step<kMine, 1>(s, seg, i, j, l, ok)) return false;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
    const float sum = over_lanes<kMine>(l, 0.f, [](float a, float b) { return a + b; });
    if (lane < kMine) c.top[warp][row0 + lane] = sum;
    ok = ok && warp_wait(c, &c.o_full[qb], (seg >> 1) & 1, p.status, kInfoAttnOut);
    if (softmax_any(group, !ok)) return false;
    tc_fence_after();
    if (key < kMine && row0 + key < rows) {
      const int r = row0 + key;
      const float sum = (c.top[0][r] + c.top[1][r]) + (c.top[2][r] + c.top[3][r]);
      // (a row whose scores were all NaN has no reference: without one its part would count as empty)
      p.ml[s.part_row + r] = make_float2(isnan(sum) ? NAN : c.m[r], sum);
    }
    // channels are lanes: a row is written 128 bytes a warp
    const uint32_t o = tmem + Geo::kOutCol + qb * kRows + lanes;
    float* dst = p.o + s.part_row * D + key;
#pragma unroll 1
    for (int r0 = row0; r0 < row0 + kMine; r0 += 8) {
      uint32_t y[8];
      tmem_ld8(o + r0, y);
      tmem_ld_wait();
      if (key < D) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (r0 + k < rows) dst[static_cast<long long>(r0 + k) * D] = __uint_as_float(y[k]);
      }
    }
    tc_fence_before();
    arrive_warp(&c.o_empty[qb]);
    softmax_sync(group);  // c.top and c.m have been read
    return true;
  }
  // A group whose rows a segment does not have goes along with the others.
  __device__ __forceinline__ bool without_rows(const Segment& s, int seg, int& i) {
    bool ok = warp_wait(c, &c.q_full, seg & 1, p.status, kInfoAttnQuery);
    for (int j = s.j0; j < s.j1 && ok; ++j, ++i) {
      const int buf = i & 1;
      const uint32_t phase = (i >> 1) & 1;
      ok = warp_wait(c, &c.s_full[buf], phase, p.status, kInfoAttnScores);
      arrive_warp(&c.s_empty[buf]);
      ok = ok && warp_wait(c, &c.p_empty[buf], phase ^ 1u, p.status, kInfoAttnProbs);
      arrive_warp(&c.p_full[buf]);
    }
    ok = ok && warp_wait(c, &c.o_full[seg & 1], (seg >> 1) & 1, p.status, kInfoAttnOut);
    if (softmax_any(group, !ok)) return false;
    arrive_warp(&c.o_empty[seg & 1]);
    return true;
  }
  __device__ void run() {
    Segment s;
    int n = 0, i = 0;
    while (true) {
      const int seg = n;
      const bool got = take(c, n, s, p.status);
      if (softmax_any(group, !got)) return;
      if (!s.live) return;
      load_queries<kBf16, D>(p, c, q_mem, s, seg);
      const int rows = (s.toks * p.G + 15) / 16 * 16, mine = rows <= 8 * kSoftGroups ? 8 : 16;
      if (group * mine >= rows ? !without_rows(s, seg, i) : mine == 8 ? !segment<8>(s, seg, i) : !segment<16>(s, seg, i)) return;
    }
  }
};

// ---------------------------------------------------------------- list (warp 3)
// Hands the segments over, each whenever its readers have made room.  (The whole warp walks.)
__device__ __forceinline__ void hand_list(const Kv4Attn& p, Control& c, int plen) {
  Walker w;
  w.begin(p, c.start, plen);
  for (int n = 0;; ++n) {
    Segment s;
    if (!w.next(p, s)) s.live = 0;
    const int e = n % kSegments;
    if (!warp_wait(c, &c.seg_empty[e], ((n / kSegments) & 1) ^ 1u, p.status, kInfoAttnList)) return;
    if ((threadIdx.x & 31) == 0) {
      c.seg[e] = s;
      mbar_arrive(&c.seg_full[e]);
    }
    __syncwarp();
    if (!s.live) return;
  }
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kThreads, 1) prefix_attention_kv4_kernel(const __grid_constant__ Kv4Attn p) {
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
      mbar_init(&c.s_full[b], 1); mbar_init(&c.s_empty[b], 4 * kSoftGroups);
      mbar_init(&c.v_full[b], 4); mbar_init(&c.v_empty[b], 1);
      mbar_init(&c.p_full[b], 4 * kSoftGroups); mbar_init(&c.p_empty[b], 1);
      mbar_init(&c.o_full[b], 1); mbar_init(&c.o_empty[b], 4 * kSoftGroups);
    }
    for (int s = 0; s < kSegments; ++s) { mbar_init(&c.seg_full[s], 1); mbar_init(&c.seg_empty[s], kReaders); }
    mbar_init(&c.q_full, 4 * kSoftGroups);
    mbar_init(&c.drain[0], 1);
    mbar_init(&c.drain[1], 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  }
  griddep_wait();               // what the previous kernel on the stream wrote is visible
  int plen = 0;
  if (p.B > kWarpRequests) plen = find_share<kThreads>(p, c.start);
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
      issue_scores<D>(p, c, smem_u32(mem + Geo::kQueriesAt) >> 4, tmem);
      __syncwarp();
      drain_mma(p, c, 0);
    } else if (warp == 2) {
      issue_outputs<D>(p, c, smem_u32(mem + Geo::kValuesAt) >> 4, smem_u32(mem + Geo::kProbsAt) >> 4, tmem);
      __syncwarp();
      drain_mma(p, c, 1);
    } else {
      if (p.B <= kWarpRequests) plen = find_share_by_warp(p, c.start);
      hand_list(p, c, plen);
      __syncwarp();
    }
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    expand<D, false>(p, c, mem + Geo::kRingAt, nullptr, tmem);
  } else if (warp < 8 + 4 * kSoftGroups) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    Softmax<kBf16, D> r{p, c, mem + Geo::kProbsAt, mem + Geo::kQueriesAt, tmem, tid & 127, (warp - 8) / 4, static_cast<uint32_t>((warp & 3) * 32) << 16};
    r.run();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
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
__global__ void __launch_bounds__(kMergeThreads) kv4_merge_kernel(const __grid_constant__ Kv4Attn p) {
  constexpr int kEach = D / 32;  // elements of a lane
  const int lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * (kMergeThreads / 32) + (threadIdx.x >> 5);
  if (unit >= static_cast<long long>(p.T) * p.Hq) return;
  const int t = static_cast<int>(unit / p.Hq), hq = static_cast<int>(unit % p.Hq), h = hq / p.G, g = hq % p.G;
  griddep_wait();
  const Plan plan = *p.plan;
  // (the search for the shares has written every token's of this call: zeros for one of no
  // request, which owns nothing; what an earlier call left is never read)
  const RequestPlan rp = p.requests[t];
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
    // parts four at a time, all that is read of them under way together
#pragma unroll 1
    for (int i0 = 0; i0 < count; i0 += 4) {
      float2 ml[4];
      float v[4][kEach];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const long long at = row + static_cast<long long>(kRows) * min(i0 + x, count - 1);
        ml[x] = __ldcg(p.ml + at);
        const float* o = p.o + at * D + lane * kEach;
        if (kEach == 4) {
          const float4 u = __ldcg(reinterpret_cast<const float4*>(o));
          v[x][0] = u.x; v[x][1] = u.y; v[x][kEach - 2] = u.z; v[x][kEach - 1] = u.w;
        } else {
          const float2 u = __ldcg(reinterpret_cast<const float2*>(o));
          v[x][0] = u.x; v[x][1] = u.y;
        }
        if (i0 + x >= count) ml[x] = make_float2(-INFINITY, 0.f);
      }
      float m1 = m;
#pragma unroll
      for (int x = 0; x < 4; ++x) m1 = isnan(m1) || isnan(ml[x].x) ? NAN : fmaxf(m1, ml[x].x);
      const float old = m == -INFINITY ? 0.f : ex2(m - m1);
      l *= old;
#pragma unroll
      for (int i = 0; i < kEach; ++i) acc[i] *= old;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (ml[x].x == -INFINITY) continue;  // saw no key (and its outputs may be of another part)
        const float a = ex2(ml[x].x - m1);
        l += a * ml[x].y;
#pragma unroll
        for (int i = 0; i < kEach; ++i) acc[i] += a * v[x][i];
      }
      m = m1;
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

// Workspace after the fixed header.  Monotone in T: a size serves every smaller call of
// the same heads.
struct Layout {
  size_t o_plan, o_req, o_ml, o_o, total;
};
Layout layout(int T, int Hq, int D, int ctas) {
  Layout L;
  const size_t rows = 2 * static_cast<size_t>(T) * Hq + static_cast<size_t>(kRows) * (ctas + 1);
  size_t o = kWsHeaderBytes;
  L.o_plan = o; o += kWsAlign;
  L.o_req = o; o += ws_align_up(sizeof(RequestPlan) * static_cast<size_t>(T));
  L.o_ml = o; o += ws_align_up(8 * rows);
  L.o_o = o; o += ws_align_up(4 * rows * D);
  L.total = o;
  return L;
}

template <typename K>
cudaError_t launch_one(K* kernel, const Kv4Attn& p, unsigned grid, int threads, size_t smem, cudaStream_t s) {
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
cudaError_t launch(const Kv4Attn& p, int few, cudaStream_t s) {
  cudaError_t e;
  if (few) {
    e = launch_kv4_few(p, few, D, kBf16, s);
  } else {
    static std::atomic<uint64_t> done{0};
    e = allow_smem(prefix_attention_kv4_kernel<kBf16, D>, Geometry<D>::kDynamic, done);
    if (e == cudaSuccess)
      e = launch_one(prefix_attention_kv4_kernel<kBf16, D>, p, static_cast<unsigned>(p.ctas), kThreads,
                     Geometry<D>::kDynamic, s);
  }
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
  return sms > 0 ? layout(T, Hq, D, sms).total : 0;
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
    const int most = kv4_few_rows(T, B, Hq / Hkv, page_size, prefix_cap, table_width);
    const long long tpt = (most ? most : kRows) / (Hq / Hkv), row_tiles = (T + tpt - 1) / tpt;
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
  const Layout L = layout(T, Hq, D, sms);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  Kv4Attn p;
  memset(&p, 0, sizeof(p));
  p.T = T; p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; 
  const int few = kv4_few_rows(T, B, p.G, page_size, prefix_cap, table_width);
  p.tpt = (few ? few : kRows) / p.G;
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
  p.ml = reinterpret_cast<float2*>(w + L.o_ml);
  p.o = reinterpret_cast<float*>(w + L.o_o);
  const cudaError_t e = dtype == MOE_DTYPE_BF16 ? (D == 64 ? launch<true, 64>(p, few, stream) : launch<true, 128>(p, few, stream))
                                                : (D == 64 ? launch<false, 64>(p, few, stream) : launch<false, 128>(p, few, stream));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
