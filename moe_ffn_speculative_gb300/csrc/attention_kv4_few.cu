// Attention over a 4-bit cache for few query rows (up to 16: single tokens, short
// blocks), where the bytes of the cache are all there is.
//
// The same transposed products as the other kernel's, S^T = K Q^T and O^T = V^T P^T, but
// on the warps' own matrix instructions (m16n8k16, 8 rows an instruction): a warp
// expands 16 keys in registers, in the very places where the instruction wants them, so
// that nothing passes through shared or tensor memory and no role waits for another.  The
// fifth-generation instruction would take operands through shared memory for 128 lanes,
// at 30 to 70 clocks each however few the rows, and its kernel's handing over costs 1500
// clocks a tile of 128 keys (measured; the tile's bytes take 740 to arrive).  Here the 128
// instructions of a tile and 8 rows take 270 clocks of an SM's tensor pipes and the
// expansion 400 of its conversion pipe. 
//
// A CTA (one per SM) takes a share of the list as there.  Its last warp walks it and copies its
// keys, 256 at a time, into a ring of stages; the others take the keys 32 at a time in turn,
// each with its own references, sums and outputs, which meet in shared memory at a
// segment's end.  (With the codes of coming steps in registers there were too few bytes
// under way, and with copies by the lanes that use them a quarter of the instructions was
// their addresses: 228 and 202 us where 640000 keys of 8 heads take 103 to read.)
//
// Places.  With lane = 4 r + q (r < 8, q < 4), of the 16 keys from `base`:
//   S^T's row r is key (r % 2) 4 + r / 2, row 8 + r that key + 8: a load's lanes touch 8
//     neighbouring keys, and the scores come out where the second product wants them.
//   The lane's channels of a key are a half of one or two groups of 32 (those that leave
//     8-byte loads with few bank conflicts); queries are laid out to match.
//   Of values the lane reads keys q, 4 + q, 8 + q, 12 + q, channels [r D/8, (r + 1) D/8):
//     4 neighbouring keys a load; two keys' channels are exchanged between registers.
//   O^T's block b: rows r and 8 + r are channels r D/8 + 2 b and + 1.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include "attention_kv4.cuh"
#include "kv4.cuh"
#include "moe.h"

namespace moe {
namespace {

// Warps that compute, beside one that walks the list: with 8 rows 16 warps of 128 registers
// a thread, with 16 rows (twice the outputs) 12 of 168.
constexpr int warps(int blocks) { return blocks == 1 ? 15 : 11; }
constexpr int threads(int blocks) { return 32 * (warps(blocks) + 1); }
constexpr int kSets = 2, kStep = 16 * kSets;     // keys of a warp at a time: sets of 16
constexpr int kUnit = 256;                       // keys of a stage
constexpr int kSegments = 4;
constexpr int kMaxStages = 12;
constexpr int kSmem = 232448;                    // 227 KB

// Shared memory: the warps' outputs at a segment's end, and as many stages as fit.
template <int D, int kBlocks>
struct Geometry {
  static constexpr int kWarps = warps(kBlocks), kThreads = threads(kBlocks);
  static constexpr int kStageBytes = kUnit * kv4_slot_bytes(D);
  static constexpr int kSlotBytes = 8 * (D + 4) * 4;
  static constexpr int kRingAt = kWarps * kSlotBytes;
  static constexpr int kFit = (kSmem - 4096 - kRingAt) / kStageBytes, kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kDynamic = kRingAt + kStages * kStageBytes;
};

struct Control {
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages], seg_full[kSegments], seg_empty[kSegments];
  Segment seg[kSegments];
  Start start;
  int abort_flag;
  float2 ml[16][8];  // the warps' (reference, sum) of 8 rows
};

__device__ __forceinline__ bool warp_wait(Control& c, uint64_t* bar, uint32_t parity, int32_t* status, int32_t info) {
  const bool ok = mbar_wait(bar, parity, &c.abort_flag);
  if (__all_sync(0xffffffffu, ok)) return true;
  if ((threadIdx.x & 31) == 0) record_failure(status, &c.abort_flag, info);
  return false;
}
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// The computing warps meet: did any of them fail?
template <int kWarps>
__device__ __forceinline__ bool warps_any(bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, "
      "q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(mine)), "n"(32 * kWarps)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
// A scale byte as f16 in both halves (255: infinite, and 0 times it NaN: its codes are 0).
__device__ __forceinline__ uint32_t scale2(uint32_t s) {
  const float f = __uint_as_float(s << 23);
  return pack_h2(f, f);
}

// A lane's codes of 16 keys with their scale bytes: of two keys, D / 4 channels; of four
// values, D / 8.
template <int D>
struct RawKeys {
  uint32_t k[2][D / 32], s[2][D / 64];
};
template <int D>
struct RawValues {
  uint32_t v[4][D / 64], s[4];
};

template <bool kBf16, int D, int kBlocks>  // kBlocks of 8 rows
struct Warp {
  static constexpr int kWarps = warps(kBlocks), kKeySteps = D / 16, kOutBlocks = D / 16, kGroups = D / 32;
  const Kv4Attn& p;
  Control& c;
  int lane, r, q, warp;
  int key;                          // r's key of 16
  uint32_t qf[kBlocks][kKeySteps][2];
  float scale[kBlocks][2];          // of rows 8 n + 2 q, + 1
  int limit[kBlocks][2];
  float m[kBlocks][2], neg[kBlocks][2], l[kBlocks][2];
  float o[kBlocks][kOutBlocks][4];

  __device__ __forceinline__ void load_queries(const Segment& s) {
    const int rows = s.toks * p.G;
#pragma unroll
    for (int n = 0; n < kBlocks; ++n) {
      const int row = 8 * n + r;
      uint4 x[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) x[i] = make_uint4(0, 0, 0, 0);
      if (row < rows) {
        const uint16_t* src = p.q + (s.tok0 + row / p.G) * p.q_stride + (s.h * p.G + row % p.G) * D + q * 16;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) x[i] = __ldg(reinterpret_cast<const uint4*>(src + i / 2 * 64) + i % 2);
      }
      float f = 1.f, back = p.scale_log2;
      if (kBf16) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          top = __vmaxu2(top, __vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu));
          top = __vmaxu2(top, __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
        }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest element goes to [2^14, 2^15); rows of zeros, infinities or NaN stay
        int e = static_cast<int>(top >> 7) - 127 - 14;
        if (top == 0 || top >= 0x7f80u) e = 0;
        e = max(e, -126);
        f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        back *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      }
#pragma unroll
      for (int t = 0; t < kKeySteps; ++t) {
        const uint32_t w[4] = {x[t / 2].x, x[t / 2].y, x[t / 2].z, x[t / 2].w};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t u = w[2 * (t % 2) + b];
          qf[n][t][b] = kBf16 ? pack_h2(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xffff0000u) * f) : u;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int mine = 8 * n + 2 * q + e;  // its scale is with lane 4 (2 q + e)
        scale[n][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * q + e));
        limit[n][e] = mine < rows ? (s.own ? max(0, min(s.keys, s.lim0 + s.tok0 + mine / p.G)) : s.keys) : s.keys;
        m[n][e] = -INFINITY;
        neg[n][e] = INFINITY;
        l[n][e] = 0.f;
      }
#pragma unroll
      for (int b = 0; b < kOutBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][b][i] = 0.f;
    }
  }

  // The lane's codes of the 16 keys from the `off`-th of a stage, of which `valid` are
  // there: the others' places may hold anything.
  __device__ __forceinline__ void take(RawKeys<D>& x, const uint8_t* stage, int off, int valid) const {
    const int local = min(p.page, kUnit), log2 = min(p.page_log2, 8);
    // the lane's half groups: half q % 2 of groups q / 2 (and q / 2 + 2)
    const int key_at = (q / 2 * local + key) * 16 + q % 2 * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = off + 8 * i, slot = at & (local - 1);
      const uint8_t* block = stage + (at >> log2) * (local * kv4_slot_bytes(D));
      const uint8_t* b = block + slot * 16 + key_at;
      const uint8_t* sc = block + kv4_scales_at(D, local, 0) + (slot + key) * kGroups + q / 2;
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
        const uint2 u = *reinterpret_cast<const uint2*>(b + w * 2 * local * 16);
        x.k[i][2 * w] = u.x;
        x.k[i][2 * w + 1] = u.y;
        x.s[i][w] = sc[2 * w];
      }
    }
    if (valid < 16) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (8 * i + key >= valid)
#pragma unroll
          for (int w = 0; w < D / 64; ++w) x.s[i][w] = x.k[i][2 * w] = x.k[i][2 * w + 1] = 0;
    }
  }
  __device__ __forceinline__ void take(RawValues<D>& x, const uint8_t* stage, int off, int valid) const {
    const int local = min(p.page, kUnit), log2 = min(p.page_log2, 8);
    const int value_at = kv4_codes_at(D, local, 1) +
                         (D == 128 ? (r / 2 * local + q) * 16 + r % 2 * 8 : (r / 4 * local + q) * 16 + r % 4 * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = off + 8 * (i / 2), slot = at & (local - 1);
      const uint8_t* block = stage + (at >> log2) * (local * kv4_slot_bytes(D));
      const uint8_t* b = block + slot * 16 + value_at + i % 2 * 64;
      if (D == 128) {
        const uint2 u = *reinterpret_cast<const uint2*>(b);
        x.v[i][0] = u.x; x.v[i][D / 64 - 1] = u.y;
      } else {
        x.v[i][0] = *reinterpret_cast<const uint32_t*>(b);
      }
      x.s[i] = block[kv4_scales_at(D, local, 1) + (slot + i % 2 * 4 + q) * kGroups + r * kGroups / 8];
    }
    if (valid < 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * i + q >= valid) {
          x.s[i] = 0;
#pragma unroll
          for (int w = 0; w < D / 64; ++w) x.v[i][w] = 0;
        }
    }
  }

  // S^T of 16 keys.
  __device__ __forceinline__ void scores(const RawKeys<D>& x, float (&s)[kBlocks][4]) const {
#pragma unroll
    for (int n = 0; n < kBlocks; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      const uint32_t f0 = scale2(x.s[0][w / 2]), f1 = scale2(x.s[1][w / 2]);
      uint32_t a[4], b[4];
      kv4_expand(x.k[0][w], a);
      kv4_expand(x.k[1][w], b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = kv4_mul2(a[i], f0);
        b[i] = kv4_mul2(b[i], f1);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
          mma(s[n], a[2 * t], b[2 * t], a[2 * t + 1], b[2 * t + 1], qf[n][2 * w + t][0], qf[n][2 * w + t][1]);
    }
  }

  // Moves the rows' references to the logits t that pass them (s: the scores), and what was
  // added up under the old ones.  A row without one has neg = infinity, so that its first
  // score comes here.
  __device__ __forceinline__ void move(const float (&s)[kSets][kBlocks][4], float (&t)[kSets][kBlocks][4]) {
#pragma unroll
    for (int n = 0; n < kBlocks; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool none = m[n][e] == -INFINITY;
        float high = -INFINITY;
#pragma unroll
        for (int k = 0; k < kSets; ++k)
#pragma unroll
          for (int i = e; i < 4; i += 2) {
            if (none && t[k][n][i] != -INFINITY) t[k][n][i] = s[k][n][i] * scale[n][e];
            high = isnan(t[k][n][i]) || isnan(high) ? NAN : fmaxf(high, t[k][n][i]);
          }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          const float v = __shfl_xor_sync(0xffffffffu, high, d);
          high = isnan(v) || isnan(high) ? NAN : fmaxf(high, v);
        }
        // (not: high > ..., so that NaN moves too)
        if (high != -INFINITY && (none || !(high <= kLift + kRescaleAt))) {
          const float was = m[n][e], now = (none ? high : was + high) - kLift, f = none ? 0.f : ex2(was - now);
          m[n][e] = now;
          neg[n][e] = -now;
          l[n][e] *= f;
#pragma unroll
          for (int b = 0; b < kOutBlocks; ++b) {
            o[n][b][e] *= f;
            o[n][b][e + 2] *= f;
          }
#pragma unroll
          for (int k = 0; k < kSets; ++k)
#pragma unroll
            for (int i = e; i < 4; i += 2)
              if (t[k][n][i] != -INFINITY) t[k][n][i] = fmaf(s[k][n][i], scale[n][e], neg[n][e]);
        }
      }
  }

  // The keys' powers, as the second product's operand.
  __device__ __forceinline__ void powers(const float (&s)[kSets][kBlocks][4], uint32_t (&pb)[kSets][kBlocks][2], int base,
                                         int least) {
    // logits relative to the reference; rows 8 n + 2 q and + 1, keys `key` and `key` + 8
    float t[kSets][kBlocks][4], top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kSets; ++k)
#pragma unroll
      for (int n = 0; n < kBlocks; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) t[k][n][i] = fmaf(s[k][n][i], scale[n][i & 1], neg[n][i & 1]);
    if (base + kStep > least) {
#pragma unroll
      for (int k = 0; k < kSets; ++k)
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (base + 16 * k + key + 8 * (i >> 1) >= limit[n][i & 1]) t[k][n][i] = -INFINITY;
    }
#pragma unroll
    for (int k = 0; k < kSets; ++k)
#pragma unroll
      for (int n = 0; n < kBlocks; ++n)
        top = fmaxf(fmaxf(top, fmaxf(t[k][n][0], t[k][n][1])), fmaxf(t[k][n][2], t[k][n][3]));
    if (__any_sync(0xffffffffu, top > kLift + kRescaleAt)) move(s, t);
#pragma unroll
    for (int k = 0; k < kSets; ++k)
#pragma unroll
      for (int n = 0; n < kBlocks; ++n) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = ex2(t[k][n][i]);
        l[n][0] += e[0] + e[2];
        l[n][1] += e[1] + e[3];
        pb[k][n][0] = transpose8(pack_h2(e[0], e[1]));
        pb[k][n][1] = transpose8(pack_h2(e[2], e[3]));
      }
  }

  // O^T of 16 keys.  Two keys' codes are exchanged, so that a byte holds a channel of both.
  __device__ __forceinline__ void outputs(const RawValues<D>& x, const uint32_t (&pb)[kBlocks][2]) {
    uint32_t f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      f[i] = pack_h2(__uint_as_float(x.s[2 * i] << 23), __uint_as_float(x.s[2 * i + 1] << 23));
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
      uint32_t a[4][4];  // even and odd channels of keys q and 4 + q, then of 8 + q and 12 + q
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t u = x.v[2 * i][w], v = x.v[2 * i + 1][w];
        kv4_expand((u & 0x0f0f0f0fu) | ((v << 4) & 0xf0f0f0f0u), a[2 * i]);
        kv4_expand(((u >> 4) & 0x0f0f0f0fu) | (v & 0xf0f0f0f0u), a[2 * i + 1]);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          a[2 * i][b] = kv4_mul2(a[2 * i][b], f[i]);
          a[2 * i + 1][b] = kv4_mul2(a[2 * i + 1][b], f[i]);
        }
      }
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int n = 0; n < kBlocks; ++n) mma(o[n][4 * w + b], a[0][b], a[1][b], a[2][b], a[3][b], pb[n][0], pb[n][1]);
    }
  }

  // kStep keys from `base`, the off-th of a stage.
  __device__ __forceinline__ void step(const uint8_t* stage, uint64_t* empty, int off, int base, int end, int least) {
    float s[kSets][kBlocks][4];
    uint32_t pb[kSets][kBlocks][2];
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      RawKeys<D> x;
      take(x, stage, off + 16 * k, end - base - 16 * k);
      scores(x, s[k]);
    }
    RawValues<D> x[kSets];
#pragma unroll
    for (int k = 0; k < kSets; ++k) take(x[k], stage, off + 16 * k, end - base - 16 * k);
    arrive_warp(empty);
    powers(s, pb, base, least);
#pragma unroll
    for (int k = 0; k < kSets; ++k) outputs(x[k], pb[k]);
  }

  // The warp's steps of a segment: every kWarps-th of those in its `units` stages, whose
  // first is the unit0-th of the CTA.  Every warp sees every stage fill and gives it back, with
  // or without a step there: one that passed stages over could come to wait for a stage's next
  // filling while the one before is still on its way (copies land in any order), which a
  // barrier's parity does not tell apart.  (Waits by a count of issued fillings, in the warps that
  // have a step alone, were 2 % faster for 8 rows and 2 % slower for 16.)
  __device__ __forceinline__ bool run(const Segment& s, const uint8_t* ring, int unit0, int units) {
    using Geo = Geometry<D, kBlocks>;
    constexpr int kSteps = kUnit / kStep;
    static_assert(kSteps <= kWarps, "a step a unit at most");
    load_queries(s);
    const int first = s.j0 * kTile, end = min(s.j1 * kTile, s.keys), base0 = first / kUnit * kUnit;
    int mine = warp;  // the warp's next step, counted from the unit's first
#pragma unroll 1
    for (int u = 0; u < units; ++u) {
      const int unit = unit0 + u, stage = unit % Geo::kStages, base = base0 + u * kUnit + mine * kStep;
      if (!warp_wait(c, &c.kv_full[stage], unit / Geo::kStages & 1, p.status, kInfoAttnStage)) return false;
      if (mine < kSteps && base >= first && base < end)
        step(ring + stage * Geo::kStageBytes, &c.kv_empty[stage], mine * kStep, base, end, s.least);
      else
        arrive_warp(&c.kv_empty[stage]);
      mine -= kSteps;
      if (mine < 0) mine += kWarps;
    }
    return true;
  }

  // The warp's references, sums and outputs of the n-th 8 rows, for the others to read.
  __device__ __forceinline__ void hand(int n, float* slot) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float t = l[n][e];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
      if (r == 0) c.ml[warp][2 * q + e] = make_float2(m[n][e], t);
      // a row of D, the lane's channels side by side
      float* dst = slot + (2 * q + e) * (D + 4) + r * (D / 8);
#pragma unroll
      for (int b = 0; b < kOutBlocks; b += 2)
        *reinterpret_cast<float4*>(dst + 2 * b) = make_float4(o[n][b][e], o[n][b][e + 2], o[n][b + 1][e], o[n][b + 1][e + 2]);
    }
  }
};

__device__ __forceinline__ int units_in(const Segment& s) {
  return (min(s.j1 * kTile, s.keys) + kUnit - 1) / kUnit - s.j0 * kTile / kUnit;
}

// The last warp: hands the segments over and copies their keys.
template <int D, int kBlocks>
__device__ __forceinline__ void produce(const Kv4Attn& p, Control& c, int plen, uint8_t* ring_mem) {
  using Geo = Geometry<D, kBlocks>;
  const int lane = threadIdx.x & 31;
  Walker w;
  w.begin(p, c.start, plen);
  Ring ring;
  int filled = 0;
  bool ok = true;
  for (int n = 0; ok; ++n) {
    Segment s;
    if (!w.next(p, s)) s.live = 0;
    const int e = n % kSegments;
    ok = warp_wait(c, &c.seg_empty[e], ((n / kSegments) & 1) ^ 1u, p.status, kInfoAttnList);
    if (!ok) break;
    if (lane == 0) {
      c.seg[e] = s;
      mbar_arrive(&c.seg_full[e]);
    }
    __syncwarp();
    if (!s.live) break;
    int first = s.j0 * kTile / kUnit * kUnit;
    Pages<kUnit> pages;
    pages.begin(p, s, lane);
    for (int u = units_in(s); u > 0; --u, first += kUnit) {
      const int page = pages.of(p, first, lane);
      ok = warp_wait(c, &c.kv_empty[ring.stage], ring.phase ^ 1u, p.status, kInfoAttnStage);
      if (!ok) break;
      copy_keys<D, kUnit>(p, s, first, page, ring_mem + ring.stage * Geo::kStageBytes, &c.kv_full[ring.stage], lane);
      ++filled;
      ring.next(Geo::kStages);
    }
  }
  // every copy that was issued has landed (also after a failure)
  for (int e = 0; e < Geo::kStages; ++e) {
    const int fills = filled / Geo::kStages + (e < filled % Geo::kStages ? 1 : 0);
    if (fills > 0 && !mbar_wait(&c.kv_full[e], (fills - 1) & 1, nullptr))
      record_failure(p.status, &c.abort_flag, kInfoAttnDrain);
  }
  __syncwarp();
}

// 8 rows of a segment from `row0` over the warps in order, a warp a row, and to the
// workspace.
template <int D, int kBlocks>
__device__ __forceinline__ void finish(const Kv4Attn& p, const Control& c, const Segment& s, int row0,
                                       const uint8_t* slots, int warp, int lane) {
  constexpr int kWarps = warps(kBlocks);
  const int row = warp;
  if (row < 8 && row0 + row < s.toks * p.G) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < kWarps) ml = c.ml[lane][row];
    float top = ml.x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float v = __shfl_xor_sync(0xffffffffu, top, d);
      top = isnan(top) || isnan(v) ? NAN : fmaxf(top, v);
    }
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
    float sum = f * ml.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    float acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      const float a = __shfl_sync(0xffffffffu, f, x);
      const float* src = reinterpret_cast<const float*>(slots + x * Geometry<D, kBlocks>::kSlotBytes) + row * (D + 4) + lane;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) acc[i] += a * src[32 * i];
    }
    float* dst = p.o + (s.part_row + row0 + row) * D + lane;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) dst[32 * i] = acc[i];
    // (a row whose scores were all NaN has no reference: without one its part would count as empty)
    if (lane == 0) p.ml[s.part_row + row0 + row] = make_float2(isnan(sum) ? NAN : top, sum);
  }
}

template <bool kBf16, int D, int kBlocks>
__global__ void __launch_bounds__(threads(kBlocks), 1) kv4_few_kernel(const __grid_constant__ Kv4Attn p) {
  using Geo = Geometry<D, kBlocks>;
  extern __shared__ uint4 dynamic[];
  __shared__ Control c;
  uint8_t* mem = reinterpret_cast<uint8_t*>(dynamic);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    c.abort_flag = 0;
    for (int s = 0; s < Geo::kStages; ++s) { mbar_init(&c.kv_full[s], 1); mbar_init(&c.kv_empty[s], Geo::kWarps); }
    for (int s = 0; s < kSegments; ++s) { mbar_init(&c.seg_full[s], 1); mbar_init(&c.seg_empty[s], Geo::kWarps); }
    fence_barrier_init();
  }
  griddep_wait();               // what the previous kernel on the stream wrote is visible
  int plen = 0;
  if (p.B > kWarpRequests) plen = find_share<Geo::kThreads>(p, c.start);
  __syncthreads();
  if (warp == Geo::kWarps) {
    if (p.B <= kWarpRequests) plen = find_share_by_warp(p, c.start);
    produce<D, kBlocks>(p, c, plen, mem + Geo::kRingAt);
    return;
  }
  const int r = lane >> 2;
  int unit = 0;
  for (int n = 0;; ++n) {
    const int e = n % kSegments;
    bool ok = warp_wait(c, &c.seg_full[e], (n / kSegments) & 1, p.status, kInfoAttnList);
    const Segment s = c.seg[e];
    arrive_warp(&c.seg_empty[e]);
    // (the vote also lets the last segment's outputs be read before this one's are written)
    if (warps_any<Geo::kWarps>(!ok) || !s.live) return;
    Warp<kBf16, D, kBlocks> u{p, c, lane, r, lane & 3, warp, (r & 1) * 4 + (r >> 1)};
    const int units = units_in(s);
    ok = u.run(s, mem + Geo::kRingAt, unit, units);
    unit += units;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      if (b > 0) warps_any<Geo::kWarps>(false);  // the last rows have been read
      u.hand(b, reinterpret_cast<float*>(mem + warp * Geo::kSlotBytes));
      if (warps_any<Geo::kWarps>(!ok)) return;
      finish<D, kBlocks>(p, c, s, 8 * b, mem, warp, lane);
    }
  }
}

template <bool kBf16, int D, int kBlocks>
cudaError_t launch(const Kv4Attn& p, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  constexpr int kBytes = Geometry<D, kBlocks>::kDynamic;
  cudaError_t e = allow_smem(kv4_few_kernel<kBf16, D, kBlocks>, kBytes, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(threads(kBlocks));
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_few_kernel<kBf16, D, kBlocks>, p);
}
template <bool kBf16, int D>
cudaError_t launch(const Kv4Attn& p, int rows, cudaStream_t s) {
  return rows > 8 ? launch<kBf16, D, 2>(p, s) : launch<kBf16, D, 1>(p, s);
}

}  // namespace

// A tile of 128 keys costs this kernel 0.55 of what the other needs for up to 64 rows where
// it has up to 8 (640000 own keys of 16 single tokens: 146 us, the other 257), 0.82 where it
// has up to 16 (4 tokens each: 212 and 257; at 80000 keys 50 and 48).  So it takes a call
// whose blocks have few rows unless a prefix shared by many of them outweighs their own keys,
// as far as the tables' sizes tell (8 blocks of 12 rows over 4096 shared keys and up to 900
// own ones: 32.8 us here, 27.8 there).
int kv4_few_rows(int T, int B, int G, int page, int prefix_cap, int table_width) {
  const int block = G * (B > 0 ? ceil_div(T, B) : T);  // rows of a request's block, on average
  if (block > 16) return 0;
  const int rows = block <= 8 ? 8 : 16;
  const long long prefix = tiles_of(prefix_cap * page), own = tiles_of(table_width * page);
  const long long few = ceil_div(T, rows / G), many = ceil_div(T, kRows / G);
  return 5 * (prefix * few + B * own) <= (rows == 8 ? 9 : 6) * (prefix * many + B * own) ? rows : 0;
}

cudaError_t launch_kv4_few(const Kv4Attn& p, int rows, int D, bool bf16, cudaStream_t s) {
  if (bf16) return D == 64 ? launch<true, 64>(p, rows, s) : launch<true, 128>(p, rows, s);
  return D == 64 ? launch<false, 64>(p, rows, s) : launch<false, 128>(p, rows, s);
}

}  // namespace moe
