// Matrix product with weights of 4 bits (moe_linear_q4): y = act(x W^T + bias) + residual,
// W[n, k] = s[n, k / g] (c[n, k] - z[n, k / g]), c and z whole numbers 0 .. 15, s 16-bit.
//
// No weight is rounded: the MMA multiplies the whole numbers c - z, which both 16-bit types
// hold exactly, and a group's fp32 sum is multiplied by its scale as it is added to the
// output's, in fp32.
//
// Bound by the bytes of the weights for few rows (4096 x 4096: 8.6 MB, 1.3 us), by the
// tensor cores for many.  In between stands the expansion: a word of 8 codes takes 11
// instructions (9 in f16) to become the operand.  As in the attention over a 4-bit cache
// the weights are the MMA's M side, so that a thread that holds a weight row expands it
// into its own lane of tensor memory, and the group's scale of that row is one register
// of the thread that adds the sums up: scales and zeros cost a multiplication a row and
// token and none a weight, and weights pass shared memory once.
//
// Layout (moe_q4_prepare, once a set of weights): for every 128 rows and 128 inputs one run
// of bytes, [4][128 rows][16 bytes] of codes (32 inputs of a row in 16 bytes, inputs 2 j and
// 2 j + 1 of every 8 in nibbles j and j + 4, where one mask finds both), then the groups'
// scales [128 / g][128 rows] and zeros.  A block is one copy, and a warp's lanes read 512
// bytes side by side.
//
// A CTA (one per SM): warp 0 copies weight blocks and token tiles into a ring of stages,
// warp 1 issues the MMAs, warpgroups 1 to 3 expand blocks in turn, warpgroup 4 adds the
// groups' sums up and runs the epilogue.  Few tiles are shared by clusters of CTAs, each a
// range of K, whose sums meet in distributed shared memory in rank order; of many, each CTA
// takes its share one after the other.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <string.h>

#include "epilogue.cuh"
#include "moe.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 640;
constexpr int kExpanders = 3;       // warpgroups that expand
constexpr int kBlock = 128;         // inputs of a block
constexpr int kRows = 128;          // weight rows of a tile
constexpr int kMaxTok = 128;        // tokens of a tile
constexpr int kSmem = 226 * 1024;
constexpr int kQ4Stages = 14;
constexpr int kMaxCluster = 8;
constexpr int kCodeBytes = kRows * kBlock / 2;
// tensor memory: the expanded blocks, then the groups' sums
constexpr uint32_t kSumsCol = kExpanders * (kBlock / 2);
constexpr int kSumsCols = 256, kMaxSums = 8;
// Registers a thread, moved between the warpgroups: 56 + 3 x 64 + 224 <= 5 x 96
constexpr int kRegsFew = 56, kRegsExpand = 64, kRegsSum = 224;

struct Q4Params {
  int M, N, K, k_blocks;
  int group, group_log2;     // inputs of a group: 32, 64 or 128
  int zeros;                 // 1: the groups have zero points (else 8)
  int block_bytes;           // of a weight block
  int n_tok, row_tiles, tok_tiles;
  int stages, cluster, sums; // sums: buffers of a group's sums in tensor memory
  const uint8_t* w;
  const uint16_t *bias, *residual;
  uint16_t* y;
  long long res_stride, y_stride;
  int act;
  int32_t* status;
};

struct Control {
  uint64_t full[kQ4Stages], empty[kQ4Stages];
  uint64_t a_full[kExpanders], a_empty[kExpanders];
  uint64_t d_full[kMaxSums], d_empty[kMaxSums], drain;
  uint32_t tmem;
  int abort_flag;
};

__host__ __device__ constexpr int block_bytes(int group, bool zeros) {
  return kCodeBytes + kBlock / group * kRows * (zeros ? 3 : 2);
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
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\ttcgen05.mma.cta_group::1."
      "kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
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
__device__ __forceinline__ uint32_t mask_or(uint32_t a, uint32_t mask, uint32_t magic) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "r"(mask), "r"(magic));
  return d;
}
// A type's numbers 2^e + z, in both halves: what is taken off a code that has been put
// into the mantissa of 2^e (bf16: 128; f16: 1024).
template <bool kBf16>
__device__ __forceinline__ uint32_t magic2(uint32_t z) {
  return (kBf16 ? 0x43004300u : 0x64006400u) + z * 0x00010001u;
}
template <bool kBf16>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  uint32_t d;
  if (kBf16) asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// 8 codes as whole numbers less z (off = magic2(z)), pairs of neighbouring inputs.  In f16
// a code may stay in the mantissa's next four bits, where it counts 16: 1024 + 16 c, of
// which a sixteenth less 64 + z (off16, negative) is exact too.
template <bool kBf16>
__device__ __forceinline__ void expand8(uint32_t w, uint32_t off, uint32_t off16, uint32_t* o) {
  if (kBf16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = sub2<true>(mask_or(w >> (4 * j), 0x000f000fu, 0x43004300u), off);
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t v = w >> (8 * j);
      o[2 * j] = sub2<false>(mask_or(v, 0x000f000fu, 0x64006400u), off);
      asm("fma.rn.f16x2 %0, %1, %2, %3;"
          : "=r"(o[2 * j + 1])
          : "r"(mask_or(v, 0x00f000f0u, 0x64006400u)), "r"(0x2c002c00u), "r"(off16));
    }
  }
}

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

// The tiles of a CTA (its cluster's, with this CTA's range of blocks of each): row tiles
// innermost, so that CTAs at work together read the same tokens.
struct Tiles {
  int at, step, end, kb0, kb1;
  __device__ Tiles(const Q4Params& p, int rank) {
    at = blockIdx.x / p.cluster;
    step = gridDim.x / p.cluster;
    end = p.row_tiles * p.tok_tiles;
    kb0 = static_cast<int>(static_cast<long long>(p.k_blocks) * rank / p.cluster);
    kb1 = static_cast<int>(static_cast<long long>(p.k_blocks) * (rank + 1) / p.cluster);
  }
};

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    linear_q4_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ Q4Params p) {
  extern __shared__ uint8_t dynamic[];
  __shared__ Control c;
  uint8_t* mem = dynamic + ((1024u - (smem_u32(dynamic) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = p.cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  const uint32_t x_bytes = p.n_tok * kBlock * 2, w_space = (p.block_bytes + 1023) / 1024 * 1024;
  const uint32_t stage_space = x_bytes + w_space;  // the token tile first: it is swizzled
  const int groups = kBlock >> p.group_log2;       // of a block
  const Tiles tiles(p, rank);

  if (tid == 0) {
    c.abort_flag = 0;
    for (int s = 0; s < p.stages; ++s) { mbar_init(&c.full[s], 1); mbar_init(&c.empty[s], 9); }
    for (int s = 0; s < kExpanders; ++s) { mbar_init(&c.a_full[s], 4); mbar_init(&c.a_empty[s], 1); }
    for (int s = 0; s < p.sums; ++s) { mbar_init(&c.d_full[s], 1); mbar_init(&c.d_empty[s], 4); }
    mbar_init(&c.drain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  // the first blocks come into L2 while the previous kernel ends (what it writes, weights
  // included, is read only after it)
  if (warp == 0 && lane < min(p.stages, tiles.kb1 - tiles.kb0) && tiles.at < tiles.end)
    bulk_prefetch_l2(p.w + (static_cast<long long>(tiles.at % p.row_tiles) * p.k_blocks + tiles.kb0 + lane) * p.block_bytes,
                     p.block_bytes);
  griddep_wait();  // what the previous kernel on the stream wrote is visible

  bool ok = true;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp == 0) {
      if (elect()) {
        const uint64_t pol = l2_evict_first_policy();
        Ring r;
        int filled = 0;
        for (int t = tiles.at; t < tiles.end && ok; t += tiles.step) {
          const uint8_t* w = p.w + static_cast<long long>(t % p.row_tiles) * p.k_blocks * p.block_bytes;
          const int t0 = t / p.row_tiles * p.n_tok;
          for (int kb = tiles.kb0; kb < tiles.kb1; ++kb) {
            ok = mbar_wait(&c.empty[r.stage], r.phase ^ 1u, &c.abort_flag);
            if (!ok) break;
            uint8_t* st = mem + r.stage * stage_space;
            mbar_arrive_expect_tx(&c.full[r.stage], x_bytes + p.block_bytes);
            // (weights that several token tiles read stay in L2)
            if (p.tok_tiles > 1) bulk_load(st + x_bytes, w + static_cast<long long>(kb) * p.block_bytes, p.block_bytes, &c.full[r.stage]);
            else bulk_load_hint(st + x_bytes, w + static_cast<long long>(kb) * p.block_bytes, p.block_bytes, &c.full[r.stage], pol);
            tma_load_2d(st, &tm_x, &c.full[r.stage], kb * kBlock, t0);
            tma_load_2d(st + x_bytes / 2, &tm_x, &c.full[r.stage], kb * kBlock + 64, t0);
            ++filled;
            r.next(p.stages);
          }
        }
        if (!ok) record_failure(p.status, &c.abort_flag, kInfoEmpty);
        // every copy that was issued has landed (also after a failure)
        for (int s = 0; s < p.stages; ++s) {
          const int fills = filled / p.stages + (s < filled % p.stages ? 1 : 0);
          if (fills > 0 && !mbar_wait(&c.full[s], (fills - 1) & 1, nullptr))
            record_failure(p.status, &c.abort_flag, kInfoDrain);
        }
      }
    } else if (warp == 1) {
      if (elect()) {
        const uint32_t id = kBf16 ? idesc_bf16(kRows, p.n_tok) : idesc_f16(kRows, p.n_tok);
        const int steps = 1 << (p.group_log2 - 4);  // MMAs of a group
        Ring r, a, d;
        for (int t = tiles.at; t < tiles.end && ok; t += tiles.step)
          for (int kb = tiles.kb0; kb < tiles.kb1 && ok; ++kb) {
            ok = mbar_wait(&c.full[r.stage], r.phase, &c.abort_flag) && mbar_wait(&c.a_full[a.stage], a.phase, &c.abort_flag);
            if (!ok) { record_failure(p.status, &c.abort_flag, kInfoFull); break; }
            const uint32_t b = kDescLoK + (smem_u32(mem + r.stage * stage_space) >> 4);
            const uint32_t at = tmem + a.stage * (kBlock / 2);
            for (int g = 0; g < groups; ++g) {
              ok = mbar_wait(&c.d_empty[d.stage], d.phase ^ 1u, &c.abort_flag);
              if (!ok) { record_failure(p.status, &c.abort_flag, kInfoAccEmpty); break; }
              tc_fence_after();
              const uint32_t sums = tmem + kSumsCol + d.stage * (kSumsCols / p.sums);
#pragma unroll 2
              for (int i = 0; i < steps; ++i) {
                const int ks = g * steps + i;
                mma_ts(sums, at + ks * 8, b + (ks / 4) * (x_bytes / 32) + (ks % 4) * 2, kDescHi, id, i > 0 ? 1u : 0u);
              }
              mma_commit(&c.d_full[d.stage]);
              d.next(p.sums);
            }
            mma_commit(&c.a_empty[a.stage]);
            mma_commit(&c.empty[r.stage]);
            a.next(kExpanders);
            r.next(p.stages);
          }
        // every MMA issued above has completed once `drain` flips
        mma_commit(&c.drain);
        if (!mbar_wait(&c.drain, 0, nullptr)) record_failure(p.status, &c.abort_flag, kInfoDrain);
      }
    }
  } else if (warp < 4 + 4 * kExpanders) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsExpand));
    // a thread a row; of three warpgroups, each takes every third block
    const int turn = warp / 4 - 1, row = tid & 127;
    const uint32_t dst = tmem + turn * (kBlock / 2) + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    Ring r;
    int n = 0;
    uint32_t phase = 1;
    for (int t = tiles.at; t < tiles.end && ok; t += tiles.step)
      for (int kb = tiles.kb0; kb < tiles.kb1; ++kb, ++n, r.next(p.stages)) {
        if (n % kExpanders != turn) {
          continue;
        }
        ok = warp_wait(c, &c.full[r.stage], r.phase, p.status, kInfoFull);
        if (!ok) break;
        ok = warp_wait(c, &c.a_empty[turn], phase, p.status, kInfoAccEmpty);
        if (!ok) break;
        phase ^= 1u;
        tc_fence_after();
        const uint8_t* st = mem + r.stage * stage_space + x_bytes;
        const uint8_t* zeros = st + kCodeBytes + groups * kRows * 2 + row;
        uint4 w = *reinterpret_cast<const uint4*>(st + row * 16);
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
          if (q < 3) w = *reinterpret_cast<const uint4*>(st + ((q + 1) * kRows + row) * 16);
          const uint32_t z = p.zeros ? zeros[(q * 32 >> p.group_log2) * kRows] : 8u;
          const uint32_t off = magic2<kBf16>(z);
          // -(64 + z) in f16: z counts 16 of its last bits
          const uint32_t off16 = 0xd400d400u + z * 0x00100010u;
          uint32_t o[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) expand8<kBf16>(x[i], off, off16, o + 4 * i);
          tmem_st16(dst + q * 16, o);
        }
        arrive_warp(&c.empty[r.stage]);
        tmem_st_wait();
        tc_fence_before();
        arrive_warp(&c.a_full[turn]);
      }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSum));
    // a thread a row: its outputs of all the tile's tokens
    const int row = tid & 127;
    const uint32_t src = tmem + kSumsCol + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    Ring r, d;
    for (int t = tiles.at; t < tiles.end && ok; t += tiles.step) {
      unsigned long long acc[kMaxTok / 2];
#pragma unroll
      for (int i = 0; i < kMaxTok / 2; ++i) acc[i] = 0ull;
      for (int kb = tiles.kb0; kb < tiles.kb1 && ok; ++kb) {
        ok = warp_wait(c, &c.full[r.stage], r.phase, p.status, kInfoFull);
        if (!ok) break;
        const uint16_t* scales =
            reinterpret_cast<const uint16_t*>(mem + r.stage * stage_space + x_bytes + kCodeBytes) + row;
        for (int g = 0; g < groups; ++g) {
          const float s = to_f<kBf16>(scales[g * kRows]);
          if (g == groups - 1) arrive_warp(&c.empty[r.stage]);
          ok = warp_wait(c, &c.d_full[d.stage], d.phase, p.status, kInfoAccFull);
          if (!ok) break;
          tc_fence_after();
          const unsigned long long s2 = pair(s, s);
          const uint32_t at = src + d.stage * (kSumsCols / p.sums);
#pragma unroll
          for (int i = 0; i < kMaxTok / 16; ++i)
            if (16 * i < p.n_tok) {
              uint32_t v[16];
              tmem_ld16(at + 16 * i, v);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 8; ++k)
                acc[8 * i + k] = fma2(pair(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), s2, acc[8 * i + k]);
            }
          tc_fence_before();
          arrive_warp(&c.d_empty[d.stage]);
          d.next(p.sums);
        }
        r.next(p.stages);
      }
      if (!ok) break;
      const int n = t % p.row_tiles * kRows + row, t0 = t / p.row_tiles * p.n_tok, toks = min(p.n_tok, p.M - t0);
      if (p.cluster == 1) {
        if (n < p.N) {
          const float bias = p.bias ? to_f<kBf16>(p.bias[n]) : 0.f;
          uint16_t* y = p.y + t0 * p.y_stride + n;
          const uint16_t* res = p.residual ? p.residual + t0 * p.res_stride + n : nullptr;
#pragma unroll
          for (int i = 0; i < kMaxTok / 2; ++i)
            if (2 * i < toks) {
              float v[2];
              unpair(acc[i], v[0], v[1]);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (2 * i + e < toks) {
                  float z = activate(v[e] + bias, p.act);
                  if (res) z += to_f<kBf16>(res[(2 * i + e) * p.res_stride]);
                  y[(2 * i + e) * p.y_stride] = from_f<kBf16>(z);
                }
            }
        }
      } else {
        // this CTA's sums, token-major, over the stages: all of them have been read (the
        // last group's sums were complete), and a cluster has one tile
        float* part = reinterpret_cast<float*>(mem);
#pragma unroll
        for (int i = 0; i < kMaxTok / 2; ++i)
          if (2 * i < toks) {
            float v[2];
            unpair(acc[i], v[0], v[1]);
            part[2 * i * kRows + row] = v[0];
            part[(2 * i + 1) * kRows + row] = v[1];
          }
      }
    }
  }
  __syncwarp();
  if (p.cluster > 1) {
    cluster_sync();
    const float* part = reinterpret_cast<const float*>(mem);
    const int n = tiles.at % p.row_tiles * kRows + lane * 4, t0 = tiles.at / p.row_tiles * p.n_tok;
    const int toks = min(p.n_tok, p.M - t0);
    const int ta = toks * rank / p.cluster, tb = toks * (rank + 1) / p.cluster;
    float bias[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.bias && n < p.N)
      for (int i = 0; i < 4; ++i) bias[i] = to_f<kBf16>(p.bias[n + i]);
    for (int t = ta + warp; t < tb; t += kThreads / 32) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t local = smem_u32(part + t * kRows + lane * 4);
      for (int q = 0; q < p.cluster; ++q) {
        const float4 f = ld_cluster4(local, q);
        v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
      }
      if (n < p.N) {
        ushort4 out;
        uint16_t* o = &out.x;
        for (int i = 0; i < 4; ++i) {
          float z = activate(v[i] + bias[i], p.act);
          if (p.residual) z += to_f<kBf16>(p.residual[(t0 + t) * p.res_stride + n + i]);
          o[i] = from_f<kBf16>(z);
        }
        *reinterpret_cast<ushort4*>(p.y + (t0 + t) * p.y_stride + n) = out;
      }
    }
    cluster_sync();  // the others have read this CTA's sums
  }
  // (y may be what a fused forward loads before it waits: see linear.cu)
  __threadfence();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- the weights' layout
// A thread a row and 32 inputs: codes two a byte, the even input in the low nibble, to
// words with inputs 2 j, 2 j + 1 in nibbles j, j + 4.  The first input of a group brings its
// scale and zero.  Rows past N and inputs past K: scale 0.
__device__ __forceinline__ uint32_t spread(uint32_t w) {
  uint32_t e = w & 0x0f0f0f0fu, o = (w >> 4) & 0x0f0f0f0fu;
  e = (e | e >> 4) & 0x00ff00ffu;
  o = (o | o >> 4) & 0x00ff00ffu;
  return ((e | e >> 8) & 0xffffu) | (((o | o >> 8) & 0xffffu) << 16);
}
__global__ void __launch_bounds__(256)
    q4_prepare_kernel(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int N, int K, int group,
                      int k_blocks, int bytes, uint8_t* out, long long units) {
  const long long u = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (u >= units) return;
  const int row = static_cast<int>(u % kRows), q = static_cast<int>(u / kRows % 4);
  const long long b = u / (4 * kRows);
  const int n = static_cast<int>(b / k_blocks) * kRows + row, k = static_cast<int>(b % k_blocks) * kBlock + q * 32;
  const bool live = n < N && k < K;
  uint8_t* block = out + b * bytes;
  uint4 w = make_uint4(0, 0, 0, 0);
  if (live) w = *reinterpret_cast<const uint4*>(codes + (static_cast<long long>(n) * K + k) / 2);
  *reinterpret_cast<uint4*>(block + (q * kRows + row) * 16) = make_uint4(spread(w.x), spread(w.y), spread(w.z), spread(w.w));
  if (q * 32 % group == 0) {
    const int g = q * 32 / group, groups = kBlock / group;
    const long long at = static_cast<long long>(n) * (K / group) + k / group;
    reinterpret_cast<uint16_t*>(block + kCodeBytes)[g * kRows + row] = live ? scales[at] : 0;
    if (zeros) (block + kCodeBytes + groups * kRows * 2)[g * kRows + row] = live ? zeros[at] : 0;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

moe_status check_weights(int N, int K, int group) {
  if (N < 1 || K < 1 || group < 1) return MOE_ERR_INVALID_ARG;
  if (N % 8 || (group != 32 && group != 64 && group != 128) || K % group || N > MOE_MAX_LINEAR || K > MOE_MAX_LINEAR)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// CTAs that share a tile: as many as the SMs hold at once, each with 4 blocks at least.
int cluster_size(int tiles, int k_blocks, int sms) {
  int c = 1;
  while (c < kMaxCluster && (c + 1) * tiles <= sms && k_blocks / (c + 1) >= 4) ++c;
  return c;
}

template <bool kBf16>
cudaError_t launch(const CUtensorMap& tm_x, const Q4Params& p, int grid, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(linear_q4_kernel<kBf16>, kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = p.cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_q4_kernel<kBf16>, tm_x, p);
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_q4_weight_bytes(int N, int K, int group, int has_zeros) {
  using namespace moe;
  if (check_weights(N, K, group) != MOE_OK) return 0;
  return static_cast<size_t>(ceil_div(N, kRows)) * ceil_div(K, kBlock) * block_bytes(group, has_zeros != 0);
}

moe_status moe_q4_prepare(const uint8_t* codes, const void* scales, const uint8_t* zeros, int N, int K, int group,
                          void* weights, size_t weight_bytes, cudaStream_t stream) {
  using namespace moe;
  const moe_status st = check_weights(N, K, group);
  if (st != MOE_OK) return st;
  if (!codes || !scales || !weights || !aligned16(codes) || !aligned16(weights)) return MOE_ERR_INVALID_ARG;
  const size_t need = moe_q4_weight_bytes(N, K, group, zeros != nullptr);
  if (weight_bytes < need) return MOE_ERR_WORKSPACE;
  const long long groups = static_cast<long long>(N) * (K / group);
  const RowSet out = {weights, 1, static_cast<long long>(need), 0};
  if (rows_meet(out, {codes, 1, static_cast<long long>(N) * K / 2, 0}) || rows_meet(out, {scales, 1, 2 * groups, 0}) ||
      rows_meet(out, {zeros, 1, groups, 0}))
    return MOE_ERR_INVALID_ARG;
  const int k_blocks = ceil_div(K, kBlock);
  const long long units = static_cast<long long>(ceil_div(N, kRows)) * k_blocks * 4 * kRows;
  if ((units + 255) / 256 > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  q4_prepare_kernel<<<static_cast<unsigned>((units + 255) / 256), 256, 0, stream>>>(
      codes, static_cast<const uint16_t*>(scales), zeros, N, K, group, k_blocks, block_bytes(group, zeros != nullptr),
      static_cast<uint8_t*>(weights), units);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_linear_q4_workspace_bytes(int M, int N, int K) {
  if (M < 0 || N < 1 || K < 1) return 0;
  if (N % 8 || K % 32 || M > MOE_MAX_LINEAR || N > MOE_MAX_LINEAR || K > MOE_MAX_LINEAR) return 0;
  return MOE_STATUS_BYTES;
}

moe_status moe_linear_q4(const void* x, long long x_stride, int M, int K, const void* weights, size_t weight_bytes, int N,
                         int group, int has_zeros, int dtype, const void* bias, int activation, const void* residual,
                         long long residual_stride, void* y, long long y_stride, void* ws, size_t ws_bytes,
                         cudaStream_t stream) {
  using namespace moe;
  if (M < 0) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_weights(N, K, group);
  if (st != MOE_OK) return st;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (has_zeros != 0 && has_zeros != 1) return MOE_ERR_INVALID_ARG;
  if (activation < MOE_ACT_NONE || activation > MOE_ACT_RELU) return MOE_ERR_INVALID_ARG;
  if (M > MOE_MAX_LINEAR) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!x || !weights || !y || x == y || weights == y) return MOE_ERR_INVALID_ARG;
  const size_t need = moe_q4_weight_bytes(N, K, group, has_zeros);
  if (weight_bytes < need) return MOE_ERR_INVALID_ARG;
  if (y_stride < N || (M > 1 && x_stride < K) || (residual && residual_stride < 0)) return MOE_ERR_INVALID_ARG;
  if (residual == y && residual_stride != y_stride) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(weights) || !aligned16(bias) || !aligned16(residual) || !aligned16(y))
    return MOE_ERR_INVALID_ARG;
  if (x_stride % 8 || y_stride % 8 || (residual && residual_stride % 8)) return MOE_ERR_UNSUPPORTED;
  const RowSet out = {y, M, 2ll * N, 2 * y_stride};
  if (rows_meet(out, {x, M, 2ll * K, 2 * x_stride}) || rows_meet(out, {weights, 1, static_cast<long long>(need), 0}) ||
      rows_meet(out, {bias, 1, 2ll * N, 0}) ||
      (residual != y && rows_meet(out, {residual, M, 2ll * N, 2 * residual_stride})))
    return MOE_ERR_INVALID_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kWsAlign) != 0 || ws_bytes < MOE_STATUS_BYTES)
    return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  Q4Params p;
  memset(&p, 0, sizeof(p));
  p.M = M; p.N = N; p.K = K;
  p.k_blocks = ceil_div(K, kBlock);
  p.group = group;
  p.group_log2 = group == 32 ? 5 : group == 64 ? 6 : 7;
  p.zeros = has_zeros;
  p.block_bytes = block_bytes(group, has_zeros != 0);
  p.row_tiles = ceil_div(N, kRows);
  p.tok_tiles = ceil_div(M, kMaxTok);
  p.n_tok = ceil_div(ceil_div(M, p.tok_tiles), 16) * 16;
  p.tok_tiles = ceil_div(M, p.n_tok);
  const long long tiles = static_cast<long long>(p.row_tiles) * p.tok_tiles;
  if (tiles > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  p.cluster = cluster_size(static_cast<int>(tiles < sms ? tiles : sms), p.k_blocks, sms);
  p.stages = (kSmem - 1024) / (p.n_tok * kBlock * 2 + ceil_div(p.block_bytes, 1024) * 1024);
  if (p.stages > kQ4Stages) p.stages = kQ4Stages;
  p.sums = kSumsCols / (p.n_tok <= 32 ? 32 : p.n_tok <= 64 ? 64 : 128);
  p.w = static_cast<const uint8_t*>(weights);
  p.bias = static_cast<const uint16_t*>(bias);
  p.residual = static_cast<const uint16_t*>(residual); p.res_stride = residual_stride;
  p.y = static_cast<uint16_t*>(y); p.y_stride = y_stride;
  p.act = activation;
  p.status = static_cast<int32_t*>(ws);
  const bool f16 = dtype == MOE_DTYPE_F16;
  CUtensorMap tm_x;
  const uint64_t xd[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(M)};
  const uint64_t xst[1] = {static_cast<uint64_t>(M > 1 ? x_stride : K) * 2};
  const uint32_t xb[2] = {64, static_cast<uint32_t>(p.n_tok)};
  if (!encode_map_16(&tm_x, f16, x, 2, xd, xst, xb)) return MOE_ERR_CUDA;
  const int grid = p.cluster * static_cast<int>(tiles < sms / p.cluster ? tiles : sms / p.cluster);
  const cudaError_t e = f16 ? launch<false>(tm_x, p, grid, stream) : launch<true>(tm_x, p, grid, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
