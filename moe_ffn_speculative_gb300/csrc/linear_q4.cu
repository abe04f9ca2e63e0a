// Matrix product with weights of 4 bits (moe_linear_q4): y = act(x W^T + bias) + residual,
// W[n, k] = s[n, k / g] (c[n, k] - z[n, k / g]), c and z whole numbers 0 .. 15, s 16-bit.
//
// No weight is rounded: (c - z) s has 12 significant bits in bf16 and 15 in f16, and goes to
// the MMA as two numbers of the type: the product rounded, and what that is too much, which
// one fused multiply-add gives exactly (its last bit is a multiple of the scale's, so that
// no range is lost) and the MMA negates.  Twice the products, but one sum a row and token
// from the first input to the last, which stays in tensor memory.  (Groups' sums of whole
// numbers, scaled as they were added up, were bound by their reading: 650 us at 2048 x 4096 x
// 12288 in groups of 64, 984 in groups of 32.)  The scales' products have to be in the type's
// range; an infinity in x meets a zero and gives NaN.
//
// The weights are the MMA's M side, so that a thread that holds a weight row expands it into
// its own lane of tensor memory: a row's scale and zero are one load a group, and weights pass
// shared memory once.  The expansion takes 19 instructions for a word of 8 codes.
//
// A CTA (one per SM): warp 0 copies weight blocks and token tiles into a ring of stages,
// warp 1 issues the MMAs, warpgroups 1 to 4 expand half a block each in turn, and
// warpgroups 5 and 6 run a tile's epilogue under the next one's products (one group: gelu took
// 317 us there).  Few tiles are shared by clusters of CTAs, each a range of K: the sums are
// written to the shared memory of the CTA that adds them up in rank order; of many, each CTA takes its share one after the
// other.
//
// Measured (floors in brackets): 2048 x 4096 x 12288, groups of 64, gelu, 236 us (106; the
// tensor cores' doubled work is 1.74 PFLOP/s, 0.9 of the measured cuBLAS rate); 72 x 4096 ->
// 6144 14.9 us (2.2), 64 x 4096 -> 4096 10.6.  There 5 us are prologue, fill and the cluster's
// meeting, the rest 0.55 us a block: of it without stores to tensor memory 0.4, without
// the arithmetic 0.42, without MMAs 0.5, with none of them 0.32, which is waits and issue.
// Six buffers of expanded weights in place of four, or two warps that issue, each with sums of
// its own, were not faster.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <string.h>

#include "epilogue.cuh"
#include "issue.cuh"
#include "linear_q4.cuh"
#include "moe.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 896;
constexpr int kExpanders = 4;       // warpgroups that expand, each with a buffer
constexpr int kHalf = kBlock / 2;   // inputs of a buffer
constexpr int kMaxTok = 128;        // tokens of a tile
constexpr int kSmem = 226 * 1024;
constexpr int kQ4Stages = 14;
constexpr int kMaxCluster = 8;
constexpr uint32_t kNegateA = 1u << 13;  // of an instruction descriptor
// tensor memory: the expanded halves (products rounded, then what they are too much), then
// two tiles' sums
constexpr uint32_t kSumsCol = kExpanders * kHalf;

struct Control {
  uint64_t full[kQ4Stages], empty[kQ4Stages];
  uint64_t a_full[kExpanders], a_empty[kExpanders];
  uint64_t d_full[2], d_empty[2], drain;
  uint32_t tmem;
  int abort_flag;
};

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// v s rounded, and what that is too much (minus = -s).
template <bool kBf16>
__device__ __forceinline__ void scale2(uint32_t v, uint32_t s, uint32_t minus, uint32_t& hi, uint32_t& over) {
  if (kBf16) {
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(v), "r"(s));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(over) : "r"(v), "r"(minus), "r"(hi));
  } else {
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(v), "r"(s));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(over) : "r"(v), "r"(minus), "r"(hi));
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
    kb0 = rank * p.blocks_each + min(rank, p.blocks_more);
    kb1 = kb0 + p.blocks_each + (rank < p.blocks_more ? 1 : 0);
  }
};

// The epilogue of a token's outputs [n, n + 4).
template <bool kBf16>
__device__ __forceinline__ void finish4(const Q4Params& p, const float4& sum, const ushort4& b, const ushort4& res, uint16_t* y) {
  float v[4] = {sum.x, sum.y, sum.z, sum.w};
  ushort4 out;
  uint16_t* o = &out.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = activate(v[i] + to_f<kBf16>((&b.x)[i]), p.act);
    o[i] = from_f<kBf16>(p.residual ? v[i] + to_f<kBf16>((&res.x)[i]) : v[i]);
  }
  *reinterpret_cast<ushort4*>(y) = out;
}

template <int kAct>
__device__ __forceinline__ void activate16(float (&v)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = activate(v[k], kAct);
}
// The epilogue of output n of tokens [t, t + m), m <= 16 (a warp's lanes: 32 outputs side by
// side).
template <bool kBf16>
__device__ __forceinline__ void finish16(const Q4Params& p, const uint32_t (&sum)[16], float b, int t, int m, int n) {
  uint16_t res[16] = {};
  if (p.residual) {
    const uint16_t* r = p.residual + t * p.res_stride + n;
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (k < m) res[k] = r[k * p.res_stride];
  }
  float v[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(sum[k]) + b;
  // (one branch for the 16)
  if (p.act == MOE_ACT_SILU) activate16<MOE_ACT_SILU>(v);
  else if (p.act == MOE_ACT_GELU) activate16<MOE_ACT_GELU>(v);
  else if (p.act == MOE_ACT_GELU_TANH) activate16<MOE_ACT_GELU_TANH>(v);
  else if (p.act == MOE_ACT_RELU) activate16<MOE_ACT_RELU>(v);
  uint16_t* y = p.y + t * p.y_stride + n;
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (k < m) y[k * p.y_stride] = from_f<kBf16>(p.residual ? v[k] + to_f<kBf16>(res[k]) : v[k]);
}

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
  float* sums = reinterpret_cast<float*>(mem + p.stages * stage_space);  // of a cluster: [rank][slots][kRows]
  const int groups = kBlock >> p.group_log2;       // of a block
  const Tiles tiles(p, rank);

  if (warp == 0) {
    if (lane < p.stages) { mbar_init(&c.full[lane], 1); mbar_init(&c.empty[lane], 9); }
    if (lane < kExpanders) { mbar_init(&c.a_full[lane], 4); mbar_init(&c.a_empty[lane], 1); }
    if (lane < 2) { mbar_init(&c.d_full[lane], 1); mbar_init(&c.d_empty[lane], 8); }
    if (lane == 0) {
      c.abort_flag = 0;
      mbar_init(&c.drain, 1);
      tma_prefetch_desc(&tm_x);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.cluster > 1) cluster_arrive_relaxed();  // the others may write to its memory
  const uint32_t tmem = c.tmem;
  // the first blocks come into L2 while the previous kernel ends (what it writes, weights
  // included, is read only after it)
  if (warp == 0 && lane < min(p.stages, tiles.kb1 - tiles.kb0) && tiles.at < tiles.end)
    bulk_prefetch_l2(p.w + (static_cast<long long>(tiles.at % p.row_tiles) * p.k_blocks + tiles.kb0 + lane) * p.block_bytes,
                     p.block_bytes);
  griddep_wait();  // what the previous kernel on the stream wrote is visible

  bool ok = true;
  if (warp < 4) {
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
      // all lanes go along, so that addresses stay uniform; one issues
      const uint32_t lead = elect() ? 1u : 0u;
      const uint32_t id = kBf16 ? idesc_bf16(kRows, p.n_tok) : idesc_f16(kRows, p.n_tok);
      const uint32_t b_base = kDescLoK + (smem_u32(mem) >> 4), b_stage = stage_space >> 4, b_half = x_bytes >> 5;
      Ring r;
      uint32_t a_phase = 0, turn = 0, tile = 0;
      for (int t = tiles.at; t < tiles.end && ok; t += tiles.step, ++tile) {
        const uint32_t d = tmem + kSumsCol + (tile & 1) * kMaxTok;
        ok = warp_wait(c, &c.d_empty[tile & 1], (tile >> 1 & 1) ^ 1u, p.status, kInfoAccEmpty);
        if (!ok) break;
        uint32_t more = 0;
        bool ready = false;
        for (int kb = tiles.kb0; kb < tiles.kb1; ++kb) {
          uint32_t b = b_base + r.stage * b_stage;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // (the expanders have seen the stage's copies land, the tokens' with the weights')
            if (!ready) ok = warp_wait(c, &c.a_full[turn], a_phase, p.status, kInfoFull);
            if (!ok) break;
            tc_fence_after();
            // the next buffer is asked after while these products are issued
            const uint32_t a = tmem + turn * kHalf, a_next = turn + 1 < kExpanders ? turn + 1 : 0;
            const uint32_t next_phase = a_next ? a_phase : a_phase ^ 1u;
            const bool next = mbar_test_wait(&c.a_full[a_next], next_phase);
#pragma unroll
            for (int i = 0; i < kHalf / 16; ++i) {
              mma_ts_by(lead, d, a + i * 8, b + i * 2, id, i ? 1u : more);
              mma_ts_by(lead, d, a + kHalf / 2 + i * 8, b + i * 2, id | kNegateA, 1u);
            }
            more = 1u;
            mma_commit_by(lead, &c.a_empty[turn]);
            b += b_half;
            turn = a_next;
            a_phase = next_phase;
            ready = __all_sync(0xffffffffu, next);
          }
          if (!ok) break;
          mma_commit_by(lead, &c.empty[r.stage]);
          r.next(p.stages);
        }
        if (ok) mma_commit_by(lead, &c.d_full[tile & 1]);
      }
      // every MMA issued above has completed once `drain` flips
      mma_commit_by(lead, &c.drain);
      if (!mbar_wait(&c.drain, 0, nullptr) && lead) record_failure(p.status, &c.abort_flag, kInfoDrain);
    }
  } else if (warp < 4 + 4 * kExpanders) {
    // a thread a row; of four warpgroups, each takes every second block's first or second half
    const int turn = warp / 4 - 1, row = tid & 127, half = turn & 1;
    const uint32_t dst = tmem + turn * kHalf + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    Ring r;
    int odd = 0;
    uint32_t phase = 1;
    for (int t = tiles.at; t < tiles.end && ok; t += tiles.step)
      for (int kb = tiles.kb0; kb < tiles.kb1; ++kb, odd ^= 1, r.next(p.stages)) {
        if (odd != turn >> 1) continue;
        // (first the products of the block before the last: then every copy up to that one has
        // landed, and the stage's parity can mean only this block's, with three stages too)
        ok = warp_wait(c, &c.a_empty[turn], phase, p.status, kInfoAccEmpty);
        if (!ok) break;
        phase ^= 1u;
        tc_fence_after();
        ok = warp_wait(c, &c.full[r.stage], r.phase, p.status, kInfoFull);
        if (!ok) break;
        const uint8_t* st = mem + r.stage * stage_space + x_bytes;
        uint4 w = *reinterpret_cast<const uint4*>(st + (half * 2 * kRows + row) * 16);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
          if (q == 0) w = *reinterpret_cast<const uint4*>(st + ((half * 2 + 1) * kRows + row) * 16);
          const int g = ((half * 2 + q) * 32 >> p.group_log2) * kRows + row;
          uint32_t s = reinterpret_cast<const uint16_t*>(st + kCodeBytes)[g];
          s |= s << 16;
          const uint32_t minus = s ^ 0x80008000u;
          const uint32_t z = p.zeros ? st[kCodeBytes + groups * kRows * 2 + g] : 8u;
          const uint32_t off = magic2<kBf16>(z);
          // -(64 + z) in f16: z counts 16 of its last bits
          const uint32_t off16 = 0xd400d400u + z * 0x00100010u;
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            uint32_t hi[8], over[8];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t v[4];
              expand8<kBf16>(x[i + e], off, off16, v);
#pragma unroll
              for (int k = 0; k < 4; ++k) scale2<kBf16>(v[k], s, minus, hi[4 * e + k], over[4 * e + k]);
            }
            tmem_st8(dst + q * 16 + i * 4, hi);
            tmem_st8(dst + kHalf / 2 + q * 16 + i * 4, over);
          }
        }
        arrive_warp(&c.empty[r.stage]);
        tmem_st_wait();
        tc_fence_before();
        arrive_warp(&c.a_full[turn]);
      }
  } else {
    // a thread a row, 16 tokens at a time, of two warpgroups each takes every second 16
    const int row = tid & 127, first = (warp / 4 - 1 - kExpanders) * 16;
    const uint32_t lanes = tmem + kSumsCol + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    uint32_t tile = 0;
    for (int t = tiles.at; t < tiles.end && ok && p.cluster == 1; t += tiles.step, ++tile) {
      ok = warp_wait(c, &c.d_full[tile & 1], tile >> 1 & 1, p.status, kInfoAccFull);
      if (!ok) break;
      tc_fence_after();
      const int t0 = t / p.row_tiles * p.n_tok, toks = min(p.n_tok, p.M - t0);
      const uint32_t src = lanes + (tile & 1) * kMaxTok;
      const int n = t % p.row_tiles * kRows + row;
      const float b = p.bias && n < p.N ? to_f<kBf16>(p.bias[n]) : 0.f;
      for (int i = first; i < toks; i += 32) {
        uint32_t v[16];
        tmem_ld16(src + i, v);
        tmem_ld_wait();
        if (n < p.N) finish16<kBf16>(p, v, b, t0 + i, min(16, toks - i), n);
        __syncwarp();
      }
      tc_fence_before();
      arrive_warp(&c.d_empty[tile & 1]);
    }
  }
  __syncwarp();
  if (p.cluster > 1) {
    // the c-th 8 tokens' sums to rank c % cluster, which adds up what the ranks write there: all
    // warpgroups but the first, 16 tokens at a time
    const int toks = min(p.n_tok, p.M - tiles.at / p.row_tiles * p.n_tok);
    cluster_wait();
    if (warp >= 4 && ok && warp_wait(c, &c.d_full[0], 0, p.status, kInfoAccFull)) {
      tc_fence_after();
      const uint32_t src = tmem + kSumsCol + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      int q = (warp / 4 - 1) * 2, slot = 0;
      for (int i = q * 8; i < toks; i += (kThreads / 128 - 1) * 16, q += (kThreads / 128 - 2) * 2) {
        uint32_t v[16];
        tmem_ld16(src + i, v);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < 2; ++h, ++q) {
          while (q >= p.cluster) { q -= p.cluster; slot += 8; }
          const uint32_t to = of_rank(smem_u32(sums + (rank * p.slots + slot) * kRows + (tid & 127)), q);
#pragma unroll
          for (int k = 0; k < 8; ++k) st_cluster(to + k * kRows * 4, __uint_as_float(v[8 * h + k]));
        }
      }
      tc_fence_before();
    }
    // this CTA's tokens, a warp each and a lane 4 outputs; what the epilogue reads comes while
    // the others finish
    constexpr int kWarps = kThreads / 32, kEach = (kMaxTok / 2 + kWarps - 1) / kWarps;
    const int n = tiles.at % p.row_tiles * kRows + lane * 4, t0 = tiles.at / p.row_tiles * p.n_tok;
    ushort4 b = make_ushort4(0, 0, 0, 0), res[kEach];
    if (p.bias && n < p.N) b = __ldg(reinterpret_cast<const ushort4*>(p.bias + n));
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int slot = warp + i * kWarps, t = ((slot >> 3) * p.cluster + rank) * 8 + (slot & 7);
      res[i] = make_ushort4(0, 0, 0, 0);
      if (p.residual && n < p.N && slot < p.slots && t < toks) res[i] = *reinterpret_cast<const ushort4*>(p.residual + (t0 + t) * p.res_stride + n);
    }
    cluster_sync();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int slot = warp + i * kWarps, t = ((slot >> 3) * p.cluster + rank) * 8 + (slot & 7);
      if (slot >= p.slots || t >= toks || n >= p.N) continue;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int q = 0; q < p.cluster; ++q) {
        const float4 f = *reinterpret_cast<const float4*>(sums + (q * p.slots + slot) * kRows + lane * 4);
        v.x += f.x; v.y += f.y; v.z += f.z; v.w += f.w;
      }
      finish4<kBf16>(p, v, b, res[i], p.y + (t0 + t) * p.y_stride + n);
    }
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

// How many clusters of c CTAs fit on the current device at once (0 on failure), asked once
// a device and size, of an empty kernel of the same shape (see linear.cu).
__global__ void __launch_bounds__(kThreads, 1) q4_shape_kernel() {}

int resident_clusters(int c) {
  static std::atomic<int> known[kMaxCluster + 1][64];
  int d = 0;
  if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= 64) return 0;
  int n = known[c][d].load(std::memory_order_relaxed);
  if (n > 0) return n;
  static std::atomic<uint64_t> done{0};
  if (allow_smem(q4_shape_kernel, kSmem, done) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(c * 1024);  // more than fit
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = c;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, q4_shape_kernel, &cfg) != cudaSuccess) return 0;
  known[c][d].store(n, std::memory_order_relaxed);
  return n;
}

// CTAs that share a tile: as many as are resident at once, each with 2 blocks at least.  (64
// x 4096 -> 4096: 21.6 us with one, 15.2 with two, 10.6 with the four that fit; 30 x 4096 ->
// 1024: 21.0, 14.4 and, with eight, 7.7.)
int cluster_size(int tiles, int k_blocks, int sms) {
  int c = 1;
  while (c < kMaxCluster && (c + 1) * tiles <= sms && k_blocks / (c + 1) >= 2 && resident_clusters(c + 1) >= tiles) ++c;
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
  p.w = static_cast<const uint8_t*>(weights);
  p.bias = static_cast<const uint16_t*>(bias);
  p.residual = static_cast<const uint16_t*>(residual); p.res_stride = residual_stride;
  p.y = static_cast<uint16_t*>(y); p.y_stride = y_stride;
  p.act = activation;
  p.status = static_cast<int32_t*>(ws);
  const bool f16 = dtype == MOE_DTYPE_F16;
  if (M <= kQ4FewRows) return launch_linear_q4_few(f16, p, x, x_stride, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  p.row_tiles = ceil_div(N, kRows);
  p.tok_tiles = ceil_div(M, kMaxTok);
  p.n_tok = ceil_div(ceil_div(M, p.tok_tiles), 16) * 16;
  p.tok_tiles = ceil_div(M, p.n_tok);
  const long long tiles = static_cast<long long>(p.row_tiles) * p.tok_tiles;
  if (tiles > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  p.cluster = cluster_size(static_cast<int>(tiles < sms ? tiles : sms), p.k_blocks, sms);
  p.blocks_each = p.k_blocks / p.cluster;
  p.blocks_more = p.k_blocks % p.cluster;
  p.slots = p.cluster > 1 ? ceil_div(p.n_tok / 8, p.cluster) * 8 : 0;
  p.stages = (kSmem - 1024 - p.slots * p.cluster * kRows * 4) / (p.n_tok * kBlock * 2 + ceil_div(p.block_bytes, 1024) * 1024);
  if (p.stages > kQ4Stages) p.stages = kQ4Stages;
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
