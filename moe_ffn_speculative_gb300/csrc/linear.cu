// Matrix product with bias, activation and residual in its epilogue
// (moe_linear): y = act(x W^T + bias) + residual, W [N, K].
//
// Few rows (few_rows): bound by the bytes of W, which are read once.  The 128 rows of a
// weight tile are the MMA's M dimension and up to 128 tokens its N dimension;
// a cluster of CTAs shares a weight tile, each taking a range of K, so that a
// layer with few tiles still occupies the SMs.  The CTAs' fp32 sums meet in
// distributed shared memory: every CTA adds its share of the tokens over the
// cluster in rank order (the result does not depend on timing) and applies
// the epilogue.
//
// A CTA: warp 0 loads weight and token tiles by TMA into a ring of stages,
// warp 1 issues the MMAs, warps 2..5 drain tensor memory.
//
// Many rows: bound by the tensor cores.  Pairs of CTAs work on tiles of 256
// tokens by up to 256 outputs (linear_many_kernel): each CTA holds 128 token
// rows and half of the tile's weight rows, and the pair's MMA reads both
// halves, so a byte of shared memory feeds twice the products.  The pairs are
// persistent; two accumulators in tensor memory let a tile's epilogue run
// under the next tile's products.  The tile's width is chosen so that the last
// wave of tiles is full.
//
// Neither kernel signals its dependents before it is complete, although its own
// start may overlap its predecessor's end: y may be the expert weights of a fused
// forward, which loads the first of them before it waits.  For the same reason
// the writers fence at their end, before the last CTA's exit lets a dependent
// start (0.15 us of 9 for 9 rows, nothing of 229 for 4096; the tables below were
// measured without it).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include "moe.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kLinThreads = 192;
// Half an SM's shared memory: two CTAs are resident, so that clusters of more CTAs
// than there are SMs run at once, and, behind a kernel that signals its dependents
// early, a launch's CTAs (and their first weights' way into L2) start while it ends.
constexpr int kLinSmem = 112 * 1024;
constexpr int kLinMaxStages = 12;
constexpr int kFewTokens = 128;          // most rows of linear_few_kernel, one tile of tokens
constexpr int kMaxCluster = 8;

struct LinearParams {
  int M, N, K, k_blocks;
  int n_tok;                 // few rows: tokens of a tile; many: its outputs (a multiple of 16)
  int stages, cluster;
  uint32_t tmem_cols;
  const uint16_t *bias, *residual;
  uint16_t* y;
  long long res_stride, y_stride;
  int act;
  int32_t* status;
};

struct LinearControl {
  uint64_t full[kLinMaxStages], empty[kLinMaxStages], acc, drain;
  uint32_t tmem;
  int abort_flag;
};

template <bool kBf16>
__device__ __forceinline__ float to_f(uint16_t u) {
  if (kBf16) return __bfloat162float(__ushort_as_bfloat16(u));
  return __half2float(__ushort_as_half(u));
}
template <bool kBf16>
__device__ __forceinline__ uint16_t from_f(float v) {
  if (kBf16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  return __half_as_ushort(__float2half_rn(v));
}

// v sigmoid(v) and the like through one exponential (the quotient is 0 where it
// has run over); erfc keeps gelu's negative tail from cancelling.
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case MOE_ACT_SILU: return __fdividef(v, 1.f + __expf(-v));
    case MOE_ACT_GELU: return 0.5f * v * erfcf(-v * 0.70710678118654752f);
    case MOE_ACT_GELU_TANH:
      return __fdividef(v, 1.f + __expf(-1.5957691216057308f * (v + 0.044715f * v * v * v)));
    case MOE_ACT_RELU: return v <= 0.f ? 0.f : v;  // NaN stays NaN (fmaxf returns the other operand)
    default: return v;
  }
}

__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t local, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

template <bool kBf16>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_few_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const __grid_constant__ LinearParams p) {
  extern __shared__ uint8_t dynamic[];
  __shared__ LinearControl c;
  uint8_t* ring_mem = dynamic + ((1024u - (smem_u32(dynamic) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = p.cluster > 1 ? cluster_rank() : 0;
  const int n0 = (blockIdx.x / p.cluster) * kHalfRows;
  const int kb0 = static_cast<int>(static_cast<long long>(p.k_blocks) * rank / p.cluster);
  const int kb1 = static_cast<int>(static_cast<long long>(p.k_blocks) * (rank + 1) / p.cluster);
  const uint32_t stage_bytes = kTileBytesA + p.n_tok * 128;

  if (tid == 0) {
    c.abort_flag = 0;
    for (int s = 0; s < p.stages; ++s) { mbar_init(&c.full[s], 1); mbar_init(&c.empty[s], 1); }
    mbar_init(&c.acc, 1);
    mbar_init(&c.drain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  // the weights' first tiles come into L2 while the previous kernel ends (what
  // it writes, weights included, is read only after it)
  if (warp == 0 && elect())
    for (int kb = kb0; kb < min(kb1, kb0 + kLinMaxStages); ++kb) tma_prefetch_2d(&tm_w, kb * kBlockK, n0);
  griddep_wait();  // what the previous kernel on the stream wrote is visible

  bool ok = true;
  if (warp == 0) {
    if (elect()) {
      const uint64_t pol = l2_evict_first_policy();
      Ring r;
      int filled = 0;
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        ok = mbar_wait(&c.empty[r.stage], r.phase ^ 1u, &c.abort_flag);
        if (!ok) break;
        uint8_t* a = ring_mem + r.stage * stage_bytes;
        mbar_arrive_expect_tx(&c.full[r.stage], stage_bytes);
        tma_load_2d_hint(a, &tm_w, &c.full[r.stage], kb * kBlockK, n0, pol);
        tma_load_2d(a + kTileBytesA, &tm_x, &c.full[r.stage], kb * kBlockK, 0);
        ++filled;
        r.next(p.stages);
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
      const uint32_t id = kBf16 ? idesc_bf16(kHalfRows, p.n_tok) : idesc_f16(kHalfRows, p.n_tok);
      Ring r;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = mbar_wait(&c.full[r.stage], r.phase, &c.abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = kDescLoK + (smem_u32(ring_mem + r.stage * stage_bytes) >> 4), b = a + kTileBytesA / 16;
#pragma unroll
        for (int ks = 0; ks < kBlockK / 16; ++ks)
          mma_ss(tmem, a + 2 * ks, kDescHi, b + 2 * ks, kDescHi, id, (kb > kb0 || ks > 0) ? 1u : 0u);
        mma_commit(&c.empty[r.stage]);
        r.next(p.stages);
      }
      if (!ok) record_failure(p.status, &c.abort_flag, kInfoFull);
      mma_commit(&c.acc);
      mma_commit(&c.drain);
      if (!mbar_wait(&c.drain, 0, nullptr)) record_failure(p.status, &c.abort_flag, kInfoDrain);
    }
  } else {
    ok = mbar_wait(&c.acc, 0, &c.abort_flag);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0) record_failure(p.status, &c.abort_flag, kInfoAccFull);
    tc_fence_after();
  }

  // the tile's rows are lanes; warp w of 2..5 reads lanes 32 (w % 4) ..
  const int row = (warp & 3) * 32 + lane;
  const int toks = p.M;
  if (p.cluster == 1) {
    if (warp >= 2 && ok) {
      const int n = n0 + row;
      const float bias = (p.bias && n < p.N) ? to_f<kBf16>(p.bias[n]) : 0.f;
      for (int t = 0; t < toks; t += 16) {
        uint32_t r[16];
        tmem_ld16(tmem + t + (static_cast<uint32_t>((warp & 3) * 32) << 16), r);
        tmem_ld_wait();
        if (n < p.N)
          for (int i = 0; i < 16 && t + i < toks; ++i) {
            float v = activate(__uint_as_float(r[i]) + bias, p.act);
            if (p.residual) v += to_f<kBf16>(p.residual[(t + i) * p.res_stride + n]);
            p.y[(t + i) * p.y_stride + n] = from_f<kBf16>(v);
          }
      }
    }
  } else {
    // this CTA's sums, token-major, over the stages (all of them consumed)
    float* part = reinterpret_cast<float*>(ring_mem);
    if (warp >= 2 && ok) {
      for (int t = 0; t < toks; t += 16) {
        uint32_t r[16];
        tmem_ld16(tmem + t + (static_cast<uint32_t>((warp & 3) * 32) << 16), r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(t + i) * kHalfRows + row] = __uint_as_float(r[i]);
      }
    }
    cluster_sync();
    const int n = n0 + lane * 4;
    const int ta = toks * static_cast<int>(rank) / p.cluster, tb = toks * static_cast<int>(rank + 1) / p.cluster;
    float bias[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.bias && n < p.N)
      for (int i = 0; i < 4; ++i) bias[i] = to_f<kBf16>(p.bias[n + i]);
    for (int t = ta + warp; t < tb; t += kLinThreads / 32) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t local = smem_u32(part + t * kHalfRows + lane * 4);
      for (int q = 0; q < p.cluster; ++q) {
        const float4 f = ld_cluster4(local, q);
        v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
      }
      if (n < p.N) {
        ushort4 out;
        uint16_t* o = &out.x;
        for (int i = 0; i < 4; ++i) {
          float z = activate(v[i] + bias[i], p.act);
          if (p.residual) z += to_f<kBf16>(p.residual[t * p.res_stride + n + i]);
          o[i] = from_f<kBf16>(z);
        }
        *reinterpret_cast<ushort4*>(p.y + t * p.y_stride + n) = out;
      }
    }
    cluster_sync();  // the others have read this CTA's sums
  }
  __threadfence();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

// ---------------------------------------------------------------- many rows: CTA pairs
constexpr int kManyThreads = 320;  // producer, issuer, 8 epilogue warps
constexpr int kManyEpiWarps = 8;
constexpr int kManyStages = 10;    // most stages: as many as fit
constexpr int kManySmem = 226 * 1024;
constexpr int kManyRows = 256;     // tokens of a tile, 128 a CTA
constexpr int kManyWide = 256;     // widest tile, in outputs

struct ManyControl {
  uint64_t full[kManyStages], empty[kManyStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int abort_flag;
};

__device__ __forceinline__ uint32_t map_rank(const void* local, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  return a;
}
// TMA load into this CTA's shared memory, counted on a barrier of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
// mma_ss over both CTAs' halves.
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, "
      "%3};\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at the same place in both CTAs of the pair when the
// MMAs issued so far are complete.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <bool kBf16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = to_f<kBf16>(static_cast<uint16_t>(w[i] & 0xffffu));
    f[2 * i + 1] = to_f<kBf16>(static_cast<uint16_t>(w[i] >> 16));
  }
}
template <bool kBf16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = static_cast<uint32_t>(from_f<kBf16>(f[2 * i])) | (static_cast<uint32_t>(from_f<kBf16>(f[2 * i + 1])) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The residual of one row's outputs [n, n + 32), those below `end` (both
// multiples of 8).
__device__ __forceinline__ void load_residual(const LinearParams& p, int t, int n, int end, uint4 (&res)[4]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    res[h] = make_uint4(0, 0, 0, 0);
    if (p.residual && t < p.M && n + 8 * h < end)
      res[h] = *reinterpret_cast<const uint4*>(p.residual + t * p.res_stride + n + 8 * h);
  }
}
// One row's outputs [n, n + 32) of those below `end`.
template <bool kBf16, int kAct>
__device__ __forceinline__ void finish32(const LinearParams& p, uint32_t taddr, int t, int n, int end,
                                         const uint4 (&res)[4]) {
  uint32_t r[32];
  tmem_ld16(taddr, *reinterpret_cast<uint32_t(*)[16]>(r));
  tmem_ld16(taddr + 16, *reinterpret_cast<uint32_t(*)[16]>(r + 16));
  tmem_ld_wait();
  if (t >= p.M) return;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    if (n + 8 * h >= end) break;
    float v[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[8 * h + i]);
    if (p.bias) {
      unpack8<kBf16>(__ldg(reinterpret_cast<const uint4*>(p.bias + n + 8 * h)), b);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += b[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = activate(v[i], kAct);
    if (p.residual) {
      unpack8<kBf16>(res[h], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += b[i];
    }
    *reinterpret_cast<uint4*>(p.y + t * p.y_stride + n + 8 * h) = pack8<kBf16>(v);
  }
}

template <bool kBf16, int kAct>
__global__ void __launch_bounds__(kManyThreads, 1)
    linear_many_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                       const __grid_constant__ LinearParams p) {
  extern __shared__ uint8_t dynamic[];
  __shared__ ManyControl c;
  uint8_t* ring_mem = dynamic + ((1024u - (smem_u32(dynamic) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const int wide = p.n_tok;  // outputs of a tile
  const int t_tiles = ceil_div(p.M, kManyRows), tiles = t_tiles * ceil_div(p.N, wide);
  const uint32_t stage_bytes = kTileBytesA + static_cast<uint32_t>(wide / 2) * 128;
  // stages start on 1024 bytes: the swizzle's period
  const uint32_t stage_space = (stage_bytes + 1023u) & ~1023u;
  const int stages = p.stages;

  if (tid == 0) {
    c.abort_flag = 0;
    for (int s = 0; s < stages; ++s) { mbar_init(&c.full[s], 1); mbar_init(&c.empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&c.acc_full[b], 1); mbar_init(&c.acc_empty[b], 2 * kManyEpiWarps); }
    mbar_init(&c.drain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&c.tmem)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are set up
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  griddep_wait();

  if (warp == 0) {
    // this CTA's 128 token rows and its half of the tile's weight rows
    if (elect()) {
      Ring r;
      int filled = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles && ok; tile += pairs) {
        const int t0 = (tile % t_tiles) * kManyRows + static_cast<int>(rank) * 128;
        const int n0 = (tile / t_tiles) * wide + static_cast<int>(rank) * (wide / 2);
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          ok = mbar_wait(&c.empty[r.stage], r.phase ^ 1u, &c.abort_flag);
          if (!ok) break;
          uint8_t* a = ring_mem + r.stage * stage_space;
          if (rank == 0) mbar_arrive_expect_tx(&c.full[r.stage], 2 * stage_bytes);
          const uint32_t bar = map_rank(&c.full[r.stage], 0);
          tma_load_2d_pair(a, &tm_x, bar, kb * kBlockK, t0);
          tma_load_2d_pair(a + kTileBytesA, &tm_w, bar, kb * kBlockK, n0);
          ++filled;
          r.next(stages);
        }
      }
      if (!ok) record_failure(p.status, &c.abort_flag, kInfoEmpty);
      // both CTAs' copies are counted on the leader's barriers
      if (rank == 0)
        for (int s = 0; s < stages; ++s) {
          const int fills = filled / stages + (s < filled % stages ? 1 : 0);
          if (fills > 0 && !mbar_wait(&c.full[s], (fills - 1) & 1, nullptr))
            record_failure(p.status, &c.abort_flag, kInfoDrain);
        }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect()) {
      const uint32_t id = kBf16 ? idesc_bf16(kManyRows, wide) : idesc_f16(kManyRows, wide);
      Ring r;
      bool ok = true;
      int i = 0;
      for (int tile = pair; tile < tiles && ok; tile += pairs, ++i) {
        const int buf = i & 1;
        ok = mbar_wait(&c.acc_empty[buf], ((i >> 1) & 1) ^ 1u, &c.abort_flag);
        if (!ok) { record_failure(p.status, &c.abort_flag, kInfoAccEmpty); break; }
        tc_fence_after();
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          ok = mbar_wait(&c.full[r.stage], r.phase, &c.abort_flag);
          if (!ok) { record_failure(p.status, &c.abort_flag, kInfoFull); break; }
          tc_fence_after();
          const uint32_t a = kDescLoK + (smem_u32(ring_mem + r.stage * stage_space) >> 4), b = a + kTileBytesA / 16;
#pragma unroll
          for (int ks = 0; ks < kBlockK / 16; ++ks)
            mma_pair(tmem + buf * kManyWide, a + 2 * ks, b + 2 * ks, id, (kb > 0 || ks > 0) ? 1u : 0u);
          commit_pair(&c.empty[r.stage]);
          r.next(stages);
        }
        commit_pair(&c.acc_full[buf]);
      }
      commit_pair(&c.drain);
      if (!mbar_wait(&c.drain, 0, nullptr)) record_failure(p.status, &c.abort_flag, kInfoDrain);
    }
  } else {
    // rows are lanes; two warps a 32-lane quarter, a half of the columns each
    const int quarter = warp & 3, half = (warp - 2) / 4;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int split = ((wide / 2 + 31) / 32) * 32;
    int i = 0;
    for (int tile = pair; tile < tiles; tile += pairs, ++i) {
      const int buf = i & 1;
      const int t = (tile % t_tiles) * kManyRows + static_cast<int>(rank) * 128 + quarter * 32 + lane;
      const int n0 = (tile / t_tiles) * wide, end = min(n0 + wide, p.N);
      const int first = n0 + (half ? split : 0), last = half ? end : min(n0 + split, end);
      // the residual, 32 columns ahead of the sums
      uint4 res[4], next[4];
      load_residual(p, t, first, last, res);
      const bool got = mbar_wait(&c.acc_full[buf], (i >> 1) & 1, &c.abort_flag);
      if (!__all_sync(0xffffffffu, got)) {
        if (lane == 0) record_failure(p.status, &c.abort_flag, kInfoAccFull);
        break;
      }
      tc_fence_after();
      for (int n = first; n < last; n += 32) {
        if (n + 32 < last) load_residual(p, t, n + 32, last, next);
        finish32<kBf16, kAct>(p, tmem + buf * kManyWide + (n - n0) + lanes, t, n, last, res);
#pragma unroll
        for (int h = 0; h < 4; ++h) res[h] = next[h];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote(map_rank(&c.acc_empty[buf], 0));
    }
    __threadfence();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA's copies, MMAs or barriers are in use
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Outputs of a tile: the width that makes the waves of tiles cheapest, a wave
// costing its width and about 24 outputs' worth of fixed time.  us at the width
// taken and at others: 256 x 4096 -> 6144: 96 16.4; 128 17.6, 192 20.8, 256 25.7.
// 1001 x 2056 -> 5000: 144 31.1; 96 35.4, 192 35.7, 256 38.3.  4096 x 4096 ->
// 12288: 256 227 to 236; 192 240, 144 260, 96 312.
int tile_width(int M, int N, int pairs) {
  int best = kManyWide;
  long long cost = -1;
  for (int w = kManyWide; w >= 64; w -= 16) {
    const long long tiles = static_cast<long long>(ceil_div(M, kManyRows)) * ceil_div(N, w);
    const long long c = (tiles + pairs - 1) / pairs * (w + 24);
    if (cost < 0 || c < cost) { cost = c; best = w; }
  }
  return best;
}

template <bool kBf16, int kAct>
cudaError_t launch_many_act(const CUtensorMap& tm_w, const CUtensorMap& tm_x, const LinearParams& p, int grid,
                            cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(linear_many_kernel<kBf16, kAct>, kManySmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kManyThreads);
  cfg.dynamicSmemBytes = kManySmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_many_kernel<kBf16, kAct>, tm_w, tm_x, p);
}
template <bool kBf16>
cudaError_t launch_many(const CUtensorMap& tm_w, const CUtensorMap& tm_x, const LinearParams& p, int grid,
                        cudaStream_t s) {
  switch (p.act) {
    case MOE_ACT_SILU: return launch_many_act<kBf16, MOE_ACT_SILU>(tm_w, tm_x, p, grid, s);
    case MOE_ACT_GELU: return launch_many_act<kBf16, MOE_ACT_GELU>(tm_w, tm_x, p, grid, s);
    case MOE_ACT_GELU_TANH: return launch_many_act<kBf16, MOE_ACT_GELU_TANH>(tm_w, tm_x, p, grid, s);
    case MOE_ACT_RELU: return launch_many_act<kBf16, MOE_ACT_RELU>(tm_w, tm_x, p, grid, s);
    default: return launch_many_act<kBf16, MOE_ACT_NONE>(tm_w, tm_x, p, grid, s);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// How many clusters of c CTAs fit on the current device at once (0 on
// failure), asked once a device and size: of an empty kernel of the same shape,
// since the query takes a kernel that allocates tensor memory to fill its SM,
// whatever it allocates (two CTAs of linear_few_kernel do share one).
__global__ void __launch_bounds__(kLinThreads, 1) shape_kernel() {}

int resident_clusters(int c) {
  static std::atomic<int> known[kMaxCluster + 1][64];
  int d = 0;
  if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= 64) return 0;
  int n = known[c][d].load(std::memory_order_relaxed);
  if (n > 0) return n;
  static std::atomic<uint64_t> done{0};
  if (allow_smem(shape_kernel, kLinSmem, done) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(c * 1024);  // more than fit
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = kLinSmem;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = c;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, shape_kernel, &cfg) != cudaSuccess) return 0;
  known[c][d].store(n, std::memory_order_relaxed);
  return n;
}

// CTAs that share a weight tile: as many as leave each at least 4 of the
// 64-input k-blocks, make at most 1.5 CTAs an SM and are resident at once.  (72
// x 4096 -> 6144, 48 tiles: 24.6, 16.5, 14.6, 13.4, 14.2, 19.7 us with 1 .. 6, of
// which 6 no longer fit; 9 x 4096 -> 4096, 32 tiles: 16.9, 11.3, 9.9, 9.1, 9.5,
// 9.2, and 9.1 with the 7 that it takes.)
int cluster_size(int tiles, int k_blocks, int sms) {
  int c = 1;
  while (c < kMaxCluster && 2 * (c + 1) * tiles <= 3 * sms && k_blocks / (c + 1) >= 4 &&
         resident_clusters(c + 1) >= tiles)
    ++c;
  return c;
}

// Which kernel: the few rows' one streams every weight once but multiplies 128
// weights with all rows in each CTA, so it pays while the rows are few or a
// weight tile has a cluster to share the reading.  us, few / many, K = 4096:
//   N = 24576 (no cluster)    48 rows 38.2 / 38.6    64 40.3 / 39.0   128 50.7 / 41.1
//   N = 12288 (cluster of 2)  64 rows 21.9 / 23.0    80 22.6 / 23.1    96 25.0 / 23.5
//   N =  6144 (4)             96 rows 15.3 / 15.5   112 15.9 / 15.7   128 16.6 / 16.1
//   N =  4096 (7)             72 rows 11.8 / 13.7   112 13.7 / 14.0   128 14.6 / 14.0
bool few_rows(int M, int cluster) { return M <= kFewTokens && M <= 32 + 16 * cluster; }

template <bool kBf16>
cudaError_t launch_few(const CUtensorMap& tm_w, const CUtensorMap& tm_x, const LinearParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(linear_few_kernel<kBf16>, kLinSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(ceil_div(p.N, kHalfRows) * p.cluster);
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = kLinSmem;
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
  return cudaLaunchKernelEx(&cfg, linear_few_kernel<kBf16>, tm_w, tm_x, p);
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_linear_workspace_bytes(int M, int N, int K) {
  if (M < 0 || N < 1 || K < 1) return 0;
  if (N % 8 || K % 8 || M > MOE_MAX_LINEAR || N > MOE_MAX_LINEAR || K > MOE_MAX_LINEAR) return 0;
  return MOE_STATUS_BYTES;
}

moe_status moe_linear(const void* x, long long x_stride, int M, int K, const void* w, int N, int dtype,
                      const void* bias, int activation, const void* residual, long long residual_stride, void* y,
                      long long y_stride, void* ws, size_t ws_bytes, cudaStream_t stream) {
  using namespace moe;
  if (M < 0 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (activation < MOE_ACT_NONE || activation > MOE_ACT_RELU) return MOE_ERR_INVALID_ARG;
  if (N % 8 || K % 8 || M > MOE_MAX_LINEAR || N > MOE_MAX_LINEAR || K > MOE_MAX_LINEAR) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!x || !w || !y || x == y || w == y) return MOE_ERR_INVALID_ARG;
  if (y_stride < N || (M > 1 && x_stride < K) || (residual && residual_stride < 0)) return MOE_ERR_INVALID_ARG;
  if (residual == y && residual_stride != y_stride) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(bias) || !aligned16(residual) || !aligned16(y))
    return MOE_ERR_INVALID_ARG;
  if (x_stride % 8 || y_stride % 8 || (residual && residual_stride % 8)) return MOE_ERR_UNSUPPORTED;
  const RowSet out = {y, M, 2ll * N, 2 * y_stride};
  if (rows_meet(out, {x, M, 2ll * K, 2 * x_stride}) || rows_meet(out, {w, 1, 2ll * N * K, 0}) ||
      rows_meet(out, {bias, 1, 2ll * N, 0}) ||
      (residual != y && rows_meet(out, {residual, M, 2ll * N, 2 * residual_stride})))
    return MOE_ERR_INVALID_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kWsAlign) != 0 || ws_bytes < MOE_STATUS_BYTES)
    return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  LinearParams p;
  memset(&p, 0, sizeof(p));
  p.M = M; p.N = N; p.K = K;
  p.k_blocks = ceil_div(K, kBlockK);
  if (M <= kFewTokens) p.cluster = cluster_size(ceil_div(N, kHalfRows), p.k_blocks, sms);
  const bool few = few_rows(M, p.cluster);
  if (few) {
    p.n_tok = ceil_div(M, 16) * 16;
    p.stages = (kLinSmem - 1024) / (kTileBytesA + p.n_tok * 128);
    if (p.stages > kLinMaxStages) p.stages = kLinMaxStages;
    p.tmem_cols = 32;
    while (p.tmem_cols < static_cast<uint32_t>(p.n_tok)) p.tmem_cols <<= 1;
  } else {
    p.n_tok = tile_width(M, N, sms / 2);
    p.stages = (kManySmem - 1024) / ((kTileBytesA + p.n_tok / 2 * 128 + 1023) / 1024 * 1024);
    if (p.stages > kManyStages) p.stages = kManyStages;
  }
  p.bias = static_cast<const uint16_t*>(bias);
  p.residual = static_cast<const uint16_t*>(residual); p.res_stride = residual_stride;
  p.y = static_cast<uint16_t*>(y); p.y_stride = y_stride;
  p.act = activation;
  p.status = static_cast<int32_t*>(ws);
  const bool f16 = dtype == MOE_DTYPE_F16;
  CUtensorMap tm_w, tm_x;
  const uint64_t wd[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N)}, wst[1] = {static_cast<uint64_t>(K) * 2};
  const uint64_t xd[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(M)};
  const uint64_t xst[1] = {static_cast<uint64_t>(M > 1 ? x_stride : K) * 2};
  const uint32_t wb[2] = {kBlockK, static_cast<uint32_t>(few ? kHalfRows : p.n_tok / 2)};
  const uint32_t xb[2] = {kBlockK, static_cast<uint32_t>(few ? p.n_tok : kManyRows / 2)};
  if (!encode_map_16(&tm_w, f16, w, 2, wd, wst, wb) || !encode_map_16(&tm_x, f16, x, 2, xd, xst, xb))
    return MOE_ERR_CUDA;
  cudaError_t e;
  if (few) {
    e = f16 ? launch_few<false>(tm_w, tm_x, p, stream) : launch_few<true>(tm_w, tm_x, p, stream);
  } else {
    const long long tiles = static_cast<long long>(ceil_div(M, kManyRows)) * ceil_div(N, p.n_tok);
    const int grid = 2 * static_cast<int>(tiles < sms / 2 ? tiles : sms / 2);
    e = f16 ? launch_many<false>(tm_w, tm_x, p, grid, stream) : launch_many<true>(tm_w, tm_x, p, grid, stream);
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
