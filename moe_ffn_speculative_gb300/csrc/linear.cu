// Matrix product with bias, activation and residual in its epilogue
// (moe_linear): y = act(x W^T + bias) + residual, W [N, K].
//
// Few rows: bound by the bytes of W, which are read once.  The 128 rows of a
// weight tile are the MMA's M dimension and up to 256 tokens its N dimension;
// a cluster of CTAs shares a weight tile, each taking a range of K, so that a
// layer with few tiles still occupies the SMs.  The CTAs' fp32 sums meet in
// distributed shared memory: every CTA adds its share of the tokens over the
// cluster in rank order (the result does not depend on timing) and applies
// the epilogue.
//
// A CTA: warp 0 loads weight and token tiles by TMA into a ring of stages,
// warp 1 issues the MMAs, warps 2..5 drain tensor memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include "moe.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kLinThreads = 192;
constexpr int kLinSmem = 232448 - 1024;  // 227 KB less the control words
constexpr int kLinMaxStages = 12;
constexpr int kLinMaxTokens = 256;       // tokens of a tile
constexpr int kMaxCluster = 8;

struct LinearParams {
  int M, N, K, k_blocks;
  int n_tok;                 // tokens of a tile: a multiple of 16
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

// v sigmoid(v) and the like through one exponential; erfc keeps gelu's
// negative tail from cancelling.
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case MOE_ACT_SILU: return v / (1.f + __expf(-v));
    case MOE_ACT_GELU: return 0.5f * v * erfcf(-v * 0.70710678118654752f);
    case MOE_ACT_GELU_TANH:
      return v / (1.f + __expf(-1.5957691216057308f * (v + 0.044715f * v * v * v)));
    case MOE_ACT_RELU: return fmaxf(v, 0.f);
    default: return v;
  }
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
  const int t0 = blockIdx.y * p.n_tok;
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
  griddep_wait();  // what the previous kernel on the stream wrote is visible
  griddep_launch_dependents();

  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = l2_evict_first_policy();
      Ring r;
      int filled = 0;
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        ok = mbar_wait(&c.empty[r.stage], r.phase ^ 1u, &c.abort_flag);
        if (!ok) break;
        uint8_t* a = ring_mem + r.stage * stage_bytes;
        mbar_arrive_expect_tx(&c.full[r.stage], stage_bytes);
        tma_load_2d_hint(a, &tm_w, &c.full[r.stage], kb * kBlockK, n0, pol);
        tma_load_2d(a + kTileBytesA, &tm_x, &c.full[r.stage], kb * kBlockK, t0);
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
    if (lane == 0) {
      const uint32_t id = kBf16 ? idesc_bf16(kHalfRows, p.n_tok) : idesc_f16(kHalfRows, p.n_tok);
      Ring r;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = mbar_wait(&c.full[r.stage], r.phase, &c.abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = smem_u32(ring_mem + r.stage * stage_bytes), b = a + kTileBytesA;
#pragma unroll
        for (int ks = 0; ks < kBlockK / 16; ++ks)
          mma_bf16(tmem, sw128_desc(a + ks * 32), sw128_desc(b + ks * 32), id, (kb > kb0 || ks > 0) ? 1u : 0u);
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
  const int toks = min(p.n_tok, p.M - t0);
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
            if (p.residual) v += to_f<kBf16>(p.residual[(t0 + t + i) * p.res_stride + n]);
            p.y[(t0 + t + i) * p.y_stride + n] = from_f<kBf16>(v);
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
          if (p.residual) z += to_f<kBf16>(p.residual[(t0 + t) * p.res_stride + n + i]);
          o[i] = from_f<kBf16>(z);
        }
        *reinterpret_cast<ushort4*>(p.y + (t0 + t) * p.y_stride + n) = out;
      }
    }
    cluster_sync();  // the others have read this CTA's sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// CTAs that share a weight tile: as many as keep the grid within the SMs and
// leave each at least 4 of the 64-input k-blocks.
int cluster_size(int tiles, int k_blocks, int sms) {
  int c = 1;
  while (c < kMaxCluster && (c + 1) * tiles <= sms && k_blocks / (c + 1) >= 4) ++c;
  return c;
}

template <bool kBf16>
cudaError_t launch_few(const CUtensorMap& tm_w, const CUtensorMap& tm_x, const LinearParams& p, cudaStream_t s) {
  cudaError_t e =
      cudaFuncSetAttribute(linear_few_kernel<kBf16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(ceil_div(p.N, kHalfRows) * p.cluster, ceil_div(p.M, p.n_tok));
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
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kWsAlign) != 0 || ws_bytes < MOE_STATUS_BYTES)
    return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  LinearParams p;
  memset(&p, 0, sizeof(p));
  p.M = M; p.N = N; p.K = K;
  p.k_blocks = ceil_div(K, kBlockK);
  const int m_tiles = ceil_div(M, kLinMaxTokens);
  p.n_tok = ceil_div(ceil_div(M, m_tiles), 16) * 16;
  p.cluster = cluster_size(ceil_div(N, kHalfRows) * ceil_div(M, p.n_tok), p.k_blocks, sms);
  p.stages = (kLinSmem - 1024) / (kTileBytesA + p.n_tok * 128);
  if (p.stages > kLinMaxStages) p.stages = kLinMaxStages;
  p.tmem_cols = 32;
  while (p.tmem_cols < static_cast<uint32_t>(p.n_tok)) p.tmem_cols <<= 1;
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
  const uint32_t wb[2] = {kBlockK, kHalfRows}, xb[2] = {kBlockK, static_cast<uint32_t>(p.n_tok)};
  if (!encode_map_16(&tm_w, f16, w, 2, wd, wst, wb) || !encode_map_16(&tm_x, f16, x, 2, xd, xst, xb))
    return MOE_ERR_CUDA;
  const cudaError_t e = f16 ? launch_few<false>(tm_w, tm_x, p, stream) : launch_few<true>(tm_w, tm_x, p, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
