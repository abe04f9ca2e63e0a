// moe_linear_q4 for few rows: bound by the weights' bytes, which every warp takes from
// memory into the registers of its own matrix instructions.
//
// A fragment of mma.m16n8k16 wants pairs of neighbouring inputs, and any order of the
// inputs will do that both operands share.  So of the 16 bytes that hold 32 inputs of a
// row four lanes take a word each, 8 inputs, which one shift, mask and subtraction a pair
// turn into the weights' side of two products, and 16 bytes of a token's inputs in the
// same places are their other side: neither passes shared memory.  A group's fp32 sums
// are whole numbers times inputs; its scales multiply them as they are added up.
//
// A CTA takes 32 weight rows, its 16 or 8 warps a block of 128 inputs each in turn, 16 rows a
// fragment; the warps' sums meet in shared memory in the warps' order.  (Fewer rows a warp
// would read the tokens' inputs more often, more would leave SMs without work at 4096 rows.)
//
// Measured: 1 row of 4096 x 4096 5.4 us (floor 1.3: launch, two dependent trips to memory and
// the joining), 4096 x 24576 17.5 us (3.0 TB/s), 16 rows 24.7: the pipe that expands is busy a
// third of the time, memory less; a warp's loads do not run under its own arithmetic.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <string.h>

#include "linear_q4.cuh"
#include "moe.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kWarpRows = 32;
constexpr int kPad = kWarpRows + 4;  // floats a token of a warp's sums (no bank twice)

template <bool kBf16>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if (kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t load_once(const void* p) {
  uint32_t v;
  asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// kTiles: 8 tokens each.
template <bool kBf16, int kTiles, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, (kTiles == 1 ? 32 : 16) / kWarps)
    linear_q4_few_kernel(const __grid_constant__ Q4Params p, const uint16_t* x, long long x_stride) {
  extern __shared__ float sums[];  // [warps][tokens][kPad]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kWarpRows, r0 = n0 % kRows;
  const uint8_t* tile = p.w + static_cast<long long>(n0 / kRows) * p.k_blocks * p.block_bytes;
  // this warp's codes come into L2 while the previous kernel ends (it may write weights)
  for (int kb = warp; kb < p.k_blocks; kb += kWarps)
    if (lane < 16)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(tile + static_cast<long long>(kb) * p.block_bytes +
                                                    (lane >> 2) * (kRows * 16) + r0 * 16 + (lane & 3) * 128));
  griddep_wait();

  float acc[2][kTiles][4] = {};
  const int log2 = p.group_log2, last = (1 << (log2 - 5)) - 1;  // 32 inputs of a group, less one
  for (int kb = warp; kb < p.k_blocks; kb += kWarps) {
    const uint8_t* block = tile + static_cast<long long>(kb) * p.block_bytes;
    const uint8_t* scales = block + kCodeBytes + (r0 + g) * 2;
    const uint8_t* zeros = block + kCodeBytes + (kBlock >> log2) * kRows * 2 + r0 + g;
    uint32_t w[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) w[q][i] = load_once(block + (q * kRows + r0 + g + 8 * i) * 16 + t * 4);
    float sum[2][kTiles][4];
    float s[4];
    uint32_t z[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = kb * kBlock + q * 32;
      if ((q & last) == 0) {
        const int at = (q * 32 >> log2) * kRows;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[i] = to_f<kBf16>(*reinterpret_cast<const uint16_t*>(scales + (at + 8 * i) * 2));
          z[i] = p.zeros ? zeros[at + 8 * i] : 8u;
        }
#pragma unroll
        for (int i = 0; i < 2 * kTiles * 4; ++i) (&sum[0][0][0])[i] = 0.f;
      }
      uint4 b[kTiles];
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        b[j] = make_uint4(0, 0, 0, 0);
        if (g + 8 * j < p.M && k < p.K)
          b[j] = __ldg(reinterpret_cast<const uint4*>(x + (g + 8 * j) * x_stride + k + t * 8));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // 16 rows
        uint32_t a[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          expand8<kBf16>(w[q][2 * h + i], magic2<kBf16>(z[2 * h + i]), 0xd400d400u + z[2 * h + i] * 0x00100010u, a[i]);
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          mma16<kBf16>(sum[h][j], a[0][0], a[1][0], a[0][1], a[1][1], b[j].x, b[j].y);
          mma16<kBf16>(sum[h][j], a[0][2], a[1][2], a[0][3], a[1][3], b[j].z, b[j].w);
        }
      }
      if ((q & last) == last)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[h][j][i] = fmaf(sum[h][j][i], s[2 * h + (i >> 1)], acc[h][j][i]);
    }
  }
  // (what the epilogue reads is on its way while the warps meet)
  constexpr int kEach = (kTiles * 8 + kWarps - 1) / kWarps;
  const int n = n0 + lane;
  uint16_t bias = 0, res[kEach] = {};
  if (n < p.N) {
    if (p.bias) bias = p.bias[n];
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (p.residual && warp + i * kWarps < p.M) res[i] = p.residual[(warp + i * kWarps) * p.res_stride + n];
  }
  // token 8 j + 2 t + (i & 1), row 16 h + g + 8 (i >> 1)
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sums[((warp * kTiles + j) * 8 + 2 * t + (i & 1)) * kPad + 16 * h + g + 8 * (i >> 1)] = acc[h][j][i];
  __syncthreads();
  if (n < p.N)
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int m = warp + e * kWarps;
      if (m >= p.M) break;
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) v += sums[(i * kTiles * 8 + m) * kPad + lane];
      if (p.bias) v += to_f<kBf16>(bias);
      v = activate(v, p.act);
      if (p.residual) v += to_f<kBf16>(res[e]);
      p.y[m * p.y_stride + n] = from_f<kBf16>(v);
    }
  __threadfence();  // (y may be what a fused forward loads before it waits: see linear.cu)
}

template <bool kBf16, int kTiles, int kWarps>
cudaError_t launch_few(const Q4Params& p, const uint16_t* x, long long x_stride, cudaStream_t s) {
  constexpr int kBytes = kWarps * kTiles * 8 * kPad * 4;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(linear_q4_few_kernel<kBf16, kTiles, kWarps>, kBytes, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.dynamicSmemBytes = kBytes;
  cfg.gridDim = dim3(ceil_div(p.N, kWarpRows));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_q4_few_kernel<kBf16, kTiles, kWarps>, p, x, x_stride);
}

// With 16 warps a CTA the weights of one are read soonest, with 8 more of them are at work at
// once.  (1 row of 4096 x 4096: 5.4 and 6.2 us, x 12288: 11.3 and 10.3, x 24576: 19.3 and 17.5;
// 16 rows: x 6144 10.8 and 9.3, x 24576 30.3 and 24.7; 12288 x 4096: 10.8 and 12.9.)
template <int kWarps>
cudaError_t launch_few(bool f16, const Q4Params& p, const uint16_t* x, long long x_stride, cudaStream_t s) {
  switch (ceil_div(p.M, 8)) {
    case 1: return f16 ? launch_few<false, 1, kWarps>(p, x, x_stride, s) : launch_few<true, 1, kWarps>(p, x, x_stride, s);
    case 2: return f16 ? launch_few<false, 2, kWarps>(p, x, x_stride, s) : launch_few<true, 2, kWarps>(p, x, x_stride, s);
    default: return f16 ? launch_few<false, 3, kWarps>(p, x, x_stride, s) : launch_few<true, 3, kWarps>(p, x, x_stride, s);
  }
}

}  // namespace

cudaError_t launch_linear_q4_few(bool f16, const Q4Params& p, const void* x, long long x_stride, cudaStream_t s) {
  const uint16_t* xs = static_cast<const uint16_t*>(x);
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorUnknown;
  return ceil_div(p.N, kWarpRows) > sms ? launch_few<8>(f16, p, xs, x_stride, s) : launch_few<16>(f16, p, xs, x_stride, s);
}

}  // namespace moe
