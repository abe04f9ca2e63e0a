// What the two kernels of moe_linear_q4 share: the weights' layout and the expansion.
//
// Layout (moe_q4_prepare, once a set of weights): for every 128 rows and 128 inputs one run
// of bytes, [4][128 rows][16 bytes] of codes (32 inputs of a row in 16 bytes, inputs 2 j and
// 2 j + 1 of every 8 in nibbles j and j + 4, where one mask finds both), then the groups'
// scales [128 / g][128 rows] and zeros.  A block is one copy, and a warp's lanes read 512
// bytes side by side.
#pragma once
#include "epilogue.cuh"

namespace moe {

constexpr int kBlock = 128;  // inputs of a block
constexpr int kRows = 128;   // weight rows of a block
constexpr int kCodeBytes = kRows * kBlock / 2;

__host__ __device__ constexpr int block_bytes(int group, bool zeros) {
  return kCodeBytes + kBlock / group * kRows * (zeros ? 3 : 2);
}

struct Q4Params {
  int M, N, K, k_blocks;
  int group, group_log2;     // inputs of a group: 32, 64 or 128
  int zeros;                 // 1: the groups have zero points (else 8)
  int block_bytes;           // of a weight block
  int n_tok, row_tiles, tok_tiles;
  int stages, cluster;
  int slots;                     // tokens of a tile that a CTA of the cluster finishes, at most
  int blocks_each, blocks_more;  // of a tile's K a CTA of the cluster takes; those that take one more
  const uint8_t* w;
  const uint16_t *bias, *residual;
  uint16_t* y;
  long long res_stride, y_stride;
  int act;
  int32_t* status;
};

// For few rows (linear_q4_few.cu): a kernel on the warps' own matrix instructions.  Where the
// two cross (us, this kernel and the other): 1 row of 4096 x 4096 5.4 and 9.8, 24 rows 7.7
// and 9.8; of 4096 x 24576 17.5 and 37, 31.5 and 37; 32 rows 9.7 and 10, 48 and 37.
constexpr int kQ4FewRows = 24;
cudaError_t launch_linear_q4_few(bool f16, const Q4Params& p, const void* x, long long x_stride, cudaStream_t s);

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

}  // namespace moe
