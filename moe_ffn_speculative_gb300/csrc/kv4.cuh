// The 4-bit cache of keys and values (kv4): geometry of a block and expansion of
// its codes.
//
// A cache is [pages][key heads][block]; the block of a page of P slots and a
// head of D channels holds, for every group of 32 channels, P runs of 16 bytes
// (the group's codes of one slot, even channel in the low nibble): the keys'
// groups, then the values'; then P x D/32 scales of the keys and as many of the
// values.  So a warp whose lanes are slots reads and writes 512 contiguous bytes
// at a time, without a bank conflict in shared memory, and a slot's scales are
// one word; and the block of a page is one copy.
#pragma once
#include "moe_internal.cuh"

namespace moe {

constexpr int kKv4Low = 104, kKv4High = 140;  // scales that moe_kv4_write writes (the FP4 experts' range)
constexpr int kKv4Nan = 255;                  // scale of a group that holds an infinity or NaN

__host__ __device__ constexpr int kv4_slot_bytes(int D) { return D + D / 16; }
__host__ __device__ constexpr int kv4_codes_at(int D, int page, int which) { return which * page * (D / 2); }
__host__ __device__ constexpr int kv4_scales_at(int D, int page, int which) {
  return page * D + which * page * (D / 32);
}

#ifdef __CUDACC__
// The scale byte's power of two in f16, in both halves.  2^-24 .. 2^15 are exact;
// smaller ones are 0, larger ones infinite and 255 NaN (no write makes them but the
// last).
__device__ __forceinline__ uint32_t kv4_scale_h2(uint32_t s) {
  const int e = static_cast<int>(s) - 127;
  uint32_t b = e >= -14 ? static_cast<uint32_t>(e + 15) << 10 : (e >= -24 ? 1u << (e + 24) : 0u);
  if (e > 15) b = s == kKv4Nan ? 0x7e00u : 0x7c00u;
  return b | (b << 16);
}
// The scale byte's power of two in fp32 (exact for all of them; 255: NaN).
__device__ __forceinline__ float kv4_scale_f(uint32_t s) {
  return __uint_as_float(s == kKv4Nan ? 0x7fc00000u : (s == 0 ? 0x00400000u : s << 23));
}
// Eight codes (byte j: channels 2j in the low nibble, 2j + 1 in the high one) in f16.
__device__ __forceinline__ void kv4_expand(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t"
      "}"
      : "=&r"(o[0]), "=&r"(o[1]), "=&r"(o[2]), "=&r"(o[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t kv4_mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
#endif

}  // namespace moe
