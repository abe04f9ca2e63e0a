// Query/key norms, position rotation and cache write of one attention layer
// in one launch (moe_qk_norm_rope).
//
// Per head row x of D elements: y = x * rsqrt(mean(x^2) + eps) * w, then the
// first R elements are rotated in pairs (a, b) -> (a c - b s, b c + a s) by
// the cosines and sines of the token's position.  Everything is held in fp32
// between the one load and the one rounding to the output type.  Query rows
// go to q_out, key rows and the untouched value rows to the token's slot of
// the paged cache.
//
// The pass reads and writes every row once, so it is bound by memory
// bandwidth for many tokens and by the latency of its two dependent loads
// (position, then table row) for few.  A head row is held by D / 8 lanes, 16
// bytes each, so the norm's sum is a shuffle over those lanes; the pair
// (i, i + R/2) is another shuffle, the pair (2i, 2i + 1) lies in one lane.  A
// block takes one token: each lane group walks the token's heads, kHeads rows
// in flight at a time, and keeps its eight cosines and sines in registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <string.h>

#include "moe.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kHeads = 4;  // head rows a lane group loads before it uses the first

struct RopeParams {
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride, q_out_stride;
  int T, Hq, Hkv;
  const uint16_t *q_weight, *k_weight;
  float eps;
  const float* rope;
  int rot, max_pos, interleaved;
  const int32_t* positions;
  uint16_t *q_out, *k_cache, *v_cache;
  const int32_t* slots;
  long long n_slots;
  int32_t* status;
};

template <bool kBf16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if (kBf16) {
    __nv_bfloat162 h;
    memcpy(&h, &u, 4);
    return __bfloat1622float2(h);
  }
  __half2 h;
  memcpy(&h, &u, 4);
  return __half22float2(h);
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
template <bool kBf16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2<kBf16>(w[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = D / 8;  // lanes of a head row
  constexpr int kGroups = kRopeThreads / kLanes;
  const int t = blockIdx.x;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int heads = p.Hq + 2 * p.Hkv;

  long long slot = t;
  if (p.slots) slot = __ldg(p.slots + t);
  int pos = 0;
  if (p.rot > 0) pos = __ldg(p.positions + t);
  bool skip = false, cached = slot >= 0;
  if (pos < 0 || (p.rot > 0 && pos >= p.max_pos)) {
    skip = true;
    if (threadIdx.x == 0) record_index(p.status, kInfoPosition);
  }
  if (slot >= p.n_slots) {
    cached = false;
    if (threadIdx.x == 0 && p.Hkv > 0) record_index(p.status, kInfoSlot);
  }
  if (skip) return;

  // this lane's cosines and (signed) sines; 1 and 0 beyond the rotated part
  const int half = p.rot / 2;
  const int e0 = lane * 8;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) { c[i] = 1.f; s[i] = 0.f; }
  int partner = threadIdx.x & 31;
  if (e0 < p.rot) {
    const float* row = p.rope + static_cast<long long>(pos) * p.rot;
    if (p.interleaved) {
      const float4 cv = __ldg(reinterpret_cast<const float4*>(row + e0 / 2));
      const float4 sv = __ldg(reinterpret_cast<const float4*>(row + half + e0 / 2));
      const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[2 * i] = c[2 * i + 1] = cc[i];
        s[2 * i] = -ss[i];
        s[2 * i + 1] = ss[i];
      }
    } else {
      const bool upper = e0 >= half;
      const int i0 = upper ? e0 - half : e0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 cv = __ldg(reinterpret_cast<const float4*>(row + i0 + 4 * j));
        const float4 sv = __ldg(reinterpret_cast<const float4*>(row + half + i0 + 4 * j));
        const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          c[4 * j + i] = cc[i];
          s[4 * j + i] = upper ? ss[i] : -ss[i];
        }
      }
      partner += upper ? -(half / 8) : half / 8;
    }
  }

  for (int base = 0; base < heads; base += kGroups * kHeads) {  // the same count in every lane
    const int h0 = base + group;
    uint4 raw[kHeads];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j * kGroups;
      raw[j] = make_uint4(0, 0, 0, 0);
      const uint16_t* src = nullptr;
      if (h < p.Hq) src = p.q + t * p.q_stride + h * D;
      else if (h < p.Hq + p.Hkv) src = p.k + t * p.k_stride + (h - p.Hq) * D;
      else if (h < heads && p.v) src = p.v + t * p.v_stride + (h - p.Hq - p.Hkv) * D;
      if (src) raw[j] = *reinterpret_cast<const uint4*>(src + e0);
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j * kGroups;
      // every lane of the warp takes part in the shuffles, whatever its head
      const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
      float x[8];
      unpack8<kBf16>(raw[j], x);
      const uint16_t* weight = is_q ? p.q_weight : p.k_weight;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (weight) {
        float w[8];
        unpack8<kBf16>(__ldg(reinterpret_cast<const uint4*>(weight + e0)), w);
        const float r = rsqrtf(sum * (1.f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
      }
      float y[8];
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i] * c[i] + x[i ^ 1] * s[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i] * c[i] + __shfl_sync(0xffffffffu, x[i], partner) * s[i];
      }
      uint4 out;
      out.x = pack2<kBf16>(y[0], y[1]);
      out.y = pack2<kBf16>(y[2], y[3]);
      out.z = pack2<kBf16>(y[4], y[5]);
      out.w = pack2<kBf16>(y[6], y[7]);
      if (is_q) {
        *reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride + h * D + e0) = out;
      } else if (h < heads && cached) {
        if (!is_v)
          *reinterpret_cast<uint4*>(p.k_cache + (slot * p.Hkv + (h - p.Hq)) * D + e0) = out;
        else if (p.v)
          *reinterpret_cast<uint4*>(p.v_cache + (slot * p.Hkv + (h - p.Hq - p.Hkv)) * D + e0) = raw[j];
      }
    }
  }
}

template <bool kBf16>
cudaError_t launch(const RopeParams& p, int D, cudaStream_t s) {
  switch (D) {
    case 64: qk_norm_rope_kernel<kBf16, 64><<<p.T, kRopeThreads, 0, s>>>(p); break;
    case 128: qk_norm_rope_kernel<kBf16, 128><<<p.T, kRopeThreads, 0, s>>>(p); break;
    default: qk_norm_rope_kernel<kBf16, 256><<<p.T, kRopeThreads, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace moe

extern "C" moe_status moe_qk_norm_rope(const void* q, long long q_stride, const void* k, long long k_stride,
                                       const void* v, long long v_stride, int T, int Hq, int Hkv, int D, int dtype,
                                       const void* q_weight, const void* k_weight, float eps, const float* rope,
                                       int rot_dim, int max_pos, int interleaved, const int32_t* positions,
                                       void* q_out, long long q_out_stride, void* k_cache, void* v_cache,
                                       const int32_t* slots, long long n_slots, void* ws, size_t ws_bytes,
                                       cudaStream_t stream) {
  using namespace moe;
  if (T < 0 || Hq < 0 || Hkv < 0 || D < 1 || rot_dim < 0 || rot_dim > D || max_pos < 0 || n_slots < 0)
    return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return MOE_ERR_INVALID_ARG;
  if (!(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if ((D != 64 && D != 128 && D != 256) || rot_dim % 16 != 0 || T > MOE_MAX_ATTN_TOKENS || Hq > 1024 || Hkv > 1024)
    return MOE_ERR_UNSUPPORTED;
  if (T == 0 || (Hq == 0 && Hkv == 0)) return MOE_OK;
  if (Hq > 0 && (!q || !q_out || q_stride < 0 || q_out_stride < static_cast<long long>(Hq) * D))
    return MOE_ERR_INVALID_ARG;
  if (Hkv > 0 && (!k || !k_cache || k_stride < 0)) return MOE_ERR_INVALID_ARG;
  if (Hkv > 0 && (!v != !v_cache || (v && v_stride < 0))) return MOE_ERR_INVALID_ARG;
  if (Hkv > 0 && !slots && n_slots < T) return MOE_ERR_INVALID_ARG;
  if (rot_dim > 0 && (!rope || !positions)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_weight) || !aligned16(k_weight) ||
      !aligned16(rope) || !aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache))
    return MOE_ERR_INVALID_ARG;
  if (q_stride % 8 || k_stride % 8 || v_stride % 8 || q_out_stride % 8) return MOE_ERR_UNSUPPORTED;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kWsAlign) != 0 || ws_bytes < MOE_STATUS_BYTES)
    return MOE_ERR_WORKSPACE;
  RopeParams p;
  memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(q); p.k = static_cast<const uint16_t*>(k); p.v = static_cast<const uint16_t*>(v);
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride; p.q_out_stride = q_out_stride;
  p.T = T; p.Hq = Hq; p.Hkv = Hkv;
  p.q_weight = static_cast<const uint16_t*>(q_weight); p.k_weight = static_cast<const uint16_t*>(k_weight);
  p.eps = eps;
  p.rope = rope; p.rot = rot_dim; p.max_pos = max_pos; p.interleaved = interleaved; p.positions = positions;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_cache = static_cast<uint16_t*>(k_cache); p.v_cache = static_cast<uint16_t*>(v_cache);
  p.slots = slots; p.n_slots = n_slots;
  p.status = static_cast<int32_t*>(ws);
  const cudaError_t e = dtype == MOE_DTYPE_BF16 ? launch<true>(p, D, stream) : launch<false>(p, D, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
