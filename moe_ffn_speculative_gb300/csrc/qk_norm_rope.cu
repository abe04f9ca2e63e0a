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
// (position, then table row) for few.  D / 8 lanes hold a head row, each four
// of its pairs: two runs of four elements R/2 apart (or of neighbours, or, past
// the rotated part, any two runs).  So a rotation needs no other lane, a lane
// four cosines and four sines, and the norm's sum one shuffle over those lanes.
// The norm's weights are multiplied into the cosines and sines once a token, for
// queries and keys: the row costs 24 multiplications a lane, its factor r last.
// A block takes one token.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <string.h>

#include "moe.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kRopeThreads = 256;  // most threads of a block
constexpr int kHeads = 4;          // query rows a lane group loads before it uses the first

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
// A lane's part of a head row: two runs of four elements.
struct Part {
  uint2 a, b;
};
__device__ __forceinline__ Part load_part(const uint16_t* row, int ea, int eb) {
  return Part{*reinterpret_cast<const uint2*>(row + ea), *reinterpret_cast<const uint2*>(row + eb)};
}
__device__ __forceinline__ void store_part(uint16_t* row, int ea, int eb, const Part& x) {
  *reinterpret_cast<uint2*>(row + ea) = x.a;
  *reinterpret_cast<uint2*>(row + eb) = x.b;
}
// Its four pairs: element k of both runs, or (kInter) neighbours.
template <bool kBf16, bool kInter>
__device__ __forceinline__ void to_pairs(const Part& x, float (&a)[4], float (&b)[4]) {
  const float2 v[4] = {unpack2<kBf16>(x.a.x), unpack2<kBf16>(x.a.y), unpack2<kBf16>(x.b.x), unpack2<kBf16>(x.b.y)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kInter) {
      a[i] = v[i].x;
      b[i] = v[i].y;
    } else {
      (i < 2 ? a : b)[2 * (i % 2)] = v[i].x;
      (i < 2 ? a : b)[2 * (i % 2) + 1] = v[i].y;
    }
  }
}
template <bool kBf16, bool kInter>
__device__ __forceinline__ Part from_pairs(const float (&a)[4], const float (&b)[4]) {
  Part x;
  if (kInter) {
    x.a = make_uint2(pack2<kBf16>(a[0], b[0]), pack2<kBf16>(a[1], b[1]));
    x.b = make_uint2(pack2<kBf16>(a[2], b[2]), pack2<kBf16>(a[3], b[3]));
  } else {
    x.a = make_uint2(pack2<kBf16>(a[0], a[1]), pack2<kBf16>(a[2], a[3]));
    x.b = make_uint2(pack2<kBf16>(b[0], b[1]), pack2<kBf16>(b[2], b[3]));
  }
  return x;
}

// The rotation of a lane's pairs with the norm's weights in it:
// (a, b) -> r (a ca - b sb, b cb + a sa); past the rotated part r (a ca, b cb),
// without a product of the one with the other (0 times an infinity is NaN).
template <bool kBf16, bool kInter, int D>
struct Turn {
  float ca[4], sb[4], cb[4], sa[4];
  bool norm, rotated;
  __device__ __forceinline__ Turn(const float (&c)[4], const float (&s)[4], bool rotated, const uint16_t* weight, int ea,
                                  int eb)
      : norm(weight != nullptr), rotated(rotated) {
    float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
    if (norm) to_pairs<kBf16, kInter>(load_part(weight, ea, eb), wa, wb);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ca[i] = wa[i] * c[i];
      sb[i] = wb[i] * s[i];
      cb[i] = wb[i] * c[i];
      sa[i] = wa[i] * s[i];
    }
  }
  // (Every lane of the warp takes part in the sum.)
  __device__ __forceinline__ Part operator()(const Part& x, float eps) const {
    float a[4], b[4], ya[4], yb[4], r = 1.f;
    to_pairs<kBf16, kInter>(x, a, b);
    if (norm) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += a[i] * a[i] + b[i] * b[i];
#pragma unroll
      for (int o = D / 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      r = rsqrtf(sum * (1.f / D) + eps);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ya[i] = (rotated ? a[i] * ca[i] - b[i] * sb[i] : a[i] * ca[i]) * r;
      yb[i] = (rotated ? b[i] * cb[i] + a[i] * sa[i] : b[i] * cb[i]) * r;
    }
    return from_pairs<kBf16, kInter>(ya, yb);
  }
};

template <bool kBf16, bool kInter, int D>
__global__ void __launch_bounds__(kRopeThreads, 4) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = D / 8;  // lanes of a head row
  const int groups = blockDim.x / kLanes, lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const long long t = blockIdx.x;
  long long slot = t;
  if (p.slots) slot = __ldg(p.slots + t);
  int pos = 0;
  if (p.rot > 0) pos = __ldg(p.positions + t);

  // this lane's runs: pairs of the rotated part first, then runs of the rest
  const int turning = p.rot / 8;  // lanes with rotated pairs
  int ea, eb;
  if (kInter || lane >= turning) {
    ea = kInter ? lane * 8 : p.rot + (lane - turning) * 8;
    eb = ea + 4;
  } else {
    ea = lane * 4;
    eb = p.rot / 2 + lane * 4;
  }
  // the first rows' loads are under way while the position is
  const uint16_t* q = p.q + t * p.q_stride;
  const uint16_t* k = p.k + t * p.k_stride;
  const uint16_t* v = p.v + t * p.v_stride;
  Part xq[kHeads], xk = {}, xv = {};
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    xq[j] = Part{};
    if (group + j * groups < p.Hq) xq[j] = load_part(q + (group + j * groups) * D, ea, eb);
  }
  if (group < p.Hkv) {
    xk = load_part(k + group * D, ea, eb);
    if (p.v) xv = load_part(v + group * D, ea, eb);
  }

  bool cached = slot >= 0;
  if (slot >= p.n_slots) {
    cached = false;
    if (threadIdx.x == 0 && p.Hkv > 0) record_index(p.status, kInfoSlot);
  }
  if (pos < 0 || (p.rot > 0 && pos >= p.max_pos)) {
    if (threadIdx.x == 0) record_index(p.status, kInfoPosition);
    return;
  }
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  if (lane < turning) {
    const float* row = p.rope + static_cast<long long>(pos) * p.rot + lane * 4;
    const float4 cv = __ldg(reinterpret_cast<const float4*>(row));
    const float4 sv = __ldg(reinterpret_cast<const float4*>(row + p.rot / 2));
    c[0] = cv.x; c[1] = cv.y; c[2] = cv.z; c[3] = cv.w;
    s[0] = sv.x; s[1] = sv.y; s[2] = sv.z; s[3] = sv.w;
  }
  {
    const Turn<kBf16, kInter, D> turn(c, s, lane < turning, p.q_weight, ea, eb);
    uint16_t* out = p.q_out + t * p.q_out_stride;
    for (int base = 0; base < p.Hq; base += groups * kHeads) {  // the same count in every lane
      if (base > 0) {
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
          const int h = base + group + j * groups;
          if (h < p.Hq) xq[j] = load_part(q + h * D, ea, eb);
        }
      }
#pragma unroll
      for (int j = 0; j < kHeads; ++j) {
        if (base + j * groups >= p.Hq) break;
        const int h = base + group + j * groups;
        const Part y = turn(xq[j], p.eps);
        if (h < p.Hq) store_part(out + h * D, ea, eb, y);
      }
    }
  }
  if (p.Hkv == 0) return;
  const Turn<kBf16, kInter, D> turn(c, s, lane < turning, p.k_weight, ea, eb);
  for (int base = 0; base < p.Hkv; base += groups) {
    const int h = base + group;
    if (base > 0 && h < p.Hkv) {
      xk = load_part(k + h * D, ea, eb);
      if (p.v) xv = load_part(v + h * D, ea, eb);
    }
    const Part y = turn(xk, p.eps);
    if (h < p.Hkv && cached) {
      const long long row = (slot * p.Hkv + h) * D;
      store_part(p.k_cache + row, ea, eb, y);
      if (p.v) store_part(p.v_cache + row, ea, eb, xv);
    }
  }
}

// Threads of a block: few tokens (a block an SM or fewer) take a lane group for
// every row, so that no row waits for another; many take eight groups, so that a
// lane's set-up is spent on several rows.  (16384 tokens of 32 + 2 x 8 heads of
// 128, with 4, 6, 8, 16 groups: 81, 90, 79, 107 us, and 72 with 64 registers a
// thread; 1003 of 40 + 2 x 8 heads of 64 with 8, 12, 16, 32: 4.0, 4.0, 4.8, 6.3.)
template <bool kBf16, bool kInter, int D>
cudaError_t launch(const RopeParams& p, cudaStream_t s) {
  int threads = 8 * (D / 8);
  if (p.T <= device_sms()) {
    const int rows = p.Hq > p.Hkv ? p.Hq : p.Hkv;
    threads = (rows * (D / 8) + 31) / 32 * 32;
    if (threads > kRopeThreads) threads = kRopeThreads;
  }
  qk_norm_rope_kernel<kBf16, kInter, D><<<p.T, threads, 0, s>>>(p);
  return cudaGetLastError();
}
template <bool kBf16, bool kInter>
cudaError_t launch(const RopeParams& p, int D, cudaStream_t s) {
  return D == 64    ? launch<kBf16, kInter, 64>(p, s)
         : D == 128 ? launch<kBf16, kInter, 128>(p, s)
                    : launch<kBf16, kInter, 256>(p, s);
}
template <bool kBf16>
cudaError_t launch(const RopeParams& p, int D, cudaStream_t s) {
  return p.interleaved ? launch<kBf16, true>(p, D, s) : launch<kBf16, false>(p, D, s);
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
  const long long q_row = 2ll * Hq * D, k_row = 2ll * Hkv * D;
  const RowSet qo = {q_out, T, q_row, 2 * q_out_stride}, kc = {k_cache, 1, k_row * n_slots, 0},
               vc = {v_cache, 1, k_row * n_slots, 0};
  if ((q_out == q && T > 1 ? q_stride != q_out_stride : q_out != q && rows_meet(qo, {q, T, q_row, 2 * q_stride})) ||
      rows_meet(qo, {k, T, k_row, 2 * k_stride}) || rows_meet(qo, {v, T, k_row, 2 * v_stride}) || rows_meet(qo, kc) ||
      rows_meet(qo, vc) || rows_meet(kc, vc))
    return MOE_ERR_INVALID_ARG;
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
