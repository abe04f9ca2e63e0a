// Attention of a batch of requests whose cached context begins with one
// prefix that all of them share, followed by pages of their own
// (moe_prefix_attention).
//
// For the query of token t (the i-th of its request's n) and head h, over the
// prefix keys and the first `seen` of the request's own keys:
//   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale q . k_j,
// with the running maximum m and both sums held in fp32.
//
// One warp per (token, head): D / 32 elements of the row a lane, one key at a
// time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include "moe.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

struct AttnParams {
  const uint16_t *q, *k, *v;
  long long q_stride;
  int T, B, Hq, Hkv, n_pages, page;
  const int32_t *q_start, *prefix_pages, *prefix_len, *page_table, *own_len;
  int prefix_cap, table_width, causal;
  float scale_log2;
  uint16_t* out;
  float* lse;
  int32_t* status;
};

// A length read on the device, held within its page table.
__device__ __forceinline__ int held(int len, int pages, int page, int32_t* status) {
  if (len >= 0 && len <= pages * page) return len;
  record_index(status, kInfoLength);
  return len < 0 ? 0 : pages * page;
}

template <bool kBf16>
__device__ __forceinline__ float to_f(uint16_t u) {
  if (kBf16) return __bfloat162float(__ushort_as_bfloat16(u));
  return __half2float(__ushort_as_half(u));
}

template <bool kBf16, int D>
__device__ void keys(const AttnParams& p, const float (&q)[D / 32], const int32_t* pages, int count, int hk, float& m,
                     float& l, float (&o)[D / 32]) {
  const int lane = threadIdx.x & 31;
  for (int j = 0; j < count; ++j) {
    const int pg = __ldg(pages + j / p.page);
    float k[D / 32], v[D / 32];
    if (pg < 0 || pg >= p.n_pages) {
      if (lane == 0) record_index(p.status, kInfoPage);
      for (int i = 0; i < D / 32; ++i) k[i] = v[i] = 0.f;
    } else {
      const long long row = ((static_cast<long long>(pg) * p.page + j % p.page) * p.Hkv + hk) * D;
      for (int i = 0; i < D / 32; ++i) {
        k[i] = to_f<kBf16>(p.k[row + lane + 32 * i]);
        v[i] = to_f<kBf16>(p.v[row + lane + 32 * i]);
      }
    }
    float s = 0.f;
    for (int i = 0; i < D / 32; ++i) s += q[i] * k[i];
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2;
    const float m1 = fmaxf(m, s);
    const float base = m1 == -INFINITY ? 0.f : m1;
    const float a = exp2f(m - base), e = exp2f(s - base);
    m = m1;
    l = l * a + e;
    for (int i = 0; i < D / 32; ++i) o[i] = o[i] * a + e * v[i];
  }
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(128) prefix_attention_kernel(const __grid_constant__ AttnParams p) {
  const int lane = threadIdx.x & 31;
  const long long row = blockIdx.x * 4ll + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(p.T) * p.Hq) return;
  const int t = static_cast<int>(row / p.Hq), h = static_cast<int>(row % p.Hq), hk = h / (p.Hq / p.Hkv);
  int b = -1, first = 0, n = 0;
  for (int i = 0; i < p.B; ++i) {
    const int a = __ldg(p.q_start + i), z = __ldg(p.q_start + i + 1);
    if (a < 0 || z < a || z > p.T) {
      if (lane == 0) record_index(p.status, kInfoStarts);
      continue;
    }
    if (t >= a && t < z) { b = i; first = a; n = z - a; }
  }
  float q[D / 32], o[D / 32], m = -INFINITY, l = 0.f;
  for (int i = 0; i < D / 32; ++i) {
    q[i] = to_f<kBf16>(p.q[t * p.q_stride + h * D + lane + 32 * i]);
    o[i] = 0.f;
  }
  if (b >= 0) {
    if (p.prefix_cap > 0) {
      const int len = held(__ldg(p.prefix_len), p.prefix_cap, p.page, p.status);
      keys<kBf16, D>(p, q, p.prefix_pages, len, hk, m, l, o);
    }
    if (p.table_width > 0) {
      const int len = held(__ldg(p.own_len + b), p.table_width, p.page, p.status);
      const int seen = p.causal ? max(0, len - n + (t - first) + 1) : len;
      keys<kBf16, D>(p, q, p.page_table + static_cast<long long>(b) * p.table_width, min(seen, len), hk, m, l, o);
    }
  }
  const float r = l > 0.f ? 1.f / l : 0.f;
  for (int i = 0; i < D / 32; ++i) {
    const float y = o[i] * r;
    p.out[row * D + lane + 32 * i] =
        kBf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(y)) : __half_as_ushort(__float2half_rn(y));
  }
  if (lane == 0 && p.lse) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// MOE_OK where a batch of this shape is within the kernels' limits.
moe_status shape_status(int T, int B, int Hq, int Hkv, int D) {
  if (T < 0 || B < 0 || Hq < 1 || Hkv < 1 || D < 1) return MOE_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return MOE_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || Hq / Hkv > 128 || Hq > 1024 || T > MOE_MAX_ATTN_TOKENS || B > MOE_MAX_REQUESTS)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t workspace_bytes() { return kWsHeaderBytes; }

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_prefix_attention_workspace_bytes(int T, int B, int Hq, int Hkv, int D) {
  if (moe::shape_status(T, B, Hq, Hkv, D) != MOE_OK) return 0;
  return moe::workspace_bytes();
}

moe_status moe_prefix_attention(const void* q, long long q_stride, int T, int B, const int32_t* q_start, int Hq,
                                int Hkv, int D, int dtype, const void* k_cache, const void* v_cache, int n_pages,
                                int page_size, const int32_t* prefix_pages, int prefix_cap, const int32_t* prefix_len,
                                const int32_t* page_table, int table_width, const int32_t* own_len, int causal,
                                float scale, void* out, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  using namespace moe;
  const moe_status st = shape_status(T, B, Hq, Hkv, D);
  if (st != MOE_OK) return st;
  if (n_pages < 0 || page_size < 1 || prefix_cap < 0 || table_width < 0) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return MOE_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale < INFINITY)) return MOE_ERR_INVALID_ARG;
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(prefix_cap) * page_size > MOE_MAX_KEYS ||
      static_cast<long long>(table_width) * page_size > MOE_MAX_KEYS)
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!q || !out || q_stride < 0) return MOE_ERR_INVALID_ARG;
  if (B > 0 && !q_start) return MOE_ERR_INVALID_ARG;
  if (prefix_cap > 0 && (!prefix_pages || !prefix_len)) return MOE_ERR_INVALID_ARG;
  if (B > 0 && table_width > 0 && (!page_table || !own_len)) return MOE_ERR_INVALID_ARG;
  if (prefix_cap + table_width > 0 && (n_pages < 1 || !k_cache || !v_cache)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || q == out)
    return MOE_ERR_INVALID_ARG;
  if (q_stride % 8) return MOE_ERR_UNSUPPORTED;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kWsAlign) != 0 || ws_bytes < workspace_bytes())
    return MOE_ERR_WORKSPACE;
  AttnParams p;
  memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(q); p.q_stride = q_stride;
  p.k = static_cast<const uint16_t*>(k_cache); p.v = static_cast<const uint16_t*>(v_cache);
  p.T = T; p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.n_pages = n_pages; p.page = page_size;
  p.q_start = q_start; p.prefix_pages = prefix_pages; p.prefix_len = prefix_len; p.page_table = page_table;
  p.own_len = own_len;
  p.prefix_cap = prefix_cap; p.table_width = table_width; p.causal = causal;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = static_cast<uint16_t*>(out); p.lse = lse;
  p.status = static_cast<int32_t*>(ws);
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(T) * Hq + 3) / 4);
  if (dtype == MOE_DTYPE_BF16) {
    if (D == 64) prefix_attention_kernel<true, 64><<<grid, 128, 0, stream>>>(p);
    else prefix_attention_kernel<true, 128><<<grid, 128, 0, stream>>>(p);
  } else {
    if (D == 64) prefix_attention_kernel<false, 64><<<grid, 128, 0, stream>>>(p);
    else prefix_attention_kernel<false, 128><<<grid, 128, 0, stream>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
