// Writes to and reads from a cache of keys and values in 4 bits (moe_kv4_write,
// moe_kv4_read).  Format and layout: kv4.cuh.
//
// A group of 32 channels x_c has the scale 2^s, the least power of two in [2^-23,
// 2^13] with max |x_c| <= 6 2^s, and the codes e2m1(x_c 2^-s), nearest, ties to
// the even code.  The product is exact in fp32 and so is what a code stands for in
// the 16-bit types, so a stored element does not depend on how it is computed.
//
// Both are bound by bytes.  Four lanes hold a group, 8 channels (16 bytes) each,
// and a warp 8 slots, so that 16-bit rows are read and written in whole sectors and
// the codes of neighbouring slots, which lie side by side, too.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <string.h>

#include "kv4.cuh"
#include "moe.h"

namespace moe {
namespace {

constexpr int kKvThreads = 256;

struct Kv4Params {
  const uint16_t *k, *v;       // write: rows of the call
  long long k_stride, v_stride;
  uint16_t *k_out, *v_out;     // read
  int T, Hkv, page, page_log2, n_pages;
  const int32_t* index;        // write: slots; read: pages (or NULL)
  uint8_t* cache;
  int32_t* status;
};

template <bool kBf16>
__device__ __forceinline__ float2 widen(uint32_t u) {
  if (kBf16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  __half2 h;
  memcpy(&h, &u, 4);
  return __half22float2(h);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t narrow(float2 f) {
  uint32_t u;
  if (kBf16) {
    const __nv_bfloat162 h = __float22bfloat162_rn(f);
    memcpy(&u, &h, 4);
  } else {
    const __half2 h = __float22half2_rn(f);
    memcpy(&u, &h, 4);
  }
  return u;
}
// Two fp32 as e2m1 codes: a in the low nibble, b in the high one.
__device__ __forceinline__ uint32_t code2(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(a), "f"(b));
  return r;
}

// 8 channels of one group in this lane, the group in 4 lanes: their codes and the
// group's scale byte.
template <bool kBf16>
__device__ __forceinline__ uint32_t encode8(const uint4& x, uint32_t& scale, bool& range) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  // magnitudes order as their bits do, infinities and NaN last
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
  top = max(top & 0xffffu, top >> 16);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  if (top >= (kBf16 ? 0x7f80u : 0x7c00u)) {
    scale = kKv4Nan;
    range = true;
    return 0;
  }
  // max = 1.m 2^e: 6 2^(e - 2) covers it up to 1.5
  const uint32_t bits = __float_as_uint(widen<kBf16>(top).x);
  int b = static_cast<int>(bits >> 23) - 2 + ((bits & 0x7fffffu) > 0x400000u ? 1 : 0);
  range |= b > kKv4High;
  b = min(max(b, kKv4Low), kKv4High);
  scale = static_cast<uint32_t>(b);
  const float f = __uint_as_float(static_cast<uint32_t>(254 - b) << 23);  // 2^-s
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = widen<kBf16>(w[i]);
    codes |= code2(p.x * f, p.y * f) << (8 * i);
  }
  return codes;
}

// A warp: 8 tokens, all D / 32 groups of the keys or values of one head.
template <bool kBf16, int D>
__global__ void __launch_bounds__(kKvThreads) kv4_write_kernel(const __grid_constant__ Kv4Params p) {
  constexpr int kGroups = D / 32;
  griddep_wait();
  const int lane = threadIdx.x & 31, part = lane & 3;
  const long long unit = static_cast<long long>(blockIdx.x) * (kKvThreads / 32) + (threadIdx.x >> 5);
  const int kinds = 2 * p.Hkv, t = static_cast<int>(unit / kinds) * 8 + (lane >> 2);
  const int which = static_cast<int>(unit % kinds) >= p.Hkv, h = static_cast<int>(unit % kinds) - which * p.Hkv;
  const bool live = t < p.T;
  uint4 x[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) x[g] = make_uint4(0, 0, 0, 0);
  int slot = -1;
  if (live) {
    const uint16_t* row = (which ? p.v + t * p.v_stride : p.k + t * p.k_stride) + h * D + part * 8;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) x[g] = *reinterpret_cast<const uint4*>(row + g * 32);
    slot = p.index ? __ldg(p.index + t) : t;
  }
  uint32_t codes[kGroups], scales = 0;
  bool range = false;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    uint32_t s;
    codes[g] = encode8<kBf16>(x[g], s, range);
    scales |= s << (8 * g);
  }
  if (slot < 0) return;
  if ((slot >> p.page_log2) >= p.n_pages) {
    record_index(p.status, kInfoSlot);
    return;
  }
  if (range) record_range(p.status, kInfoKvRange);
  const int at = slot & (p.page - 1);
  uint8_t* block = p.cache + (static_cast<long long>(slot >> p.page_log2) * p.Hkv + h) * (p.page * kv4_slot_bytes(D));
  uint8_t* dst = block + kv4_codes_at(D, p.page, which) + at * 16 + part * 4;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) *reinterpret_cast<uint32_t*>(dst + g * p.page * 16) = codes[g];
  if (part == 0) {
    uint8_t* s = block + kv4_scales_at(D, p.page, which) + at * kGroups;
    if (kGroups == 4) *reinterpret_cast<uint32_t*>(s) = scales;
    else *reinterpret_cast<uint16_t*>(s) = static_cast<uint16_t>(scales);
  }
}

// A warp: 8 slots, all groups of the keys or values of one page and head.
template <bool kBf16, int D>
__global__ void __launch_bounds__(kKvThreads) kv4_read_kernel(const __grid_constant__ Kv4Params p) {
  constexpr int kGroups = D / 32;
  griddep_wait();
  const int lane = threadIdx.x & 31, part = lane & 3;
  const long long unit = static_cast<long long>(blockIdx.x) * (kKvThreads / 32) + (threadIdx.x >> 5);
  // heads innermost: the warps of a block write neighbouring rows
  const int kinds = 2 * p.Hkv, runs = p.page / 8;
  const int kind = static_cast<int>(unit % kinds), which = kind >= p.Hkv, h = kind - which * p.Hkv;
  const long long i = unit / kinds / runs;
  if (i >= p.T) return;
  const int at = static_cast<int>(unit / kinds % runs) * 8 + (lane >> 2);
  int page = static_cast<int>(i);
  if (p.index) page = __ldg(p.index + i);
  uint16_t* out = (which ? p.v_out : p.k_out) + ((i * p.page + at) * p.Hkv + h) * D + part * 8;
  if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.n_pages)) {
    if (lane == 0) record_index(p.status, kInfoPage);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) *reinterpret_cast<uint4*>(out + g * 32) = make_uint4(0, 0, 0, 0);
    return;
  }
  const uint8_t* block = p.cache + (static_cast<long long>(page) * p.Hkv + h) * (p.page * kv4_slot_bytes(D));
  const uint8_t* src = block + kv4_codes_at(D, p.page, which) + at * 16 + part * 4;
  uint32_t codes[kGroups], scales;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) codes[g] = *reinterpret_cast<const uint32_t*>(src + g * p.page * 16);
  const uint8_t* s = block + kv4_scales_at(D, p.page, which) + at * kGroups;
  if (kGroups == 4) scales = *reinterpret_cast<const uint32_t*>(s);
  else scales = *reinterpret_cast<const uint16_t*>(s);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const float f = kv4_scale_f((scales >> (8 * g)) & 255u);
    uint32_t e[4];
    kv4_expand(codes[g], e);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 y = widen<false>(e[j]);
      e[j] = narrow<kBf16>(make_float2(y.x * f, y.y * f));
    }
    *reinterpret_cast<uint4*>(out + g * 32) = make_uint4(e[0], e[1], e[2], e[3]);
  }
}

typedef void Kernel(Kv4Params);
cudaError_t launch(Kernel* kernel, const Kv4Params& p, long long warps, cudaStream_t s) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kKvThreads / 32 - 1) / (kKvThreads / 32)));
  cfg.blockDim = dim3(kKvThreads);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

moe_status check_cache(int n_pages, int page_size, int Hkv, int D, int dtype) {
  if (n_pages < 0 || page_size < 1 || Hkv < 1 || D < 1) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0 || (D != 64 && D != 128) || Hkv > 1024)
    return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(n_pages) * page_size > INT32_MAX) return MOE_ERR_UNSUPPORTED;  // slots are int32
  return MOE_OK;
}

void fill(Kv4Params& p, int T, int Hkv, int page_size, int n_pages, const int32_t* index, void* cache, void* ws) {
  memset(&p, 0, sizeof(p));
  p.T = T; p.Hkv = Hkv; p.page = page_size; p.n_pages = n_pages;
  while ((1 << p.page_log2) < page_size) ++p.page_log2;
  p.index = index;
  p.cache = static_cast<uint8_t*>(cache);
  p.status = static_cast<int32_t*>(ws);
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_kv4_write(const void* k, long long k_stride, const void* v, long long v_stride, int T, int Hkv, int D,
                         int dtype, const int32_t* slots, void* cache, int n_pages, int page_size, void* ws,
                         size_t ws_bytes, cudaStream_t stream) {
  using namespace moe;
  if (T < 0) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_cache(n_pages, page_size, Hkv, D, dtype);
  if (st != MOE_OK) return st;
  if (T > MOE_MAX_ATTN_TOKENS) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!k || !v || k_stride < 0 || v_stride < 0 || (n_pages > 0 && !cache)) return MOE_ERR_INVALID_ARG;
  if (!slots && static_cast<long long>(n_pages) * page_size < T) return MOE_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache)) return MOE_ERR_INVALID_ARG;
  if (k_stride % 8 || v_stride % 8) return MOE_ERR_UNSUPPORTED;
  const RowSet pool = {cache, 1, static_cast<long long>(n_pages) * Hkv * page_size * kv4_slot_bytes(D), 0};
  if (rows_meet(pool, {k, T, 2ll * Hkv * D, 2 * k_stride}) || rows_meet(pool, {v, T, 2ll * Hkv * D, 2 * v_stride}) ||
      rows_meet(pool, {slots, 1, 4ll * T, 0}))
    return MOE_ERR_INVALID_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kWsAlign) != 0 || ws_bytes < MOE_STATUS_BYTES)
    return MOE_ERR_WORKSPACE;
  Kv4Params p;
  fill(p, T, Hkv, page_size, n_pages, slots, cache, ws);
  p.k = static_cast<const uint16_t*>(k); p.v = static_cast<const uint16_t*>(v);
  p.k_stride = k_stride; p.v_stride = v_stride;
  Kernel* kernel = dtype == MOE_DTYPE_BF16 ? (D == 64 ? kv4_write_kernel<true, 64> : kv4_write_kernel<true, 128>)
                                           : (D == 64 ? kv4_write_kernel<false, 64> : kv4_write_kernel<false, 128>);
  return launch(kernel, p, (T + 7) / 8 * 2ll * Hkv, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_kv4_read(const void* cache, int n_pages, int page_size, int Hkv, int D, const int32_t* pages, int n,
                        void* k, void* v, int dtype, void* ws, size_t ws_bytes, cudaStream_t stream) {
  using namespace moe;
  if (n < 0) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_cache(n_pages, page_size, Hkv, D, dtype);
  if (st != MOE_OK) return st;
  if (static_cast<long long>(n) * page_size > MOE_MAX_KEYS) return MOE_ERR_UNSUPPORTED;
  if (n == 0) return MOE_OK;
  if (!k || !v || (n_pages > 0 && !cache) || (!pages && n > n_pages)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache)) return MOE_ERR_INVALID_ARG;
  const long long bytes = 2ll * n * page_size * Hkv * D;
  const RowSet pool = {cache, 1, static_cast<long long>(n_pages) * Hkv * page_size * kv4_slot_bytes(D), 0};
  const RowSet ids = {pages, 1, 4ll * n, 0}, ko = {k, 1, bytes, 0}, vo = {v, 1, bytes, 0};
  if (rows_meet(ko, vo) || rows_meet(ko, pool) || rows_meet(vo, pool) || rows_meet(ko, ids) || rows_meet(vo, ids))
    return MOE_ERR_INVALID_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kWsAlign) != 0 || ws_bytes < MOE_STATUS_BYTES)
    return MOE_ERR_WORKSPACE;
  const long long warps = static_cast<long long>(n) * (page_size / 8) * 2 * Hkv;
  if ((warps + 7) / 8 > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  Kv4Params p;
  fill(p, n, Hkv, page_size, n_pages, pages, const_cast<void*>(cache), ws);
  p.k_out = static_cast<uint16_t*>(k); p.v_out = static_cast<uint16_t*>(v);
  Kernel* kernel = dtype == MOE_DTYPE_BF16 ? (D == 64 ? kv4_read_kernel<true, 64> : kv4_read_kernel<true, 128>)
                                           : (D == 64 ? kv4_read_kernel<false, 64> : kv4_read_kernel<false, 128>);
  return launch(kernel, p, warps, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
