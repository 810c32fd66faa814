// Shared by the attention-side operators: element conversions, packed fp32
// arithmetic and the checks of a caller's ft_kv_cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ft_internal.h"

namespace ft {

template <typename E>
struct Elem;  // two packed 16-bit elements <-> two floats
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kDtype = FT_DTYPE_BF16;
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&b);
  }
};
template <>
struct Elem<__half> {
  static constexpr int kDtype = FT_DTYPE_F16;
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __half2 b = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&b);
  }
};

// 2^x, and two fp32 numbers to an instruction.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

inline bool is_16b(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// FT_OK, or records why the cache cannot be used.
inline int check_kv_cache(const ft_kv_cache& c, bool head_256) {
  if (!c.k || !c.v) return record_error(FT_E_ARG, "the cache's k and v must not be null");
  if (c.reserved) return record_error(FT_E_ARG, "the cache's reserved field must be zero");
  if (c.dtype != FT_DTYPE_BF16 && c.dtype != FT_DTYPE_F16)
    return record_error(FT_E_ARG, "the cache's dtype must be FT_DTYPE_BF16 or FT_DTYPE_F16");
  if (c.num_pages < 1 || c.kv_heads < 1 || c.head_dim < 1 || c.page_size < 1)
    return record_error(FT_E_ARG, "num_pages, kv_heads, head_dim and page_size must be positive");
  if (c.page_size < 8 || c.page_size > 4096 || (c.page_size & (c.page_size - 1)))
    return record_error(FT_E_UNSUPPORTED, "page_size must be a power of two, 8 to 4096 (got %d)", c.page_size);
  if (c.head_dim != 64 && c.head_dim != 128 && !(head_256 && c.head_dim == 256))
    return record_error(FT_E_UNSUPPORTED, "head_dim %d is not built", c.head_dim);
  const int64_t s[6] = {c.k_page_stride, c.k_token_stride, c.k_head_stride,
                        c.v_page_stride, c.v_token_stride, c.v_head_stride};
  for (int64_t x : s)
    if (x < 0 || x % 8 || x >= (int64_t(1) << 38))
      return record_error(FT_E_ARG, "cache strides must be non-negative multiples of 8 elements below 2^38");
  if (!c.k_token_stride || !c.v_token_stride || (c.kv_heads > 1 && (!c.k_head_stride || !c.v_head_stride)) ||
      (c.num_pages > 1 && (!c.k_page_stride || !c.v_page_stride)))
    return record_error(FT_E_ARG, "the cache's rows, heads and pages must not share memory (a stride is 0)");
  if (!is_16b(c.k) || !is_16b(c.v)) return record_error(FT_E_ARG, "the cache must be 16-byte aligned");
  return FT_OK;
}

inline int sm_count() {
  static thread_local int known_dev = -1, sms = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev != known_dev) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return 1;
    known_dev = dev;
  }
  return sms;
}

}  // namespace ft
