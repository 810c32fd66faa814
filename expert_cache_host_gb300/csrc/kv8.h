// Shared by the operators on the 8-bit paged cache: e4m3 and scale-byte
// conversions and the checks of a caller's ft_kv8_cache.
#pragma once

#include "attn_side.h"

namespace ft {

// 2^i for any i (0 below 2^-149).
__device__ __forceinline__ float exp2i(int i) {
  return i >= -126 ? __uint_as_float((uint32_t)(i + 127) << 23) : i >= -149 ? __uint_as_float(1u << (i + 149)) : 0.f;
}
// What a scale byte stands for.
__device__ __forceinline__ float scale_of(uint32_t e) { return e == 255u ? __uint_as_float(0x7FC00000u) : exp2i((int)e - 127); }

// Two e4m3 numbers (the low 16 bits) as f16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("{ .reg .b16 h; cvt.u16.u32 h, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(v));
  return r;
}
// Four floats rounded to e4m3 (nearest even; past 448 in size 448, NaN 0x7F), the first in the lowest byte.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{ .reg .b16 l, h; cvt.rn.satfinite.e4m3x2.f32 l, %2, %1; cvt.rn.satfinite.e4m3x2.f32 h, %4, %3; mov.b32 %0, {l, h}; }"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// The larger magnitudes of two pairs (signs are of no account; NaN where there is one).
template <typename E>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (Elem<E>::kDtype == FT_DTYPE_BF16)
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float e4m3_value(uint8_t c) { return Elem<__half>::unpack(e4m3x2_to_f16x2(c)).x; }

// Sixteen e4m3 numbers times the power of two of scale byte e, rounded to a 16-bit
// type, for the bytes whose factor that type holds.  `sixteen` and `one` are these
// numbers, unknown to the compiler: multiplications run beside the other pipe's
// shifts and permutations, which bound this, and as shifts would join them.
template <typename E>
struct Scaled;
template <>
struct Scaled<__half> {
  // 2^-24 .. 2^15, and 0 where 448 * 2^(e - 127) rounds to it (blocks of zeros, places without a block).
  static __device__ __forceinline__ bool fast(uint32_t e, uint32_t) { return e - 103u <= 39u || e <= 93u; }
  static __device__ __forceinline__ uint32_t factor(uint32_t e) {
    const uint32_t f = e > 112u ? (e - 112u) << 10 : e >= 103u ? 1u << (e - 103u) : 0u;
    return f * 0x10001u;
  }
  static __device__ __forceinline__ uint32_t mul(uint32_t a, uint32_t f) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(f));
    return r;
  }
  static __device__ __forceinline__ void convert(const uint4& v, uint32_t f, uint32_t, uint32_t, uint32_t* o, uint32_t&) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t lo, hi;
      asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
          : "=r"(lo), "=r"(hi)
          : "r"(w[k]));
      o[2 * k] = mul(lo, f);
      o[2 * k + 1] = mul(hi, f);
    }
  }
};
template <>
struct Scaled<__nv_bfloat16> {
  // A code's bits in a bf16's places (sign, the low exponent and the high fraction bits) are 2^-120 of it, but for NaN
  // codes: these and 1 have the uppermost bit of a byte (`nan`).
  static __device__ __forceinline__ bool fast(uint32_t e, uint32_t nan) { return e <= 134u && !(nan & 0x80808080u); }
  static __device__ __forceinline__ uint32_t factor(uint32_t e) { return ((e + 120u) << 7) * 0x10001u; }  // 2^(e - 7)
  static __device__ __forceinline__ uint32_t mul(uint32_t a, uint32_t f) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(f));
    return r;
  }
  static __device__ __forceinline__ void convert(const uint4& v, uint32_t f, uint32_t sixteen, uint32_t one, uint32_t* o,
                                                 uint32_t& nan) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t size = w[k] & 0x7F7F7F7Fu, sign = w[k] & 0x80808080u;
      t[k] = size * one + 0x01010101u;
      // halves of a size in the low byte, times 16, and the sign in the high one
      o[2 * k] = mul(__byte_perm(size, 0, 0x4140) * sixteen + __byte_perm(sign, 0, 0x1404), f);
      o[2 * k + 1] = mul(__byte_perm(size, 0, 0x4342) * sixteen + __byte_perm(sign, 0, 0x3424), f);
    }
    nan |= (t[0] | t[1]) | (t[2] | t[3]);
  }
};

inline bool is_pow2(int x) { return x > 0 && !(x & (x - 1)); }
inline int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

// FT_OK, or records why the cache cannot be used.
inline int check_kv8_cache(const ft_kv8_cache& c) {
  if (!c.k || !c.v || !c.k_scale || !c.v_scale) return record_error(FT_E_ARG, "the cache's pointers must not be null");
  if (c.reserved) return record_error(FT_E_ARG, "the cache's reserved field must be zero");
  if (c.num_pages < 1 || c.kv_heads < 1 || c.head_dim < 1 || c.page_size < 1 || c.block_size < 1)
    return record_error(FT_E_ARG, "num_pages, kv_heads, head_dim, page_size and block_size must be positive");
  if (c.page_size < 16 || c.page_size > 4096 || !is_pow2(c.page_size))
    return record_error(FT_E_UNSUPPORTED, "page_size must be a power of two, 16 to 4096 (got %d)", c.page_size);
  if (c.block_size < 16 || c.block_size > 128 || !is_pow2(c.block_size) || c.block_size > c.page_size)
    return record_error(FT_E_UNSUPPORTED, "block_size must be a power of two, 16 to 128 and at most page_size (got %d)",
                        c.block_size);
  if (c.head_dim != 64 && c.head_dim != 128)
    return record_error(FT_E_UNSUPPORTED, "head_dim %d is not built", c.head_dim);
  if (c.kv_heads > 16384) return record_error(FT_E_UNSUPPORTED, "more than 16384 key heads");
  const int64_t s[6] = {c.k_page_stride, c.k_token_stride, c.k_head_stride,
                        c.v_page_stride, c.v_token_stride, c.v_head_stride};
  for (int64_t x : s)
    if (x < 0 || x % 16 || x >= (int64_t(1) << 38))
      return record_error(FT_E_ARG, "cache strides must be non-negative multiples of 16 bytes below 2^38");
  if (!c.k_token_stride || !c.v_token_stride || (c.kv_heads > 1 && (!c.k_head_stride || !c.v_head_stride)) ||
      (c.num_pages > 1 && (!c.k_page_stride || !c.v_page_stride)))
    return record_error(FT_E_ARG, "the cache's rows, heads and pages must not share memory (a stride is 0)");
  if (!is_16b(c.k) || !is_16b(c.v)) return record_error(FT_E_ARG, "the cache must be 16-byte aligned");
  return FT_OK;
}

}  // namespace ft
