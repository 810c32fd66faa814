// Per-head norms of queries and keys with the position rotation, keys and
// values written into the paged cache (ft_qk_norm_rope).
//
//   y = x / sqrt(mean(x^2) + eps) * weight, then (y_a, y_b) turned by the
//   token's angles; all in fp32, one rounding at the end.
//
// Every element is read and written once, so HBM bounds it (latency, for a
// few tokens) if the instructions per element stay few.  A head is D/8 lanes
// with 8 elements each; the mean is a shuffle sum over the head's lanes.  A
// warp takes HPW = 256/D heads at a time and ITER such sets of one token, so
// that the token's angles and the weights are loaded once for ITER*HPW heads
// and ITER 16-byte loads per lane are in flight before the first is used.
// What is left is latency: 8192 tokens with 32/4 heads of 128 (172 MB) take
// 32.0 us = 5.4 TB/s, a plain copy of the same bytes 25.9 us.
//
// With the whole head rotated in halves (i with i + D/2) a lane holds both
// members of its pairs: elements 4l..4l+3 of either half.  The weights then go
// into the angles once per token, y_a = r (x_a (w_a c) - x_b (w_b s)), and an
// element costs 1.5 packed fp32 operations beside its conversions.  Otherwise
// a lane holds 8 neighbours, and a partner half is another lane's 8 (a shuffle
// each).
#include <algorithm>

#include "attn_side.h"
#include "tma.h"

namespace ft {
namespace {

constexpr int kWarps = 4;
// Resident blocks per SM where there are many tokens (the most without spills).
// 8192 tokens, 32/4 heads of 128: 32.0 us with 6, 33.8 with 5, 34.9 with 8.
// 8000 tokens, 40/8 heads of 64, 32 rotated: 31.6 us with 5, 34.9 with 6.
constexpr int kBlocks = 6, kBlocksOther = 5;

struct Args {
  ft_qk_args a;
  int heads;       // q_heads + 2 kv_heads
  int groups;      // warps' groups of heads per token
  int log2_page;
  int64_t num_slots;
  bool vec_in, vec_out;  // rows of q, k, v / q_out are 16-byte aligned
};

__device__ __forceinline__ uint4 load8(const uint16_t* lo, const uint16_t* hi, bool split, bool vec) {
  if (vec) {
    if (!split) return *reinterpret_cast<const uint4*>(lo);
    const uint2 a = *reinterpret_cast<const uint2*>(lo), b = *reinterpret_cast<const uint2*>(hi);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t* p = (i < 2 ? lo + 2 * i : hi + 2 * (i - 2));
    w[i] = (uint32_t)p[0] | ((uint32_t)p[1] << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8(uint16_t* lo, uint16_t* hi, uint4 v, bool split, bool vec) {
  if (vec) {
    if (!split) {
      *reinterpret_cast<uint4*>(lo) = v;
    } else {
      *reinterpret_cast<uint2*>(lo) = make_uint2(v.x, v.y);
      *reinterpret_cast<uint2*>(hi) = make_uint2(v.z, v.w);
    }
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t* p = (i < 2 ? lo + 2 * i : hi + 2 * (i - 2));
    p[0] = (uint16_t)w[i];
    p[1] = (uint16_t)(w[i] >> 16);
  }
}

// Four weights as two pairs.
struct Pairs {
  uint64_t lo, hi;
};
template <typename E>
__device__ __forceinline__ Pairs weights4(const void* w, int at) {
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + at));
  const float2 a = Elem<E>::unpack(v.x), b = Elem<E>::unpack(v.y);
  return {pair2(a.x, a.y), pair2(b.x, b.y)};
}
__device__ __forceinline__ Pairs angles4(const float* p) {
  const float4 v = __ldg(reinterpret_cast<const float4*>(p));
  return {pair2(v.x, v.y), pair2(v.z, v.w)};
}
__device__ __forceinline__ Pairs operator*(Pairs a, Pairs b) { return {mul2(a.lo, b.lo), mul2(a.hi, b.hi)}; }
__device__ __forceinline__ Pairs fma4(Pairs a, Pairs b, Pairs c) { return {fma2(a.lo, b.lo, c.lo), fma2(a.hi, b.hi, c.hi)}; }

// HALVES: the whole head rotated, i with i + D/2.
template <typename E, int D, int ITER, bool HALVES>
__global__ void __launch_bounds__(kWarps * 32, ITER == 1 ? 1 : HALVES ? kBlocks : kBlocksOther) qk_norm_rope_kernel(const __grid_constant__ Args g) {
  constexpr int LPH = D / 8;      // lanes per head
  constexpr int HPW = 32 / LPH;   // heads per warp at a time
  const ft_qk_args& a = g.a;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, sub = lane % LPH;
  const int Hq = a.q_heads, Hkv = a.cache.kv_heads;
  // this lane's elements of a head: 4 at e0 and 4 at e1
  const int e0 = HALVES ? sub * 4 : sub * 8, e1 = HALVES ? D / 2 + sub * 4 : sub * 8 + 4;

  // Units (a token's group of heads) in turn; the next one's position and slot
  // are fetched beside this one's rows, so that rows and angles take one
  // latency and not three in a row.
  const uint32_t units = (uint32_t)a.T * g.groups, stride = gridDim.x * kWarps;
  uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (unit >= units) return;
  int next_t = (int)(unit / (uint32_t)g.groups), next_pos = a.positions[next_t];
  int64_t next_slot = a.slots[next_t];
#pragma unroll 1
  for (;;) {
    const int t = next_t, group = (int)(unit - (uint32_t)t * g.groups), pos = next_pos;
    const int64_t slot = next_slot;
    const bool more = ITER > 1 && units - unit > stride;
    if (more) {
      unit += stride;
      next_t = (int)(unit / (uint32_t)g.groups);
      next_pos = a.positions[next_t];
      next_slot = a.slots[next_t];
    }
    const int h0 = group * ITER * HPW + lane / LPH;
    uint4 raw[ITER];
    {
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + t * a.q_stride;
      const uint16_t* k = static_cast<const uint16_t*>(a.k) + t * a.k_stride - (int64_t)Hq * D;
      const uint16_t* v = static_cast<const uint16_t*>(a.v) + t * a.v_stride - (int64_t)(Hq + Hkv) * D;
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int h = h0 + it * HPW;
        if (h < g.heads) {
          const uint16_t* row = (h < Hq ? q : h < Hq + Hkv ? k : v) + (int64_t)h * D;
          raw[it] = load8(row + e0, row + e1, HALVES, g.vec_in);
        } else {
          raw[it] = make_uint4(0, 0, 0, 0);
        }
      }
    }
    const bool in_range = pos >= 0 && pos < a.max_pos;
    const bool keep = in_range && slot >= 0 && slot < g.num_slots;  // keys and values are written
    if (a.status && group == 0 && lane == 0) {
      if (!in_range) atomicOr(a.status, FT_ST_BAD_TOKEN);
      if (slot >= g.num_slots) atomicOr(a.status, FT_ST_BAD_SLOT);
    }
    const int64_t page = keep ? slot >> g.log2_page : 0;
    const int64_t row_in = keep ? slot & ((int64_t(1) << g.log2_page) - 1) : 0;
    uint16_t* const q_out = static_cast<uint16_t*>(a.q_out) + t * a.q_out_stride;
    uint16_t* const k_out = static_cast<uint16_t*>(a.cache.k) + page * a.cache.k_page_stride + row_in * a.cache.k_token_stride;
    uint16_t* const v_out = static_cast<uint16_t*>(a.cache.v) + page * a.cache.v_page_stride + row_in * a.cache.v_token_stride;

    // The angles and weights of this lane's elements.  Halves paired: element
    // i < rot/2 and i + rot/2 share angle i; neighbours paired: 2i and 2i+1 do.
    const int half = a.rot_dim / 2;
    const bool rotated = HALVES || sub * 8 < a.rot_dim;  // rot_dim is a multiple of 16: a lane's 8 are on one side
    const bool upper = !HALVES && sub * 8 >= half;       // this lane holds the second members of its pairs
    const float* angles = a.cos_sin + (int64_t)(in_range ? pos : 0) * a.rot_dim;
    bool for_keys = h0 >= Hq;  // whose weights are in use
    Pairs wa, wb;              // halves not in a lane: the weights
    Pairs ac, bs, bc, as;      // else w_a c, -w_b s, w_b c, w_a s
    auto take_weights = [&] {
      const void* w = for_keys ? a.k_weight : a.q_weight;
      wa = weights4<E>(w, e0), wb = weights4<E>(w, e1);
      if constexpr (HALVES) {
        const uint64_t minus = pair2(-1.f, -1.f);
        const Pairs c = angles4(angles + e0), s = angles4(angles + half + e0);
        ac = wa * c, bc = wb * c, as = wa * s;
        bs = wb * s;
        bs = bs * Pairs{minus, minus};
      }
    };
    take_weights();
    float cs[8], sn[8];
    if constexpr (!HALVES) {
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
      if (rotated) {
        if (a.interleaved) {
          const float4 c = __ldg(reinterpret_cast<const float4*>(angles + sub * 4));
          const float4 s = __ldg(reinterpret_cast<const float4*>(angles + half + sub * 4));
          cs[0] = cs[1] = c.x, cs[2] = cs[3] = c.y, cs[4] = cs[5] = c.z, cs[6] = cs[7] = c.w;
          sn[0] = sn[1] = s.x, sn[2] = sn[3] = s.y, sn[4] = sn[5] = s.z, sn[6] = sn[7] = s.w;
        } else {
          const float* p = angles + (upper ? sub * 8 - half : sub * 8);
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const float4 c = __ldg(reinterpret_cast<const float4*>(p) + v);
            const float4 s = __ldg(reinterpret_cast<const float4*>(p + half) + v);
            cs[4 * v] = c.x, cs[4 * v + 1] = c.y, cs[4 * v + 2] = c.z, cs[4 * v + 3] = c.w;
            sn[4 * v] = s.x, sn[4 * v + 1] = s.y, sn[4 * v + 2] = s.z, sn[4 * v + 3] = s.w;
          }
        }
      }
    }
    // the lane of this head with the paired elements (itself where neighbours are paired)
    const int hop = half / 8;
    const int mate = lane - sub + (a.interleaved || !rotated ? sub : (upper ? sub - hop : sub + hop));
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const int h = h0 + it * HPW;
      uint4 o = raw[it];
      if (h0 - lane / LPH + it * HPW < Hq + Hkv) {  // (warp-uniform: not a set of values alone)
        const bool key = h >= Hq;
        if (key != for_keys) {
          for_keys = key;
          take_weights();
        }
        const uint32_t rw[4] = {raw[it].x, raw[it].y, raw[it].z, raw[it].w};
        uint64_t x2[4];
        uint64_t sq = pair2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = Elem<E>::unpack(rw[i]);
          x2[i] = pair2(f.x, f.y);
          sq = fma2(x2[i], x2[i], sq);
        }
        const float2 s2 = split2(sq);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int p = 1; p < LPH; p <<= 1) ss += __shfl_xor_sync(~0u, ss, p);
        const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
        const uint64_t r2 = pair2(r, r);
        float y[8];
        if constexpr (HALVES) {
          const Pairs xa = Pairs{x2[0], x2[1]} * Pairs{r2, r2}, xb = Pairs{x2[2], x2[3]} * Pairs{r2, r2};
          const Pairs ya = fma4(xa, ac, xb * bs), yb = fma4(xb, bc, xa * as);
          const uint64_t y2[4] = {ya.lo, ya.hi, yb.lo, yb.hi};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = split2(y2[i]);
            y[2 * i] = f.x, y[2 * i + 1] = f.y;
          }
        } else {
          const uint64_t w2[4] = {wa.lo, wa.hi, wb.lo, wb.hi};
          float x[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = split2(mul2(x2[i], mul2(r2, w2[i])));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
          }
          if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              y[i] = x[i] * cs[i] - x[i + 1] * sn[i];
              y[i + 1] = x[i + 1] * cs[i] + x[i] * sn[i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float m = __shfl_sync(~0u, x[i], mate);
              y[i] = upper ? fmaf(x[i], cs[i], m * sn[i]) : fmaf(x[i], cs[i], -m * sn[i]);
            }
          }
          if (!rotated) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[i];
          }
        }
        if (h < Hq + Hkv) {
          o.x = Elem<E>::pack(y[0], y[1]);
          o.y = Elem<E>::pack(y[2], y[3]);
          o.z = Elem<E>::pack(y[4], y[5]);
          o.w = Elem<E>::pack(y[6], y[7]);
        }
      }
      if (h < Hq) {
        if (!in_range) o = make_uint4(0, 0, 0, 0);
        uint16_t* dst = q_out + (int64_t)h * D;
        store8(dst + e0, dst + e1, o, HALVES, g.vec_out);
      } else if (h < g.heads && keep) {
        const bool is_k = h < Hq + Hkv;
        uint16_t* dst = is_k ? k_out + (int64_t)(h - Hq) * a.cache.k_head_stride
                             : v_out + (int64_t)(h - Hq - Hkv) * a.cache.v_head_stride;
        store8(dst + e0, dst + e1, o, HALVES, true);
      }
    }
    if (!more) break;
  }
}

template <typename E, int D, bool HALVES>
cudaError_t launch(Args g, cudaStream_t st) {
  constexpr int HPW = 32 / (D / 8);
  const int sets = (g.heads + HPW - 1) / HPW;  // warp-wide sets of heads per token
  // Few tokens: one set per warp, so that a token spreads over the machine
  // (latency).  Many: four, so that angles and weights are loaded once for
  // four and four loads per lane are in flight, on resident warps that take
  // one unit after another (512 tokens: 3.4 us, one set per warp 4.1; below,
  // as fast).
  const bool many = (int64_t)g.a.T * sets >= (int64_t)sm_count() * 64;
  const int iter = many ? 4 : 1;
  g.groups = (sets + iter - 1) / iter;
  const int64_t units = (int64_t)g.a.T * g.groups;
  const int64_t all = (units + kWarps - 1) / kWarps, resident = sm_count() * (HALVES ? kBlocks : kBlocksOther);
  const int64_t grid = many ? std::min(all, resident) : all;
  if (units > 0x7FFFFF00) return cudaErrorInvalidValue;  // (refused before: T is limited)
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(cfg, attr, dim3((unsigned)grid), dim3(kWarps * 32), 0, st);
  return many ? cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<E, D, 4, HALVES>, g)
              : cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<E, D, 1, HALVES>, g);
}

template <typename E, int D>
cudaError_t launch_r(const Args& g, cudaStream_t st) {
  return g.a.rot_dim == D && !g.a.interleaved ? launch<E, D, true>(g, st) : launch<E, D, false>(g, st);
}

template <typename E>
cudaError_t launch_d(const Args& g, cudaStream_t st) {
  switch (g.a.cache.head_dim) {
    case 64: return launch_r<E, 64>(g, st);
    case 128: return launch_r<E, 128>(g, st);
    default: return launch_r<E, 256>(g, st);
  }
}

}  // namespace
}  // namespace ft

extern "C" int ft_qk_norm_rope(const ft_qk_args* args, void* stream) {
  using namespace ft;
  if (!args) return record_error(FT_E_ARG, "null args");
  const ft_qk_args& a = *args;
  if (int rc = check_kv_cache(a.cache, true)) return rc;
  if (a.T < 0 || a.q_heads < 1 || a.max_pos < 1) return record_error(FT_E_ARG, "bad T, q_heads or max_pos");
  if ((int64_t)a.T * ((int64_t)a.q_heads + 2 * (int64_t)a.cache.kv_heads) > 0x7FFFFF00)
    return record_error(FT_E_ARG, "T times the heads must stay below 2^31");
  if (!a.q || !a.k || !a.v || !a.q_weight || !a.k_weight || !a.positions || !a.slots || !a.q_out ||
      (!a.cos_sin && a.rot_dim))
    return record_error(FT_E_ARG, "null pointer");
  if (a.rot_dim < 0 || a.rot_dim > a.cache.head_dim)
    return record_error(FT_E_ARG, "rot_dim must be 0 to head_dim");
  if (a.rot_dim % 16) return record_error(FT_E_UNSUPPORTED, "rot_dim must be a multiple of 16");
  if (!is_16b(a.cos_sin) || !is_16b(a.q_weight) || !is_16b(a.k_weight))
    return record_error(FT_E_ARG, "cos_sin and the weights must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
       reinterpret_cast<uintptr_t>(a.q_out)) % 2)
    return record_error(FT_E_ARG, "q, k, v and q_out must be aligned to their type");
  if (!(a.eps >= 0.f)) return record_error(FT_E_ARG, "eps must not be negative");
  if (a.q_out == a.q && a.q_out_stride != a.q_stride)
    return record_error(FT_E_ARG, "q_out on top of q needs the same stride");
  if (a.q_stride < 0 || a.k_stride < 0 || a.v_stride < 0 || a.q_out_stride < 0)
    return record_error(FT_E_ARG, "strides must not be negative");
  if (a.T == 0) return FT_OK;
  Args g{};
  g.a = a;
  g.heads = a.q_heads + 2 * a.cache.kv_heads;
  while ((1 << g.log2_page) < a.cache.page_size) ++g.log2_page;
  g.num_slots = (int64_t)a.cache.num_pages * a.cache.page_size;
  g.vec_in = is_16b(a.q) && is_16b(a.k) && is_16b(a.v) && (a.q_stride | a.k_stride | a.v_stride) % 8 == 0;
  g.vec_out = is_16b(a.q_out) && a.q_out_stride % 8 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.cache.dtype == FT_DTYPE_BF16 ? launch_d<__nv_bfloat16>(g, st) : launch_d<__half>(g, st);
  if (e != cudaSuccess) return record_error(FT_E_CUDA, "norm and rotation launch failed: %s", cudaGetErrorString(e));
  return FT_OK;
}
