// Per-head norms of queries and keys with the position rotation, keys and
// values written into the paged cache (ft_qk_norm_rope).
//
//   y = x / sqrt(mean(x^2) + eps) * weight, then (y_a, y_b) turned by the
//   token's angles; all in fp32, one rounding at the end.
//
// Every element is read and written once, so HBM bounds it (latency, for a
// few tokens).  A head is D/8 lanes with 8 elements each: a row is loaded and
// stored in 16-byte pieces, the mean is a shuffle sum over the head's lanes,
// and with the halves paired (i with i + rot/2) a lane's partner elements are
// the same 8 places of one other lane, which one shuffle per element fetches.  A
// warp takes HPW = 256/D heads at a time and ITER such groups of one token, so
// the token's angles are loaded once for ITER*HPW heads and ITER 16-byte loads
// per lane are in flight before the first is used.
#include "attn_side.h"

namespace ft {
namespace {

constexpr int kWarps = 8;

struct Args {
  ft_qk_args a;
  int heads;       // q_heads + 2 kv_heads
  int groups;      // warps' groups of heads per token
  int log2_page;
  int64_t num_slots;
  bool vec_in, vec_out;  // rows of q, k, v / q_out are 16-byte aligned
};

__device__ __forceinline__ uint4 load8(const uint16_t* p, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8(uint16_t* p, uint4 v, bool vec) {
  if (vec) {
    *reinterpret_cast<uint4*>(p) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[2 * i] = (uint16_t)w[i];
    p[2 * i + 1] = (uint16_t)(w[i] >> 16);
  }
}

template <typename E, int D, int ITER>
__global__ void __launch_bounds__(kWarps * 32) qk_norm_rope_kernel(const __grid_constant__ Args g) {
  constexpr int LPH = D / 8;      // lanes per head
  constexpr int HPW = 32 / LPH;   // heads per warp at a time
  const ft_qk_args& a = g.a;
  const int lane = threadIdx.x & 31, sub = lane % LPH;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t64 = unit / g.groups;
  if (t64 >= a.T) return;
  const int t = (int)t64, group = (int)(unit - t64 * g.groups);
  const int Hq = a.q_heads, Hkv = a.cache.kv_heads;

  const int pos = a.positions[t];
  const int64_t slot = a.slots[t];
  uint4 raw[ITER];
#pragma unroll
  for (int it = 0; it < ITER; ++it) {
    const int h = (group * ITER + it) * HPW + lane / LPH;
    if (h < g.heads) {
      const uint16_t* row;
      if (h < Hq)
        row = static_cast<const uint16_t*>(a.q) + t * a.q_stride + (int64_t)h * D;
      else if (h < Hq + Hkv)
        row = static_cast<const uint16_t*>(a.k) + t * a.k_stride + (int64_t)(h - Hq) * D;
      else
        row = static_cast<const uint16_t*>(a.v) + t * a.v_stride + (int64_t)(h - Hq - Hkv) * D;
      raw[it] = load8(row + sub * 8, g.vec_in);
    } else {
      raw[it] = make_uint4(0, 0, 0, 0);
    }
  }
  const bool in_range = pos >= 0 && pos < a.max_pos;
  const bool keep = in_range && slot >= 0 && slot < g.num_slots;  // keys and values are written
  if (a.status && group == 0 && lane == 0) {
    if (!in_range) atomicOr(a.status, FT_ST_BAD_TOKEN);
    if (slot >= g.num_slots) atomicOr(a.status, FT_ST_BAD_SLOT);
  }
  const int64_t page = slot >> g.log2_page;
  const int64_t row_in = slot & ((int64_t(1) << g.log2_page) - 1);

  // The angles of this lane's 8 elements.  Halves paired: element i < rot/2
  // and i + rot/2 share angle i; neighbours paired: 2i and 2i+1 share angle i.
  const int half = a.rot_dim / 2, e0 = sub * 8;
  const bool rotated = e0 < a.rot_dim;  // rot_dim is a multiple of 16: a lane's 8 elements are on one side
  const bool upper = e0 >= half;        // halves: this lane holds the second member of its pairs
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  if (rotated && in_range) {
    const float* base = a.cos_sin + (int64_t)pos * a.rot_dim;
    if (a.interleaved) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(base + sub * 4));
      const float4 s = __ldg(reinterpret_cast<const float4*>(base + half + sub * 4));
      cs[0] = cs[1] = c.x, cs[2] = cs[3] = c.y, cs[4] = cs[5] = c.z, cs[6] = cs[7] = c.w;
      sn[0] = sn[1] = s.x, sn[2] = sn[3] = s.y, sn[4] = sn[5] = s.z, sn[6] = sn[7] = s.w;
    } else {
      const float* p = base + (upper ? e0 - half : e0);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(p) + v);
        const float4 s = __ldg(reinterpret_cast<const float4*>(p + half) + v);
        cs[4 * v] = c.x, cs[4 * v + 1] = c.y, cs[4 * v + 2] = c.z, cs[4 * v + 3] = c.w;
        sn[4 * v] = s.x, sn[4 * v + 1] = s.y, sn[4 * v + 2] = s.z, sn[4 * v + 3] = s.w;
      }
    }
  }
  // the lane of this head with the paired elements (itself where neighbours are paired)
  const int hop = half / 8;
  const int mate = lane - sub + (a.interleaved || !rotated ? sub : (upper ? sub - hop : sub + hop));
  const uint4 wq = __ldg(reinterpret_cast<const uint4*>(a.q_weight) + sub);
  const uint4 wk = __ldg(reinterpret_cast<const uint4*>(a.k_weight) + sub);

#pragma unroll
  for (int it = 0; it < ITER; ++it) {
    const int h = (group * ITER + it) * HPW + lane / LPH;
    const uint32_t rw[4] = {raw[it].x, raw[it].y, raw[it].z, raw[it].w};
    float x[8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Elem<E>::unpack(rw[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
      ss = fmaf(f.x, f.x, fmaf(f.y, f.y, ss));
    }
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(~0u, ss, o);
    const float r = 1.f / sqrtf(ss * (1.f / D) + a.eps);
    const uint4 w4 = h < Hq ? wq : wk;
    const uint32_t ww[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Elem<E>::unpack(ww[i]);
      x[2 * i] *= r * f.x;
      x[2 * i + 1] *= r * f.y;
    }
    float y[8];
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
    uint4 o = raw[it];
    if (h < Hq + Hkv) {
      o.x = Elem<E>::pack(y[0], y[1]);
      o.y = Elem<E>::pack(y[2], y[3]);
      o.z = Elem<E>::pack(y[4], y[5]);
      o.w = Elem<E>::pack(y[6], y[7]);
    }
    if (h < Hq) {
      if (!in_range) o = make_uint4(0, 0, 0, 0);
      store8(static_cast<uint16_t*>(a.q_out) + t * a.q_out_stride + (int64_t)h * D + e0, o, g.vec_out);
    } else if (h < g.heads && keep) {
      const bool is_k = h < Hq + Hkv;
      const int kh = h - Hq - (is_k ? 0 : Hkv);
      uint16_t* dst = static_cast<uint16_t*>(is_k ? a.cache.k : a.cache.v) +
                      page * (is_k ? a.cache.k_page_stride : a.cache.v_page_stride) +
                      row_in * (is_k ? a.cache.k_token_stride : a.cache.v_token_stride) +
                      kh * (is_k ? a.cache.k_head_stride : a.cache.v_head_stride) + e0;
      *reinterpret_cast<uint4*>(dst) = o;
    }
  }
}

template <typename E, int D>
cudaError_t launch(Args g, cudaStream_t st) {
  constexpr int HPW = 32 / (D / 8);
  const int sets = (g.heads + HPW - 1) / HPW;  // warp-wide sets of heads per token
  // Few tokens: one set per warp, so that a token spreads over the machine
  // (latency).  Many: four, so that angles and weights are loaded once for
  // four and four loads per lane are in flight.
  const bool many = (int64_t)g.a.T * sets >= (int64_t)sm_count() * kWarps * 8;
  const int iter = many ? 4 : 1;
  g.groups = (sets + iter - 1) / iter;
  const int64_t units = (int64_t)g.a.T * g.groups;
  const int64_t grid = (units + kWarps - 1) / kWarps;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  if (many)
    qk_norm_rope_kernel<E, D, 4><<<(unsigned)grid, kWarps * 32, 0, st>>>(g);
  else
    qk_norm_rope_kernel<E, D, 1><<<(unsigned)grid, kWarps * 32, 0, st>>>(g);
  return cudaGetLastError();
}

template <typename E>
cudaError_t launch_d(const Args& g, cudaStream_t st) {
  switch (g.a.cache.head_dim) {
    case 64: return launch<E, 64>(g, st);
    case 128: return launch<E, 128>(g, st);
    default: return launch<E, 256>(g, st);
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
  if (!a.q || !a.k || !a.v || !a.q_weight || !a.k_weight || !a.positions || !a.slots || !a.q_out ||
      (!a.cos_sin && a.rot_dim))
    return record_error(FT_E_ARG, "null pointer");
  if (a.rot_dim < 0 || a.rot_dim > a.cache.head_dim)
    return record_error(FT_E_ARG, "rot_dim must be 0 to head_dim");
  if (a.rot_dim % 16) return record_error(FT_E_UNSUPPORTED, "rot_dim must be a multiple of 16");
  if (!is_16b(a.cos_sin) || !is_16b(a.q_weight) || !is_16b(a.k_weight))
    return record_error(FT_E_ARG, "cos_sin and the weights must be 16-byte aligned");
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
