// Keys and values quantised into the 8-bit paged cache (ft_kv8_store) and rows
// of it read back in 16 bits (ft_kv8_load).
//
// A block of tokens of one head has one scale 2^(e-127), e the least byte with
// max |x| <= 448 * 2^(e-127): a power of two, so that x 2^(127-e) is exact, the
// one rounding is that to e4m3, and a block whose scale grows later keeps its
// earlier tokens exactly but for those that become subnormal.
//
// Store: a unit is (request's block, head, keys or values); W warps hold its
// rows in registers, 8 rows' stretches a lane, between the maximum and the
// codes, so that every number is read once.  Load: a lane takes 16 codes of
// kItems rows at a time.  HBM bounds the load where there are many rows (32768 of 8
// heads of 128, 202 MB: 33 us = 6.1 TB/s), latency both where there are few (64
// tokens stored: 3.3 us, 77 rows read: 2.5); the store of many comes near with its
// pipe of comparisons and conversions 57 % busy (8192 tokens, 50 MB: 10.8 us).
#include <algorithm>

#include "kv8.h"
#include "tma.h"

namespace ft {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSteps = 8;  // 16-byte stretches a lane holds
constexpr int kSpan = 4;   // requests a lane looks at together

struct StoreArgs {
  ft_kv8_store_args a;
  int log2_page, log2_block;
};

// A request's rows and the blocks they reach.
struct Rows {
  int q0, n, ctx;
};
__device__ __forceinline__ Rows rows_of(const ft_kv8_store_args& a, int b) {
  Rows r;
  r.q0 = a.q_start[b];
  r.n = r.q0 < 0 ? 0 : max(min(a.q_start[b + 1], a.max_tokens) - r.q0, 0);
  r.ctx = max(a.ctx_len[b], 0);
  return r;
}

template <typename E>
constexpr uint32_t kInf16 = Elem<E>::kDtype == FT_DTYPE_BF16 ? 0x7F80u : 0x7C00u;
// From this byte on a code of 256 would pass the type's range.
template <typename E>
constexpr int kCapByte = Elem<E>::kDtype == FT_DTYPE_BF16 ? 247 : 135;

template <typename E, int D, int W>
__global__ void __launch_bounds__(kThreads, 4) kv8_store_kernel(const __grid_constant__ StoreArgs g) {
  constexpr int LPR = D / 8, RPS = 32 / LPR;  // lanes of a row, rows of a warp's step
  const ft_kv8_store_args& a = g.a;
  __shared__ uint32_t s_max[kWarps];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The request and block of unit blockIdx.x, from sums of the requests' blocks: every warp for itself, 32 * kSpan
  // requests at a time, their lengths loaded together.
  const int bs_mask = (1 << g.log2_block) - 1;
  Rows r{};
  int b = -1, j = 0;
  for (long long base = 0, b0 = 0; b0 < a.num_reqs; b0 += 32 * kSpan) {
    Rows mine[kSpan];
    long long cnt[kSpan], sum = 0;
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
      mine[i] = Rows{};
      if (b0 + lane * kSpan + i < a.num_reqs) mine[i] = rows_of(a, (int)b0 + lane * kSpan + i);
    }
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
      cnt[i] = mine[i].n > 0 ? (((long long)mine[i].ctx + mine[i].n + bs_mask) >> g.log2_block) - (mine[i].ctx >> g.log2_block) : 0;
      sum += cnt[i];
    }
    long long x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    const uint32_t hit = __ballot_sync(~0u, base + x > (long long)blockIdx.x);
    if (hit) {
      const int from = __ffs(hit) - 1;
      long long at = (long long)blockIdx.x - (base + x - sum);  // the unit's place in the lane's requests
      int which = 0;
#pragma unroll
      for (int i = 0; i + 1 < kSpan; ++i) {
        const bool past = which == i && at >= cnt[i];
        at -= past ? cnt[i] : 0;
        which += past ? 1 : 0;
      }
#pragma unroll
      for (int i = 0; i < kSpan; ++i)
        if (which == i) r = mine[i];
      r.q0 = __shfl_sync(~0u, r.q0, from);
      r.n = __shfl_sync(~0u, r.n, from);
      r.ctx = __shfl_sync(~0u, r.ctx, from);
      j = (int)__shfl_sync(~0u, at, from);
      b = (int)b0 + from * kSpan + __shfl_sync(~0u, which, from);
      break;
    }
    base += __shfl_sync(~0u, x, 31);
  }
  if (b < 0) return;  // (the whole block)
  const long long block0 = ((long long)(r.ctx >> g.log2_block) + j) << g.log2_block;  // the block's first token
  const int lo = (int)max((long long)r.ctx - block0, 0ll);                              // its new rows are [lo, hi)
  const int hi = (int)min((long long)r.ctx + r.n - block0, (long long)bs_mask + 1);
  const int sub = blockIdx.y * (kWarps / W) + warp / W;
  const bool active = sub < 2 * a.cache.kv_heads;
  const bool values = sub >= a.cache.kv_heads;
  const int head = values ? sub - a.cache.kv_heads : sub;

  // the page (its load runs beside the rows')
  const long long col = block0 >> g.log2_page;
  const int page = col < a.table_width ? a.block_table[(int64_t)b * a.table_width + col] : -1;
  const int row0 = (warp % W) * RPS * kSteps + lane / LPR, e0 = (lane % LPR) * 8;
  uint4 x[kSteps];
  {
    const uint16_t* src = static_cast<const uint16_t*>(values ? a.v : a.k) + (int64_t)head * D + e0;
    const int64_t stride = values ? a.v_stride : a.k_stride;
    const int64_t t0 = r.q0 + (block0 - r.ctx);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int row = row0 + i * RPS;
      x[i] = make_uint4(0, 0, 0, 0);
      if (active && row >= lo && row < hi) x[i] = *reinterpret_cast<const uint4*>(src + (t0 + row) * stride);
    }
  }
  const bool there = page >= 0 && page < a.cache.num_pages;
  const int in_page = (int)(block0 & ((1 << g.log2_page) - 1));
  uint8_t* scale = (values ? a.cache.v_scale : a.cache.k_scale) +
                   ((int64_t)(there ? page : 0) * (1 << (g.log2_page - g.log2_block)) + (in_page >> g.log2_block)) *
                       a.cache.kv_heads + (active ? head : 0);
  uint32_t was = active && there && lo > 0 ? *scale : 0u;
  if (!there && a.status && tid == 0 && blockIdx.y == 0) atomicOr(a.status, FT_ST_BAD_SLOT);

  // The largest finite number, as 16 bits without the sign (ordered as whole numbers).
  constexpr uint32_t inf = kInf16<E>;
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
    m2 = max_abs2<E>(max_abs2<E>(max_abs2<E>(m2, x[i].x), x[i].y), max_abs2<E>(x[i].z, x[i].w));
  m2 &= 0x7FFF7FFFu;
  uint32_t m = __reduce_max_sync(~0u, max(m2 & 0xFFFFu, m2 >> 16));
  const bool odd = m >= inf;  // infinities or NaN among the warp's numbers
  if (odd) {
    m = 0;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t h = (w[k >> 1] >> (k & 1 ? 16 : 0)) & 0x7FFFu;
        if (h < inf) m = max(m, h);
      }
    }
    m = __reduce_max_sync(~0u, m);
  }
  if constexpr (W > 1) {
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < W; ++k) m = max(m, s_max[warp / W * W + k]);
  }
  if (!active || !there) return;

  const uint32_t bits = __float_as_uint(Elem<E>::unpack(m).x);
  const int need = max((int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0), 0);
  const bool bad = was == 255u;
  if (bad && lane == 0 && a.status) atomicOr(a.status, FT_ST_NAN);
  const int e = bad ? need : max((int)was, need);
  const int64_t page_stride = values ? a.cache.v_page_stride : a.cache.k_page_stride;
  const int64_t token_stride = values ? a.cache.v_token_stride : a.cache.k_token_stride;
  uint8_t* dst = static_cast<uint8_t*>(values ? a.cache.v : a.cache.k) + page * page_stride +
                 in_page * token_stride + head * (values ? a.cache.v_head_stride : a.cache.k_head_stride) + e0;
  if (lo > 0 && (bad || e != (int)was)) {  // the tokens already there
    const float f = bad ? __uint_as_float(0x7FC00000u) : exp2i((int)was - e);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int row = row0 + i * RPS;
      if (row >= lo) continue;
      uint2* p = reinterpret_cast<uint2*>(dst + row * token_stride);
      const uint2 c = *p;
      const uint32_t w[2] = {c.x, c.y};
      uint32_t o[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 u = Elem<__half>::unpack(e4m3x2_to_f16x2(w[k] & 0xFFFFu));
        const float2 v = Elem<__half>::unpack(e4m3x2_to_f16x2(w[k] >> 16));
        o[k] = to_e4m3x4(u.x * f, u.y * f, v.x * f, v.y * f);
      }
      *p = make_uint2(o[0], o[1]);
    }
  }
  if (lane == 0 && warp % W == 0) *scale = (uint8_t)e;
  const float f = exp2i(127 - e);
  const bool plain = e < kCapByte<E> && !odd;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int row = row0 + i * RPS;
    if (row < lo || row >= hi) continue;
    uint2* to = reinterpret_cast<uint2*>(dst + row * token_stride);
    const float2 a0 = Elem<E>::unpack(x[i].x), a1 = Elem<E>::unpack(x[i].y), a2 = Elem<E>::unpack(x[i].z), a3 = Elem<E>::unpack(x[i].w);
    *to = make_uint2(to_e4m3x4(a0.x * f, a0.y * f, a1.x * f, a1.y * f), to_e4m3x4(a2.x * f, a2.y * f, a3.x * f, a3.y * f));
  }
  if (plain) return;
  // Once more for what the conversion does not do: no code past the type's range, NaN for what is not finite.
  const float cap = e >= kCapByte<E> ? 240.f : 448.f;
#pragma unroll 1
  for (int z = 0; z < kSteps * 8; ++z) {
    const int row = row0 + z / 8 * RPS;
    if (row < lo || row >= hi) continue;
    const float v = Elem<E>::unpack(static_cast<const uint16_t*>(values ? a.v : a.k)[(r.q0 + (block0 - r.ctx) + row) *
                                        (values ? a.v_stride : a.k_stride) + (int64_t)head * D + e0 + z % 8]).x;
    const float y = v - v == 0.f ? fminf(fmaxf(v * f, -cap), cap) : __uint_as_float(0x7FC00000u);
    dst[row * token_stride + z % 8] = (uint8_t)to_e4m3x4(y, 0.f, 0.f, 0.f);
  }
}

template <typename E, int D>
cudaError_t launch_store(const StoreArgs& g, cudaStream_t st) {
  const ft_kv8_store_args& a = g.a;
  // A request's new rows reach one block more than they fill at either end.
  const int64_t units = std::min<int64_t>(a.max_tokens, a.max_tokens / a.cache.block_size + 2 * (int64_t)a.num_reqs);
  const int W = std::max(1, a.cache.block_size * D / (32 * 8 * kSteps));
  const int subs = 2 * a.cache.kv_heads, per = kWarps / W;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(cfg, attr, dim3((unsigned)units, (unsigned)((subs + per - 1) / per)), dim3(kThreads), 0, st);
  switch (W) {
    case 1: return cudaLaunchKernelEx(&cfg, kv8_store_kernel<E, D, 1>, g);
    case 2: return cudaLaunchKernelEx(&cfg, kv8_store_kernel<E, D, 2>, g);
    case 4: return cudaLaunchKernelEx(&cfg, kv8_store_kernel<E, D, 4>, g);
    default: return cudaLaunchKernelEx(&cfg, kv8_store_kernel<E, D, 8>, g);
  }
}

struct LoadArgs {
  ft_kv8_load_args a;
  int log2_page, log2_block, log2_lanes;  // lanes: pieces of 16 codes of a head
  int64_t num_slots;
  uint32_t pieces;  // of a row: keys, then values
};

constexpr int kItems = 4;

// A thread takes one piece (16 codes of a head) of kItems rows, kRowStep rows apart.
template <typename E>
__global__ void __launch_bounds__(kThreads) kv8_load_kernel(const __grid_constant__ LoadArgs g) {
  const ft_kv8_load_args& a = g.a;
  pdl_wait();
  pdl_trigger();
  const uint32_t id = blockIdx.x * kThreads + threadIdx.x, group = id / g.pieces, piece = id - group * g.pieces;
  const int64_t t0 = (int64_t)group * kItems;
  const uint32_t half = g.pieces >> 1;
  const bool values = piece >= half;
  const uint32_t p = values ? piece - half : piece, head = p >> g.log2_lanes, at = (p & ((1u << g.log2_lanes) - 1)) * 16;
  const uint8_t* codes = static_cast<const uint8_t*>(values ? a.cache.v : a.cache.k) +
                         head * (values ? a.cache.v_head_stride : a.cache.k_head_stride) + at;
  const uint8_t* scales = values ? a.cache.v_scale : a.cache.k_scale;
  const int64_t page_stride = values ? a.cache.v_page_stride : a.cache.k_page_stride;
  const int64_t token_stride = values ? a.cache.v_token_stride : a.cache.k_token_stride;
  int64_t slot[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) slot[i] = t0 + i < a.T ? a.slots[t0 + i] : -1;
  uint4 c[kItems];
  uint32_t e[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (slot[i] >= g.num_slots) {
      if (a.status && piece == 0) atomicOr(a.status, FT_ST_BAD_SLOT);
      slot[i] = -1;
    }
    c[i] = make_uint4(0, 0, 0, 0);
    e[i] = 0;
    if (slot[i] >= 0) {
      const int64_t page = slot[i] >> g.log2_page, row = slot[i] & ((1 << g.log2_page) - 1);
      c[i] = *reinterpret_cast<const uint4*>(codes + page * page_stride + row * token_stride);
      e[i] = scales[((page << (g.log2_page - g.log2_block)) + (row >> g.log2_block)) * a.cache.kv_heads + head];
    }
  }
  uint16_t* out = static_cast<uint16_t*>(values ? a.v : a.k) + (int64_t)head * (16 << g.log2_lanes) + at;
  const int64_t stride = values ? a.v_stride : a.k_stride;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (t0 + i >= a.T) break;
    const float f = scale_of(e[i]);
    const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 y = Elem<__half>::unpack(e4m3x2_to_f16x2(k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xFFFFu));
      o[k] = Elem<E>::pack(y.x * f, y.y * f);
    }
    uint4* dst = reinterpret_cast<uint4*>(out + (t0 + i) * stride);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

int check_rows(const void* k, const void* v, int64_t k_stride, int64_t v_stride, int dtype) {
  if (dtype != FT_DTYPE_BF16 && dtype != FT_DTYPE_F16)
    return record_error(FT_E_ARG, "dtype must be FT_DTYPE_BF16 or FT_DTYPE_F16");
  if (!k || !v) return record_error(FT_E_ARG, "null pointer");
  if (!is_16b(k) || !is_16b(v) || k_stride < 0 || v_stride < 0 || k_stride % 8 || v_stride % 8 ||
      k_stride >= (int64_t(1) << 38) || v_stride >= (int64_t(1) << 38))
    return record_error(FT_E_ARG, "k and v must be 16-byte aligned, row strides multiples of 8 elements below 2^38");
  return FT_OK;
}

}  // namespace
}  // namespace ft

extern "C" int ft_kv8_store(const ft_kv8_store_args* args, void* stream) {
  using namespace ft;
  if (!args) return record_error(FT_E_ARG, "null args");
  const ft_kv8_store_args& a = *args;
  if (int rc = check_kv8_cache(a.cache)) return rc;
  if (a.max_tokens < 0 || a.num_reqs < 0 || a.table_width < 0)
    return record_error(FT_E_ARG, "max_tokens, num_reqs and table_width must not be negative");
  if (int rc = check_rows(a.k, a.v, a.k_stride, a.v_stride, a.dtype)) return rc;
  if (!a.q_start || !a.ctx_len || !a.block_table) return record_error(FT_E_ARG, "null pointer");
  if (a.max_tokens == 0 || a.num_reqs == 0) return FT_OK;
  if (a.table_width < 1) return record_error(FT_E_ARG, "table_width must be positive");
  StoreArgs g{};
  g.a = a;
  g.log2_page = log2_of(a.cache.page_size);
  g.log2_block = log2_of(a.cache.block_size);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool wide = a.cache.head_dim == 128;
  const cudaError_t e =
      a.dtype == FT_DTYPE_BF16
          ? (wide ? launch_store<__nv_bfloat16, 128>(g, st) : launch_store<__nv_bfloat16, 64>(g, st))
          : (wide ? launch_store<__half, 128>(g, st) : launch_store<__half, 64>(g, st));
  if (e != cudaSuccess) return record_error(FT_E_CUDA, "cache store launch failed: %s", cudaGetErrorString(e));
  return FT_OK;
}

extern "C" int ft_kv8_load(const ft_kv8_load_args* args, void* stream) {
  using namespace ft;
  if (!args) return record_error(FT_E_ARG, "null args");
  const ft_kv8_load_args& a = *args;
  if (int rc = check_kv8_cache(a.cache)) return rc;
  if (a.T < 0) return record_error(FT_E_ARG, "T must not be negative");
  if (int rc = check_rows(a.k, a.v, a.k_stride, a.v_stride, a.dtype)) return rc;
  if (!a.slots) return record_error(FT_E_ARG, "null pointer");
  if (a.T == 0) return FT_OK;
  const int64_t row = (int64_t)a.cache.kv_heads * a.cache.head_dim;
  if (a.T > 1 && (a.k_stride < row || a.v_stride < row))
    return record_error(FT_E_ARG, "rows of k and v must not overlap");
  LoadArgs g{};
  g.a = a;
  g.log2_page = log2_of(a.cache.page_size);
  g.log2_block = log2_of(a.cache.block_size);
  g.log2_lanes = log2_of(a.cache.head_dim / 16);
  g.num_slots = (int64_t)a.cache.num_pages * a.cache.page_size;
  g.pieces = 2u * (unsigned)a.cache.kv_heads << g.log2_lanes;
  const int64_t threads = ((int64_t)a.T + kItems - 1) / kItems * g.pieces;
  if (threads > 0xFFFFFF00ll) return record_error(FT_E_UNSUPPORTED, "T times the heads is too large for one call");
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(cfg, attr, dim3((unsigned)((threads + kThreads - 1) / kThreads)), dim3(kThreads), 0,
             static_cast<cudaStream_t>(stream));
  const cudaError_t e = a.dtype == FT_DTYPE_BF16 ? cudaLaunchKernelEx(&cfg, kv8_load_kernel<__nv_bfloat16>, g)
                                                 : cudaLaunchKernelEx(&cfg, kv8_load_kernel<__half>, g);
  if (e != cudaSuccess) return record_error(FT_E_CUDA, "cache load launch failed: %s", cudaGetErrorString(e));
  return FT_OK;
}
