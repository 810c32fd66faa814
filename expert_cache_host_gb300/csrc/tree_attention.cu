// Attention of a step's tokens over the paged cache (ft_tree_attention).
//
// One warp per (row, query head): 32 keys at a time, a lane per key for the
// scores, a lane per D/32 outputs for the second product, with the running
// maximum and sum of a softmax.
#include <math_constants.h>

#include "attn_side.h"

namespace ft {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <typename E, int D>
__global__ void __launch_bounds__(kWarps * 32) tree_attention_kernel(const ft_attn_args a, int log2_page) {
  __shared__ float sq[kWarps][D];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + w;
  const int t = (int)(unit / a.q_heads), h = (int)(unit % a.q_heads);
  if (t >= a.max_tokens || t >= a.q_start[a.num_reqs]) return;
  int lo = 0, hi = a.num_reqs;  // the last request that starts at or before t and has rows
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.q_start[mid] <= t) lo = mid; else hi = mid;
  }
  const int b = lo, i = t - a.q_start[b], ctx = a.ctx_len[b];
  const int n = a.q_start[b + 1] - a.q_start[b];
  const int kh = h / (a.q_heads / a.cache.kv_heads), P = 1 << log2_page;
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + t * a.q_stride + (int64_t)h * D;
  for (int d = lane; d < D; d += 32) sq[w][d] = Elem<E>::unpack(q[d]).x;
  __syncwarp();
  const int per = D / 32;
  float m = -CUDART_INF_F, sum = 0.f, acc[per];
  for (int x = 0; x < per; ++x) acc[x] = 0.f;
  for (int k0 = 0; k0 < ctx + n; k0 += 32) {
    const int k = k0 + lane;
    bool seen = k < ctx + n && (k >> log2_page) < a.table_width;
    if (seen && k >= ctx) {
      const int j = k - ctx;
      seen = a.mask ? (j < 32 * a.mask_words && (a.mask[(int64_t)t * a.mask_words + (j >> 5)] >> (j & 31) & 1)) : j <= i;
    }
    int page = -1;
    if (seen) page = a.block_table[(int64_t)b * a.table_width + (k >> log2_page)];
    if (seen && (page < 0 || page >= a.cache.num_pages)) {
      if (a.status) atomicOr(a.status, FT_ST_BAD_SLOT);
      seen = false;
    }
    float s = -CUDART_INF_F;
    if (seen) {
      const uint4* row = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.cache.k) + page * a.cache.k_page_stride +
                                                        (k & (P - 1)) * a.cache.k_token_stride + kh * a.cache.k_head_stride);
      s = 0.f;
      for (int v = 0; v < D / 8; ++v) {
        const uint4 r = row[v];
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
        for (int e = 0; e < 4; ++e) {
          const float2 f = Elem<E>::unpack(u[e]);
          s += f.x * sq[w][v * 8 + 2 * e] + f.y * sq[w][v * 8 + 2 * e + 1];
        }
      }
      s *= a.scale;
    }
    float mx = s;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
    const float mn = fmaxf(m, mx);
    if (mn == -CUDART_INF_F) continue;
    const float keep = exp2f((m - mn) * kLog2e), p = exp2f((s - mn) * kLog2e);
    float ps = p;
    for (int o = 16; o > 0; o >>= 1) ps += __shfl_xor_sync(~0u, ps, o);
    sum = sum * keep + ps;
    m = mn;
    for (int x = 0; x < per; ++x) acc[x] *= keep;
    const unsigned live = __ballot_sync(~0u, seen);
    for (int c = 0; c < 32; ++c) {
      if (!(live >> c & 1)) continue;
      const float pc = __shfl_sync(~0u, p, c);
      const int pg = __shfl_sync(~0u, page, c), kk = k0 + c;
      const uint16_t* row = static_cast<const uint16_t*>(a.cache.v) + pg * a.cache.v_page_stride +
                            (kk & (P - 1)) * a.cache.v_token_stride + kh * a.cache.v_head_stride;
      for (int x = 0; x < per; ++x) acc[x] += pc * Elem<E>::unpack(row[x * 32 + lane]).x;
    }
  }
  uint16_t* o = static_cast<uint16_t*>(a.out) + t * a.out_stride + (int64_t)h * D;
  for (int x = 0; x < per; ++x) o[x * 32 + lane] = (uint16_t)Elem<E>::pack(sum > 0.f ? acc[x] / sum : 0.f, 0.f);
  if (a.lse && lane == 0) a.lse[(int64_t)t * a.q_heads + h] = m + logf(sum);
}

int check(const ft_attn_args& a) {
  if (int rc = check_kv_cache(a.cache, false)) return rc;
  if (a.max_tokens < 0 || a.num_reqs < 0 || a.q_heads < 1 || a.table_width < 0 || a.mask_words < 0)
    return record_error(FT_E_ARG, "max_tokens, num_reqs, table_width and mask_words must not be negative, q_heads positive");
  if (a.q_heads % a.cache.kv_heads) return record_error(FT_E_ARG, "q_heads must be a multiple of kv_heads");
  if (a.q_heads / a.cache.kv_heads > 128) return record_error(FT_E_UNSUPPORTED, "more than 128 query heads to a key head");
  return FT_OK;
}

}  // namespace
}  // namespace ft

extern "C" int ft_tree_attention_workspace(const ft_attn_args* args, uint64_t* bytes) {
  using namespace ft;
  if (!args || !bytes) return record_error(FT_E_ARG, "null pointer");
  if (int rc = check(*args)) return rc;
  *bytes = 16;
  return FT_OK;
}

extern "C" int ft_tree_attention(const ft_attn_args* args, void* stream) {
  using namespace ft;
  if (!args) return record_error(FT_E_ARG, "null args");
  const ft_attn_args& a = *args;
  if (int rc = check(a)) return rc;
  if (a.max_tokens == 0 || a.num_reqs == 0) return FT_OK;
  if (!a.q || !a.out || !a.q_start || !a.ctx_len || !a.block_table || !a.workspace)
    return record_error(FT_E_ARG, "null pointer");
  if (a.table_width < 1) return record_error(FT_E_ARG, "table_width must be positive");
  if (a.mask ? a.mask_words < 1 : a.mask_words != 0)
    return record_error(FT_E_ARG, "a mask needs mask_words >= 1; without one mask_words must be 0");
  if (!is_16b(a.q) || !is_16b(a.out) || !is_16b(a.workspace) || a.q_stride < 0 || a.out_stride < 0 || a.q_stride % 8 ||
      a.out_stride % 8)
    return record_error(FT_E_ARG, "q, out and workspace must be 16-byte aligned, row strides multiples of 8 elements");
  if (!(a.scale - a.scale == 0.f)) return record_error(FT_E_ARG, "scale must be finite");
  uint64_t need = 0;
  if (int rc = ft_tree_attention_workspace(args, &need)) return rc;
  if (a.workspace_bytes < need)
    return record_error(FT_E_ARG, "workspace of %llu bytes, %llu needed", (unsigned long long)a.workspace_bytes,
                        (unsigned long long)need);
  int log2_page = 0;
  while ((1 << log2_page) < a.cache.page_size) ++log2_page;
  const int64_t grid = ((int64_t)a.max_tokens * a.q_heads + kWarps - 1) / kWarps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = a.cache.dtype == FT_DTYPE_BF16;
  if (a.cache.head_dim == 128) {
    if (bf) tree_attention_kernel<__nv_bfloat16, 128><<<(unsigned)grid, kWarps * 32, 0, st>>>(a, log2_page);
    else tree_attention_kernel<__half, 128><<<(unsigned)grid, kWarps * 32, 0, st>>>(a, log2_page);
  } else {
    if (bf) tree_attention_kernel<__nv_bfloat16, 64><<<(unsigned)grid, kWarps * 32, 0, st>>>(a, log2_page);
    else tree_attention_kernel<__half, 64><<<(unsigned)grid, kWarps * 32, 0, st>>>(a, log2_page);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return record_error(FT_E_CUDA, "attention launch failed: %s", cudaGetErrorString(e));
  return FT_OK;
}
