// Attention of a step's tokens over the 8-bit paged cache (ft_kv8_attention).
//
// A block per row and query head; its warps take the request's keys in turn, a
// lane D/32 numbers of each, with the running maximum m and sum l of the softmax,
// and are joined at the end: the plain form of the kernel.
#include <math_constants.h>

#include "kv8.h"
#include "tma.h"

namespace ft {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

struct Args {
  ft_kv8_attn_args a;
  int log2_page, log2_block, max_new;
};

template <typename E, int D>
__global__ void __launch_bounds__(kThreads) kv8_attention_kernel(const __grid_constant__ Args g) {
  constexpr int N = D / 32;
  const ft_kv8_attn_args& a = g.a;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int lo = 0, hi = a.num_reqs;  // the last request that begins at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.q_start[mid] <= t) lo = mid; else hi = mid;
  }
  const int b = lo, q0 = a.q_start[b];
  if (q0 < 0 || t < q0) return;
  const int n = max(min(a.q_start[b + 1], a.max_tokens) - q0, 0), i = t - q0;
  if (i >= n) return;
  const int ctx = max(a.ctx_len[b], 0);
  const uint32_t keys = (uint32_t)ctx + n;
  if (n > g.max_new || keys > 0x7FFFFFFFu - 256) {
    if (a.status && tid == 0) atomicOr(a.status, n > g.max_new ? FT_ST_NO_ROOM : FT_ST_BAD_SLOT);
    return;
  }
  const int head = h / (a.q_heads / a.cache.kv_heads);
  float q[N], o[N];
  const uint16_t* qr = static_cast<const uint16_t*>(a.q) + t * a.q_stride + (int64_t)h * D + lane * N;
#pragma unroll
  for (int k = 0; k < N; ++k) q[k] = Elem<E>::unpack(qr[k]).x, o[k] = 0.f;
  auto number = [&](const uint8_t* p, float f) {  // rounded to the rows' type
    return Elem<E>::unpack(Elem<E>::pack(Elem<__half>::unpack(e4m3x2_to_f16x2(*p)).x * f, 0.f)).x;
  };
  float m = -CUDART_INF_F, l = 0.f;
  for (uint32_t key = warp; key < keys; key += kWarps) {
    if (key >= (uint32_t)ctx) {
      const int j = (int)(key - ctx);
      if (a.mask ? (j >> 5) >= a.mask_words || !(a.mask[(int64_t)t * a.mask_words + (j >> 5)] >> (j & 31) & 1) : j > i) continue;
    }
    const int col = (int)(key >> g.log2_page), row = (int)(key & ((1u << g.log2_page) - 1));
    const int page = col < a.table_width ? a.block_table[(int64_t)b * a.table_width + col] : -1;
    if (page < 0 || page >= a.cache.num_pages) {
      if (a.status && lane == 0) atomicOr(a.status, FT_ST_BAD_SLOT);
      continue;
    }
    const int64_t at = (((int64_t)page << (g.log2_page - g.log2_block)) + (row >> g.log2_block)) * a.cache.kv_heads + head;
    const uint8_t* k = static_cast<const uint8_t*>(a.cache.k) + page * a.cache.k_page_stride + row * a.cache.k_token_stride +
                       head * a.cache.k_head_stride + lane * N;
    const uint8_t* v = static_cast<const uint8_t*>(a.cache.v) + page * a.cache.v_page_stride + row * a.cache.v_token_stride +
                       head * a.cache.v_head_stride + lane * N;
    const float fk = scale_of(a.cache.k_scale[at]), fv = scale_of(a.cache.v_scale[at]);
    float s = 0.f;
#pragma unroll
    for (int z = 0; z < N; ++z) s += q[z] * number(k + z, fk);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    s *= a.scale;
    const float top = fmaxf(m, s), f = m == -CUDART_INF_F ? 0.f : expf(m - top), p = top == -CUDART_INF_F ? 0.f : expf(s - top);
    l = l * f + p;
#pragma unroll
    for (int z = 0; z < N; ++z) o[z] = o[z] * f + p * number(v + z, fv);
    m = top;
  }
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
  for (int z = 0; z < N; ++z) s_o[warp][lane * N + z] = o[z];
  __syncthreads();
  float most = -CUDART_INF_F, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) most = fmaxf(most, s_m[w]);
  if (tid < D) {
    float y = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float f = s_m[w] == -CUDART_INF_F ? 0.f : expf(s_m[w] - most);
      if (f != 0.f) sum += f * s_l[w], y += f * s_o[w][tid];  // (NaN: a seen score was NaN or +inf)
    }
    static_cast<uint16_t*>(a.out)[t * a.out_stride + (int64_t)h * D + tid] = (uint16_t)Elem<E>::pack(sum == 0.f ? 0.f : y / sum, 0.f);
    if (a.lse && tid == 0) a.lse[(int64_t)t * a.q_heads + h] = sum == 0.f ? -CUDART_INF_F : most + logf(sum);
  }
}

int check(const ft_kv8_attn_args& a) {
  if (int rc = check_kv8_cache(a.cache)) return rc;
  if (a.dtype != FT_DTYPE_BF16 && a.dtype != FT_DTYPE_F16)
    return record_error(FT_E_ARG, "dtype must be FT_DTYPE_BF16 or FT_DTYPE_F16");
  if (a.max_tokens < 0 || a.max_new < 0 || a.num_reqs < 0 || a.q_heads < 1 || a.table_width < 0 || a.mask_words < 0)
    return record_error(FT_E_ARG,
                        "max_tokens, max_new, num_reqs, table_width and mask_words must not be negative, q_heads positive");
  if (a.q_heads % a.cache.kv_heads) return record_error(FT_E_ARG, "q_heads must be a multiple of kv_heads");
  if (a.q_heads / a.cache.kv_heads > 128) return record_error(FT_E_UNSUPPORTED, "more than 128 query heads to a key head");
  return FT_OK;
}

uint64_t workspace(int grid, int D) { return (uint64_t)grid * 2 * 256 * D * 4; }

}  // namespace
}  // namespace ft

extern "C" int ft_kv8_attention_workspace(const ft_kv8_attn_args* args, uint64_t* bytes) {
  using namespace ft;
  if (!args || !bytes) return record_error(FT_E_ARG, "null pointer");
  if (int rc = check(*args)) return rc;
  *bytes = workspace(sm_count(), args->cache.head_dim);
  return FT_OK;
}

extern "C" int ft_kv8_attention(const ft_kv8_attn_args* args, void* stream) {
  using namespace ft;
  if (!args) return record_error(FT_E_ARG, "null args");
  const ft_kv8_attn_args& a = *args;
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
  if (!(fabsf(a.scale) < 1e37f)) return record_error(FT_E_ARG, "scale must be finite (below 1e37)");
  const int D = a.cache.head_dim;
  const uint64_t need = workspace(sm_count(), D);
  if (a.workspace_bytes < need)
    return record_error(FT_E_ARG, "workspace of %llu bytes, %llu needed", (unsigned long long)a.workspace_bytes,
                        (unsigned long long)need);
  Args g{};
  g.a = a;
  g.log2_page = log2_of(a.cache.page_size);
  g.log2_block = log2_of(a.cache.block_size);
  g.max_new = a.max_new ? a.max_new : a.max_tokens;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(cfg, attr, dim3((unsigned)a.max_tokens, (unsigned)a.q_heads), dim3(kThreads), 0, static_cast<cudaStream_t>(stream));
  cudaError_t e;
  if (a.dtype == FT_DTYPE_BF16)
    e = D == 128 ? cudaLaunchKernelEx(&cfg, kv8_attention_kernel<__nv_bfloat16, 128>, g)
                 : cudaLaunchKernelEx(&cfg, kv8_attention_kernel<__nv_bfloat16, 64>, g);
  else
    e = D == 128 ? cudaLaunchKernelEx(&cfg, kv8_attention_kernel<__half, 128>, g)
                 : cudaLaunchKernelEx(&cfg, kv8_attention_kernel<__half, 64>, g);
  if (e != cudaSuccess) return record_error(FT_E_CUDA, "attention launch failed: %s", cudaGetErrorString(e));
  return FT_OK;
}
