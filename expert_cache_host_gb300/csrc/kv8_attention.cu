// Attention over the 8-bit paged cache (ft_kv8_attention): checks of its
// arguments and the launch; the kernels are in kv8_few.cuh (few rows) and
// tree_attention.cuh.
#include "kv8_few.cuh"

namespace ft {
namespace {

// The call as one over a 16-bit cache of the rows' type, with strides in bytes.
ft_attn_args as_attn(const ft_kv8_attn_args& a) {
  const ft_kv8_cache& c = a.cache;
  ft_attn_args t{};
  t.q = a.q, t.out = a.out, t.lse = a.lse, t.q_start = a.q_start, t.ctx_len = a.ctx_len, t.block_table = a.block_table;
  t.mask = a.mask, t.workspace = a.workspace, t.status = a.status, t.q_stride = a.q_stride, t.out_stride = a.out_stride;
  t.workspace_bytes = a.workspace_bytes, t.max_tokens = a.max_tokens, t.num_reqs = a.num_reqs, t.q_heads = a.q_heads;
  t.table_width = a.table_width, t.mask_words = a.mask_words, t.scale = a.scale;
  t.cache.k = c.k, t.cache.v = c.v, t.cache.dtype = a.dtype, t.cache.num_pages = c.num_pages;
  t.cache.page_size = c.page_size, t.cache.kv_heads = c.kv_heads, t.cache.head_dim = c.head_dim;
  t.cache.k_page_stride = c.k_page_stride, t.cache.k_token_stride = c.k_token_stride, t.cache.k_head_stride = c.k_head_stride;
  t.cache.v_page_stride = c.v_page_stride, t.cache.v_token_stride = c.v_token_stride, t.cache.v_head_stride = c.v_head_stride;
  return t;
}

int check(const ft_kv8_attn_args& a) {
  if (int rc = check_kv8_cache(a.cache)) return rc;
  if (a.dtype != FT_DTYPE_BF16 && a.dtype != FT_DTYPE_F16)
    return record_error(FT_E_ARG, "dtype must be FT_DTYPE_BF16 or FT_DTYPE_F16");
  if (a.max_new < 0) return record_error(FT_E_ARG, "max_new must not be negative");
  return tree_attention::check_sizes(as_attn(a));
}

template <typename E>
int launch_few(const tree_attention::Args& g, int grid, int64_t rows, cudaStream_t st) {
  if (g.a.cache.head_dim == 128)
    return rows <= 8 ? kv8_few::launch<E, 128, 1>(g, grid, st) : kv8_few::launch<E, 128, 2>(g, grid, st);
  return rows <= 8 ? kv8_few::launch<E, 64, 1>(g, grid, st) : kv8_few::launch<E, 64, 2>(g, grid, st);
}

}  // namespace
}  // namespace ft

extern "C" int ft_kv8_attention_workspace(const ft_kv8_attn_args* args, uint64_t* bytes) {
  using namespace ft;
  if (!args || !bytes) return record_error(FT_E_ARG, "null pointer");
  if (int rc = check(*args)) return rc;
  *bytes = tree_attention::workspace(sm_count(), args->cache.head_dim);
  return FT_OK;
}

extern "C" int ft_kv8_attention(const ft_kv8_attn_args* args, void* stream) {
  using namespace ft;
  using namespace ft::tree_attention;
  if (!args) return record_error(FT_E_ARG, "null args");
  if (int rc = check(*args)) return rc;
  const ft_attn_args a = as_attn(*args);
  if (a.max_tokens == 0 || a.num_reqs == 0) return FT_OK;
  const int grid = sm_count(), D = a.cache.head_dim;
  if (int rc = check_rest(a, workspace(grid, D))) return rc;
  const int max_new = args->max_new ? std::min(args->max_new, a.max_tokens) : a.max_tokens;
  // Few rows: a kernel whose products take 8 or 16, on two CTAs or one an SM.
  const int64_t rows = (int64_t)max_new * (a.q_heads / a.cache.kv_heads);
  const int few = rows > 16 ? 0 : rows <= 8 || D == 64 ? 2 * grid : grid;
  Args g = few ? make_args(a, few, kv8_few::kRows) : make_args(a, grid);
  g.k_scale = args->cache.k_scale;
  g.v_scale = args->cache.v_scale;
  g.log2_block = log2_of(args->cache.block_size);
  g.max_new = max_new;
  g.sixteen = 16;
  g.one = 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (few) return args->dtype == FT_DTYPE_BF16 ? launch_few<__nv_bfloat16>(g, few, rows, st) : launch_few<__half>(g, few, rows, st);
  if (args->dtype == FT_DTYPE_BF16)
    return D == 128 ? launch<__nv_bfloat16, 128, true>(g, grid, st) : launch<__nv_bfloat16, 64, true>(g, grid, st);
  return D == 128 ? launch<__half, 128, true>(g, grid, st) : launch<__half, 64, true>(g, grid, st);
}
