// Attention over a 16-bit paged cache (ft_tree_attention): checks of its
// arguments and the launch; the kernels are in tree_attention.cuh.
#include "tree_attention.cuh"

namespace ft {
namespace {

int check(const ft_attn_args& a) {
  if (int rc = check_kv_cache(a.cache, false)) return rc;
  return tree_attention::check_sizes(a);
}

}  // namespace
}  // namespace ft

extern "C" int ft_tree_attention_workspace(const ft_attn_args* args, uint64_t* bytes) {
  using namespace ft;
  if (!args || !bytes) return record_error(FT_E_ARG, "null pointer");
  if (int rc = check(*args)) return rc;
  *bytes = tree_attention::workspace(sm_count(), args->cache.head_dim);
  return FT_OK;
}

extern "C" int ft_tree_attention(const ft_attn_args* args, void* stream) {
  using namespace ft;
  using namespace ft::tree_attention;
  if (!args) return record_error(FT_E_ARG, "null args");
  const ft_attn_args& a = *args;
  if (int rc = check(a)) return rc;
  if (a.max_tokens == 0 || a.num_reqs == 0) return FT_OK;
  const int grid = sm_count(), D = a.cache.head_dim;
  if (int rc = check_rest(a, workspace(grid, D))) return rc;
  const Args g = make_args(a, grid);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.cache.dtype == FT_DTYPE_BF16)
    return D == 128 ? launch<__nv_bfloat16, 128, false>(g, grid, st) : launch<__nv_bfloat16, 64, false>(g, grid, st);
  return D == 128 ? launch<__half, 128, false>(g, grid, st) : launch<__half, 64, false>(g, grid, st);
}
