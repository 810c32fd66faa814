// Block tables, slots, positions and ancestor masks of a step from the
// requests' lengths, in one launch (ft_kv_plan).
//
// With n_b the new tokens of request b, everything a row needs is its request
// (the last b with q_start[b] = sum_{b' < b} n_b' at or before the row) and how
// many fresh pages the requests before it take,
// sum_{b' < b} ceil((ctx+n)/P) - ceil(ctx/P), columns of the table only.  A page is fresh exactly when the
// step writes its first row, so the row with (ctx + i) % P == 0 fills the
// block-table column and no row waits for another's write.
//
// The bytes are few (a row's 12 plus its mask); what bounds it is latency: one
// launch, one load of the lengths, one block-wide scan, then the parents'
// chain.  So every CTA (256 rows) scans the requests itself, up to the last
// one it needs, instead of reading another launch's sums: requests are a few
// thousand at most and their lengths stay in L2.  64 requests with a token each
// take 2.6 us, 256 with 4400 drafted tokens 4.3 us (graph replay).
#include "attn_side.h"
#include "tma.h"

namespace ft {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;  // requests a thread scans at a time
constexpr int kBehind = kThreads;  // rows before the CTA's whose parents it keeps at hand: a tree that began there

// Exclusive sum over the block of each thread's v; `total` is the block's sum.
template <typename T>
__device__ __forceinline__ T block_exclusive(T v, T* sh, T& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[w] = x;
  __syncthreads();
  T before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    const T s = sh[i];
    if (i < w) before += s;
    all += s;
  }
  __syncthreads();
  total = all;
  return before + x - v;
}

__global__ void __launch_bounds__(kThreads) kv_plan_kernel(const ft_plan_args a, int log2_page) {
  __shared__ int sh[kThreads / 32];
  __shared__ long long shl[kThreads / 32];
  __shared__ int rec_start[kThreads], rec_req[kThreads], rec_ctx[kThreads], rec_page[kThreads], rec_n[kThreads];
  __shared__ int s_parent[kBehind + kThreads];  // of the rows from t0 - kBehind on
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int P = 1 << log2_page;
  const int t0 = blockIdx.x * kThreads, t = t0 + tid;
  const bool first = blockIdx.x == 0;  // this CTA also writes q_start and free_left
  uint32_t fault = 0;

  rec_req[tid] = -1;
  pdl_wait();
  pdl_trigger();
  if (a.parents) {
    static_assert(kBehind == kThreads, "a row in the window and one behind it per thread");
    s_parent[tid] = t >= kBehind ? a.parents[t - kBehind] : -1;  // (t - kBehind < t0, so it is a row)
    s_parent[kBehind + tid] = t < a.max_tokens ? a.parents[t] : -1;
  }
  const int free_count = *a.free_count;
  __syncthreads();

  long long tok = 0;  // sums over the requests of earlier rounds of the scan
  int page = 0;
  for (int b0 = 0; b0 < a.num_reqs; b0 += kThreads * kPer) {
    int ctx[kPer], n[kPer], fresh[kPer];
    long long start[kPer], sum = 0, total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = b0 + tid * kPer + i;
      ctx[i] = b < a.num_reqs ? a.ctx_len[b] : 0;
      n[i] = b < a.num_reqs ? a.new_len[b] : 0;
      if (ctx[i] < 0 || n[i] < 0 || (long long)ctx[i] + n[i] > 0x7FFFFFFFll - P) {
        fault |= FT_ST_NO_ROOM;
        ctx[i] = 0;
        n[i] = 0;
      }
      sum += n[i];
    }
    start[0] = tok + block_exclusive(sum, shl, total);
    int psum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i + 1 < kPer) start[i + 1] = start[i] + n[i];
      if (start[i] + n[i] > a.max_tokens) {  // cut: the rows have run out
        fault |= FT_ST_NO_ROOM;
        start[i] = min(start[i], (long long)a.max_tokens);
        n[i] = a.max_tokens - (int)start[i];
      }
      // (a column past the table takes no page: nothing would hold its id)
      fresh[i] = min((ctx[i] + n[i] + P - 1) >> log2_page, a.table_width) -
                 min((ctx[i] + P - 1) >> log2_page, a.table_width);
      psum += fresh[i];
    }
    int ptotal;
    int pb = page + block_exclusive(psum, sh, ptotal);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = b0 + tid * kPer + i;
      if (b < a.num_reqs) {
        const int s0 = (int)start[i];
        if (first) a.q_start[b] = s0;
        if (n[i] > 0 && s0 < t0 + kThreads && s0 + n[i] > t0) {
          const int at = max(s0 - t0, 0);
          rec_req[at] = b;
          rec_start[at] = s0;
          rec_ctx[at] = ctx[i];
          rec_page[at] = pb;
          rec_n[at] = n[i];
        }
      }
      pb += fresh[i];
    }
    tok += total;
    page += ptotal;
    if (!first && tok >= t0 + kThreads) break;  // every request of this CTA's rows is known
  }
  if (first && tid == 0) {
    a.q_start[a.num_reqs] = (int)min(tok, (long long)a.max_tokens);
    *a.free_left = max(free_count - page, 0);
  }
  __syncthreads();
  // Each row's request: the nearest record at or before it.
  int rec = rec_req[tid] >= 0 ? tid : -1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int r = __shfl_up_sync(~0u, rec, o);
    if (lane >= o) rec = max(rec, r);
  }
  if (lane == 31) sh[w] = rec;
  __syncthreads();
  for (int i = 0; i < w; ++i) rec = max(rec, sh[i]);
  if (t >= a.max_tokens) {
    // a row past the last: nothing to write
  } else if (rec < 0 || t >= rec_start[rec] + rec_n[rec]) {  // padding
    a.slots[t] = -1;
    a.positions[t] = 0;
    for (int i = 0; i < a.mask_words; ++i) a.mask[(size_t)t * a.mask_words + i] = 0;
  } else {
    const int b = rec_req[rec], start = rec_start[rec], ctx = rec_ctx[rec];
    const int i = t - start, at = ctx + i, col = at >> log2_page, held = (ctx + P - 1) >> log2_page;
    int pg = -1;
    if (col < a.table_width) {
      int32_t* entry = a.block_table + (size_t)b * a.table_width + col;
      if (col < held) {
        pg = *entry;
      } else {
        const int k = free_count - 1 - (rec_page[rec] + col - held);
        if (k >= 0) pg = a.free_pages[k];
        if ((at & (P - 1)) == 0) *entry = pg;
      }
    }
    if (pg < 0) fault |= FT_ST_NO_ROOM;
    a.slots[t] = pg < 0 ? -1 : (((int64_t)pg << log2_page) | (at & (P - 1)));
    int depth = i;
    if (a.parents) {
      // Ancestors come in descending order, so the mask's words are finished
      // one after another from the row's own word down.
      uint32_t* row = a.mask + (size_t)t * a.mask_words;
      int word = a.mask_words, cur = i;
      uint32_t bits = 0;
      depth = -1;
      if ((i >> 5) >= a.mask_words) fault |= FT_ST_BAD_TREE;
      while (cur >= 0) {
        ++depth;
        const int cw = cur >> 5;
        if (cw < word) {
          if (word < a.mask_words) row[word] = bits;
          for (int z = word - 1; z > cw; --z) row[z] = 0;
          word = cw;
          bits = 0;
        }
        if (cw < a.mask_words) bits |= 1u << (cur & 31);
        const int g = start + cur;
        int up = g >= t0 - kBehind ? s_parent[g - t0 + kBehind] : a.parents[g];
        if (up >= cur || up < -1) {
          fault |= FT_ST_BAD_TREE;
          up = -1;
        }
        cur = up;
      }
      if (word < a.mask_words) row[word] = bits;
      for (int z = min(word, a.mask_words) - 1; z >= 0; --z) row[z] = 0;
    }
    a.positions[t] = ctx + depth;
  }
  if (fault && a.status) atomicOr(a.status, fault);
}

}  // namespace
}  // namespace ft

extern "C" int ft_kv_plan(const ft_plan_args* args, void* stream) {
  using namespace ft;
  if (!args) return record_error(FT_E_ARG, "null args");
  const ft_plan_args& a = *args;
  if (a.reserved) return record_error(FT_E_ARG, "reserved must be zero");
  if (a.num_reqs < 0 || a.max_tokens < 0 || a.table_width < 0 || a.mask_words < 0)
    return record_error(FT_E_ARG, "num_reqs, max_tokens, table_width and mask_words must not be negative");
  if (a.page_size < 1 || a.page_size > (1 << 20) || (a.page_size & (a.page_size - 1)))
    return record_error(FT_E_ARG, "page_size must be a power of two up to 2^20");
  if (a.max_tokens > (1 << 30)) return record_error(FT_E_ARG, "max_tokens must not exceed 2^30");
  if (a.num_reqs > 0 && (!a.ctx_len || !a.new_len || !a.block_table || !a.free_pages))
    return record_error(FT_E_ARG, "null pointer");
  if (!a.q_start || !a.free_count || !a.free_left || (a.max_tokens > 0 && (!a.slots || !a.positions)))
    return record_error(FT_E_ARG, "null pointer");
  if (a.free_left == a.free_count) return record_error(FT_E_ARG, "free_left must not be free_count");
  if (a.parents ? (!a.mask || a.mask_words < 1) : a.mask_words != 0)
    return record_error(FT_E_ARG, "parents need a mask with mask_words >= 1; without them mask_words must be 0");
  int log2_page = 0;
  while ((1 << log2_page) < a.page_size) ++log2_page;
  const int grid = a.max_tokens > 0 ? (a.max_tokens + kThreads - 1) / kThreads : 1;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(cfg, attr, dim3(grid), dim3(kThreads), 0, static_cast<cudaStream_t>(stream));
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_plan_kernel, a, log2_page);
  if (e != cudaSuccess) return record_error(FT_E_CUDA, "plan launch failed: %s", cudaGetErrorString(e));
  return FT_OK;
}
