// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits in one pass (ft_token_logprobs).
//
// With m a running maximum and t = (x - m) log2(e), a row needs
//   S = sum 2^t,   U = sum t 2^t:
//   ln sum e^x = m + ln 2 log2 S,   entropy = ln 2 (log2 S - U / S),
// and when t falls by d for a larger m, U <- (U - d S) 2^-d, S <- S 2^-d.
// (x - m is formed first: with one fused product the reference m log2(e) would
// overflow for logits near the type's ends.)  Each thread keeps its own
// (m, S, U) over a batch of kVecs vectors at a time, so one maximum and one
// rescaling serve the batch; partial sums join in a fixed order.
//
// Alternatives without a second pass over HBM: order all entries by a 64-bit
// key (value, then lower id), so that no two are equal.  Each thread keeps
// only its largest value and the batch it came from.  The top_n-th largest of
// the threads' best keys is a bound: at least top_n entries reach it, and
// every entry that does belongs to one of exactly top_n threads (a thread's
// best is at least any of its entries).  So only those threads' entries are
// looked at again (from L2), a warp per thread, and merged 32 at a time into a
// sorted list in registers.  The work does not depend on the values beyond
// that, and equal logits cost nothing extra.
//
// A row goes to a cluster of CTAs, each with a stretch of it, so that a few
// rows still use many SMs; the CTAs' sums and sorted lists join through
// distributed shared memory.
#include <cooperative_groups.h>
#include <math_constants.h>

#include "attn_side.h"

namespace ft {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kVecs = 4;  // 16-byte loads of a batch
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Larger value, or the lower id among equals, is the larger key; 0 is below every entry.
__device__ __forceinline__ uint64_t make_key(float v, uint32_t id) {
  const uint32_t b = __float_as_uint(v == v ? v + 0.f : -CUDART_INF_F);  // -0 counts as +0, NaN as -inf
  const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((uint64_t)o << 32) | (0xFFFFFFFFu - id);
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ uint32_t key_id(uint64_t k) { return 0xFFFFFFFFu - (uint32_t)k; }

__device__ __forceinline__ uint64_t order_step(uint64_t k, int lane, int o, bool larger_first) {
  const uint64_t other = __shfl_xor_sync(~0u, k, o);
  const bool low = (lane & o) == 0;
  return (low == larger_first) == (k > other) ? k : other;
}
// The warp's 32 keys in descending order of lane.
__device__ __forceinline__ uint64_t warp_sort(uint64_t k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) k = order_step(k, lane, o, (lane & size) == 0 || size == 32);
  return k;
}
// The 32 largest of two descending lists, descending.
__device__ __forceinline__ uint64_t warp_merge(uint64_t a, uint64_t b, int lane) {
  const uint64_t r = __shfl_sync(~0u, b, 31 - lane);
  uint64_t k = a > r ? a : r;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) k = order_step(k, lane, o, true);
  return k;
}

struct Sums {
  float m, s, u;  // reference, sum of 2^t, sum of t 2^t
};
__device__ __forceinline__ Sums join(Sums a, Sums b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -CUDART_INF_F) return a;
  const float da = fmaxf((a.m - m) * kLog2e, -1e30f), db = fmaxf((b.m - m) * kLog2e, -1e30f);
  const float ea = ex2(da), eb = ex2(db);
  Sums r;
  r.m = m;
  r.s = a.s * ea + b.s * eb;
  // d * 2^d -> 0 as d -> -inf: a part that vanishes adds nothing
  r.u = (ea > 0.f ? (a.u + da * a.s) * ea : 0.f) + (eb > 0.f ? (b.u + db * b.s) * eb : 0.f);
  return r;
}

template <typename E>
struct Logit;  // 16 bytes of logits <-> floats, and a maximum that keeps NaN
template <>
struct Logit<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 w, float* x) {
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ float scalar(const float* p) { return __ldg(p); }
};
template <typename E>
struct Logit16 {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 w, float* x) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Elem<E>::unpack(v[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Logit<__nv_bfloat16> : Logit16<__nv_bfloat16> {
  static __device__ __forceinline__ float scalar(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};
template <>
struct Logit<__half> : Logit16<__half> {
  static __device__ __forceinline__ float scalar(const __half* p) { return __half2float(*p); }
};

struct RowShared {
  uint64_t list[kWarps][kMaxTop];
  uint64_t mine[kMaxTop];  // this CTA's best, descending (read by the cluster's first CTA)
  int cand[kMaxTop];
  Sums warp_sums[kWarps];
  Sums sums;  // this CTA's
  int nan;
};

template <typename E, int CS>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const ft_logprob_args a) {
  using L = Logit<E>;
  constexpr int N = L::N;
  __shared__ RowShared sh;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rank = CS == 1 ? 0 : (int)(blockIdx.x % CS);
  const int t = blockIdx.x / CS;
  const E* row = static_cast<const E*>(a.logits) + (int64_t)t * a.row_stride;

  // The row: up to N-1 entries before the first 16-byte boundary, whole
  // 16-byte vectors, the rest.  Vectors [v0, v1) are this CTA's.
  const int mis = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(E));
  const int head = min(mis ? N - mis : 0, a.V);
  const int nvec = (a.V - head) / N, tail0 = head + nvec * N;
  const uint4* body = reinterpret_cast<const uint4*>(row + head);
  const int per = ((nvec + CS - 1) / CS + kThreads - 1) / kThreads * kThreads;
  const int v0 = min(rank * per, nvec), v1 = min(v0 + per, nvec);

  if (tid == 0) sh.nan = 0;
  Sums q{-CUDART_INF_F, 0.f, 0.f};
  float best = -CUDART_INF_F;
  int best_vec = -1;  // first vector of the batch with this thread's largest value
  bool nan = false;
  for (int v = v0 + tid; v < v1; v += kThreads * kVecs) {
    uint4 raw[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int vi = v + i * kThreads;
      raw[i] = __ldg(body + (vi < v1 ? vi : v));  // past the end: the batch's first vector again, not counted below
    }
    float bmax = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float x[N];
      L::unpack(raw[i], x);
#pragma unroll
      for (int j = 0; j < N; ++j) bmax = fmaxf(bmax, x[j]);
    }
    if (bmax > best || best_vec < 0) best = bmax, best_vec = v;
    if (bmax > q.m) {
      const float d = fmaxf((q.m - bmax) * kLog2e, -1e30f), e = ex2(d);
      q.u = e > 0.f ? (q.u + d * q.s) * e : 0.f;
      q.s *= e;
      q.m = bmax;
    }
    const float ref = q.m == -CUDART_INF_F ? 0.f : q.m;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if (v + i * kThreads < v1) {
        float x[N];
        L::unpack(raw[i], x);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          nan |= x[j] != x[j];
          const float tt = fmaxf((x[j] - ref) * kLog2e, -1000.f);  // -inf and NaN: 2^-1000 = 0
          const float e = ex2(tt);
          q.s += e;
          q.u = fmaf(tt, e, q.u);
        }
      }
    }
  }
  // entries outside the vectors: at most N-1 on either side, one thread each
  uint64_t edge = 0;
  if (rank == 0 && tid < 32) {
    int id = -1;
    if (tid < head) id = tid;
    else if (tid >= 16 && tail0 + tid - 16 < a.V) id = tail0 + tid - 16;
    if (id >= 0) {
      const float x = L::scalar(row + id);
      nan |= x != x;
      edge = make_key(x, id);
      if (x > -CUDART_INF_F) q = join(q, Sums{x, 1.f, 0.f});
    }
  }
  // the block's sums, in a fixed order
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums b;
    b.m = __shfl_down_sync(~0u, q.m, o);
    b.s = __shfl_down_sync(~0u, q.s, o);
    b.u = __shfl_down_sync(~0u, q.u, o);
    q = join(q, b);
  }
  if (lane == 0) sh.warp_sums[w] = q;
  __syncthreads();
  if (nan) sh.nan = 1;
  if (tid == 0) {
    Sums s = sh.warp_sums[0];
    for (int i = 1; i < kWarps; ++i) s = join(s, sh.warp_sums[i]);
    sh.sums = s;
  }

  if (a.top_n > 0) {
    // this thread's best key: the first place of its largest value
    uint64_t key = 0;
    if (best_vec >= 0) {
      for (int i = kVecs - 1; i >= 0; --i) {
        const int vi = best_vec + i * kThreads;
        if (vi < v1) {
          float x[N];
          L::unpack(__ldg(body + vi), x);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const uint64_t k = make_key(x[j], head + vi * N + j);
            key = k > key ? k : key;
          }
        }
      }
    }
    const uint64_t own = key;
    uint64_t k = warp_sort(key, lane);
    sh.list[w][lane] = k;
    __syncthreads();
#pragma unroll 1
    for (int n = kWarps / 2; n > 0; n >>= 1) {
      if (w < n) sh.list[w][lane] = warp_merge(sh.list[w][lane], sh.list[w + n][lane], lane);
      __syncthreads();
    }
    const uint64_t bound = sh.list[0][a.top_n - 1];
    // the (at most top_n) threads that reach the bound, in order of their place in the list
    if (own != 0 && own >= bound) {
      int p = 0;
      while (sh.list[0][p] != own) ++p;
      sh.cand[p] = tid;
    }
    __syncthreads();
    const int n_cand = __popc(__ballot_sync(~0u, lane < a.top_n && sh.list[0][lane] != 0));
    __syncthreads();
    uint64_t top = w == 0 ? warp_sort(edge, lane) : 0;
    for (int c = w; c < n_cand; c += kWarps) {
      const int who = sh.cand[c];
      for (int base = v0 + who; base < v1; base += 32 * kThreads) {
        const int vi = base + lane * kThreads;
        float x[N];
        if (vi < v1) L::unpack(__ldg(body + vi), x);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          uint64_t e = vi < v1 ? make_key(x[j], head + vi * N + j) : 0;
          if (e < bound) e = 0;
          if (__any_sync(~0u, e != 0)) top = warp_merge(top, warp_sort(e, lane), lane);
        }
      }
    }
    sh.list[w][lane] = top;
    __syncthreads();
#pragma unroll 1
    for (int n = kWarps / 2; n > 0; n >>= 1) {
      if (w < n) sh.list[w][lane] = warp_merge(sh.list[w][lane], sh.list[w + n][lane], lane);
      __syncthreads();
    }
    if (w == 0) sh.mine[lane] = sh.list[0][lane];
  }
  if constexpr (CS > 1) {
    cg::this_cluster().sync();
  } else {
    __syncthreads();
  }
  if (rank == 0 && w == 0) {
    Sums s = sh.sums;
    int any_nan = sh.nan;
    uint64_t top = a.top_n > 0 ? sh.mine[lane] : 0;
    if constexpr (CS > 1) {
      for (int r = 1; r < CS; ++r) {
        const RowShared* o = cg::this_cluster().map_shared_rank(&sh, r);
        s = join(s, o->sums);
        any_nan |= o->nan;
        if (a.top_n > 0) top = warp_merge(top, o->mine[lane], lane);
      }
    }
    const bool empty = s.m == -CUDART_INF_F, inf = s.m == CUDART_INF_F;
    const float log2s = log2f(s.s);
    const float off = kLn2 * log2s;  // ln p of an entry x: x - m - off
    auto logp = [&](float x) {
      if (inf) return CUDART_NAN_F;
      if (empty || !(x > -CUDART_INF_F)) return -CUDART_INF_F;
      return (x - s.m) - off;
    };
    if (lane == 0) {
      if (a.status && (any_nan || inf)) atomicOr(a.status, FT_ST_NAN);
      if (a.entropy) a.entropy[t] = inf ? CUDART_NAN_F : empty ? 0.f : kLn2 * (log2s - s.u / s.s);
      if (a.logprob && a.tokens) {
        const int id = a.tokens[t];
        if (id >= a.V && a.status) atomicOr(a.status, FT_ST_BAD_TOKEN);
        a.logprob[t] = id >= 0 && id < a.V ? logp(L::scalar(row + id)) : CUDART_NAN_F;
      }
    }
    if (lane < a.top_n) {
      if (a.top_ids) a.top_ids[(int64_t)t * a.top_n + lane] = (int32_t)key_id(top);
      if (a.top_logprobs) a.top_logprobs[(int64_t)t * a.top_n + lane] = logp(key_value(top));
    }
  }
  // the first CTA has read the others' shared memory when they leave
  if constexpr (CS > 1) cg::this_cluster().sync();
}

template <typename E, int CS>
cudaError_t launch(const ft_logprob_args& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.T * CS);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CS;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CS > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<E, CS>, a);
}

template <typename E>
cudaError_t launch_cs(const ft_logprob_args& a, cudaStream_t st) {
  // enough CTAs for the machine, but no CTA with less than one batch
  const int vecs = a.V / Logit<E>::N;
  int cs = 1;
  while (cs < 8 && (int64_t)a.T * cs < 4 * sm_count() && vecs / cs > kThreads * kVecs) cs *= 2;
  switch (cs) {
    case 1: return launch<E, 1>(a, st);
    case 2: return launch<E, 2>(a, st);
    case 4: return launch<E, 4>(a, st);
    default: return launch<E, 8>(a, st);
  }
}

}  // namespace
}  // namespace ft

extern "C" int ft_token_logprobs(const ft_logprob_args* args, void* stream) {
  using namespace ft;
  if (!args) return record_error(FT_E_ARG, "null args");
  const ft_logprob_args& a = *args;
  if (a.dtype != FT_DTYPE_BF16 && a.dtype != FT_DTYPE_F16 && a.dtype != FT_DTYPE_F32)
    return record_error(FT_E_ARG, "logits must be FT_DTYPE_BF16, FT_DTYPE_F16 or FT_DTYPE_F32");
  if (a.T < 0 || a.V < 1 || a.T > (1 << 27) || a.V > (1 << 30)) return record_error(FT_E_ARG, "bad T or V");
  if (a.top_n < 0 || a.top_n > kMaxTop || a.top_n > a.V)
    return record_error(FT_E_ARG, "top_n must be 0 to min(32, V)");
  if (!a.logits) return record_error(FT_E_ARG, "null pointer");
  if (reinterpret_cast<uintptr_t>(a.logits) % (a.dtype == FT_DTYPE_F32 ? 4 : 2))
    return record_error(FT_E_ARG, "logits must be aligned to their type");
  if (a.row_stride < 0) return record_error(FT_E_ARG, "row_stride must not be negative");
  if (a.top_n > 0 && (!a.top_ids || !a.top_logprobs)) return record_error(FT_E_ARG, "top_n needs top_ids and top_logprobs");
  if ((a.logprob != nullptr) != (a.tokens != nullptr)) return record_error(FT_E_ARG, "tokens and logprob go together");
  if (a.T == 0) return FT_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.dtype == FT_DTYPE_BF16)
    e = launch_cs<__nv_bfloat16>(a, st);
  else if (a.dtype == FT_DTYPE_F16)
    e = launch_cs<__half>(a, st);
  else
    e = launch_cs<float>(a, st);
  if (e != cudaSuccess) return record_error(FT_E_CUDA, "log probability launch failed: %s", cudaGetErrorString(e));
  return FT_OK;
}
