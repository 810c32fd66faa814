// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits in one pass (ft_token_logprobs).
//
// With m a running maximum, M = m log2(e) and t = x log2(e) - M, a row needs
//   S = sum 2^t,   U = sum t 2^t:
//   ln sum e^x = m + ln 2 log2 S,   entropy = ln 2 (log2 S - U / S),
// and when t falls by d for a larger m, U <- (U - d S) 2^-d, S <- S 2^-d.  (M is
// rounded; t at x = m is that rounding, and the result takes it out again.  Past
// |m| = 2^24, where it would pass 1, t is (x - m) log2(e).)
//
// HBM bounds many rows, if a batch of logits costs few instructions: 16-bit
// logits are clamped and their maximum taken in packed pairs, the rest runs on
// packed fp32 pairs, so that an element is 1 exponential and 3.5 other
// instructions (4000 rows of 131072 bf16 without alternatives: 6.7 TB/s, the
// copy rate; 1024 rows with 8 alternatives 54 us, without 47).  A batch is
// kVecs 16-byte vectors a thread: one maximum and one rescaling serve it, and
// the next batch's loads are in flight meanwhile.
// A batch that holds NaN, or whose maximum lies past 2^24 or near the type's
// lowest value, is done again with care.
//
// Alternatives without a second pass over HBM: each thread keeps only its
// largest value.  The top_n-th largest over groups of threads is a bound that
// at least top_n entries reach, and only threads whose largest reaches it hold
// such entries: a warp looks at each such thread's entries again (from L2) and
// collects those that reach the bound, top_n and a few more.  They are ordered
// by a 64-bit key (value, then lower id).  Where they overflow the list
// (thousands of equal logits) the warps walk all entries, each merging what
// beats its own top_n-th.
//
// A row goes to a cluster of CTAs, each with a stretch of it, so that a few
// rows still use many SMs; the CTAs' sums and lists are written to the first
// one's shared memory.  All orders are fixed, so results repeat bit by bit.
#include <cooperative_groups.h>
#include <math_constants.h>

#include "attn_side.h"
#include "tma.h"

namespace ft {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kVecs = 4;     // 16-byte loads of a batch
constexpr int kList = 1024;  // entries that reach the bound
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNear = 16777216.f;  // up to here the rounding of m log2(e) is below 1

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

// Bitonic networks over a warp's lanes, larger first.
template <typename T>
__device__ __forceinline__ T order_step(T k, int lane, int o, bool larger_first) {
  const T other = __shfl_xor_sync(~0u, k, o);
  const bool low = (lane & o) == 0;
  return (low == larger_first) == (k > other) ? k : other;
}
template <typename T>
__device__ __forceinline__ T warp_sort(T k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) k = order_step(k, lane, o, (lane & size) == 0 || size == 32);
  return k;
}
// The 32 largest of two descending lists, descending.
template <typename T>
__device__ __forceinline__ T warp_merge(T a, T b, int lane) {
  const T r = __shfl_sync(~0u, b, 31 - lane);
  T k = a > r ? a : r;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) k = order_step(k, lane, o, true);
  return k;
}
// Lists [0, n) (n a power of two) merged into the first; the whole block calls it.
template <typename T>
__device__ __forceinline__ void block_merge(T (*list)[kMaxTop], int n, int w, int lane) {
#pragma unroll 1
  for (n >>= 1; n > 0; n >>= 1) {
    __syncthreads();
    if (w < n) list[w][lane] = warp_merge(list[w][lane], list[w + n][lane], lane);
  }
  __syncthreads();
}

struct Sums {
  float m, s, u;  // reference, sum of 2^t, sum of t 2^t
};
__device__ __forceinline__ bool near(float m) { return fabsf(m) <= kNear; }
// t of the reference itself: the rounding of M.
__device__ __forceinline__ float rest(float m) { return near(m) ? fmaf(m, kLog2e, -__fmul_rn(m, kLog2e)) : 0.f; }
// How far t falls when the reference moves from a to b >= a.
__device__ __forceinline__ float fall(float a, float b) {
  if (__builtin_expect(near(a) && near(b), 1)) return __fmul_rn(a, kLog2e) - __fmul_rn(b, kLog2e);
  return fmaxf((a - b) * kLog2e + (rest(b) - rest(a)), -1e30f);  // (also for -inf - -inf)
}
__device__ __forceinline__ Sums moved(Sums a, float m) {
  const float d = fall(a.m, m), e = ex2(d);
  // d 2^d -> 0 as d -> -inf: a part that vanishes adds nothing
  return Sums{m, a.s * e, e > 0.f ? fmaf(d, a.s, a.u) * e : 0.f};
}
// The sum of each N neighbouring lanes' parts, in a fixed order: to their maximum, then added.
template <int N>
__device__ __forceinline__ Sums lanes_sum(Sums q) {
  float m = q.m;
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  if (m != -CUDART_INF_F) q = moved(q, m);
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    q.s += __shfl_xor_sync(~0u, q.s, o);
    q.u += __shfl_xor_sync(~0u, q.u, o);
  }
  return q;
}
// One entry with care: any value.
__device__ __forceinline__ void add_entry(Sums& q, float x) {
  if (!(x > -CUDART_INF_F)) return;  // -inf adds nothing, NaN counts as -inf
  if (x > q.m) q = moved(q, x);
  const float t = near(q.m) ? fmaf(x, kLog2e, -__fmul_rn(q.m, kLog2e)) : (x - q.m) * kLog2e;
  const float e = ex2(fmaxf(t, -1e30f));
  q.s += e;
  if (e > 0.f) q.u = fmaf(t, e, q.u);
}

template <typename E>
struct Logit;  // 16 bytes of logits
template <>
struct Logit<float> {
  static constexpr int N = 4;
  static constexpr float kLow = -kNear;
  static __device__ __forceinline__ void unpack(uint4 w, float* x) {
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
  }
  // every value at least a little below kLow, NaN kept
  static __device__ __forceinline__ void unpack_clamped(uint4 w, float* x) {
    unpack(w, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("max.NaN.f32 %0, %0, %1;" : "+f"(x[j]) : "f"(-1e30f));
  }
  // maximum of a batch's values that are not NaN
  static __device__ __forceinline__ float largest(const uint4* v) {
    float m = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v[i].x), __uint_as_float(v[i].y)),
                         fmaxf(__uint_as_float(v[i].z), __uint_as_float(v[i].w))));
    return m;
  }
  static __device__ __forceinline__ float scalar(const float* p) { return __ldg(p); }
};
template <typename E, typename E2>
struct Logit16 {
  static constexpr int N = 8;
  static __device__ __forceinline__ E2 as2(uint32_t w) { return *reinterpret_cast<E2*>(&w); }
  static __device__ __forceinline__ uint32_t bits(E2 w) { return *reinterpret_cast<uint32_t*>(&w); }
  static __device__ __forceinline__ void unpack(uint4 w, float* x) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Elem<E>::unpack(v[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void unpack_clamped(uint4 w, float* x) {
    const E2 low = as2(Logit<E>::kClamp);
    unpack(make_uint4(bits(__hmax2_nan(as2(w.x), low)), bits(__hmax2_nan(as2(w.y), low)),
                      bits(__hmax2_nan(as2(w.z), low)), bits(__hmax2_nan(as2(w.w), low))),
           x);
  }
  static __device__ __forceinline__ float largest(const uint4* v) {
    E2 m = __hmax2(__hmax2(as2(v[0].x), as2(v[0].y)), __hmax2(as2(v[0].z), as2(v[0].w)));
#pragma unroll
    for (int i = 1; i < kVecs; ++i)
      m = __hmax2(m, __hmax2(__hmax2(as2(v[i].x), as2(v[i].y)), __hmax2(as2(v[i].z), as2(v[i].w))));
    const float2 f = Elem<E>::unpack(bits(m));
    const float top = fmaxf(f.x, f.y);
    return top == top ? top : -CUDART_INF_F;
  }
};
template <>
struct Logit<__nv_bfloat16> : Logit16<__nv_bfloat16, __nv_bfloat162> {
  static constexpr uint32_t kClamp = 0xF149F149u;  // about -1e30
  static constexpr float kLow = -kNear;
  static __device__ __forceinline__ float scalar(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};
template <>
struct Logit<__half> : Logit16<__half, __half2> {
  static constexpr uint32_t kClamp = 0xFBFFFBFFu;  // -65504
  static constexpr float kLow = -6e4f;
  static __device__ __forceinline__ float scalar(const __half* p) { return __half2float(*p); }
};

struct RowShared {
  uint64_t keys[kList];
  uint64_t list[kWarps][kMaxTop];
  uint64_t from[kMaxCluster][kMaxTop];  // the first CTA's: each CTA's best, descending
  Sums from_sums[kMaxCluster];
  int from_nan[kMaxCluster];
  float best[64];          // largest of each 4 threads
  uint8_t who[kThreads];   // threads whose largest reaches the bound
  Sums warp_sums[kWarps];
  int warp_nan[kWarps];    // the warp met a NaN
  int n_who, count;
};

template <typename E, int CS>
__global__ void __launch_bounds__(kThreads, 4) token_logprobs_kernel(const ft_logprob_args a) {
  using L = Logit<E>;
  constexpr int N = L::N;
  __shared__ RowShared sh;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const int rank = CS == 1 ? 0 : (int)(blockIdx.x % CS);
  const int t = blockIdx.x / CS;
  const E* row = static_cast<const E*>(a.logits) + (int64_t)t * a.row_stride;
  if (tid == 0) sh.n_who = sh.count = 0;  // (used after the barrier that follows the bound)
  if constexpr (CS > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // waited for before remote writes

  // The given token's logit, on its way while the row is read.
  int token = -1;
  float token_x = 0.f;
  if (rank == 0 && tid == 0 && a.tokens) {
    token = a.tokens[t];
    if (token >= 0 && token < a.V) token_x = L::scalar(row + token);
  }

  // The row: up to N-1 entries before the first 16-byte boundary, whole
  // 16-byte vectors, the rest.  Vectors [v0, v1) are this CTA's.
  const int mis = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(E));
  const int head = min(mis ? N - mis : 0, a.V);
  const int nvec = (a.V - head) / N, tail0 = head + nvec * N;
  const uint4* body = reinterpret_cast<const uint4*>(row + head);
  const int per = ((nvec + CS - 1) / CS + kThreads - 1) / kThreads * kThreads;
  const int v0 = min(rank * per, nvec), v1 = min(v0 + per, nvec);

  Sums q{-CUDART_INF_F, 0.f, 0.f};
  bool nan = false;
  uint4 raw[kVecs];
  // past the end: the batch's first vector again, left out of the sums
  auto load = [&](int v) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) raw[i] = __ldg(body + (v + i * kThreads < v1 ? v + i * kThreads : v));
  };
  if (v0 + tid < v1) load(v0 + tid);
  for (int v = v0 + tid; v < v1; v += kThreads * kVecs) {
    uint4 cur[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) cur[i] = raw[i];
    if (v + kThreads * kVecs < v1) load(v + kThreads * kVecs);
    const float top = L::largest(cur);
    if (top > q.m) q = moved(q, top);
    const uint64_t m2 = pair2(-__fmul_rn(q.m, kLog2e), -__fmul_rn(q.m, kLog2e)), l2 = pair2(kLog2e, kLog2e);
    uint64_t s2[2] = {}, u2[2] = {};
    const int left = (v1 - v + kThreads - 1) / kThreads;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if (i < left) {
        float x[N];
        L::unpack_clamped(cur[i], x);
#pragma unroll
        for (int j = 0; j < N; j += 2) {
          const uint64_t t2 = fma2(pair2(x[j], x[j + 1]), l2, m2);
          const float2 f = split2(t2);
          const uint64_t e2 = pair2(ex2(f.x), ex2(f.y));
          s2[(j >> 1) & 1] = add2(s2[(j >> 1) & 1], e2);
          u2[(j >> 1) & 1] = fma2(t2, e2, u2[(j >> 1) & 1]);
        }
      }
    }
    const float2 s = split2(add2(s2[0], s2[1])), u = split2(add2(u2[0], u2[1]));
    const float bs = s.x + s.y;
    if (bs == bs && q.m >= L::kLow && q.m <= kNear) {
      q.s += bs;
      q.u += u.x + u.y;
    } else {
#pragma unroll 1
      for (int i = 0; i < kVecs && i < left; ++i) {
        float x[N];
        L::unpack(__ldg(body + v + i * kThreads), x);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          nan |= x[j] != x[j];
          add_entry(q, x[j]);
        }
      }
    }
  }
  const float best = v0 + tid < v1 ? q.m : CUDART_NAN_F;  // NaN: this thread has no vector
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
      add_entry(q, x);
    }
  }
  q = lanes_sum<32>(q);
  nan = __any_sync(~0u, nan);
  if (lane == 0) {
    sh.warp_sums[w] = q;
    sh.warp_nan[w] = nan;
  }

  if (a.top_n > 0) {
    // The bound: the top_n-th largest of 64 groups of 4 threads, or 32 of 8 where
    // that leaves enough groups above it (-inf: fewer groups have vectors).
    // Of g groups about g ln(g / (g - top_n)) entries reach the bound: 9 for 8
    // and 22 for 16 of 32, 44 for 32 of 64 (all 32 of 32 would be some 130).
    float most = best == best ? best : -CUDART_INF_F;
    most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
    most = fmaxf(most, __shfl_xor_sync(~0u, most, 2));
    if ((lane & 3) == 0) sh.best[w * 8 + (lane >> 2)] = most;
    __syncthreads();
    float order = sh.best[lane], other = sh.best[lane + 32];
    if (a.top_n <= 16)
      order = warp_sort(fmaxf(order, other), lane);
    else
      order = warp_merge(warp_sort(order, lane), warp_sort(other, lane), lane);
    const float bound = __shfl_sync(~0u, order, a.top_n - 1);
    // the threads with entries that reach it, shared out over the warps
    if (best >= bound) sh.who[atomicAdd(&sh.n_who, 1)] = (uint8_t)tid;
    __syncthreads();
    const int n_who = sh.n_who;
    for (int c = w; c < n_who; c += kWarps) {
      const int first = v0 + sh.who[c];
#pragma unroll 2
      for (int v = first + lane * kThreads; v < v1; v += 32 * kThreads) {
        float x[N];
        L::unpack(__ldg(body + v), x);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (!(x[j] < bound)) {  // NaN too: it counts as -inf, which may be the bound
            const uint64_t key = make_key(x[j], head + v * N + j);
            if (key_value(key) >= bound) {
              const int at = atomicAdd(&sh.count, 1);
              if (at < kList) sh.keys[at] = key;
            }
          }
        }
      }
    }
    if (edge && key_value(edge) >= bound) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kList) sh.keys[at] = edge;
    }
    if (tid < kMaxTop) sh.list[0][tid] = 0;
    __syncthreads();
    const int count = sh.count;
    if (count <= kList) {
      // each key's place is how many are larger
      for (int i = tid; i < count; i += kThreads) {
        const uint64_t key = sh.keys[i];
        int place = 0;
        for (int j = 0; j < count; ++j) place += sh.keys[j] > key;
        if (place < a.top_n) sh.list[0][place] = key;
      }
      __syncthreads();
    } else {
      // too many equal entries for the list: all entries, a warp's 32 vectors at a time
      uint64_t top = w == 0 ? warp_sort(edge, lane) : 0;
      for (int v = v0 + w * 32; v < v1; v += kThreads) {
        float x[N];
        if (v + lane < v1) L::unpack(__ldg(body + v + lane), x);
        const uint64_t cut = __shfl_sync(~0u, top, a.top_n - 1);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint64_t k = v + lane < v1 ? make_key(x[j], head + (v + lane) * N + j) : 0;
          if (__any_sync(~0u, k > cut)) top = warp_merge(top, warp_sort(k, lane), lane);
        }
      }
      sh.list[w][lane] = top;
      block_merge(sh.list, kWarps, w, lane);
    }
  } else {
    __syncthreads();
  }
  // this CTA's sums and list, into the first CTA's shared memory
  if (w == 0) {
    const Sums s = lanes_sum<kWarps>(sh.warp_sums[lane % kWarps]);
    const bool any_nan = __any_sync(~0u, sh.warp_nan[lane % kWarps] != 0);
    RowShared* to = &sh;
    if constexpr (CS > 1) {
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster has started
      to = cg::this_cluster().map_shared_rank(&sh, 0);
    }
    if (a.top_n > 0) to->from[rank][lane] = sh.list[0][lane];
    if (lane == 0) {
      to->from_sums[rank] = s;
      to->from_nan[rank] = any_nan;
    }
  } else if constexpr (CS > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  }
  if constexpr (CS > 1) {
    cg::this_cluster().sync();
  } else {
    __syncthreads();
  }
  if (rank != 0) return;
  if (CS > 1 && a.top_n > 0) block_merge(sh.from, CS, w, lane);
  if (w == 0) {
    const Sums s = lanes_sum<CS>(sh.from_sums[lane % CS]);
    const bool any_nan = __any_sync(~0u, sh.from_nan[lane % CS] != 0);
    const bool empty = s.m == -CUDART_INF_F, inf = s.m == CUDART_INF_F;
    const float log2s = log2f(s.s);
    const float off = kLn2 * (log2s - rest(s.m));  // ln p of an entry x: x - m - off
    auto logp = [&](float x) {
      if (inf) return CUDART_NAN_F;
      if (empty || !(x > -CUDART_INF_F)) return -CUDART_INF_F;
      return fminf((x - s.m) - off, 0.f);  // (a row of one entry: off is a rounding of either sign)
    };
    if (lane == 0) {
      if (a.status && (any_nan || inf)) atomicOr(a.status, FT_ST_NAN);
      if (a.entropy) a.entropy[t] = inf ? CUDART_NAN_F : empty ? 0.f : fmaxf(kLn2 * (log2s - s.u / s.s), 0.f);
      if (a.logprob && a.tokens) {
        if (token >= a.V && a.status) atomicOr(a.status, FT_ST_BAD_TOKEN);
        a.logprob[t] = token >= 0 && token < a.V ? logp(token_x) : CUDART_NAN_F;
      }
    }
    if (lane < a.top_n) {
      const uint64_t top = sh.from[0][lane];
      a.top_ids[(int64_t)t * a.top_n + lane] = (int32_t)key_id(top);
      a.top_logprobs[(int64_t)t * a.top_n + lane] = logp(key_value(top));
    }
  }
}

template <typename E, int CS>
cudaError_t launch(const ft_logprob_args& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.T * CS);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CS;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CS > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<E, CS>, a);
}

template <typename E>
cudaError_t launch_cs(const ft_logprob_args& a, cudaStream_t st) {
  // A CTA for every SM, but a row is halved again only where its stretches hold
  // more than one batch each.  More CTAs shorten the read of a row and repeat the
  // search for its alternatives: 61 rows of
  // 50021 fp32 with 20 alternatives take 7.7 us with 4 CTAs a row, 9.1 with 8
  // and 11.1 with one, 300 rows of 131072 bf16 with 8 alternatives 18.8 us with
  // one and 27.1 us with 4.
  const int vecs = a.V / Logit<E>::N;
  int cs = 1;
  while (cs < kMaxCluster && (int64_t)a.T * cs < sm_count() && vecs / cs > kThreads * kVecs) cs *= 2;
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
