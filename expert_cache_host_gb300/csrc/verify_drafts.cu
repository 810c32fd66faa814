// Drafted tokens accepted or rejected against the target's probabilities, and
// the token that follows (ft_verify_drafts).
//
// A child x of the row reached is accepted if u q(x) A < a(x); a rejection turns
// a into max(a - A q, 0) and A into its sum; the last a is drawn from by its
// running sum.  Whether a child is accepted takes single entries, so the walk
// down the tree gathers those (all rows' entries at once); only a rejection
// followed by another child, and the draw at the end, read a row of V entries.
// One row of either kind and request is what the call cannot do without, HBM
// bounds large batches, latency a single request.
//
// The token is a whole number next to borders of the running sum: fp32 sums over
// 131072 entries would move the borders by more than many entries are wide, and
// 64-bit floating point runs at a sixty-fourth of the rate.  So entries are cut into
// whole numbers at three levels (multiples of 2^-22, 2^-40 and 2^-59; adding a
// constant leaves each level's number in the sum's low bits) and added as such:
// sums do not depend on their order.  After k rejections
//   a = max(p - q B, 0),  B = 1 + A_1 + .. + A_(k-1)
// (what one step cuts off at 0 the next ones would take below it), so a is never
// stored and takes one product, in two fp32 numbers: exact to 2^-46.
//
// A cluster of CTAs shares a request.  CTA 0 walks and says what the cluster
// does next; every warp sums one stretch of the row and keeps its pieces' sums,
// and the piece that holds the drawn point is gone through once more.
#include <cooperative_groups.h>

#include "attn_side.h"
#include "tma.h"

namespace ft {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kNodes = 512;  // rows of a request whose entries are gathered ahead
constexpr int kRejected = 64;
constexpr int kUnit = 59;  // sums are in units of 2^-59
constexpr int kBatch = 4;  // vectors a lane loads before it uses the first
constexpr int kPieces = 64;  // of a warp's stretch

template <typename E>
struct Prob {  // a 16-byte vector of a row
  static constexpr int N = 8;
  static __device__ __forceinline__ float one(const void* p, int64_t i) {
    return Elem<E>::unpack(static_cast<const uint16_t*>(p)[i]).x;
  }
  static __device__ __forceinline__ void all(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = Elem<E>::unpack(w[i]);
      f[2 * i] = t.x, f[2 * i + 1] = t.y;
    }
  }
};
template <>
struct Prob<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
  static __device__ __forceinline__ void all(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
};

__device__ __forceinline__ bool in_range(float v) { return v >= 0.f && v <= 2.f; }
// A random number as it is used.
__device__ __forceinline__ float below_one(float u) { return u > 0.f ? fminf(u, 0.99999994f) : 0.f; }

// Sums of numbers hi + lo in [0, 2] (|lo| <= 2^-24 hi) as whole numbers at three
// levels; each counts the constants' bits once a number.
struct Levels {
  uint32_t a = 0, b = 0, c = 0;
  static constexpr float kA = 2.f, kB = 0x1.8p-17f, kC = 0x1.8p-36f;
  __device__ __forceinline__ void add(float hi, float lo) {
    const float s = hi + kA, r = (hi - (s - kA)) + lo;
    const float t = r + kB, q = r - (t - kB);
    a += __float_as_uint(s);
    b += __float_as_uint(t);
    c += __float_as_uint(q + kC);
  }
  // What `n` numbers gave, without the constants.
  __device__ __forceinline__ void finish(uint32_t n) {
    a -= n * __float_as_uint(kA);
    b -= n * __float_as_uint(kB);
    c -= n * __float_as_uint(kC);
  }
  __device__ __forceinline__ uint64_t value() const {
    return ((uint64_t)a << (kUnit - 22)) + ((int64_t)(int32_t)b << (kUnit - 40)) + (int64_t)(int32_t)c;
  }
};

struct Node {
  int parent, token;
  float u, p, q;
};

enum Command : int { kSum, kDraw };

struct Shared {
  Node nodes[kNodes];
  // what CTA 0 says
  int command, row, k;  // the row that is read (in the batch), rejections so far
  float b_hi, b_lo;     // B
  int gone[kRejected];  // rejected tokens
  // sums of a pass: of a warp's pieces, of this CTA's warps, of all CTAs
  uint64_t piece[kWarps][kPieces];
  uint64_t warp_sum[kWarps], cta_sum[kMaxCluster];
  float warp_size[kWarps], cta_size[kMaxCluster];
};

struct Row {  // a request's row of probabilities, and the draft's beside it
  const void* p;
  const void* q;
  int off;       // index of the first element on a 16-byte boundary of both; -1: there is none
  int groups;    // vectors, the first holding elements [off - N, off)
};

template <typename E>
__device__ __forceinline__ Row row_at(const ft_verify_args& a, int64_t t) {
  constexpr int N = Prob<E>::N, size = 16 / N;
  Row r;
  r.p = static_cast<const uint8_t*>(a.probs) + t * a.probs_stride * size;
  r.q = a.draft_probs ? static_cast<const uint8_t*>(a.draft_probs) + t * a.draft_stride * size : nullptr;
  const int mis = (int)(reinterpret_cast<uintptr_t>(r.p) % 16) / size;
  r.off = mis ? N - mis : 0;
  r.groups = (a.V - r.off + N - 1) / N + 1;
  if (r.q && (int)(reinterpret_cast<uintptr_t>(r.q) % 16) / size != mis) r.off = -1;
  if (r.off < 0) r.groups = (a.V + N - 1) / N + 1;
  return r;
}

// Group g of a row: elements first(g) .. + N - 1, those outside [0, V) as 0.
template <typename E>
__device__ __forceinline__ uint4 load(const void* row, bool vec, int first, int V) {
  constexpr int N = Prob<E>::N;
  if (vec && first >= 0 && first + N <= V)
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + (int64_t)first * (16 / N)));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (first + i < 0 || first + i >= V) continue;
    if constexpr (N == 4)
      w[i] = static_cast<const uint32_t*>(row)[first + i];
    else
      w[i >> 1] |= (uint32_t)static_cast<const uint16_t*>(row)[first + i] << (i & 1 ? 16 : 0);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What is left of a group's elements, as hi + lo.
template <typename E>
struct Weights {
  float hi[Prob<E>::N], lo[Prob<E>::N];
  bool bad;
  __device__ __forceinline__ void make(const Shared& sh, const uint4& vp, const uint4& vq, bool draft, int first, int k,
                                       float b_hi, float b_lo) {
    constexpr int N = Prob<E>::N;
    Prob<E>::all(vp, hi);
    bad = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool ok = in_range(hi[i]);
      bad |= !ok;
      hi[i] = ok ? hi[i] : 0.f;
      lo[i] = 0.f;
    }
    if (k == 0) return;
    if (!draft) {
      for (int j = 0; j < k; ++j) {
        const uint32_t at = (uint32_t)(sh.gone[j] - first);
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (at == (uint32_t)i) hi[i] = 0.f;
      }
      return;
    }
    float q[N];
    Prob<E>::all(vq, q);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool ok = in_range(q[i]);
      bad |= !ok;
      const float f = ok ? q[i] : 0.f;
      const float t = f * b_hi, e = fmaf(f, b_lo, fmaf(f, b_hi, -t));  // f B = t + e
      const float d = hi[i] - t, v = d - hi[i];
      const float l = ((hi[i] - (d - v)) - (t + v)) - e;  // hi - t = d + the first difference, exactly
      const bool some = d + l > 0.f;
      hi[i] = some ? d : 0.f;
      lo[i] = some ? l : 0.f;
    }
  }
};

template <typename T>
__device__ __forceinline__ T warp_sum(T x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// The walk's state, in CTA 0's first warp (every lane the same).
struct Walk {
  int at, last, k, count;  // row reached, last child tried, rejections at `at`, accepted rows
  bool known;              // A after k rejections is
  double A, B;             // it, and those before it together
};

template <typename E, int CS>
__global__ void __launch_bounds__(kThreads, 3) verify_drafts_kernel(const __grid_constant__ ft_verify_args a) {
  __shared__ Shared sh;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / CS, rank = CS > 1 ? (int)(blockIdx.x % CS) : 0;
  auto everyone = [&] {
    if constexpr (CS > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
  };
  auto peer = [&](int r) -> Shared* {
    if constexpr (CS > 1) return cg::this_cluster().map_shared_rank(&sh, r);
    return &sh;
  };
  const int q0 = a.q_start[b], end = min(a.q_start[b + 1], a.max_tokens);
  const int n = q0 < 0 ? 0 : max(end - q0, 0);
  if (n == 0) {  // (the whole cluster)
    if (rank == 0 && tid == 0) a.n_accepted[b] = 0, a.next_token[b] = -1;
    return;
  }
  auto node_at = [&](int i, int at) {  // row i; its entries if its parent is `at` (or whatever it is, at < 0)
    Node x;
    x.parent = a.parents ? a.parents[q0 + i] : i - 1;
    x.token = a.tokens[q0 + i];
    x.u = a.accept_u[q0 + i];
    x.p = 0.f, x.q = 1.f;
    const int from = at < 0 ? x.parent : at;
    if (x.token >= 0 && x.token < a.V && from >= 0 && from < i) {
      const Row r = row_at<E>(a, q0 + from);
      x.p = Prob<E>::one(r.p, x.token);
      if (r.q) x.q = Prob<E>::one(r.q, x.token);
    }
    return x;
  };
  if constexpr (CS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (rank == 0) {
    for (int i = tid; i < min(n, kNodes); i += kThreads)
      if (i > 0) sh.nodes[i] = node_at(i, -1);
    __syncthreads();
  }
  if constexpr (CS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA has started
  Walk w{0, 0, 0, 0, true, 1.0, 0.0};
  bool bad = false, bad_token = false, bad_tree = false;
  for (;;) {
    if (rank == 0 && warp == 0) {
      int command = kDraw;
      for (;;) {
        // the next child of w.at
        int child = -1;
        for (int i0 = w.last + 1; i0 < n && child < 0; i0 += 32) {
          const int i = i0 + lane;
          int parent = -1;
          if (i < n) parent = i < kNodes ? sh.nodes[i].parent : a.parents ? a.parents[q0 + i] : i - 1;
          const uint32_t hit = __ballot_sync(~0u, i < n && parent == w.at);
          if (hit) child = i0 + __ffs(hit) - 1;
        }
        if (child < 0) break;
        Node x;
        if (child < kNodes)
          x = sh.nodes[child];
        else
          x = node_at(child, w.at);
        if (x.token < 0 || x.token >= a.V) {
          bad_token = true;
          w.last = child;
          continue;
        }
        if (w.k == kRejected) {
          bad_tree = true;
          w.last = child;
          continue;
        }
        if (!w.known) {
          command = kSum;
          break;
        }
        const bool ok_p = in_range(x.p), ok_q = in_range(x.q);
        bad |= !ok_p || !ok_q;
        const double p = ok_p ? x.p : 0.f, q = ok_q ? x.q : 0.f, u = below_one(x.u);
        double left = p;
        if (a.draft_probs) {
          left = fmax(p - q * w.B, 0.0);
        } else {
          for (int j = 0; j < w.k; ++j)
            if (sh.gone[j] == x.token) left = 0.0;
        }
        w.last = child;
        if (u * q * w.A < left) {  // (exact before the first rejection: two fp32 numbers' product)
          if (lane == 0) a.accepted[q0 + w.count] = child;
          w = Walk{child, child, 0, w.count + 1, true, 1.0, 0.0};
        } else {
          if (lane == 0) sh.gone[w.k] = x.token;
          __syncwarp();
          w.B += w.A;
          // without draft probabilities the next A is known once one sum is
          w.known = w.k > 0 && !a.draft_probs;
          if (w.known) w.A -= left;
          ++w.k;
        }
      }
      // what the cluster does next: sums of a at (at, k), then the draw
      if (lane < CS) {
        Shared* to = peer(lane);
        to->command = command;
        to->row = w.at;
        to->k = w.k;
        to->b_hi = (float)w.B;
        to->b_lo = (float)(w.B - (double)(float)w.B);
        for (int j = 0; j < w.k; ++j) to->gone[j] = sh.gone[j];
      }
    }
    everyone();
    const int command = sh.command;
    int k = sh.k;
    const Row r = row_at<E>(a, q0 + sh.row);
    constexpr int N = Prob<E>::N;
    const int per = (r.groups + CS * kWarps - 1) / (CS * kWarps);
    const int g0 = (rank * kWarps + warp) * per, g1 = min(g0 + per, r.groups);
    const bool vec = r.off >= 0;
    const int base = (vec ? r.off : 0) - N;  // first element of group 0
    // A stretch is gone through kBatch vectors a lane at a time; a piece is one such step, or several of a long one.
    const int steps = (per + 32 * kBatch - 1) / (32 * kBatch), to_piece = (steps + kPieces - 1) / kPieces;
    const float b_hi = sh.b_hi, b_lo = sh.b_lo;
    uint64_t total = 0;
    for (;;) {
      uint64_t sum = 0, piece = 0;
      float size = 0.f;
      for (int step = 0; step < steps; ++step) {
        const int g = g0 + step * 32 * kBatch + lane;
        uint4 vp[kBatch], vq[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int first = base + (g + 32 * i) * N;
          vp[i] = vq[i] = make_uint4(0, 0, 0, 0);
          if (g + 32 * i < g1) {
            vp[i] = load<E>(r.p, vec, first, a.V);
            if (r.q && k > 0) vq[i] = load<E>(r.q, vec, first, a.V);
          }
        }
        Levels s;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          Weights<E> x;
          x.make(sh, vp[i], vq[i], r.q != nullptr, base + (g + 32 * i) * N, k, b_hi, b_lo);
          bad |= x.bad;
#pragma unroll
          for (int j = 0; j < N; ++j) s.add(x.hi[j], x.lo[j]);
        }
        s.finish(kBatch * N);
        // (the first level's number in two parts: a warp's could pass 32 bits)
        const uint32_t up = __reduce_add_sync(~0u, s.a >> 12), low = __reduce_add_sync(~0u, s.a & 0xFFFu);
        const int32_t b32 = __reduce_add_sync(~0u, (int32_t)s.b), c32 = __reduce_add_sync(~0u, (int32_t)s.c);
        piece += (((uint64_t)up << 12) + low << (kUnit - 22)) + ((int64_t)b32 << (kUnit - 40)) + (int64_t)c32;
        size += (float)up * 0x1p-10f;
        if (step + 1 == steps || (step + 1) % to_piece == 0) {
          if (lane == 0) sh.piece[warp][step / to_piece] = piece;
          sum += piece;
          piece = 0;
        }
      }
      if (lane == 0) sh.warp_sum[warp] = sum, sh.warp_size[warp] = size;
      __syncthreads();
      if (tid < CS) {
        uint64_t s = 0;
        float z = 0.f;
        for (int i = 0; i < kWarps; ++i) s += sh.warp_sum[i], z += sh.warp_size[i];
        Shared* to = peer(tid);
        to->cta_sum[rank] = s;
        to->cta_size[rank] = z;
      }
      everyone();
      float whole = 0.f;
      total = 0;
      for (int i = 0; i < CS; ++i) total += sh.cta_sum[i], whole += sh.cta_size[i];
      if (whole > 8.f) {
        total = 0;
        bad = true;
      }
      if (command == kSum || total > 0 || k == 0) break;
      k = 0;  // nothing is left of a: the draw is from p
      everyone();
    }
    if (command == kSum) {
      if (rank == 0 && warp == 0) {
        w.A = (double)total * 0x1p-59;
        w.known = true;
      }
      everyone();  // (the sums have been read)
      continue;
    }
    // the draw
    if (total == 0) {
      bad = true;
      if (rank == 0 && tid == 0) a.next_token[b] = -1;
    } else {
      // floor(u total): a whole running sum is above u total where it is above that
      const uint32_t bits = __float_as_uint(below_one(a.draw_u[b]));
      const int shift = 150 - max((int)(bits >> 23), 1);
      const uint32_t m = (bits & 0x7FFFFFu) | (bits >> 23 ? 0x800000u : 0u);
      const uint64_t point = shift >= 128 ? 0 : (uint64_t)(((unsigned __int128)total * m) >> shift);
      uint64_t before = 0;
      for (int i = 0; i < rank; ++i) before += sh.cta_sum[i];
      if (point >= before && point - before < sh.cta_sum[rank]) {
        uint64_t left = point - before;
        for (int i = 0; i < warp; ++i) {
          if (left < sh.warp_sum[i]) {
            left = ~0ull;
            break;
          }
          left -= sh.warp_sum[i];
        }
        if (left != ~0ull && left < sh.warp_sum[warp]) {  // this warp's stretch holds the point
          int step = 0;
          for (int at = 0; left >= sh.piece[warp][at]; ++at) {  // (their sum is above it)
            left -= sh.piece[warp][at];
            step += to_piece;
          }
          bool found = false;
          for (; step < steps && !found; ++step) {
            const int gg = g0 + step * 32 * kBatch + lane;
            uint4 vp[kBatch], vq[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int first = base + (gg + 32 * i) * N;
              vp[i] = vq[i] = make_uint4(0, 0, 0, 0);
              if (gg + 32 * i < g1) {
                vp[i] = load<E>(r.p, vec, first, a.V);
                if (r.q && k > 0) vq[i] = load<E>(r.q, vec, first, a.V);
              }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              if (found) break;
              const int first = base + (gg + 32 * i) * N;
              Weights<E> x;
              x.make(sh, vp[i], vq[i], r.q != nullptr, first, k, b_hi, b_lo);
              auto value = [&](int j) {
                Levels s;
                s.add(x.hi[j], x.lo[j]);
                s.finish(1);
                return s.value();
              };
              uint64_t mine = 0;
#pragma unroll
              for (int j = 0; j < N; ++j) mine += value(j);
              uint64_t upto = mine;
#pragma unroll
              for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(~0u, upto, o);
                if (lane >= o) upto += y;
              }
              const uint32_t hit = __ballot_sync(~0u, upto > left);
              if (hit) {
                if (lane == __ffs(hit) - 1) {
                  uint64_t c = upto - mine;
                  int token = -1;
#pragma unroll
                  for (int j = 0; j < N; ++j) {
                    c += value(j);
                    if (token < 0 && c > left) token = first + j;
                  }
                  a.next_token[b] = token;
                }
                found = true;
              } else {
                left -= __shfl_sync(~0u, upto, 31);
              }
            }
          }
        }
      }
    }
    break;
  }
  if (rank == 0 && warp == 0) {
    if (lane == 0) a.n_accepted[b] = w.count;
    for (int i = w.count + lane; i < n; i += 32) a.accepted[q0 + i] = -1;
  }
  if (a.status) {
    const uint32_t said = (bad ? FT_ST_NAN : 0u) | (bad_token ? FT_ST_BAD_TOKEN : 0u) | (bad_tree ? FT_ST_BAD_TREE : 0u);
    if (said) atomicOr(a.status, said);
  }
  everyone();  // no CTA leaves while another may still write into its shared memory
}

template <typename E, int CS>
cudaError_t launch(const ft_verify_args& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.num_reqs * CS);
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
  return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<E, CS>, a);
}

template <typename E>
cudaError_t launch_cs(const ft_verify_args& a, cudaStream_t st) {
  int cs = 1;
  while (cs < kMaxCluster && (int64_t)a.num_reqs * cs < 4 * sm_count() && a.V / Prob<E>::N / cs > kThreads * kBatch) cs *= 2;
  switch (cs) {
    case 1: return launch<E, 1>(a, st);
    case 2: return launch<E, 2>(a, st);
    case 4: return launch<E, 4>(a, st);
    default: return launch<E, 8>(a, st);
  }
}

}  // namespace
}  // namespace ft

extern "C" int ft_verify_drafts(const ft_verify_args* args, void* stream) {
  using namespace ft;
  if (!args) return record_error(FT_E_ARG, "null args");
  const ft_verify_args& a = *args;
  if (a.dtype != FT_DTYPE_BF16 && a.dtype != FT_DTYPE_F16 && a.dtype != FT_DTYPE_F32)
    return record_error(FT_E_ARG, "probabilities must be FT_DTYPE_F32, FT_DTYPE_BF16 or FT_DTYPE_F16");
  if (a.max_tokens < 0 || a.num_reqs < 0 || a.num_reqs > (1 << 27) || a.V < 1 || a.V > (1 << 30))
    return record_error(FT_E_ARG, "bad max_tokens, num_reqs or V");
  if (!a.probs || !a.tokens || !a.accept_u || !a.draw_u || !a.q_start || !a.accepted || !a.n_accepted || !a.next_token)
    return record_error(FT_E_ARG, "null pointer");
  if ((reinterpret_cast<uintptr_t>(a.probs) | reinterpret_cast<uintptr_t>(a.draft_probs)) % (a.dtype == FT_DTYPE_F32 ? 4 : 2))
    return record_error(FT_E_ARG, "probabilities must be aligned to their type");
  if (a.probs_stride < 0 || a.draft_stride < 0) return record_error(FT_E_ARG, "strides must not be negative");
  if (a.num_reqs == 0) return FT_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.dtype == FT_DTYPE_BF16)
    e = launch_cs<__nv_bfloat16>(a, st);
  else if (a.dtype == FT_DTYPE_F16)
    e = launch_cs<__half>(a, st);
  else
    e = launch_cs<float>(a, st);
  if (e != cudaSuccess) return record_error(FT_E_CUDA, "draft verification launch failed: %s", cudaGetErrorString(e));
  return FT_OK;
}
