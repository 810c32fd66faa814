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
// whole numbers at two levels (multiples of 2^-22 and 2^-44; adding a constant
// leaves each level's number in the sum's low bits) and added as such: sums do not
// depend on their order.  After k rejections
//   a = max(p - q B, 0),  B = 1 + A_1 + .. + A_(k-1)
// (what one step cuts off at 0 the next ones would take below it), so a is never
// stored and takes one product, in two fp32 numbers (to 2^-46).
//
// A cluster of CTAs shares a request.  CTA 0 walks, a row of the request a lane,
// and says what the cluster does next; every warp sums one stretch of the row and
// keeps its pieces' sums, and the piece that holds the drawn point is gone through
// once more.  Vectors come through shared memory (a thread's own, kDepth rounds
// ahead).  64 trees of 9..17 tokens over 131072 fp32 entries take 43..50 us (67 MB of
// rows; the last requests go through theirs four times), one request 9.6.  One
// request is bound by latency, so the loop over them has no branches but for unusual
// numbers (with them a round of 8 numbers took 2400 cycles) and its code is short.
#include <cooperative_groups.h>

#include <type_traits>

#include "attn_side.h"
#include "tma.h"

namespace ft {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kRejected = 64;
constexpr int kUnit = 44;     // sums are in units of 2^-44
constexpr double kUnits = 1ull << kUnit;
constexpr int kNumbers = 16;  // of a thread in a round
constexpr int kDepth = 2;     // rounds on their way
constexpr int kResident = 2;  // CTAs of an SM
constexpr int kPieces = 64;   // of a warp's stretch at most
constexpr int kPiece = 4;     // rounds of a piece, or a multiple

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

// Sums of pairs of numbers hi + lo in [0, 2], hi the fp32 number next to the pair
// (|lo| <= 2^-24), as whole numbers at two levels; each counts the constants' bits
// once a number.  The first level leaves at most 2^-23 of hi, so that the second
// takes less than 2^-22 in size: kB and it stay in one binade, whose numbers are
// 2^-44 apart.  (With 0x1.8p-22 and 2^-45 there is room for 2^-23 alone: where lo
// came on top, after a rejection, entries were off by up to 2^-24.)
struct Levels {
  uint32_t a = 0, b = 0;
  static constexpr float kA = 2.f, kB = 0x1.8p-21f;
  __device__ __forceinline__ void add(uint64_t hi, uint64_t lo) {
    const uint64_t minus = pair2(-1.f, -1.f);
    const uint64_t s = add2(hi, pair2(kA, kA));
    const uint64_t r = add2(fma2(add2(s, pair2(-kA, -kA)), minus, hi), lo);
    const float2 x = split2(s), y = split2(add2(r, pair2(kB, kB)));
    a += __float_as_uint(x.x) + __float_as_uint(x.y);
    b += __float_as_uint(y.x) + __float_as_uint(y.y);
  }
  // What `n` numbers gave, without the constants.
  __device__ __forceinline__ void finish(uint32_t n) {
    a -= n * __float_as_uint(kA);
    b -= n * __float_as_uint(kB);
  }
  __device__ __forceinline__ uint64_t value() const { return ((uint64_t)a << (kUnit - 22)) + (int64_t)(int32_t)b; }
};

enum Command : int { kSum, kDraw };

struct Shared {
  uint4 ring[kDepth][2][kNumbers / 4][kThreads];
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

// Elements first .. first + N - 1 of a row, those outside [0, V) as 0.
template <typename E>
__device__ __noinline__ uint4 load_edge(const void* row, int first, int V) {
  constexpr int N = Prob<E>::N;
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

// Numbers outside [0, 2] become 0.
template <int COUNT>
__device__ __noinline__ void mend(float* f) {
  for (int i = 0; i < COUNT; ++i) f[i] = in_range(f[i]) ? f[i] + 0.f : 0.f;  // (-0 is 0)
}

__device__ __forceinline__ void copy16(const void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The walk's state, in CTA 0's first warp (every lane the same).
struct Walk {
  int at, last, k, count;  // row reached, last child tried, rejections at `at`, accepted rows
  bool known;              // A after k rejections is
  double A, B;             // it, and those before it together
};

template <typename E, int CS>
__global__ void __launch_bounds__(kThreads, kResident) verify_drafts_kernel(const __grid_constant__ ft_verify_args a) {
  constexpr int N = Prob<E>::N;
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
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
  // (CTA 0 may write into another's shared memory once all have started)
  if constexpr (CS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  Walk w{0, 0, 0, 0, true, 1.0, 0.0};
  // A lane's row of the window of 32 that is looked at: its parent, token, number and entries.
  int window = -32, parent = -1, token = -1;
  float u = 0.f, px = 0.f, qx = 1.f;
  bool bad = false, bad_token = false, bad_tree = false, started = CS == 1;
  for (;;) {
    if (rank == 0 && warp == 0) {
      int command = kDraw;
      for (;;) {
        // the next child of w.at (a child's row comes after its parent's)
        const uint32_t hit = __ballot_sync(~0u, parent == w.at && window + lane > w.last);
        if (!hit) {
          if (window + 32 >= n) break;
          window += 32;
          const int i = window + lane;
          parent = token = -1;
          if (i < n && i > 0) {
            parent = a.parents ? a.parents[q0 + i] : i - 1;
            token = a.tokens[q0 + i];
            u = below_one(a.accept_u[q0 + i]);
            px = 0.f, qx = 1.f;
            if (token >= 0 && token < a.V && parent >= 0 && parent < i) {
              const Row r = row_at<E>(a, q0 + parent);
              px = Prob<E>::one(r.p, token);
              if (r.q) qx = Prob<E>::one(r.q, token);
            }
          }
          continue;
        }
        const int from = __ffs(hit) - 1, child = window + from;
        const int x = __shfl_sync(~0u, token, from);
        const float ux = __shfl_sync(~0u, u, from);
        float p = __shfl_sync(~0u, px, from), q = __shfl_sync(~0u, qx, from);
        if (x < 0 || x >= a.V) {
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
        if (!in_range(p)) p = 0.f, bad = true;
        if (!in_range(q)) q = 0.f, bad = true;
        bool yes;
        double left = 0.0;
        if (w.k == 0) {  // u q < p, exactly: the product is t + e
          const float t = ux * q, e = fmaf(ux, q, -t);
          yes = t < p || (t == p && e < 0.f);
        } else {
          left = p;
          if (a.draft_probs) {
            left = fmax(p - q * w.B, 0.0);
          } else {
            for (int j = 0; j < w.k; ++j)
              if (sh.gone[j] == x) left = 0.0;
          }
          yes = (double)ux * q * w.A < left;
        }
        w.last = child;
        if (yes) {
          if (lane == 0) a.accepted[q0 + w.count] = child;
          w = Walk{child, child, 0, w.count + 1, true, 1.0, 0.0};
        } else {
          if (lane == 0) sh.gone[w.k] = x;
          __syncwarp();
          w.B += w.A;
          // without draft probabilities the next A is known once one sum is
          w.known = w.k > 0 && !a.draft_probs;
          if (w.known) w.A -= rint(left * kUnits) / kUnits;  // (as it was added)
          ++w.k;
        }
      }
      if constexpr (CS > 1) {
        if (!started) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
    } else if constexpr (CS > 1) {
      if (!started) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    started = true;
    everyone();
    const int command = sh.command;
    const float b_hi = sh.b_hi, b_lo = sh.b_lo;
    int k = sh.k;
    const Row r = row_at<E>(a, q0 + sh.row);
    const int per = (r.groups + CS * kWarps - 1) / (CS * kWarps);
    const int g0 = (rank * kWarps + warp) * per, g1 = min(g0 + per, r.groups);
    const bool vec = r.off >= 0;
    const int base = (vec ? r.off : 0) - N;  // first element of group 0
    // A lane takes every 32nd vector of its warp's stretch, kVecs of them a round.
    constexpr int kVecs = kNumbers / N;
    const int rounds = (per + 32 * kVecs - 1) / (32 * kVecs), piece = (rounds + kPieces * kPiece - 1) / (kPieces * kPiece) * kPiece;
    const int limit = base + g1 * N;  // of the stretch
    auto first_of = [&](int round, int v) { return base + (g0 + (round * kVecs + v) * 32 + lane) * N; };
    auto copy = [&](int round) {
      if (round >= rounds) return copy_commit();
      const int first = first_of(round, 0);
      uint4* to = &sh.ring[round % kDepth][0][0][tid];
      const bool q = r.q && k > 0;
      const int last = first - lane * N + (kVecs * 32 - 1) * N;  // the round's last vector
      if (vec && first >= lane * N && last + N <= a.V && last < limit) {
        const uint8_t* from = static_cast<const uint8_t*>(r.p) + (int64_t)first * (16 / N);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) copy16(to + v * kThreads, from + v * 512);
        if (q) {
          from = static_cast<const uint8_t*>(r.q) + (int64_t)first * (16 / N);
#pragma unroll
          for (int v = 0; v < kVecs; ++v) copy16(to + (kNumbers / 4 + v) * kThreads, from + v * 512);
        }
      } else {
#pragma unroll 1
        for (int v = 0; v < kVecs; ++v) {
          const int at = first + v * 32 * N;
          const bool inside = vec && at >= 0 && at + N <= a.V, some = at < limit;
#pragma unroll 1
          for (int z = 0; z < (q ? 2 : 1); ++z) {
            uint4* slot = to + (z * (kNumbers / 4) + v) * kThreads;
            const void* row = z ? r.q : r.p;
            if (some && inside)
              copy16(slot, static_cast<const uint8_t*>(row) + (int64_t)at * (16 / N));
            else
              *slot = some ? load_edge<E>(row, at, a.V) : make_uint4(0, 0, 0, 0);
          }
        }
      }
      copy_commit();
    };
    // A round's numbers from slot z of the ring; where one is outside [0, 2], mended and reported.
    auto numbers = [&](int round, int z, float* f) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) Prob<E>::all(sh.ring[round % kDepth][z][v][tid], f + v * N);
      uint32_t most = 0;  // (as whole numbers: above 2's bits if negative or NaN)
#pragma unroll
      for (int i = 0; i < kNumbers; ++i) most = max(most, __float_as_uint(f[i]));
      if (most > 0x40000000u) {
        float t[kNumbers];
        bool odd = false;
#pragma unroll
        for (int i = 0; i < kNumbers; ++i) t[i] = f[i], odd |= !in_range(f[i]);
        mend<kNumbers>(t);
        bad |= odd;
#pragma unroll
        for (int i = 0; i < kNumbers; ++i) f[i] = t[i];
      }
    };
    // What is left of a round's numbers, as hi + lo: pairs of neighbours.  `how`: nothing rejected, drafts without or
    // with probabilities.
    auto weights = [&](auto how, int round, uint64_t* hi, uint64_t* lo) {
      float p[kNumbers];
      numbers(round, 0, p);
      if constexpr (how == 1) {
        for (int j = 0; j < k; ++j) {
#pragma unroll
          for (int v = 0; v < kVecs; ++v) {
            const uint32_t at = (uint32_t)(sh.gone[j] - first_of(round, v));
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (at == (uint32_t)i) p[v * N + i] = 0.f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kNumbers / 2; ++i) hi[i] = pair2(p[2 * i], p[2 * i + 1]), lo[i] = 0;
      if constexpr (how == 2) {
        float q[kNumbers];
        numbers(round, 1, q);
        const uint64_t bh = pair2(b_hi, b_hi), bl = pair2(b_lo, b_lo), mh = pair2(-b_hi, -b_hi), minus = pair2(-1.f, -1.f);
#pragma unroll
        for (int i = 0; i < kNumbers / 2; ++i) {
          const uint64_t f = pair2(q[2 * i], q[2 * i + 1]), t = mul2(f, mh);  // q B = -t + e
          const uint64_t e = fma2(f, bl, fma2(f, bh, t));
          const uint64_t d = add2(hi[i], t);
          const uint64_t l = fma2(e, minus, add2(fma2(d, minus, hi[i]), t));  // d + l = p - q B, l rounded
          const uint64_t s = add2(d, l);  // and the number next to it: l holds both roundings above, up to 2^-22 where p > 1
          const float2 z = split2(s), y = split2(fma2(fma2(d, minus, s), minus, l));
          hi[i] = pair2(z.x > 0.f ? z.x : 0.f, z.y > 0.f ? z.y : 0.f);
          lo[i] = pair2(z.x > 0.f ? y.x : 0.f, z.y > 0.f ? y.y : 0.f);
        }
      }
    };
    const std::integral_constant<int, 0> plain;
    const std::integral_constant<int, 1> without;
    const std::integral_constant<int, 2> with;
    for (;;) {
      uint64_t whole_sum = 0;
      float size = 0.f;
      auto pass = [&](auto how) {
        uint64_t piece_sum = 0;
        int left = piece, at = 0;
        Levels sum;
        uint32_t count = 0;
#pragma unroll 1
        for (int i = 0; i < kDepth; ++i) copy(i);
#pragma unroll 1
        for (int round = 0; round < rounds; ++round) {
          copy_wait<kDepth - 1>();
          uint64_t hi[kNumbers / 2], lo[kNumbers / 2];
          weights(how, round, hi, lo);
#pragma unroll
          for (int i = 0; i < kNumbers / 2; ++i) sum.add(hi[i], lo[i]);
          count += kNumbers;
          copy(round + kDepth);
          if ((round + 1) % kPiece != 0 && round + 1 != rounds) continue;
          sum.finish(count);
          // (in two parts each: a thread's 64 numbers stay below 2^29 and 2^28 in size, a warp's could pass 32 bits)
          const uint32_t up = __reduce_add_sync(~0u, sum.a >> 12), low = __reduce_add_sync(~0u, sum.a & 0xFFFu);
          const int32_t b = (int32_t)sum.b;
          const int32_t b_up = __reduce_add_sync(~0u, b >> 12), b_low = __reduce_add_sync(~0u, b & 0xFFF);
          piece_sum += ((((uint64_t)up << 12) + low) << (kUnit - 22)) + (((int64_t)b_up << 12) + b_low);
          size += (float)up * 0x1p-10f;
          sum = Levels();
          count = 0;
          left -= kPiece;
          if (left == 0 || round + 1 == rounds) {
            if (lane == 0) sh.piece[warp][at] = piece_sum;
            whole_sum += piece_sum;
            piece_sum = 0;
            left = piece;
            ++at;
          }
        }
      };
      if (k == 0)
        pass(plain);
      else if (!r.q)
        pass(without);
      else
        pass(with);
      copy_wait<0>();
      if (lane == 0) sh.warp_sum[warp] = whole_sum, sh.warp_size[warp] = size;
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
      uint64_t total = 0, before = 0;
      float whole = 0.f;
#pragma unroll 1
      for (int i = 0; i < CS; ++i) {
        if (i == rank) before = total;
        total += sh.cta_sum[i];
        whole += sh.cta_size[i];
      }
      if (whole > 8.f) {
        total = 0;
        bad = true;
      }
      if (command == kSum) {
        w.A = (double)total / kUnits;
        w.known = true;
        break;
      }
      if (total == 0 && k > 0) {  // nothing is left of a: the draw is from p
        k = 0;
        everyone();
        continue;
      }
      if (total == 0) {
        bad = true;
        if (rank == 0 && tid == 0) a.next_token[b] = -1;
        break;
      }
      // floor(u total): a whole running sum is above u total where it is above that
      const uint32_t bits = __float_as_uint(below_one(a.draw_u[b]));
      const int shift = 150 - max((int)(bits >> 23), 1);
      const uint32_t m = (bits & 0x7FFFFFu) | (bits >> 23 ? 0x800000u : 0u);
      const uint64_t point = shift >= 128 ? 0 : (uint64_t)(((unsigned __int128)total * m) >> shift);
      if (point < before || point - before >= sh.cta_sum[rank]) break;
      uint64_t left = point - before;
      bool mine = true;
#pragma unroll 1
      for (int i = 0; i < warp && mine; ++i) {
        mine = left >= sh.warp_sum[i];
        left -= sh.warp_sum[i];
      }
      if (!mine || left >= sh.warp_sum[warp]) break;
      // this warp's stretch holds the point
      int round = 0;
      for (int i = 0; left >= sh.piece[warp][i]; ++i) {  // (their sum is above it)
        left -= sh.piece[warp][i];
        round += piece;
      }
      bool found = false;
#pragma unroll 1
      for (; !found && round < rounds; ++round) {
        copy(round);
        copy_wait<0>();
        uint64_t hi[kNumbers / 2], lo[kNumbers / 2];
        if (k == 0)
          weights(plain, round, hi, lo);
        else if (!r.q)
          weights(without, round, hi, lo);
        else
          weights(with, round, hi, lo);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
          if (found) break;
          Levels sum;
#pragma unroll
          for (int i = 0; i < N / 2; ++i) sum.add(hi[v * (N / 2) + i], lo[v * (N / 2) + i]);
          sum.finish(N);
          const uint64_t own = sum.value();
          uint64_t upto = own;
#pragma unroll 1
          for (int o = 1; o < 32; o <<= 1) {
            const uint64_t y = __shfl_up_sync(~0u, upto, o);
            if (lane >= o) upto += y;
          }
          const uint32_t hit = __ballot_sync(~0u, upto > left);
          if (hit && lane == __ffs(hit) - 1) {
            uint64_t c = upto - own;
            int next = -1;
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const float2 x = split2(hi[(v * N + i) / 2]), y = split2(lo[(v * N + i) / 2]);
              Levels one;
              one.add(pair2(i & 1 ? x.y : x.x, 0.f), pair2(i & 1 ? y.y : y.x, 0.f));
              one.finish(2);
              c += one.value();
              if (next < 0 && c > left) next = first_of(round, v) + i;
            }
            a.next_token[b] = next;
          }
          found = hit != 0;
          left -= __shfl_sync(~0u, upto, 31);
        }
      }
      break;
    }
    if (command == kDraw) break;
    everyone();  // (the sums have been read)
  }
  if (rank == 0 && warp == 0) {
    if (lane == 0) a.n_accepted[b] = w.count;
    for (int i = w.count + lane; i < n; i += 32) a.accepted[q0 + i] = -1;
  }
  if (a.status) {
    const uint32_t said = (bad ? FT_ST_NAN : 0u) | (bad_token ? FT_ST_BAD_TOKEN : 0u) | (bad_tree ? FT_ST_BAD_TREE : 0u);
    if (said) atomicOr(a.status, said);
  }
}

template <typename E, int CS>
void configure(const ft_verify_args& a, cudaStream_t st, cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr) {
  cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3((unsigned)a.num_reqs * CS);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CS;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CS > 1 ? 2 : 1;
}

template <typename E, int CS>
cudaError_t prepare() {
  static thread_local int configured = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured == dev) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(verify_drafts_kernel<E, CS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
  if (e == cudaSuccess && CS > 8)
    e = cudaFuncSetAttribute(verify_drafts_kernel<E, CS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) configured = dev;
  return e;
}

template <typename E, int CS>
cudaError_t launch(const ft_verify_args& a, cudaStream_t st) {
  if (const cudaError_t e = prepare<E, CS>()) return e;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  configure<E, CS>(a, st, cfg, attr);
  return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<E, CS>, a);
}

// Clusters of kMaxCluster CTAs that run at once (0 where there are none).
template <typename E>
int room(const ft_verify_args& a) {
  static thread_local int known_dev = -1, clusters = 0;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != known_dev) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    configure<E, kMaxCluster>(a, nullptr, cfg, attr);
    if (prepare<E, kMaxCluster>() != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&clusters, verify_drafts_kernel<E, kMaxCluster>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      clusters = 0;
    }
    known_dev = dev;
  }
  return clusters;
}

template <typename E>
cudaError_t launch_cs(const ft_verify_args& a, cudaStream_t st) {
  // As many CTAs a request as run at once, while a lane has more than one vector of a row.  A cluster lies in one GPC, and
  // of 16 CTAs there is room for 14; a few more wait for the first to end.  Three batches each of trees over 131072 fp32
  // entries, in us: 16 requests 18, 17, 25 with 16 CTAs and 24, 21, 31 with 8; 17 requests 25, 37, 37 and 22, 36, 39; 18
  // requests 24, 29, 35 and 24, 33, 33.  Rows of 50021 16-bit entries: 14 requests 16, 14, 13 and 16, 14, 14; 16 requests
  // 16, 17, 19 and 14, 14, 15; 37 requests 23 and 18.
  int cs = 1;
  while (cs < kMaxCluster && a.V / Prob<E>::N / cs > kThreads &&
         (cs < 8 ? (int64_t)a.num_reqs * cs * 2 <= (int64_t)sm_count() * kResident : a.num_reqs * 4ll <= room<E>(a) * 5ll))
    cs *= 2;
  switch (cs) {
    case 1: return launch<E, 1>(a, st);
    case 2: return launch<E, 2>(a, st);
    case 4: return launch<E, 4>(a, st);
    case 8: return launch<E, 8>(a, st);
    default: return launch<E, 16>(a, st);
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
