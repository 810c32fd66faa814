// Attention over the 8-bit paged cache where a request has few rows (new tokens
// times the query heads of a key head: 16 at most), single tokens above all.
//
// Keys and values are read once for a handful of rows, so HBM bounds it and
// everything else has to stay out of its way: 128 keys of a head are 32 KB at D =
// 128, 0.75 us of one SM's share.  Tensor-core instructions with 128 rows would
// need the codes as 16-bit numbers in shared memory (twice the bytes written and
// read again); instead a warp takes 16 keys at a time from shared memory into
// registers, where one instruction turns two codes into f16, as the operand with
// 16 rows of m16n8k16, and the few query rows are the operand with 8:
//   S^T = K Q^T [16 keys x 8 rows], O^T += V^T P^T [D x 8 rows]
// The order of the head's numbers within a product is free, so a lane takes 16
// contiguous codes of a key at a time and Q's fragments follow suit; P^T is
// transposed within the warp.
//
// Scales stay out of the products: 16 keys lie in one block, so a chunk has one
// scale for its keys, which the scores take, and one for its values, which the
// probabilities take.  With X = s 2^ek, row maximum M and row offset mo:
//   p = 2^(c (X - M)), l += p          and      P = 2^(c (X - M) + ev - mo + 11)
// P in f16, where mo follows the maximum of c (X - M) + ev, so that a value's
// weight is held relative to the largest weight times scale.  Queries are f16 too,
// bf16 ones times a power of two of their row.  The largest lies in [2^10, 2^11)
// then, where f16 holds all 8 bits of a bf16 number from 2^-17 on: numbers below
// 2^-27 of the row's largest are rounded to multiples of at most 2^-34 of it.
//
// A CTA's eight warps take the eight chunks of a 128-key tile, each with a ring of
// its own (TMA) and no barrier of the CTA before an item's end, where they are
// joined.  All waits are bounded, as in tree_attention.cuh.
//
// 64 single tokens over 16384 keys, 32/4 heads of 128, 1.08 GB: 174 us = 6.2 TB/s;
// over 100..16384 keys, 0.5 GB: 90 us = 5.5 TB/s; one over 4096: 10.3 us, latency.
// With 16 rows (64 heads) 231 us: 8 warps of an SM instead of 16, for the registers.
#pragma once

#include "tree_attention.cuh"

namespace ft {
namespace kv8_few {

using tree_attention::Args;
using tree_attention::Cut;
using tree_attention::Deal;
using tree_attention::Held;
using tree_attention::kLn2;
using tree_attention::KT;
using tree_attention::Req;
using tree_attention::uniform;
using tree_attention::Walk;

constexpr int kWarps = 8, kThreads = kWarps * 32, kChunk = 16;
constexpr int kRows = 16;  // of a part
constexpr float kUp = 11.f, kLagP = 4.f, kLagL = 8.f;  // P <= 2^15, p <= 2^8

template <int D, int NB>
struct Cfg {
  static constexpr int R = 8 * NB;                        // rows
  static constexpr int CTAS = NB == 1 || D == 64 ? 2 : 1;  // of an SM: what the registers allow
  static constexpr int HALF = kChunk * D;                 // bytes of a chunk's keys or values
  // Two chunks a warp: with three, 128 KB of an SM in flight, 64 requests of 16384 keys took 184 us in place of 174 (and 95
  // in place of 89 of the ragged ones).
  static constexpr int STAGES = 2;
  static constexpr int RING = kWarps * STAGES * 2 * HALF;
  static constexpr int LINE = D + 4;                      // floats of a row's output: rows 2 t4 apart by 8 banks
  static constexpr int JOIN = kWarps * R * LINE * 4;      // the warps' outputs, in the ring's place
  static constexpr int SMEM = RING > JOIN ? RING : JOIN;  // and Shared
};

template <int R, int S>
struct Shared {
  uint64_t full[kWarps][S];
  long long red[kWarps];
  Walk<true> start;
  float m[kWarps][R], l[kWarps][R], mo[kWarps][R];
  float f[kWarps][R];               // a warp's weight in the row
  float most[R], sum[R], norm[R];   // the row's maximum and sum, and what its output is multiplied by, twice
};

__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Four codes as f16: the lower two, the upper two.
__device__ __forceinline__ void halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Where a row's 16-byte piece lies in its chunk (the swizzle of D bytes).  The
// lanes that read together (keys: two rows, every second or every piece; values:
// every second row, two pieces) meet in no bank at D = 128, values' in twos at 64.
template <int D>
__device__ __forceinline__ uint32_t place(int row, int piece) {
  if constexpr (D == 128) return row * 128 + ((piece ^ (row & 7)) << 4);
  return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}

template <typename E, int D, int NB>
__global__ void __launch_bounds__(kThreads, (Cfg<D, NB>::CTAS)) few_rows_kernel(const __grid_constant__ CUtensorMap map_k,
                                                                                     const __grid_constant__ CUtensorMap map_v,
                                                                                     const __grid_constant__ Args g) {
  using C = Cfg<D, NB>;
  constexpr int R = C::R, S = C::STAGES, KS = D / 16, MT = D / 16;  // k steps of K Q^T, row tiles of V^T
  constexpr bool BF = Elem<E>::kDtype == FT_DTYPE_BF16;
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared<R, S>& sh = *reinterpret_cast<Shared<R, S>*>(smem + C::SMEM);
  const ft_attn_args& a = g.a;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31, gid = lane >> 2, t4 = lane & 3;
  if (lane < S) mbar_init(&sh.full[warp][lane], 1);
  mbar_init_fence();
  if (tid < 2) tree_attention::prefetch_map(tid ? &map_v : &map_k);
  pdl_wait();
  pdl_trigger();
  long long lo = 0;
  Deal deal(0, 1);
  tree_attention::schedule<true, kThreads>(g, sh.red, sh.start, lo, deal);
  __syncthreads();
  Walk<true> wk = sh.start;
  const int share = wk.left;
  bool has_cut = false, late = false;
  uint32_t parity = 0;  // a bit per stage: of its next filling
  uint8_t* const ring = smem + warp * S * 2 * C::HALF;
  const int page_mask = (1 << g.log2_page) - 1;
  // This lane's pieces of a chunk: of keys gid (and 8 rows on, gid + 8), of values in rows 2 t4 (and 1, 8, 9 on).
  uint32_t k_at[D / 64], v_at[2];
#pragma unroll
  for (int k = 0; k < D / 64; ++k) k_at[k] = place<D>(gid, D == 128 ? 2 * t4 + k : t4);
#pragma unroll
  for (int k = 0; k < 2; ++k)
    v_at[k] = C::HALF + (D == 128 ? place<D>(2 * t4 + k, gid) : place<D>(2 * t4 + k, gid >> 1) + (gid & 1) * 8);
  constexpr uint32_t kOn = 8 * D;  // 8 rows on, in the same places of the swizzle

  while (wk.next(g)) {
    const Req& r = wk.r;
    const int keys = r.ctx + r.n, rows = r.n * g.G, tiles = wk.t1 - wk.t0;
    const int32_t* table = a.block_table + (int64_t)wk.b * a.table_width;
    // Queries, as the lane's numbers come in K's: D / 4 from D / 4 t4 on (loaded before the pages are known).
    uint4 qw[NB][D / 32];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = nb * 8 + gid, i = row / g.G;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) qw[nb][k] = make_uint4(0, 0, 0, 0);
      if (row < rows) {
        const uint16_t* q = static_cast<const uint16_t*>(a.q) + (r.q0 + i) * a.q_stride + (int64_t)(wk.h * g.G + row - i * g.G) * D;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) qw[nb][k] = *reinterpret_cast<const uint4*>(q + t4 * (D / 4) + k * 8);
      }
    }

    // A window of 32 tiles: lane i has the page of the warp's chunk of tile `window` + i, and its scale bytes (or that
    // there is none).  The next window's are fetched on the way through this one, the last one's bytes kept for the
    // chunks that are still to be read.
    constexpr uint32_t kNone = 1u << 16;
    int window = wk.t0, window_read = wk.t0;
    auto page_at = [&](int first) {  // of tile first + lane; -1: none
      if (first + lane >= wk.t1) return -1;
      const int key0 = (first + lane) * KT + warp * kChunk, col = key0 >> g.log2_page;
      if (key0 >= keys) return -1;
      const int pg = col < a.table_width ? table[col] : -1;
      if (pg >= 0 && pg < a.cache.num_pages) return pg;
      if (a.status) atomicOr(a.status, FT_ST_BAD_SLOT);
      return -1;
    };
    auto bytes_at = [&](int first, int pg) -> uint32_t {
      if (pg < 0) return kNone;
      const int64_t at = tree_attention::scale_index(g, pg, ((first + lane) * KT + warp * kChunk) & page_mask, wk.h);
      return g.k_scale[at] | (uint32_t)g.v_scale[at] << 8;
    };
    int page = page_at(wk.t0), page_next = -1;
    uint32_t bytes = bytes_at(wk.t0, page), bytes_next = kNone;
    // The warp's chunk of tile t on its way into stage st.
    auto issue = [&](int t, int st) {
      if (t >= wk.t1) return;
      if (t == window + 16) page_next = page_at(window + 32);
      if (t == window + 24) bytes_next = bytes_at(window + 32, page_next);
      if (t == window + 32) window = t, page = page_next;
      const int pg = __shfl_sync(~0u, page, t - window), row0 = (t * KT + warp * kChunk) & page_mask;
      if (pg < 0 || late) return;
      if (lane == 0) {
        mbar_expect_tx(&sh.full[warp][st], 2 * C::HALF);
        tensor_g2s_4d(ring + st * 2 * C::HALF, &map_k, 0, row0, wk.h, pg, &sh.full[warp][st]);
        tensor_g2s_4d(ring + st * 2 * C::HALF + C::HALF, &map_v, 0, row0, wk.h, pg, &sh.full[warp][st]);
      }
    };
#pragma unroll
    for (int k = 0; k < S; ++k) issue(wk.t0 + k, k);

    uint32_t qf[NB][KS][2];
    int qe[NB];  // q = qf * 2^-qe
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      uint32_t u[D / 8];
#pragma unroll
      for (int k = 0; k < D / 32; ++k) u[4 * k] = qw[nb][k].x, u[4 * k + 1] = qw[nb][k].y, u[4 * k + 2] = qw[nb][k].z, u[4 * k + 3] = qw[nb][k].w;
      qe[nb] = 0;
      if constexpr (BF) {
        uint32_t two = 0;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) two = max_abs2<E>(two, u[k]);
        two &= 0x7FFF7FFFu;
        uint32_t most = max(two & 0xFFFFu, two >> 16);  // the largest number's bits
        if (most >= 0x7F80u) {                          // (of the finite ones)
          most = 0;
#pragma unroll 1
          for (int k = 0; k < D / 4; ++k) {
            const int row = nb * 8 + gid, i = row / g.G;
            const uint32_t x = static_cast<const uint16_t*>(a.q)[(r.q0 + i) * a.q_stride +
                                                                (int64_t)(wk.h * g.G + row - i * g.G) * D + t4 * (D / 4) + k] & 0x7FFFu;
            if (x < 0x7F80u) most = max(most, x);
          }
        }
        most = max(most, __shfl_xor_sync(~0u, most, 1));
        most = max(most, __shfl_xor_sync(~0u, most, 2));
        qe[nb] = most ? 137 - (int)max(most >> 7, 1u) : 0;  // the largest becomes 2^10 ..
        const float f1 = exp2i(qe[nb] / 2), f2 = exp2i(qe[nb] - qe[nb] / 2);
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const float2 y = Elem<E>::unpack(u[k]);
          u[k] = Elem<__half>::pack(y.x * f1 * f2, y.y * f1 * f2);
        }
      }
      if (g.neg) {
#pragma unroll
        for (int k = 0; k < D / 8; ++k) u[k] ^= 0x80008000u;
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) qf[nb][k][0] = u[2 * k], qf[nb][k][1] = u[2 * k + 1];
    }
    // This thread's rows of the products, 2 t4 and 2 t4 + 1 of every eight: their queries' exponents, and which new
    // tokens they see (16 at most).
    float rf[NB][2];
    uint32_t vis[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        rf[nb][j] = exp2i(-__shfl_sync(~0u, qe[nb], (2 * t4 + j) * 4));
        const int row = nb * 8 + 2 * t4 + j, i = row / g.G;
        vis[nb][j] = 0;
        if (row < rows)
          vis[nb][j] = (a.mask ? a.mask[(int64_t)(r.q0 + i) * a.mask_words] : (2u << i) - 1) & ((1u << r.n) - 1);
      }
    }

    // A row's maximum and offset as they are and (0 where there is none yet) as they are used.
    float M[NB][2], mo[NB][2], l[NB][2], Mr[NB][2], up[NB][2];
    float o[MT][NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int j = 0; j < 2; ++j) M[nb][j] = mo[nb][j] = -CUDART_INF_F, l[nb][j] = Mr[nb][j] = 0.f, up[nb][j] = kUp;
    }
#pragma unroll
    for (int k = 0; k < MT; ++k)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int z = 0; z < 4; ++z) o[k][nb][z] = 0.f;

    int st = 0;
#pragma unroll 1
    for (int n = 0; n < tiles; ++n) {
      const int t = wk.t0 + n, key0 = t * KT + warp * kChunk;
      if (t == window_read + 32) window_read = t, bytes = bytes_next;
      const uint32_t scales = __shfl_sync(~0u, bytes, t - window_read);
      if (!(scales & kNone)) {
        if (__any_sync(~0u, !mbar_wait(&sh.full[warp][st], parity >> st & 1, late))) late = true;
        parity ^= 1u << st;
        const uint8_t* kc = ring + st * 2 * C::HALF;
        // scores of keys gid and gid + 8
        float x[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int z = 0; z < 4; ++z) x[nb][z] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          const uint4 p = *reinterpret_cast<const uint4*>(kc + k_at[k]);
          const uint4 q = *reinterpret_cast<const uint4*>(kc + kOn + k_at[k]);
          const uint32_t pw[4] = {p.x, p.y, p.z, p.w}, qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a0, a1, a2, a3;
            halves(pw[w], a0, a2);
            halves(qw[w], a1, a3);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma(x[nb], a0, a1, a2, a3, qf[nb][k * 4 + w][0], qf[nb][k * 4 + w][1]);
          }
        }
        const uint32_t ek = scales & 255u, ev = scales >> 8 & 255u;
        const float kf = scale_of(ek), shift = ev == 255u ? 0.f : (float)((int)ev - 127);
        const bool special = key0 + kChunk > r.ctx;  // new keys, or rows past the end
        uint32_t seen[NB][2];                        // the row's keys of the chunk
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float f = ek == 255u ? kf : fminf(kf * rf[nb][j], 3e38f);
            x[nb][j] *= f;
            x[nb][2 + j] *= f;
          }
        }
        if (special) {
          const int off = key0 - r.ctx;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              seen[nb][j] = off < 0 ? vis[nb][j] << -off | ((1u << -off) - 1) : vis[nb][j] >> off;
              if (nb * 8 + 2 * t4 + j >= rows) seen[nb][j] = 0;
              if (!(seen[nb][j] >> gid & 1)) x[nb][j] = -CUDART_INF_F;
              if (!(seen[nb][j] >> (gid + 8) & 1)) x[nb][2 + j] = -CUDART_INF_F;
            }
          }
        }
        float y[NB][4];
        bool grow = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          // (before a row's first key mo is -inf, and any score is above)
          const float most[2] = {fminf(kLagL, mo[nb][0] + (kLagP - shift)), fminf(kLagL, mo[nb][1] + (kLagP - shift))};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            y[nb][z] = (x[nb][z] - Mr[nb][z & 1]) * g.c;
            grow |= y[nb][z] > most[z & 1];
          }
        }
        if (__any_sync(~0u, grow)) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float top = fmaxf(x[nb][j], x[nb][2 + j]);
              top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
              top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
              top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
              const float was = M[nb][j], m = fmaxf(was, top);
              if (m > -CUDART_INF_F) {
                const float down = was == -CUDART_INF_F ? 0.f : (was - m) * g.c;
                const float before = mo[nb][j] + down, now = fmaxf(before, (top - m) * g.c + shift);
                const float f = before == -CUDART_INF_F ? 1.f : ex2(before - now);
                M[nb][j] = Mr[nb][j] = m;
                mo[nb][j] = now;
                up[nb][j] = kUp - (now == -CUDART_INF_F ? 0.f : now);
                l[nb][j] *= ex2(down);
#pragma unroll
                for (int k = 0; k < MT; ++k) o[k][nb][j] *= f, o[k][nb][2 + j] *= f;
              }
              y[nb][j] = (x[nb][j] - Mr[nb][j]) * g.c;
              y[nb][2 + j] = (x[nb][2 + j] - Mr[nb][j]) * g.c;
            }
          }
        }
        uint32_t pf[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float w[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            l[nb][z & 1] += ex2(y[nb][z]);
            // 16 bits are what the product takes; the sum keeps all 32
            w[z] = ex2(y[nb][z] + (shift + up[nb][z & 1]));
          }
          if (ev == 255u) {  // NaN to the rows that see the key
#pragma unroll
            for (int z = 0; z < 4; ++z) w[z] = x[nb][z] == -CUDART_INF_F ? 0.f : CUDART_NAN_F;
          }
          pf[nb][0] = transpose8(Elem<__half>::pack(w[0], w[1]));
          pf[nb][1] = transpose8(Elem<__half>::pack(w[2], w[3]));
        }
        // values of keys 2 t4, 2 t4 + 1 and both + 8: the lane's D / 8 numbers from D / 8 gid on
        uint32_t v[4][D / 32];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const uint8_t* from = kc + (z < 2 ? 0 : kOn) + v_at[z & 1];
          if constexpr (D == 128) {
            const uint4 u = *reinterpret_cast<const uint4*>(from);
            v[z][0] = u.x, v[z][1] = u.y, v[z][2] = u.z, v[z][3] = u.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(from);
            v[z][0] = u.x, v[z][1] = u.y;
          }
        }
        if (special) {
          // NaN codes of new tokens: out of the product (0 x NaN), and into the outputs of the rows that see them
          uint32_t nan = 0;
#pragma unroll
          for (int z = 0; z < 4; ++z)
#pragma unroll
            for (int w = 0; w < D / 32; ++w) nan |= ((v[z][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          if (__any_sync(~0u, nan != 0)) {
#pragma unroll
            for (int z = 0; z < 4; ++z)
#pragma unroll
              for (int w = 0; w < D / 32; ++w)
                v[z][w] &= ~((((v[z][w] & 0x7F7F7F7Fu) + 0x01010101u) >> 7 & 0x01010101u) * 0xFFu);
#pragma unroll 1
            for (int key = 0; key < kChunk; ++key) {
#pragma unroll
              for (int b = 0; b < D / 8; ++b) {
                const int d = gid * (D / 8) + b;
                if ((kc[C::HALF + place<D>(key, d >> 4) + (d & 15)] & 0x7F) != 0x7F) continue;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                  for (int j = 0; j < 2; ++j)
                    if (seen[nb][j] >> key & 1) o[b >> 1][nb][(b & 1) * 2 + j] = CUDART_NAN_F;
              }
            }
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint32_t p0 = __byte_perm(v[0][w], v[1][w], 0x5140), p1 = __byte_perm(v[0][w], v[1][w], 0x7362);
          const uint32_t q0 = __byte_perm(v[2][w], v[3][w], 0x5140), q1 = __byte_perm(v[2][w], v[3][w], 0x7362);
          uint32_t f0[4], f1[4];
          halves(p0, f0[0], f0[1]);
          halves(q0, f0[2], f0[3]);
          halves(p1, f1[0], f1[1]);
          halves(q1, f1[2], f1[3]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma(o[2 * w][nb], f0[0], f0[1], f0[2], f0[3], pf[nb][0], pf[nb][1]);
            mma(o[2 * w + 1][nb], f1[0], f1[1], f1[2], f1[3], pf[nb][0], pf[nb][1]);
          }
        }
      }
      proxy_fence_reads();
      __syncwarp();
      issue(t + S, st);
      if (++st == S) st = 0;
    }

    // The warps' sums joined: in the rings' place, [warp][row][pair of a lane][gid][2].
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float s = l[nb][j];
        s += __shfl_xor_sync(~0u, s, 4);
        s += __shfl_xor_sync(~0u, s, 8);
        s += __shfl_xor_sync(~0u, s, 16);
        const int row = nb * 8 + 2 * t4 + j;
        if (gid == 0) sh.m[warp][row] = M[nb][j], sh.l[warp][row] = s, sh.mo[warp][row] = mo[nb][j];
      }
    }
    __syncthreads();  // the rings are empty
    float* const outs = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int k = 0; k < MT; ++k) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float* to = outs + (warp * R + nb * 8 + 2 * t4) * C::LINE + k * 16 + gid * 2;
        *reinterpret_cast<float2*>(to) = make_float2(o[k][nb][0], o[k][nb][2]);
        *reinterpret_cast<float2*>(to + C::LINE) = make_float2(o[k][nb][1], o[k][nb][3]);
      }
    }
    if (tid < R) {
      float m = -CUDART_INF_F, sum = 0.f, off = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sh.m[w][tid]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = sh.m[w][tid];
        const bool some = mw != -CUDART_INF_F || sh.l[w][tid] != 0.f;
        const float down = mw == -CUDART_INF_F ? 0.f : (mw - m) * g.c;
        if (some) sum += sh.l[w][tid] * ex2(down);
        off = fmaxf(off, sh.mo[w][tid] + down);
      }
      if (off == -CUDART_INF_F) off = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = sh.m[w][tid], down = mw == -CUDART_INF_F ? 0.f : (mw - m) * g.c;
        const bool some = mw != -CUDART_INF_F || sh.l[w][tid] != 0.f;
        const float at = sh.mo[w][tid] == -CUDART_INF_F ? 0.f : sh.mo[w][tid] + down - off;
        sh.f[w][tid] = some ? ex2(at) : -1.f;  // (-1: nothing to add)
      }
      sh.most[tid] = m;
      sh.sum[tid] = sum;
      sh.norm[tid] = ex2(0.5f * (off - kUp));  // (its square may be below what fp32 holds)
    }
    __syncthreads();
    const bool whole = wk.t0 == 0 && wk.t1 == r.tiles;
    const int slot = blockIdx.x * 2 + (wk.t0 == 0 ? 1 : 0);
    for (int z = tid; z < rows * (D / 4); z += kThreads) {
      const int row = z / (D / 4), quad = z % (D / 4);
      float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = sh.f[w][row];
        const float4 x = *reinterpret_cast<const float4*>(outs + (w * R + row) * C::LINE + quad * 4);
        if (f == -1.f) continue;
        y[0] += f * x.x, y[1] += f * x.y, y[2] += f * x.z, y[3] += f * x.w;
      }
      const float sum = sh.sum[row], norm = sh.norm[row];
      const bool some = sum > 0.f || sum != sum;
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = some ? y[k] * norm / sum * norm : 0.f;
      const int i = row / g.G, head = wk.h * g.G + row - i * g.G;
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // two neighbours of one lane, and of the next
        const int d = (quad % 4 * 2 + k) * (D / 8) + quad / 4 * 2;
        if (whole)
          *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + (r.q0 + i) * a.out_stride + (int64_t)head * D + d) =
              Elem<E>::pack(y[2 * k], y[2 * k + 1]);
        else
          reinterpret_cast<float2*>(g.part_o + ((int64_t)slot * (D / 4) + d / 4) * kRows + row)[d / 2 % 2] =
              make_float2(y[2 * k], y[2 * k + 1]);
      }
      if (quad == 0) {
        if (!whole)
          g.part_ml[slot * kRows + row] =
              make_float2(some ? sh.most[row] : -CUDART_INF_F, sum * (Held<E>::kUp == 0.f ? 1.f : 2048.f));
        else if (a.lse)
          a.lse[(int64_t)(r.q0 + i) * a.q_heads + head] = some ? (sh.most[row] * g.c + log2f(sum)) * kLn2 : -CUDART_INF_F;
      }
    }
    if (!whole && wk.t0 == 0) {
      has_cut = true;
      if (tid == 0) {
        // the CTA that owns the first unit of the item's last tile
        const long long it = lo + (share - wk.left) - wk.unit + (long long)(r.tiles - 1) * wk.weight();
        g.cut[blockIdx.x] = Cut{deal.owner(it) - (int)blockIdx.x + 1, rows, r.q0, wk.h};
      }
    }
    proxy_fence_reads();
    late = __syncthreads_or(late);  // the outputs have been read
  }
  if (tid == 0 && !has_cut) g.cut[blockIdx.x].parts = 0;
  if (late) {
    // Every copy has been waited for unless a wait ran out; those still in flight get kDrainNs.
    for (const uint64_t t0 = global_ns(); global_ns() - t0 < tree_attention::kDrainNs;) __nanosleep(1000);
    if (tid == 0 && a.status) atomicOr(a.status, FT_ST_TIMEOUT);
  }
}

// (L2 fetches a row and no more: the head beside it is another CTA's, and with 256 bytes 64 requests of 16384 keys took
// 244 us in place of 177)
inline bool chunk_map(CUtensorMap* map, void* base, const ft_kv_cache& c, int64_t page, int64_t token, int64_t head, char* msg,
                      size_t len) {
  const uint64_t dims[4] = {(uint64_t)c.head_dim, (uint64_t)c.page_size, (uint64_t)c.kv_heads, (uint64_t)c.num_pages};
  const uint64_t strides[3] = {(uint64_t)token, (uint64_t)(c.kv_heads > 1 ? head : c.head_dim),
                               (uint64_t)(c.num_pages > 1 ? page : c.head_dim)};
  const uint32_t box[4] = {(uint32_t)c.head_dim, kChunk, 1, 1};
  return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box, msg, len, c.head_dim, c.head_dim);
}

template <typename E, int D, int NB>
int launch(const Args& g, int grid, cudaStream_t st) {
  using C = Cfg<D, NB>;
  constexpr int smem = C::SMEM + (int)sizeof(Shared<C::R, C::STAGES>);
  static_assert(smem * C::CTAS <= 227 * 1024, "the CTAs of an SM must fit its shared memory");
  static_assert(Held<__half>::kUp == 11.f && Held<__nv_bfloat16>::kUp == 0.f, "parts' sums are scaled by 2^kUp");
  const ft_kv_cache& c = g.a.cache;
  CUtensorMap mk, mv;
  char msg[128] = "";
  if (!chunk_map(&mk, c.k, c, c.k_page_stride, c.k_token_stride, c.k_head_stride, msg, sizeof(msg)) ||
      !chunk_map(&mv, c.v, c, c.v_page_stride, c.v_token_stride, c.v_head_stride, msg, sizeof(msg)))
    return record_error(FT_E_CUDA, "%s", msg);
  static thread_local int configured = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured != dev) {
    const cudaError_t e = cudaFuncSetAttribute(few_rows_kernel<E, D, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return record_error(FT_E_CUDA, "attention setup failed: %s", cudaGetErrorString(e));
    configured = dev;
  }
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(cfg, attr, dim3(grid), dim3(kThreads), smem, st);
  cudaError_t e = cudaLaunchKernelEx(&cfg, few_rows_kernel<E, D, NB>, mk, mv, g);
  if (e == cudaSuccess) e = tree_attention::launch_join<E, D, kRows>(g, grid, st);
  if (e != cudaSuccess) return record_error(FT_E_CUDA, "attention launch failed: %s", cudaGetErrorString(e));
  return FT_OK;
}

}  // namespace kv8_few
}  // namespace ft
