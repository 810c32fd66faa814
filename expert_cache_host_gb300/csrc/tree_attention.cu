// Attention of a step's tokens over the paged cache (ft_tree_attention) on the
// fifth-generation tensor cores.
//
// For one request and key head, the rows that read the same keys are the
// step's tokens times the query heads of the group (r = token * G + head).  A
// tile is 128 rows x 128 keys: S = Q K^T, p = 2^(c S - m) with the running row
// maximum m (c = scale log2 e), O += P V.  S, P and O live in tensor memory; P
// takes S's place as packed 16-bit pairs and is the A operand of the second
// product from there.
//
// What bounds it: K and V are read once from HBM and serve 128 or 256 rows;
// a few rows leave it HBM-bound (a 128-key tile is 64 KB at D = 128, about 3000
// cycles of one SM's share, its two products about 1000), 256 rows and more
// bring the products level with the reads.  So:
//  - a work item (request, key head, block of up to 256 rows) is cut along the
//    keys wherever the machine's even share ends: every CTA takes the same
//    number of key tiles of the flattened list of items, whatever the lengths;
//    an item cut over several CTAs leaves partial outputs in the workspace and
//    the last CTA to finish joins them in order.
//  - two streams of (S, softmax, O) per CTA: while the four softmax warps of
//    one work, the tensor cores run the other's products.  With more than 128
//    rows the streams are the two row tiles and share every K and V tile; with
//    fewer they are the even and the odd key tiles, joined at the end.
//  - K and V come through one ring of 128-key stages filled by TMA, a box per
//    page (or per half of a head's 128 numbers), running ahead across items.
//
// Warps 0-3 and 4-7: softmax of stream 0 and 1 (a thread per row); warp 8: TMA;
// warp 9: tensor-core issue.  All waits are bounded (FT_ST_TIMEOUT).
//
// Keys a row does not see get S = -inf by selection, so their bits do not
// matter.  For V the product would turn 0 x NaN into NaN: rows of V past the
// request's keys, of absent pages, and non-finite numbers of new tokens are
// replaced by zero in shared memory before the product (only tiles that can
// hold such rows are looked at); a row that does see a non-finite new value
// adds it in the epilogue.
#include <math_constants.h>

#include "attn_side.h"
#include "tcgen05.h"

namespace ft {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int KT = 128;        // keys of a tile
constexpr int kThreads = 384;  // 8 softmax warps, TMA, issue, two that only fill their warpgroup
// Registers a thread: 168 at launch; the softmax warpgroups hold a row of S (128) and take the third's.
constexpr int kSoftmaxRegs = 224, kOtherRegs = 56;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * 168, "the split must fit the launch's registers");
constexpr int kProducer = 8, kIssuer = 9;  // warps
// The running maximum may lag behind by this much (in log2 units) before O is
// rescaled: p <= 2^8 stays exact in fp32 sums and in range of f16.
constexpr float kLag = 8.f;

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;            // 128-byte column blocks of a row
  static constexpr int TILE = 128 * D * 2;         // bytes of a Q, K or V tile
  static constexpr int BLOCK = 128 * 128;          // bytes of one column block of a tile
  static constexpr int NST = D == 128 ? 5 : 12;    // ring stages: what a CTA's 227 KB hold beside two Q tiles
  static constexpr int SMEM = 2 * TILE + NST * TILE;  // and Shared
};

struct Args {
  ft_attn_args a;
  int log2_page, G, tpt;  // query heads per key head; tokens per 128-row tile
  float c;                // |scale| log2 e
  bool neg;               // scale < 0
  float* part_o;          // [2 grid][256][D]
  float* part_lse;        // [2 grid][256], log2 units
  unsigned int* count;    // [grid] parts done of the item that begins to be cut at this CTA
};

__host__ __device__ constexpr size_t count_bytes(int grid) { return ((size_t)grid * 4 + 255) / 256 * 256; }
__host__ __device__ constexpr size_t lse_bytes(int grid) { return (size_t)grid * 2 * 256 * 4; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Requests' sizes and the walk over this CTA's work.
struct Req {
  int q0, n, ctx, tiles, blocks;
};
__device__ __forceinline__ Req request(const Args& g, int b) {
  Req r;
  r.q0 = g.a.q_start[b];
  r.n = max(min(g.a.q_start[b + 1], g.a.max_tokens) - r.q0, 0);
  r.ctx = max(g.a.ctx_len[b], 0);
  r.tiles = (int)(((long long)r.ctx + r.n + KT - 1) / KT);
  r.blocks = (r.n + 2 * g.tpt - 1) / (2 * g.tpt);
  return r;
}
__device__ __forceinline__ long long units(const Args& g, int b) {
  const Req r = request(g, b);
  return (long long)r.tiles * r.blocks * g.a.cache.kv_heads;
}

struct Walk {
  long long at, end, total;  // in tiles of the flattened list
  int grid;                  // CTAs that share it
  int b, h, blk, tile;       // the next tile
  Req r;
  // the current item
  int t0, t1;                // its tiles [t0, t1) are this CTA's
  int rows;                  // valid rows of the block (tokens * G)
  bool pair;                 // two row tiles
  __device__ __forceinline__ bool next(const Args& g) {
    if (at >= end) return false;
    while (tile >= r.tiles || r.n == 0) {
      tile = 0;
      if (r.n == 0 || ++blk >= r.blocks) {
        blk = 0;
        if (r.n == 0 || ++h >= g.a.cache.kv_heads) {
          h = 0;
          r = request(g, ++b);
        }
      }
    }
    t0 = tile;
    t1 = (int)min((long long)r.tiles, tile + (end - at));
    at += t1 - t0;
    tile = t1;
    const int tok = min(r.n - blk * 2 * g.tpt, 2 * g.tpt);
    rows = tok * g.G;
    pair = tok > g.tpt;
    return true;
  }
  // key tiles of a stream, and a stream's j-th
  __device__ __forceinline__ int count(int s) const { return pair ? t1 - t0 : (t1 - t0 + 1 - s) / 2; }
  __device__ __forceinline__ int tile_of(int s, int j) const { return pair ? t0 + j : t0 + 2 * j + s; }
};

struct Shared {
  uint64_t full[12], empty[12];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], o_full[2];
  uint32_t tmem;
  uint32_t pages[12];      // per stage: which pages of the tile are there
  uint32_t s_pages[2];     // of the K tile behind a stream's S
  uint32_t nonfinite[2];   // per item parity: a new token's values held inf or NaN
  long long red[kThreads / 32];
  long long at, total;     // start of this CTA's share: units into request b
  int b;
  int last;                // this CTA joins the parts
  float lse[2][128], inv[2][128];  // a row's streams: log2 sum with its maximum, 1 / sum
};

// The 32 bits of a token's visibility that begin at new token `off` (bits
// before token 0 are the context: set).
__device__ __forceinline__ uint32_t mask_bits(const Args& g, const uint32_t* row, int i, int off) {
  if (off <= -32) return ~0u;
  auto word = [&](int w) -> uint32_t {
    if (row) return w < g.a.mask_words ? row[w] : 0u;
    const int left = i + 1 - 32 * w;  // without a mask: tokens 0 .. i
    return left <= 0 ? 0u : left >= 32 ? ~0u : (1u << left) - 1;
  };
  if (off < 0) return (word(0) << -off) | ((1u << -off) - 1);
  const int w = off >> 5, s = off & 31;
  return s ? (word(w) >> s) | (word(w + 1) << (32 - s)) : word(w);
}

// Which of the 32 keys from key0 on row i of the request sees.
__device__ __forceinline__ uint32_t visible(const Args& g, const Req& r, const uint32_t* row, int i, int key0, int w,
                                            uint32_t pages) {
  const int off = key0 - r.ctx, left = r.n - off;
  if (left <= 0) return 0;
  uint32_t v = mask_bits(g, row, i, off);
  if (left < 32) v &= (1u << left) - 1;
  // pages of the tile, in groups of min(page_size, 32) keys
  const int per = 1 << g.log2_page;
  if (per >= 32) {
    if (!(pages >> ((w * 32) >> g.log2_page) & 1)) v = 0;
  } else {
    for (int k = 0; k < 32; k += per)
      if (!(pages >> ((w * 32 + k) >> g.log2_page) & 1)) v &= ~(((1u << per) - 1) << k);
  }
  return v;
}

template <typename E, int D>
__device__ __forceinline__ bool any_nonfinite(uint32_t w) {
  constexpr uint32_t x = Elem<E>::kDtype == FT_DTYPE_BF16 ? 0x7F80u : 0x7C00u;
  return (w & x) == x || (w >> 16 & x) == x;
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Args g) {
  using C = Cfg<D>;
  constexpr int NST = C::NST;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sq = smem;
  uint8_t* ring = sq + 2 * C::TILE;
  Shared& sh = *reinterpret_cast<Shared*>(smem + C::SMEM);
  const ft_attn_args& a = g.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.s_full[s], 2);  // the products and the issuer's word on the pages
      mbar_init(&sh.p_full[s], 4);
      mbar_init(&sh.o_full[s], 2);
      sh.nonfinite[s] = 0;
    }
    mbar_init_fence();
  }
  if (warp == kIssuer) tmem_alloc(&sh.tmem, 512);

  // Total work and where this CTA's share begins.
  Walk wk;
  {
    long long mine = 0;
    for (int b = tid; b < a.num_reqs; b += kThreads) mine += units(g, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(~0u, mine, o);
    if (lane == 0) sh.red[warp] = mine;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kThreads / 32; ++w) total += sh.red[w];
    wk.total = total;
    wk.grid = (int)min((long long)gridDim.x, total);
    const int c = blockIdx.x;
    wk.at = c < wk.grid ? total * c / wk.grid : 0;
    wk.end = c < wk.grid ? total * (c + 1) / wk.grid : 0;
    long long base = 0;
    for (int b0 = 0; b0 < a.num_reqs && base <= wk.at; b0 += kThreads) {
      const long long u = b0 + tid < a.num_reqs ? units(g, b0 + tid) : 0;
      long long x = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) sh.red[warp] = x;
      __syncthreads();
      long long before = base, all = 0;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sh.red[w];
        all += sh.red[w];
      }
      const long long first = before + x - u;
      if (wk.at >= first && wk.at < first + u) {
        sh.b = b0 + tid;
        sh.at = wk.at - first;
      }
      base += all;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wk.b = sh.b;
    wk.h = wk.blk = wk.tile = 0;
    if (wk.at < wk.end) {
      wk.r = request(g, wk.b);
      const long long per_head = (long long)wk.r.tiles * wk.r.blocks;
      wk.h = (int)(sh.at / per_head);
      const long long in_head = sh.at - wk.h * per_head;
      wk.blk = (int)(in_head / wk.r.tiles);
      wk.tile = (int)(in_head - (long long)wk.blk * wk.r.tiles);
    }
  }
  const uint32_t tmem = sh.tmem;
  bool late = false;

  if (warp >= kProducer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kProducer) {
    const int per_tile = g.log2_page >= 7 ? 1 : KT >> g.log2_page;  // pages of a tile
    const int box_rows = KT / per_tile;
    const uint32_t box_bytes = (uint32_t)box_rows * 128 * C::HALVES;
    uint32_t it = 0;
    int item = 0;
    for (; wk.next(g); ++item) {
      if (item > 0 && !mbar_wait(&sh.q_empty, (uint32_t)((item - 1) & 1), late)) late = true;
      const int q_tiles = wk.pair ? 2 : 1;
      if (lane == 0) {
        mbar_expect_tx(&sh.q_full, (uint32_t)(q_tiles * g.tpt * g.G * D * 2));
        for (int s = 0; s < q_tiles; ++s)
          for (int hf = 0; hf < C::HALVES; ++hf)
            tensor_g2s_3d(sq + s * C::TILE + hf * C::BLOCK, &map_q, hf * 64, wk.h * g.G,
                          wk.r.q0 + (wk.blk * 2 + s) * g.tpt, &sh.q_full);
      }
      const int32_t* row = a.block_table + (int64_t)wk.b * a.table_width;
      const int len = wk.r.ctx + wk.r.n;
      auto page_of = [&](int t) {
        const long long col = (((long long)t * KT) >> g.log2_page) + lane;
        return lane < per_tile && t < wk.t1 && col < a.table_width ? row[col] : -1;
      };
      int page = page_of(wk.t0);
      for (int t = wk.t0; t < wk.t1; ++t) {
        const int next_page = page_of(t + 1);
        const int key = t * KT + lane * box_rows;  // first key of this lane's page
        const bool used = lane < per_tile && key < len;
        const bool there = used && page >= 0 && page < a.cache.num_pages;
        if (used && !there && a.status) atomicOr(a.status, FT_ST_BAD_SLOT);
        const uint32_t pages = __ballot_sync(~0u, there);
        const int y = g.log2_page >= 7 ? (t * KT) & ((1 << g.log2_page) - 1) : 0;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const int st = it % NST;
          if (it >= NST && !mbar_wait(&sh.empty[st], (uint32_t)(((it / NST) - 1) & 1), late)) late = true;
          uint8_t* dst = ring + st * C::TILE + lane * box_rows * 128;
          if (lane == 0) {
            sh.pages[st] = pages;
            mbar_expect_tx(&sh.full[st], (uint32_t)__popc(pages) * box_bytes);
          }
          __syncwarp();
          if (there) {
#pragma unroll
            for (int hf = 0; hf < C::HALVES; ++hf)
              tensor_g2s_4d(dst + hf * C::BLOCK, kv ? &map_v : &map_k, hf * 64, y, wk.h, page, &sh.full[st]);
          }
        }
        page = next_page;
      }
    }
  } else if (warp == kIssuer) {
    constexpr bool BF = Elem<E>::kDtype == FT_DTYPE_BF16;
    constexpr uint32_t id_qk = umma_idesc_f16(BF, 128, KT, false), id_pv = umma_idesc_f16(BF, 128, D, true);
    uint32_t base = 0;     // ring position of the item's first stage
    uint32_t done[2] = {};  // tiles of each stream so far (barrier phases)
    int item = 0;
    for (; wk.next(g); ++item) {
      if (lane == 0) sh.nonfinite[item & 1] = 0;
      if (!mbar_wait(&sh.q_full, (uint32_t)(item & 1), late)) late = true;
      tc_fence_after();
      const int cnt[2] = {wk.count(0), wk.count(1)};
      auto qk = [&](int s, int j) {
        const uint32_t pos = base + 2 * (wk.tile_of(s, j) - wk.t0);
        const int st = pos % NST;
        if (!mbar_wait(&sh.full[st], (pos / NST) & 1, late)) late = true;
        tc_fence_after();
        if (lane == 0) {
          sh.s_pages[s] = sh.pages[st];
          mbar_arrive_cta(&sh.s_full[s]);
          const uint32_t qa = smem_u32(sq + (wk.pair ? s : 0) * C::TILE), ka = smem_u32(ring + st * C::TILE);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * C::BLOCK + (kk & 3) * 32;
            umma_bf16(tmem + 256 + s * 128, umma_desc_sw128(qa + off), umma_desc_sw128(ka + off), id_qk, kk ? 1u : 0u);
          }
          umma_commit(&sh.s_full[s]);
          if (!wk.pair || s == 1) umma_commit(&sh.empty[st]);
        }
        __syncwarp();
      };
      auto pv = [&](int s, int j) {
        const int t = wk.tile_of(s, j);
        const uint32_t pos = base + 2 * (t - wk.t0) + 1;
        const int st = pos % NST;
        if (!mbar_wait(&sh.full[st], (pos / NST) & 1, late)) late = true;
        uint8_t* v = ring + st * C::TILE;
        if (!wk.pair || s == 0) {
          // rows of V that must not reach the product
          const uint32_t pages = sh.pages[st];
          const int per_tile = g.log2_page >= 7 ? 1 : KT >> g.log2_page;
          const int left = wk.r.ctx + wk.r.n - t * KT;  // keys of the request in this tile
          const bool whole = left >= KT && pages == (per_tile == 32 ? ~0u : (1u << per_tile) - 1);
          const int fresh = max(wk.r.ctx - t * KT, 0);  // first row of a new token
          if (!whole || fresh < KT) {
            const int row_shift = min(g.log2_page, 7);
            uint32_t found = 0;
            for (int x = lane; x < 128 * 8 * C::HALVES; x += 32) {
              const int row = (x >> 3) & 127, hf = x >> 10;
              uint4* p = reinterpret_cast<uint4*>(v + hf * C::BLOCK + row * 128 + (x & 7) * 16);
              if (row >= left || !(pages >> (row >> row_shift) & 1)) {
                *p = make_uint4(0, 0, 0, 0);
              } else if (row >= fresh) {
                uint4 u = *p;
                uint32_t* e = reinterpret_cast<uint32_t*>(&u);
                bool hit = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if (any_nonfinite<E, D>(e[i])) {
                    constexpr uint32_t inf = BF ? 0x7F80u : 0x7C00u;
                    if ((e[i] & inf) == inf) e[i] &= 0xFFFF0000u;
                    if ((e[i] >> 16 & inf) == inf) e[i] &= 0xFFFFu;
                    hit = true;
                  }
                }
                if (hit) {
                  *p = u;
                  found = 1;
                }
              }
            }
            proxy_fence_writes();
            if (__any_sync(~0u, found) && lane == 0) sh.nonfinite[item & 1] = 1;
            __syncwarp();
          }
        }
        if (!mbar_wait(&sh.p_full[s], (done[s] + j) & 1, late)) late = true;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t va = smem_u32(v);
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk)
            umma_f16_ta(tmem + s * 128, tmem + 256 + s * 128 + kk * 8, umma_desc_sw128_mn(va + kk * 2048, C::BLOCK),
                        id_pv, (j | kk) ? 1u : 0u);
          if (!wk.pair || s == 1) umma_commit(&sh.empty[st]);
          if (j + 1 == cnt[s]) {
            umma_commit(&sh.o_full[s]);
            mbar_arrive_cta(&sh.o_full[s]);
          }
        }
        __syncwarp();
      };
      for (int s = 0; s < 2; ++s)
        if (cnt[s] > 0) qk(s, 0);
      bool q_done = false;
      for (int j = 0; j < cnt[0]; ++j) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (j < cnt[s]) {
            pv(s, j);
            if (j + 1 < cnt[s]) qk(s, j + 1);
          }
        }
        if (!q_done && j + 2 >= cnt[0]) {  // every product with Q has been issued
          q_done = true;
          if (lane == 0) umma_commit(&sh.q_empty);
        }
      }
      done[0] += cnt[0];
      done[1] += cnt[1];
      base += 2 * (wk.t1 - wk.t0);
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int s = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + 256 + s * 128 + lanes, t_o = tmem + lanes;
    uint32_t tiles_done = 0, items_of_stream = 0;
    for (int item = 0; wk.next(g); ++item) {
      const Req& r = wk.r;
      const int first_tok = (wk.blk * 2 + (wk.pair ? s : 0)) * g.tpt;
      const int tok = row / g.G, i = first_tok + tok;
      const bool valid = tok < g.tpt && i < r.n;
      const bool warp_live = __any_sync(~0u, valid);
      const uint32_t* mrow = a.mask ? a.mask + (int64_t)(r.q0 + (valid ? i : 0)) * a.mask_words : nullptr;
      const int cnt = wk.count(s);
      float m = -CUDART_INF_F, l = 0.f;
      for (int j = 0; j < cnt; ++j, ++tiles_done) {
        if (!mbar_wait(&sh.s_full[s], tiles_done & 1, late)) late = true;
        tc_fence_after();
        const int t = wk.tile_of(s, j);
        const uint32_t pages = sh.s_pages[s];
        if (warp_live) {
          uint32_t u[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_async(t_s + c * 32, u + c * 32);
          tmem_wait_ld();
          float* x = reinterpret_cast<float*>(u);
          if (g.neg) {
#pragma unroll
            for (int c = 0; c < 128; ++c) x[c] = -x[c];
          }
          const int per_tile = g.log2_page >= 7 ? 1 : KT >> g.log2_page;
          if ((t + 1) * KT > r.ctx || pages != (1u << per_tile) - 1) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t vis = valid ? visible(g, r, mrow, i, t * KT + w * 32, w, pages) : 0u;
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(vis >> c & 1)) x[w * 32 + c] = -CUDART_INF_F;
            }
          }
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int c = 4; c < 128; ++c) mx[c & 3] = fmaxf(mx[c & 3], x[c]);
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const bool grow = (top - m) * g.c > kLag || m == -CUDART_INF_F;  // also the first tile with a key
          if (__any_sync(~0u, grow)) {
            const float f = grow ? (top == -CUDART_INF_F ? 1.f : ex2((m - top) * g.c)) : 1.f;
            if (j > 0) {
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32_async(t_o + s * 128 + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st32(t_o + s * 128 + c, o);
              }
            }
            l *= f;
            if (grow) m = top;
          }
          const float ref = m == -CUDART_INF_F ? 0.f : m * g.c;
          float sum[4] = {};
#pragma unroll
          for (int c = 0; c < 128; c += 2) {
            const float p0 = ex2(fmaf(x[c], g.c, -ref)), p1 = ex2(fmaf(x[c + 1], g.c, -ref));
            sum[(c >> 1) & 3] += p0 + p1;
            u[c >> 1] = Elem<E>::pack(p0, p1);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_st32(t_s, u);
          tmem_st32(t_s + 32, u + 32);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&sh.p_full[s]);
      }
      if (cnt > 0) {
        if (!mbar_wait(&sh.o_full[s], items_of_stream & 1, late)) late = true;
        ++items_of_stream;
        tc_fence_after();
      }
      const bool nonfinite = cnt > 0 && sh.nonfinite[item & 1];
      // Rows' output: with a row tile per stream the thread's own; else the two
      // streams' halves of the keys joined, each warpgroup half of the columns.
      float w0 = s == 0 ? 1.f : 0.f, w1 = 1.f - w0, lse = l > 0.f || l != l ? m * g.c + log2f(l) : -CUDART_INF_F;
      int c0 = 0, c1 = D;
      float inv = lse == -CUDART_INF_F ? 0.f : 1.f / l;
      bool use0 = s == 0, use1 = s == 1;
      if (!wk.pair) {
        sh.lse[s][row] = cnt > 0 ? lse : -CUDART_INF_F;
        sh.inv[s][row] = inv;
        bar_sync(1, 256);
        const float l0 = sh.lse[0][row], l1 = sh.lse[1][row];
        float top = fmaxf(l0, l1);
        if (l0 != l0 || l1 != l1) top = CUDART_NAN_F;
        if (top == -CUDART_INF_F) {
          w0 = w1 = 0.f;
          lse = top;
        } else {
          const float e0 = ex2(l0 - top), e1 = ex2(l1 - top);
          lse = top + log2f(e0 + e1);
          w0 = e0 / (e0 + e1) * sh.inv[0][row];
          w1 = e1 / (e0 + e1) * sh.inv[1][row];
        }
        use0 = l0 != -CUDART_INF_F;
        use1 = l1 != -CUDART_INF_F;
        c0 = s * (D / 2);
        c1 = c0 + D / 2;
        inv = 1.f;
      }
      use0 = use0 && wk.count(0) > 0;
      use1 = use1 && wk.count(1) > 0;
      const bool whole = wk.t0 == 0 && wk.t1 == r.tiles;
      const int slot = blockIdx.x * 2 + (wk.t0 == 0 ? 1 : 0);
      const int part_row = slot * 256 + (wk.pair ? s * 128 : 0) + row;
      const int h0 = wk.h * g.G + row % g.G;
      if (warp_live) {
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          uint32_t o[32], o2[32];
          tmem_ld32_async(t_o + (wk.pair && s ? 128 : 0) + c, o);
          if (!wk.pair) tmem_ld32_async(t_o + 128 + c, o2);
          tmem_wait_ld();
          float y[32];
          if (wk.pair) {
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = inv == 0.f ? 0.f : __uint_as_float(o[k]) * inv;
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              y[k] = (use0 ? __uint_as_float(o[k]) * w0 : 0.f) + (use1 ? __uint_as_float(o2[k]) * w1 : 0.f);
          }
          if (nonfinite && valid) {
            // new tokens' infinities and NaN that this row sees
            for (int key = max(r.ctx, wk.t0 * KT); key < min(r.ctx + r.n, wk.t1 * KT); ++key) {
              const int jn = key - r.ctx;
              if (!(mask_bits(g, mrow, i, jn) & 1)) continue;
              const long long col = key >> g.log2_page;
              const int pg = col < a.table_width ? a.block_table[(int64_t)wk.b * a.table_width + col] : -1;
              if (pg < 0 || pg >= a.cache.num_pages) continue;
              const uint16_t* vr = static_cast<const uint16_t*>(a.cache.v) + pg * a.cache.v_page_stride +
                                   (key & ((1 << g.log2_page) - 1)) * a.cache.v_token_stride +
                                   wk.h * a.cache.v_head_stride + c;
              for (int k = 0; k < 32; ++k) {
                const float f = Elem<E>::unpack(vr[k]).x;
                if (!(f - f == 0.f)) {
#pragma unroll
                  for (int z = 0; z < 32; ++z)
                    if (z == k) y[z] += f;
                }
              }
            }
          }
          if (valid) {
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (int64_t)(r.q0 + i) * a.out_stride +
                                                    (int64_t)h0 * D + c);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                dst[k] = make_uint4(Elem<E>::pack(y[8 * k], y[8 * k + 1]), Elem<E>::pack(y[8 * k + 2], y[8 * k + 3]),
                                    Elem<E>::pack(y[8 * k + 4], y[8 * k + 5]), Elem<E>::pack(y[8 * k + 6], y[8 * k + 7]));
            } else {
              float4* dst = reinterpret_cast<float4*>(g.part_o + (int64_t)part_row * D + c);
#pragma unroll
              for (int k = 0; k < 8; ++k) dst[k] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
            }
          }
        }
      }
      if (valid && (wk.pair || s == 0)) {
        if (!whole)
          g.part_lse[part_row] = lse;
        else if (a.lse)
          a.lse[(int64_t)(r.q0 + i) * a.q_heads + h0] = lse * kLn2;
      }
      tc_fence_before();
      if (!whole) {
        // The CTAs that share the item: the one with its first tile counts.
        const long long start = wk.at - wk.t1, G64 = wk.grid;  // the item's first unit
        const int ca = (int)(((start + 1) * G64 - 1) / wk.total), cb = (int)(((start + r.tiles) * G64 - 1) / wk.total);
        __threadfence();
        bar_sync(1, 256);
        if (tid == 0) {
          const unsigned before = atomicAdd(&g.count[ca], 1u);
          sh.last = before == (unsigned)(cb - ca);
          if (sh.last) g.count[ca] = 0;
          __threadfence();
        }
        bar_sync(1, 256);
        if (sh.last) {
          constexpr int LPR = D / 4;  // lanes per row
          const int col = (tid % LPR) * 4;
          const int tile_rows = g.tpt * g.G;
          for (int x = tid / LPR; x < wk.rows; x += 256 / LPR) {
            const int tile_s = x >= tile_rows ? 1 : 0, rr = x - tile_s * tile_rows;
            const int prow = tile_s * 128 + rr;
            float top = -CUDART_INF_F;
            bool nan = false;
            for (int c = ca; c <= cb; ++c) {
              const float v = __ldcg(&g.part_lse[(c * 2 + (c == ca ? 1 : 0)) * 256 + prow]);
              nan |= v != v;
              top = fmaxf(top, v);
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
            if (nan) top = CUDART_NAN_F;
            if (top != -CUDART_INF_F) {
#pragma unroll 4
              for (int c = ca; c <= cb; ++c) {
                const int pr = (c * 2 + (c == ca ? 1 : 0)) * 256 + prow;
                const float e = ex2(__ldcg(&g.part_lse[pr]) - top);
                const float4 o = __ldcg(reinterpret_cast<const float4*>(g.part_o + (int64_t)pr * D + col));
                if (e != 0.f) {
                  sum += e;
                  acc.x = fmaf(e, o.x, acc.x), acc.y = fmaf(e, o.y, acc.y);
                  acc.z = fmaf(e, o.z, acc.z), acc.w = fmaf(e, o.w, acc.w);
                }
              }
            }
            const float iv = top == -CUDART_INF_F ? 0.f : 1.f / sum;
            const int ti = wk.blk * 2 * g.tpt + tile_s * g.tpt + rr / g.G, hh = wk.h * g.G + rr % g.G;
            uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (int64_t)(r.q0 + ti) * a.out_stride +
                                                  (int64_t)hh * D + col);
            *dst = make_uint2(Elem<E>::pack(acc.x * iv, acc.y * iv), Elem<E>::pack(acc.z * iv, acc.w * iv));
            if (a.lse && col == 0)
              a.lse[(int64_t)(r.q0 + ti) * a.q_heads + hh] =
                  top == -CUDART_INF_F ? top : (top + log2f(sum)) * kLn2;
          }
        }
      }
      // both warpgroups have read O (and the joined rows' numbers) before either goes on
      bar_sync(1, 256);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
  if (late && a.status) atomicOr(a.status, FT_ST_TIMEOUT);
}

int check(const ft_attn_args& a) {
  if (int rc = check_kv_cache(a.cache, false)) return rc;
  if (a.max_tokens < 0 || a.num_reqs < 0 || a.q_heads < 1 || a.table_width < 0 || a.mask_words < 0)
    return record_error(FT_E_ARG, "max_tokens, num_reqs, table_width and mask_words must not be negative, q_heads positive");
  if (a.q_heads % a.cache.kv_heads) return record_error(FT_E_ARG, "q_heads must be a multiple of kv_heads");
  if (a.q_heads / a.cache.kv_heads > 128) return record_error(FT_E_UNSUPPORTED, "more than 128 query heads to a key head");
  return FT_OK;
}

uint64_t workspace(int grid, int D) { return count_bytes(grid) + lse_bytes(grid) + (uint64_t)grid * 2 * 256 * D * 4; }

bool cache_map(CUtensorMap* map, void* base, const ft_kv_cache& c, int64_t page, int64_t token, int64_t head, char* msg,
               size_t len) {
  const uint64_t dims[4] = {(uint64_t)c.head_dim, (uint64_t)c.page_size, (uint64_t)c.kv_heads, (uint64_t)c.num_pages};
  const uint64_t strides[3] = {(uint64_t)token * 2, (uint64_t)(c.kv_heads > 1 ? head : c.head_dim) * 2,
                               (uint64_t)(c.num_pages > 1 ? page : c.head_dim) * 2};
  const uint32_t box[4] = {64, (uint32_t)(c.page_size < KT ? c.page_size : KT), 1, 1};
  return encode_tensor_map(map, c.dtype == FT_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                           4, base, dims, strides, box, msg, len, true);
}

template <typename E, int D>
int launch(const Args& g, int grid, cudaStream_t st) {
  using C = Cfg<D>;
  const ft_attn_args& a = g.a;
  const ft_kv_cache& c = a.cache;
  CUtensorMap mq, mk, mv;
  char msg[128] = "";
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.q_heads, (uint64_t)a.max_tokens};
  const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)(a.max_tokens > 1 ? a.q_stride : (int64_t)a.q_heads * D) * 2};
  const uint32_t box[3] = {64, (uint32_t)g.G, (uint32_t)g.tpt};
  if (!encode_tensor_map(&mq, Elem<E>::kDtype == FT_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                         3, const_cast<void*>(a.q), dims, strides, box, msg, sizeof(msg), true) ||
      !cache_map(&mk, c.k, c, c.k_page_stride, c.k_token_stride, c.k_head_stride, msg, sizeof(msg)) ||
      !cache_map(&mv, c.v, c, c.v_page_stride, c.v_token_stride, c.v_head_stride, msg, sizeof(msg)))
    return record_error(FT_E_CUDA, "%s", msg);
  static thread_local int configured = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured != dev) {
    const cudaError_t e =
        cudaFuncSetAttribute(tree_attention_kernel<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(C::SMEM + sizeof(Shared)));
    if (e != cudaSuccess) return record_error(FT_E_CUDA, "attention setup failed: %s", cudaGetErrorString(e));
    configured = dev;
  }
  tree_attention_kernel<E, D><<<grid, kThreads, C::SMEM + sizeof(Shared), st>>>(mq, mk, mv, g);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return record_error(FT_E_CUDA, "attention launch failed: %s", cudaGetErrorString(e));
  return FT_OK;
}

}  // namespace
}  // namespace ft

extern "C" int ft_tree_attention_workspace(const ft_attn_args* args, uint64_t* bytes) {
  using namespace ft;
  if (!args || !bytes) return record_error(FT_E_ARG, "null pointer");
  if (int rc = check(*args)) return rc;
  *bytes = workspace(sm_count(), args->cache.head_dim);
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
  const int grid = sm_count(), D = a.cache.head_dim;
  const uint64_t need = workspace(grid, D);
  if (a.workspace_bytes < need)
    return record_error(FT_E_ARG, "workspace of %llu bytes, %llu needed", (unsigned long long)a.workspace_bytes,
                        (unsigned long long)need);
  Args g{};
  g.a = a;
  while ((1 << g.log2_page) < a.cache.page_size) ++g.log2_page;
  g.G = a.q_heads / a.cache.kv_heads;
  g.tpt = 128 / g.G;
  g.neg = a.scale < 0.f;
  // a scale of 0 keeps seen (0) and unseen (-inf) scores apart
  const float c = (g.neg ? -a.scale : a.scale) * kLog2e;
  g.c = c > 1e-30f ? c : 1e-30f;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  g.count = reinterpret_cast<unsigned int*>(ws);
  g.part_lse = reinterpret_cast<float*>(ws + count_bytes(grid));
  g.part_o = reinterpret_cast<float*>(ws + count_bytes(grid) + lse_bytes(grid));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.cache.dtype == FT_DTYPE_BF16)
    return D == 128 ? launch<__nv_bfloat16, 128>(g, grid, st) : launch<__nv_bfloat16, 64>(g, grid, st);
  return D == 128 ? launch<__half, 128>(g, grid, st) : launch<__half, 64>(g, grid, st);
}
