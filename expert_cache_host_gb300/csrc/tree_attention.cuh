// Attention of a step's tokens over the paged cache on the fifth-generation tensor
// cores: ft_tree_attention, and (Q8) ft_kv8_attention where a request has more than
// a few rows.
//
// For one request and key head, the rows that read the same keys are the
// step's tokens times the query heads of the group (r = token * G + head).  A
// tile is 128 rows x 128 keys: S = Q K^T, p = 2^(c S - m) with the running row
// maximum m (c = scale log2 e; f16 holds p times 2^11), O += P V.  S, P and O live in tensor memory; P
// takes S's place as packed 16-bit pairs and is the A operand of the second
// product from there.
//
// What bounds it: K and V are read once from HBM and serve 128 or 256 rows.  A
// 128-key tile is 64 KB at D = 128, 1.49 us of one SM's share of HBM; its two
// products take 1031 cycles per 128 rows.  So few rows leave it HBM-bound (32
// single tokens over 16K keys, 1.07 GB: 168 us = 6.4 TB/s).  With 256 rows the
// products take as long as the reads, and the chain from Q K^T over the softmax
// (1320 cycles a row tile) to P V longer than either: 32 trees of 24..32 tokens
// over 8K..32K keys, 1.37 GB, 0.30 TFLOP, take 248..257 us at best and
// 271..289 us one call after another under the power cap (285 us at 1612 MHz: 4.8
// TB/s, 1045 TFLOP/s), 2 us a tile where the reads need 1.49 us and the products
// 1.28 us.  So:
//  - a work item (request, key head, block of up to 256 rows) is cut along the
//    keys wherever the machine's even share ends: every CTA takes the same
//    amount of the flattened list of items, whatever the lengths (24 requests of
//    100..8192 keys, 160 MB: 40 us, of which 6 the join's); an item cut over
//    several CTAs leaves partial outputs in the workspace, which a second small
//    kernel joins in order.
//  - two streams of (S, softmax, O) per CTA: while the four softmax warps of
//    one work, the tensor cores run the other's products.  With more than 128
//    rows the streams are the two row tiles and share every K and V tile; with
//    fewer they are the even and the odd key tiles, joined at the end.
//  - K and V come through one ring of 128-key stages filled by TMA, a box per
//    page (or per half of a head's 128 numbers), running ahead across items.
//
// Warps 0-3 and 4-7: softmax of stream 0 and 1 (a thread per row); warp 8: TMA;
// warp 9: tensor-core issue; warp 10: V rows (below).  All waits are bounded:
// where one runs out (FT_ST_TIMEOUT) nothing more is loaded, and the CTA ends a
// while after all its warps have come to theirs, with no copy or product in flight.
//
// Keys a row does not see get S = -inf by selection, so their bits do not
// matter.  For V the product would turn 0 x NaN into NaN: rows of V past the
// request's keys, of absent pages, and non-finite numbers of new tokens are
// replaced by zero in shared memory before the product; a row that does see a
// non-finite new value adds it in the epilogue.  Only tiles that can hold such
// rows go through warp 10: their V lands on the stage's `raw` barrier, and the
// warp passes it on to `full`.
//
// Q8: tiles come as 8-bit codes through a ring of their own, and four more warps
// turn them into the 16-bit tiles of the products (code * 2^(e-127), exact but for
// f16's numbers below 2^-14; V's rows are looked over by them too).  The products
// and the conversion, not the bytes, then bound long trees: 32 of 24..32 tokens
// over 8K..32K keys, 0.69 GB, 0.30 TFLOP, take 325..331 us in bf16 and 314..324 in
// f16, where the 16-bit cache takes 254..260.  A tile is written twice and read
// twice in shared memory, 1000 cycles besides the products' 1500, and a warp's 32
// rows of it take 1400 cycles in bf16 and 820 in f16: shifts, permutations and
// 8-bit conversions share one pipe, 2 cycles a warp instruction; f16 takes one such
// conversion for two codes, bf16, for which there is none, 3.3 such instructions
// and 1.3 on the multipliers' pipe.
#pragma once

#include <math_constants.h>

#include <algorithm>
#include <limits>
#include <type_traits>

#include "kv8.h"
#include "tcgen05.h"

namespace ft {
namespace tree_attention {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int KT = 128;        // keys of a tile
constexpr int kProducer = 8, kIssuer = 9, kFixer = 10;  // warps
constexpr int kConverters = 12;                         // Q8: the first of four
// The running maximum m may lag behind by kLag (in log2 units) before O is
// rescaled, and probabilities are held times 2^kUp, p = 2^(c S - m + kUp), so
// that p <= 2^(kLag + kUp).  bf16 has fp32's range.  f16 has a fixed spacing of
// 2^-24 below 2^-14, so its probabilities take the range up to 2^15: those of
// 2^-25 of a row's largest still have all their bits, and 2^-36 is the least
// that is not lost.  (Held as p <= 1, keys of 2^-25 each beside one large score
// vanished from the output: half of it over 16K keys.)
template <typename E>
struct Held;
template <>
struct Held<__nv_bfloat16> {
  static constexpr float kLag = 8.f, kUp = 0.f;
};
template <>
struct Held<__half> {
  static constexpr float kLag = 4.f, kUp = 11.f;
};
// The exponents c x - fl(c m) hold the rounding of c m, and every maximum a row
// has had, in either stream and in every part, has one of its own: up to here
// two of them put a key's weight off by 2^-16 ln 2 at most.  Past it the
// exponents are c (x - m), 128 more subtractions a row and tile: 32 long trees
// 287 us instead of 271, 24 requests 41.7 instead of 40.5.  (With 2^20 in place
// of 256 weights were off by up to 4 %.)
constexpr float kFar = 256.f;

template <int D, bool Q8>
struct Cfg {
  // 8 softmax warps, TMA, issue, V fixer, one that only fills its warpgroup; Q8: four converters.
  static constexpr int THREADS = Q8 ? 512 : 384;
  // Registers a thread: 168 (Q8: 128) at launch; the softmax warpgroups hold a row of S (128) and take the others'.
  static constexpr int SOFTMAX_REGS = Q8 ? 208 : 224, OTHER_REGS = Q8 ? 48 : 56;
  static_assert(2 * SOFTMAX_REGS + (THREADS / 128 - 2) * OTHER_REGS <= THREADS / 128 * (Q8 ? 128 : 168),
                "the split must fit the launch's registers");
  static constexpr int HALVES = D / 64;            // 128-byte column blocks of a row
  static constexpr int TILE = 128 * D * 2;         // bytes of a Q, K or V tile
  static constexpr int BLOCK = 128 * 128;          // bytes of one column block of a tile
  static constexpr int TILE8 = 128 * D;            // bytes of an 8-bit tile
  // Ring stages: what a CTA's 227 KB hold beside two Q tiles; Q8: of converted tiles, and of tiles as they come.
  static constexpr int NST = Q8 ? (D == 128 ? 3 : 6) : D == 128 ? 5 : 12;
  static constexpr int NST8 = Q8 ? (D == 128 ? 4 : 8) : 0;
  static constexpr int SMEM = 2 * TILE + NST * TILE + NST8 * TILE8;  // and Shared
};

struct Args {
  ft_attn_args a;
  int log2_page, G, tpt;  // query heads per key head; tokens per 128-row tile
  float c;                // |scale| log2 e
  bool neg;               // scale < 0
  float4* part_o;         // [2 grid][2 row tiles][D / 4][128 rows] of 4 outputs: a warp's rows are contiguous
  float2* part_ml;        // [2 grid][256] a part's maximum m and sum l = sum 2^(c (S - m)), times 2^kUp
  struct Cut* cut;        // [grid] the item that begins at this CTA and goes on at the next
  // Q8: the cache's strides are bytes, and
  const uint8_t *k_scale, *v_scale;
  int log2_block, max_new;
  uint32_t sixteen, one;  // as convert_rows wants them
};

// An item cut over several CTAs: parts = 0 where there is none.
struct Cut {
  int parts, rows, token0, h;
};

__host__ __device__ constexpr size_t cut_bytes(int grid) { return ((size_t)grid * sizeof(Cut) + 255) / 256 * 256; }
__host__ __device__ constexpr size_t ml_bytes(int grid, int rows = 256) { return (size_t)grid * 2 * rows * sizeof(float2); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(~0u, x, 0); }
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// A tile costs a CTA this many units: with two row tiles the products and both
// streams' softmax take 2700 cycles, with one 1750 (measured at D = 128; used at
// 64 too, where reads and products are half and the softmax is not).
constexpr int kPairUnits = 3, kSingleUnits = 2;
// An item costs this much besides (its Q, the first tile's way through the
// pipeline, its output), counted after its tiles.  24 requests of 100..8192
// keys: 40.2 us with 6, 41.5 with 3, 47.9 with 0; 40 requests of up to 3001 keys
// and 37 tokens, f16, D = 64: 55.9, 64.4, 71.5.
constexpr int kItemUnits = 6;
// Requests' sizes and the walk over this CTA's work.
struct Req {
  int q0, n, ctx, tiles, blocks;
};
// What copies and products in flight are given after a wait has run out; they take microseconds.
constexpr uint64_t kDrainNs = 100000000;
// Beyond this many keys a tile's end would not fit 31 bits.
constexpr uint32_t kMostKeys = 0x7FFFFFFFu - 2 * KT;
template <bool Q8>
__device__ __forceinline__ Req request(const Args& g, int b) {
  Req r;
  r.q0 = g.a.q_start[b];
  r.n = r.q0 < 0 ? 0 : max(min(g.a.q_start[b + 1], g.a.max_tokens) - r.q0, 0);
  r.ctx = max(g.a.ctx_len[b], 0);
  const uint32_t keys = (uint32_t)r.ctx + r.n;
  r.tiles = (int)((keys + KT - 1) / KT);
  r.blocks = (r.n + 2 * g.tpt - 1) / (2 * g.tpt);
  if (Q8 && r.n > g.max_new) {
    if (g.a.status) atomicOr(g.a.status, FT_ST_NO_ROOM);
    r.n = r.tiles = r.blocks = 0;
  }
  // (a head's units must fit 31 bits too)
  if (keys > kMostKeys || __umulhi((uint32_t)(r.tiles * kPairUnits + kItemUnits), 2u * r.blocks) != 0) {
    if (g.a.status) atomicOr(g.a.status, FT_ST_BAD_SLOT);
    r.n = r.tiles = r.blocks = 0;
  }
  return r;
}
// Units of all but the last block, and of the last, per tile.
__device__ __forceinline__ int last_weight(const Args& g, const Req& r) {
  return r.n - (r.blocks - 1) * 2 * g.tpt > g.tpt ? kPairUnits : kSingleUnits;
}
__device__ __forceinline__ long long head_units(const Args& g, const Req& r) {
  return r.blocks ? (long long)r.tiles * (kPairUnits * (r.blocks - 1) + last_weight(g, r)) + kItemUnits * r.blocks : 0;
}

template <bool Q8>
struct Walk {
  int left;               // units of this CTA's share still to come
  int b, h, blk, unit;    // the next unit: place in its block
  Req r;
  // the current item
  int t0, t1;             // its tiles [t0, t1) are this CTA's: those whose first unit is
  bool pair;              // two row tiles
  __device__ __forceinline__ bool next(const Args& g) {
    for (;;) {
      if (left <= 0) return false;
      pair = r.n - blk * 2 * g.tpt > g.tpt;
      const int size = r.tiles * weight() + kItemUnits;
      if (r.n > 0 && unit < size) {
        const int end = min(size, unit + left);
        t0 = tiles_before(unit);
        t1 = tiles_before(end);
        left -= end - unit;
        unit = end;
        if (t1 > t0) return true;
      } else {
        unit = 0;
        if (++blk >= r.blocks) {
          blk = 0;
          if (r.n == 0 || ++h >= g.a.cache.kv_heads) {
            h = 0;
            r = request<Q8>(g, ++b);
          }
        }
      }
    }
  }
  __device__ __forceinline__ int weight() const { return pair ? kPairUnits : kSingleUnits; }
  // tiles of the block whose first unit lies before `u`
  __device__ __forceinline__ int tiles_before(int u) const {
    return min(r.tiles, pair ? (u + kPairUnits - 1) / kPairUnits : (u + kSingleUnits - 1) / kSingleUnits);
  }
  // key tiles of a stream, and a stream's j-th
  __device__ __forceinline__ int count(int s) const { return pair ? t1 - t0 : (t1 - t0 + 1 - s) / 2; }
  __device__ __forceinline__ int tile_of(int s, int j) const { return pair ? t0 + j : t0 + 2 * j + s; }
};

// a / b.  Below 2^21 through fp32: (a + 1/2) / b is at least 1/(2b) from a whole
// number and the quotient's error is below 2^-22 a / b.  (An integer division is
// some hundred cycles, several in a row at the head of every CTA.)
__device__ __forceinline__ uint32_t quotient(uint32_t a, uint32_t b) {
  return (a | b) < (1u << 21) ? (uint32_t)__fdividef((float)a + 0.5f, (float)b) : a / b;
}

// Units are dealt to `grid` CTAs in order, `per` each and one more to the first `extra`.
struct Deal {
  int per, extra, grid;
  __device__ __forceinline__ Deal(long long total, int ctas) {
    // A share is never less than a tile's units, so every CTA between an item's
    // first and last has a tile of it (the join counts on that).
    const uint32_t t = (uint32_t)min(total, 0x7FFFFFFFll);  // more than 2^31 units: the last CTA takes what is left
    grid = max(1, min(ctas, (int)(t / kPairUnits)));
    per = (int)quotient(t, grid);
    extra = (int)(t - (uint32_t)per * grid);
  }
  __device__ __forceinline__ long long first(int c) const { return (long long)c * per + min(c, extra); }
  __device__ __forceinline__ int owner(long long unit) const {
    const uint32_t u = (uint32_t)min(unit, 0x7FFFFFFFll), wide = (uint32_t)extra * (per + 1);
    const int c = u < wide ? (int)quotient(u, per + 1) : extra + (int)quotient(u - wide, max(per, 1));
    return min(c, grid - 1);
  }
};

template <bool Q8>
struct Shared {
  static constexpr int kStages = Q8 ? 8 : 12, kWarps = Q8 ? 16 : 12;
  uint64_t full[kStages], empty[kStages];
  uint64_t raw[Q8 ? 8 : kStages];  // the stage's V has landed but is not fit for the product yet; Q8: an 8-bit stage has
  uint64_t raw_empty[Q8 ? 8 : 1];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2];  // p_half: P's first 64 keys
  uint32_t tmem;
  uint32_t pages[kStages];          // per stage: which pages of the tile are there
  uint32_t raw_pages[Q8 ? 8 : 1];
  uint8_t raw_scale[Q8 ? 8 : 1][8];  // per 8-bit stage: the scale bytes of its blocks
  uint32_t s_pages[2];     // of the K tile behind a stream's S
  uint32_t nonfinite[4][Q8 ? 4 : 1];  // per item (mod 4): a new token's values held inf or NaN (Q8: of a converter's rows)
  long long red[kWarps];
  Walk<Q8> start;              // where this CTA's share starts
  float m[2][128], l[2][128];  // a row's streams: maximum and sum
};

// Total work and where this CTA's share begins, from inclusive sums of the
// requests' units: by warp 0 where its lanes hold all requests, else over the
// block, kThreads requests at a time.
// (`red`: a number a warp; a barrier has to follow before `start` is read)
template <bool Q8, int kThreads>
__device__ __forceinline__ void schedule(const Args& g, long long* red, Walk<Q8>& start, long long& lo, Deal& deal) {
  const ft_attn_args& a = g.a;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  long long total = 0;  // units of all items
  {
    const int c = blockIdx.x;
    auto share_of = [&] {
      deal = Deal(total, gridDim.x);
      lo = deal.first(c);
      return c >= deal.grid ? 0 : c == deal.grid - 1 ? (int)min(total - lo, 0x7FFFFFFFll) : deal.per + (c < deal.extra);
    };
    // The walk's start, `at` units into request b.
    auto place = [&](Walk<Q8>& w, const Req& r, int b, uint32_t at) {
      const uint32_t per_head = (uint32_t)head_units(g, r), per_block = (uint32_t)r.tiles * kPairUnits + kItemUnits;
      w.b = b;
      w.r = r;
      w.h = (int)quotient(at, per_head);
      const uint32_t in_head = at - w.h * per_head;
      w.blk = min((int)quotient(in_head, per_block), r.blocks - 1);
      w.unit = (int)(in_head - w.blk * per_block);
    };
    Req r{};
    long long u = 0, x = 0;
    auto warp_scan = [&](int b) {
      r = Req{};
      if (b < a.num_reqs) r = request<Q8>(g, b);
      u = head_units(g, r) * a.cache.kv_heads;
      x = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
      }
    };
    if (a.num_reqs <= 32) {
      if (warp == 0) {
        warp_scan(lane);
        total = __shfl_sync(~0u, x, 31);
        const int share = share_of();
        if (share > 0 && lo >= x - u && lo < x) place(start, r, lane, (uint32_t)(lo - (x - u)));
        if (lane == 0) start.left = share;
      }
    } else {
      auto scan = [&](int b0) {
        warp_scan(b0 + tid);
        __syncthreads();
        if (lane == 31) red[warp] = x;
        __syncthreads();
        long long all = 0, before = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
          const long long y = red[w];
          if (w < warp) before += y;
          all += y;
        }
        x += before;
        return all;
      };
      for (int b0 = 0; b0 < a.num_reqs; b0 += kThreads) total += scan(b0);
      const int share = share_of();
      long long base = 0;
      for (int b0 = 0; b0 < a.num_reqs && base <= lo; b0 += kThreads) {
        const long long all = a.num_reqs > kThreads ? scan(b0) : total;
        const long long first = base + x - u;
        if (share > 0 && lo >= first && lo < first + u) place(start, r, b0 + tid, (uint32_t)(lo - first));
        base += all;
      }
      if (tid == 0) start.left = share;
    }
  }
}

// The 32 bits of a token's visibility that begin at new token `off` (bits
// before token 0 are the context: set).  `first`: the row's first two words.
__device__ __forceinline__ uint32_t mask_bits(const Args& g, const uint32_t* row, uint2 first, int i, int off) {
  if (off <= -32) return ~0u;
  auto word = [&](int w) -> uint32_t {
    if (row) return w >= g.a.mask_words ? 0u : w == 0 ? first.x : w == 1 ? first.y : row[w];
    const int left = i + 1 - 32 * w;  // without a mask: tokens 0 .. i
    return left <= 0 ? 0u : left >= 32 ? ~0u : (1u << left) - 1;
  };
  if (off < 0) return (word(0) << -off) | ((1u << -off) - 1);
  const int w = off >> 5, s = off & 31;
  return s ? (word(w) >> s) | (word(w + 1) << (32 - s)) : word(w);
}

// Which of the 32 keys from key0 on row i of the request sees.
__device__ __forceinline__ uint32_t visible(const Args& g, const Req& r, const uint32_t* row, uint2 first, int i, int key0, int w,
                                            uint32_t pages) {
  const int off = key0 - r.ctx, left = r.n - off;
  if (left <= 0) return 0;
  uint32_t v = mask_bits(g, row, first, i, off);
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

// Rows of a V tile that must not reach the product: rows [left, last) past the
// request's keys and rows of absent pages become zero, and so do non-finite
// numbers in the new tokens' rows [fresh, left); returns whether there were any.
// One warp, the tile's rows [from, to).
template <typename E, int HALVES, int BLOCK>
__device__ __forceinline__ uint32_t fix_v(uint8_t* v, int lane, int row_shift, uint32_t pages, int left, int last,
                                          int fresh, int from = 0, int to = KT) {
  constexpr uint32_t x = Elem<E>::kDtype == FT_DTYPE_BF16 ? 0x7F807F80u : 0x7C007C00u;  // both exponents
  const int rows = max(min(left, to), from);
  last = min(last, to);
  fresh = max(fresh, from);
  auto chunk = [&](int row0, int i) {
    return reinterpret_cast<uint4*>(v + (HALVES == 1 ? 0 : ((i >> 3) & 1) * BLOCK) +
                                    (row0 + i / (8 * HALVES)) * 128 + (i & 7) * 16);
  };
  for (int i = lane; i < (last - rows) * 8 * HALVES; i += 32) *chunk(rows, i) = make_uint4(0, 0, 0, 0);
  const uint32_t used = (rows + (1 << row_shift) - 1) >> row_shift;
  if ((pages & ((1u << used) - 1)) != (1u << used) - 1) {
    for (int i = lane + from * 8 * HALVES; i < rows * 8 * HALVES; i += 32)
      if (!(pages >> ((i / (8 * HALVES)) >> row_shift) & 1)) *chunk(0, i) = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }
  bool hit = false;
#pragma unroll 4
  for (int i = lane; i < (rows - fresh) * 8 * HALVES; i += 32) {
    uint4 u = *chunk(fresh, i);
    uint32_t* e = reinterpret_cast<uint32_t*>(&u);
    uint32_t all = 0;  // a half with a zero: that exponent is all ones
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t y = (e[k] & x) ^ x;
      all |= (y - 0x00010001u) & ~y & 0x80008000u;
    }
    if (all) {  // (a borrow from the lower half can raise the upper's flag: looked at exactly here)
      bool bad = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if ((e[k] & x & 0xFFFFu) == (x & 0xFFFFu)) e[k] &= 0xFFFF0000u, bad = true;
        if ((e[k] & x & 0xFFFF0000u) == (x & 0xFFFF0000u)) e[k] &= 0xFFFFu, bad = true;
      }
      if (bad) *chunk(fresh, i) = u;
      hit |= bad;
    }
  }
  proxy_fence_writes();
  return __any_sync(~0u, hit);
}

// The place of a row's scale byte.
__device__ __forceinline__ int64_t scale_index(const Args& g, int page, int in_page, int head) {
  return (((int64_t)page << (g.log2_page - g.log2_block)) + (in_page >> g.log2_block)) * g.a.cache.kv_heads + head;
}

// Rows [from, from + 32) of it, as a call: what few tiles need stays out of the loops' instructions.
template <typename E, int HALVES, int BLOCK>
__device__ __noinline__ uint32_t fix_v_rows(uint8_t* v, int lane, int row_shift, uint32_t pages, int left, int fresh, int from) {
  return fix_v<E, HALVES, BLOCK>(v, lane, row_shift, pages, left, KT, fresh, from, from + 32);
}

// What convert_rows does, for any factor and any code: a lane's, one after another.
template <typename E, int D>
__device__ __noinline__ void convert_unusual(const uint8_t* in, uint8_t* out, uint32_t e_lo, uint32_t e_hi, int half, int lo,
                                             int hi) {
  constexpr int COLS = D / 64;
#pragma unroll 1
  for (int z = 0; z < 4 * COLS * 16; ++z) {
    const int g = z / (COLS * 16), k = z / 16 % COLS, q = z % 16;
    const uint8_t code = in[g * 8 * D + (COLS == 2 ? (half ^ k) * 64 : 0) + q];
    *reinterpret_cast<uint16_t*>(out + g * (8 * 128) + (COLS == 2 ? (half ^ k) * (128 * 128) : 0) + (q < 8 ? lo : hi) + (q & 7) * 2) =
        (uint16_t)Elem<E>::pack(e4m3_value(code) * scale_of(g < 2 ? e_lo : e_hi), 0.f);
  }
}

// One warp: 32 rows of an 8-bit tile (rows of D bytes, one after another) as
// 16-bit numbers code * 2^(e-127) in the 128-byte swizzle layout.  A lane takes
// 16 codes of one of 8 rows at a time; an eighth of the warp passes two rows of
// half their columns each, so that neither the loads nor the stores meet in a
// bank.  The rows lie in two blocks at most: e_lo is the scale byte of the first 16,
// e_hi that of the last 16 (both warp-uniform).
template <typename E, int D>
__device__ __forceinline__ void convert_rows(const uint8_t* src, uint8_t* dst, uint32_t e_lo, uint32_t e_hi, int lane,
                                             uint32_t sixteen, uint32_t one) {
  constexpr int COLS = D / 64;  // passes over 8 rows
  // this lane's row of 8, and its columns in the first pass (in the second the others)
  const int row = D == 128 ? (lane >> 3) * 2 + ((lane >> 2) & 1) : lane >> 2;
  const int half = D == 128 ? (lane >> 2) & 1 : 0, c = lane & 3, x = row & 7;
  const uint8_t* in = src + row * D + c * 16;
  uint8_t* out = dst + row * 128;
  const int lo = ((2 * c) ^ x) * 16, hi = ((2 * c + 1) ^ x) * 16;
  auto load = [&](int g, int k) { return *reinterpret_cast<const uint4*>(in + g * 8 * D + (COLS == 2 ? (half ^ k) * 64 : 0)); };
  uint32_t nan = 0;
  // (rolled, without a branch, and with the unusual in calls: the softmax warps' code fills the instruction cache.  32
  // long trees, bf16: 325 us, with the calls inlined 352, a branch for unusual codes in the loop 386, the loop unrolled
  // twice 391 and four times 430)
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    uint4 v[COLS];
#pragma unroll
    for (int k = 0; k < COLS; ++k) v[k] = load(g, k);
    const uint32_t f = Scaled<E>::factor(g < 2 ? e_lo : e_hi);
#pragma unroll
    for (int k = 0; k < COLS; ++k) {
      uint32_t o[8];
      Scaled<E>::convert(v[k], f, sixteen, one, o, nan);
      uint8_t* to = out + g * (8 * 128) + (COLS == 2 ? (half ^ k) * (128 * 128) : 0);
      *reinterpret_cast<uint4*>(to + lo) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(to + hi) = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
  if (Scaled<E>::fast(e_lo, nan) && Scaled<E>::fast(e_hi, nan)) return;
  convert_unusual<E, D>(in, out, e_lo, e_hi, half, lo, hi);
}

template <typename E, int D, bool Q8>
__global__ void __launch_bounds__(Cfg<D, Q8>::THREADS, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Args g) {
  using C = Cfg<D, Q8>;
  constexpr int NST = C::NST, kThreads = C::THREADS;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sq = smem;
  uint8_t* ring = sq + 2 * C::TILE;
  uint8_t* ring8 = ring + NST * C::TILE;
  Shared<Q8>& sh = *reinterpret_cast<Shared<Q8>*>(smem + C::SMEM);
  const ft_attn_args& a = g.a;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

  if (warp == kIssuer) tmem_alloc(&sh.tmem, 512);
  if (warp == kProducer) {
    if constexpr (Q8) {
      if (lane < C::NST8) {
        mbar_init(&sh.raw[lane], 2);  // the copies, and the scale bytes
        mbar_init(&sh.raw_empty[lane], 4);
      }
    }
    if (lane < NST) {
      mbar_init(&sh.full[lane], Q8 ? 4 : 1);
      mbar_init(&sh.empty[lane], 1);
      if constexpr (!Q8) mbar_init(&sh.raw[lane], 1);
    } else if (lane < NST + 2) {
      const int s = lane - NST;
      mbar_init(&sh.s_full[s], 2);  // the products and the issuer's word on the pages
      mbar_init(&sh.p_half[s], 4);
      mbar_init(&sh.p_full[s], 4);
      mbar_init(&sh.o_full[s], 2);
    } else if (lane == NST + 2) {
      mbar_init(&sh.q_full, 1);
      mbar_init(&sh.q_empty, 1);
    }
    mbar_init_fence();
    if (lane < 3) prefetch_map(lane == 0 ? &map_q : lane == 1 ? &map_k : &map_v);
  }
  // What follows reads what earlier kernels of the stream wrote.
  pdl_wait();
  pdl_trigger();  // the join kernel may be set up; it waits for this grid's end

  long long lo = 0;  // the first unit of this CTA's share (warp 0 knows)
  Deal deal(0, 1);
  schedule<Q8, kThreads>(g, sh.red, sh.start, lo, deal);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  Walk<Q8> wk = sh.start;
  const uint32_t tmem = uniform(sh.tmem);
  bool late = false;

  if (warp >= kProducer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    const int per_tile = g.log2_page >= 7 ? 1 : KT >> g.log2_page;  // pages of a tile
    const int box_rows = KT / per_tile;
    const uint32_t full_pages = (1u << per_tile) - 1;
    // A lane per page of a tile: the page's id, and whether it is there.  Q8: lanes 16 .. 23 and 24 .. 31 have the
    // pages of its blocks.
    auto page_of = [&](int t) {
      long long col = (((long long)t * KT) >> g.log2_page) + lane;
      bool has = lane < per_tile;
      if constexpr (Q8) {
        const int row = (lane & 7) << g.log2_block;
        if (lane >= 16) {
          col = ((long long)t * KT + row) >> g.log2_page;
          has = row < KT;
        }
      }
      return has && t < wk.t1 && col < a.table_width ? a.block_table[(int64_t)wk.b * a.table_width + col] : -1;
    };
    // Q8, lanes from 16 on: the scale byte of a block of keys (24 on: of values); 0 where there is none.
    auto byte_of = [&](int t, int page) -> uint32_t {
      const int row = (lane & 7) << g.log2_block;
      if (lane < 16 || page < 0 || page >= a.cache.num_pages || t >= wk.t1 || t * KT + row >= wk.r.ctx + wk.r.n) return 0;
      const uint8_t* s = lane & 8 ? g.v_scale : g.k_scale;
      return s[scale_index(g, page, (t * KT + row) & ((1 << g.log2_page) - 1), wk.h)];
    };
    auto used = [&](int t) { return lane < per_tile && t * KT + lane * box_rows < wk.r.ctx + wk.r.n; };
    auto there = [&](int t, int page) { return used(t) && page >= 0 && page < a.cache.num_pages; };
    // V tiles that fix_v looks at: new tokens, the end of the request, absent pages
    auto special = [&](int t, uint32_t pages) { return (t + 1) * KT > wk.r.ctx || pages != full_pages; };

    if (warp == kProducer) {
      const uint32_t box_bytes = (uint32_t)box_rows * (Q8 ? D : 128 * C::HALVES);
      uint32_t st = 0, phase = 1;  // the stage to fill and the parity of its last emptying
      int item = 0;
      for (; wk.next(g); ++item) {
        int page = page_of(wk.t0);
        if (item > 0 && !mbar_wait(&sh.q_empty, (uint32_t)((item - 1) & 1), late)) late = true;
        const int q_tiles = wk.pair ? 2 : 1;
        if (lane == 0) {
          mbar_expect_tx(&sh.q_full, (uint32_t)(q_tiles * g.tpt * g.G * D * 2));
          for (int s = 0; s < q_tiles; ++s)
            for (int hf = 0; hf < C::HALVES; ++hf)
              tensor_g2s_3d(sq + s * C::TILE + hf * C::BLOCK, &map_q, hf * 64, wk.h * g.G,
                            wk.r.q0 + (wk.blk * 2 + s) * g.tpt, &sh.q_full);
        }
        if constexpr (Q8) {
          // Two pages ahead, so that a block's scale byte can be fetched one tile ahead.
          int next_page = page_of(wk.t0 + 1);
          uint32_t scale = byte_of(wk.t0, page);
          for (int t = wk.t0; t < wk.t1; ++t) {
            const int page_after = page_of(t + 2);
            const uint32_t next_scale = byte_of(t + 1, next_page);
            const bool load = there(t, page);
            if (used(t) && !load && a.status) atomicOr(a.status, FT_ST_BAD_SLOT);
            const uint32_t pages = __ballot_sync(~0u, load);
            const int y = g.log2_page >= 7 ? (t * KT) & ((1 << g.log2_page) - 1) : 0;
            const uint32_t first = st;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              if (!mbar_wait(&sh.raw_empty[st], phase, late)) late = true;  // the first round passes at once
              if (lane == 0) {
                sh.raw_pages[st] = pages;
                mbar_expect_tx(&sh.raw[st], (uint32_t)__popc(pages) * box_bytes);
              }
              __syncwarp();
              if (load)
                tensor_g2s_4d(ring8 + st * C::TILE8 + lane * box_rows * D, kv ? &map_v : &map_k, 0, y, wk.h, page, &sh.raw[st]);
              if (++st == C::NST8) st = 0, phase ^= 1;
            }
            if (lane >= 16) sh.raw_scale[(lane & 8) ? (first + 1 == C::NST8 ? 0 : first + 1) : first][lane & 7] = (uint8_t)scale;
            __syncwarp();
            if (lane < 2) mbar_arrive_cta(&sh.raw[lane ? (first + 1 == C::NST8 ? 0 : first + 1) : first]);
            page = next_page;
            next_page = page_after;
            scale = next_scale;
            if (__any_sync(~0u, late)) wk.left = 0, wk.t1 = t;  // load nothing more
          }
        } else {
          for (int t = wk.t0; t < wk.t1; ++t) {
            const int next_page = page_of(t + 1);
            const bool load = there(t, page);
            if (used(t) && !load && a.status) atomicOr(a.status, FT_ST_BAD_SLOT);
            const uint32_t pages = __ballot_sync(~0u, load);
            const int y = g.log2_page >= 7 ? (t * KT) & ((1 << g.log2_page) - 1) : 0;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              if (!mbar_wait(&sh.empty[st], phase, late)) late = true;  // the first round passes at once
              uint64_t* bar = kv && special(t, pages) ? &sh.raw[st] : &sh.full[st];
              if (lane == 0) {
                sh.pages[st] = pages;
                mbar_expect_tx(bar, (uint32_t)__popc(pages) * box_bytes);
              }
              __syncwarp();
              if (load) {
                uint8_t* dst = ring + st * C::TILE + lane * box_rows * 128;
#pragma unroll
                for (int hf = 0; hf < C::HALVES; ++hf)
                  tensor_g2s_4d(dst + hf * C::BLOCK, kv ? &map_v : &map_k, hf * 64, y, wk.h, page, bar);
              }
              if (++st == NST) st = 0, phase ^= 1;
            }
            page = next_page;
            if (__any_sync(~0u, late)) wk.left = 0, wk.t1 = t;  // load nothing more
          }
        }
      }
    } else if (Q8 && warp >= kConverters) {
      // 8-bit tiles become the 16-bit tiles that the products take; each warp 32 rows.
      uint32_t st = 0, st8 = 0, phase = 1, phase8 = 0;
      const int first_row = (warp - kConverters) * 32;
      for (int item = 0; wk.next(g); ++item) {
        uint32_t found = 0;
        for (int t = wk.t0; t < wk.t1; ++t) {
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            if (!mbar_wait(&sh.raw[st8], phase8, late)) late = true;
            if (!mbar_wait(&sh.empty[st], phase, late)) late = true;  // the first round passes at once
            const uint32_t pages = sh.raw_pages[st8];
            convert_rows<E, D>(ring8 + st8 * C::TILE8 + first_row * D, ring + st * C::TILE + first_row * 128,
                               uniform(sh.raw_scale[st8][first_row >> g.log2_block]),
                               uniform(sh.raw_scale[st8][(first_row + 16) >> g.log2_block]), lane, g.sixteen, g.one);
            if (kv && special(t, pages)) {
              const int left = wk.r.ctx + wk.r.n - t * KT;
              __syncwarp();
              found |= fix_v_rows<E, C::HALVES, C::BLOCK>(ring + st * C::TILE, lane, min(g.log2_page, 7), pages, left,
                                                          max(wk.r.ctx - t * KT, 0), first_row);
              if (lane == 0) sh.nonfinite[item & 3][warp - kConverters] = found;
            }
            if (warp == kConverters && lane == 0) sh.pages[st] = pages;
            proxy_fence_writes();  // (and of the 8-bit stage's reads before its refill)
            __syncwarp();
            if (lane == 0) {
              mbar_arrive_cta(&sh.full[st]);
              mbar_arrive_cta(&sh.raw_empty[st8]);
            }
            if (++st == NST) st = 0, phase ^= 1;
            if (++st8 == C::NST8) st8 = 0, phase8 ^= 1;
          }
        }
      }
    } else if (!Q8 && warp == kFixer) {
      uint32_t st = 0, rounds = 0;  // the stage of a tile's V; a bit per stage: parity of its next raw phase
      for (int item = 0; wk.next(g); ++item) {
        uint32_t found = 0;
        for (int t = wk.t0; t < wk.t1; ++t) {
          if (++st == NST) st = 0;  // past the tile's K
          const uint32_t pages = __ballot_sync(~0u, there(t, page_of(t)));
          if (special(t, pages)) {
            if (!mbar_wait(&sh.raw[st], (rounds >> st) & 1, late)) late = true;
            rounds ^= 1u << st;
            const int left = wk.r.ctx + wk.r.n - t * KT;
            found |= fix_v<E, C::HALVES, C::BLOCK>(ring + st * C::TILE, lane, min(g.log2_page, 7), pages, left,
                                                   min(KT, (left + 15) & ~15), max(wk.r.ctx - t * KT, 0));
            if (lane == 0) {
              sh.nonfinite[item & 3][0] = found;
              mbar_arrive_cta(&sh.full[st]);
            }
          }
          if (++st == NST) st = 0;
        }
      }
    } else if (warp == kIssuer) {
      // The whole warp keeps the loop's state and one elected lane issues: with
      // warp-uniform numbers the descriptors stay in uniform registers.
      const bool one = elect_one();
      constexpr bool BF = Elem<E>::kDtype == FT_DTYPE_BF16;
      constexpr uint32_t id_qk = umma_idesc_f16(BF, 128, KT, false), id_pv = umma_idesc_f16(BF, 128, D, true);
      const uint64_t dq0 = umma_desc_sw128(smem_u32(sq));
      const uint64_t dk0 = umma_desc_sw128(smem_u32(ring)), dv0 = umma_desc_sw128_mn(smem_u32(ring), C::BLOCK);
      uint32_t base = 0;             // ring position of the item's first stage
      uint32_t done0 = 0, done1 = 0;  // tiles of each stream so far (barrier phases)
      for (int item = 0; wk.next(g); ++item) {
        const bool pair = uniform(wk.pair);
        const int n_tiles = uniform(wk.t1 - wk.t0), c0 = uniform(wk.count(0)), c1 = uniform(wk.count(1));
        // 16-key steps of the item's last tile: past the request's keys nothing is multiplied
        const int last_steps = uniform(
            wk.t1 == wk.r.tiles ? (min(KT, wk.r.ctx + wk.r.n - (wk.t1 - 1) * KT) + 15) >> 4 : KT / 16);
        if (!mbar_wait(&sh.q_full, (uint32_t)(item & 1), late)) late = true;
        auto qk = [&](auto stream, int j) {
          constexpr int s = decltype(stream)::value;
          const uint32_t pos = base + 2 * (pair ? j : 2 * j + s), st = pos % NST;
          // (a row tile pair's second stream finds the tile its first has waited for)
          if ((!pair || s == 0) && !mbar_wait(&sh.full[st], (pos / NST) & 1, late)) late = true;
          tc_fence_after();
          const uint64_t dq = dq0 + (uint32_t)((pair ? s : 0) * (C::TILE >> 4)), dk = dk0 + st * (C::TILE >> 4);
          if (one) {
            sh.s_pages[s] = sh.pages[st];
            mbar_arrive_cta(&sh.s_full[s]);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * C::BLOCK + (kk & 3) * 32) >> 4;
              umma_bf16(tmem + 256 + s * 128, dq + off, dk + off, id_qk, kk ? 1u : 0u);
            }
            umma_commit(&sh.s_full[s]);
            if (!pair || s == 1) umma_commit(&sh.empty[st]);
          }
          __syncwarp();
        };
        auto pv = [&](auto stream, int j) {
          constexpr int s = decltype(stream)::value;
          const int i = pair ? j : 2 * j + s;
          const uint32_t pos = base + 2 * i + 1, st = pos % NST;
          if ((!pair || s == 0) && !mbar_wait(&sh.full[st], (pos / NST) & 1, late)) late = true;
          const uint32_t phase = ((s ? done1 : done0) + j) & 1;
          const uint64_t dv = dv0 + st * (C::TILE >> 4);
          const int steps = i + 1 == n_tiles ? last_steps : KT / 16;
          // P comes in two halves, so that the first half's products run beside
          // the second half's exponentials.
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!mbar_wait(half ? &sh.p_full[s] : &sh.p_half[s], phase, late)) late = true;
            tc_fence_after();
            if (one) {
#pragma unroll
              for (int k = 0; k < KT / 32; ++k) {
                const int kk = half * (KT / 32) + k;
                if (kk < steps)
                  umma_f16_ta(tmem + s * 128, tmem + 256 + s * 128 + kk * 8, dv + kk * (2048 >> 4), id_pv,
                              kk ? 1u : (j ? 1u : 0u));
              }
            }
          }
          if (one) {
            if (!pair || s == 1) umma_commit(&sh.empty[st]);
            if (j + 1 == (s ? c1 : c0)) {  // the item's output is complete
              umma_commit(&sh.o_full[s]);
              mbar_arrive_cta(&sh.o_full[s]);
            }
          }
          __syncwarp();
        };
        const std::integral_constant<int, 0> S0;
        const std::integral_constant<int, 1> S1;
        qk(S0, 0);
        if (c1 > 0) qk(S1, 0);
        if (c0 == 1 && one) umma_commit(&sh.q_empty);  // every product with Q has been issued
        for (int j = 0; j < c0; ++j) {
          pv(S0, j);
          if (j + 1 < c0) qk(S0, j + 1);
          if (j < c1) pv(S1, j);
          if (j + 1 < c1) qk(S1, j + 1);
          if (j + 2 == c0 && one) umma_commit(&sh.q_empty);
        }
        done0 += c0;
        done1 += c1;
        base += 2 * n_tiles;
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX_REGS));
    const int s = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + 256 + s * 128 + lanes, t_o = tmem + lanes;
    const uint32_t full_pages = g.log2_page >= 7 ? 1u : (1u << (KT >> g.log2_page)) - 1;
    const int tok = row / g.G, head = row - tok * g.G;  // this thread's row in any block
    uint32_t tiles_done = 0, items_of_stream = 0;
    bool has_cut = false;
    const int share = wk.left;
    for (int item = 0; wk.next(g); ++item) {
      const Req& r = wk.r;
      const int first_tok = (wk.blk * 2 + (wk.pair ? s : 0)) * g.tpt;
      const int i = first_tok + tok;
      const bool valid = tok < g.tpt && i < r.n;
      const bool warp_live = __any_sync(~0u, valid);
      const uint32_t* mrow = a.mask ? a.mask + (int64_t)(r.q0 + (valid ? i : 0)) * a.mask_words : nullptr;
      uint2 first = make_uint2(0, 0);  // (loaded while the tiles are on their way)
      if (mrow && wk.t1 * KT > r.ctx) {
        first.x = mrow[0];
        if (a.mask_words > 1) first.y = mrow[1];
      }
      const int cnt = wk.count(s);
      float m = -CUDART_INF_F, l = 0.f;
      bool far = false;  // one of the warp's rows has m past kFar
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
          if ((t + 1) * KT > r.ctx || pages != full_pages) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t vis = valid ? visible(g, r, mrow, first, i, t * KT + w * 32, w, pages) : 0u;
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(vis >> c & 1)) x[w * 32 + c] = -CUDART_INF_F;
            }
          }
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int c = 4; c < 124; c += 2) mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], x[c], x[c + 1]);
          const float top = max3(max3(mx[0], mx[1], x[124]), max3(mx[2], mx[3], x[125]), fmaxf(x[126], x[127]));
          const bool grow = (top - m) * g.c > Held<E>::kLag || m == -CUDART_INF_F;  // also the first tile with a key
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
            // (rows that are not this request's hold a neighbour's queries or none: no say in how these are rounded)
            far = __any_sync(~0u, valid && fabsf(m) * g.c > kFar && m != -CUDART_INF_F);
          }
          float ref = m == -CUDART_INF_F ? 0.f : m * g.c;
          if (far) {
            const float from = ref == 0.f ? 0.f : m;
#pragma unroll
            for (int c = 0; c < 128; ++c) x[c] -= from;
            ref = 0.f;
          }
          const uint64_t c2 = pair2(g.c, g.c), ref2 = pair2(Held<E>::kUp - ref, Held<E>::kUp - ref);
          uint64_t sum[4] = {};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int c = half * 64; c < half * 64 + 64; c += 2) {
              const float2 t2 = split2(fma2(pair2(x[c], x[c + 1]), c2, ref2));
              const float p0 = ex2(t2.x), p1 = ex2(t2.y);
              sum[(c >> 1) & 3] = add2(sum[(c >> 1) & 3], pair2(p0, p1));
              // 16 bits are what the second product takes; the sum keeps all 32.  Outputs are 2.3e-3 from 64 bits in
              // bf16 and 2.8e-4 in f16, with 32-bit probabilities 1.7e-3 and 2.1e-4 (the output's own rounding).
              u[c >> 1] = Elem<E>::pack(p0, p1);
            }
            tmem_st32(t_s + half * 32, u + half * 32);
            tmem_wait_st();
            tc_fence_before();
            if (half == 0) {
              __syncwarp();
              if (lane == 0) mbar_arrive_cta(&sh.p_half[s]);
            }
          }
          const float2 part = split2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
          l += part.x + part.y;
        } else if (lane == 0) {
          mbar_arrive_cta(&sh.p_half[s]);
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
      // Rows' output: with a row tile per stream the thread's own; else the two
      // streams' halves of the keys joined, each warpgroup half of the columns.
      // A sum is joined as its maximum and its sum: as one logarithm c m + log2 l
      // it would lose l's bits to a large m (all of them at c m = 2^27).
      float w0 = 0.f, w1 = 0.f;
      int c0 = 0, c1 = D;
      bool use0 = s == 0, use1 = s == 1;
      if (!wk.pair) {
        sh.m[s][row] = cnt > 0 ? m : -CUDART_INF_F;
        sh.l[s][row] = l;
        bar_sync(1, 256);
        const float m0 = sh.m[0][row], m1 = sh.m[1][row], l0 = sh.l[0][row], l1 = sh.l[1][row];
        m = fmaxf(m0, m1);
        use0 = m0 != -CUDART_INF_F;
        use1 = m1 != -CUDART_INF_F;
        w0 = use0 ? ex2((m0 - m) * g.c) : 0.f;
        w1 = use1 ? ex2((m1 - m) * g.c) : 0.f;
        l = (use0 ? w0 * l0 : 0.f) + (use1 ? w1 * l1 : 0.f);
        c0 = s * (D / 2);
        c1 = c0 + D / 2;
      }
      const bool some = l > 0.f || l != l;  // NaN: a seen score was NaN or +inf
      const float inv = some ? __fdividef(1.f, l) : 0.f;
      const float lse = some ? m * g.c + (__log2f(l) - Held<E>::kUp) : -CUDART_INF_F;
      w0 *= inv;
      w1 *= inv;
      // Written where an item has new keys, before the product of their tile: without row tile pairs the other
      // stream's warps know that it is only past the barrier above.
      bool nonfinite = wk.t1 * KT > r.ctx && sh.nonfinite[item & 3][0];
      if constexpr (Q8) {
#pragma unroll
        for (int k = 1; k < 4; ++k) nonfinite |= wk.t1 * KT > r.ctx && sh.nonfinite[item & 3][k];
      }
      use0 = use0 && wk.count(0) > 0;
      use1 = use1 && wk.count(1) > 0;
      const bool whole = wk.t0 == 0 && wk.t1 == r.tiles;
      const int slot = blockIdx.x * 2 + (wk.t0 == 0 ? 1 : 0);
      const int part_row = slot * 256 + (wk.pair ? s * 128 : 0) + row;
      const int h0 = wk.h * g.G + head;
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
              if (!(mask_bits(g, mrow, first, i, jn) & 1)) continue;
              const long long col = key >> g.log2_page;
              const int pg = col < a.table_width ? a.block_table[(int64_t)wk.b * a.table_width + col] : -1;
              if (pg < 0 || pg >= a.cache.num_pages) continue;
              using V = std::conditional_t<Q8, uint8_t, uint16_t>;
              const int in_page = key & ((1 << g.log2_page) - 1);
              const V* vr = static_cast<const V*>(a.cache.v) + pg * a.cache.v_page_stride +
                            in_page * a.cache.v_token_stride + wk.h * a.cache.v_head_stride + c;
              float scale = 1.f;
              if constexpr (Q8) scale = scale_of(g.v_scale[scale_index(g, pg, in_page, wk.h)]);
              for (int k = 0; k < 32; ++k) {
                float f;
                if constexpr (Q8)
                  f = Elem<E>::unpack(Elem<E>::pack(e4m3_value(vr[k]) * scale, 0.f)).x;
                else
                  f = Elem<E>::unpack(vr[k]).x;
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
              float4* dst = g.part_o + ((int64_t)(slot * 2 + (wk.pair ? s : 0)) * (D / 4) + c / 4) * 128 + row;
#pragma unroll
              for (int k = 0; k < 8; ++k) dst[k * 128] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
            }
          }
        }
      }
      if (valid && (wk.pair || s == 0)) {
        if (!whole)
          g.part_ml[part_row] = make_float2(some ? m : -CUDART_INF_F, l);
        else if (a.lse)
          a.lse[(int64_t)(r.q0 + i) * a.q_heads + h0] = lse * kLn2;
      }
      if (!whole && wk.t0 == 0) {
        has_cut = true;
        if (tid == 0) {
          // the CTA that owns the first unit of the item's last tile
          const long long it = lo + (share - wk.left) - wk.unit + (long long)(r.tiles - 1) * wk.weight();
          const int cb = deal.owner(it);
          const int rows = min(r.n - wk.blk * 2 * g.tpt, 2 * g.tpt) * g.G;
          g.cut[blockIdx.x] = Cut{cb - (int)blockIdx.x + 1, rows, r.q0 + wk.blk * 2 * g.tpt, wk.h};
        }
      }
      tc_fence_before();
      // both warpgroups have read O before either goes on
      bar_sync(1, 256);
    }
    if (tid == 0 && !has_cut) g.cut[blockIdx.x].parts = 0;
  }
  tc_fence_before();
  const bool any_late = __syncthreads_or(late);
  tc_fence_after();
  if (any_late) {
    // Every copy and product that was issued has been waited for unless a wait
    // ran out; those still in flight get kDrainNs.
    for (const uint64_t t0 = global_ns(); global_ns() - t0 < kDrainNs;) __nanosleep(1000);
    if (late && a.status) atomicOr(a.status, FT_ST_TIMEOUT);
    __syncthreads();
  }
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
}

// Joins the parts of the items that were cut; the blocks of a column share an
// item.  With m_c, l_c a part's maximum and sum and O_c its normalised output,
// M = max m_c, L = sum l_c 2^(c (m_c - M)), out = sum (l_c 2^(c (m_c - M)) / L) O_c
// and ln sum = ln 2 (c M + log2 L).  The parts are in L2 and the
// kernel is latency, so a batch's loads are all in flight before the first is
// used, and where the item has few outputs several lanes share one (its parts in
// stretches, joined in order).  A lane takes 4 outputs of a row.  Launched as a
// programmatic dependent of the kernel above.
constexpr int kJoinThreads = 128, kJoinBlocks = 24, kJoinBatch = 8, kJoinSplit = 4;

struct Part {
  float m, l;  // maximum, sum
  float4 acc;  // normalised output
  __device__ __forceinline__ void scale(float w) { acc.x *= w, acc.y *= w, acc.z *= w, acc.w *= w; }
  __device__ __forceinline__ void add(float w, const float4& o) {  // (o is not looked at where its weight is 0)
    if (w > 0.f) acc.x = fmaf(w, o.x, acc.x), acc.y = fmaf(w, o.y, acc.y), acc.z = fmaf(w, o.z, acc.z), acc.w = fmaf(w, o.w, acc.w);
  }
};

// ROWS: of a row tile in the parts; 128 of two tiles, or fewer of one.
template <typename E, int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) tree_attention_join_kernel(const __grid_constant__ Args g) {
  pdl_wait();
  const int c0 = blockIdx.x;
  const Cut cut = g.cut[c0];
  if (cut.parts == 0) return;
  const ft_attn_args& a = g.a;
  const int tile_rows = g.tpt * g.G, outputs = cut.rows * (D / 4), warps = gridDim.y * (kJoinThreads / 32);
  const int lane = threadIdx.x & 31, w = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5);
  int split = 1;
  while (split < kJoinSplit && outputs * split * 2 <= warps * 32 && split < cut.parts) split *= 2;
  const int per = 32 / split, slice = lane / per;  // outputs of a warp; this lane's stretch of the parts
  const int first = cut.parts * slice / split, last = cut.parts * (slice + 1) / split;
  auto slot = [&](int p) { return (c0 + p) * 2 + (p == 0 ? 1 : 0); };
  for (int x0 = w * per; x0 < outputs; x0 += warps * per) {
    const int x = min(x0 + lane % per, outputs - 1);
    const int col = x / cut.rows, rr = x - col * cut.rows;  // rows fastest: contiguous in the parts
    const int tile = rr >= tile_rows ? 1 : 0, row = rr - tile * tile_rows;
    Part q{-CUDART_INF_F, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    bool nan = false;
    for (int p0 = first; p0 < last; p0 += kJoinBatch) {
      float2 ml[kJoinBatch];
      float4 o[kJoinBatch];
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) {
        ml[i] = make_float2(-CUDART_INF_F, 0.f);
        if (p0 + i < last) {
          const int at = slot(p0 + i);
          const int64_t part = ROWS == 128 ? at * 2 + tile : at;
          ml[i] = __ldcg(&g.part_ml[part * ROWS + row]);
          o[i] = __ldcg(&g.part_o[(part * (D / 4) + col) * ROWS + row]);
        }
      }
      float most = q.m;
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) {
        nan |= ml[i].y != ml[i].y;
        most = fmaxf(most, ml[i].x);
      }
      if (most == -CUDART_INF_F) continue;
      const float was = q.l * ex2((q.m - most) * g.c);
      float e[kJoinBatch], l = was;
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) {
        e[i] = ml[i].y * ex2((ml[i].x - most) * g.c);
        l += e[i];
      }
      const float inv = __fdividef(1.f, l);
      q.scale(was * inv);
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) q.add(e[i] * inv, o[i]);
      q.m = most, q.l = l;
    }
    // the stretches, lower parts first
    for (int s = per; s < 32; s *= 2) {
      Part r;
      r.m = __shfl_down_sync(~0u, q.m, s);
      r.l = __shfl_down_sync(~0u, q.l, s);
      r.acc.x = __shfl_down_sync(~0u, q.acc.x, s), r.acc.y = __shfl_down_sync(~0u, q.acc.y, s);
      r.acc.z = __shfl_down_sync(~0u, q.acc.z, s), r.acc.w = __shfl_down_sync(~0u, q.acc.w, s);
      nan |= __shfl_down_sync(~0u, (int)nan, s) != 0;
      const float most = fmaxf(q.m, r.m);
      if (most != -CUDART_INF_F) {
        const float a = q.l * ex2((q.m - most) * g.c), b = r.l * ex2((r.m - most) * g.c);
        const float inv = __fdividef(1.f, a + b);
        q.scale(a * inv);
        q.add(b * inv, r.acc);
        q.m = most, q.l = a + b;
      }
    }
    if (slice != 0 || x0 + lane >= outputs) continue;
    if (nan) q.l = CUDART_NAN_F;  // a part's scores held NaN: the row is NaN
    const float one = q.l != q.l ? q.l : 1.f;
    const int h = cut.h * g.G + row % g.G;
    const int64_t t = cut.token0 + tile * g.tpt + row / g.G;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + t * a.out_stride + (int64_t)h * D + col * 4) =
        make_uint2(Elem<E>::pack(q.acc.x * one, q.acc.y * one), Elem<E>::pack(q.acc.z * one, q.acc.w * one));
    if (a.lse && col == 0)
      a.lse[t * a.q_heads + h] = q.l == 0.f ? -CUDART_INF_F : (q.m * g.c + (log2f(q.l) - Held<E>::kUp)) * kLn2;
  }
}

inline uint64_t workspace(int grid, int D) { return cut_bytes(grid) + ml_bytes(grid) + (uint64_t)grid * 2 * 256 * D * 4; }

template <bool Q8>
bool cache_map(CUtensorMap* map, void* base, const ft_kv_cache& c, int64_t page, int64_t token, int64_t head, char* msg,
               size_t len) {
  const uint64_t dims[4] = {(uint64_t)c.head_dim, (uint64_t)c.page_size, (uint64_t)c.kv_heads, (uint64_t)c.num_pages};
  const uint64_t size = Q8 ? 1 : 2;
  const uint64_t strides[3] = {(uint64_t)token * size, (uint64_t)(c.kv_heads > 1 ? head : c.head_dim) * size,
                               (uint64_t)(c.num_pages > 1 ? page : c.head_dim) * size};
  const uint32_t box[4] = {Q8 ? (uint32_t)c.head_dim : 64, (uint32_t)(c.page_size < KT ? c.page_size : KT), 1, 1};
  if (Q8) return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box, msg, len, 0, c.head_dim);
  return encode_tensor_map(map, c.dtype == FT_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                           4, base, dims, strides, box, msg, len, 128);
}

template <typename E, int D, int ROWS>
cudaError_t launch_join(const Args& g, int grid, cudaStream_t st) {
  // blocks for the most rows an item can have, so that its outputs can be shared by kJoinSplit lanes
  const int most = std::min(std::min(g.a.max_tokens, 2 * g.tpt) * g.G, ROWS == 128 ? 256 : ROWS) * (D / 4) * kJoinSplit;
  const int blocks = std::min((most + kJoinThreads - 1) / kJoinThreads, kJoinBlocks);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(cfg, attr, dim3(grid, blocks), dim3(kJoinThreads), 0, st);
  return cudaLaunchKernelEx(&cfg, tree_attention_join_kernel<E, D, ROWS>, g);
}

template <typename E, int D, bool Q8>
int launch(const Args& g, int grid, cudaStream_t st) {
  using C = Cfg<D, Q8>;
  const ft_attn_args& a = g.a;
  const ft_kv_cache& c = a.cache;
  CUtensorMap mq, mk, mv;
  char msg[128] = "";
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.q_heads, (uint64_t)a.max_tokens};
  const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)(a.max_tokens > 1 ? a.q_stride : (int64_t)a.q_heads * D) * 2};
  const uint32_t box[3] = {64, (uint32_t)g.G, (uint32_t)g.tpt};
  if (!encode_tensor_map(&mq, Elem<E>::kDtype == FT_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                         3, const_cast<void*>(a.q), dims, strides, box, msg, sizeof(msg), 128) ||
      !cache_map<Q8>(&mk, c.k, c, c.k_page_stride, c.k_token_stride, c.k_head_stride, msg, sizeof(msg)) ||
      !cache_map<Q8>(&mv, c.v, c, c.v_page_stride, c.v_token_stride, c.v_head_stride, msg, sizeof(msg)))
    return record_error(FT_E_CUDA, "%s", msg);
  static thread_local int configured = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured != dev) {
    const cudaError_t e =
        cudaFuncSetAttribute(tree_attention_kernel<E, D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(C::SMEM + sizeof(Shared<Q8>)));
    if (e != cudaSuccess) return record_error(FT_E_CUDA, "attention setup failed: %s", cudaGetErrorString(e));
    configured = dev;
  }
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(cfg, attr, dim3(grid), dim3(C::THREADS), C::SMEM + sizeof(Shared<Q8>), st);
  cudaError_t e = cudaLaunchKernelEx(&cfg, tree_attention_kernel<E, D, Q8>, mq, mk, mv, g);
  if (e == cudaSuccess) e = launch_join<E, D, 128>(g, grid, st);
  if (e != cudaSuccess) return record_error(FT_E_CUDA, "attention launch failed: %s", cudaGetErrorString(e));
  return FT_OK;
}

// ---- Checks of a call but for its cache, and its arguments

inline int check_sizes(const ft_attn_args& a) {
  if (a.max_tokens < 0 || a.num_reqs < 0 || a.q_heads < 1 || a.table_width < 0 || a.mask_words < 0)
    return record_error(FT_E_ARG, "max_tokens, num_reqs, table_width and mask_words must not be negative, q_heads positive");
  if (a.q_heads % a.cache.kv_heads) return record_error(FT_E_ARG, "q_heads must be a multiple of kv_heads");
  if (a.q_heads / a.cache.kv_heads > 128) return record_error(FT_E_UNSUPPORTED, "more than 128 query heads to a key head");
  return FT_OK;
}

// (of a call with rows)
inline int check_rest(const ft_attn_args& a, uint64_t need) {
  if (!a.q || !a.out || !a.q_start || !a.ctx_len || !a.block_table || !a.workspace)
    return record_error(FT_E_ARG, "null pointer");
  if (a.table_width < 1) return record_error(FT_E_ARG, "table_width must be positive");
  if (a.mask ? a.mask_words < 1 : a.mask_words != 0)
    return record_error(FT_E_ARG, "a mask needs mask_words >= 1; without one mask_words must be 0");
  if (!is_16b(a.q) || !is_16b(a.out) || !is_16b(a.workspace) || a.q_stride < 0 || a.out_stride < 0 || a.q_stride % 8 ||
      a.out_stride % 8)
    return record_error(FT_E_ARG, "q, out and workspace must be 16-byte aligned, row strides multiples of 8 elements");
  if (!(fabsf(a.scale) < 1e37f)) return record_error(FT_E_ARG, "scale must be finite (below 1e37)");
  if (a.workspace_bytes < need)
    return record_error(FT_E_ARG, "workspace of %llu bytes, %llu needed", (unsigned long long)a.workspace_bytes,
                        (unsigned long long)need);
  return FT_OK;
}

// `rows`: of an item at most.
inline Args make_args(const ft_attn_args& a, int grid, int rows = 256) {
  Args g{};
  g.a = a;
  g.log2_page = log2_of(a.cache.page_size);
  g.G = a.q_heads / a.cache.kv_heads;
  g.tpt = 128 / g.G;
  g.neg = a.scale < 0.f;
  // a scale of 0 becomes the least positive number: -inf stays -inf and the largest finite score is 5e-7
  const float c = (g.neg ? -a.scale : a.scale) * kLog2e;
  g.c = c > 0.f ? c : std::numeric_limits<float>::denorm_min();
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  g.cut = reinterpret_cast<Cut*>(ws);
  g.part_ml = reinterpret_cast<float2*>(ws + cut_bytes(grid));
  g.part_o = reinterpret_cast<float4*>(ws + cut_bytes(grid) + ml_bytes(grid, rows));
  return g;
}

}  // namespace tree_attention
}  // namespace ft
