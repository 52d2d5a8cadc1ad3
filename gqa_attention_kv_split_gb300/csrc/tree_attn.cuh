// tree_attn.cuh -- attention of several new tokens per sequence over a paged K/V cache
// (f16, bf16 or E4M3 pages): drafted tokens in a tree or a chain, grouped queries, split
// over the cache's length and joined, on tcgen05 with accumulators in TMEM, for sm_103a.
//
// Mathematics.  Sequence b has n new tokens whose keys and values are in the cache already,
// behind base = len - n others.  Row (i, h), token i and query head h over KV head g, is
//   s_t = cap( (q_ih . K_t) * scale ),  out = v_scale * sum_t w_t V_t / sum_t w_t,
//   w_t = exp(s_t - m),  lse = ln sum_t exp(s_t)
// over the cached tokens t < base within its window (or among the sinks) and the drafted ones
// base + j whose bit j its mask has; without masks over t <= base + i.  A range of tokens is
// summed as (m, l, o) and ranges join by rescaling to the larger m.
//
// What bounds it: a K/V byte serves n G / 2 products of 16 bits (G heads a KV head), so HBM does up to
// about 256 rows n G, the tensor cores from there on.  The rows of a KV head are packed into
// the MMA's M = 128 (row = token * G + head): S = Q K^T with the keys on N, O = P V with the
// weights as TMEM operand.  With 128 rows or fewer a tile of 128 tokens (64 KB in bf16, head
// dim 128: 1.5 us of an SM's share of HBM) keeps the tensor pipe busy for 0.8 us, however few
// rows there are, and the softmax for less:
//  * Copies.  With 64 (32) rows or fewer each row stands in the M dimension twice (four times; twice too at head dim 256,
//    whose tiles have two parts), if there is more than one tile,
//    and each copy weighs a half (a quarter) of a tile's tokens, with zeros in P for the
//    others: the warps share the softmax evenly, as independent (m, l, o) that join at the end.
//  * S in two TMEM buffers (three at head dim 64): S of the next tile is computed while the softmax works on this one;
//    P overwrites the S it came from (32 tokens' weights: 16 columns of their first terms, 16
//    of their second ones).
//  * Weights enter the product with V as two terms of 16 bits (22 bits in f16, 16 in bf16).
//  * O leaves TMEM every 16384 tokens for sums that round to nearest (fold_out).
//  * The maximum is raised (and O rescaled in TMEM) only when a row's passes the one in use by
//    more than 2^8: weights then stay within f16, whose terms keep 2^-31 of the largest.
//
//  * Grid: one block per SM, in gangs of up to 8 with equal shares of the sequences' tokens,
//    counted on the device from the lengths, as the one-token attention's (paged_attn.cuh):
//    the blocks of a gang read the same tokens for other heads or other row blocks.  Pieces of
//    units that lie in several blocks go to the workspace and a second kernel joins them.
//  * Warps: 0 and 3 copy K and V (tensor-map TMA, one 128-byte chunk of a head's row for a page
//    or a tile at a time, into the 128-byte-swizzled layout that both products read), 1 issues the
//    products (S with the queries as TMEM operand), 4-11 load the queries, do the softmax (one
//    thread a TMEM lane, two groups in turn) and write the results.  E4M3 pages: 12-15 widen K and V to f16,
//    exactly.
//  * Every wait is bounded; a block whose wait expires drains what it started and leaves.
//
// Measured on GB300 (time in a graph of 21 calls): 16 sequences of 16384 tokens, 32/8 heads of 128, bf16, 8 drafts: 164 us,
// 6.55 TB/s; 64 drafts: 294 us, 935 TFLOP/s; 8 of 65536, f16, 64 drafts: 617-630 us at the power limit, 570 before it, 965
// TFLOP/s; 48 of up to 16001, 64/8 heads, E4M3, up to 16 drafts: 233 us, 3.4 TB/s; 200 of up to 600, bf16, up to 8 drafts: 93 us;
// one of 2048 tokens, 8 drafts: 13.6 us.  (Times beside single steps below are of graphs of one call, which take 3 us more.)
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "softcap.cuh"
#include "tcgen05.cuh"
#include "tree_attn_host.h"

namespace gqa {
namespace ta {

namespace {

__device__ uint32_t g_tree_attn_err;  // of this translation unit's kernels

}  // namespace

template <int kCache, int D>
struct Shape {
  static constexpr bool kFp8 = kCache >= kCacheE4m3;
  static constexpr int kTile = tile_of(D);
  static constexpr int kChunks = D / 64;              // 128-byte chunks of a 16-bit row
  static constexpr int kSlot = kTile * D * 2;         // a tile of K (or of V) as the products read it
  static constexpr int kRaw = kTile * D;              // an E4M3 tile as it is copied
  // Slots of K and V, and of tiles yet to be widened.
  static constexpr int kNK = kFp8 ? (D == 64 ? 3 : 2) : (D == 64 ? 5 : 3);
  static constexpr int kNV = kNK;  // (the widening warps count both with one number)
  static constexpr int kNR = kFp8 ? (D == 64 ? 4 : 2) : 0;
  static constexpr int kThreads = kFp8 ? 512 : 384;
  static constexpr int kData = (kNK + kNV) * kSlot + 2 * kNR * kRaw;
  // TMEM columns: O, the buffers of S (where they fit three, so that a group's next scores are there when
  // it has done with a tile), and the queries (two elements a column).
  static constexpr int kBufs = D == 64 ? 3 : 2;
  static constexpr uint32_t kO = 0, kS = D, kQ = D + kBufs * kTile;
  // What starting and ending a unit costs, in tiles.  (E4M3: 40 sequences of up to 3000 tokens with up to 30 drafts
  // 67.2 us with 3, 63.3 with 6, 20 of up to 8000 58.3 with 6, 62.3 with 10.  bf16: 200 of up to 600 100.8 us
  // with 2, 98.0 with 4, 96.7 with 5, 96.9 with 8; 20 of up to 8000 67.7, 65.0, 64.4, 66.7.)
  static constexpr int kUnitWork = kFp8 ? 6 : 5;
  // Tiles whose products O takes before it goes to a sum outside TMEM (an even number).
  static constexpr int kFold = 16384 / kTile;
};

struct Bars {
  uint64_t k_full[5], k_free[5], v_full[5], v_free[5];      // tiles as the products read them
  uint64_t kr_full[4], kr_free[4], vr_full[4], vr_free[4];  // E4M3 tiles
  uint64_t s_full[3], p_full[3][2], p_free[3];              // buffers of S and P; P by halves of a tile
  uint64_t q_ready, drain;
};

template <int kThreads>
struct Smem {
  Bars bar;
  alignas(16) float stage[2][kRows][20];  // 16 columns of the copies' sums, for each half of the columns
  float m_used[kRows];                 // the maximum that the last tile's weights are relative to
  float m[2][kRows], l[2][kRows];      // of the groups' copies, at a unit's end (and their queries' largest elements)
  float m_fold[kRows];                 // the maximum that the sums outside TMEM are relative to
  int64_t scan_work[kThreads / 32], scan_turns[kThreads / 32];
  int most[kThreads / 32];
  int64_t total, end, rem;
  int n_gangs, b0;
  uint32_t tmem;
};

// (32-bit divisions where they do)
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  return (x | y) >> 32 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
}
__device__ __forceinline__ int64_t share_begin(int i, int64_t total, int n) { return quotient(total * i, n); }
// The gang that has a piece of work: the last one whose share begins at or before it.
__device__ __forceinline__ int share_of(int64_t at, int64_t total, int n) { return (int)quotient((at + 1) * n + total - 1, total) - 1; }

// A sequence: its new tokens, and its tiles in the order in which they are gone through
// (those of the sinks, then those from the window's first on, `gap` further).
template <int kTile>
struct Seq {
  int64_t row0;                  // of its first new token
  int n, len, base;              // new tokens; cached ones in all, and before the new ones
  int first, sinks;              // no row sees the tokens in [sinks, first)
  int sink_tiles, gap, tiles;
  int rows, blocks;              // rows of a KV head, and blocks of kRows of them
  bool bad;
  __device__ __forceinline__ Seq(const Params& p, int b) {
    const int64_t lo = p.indptr[b], hi = p.indptr[b + 1];
    bad = lo < 0 || hi < lo || hi > p.total;
    row0 = lo;
    n = bad ? 0 : (int)(hi - lo);
    const int64_t cap = p.max_pages << p.page_shift, x = p.kv_lens[b];
    len = (int)(x < 0 ? 0 : x > cap ? cap : x);  // (a capacity is at most 2^30)
    base = len - n;
    rows = n * p.group;
    blocks = (rows + kRows - 1) / kRows;
    first = p.window > 0 && base >= p.window ? base + 1 - p.window : 0;
    sinks = p.sinks < first ? p.sinks : 0;
    if (first > 0 && p.sinks >= first) first = 0;  // the sinks reach the window
    sink_tiles = (sinks + kTile - 1) / kTile;
    gap = max(0, first / kTile - sink_tiles);
    tiles = n > 0 ? (len + kTile - 1) / kTile - gap : 0;
  }
  __device__ __forceinline__ int place(int tile) const { return tile < sink_tiles ? tile : tile + gap; }
  __device__ __forceinline__ bool hidden(int key) const { return key >= len || (key < first && key >= sinks); }
  // Is any of the tokens [key, key + count) in no row's sight?
  __device__ __forceinline__ bool edge(int key, int count) const { return key + count > len || (key < first && key + count > sinks); }
};

// Walks the units of a block's share (paged_attn.cuh's walk, with units that depend on the
// sequence): work is counted in a unit's tiles and kUnitWork before them, or, by_unit, in
// whole units.  Unit u of a sequence is row block u % blocks of KV head u / blocks: a gang's
// blocks, which have neighbouring units, share the tokens that several row blocks read.
template <int kTile, int kUnitWork>
struct Walk {
  int left, b, unit, t_beg, t_end;
  bool by_unit, chain;
  Seq<kTile> seq;
  __device__ __forceinline__ Walk(const Params& p, int share, int b_, int64_t rem, bool by_unit_)
      : b(b_), by_unit(by_unit_), chain(!p.mask), seq(p, b_) {
    if (by_unit) {
      unit = (int)rem;
      t_beg = 0;
      t_end = seq.tiles;
      left = share - 1;
    } else {
      const int work = seq.tiles + kUnitWork;
      unit = (int)quotient(rem, work);
      const int at = (int)(rem - (int64_t)unit * work);
      t_beg = max(0, at - kUnitWork);
      left = share - max(0, kUnitWork - at);
      t_end = min(seq.tiles, t_beg + left);
    }
    unit = (unit << p.gang_shift) + ((int)blockIdx.x & ((1 << p.gang_shift) - 1));
  }
  __device__ __forceinline__ bool valid() const { return by_unit || left > 0; }
  __device__ __forceinline__ bool next(const Params& p) {
    left -= by_unit ? 1 : t_end - t_beg + kUnitWork;
    if (by_unit ? left < 0 : left <= 0) return false;
    t_beg = 0;
    unit += 1 << p.gang_shift;
    if (unit >= p.hkv * seq.blocks) {
      unit -= p.hkv * seq.blocks;
      do {
        if (++b >= p.batch) return false;
        seq = Seq<kTile>(p, b);
      } while (seq.tiles == 0);
    }
    t_end = by_unit ? seq.tiles : min(seq.tiles, left);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return t_beg == 0 && t_end == seq.tiles; }
  __device__ __forceinline__ int kv_head() const { return unit / seq.blocks; }
  __device__ __forceinline__ int row_begin() const { return (unit - unit / seq.blocks * seq.blocks) * kRows; }
  __device__ __forceinline__ int rows() const { return min(kRows, seq.rows - row_begin()); }
  // Tiles of this piece that a row of it can see: in a chain none behind its last token's.
  __device__ __forceinline__ int count(const Params& p) const {
    int e = t_end;
    if (chain) {
      const int last = seq.base + (row_begin() + rows() - 1) / p.group;
      if (last < 0) return 0;
      const int tile = last / kTile;
      e = min(e, (tile < seq.sink_tiles ? tile : tile - seq.gap) + 1);
    }
    return max(0, e - t_beg);
  }
};

// ---- the products -------------------------------------------------------------

// Instruction descriptor, kind::f16, f32 accumulators: the operands' type at bits 7 and 10
// (0 f16, 1 bf16), B's major at 16 (1: MN), N >> 3 at 17, M >> 4 at 24.
__host__ __device__ constexpr uint32_t idesc(bool bf16, int n, bool b_mn_major) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn_major ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}

__device__ __forceinline__ void tma_5d(uint32_t dst, const CUtensorMap* map, int slot, int chunk, int head, int page, uint32_t bar,
                                       uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
      "l"(map), "r"(0), "r"(slot), "r"(chunk), "r"(head), "r"(page), "r"(bar), "l"(policy)
      : "memory");
}

// Four E4M3 bytes -> four f16, exactly.
__device__ __forceinline__ uint2 widen(uint32_t four) {
  uint2 d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d.x) : "h"((uint16_t)(four & 0xffffu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d.y) : "h"((uint16_t)(four >> 16)));
  return d;
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  if (kBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool kBf16>
__device__ __forceinline__ float2 unpack(uint32_t x) {
  if (kBf16) return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Arrives at a named barrier that other threads wait at.
__device__ __forceinline__ void named_bar_arrive(uint32_t id, uint32_t count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// Bits of the tokens key .. key + 31 that lie in [lo, hi).
__device__ __forceinline__ uint32_t range_bits(int key, int lo, int hi) {
  const int a = lo - key, z = hi - key;
  if (z <= 0 || a >= 32) return 0u;
  const uint32_t below = z >= 32 ? ~0u : (1u << z) - 1u;
  return a <= 0 ? below : below & (~0u << a);
}

// What a row sees.
struct Sight {
  int lo, hi, sinks;          // cached tokens in [lo, hi) and [0, sinks)
  int base, words, len;       // drafted token j, at base + j: bit j of mask
  const int32_t* mask;        // null: none
  __device__ __forceinline__ uint32_t bits(int key) const {
    if (lo <= key && key + 32 <= hi) return ~0u;
    uint32_t v = range_bits(key, lo, hi) | range_bits(key, 0, sinks);
    if (mask && key + 32 > base) {
      const int j = key - base, w = j >> 5;
      const uint32_t a = w >= 0 && w < words ? (uint32_t)mask[w] : 0u;
      const uint32_t z = w >= -1 && w + 1 < words ? (uint32_t)mask[w + 1] : 0u;
      v |= __funnelshift_r(a, z, j & 31) & range_bits(key, base, len);
    }
    return v;
  }
};

namespace {

// The tensor cores cut off what does not fit their f32 sums, two of them for 16 tokens, so that a long sum drifts towards
// 0 (1.2e-3 of sum w |V| over 2^20 tokens).  So O goes to sums outside TMEM (in the workspace, where nothing lies yet that is read
// later), whose f32 additions round to nearest, every 16384 tokens.  (8 x 65536 f16 tokens with 64 drafts: 2.1e-4 off the
// 64-bit form, as f32 rounded to f16 is, 2.3e-4 without; 605 -> 613 us.  Every 8192 tokens 2.08e-4, 625 us, and pieces of
// fewer than 16384 tokens pay too, 163 -> 167 us; every 4096 the same error, 665 us.)
//
// Adds a lane's columns of O, times alpha, to its sums (times f; there are none yet at the first time).
template <int D>
__device__ __forceinline__ void fold_out(uint32_t t_o, float4* sums, float alpha, float f, bool first) {
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t o[16];
    tc::ld16(t_o + c, o);
    tc::ld_wait();
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      float4 y = make_float4(__uint_as_float(o[e]) * alpha, __uint_as_float(o[e + 1]) * alpha, __uint_as_float(o[e + 2]) * alpha,
                             __uint_as_float(o[e + 3]) * alpha);
      float4* const at = sums + (c + e) / 4 * kRows;
      if (!first) {
        const float4 x = *at;
        y = make_float4(fmaf(x.x, f, y.x), fmaf(x.y, f, y.y), fmaf(x.z, f, y.z), fmaf(x.w, f, y.w));
      }
      *at = y;
    }
  }
}

// And back: the sums, times g, join kCols of a lane's columns of O.
template <int kCols>
__device__ __forceinline__ void unfold_out(uint32_t t_o, const float4* sums, float g) {
  constexpr int kBatch = 32;  // columns whose loads are in flight together (with 64 registers are spilled)
#pragma unroll 1
  for (int c0 = 0; c0 < kCols; c0 += kBatch) {
    float4 x[kBatch / 4];
#pragma unroll
    for (int e = 0; e < kBatch / 4; ++e) x[e] = sums[(c0 / 4 + e) * kRows];
#pragma unroll
    for (int c = 0; c < kBatch; c += 16) {
      uint32_t o[16];
      tc::ld16(t_o + c0 + c, o);
      tc::ld_wait();
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 y = x[(c + e) / 4];
        o[e] = __float_as_uint(fmaf(y.x, g, __uint_as_float(o[e])));
        o[e + 1] = __float_as_uint(fmaf(y.y, g, __uint_as_float(o[e + 1])));
        o[e + 2] = __float_as_uint(fmaf(y.z, g, __uint_as_float(o[e + 2])));
        o[e + 3] = __float_as_uint(fmaf(y.w, g, __uint_as_float(o[e + 3])));
      }
      tc::st16(t_o + c0 + c, o);
    }
  }
}

template <int kCache, int D, bool kCap>
__global__ void __launch_bounds__(Shape<kCache, D>::kThreads, 1)
    tree_attn_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
  using S = Shape<kCache, D>;
  constexpr bool kFp8 = S::kFp8, kBf16 = kCache == kCacheBf16;    // the pages; the products' type
  constexpr bool kQBf16 = kBf16 || kCache == kCacheE4m3;          // q and out
  constexpr int kTile = S::kTile, kThreads = S::kThreads;
  constexpr int kTileShift = kTile == 64 ? 6 : 7;
  constexpr float kRaise = 8.f, kShift = kBf16 ? 0.f : 6.f;       // weights are at most 2^(kRaise + kShift)
  uint32_t* const err = &g_tree_attn_err;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const sk = smem_raw;
  uint8_t* const sv = sk + S::kNK * S::kSlot;
  uint8_t* const skr = sv + S::kNV * S::kSlot;
  uint8_t* const svr = skr + S::kNR * S::kRaw;
  Smem<kThreads>& sm = *reinterpret_cast<Smem<kThreads>*>(smem_raw + S::kData);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gang = (int)blockIdx.x >> p.gang_shift, gangs = kGrid >> p.gang_shift;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 5; ++i) {
      mbar_init(smem_u32(&sm.bar.k_full[i]), kFp8 ? 4 : 1);
      mbar_init(smem_u32(&sm.bar.k_free[i]), 1);
      mbar_init(smem_u32(&sm.bar.v_full[i]), kFp8 ? 4 : 1);
      mbar_init(smem_u32(&sm.bar.v_free[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&sm.bar.kr_full[i]), 1);
      mbar_init(smem_u32(&sm.bar.kr_free[i]), 4);
      mbar_init(smem_u32(&sm.bar.vr_full[i]), 1);
      mbar_init(smem_u32(&sm.bar.vr_free[i]), 4);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(smem_u32(&sm.bar.s_full[i]), 1);
      mbar_init(smem_u32(&sm.bar.p_full[i][0]), 4);
      mbar_init(smem_u32(&sm.bar.p_full[i][1]), 4);
      mbar_init(smem_u32(&sm.bar.p_free[i]), 1);
    }
    mbar_init(smem_u32(&sm.bar.drain), 1);
    mbar_init(smem_u32(&sm.bar.q_ready), 8);
    fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(smem_u32(&sm.tmem), 512);
    tc::tmem_relinquish();
  }
  // Launched as a programmatic dependent: what went before on the stream (the append of
  // this step) has ended and is visible from here on.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0 && p.record) p.record[blockIdx.x].last = -1;

  // ---- this block's share ------------------------------------------------------
  // Work is counted and scanned over the sequences; the share's first piece of work lies in the sequence
  // whose work covers it.
  using SeqT = Seq<kTile>;
  auto turns_of = [&](const SeqT& s) { return s.tiles == 0 ? 0 : (p.hkv * s.blocks) >> p.gang_shift; };
  auto flag = [&](const SeqT& s, int64_t b) {
    if (blockIdx.x == 0 && (s.bad || (b == 0 && s.row0 != 0))) atomicOr(err, kErrBadIndptr);
  };
  bool by_unit, bare = false;  // in whole units; a sequence without a cached token?
  int n_gangs, b0 = 0;         // gangs with a share: none is empty; the share's first sequence
  int64_t total, beg, end, rem = 0;
  auto shares = [&](int most, int64_t total_w, int64_t total_t) {
    // (without a record nothing would be joined: the host has seen that no unit needs to be split, but where offsets fall
    // the sequences between may have more rows than it counted)
    by_unit = !p.record || (most <= kWholeTiles && total_t <= gangs);
    total = by_unit ? total_t : total_w;
    // (offsets that fall again and again can make sequences in order of any number of rows, where the host has counted
    // each row once: no share may pass the 31 bits that it is counted in)
    if (total > (kTreeMostWork >> p.gang_shift)) {
      if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(err, kErrBadIndptr);
      total = 0;
    }
    n_gangs = total < gangs ? (int)total : gangs;
    beg = gang < n_gangs ? share_begin(gang, total, n_gangs) : 0;
    end = gang < n_gangs ? share_begin(gang + 1, total, n_gangs) : 0;
  };
  if (p.few) {
    // Up to 32 sequences, less than 2^31 of work: a lane each, and each warp for itself (nothing to meet for:
    // one sequence of 2048 tokens 18.5 -> 17.8 us).
    const bool in = lane < p.batch;
    const SeqT s(p, in ? lane : 0);
    if (in && warp == 0) flag(s, lane);
    const int t = in ? turns_of(s) : 0, w = t * (s.tiles + S::kUnitWork);
    int it = t, iw = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, it, d), c = __shfl_up_sync(0xffffffffu, iw, d);
      if (lane >= d) {
        it += a;
        iw += c;
      }
    }
    bare = __any_sync(0xffffffffu, in && s.n > 0 && s.tiles == 0);
    shares(__reduce_max_sync(0xffffffffu, in ? s.tiles : 0), __shfl_sync(0xffffffffu, iw, 31), __shfl_sync(0xffffffffu, it, 31));
    const int mine = by_unit ? t : w, before = (by_unit ? it : iw) - mine;
    const uint32_t who = __ballot_sync(0xffffffffu, beg < end && beg >= before && beg < before + mine);
    if (who) b0 = __ffs(who) - 1;
    rem = beg - __shfl_sync(0xffffffffu, before, b0);
  } else {
    // Each thread sums the work of a contiguous range of sequences; a scan over the threads
    // gives the ranges' starts, and the range that holds the share's first piece of work is
    // walked by its thread.
    const int64_t per = (p.batch + kThreads - 1) / kThreads;
    const int64_t s0 = threadIdx.x * per < p.batch ? threadIdx.x * per : p.batch;
    const int64_t s1 = s0 + per < p.batch ? s0 + per : p.batch;
    int64_t work = 0, turns = 0;
    int most = 0;
    for (int64_t b = s0; b < s1; ++b) {
      const SeqT s(p, (int)b);
      flag(s, b);
      const int64_t t = turns_of(s);
      turns += t;
      work += t * (s.tiles + S::kUnitWork);
      most = max(most, s.tiles);
      bare |= s.n > 0 && s.tiles == 0;
    }
    int64_t iw = work, it = turns;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, iw, d), c = __shfl_up_sync(0xffffffffu, it, d);
      if (lane >= d) {
        iw += a;
        it += c;
      }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 31) {
      sm.scan_work[warp] = iw;
      sm.scan_turns[warp] = it;
      sm.most[warp] = most;
    }
    bare = __syncthreads_or(bare);
    int64_t before_w = 0, before_t = 0, total_w = 0, total_t = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) {
        before_w += sm.scan_work[w];
        before_t += sm.scan_turns[w];
      }
      total_w += sm.scan_work[w];
      total_t += sm.scan_turns[w];
      most = max(most, sm.most[w]);
    }
    shares(most, total_w, total_t);
    const int64_t before = by_unit ? before_t + it - turns : before_w + iw - work, mine = by_unit ? turns : work;
    if (beg < end && beg >= before && beg < before + mine) {
      int64_t left = beg - before;
      int64_t b = s0;
      for (;; ++b) {
        const SeqT s(p, (int)b);
        const int64_t t = turns_of(s), w = by_unit ? t : t * (s.tiles + S::kUnitWork);
        if (left < w) break;
        left -= w;
      }
      sm.b0 = (int)b;
      sm.rem = left;
    }
  }
  if (threadIdx.x == 0) {
    sm.total = total;
    sm.n_gangs = n_gangs;
    sm.end = end;
  }
  // Rows of sequences without a cached token: zeros.
  for (int64_t b = blockIdx.x; bare && b < p.batch; b += kGrid) {
    const SeqT s(p, (int)b);
    if (s.tiles > 0 || s.n == 0) continue;
    const int64_t r0 = s.row0 * p.hq, rows = (int64_t)s.n * p.hq;
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + r0 * D * 2);
    for (int64_t i = threadIdx.x; i < rows * (D / 8); i += kThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t i = threadIdx.x; p.lse && i < rows; i += kThreads) p.lse[r0 + i] = -INFINITY;
  }
  tc::fence_before_thread_sync();
  __syncthreads();
  tc::fence_after_thread_sync();
  const uint32_t tmem = sm.tmem;
  const bool has_share = beg < end;
  if (!p.few && has_share) {
    b0 = sm.b0;
    rem = sm.rem;
  }
  Walk<kTile, S::kUnitWork> walk(p, has_share ? (int)(end - beg) : 0, b0, has_share ? rem : 0, by_unit);
  if (!has_share || !walk.valid()) {  // (or a share that lies before a unit's first tile)
    if (warp == 1) tc::tmem_dealloc(tmem, 512);
    return;
  }
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return (bool)__all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, err));
  };
  bool failed = false;  // a wait of this thread's role expired
  int issued = 0;       // producers: stages issued, up to all of them

  if (warp == 0 || warp == 3) {
    // ---------------------------------------------------------------- producers
    const bool is_v = warp == 3;
    constexpr int kStagesK = kFp8 ? S::kNR : S::kNK, kStagesV = kFp8 ? S::kNR : S::kNV;
    const int stages = is_v ? kStagesV : kStagesK;
    uint64_t* const full = kFp8 ? (is_v ? sm.bar.vr_full : sm.bar.kr_full) : (is_v ? sm.bar.v_full : sm.bar.k_full);
    uint64_t* const free_ = kFp8 ? (is_v ? sm.bar.vr_free : sm.bar.kr_free) : (is_v ? sm.bar.v_free : sm.bar.k_free);
    constexpr int kStage = kFp8 ? S::kRaw : S::kSlot;
    constexpr int kParts = kFp8 ? 1 : S::kChunks;  // copies for one box: the chunks of its rows
    const uint32_t base = smem_u32(kFp8 ? (is_v ? svr : skr) : (is_v ? sv : sk));
    const CUtensorMap* const map = is_v ? &v_map : &k_map;
    const int box_shift = p.box_shift, boxes = kTile >> box_shift, box_bytes = (kFp8 ? D : 128) << box_shift;
    const int my_box = lane & (boxes - 1), my_part = lane >> (kTileShift - box_shift);
    const uint32_t my_dst = base + my_part * (kTile * 128) + my_box * box_bytes;
    int st = 0, ph = 1;
    do {
      const SeqT& s = walk.seq;
      const int n = p.starve ? 0 : walk.count(p), head = walk.kv_head();
      // (row blocks that read the same tokens find them in L2)
      const uint64_t pol = s.blocks > 1 ? policy_evict_last() : policy_evict_first();
      const int32_t* row = p.block_table + (int64_t)walk.b * p.max_pages;
      // Copies are counted along the unit's tiles; place() says where in the sequence one lies.
      auto place = [&](int c) { return (s.place(c >> (kTileShift - box_shift)) << (kTileShift - box_shift)) + (c & (boxes - 1)); };
      auto wanted = [&](int c) {
        const int64_t key = (int64_t)c << box_shift;
        return key < s.len && (key + (1 << box_shift) > s.first || key < s.sinks);
      };
      auto page_of = [&](int c) {
        c = place(c);
        if (!wanted(c)) return 0;
        int g = row[c >> (p.page_shift - box_shift)];
        if (g < 0 || g >= p.num_pages) {
          atomicOr(err, kErrBadIndex);
          g = 0;
        }
        return g;
      };
      // Page numbers, 32 copies' worth at a time and one such group ahead (lane l has those of copy l).
      int c = walk.t_beg << (kTileShift - box_shift);
      int cur = n > 0 ? page_of(c + lane) : 0, nxt = n > 0 ? page_of(c + 32 + lane) : 0, at = 0;
      for (int j = 0; j < n; ++j) {
        if (!wait_all(&free_[st], ph)) {
          failed = true;
          break;
        }
        const int pg = __shfl_sync(0xffffffffu, cur, at + my_box);
        const int mine_at = place(c + my_box);
        const bool live = my_part < kParts && wanted(mine_at);
        const uint32_t bar = smem_u32(&full[st]);
        const uint32_t bytes = box_bytes * __popc(__ballot_sync(0xffffffffu, live));
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        if (live) tma_5d(my_dst + st * kStage, map, (mine_at << box_shift) & ((1 << p.page_shift) - 1), my_part, head, pg, bar, pol);
        c += boxes;
        at += boxes;
        if (at == 32) {
          at = 0;
          cur = nxt;
          nxt = page_of(c + 32 + lane);
        }
        issued = min(issued + 1, stages);
        if (++st == stages) {
          st = 0;
          ph ^= 1;
        }
      }
    } while (!failed && walk.next(p));
    // No copy may land after the block has gone (the stages before st were filled in the present
    // round, the others in the one before).
    if (lane == 0)
      for (int i = 0; i < issued; ++i)
        if (!mbar_wait(smem_u32(&full[i]), i < st ? ph ^ 1 : ph, err)) break;
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    // S of kBufs tiles ahead, and then O of each tile followed by the S that goes into the buffer
    // which that O has read: the tensor pipe takes them in this order, so that nothing waits
    // for a product's end but the softmax.
    constexpr uint32_t id_s = idesc(kBf16, kTile, false), id_o = idesc(kBf16, D, true);
    const uint64_t dk0 = tc::sw128_desc(smem_u32(sk)), dv0 = tc::sw128_desc_lbo(smem_u32(sv), kTile * 128);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    int ks = 0, kph = 0, vs = 0, vph = 0, units = 0;  // slots of K and V and their parities; units so far
    int sb = 0, pb = 0, pph = 0;                      // buffers of the next S and of the next P, and its parity
    auto issue_s = [&] {
      if (!wait_all(&sm.bar.k_full[ks], kph)) return false;
      tc::fence_after_thread_sync();
      const uint64_t dk = dk0 + (uint64_t)(ks * (S::kSlot >> 4));
      const uint32_t ts = tm + S::kS + (uint32_t)sb * kTile;
      if (tc::elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_f16_tmem_a(ts, tm + S::kQ + 8 * k, dk + (k / 4) * (kTile * 128 >> 4) + 2 * (k % 4), id_s, k > 0);
        tc::commit(smem_u32(&sm.bar.s_full[sb]));
        tc::commit(smem_u32(&sm.bar.k_free[ks]));
      }
      __syncwarp();
      if (++sb == S::kBufs) sb = 0;
      if (++ks == S::kNK) {
        ks = 0;
        kph ^= 1;
      }
      return true;
    };
    do {
      const int n = walk.count(p);
      if (n == 0) continue;
      if (!wait_all(&sm.bar.q_ready, units & 1)) {
        failed = true;
        break;
      }
      ++units;
      for (int i = 0; i < S::kBufs && i < n && !failed; ++i) failed = !issue_s();
      for (int i = 0; i < n && !failed; ++i) {
        if (!wait_all(&sm.bar.v_full[vs], vph)) {
          failed = true;
          break;
        }
        if (!kFp8) {
          // Rows that nothing sees may hold anything; 0 * NaN is NaN, so they are zeroed.
          const int key0 = walk.seq.place(walk.t_beg + i) * kTile;
          if (walk.seq.edge(key0, kTile)) {
            for (int x = lane; x < kTile * 8; x += 32) {
              if (!walk.seq.hidden(key0 + (x >> 3))) continue;
#pragma unroll
              for (int ch = 0; ch < S::kChunks; ++ch)
                *reinterpret_cast<uint4*>(sv + vs * S::kSlot + ch * (kTile * 128) + x * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
          }
        }
        const uint64_t dv = dv0 + (uint64_t)(vs * (S::kSlot >> 4));
        const uint32_t tp = tm + S::kS + (uint32_t)pb * kTile;
        bool ok = true;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ok = ok && wait_all(&sm.bar.p_full[pb][h], pph);
          if (!ok) break;
          tc::fence_after_thread_sync();
          if (tc::elect_one()) {
            // K = 16 tokens a product: 8 columns of P (first terms, then second ones), 2048 bytes of V
#pragma unroll
            for (int k = h * (kTile / 32); k < (h + 1) * (kTile / 32); ++k) {
              const uint32_t a = tp + 32 * (k / 2) + 8 * (k % 2);
              tc::mma_f16_tmem_a(tm + S::kO, a, dv + 128 * k, id_o, (i % S::kFold > 0 || k > 0) ? 1u : 0u);
              tc::mma_f16_tmem_a(tm + S::kO, a + 16, dv + 128 * k, id_o, 1u);
            }
            if (h == 1) {
              tc::commit(smem_u32(&sm.bar.p_free[pb]));
              tc::commit(smem_u32(&sm.bar.v_free[vs]));
            }
          }
          __syncwarp();
        }
        if (!ok || (i + S::kBufs < n && !issue_s())) {
          failed = true;
          break;
        }
        if (++pb == S::kBufs) {
          pb = 0;
          pph ^= 1;
        }
        if (++vs == S::kNV) {
          vs = 0;
          vph ^= 1;
        }
      }
    } while (!failed && walk.next(p));
  } else if (warp == 2) {
    // (holds its place: groups of four warps read TMEM by their numbers)
  } else if (warp < 12) {
    // ---------------------------------------------------------------- softmax
    // Two groups of four warps take the tiles in turn (and a half of the columns of O and of the
    // queries each); a thread is a TMEM lane.  A tile's group hands the maximum that it used to
    // the next one's, so that O has one reference: the groups' phases drift apart, and one loads
    // scores or waits while the other computes (256 rows of 65536 f16 tokens, 8 sequences: 660 us with
    // both groups on one tile, half the tokens each; 565 so).
    const int group = (warp - 4) >> 2, quad = warp & 3, L = 32 * quad + lane;
    const uint32_t t_lane = tmem + ((uint32_t)(32 * quad) << 16);
    constexpr int kParts = kTile / 32;
    int j = 0, seg = 0;     // tiles so far; pieces begun
    int buf = 0, bph = 0;   // the next tile's buffer and its parity
    auto last_buf = [&] { return buf == 0 ? S::kBufs - 1 : buf - 1; };  // the buffer before it
    auto last_ph = [&] { return buf == 0 ? bph ^ 1 : bph; };
    // Once a wait has expired (failed) nothing more is waited for, computed or written, but the
    // warps go on meeting.
    do {
      const SeqT& s = walk.seq;
      const int n = walk.count(p), kvh = walk.kv_head(), r0 = walk.row_begin(), rows = walk.rows();
      // Copies of each row, a power of two, of `span` rows each; copy `rep` weighs the 32-token
      // parts of a tile that are rep modulo their number.
      // (None for one tile: adding them up would take longer than they save, 12.4 against 11.5 us for 100 tokens.)
      const int rep_shift = rows > 64 || n < 2 ? 0 : rows > 32 || kTile == 64 ? 1 : 2;
      const int copies = 1 << rep_shift, span = kRows >> rep_shift, rep = L / span, row = L - rep * span;
      const bool live = row < rows;
      const int token = (r0 + (live ? row : 0)) / p.group, head = kvh * p.group + (r0 + (live ? row : 0)) - token * p.group;
      ++seg;
      float scale = fabsf(p.scale_log2);  // (its sign goes into the queries)
      if (n > 0 && !failed) {
        // ---- queries: half a row a thread
        constexpr int kVec = D / 16;  // 16-byte pieces
        uint4 v[kVec];
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.q) +
                                                          ((s.row0 + token) * p.q_tok + head * p.q_head + group * (D / 2)) * 2);
#pragma unroll
        for (int k = 0; k < kVec; ++k) v[k] = live ? src[k] : make_uint4(0u, 0u, 0u, 0u);
        uint32_t* w = reinterpret_cast<uint32_t*>(v);
        if (kFp8 && kQBf16) {
          // bf16 rows enter the f16 product scaled by a power of two that brings their largest
          // element into [2^15, 2^16): exact but for elements below 2^-29 of it, whose
          // rounding is at most 2^-40 of the largest.
          uint32_t mx = 0;
#pragma unroll
          for (int k = 0; k < 4 * kVec; ++k) mx = max(mx, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
          sm.m[group][L] = __uint_as_float(mx);
          named_bar_sync(12 + quad, 64);
          mx = max(mx, __float_as_uint(sm.m[1 - group][L]));
          named_bar_sync(12 + quad, 64);
          const int ex = min(max((int)(mx >> 7), 16), 254);  // biased exponent
          const float down = __uint_as_float((uint32_t)(269 - ex) << 23);
#pragma unroll
          for (int k = 0; k < 4 * kVec; ++k) {
            const float2 f = unpack<true>(w[k]);
            w[k] = pack<false>(f.x * down, f.y * down);
          }
          scale = fmaxf(scale * __uint_as_float((uint32_t)(ex - 15) << 23), 1.17549435e-38f);  // (not 0: hidden scores are infinities)
        }
        if (p.scale_log2 < 0.f) {
#pragma unroll
          for (int k = 0; k < 4 * kVec; ++k) w[k] ^= 0x80008000u;
        }
#pragma unroll
        for (int c = 0; c < 4 * kVec; c += 16)
          tc::st16(t_lane + S::kQ + group * (D / 4) + c, *reinterpret_cast<uint32_t(*)[16]>(w + c));
        tc::st_wait();
        tc::fence_before_thread_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.bar.q_ready));
      } else if (n > 0 && kFp8 && kQBf16) {
        named_bar_sync(12 + quad, 64);
        named_bar_sync(12 + quad, 64);
      }
      // ---- what this row sees
      Sight see;
      see.base = s.base;
      see.len = s.len;
      see.words = p.words;
      see.mask = nullptr;
      const int at = s.base + token;  // its place in the cache
      int pos = at;
      see.hi = p.mask ? s.base : at + 1;
      if (p.mask && live) {
        see.mask = p.mask + (s.row0 + token) * p.words;
        if (p.window > 0) pos = max(s.base, p.positions[s.row0 + token]);
      }
      see.lo = p.window > 0 && pos >= p.window ? pos + 1 - p.window : 0;
      see.sinks = p.window > 0 ? min(p.sinks, see.hi) : 0;
      if (!live) {  // a row that is not there: its sums (of zero queries) go nowhere
        see.lo = 0;
        see.hi = 0x7fffffff;
      }

      // The piece's place in the workspace; until it is written there the sums outside TMEM, four columns of
      // each lane after the other.
      auto piece = [&] { return ((int)blockIdx.x * 2 + (seg == 1 ? 0 : 1)) * kRows; };
      auto folded = [&](int c) { return reinterpret_cast<float4*>(p.part_o + (int64_t)piece() * D) + c / 4 * kRows + L; };
      float m = -INFINITY, l = 0.f;
      auto advance = [&] {
        ++j;
        if (++buf == S::kBufs) {
          buf = 0;
          bph ^= 1;
        }
      };
      for (int i = 0; i < n; ++i, advance()) {
        if ((j & 1) != group) continue;
        if (!failed && !wait_all(&sm.bar.s_full[buf], bph)) failed = true;
        tc::fence_after_thread_sync();
        const uint32_t ts = t_lane + S::kS + (uint32_t)buf * kTile;
        const int key0 = s.place(walk.t_beg + i) * kTile;
        const bool plain = __all_sync(0xffffffffu, see.lo <= key0 && key0 + kTile <= see.hi);  // nothing is hidden
        auto hide = [&](uint32_t (&x)[32], int c) {
          const uint32_t vis = see.bits(key0 + 32 * c);
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = vis >> e & 1u ? x[e] : 0xff800000u;  // -infinity
        };
        // ---- the tile's maximum
        float mx = -INFINITY;
        if (!failed) {
          float y[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // (four chains)
#pragma unroll 1
          for (int c = rep; c < kParts; c += copies) {
            uint32_t v[32];
            tc::ld32(ts + 32 * c, v);
            tc::ld_wait();
            if (!plain) hide(v, c);
#pragma unroll
            for (int e = 0; e < 32; e += 2) y[e / 2 % 4] = max3(y[e / 2 % 4], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
          }
          mx = max3(fmaxf(y[0], y[1]), y[2], y[3]);
          if (mx != -INFINITY) mx = kCap ? capped(mx * scale, p.cap_out, p.cap_inv) : mx * scale;
        }
        // ---- the maximum in use: what the tile before this one left, raised if it is passed by far
        if (i > 0) {
          named_bar_sync(2 + 2 * quad + (j & 1), 64);
          const float last = sm.m_used[L];
          l *= m == -INFINITY ? 0.f : fast_exp2(m - last);
          m = last;
        }
        const bool raise = mx > m + kRaise || (m == -INFINITY && mx > m);
        const float alpha = raise ? fast_exp2(m - mx) : 1.f;  // 0 where m was -inf
        if (raise) {
          l *= alpha;
          m = mx;
        }
        if (i + 1 < n) {
          sm.m_used[L] = m;
          named_bar_arrive(2 + 2 * quad + ((j + 1) & 1), 64);
        }
        if (i > 0 && i % S::kFold == 0) {
          // O goes to the sums outside TMEM and begins anew.  (kFold is even: one group does this for a whole piece.)
          if (!failed && !wait_all(&sm.bar.p_free[last_buf()], last_ph())) failed = true;
          tc::fence_after_thread_sync();
          const bool first = i == S::kFold;
          const float f = first || m == -INFINITY ? 0.f : fast_exp2(sm.m_fold[L] - m);
          if (!failed) fold_out<D>(t_lane + S::kO, folded(0), alpha, f, first);
          sm.m_fold[L] = m;
        } else if (i > 0 && !failed && __any_sync(0xffffffffu, raise)) {
          // O holds the products of the tiles before this one
          if (!wait_all(&sm.bar.p_free[last_buf()], last_ph())) failed = true;
          tc::fence_after_thread_sync();
#pragma unroll 1
          for (int c = 0; c < D && !failed; c += 16) {  // (16 columns at a time: the tile's scores are live)
            uint32_t o[16];
            tc::ld16(t_lane + S::kO + c, o);
            tc::ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::st16(t_lane + S::kO + c, o);
          }
        }
        if (failed) continue;
        // ---- weights, in two terms, over the scores that they came from
        const float sub = m == -INFINITY ? 0.f : m - kShift;
        float2 sum = make_float2(0.f, 0.f);
        const float2 ss = make_float2(kCap ? 1.f : scale, kCap ? 1.f : scale), nn = make_float2(-sub, -sub);
        // (A loop that is not unrolled: with 64 or 128 tokens in one piece of code, or loads ahead of the part
        // in work, registers are spilled, 608, 748 and 679 us for 565 of the same case.)
#pragma unroll 1
        for (int c = 0; c < kParts; ++c) {
          uint32_t w[32];
          if ((c & (copies - 1)) == rep) {
            uint32_t v[32];
            tc::ld32(ts + 32 * c, v);
            tc::ld_wait();
            if (kCap) {
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(capped(__uint_as_float(v[e]) * scale, p.cap_out, p.cap_inv));
            }
            if (!plain) hide(v, c);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 z = __ffma2_rn(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), ss, nn);
              z.x = fast_exp2(z.x);
              z.y = fast_exp2(z.y);
              w[e] = pack<kBf16>(z.x, z.y);
              const float2 low = __ffma2_rn(unpack<kBf16>(w[e]), make_float2(-1.f, -1.f), z);
              w[16 + e] = pack<kBf16>(low.x, low.y);
              sum = __fadd2_rn(sum, z);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = 0u;
          }
          tc::st32(ts + 32 * c, w);
          if (c % (kParts / 2) == kParts / 2 - 1) {  // a half of the tile: its product may begin
            tc::st_wait();
            tc::fence_before_thread_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.bar.p_full[buf][c / (kParts / 2)]));
          }
        }
        l += sum.x + sum.y;
      }
      // ---- the unit's (or its piece's) end
      if (n > 0 && !failed) {
        if (!wait_all(&sm.bar.p_free[last_buf()], last_ph())) failed = true;
        tc::fence_after_thread_sync();
      }
      // The copies of a row, and the groups' sums: O is relative to the later group's maximum
      sm.m[group][L] = m;
      sm.l[group][L] = l;
      named_bar_sync(1, 256);
      const float own = fmaxf(sm.m[0][L], sm.m[1][L]);
      float mm = -INFINITY, ll = 0.f;
      for (int x = row; x < kRows; x += span) mm = max3(mm, sm.m[0][x], sm.m[1][x]);
      for (int x = row; x < kRows; x += span)
        for (int g = 0; g < 2; ++g) ll = fmaf(sm.l[g][x], sm.m[g][x] == -INFINITY ? 0.f : fast_exp2(sm.m[g][x] - mm), ll);
      float f = own == -INFINITY ? 0.f : fast_exp2(own - mm);  // what this copy's sums are multiplied by
      m = mm;
      l = ll;
      if (n > S::kFold && !failed) {
        const float g = sm.m_fold[L] == -INFINITY ? 0.f : fast_exp2(sm.m_fold[L] - own);
        unfold_out<D / 2>(t_lane + S::kO + group * (D / 2), folded(group * (D / 2)), g);
        tc::st_wait();
      }
      named_bar_sync(1, 256);  // (they are written again at the next unit's end, and the piece takes the folded sums' place)
      const bool summed = n > 0 && !failed;  // there is something in O
      if (!summed) f = 0.f;
      const bool whole = walk.whole(), writes = live && rep == 0 && !failed;
      if (whole) f = l == 0.f ? 0.f : f * (p.v_scale / l);
      const int64_t out_row = (s.row0 + token) * p.hq + head;
#pragma unroll 1
      for (int c = group * (D / 2); c < (group + 1) * (D / 2); c += 16) {
        uint32_t o[16];
        if (summed) {
          tc::ld16(t_lane + S::kO + c, o);
          tc::ld_wait();
        }
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = f == 0.f ? 0.f : __uint_as_float(o[e]) * f;
        if (rep_shift > 0) {
          // Copies: the group's threads add them up, four columns of a row each
          if (live) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(&sm.stage[group][L][e]) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
          }
          named_bar_sync(10 + group, 128);
          for (int y = L >> 2; y < rows && !failed; y += 32) {
            const float* const from = &sm.stage[group][y][4 * (L & 3)];
            auto copy = [&](int n) { return *reinterpret_cast<const float4*>(from + n * span * 20); };
            float4 u = copy(0);
            const float4 w = copy(1);
            u = make_float4(u.x + w.x, u.y + w.y, u.z + w.z, u.w + w.w);
            if (rep_shift > 1) {
              const float4 a = copy(2), b = copy(3);
              u = make_float4(u.x + (a.x + b.x), u.y + (a.y + b.y), u.z + (a.z + b.z), u.w + (a.w + b.w));
            }
            const int d = c + 4 * (L & 3);
            if (whole) {
              const int t = (r0 + y) / p.group, h = kvh * p.group + r0 + y - t * p.group;
              *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + (((s.row0 + t) * p.hq + h) * D + d) * 2) =
                  make_uint2(pack<kQBf16>(u.x, u.y), pack<kQBf16>(u.z, u.w));
            } else {
              *reinterpret_cast<float4*>(p.part_o + (int64_t)(piece() + y) * D + d) = u;
            }
          }
          named_bar_sync(10 + group, 128);
          continue;
        }
        if (!writes) continue;
        if (whole) {
          uint4 u[2];
          uint32_t* w = reinterpret_cast<uint32_t*>(u);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = pack<kQBf16>(x[2 * e], x[2 * e + 1]);
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + (out_row * D + c) * 2);
          dst[0] = u[0];
          dst[1] = u[1];
        } else {
          float4* dst = reinterpret_cast<float4*>(p.part_o + (int64_t)(piece() + row) * D + c);
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        }
      }
      if (writes && group == 0) {
        if (!whole)
          p.part_ml[piece() + row] = make_float2(m - kShift, l);
        else if (p.lse)
          p.lse[out_row] = l == 0.f ? -INFINITY : (m - kShift) * 0.6931471805599453f + logf(l);
      }
      if (p.record && L == 0 && group == 0 && walk.t_beg == 0 && !whole && !failed) {
        // The unit begins here; it ends in the gang that has its last tile.
        const int64_t last = sm.end - walk.left + s.tiles - 1;
        p.record[blockIdx.x] = Record{s.row0, kvh, r0, rows, walk.unit & ((1 << p.gang_shift) - 1), gang, share_of(last, sm.total, sm.n_gangs),
                                      seg == 1 ? 0 : 1};
      }
      tc::fence_before_thread_sync();  // (O has been read before the next unit's first weights are there)
    } while (walk.next(p));
  } else {
    // ---------------------------------------------------------------- E4M3 -> f16
    // K and then V of each tile.
    if constexpr (kFp8) {
      // A thread's 16-byte pieces of a tile: one column of them, every kRowStep-th row (a multiple of 8, so
      // that its place in a swizzled row is the same), each two pieces of f16.  Eight lanes have four pieces of a
      // row's chunk and four of the next row's other chunk: they fill all banks when they load, and, as the swizzle
      // puts an odd row's first halves where an even one's second ones lie, when they store either half.
      constexpr int kRowStep = 128 / (D / 16), kMine = kTile / kRowStep;
      const int t = threadIdx.x & 127, odd = (t >> 2) & 1, chunk = (t >> 3) % S::kChunks ^ (S::kChunks > 1 ? odd : 0);
      const int row0 = 2 * ((t >> 3) / S::kChunks) + odd, piece0 = row0 * (D / 16) + chunk * 4 + (t & 3);
      const uint32_t first = (uint32_t)(chunk * (kTile * 128) + row0 * 128 + ((2 * (t & 3) ^ (row0 & 7)) << 4));
      int rs = 0, rph = 0, st = 0, ph = 1;
      do {
        const int n = walk.count(p);
        for (int i = 0; i < n && !failed; ++i) {
          const int key0 = walk.seq.place(walk.t_beg + i) * kTile;
          const bool edge = walk.seq.edge(key0, kTile);
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            uint64_t* const raw_full = (kv ? sm.bar.vr_full : sm.bar.kr_full) + rs;
            uint64_t* const free_ = (kv ? sm.bar.v_free : sm.bar.k_free) + st;
            if (!wait_all(raw_full, rph)) {
              failed = true;
              break;
            }
            const uint4* src = reinterpret_cast<const uint4*>((kv ? svr : skr) + rs * S::kRaw);
            uint8_t* dst = (kv ? sv : sk) + st * S::kSlot;
            // (all loads before the first store: the compiler cannot know that they are of other bytes)
            uint4 v[kMine];
#pragma unroll
            for (int k = 0; k < kMine; ++k) v[k] = src[piece0 + 128 * k];
            if (!wait_all(free_, ph)) {
              failed = true;
              break;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32((kv ? sm.bar.vr_free : sm.bar.kr_free) + rs));  // (it is in registers)
            if (edge && kv) {
              // Rows of V that nothing sees may hold anything; 0 * NaN is NaN, so they are zeroed.
#pragma unroll
              for (int k = 0; k < kMine; ++k)
                if (walk.seq.hidden(key0 + row0 + kRowStep * k)) v[k] = make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int k = 0; k < kMine; ++k) {
              const uint2 a = widen(v[k].x), b = widen(v[k].y), c = widen(v[k].z), d = widen(v[k].w);
              uint8_t* to = dst + k * (kRowStep * 128);
              *reinterpret_cast<uint4*>(to + first) = make_uint4(a.x, a.y, b.x, b.y);
              *reinterpret_cast<uint4*>(to + (first ^ 16)) = make_uint4(c.x, c.y, d.x, d.y);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32((kv ? sm.bar.v_full : sm.bar.k_full) + st));
          }
          if (++rs == S::kNR) {
            rs = 0;
            rph ^= 1;
          }
          if (++st == S::kNK) {
            st = 0;
            ph ^= 1;
          }
        }
      } while (!failed && walk.next(p));
    }
  }

  // ---------------------------------------------------------------- teardown
  tc::fence_before_thread_sync();
  if (__syncthreads_or(failed)) {
    // A wait expired: let the products that the issuer started complete before TMEM is freed.
    if (warp == 1) {
      if (tc::elect_one()) tc::commit(smem_u32(&sm.bar.drain));
      __syncwarp();
      mbar_wait(smem_u32(&sm.bar.drain), 0, err);
    }
    tc::fence_before_thread_sync();
    __syncthreads();
  }
  if (warp == 1) {
    tc::fence_after_thread_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// (volatile: the compiler would otherwise put each load next to its use)
template <int kN>
__device__ __forceinline__ void load_l2(const float* p, float (&v)[kN]) {
  if constexpr (kN == 2)
    asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "l"(p));
  else
#pragma unroll
    for (int i = 0; i < kN; i += 4)
      asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3]) : "l"(p + i));
}

// Joins the pieces of the units that lie in several blocks' shares, in the order of their
// tiles: a warp per row.  Up to 32 pieces' maxima and sums come at once, a lane each, and their
// outputs kBatch at a time, none of which waits for another.  Two at a time where units have few pieces (16
// sequences of 16384 tokens, 32 drafts, head dim 64, graphs of 21 calls: 132.2 us; 134.2 with 8), eight for long
// lists (one of 2048 tokens, up to 14 pieces a unit: 13.7 us, 15.1 with 2; of 8192: 18.8, 20.2).
template <int D, bool kQBf16, int kBatch>
__global__ void __launch_bounds__(256) tree_attn_join_kernel(const __grid_constant__ Params p) {
  constexpr int kN = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Record u = p.record[blockIdx.x];
  const int lane = threadIdx.x & 31, row = (int)blockIdx.y * 8 + ((int)threadIdx.x >> 5);
  if (u.last < 0 || row >= u.rows) return;
  auto piece = [&](int c) { return (int64_t)(2 * ((c << p.gang_shift) + u.lane) + (c == u.first ? u.first_slot : 0)) * kRows + row; };
  float m = -INFINITY, l = 0.f, x[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) x[i] = 0.f;
  for (int c1 = u.first; c1 <= u.last; c1 += 32) {
    const int count = min(32, u.last + 1 - c1);
    float ml[2] = {-INFINITY, 0.f};
    if (lane < count) load_l2<2>(reinterpret_cast<const float*>(p.part_ml + piece(c1 + lane)), ml);
    float f = 1.f, g = 0.f;  // what the sums so far, and this lane's piece, are multiplied by
    for (int c0 = 0; c0 < count; c0 += kBatch) {
      float v[kBatch][kN];
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
        if (c0 + e < count) load_l2<kN>(p.part_o + piece(c1 + c0 + e) * D + lane * kN, v[e]);
      if (c0 == 0) {
        float mn = fmaxf(m, ml[0]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        f = m == -INFINITY ? 0.f : fast_exp2(m - mn);
        g = ml[0] == -INFINITY ? 0.f : fast_exp2(ml[0] - mn);
        m = mn;
        float sum = ml[1] * g;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = fmaf(l, f, sum);
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] *= f;
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        if (c0 + e >= count) break;
        const float w = __shfl_sync(0xffffffffu, g, c0 + e);
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = fmaf(v[e][i], w, x[i]);
      }
    }
  }
  const int r = u.row + row, token = r / p.group, head = u.kv_head * p.group + r - token * p.group;
  const int64_t out_row = (u.row0 + token) * p.hq + head;
  const float inv = l == 0.f ? 0.f : p.v_scale / l;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + (out_row * D + lane * kN) * 2);
#pragma unroll
  for (int i = 0; i < kN; i += 2) dst[i / 2] = pack<kQBf16>(x[i] * inv, x[i + 1] * inv);
  if (lane == 0 && p.lse) p.lse[out_row] = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

template <int kCache, int D, bool kCap>
cudaError_t launch_instance(const Params& p, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
  using S = Shape<kCache, D>;
  constexpr size_t smem = S::kData + sizeof(Smem<S::kThreads>);
  static_assert(smem <= 227 * 1024, "shared memory");
  static_assert(S::kNK <= 5 && S::kNV <= 5 && S::kNR <= 4, "barrier arrays");
  static_assert(S::kQ + D / 2 <= 512, "TMEM columns");
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(tree_attn_kernel<kCache, D, kCap>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kGrid);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, tree_attn_kernel<kCache, D, kCap>, p, k_map, v_map)) != cudaSuccess || !p.record) return e;
  cfg.gridDim = dim3(kGrid, p.row_groups);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  constexpr bool kQBf16 = kCache == kCacheBf16 || kCache == kCacheE4m3;
  return cudaLaunchKernelEx(&cfg, p.long_lists ? tree_attn_join_kernel<D, kQBf16, D == 256 ? 4 : 8> : tree_attn_join_kernel<D, kQBf16, 2>, p);
}

template <int kCache>
cudaError_t launch_cache(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
  const bool cap = p.cap_out != 0.f;
  switch (d) {
    case 64: return cap ? launch_instance<kCache, 64, true>(p, k_map, v_map, stream) : launch_instance<kCache, 64, false>(p, k_map, v_map, stream);
    case 128: return cap ? launch_instance<kCache, 128, true>(p, k_map, v_map, stream) : launch_instance<kCache, 128, false>(p, k_map, v_map, stream);
    default: return cap ? launch_instance<kCache, 256, true>(p, k_map, v_map, stream) : launch_instance<kCache, 256, false>(p, k_map, v_map, stream);
  }
}

cudaError_t read_errors_here(uint32_t* word) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(word, g_tree_attn_err, sizeof(uint32_t));
  return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_tree_attn_err, &zero, sizeof(uint32_t));
}

}  // namespace

}  // namespace ta
}  // namespace gqa
