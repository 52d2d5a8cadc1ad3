// paged_attn.cuh -- attention of one new token per sequence over a paged K/V
// cache (f16, bf16 or E4M3 pages), grouped queries, split over the cache's
// length and joined, for sm_103a.
//
// Mathematics.  For sequence b, query head h and KV head g = h / G,
//   s_t = cap( (q . K_t) * scale ),  cap(x) = softcap * tanh(x / softcap) if softcap > 0,
//   out = v_scale * sum_t exp(s_t - m) V_t / sum_t exp(s_t - m),  lse = ln sum_t exp(s_t)
// over max(0, len - window) <= t < len.  A range of tokens is summed as
// (m, l, o) with the running maximum m, l = sum exp(s - m) and o = sum exp(s -
// m) V in f32; ranges join by rescaling to the larger m.
//
// What bounds it: HBM -- every K/V byte is read once for 4 G / w flops (w bytes
// per element).  FMA units keep up only to G of about 6 at 16 bits, so both
// products run on the tensor cores, transposed: S^T = K Q^T and O^T = V^T P^T,
// with 16 keys (then 16 output elements) on the M side and 8 heads on the N
// side.  The cache is the A operand straight from shared memory, a group of up
// to 8 heads costs the same as one, and the accumulators of the output are D / 4
// registers for each 8 heads.  Up to 8 heads the warp-level mma is enough: at HBM
// speed the tensor pipe is busy for 14 % (bf16) or 26 % (E4M3) of the cycles.
// From 16 heads on E4M3 pages are bound by the widening and the products (64 x
// 60000 on one KV head: 96 us for 73 of HBM), and more than 16 heads by going
// through a tile once for each 16 (32 heads: 208 us in bf16 for 145 of HBM, 179
// in E4M3); accumulators in TMEM, with the keys on the M side, are not tried here.
//
//  * Grid: one block per SM, each with an equal share of the work of all
//    (sequence, KV head, block of heads) units, whatever the lengths -- the
//    shares are computed on the device from seq_lens.  Blocks go in gangs of 8 (fewer if
//    8 does not divide the units of a sequence): a gang has a share of the sequences'
//    tokens, in order, and each of its blocks goes through them for other units, so
//    that the heads of a token are read at the same time (rows of different heads side
//    by side in DRAM, and two blocks of heads that need the same K and V: 48 sequences
//    of up to 16001 tokens, token-major E4M3, 137 us without gangs, 124 with (one term a
//    weight); 64 x 8192 head-major 160 and 155; 32 heads on one KV head, 64 x 60000, 276
//    and 223; against 0.1 us of a small call, and 24.3 and 24.8 us for 190 sequences of
//    128 tokens).
//    A unit that lies inside one block is written by it; the pieces of one that does not
//    go to the workspace (at most two per block), and a second kernel joins them.
//  * Producer warps move tiles of 32 to 128 tokens with tensor-map TMA copies
//    into a ring of 128 KB: any page size and cache order is a box of the
//    map.  The 128-byte (64-byte) swizzle makes every ldmatrix conflict-free.
//  * Eight consumer warps (four at head dim 256), each with its own 32 (16) keys of
//    a tile and its own (m, l, o); groups of warps take tiles in turn, so that one
//    tile's softmax overlaps another one's products.  They meet at the end of a
//    unit only.
//
// Measured on GB300 (time in a graph): 64 sequences of up to 8192 tokens, 32/8 heads,
// bf16: 155 us, 6.94 TB/s; 20 of 8192: 99 us, 6.75 TB/s; 48 of up to 16001, 64/8 heads,
// E4M3: 126 us, 6.27 TB/s; 8 of 131072, f16: 585 us, 7.34 TB/s.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "paged_attn_host.h"

namespace gqa {
namespace pa {

namespace {

__device__ uint32_t g_paged_attn_err;  // of this translation unit's kernels

}  // namespace

template <int kCache, int D, int NT>
struct Shape {
  static constexpr int kEsz = kCache >= kCacheE4m3 ? 1 : 2;
  static constexpr int kRow = D * kEsz;                     // bytes of a token's row
  static constexpr int kChunk = kRow < 128 ? kRow : 128;    // bytes of a swizzled row in shared memory
  static constexpr int kTile = tile_of(kRow);                // tokens per stage
  // Consumer warps: eight, or four where the accumulators need more than the 168
  // registers a thread that twelve warps leave.
  static constexpr int kWarps = D > 128 ? 4 : 8;
  // Four producer warps: for K and V, and for the even and the odd tiles.  (An issued
  // copy takes its warp about 130 cycles; with pages of 16 tokens a tile of E4M3 has
  // eight: 197 us with one producer, 177 with two, 162 with four on 48 sequences of up to
  // 16001 tokens.  They cost no registers: nine warps leave as many a thread as twelve.)
  static constexpr int kProducers = 4;
  static constexpr int kThreads = (kWarps + kProducers) * 32;
  // 16-key blocks that a warp takes of a tile: two give it two independent sums of
  // products and one reduction for 32 keys (1.28x over one block on 48 sequences of up to
  // 16001 tokens in E4M3 pages of 64; 16 heads on one KV head, 64 x 60000: 95 us with two,
  // 106 with one); with 16 heads and long rows the registers that the second one needs would
  // spill (64 x 8192 tokens in bf16, 16 heads a KV head: 184 us with two, 164 with one).
  static constexpr int kBlocks = NT == 2 && D > (kEsz == 1 ? 128 : 64) ? 1 : 2;
  static constexpr int kGroupWarps = kTile / (16 * kBlocks);  // warps that share a tile
  static constexpr int kGroups = kWarps / kGroupWarps;      // tiles in work at a time
  static constexpr int kHalf = kTile * kRow;                // bytes of K (and of V) of a stage
  // What starting and ending a unit costs, in tiles: about the time of 96 KB of K and V
  // for 8 heads, twice that for 16.  (12 sequences of up to 8192 tokens in bf16: 43.0 us
  // without it, 38.3 with 2 or 8 tiles; with 16 heads a KV head 62.6 us, 47.5 with 2,
  // 43.9 with 8; 48 of up to 16001 in E4M3: 147.4, 140.5 with 2, 136.4 with 8.  These before
  // blocks went in gangs; with them 35.9, 40.6 and, one term a weight as before, 124 us, and the
  // same with 64 or 144 KB.)
  static constexpr int kUnitWork = NT * 96 * 1024 / (2 * kHalf);
  static constexpr int kRoom = 128 * 1024;  // the warps' join takes up to 68 KB
  // A whole number of groups' turns, so that a stage always belongs to one group (a
  // wait on its barrier can then never be a phase behind).
  static constexpr int kStages = kRoom / (2 * kHalf) / kGroups * kGroups;
  static_assert(kStages >= kGroups && kStages % (kProducers / 2) == 0, "whole turns of groups and producers");
};

// Gang i of n has the work [total * i / n, total * (i + 1) / n).  (32-bit divisions where they do.)
__device__ __forceinline__ int64_t share_begin(int i, int64_t total, int n) {
  const int64_t x = total * i;
  return x >> 32 ? x / n : (int64_t)((uint32_t)x / (uint32_t)n);
}
// The gang that has a tile: the last one whose share begins at or before it.
__device__ __forceinline__ int share_of(int64_t tile, int64_t total, int n) {
  const int64_t x = (tile + 1) * n + total - 1;
  return (int)(x >> 32 ? x / total : (int64_t)((uint32_t)x / (uint32_t)total)) - 1;
}

template <int kWarps, int D, int NT>
struct Smem {
  static constexpr int kRows = 8 * NT;
  alignas(16) uint8_t q[2][kRows][D * 2 + 16];
  alignas(16) float o[kWarps][kRows][D + 4];  // (the odd row length spreads the banks)
  float m[kWarps][kRows];
  float l[kWarps][kRows];
  alignas(8) uint64_t full[32];
  uint64_t empty[32];
  uint64_t q_full[2];
  uint64_t q_empty[2];
  int64_t scan[kWarps + 4];
  int most[kWarps + 4];
  int64_t total;  // work of one block of each gang
  int n_gangs;    // gangs with a share
  int64_t end;    // of this block's share
  int64_t rem;    // the share's first tile within its first sequence,
  int b0;         // and that sequence
};

__device__ __forceinline__ void ldsm4(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool kBf16>
__device__ __forceinline__ void mma(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  if (kBf16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)two));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float f16_lo(uint32_t x) { return __half2float(__ushort_as_half((unsigned short)x)); }
__device__ __forceinline__ float f16_hi(uint32_t x) { return __half2float(__ushort_as_half((unsigned short)(x >> 16))); }
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

__device__ __forceinline__ void tma_5d(uint32_t dst, const CUtensorMap* map, int slot, int head, int page, uint32_t bar,
                                       uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
      "l"(map), "r"(0), "r"(slot), "r"(0), "r"(head), "r"(page), "r"(bar), "l"(policy)
      : "memory");
}

// Which of its gang's blocks a block is, or the one that has a unit.
__device__ __forceinline__ int lane_of_gang(const Params& p, int i) { return i & ((1 << p.gang_shift) - 1); }

// First token and number of tiles of a sequence of the given length.
template <int kTile>
struct Span {
  int len, first, tile0, tiles;
  __device__ __forceinline__ Span(const Params& p, int32_t seq_len) {
    const int64_t cap = p.max_pages << p.page_shift;
    const int64_t n = seq_len;
    len = (int)(n < 0 ? 0 : (n > cap ? cap : n));
    first = p.window > 0 && len > p.window ? len - p.window : 0;
    tile0 = first / kTile;
    tiles = (len + kTile - 1) / kTile - tile0;  // (a capacity is at most 2^30 tokens)
  }
};

// Walks the units of a block's share.  Shares are counted in the work of a unit: its
// tiles and, before them, what starting and ending a unit costs in tiles (kUnitWork);
// or, by_unit, in whole units.  (A share has less than 2^31: the host sees to it.)
template <int kTile, int kUnitWork>
struct Walk {
  int left;   // of the share: from the piece's first tile on; by_unit: units behind this one
  int b;      // sequence
  int unit;   // within the sequence: kv head * head blocks + head block; the next one is 2^gang_shift further
  int t_beg;  // first tile of the piece within the unit, and one past its last
  int t_end;
  Span<kTile> span;
  bool by_unit;
  // From `rem` into the sequence's work (of one block of a gang) on; valid() says whether there is a tile.
  __device__ __forceinline__ Walk(const Params& p, int share, int b_, int64_t rem, bool by_unit_)
      : b(b_), span(p, p.seq_lens[b_]), by_unit(by_unit_) {
    if (by_unit) {
      unit = (int)rem;
      t_beg = 0;
      t_end = span.tiles;
      left = share - 1;
    } else {
      const int work = span.tiles + kUnitWork;
      unit = (int)(rem / work);
      const int at = (int)(rem - (int64_t)unit * work);
      t_beg = max(0, at - kUnitWork);
      left = share - max(0, kUnitWork - at);
      t_end = min(span.tiles, t_beg + left);
    }
    unit = (unit << p.gang_shift) + lane_of_gang(p, blockIdx.x);
  }
  __device__ __forceinline__ bool valid() const { return by_unit || left > 0; }
  // To the next piece; false at the end of the share.
  __device__ __forceinline__ bool next(const Params& p) {
    left -= by_unit ? 1 : t_end - t_beg + kUnitWork;
    if (by_unit ? left < 0 : left <= 0) return false;
    t_beg = 0;
    unit += 1 << p.gang_shift;
    if (unit >= p.hkv * p.head_blocks) {
      unit -= p.hkv * p.head_blocks;
      do {
        if (++b >= p.batch) return false;
        span = Span<kTile>(p, p.seq_lens[b]);
      } while (span.tiles == 0);
    }
    t_end = by_unit ? span.tiles : min(span.tiles, left);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return t_beg == 0 && t_end == span.tiles; }
};

// cap * tanh(s / cap), to 2^-19 of itself.  With u = s / cap and |u| >= 1/4, tanh u = 1 - 2 /
// (exp(2 u) + 1), whose error of up to 1.6 * 2^-22 (the exponential's and the reciprocal's) is
// 2^-19 of it at 1/4 and would be any multiple of it nearer to 0.  There the series u - u^3 / 3
// + 2 u^5 / 15 - 17 u^7 / 315 + 62 u^9 / 2835 is taken, 2^-26 off at 1/4, as s (1 + u^2 (...)):
// under a cap far above the scores u may be denormal, and s stays as it is.  (Both are formed
// and one is chosen: the window case with its cap 50 109.7 us, 48 x 16001 over E4M3 pages with
// cap 30 128.7 us; 109.1 and 127.2 with the exponential alone, 115.5 and 134.5 with tanhf.)
__device__ __forceinline__ float capped(const Params& p, float s) {
  const float u = s * p.cap_inv, w = u * u;
  const float series = fmaf(fmaf(fmaf(62.f / 2835.f, w, -17.f / 315.f), w, 2.f / 15.f), w, -1.f / 3.f);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fast_exp2(u * 2.8853900817779268f) + 1.f));
  const float far = fmaf(-2.f * p.cap_out, r, p.cap_out);
  return fabsf(u) < 0.25f ? fmaf(s * w, series, s) : far;
}

// Elements d, d + 1 of a head's output from sums relative to exp2(mm), and its lse.
template <int D, bool kQBf16>
__device__ __forceinline__ void store_out(const Params& p, int64_t row, int d, float x, float y, float mm, float l) {
  const float inv = p.v_scale / l;
  const uint32_t pk = kQBf16 ? pack_bf16(x * inv, y * inv) : pack_f16(x * inv, y * inv);
  *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + (row * D + d) * 2) = pk;
  if (d == 0 && p.lse) p.lse[row] = mm * 0.6931471805599453f + logf(l);
}

namespace {

// (volatile: the compiler would otherwise put each load next to its use)
__device__ __forceinline__ float2 load_l2(const float2* p) {
  float2 v;
  asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}

template <int kCache, int D, int NT>
__global__ void __launch_bounds__(Shape<kCache, D, NT>::kThreads, 1)
    paged_attn_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map) {
  uint32_t* const err = &g_paged_attn_err;
  using S = Shape<kCache, D, NT>;
  constexpr bool kBf16 = kCache == kCacheBf16;
  constexpr bool kFp8 = kCache >= kCacheE4m3;
  constexpr bool kQBf16 = kBf16 || kCache == kCacheE4m3;  // the type of q and of the output
  // A weight enters the product with V as two terms of the pages' type (f16 for E4M3 ones): 22
  // bits of it, 16 in bf16, so that its rounding stays far below the output's.  (One f16 term
  // of 11 bits, over E4M3 pages: 48 sequences of up to 16001 tokens 124 us instead of 126,
  // with 16 heads a KV head 84 instead of 95; but outputs 2e-4 off the f32 form's.)
  constexpr int kUnitWork = S::kUnitWork;
  constexpr int kTile = S::kTile, kWarps = S::kWarps, kThreads = S::kThreads;
  constexpr int kRows = 8 * NT;
  constexpr int kTileShift = kTile == 32 ? 5 : kTile == 64 ? 6 : 7;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = smem_raw;
  Smem<S::kWarps, D, NT>& sm = *reinterpret_cast<Smem<S::kWarps, D, NT>*>(smem_raw + S::kStages * 2 * S::kHalf);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = p.hkv * p.head_blocks;
  const int turns = units >> p.gang_shift, gang = (int)blockIdx.x >> p.gang_shift, gangs = kGrid >> p.gang_shift;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(smem_u32(&sm.full[i]), 2);
      mbar_init(smem_u32(&sm.empty[i]), S::kGroupWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.q_full[i]), 1);
      mbar_init(smem_u32(&sm.q_empty[i]), kWarps);
    }
    fence_mbar_init();
  }
  // Query rows that a unit does not have stay zero or hold an older row: each head is a
  // column of its own in both products.
  for (int i = threadIdx.x; i < (int)sizeof(sm.q) / 16; i += kThreads)
    reinterpret_cast<uint4*>(sm.q)[i] = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  // Launched as a programmatic dependent: what went before on the stream (the append of
  // this step) has ended and is visible from here on.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0 && p.record && !p.record_by_unit) p.record[blockIdx.x].last = -1;

  // ---- this block's share: of the work of every 2^gang_shift-th unit, [T * gang / n, T *
  // (gang + 1) / n), or one whole unit if there are no more units than blocks and none has more than kWholeTiles tiles:
  // to read them takes less time than to join the pieces of a split unit (2 sequences
  // of up to 200 tokens, 8 KV heads: 8.8 us split, 5.6 us whole; 16 of 512: 14.7 and 10.1).
  // Each thread sums the tiles of a contiguous range of sequences; a scan over the
  // threads gives the ranges' starts, and the range that holds the share's first tile
  // is walked by its thread.
  const int64_t per = (p.batch + kThreads - 1) / kThreads;
  const int64_t s0 = threadIdx.x * per < p.batch ? threadIdx.x * per : p.batch;
  const int64_t s1 = s0 + per < p.batch ? s0 + per : p.batch;
  constexpr int kCountAt = 46;  // a sum holds tiles below, and sequences that have any above
  int64_t mine = 0;
  int most = 0;
  for (int64_t b = s0; b < s1; ++b) {
    const Span<kTile> sp(p, p.seq_lens[b]);
    mine += sp.tiles + (sp.tiles ? int64_t(1) << kCountAt : 0);
    most = max(most, sp.tiles);
    if (sp.tiles == 0 && b % kGrid == blockIdx.x) {  // no token: a zero row
      for (int h = 0; h < p.hq; ++h) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + ((int64_t)b * p.hq + h) * D * 2);
        for (int i = 0; i < D / 8; ++i) o[i] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse) p.lse[(int64_t)b * p.hq + h] = -INFINITY;
      }
      if (p.record && p.record_by_unit)
        for (int u = 0; u < units; ++u) p.record[b * units + u].last = -1;
    }
  }
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) {
    sm.scan[warp] = incl;
    sm.most[warp] = most;
  }
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sm.scan[w];
    total += sm.scan[w];
    most = max(most, sm.most[w]);
  }
  before += incl - mine;
  const bool by_unit = most <= kWholeTiles && (total >> kCountAt) * turns <= gangs;
  auto counted = [&](int64_t sum) {
    const int64_t n = sum >> kCountAt;
    return (by_unit ? n : (sum & ((int64_t(1) << kCountAt) - 1)) + n * kUnitWork) * turns;
  };
  before = counted(before);
  total = counted(total);
  mine = counted(mine);
  const int n_gangs = total < gangs ? (int)total : gangs;  // gangs with a share: none is empty
  const bool has_share = gang < n_gangs;
  const int64_t beg = has_share ? share_begin(gang, total, n_gangs) : 0;
  const int64_t end = has_share ? share_begin(gang + 1, total, n_gangs) : 0;
  if (threadIdx.x == 0) {
    sm.total = total;
    sm.n_gangs = n_gangs;
    sm.end = end;
  }
  if (beg < end && beg >= before && beg < before + mine) {
    int64_t rem = beg - before;
    int64_t b = s0;
    for (;; ++b) {
      const int tiles = Span<kTile>(p, p.seq_lens[b]).tiles;
      const int64_t n = (int64_t)(tiles == 0 ? 0 : by_unit ? 1 : tiles + kUnitWork) * turns;
      if (rem < n) break;
      rem -= n;
    }
    sm.b0 = (int)b;
    sm.rem = rem;
  }
  __syncthreads();
  if (beg >= end) return;
  Walk<kTile, kUnitWork> walk(p, (int)(end - beg), sm.b0, sm.rem, by_unit);
  if (!walk.valid()) return;  // (a share that lies before a unit's first tile)

  if (warp >= kWarps) {
    // ---------------- producer ------------------------------------------------
    if (p.starve) return;
    const bool is_v = (warp - kWarps) & 1;
    const int pair = (warp - kWarps) >> 1;
    constexpr int kPairs = S::kProducers / 2;
    // (K and V make room for others in L2 first, also where two blocks of heads read them: the
    // gang reads them at nearly the same time.  Kept last, 32 heads on one KV head, 64 x 60000
    // in bf16, take 209 us instead of 207.6, 20 heads 204 instead of 202.)
    const uint64_t pol = policy_evict_first();
    // (a box and a page are powers of two: the loop below has no division)
    const int box_shift = p.box_shift, page_shift = p.page_shift;
    const int boxes = kTile >> box_shift;  // copies per tile of K (and of V)
    const uint32_t box_bytes = (uint32_t)S::kRow << box_shift;
    const uint32_t lane_dst = smem_u32(ring) + lane * box_bytes;
    int st = pair, ph = 1;  // this pair's next stage, and the parity of the phase that frees it (the first one is free)
    int skip = pair;        // tiles to this pair's next one
    int issued = 0;         // stages issued, up to all of this pair's
    int seg = 0;            // pieces begun
    bool ok = true;
    do {
      const int kvh = walk.unit / p.head_blocks;
      const int h0 = kvh * p.group + (walk.unit - kvh * p.head_blocks) * kRows;
      const int heads = min(kRows, (kvh + 1) * p.group - h0);
      if (warp == kWarps) {
        const int qb = seg & 1;
        if (seg >= 2 && !__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.q_empty[qb]), ((seg >> 1) - 1) & 1, err))) break;
        const uint32_t qf = smem_u32(&sm.q_full[qb]);
        if (lane == 0) mbar_arrive_expect_tx(qf, (uint32_t)heads * D * 2);
        __syncwarp();
        if (lane < heads)
          bulk_g2s_hint(smem_u32(sm.q[qb][lane]),
                        static_cast<const uint8_t*>(p.q) + ((int64_t)walk.b * p.q_seq + (h0 + lane) * p.q_head) * 2, D * 2, qf,
                        policy_evict_last());
      }
      ++seg;
      // Page numbers, 32 copies' worth at a time and one such group ahead (lane l has those of copy l).
      const int32_t* row = p.block_table + (int64_t)walk.b * p.max_pages;
      // This lane's copy, counted from the sequence's first token; copies behind the last
      // token are not made, nor those before the window.
      int c = ((walk.span.tile0 + walk.t_beg + skip) << (kTileShift - box_shift)) + lane;
      const int c_end = ((walk.span.len - 1) >> box_shift) + 1;
      const int c_first = walk.span.first >> box_shift;
      auto page_of = [&](int copy) {
        if (copy < c_first || copy >= c_end) return 0;
        int g = row[copy >> (page_shift - box_shift)];
        if (g < 0 || g >= p.num_pages) {
          atomicOr(err, kErrBadIndex);
          g = 0;
        }
        return g;
      };
      int cur = page_of(c), nxt = page_of(c + 32);
      int at = 0;  // copies of this piece so far, within a group of 32
      int t = walk.t_beg + skip;
      for (; t < walk.t_end; t += kPairs) {
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.empty[st]), ph, err))) {
          ok = false;
          break;
        }
        const int pg = __shfl_sync(0xffffffffu, cur, (at + lane) & 31);
        const bool live = lane < boxes && c >= c_first && c < c_end;
        const uint32_t bar = smem_u32(&sm.full[st]);
        const uint32_t bytes = box_bytes * __popc(__ballot_sync(0xffffffffu, live));
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        if (live) {
          const uint32_t dst = lane_dst + st * 2 * S::kHalf;
          const int slot = (c << box_shift) & ((1 << page_shift) - 1);
          if (is_v)
            tma_5d(dst + S::kHalf, &v_map, slot, kvh, pg, bar, pol);
          else
            tma_5d(dst, &k_map, slot, kvh, pg, bar, pol);
        }
        c += kPairs * boxes;
        at += kPairs * boxes;
        if (at == 32) {
          at = 0;
          cur = nxt;
          nxt = page_of(c + 32);
        }
        issued = min(issued + 1, S::kStages / kPairs);
        st += kPairs;
        if (st >= S::kStages) {
          st = pair;
          ph ^= 1;
        }
      }
      skip = t - walk.t_end;
    } while (ok && walk.next(p));
    // No copy may land after the block has gone.
    if (lane == 0) {
      // (stages before st were last filled in the present round, the others in the one
      // before; an expired wait has waited long enough for the copies behind it too)
      for (int i = pair; i < pair + kPairs * issued; i += kPairs)
        if (!mbar_wait(smem_u32(&sm.full[i]), i < st ? ph ^ 1 : ph, err)) break;
      for (int i = seg > 2 ? seg - 2 : 0; warp == kWarps && i < seg; ++i) mbar_wait(smem_u32(&sm.q_full[i & 1]), (i >> 1) & 1, err);
    }
    return;
  }

  // ---------------- consumers --------------------------------------------------
  const int grp = warp / S::kGroupWarps;
  constexpr int kBlocks = S::kBlocks, kKeys = 16 * kBlocks;
  const int row0 = (warp % S::kGroupWarps) * kKeys;  // this warp's keys of a tile
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  const uint32_t ring_u = smem_u32(ring);
  // This warp's 16-key blocks: the base of the block's copy and its first row in it
  const int box = 1 << p.box_shift;
  uint32_t blk[kBlocks];
#pragma unroll
  for (int j = 0; j < kBlocks; ++j) {
    const int r = row0 + 16 * j;
    blk[j] = (uint32_t)(r / box) * box * S::kRow + (uint32_t)(r % box) * S::kChunk;
  }
  const uint32_t chunk_step = (uint32_t)box * S::kChunk;
  // ldmatrix row of this lane: K rows 0-15 (A operand), V rows 0-15 (transposed A operand)
  const int k_row = (lane & 7) + ((lane >> 3) & 1) * 8;
  const int v_row = kFp8 ? k_row : (lane & 7) + (lane >> 4) * 8;
  const int k_sel = lane >> 4, v_sel = kFp8 ? lane >> 4 : (lane >> 3) & 1;  // which 16 bytes of a 32-byte step
  auto swz = [](int row, int c16) { return S::kChunk == 128 ? (c16 ^ (row & 7)) : (c16 ^ ((row >> 1) & 3)); };
  // 16-byte column c16 of the whole row -> offset within the block
  auto col = [&](int row, int c16) {
    constexpr int kPer = S::kChunk / 16;
    return (uint32_t)(c16 / kPer) * chunk_step + (uint32_t)row * S::kChunk + (uint32_t)swz(row, c16 % kPer) * 16;
  };
  // P keeps f16's full precision down to 2^-28 of the largest weight.
  constexpr float kShift = kBf16 ? 0.f : 14.f;

  int st = grp, ph = 0;  // this group's next stage and the parity that fills it
  int skip = grp;        // tiles to this group's next one
  int seg = 0;
  bool dead = false;  // a wait has expired: nothing more is waited for or computed
  do {
    const int kvh = walk.unit / p.head_blocks;
    const int h0 = kvh * p.group + (walk.unit - kvh * p.head_blocks) * kRows;
    const int heads = min(kRows, (kvh + 1) * p.group - h0);
    const int qb = seg & 1;
    if (!dead && !__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.q_full[qb]), (seg >> 1) & 1, err))) dead = true;
    // Q as the B operand of S^T = K Q^T: column g = head, rows = head-dim elements (for
    // E4M3 pages in the order in which a widened 32-bit word of K gives them).
    uint32_t qf[NT][D / 16][2];
    float sc[NT][2];  // scale of the scores of heads c2, c2 + 1
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint8_t* qr = sm.q[qb][8 * t + g];
      if (!kFp8) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[t][k][0] = *reinterpret_cast<const uint32_t*>(qr + (16 * k + c2) * 2);
          qf[t][k][1] = *reinterpret_cast<const uint32_t*>(qr + (16 * k + c2 + 8) * 2);
        }
      } else {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint2 w = *reinterpret_cast<const uint2*>(qr + (16 * k + 2 * c2) * 2);
          qf[t][k][0] = w.x;
          qf[t][k][1] = w.y;
        }
      }
      sc[t][0] = sc[t][1] = 1.f;
      if (kFp8 && kQBf16) {
        // bf16 rows enter the f16 product scaled by a power of two that brings their
        // largest element into [2^15, 2^16) (65280 is the largest bf16 number there, 65504
        // f16's; the products are summed in f32): exact but for elements below 2^-29 of it,
        // whose rounding is at most 2^-40 of the largest.
        uint32_t mx = 0;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mx = max(mx, qf[t][k][i] & 0x7fffu);
            mx = max(mx, (qf[t][k][i] >> 16) & 0x7fffu);
          }
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int ex = min(max((int)(mx >> 7), 16), 254);  // biased exponent
        const float down = __uint_as_float((uint32_t)(269 - ex) << 23);
        const float up = __uint_as_float((uint32_t)(ex - 15) << 23);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qf[t][k][i] = pack_f16(bf16_lo(qf[t][k][i]) * down, bf16_hi(qf[t][k][i]) * down);
        sc[t][0] = __shfl_sync(0xffffffffu, up, c2 * 4);
        sc[t][1] = __shfl_sync(0xffffffffu, up, c2 * 4 + 4);
      }
      sc[t][0] *= p.scale_log2;
      sc[t][1] *= p.scale_log2;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.q_empty[qb]));
    ++seg;

    float o[NT][D / 16][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }

    int tile = walk.t_beg + skip;
    for (; tile < walk.t_end; tile += S::kGroups) {
      if (dead) continue;
      const int key0 = (walk.span.tile0 + tile) * kTile + row0;  // this warp's first key
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.full[st]), ph, err))) {
        dead = true;
        continue;
      }
      const uint32_t kb = ring_u + st * 2 * S::kHalf, vb = kb + S::kHalf;
      if (key0 < walk.span.len && key0 + kKeys > walk.span.first) {
        const bool edge = key0 + kKeys > walk.span.len || key0 < walk.span.first;
        // ---- S^T = K Q^T
        float s[kBlocks][NT][4];
#pragma unroll
        for (int j = 0; j < kBlocks; ++j)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][t][e] = 0.f;
        if (!kFp8) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int j = 0; j < kBlocks; ++j) {
              uint32_t a[4];
              ldsm4(a, kb + blk[j] + col(k_row, 2 * k + k_sel));
#pragma unroll
              for (int t = 0; t < NT; ++t) mma<kBf16>(s[j][t], a, qf[t][k][0], qf[t][k][1]);
            }
        } else {
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
#pragma unroll
            for (int j = 0; j < kBlocks; ++j) {
              uint32_t w[4];
              ldsm4(w, kb + blk[j] + col(k_row, 2 * k + k_sel));
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t a[4] = {e4m3_to_f16x2(w[2 * i] & 0xffffu), e4m3_to_f16x2(w[2 * i + 1] & 0xffffu),
                                       e4m3_to_f16x2(w[2 * i] >> 16), e4m3_to_f16x2(w[2 * i + 1] >> 16)};
#pragma unroll
                for (int t = 0; t < NT; ++t) mma<false>(s[j][t], a, qf[t][2 * k + i][0], qf[t][2 * k + i][1]);
              }
            }
        }
        if (edge) {
          // V rows outside the sequence may hold anything; 0 * NaN is NaN, so they are zeroed.
#pragma unroll
          for (int j = 0; j < kBlocks; ++j)
            for (int i = lane; i < 16 * (S::kRow / 16); i += 32) {
              const int r = i % 16, c16 = i / 16, key = key0 + 16 * j + r;
              if (key >= walk.span.len || key < walk.span.first)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + blk[j] + col(r, c16)), "r"(0) : "memory");
            }
          __syncwarp();
        }
        // ---- softmax weights: rows (keys) g, g + 8 of each block; columns (heads) c2, c2 + 1
        bool grow = false;  // has a score passed its head's maximum?
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < kBlocks; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float& v = s[j][t][e];
              v *= sc[t][e & 1];
              if (p.cap_out != 0.f) v = capped(p, v);
            }
            if (edge) {
              const int ka = key0 + 16 * j + g, kc = ka + 8;
              if (ka >= walk.span.len || ka < walk.span.first) s[j][t][0] = s[j][t][1] = -INFINITY;
              if (kc >= walk.span.len || kc < walk.span.first) s[j][t][2] = s[j][t][3] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) grow |= s[j][t][e] > m[t][e & 1];
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float alpha[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float x = m[t][i];
#pragma unroll
              for (int j = 0; j < kBlocks; ++j) x = fmaxf(x, fmaxf(s[j][t][i], s[j][t][i + 2]));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
              alpha[i] = x == -INFINITY ? 0.f : fast_exp2(m[t][i] - x);
              m[t][i] = x;
              l[t][i] *= alpha[i];
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[t][i][e] *= alpha[e & 1];
          }
        }
        uint32_t pb[kBlocks][NT][2], pl[kBlocks][NT][2];  // the weights' two terms
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float sub = m[t][i] == -INFINITY ? 0.f : m[t][i];
#pragma unroll
            for (int j = 0; j < kBlocks; ++j) {
              s[j][t][i] = fast_exp2(s[j][t][i] - sub + kShift);
              s[j][t][i + 2] = fast_exp2(s[j][t][i + 2] - sub + kShift);
              l[t][i] += s[j][t][i] + s[j][t][i + 2];
            }
          }
          // P^T as the B operand of O^T = V^T P^T: rows = keys, columns = heads
#pragma unroll
          for (int j = 0; j < kBlocks; ++j) {
            const float* v = s[j][t];
            if (kBf16) {
              const uint32_t x0 = pack_bf16(v[0], v[1]), x1 = pack_bf16(v[2], v[3]);
              pb[j][t][0] = movm_t(x0);
              pb[j][t][1] = movm_t(x1);
              pl[j][t][0] = movm_t(pack_bf16(v[0] - bf16_lo(x0), v[1] - bf16_hi(x0)));
              pl[j][t][1] = movm_t(pack_bf16(v[2] - bf16_lo(x1), v[3] - bf16_hi(x1)));
            } else {
              const uint32_t x0 = pack_f16(v[0], v[1]), x1 = pack_f16(v[2], v[3]);
              pb[j][t][0] = movm_t(x0);
              pb[j][t][1] = movm_t(x1);
              pl[j][t][0] = movm_t(pack_f16(v[0] - f16_lo(x0), v[1] - f16_hi(x0)));
              pl[j][t][1] = movm_t(pack_f16(v[2] - f16_lo(x1), v[3] - f16_hi(x1)));
            }
          }
        }
        // ---- O^T += V^T P^T
        if (!kFp8) {
#pragma unroll
          for (int j = 0; j < kBlocks; ++j)
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              uint32_t a[4];
              ldsm4_t(a, vb + blk[j] + col(v_row, 2 * i + v_sel));
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                mma<kBf16>(o[t][i], a, pb[j][t][0], pb[j][t][1]);
                mma<kBf16>(o[t][i], a, pl[j][t][0], pl[j][t][1]);
              }
            }
        } else {
#pragma unroll
          for (int j = 0; j < kBlocks; ++j)
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              uint32_t w[4];
              ldsm4_t(w, vb + blk[j] + col(v_row, 2 * k + v_sel));
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                // two keys of two neighbouring elements -> the two keys of each element
                const uint32_t lo = __byte_perm(w[2 * i], 0u, 0x3120), hi = __byte_perm(w[2 * i + 1], 0u, 0x3120);
                const uint32_t a[4] = {e4m3_to_f16x2(lo & 0xffffu), e4m3_to_f16x2(lo >> 16), e4m3_to_f16x2(hi & 0xffffu),
                                       e4m3_to_f16x2(hi >> 16)};
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                  mma<false>(o[t][2 * k + i], a, pb[j][t][0], pb[j][t][1]);
                  mma<false>(o[t][2 * k + i], a, pl[j][t][0], pl[j][t][1]);
                }
              }
            }
        }
        if (edge) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.empty[st]));
      st += S::kGroups;
      if (st >= S::kStages) {
        st = grp;
        ph ^= 1;
      }
    }
    skip = tile - walk.t_end;

    // ---- join the warps: (m, l) and o as they are, put together by the reading threads ----
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 4);
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 8);
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 16);
      }
    const bool whole = walk.whole();
    const int slot = seg == 1 ? 0 : 1;
    const int64_t piece = ((int64_t)blockIdx.x * 2 + slot) * kRows;
    if (seg > 1) named_bar_sync(1, kWarps * 32);  // the last unit has been read
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (8 * t + c2 >= heads) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (g == 0) {
          sm.m[warp][8 * t + c2 + i] = m[t][i];
          sm.l[warp][8 * t + c2 + i] = l[t][i];
        }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // element of the head dim in row g (+ 8) of this 16-row block
          const int d = kFp8 ? 16 * i + 2 * g + (e >> 1) : 16 * i + g + 8 * (e >> 1);
          sm.o[warp][8 * t + c2 + (e & 1)][d] = o[t][i][e];
        }
    }
    named_bar_sync(1, kWarps * 32);
    for (int i = threadIdx.x; i < heads * (D / 2); i += kWarps * 32) {
      const int r = i / (D / 2), d = (i % (D / 2)) * 2;
      float mw[kWarps], mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        mw[w] = sm.m[w][r];
        mm = fmaxf(mm, mw[w]);
      }
      float ll = 0.f, x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = mw[w] == -INFINITY ? 0.f : fast_exp2(mw[w] - mm);  // 0: a warp that saw no key
        const float2 u = *reinterpret_cast<const float2*>(&sm.o[w][r][d]);
        ll = fmaf(sm.l[w][r], f, ll);
        x = fmaf(u.x, f, x);
        y = fmaf(u.y, f, y);
      }
      if (dead) continue;
      if (whole) {
        store_out<D, kQBf16>(p, (int64_t)walk.b * p.hq + h0 + r, d, x, y, mm - kShift, ll);
      } else {
        *reinterpret_cast<float2*>(p.part_o + (piece + r) * D + d) = make_float2(x, y);
        if (d == 0) p.part_ml[piece + r] = make_float2(mm - kShift, ll);
      }
    }
    if (p.record && threadIdx.x == 0 && walk.t_beg == 0 && (!whole || p.record_by_unit)) {
      // The unit begins here; it ends in the gang that has its last tile.
      const int64_t last_tile = sm.end - walk.left + walk.span.tiles - 1;
      Record r{walk.b, walk.unit, gang, -1, slot};
      if (!whole) r.last = share_of(last_tile, sm.total, sm.n_gangs);
      p.record[p.record_by_unit ? walk.b * units + walk.unit : (int)blockIdx.x] = r;
    }
  } while (walk.next(p));
}

// Joins the pieces of the units that lie in several blocks' shares, in the order of their
// tiles: one block per record and row, in which four groups of threads take every fourth
// piece each, eight loads of a thread in flight.  (A kernel of its own: the main kernel's
// block that ends last would take longer than this launch to read them -- 6 units of 25
// pieces, 16 heads of 256 elements: 60 us against 26; one unit: 21 against 11.)
template <int D, int NT, bool kQBf16>
__global__ void __launch_bounds__(2 * D) paged_attn_join_kernel(const __grid_constant__ Params p) {
  constexpr int kGroups = 4, kBatch = 8;
  __shared__ float4 part[kGroups][D / 2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Record u = p.record[blockIdx.x];
  if (u.last < 0) return;
  const int kvh = u.unit / p.head_blocks, r = blockIdx.y, first = u.first, lane = lane_of_gang(p, u.unit);
  const int head = kvh * p.group + (u.unit - kvh * p.head_blocks) * 8 * NT + r;
  if (head >= (kvh + 1) * p.group) return;
  const int grp = threadIdx.x / (D / 2), i = threadIdx.x % (D / 2);
  float m = -INFINITY, l = 0.f, x = 0.f, y = 0.f;
  auto add = [&](float m2, float l2, float x2, float y2) {
    const float mn = fmaxf(m, m2);
    const float f = m == -INFINITY ? 0.f : fast_exp2(m - mn), g = m2 == -INFINITY ? 0.f : fast_exp2(m2 - mn);
    m = mn;
    l = fmaf(l, f, l2 * g);
    x = fmaf(x, f, x2 * g);
    y = fmaf(y, f, y2 * g);
  };
  for (int c0 = first + grp; c0 <= u.last; c0 += kGroups * kBatch) {
    float2 ml[kBatch], v[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int c = min(c0 + e * kGroups, u.last);
      const int64_t at = (int64_t)(2 * ((c << p.gang_shift) + lane) + (c == first ? u.first_slot : 0)) * (8 * NT) + r;
      ml[e] = load_l2(p.part_ml + at);
      v[e] = load_l2(reinterpret_cast<const float2*>(p.part_o + at * D + 2 * i));
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (c0 + e * kGroups <= u.last) add(ml[e].x, ml[e].y, v[e].x, v[e].y);
  }
  part[grp][i] = make_float4(m, l, x, y);
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int g = 1; g < kGroups; ++g) {
    const float4 o = part[g][i];
    add(o.x, o.y, o.z, o.w);
  }
  store_out<D, kQBf16>(p, (int64_t)u.b * p.hq + head, 2 * i, x, y, m, l);
}

template <int kCache, int D, int NT>
cudaError_t launch_instance(const Params& p, const CUtensorMap& k_map, const CUtensorMap& v_map,
                            cudaStream_t stream) {
  using S = Shape<kCache, D, NT>;
  constexpr size_t smem = S::kStages * 2 * S::kHalf + sizeof(Smem<S::kWarps, D, NT>);
  static_assert(smem <= 227 * 1024, "shared memory");
  static_assert(S::kStages <= 32, "barrier arrays");
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(paged_attn_kernel<kCache, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
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
  if ((e = cudaLaunchKernelEx(&cfg, paged_attn_kernel<kCache, D, NT>, p, k_map, v_map)) != cudaSuccess || !p.record) return e;
  cfg.gridDim = dim3((unsigned)p.records, p.group < 8 * NT ? p.group : 8 * NT);
  cfg.blockDim = dim3(2 * D);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_attn_join_kernel<D, NT, kCache == kCacheBf16 || kCache == kCacheE4m3>, p);
}

template <int kCache>
cudaError_t launch_cache(const Params& p, int d, const CUtensorMap& k_map, const CUtensorMap& v_map,
                         cudaStream_t stream) {
  const bool two = p.group > 8;
  switch (d) {
    case 64:
      return two ? launch_instance<kCache, 64, 2>(p, k_map, v_map, stream)
                 : launch_instance<kCache, 64, 1>(p, k_map, v_map, stream);
    case 128:
      return two ? launch_instance<kCache, 128, 2>(p, k_map, v_map, stream)
                 : launch_instance<kCache, 128, 1>(p, k_map, v_map, stream);
    default:
      return two ? launch_instance<kCache, 256, 2>(p, k_map, v_map, stream)
                 : launch_instance<kCache, 256, 1>(p, k_map, v_map, stream);
  }
}

cudaError_t read_errors_here(uint32_t* word) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(word, g_paged_attn_err, sizeof(uint32_t));
  return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_paged_attn_err, &zero, sizeof(uint32_t));
}

}  // namespace

}  // namespace pa
}  // namespace gqa
