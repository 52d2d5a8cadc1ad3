// append.cu -- rotary embedding of new query and key rows and the append of
// the keys and values to a paged cache: 16-bit pages, E4M3 pages, and NVFP4
// pages (E2M1 codes with one E4M3 scale per 16 elements, the pages that
// nvfp4_paged_ctx_attn reads).
//
// Mathematics.  Token t of sequence b sits at position
//   pos = kv_lens[b] - (indptr[b+1] - t),
// and a rotated pair (x, y) of a q or k row becomes (x c - y s, y c + x s) with
// c = rope[pos, i], s = rope[pos, rot/2 + i] -- pairs (i, i + rot/2), or
// (2i, 2i + 1) interleaved.  Products and sums are formed in f32, each rounded
// once (no contraction), and the result is rounded once to its stored type.
// NVFP4: sf = E4M3(amax / 6) of a 16-element block, codes = E2M1(x / sf), what f32
// divisions give, so a plain f32 evaluation gives the same bits.
//
// What bounds it: HBM for prompts (each input read once, each output written
// once, 3 flops per rotated element), latency for single tokens -- a chain of
// dependent loads (lengths, then the table entry and the angles).  Hence:
//  * one thread owns one pair of 16-byte vectors of a row (the two halves of a
//    rotation when it is a half-split one), so a rotation needs no exchange;
//  * the row data, which depend on no metadata, are loaded before the token's
//    sequence, position and page are looked up;
//  * a warp looks up one token (a 32-way search of indptr: two probes for up
//    to 1024 sequences), and a block's warps look up its tokens side by side.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "paged.h"

namespace gqa {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kMaxTok = kAppendThreads / 32;  // tokens per block: one looked up by each warp

__device__ uint32_t g_append_err;

// Where a block's token goes: its position, and its page and slot; pos < 0: not written.
struct TokenPlace {
  int64_t page;
  int64_t pos;
  int slot;
};

__device__ __forceinline__ void unpack8(const uint4& u, float f[8], __half) {
  const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ void unpack8(const uint4& u, float f[8], __nv_bfloat16) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float f[8], __half) {
  uint4 u;
  __half2* h = reinterpret_cast<__half2*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
  return u;
}
__device__ __forceinline__ uint4 pack8(const float f[8], __nv_bfloat16) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return u;
}

// Two f32 operations in one instruction, each rounded as by itself: issue slots bound the
// NVFP4 append (8192 tokens: 32.9 us with single operations, 30.8 with these).  Sums of
// products are left single: a packed product and a packed sum come out as one rounding.
struct Two {
  uint64_t v;
  __device__ __forceinline__ Two() {}
  __device__ __forceinline__ Two(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ void split(float& lo, float& hi) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
};
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ void sum(Two a, Two b, float* r) {
  float a0, a1, b0, b1;
  a.split(a0, a1);
  b.split(b0, b1);
  r[0] = __fadd_rn(a0, b0);
  r[1] = __fadd_rn(a1, b1);
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Two f32 -> two E4M3 bytes (lo in the low byte), RNE, saturating; NaN stays NaN.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 pack8_e4m3(const float f[8], float inv_scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    mul2(Two(f[2 * i], f[2 * i + 1]), Two(inv_scale, inv_scale)).split(lo, hi);
    w[i] = f32x2_to_e4m3x2(lo, hi);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Two f32 -> one byte of E2M1 codes (lo in the low nibble), RNE, saturating.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "cvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float amax8(const float f[8]) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(f[i]));
  return m;
}
// x / s by one multiplication with r, 1 / s to a few f32 spacings, and one correction step
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990): within 2^-44 of the quotient before its rounding to f32.  Rounded to E2M1 (s a
// scale) or to E4M3 (s = 6) it gives what the f32 division gives: for a border t between
// two codes, t * s is an f32 number (of 7 significant bits at most), so that x either is
// t * s, and the step gives t, or is at least one f32 spacing away from it, and the
// quotient more than half a spacing (by 2^-31 of it) away from t.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = __fmul_rn(x, r);
  return __fmaf_rn(__fmaf_rn(-q, s, x), r, q);
}
// E4M3 scale byte of a block's largest magnitude, and the scale's value.
__device__ __forceinline__ uint32_t block_scale(float amax, float* value) {
  const float x = amax > 4096.f ? 4096.f : amax;  // (saturates all the same, and is no infinity; NaN stays)
  const uint32_t byte = f32x2_to_e4m3x2(quotient(x, 6.f, 1.f / 6.f), 0.f);
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)byte));
  *value = __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
  return byte & 0xffu;
}
// Eight elements -> 4 bytes of codes; all codes 0 where the scale is 0 or NaN.
__device__ __forceinline__ uint32_t codes8(const float f[8], float scale) {
  if (!(scale > 0.f)) return 0u;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Two x(f[2 * i], f[2 * i + 1]), by(inv, inv), q = mul2(x, by);
    float lo, hi;
    fma2(fma2(q, Two(-scale, -scale), x), by, q).split(lo, hi);  // (quotient, two at a time)
    r |= f32x2_to_e2m1x2(lo, hi) << (8 * i);
  }
  if (scale == 448.f) {  // the largest scale: there may be infinities, whose correction is NaN
    r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r |= f32x2_to_e2m1x2(__fdiv_rn(f[2 * i], scale), __fdiv_rn(f[2 * i + 1], scale)) << (8 * i);
  }
  return r;
}

// (x, y) -> (x c - y s, y c + x s), each product and sum rounded by itself: the two pairs
// (x[0], y[0]) and (x[1], y[1]), or one that lies together.
__device__ __forceinline__ void turn_pairs(float* x, float* y, float c0, float s0, float c1, float s1) {
  const Two u(x[0], x[1]), w(y[0], y[1]), c(c0, c1), s(s0, s1), minus_s(-s0, -s1);
  sum(mul2(u, c), mul2(w, minus_s), x);
  sum(mul2(w, c), mul2(u, s), y);
}
__device__ __forceinline__ void turn_pair(float* z, float c, float s) {
  sum(mul2(Two(z[0], z[1]), Two(c, c)), mul2(Two(z[1], z[0]), Two(-s, s)), z);
}

// The sequence of token t: the last b with indptr[b] <= t (the whole warp).
// Each step probes 32 evenly spaced entries; every probe lies in [lo, hi).
__device__ __forceinline__ int64_t find_sequence(const int32_t* indptr, int64_t batch, int64_t t, int lane) {
  int64_t lo = 0, hi = batch;  // the answer is in [lo, hi) if indptr[0] <= t
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 31) / 32;
    const int64_t at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && indptr[at] <= t);
    const int k = le ? 31 - __clz(le) : 0;
    lo += k * step;
    hi = hi < lo + step ? hi : lo + step;
  }
  return lo;
}

// Position, page and slot of token t, and its cosines and sines into `angles` (the whole
// warp; the result is the same in every lane).
__device__ __forceinline__ TokenPlace place_token(const AppendArgs& a, int64_t t, int lane, float4* angles) {
  TokenPlace p{0, -1, 0};
  int64_t b = t, behind = 1;  // tokens from t to the end of its sequence's new ones
  if (a.indptr) {
    b = find_sequence(a.indptr, a.batch, t, lane);
    const int64_t lo = a.indptr[b], hi = a.indptr[b + 1];
    if (t < lo || t >= hi) return p;  // behind the last sequence (a padded batch), or check_offsets flags it
    behind = hi - t;
  }
  const int64_t pos = (int64_t)a.kv_lens[b] - behind;
  if (pos < 0) return p;  // an inactive sequence
  const int64_t lp = (uint32_t)pos / (uint32_t)a.page_size;  // (a length is an int32)
  int64_t page = -1;
  if (lp < a.max_pages_per_seq) page = a.block_table[b * a.max_pages_per_seq + lp];
  const bool known = !a.rope || pos < a.rope_len;
  if (a.rope && known)
    for (int i = lane; i < a.rot / 4; i += 32) angles[i] = reinterpret_cast<const float4*>(a.rope + pos * a.rot)[i];
  if (page < 0 || page >= a.num_pages || !known) {
    if (lane == 0) atomicOr(&g_append_err, kErrBadIndex);
    return p;
  }
  p.page = page;
  p.pos = pos;
  p.slot = (int)(pos - lp * a.page_size);
  return p;
}

// The offsets run from 0 upwards and end within the inputs: all of them are looked at, the
// grid's threads taking one each (the last warps first, which place no token in a small call).
__device__ __forceinline__ void check_offsets(const AppendArgs& a) {
  const int64_t me = (int64_t)blockIdx.x * kAppendThreads + (kAppendThreads - 1 - threadIdx.x);
  bool bad = me == 0 && (a.indptr[0] != 0 || a.indptr[a.batch] > a.total);
  for (int64_t b = me; b < a.batch; b += (int64_t)gridDim.x * kAppendThreads) bad |= a.indptr[b] > a.indptr[b + 1];
  if (bad) atomicOr(&g_append_err, kErrBadIndptr);
}

// kMode: kAppendSame (pages of the inputs' type), kAppendE4m3, kAppendNvfp4.
template <typename T, int D, int kMode>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / 16;  // threads per row, each with two 16-byte vectors
  __shared__ TokenPlace place[kMaxTok];
  __shared__ float4 angles[kMaxTok][D / 4];
  asm volatile("griddepcontrol.launch_dependents;");  // (the attention of this step may start; it waits for this grid's end)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = (int64_t)blockIdx.x * a.tok_per_block;
  const int n_tok = (int)(a.total < t0 + a.tok_per_block ? a.total - t0 : a.tok_per_block);
  const int rows = (a.q ? a.hq : 0) + 2 * a.hkv;  // of one token: q heads, k heads, v heads
  const int hq = a.q ? a.hq : 0;
  const int turned = a.rope ? a.rot / 16 : 0;  // lanes of a row that rotate

  // A thread's rows: kStep apart, over the block's tokens.
  constexpr int kStep = kAppendThreads / kLanes;
  const int j = threadIdx.x % kLanes;
  struct Row {
    int tok, row;
    uint4 lo, hi;
  };
  auto split = [&](int row) { return row < hq + a.hkv && j < turned && !a.interleaved; };  // a half-split rotation
  auto load = [&](Row& x) {
    while (x.row >= rows) {
      x.row -= rows;
      ++x.tok;
    }
    if (x.tok >= n_tok) return;
    const T* src;
    if (x.row < hq)
      src = static_cast<const T*>(a.q) + (t0 + x.tok) * a.q_tok + x.row * a.q_head;
    else if (x.row < hq + a.hkv)
      src = static_cast<const T*>(a.k) + (t0 + x.tok) * a.k_tok + (x.row - hq) * a.k_head;
    else
      src = static_cast<const T*>(a.v) + (t0 + x.tok) * a.v_tok + (x.row - hq - a.hkv) * a.v_head;
    const bool sp = split(x.row);
    x.lo = *reinterpret_cast<const uint4*>(src + 8 * (sp ? j : 2 * j));
    x.hi = *reinterpret_cast<const uint4*>(src + 8 * (sp ? j + turned : 2 * j + 1));
  };

  Row next{0, (int)threadIdx.x / kLanes, make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  load(next);
  if (warp < n_tok) {
    const TokenPlace p = place_token(a, t0 + warp, lane, angles[warp]);
    if (lane == 0) place[warp] = p;
  }
  if (a.indptr) check_offsets(a);
  __syncthreads();
  // (NVFP4: a warp's four rows are of one token and one kind -- 32 or 0 q heads, 8 of k and
  // 8 of v -- so that its lanes take every branch together and the shuffles are whole.)
  while (next.tok < n_tok) {
    const Row cur = next;
    next.row += kStep;
    load(next);
    const TokenPlace p = place[cur.tok];
    if (p.pos < 0) continue;
    const int row = cur.row;
    const bool sp = split(row);
    const int v0 = sp ? j : 2 * j, v1 = sp ? j + turned : 2 * j + 1;
    const bool is_q = row < hq, is_v = row >= hq + a.hkv;
    const int h = is_q ? row : is_v ? row - hq - a.hkv : row - hq;
    const bool turn = !is_v && j < turned;
    if (kMode == kAppendSame && !turn) {  // as it is
      T* dst = is_q ? static_cast<T*>(a.q_out) + (t0 + cur.tok) * a.qo_tok + h * a.qo_head
               : is_v ? static_cast<T*>(a.v_pages) + p.page * a.vp_page + h * a.vp_head + p.slot * a.vp_slot
                      : static_cast<T*>(a.k_pages) + p.page * a.kp_page + h * a.kp_head + p.slot * a.kp_slot;
      *reinterpret_cast<uint4*>(dst + 16 * j) = cur.lo;
      *reinterpret_cast<uint4*>(dst + 16 * j + 8) = cur.hi;
      continue;
    }
    float x[8], y[8];
    unpack8(cur.lo, x, T());
    unpack8(cur.hi, y, T());
    if (turn) {
      const float4* cs = &angles[cur.tok][2 * j];
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // four angles at a time
        const float4 c4 = cs[i], s4 = cs[a.rot / 8 + i];
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
        if (a.interleaved) {
          float* z = i ? y : x;
#pragma unroll
          for (int e = 0; e < 4; ++e) turn_pair(z + 2 * e, c[e], s[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; e += 2) turn_pairs(x + 4 * i + e, y + 4 * i + e, c[e], s[e], c[e + 1], s[e + 1]);
        }
      }
    }
    if (is_q) {
      if (kMode == kAppendNvfp4) {
        uint8_t* dst = static_cast<uint8_t*>(a.q_out) + (t0 + cur.tok) * a.qo_tok + h * a.qo_head;
        *reinterpret_cast<uint2*>(dst + 8 * v0) = pack8_e4m3(x, a.inv_q);
        *reinterpret_cast<uint2*>(dst + 8 * v1) = pack8_e4m3(y, a.inv_q);
      } else {
        T* dst = static_cast<T*>(a.q_out) + (t0 + cur.tok) * a.qo_tok + h * a.qo_head;
        *reinterpret_cast<uint4*>(dst + 8 * v0) = pack8(x, T());
        *reinterpret_cast<uint4*>(dst + 8 * v1) = pack8(y, T());
      }
      continue;
    }
    if (kMode == kAppendNvfp4) {
      const int64_t r = (p.page * kHkv + h) * kPage + p.slot;
      uint8_t* codes = static_cast<uint8_t*>(is_v ? a.v_pages : a.k_pages) + r * (D / 2);
      uint8_t* sf = (is_v ? a.v_sf : a.k_sf) + r * (D / 16);
      // A rotated half-split row has its blocks in two neighbouring lanes (rot is a
      // multiple of 32: lanes 2i and 2i+1 hold the halves of one block, twice);
      // otherwise a lane has a whole one.
      float ax = amax8(x), ay = amax8(y), sx, sy;
      const float ox = __shfl_xor_sync(0xffffffffu, ax, 1), oy = __shfl_xor_sync(0xffffffffu, ay, 1);
      if (sp) {
        const uint32_t bx = block_scale(max_nan(ax, ox), &sx), by = block_scale(max_nan(ay, oy), &sy);
        *reinterpret_cast<uint32_t*>(codes + 4 * v0) = codes8(x, sx);
        *reinterpret_cast<uint32_t*>(codes + 4 * v1) = codes8(y, sy);
        if ((j & 1) == 0) {
          sf[v0 / 2] = (uint8_t)bx;
          sf[v1 / 2] = (uint8_t)by;
        }
      } else {
        sf[j] = (uint8_t)block_scale(max_nan(ax, ay), &sx);
        *reinterpret_cast<uint2*>(codes + 8 * j) = make_uint2(codes8(x, sx), codes8(y, sx));
      }
    } else {
      const int64_t off = is_v ? p.page * a.vp_page + h * a.vp_head + p.slot * a.vp_slot
                               : p.page * a.kp_page + h * a.kp_head + p.slot * a.kp_slot;
      void* base = is_v ? a.v_pages : a.k_pages;
      if (kMode == kAppendE4m3) {
        const float inv = is_v ? a.inv_v : a.inv_k;
        uint8_t* dst = static_cast<uint8_t*>(base) + off;
        *reinterpret_cast<uint2*>(dst + 8 * v0) = pack8_e4m3(x, inv);
        *reinterpret_cast<uint2*>(dst + 8 * v1) = pack8_e4m3(y, inv);
      } else {
        T* dst = static_cast<T*>(base) + off;
        *reinterpret_cast<uint4*>(dst + 8 * v0) = pack8(x, T());
        *reinterpret_cast<uint4*>(dst + 8 * v1) = pack8(y, T());
      }
    }
  }
}

template <typename T, int kMode>
cudaError_t launch_d(const AppendArgs& a, unsigned grid, cudaStream_t stream) {
  if constexpr (kMode == kAppendNvfp4) {
    append_kernel<T, kD, kMode><<<grid, kAppendThreads, 0, stream>>>(a);
  } else {
    switch (a.d) {
      case 64: append_kernel<T, 64, kMode><<<grid, kAppendThreads, 0, stream>>>(a); break;
      case 128: append_kernel<T, 128, kMode><<<grid, kAppendThreads, 0, stream>>>(a); break;
      default: append_kernel<T, 256, kMode><<<grid, kAppendThreads, 0, stream>>>(a); break;
    }
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_mode(const AppendArgs& a, unsigned grid, cudaStream_t stream) {
  switch (a.mode) {
    case kAppendSame: return launch_d<T, kAppendSame>(a, grid, stream);
    case kAppendE4m3: return launch_d<T, kAppendE4m3>(a, grid, stream);
    default: return launch_d<T, kAppendNvfp4>(a, grid, stream);
  }
}

}  // namespace

cudaError_t launch_append(AppendArgs a, cudaStream_t stream) {
  // Tokens per block: one for each warp at most (they share the block's start), and as
  // few as make whole turns of the blocks that run at a time, four on each SM (8192
  // tokens of 32 + 8 + 8 heads: 7 a block in 36.1 us, 8 in 37.0).
  const int64_t at_once = 4 * 152;
  const int64_t turns = (a.total + at_once * kMaxTok - 1) / (at_once * kMaxTok);
  const int64_t per = (a.total + at_once * turns - 1) / (at_once * turns);
  a.tok_per_block = (int)per;
  const int64_t grid = (a.total + per - 1) / per;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return a.bf16 ? launch_mode<__nv_bfloat16>(a, (unsigned)grid, stream) : launch_mode<__half>(a, (unsigned)grid, stream);
}

cudaError_t append_read_errors(uint32_t* word) {
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return e;
  uint32_t zero = 0;
  if ((e = cudaMemcpyFromSymbol(word, g_append_err, sizeof(uint32_t))) != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_append_err, &zero, sizeof(uint32_t));
}

}  // namespace gqa
