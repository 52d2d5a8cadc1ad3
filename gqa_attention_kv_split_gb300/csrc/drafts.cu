// drafts.cu -- what a step with drafted tokens needs around its attention: the
// trees' visibility bits and positions, and the accepted tokens' cache rows moved
// together.
//
// Trees.  Token i of a tree (parent[i] < i, or -1: it follows the last cached
// token) sees itself and the tokens above it; its depth counts those, and its
// position is (cached tokens) + depth.  Nothing is computed but the walk up: one
// thread a token, the parents in shared memory, about 30 cycles a step, twice where
// a window has to know the depth first.  (Pointer doubling needs fewer steps from a
// depth of about 8 on but a barrier or two for each, and its words in shared memory;
// trees of drafted tokens are 4 to 10 deep.)  Ancestors come in falling order, so
// that a row's words are finished one after the other and go straight to memory.
// What bounds it is the launch and three dependent loads (time in a graph of 21 calls: one tree of 16
// tokens 1.8 us, 256 of up to 64 under a window 3.0 us).
//
// Compaction.  The rows kept[b][0 .. n) of a sequence's drafted tokens (rising) go to
// its first n drafted places.  A thread owns 16 bytes of a row (8 where a tensor's
// rows are no multiple of 16) in one head, layer and tensor and moves them for all kept
// tokens in order, kBatch at a time, loads before stores: a place is never written
// before it has been read, since kept[j] > kept[i] >= i for j > i, and no thread reads
// what another one writes.  HBM bounds it where there are many rows (each is read
// once and written once), latency otherwise: lengths, then table entries, then rows
// (one sequence in one layer 3.5 us; 64 in 16 layers, 30 MB read and written: 9.3 us).
#include <cuda_runtime.h>

#include "common.cuh"
#include "paged.h"

namespace gqa {
namespace {

__device__ uint32_t g_drafts_err;

__global__ void __launch_bounds__(kMaxTreeTokens) tree_mask_kernel(const TreeMaskArgs a) {
  __shared__ int16_t parent[kMaxTreeTokens];
  const int64_t b = blockIdx.x;
  const int64_t lo = a.indptr[b], hi = a.indptr[b + 1];
  const int len = a.kv_lens[b];
  if (lo < 0 || hi < lo || hi > a.total || (b == 0 && lo != 0)) {
    if (threadIdx.x == 0) atomicOr(&g_drafts_err, kErrBadIndptr);
    if (lo < 0 || hi < lo || hi > a.total) return;
  }
  int n = (int)(hi - lo);
  const int base = len - n;  // cached tokens before the tree
  bool bad = n > 32 * a.words;
  n = min(n, 32 * a.words);  // (those behind are left alone)
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    int p = a.parents[lo + i];
    if (p < -1 || p >= i) {
      bad = true;
      p = -1;
    }
    parent[i] = (int16_t)p;
  }
  if (bad) atomicOr(&g_drafts_err, kErrBadIndex);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    int depth = 0;
    if (a.window > 0)
      for (int j = parent[i]; j >= 0; j = parent[j]) ++depth;
    uint32_t* row = a.mask + (lo + i) * a.words;
    int w = a.words - 1, above = 0;
    uint32_t bits = 0;
    for (int j = i; j >= 0; j = parent[j], ++above) {
      for (; w > j >> 5; --w, bits = 0) row[w] = bits;
      const bool seen = a.window <= 0 || above < a.window || base + depth - above < a.sinks;
      bits |= (uint32_t)seen << (j & 31);
    }
    for (; w >= 0; --w, bits = 0) row[w] = bits;
    a.positions[lo + i] = base + above - 1;
  }
}

constexpr int kKeepThreads = 256;
constexpr int kKeepList = 128;  // kept tokens resolved at a time
constexpr int kKeepBatch = 8;   // rows of a thread in flight

struct Move {
  int64_t src_page, dst_page;  // src_page < 0: not moved
  int src_slot, dst_slot;
};

__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const __grid_constant__ KeepArgs a) {
  __shared__ Move move[kKeepList];
  const int64_t b = blockIdx.y;
  const int64_t lo = a.indptr[b], hi = a.indptr[b + 1];
  const int32_t len = a.kv_lens[b];
  const int64_t n = hi - lo, base = len - n;  // drafted tokens, cached ones before them
  const int64_t count = a.num_kept[b];
  const int32_t* kept = a.kept + b * a.max_kept;
  const int64_t most = n < a.max_kept ? n : a.max_kept;
  // A sequence whose numbers make no sense is left as it is: its offsets, its length,
  // more kept tokens than there are, or kept ones that do not rise.
  const bool offsets = lo >= 0 && n >= 0 && (b > 0 || lo == 0);
  bool ok = offsets && count >= 0 && count <= (n > 0 ? most : 0);
  bool rises = true;
  if (ok)
    for (int64_t i = threadIdx.x; i < count; i += kKeepThreads) {
      const int32_t k = kept[i];
      rises &= k >= 0 && k < n && (i == 0 || kept[i - 1] < k);
    }
  rises = __syncthreads_and(rises);
  ok &= rises && (base >= 0 || count == 0);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (!offsets) atomicOr(&g_drafts_err, kErrBadIndptr);
    if (offsets && !ok) atomicOr(&g_drafts_err, kErrBadIndex);
    a.new_lens[b] = ok && base >= 0 ? (int32_t)(base + count) : len;
  }
  if (!ok || count == 0) return;

  // This thread's piece of a row: column, head, layer, tensor.
  int64_t item = (int64_t)blockIdx.x * kKeepThreads + threadIdx.x;
  int t = 0;
  while (t < a.tensors && item >= a.t[t].items) item -= a.t[t++].items;
  const bool mine = t < a.tensors;
  const KeepTensor& kt = a.t[mine ? t : 0];
  const int64_t row = item / kt.pieces, col = item - row * kt.pieces;
  const int64_t layer = row / kt.heads, head = row - layer * kt.heads;
  uint8_t* at = kt.data + layer * kt.s_layer + head * kt.s_head + col * kt.vec;

  for (int64_t i0 = 0; i0 < count; i0 += kKeepList) {
    const int m = (int)(count - i0 < kKeepList ? count - i0 : kKeepList);
    if (i0 > 0) __syncthreads();
    for (int i = threadIdx.x; i < m; i += kKeepThreads) {
      Move r{-1, 0, 0, 0};
      const int64_t src = base + kept[i0 + i], dst = base + i0 + i;
      if (src != dst) {
        const int64_t sp = src / a.page_size, dp = dst / a.page_size;
        const bool in = sp < a.max_pages;  // (dst < src)
        const int64_t p = in ? a.block_table[b * a.max_pages + sp] : -1, q = in ? a.block_table[b * a.max_pages + dp] : -1;
        if (p >= 0 && p < a.num_pages && q >= 0 && q < a.num_pages)
          r = {p, q, (int)(src - sp * a.page_size), (int)(dst - dp * a.page_size)};
        else if (blockIdx.x == 0)
          atomicOr(&g_drafts_err, kErrBadIndex);
      }
      move[i] = r;
    }
    __syncthreads();
    if (!mine) continue;
    for (int i = 0; i < m; i += kKeepBatch) {
      uint4 x[kKeepBatch];
#pragma unroll
      for (int e = 0; e < kKeepBatch; ++e) {
        if (i + e >= m || move[i + e].src_page < 0) continue;
        const uint8_t* p = at + move[i + e].src_page * kt.s_page + move[i + e].src_slot * kt.s_slot;
        if (kt.vec == 16) {
          x[e] = *reinterpret_cast<const uint4*>(p);
        } else {
          const uint2 y = *reinterpret_cast<const uint2*>(p);
          x[e].x = y.x;
          x[e].y = y.y;
        }
      }
#pragma unroll
      for (int e = 0; e < kKeepBatch; ++e) {
        if (i + e >= m || move[i + e].src_page < 0) continue;
        uint8_t* p = at + move[i + e].dst_page * kt.s_page + move[i + e].dst_slot * kt.s_slot;
        if (kt.vec == 16)
          *reinterpret_cast<uint4*>(p) = x[e];
        else
          *reinterpret_cast<uint2*>(p) = make_uint2(x[e].x, x[e].y);
      }
    }
  }
}

}  // namespace

cudaError_t launch_tree_mask(const TreeMaskArgs& a, cudaStream_t stream) {
  // A thread for each token that the masks have a bit for.
  tree_mask_kernel<<<(unsigned)a.batch, 32 * a.words, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_keep(const KeepArgs& a, cudaStream_t stream) {
  int64_t items = 0;
  for (int i = 0; i < a.tensors; ++i) items += a.t[i].items;
  const int64_t blocks = items > 0 ? (items + kKeepThreads - 1) / kKeepThreads : 1;
  if (blocks > 0x7fffffffLL || a.batch > 65535) return cudaErrorInvalidConfiguration;
  keep_kernel<<<dim3((unsigned)blocks, (unsigned)a.batch), kKeepThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t drafts_read_errors(uint32_t* word) {
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return e;
  uint32_t zero = 0;
  if ((e = cudaMemcpyFromSymbol(word, g_drafts_err, sizeof(uint32_t))) != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_drafts_err, &zero, sizeof(uint32_t));
}

}  // namespace gqa
