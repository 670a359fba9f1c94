// What the tensor-core kernels of kdtv_project share: which adapters a tile has, and where its columns and A x lie.
#pragma once

#include "kdtv_guard.cuh"
#include "kdtv_proj.cuh"

namespace kdtv {
namespace {

constexpr int kUnitBytes = 128;            // of d_in in a unit
constexpr int kWords = KDTV_MAX_ADAPTERS / 32;

// ---- which adapters a tile has -------------------------------------------------------------
// Adapters of a group of requests that have live rows, as a bitmap in shared
// memory (by a warp); their places are the order of their numbers.
__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

__device__ __forceinline__ int group_bitmap(const ProjArgs& a, int g, uint32_t* bits, bool* live) {
  const int lane = threadIdx.x & 31, words = (a.adapters + 31) / 32;
  for (int w = lane; w < words; w += 32) bits[w] = 0u;
  __syncwarp();
  bool any = false;
  constexpr int kAtOnce = 2;                // a lane's requests whose loads are under way together
  for (int b0 = g * a.requests + lane; b0 < min(a.B, (g + 1) * a.requests); b0 += 32 * kAtOnce) {
    int n[kAtOnce], raw[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int b = b0 + 32 * k;
      const bool in = b < min(a.B, (g + 1) * a.requests);
      n[k] = in ? live_rows(a.n_live, b, a.N) : 0;
      raw[k] = in && a.adapter ? a.adapter[b] : -1;
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (n[k] <= 0) continue;
      const int id = proj_adapter(a, raw[k]);
      any |= id != -2;
      if (id >= 0) atomicOr(&bits[id >> 5], 1u << (id & 31));
    }
  }
  *live = __any_sync(0xffffffffu, any);
  __syncwarp();
  int count = 0;
  for (int w = lane; w < words; w += 32) count += __popc(bits[w]);
  return warp_sum(count);
}

// A request's n rows in blocks as even as they can be, so that its last one is not a small rest: rows of half a
// block.  (Tiles of several requests: all N rows.)
__device__ __forceinline__ int half_rows_of(const ProjArgs& a, int n) {
  if (!a.by_rows_of) return a.N;
  const int blocks = max(1, (n + 2 * a.half_rows - 1) / (2 * a.half_rows));
  return max(1, ((n + blocks - 1) / blocks + 1) / 2);
}
// Columns of half a tile whose half blocks have hr rows.
__device__ __forceinline__ int half_cols_of(const ProjArgs& a, int hr) { return (a.half_requests * hr + 15) & ~15; }

// The request and row of a tile's column; false: the column is not in use.
__device__ __forceinline__ bool column(const ProjArgs& a, int g, int j, int hr, int c, int* b, int* i) {
  const int hc = half_cols_of(a, hr), h = c >= hc, e = c - (h ? hc : 0);
  if (a.by_rows_of) {
    *b = g;
    *i = (2 * j + h) * hr + e;
    return e < hr && *i < a.N;
  }
  const int rq = (int)divide(e, a.by_N);
  *b = g * a.requests + h * a.half_requests + rq;
  *i = e - rq * a.N;
  return rq < a.half_requests && *b < a.B;
}
// Where the 16 ranks of chunk c, part p of row i of request b start; their two 16-byte halves lie swizzled: `flip`
// is the one that comes second.  hr: of the request.
__device__ __forceinline__ char* part_row(const ProjArgs& a, int b, int i, int hr, int c, int p, int* flip) {
  int g, j, h, col;
  if (a.by_rows_of) {
    g = b;
    const int half = i / hr;
    j = half >> 1;
    h = half & 1;
    col = i - half * hr;
  } else {
    g = (int)divide(b, a.by_requests);
    const int rq = b - g * a.requests;
    j = 0;
    h = rq >= a.half_requests;
    col = (rq - (h ? a.half_requests : 0)) * a.N + i;
  }
  *flip = (col >> 2) & 1;
  return a.parts + (((long long)(g * a.blocks + j) * a.pairs + (c >> 1)) * 2 + h) * proj_half_bytes(a) +
         (long long)((c & 1) * 2 + p) * a.half_cols * 32 + col * 32;
}

// Exponent bytes at .. at + 4 W - 1 of a row of `bytes` at any address, as words; 127 behind the row.  From the aligned
// words that hold them, where those lie within the tensor (it ends at `end`).
template <int W>
__device__ __forceinline__ void exponent_words(const uint8_t* row, int at, int bytes, const uint8_t* end, uint32_t (&x)[W]) {
  const int left = bytes - at;                 // of the row
  const uint8_t* p = row + at;
  if (left > 0 && p + 4 * W + 4 <= end) {
    const uint32_t shift = ((uint32_t)reinterpret_cast<uintptr_t>(p) & 3u) * 8u;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(3));
    uint32_t raw[W + 1];
#pragma unroll
    for (int k = 0; k <= W; ++k) raw[k] = words[k];
#pragma unroll
    for (int k = 0; k < W; ++k) x[k] = __funnelshift_r(raw[k], raw[k + 1], shift);
  } else {
#pragma unroll
    for (int k = 0; k < W; ++k) {
      x[k] = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * k + e < left) x[k] |= (uint32_t)p[4 * k + e] << (8 * e);
    }
  }
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const int valid = min(max(left - 4 * k, 0), 4);
    if (valid < 4) x[k] = (x[k] & ((1u << (8 * valid)) - 1u)) | (0x7f7f7f7fu << (8 * valid));
  }
}

}  // namespace

// v = s_a A_a x of all tokens into a.parts, on the current device.
cudaError_t launch_proj_low(const ProjArgs& a, int sms, cudaStream_t st);

// An SM divides its memory between L1 and shared memory once for all blocks that it holds: what is to run
// beside the projection asks for the division that the projection needs.
template <typename... KArgs>
cudaError_t beside(void (*kernel)(KArgs...)) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
}

}  // namespace kdtv
