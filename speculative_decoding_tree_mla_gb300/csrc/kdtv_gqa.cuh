// Shared by the CUDA-core and tensor-core paths of kdtv_gqa_verify_attn.
#pragma once

#include "kdtv_rope.cuh"

namespace kdtv {

// Device-side view of a call.  A unit of output rows is (request, key/value
// head, row): row r of a key/value head is node r / G, query head kvh * G +
// r % G, so the rows that share keys are neighbours.
struct GqaArgs {
  int B, N, H, Hkv, G, d, dtype;
  int page_size, t_stride, max_pages, num_pages;
  float scale;
  const void *q, *k, *v;
  const uint8_t *k_scale, *v_scale;
  const int32_t *parent, *prefix_len, *n_nodes, *page_table;
  void* out;
  unsigned int* status;
  float* part_o;               // partial rows (unnormalised), fp32
  float2* part_ml;             // {reference maximum (log2 units), sum}; sum < 0: the row is not written
  int* plan;                   // tensor cores: units per group of CTAs, then each request's first unit
  int chunk, splits;           // CUDA cores: keys per split, splits
  long long cap;               // rows a request may have
  // tensor cores: heads side by side in a group of CTAs, groups, nodes per 128-row tile (128 / G),
  // log2 of page_size, blocks of hg heads, row tiles
  int hg, groups, npt, page_shift, blocks, tiles;
  Divisor by_hg, by_groups, by_pair, by_G, by_tiles;   // (pair: two tiles' nodes)
};

__device__ __forceinline__ void gqa_error(const GqaArgs& a, unsigned int code) {
  atomicCAS(a.status, 0u, code);
}

// Prefix L and live nodes n of request b; n = 0 (and an error recorded) if its
// rows do not fit the cache.
__device__ __forceinline__ void gqa_request(const GqaArgs& a, int b, int* L, int* n) {
  *L = a.prefix_len[b];
  *n = live_rows(a.n_nodes, b, a.N);
  if (*n > 0 && (*L < 0 || (long long)*L + *n > a.cap)) {
    gqa_error(a, KDTV_ERR_BAD_PREFIX);
    *n = 0;
  }
}

// Cache row (without heads) of position t of request b; -1: page out of range.
__device__ __forceinline__ long long gqa_row(const GqaArgs& a, int b, int t) {
  if (!a.page_size) return (long long)b * a.t_stride + t;
  const int page = a.page_table[(long long)b * a.max_pages + t / a.page_size];
  if (page < 0 || page >= a.num_pages) return -1;
  return (long long)page * a.page_size + t % a.page_size;
}

// Node i's root path as a bit mask, i included; false if it is malformed.
// parent[j] < j bounds the walk.
__device__ __forceinline__ bool gqa_path(const GqaArgs& a, int b, int i, uint32_t (&mask)[4]) {
  const int32_t* par = a.parent + (long long)b * a.N;
  mask[0] = mask[1] = mask[2] = mask[3] = 0u;
  for (;;) {
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if ((i >> 5) == w) mask[w] |= 1u << (i & 31);
    const int p = par[i];
    if (i == 0) return p == -1;
    if (p < 0 || p >= i) return false;
    i = p;
  }
}

// 32 visibility bits of keys t0 .. t0 + 31 for a row with this path mask:
// everything before L, its path from L on (bits behind the live nodes are 0).
__device__ __forceinline__ uint32_t gqa_visible(const uint32_t (&mask)[4], int t0, int L) {
  const int j = t0 - L;
  if (j <= -32) return 0xffffffffu;
  if (j < 0) return (mask[0] << -j) | ((1u << -j) - 1u);
  const int w = j >> 5;
  const uint32_t lo = w == 0 ? mask[0] : w == 1 ? mask[1] : w == 2 ? mask[2] : w == 3 ? mask[3] : 0u;
  const uint32_t hi = w == 0 ? mask[1] : w == 1 ? mask[2] : w == 2 ? mask[3] : 0u;
  return __funnelshift_r(lo, hi, j & 31);
}

__device__ __forceinline__ float gqa_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

int gqa_tc_supported(const kdtv_gqa_dims* d);
size_t gqa_tc_workspace(const kdtv_gqa_dims* d, int sms, GqaArgs* a);   // sets a's plan; 0: too large
int launch_gqa_tc(const GqaArgs& a, bool stall, cudaStream_t st);

}  // namespace kdtv
