// Shared by the CUDA-core and tensor-core paths of kdtv_project.
#pragma once

#include "kdtv_rope.cuh"

namespace kdtv {

// Device-side view of a call.
struct ProjArgs {
  int B, N, K, M, R, adapters, dtype;      // d_in, d_out, rank
  const void *x, *W, *A, *Bm;
  const uint8_t *x_scale, *W_scale;
  const float* adapter_scale;
  const int32_t *adapter, *n_live;
  void* y;
  unsigned int* status;
  long long xs[2], ys[2];                  // elements between requests, rows
  Divisor by_N;
  float* low;                              // CUDA cores: s_a A_a x, [B * N, R]
};

__device__ __forceinline__ void proj_error(const ProjArgs& a, unsigned int code) { atomicCAS(a.status, 0u, code); }

// Adapter of request b: -1 for none, -2 (and an error recorded) for an index out of range.
__device__ __forceinline__ int proj_adapter(const ProjArgs& a, int b) {
  if (!a.adapter) return -1;
  const int id = a.adapter[b];
  if (id >= -1 && id < a.adapters) return id;
  proj_error(a, KDTV_ERR_BAD_ADAPTER);
  return -2;
}

}  // namespace kdtv
