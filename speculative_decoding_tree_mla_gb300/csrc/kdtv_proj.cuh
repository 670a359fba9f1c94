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

  // Tensor cores.  A token tile is one request's block of rows, or all rows of several requests, in two
  // halves, one for each CTA of a pair: half of the rows, or of the requests.  A half's columns are
  // request-major; behind them come unused ones, up to a multiple of 16, half_cols at most.
  int requests, blocks, groups;            // requests of a tile, most row blocks of a request, groups of requests
  int half_requests, half_rows, half_cols; // the largest half
  bool by_rows_of;                         // the halves are halves of a request's rows
  int base;                                // units (128 bytes of d_in each) of a tile without adapters
  int chunks;                              // 16-rank chunks of an adapter
  int pairs;                               // most pairs of chunks that a tile may have
  int features;                            // 256-row tiles of W
  int stages, scale_mode;                  // ring entries; how scale rows may be read
  int shared;                              // columns that the two accumulators have in common
  bool wide;                               // rows of y are written 16 bytes at a time
  char* parts;                             // A x in two bf16 parts: [tile][pair][half][chunk][part][half_cols][16]
  float* partial;                          // [pair][2 places][CTA][2 half_cols][128] sums of cut tiles
  int* plan;                               // what was cut: see CutTile
  Divisor by_requests, by_chunks;
};

__device__ __forceinline__ void proj_error(const ProjArgs& a, unsigned int code) { atomicCAS(a.status, 0u, code); }

// A request's adapter from its index: -1 for none, -2 (and an error recorded) for one out of range.
__device__ __forceinline__ int proj_adapter(const ProjArgs& a, int id) {
  if (id >= -1 && id < a.adapters) return id;
  proj_error(a, KDTV_ERR_BAD_ADAPTER);
  return -2;
}

// Bytes of A x of one pair of chunks, of one half of a tile.
__host__ __device__ inline long long proj_half_bytes(const ProjArgs& a) { return (long long)a.half_cols * 128; }

// Whether the tensor cores take these sizes, and the tiles; the workspace they need.
bool proj_tc_sizes(const kdtv_project_dims* d, int sms, ProjArgs* a);
size_t proj_tc_workspace(const ProjArgs& a, int sms);
int proj_tc_launches(const ProjArgs& a);      // (with adapters in use)
int launch_proj_tc(const ProjArgs& a, int sms, bool stall, cudaStream_t st);

}  // namespace kdtv
