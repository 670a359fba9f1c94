// v = s_a A_a x, the inner products of kdtv_project's adapters on tensor cores,
// laid out as the projection's operands are to lie in shared memory: two bf16
// parts of the fp32 sums.
//
// mma.sync products of 16 ranks and 8 tokens.  The order of d_in within a
// product does not matter as long as both operands have the same, so a lane's
// 16 bytes of a row (8 elements) are two products' fragments: lane 4 g + q has
// elements 8 q .. 8 q + 7 of 32 of row g.  (tcgen05 would need 128 rows of one
// adapter, and x in bf16: one-byte x is widened on its way into the registers.)

#include <cuda.h>

#include "kdtv_proj_tc.cuh"
#include "kdtv_tmap.cuh"

namespace kdtv {
namespace {

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 32 elements of d_in: rows g and g + 8 of A, row g of x.
__device__ __forceinline__ void mma_32(float (&d)[4], const uint4& lo, const uint4& hi, const uint4& x) {
  mma_16x8x16(d, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
  mma_16x8x16(d, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
}

// Eight E4M3 bytes times 2^(byte - 127) as four bf16 pairs (exact where bf16 reaches).
__device__ __forceinline__ uint4 widen8(uint2 w, uint32_t byte) {
  const float f = scale_of_byte(byte);
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 v = widen2(((k < 2 ? w.x : w.y) >> (16 * (k & 1))) & 0xffffu);
    o[k] = pack_bf16x2(v.x * f, v.y * f);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A block's request: its rows, and where its adapter stands among the tile's.
struct Low {
  int b, n, id, hr;                        // request, live rows, adapter, rows of half a block
  int first, chunks;                       // its adapter's first chunk, chunks of the tile
  float s;
};
__device__ __forceinline__ char* low_place(const ProjArgs& a, const Low& w, int i, int c, int p, int h) {
  int flip;
  char* at = part_row(a, w.b, i, w.hr, c, p, &flip);
  return at + ((h ^ flip) << 4);
}
// False: nothing to do (the same for all of the block).  All of the block comes along.
__device__ __forceinline__ bool low_request(const ProjArgs& a, int b, int i0, Low& w) {
  __shared__ uint32_t bits[kWords];
  __shared__ int s_slot, s_slots;
  w.b = b;
  w.n = live_rows(a.n_live, b, a.N);
  const int raw = a.adapter[b];                            // (both loads under way)
  if (i0 >= w.n) return false;
  w.id = proj_adapter(a, raw);
  if (w.id == -2 || (w.id < 0 && a.requests == 1)) return false;
  w.hr = half_rows_of(a, w.n);
  if (a.requests == 1) {
    w.first = 0;
    w.chunks = a.chunks;
  } else {
    // the tile's adapters, a request a thread
    const int words = (a.adapters + 31) / 32, g = (int)divide(b, a.by_requests);
    for (int k = threadIdx.x; k < words; k += blockDim.x) bits[k] = 0u;
    __syncthreads();
    for (int c = g * a.requests + threadIdx.x; c < min(a.B, (g + 1) * a.requests); c += blockDim.x) {
      const int n = live_rows(a.n_live, c, a.N), id = a.adapter[c];
      if (n > 0 && id >= 0 && id < a.adapters) atomicOr(&bits[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      int below = 0, slots = 0;
      for (int k = lane; k < words; k += 32) {
        slots += __popc(bits[k]);
        if (32 * k <= w.id) below += __popc(k == w.id >> 5 ? bits[k] & ((1u << (w.id & 31)) - 1u) : bits[k]);
      }
      below = warp_sum(below);
      slots = warp_sum(slots);
      if (lane == 0) s_slot = below, s_slots = slots;
    }
    __syncthreads();
    w.first = s_slot * a.chunks;
    w.chunks = s_slots * a.chunks;
  }
  w.s = w.id >= 0 && a.adapter_scale ? a.adapter_scale[w.id] : 1.f;
  return true;
}
// Zeros for the tile's other adapters in rows i0 .. i1 - 1.
__device__ __forceinline__ void low_zeros(const ProjArgs& a, const Low& w, int i0, int i1) {
  const int others = w.chunks - (w.id < 0 ? 0 : a.chunks);
  for (int e = threadIdx.x; e < (i1 - i0) * others * 4; e += blockDim.x) {
    const int i = e / (others * 4), r = e - i * (others * 4), c = r >> 2;
    *reinterpret_cast<uint4*>(low_place(a, w, i0 + i, w.id >= 0 && c >= w.first ? c + a.chunks : c, (r >> 1) & 1, r & 1)) =
        make_uint4(0u, 0u, 0u, 0u);
  }
}
// A lane's sums of 16 ranks from rank0 on and 8 tokens from row t0 on, in two parts (16 significant bits).
__device__ __forceinline__ void low_store(const ProjArgs& a, const Low& w, const float (&acc)[4], int rank0, int t0) {
  const int lane = threadIdx.x & 31, c = rank0 >> 4;       // (rank0 is a multiple of 16)
  if (c >= a.chunks) return;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = t0 + 2 * (lane & 3) + e;
    if (i >= w.n) continue;
    int flip;
    char* const row = part_row(a, w.b, i, w.hr, w.first + c, 0, &flip) + (lane >> 2) * 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // (ranks that fill up the last 16: 0, not the NaN of an infinite x times A's zeros behind the rank, a multiple of 8)
      const float v = rank0 + 8 * h < a.R ? w.s * acc[2 * h + e] : 0.f;
      // (bf16's largest value for what would round beyond it: the other part has the rest)
      constexpr float most = 0x1.fep127f;
      const __nv_bfloat16 hi = __float2bfloat16_rn(fabsf(v) < INFINITY ? fminf(fmaxf(v, -most), most) : v);
      const float left = v - __bfloat162float(hi);         // exact; not a number where v is not finite
      char* const at = row + ((h ^ flip) << 4);
      *reinterpret_cast<__nv_bfloat16*>(at) = hi;
      *reinterpret_cast<__nv_bfloat16*>(at + (long long)a.half_cols * 32) = __float2bfloat16_rn(fabsf(left) < INFINITY ? left : 0.f);
    }
  }
}
// The sums of a cluster's blocks to its first one, in their order.
template <int V>
__device__ __forceinline__ void low_join(float (&acc)[V], float (*red)[32], bool mine, int part, int split) {
  const int lane = threadIdx.x & 31;
  if (mine && part > 0)
#pragma unroll
    for (int k = 0; k < V; ++k) red[k][lane] = acc[k];
  cluster_sync();
  if (mine && part == 0)
    for (int c = 1; c < split; ++c)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        float v;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa(smem_u32(&red[k][lane]), c)) : "memory");
        acc[k] += v;
      }
  cluster_sync();                                          // (the others' memory is read)
}

// ---- few rows of a request ---------------------------------------------------------------------
// A block has 16 ranks and up to 8 rows of a request; its eight warps every
// eighth 32 elements of d_in each, the next kAhead of them on their way from
// global memory to registers while these are multiplied; `split` blocks of a
// cluster share d_in.  Little shared memory and few registers, since it runs
// beside the projection's CTAs.  Bound by the latency of its loads (64 requests of one row, 8192
// elements, 16 ranks: 13 us from a cold cache, of eight one-byte rows and 32 ranks 18; hidden beside the projection).
constexpr int kFew = 8, kWays = 8, kAhead = 2;

template <bool kOneByte>
__global__ void __launch_bounds__(32 * kWays, 3) proj_low_few_kernel(const __grid_constant__ ProjArgs a, int split) {
  __shared__ float red[kWays / 2][4][32];
  grid_dep_launch();                 // the projection may be launched; its adapters' units wait for this grid
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = blockIdx.x, q = lane & 3, g = lane >> 2;
  Low w;
  if (!low_request(a, blockIdx.z, 0, w)) return;
  if (blockIdx.y == 0 && part == 0 && a.requests > 1) low_zeros(a, w, 0, w.n);
  if (w.id < 0) return;
  const int rank0 = blockIdx.y * 16;
  float acc[4] = {};
  const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(a.A) + ((long long)w.id * a.R + rank0 + g) * a.K + 8 * q;
  const char* x = static_cast<const char*>(a.x) + (w.b * a.xs[0] + g * a.xs[1] + 8 * q) * (kOneByte ? 1 : 2);
  const uint8_t* xe = a.x_scale + ((long long)w.b * a.N + g) * (a.K / KDTV_GROUP);
  struct Step {
    uint4 lo[kAhead], hi[kAhead], x[kAhead];             // (one-byte x: in the first two words)
    uint32_t e[kAhead];
  };
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  const int stride = split * kWays * 32 * kAhead;
  auto load = [&](Step& s, int k0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = k0 + u * kWays * 32;
      const bool in = k + 8 * q < a.K, on = in && g < w.n;
      s.lo[u] = in && rank0 + g < a.R ? *reinterpret_cast<const uint4*>(A + k) : none;
      s.hi[u] = in && rank0 + g + 8 < a.R ? *reinterpret_cast<const uint4*>(A + 8ll * a.K + k) : none;
      s.x[u] = none;
      if constexpr (kOneByte) {
        s.e[u] = 127u;
        if (on) {
          const uint2 v = *reinterpret_cast<const uint2*>(x + k);
          s.x[u].x = v.x;
          s.x[u].y = v.y;
          s.e[u] = xe[k / KDTV_GROUP];
        }
      } else if (on) {
        s.x[u] = *reinterpret_cast<const uint4*>(x + 2 * k);
      }
    }
  };
  auto multiply = [&](const Step& s) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      mma_32(acc, s.lo[u], s.hi[u], kOneByte ? widen8(make_uint2(s.x[u].x, s.x[u].y), s.e[u]) : s.x[u]);
  };
  const int start = part * kWays * 32 * kAhead + warp * 32;
  Step s0, s1;
  load(s0, start);
#pragma unroll 1
  for (int k0 = start; k0 < a.K; k0 += 2 * stride) {       // (loads behind d_in are zeros)
    load(s1, k0 + stride);
    multiply(s0);
    load(s0, k0 + 2 * stride);
    multiply(s1);
  }
#pragma unroll
  for (int half = kWays / 2; half > 0; half /= 2) {        // the upper half's sums to the lower half
    if (warp >= half && warp < 2 * half)
#pragma unroll
      for (int k = 0; k < 4; ++k) red[warp - half][k][lane] = acc[k];
    __syncthreads();
    if (warp < half)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] += red[warp][k][lane];
    __syncthreads();
  }
  if (split > 1) low_join(acc, red[0], warp == 0, part, split);
  if (warp == 0 && part == 0) low_store(a, w, acc, rank0, 0);
}

// ---- many rows ---------------------------------------------------------------------------------
// A block has 64 rows of a request and 16 WR MR ranks; TMA brings both operands
// to a ring in shared memory, and eight warps (WR of them along the ranks)
// multiply all of a stage.  `split` blocks of a cluster share d_in.  Its blocks take an SM
// for themselves and the projection's follow them: loads from global memory
// to registers, beside the projection, took 57 us for 6000 rows of 4096 and
// 64 ranks, where this takes 32 by itself from a cold cache and leaves x in L2.
// Bound by the reads of shared memory (48 KiB for each 16 that land, with 64 ranks).
constexpr int kRows = 64, kRowStages = 12;

template <bool kOneByte, int WR, int MR>
__global__ void __launch_bounds__(288, 1)
proj_low_rows_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_a,
                     const __grid_constant__ ProjArgs a, int split, int stages) {
  constexpr int NT = WR, kRanks = 16 * WR * MR, kBoxes = kOneByte ? 2 : 1;     // tokens' eights of a warp; boxes of A
  constexpr int kXBytes = kRows * kUnitBytes, kABytes = kRanks * kUnitBytes, kStage = kXBytes + kBoxes * kABytes;
  extern __shared__ unsigned char low_smem[];
  float (*red)[MR * NT * 4][32] = reinterpret_cast<float (*)[MR * NT * 4][32]>(low_smem);      // [8]
  uint64_t* bars = reinterpret_cast<uint64_t*>(low_smem + 8 * sizeof(red[0]));               // [2 kRowStages]
  uint32_t& s_abort = *reinterpret_cast<uint32_t*>(bars + 2 * kRowStages);
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = blockIdx.x % split, i0 = blockIdx.x / split * kRows;
  const uint32_t ring = (smem_u32(&s_abort) + 4 + 1023) & ~1023u, full = smem_u32(bars), empty = full + 8 * kRowStages;
  const Guard guard{&s_abort, a.status, 2000000000u};
  if (threadIdx.x < (unsigned)stages) {
    mbar_init(full + 8 * threadIdx.x, 1);
    mbar_init(empty + 8 * threadIdx.x, 8);
  }
  if (threadIdx.x == 0) s_abort = 0u;
  fence_mbar_init();
  Low w;
  if (!low_request(a, blockIdx.z, i0, w)) return;
  if (blockIdx.y == 0 && part == 0 && a.requests > 1) low_zeros(a, w, i0, min(i0 + kRows, w.n));
  if (w.id < 0) return;
  __syncthreads();
  const int rank0 = blockIdx.y * kRanks;
  const int u0 = (int)((long long)a.base * part / split), u1 = (int)((long long)a.base * (part + 1) / split);
  constexpr int kElems = kOneByte ? 128 : 64;              // of d_in in a unit
  float acc[MR * NT * 4] = {};
  int slot = 0;
  uint32_t phase = 0u;
  auto advance = [&]() {
    if (++slot == stages) {
      slot = 0;
      phase ^= 1u;
    }
  };
  if (warp == 8) {
    if (lane == 0) {
      int loads = 0;
      for (int u = u0; u < u1; ++u, ++loads) {
        if (!wait(guard, empty + 8 * slot, phase ^ 1u)) break;
        const uint32_t bar = full + 8 * slot, dst = ring + slot * kStage;
        mbar_expect_tx(bar, kStage);
        tma_load_3d(dst, &tm_x, bar, u * kElems, i0, w.b);
        for (int k = 0; k < kBoxes; ++k) tma_load_3d(dst + kXBytes + k * kABytes, &tm_a, bar, u * kElems + 64 * k, rank0, w.id);
        advance();
      }
      for (int k = loads > stages ? loads - stages : 0; k < loads; ++k) drain(guard, full + 8 * (k % stages), (k / stages) & 1);
    }
    __syncwarp();
  } else {
    const int wr = warp % WR, wt = warp / WR, q = lane & 3, g = lane >> 2, row_bytes = a.K / KDTV_GROUP;
    auto lds = [](uint32_t at, int row, int chunk) -> uint4 {         // 16 bytes of a swizzled row
      uint4 v;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at + row * 128 + ((chunk ^ (row & 7)) << 4)) : "memory");
      return v;
    };
    // one byte: the exponents of a row's four groups, two units ahead
    const uint8_t* xe[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int i = i0 + (wt * NT + j) * 8 + g;
      xe[j] = kOneByte && i < w.n ? a.x_scale + ((long long)w.b * a.N + i) * row_bytes : nullptr;
    }
    auto exponents = [&](int j, int u) -> uint32_t {
      if (!kOneByte || !xe[j] || u >= u1) return 0x7f7f7f7fu;
      if (a.scale_mode) return *reinterpret_cast<const uint32_t*>(xe[j] + 4 * u);
      uint32_t v[1];
      exponent_words(xe[j], 4 * u, row_bytes, a.x_scale + (long long)a.B * a.N * row_bytes, v);
      return v[0];
    };
    uint32_t now[NT], soon[NT], later[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      soon[j] = exponents(j, u0);
      later[j] = exponents(j, u0 + 1);
    }
    for (int u = u0; u < u1; ++u) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        now[j] = soon[j];
        soon[j] = later[j];
        later[j] = exponents(j, u + 2);
      }
      if (!wait_warp(guard, full + 8 * slot, phase)) break;
      const uint32_t xs = ring + slot * kStage, as = xs + kXBytes;
      // 32 elements a step: lane q's are 16 q + 8 (step % 2) .. + 7 of 64, every other 16 bytes of A's rows, so that two rows'
      // lie in different banks (with 8 q .. + 7 of 32 every read took twice as long).
      uint4 both[NT];                          // one byte: two steps' elements of x
#pragma unroll
      for (int step = 0; step < kElems / 32; ++step) {
        const int h = step & 1, box = step >> 1;
        uint4 x[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int row = (wt * NT + j) * 8 + g;
          if constexpr (kOneByte) {
            if (h == 0) both[j] = lds(xs, row, 4 * box + q);
            x[j] = widen8(h ? make_uint2(both[j].z, both[j].w) : make_uint2(both[j].x, both[j].y),
                          (now[j] >> (8 * (2 * box + (q >> 1)))) & 0xffu);
          } else {
            x[j] = lds(xs, row, 2 * q + h);
          }
        }
#pragma unroll
        for (int m = 0; m < MR; ++m) {
          const int row = (wr * MR + m) * 16 + g;
          const uint32_t at = as + box * kABytes;          // (bf16: one box)
          const uint4 lo = lds(at, row, 2 * q + h), hi = lds(at, row + 8, 2 * q + h);
#pragma unroll
          for (int j = 0; j < NT; ++j) mma_32(reinterpret_cast<float(&)[4]>(acc[(m * NT + j) * 4]), lo, hi, x[j]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * slot);
      advance();
    }
  }
  if (split > 1) low_join(acc, red[warp & 7], warp < 8, part, split);
  if (warp < 8 && part == 0) {
    const int wr = warp % WR, wt = warp / WR;
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        low_store(a, w, reinterpret_cast<float(&)[4]>(acc[(m * NT + j) * 4]), rank0 + (wr * MR + m) * 16, i0 + (wt * NT + j) * 8);
  }
}

// d_in over as many blocks of a cluster, `cap` at most, as keep the grid within `most`, 512 elements each at least.
int split_of(const ProjArgs& a, long long blocks, long long most, int cap) {
  int split = 1;
  while (split < cap && blocks * split * 2 <= most && a.K / (2 * split) >= 512) split *= 2;
  return split;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_split(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, int split, cudaStream_t st, Args&&... args) {
  const cudaError_t err = beside(kernel);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)split, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

template <bool kOneByte, int WR, int MR>
cudaError_t launch_rows(const ProjArgs& a, int sms, cudaStream_t st) {
  constexpr uint64_t e = kOneByte ? 1 : 2;
  constexpr int ranks = 16 * WR * MR, stage = (kRows + (kOneByte ? 2 : 1) * ranks) * kUnitBytes;
  CUtensorMap tx, ta;
  const uint64_t row = (a.K * e + 15) / 16 * 16;           // strides of single rows do not matter
  const uint64_t xdims[3] = {(uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.B};
  const uint64_t xstrides[2] = {a.N > 1 ? a.xs[1] * e : row, a.B > 1 ? a.xs[0] * e : row * a.N};
  const uint32_t xbox[3] = {(uint32_t)(kUnitBytes / e), kRows, 1};
  const uint64_t adims[3] = {(uint64_t)a.K, (uint64_t)a.R, (uint64_t)a.adapters};
  const uint64_t astrides[2] = {(uint64_t)a.K * 2, (uint64_t)a.R * a.K * 2};
  const uint32_t abox[3] = {64, ranks, 1};
  if (encode_nd(&tx, a.x, 3, xdims, xstrides, xbox, (int)e, 128) != CUDA_SUCCESS ||
      encode_nd(&ta, a.A, 3, adims, astrides, abox, 2, 128) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const int blocks = (a.N + kRows - 1) / kRows, rank_blocks = (a.R + ranks - 1) / ranks;
  const long long all = (long long)blocks * rank_blocks * a.B;
  // (8000 rows of 4096, 64 ranks, a call with 256 outputs: 128 blocks 64 us, twice as many that share d_in 69; 1003 rows of
  // 6656, one byte: four share d_in 35 us, eight 36.)  Where some of the rows may not be live, long sums are shared more:
  // (4 x up to 2000 rows of 4096, half of them live, 12288 outputs: 378 us, 367 with that.)
  const int split = split_of(a, all, a.n_live && a.base >= 32 ? 2 * sms : sms, 4);
  // one block an SM: a deep ring; more: two of them
  int stages = (all * split <= sms ? 190 : 92) * 1024 / stage;
  stages = stages < kRowStages ? stages : kRowStages;
  const size_t smem = (size_t)stages * stage + 8 * (MR * WR * 4 * 32 * 4) + 2 * kRowStages * 8 + 4 + 1023;
  const auto kern = proj_low_rows_kernel<kOneByte, WR, MR>;
  const cudaError_t err = allow_smem(kern, smem);
  if (err != cudaSuccess) return err;
  return launch_split(kern, dim3((unsigned)(blocks * split), (unsigned)rank_blocks, (unsigned)a.B), 288, smem,
                      split, st, tx, ta, a, split, stages);
}

template <bool kOneByte>
cudaError_t launch_t(const ProjArgs& a, int sms, cudaStream_t st) {
  if (a.N <= kFew) {
    const int ranks = (a.R + 15) / 16, split = split_of(a, (long long)ranks * a.B, sms, 8);
    return launch_split(proj_low_few_kernel<kOneByte>, dim3((unsigned)split, (unsigned)ranks, (unsigned)a.B), 32 * kWays, 0, split, st, a, split);
  }
  if (a.R <= 16) return launch_rows<kOneByte, 1, 1>(a, sms, st);
  if (a.R <= 32) return launch_rows<kOneByte, 2, 1>(a, sms, st);
  return launch_rows<kOneByte, 2, 2>(a, sms, st);
}

}  // namespace

cudaError_t launch_proj_low(const ProjArgs& a, int sms, cudaStream_t st) {
  return a.dtype == KDTV_BF16_FP8KV ? launch_t<true>(a, sms, st) : launch_t<false>(a, sms, st);
}

}  // namespace kdtv
