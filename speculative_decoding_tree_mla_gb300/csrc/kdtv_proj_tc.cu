// Tensor-core (tcgen05) path of kdtv_project: bf16, or one-byte inputs and
// weights with an exponent byte per 32 elements.
//
// Mathematics.  y = W x + Bm_a (s_a A_a x), a the request's adapter.  Outputs are
// the rows (TMEM lanes) of a product, tokens its columns: D[f, t] = sum_k W[f, k]
// x[t, k], so that one token costs a 16-column product, not a 128-row one.  The
// adapters are more of the same sum: with the adapters of a tile's requests
// side by side, [W | Bm_0 | Bm_1 ..] [x ; v_0 ; v_1 ..], where v_a = s_a A_a x for the
// tokens of adapter a and 0 for the others.  v is fp32, split into two bf16 parts
// (16 significant bits), each multiplied with Bm.  0 * infinity must not carry
// one adapter's values into another's tokens: an output that is not finite, in a
// tile with several adapters, is computed again on its own.
//
// Kernels: proj_low_kernel (v of all tokens, in the tiles' order, as the second
// kernel's operands lie in shared memory) and proj_tc_kernel (everything else),
// launched while the first runs; only the adapters' units wait for it.
//
// Work.  A unit is 128 bytes of d_in (64 bf16, 128 one-byte elements) or two
// chunks of 16 ranks, for one tile of 128 outputs and up to 256 (one byte: 224)
// tokens.  Whole tiles go round the CTAs; what does not fill a round is cut
// evenly by units (at least one round, so that no CTA gets little).  A tile
// that several CTAs share: each leaves its sums, and the last to come adds them in
// the order of the units, so that the result does not depend on who that is.
//
// One byte: exponent bytes travel as they are to the tensor cores, which take
// one per 32 elements and operand row (block-scaled products), so sums are in true
// units and the adapters' bf16 products add to them.

#include <cuda.h>

#include "kdtv_guard.cuh"
#include "kdtv_proj.cuh"
#include "kdtv_tmap.cuh"

#include <string.h>

namespace kdtv {
namespace {

using namespace ptx;

constexpr int kFeatures = 128;             // outputs of a tile
constexpr int kUnitBytes = 128;            // of d_in in a unit
constexpr int kWBytes = kFeatures * kUnitBytes;
constexpr int kMaxStages = 12;
constexpr int kMaxGroups = 1024;           // groups of requests in a launch
constexpr int kMaxCtas = 256;
constexpr int kWords = KDTV_MAX_ADAPTERS / 32;
constexpr int kScaleBytes = 3 * 512;       // a stage's exponent bytes: W, tokens 0 - 127, the others
constexpr int kSuper = 8;                  // token tiles that share a W tile in a row

// ---- which adapters a tile has -------------------------------------------------------------
// Adapters of a group of requests that have live rows, as a bitmap in shared
// memory (by a warp); their places are the order of their numbers.
__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

__device__ __forceinline__ int group_bitmap(const ProjArgs& a, int g, uint32_t* bits, bool* live) {
  const int lane = threadIdx.x & 31, words = (a.adapters + 31) / 32;
  for (int w = lane; w < words; w += 32) bits[w] = 0u;
  __syncwarp();
  bool any = false;
  for (int b = g * a.requests + lane; b < min(a.B, (g + 1) * a.requests); b += 32) {
    if (live_rows(a.n_live, b, a.N) <= 0) continue;
    const int id = proj_adapter(a, b);
    any |= id != -2;
    if (id >= 0) atomicOr(&bits[id >> 5], 1u << (id & 31));
  }
  *live = __any_sync(0xffffffffu, any);
  __syncwarp();
  int count = 0;
  for (int w = lane; w < words; w += 32) count += __popc(bits[w]);
  return warp_sum(count);
}

// ---- v = s_a A_a x ---------------------------------------------------------------------------
// mma.sync products of 16 ranks and 8 tokens, straight from global memory: the
// order of d_in within a product does not matter as long as both operands have
// the same, so a lane's 16-byte load (8 elements of a row) is two products'
// fragments.  A warp has 16 MR ranks, 8 NT tokens and every KW-th 32 elements
// of d_in; KW warps' sums meet in shared memory, in their order.  Bound by the
// latency of its loads (few tokens) or L2 (many); it runs beside the
// first units of the projection.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

template <bool kOneByte, int MR, int NT, int TW, int KW>
__global__ void __launch_bounds__(32 * TW * KW) proj_low_kernel(const __grid_constant__ ProjArgs a) {
  __shared__ uint32_t bits[kWords];
  __shared__ int s_slot, s_slots;
  __shared__ float red[(KW - 1) * TW][MR * NT * 4][32];
  grid_dep_launch();                 // the projection may be launched; its adapters' units wait for this grid
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
    for (int i = threadIdx.x; i < a.n_counters; i += 32 * TW * KW) a.counters[i] = 0u;
  if (!a.adapter) return;
  constexpr int kTokens = 8 * NT * TW;
  const int b = blockIdx.z, i0 = blockIdx.x * kTokens, n = live_rows(a.n_live, b, a.N);
  if (i0 >= n) return;
  const int id = proj_adapter(a, b);
  if (id == -2) return;
  const int g = (int)divide(b, a.by_requests), rq = b - g * a.requests;
  if (a.requests == 1) {
    if (id < 0) return;
    if (threadIdx.x == 0) s_slot = 0, s_slots = 1;
  } else if (warp == 0) {
    bool live;
    const int slots = group_bitmap(a, g, bits, &live);
    int below = 0;
    for (int w = lane; w < kWords && 32 * w <= id; w += 32)
      below += __popc(w == id >> 5 ? bits[w] & ((1u << (id & 31)) - 1u) : bits[w]);
    below = warp_sum(below);
    if (lane == 0) s_slot = below, s_slots = slots;
  }
  __syncthreads();
  const int first = s_slot * a.chunks, chunks = s_slots * a.chunks, rows = min(kTokens, n - i0);
  // Where row i's 16 ranks of chunk c, part p start; its two 16-byte halves h lie swizzled.
  auto place = [&](int i, int c, int p, int h) {
    const int j = (int)divide(i, a.by_rows), col = rq * a.rows + i - j * a.rows;
    return a.parts + ((long long)(g * a.blocks + j) * a.pairs + (c >> 1)) * proj_pair_bytes(a) +
           (long long)((c & 1) * 2 + p) * a.cols * 32 + col * 32 + ((h ^ ((col >> 2) & 1)) << 4);
  };
  if (blockIdx.y == 0 && a.requests > 1) {              // the other adapters' chunks
    const int others = chunks - (id < 0 ? 0 : a.chunks);
    for (int e = threadIdx.x; e < rows * others * 4; e += 32 * TW * KW) {
      const int i = e / (others * 4), r = e - i * (others * 4), c = r >> 2;
      *reinterpret_cast<uint4*>(place(i0 + i, id >= 0 && c >= first ? c + a.chunks : c, (r >> 1) & 1, r & 1)) =
          make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (id < 0) return;

  const int tw = warp % TW, kw = warp / TW, q = lane & 3, gr = lane >> 2;
  const int rank0 = blockIdx.y * 16 * MR, t0 = i0 + tw * 8 * NT;
  const bool busy = t0 < n;
  float acc[MR][NT][4] = {};
  if (busy) {
    const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(a.A) + ((long long)id * a.R + rank0 + gr) * a.K + 8 * q;
    const char* x = static_cast<const char*>(a.x) + (b * a.xs[0] + (t0 + gr) * a.xs[1] + 8 * q) * (kOneByte ? 1 : 2);
    const uint8_t* xe = a.x_scale + ((long long)b * a.N + t0 + gr) * (a.K / KDTV_GROUP);
    const long long xrow = 8 * a.xs[1] * (kOneByte ? 1 : 2);
    constexpr int U = MR * NT >= 8 ? 1 : 4;               // steps whose loads are under way together
    for (int k0 = kw * 32; k0 < a.K; k0 += KW * 32 * U) {
      uint4 va[U][MR][2], vx[U][NT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * KW * 32;
        const bool in = k + 8 * q < a.K;
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            va[u][m][h] = in && rank0 + 16 * m + 8 * h + gr < a.R
                              ? *reinterpret_cast<const uint4*>(A + (long long)(16 * m + 8 * h) * a.K + k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const bool on = in && t0 + 8 * j + gr < n;
          if constexpr (kOneByte) {
            const uint2 w = on ? *reinterpret_cast<const uint2*>(x + j * xrow + k) : make_uint2(0u, 0u);
            vx[u][j] = widen8(w, on ? xe[(long long)8 * j * (a.K / KDTV_GROUP) + k / KDTV_GROUP] : 127u);
          } else {
            vx[u][j] = on ? *reinterpret_cast<const uint4*>(x + j * xrow + 2 * k) : make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma_16x8x16(acc[m][j], va[u][m][0].x, va[u][m][1].x, va[u][m][0].y, va[u][m][1].y, vx[u][j].x, vx[u][j].y);
            mma_16x8x16(acc[m][j], va[u][m][0].z, va[u][m][1].z, va[u][m][0].w, va[u][m][1].w, vx[u][j].z, vx[u][j].w);
          }
    }
    if (kw > 0)
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) red[(kw - 1) * TW + tw][(m * NT + j) * 4 + k][lane] = acc[m][j][k];
  }
  __syncthreads();
  if (kw > 0 || !busy) return;
  const float s = a.adapter_scale ? a.adapter_scale[id] : 1.f;
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v = acc[m][j][k];
        for (int w = 0; w < KW - 1; ++w) v += red[w * TW + tw][(m * NT + j) * 4 + k][lane];
        v *= s;
        const int rank = rank0 + 16 * m + gr + (k >> 1) * 8, i = t0 + 8 * j + 2 * q + (k & 1), c = rank >> 4;
        if (i >= n || c >= a.chunks) continue;
        const __nv_bfloat16 hi = __float2bfloat16_rn(v);
        const float left = v - __bfloat162float(hi);       // exact; not a number where v is not finite
        const int h = (rank >> 3) & 1, at = (rank & 7) * 2;
        *reinterpret_cast<__nv_bfloat16*>(place(i, first + c, 0, h) + at) = hi;
        *reinterpret_cast<__nv_bfloat16*>(place(i, first + c, 1, h) + at) =
            __float2bfloat16_rn(fabsf(left) < INFINITY ? left : 0.f);
      }
}

// ---- the projection --------------------------------------------------------------------------
enum {
  B_FULL = 0, B_EMPTY = B_FULL + kMaxStages, B_ACC_FULL = B_EMPTY + kMaxStages, B_ACC_EMPTY = B_ACC_FULL + 2,
  B_DONE = B_ACC_EMPTY + 2, B_STALL, B_COUNT
};

constexpr int kWarpTma = 0, kWarpMma = 1, kWarpOut = 4, kWarpScale = 8;   // (2, 3: planning only)
__host__ __device__ constexpr int threads_of(bool one_byte) { return one_byte ? 384 : 256; }
__host__ __device__ constexpr int acc_columns(bool one_byte) { return one_byte ? 224 : 256; }
constexpr uint32_t kScaleColumn = 448;      // one byte: exponents behind the two accumulators

// Shared memory behind the ring.
struct ProjShared {
  uint64_t bars[B_COUNT];
  uint32_t tmem, abort, last[2];
  int total_tiles, cut, share, pad;         // token tiles times outputs' tiles; cut tiles; units of a CTA's share
  int first[kMaxGroups + 1];                // token tiles before each group
  int chunks[kMaxGroups];                   // 16-rank chunks of its tiles' adapters
  int start[2 * kMaxCtas + 1];              // units before each cut tile
  long long y_at[256];                      // offset of each column's output row, -1: none
  uint32_t bits[kWords];
  uint16_t ids[256];                        // the adapters of the producer's tile
};

// A part of a tile: units k0 .. k1 - 1; behind a.base of d_in come pairs of chunks.
struct Item {
  int g, j, f, k0, k1, chunks;
  int cut, seg, segs;                       // cut tile's number (-1: whole), place among its segments
};

// The items of CTA c, in the order in which every role sees them: its share of
// the cut tiles, then whole tiles.
struct Walk {
  int u, u_end, tile, s;                    // next unit of the share, next whole tile, current cut tile
};

__device__ __forceinline__ int units_of(const ProjArgs& a, int chunks) { return a.base + (chunks + 1) / 2; }

__device__ __forceinline__ void locate(const ProjArgs& a, const ProjShared& sh, int order, Item& it) {
  const int n = sh.first[a.groups], super = order / (kSuper * a.features), r = order - super * kSuper * a.features;
  const int w = min(kSuper, n - kSuper * super);
  it.f = r / w;
  const int t = kSuper * super + r - it.f * w;
  int lo = 0, hi = a.groups - 1;            // the last group with first <= t that has tiles
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sh.first[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  it.g = lo;
  it.j = t - sh.first[lo];
  it.chunks = sh.chunks[lo];
}

__device__ __forceinline__ Walk walk(const ProjShared& sh) {
  Walk w;
  const int all = sh.cut ? sh.start[sh.cut] : 0;
  w.u = min(all, (int)blockIdx.x * sh.share);
  w.u_end = min(all, w.u + sh.share);
  w.tile = sh.cut + blockIdx.x;
  int lo = 0, hi = sh.cut - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sh.start[mid] <= w.u) lo = mid;
    else hi = mid - 1;
  }
  w.s = lo;
  return w;
}

__device__ __forceinline__ bool next(const ProjArgs& a, const ProjShared& sh, Walk& w, Item& it) {
  if (w.u < w.u_end) {
    locate(a, sh, w.s, it);
    const int start = sh.start[w.s], end = sh.start[w.s + 1], stop = min(end, w.u_end);
    it.k0 = w.u - start;
    it.k1 = stop - start;
    const int c0 = start / sh.share;
    it.segs = (end - 1) / sh.share - c0 + 1;
    it.seg = (int)blockIdx.x - c0;
    it.cut = it.segs > 1 ? w.s : -1;
    w.u = stop;
    if (stop == end) ++w.s;
    return true;
  }
  if (w.tile >= sh.total_tiles) return false;
  locate(a, sh, w.tile, it);
  it.k0 = 0;
  it.k1 = units_of(a, it.chunks);
  it.cut = -1;
  it.seg = 0;
  it.segs = 1;
  w.tile += gridDim.x;
  return true;
}

// Partial of segment `seg` of a cut tile whose first segment is CTA c0's: a CTA has two
// places, one for the tile that its share begins in.
__device__ __forceinline__ float* partial_of(const ProjArgs& a, int c0, int seg) {
  return a.partial + (2ll * (c0 + seg) + (seg == 0 ? 1 : 0)) * a.cols * kFeatures;
}

// D[tmem] (+)= A[smem desc] * B[smem desc]^T of E4M3 elements with an exponent
// byte per 32 of each row (in TMEM), 32 elements deep, fp32 accumulation.
__device__ __forceinline__ void mma_scaled(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t a_scale, uint32_t b_scale, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\t"
               "setp.ne.b32 p, %6, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
               :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
               : "memory");
}
// E4M3 A and B, exponent bytes as scales; bits 4 and 29 on: which byte of a word.
__device__ __forceinline__ uint32_t idesc_scaled(int N, int byte) {
  return ((uint32_t)byte << 4) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(kFeatures >> 4) << 24) |
         ((uint32_t)byte << 29);
}
// 512 bytes of exponents: four words of 32 lanes, the same in each quarter of TMEM's lanes.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t smem) {
  uint64_t d = 0;                           // no swizzle, 8-row groups 128 bytes apart
  d |= (uint64_t)((smem >> 4) & 0x3FFFu);
  d |= (uint64_t)(128u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(tmem), "l"(d) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// One output by itself, for a value that is not finite where several adapters share a tile.
template <bool kOneByte>
__device__ __noinline__ float alone(const ProjArgs& a, int b, int i, int f) {
  float sum = 0.f;
  for (int k = 0; k < a.K; ++k) {
    float x, w;
    if constexpr (kOneByte) {
      const int groups = a.K / KDTV_GROUP;
      x = to_f32(static_cast<const __nv_fp8_e4m3*>(a.x)[b * a.xs[0] + i * a.xs[1] + k]) *
          scale_of_byte(a.x_scale[((long long)b * a.N + i) * groups + k / KDTV_GROUP]);
      w = to_f32(static_cast<const __nv_fp8_e4m3*>(a.W)[(long long)f * a.K + k]) *
          scale_of_byte(a.W_scale[(long long)f * groups + k / KDTV_GROUP]);
    } else {
      x = to_f32(static_cast<const __nv_bfloat16*>(a.x)[b * a.xs[0] + i * a.xs[1] + k]);
      w = to_f32(static_cast<const __nv_bfloat16*>(a.W)[(long long)f * a.K + k]);
    }
    sum = fmaf(x, w, sum);
  }
  const int id = a.adapter[b];
  if (id < 0) return sum;
  // this request's v, from its place among the tile's adapters
  const int g = (int)divide(b, a.by_requests), col = (b - g * a.requests) * a.rows + i;
  int slot = 0;
  for (int c = g * a.requests; c < min(a.B, (g + 1) * a.requests); ++c) {
    const int other = a.adapter[c];
    if (other < 0 || other >= id || live_rows(a.n_live, c, a.N) <= 0) continue;
    bool seen = false;
    for (int e = g * a.requests; e < c; ++e) seen |= a.adapter[e] == other && live_rows(a.n_live, e, a.N) > 0;
    slot += !seen;
  }
  for (int r = 0; r < a.R; ++r) {
    const int c = slot * a.chunks + (r >> 4);
    const char* at = a.parts + ((long long)g * a.pairs + (c >> 1)) * proj_pair_bytes(a) +
                     (long long)(c & 1) * 2 * a.cols * 32 + col * 32 + ((((r >> 3) & 1) ^ ((col >> 2) & 1)) << 4) + (r & 7) * 2;
    const float v = to_f32(*reinterpret_cast<const __nv_bfloat16*>(at)) +
                    to_f32(*reinterpret_cast<const __nv_bfloat16*>(at + (long long)a.cols * 32));
    sum = fmaf(v, to_f32(static_cast<const __nv_bfloat16*>(a.Bm)[((long long)id * a.M + f) * a.R + r]), sum);
  }
  return sum;
}

template <bool kOneByte>
__global__ void __launch_bounds__(threads_of(kOneByte), 1)
proj_tc_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
               const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ ProjArgs a, int stall) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x_bytes = a.cols * kUnitBytes, stage_bytes = kWBytes + x_bytes;
  ProjShared& sh = *reinterpret_cast<ProjShared*>(smem + (size_t)a.stages * (stage_bytes + (kOneByte ? kScaleBytes : 0)));
  const uint32_t ring = smem_u32(smem), scales = ring + a.stages * stage_bytes, bars = smem_u32(sh.bars);
  auto BAR = [&](int i) { return bars + 8u * i; };
  const Guard guard{&sh.abort, a.status, stall ? 20000000u : 2000000000u};

  // ---- set up, and plan: every CTA derives the same tiles from n_live and adapter ------------------
  if (threadIdx.x < B_COUNT) {
    const int i = threadIdx.x;
    mbar_init(BAR(i), i < B_EMPTY ? (kOneByte ? 5 : 1) : i >= B_ACC_EMPTY && i < B_DONE ? 4 : 1);
  }
  if (threadIdx.x == 0) sh.abort = 0u;
  fence_mbar_init();
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  if (warp == kWarpTma && lane == 0) {
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_x);
    if (a.adapter) prefetch_tmap(&tm_b);
  }
  if (a.requests == 1) {
    for (int g = threadIdx.x; g < a.groups; g += threads_of(kOneByte)) {
      const int n = live_rows(a.n_live, g, a.N), id = n > 0 ? proj_adapter(a, g) : -1;
      sh.first[g] = id == -2 ? 0 : (int)divide(n + a.rows - 1, a.by_rows);
      sh.chunks[g] = id >= 0 ? a.chunks : 0;
    }
  } else {
    uint32_t* bits = reinterpret_cast<uint32_t*>(smem) + warp * kWords;     // (the ring is not in use yet)
    for (int g = warp; g < a.groups; g += threads_of(kOneByte) / 32) {
      bool live;
      const int slots = group_bitmap(a, g, bits, &live);
      __syncwarp();
      if (lane == 0) {
        sh.first[g] = live ? 1 : 0;
        sh.chunks[g] = slots * a.chunks;
      }
    }
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    int sum = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 32) {
      const int own = g0 + lane < a.groups ? sh.first[g0 + lane] : 0;
      int incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (g0 + lane < a.groups) sh.first[g0 + lane] = sum + incl - own;
      sum += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) sh.first[a.groups] = sum;
    __syncwarp();
    // Whole rounds of whole tiles but the last, and what is left cut into equal shares.  Tiles of few
    // units are not cut, nor are almost full rounds.
    const int tiles = sum * a.features, ctas = gridDim.x;
    int cut = tiles % ctas == 0 ? 0 : tiles < 2 * ctas ? tiles : tiles % ctas + ctas;
    if (a.base < 16 || (tiles < ctas && tiles * 20 > ctas * 19)) cut = 0;
    Item it;
    int u = 0;
    for (int t0 = 0; t0 < cut; t0 += 32) {
      int own = 0;
      if (t0 + lane < cut) {
        locate(a, sh, t0 + lane, it);
        own = units_of(a, it.chunks);
      }
      int incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (t0 + lane < cut) sh.start[t0 + lane] = u + incl - own;
      u += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      sh.start[cut] = u;
      sh.cut = cut;
      sh.total_tiles = tiles;
      sh.share = max(8, (u + ctas - 1) / ctas);
    }
  }
  __syncthreads();
  const uint32_t tmem = sh.tmem;
  Walk w = walk(sh);
  Item it;
  int slot = 0;
  uint32_t phase = 0u;
  auto advance = [&]() {
    if (++slot == a.stages) {
      slot = 0;
      phase ^= 1u;
    }
  };

  if (warp == kWarpTma) {
    // ---- TMA producer --------------------------------------------------------------------------
    bool alive = true, waited = false;
    int loads = 0, listed = -1;
    if (stall) alive = wait_warp(guard, BAR(B_STALL), 0);
    while (alive && next(a, sh, w, it)) {
      if (it.k1 > a.base) {                    // the tile's adapters, once their units come
        if (a.requests == 1) {
          if (lane == 0) sh.ids[0] = (uint16_t)a.adapter[it.g];
        } else if (listed != it.g) {
          bool live;
          group_bitmap(a, it.g, sh.bits, &live);
          int before = 0;
          for (int w0 = 0; w0 < (a.adapters + 31) / 32; w0 += 32) {
            uint32_t m = w0 + lane < (a.adapters + 31) / 32 ? sh.bits[w0 + lane] : 0u;
            int incl = __popc(m);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int v = __shfl_up_sync(0xffffffffu, incl, o);
              if (lane >= o) incl += v;
            }
            int at = before + incl - __popc(m);
            for (; m; m &= m - 1) sh.ids[at++] = (uint16_t)((w0 + lane) * 32 + __ffs(m) - 1);
            before += __shfl_sync(0xffffffffu, incl, 31);
          }
          listed = it.g;
        }
        __syncwarp();
      }
      for (int k = it.k0; k < it.k1; ++k) {
        alive = wait_warp(guard, BAR(B_EMPTY + slot), phase ^ 1u);
        if (!alive) break;
        if (k >= a.base && !waited) {
          grid_dep_wait();                     // v is written
          waited = true;
        }
        if (lane == 0) {
          const uint32_t full = BAR(B_FULL + slot), dst = ring + slot * stage_bytes;
          if (k < a.base) {
            mbar_expect_tx(full, kWBytes + a.requests * a.rows * kUnitBytes);
            tma_load_2d(dst, &tm_w, full, k * (kOneByte ? 128 : 64), it.f * kFeatures);
            tma_load_3d(dst + kWBytes, &tm_x, full, k * (kOneByte ? 128 : 64), it.j * a.rows, it.g * a.requests);
          } else {
            const int p = k - a.base, two = min(2, it.chunks - 2 * p);
            mbar_expect_tx(full, two * (kFeatures * 32 + a.cols * 64));
            for (int c = 2 * p; c < 2 * p + two; ++c) {
              const int s = (int)divide(c, a.by_chunks);
              tma_load_3d(dst + (c & 1) * (kFeatures * 32), &tm_b, full, (c - s * a.chunks) * 16, it.f * kFeatures, sh.ids[s]);
            }
            bulk_load(dst + kWBytes, a.parts + ((long long)(it.g * a.blocks + it.j) * a.pairs + p) * proj_pair_bytes(a),
                      two * a.cols * 64, full);
          }
        }
        __syncwarp();
        advance();
        ++loads;
      }
      __syncwarp();
    }
    for (int x = loads > a.stages ? loads - a.stages : 0; x < loads; ++x)    // every copy has landed
      drain(guard, BAR(B_FULL + x % a.stages), (x / a.stages) & 1);
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ---- products ------------------------------------------------------------------------------
    if (lane == 0) {
      bool alive = true;
      const uint32_t idesc = idesc_bf16(kFeatures, a.cols, 0, 0);
      for (int n = 0; alive && next(a, sh, w, it); ++n) {
        const uint32_t d = tmem + (n & 1) * acc_columns(kOneByte);
        alive = wait(guard, BAR(B_ACC_EMPTY + (n & 1)), ((n >> 1) & 1) ^ 1u);
        uint32_t acc = 0u;
        for (int k = it.k0; alive && k < it.k1; ++k) {
          alive = wait(guard, BAR(B_FULL + slot), phase);
          if (!alive) break;
          tc_fence_after();
          const uint32_t at = ring + slot * stage_bytes;
          if (k < a.base) {
            const uint64_t ad = smem_desc(at, 16, 1024), bd = smem_desc(at + kWBytes, 16, 1024);
            if constexpr (kOneByte) {
              const uint32_t sc = tmem + kScaleColumn + (slot & 3) * 16, ss = scales + slot * kScaleBytes;
              copy_scales(sc, ss);
              copy_scales(sc + 4, ss + 512);
              if (a.cols > 128) copy_scales(sc + 8, ss + 1024);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                mma_scaled(d, ad + 2 * kk, bd + 2 * kk, idesc_scaled(a.cols, kk), sc, sc + 4, acc);
                acc = 1u;
              }
            } else {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                mma_bf16(d, ad + 2 * kk, bd + 2 * kk, idesc, acc);
                acc = 1u;
              }
            }
          } else {
            const int two = min(2, it.chunks - 2 * (k - a.base));
            for (int c = 0; c < two; ++c)
              for (int p = 0; p < 2; ++p) {
                mma_bf16(d, smem_desc_sw32(at + c * (kFeatures * 32)), smem_desc_sw32(at + kWBytes + (c * 2 + p) * a.cols * 32), idesc, acc);
                acc = 1u;
              }
          }
          mma_commit(BAR(B_EMPTY + slot));
          advance();
        }
        if (alive) mma_commit(BAR(B_ACC_FULL + (n & 1)));
      }
      mma_commit(BAR(B_DONE));                 // every product has finished before TMEM is freed
      drain(guard, BAR(B_DONE), 0);
    }
    __syncwarp();
  } else if (warp >= kWarpOut && warp < kWarpOut + 4) {
    // ---- sums to outputs: warp q has TMEM lanes 32 q .., one output each -------------------------------
    const int q = warp - kWarpOut, t = threadIdx.x - 32 * kWarpOut;
    auto meet = [&]() { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    auto agree = [&](bool ok) {                // of the four warps
      uint32_t r;
      asm volatile("{\n\t.reg .pred p, r;\n\tsetp.ne.b32 p, %1, 0;\n\t"
                   "bar.red.and.pred r, 1, 128, p;\n\tselp.u32 %0, 1, 0, r;\n\t}"
                   : "=r"(r) : "r"((uint32_t)ok) : "memory");
      return r != 0u;
    };
    grid_dep_wait();                           // the counters are clear; and no CTA ends before that grid
    for (int n = 0; next(a, sh, w, it); ++n) {
      meet();                                  // the last tile's columns are read
      for (int c = t; c < a.cols; c += 128) {
        const int rq = (int)divide(c, a.by_rows), r = c - rq * a.rows, b = it.g * a.requests + rq, i = it.j * a.rows + r;
        long long at = -1;
        if (rq < a.requests && b < a.B && i < live_rows(a.n_live, b, a.N)) {
          const int id = a.adapter ? a.adapter[b] : -1;
          if (id >= -1 && id < a.adapters) at = b * a.ys[0] + i * a.ys[1];
        }
        sh.y_at[c] = at;
      }
      if (!agree(wait_warp(guard, BAR(B_ACC_FULL + (n & 1)), (n >> 1) & 1))) break;
      tc_fence_after();
      const uint32_t acc = tmem + (n & 1) * acc_columns(kOneByte) + ((uint32_t)(32 * q) << 16);
      const int f = it.f * kFeatures + 32 * q + lane;
      const bool mixed = a.requests > 1 && it.chunks > 0;
      auto put = [&](int c, float v) {
        const long long at = sh.y_at[c];
        if (at < 0 || f >= a.M) return;
        if (mixed && !(fabsf(v) < INFINITY)) {
          const int rq = (int)divide(c, a.by_rows);
          v = alone<kOneByte>(a, it.g * a.requests + rq, c - rq * a.rows, f);
        }
        static_cast<__nv_bfloat16*>(a.y)[at + f] = __float2bfloat16_rn(v);
      };
      auto released = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_ACC_EMPTY + (n & 1)));
      };
      if (it.cut < 0) {
#pragma unroll 1
        for (int c0 = 0; c0 < a.cols; c0 += 16) {
          float v[16];
          __syncwarp();
          tmem_ld16(acc + c0, v);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; ++c) put(c0 + c, v[c]);
        }
        released();
        continue;
      }
      const int c0_cta = (int)blockIdx.x - it.seg;
      float* mine = partial_of(a, c0_cta, it.seg) + 32 * q + lane;
#pragma unroll 1
      for (int c0 = 0; c0 < a.cols; c0 += 16) {
        float v[16];
        __syncwarp();
        tmem_ld16(acc + c0, v);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c)
          if (sh.y_at[c0 + c] >= 0) mine[(c0 + c) * kFeatures] = v[c];
      }
      released();
      __threadfence();
      meet();
      if (t == 0) sh.last[0] = (int)atomicAdd(&a.counters[it.cut], 1u) == it.segs - 1;
      meet();
      if (!sh.last[0]) continue;
      __threadfence();
#pragma unroll 1
      for (int c0 = 0; c0 < a.cols; c0 += 16) {
        float v[16] = {};
#pragma unroll 1
        for (int s = 0; s < it.segs; ++s) {
          const float* part = partial_of(a, c0_cta, s) + c0 * kFeatures + 32 * q + lane;
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (sh.y_at[c0 + c] >= 0) v[c] += __ldcg(part + c * kFeatures);
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) put(c0 + c, v[c]);
      }
    }
  } else if (kOneByte && warp >= kWarpScale) {
    // ---- exponent bytes: a thread has a row of W and up to two tokens, four units' bytes at a time ------
    const int t = threadIdx.x - 32 * kWarpScale, row_bytes = a.K / KDTV_GROUP;
    auto window = [&](const uint8_t* row, int u) -> uint4 {       // units 4 u .. 4 u + 3
      uint32_t x[4] = {0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu};
      if (row && 4 * u < a.base) {
        if (a.scale_mode == 2) return *reinterpret_cast<const uint4*>(row + 16 * u);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = 16 * u + 4 * k;
          if (a.scale_mode == 1) {
            if (at < row_bytes) x[k] = *reinterpret_cast<const uint32_t*>(row + at);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (at + e < row_bytes) x[k] = (x[k] & ~(0xffu << (8 * e))) | ((uint32_t)row[at + e] << (8 * e));
          }
        }
      }
      return make_uint4(x[0], x[1], x[2], x[3]);
    };
    auto word = [](const uint4& v, int k) { return k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w; };
    const uint32_t at = (t & 31) * 16 + (t >> 5) * 4;
    bool alive = true;
    while (alive && next(a, sh, w, it)) {
      const uint8_t* rows[3] = {nullptr, nullptr, nullptr};
      if (it.f * kFeatures + t < a.M) rows[0] = a.W_scale + (long long)(it.f * kFeatures + t) * row_bytes;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = t + 128 * h, rq = (int)divide(c, a.by_rows), r = c - rq * a.rows;
        const int b = it.g * a.requests + rq, i = it.j * a.rows + r;
        if (c < a.cols && rq < a.requests && b < a.B && i < a.N) rows[1 + h] = a.x_scale + ((long long)b * a.N + i) * row_bytes;
      }
      uint4 now[3], then[3];
#pragma unroll
      for (int r = 0; r < 3; ++r) then[r] = window(rows[r], it.k0 >> 2);
      for (int k = it.k0; k < it.k1; ++k) {
        if (k < a.base && (k == it.k0 || (k & 3) == 0))
#pragma unroll
          for (int r = 0; r < 3; ++r) {
            now[r] = then[r];
            then[r] = window(rows[r], (k >> 2) + 1);
          }
        alive = wait_warp(guard, BAR(B_EMPTY + slot), phase ^ 1u);
        if (!alive) break;
        if (k < a.base) {
          const uint32_t to = scales + slot * kScaleBytes + at;
#pragma unroll
          for (int r = 0; r < 3; ++r)
            asm volatile("st.shared.b32 [%0], %1;" :: "r"(to + 512 * r), "r"(word(now[r], k & 3)) : "memory");
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_FULL + slot));
        advance();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
int launch_groups(const ProjArgs& a) { return a.groups < kMaxGroups ? a.groups : kMaxGroups; }
int ctas_of(int sms) { return sms < kMaxCtas ? sms : kMaxCtas; }

template <bool kOneByte, int MR, int NT, int TW, int KW>
cudaError_t launch_low(const ProjArgs& a, cudaStream_t st) {
  const int tokens = 8 * NT * TW;
  const dim3 grid = a.adapter ? dim3((unsigned)((a.N + tokens - 1) / tokens), (unsigned)((a.R + 16 * MR - 1) / (16 * MR)), (unsigned)a.B)
                              : dim3(1);
  proj_low_kernel<kOneByte, MR, NT, TW, KW><<<grid, 32 * TW * KW, 0, st>>>(a);
  return cudaGetLastError();
}

template <bool kOneByte>
int launch_t(const ProjArgs& a, int sms, bool stall, cudaStream_t st) {
  constexpr uint64_t e = kOneByte ? 1 : 2;
  CUtensorMap tw, tx, tb;
  {
    const uint64_t dims[2] = {(uint64_t)a.K, (uint64_t)a.M}, strides[1] = {a.K * e};
    const uint32_t box[2] = {(uint32_t)(kUnitBytes / e), kFeatures};
    if (encode_nd(&tw, a.W, 2, dims, strides, box, (int)e, 128) != CUDA_SUCCESS) return KDTV_ERR_CUDA;
  }
  {
    const uint64_t row = (a.K * e + 15) / 16 * 16;         // strides of single rows do not matter
    const uint64_t dims[3] = {(uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.B};
    const uint64_t strides[2] = {a.N > 1 ? a.xs[1] * e : row, a.B > 1 ? a.xs[0] * e : row * a.N};
    const uint32_t box[3] = {(uint32_t)(kUnitBytes / e), (uint32_t)a.rows, (uint32_t)a.requests};
    if (encode_nd(&tx, a.x, 3, dims, strides, box, (int)e, 128) != CUDA_SUCCESS) return KDTV_ERR_CUDA;
  }
  tb = tx;
  if (a.adapter) {
    const uint64_t dims[3] = {(uint64_t)a.R, (uint64_t)a.M, (uint64_t)a.adapters};
    const uint64_t strides[2] = {(uint64_t)a.R * 2, (uint64_t)a.M * a.R * 2};
    const uint32_t box[3] = {16, kFeatures, 1};
    if (encode_nd(&tb, a.Bm, 3, dims, strides, box, 2, 32) != CUDA_SUCCESS) return KDTV_ERR_CUDA;
  }
  // Few rows of a request: one rank chunk and 16 ways along d_in a block; many: 64 rows.
  cudaError_t err;
  if (a.N <= 8 || !a.adapter) err = launch_low<kOneByte, 1, 1, 1, 16>(a, st);
  else if (a.R <= 16) err = launch_low<kOneByte, 1, 2, 4, 2>(a, st);
  else if (a.R <= 32) err = launch_low<kOneByte, 2, 2, 4, 2>(a, st);
  else err = launch_low<kOneByte, 4, 2, 4, 2>(a, st);
  if (err != cudaSuccess) return KDTV_ERR_CUDA;
  const size_t smem = (size_t)a.stages * (kWBytes + a.cols * kUnitBytes + (kOneByte ? kScaleBytes : 0)) + sizeof(ProjShared);
  const auto kern = proj_tc_kernel<kOneByte>;
  if (allow_smem(kern, smem) != cudaSuccess) return KDTV_ERR_CUDA;
  if (launch_ex(kern, dim3((unsigned)ctas_of(sms)), dim3(threads_of(kOneByte)), smem, st, true, tw, tx, tb, a, stall ? 1 : 0) !=
      cudaSuccess)
    return KDTV_ERR_CUDA;
  return KDTV_OK;
}

}  // namespace

bool proj_tc_sizes(const kdtv_project_dims* d, int sms, ProjArgs* a) {
  const bool one_byte = d->dtype == KDTV_BF16_FP8KV;
  if (d->dtype == KDTV_F32 || (d->flags & KDTV_FLAG_SIMT)) return false;
  if (!one_byte && d->d_in % 8) return false;
  if (d->adapters > 0 && d->rank % 8) return false;
  const int cap = acc_columns(one_byte);
  if (2 * d->N > cap) {                       // row blocks of one request, as even as multiples of 8 allow
    a->requests = 1;
    a->groups = d->B;
    a->blocks = (d->N + cap - 1) / cap;
    a->rows = ((d->N + a->blocks - 1) / a->blocks + 7) / 8 * 8;
    a->blocks = (d->N + a->rows - 1) / a->rows;
  } else {
    const int most = cap / d->N;
    a->groups = (d->B + most - 1) / most;
    a->requests = (d->B + a->groups - 1) / a->groups;
    a->groups = (d->B + a->requests - 1) / a->requests;
    a->blocks = 1;
    a->rows = d->N;
  }
  a->cols = (a->requests * a->rows + 15) / 16 * 16;
  a->base = (int)(((long long)d->d_in * (one_byte ? 1 : 2) + kUnitBytes - 1) / kUnitBytes);
  a->chunks = d->adapters > 0 ? (d->rank + 15) / 16 : 0;
  a->pairs = ((a->requests < d->adapters ? a->requests : d->adapters) * a->chunks + 1) / 2;
  a->features = (d->d_out + kFeatures - 1) / kFeatures;
  if ((long long)a->groups * a->blocks * a->features > 0x3fffffffll) return false;
  const int stage = kWBytes + a->cols * kUnitBytes + (one_byte ? kScaleBytes : 0);
  // As many stages as leave room for the first kernel's blocks beside this one's (up to 17 KiB).
  a->stages = (int)((225 * 1024 - 18 * 1024 - sizeof(ProjShared)) / stage);
  if (a->stages > kMaxStages) a->stages = kMaxStages;
  a->n_counters = 2 * ctas_of(sms);
  a->by_requests = divisor((unsigned)a->requests);
  a->by_rows = divisor((unsigned)a->rows);
  a->by_chunks = divisor((unsigned)(a->chunks > 0 ? a->chunks : 1));
  return true;
}

// Counters, A x, partial sums.
size_t proj_tc_workspace(const ProjArgs& a, int sms) {
  return align256((size_t)a.n_counters * 4) + align256((size_t)launch_groups(a) * a.blocks * a.pairs * proj_pair_bytes(a)) +
         (size_t)2 * ctas_of(sms) * a.cols * kFeatures * 4;
}

int proj_tc_launches(const ProjArgs& a) { return (a.groups + kMaxGroups - 1) / kMaxGroups; }

int launch_proj_tc(const ProjArgs& call, int sms, bool stall, cudaStream_t st) {
  ProjArgs a = call;
  const bool one_byte = a.dtype == KDTV_BF16_FP8KV;
  char* at = reinterpret_cast<char*>(call.low);
  a.counters = reinterpret_cast<unsigned int*>(at);
  at += align256((size_t)a.n_counters * 4);
  a.parts = at;
  at += align256((size_t)launch_groups(a) * a.blocks * a.pairs * proj_pair_bytes(a));
  a.partial = reinterpret_cast<float*>(at);
  a.scale_mode = 0;
  if (one_byte) {
    const uintptr_t both = reinterpret_cast<uintptr_t>(a.x_scale) | reinterpret_cast<uintptr_t>(a.W_scale);
    a.scale_mode = a.K % 512 == 0 && both % 16 == 0 ? 2 : a.K % 128 == 0 && both % 4 == 0 ? 1 : 0;
  }
  // As many requests at a time as the plan in shared memory has places for.
  for (long long b0 = 0; b0 < call.B; b0 += (long long)kMaxGroups * a.requests) {
    a.B = (int)(call.B - b0 < (long long)kMaxGroups * a.requests ? call.B - b0 : (long long)kMaxGroups * a.requests);
    a.groups = (a.B + a.requests - 1) / a.requests;
    a.x = static_cast<const char*>(call.x) + b0 * a.xs[0] * (one_byte ? 1 : 2);
    a.y = static_cast<__nv_bfloat16*>(call.y) + b0 * a.ys[0];
    if (one_byte) a.x_scale = call.x_scale + b0 * a.N * (a.K / KDTV_GROUP);
    if (call.adapter) a.adapter = call.adapter + b0;
    if (call.n_live) a.n_live = call.n_live + b0;
    const int rc = one_byte ? launch_t<true>(a, sms, stall, st) : launch_t<false>(a, sms, stall, st);
    if (rc != KDTV_OK) return rc;
  }
  return KDTV_OK;
}

}  // namespace kdtv
