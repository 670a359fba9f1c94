// Tensor-core (tcgen05) path of kdtv_project: bf16, or one-byte inputs and
// weights with an exponent byte per 32 elements.
//
// Mathematics.  y = W x + Bm_a (s_a A_a x), a the request's adapter.  Outputs are
// the rows (TMEM lanes) of a product, tokens its columns: D[f, t] = sum_k W[f, k]
// x[t, k], so that one token costs a 32-column product, not a 256-row one.  The
// adapters are more of the same sum: with the adapters of a tile's requests
// side by side, [W | Bm_0 | Bm_1 ..] [x ; v_0 ; v_1 ..], where v_a = s_a A_a x for the
// tokens of adapter a and 0 for the others.  v is fp32, split into two bf16 parts
// (16 significant bits), each multiplied with Bm.  0 * infinity must not carry
// one adapter's values into another's tokens, and infinity times a part that is 0 or
// of the other sign is not infinity times v: an output that is not finite, in a
// tile with adapters, is computed again on its own.
//
// Kernels: one of kdtv_proj_low.cu (v of all tokens, in the tiles' order, as the
// second kernel's operands lie in shared memory), proj_tc_kernel (everything else),
// launched while the first runs, of which only the adapters' units wait for it, and
// proj_combine_kernel for tiles that were cut.
//
// Work.  A unit is 128 bytes of d_in (64 bf16, 128 one-byte elements) or two
// chunks of 16 ranks, for one tile of 256 outputs and up to 256 tokens.  A pair of
// CTAs works on a tile: each has 128 outputs, loads those rows of W and half of the
// tokens, and the products read both halves (cta_group::2), so that a unit costs
// each SM 32 KiB where a CTA by itself with as many products would load 48 (prompts
// 595 us with single CTAs, 403 with pairs and whole tiles first).  Whole tiles go
// round the pairs; what does not fill a round is cut evenly by units, where that is
// sooner done.  A tile that several pairs share: each leaves its sums, and
// proj_combine_kernel adds them in the order of the units.
//
// Bound by the tensor cores for prompts (4 x up to 2000 rows, 4096 x 12288, rank 64:
// 364 us, 1620 TFLOP/s; one byte, 8192 rows, 8192 x 8192: 410 us, 2690), by
// DRAM and some 12 us of ways in and out for few tokens (one, 8192 x 10240: 38.8 us;
// twice the outputs 64, four times 111).  Of those 12: 2.5 to plan, 1 to the first
// load and 1 until it is there, 1.5 to write, 3 to join, the rest launches; code that
// runs once comes from a cold cache, so what every call passes through is kept short.
//
// One byte: exponent bytes travel as they are to the tensor cores, which take
// one per 32 elements and operand row (block-scaled products), so sums are in true
// units and the adapters' bf16 products add to them.  They read them from TMEM, a
// row's four bytes of a unit a word, rows 32 j + l in lane l of column j, the same in
// each quarter of the lanes: four warps bring them there, and a unit is complete
// when its operands have landed and both CTAs' exponents are in place.
// (Copies from shared memory by the tensor cores' own pipe, tcgen05.cp, kept it from
// multiplying for 20 % of the time.)

#include <cuda.h>

#include "kdtv_proj_tc.cuh"
#include "kdtv_tmap.cuh"

#include <string.h>

namespace kdtv {
namespace {

using namespace ptx;

constexpr int kFeatures = 128;             // outputs of a CTA: half of a tile
constexpr int kWBytes = kFeatures * kUnitBytes;
constexpr int kMaxStages = 12;
constexpr int kMaxGroups = 512;            // groups of requests in a launch
constexpr int kMaxPairs = 128;
constexpr int kScaleBytes = 3 * 512;       // a unit's exponent bytes: W, tokens 0 - 127, the others
constexpr int kWindow = 4;                 // units whose exponent bytes are loaded together (16 bytes of a row)
constexpr int kScaleColumns = 12;          // a unit's exponents in TMEM: W's, tokens 0 - 127, the others
constexpr int kSuper = 8;                  // token tiles that share a W tile in a row

// ---- the projection --------------------------------------------------------------------------
enum {
  B_FULL = 0, B_EMPTY = B_FULL + kMaxStages, B_ACC_FULL = B_EMPTY + kMaxStages, B_ACC_EMPTY = B_ACC_FULL + 2,
  B_ACC_PART = B_ACC_EMPTY + 2,                // one byte: the shared columns are read
  B_DONE = B_ACC_PART + 2, B_STALL, B_COUNT
};

// Arrivals of a barrier's phase.
__device__ __forceinline__ uint32_t arrivals(bool one_byte, int i) {
  if (i < B_EMPTY) return one_byte ? 10 : 2;                // both CTAs' producers, and their four warps
  return i >= B_ACC_EMPTY && i < B_DONE ? 8 : 1;            // both CTAs' four warps
}

constexpr int kWarpTma = 0, kWarpMma = 1, kWarpOut = 4, kWarpScale = 8;   // (2, 3: planning only)
__host__ __device__ constexpr int threads_of(bool one_byte) { return one_byte ? 384 : 256; }
// Two accumulators of 256 columns take turns.  One byte: the exponents need 72 of TMEM's 512 columns, so those of
// more than 128 columns share kShared of theirs (the first one's last are the second one's first).  They are read first and
// given back at once, so that the next tile's products wait for that only.  (Tiles of 192 tokens without sharing: 435
// us where 256 take 328, both without exponents, for 8192 tokens, 8192 x 8192.)
constexpr int kTokens = 256, kShared = 80;
__device__ __forceinline__ uint32_t acc_at(const ProjArgs& a, int n) { return (n & 1) * (kTokens - a.shared); }
// The exponents of a ring entry: behind the accumulators, or, where those have 128 columns, between them and behind.
__device__ __forceinline__ uint32_t scale_at(const ProjArgs& a, int slot) {
  return a.shared ? 2 * kTokens - kShared + slot * kScaleColumns : (slot & 1) * kTokens + kTokens / 2 + (slot >> 1) * kScaleColumns;
}

constexpr int kRowPitch = 80;               // 64 bytes, set apart so that eight rows' 16 bytes lie in different banks

// Shared memory behind the ring.
struct ProjShared {
  uint64_t bars[B_COUNT];
  uint32_t tmem, abort;
  int total_tiles, cut, share, pad;         // token tiles times outputs' tiles; cut tiles; units of a pair's share
  int first[kMaxGroups + 1];                // token tiles before each group
  uint32_t tile[kMaxGroups];                // 16-rank chunks of its tiles' adapters, and 2^20 rows of half a block
  int start[kMaxPairs + 1];              // units before each cut tile
  long long y_at[256];                      // offset of each column's output row, -1: none
  uint32_t bits[kWords];
  uint16_t ids[256];                        // the adapters of the producer's tile
  __align__(16) unsigned char rows[4][16 * kRowPitch];   // an output warp's 32 outputs of 16 tokens
};

// A part of a tile: units k0 .. k1 - 1; behind a.base of d_in come pairs of chunks.
struct Item {
  int g, j, f, k0, k1, chunks, hr;
  int cut, seg, segs;                       // cut tile's number (-1: whole), place among its segments
};

// The items of pair c, in the order in which every role sees them: whole tiles, then its share of the cut
// ones from its end on: tiles begin with d_in, and the first kernel has until their adapters' units come.
struct Walk {
  int tile, u0, u, s;                       // next whole tile; start and end of what is left of the share, its last tile
};

// Tiles of few units are not cut.
__host__ __device__ __forceinline__ bool may_cut(const ProjArgs& a) { return a.base >= 16; }
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
  it.chunks = (int)(sh.tile[lo] & 0xfffffu);
  it.hr = (int)(sh.tile[lo] >> 20);
}

__device__ __forceinline__ Walk walk(const ProjShared& sh) {
  Walk w;
  const int pair = blockIdx.x >> 1, all = sh.cut ? sh.start[sh.cut] : 0;
  w.tile = sh.cut + pair;
  w.u0 = min(all, pair * sh.share);
  w.u = min(all, w.u0 + sh.share);
  int lo = 0, hi = sh.cut - 1;              // the last tile that starts before w.u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sh.start[mid] < w.u) lo = mid;
    else hi = mid - 1;
  }
  w.s = lo;
  return w;
}

__device__ __forceinline__ bool next(const ProjArgs& a, const ProjShared& sh, Walk& w, Item& it) {
  if (w.tile < sh.total_tiles) {
    locate(a, sh, w.tile, it);
    it.k0 = 0;
    it.k1 = units_of(a, it.chunks);
    it.cut = -1;
    it.seg = 0;
    it.segs = 1;
    w.tile += gridDim.x >> 1;
    return true;
  }
  if (w.u <= w.u0) return false;
  locate(a, sh, w.s, it);
  const int start = sh.start[w.s], end = sh.start[w.s + 1], from = max(start, w.u0), c0 = start / sh.share;
  it.k0 = from - start;
  it.k1 = w.u - start;
  it.segs = (end - 1) / sh.share - c0 + 1;
  it.seg = (int)(blockIdx.x >> 1) - c0;
  it.cut = it.segs > 1 ? w.s : -1;
  w.u = from;
  --w.s;
  return true;
}

// Pair c's sums of segment `seg` of a cut tile, those of CTA `rank`: a pair has two places, one for the tile
// that its share begins in.
__device__ __forceinline__ float* partial_of(const ProjArgs& a, int c, int seg, int rank) {
  return a.partial + ((2ll * c + (seg == 0 ? 1 : 0)) * 2 + rank) * (2 * a.half_cols) * kFeatures;
}

// What the combine kernel needs to know of a cut tile; a.plan holds their number, then these.
struct __align__(16) CutTile {
  int first, segs, g, j;                    // pair of the first segment (segs 1: whole, nothing to do)
  int f, chunks, hr, pad;
};
__device__ __forceinline__ void leave_plan(const ProjArgs& a, const ProjShared& sh, int t) {
  if (t == 0) a.plan[0] = sh.cut;
  CutTile* out = reinterpret_cast<CutTile*>(a.plan + 4);
  for (int s = t; s < sh.cut; s += 128) {
    Item it;
    locate(a, sh, s, it);
    const int first = sh.start[s] / sh.share;
    out[s] = CutTile{first, (sh.start[s + 1] - 1) / sh.share - first + 1, it.g, it.j, it.f, it.chunks, it.hr, 0};
  }
}

// D[tmem] (+)= A[smem desc] * B[smem desc]^T of E4M3 elements with an exponent
// byte per 32 of each row (in TMEM), 32 elements deep, fp32 accumulation.
__device__ __forceinline__ void mma_scaled(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t a_scale, uint32_t b_scale, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\t"
               "setp.ne.b32 p, %6, 0;\n\t"
               "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
               :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
               : "memory");
}
// E4M3 A and B, exponent bytes as scales; bits 4 and 29 on: which byte of a word.
__device__ __forceinline__ uint32_t idesc_scaled(int N, int byte) {
  return ((uint32_t)byte << 4) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(2 * kFeatures >> 4) << 24) |
         ((uint32_t)byte << 29);
}
// Words of a lane, one a column.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint4& v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};"
               :: "r"(taddr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint4& v, const uint4& w) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "r"(taddr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Four warps meet at named barrier `id`: whether all of them say so.
__device__ __forceinline__ bool all_of(int id, bool ok) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
               "bar.red.and.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r) : "r"((uint32_t)ok), "r"(id) : "memory");
  return r != 0u;
}

// Sixteen exponent bytes of a row that is not 16-byte aligned.  (By itself: nine copies of it made the first loads, whose
// code comes from a cold cache, us later.)
__device__ __noinline__ uint4 exponent_window(const uint8_t* row, int at, int bytes, const uint8_t* end, int mode) {
  uint32_t x[4] = {0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu};
  if (mode == 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at + 4 * k < bytes) x[k] = *reinterpret_cast<const uint32_t*>(row + at + 4 * k);
  } else {
    exponent_words(row, at, bytes, end, x);
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// 16 tokens' 32 outputs from shared memory, an output a lane: rows of y that are not 16-byte aligned; whether one of the
// lane's is not finite.  (By itself, so that the aligned rows' code stays short: inlined it cost 64 drafts of 8 two us of 52.)
__device__ __noinline__ bool write_narrow(uint32_t rows, const long long* y_at, unsigned short* y, bool on) {
  const int lane = threadIdx.x & 31;
  bool odd = false;
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(rows + c * kRowPitch + lane * 2) : "memory");
    const long long to = y_at[c];
    if (on && to >= 0) {
      y[to + lane] = v;
      odd |= (v & 0x7f80u) == 0x7f80u;
    }
  }
  return odd;
}

// Whether request b's row of Bm for output f has an infinity: in a tile of one request a NaN of that output may have been
// made by the two parts of v.
__device__ __noinline__ bool infinite_row(const ProjArgs& a, int b, int f) {
  const uint4* row = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.Bm) + ((long long)a.adapter[b] * a.M + f) * a.R);
  bool found = false;
  for (int r = 0; r < a.R / 8; ++r) {          // (the rank is a multiple of 8, and Bm is 16-byte aligned)
    const uint4 w = row[r];
    for (uint32_t two : {w.x, w.y, w.z, w.w}) found |= (two & 0x7fffu) == 0x7f80u || (two & 0x7fff0000u) == 0x7f800000u;
  }
  return found;
}

// One output by itself, for a value that is not finite in a tile with adapters.  Slow (a thread's loop over d_in and the
// tile's requests), so a tile of one request takes it for a NaN beside an infinity in Bm only, not for rows of x that
// are NaN.
template <bool kOneByte>
__device__ __noinline__ float alone(const ProjArgs& a, int b, int i, int f) {
  constexpr int E = kOneByte ? 1 : 2;
  const char* x = static_cast<const char*>(a.x) + (b * a.xs[0] + i * a.xs[1]) * E;
  const char* w = static_cast<const char*>(a.W) + (long long)f * a.K * E;
  float sum = 0.f;
#pragma unroll 4
  for (int k = 0; k < a.K; k += 8) {         // (d_in is a multiple of 8, and rows are 16-byte aligned)
    float u[8], v[8], scale = 1.f;
    if constexpr (kOneByte) {
      const int groups = a.K / KDTV_GROUP;
      const uint2 p = *reinterpret_cast<const uint2*>(x + k), q = *reinterpret_cast<const uint2*>(w + k);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 y = widen2(((e < 2 ? p.x : p.y) >> (16 * (e & 1))) & 0xffffu);
        const float2 z = widen2(((e < 2 ? q.x : q.y) >> (16 * (e & 1))) & 0xffffu);
        u[2 * e] = y.x;
        u[2 * e + 1] = y.y;
        v[2 * e] = z.x;
        v[2 * e + 1] = z.y;
      }
      scale = scale_of_byte(a.x_scale[((long long)b * a.N + i) * groups + k / KDTV_GROUP]);
      const float scale_w = scale_of_byte(a.W_scale[(long long)f * groups + k / KDTV_GROUP]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= scale_w;
    } else {
      load_v<8>(reinterpret_cast<const __nv_bfloat16*>(x) + k, u);
      load_v<8>(reinterpret_cast<const __nv_bfloat16*>(w) + k, v);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(u[e] * scale, v[e], sum);
  }
  const int id = a.adapter[b];
  if (id < 0) return sum;
  // this request's v, from its place among the tile's adapters
  const int g = (int)divide(b, a.by_requests);
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
    int flip;
    const char* hi = part_row(a, b, i, half_rows_of(a, live_rows(a.n_live, b, a.N)), c, 0, &flip);
    hi += (((r >> 3) & 1) ^ flip) * 16 + (r & 7) * 2;
    const float v = to_f32(*reinterpret_cast<const __nv_bfloat16*>(hi)) +
                    to_f32(*reinterpret_cast<const __nv_bfloat16*>(hi + (long long)a.half_cols * 32));
    sum = fmaf(v, to_f32(static_cast<const __nv_bfloat16*>(a.Bm)[((long long)id * a.M + f) * a.R + r]), sum);
  }
  return sum;
}

// A tile with adapters in which something is not finite, once it is written: such outputs of a warp's 32, from f0 on, an
// output a lane, are computed by themselves where they may be wrong.  All of the warp comes along.
template <bool kOneByte>
__device__ __noinline__ void look_again(const ProjArgs& a, const long long* y_at, int g, int j, int hr, int f0, int cols) {
  const int f = f0 + (threadIdx.x & 31);
  __syncwarp();                                // (the other lanes' stores)
  if (f < a.M && (a.requests > 1 || infinite_row(a, g, f))) {
#pragma unroll 1
    for (int c = 0; c < cols; ++c) {
      const long long to = y_at[c];
      if (to < 0) continue;
      __nv_bfloat16* const y = static_cast<__nv_bfloat16*>(a.y) + to + f;
      const float x = __bfloat162float(*y);
      if (a.requests > 1 ? fabsf(x) < INFINITY : x == x) continue;
      int b, i;
      column(a, g, j, hr, c, &b, &i);
      *y = __float2bfloat16_rn(alone<kOneByte>(a, b, i, f));
    }
  }
  __syncwarp();
}

// (Registers that leave room for a block of the first kernel beside this one's.)
template <bool kOneByte>
__global__ void __maxnreg__(kOneByte ? 112 : 128)
proj_tc_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
               const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ ProjArgs a, int stall) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stage_bytes = kWBytes + a.half_cols * kUnitBytes;
  const uint32_t rank = cluster_ctarank();
  ProjShared& sh = *reinterpret_cast<ProjShared*>(smem + (size_t)a.stages * stage_bytes + (kOneByte ? 2 * kWindow * kScaleBytes : 0));
  const uint32_t ring = smem_u32(smem), scales = ring + a.stages * stage_bytes, bars = smem_u32(sh.bars);
  auto BAR = [&](int i) { return bars + 8u * i; };
  const Guard guard{&sh.abort, a.status, stall ? 20000000u : 2000000000u};
  grid_dep_launch();                           // the combine kernel may be launched; it waits for this grid

  // ---- set up, and plan: every CTA derives the same tiles from n_live and adapter ------------------
  if (threadIdx.x < B_COUNT) {
    const int i = threadIdx.x;
    mbar_init(BAR(i), arrivals(kOneByte, i));
  }
  if (threadIdx.x == 0) sh.abort = 0u;
  fence_mbar_init();
  __syncthreads();
  cluster_arrive();                            // this CTA's barriers are set up
  if (warp == kWarpTma && lane == 0) {
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_x);
    if (a.adapter) {
      prefetch_tmap(&tm_b);
      prefetch_tmap(&tm_v);
    }
  }
  if (a.requests == 1) {
    for (int g = threadIdx.x; g < a.groups; g += threads_of(kOneByte)) {
      const int n = live_rows(a.n_live, g, a.N), raw = a.adapter ? a.adapter[g] : -1;   // (both loads under way)
      const int id = n > 0 ? proj_adapter(a, raw) : -1;
      const int hr = half_rows_of(a, n);
      sh.first[g] = id == -2 ? 0 : (n + 2 * hr - 1) / (2 * hr);
      sh.tile[g] = (id >= 0 ? (uint32_t)a.chunks : 0u) | ((uint32_t)hr << 20);
    }
  } else {
    uint32_t* bits = reinterpret_cast<uint32_t*>(smem) + warp * kWords;     // (the ring is not in use yet)
    for (int g = warp; g < a.groups; g += threads_of(kOneByte) / 32) {
      bool live;
      const int slots = group_bitmap(a, g, bits, &live);
      __syncwarp();
      if (lane == 0) {
        sh.first[g] = live ? 1 : 0;
        sh.tile[g] = (uint32_t)(slots * a.chunks) | ((uint32_t)a.N << 20);
      }
    }
    fence_async_smem();
  }
  __syncthreads();
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
    // Whole rounds of whole tiles, and what is left cut into equal shares, where that is sooner done than whole
    // tiles that leave pairs idle.
    const int tiles = sum * a.features, pairs = gridDim.x >> 1;
    int cut = tiles % pairs;
    // (In ns, as measured: a unit takes 300, joining cut tiles 4000 and what reading their sums takes at 3500 GB/s.)
    if (may_cut(a) && cut > 0) {
      const long long idle = (long long)(pairs - cut) * 300 * a.base / pairs;
      const long long join = 4000 + (long long)(pairs + cut) * 2 * a.half_cols * (2 * kFeatures * 4) / 3500;
      if (idle < join) cut = 0;
    } else {
      cut = 0;
    }
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
      sh.share = max(8, (u + pairs - 1) / pairs);
    }
  }
  __syncthreads();
  cluster_wait();                              // the pair's barriers are set up
  // TMEM, for all but the producer, which is at work meanwhile.
  uint32_t tmem = 0u;
  if (warp != kWarpTma) {
    if (warp == kWarpMma) {
      tmem_alloc_pair(smem_u32(&sh.tmem), 512);
      tmem_relinquish_pair();
    }
    tc_fence_before();
    asm volatile("bar.sync 3, %0;" :: "n"(threads_of(kOneByte) - 32) : "memory");
    tc_fence_after();
    tmem = sh.tmem;
  }
  const uint32_t lead = mapa(bars, 0);         // the first CTA's barriers: it issues the products
  auto LEAD = [&](int i) { return lead + 8u * i; };
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
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        const int first = min(min(it.k1, max(it.k0, a.base)), it.k0 + a.stages);
        const int from = part ? first : it.k0, to = part ? it.k1 : first;
        if (from >= to) continue;
        if (part && it.k1 > a.base) {          // the tile's adapters, while a ring full of d_in is on its way
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
        if (lane == 0)
          for (int k = from; alive && k < to; ++k) {
            alive = wait_poll(guard, BAR(B_EMPTY + slot), phase ^ 1u);
            if (!alive) break;
            const uint32_t full = LEAD(B_FULL + slot), dst = ring + slot * stage_bytes;
            const int f = (2 * it.f + rank) * kFeatures;
            if (k < a.base) {
              mbar_expect_tx_cluster(full, kWBytes + a.half_requests * a.half_rows * kUnitBytes);
              tma_load_2d_pair(dst, &tm_w, full, k * (kOneByte ? 128 : 64), f);
              tma_load_3d_pair(dst + kWBytes, &tm_x, full, k * (kOneByte ? 128 : 64), a.by_rows_of ? (2 * it.j + rank) * it.hr : 0,
                               it.g * a.requests + (a.by_rows_of ? 0 : rank * a.half_requests));
            } else {
              if (!waited) grid_dep_wait();      // v is written
              waited = true;
              const int p = k - a.base, two = min(2, it.chunks - 2 * p);
              mbar_expect_tx_cluster(full, two * (kFeatures * 32) + a.half_cols * 128);
              for (int c = 2 * p; c < 2 * p + two; ++c) {
                const int s = (int)divide(c, a.by_chunks);
                tma_load_3d_pair(dst + (c & 1) * (kFeatures * 32), &tm_b, full, (c - s * a.chunks) * 16, f, sh.ids[s]);
              }
              tma_load_2d_pair(dst + kWBytes, &tm_v, full, 0,
                               (int)((((long long)(it.g * a.blocks + it.j) * a.pairs + p) * 2 + rank) * (a.half_cols / 2)));
            }
            advance();
            ++loads;
          }
        __syncwarp();
      }
      alive = __shfl_sync(0xffffffffu, (int)alive, 0) != 0;
    }
    if (lane == 0)                             // every copy has landed, and is used up
      for (int x = loads > a.stages ? loads - a.stages : 0; x < loads; ++x)
        drain(guard, BAR(B_EMPTY + x % a.stages), (x / a.stages) & 1);
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ---- products ------------------------------------------------------------------------------
    if (lane == 0 && rank == 0) {
      bool alive = true;
      for (int n = 0; alive && next(a, sh, w, it); ++n) {
        const uint32_t d = tmem + acc_at(a, n);
        alive = wait(guard, BAR(B_ACC_EMPTY + (n & 1)), ((n >> 1) & 1) ^ 1u) &&
                (!kOneByte || n == 0 || wait_poll(guard, BAR(B_ACC_PART + ((n - 1) & 1)), ((n - 1) >> 1) & 1));
        tc_fence_after();
        const int cols = 2 * half_cols_of(a, it.hr);
        const uint32_t idesc = idesc_bf16(2 * kFeatures, cols, 0, 0);
        uint32_t acc = 0u;
        for (int k = it.k0; alive && k < it.k1; ++k) {
          alive = wait_poll(guard, BAR(B_FULL + slot), phase);
          if (!alive) break;
          tc_fence_after();
          const uint32_t at = ring + slot * stage_bytes;
          if (k < a.base) {
            const uint64_t ad = smem_desc(at, 16, 1024), bd = smem_desc(at + kWBytes, 16, 1024);
            if constexpr (kOneByte) {
              const uint32_t sc = tmem + scale_at(a, slot);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                mma_scaled(d, ad + 2 * kk, bd + 2 * kk, idesc_scaled(cols, kk), sc, sc + 4, acc);
                acc = 1u;
              }
            } else {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                mma_bf16_pair(d, ad + 2 * kk, bd + 2 * kk, idesc, acc);
                acc = 1u;
              }
            }
          } else {
            const int two = min(2, it.chunks - 2 * (k - a.base));
            for (int c = 0; c < two; ++c)
              for (int p = 0; p < 2; ++p) {
                mma_bf16_pair(d, smem_desc_sw32(at + c * (kFeatures * 32)),
                              smem_desc_sw32(at + kWBytes + (c * 2 + p) * a.half_cols * 32), idesc, acc);
                acc = 1u;
              }
          }
          mma_commit_pair(BAR(B_EMPTY + slot), 3);
          advance();
        }
        if (alive) mma_commit_pair(BAR(B_ACC_FULL + (n & 1)), 3);
      }
      mma_commit_pair(BAR(B_DONE), 1);         // every product has finished before TMEM is freed
      drain(guard, BAR(B_DONE), 0);
    }
    __syncwarp();
  } else if (warp >= kWarpOut && warp < kWarpOut + 4) {
    // ---- sums to outputs: warp q has TMEM lanes 32 q .., one output each -------------------------------
    const int q = warp - kWarpOut, t = threadIdx.x - 32 * kWarpOut;
    auto meet = [&]() { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    auto agree = [&](bool ok) { return all_of(1, ok); };
    if (blockIdx.x == 0) leave_plan(a, sh, t);
    for (int n = 0; next(a, sh, w, it); ++n) {
      meet();                                  // the last tile's columns are read
      const int cols = 2 * half_cols_of(a, it.hr);
      for (int c = t; c < cols; c += 128) {
        int b, i;
        long long at = -1;
        if (column(a, it.g, it.j, it.hr, c, &b, &i) && i < live_rows(a.n_live, b, a.N)) {
          const int id = a.adapter ? a.adapter[b] : -1;
          if (id >= -1 && id < a.adapters) at = b * a.ys[0] + i * a.ys[1];
        }
        sh.y_at[c] = at;
      }
      if (!agree(wait_warp(guard, BAR(B_ACC_FULL + (n & 1)), (n >> 1) & 1))) break;
      tc_fence_after();
      const uint32_t acc = tmem + acc_at(a, n) + ((uint32_t)(32 * q) << 16);
      const int f0 = (2 * it.f + rank) * kFeatures + 32 * q;
      const bool adapted = it.chunks > 0;
      auto released = [&](int bar) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(LEAD(bar + (n & 1)));
      };
      // Columns that the next tile's accumulator has too come first, then the others.
      const int first0 = (n & 1) ? 0 : min(cols, kTokens - a.shared), first1 = (n & 1) ? min(cols, a.shared) : cols;
      const int rest0 = first0 == 0 ? first1 : 0, rest1 = first0 == 0 ? cols : first0;
      if (it.cut >= 0) {                       // sums, for the combine kernel: an output a lane
        float* mine = partial_of(a, (int)(blockIdx.x >> 1), it.seg, rank) + 32 * q + lane;
        auto copy = [&](int c0, int c1) {
#pragma unroll 1
          for (; c0 < c1; c0 += 16) {
            float v[16];
            __syncwarp();
            tmem_ld16(acc + c0, v);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) mine[(c0 + c) * kFeatures] = v[c];
          }
        };
        copy(first0, first1);
        if (kOneByte) released(B_ACC_PART);
        copy(rest0, rest1);
        released(B_ACC_EMPTY);
        continue;
      }
      // 16 columns as the products of 8 x 8 matrices hold them: value (k, h, j, e) is output f0 + 16 h + 8 j + lane /
      // 4 of token c0 + 8 k + 2 (lane % 4) + e; p: pairs over e, rounded.
      auto fetch = [&](int c0, uint32_t (&p)[2][4]) {
        float v[2][8];                         // [h][4 k + 2 j + e]
        __syncwarp();
        tmem_ld_16x256b_x2(acc + c0, v[0]);
        tmem_ld_16x256b_x2(acc + (16u << 16) + c0, v[1]);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int m = 0; m < 4; ++m) p[k][m] = pack_bf16x2(v[m >> 1][4 * k + 2 * (m & 1)], v[m >> 1][4 * k + 2 * (m & 1) + 1]);
      };
      // To shared memory, transposed, and from there 8 outputs of a token a lane.
      const uint32_t rows = smem_u32(sh.rows[q]);
      uint32_t zero = 0u;                      // 0 times all that is written, in pairs: NaN where one is not finite
      auto write = [&](int c0, const uint32_t (&p)[2][4]) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 2; ++k)
          stmatrix_x4_trans(rows + (8 * k + (lane & 7)) * kRowPitch + (lane >> 3) * 16, p[k][0], p[k][1], p[k][2], p[k][3]);
        __syncwarp();
        if (!a.wide) {
          if (write_narrow(rows, sh.y_at + c0, static_cast<unsigned short*>(a.y) + f0, f0 + lane < a.M)) zero = 0x7fffu;
          return;
        }
        const int f = f0 + (lane & 3) * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = h * 8 + (lane >> 2);
          const long long to = sh.y_at[c0 + c];
          const uint4 v = lds128(rows + c * kRowPitch + (lane & 3) * 16);
          if (to >= 0 && f < a.M) {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.y) + to + f) = v;
            for (uint32_t two : {v.x, v.y, v.z, v.w}) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(zero) : "r"(two), "r"(0u));
          }
        }
      };
      // One byte, another tile behind this one: the shared columns are read and rounded, then given back, then written.
      // (Where none is, one copy of the code for all columns: it runs once, from a cold cache; 64 drafts of 8: 3.3 us.)
      const bool more = w.tile < sh.total_tiles || w.u > w.u0;
      if (kOneByte && more) {
        uint32_t p[kShared / 16][2][4];
#pragma unroll
        for (int k = 0; k < kShared / 16; ++k)
          if (first0 + 16 * k < first1) fetch(first0 + 16 * k, p[k]);
        released(B_ACC_PART);
#pragma unroll
        for (int k = 0; k < kShared / 16; ++k)
          if (first0 + 16 * k < first1) write(first0 + 16 * k, p[k]);
      }
#pragma unroll 1
      for (int c0 = more ? rest0 : 0; c0 < (more ? rest1 : cols); c0 += 16) {
        uint32_t p[2][4];
        fetch(c0, p);
        write(c0, p);
      }
      released(B_ACC_EMPTY);
      if (adapted && __any_sync(0xffffffffu, (zero & 0x7fff7fffu) != 0u)) look_again<kOneByte>(a, sh.y_at, it.g, it.j, it.hr, f0, cols);
    }
    grid_dep_wait();                           // no CTA ends before the first kernel
  } else if (kOneByte && warp >= kWarpScale) {
    // ---- exponent bytes: a thread has a row of W and up to two tokens, four units' bytes at a time ------
    const int t = threadIdx.x - 32 * kWarpScale, row_bytes = a.K / KDTV_GROUP;
    const uint8_t* const x_end = a.x_scale + (long long)a.B * a.N * row_bytes;
    const uint8_t* const w_end = a.W_scale + (long long)a.M * row_bytes;
    auto bytes = [&](const uint8_t* row, int u, const uint8_t* end) -> uint4 {      // of window u
      if (!row || 4 * u >= a.base) return make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
      if (a.scale_mode == 2) return *reinterpret_cast<const uint4*>(row + 16 * u);
      return exponent_window(row, 16 * u, row_bytes, end, a.scale_mode);
    };
    auto sts32 = [](uint32_t to, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" :: "r"(to), "r"(v) : "memory"); };
    const uint32_t at = (t & 31) * 16 + (t >> 5) * 4;
    // (all four warps go on, or none: they meet)
    auto agree = [&](bool ok) { return all_of(2, ok); };
    bool alive = true;
    int staged = 0;
    uint32_t stage = scales;
    while (agree(alive) && next(a, sh, w, it)) {
      const int cols = 2 * half_cols_of(a, it.hr);
      const uint8_t* rows[3] = {nullptr, nullptr, nullptr};
      if ((2 * it.f + (int)rank) * kFeatures + t < a.M) rows[0] = a.W_scale + (long long)((2 * it.f + rank) * kFeatures + t) * row_bytes;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int b, i;
        if (t + 128 * h < cols && column(a, it.g, it.j, it.hr, t + 128 * h, &b, &i))
          rows[1 + h] = a.x_scale + ((long long)b * a.N + i) * row_bytes;
      }
      uint4 now[3], soon[3], later[3];         // two windows ahead: they come from DRAM
#pragma unroll
      for (int r = 0; r < 3; ++r) {
        soon[r] = bytes(rows[r], it.k0 / kWindow, r ? x_end : w_end);
        later[r] = bytes(rows[r], it.k0 / kWindow + 1, r ? x_end : w_end);
      }
      for (int k = it.k0; k < it.k1; ++k) {
        if (k < a.base && (k == it.k0 || k % kWindow == 0)) {
#pragma unroll
          for (int r = 0; r < 3; ++r) {
            now[r] = soon[r];
            soon[r] = later[r];
            later[r] = bytes(rows[r], k / kWindow + 2, r ? x_end : w_end);
          }
          // (The next window is staged beside this one; the one after it when all four warps are past the next
          // meeting.)
          stage = scales + (staged++ & 1) * (kWindow * kScaleBytes);
#pragma unroll
          for (int r = 0; r < 3; ++r) {
            sts32(stage + at + 512 * r, now[r].x);
            sts32(stage + at + 512 * r + kScaleBytes, now[r].y);
            sts32(stage + at + 512 * r + 2 * kScaleBytes, now[r].z);
            sts32(stage + at + 512 * r + 3 * kScaleBytes, now[r].w);
          }
          if (!agree(alive)) break;
        }
        // W's words, those of tokens 0 - 127, of the others: at hand when their place is free.
        const uint32_t from = stage + (k % kWindow) * kScaleBytes + lane * 16;
        const uint4 w0 = lds128(from), w1 = lds128(from + 512), w2 = lds128(from + 1024);
        alive = alive && wait_warp(guard, BAR(B_EMPTY + slot), phase ^ 1u);
        if (!alive) continue;                  // (until the next meeting)
        if (k < a.base) {
          tc_fence_after();
          const uint32_t to = tmem + ((uint32_t)((warp & 3) * 32) << 16) + scale_at(a, slot);
          tmem_st8(to, w0, w1);
          if (cols > 128) tmem_st4(to + 8, w2);
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(LEAD(B_FULL + slot));
        advance();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                              // neither CTA arrives at the other's barriers any more
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc_pair(tmem, 512);
}

// ---- outputs of cut tiles ---------------------------------------------------------------------
// A warp has kCombineCols tokens of a tile and 128 outputs, four of a token a lane; the sums of kAtOnce segments
// of all of them are under way together.  Latency bound: the plan, the tile's record, then everything else at once.
// (The last pair to come adding the sums up by itself, with four warps, took 32 us of 53 for 64 tokens; blocks
// of 128 outputs and 16 tokens each, those of tiles that are not there among them, 14 us of 61 for 64 drafts of 8.)
constexpr int kCombineCols = 2, kAtOnce = 4, kCombineWarps = 8;

template <bool kOneByte>
__global__ void __launch_bounds__(32 * kCombineWarps) proj_combine_kernel(const __grid_constant__ ProjArgs a) {
  const int lane = threadIdx.x & 31, per_tile = 2 * (2 * a.half_cols / kCombineCols);
  grid_dep_wait();
  int item = blockIdx.x * kCombineWarps + (threadIdx.x >> 5);
  const unsigned int status = *reinterpret_cast<volatile unsigned int*>(a.status);
  const int items = a.plan[0] * per_tile;
  // (the first record at the same time: its place is there, if not the tile, since the grid covers no more of them)
  const CutTile* records = reinterpret_cast<const CutTile*>(a.plan + 4);
  CutTile it = records[item / per_tile];
  // (a wait that ran out: some sums were never written)
  if (status == KDTV_ERR_DEVICE_TIMEOUT) return;
  for (bool first = true; item < items; item += gridDim.x * kCombineWarps, first = false) {
    const int tile = item / per_tile, r = item - tile * per_tile, rank = r & 1, c0 = (r >> 1) * kCombineCols;
    if (!first) it = records[tile];
    if (it.segs < 2 || c0 >= 2 * half_cols_of(a, it.hr)) continue;
    long long at[kCombineCols];                // offset of each token's output row, -1: none
    int b[kCombineCols], i[kCombineCols];
    bool any = false;
#pragma unroll
    for (int c = 0; c < kCombineCols; ++c) {
      at[c] = -1;
      if (!column(a, it.g, it.j, it.hr, c0 + c, &b[c], &i[c])) continue;
      any = true;
      const int n = live_rows(a.n_live, b[c], a.N), id = a.adapter ? a.adapter[b[c]] : -1;
      if (i[c] < n && id >= -1 && id < a.adapters) at[c] = b[c] * a.ys[0] + i[c] * a.ys[1];
    }
    if (!any) continue;
    float4 sum[kCombineCols] = {};
#pragma unroll 1
    for (int s0 = 0; s0 < it.segs; s0 += kAtOnce) {
      float4 v[kAtOnce][kCombineCols];
#pragma unroll
      for (int s = 0; s < kAtOnce; ++s) {
        const float* part = partial_of(a, it.first + s0 + s, s0 + s, rank) + c0 * kFeatures + 4 * lane;
#pragma unroll
        for (int c = 0; c < kCombineCols; ++c)
          v[s][c] = s0 + s < it.segs ? *reinterpret_cast<const float4*>(part + c * kFeatures) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int s = 0; s < kAtOnce; ++s)
#pragma unroll
        for (int c = 0; c < kCombineCols; ++c) {
          sum[c].x += v[s][c].x;
          sum[c].y += v[s][c].y;
          sum[c].z += v[s][c].z;
          sum[c].w += v[s][c].w;
        }
    }
    const bool adapted = it.chunks > 0;
    const int f = (2 * it.f + rank) * kFeatures + 4 * lane;
#pragma unroll
    for (int c = 0; c < kCombineCols; ++c) {
      if (at[c] < 0 || f >= a.M) continue;
      float v[4] = {sum[c].x, sum[c].y, sum[c].z, sum[c].w};
      if (adapted && !(fabsf(v[0]) < INFINITY && fabsf(v[1]) < INFINITY && fabsf(v[2]) < INFINITY && fabsf(v[3]) < INFINITY)) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (f + k < a.M && (a.requests > 1 ? !(fabsf(v[k]) < INFINITY) : v[k] != v[k] && infinite_row(a, b[c], f + k)))
            v[k] = alone<kOneByte>(a, b[c], i[c], f + k);
      }
      __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + at[c] + f;
      if (a.wide) {
        *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (f + k < a.M) y[k] = __float2bfloat16_rn(v[k]);
      }
    }
  }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
int launch_groups(const ProjArgs& a) { return a.groups < kMaxGroups ? a.groups : kMaxGroups; }
int pairs_of(int sms) { return sms / 2 < 1 ? 1 : sms / 2 < kMaxPairs ? sms / 2 : kMaxPairs; }

size_t plan_bytes(int sms) { return align256(16 + (size_t)pairs_of(sms) * sizeof(CutTile)); }

template <bool kOneByte>
int launch_t(const ProjArgs& a, int sms, bool stall, cudaStream_t st) {
  constexpr uint64_t e = kOneByte ? 1 : 2;
  CUtensorMap tw, tx, tb, tv;
  {
    const uint64_t dims[2] = {(uint64_t)a.K, (uint64_t)a.M}, strides[1] = {a.K * e};
    const uint32_t box[2] = {(uint32_t)(kUnitBytes / e), kFeatures};
    if (encode_nd(&tw, a.W, 2, dims, strides, box, (int)e, 128) != CUDA_SUCCESS) return KDTV_ERR_CUDA;
  }
  {
    const uint64_t row = (a.K * e + 15) / 16 * 16;         // strides of single rows do not matter
    const uint64_t dims[3] = {(uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.B};
    const uint64_t strides[2] = {a.N > 1 ? a.xs[1] * e : row, a.B > 1 ? a.xs[0] * e : row * a.N};
    const uint32_t box[3] = {(uint32_t)(kUnitBytes / e), (uint32_t)a.half_rows, (uint32_t)a.half_requests};
    if (encode_nd(&tx, a.x, 3, dims, strides, box, (int)e, 128) != CUDA_SUCCESS) return KDTV_ERR_CUDA;
  }
  tb = tv = tx;
  if (a.adapter) {
    const uint64_t dims[3] = {(uint64_t)a.R, (uint64_t)a.M, (uint64_t)a.adapters};
    const uint64_t strides[2] = {(uint64_t)a.R * 2, (uint64_t)a.M * a.R * 2};
    const uint32_t box[3] = {16, kFeatures, 1};
    if (encode_nd(&tb, a.Bm, 3, dims, strides, box, 2, 32) != CUDA_SUCCESS) return KDTV_ERR_CUDA;
    // v lies as it is to lie in shared memory: rows of 256 bytes, copied as they are
    const uint64_t rows = (uint64_t)launch_groups(a) * a.blocks * a.pairs * a.half_cols;
    const uint64_t vdims[2] = {128, rows}, vstrides[1] = {256};
    const uint32_t vbox[2] = {128, (uint32_t)a.half_cols / 2};
    if (encode_nd(&tv, a.parts, 2, vdims, vstrides, vbox, 2, 0) != CUDA_SUCCESS) return KDTV_ERR_CUDA;
  }
  if (a.adapter && launch_proj_low(a, sms, st) != cudaSuccess) return KDTV_ERR_CUDA;
  const size_t smem = (size_t)a.stages * (kWBytes + a.half_cols * kUnitBytes) +
                      (kOneByte ? 2 * kWindow * kScaleBytes : 0) + sizeof(ProjShared);
  const auto kern = proj_tc_kernel<kOneByte>;
  if (allow_smem(kern, smem) != cudaSuccess) return KDTV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs_of(sms)));
  cfg.blockDim = dim3(threads_of(kOneByte));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {2, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.adapter ? 2 : 1;           // beside the first kernel, where there is one
  if (cudaLaunchKernelEx(&cfg, kern, tw, tx, tb, tv, a, stall ? 1 : 0) != cudaSuccess) return KDTV_ERR_CUDA;
  if (!may_cut(a)) return KDTV_OK;
  const long long tiles = (long long)a.groups * a.blocks * a.features, most = pairs_of(sms) - 1;
  const long long items = (tiles < most ? tiles : most) * 2 * (2 * a.half_cols / kCombineCols);
  if (items == 0) return KDTV_OK;
  if (beside(proj_combine_kernel<kOneByte>) != cudaSuccess) return KDTV_ERR_CUDA;
  const long long blocks = (items + kCombineWarps - 1) / kCombineWarps;
  return launch_ex(proj_combine_kernel<kOneByte>, dim3((unsigned)(blocks < 4ll * sms ? blocks : 4ll * sms)), dim3(32 * kCombineWarps), 0,
                   st, true, a) == cudaSuccess ? KDTV_OK : KDTV_ERR_CUDA;
}

}  // namespace

bool proj_tc_sizes(const kdtv_project_dims* d, int sms, ProjArgs* a) {
  const bool one_byte = d->dtype == KDTV_BF16_FP8KV;
  if (d->dtype == KDTV_F32 || (d->flags & KDTV_FLAG_SIMT)) return false;
  if (!one_byte && d->d_in % 8) return false;
  if (d->d_in > 65536) return false;          // (an output computed by itself has to be ready while others wait)
  if (d->adapters > 0 && d->rank % 8) return false;
  const int cap = kTokens / 2;                // columns of a half
  a->by_rows_of = d->B == 1 || d->N > cap;
  if (a->by_rows_of) {                        // row blocks of one request
    a->requests = a->half_requests = 1;
    a->groups = d->B;
    a->half_rows = (d->N + 1) / 2 < cap ? (d->N + 1) / 2 : cap;
    a->blocks = (d->N + 2 * a->half_rows - 1) / (2 * a->half_rows);
  } else {
    a->groups = (d->B + cap / d->N * 2 - 1) / (cap / d->N * 2);
    a->half_requests = ((d->B + a->groups - 1) / a->groups + 1) / 2;
    a->requests = 2 * a->half_requests;
    a->groups = (d->B + a->requests - 1) / a->requests;
    a->blocks = 1;
    a->half_rows = d->N;
  }
  a->half_cols = (a->half_requests * a->half_rows + 15) / 16 * 16;
  a->base = (int)(((long long)d->d_in * (one_byte ? 1 : 2) + kUnitBytes - 1) / kUnitBytes);
  a->chunks = d->adapters > 0 ? (d->rank + 15) / 16 : 0;
  a->pairs = ((a->requests < d->adapters ? a->requests : d->adapters) * a->chunks + 1) / 2;
  a->features = (d->d_out + 2 * kFeatures - 1) / (2 * kFeatures);
  if ((long long)a->groups * a->blocks * a->features > 0x3fffffffll) return false;
  // As many stages as leave room for a block of the first kernel beside this one's (4 KiB; and 1 KiB each).
  a->stages = (int)((228 * 1024 - 7 * 1024 - sizeof(ProjShared) - (one_byte ? 2 * kWindow * kScaleBytes : 0)) /
                    (kWBytes + a->half_cols * kUnitBytes));
  a->shared = one_byte && a->half_cols > kTokens / 4 ? kShared : 0;
  if (a->shared && a->stages > kShared / kScaleColumns) a->stages = kShared / kScaleColumns;
  if (a->stages > kMaxStages) a->stages = kMaxStages;
  a->by_requests = divisor((unsigned)a->requests);
  a->by_N = divisor((unsigned)d->N);
  a->by_chunks = divisor((unsigned)(a->chunks > 0 ? a->chunks : 1));
  return true;
}

// The plan, A x, partial sums.
size_t proj_tc_workspace(const ProjArgs& a, int sms) {
  return plan_bytes(sms) + align256((size_t)launch_groups(a) * a.blocks * a.pairs * 2 * proj_half_bytes(a)) +
         (size_t)4 * pairs_of(sms) * 2 * a.half_cols * kFeatures * 4;
}

int proj_tc_launches(const ProjArgs& a) {
  return (a.groups + kMaxGroups - 1) / kMaxGroups * (1 + (a.chunks > 0) + may_cut(a));
}

int launch_proj_tc(const ProjArgs& call, int sms, bool stall, cudaStream_t st) {
  ProjArgs a = call;
  const bool one_byte = a.dtype == KDTV_BF16_FP8KV;
  char* at = reinterpret_cast<char*>(call.low);
  a.plan = reinterpret_cast<int*>(at);
  at += plan_bytes(sms);
  a.parts = at;
  at += align256((size_t)launch_groups(a) * a.blocks * a.pairs * 2 * proj_half_bytes(a));
  a.partial = reinterpret_cast<float*>(at);
  a.wide = reinterpret_cast<uintptr_t>(call.y) % 16 == 0 && call.ys[0] % 8 == 0 && call.ys[1] % 8 == 0 && call.M % 8 == 0;
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
