// Tensor-core (tcgen05) path of kdtv_gqa_verify_attn: bf16 queries, bf16 or
// one-byte caches, head dims 64 and 128.
//
// Mathematics.  o = sum_t p_t v_t / sum_t p_t over the keys a node sees, p_t =
// 2^(scale log2(e) q.k_t - m), with a running reference m per row: it moves only
// when a tile's maximum is over 8 above it, so weights stay below 2^8 and O is
// rescaled rarely.  Scores, m, sums and O are fp32; a weight is rounded to bf16
// (to nearest, 2^-8) where it becomes an operand of the tensor cores.
//
// Work.  The query rows of a key/value head are (node, query head) pairs, cut
// into tiles of npt = 128 / G nodes (at most 128 rows, one per TMEM lane).  An
// item is (request, block of hg heads, pair of tiles); its work is its 128-key
// tiles.  All (item, key tile) units form one sequence and group c of hg CTAs
// takes the W consecutive units [cW, (c + 1)W), so ragged batches and few long
// requests spread evenly; CTA h of the group works on head h of the block.  The
// heads of a cache row are neighbours in memory, and the group reads them at
// about the same time (most of a step from 695 to 474 us for 64 requests over
// one-byte caches).  A piece (the part of an item in one CTA) that is not the
// whole item leaves a partial {max, sum, O} that the combine kernel merges.
// One warp of each CTA derives the sequence from prefix_len: no plan kernel.
//
// A CTA runs two score streams s = 0, 1, each with a 128 x 128 score tile, an
// output accumulator in TMEM, four softmax warps and an issuing warp, so that one
// stream's products run while the other's softmax does:
//   two tiles of rows: stream s holds tile s, both read the same keys;
//   one tile: both hold it, stream s takes the key tiles of parity s, and
//             their results are merged at the end of the piece.
// P replaces its scores in TMEM (bf16) and is the A operand of P.V, so only
// keys, values and Q pass through shared memory.  The issuers take turns: a step's
// products (P.V of one tile, Q.K^T of the next) run as one, since products that
// share the tensor cores end together, and then so do the softmaxes (taking turns:
// 258 -> 226 us for 128 nodes over 65536 keys).  A softmax hands its weights over
// in two halves, so that the first half's products run beside the rest of it.
//
// Keys and values enter one ring in the order in which the products need
// them.  With lag = 1 (two tiles) or 2 (one tile), step i of a piece multiplies
// P.V of tile i - lag, then Q.K^T of tile i; the entry number of K_i within the
// piece is i + max(0, i - lag + 1) and of V_i is i + min(n, i + lag).
//
// One-byte caches.  Keys go to the tensor cores as they lie: a query row, scaled
// by a power of two so that its largest element lies in [2^14, 2^15), is the sum of
// three E5M2 parts (three significant bits each, of a bf16's eight; exact down
// to 2^-23 of the row's largest element, and what lies below is off by 2^-31 of
// it), S = (Q0 + Q1 + Q2) K^T costs 1.5 times what bf16 would, and a key's scale
// multiplies its column of scores in the softmax.  (Two E4M3 parts had the bits but
// not the range: elements below 2^-9 of the row's largest lost theirs.  The third
// costs 391 -> 394 us for 64 requests and 310 -> 327 for 128 nodes over 65536
// keys, where the rings of raw keys and values gave up a third of their room to
// it as well.)  Values: TMA brings
// raw rows into a ring of their own, and four warps widen them to bf16 with the
// row's power-of-two scale (exact) into the operand ring.  bf16 caches: the same
// warps touch only the last key tiles, where they zero the value rows behind the
// tree, and (both) replace values that are not finite in the tree's own rows by
// 0, noting the keys: 0 * inf must not reach nodes that do not see them.  The
// epilogue adds them back to the rows that do.
//
// What bounds it (of a measured 1931 TFLOP/s and 6785 GB/s; eight calls in a graph).
// Many rows, long prefixes: the tensor cores, 1280 TFLOP/s at 128 nodes x 64 heads
// over 65536 keys in bf16 (215 us; 1415 between 32768 and 65536 keys, the rest is
// the way in and out; 1155 in a long row of calls, at the card's power limit) and
// 840 from a one-byte cache, where widening and a two-pass softmax share the issue
// slots.  Few rows: loads in flight and the chain load -> product -> softmax ->
// product of a tile, 5090 GB/s at one node over 65536 keys, bf16.  Short calls:
// latency, 13.0 us for one token over 4096 keys, of which planning takes 2 and the
// combine kernel 4.  Measured and not kept: a two-pass softmax for bf16 (284 us
// where one pass took 258); 64 columns at a time for one-byte keys (447 us where 32
// took 432: instruction cache); issuing loops rolled up (474 for 432); prefetching
// scales to L2.
//
// Every wait has a time limit; one that runs out records
// KDTV_ERR_DEVICE_TIMEOUT, whatever the status word held, and ends the CTA's work.

#include <cuda.h>

#include "kdtv_gqa.cuh"
#include "kdtv_ptx.cuh"
#include "kdtv_tmap.cuh"

namespace kdtv {
namespace {

using namespace ptx;

constexpr int kTile = 128;                  // rows of a score tile, keys of a key tile
constexpr int kThreads = 512;
constexpr int kWarpAux = 8, kWarpTma = 12, kWarpPlan = 13, kWarpMma = 14;   // (14, 15: one per stream)
constexpr int kRing = 6;                    // bound on ring sizes (barriers)
constexpr int kPieces = 8;                  // pieces that may be in flight

// barriers
enum {
  // bf16 caches: one ring of keys and values, and the values of the last tiles on their way
  // through the four warps.  One-byte caches: widened values, raw values, raw keys.
  B_KV_FULL = 0, B_KV_EMPTY = B_KV_FULL + kRing, B_TAIL = B_KV_EMPTY + kRing,
  B_RAW_FULL = B_TAIL, B_RAW_EMPTY = B_RAW_FULL + kRing, B_K_FULL = B_RAW_EMPTY + kRing,
  B_K_EMPTY = B_K_FULL + kRing, B_Q_FULL = B_K_EMPTY + kRing,
  B_Q_READY, B_Q_EMPTY, B_S_FULL, B_P_HALF = B_S_FULL + 2, B_P_READY = B_P_HALF + 2,
  B_O_FULL = B_P_READY + 2, B_ML = B_O_FULL + 2, B_O1_FREE, B_MMA_DONE, B_STALL, B_TURN,
  B_SCALE_FREE = B_TURN + 2, B_SCALE_FULL = B_SCALE_FREE + 2, B_AUX = B_SCALE_FULL + 2, B_PIECE,
  B_PIECE_READ = B_PIECE + kPieces,
  B_COUNT = B_PIECE_READ + kPieces
};

// Arrivals of a barrier's phase.
template <bool kFp8>
__device__ __forceinline__ uint32_t arrivals(int i) {
  if (i < B_KV_EMPTY) return kFp8 ? 4 : 1;                  // (widened by four warps)
  if (i < B_TAIL) return 2;                                 // both issuers
  if (i < B_RAW_EMPTY) return 1;
  if (i < B_K_FULL) return 4;
  if (i < B_K_EMPTY) return 1;
  if (i < B_Q_FULL) return 2;
  if (i == B_Q_READY || i == B_ML || i == B_O1_FREE || i == B_AUX) return 4;
  if (i == B_Q_EMPTY || i == B_MMA_DONE) return 2;
  if (i >= B_P_HALF && i < B_O_FULL) return 4;              // (and B_P_READY)
  if (i >= B_SCALE_FREE && i < B_SCALE_FULL) return 8;
  if (i >= B_SCALE_FULL && i < B_AUX) return 4;
  if (i >= B_PIECE_READ) return 15;                         // producer, two issuers, 4 + 8 warps
  return 1;
}

constexpr int kQParts = 3;                  // one-byte keys: E5M2 parts of a query row

template <int D, bool kFp8>
struct Cfg {
  static constexpr int kTileBytes = kTile * D * 2;            // Q or V tile (bf16 caches: K too) in bf16
  static constexpr int kChunk = kTile * 128;                  // its 64 columns, 128-byte rows
  static constexpr int kRawBytes = kTile * D;                 // one-byte K or V tile, part of a Q tile
  static constexpr int kQBytes = kFp8 ? kQParts * kRawBytes : kTileBytes;   // (bf16 first, then its parts)
  // D = 128: Q 64 KiB, then 5 tiles of 32 KiB; or Q 96 KiB, 2 tiles of widened values, 2 raw ones
  // of 16 KiB and 2 of keys
  static constexpr int kSlots = kFp8 ? (D == 128 ? 2 : 4) : (D == 128 ? 5 : 6);
  static constexpr int kRaw = kFp8 ? (D == 128 ? 2 : 6) : 0;
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = 2 * kQBytes;
  static constexpr int kOffRaw = kOffKV + kSlots * kTileBytes;
  static constexpr int kOffK = kOffRaw + kRaw * kRawBytes;    // (the key ring has kRaw entries too)
  static constexpr int kOffMisc = kOffK + kRaw * kRawBytes;
  // barriers (padded to 16 bytes), TMEM address and abort flag, then per piece its record, the
  // page flag and the key mask, stream 1's {max, sum}, the key scales of two tiles
  static constexpr int kBarBytes = (B_COUNT * 8 + 15) / 16 * 16;
  static constexpr int kOffMl = kOffMisc + kBarBytes + 16 + kPieces * (32 + 16 + 4);
  static constexpr int kOffScale = kOffMl + kTile * 8;
  static constexpr int kSmem = kOffScale + (kFp8 ? 2 * kTile * 4 : 0);
  static_assert(kSmem <= 227 * 1024 && kRing >= kSlots && kRing >= kRaw, "shared memory");
  static constexpr uint32_t kColS = 0, kColO = 2 * kTile;     // S0, S1, O0, O1
};

// A place in a ring of N entries; its barriers' phase.  (A fresh barrier counts
// as having completed a phase of parity 1, so the first round finds it empty.)
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0u;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];"
      :: "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint32_t bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];"
      :: "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// ---- the sequence of units ---------------------------------------------------------------
__device__ __forceinline__ int key_tiles(int L, int n) { return (L + n + kTile - 1) / kTile; }
__device__ __forceinline__ int row_pairs(const GqaArgs& a, int n) {
  return (int)divide((unsigned)(n + 2 * a.npt - 1), a.by_pair);
}
__device__ __forceinline__ int units_of(const GqaArgs& a, int b, int* L, int* n) {
  gqa_request(a, b, L, n);
  return *n > 0 ? a.blocks * row_pairs(a, *n) * key_tiles(*L, *n) : 0;
}

// A piece: the part of an item in one CTA.  The planning warp walks the CTA's
// units and hands the pieces to the other roles through a ring in shared memory.
struct __align__(16) Piece {
  int b, L, n, kvh;          // request, its prefix and live nodes, key/value head
  int node0, t0, t1, flags;  // first node of its first tile, key tiles
  __device__ __forceinline__ bool two() const { return flags & 1; }      // two tiles of rows
  __device__ __forceinline__ bool whole() const { return flags & 2; }    // all key tiles of the item
  __device__ __forceinline__ bool tail() const { return flags & 4; }     // reaches past the prefix
  __device__ __forceinline__ bool later() const { return flags & 8; }    // not at the CTA's first unit
};
constexpr int kEnd = 16;     // flag: no piece is left

// ---- bounded waits -------------------------------------------------------------------------
struct Guard {
  volatile uint32_t* abort;      // shared memory
  unsigned int* status;
  uint32_t limit;                // ns, below 2^32
};
__device__ __forceinline__ uint32_t timer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
// Short code: a wait stands at some thirty places of loops that share an
// instruction cache.
__device__ __forceinline__ bool wait(const Guard& g, uint32_t bar, uint32_t parity) {
  if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
  const uint32_t t0 = timer_lo();
#pragma unroll 1
  while (!mbar_try_wait_sleep(bar, parity, 20000u)) {
    if (*g.abort) return false;
    if (timer_lo() - t0 > g.limit) {
      atomicExch(g.status, (unsigned)KDTV_ERR_DEVICE_TIMEOUT);   // over any other code: the combine kernel asks
      *g.abort = 1u;
      return false;
    }
  }
  return true;
}
// Waits for asynchronous work that is in flight and will finish (limited all the same).
__device__ __forceinline__ void drain(const Guard& g, uint32_t bar, uint32_t parity) {
  const uint32_t t0 = timer_lo();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity))
    if (timer_lo() - t0 > g.limit) return;
}
__device__ __forceinline__ bool wait_warp(const Guard& g, uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(g, bar, parity));
}

// Four E4M3 bytes as bf16 pairs of their values times 2^-120: a code's exponent
// and mantissa bits moved to bf16's places (also of its subnormals, which become
// bf16's).  A byte and its sign, spread over the next one, are one permute; the
// conversion instructions, through f16 and fp32, took 1.8 times as long.  NaN is
// a number here (480): see has_nan_code.
__device__ __forceinline__ uint2 spread4(uint32_t w) {
  uint32_t a, b;
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(a) : "r"(w));   // {b0, its sign, b1, its sign}
  asm("prmt.b32 %0, %1, 0, 0xb3a2;" : "=r"(b) : "r"(w));
  return make_uint2((a << 4) & 0x87f087f0u, (b << 4) & 0x87f087f0u);
}
// Bit 7 of each byte whose code is NaN (other bits: anything).
__device__ __forceinline__ uint32_t has_nan_code(uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; }
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t f) {
  uint32_t y;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(f));
  return y;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// D[tmem] (+)= A[smem desc] * B[smem desc]^T, one-byte operands, 32 elements deep, fp32 accumulation.
__device__ __forceinline__ void mma_fp8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\t"
               "setp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
               :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// A in E5M2, B in E4M3.
__host__ __device__ constexpr uint32_t idesc_fp8(int M, int N) {
  return (1u << 4) | (1u << 7) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Exponent k of a query row's scale 2^k, from the largest finite magnitude of its bf16 bits: the
// largest element lands in [2^14, 2^15), below E5M2's 57344.  (bf16's smallest steps, 2^-133, are
// E5M2's too at 2^127.)
__device__ __forceinline__ int q_exponent(uint32_t max_bits) {
  return min(141 - (int)(max_bits >> 7), 127);
}
// A product of such a row and a key is taken back by 2^-kBack before it meets the key's scale, so
// that scales up to 2^100 leave it finite (448 * 2^15 * 128 terms are below 2^31).
constexpr int kBack = 7;
// Largest finite magnitude (bits) of a bf16 pair and one so far.
__device__ __forceinline__ uint32_t max_finite(uint32_t w, uint32_t m) {
  const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  if (lo < 0x7f80u) m = max(m, lo);
  if (hi < 0x7f80u) m = max(m, hi);
  return m;
}
// Four floats as E5M2 bytes, and what the bytes leave of them (exact in fp32).
__device__ __forceinline__ uint32_t take_e5m2(float (&x)[4]) {
  uint32_t w = 0u;
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(x[k], x[k + 1]), __NV_SATFINITE, __NV_E5M2);
    const float2 g = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E5M2)));
    x[k] -= g.x;
    x[k + 1] -= g.y;
    w |= two << (8 * k);
  }
  return w;
}
// Four bf16 (two words), times f, as E5M2 parts.  A part is nearest what the earlier ones leave, so
// after the first an element has five bits left, and after the second one.  Infinities become NaN,
// as their scores would.
__device__ __forceinline__ void split_e5m2(uint32_t w0, uint32_t w1, float f, uint32_t (&part)[kQParts]) {
  float x[4] = {__uint_as_float(w0 << 16) * f, __uint_as_float(w0 & 0xffff0000u) * f,
                __uint_as_float(w1 << 16) * f, __uint_as_float(w1 & 0xffff0000u) * f};
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = fabsf(x[k]) < INFINITY ? x[k] : __uint_as_float(0x7fffffffu);
#pragma unroll
  for (int k = 0; k < kQParts; ++k) part[k] = take_e5m2(x);
}
// Zeroes the elements of a bf16 pair that are not finite; true if there were any.
__device__ __forceinline__ bool drop_nonfinite(uint32_t& w) {
  const bool lo = (w & 0x00007f80u) == 0x00007f80u, hi = (w & 0x7f800000u) == 0x7f800000u;
  if (lo) w &= 0xffff0000u;
  if (hi) w &= 0x0000ffffu;
  return lo || hi;
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// What of a tree node's value row is not finite, added to the output row that a
// thread has just written (o: bf16 output, or fp32 partial).  Rare: out of line.
// Its elements 8 i .. 8 i + 7 stand `step` elements from the previous eight.
// (One-byte caches: NaN codes, and codes whose value at the row's scale is above the largest
// bf16, which is where fp32 overflows too: a code has four significant bits.)
template <int D, bool kFp8, typename T>
__device__ __noinline__ void add_nonfinite(const GqaArgs& a, int b, int kvh, int t, T* o, int step) {
  const long long row = gqa_row(a, b, t);
  if (row < 0) return;
  const long long at = (row * a.Hkv + kvh) * D;
  const float scale = kFp8 ? scale_of_byte(a.v_scale[row * a.Hkv + kvh]) : 1.f;
#pragma unroll 1
  for (int k = 0; k < D; ++k) {
    const float x = kFp8 ? to_f32(static_cast<const __nv_fp8_e4m3*>(a.v)[at + k]) * scale
                         : to_f32(static_cast<const __nv_bfloat16*>(a.v)[at + k]);
    if (fabsf(x) < INFINITY) continue;
    T* at_k = o + (k >> 3) * step + (k & 7);
    const float y[1] = {to_f32(*at_k) + x};
    store_v<1>(at_k, y);
  }
}
// A row of values in shared memory with NaN codes (src: the codes; dst: bf16, swizzled, 64 columns
// a chunk): they become NaN, or 0 if `drop`.  Rare: out of line.
template <int D, int kChunk>
__device__ __noinline__ void put_nan(uint32_t src, uint32_t dst, int swz, bool drop) {
#pragma unroll 1
  for (int e = 0; e < D; ++e) {
    uint32_t code;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(code) : "r"(src + e) : "memory");
    if ((code & 0x7fu) != 0x7fu) continue;
    const uint32_t at = dst + (e >> 6) * kChunk + ((((e >> 3) & 7) ^ swz) << 4) + (e & 7) * 2;
    asm volatile("st.shared.u16 [%0], %1;" :: "r"(at), "h"((unsigned short)(drop ? 0 : 0x7fff)) : "memory");
  }
}
// Register split with bf16 caches: the launch has 512 x 128; the softmax warps
// take most (a row's 128 scores stay in registers).  With one-byte caches the
// scores come in chunks and every role keeps its 128: 64 for the warps that
// widen the values spilled, and 64 requests took 467 us instead of 426.
constexpr int kRegsSoftmax = 192, kRegsAux = 64, kRegsControl = 64;
static_assert(256 * kRegsSoftmax + 128 * kRegsAux + 128 * kRegsControl <= 512 * 128, "registers of the launch");
template <int R>
__device__ __forceinline__ void reg_grow() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(R));
}
template <int R>
__device__ __forceinline__ void reg_shrink() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(R));
}
template <int N>
__device__ __forceinline__ void pin(float (&v)[N]) {     // values loaded from TMEM: not before the wait
#pragma unroll
  for (int k = 0; k < N; ++k) asm volatile("" : "+f"(v[k]));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(y.x), "=f"(y.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return y;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(y.x), "=f"(y.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(y.x), "=f"(y.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
gqa_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ GqaArgs a, int stall) {
  using C = Cfg<D, kFp8>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffMisc);
  const uint32_t bar0 = smem_u32(bars);
  auto BAR = [&](int i) { return bar0 + 8u * i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kOffMisc + C::kBarBytes);   // [0] tmem, [1] abort
  Piece* pieces = reinterpret_cast<Piece*>(misc + 4);                 // [kPieces]
  uint4* nonfinite = reinterpret_cast<uint4*>(pieces + kPieces);      // [kPieces] keys of the tree
  volatile uint32_t* bad_page = reinterpret_cast<uint32_t*>(nonfinite + kPieces);   // [kPieces]
  float2* ml1 = reinterpret_cast<float2*>(smem + C::kOffMl);          // [128] stream 1's {max, sum}
  const Guard guard{misc + 1, a.status, stall ? 20000000u : 2000000000u};

  grid_dep_launch();               // the combine kernel may be launched; it waits for this grid
  // The planner's first 32 requests are on their way while barriers and TMEM are set up.
  int L0 = 0, n0 = 0, u0 = 0;
  if (warp == kWarpPlan && lane < a.B) u0 = units_of(a, lane, &L0, &n0);
  if (threadIdx.x < B_COUNT) mbar_init(BAR(threadIdx.x), arrivals<kFp8>(threadIdx.x));
  if (threadIdx.x == 0) misc[1] = 0u;
  fence_mbar_init();
  if (threadIdx.x < kPieces) bad_page[threadIdx.x] = 0u;
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
  }
  if (warp == kWarpTma && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];

  // The k-th piece (k counts up in every role); false: none is left, or the CTA gave up.
  auto get_piece = [&](int k, Piece& p) -> bool {
    if (!wait_warp(guard, BAR(B_PIECE + k % kPieces), (k / kPieces) & 1)) return false;
    p = pieces[k % kPieces];
    __syncwarp();
    if (lane == 0) mbar_arrive(BAR(B_PIECE_READ + k % kPieces));
    return !(p.flags & kEnd);
  };

  // (the split is the first statement of each branch: the compiler allocates by branch)
  if (warp >= kWarpTma) {
  if constexpr (!kFp8) reg_shrink<kRegsControl>();
  if (warp == kWarpPlan) {
    // ---- planner: W and this CTA's first unit, then its pieces.  All else waits for the first
    // piece, and the code is cold: the first 32 requests stay in registers, and what a launch knows
    // is divided by multiplication (together 1.2 us of a call).
    int sum = u0;
#pragma unroll 1
    for (int b = lane + 32; b < a.B; b += 32) {
      int Lb, nb;
      sum += units_of(a, b, &Lb, &nb);
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    const int W = (int)divide((unsigned)(sum + a.groups - 1), a.by_groups);
    const int group = (int)divide(blockIdx.x, a.by_hg), my_head = blockIdx.x - group * a.hg;
    const long long first = (long long)group * W;
    const int end = first < sum ? (int)(first + W < sum ? first + W : sum) : 0;
    int at = first < sum ? (int)first : 0, b = 0, off = 0;
    if (end > 0) {
      int before = 0;
      if (blockIdx.x == 0 && lane == 0) a.plan[0] = W;          // for the combine kernel
#pragma unroll 1
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        int Lb, nb;
        const int u = b0 == 0 ? u0 : b0 + lane < a.B ? units_of(a, b0 + lane, &Lb, &nb) : 0;
        int scan = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, scan, o);
          if (lane >= o) scan += x;
        }
        const int lo = before + scan - u;
        if (blockIdx.x == 0 && b0 + lane < a.B) a.plan[1 + b0 + lane] = lo;
        const uint32_t here = __ballot_sync(0xffffffffu, u > 0 && at >= lo && at < lo + u);
        if (here) {
          b = b0 + __ffs(here) - 1;
          off = at - __shfl_sync(0xffffffffu, lo, __ffs(here) - 1);
          if (blockIdx.x > 0) break;               // (the first CTA goes on: it writes the plan)
        }
        before += __shfl_sync(0xffffffffu, scan, 31);
      }
    }
    int L = __shfl_sync(0xffffffffu, L0, b & 31), n = __shfl_sync(0xffffffffu, n0, b & 31);
    int nt = 1, rps = 1, hb = 0, pair = 0, t0 = 0;
    if (end > 0) {
      if (b >= 32) gqa_request(a, b, &L, &n);
      nt = key_tiles(L, n);
      rps = row_pairs(a, n);
      if (off > 0) {
        const int item = off / nt;
        t0 = off - item * nt;
        hb = item / rps;
        pair = item - hb * rps;
      }
    }
    for (int k = 0;; ++k) {
      if (k >= kPieces && !wait_warp(guard, BAR(B_PIECE_READ + k % kPieces), (k / kPieces - 1) & 1)) break;
      const int t1 = min(nt, t0 + end - at);
      if (lane == 0) {
        Piece p;
        p.b = b; p.L = L; p.n = n; p.kvh = hb * a.hg + my_head;
        p.node0 = pair * 2 * a.npt;
        p.t0 = t0; p.t1 = t1;
        p.flags = (n - p.node0 > a.npt ? 1 : 0) | (t0 == 0 && t1 == nt ? 2 : 0) |
                  (t1 == nt || t1 * kTile > L ? 4 : 0) | (k > 0 ? 8 : 0) | (at >= end ? kEnd : 0);
        pieces[k % kPieces] = p;
        mbar_arrive(BAR(B_PIECE + k % kPieces));
      }
      __syncwarp();
      if (at >= end) break;
      at += t1 - t0;
      t0 = 0;
      if (at < end && ++pair == rps) {
        pair = 0;
        if (++hb == a.blocks) {
          hb = 0;
          do {
            gqa_request(a, ++b, &L, &n);         // units are left, so a request with some exists
          } while (n == 0);
          nt = key_tiles(L, n);
          rps = row_pairs(a, n);
        }
      }
    }
  } else if (warp == kWarpTma) {
    // ---- TMA producer: the warp's lanes hold page ids; lane l loads box l of a tile ---------
    const int boxes = a.page_size ? kTile / a.page_size : 1;      // page_size divides 128
    const int box_rows = kTile / boxes;
    Piece p;
    bool alive = true;
    if (stall) alive = wait_warp(guard, BAR(B_STALL), 0);
    Ring<C::kSlots> ring;                         // bf16
    Ring<kFp8 ? C::kRaw : 1> kring, vring;        // one byte
    int entries = 0, k_entries = 0, v_entries = 0, q_loads = 0;
    for (int index = 0; alive && get_piece(index, p); ++index) {
      const int kvh = p.kvh, n = p.t1 - p.t0, T = p.L + p.n;
      const bool two = p.two();
      const int lag = two ? 1 : 2;
      // Q once its previous contents are used up.  Keys and values come first where they have room:
      // the next piece's are on their way while the last one's products run.
      bool q_pending = true;
      auto load_q = [&]() -> bool {
        q_pending = false;
        if (index > 0 && !wait_warp(guard, BAR(B_Q_EMPTY), (index - 1) & 1)) return false;
        if (lane == 0) {
          const uint32_t bytes = (uint32_t)a.npt * a.G * 128;
          mbar_expect_tx(BAR(B_Q_FULL), bytes * (D / 64) * (two ? 2 : 1));
          for (int s = 0; s < (two ? 2 : 1); ++s)
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(sbase + C::kOffQ + s * C::kQBytes + c * C::kChunk, &tm_q, BAR(B_Q_FULL), 64 * c,
                          kvh * a.G, p.b * a.N + p.node0 + s * a.npt);
        }
        ++q_loads;
        return true;
      };
      // windows of 32 page ids, the next one loaded ahead; a page out of range is read as page 0
      // and marks the piece
      const int32_t* table = a.page_table + (long long)p.b * a.max_pages;
      auto page_at = [&](int k) {                 // k-th box of the piece
        const int box = p.t0 * boxes + k;
        if (!a.page_size || (long long)box * box_rows >= T) return 0;
        return table[box];
      };
      int win = page_at(lane), win_next = page_at(32 + lane);
      if (index == 0) alive = load_q();           // (while the page ids are under way)
      int page0 = 0, page1 = 0, page2 = 0;        // of tiles i, i - 1, i - 2
      uint32_t bad = 0;
      for (int i = 0; alive && i < n + lag; ++i) {
        page2 = page1;
        page1 = page0;
        if (i < n) {
          const int k = i * boxes;
          if (k > 0 && (k & 31) == 0) {
            win = win_next;
            win_next = page_at(k + 32 + lane);
          }
          page0 = __shfl_sync(0xffffffffu, win, (k + lane) & 31);
          if (page0 < 0 || page0 >= (a.page_size ? a.num_pages : 1)) {
            if (lane < boxes) bad = 1;
            page0 = 0;
          }
          if (i == n - 1) {                       // before the piece's last loads: seen by its epilogue
            const bool any = __any_sync(0xffffffffu, bad);
            if (lane == 0) {
              bad_page[index % kPieces] = any ? 1u : 0u;
              if (any) gqa_error(a, KDTV_ERR_BAD_PAGE);
            }
          }
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {          // V of tile i - lag, then K of tile i
          const int kt = kv == 0 ? i - lag : i;
          if (kt < 0 || kt >= n) continue;
          const int slot = kFp8 ? (kv == 0 ? vring.slot : kring.slot) : ring.slot;
          const uint32_t phase = kFp8 ? (kv == 0 ? vring.phase : kring.phase) : ring.phase;
          const uint32_t empty = BAR((kFp8 ? (kv == 0 ? B_RAW_EMPTY : B_K_EMPTY) : B_KV_EMPTY) + slot);
          if (q_pending && (__all_sync(0xffffffffu, mbar_test_wait(BAR(B_Q_EMPTY), (index - 1) & 1)) ||
                            !__all_sync(0xffffffffu, mbar_test_wait(empty, phase ^ 1u))))
            alive = load_q();
          alive = alive && wait_warp(guard, empty, phase ^ 1u);
          if (!alive) break;
          const int t = (p.t0 + kt) * kTile;
          const int live = a.page_size ? min(boxes, (T - t + box_rows - 1) / box_rows) : 1;
          // bf16 values of a tile that reaches past the prefix go to the four warps first, which
          // then arrive on the entry's full barrier (every wait sees each phase of its barrier)
          const bool to_aux = !kFp8 && kv == 0 && t + kTile > p.L;
          const uint32_t bar =
              BAR((kFp8 ? (kv == 0 ? B_RAW_FULL : B_K_FULL) : (to_aux ? B_TAIL : B_KV_FULL)) + slot);
          const uint32_t dst = sbase + (kFp8 ? (kv == 0 ? C::kOffRaw : C::kOffK) + slot * C::kRawBytes
                                             : C::kOffKV + slot * C::kTileBytes);
          if (lane == 0) mbar_expect_tx(bar, (uint32_t)live * box_rows * D * (kFp8 ? 1 : 2));
          __syncwarp();
          if (lane < live) {
            const int page = kv == 1 ? page0 : (lag == 1 ? page1 : page2);
            const void* map = kv == 0 ? &tm_v : &tm_k;
            const int y = a.page_size ? 0 : t, z = a.page_size ? page : p.b;
            if constexpr (kFp8) {
              tma_load_4d(dst + lane * box_rows * D, map, bar, 0, kvh, y, z);
            } else {
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(dst + c * C::kChunk + lane * box_rows * 128, map, bar, 64 * c, kvh, y, z);
            }
          }
          if constexpr (kFp8) {
            if (kv == 0) {
              vring.next();
              ++v_entries;
            } else {
              kring.next();
              ++k_entries;
            }
          } else {
            ring.next();
            ++entries;
          }
        }
      }
      if (alive && q_pending) alive = load_q();
    }
    // every copy has landed before the CTA may exit
    if (q_loads) drain(guard, BAR(B_Q_FULL), (q_loads - 1) & 1);
    auto drain_ring = [&](uint32_t full, int count, int size) {
      for (int x = count > size ? count - size : 0; x < count; ++x)
        drain(guard, BAR(full + x % size), (x / size) & 1);
    };
    if constexpr (kFp8) {
      drain_ring(B_K_FULL, k_entries, C::kRaw);
      drain_ring(B_RAW_FULL, v_entries, C::kRaw);
    } else {
      drain_ring(B_KV_FULL, entries, C::kSlots);
    }
    __syncwarp();
  } else {
    // ---- MMA issuers: warp 14 + s issues stream s (one lane of it; the others follow piece by
    // piece).  A thread needs a few hundred cycles from a wait to its next product, about as long
    // as the products it then issues take, so the streams' issuers are two warps.  Each waits on
    // every entry of the ring, also the other stream's, so that it sees each phase of the barriers.
    const int s = warp - kWarpMma;
    constexpr uint32_t kIdescS = kFp8 ? idesc_fp8(kTile, kTile) : idesc_bf16(kTile, kTile, 0, 0);
    constexpr uint32_t kIdescO = idesc_bf16(kTile, D, 0, 1);
    // operands at fixed places, as descriptors to which a byte offset / 16 is added
    // (one-byte keys: rows of D bytes, 128- or 64-byte swizzle)
    const bool narrow = kFp8 && D == 64;
    const uint64_t q_desc = narrow ? smem_desc_sw64(sbase + C::kOffQ, 16, 512) : smem_desc(sbase + C::kOffQ, 16, 1024);
    const uint32_t k_at = sbase + (kFp8 ? C::kOffK : C::kOffKV);
    const uint64_t k_desc = narrow ? smem_desc_sw64(k_at, 16, 512) : smem_desc(k_at, 16, 1024);
    const uint64_t v_desc = smem_desc(sbase + C::kOffKV, C::kChunk, 1024);
    const uint32_t dS = tmem + C::kColS + kTile * s, dO = tmem + C::kColO + D * s;
    Piece p;
    bool alive = true;
    Ring<C::kSlots> ring;
    Ring<kFp8 ? C::kRaw : 1> kring;
    uint32_t p_phase = 0u, turn = s == 0 ? 1u : 0u;   // (stream 0 begins)
    for (int index = 0; __all_sync(0xffffffffu, alive) && get_piece(index, p); ++index) {
      const int n = p.t1 - p.t0;
      const bool two = p.two();
      const int lag = two ? 1 : 2;
      if (lane != 0) continue;
      const uint64_t ad = q_desc + (uint32_t)(two ? s * (C::kQBytes >> 4) : 0);
      alive = wait(guard, BAR(kFp8 ? B_Q_READY : B_Q_FULL), index & 1);
      // The streams take turns: a step's products run as one, and beside the other stream's softmax.
      // (Products that share the tensor cores end together, and then so do the softmaxes.)  In a
      // one-tile piece the steps alternate between the streams; an even number of them, so that the
      // next piece begins with stream 0 again.
      const int steps = two ? n + lag : (n + lag + 1) & ~1;
      for (int i = 0; alive && i < steps; ++i) {
        const int vt = i - lag;
        const bool mine = two || (i & 1) == s, has_v = vt >= 0 && vt < n, has_k = i < n;
        // the entries first (loaded long ago), then the softmax: from there on the products follow
        // one another
        // the entries and the softmax; one look at all three, because each costs its latency
        const int v_slot = ring.slot;
        const uint32_t v_full = BAR(B_KV_FULL + v_slot), v_phase = ring.phase;
        if (has_v) ring.next();
        const int k_slot = kFp8 ? kring.slot : ring.slot;
        const uint32_t k_full = BAR((kFp8 ? B_K_FULL : B_KV_FULL) + k_slot), k_phase = kFp8 ? kring.phase : ring.phase;
        const uint32_t k_empty = BAR((kFp8 ? B_K_EMPTY : B_KV_EMPTY) + k_slot), p_half = BAR(B_P_HALF + s);
        if (has_k) {
          if constexpr (kFp8) kring.next();
          else ring.next();
        }
        const bool v_ok = mbar_try_wait(v_full, v_phase) || !has_v, k_ok = mbar_try_wait(k_full, k_phase) || !has_k;
        const bool p_ok = mbar_try_wait(p_half, p_phase) || !(has_v && mine);
        if (!(v_ok && k_ok && p_ok))
          alive = (v_ok || wait(guard, v_full, v_phase)) && (k_ok || wait(guard, k_full, k_phase)) &&
                  (p_ok || wait(guard, p_half, p_phase));
        bool all_ready = false;
        if (mine) {
          alive = alive && wait(guard, BAR(B_TURN + s), turn);
          turn ^= 1u;
          all_ready = mbar_try_wait(BAR(B_P_READY + s), p_phase);
        }
        if (!alive) break;
        if (!mine) {
          if (has_v) mbar_arrive(BAR(B_KV_EMPTY + v_slot));
          if (has_k) mbar_arrive(k_empty);
        } else {
          if (has_v) {                                          // O_s (+)= P_s V
            const uint64_t bd = v_desc + (uint32_t)(v_slot * (C::kTileBytes >> 4));
            const uint32_t acc = two ? vt > 0 : vt > 1;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ts(dO, dS + 8 * kk, bd + kk * 128, kIdescO, kk > 0 ? 1u : acc);
            if (!all_ready) {                                   // the second half, looked at before the turn
              alive = wait(guard, BAR(B_P_READY + s), p_phase);
              if (!alive) break;
              tc_fence_after();
            }
            p_phase ^= 1u;
#pragma unroll
            for (int kk = 4; kk < 8; ++kk) mma_bf16_ts(dO, dS + 8 * kk, bd + kk * 128, kIdescO, 1u);
          }
          if (has_k) {                                          // S_s = Q K^T, over P_s
            const uint64_t bd = k_desc + (uint32_t)(k_slot * ((kFp8 ? C::kRawBytes : C::kTileBytes) >> 4));
            tc_fence_after();
            if constexpr (kFp8) {                               // the queries' parts, 32 columns a product
#pragma unroll
              for (int kk = 0; kk < kQParts * D / 32; ++kk) {
                const uint32_t part = (kk / (D / 32)) * (C::kRawBytes >> 4), off = (kk % (D / 32)) * 2;
                mma_fp8(dS, ad + part + off, bd + off, kIdescS, kk > 0);
                // the other stream's issuer needs about as long to begin as the rest takes
                if (kk == (kQParts - 1) * D / 32) mbar_arrive(BAR(B_TURN + 1 - s));
              }
            } else {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                constexpr uint32_t kC = C::kChunk >> 4;
                const uint32_t off = (kk >> 2) * kC + (kk & 3) * 2;
                mma_bf16(dS, ad + off, bd + off, kIdescS, kk > 0);
                if (kk == D / 32) mbar_arrive(BAR(B_TURN + 1 - s));   // (as above)
              }
            }
            mma_commit(BAR(B_S_FULL + s));
            mma_commit(k_empty);
          } else {
            mbar_arrive(BAR(B_TURN + 1 - s));
          }
          if (has_v) {
            mma_commit(BAR(B_KV_EMPTY + v_slot));
            if (vt + (two ? 1 : 2) >= n) mma_commit(BAR(B_O_FULL + s));
          }
        }
        if (i == n - 1) mma_commit(BAR(B_Q_EMPTY));
      }
    }
    if (lane == 0) {
      mma_commit(BAR(B_MMA_DONE));                 // every product has finished before TMEM is freed
      drain(guard, BAR(B_MMA_DONE), 0);
    }
    __syncwarp();
  }
  } else if (warp >= kWarpAux) {
    if constexpr (!kFp8) reg_shrink<kRegsAux>();
    // ---- widening (one-byte caches) and the last tiles: thread = key row of the tile -----------
    const int row = threadIdx.x - kWarpAux * 32;
    const int swz = row & 7;
    Piece p;
    bool alive = true;
    int g = 0;
    uint32_t tail_phase = 0u, aux_phase = 0u;
    // The four warps meet (with a time limit, which a named barrier does not have: a warp may have
    // given up).
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_AUX));
      const bool ok = wait_warp(guard, BAR(B_AUX), aux_phase);
      aux_phase ^= 1u;
      return ok;
    };
    Ring<kFp8 ? C::kRaw : 1> vring;
    Ring<C::kSlots> ring;
    Ring<2> sring;                                // of key scales
    float* scales = reinterpret_cast<float*>(smem + C::kOffScale);
    for (int index = 0; alive && get_piece(index, p); ++index) {
      const int kvh = p.kvh, n = p.t1 - p.t0, T = p.L + p.n;
      const int lag = p.two() ? 1 : 2;
      uint32_t* nf = reinterpret_cast<uint32_t*>(nonfinite + index % kPieces);
      if (row < 4) nf[row] = 0u;
      alive = meet();
      if (!alive) break;
      if constexpr (kFp8) {
        // The scale bytes of tile i + 2 are loaded at the end of step i, with a page id loaded a step
        // before: behind the step's proxy fence, which waits for every load that is under way.
        // (Positions behind the last are read as the last: every address is one of the request's.)
        const int32_t* table = a.page_table + (long long)p.b * a.max_pages;
        const uint8_t* ks = a.k_scale + kvh;
        const uint8_t* vs = a.v_scale + kvh;
        int t_at = p.t0 * kTile + row;                // of the tile whose page id is loaded next
        auto next_page = [&]() -> int {
          const int t = min(t_at, T - 1);
          return a.page_size ? table[t >> a.page_shift] : 0;
        };
        auto row_of_scale = [&](int page) -> long long {   // of t_at's row; moves on to the next tile
          const int t = min(t_at, T - 1);
          t_at += kTile;
          const int pg = (unsigned)page < (unsigned)a.num_pages ? page : 0;
          const long long r = a.page_size ? ((long long)pg << a.page_shift) + (t & (a.page_size - 1))
                                          : (long long)p.b * a.t_stride + t;
          return r * a.Hkv;
        };
        long long at = row_of_scale(next_page());
        int k0 = ks[at], v0 = vs[at];                      // of tiles i, i + 1
        at = row_of_scale(next_page());
        int k1 = ks[at], v1 = vs[at], vm1 = 0, vm2 = 0;    // values: of tiles i + 1 .. i - 2
        int page_next = next_page();

        // Q: each row's E5M2 parts over and behind its bf16 (while the scale bytes arrive)
        alive = wait_warp(guard, BAR(B_Q_FULL), index & 1);
        if (!alive) break;
#pragma unroll 1
        for (int tile = 0; tile < (p.two() ? 2 : 1); ++tile) {
          const uint32_t q0 = sbase + C::kOffQ + tile * C::kQBytes, qr = q0 + row * 128;
          uint32_t mxb = 0u;
#pragma unroll 2
          for (int u = 0; u < D / 8; ++u) {
            const uint4 w = lds128(qr + (u >> 3) * C::kChunk + (((u & 7) ^ swz) << 4));
            mxb = max_finite(w.w, max_finite(w.z, max_finite(w.y, max_finite(w.x, mxb))));
          }
          const float f = __uint_as_float((uint32_t)(q_exponent(mxb) + 127) << 23);
          // Part k lies at k kRawBytes, so the second of a 128-wide row's first half lies over its second
          // half, which is read before; a 64-wide row's parts lie over other rows.
          uint4 held[4];
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint4 w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) w[u] = lds128(qr + c * C::kChunk + ((u ^ swz) << 4));
            if (D == 64) {
              alive = meet();
              if (!alive) break;
            }
            if (c == 1)
#pragma unroll
              for (int u = 0; u < 4; ++u) sts128(qr + C::kRawBytes + ((u ^ swz) << 4), held[u].x, held[u].y, held[u].z, held[u].w);
#pragma unroll
            for (int u = 0; u < 4; ++u) {           // 16 elements: 16 bytes of each part
              uint32_t x[4][kQParts];
              split_e5m2(w[2 * u].x, w[2 * u].y, f, x[0]);
              split_e5m2(w[2 * u].z, w[2 * u].w, f, x[1]);
              split_e5m2(w[2 * u + 1].x, w[2 * u + 1].y, f, x[2]);
              split_e5m2(w[2 * u + 1].z, w[2 * u + 1].w, f, x[3]);
              // (D = 64: 64-byte rows, chunk u at u ^ ((row >> 1) & 3))
              const uint32_t at = D == 128 ? qr + (((4 * c + u) ^ swz) << 4) : q0 + row * 64 + ((u ^ ((row >> 1) & 3)) << 4);
#pragma unroll
              for (int k = 0; k < kQParts; ++k) {
                if (D == 128 && c == 0 && k == 1) held[u] = make_uint4(x[0][k], x[1][k], x[2][k], x[3][k]);
                else sts128(at + k * C::kRawBytes, x[0][k], x[1][k], x[2][k], x[3][k]);
              }
            }
          }
          if (!alive) break;
        }
        if (!alive) break;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_Q_READY));

        for (int i = 0; alive && i < n + lag; ++i) {
          if (i >= lag) {
          // the values of tile i - lag
          const bool full = mbar_try_wait(BAR(B_RAW_FULL + vring.slot), vring.phase);
          const bool empty = mbar_try_wait(BAR(B_KV_EMPTY + ring.slot), ring.phase ^ 1u);
          if (!__all_sync(0xffffffffu, full && empty))
            alive = wait_warp(guard, BAR(B_RAW_FULL + vring.slot), vring.phase) &&
                    wait_warp(guard, BAR(B_KV_EMPTY + ring.slot), ring.phase ^ 1u);
          if (!alive) break;
          // the row's scale times 2^120; above 2^127 the rest follows in a second pass (rare), where
          // what overflows in the tree's own rows becomes 0 and is noted for the epilogue
          const int byte = lag == 1 ? vm1 : vm2, low = min(byte, 134);
          const uint32_t f = (uint32_t)(low + 120) * 0x00800080u;
          const uint32_t src = sbase + C::kOffRaw + vring.slot * C::kRawBytes + row * D;
          const uint32_t dst = sbase + C::kOffKV + ring.slot * C::kTileBytes + row * 128;
          const int t = (p.t0 + i - lag) * kTile + row;
          const bool zero = t >= T;                 // values behind the tree: 0
          uint32_t nan = 0u;
          // 16-byte chunk c of the row at its XOR-permuted turn: no bank conflicts, for the
          // reads (rows D bytes apart) nor for the swizzled writes.  Two chunks are read before
          // the first is widened: one warp a scheduler has to hide its own latencies.
#pragma unroll 1
          for (int k2 = 0; k2 < D / 16; k2 += 2) {
            uint4 w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              w[k] = lds128(src + 16 * ((k2 + k) ^ (D == 128 ? swz : swz & 3)));
              if (zero) w[k] = make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int c = (k2 + k) ^ (D == 128 ? swz : swz & 3);
              const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
              uint32_t y[8];
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                const uint2 z = spread4(u[m]);
                nan |= has_nan_code(u[m]);
                y[2 * m] = mul_bf16x2(z.x, f);
                y[2 * m + 1] = mul_bf16x2(z.y, f);
              }
              const uint32_t half = dst + (c >> 2) * C::kChunk;
              const int j = (2 * c) & 7;
              sts128(half + ((j ^ swz) << 4), y[0], y[1], y[2], y[3]);
              sts128(half + (((j + 1) ^ swz) << 4), y[4], y[5], y[6], y[7]);
            }
          }
          if (byte > low) {
            const uint32_t f2 = (uint32_t)(byte - low + 127) * 0x00800080u;
#pragma unroll 1
            for (int c = 0; c < D / 8; ++c) {
              const uint32_t addr = dst + (c >> 3) * C::kChunk + (((c & 7) ^ swz) << 4);
              uint4 x = lds128(addr);
              x = make_uint4(mul_bf16x2(x.x, f2), mul_bf16x2(x.y, f2), mul_bf16x2(x.z, f2), mul_bf16x2(x.w, f2));
              if (t >= p.L) {
                bool any = drop_nonfinite(x.x);
                any |= drop_nonfinite(x.y);
                any |= drop_nonfinite(x.z);
                any |= drop_nonfinite(x.w);
                if (any) atomicOr(&nf[(t - p.L) >> 5], 1u << ((t - p.L) & 31));
              }
              sts128(addr, x.x, x.y, x.z, x.w);
            }
          }
          // NaN in the tree's own rows becomes 0, noted for the epilogue
          if (nan & 0x80808080u) {
            const bool drop = t >= p.L;
            put_nan<D, C::kChunk>(src, dst, swz, drop);
            if (drop) atomicOr(&nf[(t - p.L) >> 5], 1u << ((t - p.L) & 31));
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(BAR(B_KV_FULL + ring.slot));
            mbar_arrive(BAR(B_RAW_EMPTY + vring.slot));
          }
          vring.next();
          ring.next();
          }
          // Tile i's key scales, for the softmax: after the values, because the place is that of
          // tile i - 2, whose softmax may still be at work while its values are widened.  (Only tile i's
          // softmax waits for them: as part of the key entry they held tile i - 2's products back.)
          if (i < n) {
            alive = wait_warp(guard, BAR(B_SCALE_FREE + sring.slot), sring.phase ^ 1u);
            if (!alive) break;
            scales[sring.slot * kTile + row] = scale_of_byte(k0) * (1.f / (1 << kBack));
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(B_SCALE_FULL + sring.slot));
            sring.next();
          }
          k0 = k1;
          vm2 = vm1;
          vm1 = v0;
          v0 = v1;
          at = row_of_scale(page_next);
          k1 = ks[at];
          v1 = vs[at];
          page_next = next_page();
        }
      } else {
        const int from = max(p.t0, p.L / kTile);          // the first key tile that reaches past the prefix
        for (int kt = from; alive && kt < p.t1; ++kt) {
          const int i = kt - p.t0, slot = (g + i + min(n, i + lag)) % C::kSlots;
          alive = wait_warp(guard, BAR(B_TAIL + slot), (tail_phase >> slot) & 1);
          if (!alive) break;
          tail_phase ^= 1u << slot;
          const int t = kt * kTile + row;
          if (t >= p.L) {
            const uint32_t dst = sbase + C::kOffKV + slot * C::kTileBytes + row * 128;
            bool found = false;
#pragma unroll 2
            for (int k = 0; k < D / 8; ++k) {
              const uint32_t addr = dst + (k >> 3) * C::kChunk + (((k & 7) ^ swz) << 4);
              if (t >= T) {
                sts128(addr, 0u, 0u, 0u, 0u);
              } else {
                uint4 w = lds128(addr);
                bool any = drop_nonfinite(w.x);
                any |= drop_nonfinite(w.y);
                any |= drop_nonfinite(w.z);
                any |= drop_nonfinite(w.w);
                if (any) sts128(addr, w.x, w.y, w.z, w.w);
                found |= any;
              }
            }
            if (found) atomicOr(&nf[(t - p.L) >> 5], 1u << ((t - p.L) & 31));
          }
          fence_async_smem();
          alive = meet();
          if (!alive) break;
          if (row == 0) mbar_arrive(BAR(B_KV_FULL + slot));
        }
        g += 2 * n;
      }
    }
  } else {
    if constexpr (!kFp8) reg_grow<kRegsSoftmax>();
    // ---- softmax and epilogue: thread = row 32 q + lane of stream s -----------------------------
    const int s = warp >> 2, q = warp & 3, r = 32 * q + lane;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const uint32_t tS = tmem + lanes + C::kColS + kTile * s, tO = tmem + lanes + C::kColO + D * s;
    const float sl2 = a.scale * 1.4426950408889634f;      // base-2 exponentials
    const int r_node = (int)divide(r, a.by_G), r_head = r - r_node * a.G;
    Piece p;
    bool alive = true;
    uint32_t s_phase = 0u, o_phase = 0u, one_pieces = 0u;
    int k_tiles = 0;                              // of the pieces before: the parity of their scales' places
    for (int index = 0; alive && get_piece(index, p); ++index) {
      const int n = p.t1 - p.t0, kvh = p.kvh;
      const bool two = p.two();
      const int node = p.node0 + (two && s ? a.npt : 0) + r_node;
      const bool valid = r_node < a.npt && node < p.n;
      uint32_t path[4] = {0u, 0u, 0u, 0u};
      bool dead = false;
      if (valid && p.tail()) {
        dead = !gqa_path(a, p.b, node, path);
        if (dead) gqa_error(a, KDTV_ERR_BAD_TREE);
      }
      const bool any_valid = __any_sync(0xffffffffu, valid);
      // One-byte keys: the row's queries were scaled by 2^k (the four warps found the same k in
      // their copy of the row)
      float row_scale = sl2;
      if constexpr (kFp8) {
        uint32_t mxb = 0u;
        if (valid) {
          const uint4* qrow = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
              (((long long)p.b * a.N + node) * a.H + (long long)kvh * a.G + r_head) * D);
#pragma unroll 4
          for (int u = 0; u < D / 8; ++u) {
            const uint4 w = qrow[u];
            mxb = max_finite(w.w, max_finite(w.z, max_finite(w.y, max_finite(w.x, mxb))));
          }
        }
        row_scale *= __uint_as_float((uint32_t)(127 + kBack - q_exponent(mxb)) << 23);
      }
      float m = -INFINITY, l = 0.f;
      bool first = true, o1_check = s == 1 && one_pieces > 0;
      for (int i = two ? 0 : s; i < n; i += two ? 1 : 2) {
        const int t0 = (p.t0 + i) * kTile;
        alive = wait_warp(guard, BAR(B_S_FULL + s), s_phase & 1);
        ++s_phase;
        if (!alive) break;
        if constexpr (kFp8) {                    // the tile's key scales
          alive = wait_warp(guard, BAR(B_SCALE_FULL + ((k_tiles + i) & 1)), ((k_tiles + i) >> 1) & 1);
          if (!alive) break;
        }
        if (!any_valid) {                        // no row of this warp is written: its weights may be anything
          if (o1_check) {
            o1_check = false;
            alive = wait_warp(guard, BAR(B_O1_FREE), (one_pieces - 1) & 1);
            if (!alive) break;
          }
          if (lane == 0) {
            if constexpr (kFp8)
              for (int k = 0; k < (two ? 1 : 2); ++k) mbar_arrive(BAR(B_SCALE_FREE + ((k_tiles + i) & 1)));
            mbar_arrive(BAR(B_P_HALF + s));
            mbar_arrive(BAR(B_P_READY + s));
          }
          __syncwarp();
          continue;
        }
        tc_fence_after();
        const bool masked = t0 + kTile > p.L;
        // bf16 keys: a row's 128 scores stay in registers.  One-byte keys: two passes over them, a
        // chunk at a time; this instance has more roles at work, and their loops together must stay
        // in the SM's instruction cache.
        float v[kFp8 ? 32 : kTile];
        auto load_chunk = [&](int c) {
          tmem_ld32(tS + 32 * c, reinterpret_cast<float(&)[32]>(v[0]));
          tmem_wait_ld();
          pin(v);
          const uint32_t at = sbase + C::kOffScale + ((k_tiles + i) & 1) * (kTile * 4) + c * (32 * 4);
#pragma unroll
          for (int k = 0; k < 32; k += 4) {   // a column's power of two, one for all rows
            const uint4 f = lds128(at + 4 * k);
            const float2 x = mul2(make_float2(v[k], v[k + 1]), make_float2(__uint_as_float(f.x), __uint_as_float(f.y)));
            const float2 y = mul2(make_float2(v[k + 2], v[k + 3]), make_float2(__uint_as_float(f.z), __uint_as_float(f.w)));
            v[k] = x.x; v[k + 1] = x.y; v[k + 2] = y.x; v[k + 3] = y.y;
          }
          if (masked) {                          // dropped, whatever it is: a masked score may be NaN
            const uint32_t see = gqa_visible(path, t0 + 32 * c, p.L);
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = (see >> k) & 1u ? v[k] : -INFINITY;
          }
        };
        float mx = -INFINITY;
        if constexpr (kFp8) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            load_chunk(c);
            float mc[4] = {mx, v[0], v[1], v[2]};
#pragma unroll
            for (int k = 3; k + 1 < 32; k += 2) mc[(k / 2) & 3] = max3(mc[(k / 2) & 3], v[k], v[k + 1]);
            mx = max3(max3(mc[0], mc[1], mc[2]), mc[3], v[31]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, reinterpret_cast<float(&)[32]>(v[32 * c]));
          tmem_wait_ld();
          pin(v);
          if (masked) {                            // dropped, whatever it is: a masked score may be NaN
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t see = gqa_visible(path, t0 + 32 * c, p.L);
#pragma unroll
              for (int k = 0; k < 32; ++k) v[32 * c + k] = (see >> k) & 1u ? v[32 * c + k] : -INFINITY;
            }
          }
          float mc[8];                             // eight chains
#pragma unroll
          for (int c = 0; c < 8; ++c) mc[c] = max3(v[16 * c], v[16 * c + 1], v[16 * c + 2]);
#pragma unroll
          for (int k = 3; k < 15; k += 2)
#pragma unroll
            for (int c = 0; c < 8; ++c) mc[c] = max3(mc[c], v[16 * c + k], v[16 * c + k + 1]);
#pragma unroll
          for (int c = 0; c < 8; ++c) mc[c] = fmaxf(mc[c], v[16 * c + 15]);
          mx = max3(max3(mc[0], mc[1], mc[2]), max3(mc[3], mc[4], mc[5]), fmaxf(mc[6], mc[7]));
        }
        mx *= row_scale;
        // The reference maximum moves only when the tile's is over 2^8 above it: a weight
        // stays below 2^8, and O is rescaled rarely.  O is at rest: the commit that made these
        // scores visible came after this stream's previous P.V.
        float alpha = 1.f;
        if (mx > m + 8.f) {
          if (m != -INFINITY) alpha = ex2(m - mx);
          m = mx;
        }
        if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
          l *= alpha;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float v[32];
            tmem_ld32(tO + 32 * c, v);
            tmem_wait_ld();
            pin(v);
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] *= alpha;
            tmem_st32(tO + 32 * c, v);
          }
        }
        first = false;
        const float ref = m == -INFINITY ? 0.f : -m;
        const float2 scale2 = make_float2(row_scale, row_scale), ref2 = make_float2(ref, ref);
        float2 sum[4] = {};
        if (o1_check) {
          // stream 1's accumulator: stream 0's warps must have merged the last one-tile piece
          o1_check = false;
          alive = wait_warp(guard, BAR(B_O1_FREE), (one_pieces - 1) & 1);
          if (!alive) break;
        }
        auto weights = [&](const float (&x32)[32], int c) {   // of 32 columns, over scores that are read already
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float2 x = fma2(make_float2(x32[k], x32[k + 1]), scale2, ref2);
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            sum[(k / 2) & 3] = add2(sum[(k / 2) & 3], x);
            w[k / 2] = pack_bf16x2(x.x, x.y);    // bf16: the tensor cores' operand type
          }
          tmem_st16u(tS + 16 * c, w);
        };
        auto half_ready = [&]() {                // half of the keys: their products may start
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(B_P_HALF + s));
        };
        if constexpr (kFp8) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            load_chunk(c);
            weights(reinterpret_cast<const float(&)[32]>(v[0]), c);
            if (c == 1) half_ready();
          }
          if (lane == 0)                         // the scales' place: two streams arrive, or one twice
            for (int k = 0; k < (two ? 1 : 2); ++k) mbar_arrive(BAR(B_SCALE_FREE + ((k_tiles + i) & 1)));
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            weights(reinterpret_cast<const float(&)[32]>(v[32 * c]), c);
            if (c == 1) half_ready();
          }
        }
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += sum[0].x + sum[0].y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_P_READY + s));
      }
      if (!alive) break;
      k_tiles += n;

      // ---- the end of the piece ---------------------------------------------------------------
      const bool mine = two || n > s;              // this stream had a tile
      if (mine) {
        alive = wait_warp(guard, BAR(B_O_FULL + s), o_phase & 1);
        ++o_phase;
        if (!alive) break;
        tc_fence_after();
      }
      if (!two && s == 1) {
        if (o1_check) {                            // no tile of its own: not waited for above
          alive = wait_warp(guard, BAR(B_O1_FREE), (one_pieces - 1) & 1);
          if (!alive) break;
        }
        ml1[r] = make_float2(m, l);
        __syncwarp();
        tc_fence_before();
        if (lane == 0) mbar_arrive(BAR(B_ML));
        ++one_pieces;
      } else {
        float w0 = 1.f, w1 = 0.f;
        bool merge = false;
        if (!two) {
          alive = wait_warp(guard, BAR(B_ML), one_pieces & 1);
          if (!alive) break;
          tc_fence_after();
          const float2 o = ml1[r];
          merge = n > 1;
          if (merge) {
            const float mm = fmaxf(m, o.x), ref = mm == -INFINITY ? 0.f : mm;
            w0 = ex2(m - ref);
            w1 = ex2(o.x - ref);
            l = l * w0 + o.y * w1;
            m = mm;
          }
        }
        const bool bad = bad_page[index % kPieces] != 0u;
        const bool whole = p.whole();
        const bool write = valid && !bad && !dead;
        const float inv = 1.f / l;
        const long long orow = ((long long)p.b * a.N + node) * a.H + (long long)kvh * a.G + r_head;
        const long long slot = 2ll * blockIdx.x + p.later();
        const long long block = slot * 2 + (two ? s : 0);   // of 128 partial rows
        const long long prow = block * kTile + r;
        float* part = a.part_o + (block * (D / 8) * kTile + r) * 8;
        if (!whole && valid) a.part_ml[prow] = make_float2(m, write ? l : -1.f);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float v[32];
          __syncwarp();                            // lanes without a row to write rejoin
          tmem_ld32(tO + 32 * c, v);
          tmem_wait_ld();
          pin(v);
          if (merge) {
            float u[32];
            tmem_ld32(tO + D + 32 * c, u);
            tmem_wait_ld();
            pin(u);
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = v[k] * w0 + u[k] * w1;
          }
          if (!write) continue;
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + orow * D + 32 * c);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[k] = make_uint4(pack_bf16x2(v[8 * k] * inv, v[8 * k + 1] * inv),
                                  pack_bf16x2(v[8 * k + 2] * inv, v[8 * k + 3] * inv),
                                  pack_bf16x2(v[8 * k + 4] * inv, v[8 * k + 5] * inv),
                                  pack_bf16x2(v[8 * k + 6] * inv, v[8 * k + 7] * inv));
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              store8(part + (4 * c + k) * (kTile * 8), reinterpret_cast<const float(&)[8]>(v[8 * k]));
          }
        }
        if (write && p.tail()) {
          const uint4 nf = nonfinite[index % kPieces];
          uint32_t x[4] = {nf.x & path[0], nf.y & path[1], nf.z & path[2], nf.w & path[3]};
          if (x[0] | x[1] | x[2] | x[3]) {
#pragma unroll 1
            for (int j = 0; j < p.n; ++j) {
              const uint32_t word = j < 32 ? x[0] : j < 64 ? x[1] : j < 96 ? x[2] : x[3];
              if (!((word >> (j & 31)) & 1u)) continue;
              if (whole) add_nonfinite<D, kFp8>(a, p.b, kvh, p.L + j, static_cast<__nv_bfloat16*>(a.out) + orow * D, 8);
              else add_nonfinite<D, kFp8>(a, p.b, kvh, p.L + j, part, kTile * 8);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (!two) {
          ++one_pieces;
          if (lane == 0) mbar_arrive(BAR(B_O1_FREE));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

// ---- combine --------------------------------------------------------------------------------
// Output rows of items that were cut into pieces: the pieces' sums and outputs
// meet at their common maximum.  Item [S, S + nt) was cut at the multiples of W;
// a CTA's piece that starts its range is partial 2 cta, one that starts later
// 2 cta + 1.  W and the requests' first units were left by the attention kernel.
// Partial rows lie [block of 128 rows][D / 8][row][8 elements], so that the
// attention warps, a row per lane, write whole lines (row by row, the 32 lines
// of a store took 4 us at the end of a call).  Here a warp takes 64 columns of
// four rows, whose eight elements of a column are a line too; lane (column / 8 %
// 4, row, half).
// Latency bound: the first pieces' rows are loaded along with their {max, sum}.
// (Rows of a CTA, pieces under way together, one token and 8 trees of 32 nodes: 16, 4: 13.6 and 43.8
// us; 16, 8: 14.0 and 45.0; 8, 4: 14.8 and 43.1; 32, 4: 14.4 and 43.8.)
constexpr int kRowsCombine = 16, kInFlight = 4;
__host__ __device__ constexpr int combine_threads(int d) { return kRowsCombine / 4 * 32 * (d / 64); }

template <int D>
__global__ void __launch_bounds__(combine_threads(D)) gqa_combine_kernel(const __grid_constant__ GqaArgs a) {
  const int b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = (int)divide(blockIdx.x, a.by_tiles), tile = blockIdx.x - kvh * a.tiles;
  const int r0 = blockIdx.y * kRowsCombine + warp / (D / 64) * 4;
  int L, n;
  gqa_request(a, b, &L, &n);
  const int rows = min(a.npt, n - tile * a.npt) * a.G;           // of the tile
  const int hb = (int)divide(kvh, a.by_hg), head = kvh - hb * a.hg;
  // The partials and the plan are written.  (Blocks without rows wait as well: what comes next in
  // the stream may start when this grid has ended.)
  grid_dep_wait();
  if (r0 >= rows) return;
  // (a wait that ran out: some partials were never written.  Its code replaces any other, and no other
  // replaces it.)
  if (*reinterpret_cast<volatile unsigned int*>(a.status) == KDTV_ERR_DEVICE_TIMEOUT) return;
  const int W = a.plan[0], nt = key_tiles(L, n);
  const int start = a.plan[1 + b] + (hb * row_pairs(a, n) + tile / 2) * nt;
  const int c0 = start / W, count = (start + nt - 1) / W - c0 + 1;
  if (count == 1) return;                          // whole: written by its CTA
  const bool later = start != c0 * W;              // of the first piece; the others start their CTA's range
  auto block = [&](int k) {                        // 128 partial rows of piece k
    return (2ll * ((c0 + k) * a.hg + head) + (k == 0 && later)) * 2 + (tile & 1);
  };
  constexpr int T = 2;                             // fours of elements per lane
  const int sub = (lane >> 1) & 3, r = r0 + sub, column = warp % (D / 64) * 64 + (lane >> 3) * 8, half = (lane & 1) * 4;
  const bool live = r < rows, ml_live = lane < 4 * kInFlight && r0 + (lane & 3) < rows;
  // lanes 4 k + i < 16: piece k of row r0 + i
  float m2 = -INFINITY, l2 = 0.f, m = -INFINITY, o[4 * T];
  bool skip = false;
#pragma unroll
  for (int k = 0; k < 4 * T; ++k) o[k] = 0.f;
#pragma unroll 1
  for (int base = 0; base < count; base += kInFlight) {   // a running maximum over these
    float4 x[kInFlight][T];
    const float2 ml = ml_live && base + (lane >> 2) < count
                          ? a.part_ml[block(base + (lane >> 2)) * kTile + r0 + (lane & 3)] : make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int k = 0; k < kInFlight; ++k)
      if (live && base + k < count) {
        const float* src = a.part_o + (block(base + k) * (D / 8) * kTile + r) * 8 + half;
#pragma unroll
        for (int t = 0; t < T; ++t)
          x[k][t] = *reinterpret_cast<const float4*>(src + (4 * t + column / 8) * (kTile * 8));
      }
    skip |= ml.y < 0.f;
    float mx = ml.x;
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
    mx = fmaxf(m2, mx);
    const float ref2 = mx == -INFINITY ? 0.f : mx, weight = ex2(ml.x - ref2);
    l2 = l2 * ex2(m2 - ref2) + ml.y * weight;      // lanes hold parts of the sum
    m2 = mx;
    const float mo = __shfl_sync(0xffffffffu, mx, sub), ref = mo == -INFINITY ? 0.f : mo, alpha = ex2(m - ref);
    m = mo;
#pragma unroll
    for (int k = 0; k < 4 * T; ++k) o[k] *= alpha;
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const float w = __shfl_sync(0xffffffffu, weight, 4 * k + sub);
      if (base + k < count)
#pragma unroll
        for (int t = 0; t < T; ++t) {
          o[4 * t] = fmaf(x[k][t].x, w, o[4 * t]);
          o[4 * t + 1] = fmaf(x[k][t].y, w, o[4 * t + 1]);
          o[4 * t + 2] = fmaf(x[k][t].z, w, o[4 * t + 2]);
          o[4 * t + 3] = fmaf(x[k][t].w, w, o[4 * t + 3]);
        }
    }
  }
  l2 += __shfl_xor_sync(0xffffffffu, l2, 4);
  l2 += __shfl_xor_sync(0xffffffffu, l2, 8);
  const float inv = 1.f / __shfl_sync(0xffffffffu, l2, sub);
  const uint32_t dropped = __ballot_sync(0xffffffffu, skip);
  if (!live || (dropped & (0x1111u << sub))) return;
  const int i = (int)divide(r, a.by_G), node = tile * a.npt + i, h = kvh * a.G + r - i * a.G;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (((long long)b * a.N + node) * a.H + h) * D + column + half;
#pragma unroll
  for (int t = 0; t < T; ++t)
    *reinterpret_cast<uint2*>(dst + 32 * t) = make_uint2(pack_bf16x2(o[4 * t] * inv, o[4 * t + 1] * inv),
                                                         pack_bf16x2(o[4 * t + 2] * inv, o[4 * t + 3] * inv));
}

template <int D, bool kFp8>
int launch_t(const GqaArgs& a, bool stall, cudaStream_t st) {
  using C = Cfg<D, kFp8>;
  CUtensorMap tq, tk, tv;
  {
    // Q: [B * N, H, d]; a box is the G heads of npt nodes, 64 columns
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.H, (uint64_t)a.B * a.N};
    const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)a.H * D * 2};
    const uint32_t box[3] = {64, (uint32_t)a.G, (uint32_t)a.npt};
    if (encode_nd(&tq, a.q, 3, dims, strides, box, 2, 128) != CUDA_SUCCESS) return KDTV_ERR_CUDA;
  }
  const uint64_t es = kFp8 ? 1 : 2;
  const uint64_t rows = a.page_size ? a.page_size : a.t_stride, blocks = a.page_size ? a.num_pages : a.B;
  const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.Hkv, rows, blocks};
  const uint64_t strides[3] = {D * es, (uint64_t)a.Hkv * D * es, rows * a.Hkv * D * es};
  const uint32_t box[4] = {kFp8 ? (uint32_t)D : 64u, 1u, a.page_size ? (uint32_t)a.page_size : (uint32_t)kTile, 1u};
  if (encode_nd(&tk, a.k, 4, dims, strides, box, (int)es, kFp8 && D == 64 ? 64 : 128) != CUDA_SUCCESS ||
      encode_nd(&tv, a.v, 4, dims, strides, box, (int)es, kFp8 ? 0 : 128) != CUDA_SUCCESS)
    return KDTV_ERR_CUDA;
  const auto kern = gqa_tc_kernel<D, kFp8>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
    return KDTV_ERR_CUDA;
  if (launch_ex(kern, dim3((unsigned)(a.groups * a.hg)), dim3(kThreads), C::kSmem, st, false, tq, tk, tv, a, stall ? 1 : 0) !=
      cudaSuccess)
    return KDTV_ERR_CUDA;
  const int most = (a.N < a.npt ? a.N : a.npt) * a.G;          // rows of a tile
  const dim3 grid((unsigned)(a.Hkv * a.tiles), (unsigned)((most + kRowsCombine - 1) / kRowsCombine), (unsigned)a.B);
  if (launch_ex(gqa_combine_kernel<D>, grid, dim3(combine_threads(D)), 0, st, true, a) != cudaSuccess)
    return KDTV_ERR_CUDA;
  return KDTV_OK;
}

}  // namespace

// Wherever these shapes allow it: from one node over 32 keys (9.1 us, CUDA cores 15.0; one byte 12.5,
// 16.8) and 1024 requests of 64 keys (301, 359; 451, 479) to 256 requests of 1024 (191, 1003; 275,
// 1463) the CUDA cores were never ahead.
int gqa_tc_supported(const kdtv_gqa_dims* d) {
  if (d->dtype != KDTV_BF16 && d->dtype != KDTV_BF16_FP8KV) return 0;
  if (d->d != 64 && d->d != 128) return 0;
  if (d->H / d->H_kv > kTile) return 0;
  const int ps = d->page_size;
  return ps == 0 || ps == 16 || ps == 32 || ps == 64 || ps == 128;
}

size_t gqa_tc_workspace(const kdtv_gqa_dims* d, int sms, GqaArgs* a) {
  a->npt = kTile / a->G;
  a->page_shift = 0;
  while ((1 << a->page_shift) < d->page_size) ++a->page_shift;
  // heads side by side: the largest divisor of H_kv up to 8 (and the CTAs there are)
  a->hg = 8 < sms ? 8 : sms;
  while (d->H_kv % a->hg) --a->hg;
  a->groups = sms / a->hg;
  a->blocks = d->H_kv / a->hg;
  a->tiles = (d->N + a->npt - 1) / a->npt;
  a->by_hg = divisor(a->hg);
  a->by_groups = divisor(a->groups);
  a->by_pair = divisor(2 * a->npt);
  a->by_G = divisor(a->G);
  a->by_tiles = divisor(a->tiles);
  const long long cap = a->cap;
  const long long units = (long long)d->B * d->H_kv * ((d->N + 2 * a->npt - 1) / (2 * a->npt)) *
                          ((cap + kTile - 1) / kTile);
  if (units >= (1ll << 30)) return 0;               // 32-bit unit numbers
  return (size_t)2 * a->groups * a->hg * 2 * kTile;
}

int launch_gqa_tc(const GqaArgs& a, bool stall, cudaStream_t st) {
  if (a.dtype == KDTV_BF16_FP8KV)
    return a.d == 128 ? launch_t<128, true>(a, stall, st) : launch_t<64, true>(a, stall, st);
  return a.d == 128 ? launch_t<128, false>(a, stall, st) : launch_t<64, false>(a, stall, st);
}

}  // namespace kdtv
