// Rotary positions of queries, and rows written to and read back from a cache
// (rotated, quantised).  All three move each byte once, so DRAM bounds them at
// prompt sizes and launch latency at a few rows.

#include "kdtv_rope.cuh"

#include <math.h>
#include <string.h>

#include <type_traits>

namespace kdtv {
namespace {

constexpr int kThreads = 256;

// ---- rotary ---------------------------------------------------------------------------
struct RopeArgs {
  int N, H, rot_off, rot;
  int rot_items, copy_items;   // per row and head
  unsigned rot_blocks;         // blocks of rotated items; the copied ones follow
  int heads, hgroups;          // heads per thread, groups of them
  unsigned rows;               // B * N
  long long xs[3], ys[3], rs[3];
  const void* x;
  void* y;
  void* rest;
  const int32_t *prefix_len, *depth, *n_live;
};

// Thread = (row, group of heads, item); neighbouring threads hold neighbouring
// items, so a head's elements are read and written in 16-byte pieces by
// neighbouring lanes.  An item is one vector of V elements (interleaved), a
// vector and its partner rot / 2 further (half), or a vector that is only
// copied; a block has rotated or copied items, so its warps do not diverge.
// The angles of an item are computed once and serve all heads of the group; the
// loads of a batch of heads are issued before their stores, which also makes
// x == y safe: no other thread touches the item's elements.  Four blocks an SM:
// bound by DRAM at prompt sizes, and by the loads in flight.
template <typename T, int V, bool kHalf>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const __grid_constant__ kdtv_rope_table tab,
                                                           const __grid_constant__ RopeArgs a) {
  const bool copied = blockIdx.x >= a.rot_blocks;
  const unsigned t = (blockIdx.x - (copied ? a.rot_blocks : 0u)) * kThreads + threadIdx.x;   // < 2^32 (host)
  const unsigned items = (unsigned)(copied ? a.copy_items : a.rot_items);
  const int item = (int)(t % items);
  const unsigned u = t / items;
  const int hg = (int)(u % (unsigned)a.hgroups);
  const unsigned row = u / (unsigned)a.hgroups;
  if (row >= a.rows) return;
  const int b = (int)(row / (unsigned)a.N), i = (int)(row % (unsigned)a.N);
  if (i >= live_rows(a.n_live, b, a.N)) return;
  const T* x = static_cast<const T*>(a.x) + b * a.xs[0] + i * a.xs[1];
  T* y = static_cast<T*>(a.y) + b * a.ys[0] + i * a.ys[1];
  const int h0 = hg * a.heads, h1 = min(h0 + a.heads, a.H);
  if (copied) {
    constexpr int kBatch = 4;
    const int c = item * V;                             // among the elements that are copied
    const int e = c < a.rot_off ? c : c + a.rot;
    T* dst;
    long long dh;
    if (a.rest) {
      dst = static_cast<T*>(a.rest) + b * a.rs[0] + i * a.rs[1] + c;
      dh = a.rs[2];
    } else {
      dst = y + e;
      dh = a.ys[2];
    }
    for (int h = h0; h < h1; h += kBatch) {
      float v[kBatch][V];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (h + k < h1) load_v<V>(x + (h + k) * a.xs[2] + e, v[k]);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (h + k < h1) store_v<V>(dst + (h + k) * dh, v[k]);
    }
    return;
  }
  const long long pos = (long long)(a.prefix_len ? a.prefix_len[b] : 0) + (a.depth ? a.depth[row] : i);
  if (!a.rest) y += a.rot_off;
  x += a.rot_off;
  constexpr int kBatch = 2;
  if constexpr (kHalf || V == 1) {
    // u elements at e0, their partners at e1
    const int e0 = kHalf ? item * V : 2 * item;
    const int e1 = kHalf ? e0 + a.rot / 2 : e0 + 1;
    float2 cs[V];
#pragma unroll
    for (int k = 0; k < V; ++k) cs[k] = rope_cos_sin(tab.turn[item * V + k], pos, tab.amp);
    for (int h = h0; h < h1; h += kBatch) {
      float p[kBatch][V], q[kBatch][V];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (h + k < h1) {
          load_v<V>(x + (h + k) * a.xs[2] + e0, p[k]);
          load_v<V>(x + (h + k) * a.xs[2] + e1, q[k]);
        }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (h + k < h1) {
#pragma unroll
          for (int m = 0; m < V; ++m) {
            const float o = p[k][m] * cs[m].x - q[k][m] * cs[m].y;
            q[k][m] = q[k][m] * cs[m].x + p[k][m] * cs[m].y;
            p[k][m] = o;
          }
          store_v<V>(y + (h + k) * a.ys[2] + e0, p[k]);
          store_v<V>(y + (h + k) * a.ys[2] + e1, q[k]);
        }
    }
  } else {
    float2 cs[V / 2];
#pragma unroll
    for (int k = 0; k < V / 2; ++k) cs[k] = rope_cos_sin(tab.turn[item * (V / 2) + k], pos, tab.amp);
    for (int h = h0; h < h1; h += 2 * kBatch) {
      float p[2 * kBatch][V];
#pragma unroll
      for (int k = 0; k < 2 * kBatch; ++k)
        if (h + k < h1) load_v<V>(x + (h + k) * a.xs[2] + item * V, p[k]);
#pragma unroll
      for (int k = 0; k < 2 * kBatch; ++k)
        if (h + k < h1) {
#pragma unroll
          for (int m = 0; m < V / 2; ++m) {
            const float o = p[k][2 * m] * cs[m].x - p[k][2 * m + 1] * cs[m].y;
            p[k][2 * m + 1] = p[k][2 * m + 1] * cs[m].x + p[k][2 * m] * cs[m].y;
            p[k][2 * m] = o;
          }
          store_v<V>(y + (h + k) * a.ys[2] + item * V, p[k]);
        }
    }
  }
}

// ---- cache rows -------------------------------------------------------------------------
struct KvPart {
  void* cache;
  uint8_t* scale;
  const void* src;
  void* out;
  long long ss[3];
  int heads, dim, rotate, rot_off;
  int group;                   // append: lanes of one head's row (a power of two)
  Divisor by_vecs, by_dim;     // read: vectors of a row, elements of a head
};
struct KvArgs {
  int B, N, page_size, t_stride, max_pages, num_pages, parts, hgroups;
  float kv_scale, kv_inv;      // kv_inv: 1 / kv_scale if that is exact (a power of two), else 0
  Divisor by_page;
  const int32_t *prefix_len, *depth, *n_live, *page_table;
  unsigned int* status;
  KvPart part[2];
};

// Whether rows L .. L + n - 1 of request b lie in the cache and on pages in
// range; the block's threads check the pages together.  Uniform per block.
__device__ __forceinline__ bool rows_ok(const KvArgs& a, int b, int L, int n) {
  const long long cap = a.page_size ? (long long)a.max_pages * a.page_size : a.t_stride;
  if (L < 0 || (long long)L + n > cap) {
    if (threadIdx.x == 0) atomicCAS(a.status, 0u, (unsigned)KDTV_ERR_BAD_PREFIX);
    return false;
  }
  if (!a.page_size) return true;
  int bad = 0;
  for (int p = L / a.page_size + threadIdx.x; p <= (L + n - 1) / a.page_size; p += kThreads) {
    const int pg = a.page_table[(long long)b * a.max_pages + p];
    bad |= pg < 0 || pg >= a.num_pages;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) atomicCAS(a.status, 0u, (unsigned)KDTV_ERR_BAD_PAGE);
    return false;
  }
  return true;
}
__device__ __forceinline__ long long row_of(const KvArgs& a, int b, int t) {
  if (!a.page_size) return (long long)b * a.t_stride + t;
  const int p = (int)divide((unsigned)t, a.by_page);
  return (long long)a.page_table[(long long)b * a.max_pages + p] * a.page_size + (t - p * a.page_size);
}

// Largest magnitude of a lane's elements (fmaxf passes NaN by), and the largest finite one.
template <int V, int P>
__device__ __forceinline__ float max_magnitude(const float (&y)[P][V]) {
  float mx = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int k = 0; k < V; ++k) mx = fmaxf(mx, fabsf(y[p][k]));
  return mx;
}
template <int V, int P>
__device__ __forceinline__ float max_finite(const float (&y)[P][V]) {
  float mx = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int k = 0; k < V; ++k) mx = fabsf(y[p][k]) < INFINITY ? fmaxf(mx, fabsf(y[p][k])) : mx;
  return mx;
}
// The maxima of J heads over the lanes of a group (all lanes of the warp come along).
template <int J>
__device__ __forceinline__ void reduce_group(float (&mx)[J], int group) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < group)
#pragma unroll
      for (int j = 0; j < J; ++j) mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], o));
}
// The smallest e with mx <= 448 * 2^e = 1.75 * 2^(e + 8), from mx's bits.
__device__ __forceinline__ int exponent_of(float mx) {
  const uint32_t bits = __float_as_uint(mx);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return max(-117, min(119, e));
}

// A lane's elements of one head's row as they are to be rounded; mx: the row's largest finite
// magnitude.  2^-e is a power of two, so x * 2^-e loses nothing; a power also makes a code's value
// exact in bf16.
template <typename D, bool kScaled, int V, int P>
__device__ __forceinline__ void convert(const KvArgs& a, float (&y)[P][V], float mx, bool put_scale, uint8_t* scale) {
  if constexpr (sizeof(D) == 1) {
    float f = a.kv_inv;
    if constexpr (kScaled) {
      const int e = exponent_of(mx);
      f = __uint_as_float((uint32_t)(127 - e) << 23);
      if (put_scale) *scale = (uint8_t)(e + 127);
    }
    if (kScaled || f != 0.f) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int k = 0; k < V; ++k) y[p][k] *= f;
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int k = 0; k < V; ++k) y[p][k] = __fdiv_rn(y[p][k], a.kv_scale);
    }
  }
}

// Rows of a part are taken by groups of `group` lanes, a row at a time, heads
// h0 .. h1 one after the other; a block has a span of rows, so that looking its
// request up does not count.  Every lane of a warp goes through the same turns
// (shuffles).
struct Rows {
  int b, L, i0, i1, h0, h1, group;
};
__device__ __forceinline__ int partner(const KvPart& part, int rot_dim, bool half, int e) {
  // distance from element e to its rotation partner (0: not rotated)
  const int r0 = e - part.rot_off;
  if (!part.rotate || r0 < 0 || r0 >= rot_dim) return 0;
  return half ? (r0 < rot_dim / 2 ? rot_dim / 2 : -(rot_dim / 2)) : ((r0 & 1) ? -1 : 1);
}
__device__ __forceinline__ long long position(const KvArgs& a, const Rows& r, int i) {
  return (long long)r.L + (a.depth ? a.depth[(long long)r.b * a.N + i] : i);
}

enum { kPlain = 0, kHalves = 1, kPairs = 2 };          // a part's rotation

// Heads of up to 256 elements, 16-byte accesses: a lane has eight elements of a
// head.  The vectors of kBatch heads are loaded together, the next ones while
// the last are converted, and the first before the request is looked up; the
// half layout's rotation partners come from the lane that holds them; the angles
// are computed once per row.  Bound by instructions more than by DRAM at prompt
// sizes (the rotation, the search for the largest magnitude), so what a part needs
// is known at compile time: 13000 rows of 8 + 8 heads of 128 from bf16 into a
// one-byte cache take 21 us, 30 with one code for all parts; DRAM alone would
// need 12.  Three blocks an SM (two: 3 us more).
template <typename S, typename D, int kRot, bool kScaled>
__device__ __forceinline__ void append_rows(const KvArgs& a, const KvPart& part, const Rows& r, int n, int rot_dim,
                                            float amp, const uint64_t* turn_of) {
  constexpr int kWords = 8 * sizeof(S) / 16, kBatch = 4 / kWords;
  const int lane = threadIdx.x % r.group, groups = kThreads / r.group;
  const bool in_dim = lane * 8 < part.dim;
  uint4 raw[kBatch][kWords];
  auto load_heads = [&](int i, int hh) {
    const S* src = static_cast<const S*>(part.src) + r.b * part.ss[0] + i * part.ss[1] + hh * part.ss[2] + lane * 8;
    const bool row = i < r.i1 && in_dim;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
#pragma unroll
      for (int w = 0; w < kWords; ++w)
        raw[j][w] = row && hh + j < r.h1 ? reinterpret_cast<const uint4*>(src + j * part.ss[2])[w]
                                         : make_uint4(0u, 0u, 0u, 0u);
  };
  int i = r.i0 + threadIdx.x / r.group;
  load_heads(i, r.h0);
  // (every block looks the whole request up: it is written as a whole or not at all)
  if (!rows_ok(a, r.b, r.L, n)) return;
  if constexpr (kRot != kPlain) __syncthreads();      // the table
  const int mate = kRot == kPlain ? 0 : partner(part, rot_dim, kRot == kHalves, lane * 8);
  const int from = threadIdx.x % 32 + (kRot == kHalves ? mate / 8 : 0);   // lane with the partners
  long long row = i < r.i1 ? row_of(a, r.b, r.L + i) : 0;
  for (int i_turn = r.i0; i_turn < r.i1; i_turn += groups, i += groups) {
    const bool on = i < r.i1;
    D* dst = static_cast<D*>(part.cache) + row * part.heads * part.dim + lane * 8;
    uint8_t* scale = kScaled ? part.scale + row * part.heads : nullptr;
    row = i + groups < r.i1 ? row_of(a, r.b, r.L + i + groups) : 0;    // of the next turn
    float2 cs[8];                                     // (pairs: four of them)
    if (kRot != kPlain && mate != 0 && on) {
      const long long pos = position(a, r, i);
      const int r0 = lane * 8 - part.rot_off, first = kRot == kPairs ? r0 / 2 : r0 < rot_dim / 2 ? r0 : r0 - rot_dim / 2;
#pragma unroll
      for (int k = 0; k < (kRot == kPairs ? 4 : 8); ++k) {
        cs[k] = rope_cos_sin(turn_of[first + k], pos, amp);
        if (kRot == kHalves && mate < 0) cs[k].y = -cs[k].y;          // the second of its pair
      }
    }
    for (int hh = r.h0; hh < r.h1; hh += kBatch) {
      float y[kBatch][1][8], mx[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        unpack8<S>(raw[j], y[j][0]);
        if constexpr (kRot == kHalves) {
          uint4 other[kWords];
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            other[w].x = __shfl_sync(0xffffffffu, raw[j][w].x, from);
            other[w].y = __shfl_sync(0xffffffffu, raw[j][w].y, from);
            other[w].z = __shfl_sync(0xffffffffu, raw[j][w].z, from);
            other[w].w = __shfl_sync(0xffffffffu, raw[j][w].w, from);
          }
          float m[8];
          unpack8<S>(other, m);
          if (mate != 0)
#pragma unroll
            for (int k = 0; k < 8; ++k) y[j][0][k] = y[j][0][k] * cs[k].x - m[k] * cs[k].y;
        } else if (kRot == kPairs && mate != 0) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float u = y[j][0][2 * k], v = y[j][0][2 * k + 1];
            y[j][0][2 * k] = u * cs[k].x - v * cs[k].y;
            y[j][0][2 * k + 1] = v * cs[k].x + u * cs[k].y;
          }
        }
      }
      if (hh + kBatch < r.h1) load_heads(i, hh + kBatch);
      else load_heads(i + groups, r.h0);
      if constexpr (kScaled) {
        bool inf = false;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) mx[j] = max_magnitude(y[j]);
        reduce_group(mx, r.group);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) inf |= !(mx[j] < INFINITY);
        if (__any_sync(0xffffffffu, inf)) {           // rare: over the finite elements
#pragma unroll
          for (int j = 0; j < kBatch; ++j) mx[j] = max_finite(y[j]);
          reduce_group(mx, r.group);
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (hh + j < r.h1) {
          convert<D, kScaled>(a, y[j], kScaled ? mx[j] : 0.f, on && lane == 0, scale + (hh + j));
          if (on && in_dim) store_v<8>(dst + (hh + j) * part.dim, y[j][0]);
        }
    }
  }
}

// Otherwise (longer heads, P > 1; odd sizes or addresses, V = 1) one head at a
// time, the partners read again.  Lane l holds elements (p * group + l) * V + k,
// p < P, k < V, of the head.
template <typename S, typename D, int V, int P>
__device__ __forceinline__ void append_rows_any(const KvArgs& a, const KvPart& part, const Rows& r, int n, int rot_dim,
                                                bool half, float amp, const uint64_t* turn_of) {
  if (!rows_ok(a, r.b, r.L, n)) return;
  __syncthreads();                                   // the table
  const int group = r.group, lane = threadIdx.x % group, groups = kThreads / group;
  int mate[P];
#pragma unroll
  for (int p = 0; p < P; ++p) mate[p] = partner(part, rot_dim, half, (p * group + lane) * V);
  int i = r.i0 + threadIdx.x / group;
  for (int i_turn = r.i0; i_turn < r.i1; i_turn += groups, i += groups) {
    const bool on = i < r.i1;
    const long long row = on ? row_of(a, r.b, r.L + i) : 0;
    const S* src = static_cast<const S*>(part.src) + r.b * part.ss[0] + (on ? i : r.i0) * part.ss[1] + lane * V;
    D* dst = static_cast<D*>(part.cache) + row * part.heads * part.dim + lane * V;
    uint8_t* scale = part.scale ? part.scale + row * part.heads : nullptr;
    float2 cs[P][V];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (mate[p] == 0 || !on) continue;
      const int r0 = (p * group + lane) * V - part.rot_off, hd = rot_dim / 2;
      const long long pos = position(a, r, i);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if (half) cs[p][k] = rope_cos_sin(turn_of[(r0 < hd ? r0 : r0 - hd) + k], pos, amp);
        else if (V == 1 || (k & 1) == 0) cs[p][k] = rope_cos_sin(turn_of[(r0 + k) / 2], pos, amp);
        else cs[p][k] = cs[p][k - 1];
        if (mate[p] < 0 && (half || V == 1)) cs[p][k].y = -cs[p][k].y;   // the second of its pair
      }
    }
    for (int h = r.h0; h < r.h1; ++h) {
      float y[P][V];
#pragma unroll
      for (int p = 0; p < P; ++p) {
#pragma unroll
        for (int k = 0; k < V; ++k) y[p][k] = 0.f;
        const int e = p * group * V;
        if (!on || e + lane * V >= part.dim) continue;
        const S* s = src + h * part.ss[2] + e;
        load_v<V>(s, y[p]);
        if (mate[p] == 0) continue;
        if (half || V == 1) {
          float m[V];
          load_v<V>(s + mate[p], m);
#pragma unroll
          for (int k = 0; k < V; ++k) y[p][k] = y[p][k] * cs[p][k].x - m[k] * cs[p][k].y;
        } else {
#pragma unroll
          for (int k = 0; k + 1 < V; k += 2) {
            const float u = y[p][k], v = y[p][k + 1];
            y[p][k] = u * cs[p][k].x - v * cs[p][k].y;
            y[p][k + 1] = v * cs[p][k].x + u * cs[p][k].y;
          }
        }
      }
      if (part.scale) {
        float mx[1] = {max_finite(y)};
        reduce_group(mx, group);
        convert<D, true>(a, y, mx[0], on && lane == 0, scale + h);
      } else {
        convert<D, false>(a, y, 0.f, false, scale);
      }
      if (on)
#pragma unroll
        for (int p = 0; p < P; ++p)
          if ((p * group + lane) * V < part.dim) store_v<V>(dst + h * part.dim + p * group * V, y[p]);
    }
  }
}

template <typename S, typename D, int V, int P>
__global__ void __launch_bounds__(kThreads, V == 8 && P == 1 ? 3 : 1)
kv_append_kernel(const __grid_constant__ kdtv_rope_table tab, const __grid_constant__ KvArgs a, int span) {
  __shared__ uint64_t turn_of[KDTV_ROPE_MAX_DIM / 2];
  const KvPart& part = a.part[blockIdx.z];
  const int b = blockIdx.y;
  const int n = live_rows(a.n_live, b, a.N);
  const int i0 = (int)(blockIdx.x / a.hgroups) * span, i1 = min(n, i0 + span);
  const int per = (part.heads + a.hgroups - 1) / a.hgroups;
  const int h0 = (int)(blockIdx.x % a.hgroups) * per, h1 = min(h0 + per, part.heads);
  if (i0 >= i1 || h0 >= h1) return;
  const Rows r{b, a.prefix_len ? a.prefix_len[b] : 0, i0, i1, h0, h1, part.group};
  if (part.rotate)                                   // (lanes want different entries)
    for (int j = threadIdx.x; j < tab.rot_dim / 2; j += kThreads) turn_of[j] = tab.turn[j];
  const bool half = tab.layout == KDTV_ROPE_HALF;
  if constexpr (V == 8 && P == 1) {
    auto run = [&](auto scaled) {
      constexpr bool kScaled = decltype(scaled)::value;
      if (!part.rotate) append_rows<S, D, kPlain, kScaled>(a, part, r, n, 0, 1.f, turn_of);
      else if (half) append_rows<S, D, kHalves, kScaled>(a, part, r, n, tab.rot_dim, tab.amp, turn_of);
      else append_rows<S, D, kPairs, kScaled>(a, part, r, n, tab.rot_dim, tab.amp, turn_of);
    };
    if constexpr (sizeof(D) == 1) {
      if (part.scale) {
        run(std::true_type{});
        return;
      }
    }
    run(std::false_type{});
  } else {
    append_rows_any<S, D, V, P>(a, part, r, n, tab.rot_dim, half, tab.amp, turn_of);
  }
}

// A request's rows of one part are contiguous in out, and row by row in the
// cache.  A block takes a span of vectors of V elements, kBatch of them per
// thread under way together; the spans are long enough that looking the
// request up does not count, and as many as fill the SMs.
template <typename C, typename O, int V>
__global__ void __launch_bounds__(kThreads, 4) kv_read_kernel(const __grid_constant__ KvArgs a, unsigned span) {
  constexpr int kBatch = 4;
  const KvPart& part = a.part[blockIdx.z];
  const int b = blockIdx.y;
  const int n = live_rows(a.n_live, b, a.N);
  if (n == 0) return;
  const unsigned width = (unsigned)(part.heads * part.dim), vecs = width / V;
  const unsigned total = (unsigned)n * vecs, t0 = blockIdx.x * span, t1 = min(total, t0 + span);   // < 2^31 (host)
  const int L = a.prefix_len ? a.prefix_len[b] : 0;
  if (!rows_ok(a, b, L, n)) return;
  const C* cache = static_cast<const C*>(part.cache);
  O* out = static_cast<O*>(part.out) + (long long)b * a.N * width;
  for (unsigned t = t0 + threadIdx.x; t < t1; t += kBatch * kThreads) {
    // 16-byte vectors stay as they are until they are stored
    float x[kBatch][V == 16 ? 1 : V], s[kBatch];
    uint4 raw[V == 16 ? kBatch : 1];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const unsigned tk = t + k * kThreads;
      if (tk >= t1) continue;
      const unsigned i = divide(tk, part.by_vecs), c = (tk - i * vecs) * V;
      const long long row = row_of(a, b, L + (int)i);
      if constexpr (V == 16) raw[k] = *reinterpret_cast<const uint4*>(cache + row * width + c);
      else load_v<V>(cache + row * width + c, x[k]);
      s[k] = 1.f;
      if constexpr (sizeof(C) == 1)
        s[k] = part.scale ? scale_of_byte(part.scale[row * part.heads + divide(c, part.by_dim)]) : a.kv_scale;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const unsigned tk = t + k * kThreads;
      if (tk >= t1) continue;
      O* dst = out + (long long)tk * V;
      if constexpr (V == 16) {
        const uint32_t u[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float y[8];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 f = widen2(u[2 * h + j] & 0xffffu), g = widen2(u[2 * h + j] >> 16);
            y[4 * j] = f.x * s[k]; y[4 * j + 1] = f.y * s[k]; y[4 * j + 2] = g.x * s[k]; y[4 * j + 3] = g.y * s[k];
          }
          store_v<8>(dst + 8 * h, y);
        }
      } else {
        if constexpr (sizeof(C) == 1)
#pragma unroll
          for (int m = 0; m < V; ++m) x[k][m] *= s[k];
        store_v<V>(dst, x[k]);
      }
    }
  }
}

// SMs of the current device (a GB300's, where there is none).
long long sms() { return device_sm_count() > 0 ? device_sm_count() : 152; }
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool multiple(const long long (&s)[3], int v) { return s[0] % v == 0 && s[1] % v == 0 && s[2] % v == 0; }
// Element strides; {0, 0, 0} is contiguous.
void strides(const int64_t (&in)[3], long long N, long long H, long long dim, long long (&out)[3]) {
  const bool given = in[0] || in[1] || in[2];
  out[0] = given ? in[0] : N * H * dim;
  out[1] = given ? in[1] : H * dim;
  out[2] = given ? in[2] : dim;
}

template <typename T>
int launch_rope(const kdtv_rope_table& tab, RopeArgs& a, int dim, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const bool half = tab.layout == KDTV_ROPE_HALF;
  // 16-byte accesses where every address that they would have is a multiple of 16.
  bool vec = aligned(a.x, 16) && aligned(a.y, 16) && aligned(a.rest, 16) && multiple(a.xs, V) &&
             multiple(a.ys, V) && (!a.rest || multiple(a.rs, V)) && dim % V == 0 &&
             a.rot_off % V == 0 && (half ? a.rot / 2 : a.rot) % V == 0;
  const int v = vec ? V : 1;
  a.rot_items = half || !vec ? a.rot / 2 / v : a.rot / v;
  const bool in_place = a.x == a.y && !a.rest;
  a.copy_items = in_place ? 0 : (dim - a.rot) / v;
  // Heads per thread: an item's angles cost about as much as four heads' moves,
  // but threads come first.  (64 heads, 8000 rows: 4 heads 90 us, 8 82, 16 76.)
  const long long threads = (long long)a.rows * (a.rot_items + a.copy_items) * a.H;
  a.heads = 1;
  const long long enough = sms() * 1024;
  while (a.heads < 16 && a.heads < a.H && threads / (2 * a.heads) >= enough) a.heads *= 2;
  a.hgroups = (a.H + a.heads - 1) / a.heads;
  const long long per = (long long)a.rows * a.hgroups;
  const long long rot_blocks = (per * a.rot_items + kThreads - 1) / kThreads;
  const long long blocks = rot_blocks + (per * a.copy_items + kThreads - 1) / kThreads;
  if (blocks > (1ll << 32) / kThreads - 1) return KDTV_ERR_UNSUPPORTED;   // 32-bit thread indices
  a.rot_blocks = (unsigned)rot_blocks;
  auto kern = vec ? (half ? rope_kernel<T, V, true> : rope_kernel<T, V, false>)
                  : (half ? rope_kernel<T, 1, true> : rope_kernel<T, 1, false>);
  kern<<<(unsigned)blocks, kThreads, 0, st>>>(tab, a);
  return cudaGetLastError() == cudaSuccess ? KDTV_OK : KDTV_ERR_CUDA;
}

template <typename S, typename D>
cudaError_t launch_append(const kdtv_rope_table& tab, KvArgs& a, cudaStream_t st) {
  bool vec = true, wide = false;
  int heads = 1;
  for (int k = 0; k < a.parts; ++k) {
    const KvPart& p = a.part[k];
    vec = vec && aligned(p.src, 16) && aligned(p.cache, 16) && p.dim % 8 == 0 && multiple(p.ss, 8) &&
          (!p.rotate || (p.rot_off % 8 == 0 &&
                         (tab.layout == KDTV_ROPE_HALF ? tab.rot_dim / 2 : tab.rot_dim) % 8 == 0));
    wide = wide || p.dim > 256;
    heads = p.heads > heads ? p.heads : heads;
  }
  int lanes = 1;
  for (int k = 0; k < a.parts; ++k) {
    KvPart& p = a.part[k];
    p.group = 32;
    if (vec)
      while (p.group > 1 && p.group / 2 * 8 >= p.dim) p.group /= 2;
    lanes = p.group > lanes ? p.group : lanes;
  }
  // A few rows are spread over more blocks by heads; many rows get spans of them, about eight
  // blocks an SM in all.
  const int rows_turn = kThreads / lanes;                    // rows a block has at a time
  const long long n_sms = sms();
  a.hgroups = 1;
  while (2 * a.hgroups <= heads && (long long)a.B * a.N * a.hgroups * lanes < n_sms * 1024) a.hgroups *= 2;
  long long blocks = 8 * n_sms / ((long long)a.B * a.parts * a.hgroups);
  blocks = blocks < 1 ? 1 : blocks;
  const int span = (int)(((a.N + blocks - 1) / blocks + rows_turn - 1) / rows_turn * rows_turn);
  const dim3 grid((unsigned)((a.N + span - 1) / span * a.hgroups), (unsigned)a.B, (unsigned)a.parts);
  auto kern = !vec ? kv_append_kernel<S, D, 1, 16>
                   : (wide ? kv_append_kernel<S, D, 8, 2> : kv_append_kernel<S, D, 8, 1>);
  kern<<<grid, kThreads, 0, st>>>(tab, a, span);
  return cudaGetLastError();
}

template <typename C, typename O>
cudaError_t launch_read(KvArgs& a, cudaStream_t st) {
  constexpr int kWide = sizeof(C) == 1 ? 16 : 8;
  bool vec = true;
  long long width = 1;
  for (int k = 0; k < a.parts; ++k) {
    const KvPart& p = a.part[k];
    vec = vec && aligned(p.cache, 16) && aligned(p.out, 16) && p.dim % kWide == 0;
    const long long w = (long long)p.heads * p.dim;
    width = w > width ? w : width;
  }
  // Spans of at least one turn of the block's threads, else about 12 blocks an SM in all: one long
  // prefix wants fewer (65536 rows of 8 + 8 heads of 128, with 8 / 12 / 24 an SM: 71 / 73 / 74 us),
  // ragged ones more (8 of up to 8192 latent rows: 20.0 / 17.3 / 17.9).
  for (int k = 0; k < a.parts; ++k) {
    KvPart& p = a.part[k];
    p.by_vecs = divisor((unsigned)(p.heads * p.dim / (vec ? kWide : 1)));
    p.by_dim = divisor((unsigned)p.dim);
  }
  const long long total = a.N * (width / (vec ? kWide : 1)), turn = 4 * kThreads;
  long long blocks = 12 * sms() / ((long long)a.B * a.parts);
  blocks = blocks < 1 ? 1 : blocks;
  const long long span = ((total + blocks - 1) / blocks + turn - 1) / turn * turn;
  const dim3 grid((unsigned)((total + span - 1) / span), (unsigned)a.B, (unsigned)a.parts);
  auto kern = vec ? kv_read_kernel<C, O, kWide> : kv_read_kernel<C, O, 1>;
  kern<<<grid, kThreads, 0, st>>>(a, (unsigned)span);
  return cudaGetLastError();
}

// Host checks that append and read share.
int kv_args(const kdtv_kv_dims* d, const kdtv_kv_part* parts, const int32_t* page_table,
            unsigned int* status, KvArgs* a) {
  if (!d || !parts || !status) return KDTV_ERR_INVALID_ARG;
  if (d->B <= 0 || d->N <= 0 || d->parts < 1 || d->parts > 2) return KDTV_ERR_INVALID_ARG;
  if (d->dtype != KDTV_F32 && d->dtype != KDTV_BF16) return KDTV_ERR_INVALID_ARG;
  if (d->cache_dtype != KDTV_F32 && d->cache_dtype != KDTV_BF16 && d->cache_dtype != KDTV_BF16_FP8KV)
    return KDTV_ERR_INVALID_ARG;
  if (d->page_size < 0 || (d->page_size > 0) != (page_table != nullptr)) return KDTV_ERR_INVALID_ARG;
  if (d->page_size == 0 ? d->t_stride <= 0 : (d->max_pages <= 0 || d->num_pages <= 0))
    return KDTV_ERR_INVALID_ARG;
  if (d->page_size > 0 && (long long)d->max_pages * d->page_size > (1ll << 30)) return KDTV_ERR_INVALID_ARG;
  if (d->B > 65535) return KDTV_ERR_UNSUPPORTED;      // one grid row each
  memset(a, 0, sizeof(*a));
  for (int k = 0; k < d->parts; ++k) {
    const kdtv_kv_part& p = parts[k];
    if (!p.cache || p.heads <= 0 || p.dim <= 0) return KDTV_ERR_INVALID_ARG;
    if (p.scale && d->cache_dtype != KDTV_BF16_FP8KV) return KDTV_ERR_INVALID_ARG;
    if (p.dim > 512 || p.heads > (1 << 16) || (long long)d->N * p.heads * p.dim > (1ll << 31))
      return KDTV_ERR_UNSUPPORTED;                      // 32-bit indices within a request's rows
    KvPart& o = a->part[k];
    o.cache = p.cache; o.scale = p.scale; o.src = p.src; o.out = p.out;
    o.heads = p.heads; o.dim = p.dim; o.rotate = p.rotate != 0; o.rot_off = p.rot_off;
    strides(p.src_stride, d->N, p.heads, p.dim, o.ss);
  }
  a->B = d->B; a->N = d->N; a->page_size = d->page_size; a->t_stride = d->t_stride;
  a->max_pages = d->max_pages; a->num_pages = d->num_pages; a->parts = d->parts;
  a->kv_scale = d->kv_scale > 0.f ? d->kv_scale : 1.f;
  int k2;
  a->kv_inv = frexpf(a->kv_scale, &k2) == 0.5f && isnormal(1.f / a->kv_scale) ? 1.f / a->kv_scale : 0.f;
  if (d->page_size > 0) a->by_page = divisor((unsigned)d->page_size);
  a->page_table = page_table;
  a->status = status;
  return KDTV_OK;
}

bool table_ok(const kdtv_rope_table* t) {
  return t && t->rot_dim >= 2 && t->rot_dim <= KDTV_ROPE_MAX_DIM && t->rot_dim % 2 == 0 &&
         (t->layout == KDTV_ROPE_HALF || t->layout == KDTV_ROPE_INTERLEAVED);
}

}  // namespace
}  // namespace kdtv

using namespace kdtv;

extern "C" int kdtv_rope_init(const kdtv_rope_config* c, kdtv_rope_table* t) {
  if (!c || !t) return KDTV_ERR_INVALID_ARG;
  if (c->rot_dim < 2 || c->rot_dim % 2) return KDTV_ERR_INVALID_ARG;
  if (c->rot_dim > KDTV_ROPE_MAX_DIM) return KDTV_ERR_UNSUPPORTED;
  if (c->layout != KDTV_ROPE_HALF && c->layout != KDTV_ROPE_INTERLEAVED) return KDTV_ERR_INVALID_ARG;
  if (c->scaling < KDTV_ROPE_PLAIN || c->scaling > KDTV_ROPE_YARN) return KDTV_ERR_INVALID_ARG;
  if (!(c->base > 1.0) || !isfinite(c->base)) return KDTV_ERR_INVALID_ARG;
  if (c->scaling != KDTV_ROPE_PLAIN && (!(c->factor >= 1.0) || !isfinite(c->factor)))
    return KDTV_ERR_INVALID_ARG;
  const int r = c->rot_dim;
  double base = c->base, amp = 1.0, lo = 0.0, hi = 0.0;
  if (c->scaling == KDTV_ROPE_NTK) {
    if (r < 4) return KDTV_ERR_INVALID_ARG;
    base *= pow(c->factor, r / (r - 2.0));
    if (!isfinite(base)) return KDTV_ERR_INVALID_ARG;
  }
  if (c->scaling == KDTV_ROPE_YARN) {
    if (c->orig_ctx <= 0) return KDTV_ERR_INVALID_ARG;
    const double fast = c->beta_fast > 0.0 ? c->beta_fast : 32.0;
    const double slow = c->beta_slow > 0.0 ? c->beta_slow : 1.0;
    if (!(slow <= fast) || !isfinite(fast)) return KDTV_ERR_INVALID_ARG;
    // Pair j turns orig_ctx f_j / 2 pi times over the original context; the
    // pairs at which that is `fast` and `slow` bound the ramp.
    const double two_pi = 6.283185307179586;
    lo = floor(r * log(c->orig_ctx / (fast * two_pi)) / (2.0 * log(base)));
    hi = ceil(r * log(c->orig_ctx / (slow * two_pi)) / (2.0 * log(base)));
    lo = lo > 0.0 ? lo : 0.0;
    hi = hi < r - 1.0 ? hi : r - 1.0;
    amp = c->attn_factor > 0.0 ? c->attn_factor : 0.1 * log(c->factor) + 1.0;
    if (!isfinite(amp)) return KDTV_ERR_INVALID_ARG;
  }
  memset(t, 0, sizeof(*t));
  t->rot_dim = r;
  t->layout = c->layout;
  t->amp = (float)amp;
  for (int j = 0; j < r / 2; ++j) {
    double f = pow(base, -2.0 * j / r);
    if (c->scaling == KDTV_ROPE_LINEAR) f /= c->factor;
    if (c->scaling == KDTV_ROPE_YARN) {
      const double span = hi - lo > 0.001 ? hi - lo : 0.001;
      double ramp = (j - lo) / span;
      ramp = ramp < 0.0 ? 0.0 : (ramp > 1.0 ? 1.0 : ramp);
      f = f / c->factor * ramp + f * (1.0 - ramp);
    }
    // f / 2 pi < 1/6 in two doubles (1 / 2 pi is known to 2^-109), then in 2^-64 turns.
    const double inv_hi = 0.15915494309189535, inv_lo = -9.839338337591243e-18;
    const double hi_t = f * inv_hi, lo_t = fma(f, inv_hi, -hi_t) + f * inv_lo;
    t->turn[j] = (uint64_t)(hi_t * 0x1p64) + (uint64_t)(int64_t)llrint(lo_t * 0x1p64);
  }
  return KDTV_OK;
}

extern "C" int kdtv_rope(const kdtv_rope_table* t, const kdtv_rope_args* d, const void* x, void* y,
                         void* rest, const int32_t* prefix_len, const int32_t* depth,
                         const int32_t* n_live, cudaStream_t stream) {
  if (!table_ok(t) || !d || !x || !y) return KDTV_ERR_INVALID_ARG;
  if (d->B <= 0 || d->N <= 0 || d->H <= 0 || d->dim <= 0 || d->rot_off < 0 ||
      (long long)d->rot_off + t->rot_dim > d->dim)
    return KDTV_ERR_INVALID_ARG;
  if (d->dtype != KDTV_F32 && d->dtype != KDTV_BF16) return KDTV_ERR_INVALID_ARG;
  if (rest && (rest == x || rest == y || x == y)) return KDTV_ERR_INVALID_ARG;
  if (d->dim > 65536 || d->H > 65536 || (long long)d->B * d->N > 0x7fffffffll) return KDTV_ERR_UNSUPPORTED;
  RopeArgs a;
  memset(&a, 0, sizeof(a));
  a.N = d->N; a.H = d->H; a.rot_off = d->rot_off; a.rot = t->rot_dim;
  a.rows = (unsigned)((long long)d->B * d->N);
  a.x = x; a.y = y; a.rest = rest;
  a.prefix_len = prefix_len; a.depth = depth; a.n_live = n_live;
  strides(d->x_stride, d->N, d->H, d->dim, a.xs);
  strides(d->y_stride, d->N, d->H, rest ? t->rot_dim : d->dim, a.ys);
  strides(d->rest_stride, d->N, d->H, d->dim - t->rot_dim, a.rs);
  // in place is element by element: another stride would overwrite what is still to be read
  if (x == y && (a.xs[0] != a.ys[0] || a.xs[1] != a.ys[1] || a.xs[2] != a.ys[2])) return KDTV_ERR_INVALID_ARG;
  return d->dtype == KDTV_BF16 ? launch_rope<__nv_bfloat16>(*t, a, d->dim, stream)
                               : launch_rope<float>(*t, a, d->dim, stream);
}

extern "C" int kdtv_kv_append(const kdtv_kv_dims* d, const kdtv_kv_part* parts,
                              const kdtv_rope_table* rope, const int32_t* prefix_len,
                              const int32_t* depth, const int32_t* n_live,
                              const int32_t* page_table, unsigned int* status,
                              cudaStream_t stream) {
  KvArgs a;
  const int rc = kv_args(d, parts, page_table, status, &a);
  if (rc != KDTV_OK) return rc;
  kdtv_rope_table tab;
  memset(&tab, 0, sizeof(tab));
  for (int k = 0; k < a.parts; ++k) {
    const KvPart& p = a.part[k];
    if (!p.src) return KDTV_ERR_INVALID_ARG;
    if (!p.rotate) continue;
    if (!table_ok(rope) || p.rot_off < 0 || (long long)p.rot_off + rope->rot_dim > p.dim)
      return KDTV_ERR_INVALID_ARG;
    tab = *rope;
  }
  a.prefix_len = prefix_len; a.depth = depth; a.n_live = n_live;
  const bool f32 = d->dtype == KDTV_F32;
  cudaError_t e;
  if (d->cache_dtype == KDTV_F32)
    e = f32 ? launch_append<float, float>(tab, a, stream) : launch_append<__nv_bfloat16, float>(tab, a, stream);
  else if (d->cache_dtype == KDTV_BF16)
    e = f32 ? launch_append<float, __nv_bfloat16>(tab, a, stream)
            : launch_append<__nv_bfloat16, __nv_bfloat16>(tab, a, stream);
  else
    e = f32 ? launch_append<float, __nv_fp8_e4m3>(tab, a, stream)
            : launch_append<__nv_bfloat16, __nv_fp8_e4m3>(tab, a, stream);
  return e == cudaSuccess ? KDTV_OK : KDTV_ERR_CUDA;
}

extern "C" int kdtv_kv_read(const kdtv_kv_dims* d, const kdtv_kv_part* parts, const int32_t* start,
                            const int32_t* n_live, const int32_t* page_table,
                            unsigned int* status, cudaStream_t stream) {
  KvArgs a;
  const int rc = kv_args(d, parts, page_table, status, &a);
  if (rc != KDTV_OK) return rc;
  for (int k = 0; k < a.parts; ++k)
    if (!a.part[k].out) return KDTV_ERR_INVALID_ARG;
  a.prefix_len = start; a.n_live = n_live;
  const bool f32 = d->dtype == KDTV_F32;
  cudaError_t e;
  if (d->cache_dtype == KDTV_F32)
    e = f32 ? launch_read<float, float>(a, stream) : launch_read<float, __nv_bfloat16>(a, stream);
  else if (d->cache_dtype == KDTV_BF16)
    e = f32 ? launch_read<__nv_bfloat16, float>(a, stream)
            : launch_read<__nv_bfloat16, __nv_bfloat16>(a, stream);
  else
    e = f32 ? launch_read<__nv_fp8_e4m3, float>(a, stream)
            : launch_read<__nv_fp8_e4m3, __nv_bfloat16>(a, stream);
  return e == cudaSuccess ? KDTV_OK : KDTV_ERR_CUDA;
}
