// kdtv_rmsnorm: the residual's addition and the root-mean-square norm of rows,
// to the inputs' type or to E4M3 bytes with an exponent byte per 32 elements.

#include "kdtv_ptx.cuh"
#include "kdtv_rope.cuh"

#include <math.h>
#include <string.h>

namespace kdtv {
namespace {

struct NormArgs {
  unsigned rows;                 // B * N * H
  int N, dim, chunks;            // chunks of V elements in a row
  const void *x, *residual, *weight;
  void *residual_out, *y;
  uint8_t* y_scale;
  const int32_t* n_live;
  float eps, weight_offset;
  long long xs[3], rs[3], ros[3], ys[3];
  Divisor by_heads, by_N;
  int H, per_row, rows_block;    // threads of a row, rows of a block
};

// Two elements an instruction where there are eight.
template <int V>
__device__ __forceinline__ void add_v(float (&x)[V], const float (&y)[V]) {
  if constexpr (V == 1) {
    x[0] += y[0];
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      const float2 s = ptx::add2(make_float2(x[k], x[k + 1]), make_float2(y[k], y[k + 1]));
      x[k] = s.x;
      x[k + 1] = s.y;
    }
  }
}
// Eight elements to their 16-byte words (exact: they come from there).
template <typename T>
__device__ __forceinline__ void pack8(const float (&x)[8], uint4* w) {
  if constexpr (sizeof(T) == 2) {
    auto two = [](float lo, float hi) { return (__float_as_uint(lo) >> 16) | (__float_as_uint(hi) & 0xffff0000u); };
    w[0] = make_uint4(two(x[0], x[1]), two(x[2], x[3]), two(x[4], x[5]), two(x[6], x[7]));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[h] = make_uint4(__float_as_uint(x[4 * h]), __float_as_uint(x[4 * h + 1]), __float_as_uint(x[4 * h + 2]), __float_as_uint(x[4 * h + 3]));
  }
}
template <int V>
__device__ __forceinline__ void scale_v(float (&x)[V], float f) {
  if constexpr (V == 1) {
    x[0] *= f;
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      const float2 s = ptx::mul2(make_float2(x[k], x[k + 1]), make_float2(f, f));
      x[k] = s.x;
      x[k + 1] = s.y;
    }
  }
}
template <int V>
__device__ __forceinline__ void offset_v(float (&w)[V], float offset) {
#pragma unroll
  for (int k = 0; k < V; ++k) w[k] += offset;
}
// x (w + offset)
template <int V>
__device__ __forceinline__ void weigh_v(float (&x)[V], const float (&w)[V], float offset) {
  if constexpr (V == 1) {
    x[0] *= w[0] + offset;
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      const float2 s = ptx::mul2(make_float2(x[k], x[k + 1]), ptx::add2(make_float2(w[k], w[k + 1]), make_float2(offset, offset)));
      x[k] = s.x;
      x[k + 1] = s.y;
    }
  }
}
// x (r + lo) w, rounded once (not weighted: w is 1); x becomes x r rounded.  Two products' roundings are brought along.
template <int V>
__device__ __forceinline__ void product(float (&x)[V], float r, float lo, const float (&w)[V], bool weighted, float (&y)[V]) {
  if constexpr (V == 1) {
    const float t = x[0] * r, e = fmaf(x[0], lo, fmaf(x[0], r, -t));
    y[0] = weighted ? fmaf(t, w[0], e * w[0]) : t + e;
    x[0] = t;
  } else {
    const float2 r2 = make_float2(r, r), n2 = make_float2(-r, -r), lo2 = make_float2(lo, lo);
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      const float2 v = make_float2(x[k], x[k + 1]), t = ptx::mul2(v, r2);
      const float2 e = ptx::fma2(v, lo2, ptx::fma2(v, r2, ptx::mul2(v, n2)));
      const float2 f = make_float2(w[k], w[k + 1]), s = weighted ? ptx::fma2(t, f, ptx::mul2(e, f)) : ptx::add2(t, e);
      x[k] = t.x;
      x[k + 1] = t.y;
      y[k] = s.x;
      y[k + 1] = s.y;
    }
  }
}
// Sum of the squares of f x.
template <int V>
__device__ __forceinline__ float squares(const float (&x)[V], float f) {
  if constexpr (V == 1) {
    return x[0] * f * (x[0] * f);
  } else {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      const float2 v = f == 1.f ? make_float2(x[k], x[k + 1]) : ptx::mul2(make_float2(x[k], x[k + 1]), make_float2(f, f));
      sum = ptx::fma2(v, v, sum);
    }
    return sum.x + sum.y;
  }
}

// h = x + r stays in registers: x and r are read once, all of a row's loads
// are under way together, and the second pass (scale and round) reads nothing
// but the weights, which L1 or L2 holds.  A row has a part of a warp, or a
// block; a thread has CH chunks of V elements, per_row chunks apart, so that
// a warp's accesses are whole lines.
// Bound by DRAM where there are rows enough (8000 bf16 rows of 8192 with the
// residual 79 us, 6640 GB/s, to one byte 75, 6100; before its arithmetic took two
// elements an instruction and its loads waited as they lie in memory, 81 and 82), else by
// the latency of one load, one reduction and one store (one row 3.3 us).
// The statistics are fp32; y is (h * (1 / sqrt(mean + eps))) * w, each step
// rounded to fp32, and rounded once more to its type.
// kShifted: rows that start anywhere, all of a row's tensors at the same distance behind a multiple of 16 bytes: the
// chunks are those of memory, of which the first and the last may lie in the row in part.
template <typename T, typename O, int V, int CH, bool kShifted = false>
__global__ void __launch_bounds__(1024, 1) rmsnorm_kernel(const __grid_constant__ NormArgs a) {
  const int row_in = threadIdx.x / a.per_row, t = threadIdx.x - row_in * a.per_row;
  const unsigned r = blockIdx.x * (unsigned)a.rows_block + row_in;
  const unsigned bi = divide(min(r, a.rows - 1), a.by_heads), head = min(r, a.rows - 1) - bi * a.H;
  const unsigned b = divide(bi, a.by_N), i = bi - b * a.N;
  const bool live = r < a.rows && (int)i < live_rows(a.n_live, b, a.N);

  static_assert(!kShifted || (V == 8 && sizeof(O) == sizeof(T)), "whole chunks");
  const T* const xrow = static_cast<const T*>(a.x) + b * a.xs[0] + i * a.xs[1] + head * a.xs[2];
  // Elements of chunk 0 before the row; a chunk's first element; whether all of it, or of its element k, lies in the row.
  const int off = kShifted ? (int)(reinterpret_cast<uintptr_t>(xrow) % 16 / sizeof(T)) : 0;
  auto whole = [&](int at) { return !kShifted || (at * V >= off && at * V - off + V <= a.dim); };
  auto within = [&](int at, int k) { return (unsigned)(at * V - off + k) < (unsigned)a.dim; };
  // (as they lie in memory until all of them are there: half the registers)
  constexpr int kWords = V == 8 ? (int)sizeof(T) / 2 : 1;
  uint4 words[2][CH][kWords];
  float single[2][CH];
  auto load = [&](const T* p, uint4 (&w)[CH][kWords], float (&s)[CH]) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = c * a.per_row + t;
      s[c] = 0.f;
#pragma unroll
      for (int k = 0; k < kWords; ++k) w[c][k] = make_uint4(0u, 0u, 0u, 0u);
      if (!live || at >= a.chunks) continue;
      if constexpr (V == 8) {
        const T* const q = p + ((long long)at * V - off);
        if (whole(at)) {
#pragma unroll
          for (int k = 0; k < kWords; ++k) w[c][k] = reinterpret_cast<const uint4*>(q)[k];
        } else {
          float v[V];
#pragma unroll
          for (int k = 0; k < V; ++k) v[k] = within(at, k) ? to_f32(q[k]) : 0.f;
          pack8<T>(v, w[c]);
        }
      } else {
        s[c] = to_f32(p[at]);
      }
    }
  };
  auto floats = [&](const uint4 (&w)[kWords], float s, float (&x)[V]) {
    if constexpr (V == 8) unpack8<T>(w, x);
    else x[0] = s;
  };
  load(xrow, words[0], single[0]);
  if (a.residual) load(static_cast<const T*>(a.residual) + b * a.rs[0] + i * a.rs[1] + head * a.rs[2], words[1], single[1]);
  auto store = [&](auto* p, int at, const float (&x)[V]) {
    if (whole(at)) {
      store_v<V>(p + ((long long)at * V - off), x);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float one[1] = {x[k]};
        if (within(at, k)) store_v<1>(p + ((long long)at * V - off + k), one);
      }
    }
  };
  float h[CH][V];
#pragma unroll
  for (int c = 0; c < CH; ++c) floats(words[0][c], single[0][c], h[c]);
  if (a.residual) {
    T* out = static_cast<T*>(a.residual_out) + b * a.ros[0] + i * a.ros[1] + head * a.ros[2];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = c * a.per_row + t;
      float u[V];
      floats(words[1][c], single[1][c], u);
      add_v<V>(h[c], u);
      if (a.residual_out && live && at < a.chunks) store(out, at, h[c]);
    }
  }

  __shared__ float part[32];
  const int lanes = min(a.per_row, 32), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto mean_square = [&](float f) -> float {         // of the row times f
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) sum += squares<V>(h[c], f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < lanes) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (a.per_row > 32) {                             // one row in the block
      if (lane == 0) part[warp] = sum;
      __syncthreads();
      sum = lane < (int)(blockDim.x >> 5) ? part[lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    return sum / (float)a.dim;
  };
  float mean = mean_square(1.f) + a.eps, up = 1.f;
  // Squares beyond fp32's range, or too small for it: of the row times a power of two, whose square goes to eps.  Rows of
  // subnormals, whose squares are still too small then, take a second, larger one: the mean is a normal number in the end
  // (at least (2^-23)^2 / 32768), and a row of which one power makes too little is below 2^-97, so that the other makes
  // no square too large.
  float s = !(mean <= 0x1p100f) ? 0x1p-72f : mean < 0x1p-60f ? 0x1p75f : 1.f;
#pragma unroll 1
  while (__any_sync(0xffffffffu, s != up)) {          // (a row of more than a warp: the same for all of the block)
    if (a.per_row > 32) __syncthreads();              // (the last sums are read)
    mean = mean_square(s) + a.eps * s * s;
    up = s;
    if (up > 1.f && mean < 0x1p-60f) s = 0x1p126f;
  }
  float inv = 1.f / sqrtf(mean), left = 0.f;
  // One byte: what the root's reciprocal lost, by a step of Newton's method.  (Values near the middle between two codes
  // are told apart as well as fp32 sums allow: without this and the products' 298 of 441 million codes were not the
  // nearest, 220 with them, for 6 of 105 us.)
  if (sizeof(O) == 1 && mean < INFINITY && inv < INFINITY) {
    const float p = mean * inv;
    left = -0.5f * inv * fmaf(fmaf(mean, inv, -p), inv, fmaf(p, inv, -1.f));
  }
  // The power of two, to the row where the reciprocal may be more than fp32 holds; a large row's to both, since its
  // reciprocal may be subnormal: what 2^-24 makes subnormal of a row above 2^50 is 0 in the result.
  if (up < 1.f) {
    inv *= up * 0x1p24f;
    left *= up * 0x1p24f;
  }
  if (up != 1.f)
#pragma unroll
    for (int c = 0; c < CH; ++c) scale_v<V>(h[c], up < 1.f ? 0x1p-24f : up);

  const T* weight = static_cast<const T*>(a.weight);
  O* y = static_cast<O*>(a.y) + b * a.ys[0] + i * a.ys[1] + head * a.ys[2];
  uint8_t* scale = a.y_scale + (long long)min(r, a.rows - 1) * (a.dim / KDTV_GROUP);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int at = c * a.per_row + t;
    const bool on = live && at < a.chunks;
    float w[V];
#pragma unroll
    for (int k = 0; k < V; ++k) w[k] = 1.f;
    if (weight && at < a.chunks) {
      if constexpr (kShifted) {
#pragma unroll
        for (int k = 0; k < V; ++k) w[k] = within(at, k) ? to_f32(weight[at * V - off + k]) : 0.f;
      } else {
        load_v<V>(weight + at * V, w);
      }
    }
    if constexpr (sizeof(O) == 1) {                   // 32 / V lanes share an exponent
      if (weight) offset_v<V>(w, a.weight_offset);
      float z[V];
      product<V>(h[c], inv, left, w, weight != nullptr, z);
      uint32_t top = 0u;                              // (magnitudes in the order of their bits)
#pragma unroll
      for (int k = 0; k < V; ++k) top = max(top, __float_as_uint(z[k]) & 0x7fffffffu);
#pragma unroll
      for (int o = 1; o < KDTV_GROUP / V; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (__any_sync(0xffffffffu, top >= 0x7f800000u)) {        // the finite ones only
        top = 0u;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          if (!(fabsf(z[k]) < INFINITY)) z[k] = weight ? h[c][k] * w[k] : h[c][k];      // (0 times infinity was not meant)
          const uint32_t bits = __float_as_uint(z[k]) & 0x7fffffffu;
          top = max(top, bits < 0x7f800000u ? bits : 0u);
        }
#pragma unroll
        for (int o = 1; o < KDTV_GROUP / V; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      const int e = exponent_of(__uint_as_float(top));
      scale_v<V>(z, __uint_as_float((uint32_t)(127 - e) << 23));
      if (on && at % (KDTV_GROUP / V) == 0) scale[at / (KDTV_GROUP / V)] = (uint8_t)(e + 127);
      if (on) store(y, at, z);
    } else {
      scale_v<V>(h[c], inv);
      if (weight) weigh_v<V>(h[c], w, a.weight_offset);
      if (on) store(y, at, h[c]);
    }
  }
}

bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool multiple(const long long (&s)[3], int v) { return s[0] % v == 0 && s[1] % v == 0 && s[2] % v == 0; }
// (Of a dimension of one element: 0, whatever was given.)
void strides(const int64_t (&in)[3], const kdtv_norm_args& d, long long (&out)[3]) {
  const bool given = in[0] || in[1] || in[2];
  out[0] = d.B == 1 ? 0 : given ? in[0] : (long long)d.N * d.H * d.dim;
  out[1] = d.N == 1 ? 0 : given ? in[1] : (long long)d.H * d.dim;
  out[2] = d.H == 1 ? 0 : given ? in[2] : d.dim;
}
bool same(const long long (&s)[3], const long long (&t)[3]) { return s[0] == t[0] && s[1] == t[1] && s[2] == t[2]; }

template <typename T, typename O, int V, bool kShifted = false>
int launch_v(NormArgs& a, cudaStream_t st) {
  a.chunks = kShifted ? (a.dim + 16 / (int)sizeof(T) - 1 + V - 1) / V : a.dim / V;
  // Threads of a row: chunks each so that a thread has 128 bytes on their way (up to 32 where a chunk is one
  // element), or one each where the rows are too few to fill the device.  (8192 elements a row: 8000 bf16 rows with the
  // residual, to one byte, 2, 4, 8 chunks 103, 70, 76 us when products were rounded as they came (4 take 75 since),
  // without the residual -, 50, 58; 4000 fp32 rows, 2 and 4 chunks, with the residual 80 and 91, without it 56 and 46.)
  constexpr int most = V == 1 ? 32 : 4;
  const int some = V == 1 ? 8 : sizeof(T) == 4 && a.residual ? 2 : 4;
  const int least = sizeof(O) == 1 ? KDTV_GROUP / V : 1;       // lanes that share an exponent stay together
  const int sms = device_sm_count() > 0 ? device_sm_count() : 152;
  int ch = a.rows <= 2u * sms ? 1 : some;
  while ((a.chunks + ch - 1) / ch > 1024) ch *= 2;
  if (ch > most) return KDTV_ERR_UNSUPPORTED;
  int per = (a.chunks + ch - 1) / ch;
  if (per > 32) {
    per = (per + 31) / 32 * 32;
    a.rows_block = 1;
  } else {
    int p = least;
    while (p < per) p *= 2;
    per = p;
    a.rows_block = (a.rows <= 2u * sms ? 32 : 256) / per;
  }
  a.per_row = per;
  const unsigned blocks = (unsigned)((a.rows + (long long)a.rows_block - 1) / a.rows_block);
  const unsigned threads = (unsigned)(per * a.rows_block);
  auto go = [&](auto kern) {
    kern<<<blocks, threads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? KDTV_OK : KDTV_ERR_CUDA;
  };
  if constexpr (V == 1) {
    return ch <= 1 ? go(rmsnorm_kernel<T, O, 1, 1>) : ch <= 8 ? go(rmsnorm_kernel<T, O, 1, 8>) : go(rmsnorm_kernel<T, O, 1, 32>);
  } else {
    return ch == 1 ? go(rmsnorm_kernel<T, O, V, 1, kShifted>)
                   : ch == 2 ? go(rmsnorm_kernel<T, O, V, 2, kShifted>) : go(rmsnorm_kernel<T, O, V, 4, kShifted>);
  }
}

template <typename T, typename O>
int launch(NormArgs& a, cudaStream_t st) {
  // 16-byte accesses (8-byte ones of bytes) where every address that they would have allows them.
  const int v = 16 / sizeof(T) < 8 ? 4 : 8;
  const bool vec = a.dim % 8 == 0 && aligned(a.x, 16) && aligned(a.residual, 16) && aligned(a.residual_out, 16) &&
                   aligned(a.weight, 16) && aligned(a.y, sizeof(O) == 1 ? 8 : 16) && multiple(a.xs, v) &&
                   (!a.residual || multiple(a.rs, v)) && (!a.residual_out || multiple(a.ros, v)) &&
                   multiple(a.ys, sizeof(O) == 1 ? 8 : v);
  if (vec) return launch_v<T, O, 8>(a, st);
  // Rows that start anywhere, the same distance behind 16 bytes in all tensors (8000 bf16 rows of 8190 with the residual 112 us,
  // element by element 253; 7134 of 4365 56 and 107; 12000 of 101 7.6 and 6.8).
  if constexpr (sizeof(O) == sizeof(T)) {
    auto together = [&](const void* p, const long long (&s)[3]) {
      if (!p) return true;
      bool ok = (reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(a.x)) % 16 == 0;
      for (int k = 0; k < 3; ++k) ok = ok && (s[k] - a.xs[k]) % v == 0;
      return ok;
    };
    if (a.dim >= 256 && reinterpret_cast<uintptr_t>(a.x) % sizeof(T) == 0 && together(a.residual, a.rs) &&
        together(a.residual_out, a.ros) && together(a.y, a.ys) && a.dim <= 32768 - 16)
      return launch_v<T, O, 8, true>(a, st);
  }
  return launch_v<T, O, 1>(a, st);
}

}  // namespace
}  // namespace kdtv

using namespace kdtv;

extern "C" int kdtv_rmsnorm(const kdtv_norm_args* d, const void* x, const void* residual,
                            void* residual_out, const void* weight, void* y, uint8_t* y_scale,
                            const int32_t* n_live, cudaStream_t stream) {
  if (!d || !x || !y || (residual_out && !residual)) return KDTV_ERR_INVALID_ARG;
  if (d->B <= 0 || d->N <= 0 || d->H <= 0 || d->dim <= 0) return KDTV_ERR_INVALID_ARG;
  if (d->dtype != KDTV_F32 && d->dtype != KDTV_BF16) return KDTV_ERR_INVALID_ARG;
  const bool one_byte = d->out_dtype == KDTV_BF16_FP8KV;
  if (!one_byte && d->out_dtype != d->dtype) return KDTV_ERR_INVALID_ARG;
  if (one_byte != (y_scale != nullptr) || (one_byte && d->dim % KDTV_GROUP)) return KDTV_ERR_INVALID_ARG;
  if (!(d->eps >= 0.f) || !isfinite(d->eps) || !isfinite(d->weight_offset)) return KDTV_ERR_INVALID_ARG;
  if (d->dim > 32768 || (long long)d->B * d->N * d->H > 0x7fffffffll) return KDTV_ERR_UNSUPPORTED;
  if ((const void*)y == weight || (residual_out && (residual_out == y || residual_out == weight)))
    return KDTV_ERR_INVALID_ARG;
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.rows = (unsigned)((long long)d->B * d->N * d->H);
  a.N = d->N; a.H = d->H; a.dim = d->dim;
  a.x = x; a.residual = residual; a.residual_out = residual_out; a.weight = weight;
  a.y = y; a.y_scale = y_scale; a.n_live = n_live;
  a.eps = d->eps; a.weight_offset = d->weight_offset;
  strides(d->x_stride, *d, a.xs);
  strides(d->r_stride, *d, a.rs);
  strides(d->ro_stride, *d, a.ros);
  strides(d->y_stride, *d, a.ys);
  a.by_heads = divisor((unsigned)d->H);
  a.by_N = divisor((unsigned)d->N);
  // Rows of a result over one another.
  for (const auto* s : {&a.ys, &a.ros})
    if ((d->B > 1 && !(*s)[0]) || (d->N > 1 && !(*s)[1]) || (d->H > 1 && !(*s)[2])) return KDTV_ERR_INVALID_ARG;
  // In place is element by element: other strides or element sizes would overwrite what is still to be
  // read.
  if ((const void*)y == x && (one_byte || !same(a.xs, a.ys))) return KDTV_ERR_INVALID_ARG;
  if ((const void*)y == residual && (one_byte || !same(a.rs, a.ys))) return KDTV_ERR_INVALID_ARG;
  if (residual_out && residual_out == residual && !same(a.rs, a.ros)) return KDTV_ERR_INVALID_ARG;
  if (residual_out && (const void*)residual_out == x && !same(a.xs, a.ros)) return KDTV_ERR_INVALID_ARG;
  if (d->dtype == KDTV_F32)
    return one_byte ? launch<float, __nv_fp8_e4m3>(a, stream) : launch<float, float>(a, stream);
  return one_byte ? launch<__nv_bfloat16, __nv_fp8_e4m3>(a, stream) : launch<__nv_bfloat16, __nv_bfloat16>(a, stream);
}
