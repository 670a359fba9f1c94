// Rotary angles, 16-byte accesses and divisions by what a launch knows, shared by the rotary, cache
// and GQA kernels.
#pragma once

#include "kdtv_internal.cuh"

namespace kdtv {

// cos and sin of position * f_j, times amp.  The table holds f_j / 2 pi in
// units of 2^-64 turns, so the product modulo 2^64 is the fraction of a turn:
// whole turns fall off the top and the reduction is exact for any position.
// Its upper 32 bits (2^-32 turns: 1.5e-9 of angle) split into the nearest
// quarter turn and a remainder within an eighth of a turn, pi / 4, where the
// Taylor polynomials up to x^9 and x^10 leave less than 2e-9.
__device__ __forceinline__ float2 rope_cos_sin(uint64_t turn, long long pos, float amp) {
  const uint32_t x = (uint32_t)((turn * (uint64_t)pos) >> 32);
  const uint32_t q = (x + (1u << 29)) >> 30;
  const float t = (float)(int)(x - (q << 30)) * 1.4629180792671596e-9f;   // 2 pi 2^-32
  const float z = t * t;
  const float s = fmaf(t * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), t);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f),
                                       1.f / 24.f), -0.5f), 1.f);
  const float cq = (q & 1) ? -s : c, sq = (q & 1) ? c : s;
  const float sign = (q & 2) ? -amp : amp;
  return make_float2(cq * sign, sq * sign);
}

// V elements of type T as floats: one 16-byte access (two for 8 floats), or a
// scalar for V = 1.
template <int V>
__device__ __forceinline__ void load_v(const __nv_bfloat16* p, float (&x)[V]) {
  if constexpr (V == 8) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(u[k] << 16);
      x[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) x[k] = __bfloat162float(p[k]);
  }
}
// Eight elements from their 16-byte words.
template <typename S>
__device__ __forceinline__ void unpack8(const uint4* w, float (&x)[8]) {
  if constexpr (sizeof(S) == 2) {
    const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(u[k] << 16);
      x[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x[4 * h] = __uint_as_float(w[h].x);
      x[4 * h + 1] = __uint_as_float(w[h].y);
      x[4 * h + 2] = __uint_as_float(w[h].z);
      x[4 * h + 3] = __uint_as_float(w[h].w);
    }
  }
}
template <int V>
__device__ __forceinline__ void load_v(const float* p, float (&x)[V]) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const float4 w = *reinterpret_cast<const float4*>(p + k);
      x[k] = w.x; x[k + 1] = w.y; x[k + 2] = w.z; x[k + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) x[k] = p[k];
  }
}
template <int V>
__device__ __forceinline__ void store_v(__nv_bfloat16* p, const float (&x)[V]) {
  if constexpr (V == 8) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b = __float22bfloat162_rn(make_float2(x[2 * k], x[2 * k + 1]));
      u[k] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) p[k] = __float2bfloat16_rn(x[k]);
  }
}
template <int V>
__device__ __forceinline__ void store_v(float* p, const float (&x)[V]) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int k = 0; k < V; k += 4)
      *reinterpret_cast<float4*>(p + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) p[k] = x[k];
  }
}
// E4M3 bytes (to nearest even, saturating).
template <int V>
__device__ __forceinline__ void store_v(__nv_fp8_e4m3* p, const float (&x)[V]) {
  if constexpr (V == 8) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      u[k] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * k], x[2 * k + 1]), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint2*>(p) = make_uint2(u[0] | (u[1] << 16), u[2] | (u[3] << 16));
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) p[k].__x = __nv_cvt_float_to_fp8(x[k], __NV_SATFINITE, __NV_E4M3);
  }
}
// Two E4M3 bytes (the low 16 bits) as floats.
__device__ __forceinline__ float2 widen2(uint32_t two) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)));
}
// (16 bytes at a time are widened by their reader.)
template <int V>
__device__ __forceinline__ void load_v(const __nv_fp8_e4m3* p, float (&x)[V]) {
  static_assert(V == 1, "one byte");
  x[0] = to_f32(*p);
}

// n / d for 0 <= n < 2^31 by a multiplication: with 2^(s-1) < d <= 2^s and
// m = floor(2^32 (2^s - d) / d) + 1 the quotient is (n + floor(m n / 2^32)) >> s
// (Granlund and Montgomery, 1994).
struct Divisor {
  uint32_t m, s;
};
inline Divisor divisor(uint32_t d) {
  Divisor r{0u, 0u};
  while ((1ull << r.s) < d) ++r.s;
  r.m = (uint32_t)((((1ull << r.s) - d) << 32) / d + 1);
  return r;
}
__device__ __forceinline__ unsigned divide(unsigned n, Divisor d) { return (n + __umulhi(n, d.m)) >> d.s; }

// Live rows of request b.
__device__ __forceinline__ int live_rows(const int32_t* n_live, int b, int N) {
  if (!n_live) return N;
  const int n = n_live[b];
  return n < 0 ? 0 : (n > N ? N : n);
}
// The smallest e with mx <= 448 * 2^e = 1.75 * 2^(e + 8), from mx's bits.
__device__ __forceinline__ int exponent_of(float mx) {
  const uint32_t bits = __float_as_uint(mx);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return max(-117, min(119, e));
}
// Value of exponent byte e + 127 (2^e, e in [-126, 127]).
__device__ __forceinline__ float scale_of_byte(unsigned int byte) {
  return __uint_as_float(byte << 23);
}

}  // namespace kdtv
