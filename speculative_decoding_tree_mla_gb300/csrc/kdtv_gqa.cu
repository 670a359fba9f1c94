// kdtv_gqa_verify_attn: tree-verify attention over a cache of keys and values
// per head.  Host side, and the CUDA-core path (fp32, and what the tensor
// cores do not take).

#include "kdtv_gqa.cuh"
#include "kdtv_ptx.cuh"

#include <math.h>
#include <string.h>

namespace kdtv {
namespace {

// ---- CUDA cores -----------------------------------------------------------------------
// A CTA of 4 warps takes 16 rows of one key/value head and one split of the
// keys, 32 keys at a time: K and V staged in shared memory as fp32 (a warp per
// key row, rows padded with zeros to dp = 8 ceil(d / 8) elements and set 16
// bytes apart from a multiple of the banks), each warp four rows.  Scores: a
// lane per key, four elements an access, four rows share each K access.
// Softmax: online, across the lanes.  Output: a lane holds elements lane + 32 k
// of the four rows; four rows' weights of a key are one 16-byte read.  Bound by
// the fp32 pipe and shared-memory reads; the path exists for fp32 and for head
// dims outside the tensor-core instances.
constexpr int kRowsCta = 16, kRowsWarp = 4, kKeys = 32, kSimtThreads = 128;
__host__ __device__ constexpr int simt_padded(int d) { return (d + 7) / 8 * 8; }
__host__ __device__ constexpr int simt_words(int d) {     // of shared memory
  return 2 * kKeys * (simt_padded(d) + 4) + kRowsCta * simt_padded(d) + 4 * kKeys * kRowsWarp;
}

template <typename T, typename C, int DK>     // DK = ceil(d / 32), rounded up to an instance
__global__ void __launch_bounds__(kSimtThreads) gqa_simt_kernel(const __grid_constant__ GqaArgs a) {
  extern __shared__ __align__(16) float sm[];
  const int d = a.d, dp = simt_padded(d), ld = dp + 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ptx::grid_dep_launch();          // the combine kernel may be launched; it waits for this grid
  float* ks = sm;                                  // [kKeys][ld]
  float* vs = ks + kKeys * ld;                     // [kKeys][ld]
  float* qs = vs + kKeys * ld;                     // [kRowsCta][dp]
  float4* ps = reinterpret_cast<float4*>(qs + kRowsCta * dp) + warp * kKeys;   // this warp's weights, [kKeys]
  __shared__ uint32_t s_mask[kRowsCta][4];
  __shared__ int s_dead[kRowsCta];                 // 1: not a live row, 2: malformed root path
  const int b = blockIdx.z / a.Hkv, kvh = blockIdx.z % a.Hkv;
  int L, n;
  gqa_request(a, b, &L, &n);
  const int rows = n * a.G, r0 = blockIdx.y * kRowsCta;
  if (r0 >= rows) return;
  const int T_end = L + n;
  const int t_lo = blockIdx.x * a.chunk, t_hi = min(T_end, t_lo + a.chunk);
  if (t_lo >= t_hi) return;

  if (threadIdx.x < kRowsCta) {
    const int r = r0 + threadIdx.x;
    uint32_t m[4] = {0u, 0u, 0u, 0u};
    int dead = r >= rows ? 1 : 0;
    if (!dead && !gqa_path(a, b, r / a.G, m)) {
      dead = 2;
      gqa_error(a, KDTV_ERR_BAD_TREE);
    }
    for (int w = 0; w < 4; ++w) s_mask[threadIdx.x][w] = m[w];
    s_dead[threadIdx.x] = dead;
  }
  auto out_row = [&](int r) {
    return ((long long)b * a.N + r / a.G) * a.H + (long long)kvh * a.G + r % a.G;
  };
  for (int j = warp; j < kRowsCta; j += 4) {
    const T* src = static_cast<const T*>(a.q) + out_row(min(r0 + j, rows - 1)) * d;
    for (int e = lane; e < dp; e += 32) qs[j * dp + e] = e < d ? to_f32(src[e]) : 0.f;
  }
  __syncthreads();

  const float sl2 = a.scale * 1.4426950408889634f;   // base-2 exponentials
  float m[kRowsWarp], l[kRowsWarp], o[kRowsWarp][DK];
  uint32_t mask[kRowsWarp][4];
#pragma unroll
  for (int r = 0; r < kRowsWarp; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int k = 0; k < DK; ++k) o[r][k] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) mask[r][w] = s_mask[warp * kRowsWarp + r][w];
  }
  int bad_page = 0;
  for (int t0 = t_lo; t0 < t_hi; t0 += kKeys) {
    __syncthreads();
    const int nk = min(kKeys, t_hi - t0);
#pragma unroll 1
    for (int j0 = 0; j0 < kKeys; j0 += 16) {         // a warp's four rows of these: under way together
      float kx[4][DK], vx[4][DK];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + 4 * u + warp;
        const long long row = j < nk ? gqa_row(a, b, t0 + j) : 0;
        if (row < 0) bad_page = 1;
        const bool on = j < nk && row >= 0;
        const long long at = (row * a.Hkv + kvh) * d;
        float fk = 1.f, fv = 1.f;
        if constexpr (sizeof(C) == 1) {
          if (on) {
            fk = scale_of_byte(a.k_scale[row * a.Hkv + kvh]);
            fv = scale_of_byte(a.v_scale[row * a.Hkv + kvh]);
          }
        }
#pragma unroll
        for (int k = 0; k < DK; ++k) {
          const int e = lane + 32 * k;
          kx[u][k] = on && e < d ? to_f32(static_cast<const C*>(a.k)[at + e]) : 0.f;
          vx[u][k] = on && e < d ? to_f32(static_cast<const C*>(a.v)[at + e]) : 0.f;
          if constexpr (sizeof(C) == 1) {
            kx[u][k] *= fk;
            vx[u][k] *= fv;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int k = 0; k < DK; ++k)
          if (lane + 32 * k < dp) {
            ks[(j0 + 4 * u + warp) * ld + lane + 32 * k] = kx[u][k];
            vs[(j0 + 4 * u + warp) * ld + lane + 32 * k] = vx[u][k];
          }
    }
    __syncthreads();
    float s[kRowsWarp];
#pragma unroll
    for (int r = 0; r < kRowsWarp; ++r) s[r] = 0.f;
    const float4* kr = reinterpret_cast<const float4*>(ks + lane * ld);
    const float4* qr = reinterpret_cast<const float4*>(qs + warp * kRowsWarp * dp);
#pragma unroll 4
    for (int e = 0; e < dp / 4; ++e) {
      const float4 x = kr[e];
#pragma unroll
      for (int r = 0; r < kRowsWarp; ++r) {
        const float4 y = qr[r * (dp / 4) + e];
        s[r] = fmaf(y.x, x.x, s[r]);
        s[r] = fmaf(y.y, x.y, s[r]);
        s[r] = fmaf(y.z, x.z, s[r]);
        s[r] = fmaf(y.w, x.w, s[r]);
      }
    }
    uint32_t see[kRowsWarp], any = 0u;
    float p[kRowsWarp];
#pragma unroll
    for (int r = 0; r < kRowsWarp; ++r) {
      see[r] = gqa_visible(mask[r], t0, L);
      if (nk < 32) see[r] &= (1u << nk) - 1u;
      any |= see[r];
      const float x = (see[r] >> lane) & 1u ? s[r] * sl2 : -INFINITY;
      float mx = x;
#pragma unroll
      for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[r], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;
      p[r] = gqa_ex2(x - ref);
      const float alpha = gqa_ex2(m[r] - ref);
      l[r] = l[r] * alpha + p[r];                    // lanes keep parts of the sum
      m[r] = mn;
#pragma unroll
      for (int k = 0; k < DK; ++k) o[r][k] *= alpha;
    }
    __syncwarp();
    ps[lane] = make_float4(p[0], p[1], p[2], p[3]);
    __syncwarp();
    if (t0 + kKeys <= min(L, t_hi)) {                // all rows see all keys
#pragma unroll 4
      for (int j = 0; j < kKeys; ++j) {
        const float4 w = ps[j];
#pragma unroll
        for (int k = 0; k < DK; ++k) {
          const float v = lane + 32 * k < dp ? vs[j * ld + lane + 32 * k] : 0.f;
          o[0][k] = fmaf(w.x, v, o[0][k]);
          o[1][k] = fmaf(w.y, v, o[1][k]);
          o[2][k] = fmaf(w.z, v, o[2][k]);
          o[3][k] = fmaf(w.w, v, o[3][k]);
        }
      }
      continue;
    }
    // only what a row sees: a masked value may be infinite or NaN
    while (any) {
      const int j = __ffs(any) - 1;
      any &= any - 1;
      const float4 w = ps[j];
      float v[DK];
#pragma unroll
      for (int k = 0; k < DK; ++k) v[k] = lane + 32 * k < dp ? vs[j * ld + lane + 32 * k] : 0.f;
#pragma unroll
      for (int r = 0; r < kRowsWarp; ++r)
        if ((see[r] >> j) & 1u)
#pragma unroll
          for (int k = 0; k < DK; ++k) o[r][k] = fmaf(r == 0 ? w.x : r == 1 ? w.y : r == 2 ? w.z : w.w, v[k], o[r][k]);
    }
  }
  const bool bad = __syncthreads_or(bad_page);
  if (bad && threadIdx.x == 0) gqa_error(a, KDTV_ERR_BAD_PAGE);
#pragma unroll
  for (int r = 0; r < kRowsWarp; ++r) {
#pragma unroll
    for (int w = 16; w; w >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], w);
    const int rr = r0 + warp * kRowsWarp + r;
    const int dead = s_dead[warp * kRowsWarp + r];
    if (dead == 1) continue;
    const bool skip = bad || dead == 2;
    if (a.splits == 1) {
      if (skip) continue;
#pragma unroll
      for (int k = 0; k < DK; ++k)
        if (lane + 32 * k < d) {
          const float x[1] = {o[r][k] / l[r]};
          store_v<1>(static_cast<T*>(a.out) + out_row(rr) * d + lane + 32 * k, x);
        }
    } else {
      const long long slot = ((long long)blockIdx.x * a.B * a.N) * a.H + out_row(rr);
      if (lane == 0) a.part_ml[slot] = make_float2(m[r], skip ? -1.f : l[r]);
      if (skip) continue;
#pragma unroll
      for (int k = 0; k < DK; ++k)
        if (lane + 32 * k < d) a.part_o[slot * d + lane + 32 * k] = o[r][k];
    }
  }
}

// Merges the splits of an output row; a warp per row, lane k the {max, sum} of
// splits k and k + 32, four splits' elements under way together.
template <typename T>
__global__ void __launch_bounds__(256) gqa_simt_combine_kernel(const __grid_constant__ GqaArgs a) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long all = (long long)a.B * a.N * a.H;
  int L = 0, n = 0, i = 0;
  if (row < all) {
    const int b = (int)(row / ((long long)a.N * a.H));
    i = (int)(row / a.H % a.N);
    gqa_request(a, b, &L, &n);
  }
  // (warps without a row wait as well: what comes next in the stream may start when this grid has
  // ended)
  ptx::grid_dep_wait();
  if (i >= n) return;
  const int pieces = (L + n + a.chunk - 1) / a.chunk;       // <= 64
  const float2 none = make_float2(-INFINITY, 0.f);
  const float2 x0 = lane < pieces ? a.part_ml[lane * all + row] : none;
  const float2 x1 = lane + 32 < pieces ? a.part_ml[(lane + 32) * all + row] : none;
  if (__any_sync(0xffffffffu, x0.y < 0.f || x1.y < 0.f)) return;
  float m = fmaxf(x0.x, x1.x);
#pragma unroll
  for (int w = 16; w; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  const float ref = m == -INFINITY ? 0.f : m, w0 = gqa_ex2(x0.x - ref), w1 = gqa_ex2(x1.x - ref);
  float l = x0.y * w0 + x1.y * w1;
#pragma unroll
  for (int w = 16; w; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  for (int e0 = 0; e0 < a.d; e0 += 32) {
    const int e = e0 + lane;
    float o = 0.f;
    for (int p = 0; p < pieces; p += 4) {
      float x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = p + k < pieces && e < a.d ? a.part_o[((p + k) * all + row) * a.d + e] : 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float w = __shfl_sync(0xffffffffu, p + k < 32 ? w0 : w1, (p + k) & 31);
        if (p + k < pieces) o = fmaf(x[k], w, o);
      }
    }
    const float y[1] = {o / l};
    if (e < a.d) store_v<1>(static_cast<T*>(a.out) + row * a.d + e, y);
  }
}

template <typename T, typename C>
int launch_simt_t(const GqaArgs& a, cudaStream_t st) {
  const int dk = (a.d + 31) / 32;
  const size_t smem = sizeof(float) * simt_words(a.d);
  auto kern = dk <= 2 ? gqa_simt_kernel<T, C, 2> : dk <= 4 ? gqa_simt_kernel<T, C, 4> : gqa_simt_kernel<T, C, 8>;
  if (allow_smem(kern, smem) != cudaSuccess) return KDTV_ERR_CUDA;
  const dim3 grid((unsigned)a.splits, (unsigned)((a.N * a.G + kRowsCta - 1) / kRowsCta),
                  (unsigned)(a.B * a.Hkv));
  kern<<<grid, kSimtThreads, smem, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return KDTV_ERR_CUDA;
  if (a.splits > 1) {
    const long long rows = (long long)a.B * a.N * a.H;
    if (launch_ex(gqa_simt_combine_kernel<T>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, true, a) !=
        cudaSuccess)
      return KDTV_ERR_CUDA;
  }
  return KDTV_OK;
}

int launch_gqa_simt(const GqaArgs& a, cudaStream_t st) {
  if (a.dtype == KDTV_F32) return launch_simt_t<float, float>(a, st);
  if (a.dtype == KDTV_BF16) return launch_simt_t<__nv_bfloat16, __nv_bfloat16>(a, st);
  return launch_simt_t<__nv_bfloat16, __nv_fp8_e4m3>(a, st);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int check(const kdtv_gqa_dims* d) {
  if (!d) return KDTV_ERR_INVALID_ARG;
  if (d->B <= 0 || d->N <= 0 || d->H <= 0 || d->H_kv <= 0 || d->d <= 0 || d->H % d->H_kv)
    return KDTV_ERR_INVALID_ARG;
  if (d->dtype != KDTV_F32 && d->dtype != KDTV_BF16 && d->dtype != KDTV_BF16_FP8KV)
    return KDTV_ERR_INVALID_ARG;
  if (d->page_size < 0) return KDTV_ERR_INVALID_ARG;
  if (d->page_size == 0) {
    if (d->t_stride <= 0) return KDTV_ERR_INVALID_ARG;
  } else {
    if (d->max_pages <= 0 || d->num_pages <= 0) return KDTV_ERR_INVALID_ARG;
    if ((long long)d->max_pages * d->page_size > (1ll << 30)) return KDTV_ERR_INVALID_ARG;
  }
  if (d->N > kMaxNodes || d->d > 256) return KDTV_ERR_UNSUPPORTED;
  if ((long long)d->B * d->H_kv > 65535) return KDTV_ERR_UNSUPPORTED;
  if ((long long)d->B * d->N * d->H > (1ll << 28)) return KDTV_ERR_UNSUPPORTED;
  // 32-bit positions; a grid row per 16 query rows of a key/value head
  if (d->t_stride > (1 << 30) && d->page_size == 0) return KDTV_ERR_UNSUPPORTED;
  if ((long long)d->N * (d->H / d->H_kv) > 65535ll * kRowsCta) return KDTV_ERR_UNSUPPORTED;
  return KDTV_OK;
}

bool on_tensor_cores(const kdtv_gqa_dims* d) {
  return !(d->flags & KDTV_FLAG_SIMT) && gqa_tc_supported(d);
}

// Fills the plan of `a` and the offsets of its partials; the status a call returns.
int make_plan(const kdtv_gqa_dims* d, GqaArgs* a, size_t* off_ml, size_t* off_plan, size_t* total) {
  const int rc = check(d);
  if (rc != KDTV_OK) return rc;
  memset(a, 0, sizeof(*a));
  a->B = d->B; a->N = d->N; a->H = d->H; a->Hkv = d->H_kv; a->G = d->H / d->H_kv; a->d = d->d;
  a->dtype = d->dtype; a->page_size = d->page_size; a->t_stride = d->t_stride;
  a->max_pages = d->max_pages; a->num_pages = d->num_pages;
  a->cap = d->page_size ? (long long)d->max_pages * d->page_size : d->t_stride;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 152;
  size_t rows;                                     // partial rows
  if (on_tensor_cores(d)) {
    rows = gqa_tc_workspace(d, sms, a);
    if (!rows) return KDTV_ERR_UNSUPPORTED;
  } else {
    // Splits until the grid holds four CTAs per SM, each of 64 keys or more.
    const long long cap = a->cap;
    const long long ctas = (long long)d->B * d->H_kv * ((d->N * a->G + kRowsCta - 1) / kRowsCta);
    long long splits = (4ll * sms + ctas - 1) / ctas;
    const long long most = (cap + 63) / 64;
    if (splits > most) splits = most;
    if (splits > 64) splits = 64;
    a->chunk = (int)(((cap + splits - 1) / splits + kKeys - 1) / kKeys * kKeys);
    a->splits = (int)((cap + a->chunk - 1) / a->chunk);
    rows = a->splits > 1 ? (size_t)a->splits * d->B * d->N * d->H : 0;
  }
  *off_ml = align256(rows * d->d * sizeof(float));
  *off_plan = *off_ml + align256(rows * sizeof(float2));
  *total = *off_plan + align256((size_t)(1 + d->B) * sizeof(int));
  return KDTV_OK;
}

}  // namespace

}  // namespace kdtv

using namespace kdtv;

extern "C" size_t kdtv_gqa_workspace_size(const kdtv_gqa_dims* d) {
  GqaArgs a;
  size_t off, plan, total;
  return make_plan(d, &a, &off, &plan, &total) == KDTV_OK ? total : 0;
}

extern "C" int kdtv_gqa_launches_per_call(const kdtv_gqa_dims* d) {
  GqaArgs a;
  size_t off, plan, total;
  if (make_plan(d, &a, &off, &plan, &total) != KDTV_OK) return -1;
  return on_tensor_cores(d) ? 2 : (a.splits > 1 ? 2 : 1);
}

extern "C" int kdtv_gqa_verify_attn(const kdtv_gqa_dims* d, const void* q, const void* k,
                                    const void* v, const uint8_t* k_scale, const uint8_t* v_scale,
                                    const int32_t* parent, const int32_t* prefix_len,
                                    const int32_t* n_nodes, const int32_t* page_table, void* out,
                                    unsigned int* status, cudaStream_t stream) {
  GqaArgs a;
  size_t off_ml, off_plan, total;
  const int rc = make_plan(d, &a, &off_ml, &off_plan, &total);
  if (rc != KDTV_OK) return rc;
  if (!q || !k || !v || !parent || !prefix_len || !out || !status) return KDTV_ERR_INVALID_ARG;
  if ((d->page_size > 0) != (page_table != nullptr)) return KDTV_ERR_INVALID_ARG;
  const bool fp8 = d->dtype == KDTV_BF16_FP8KV;
  if (fp8 != (k_scale != nullptr) || fp8 != (v_scale != nullptr)) return KDTV_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, static_cast<const void*>(out)})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return KDTV_ERR_INVALID_ARG;
  if (!d->workspace || (reinterpret_cast<uintptr_t>(d->workspace) & 255u) || d->workspace_bytes < total)
    return KDTV_ERR_INVALID_ARG;
  a.scale = d->scale > 0.f ? d->scale : 1.0f / sqrtf((float)d->d);
  a.q = q; a.k = k; a.v = v; a.k_scale = k_scale; a.v_scale = v_scale;
  a.parent = parent; a.prefix_len = prefix_len; a.n_nodes = n_nodes; a.page_table = page_table;
  a.out = out;
  a.status = status;
  a.part_o = static_cast<float*>(d->workspace);
  a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(d->workspace) + off_ml);
  a.plan = reinterpret_cast<int*>(static_cast<char*>(d->workspace) + off_plan);
  if (on_tensor_cores(d)) return launch_gqa_tc(a, (d->flags & KDTV_FLAG_TEST_STALL) != 0, stream);
  return launch_gqa_simt(a, stream);
}
