// kdtv_gqa_verify_attn: tree-verify attention over a cache of keys and values
// per head.  Host side, and the CUDA-core path (fp32, and what the tensor
// cores do not take).

#include "kdtv_gqa.cuh"

#include <math.h>
#include <string.h>

namespace kdtv {
namespace {

// ---- CUDA cores -----------------------------------------------------------------------
// A CTA of 4 warps takes 16 rows of one key/value head and one split of the
// keys, 32 keys at a time: K and V staged in shared memory as fp32, each warp
// four rows.  Scores: a lane per key (K rows padded by one word against bank
// conflicts, four rows share each K load).  Softmax: online, across the lanes.
// Output: a lane holds elements lane + 32 k of the four rows.  Bound by the
// fp32 pipe and shared-memory reads; the path exists for fp32 and for head
// dims outside the tensor-core instances, not for speed.
constexpr int kRowsCta = 16, kRowsWarp = 4, kKeys = 32, kSimtThreads = 128;

template <typename T, typename C, int DK>     // DK = ceil(d / 32)
__global__ void __launch_bounds__(kSimtThreads) gqa_simt_kernel(const __grid_constant__ GqaArgs a) {
  extern __shared__ __align__(16) float sm[];
  const int d = a.d, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* ks = sm;                                  // [kKeys][d + 1]
  float* vs = ks + kKeys * (d + 1);                // [kKeys][d]
  float* qs = vs + kKeys * d;                      // [kRowsCta][d]
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
  for (int i = threadIdx.x; i < kRowsCta * d; i += kSimtThreads) {
    const int r = r0 + i / d;
    qs[i] = r < rows ? to_f32(static_cast<const T*>(a.q)[out_row(r) * d + i % d]) : 0.f;
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
    for (int i = threadIdx.x; i < kKeys * d; i += kSimtThreads) {
      const int j = i / d, e = i % d;
      float kx = 0.f, vx = 0.f;
      if (j < nk) {
        const long long row = gqa_row(a, b, t0 + j);
        if (row < 0) {
          bad_page = 1;
        } else {
          const long long at = (row * a.Hkv + kvh) * d + e;
          kx = to_f32(static_cast<const C*>(a.k)[at]);
          vx = to_f32(static_cast<const C*>(a.v)[at]);
          if constexpr (sizeof(C) == 1) {
            kx *= scale_of_byte(a.k_scale[row * a.Hkv + kvh]);
            vx *= scale_of_byte(a.v_scale[row * a.Hkv + kvh]);
          }
        }
      }
      ks[j * (d + 1) + e] = kx;
      vs[j * d + e] = vx;
    }
    __syncthreads();
    float s[kRowsWarp];
#pragma unroll
    for (int r = 0; r < kRowsWarp; ++r) s[r] = 0.f;
    const float* kr = ks + lane * (d + 1);
    const float* qr = qs + warp * kRowsWarp * d;
    for (int e = 0; e < d; ++e) {
      const float x = kr[e];
#pragma unroll
      for (int r = 0; r < kRowsWarp; ++r) s[r] = fmaf(qr[r * d + e], x, s[r]);
    }
#pragma unroll
    for (int r = 0; r < kRowsWarp; ++r) {
      uint32_t see = gqa_visible(mask[r], t0, L);
      if (nk < 32) see &= (1u << nk) - 1u;
      const float x = (see >> lane) & 1u ? s[r] * sl2 : -INFINITY;
      float mx = x;
#pragma unroll
      for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[r], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float p = gqa_ex2(x - ref), alpha = gqa_ex2(m[r] - ref);
      float ps = p;
#pragma unroll
      for (int w = 16; w; w >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, w);
      l[r] = l[r] * alpha + ps;
      m[r] = mn;
#pragma unroll
      for (int k = 0; k < DK; ++k) o[r][k] *= alpha;
      // only what the row sees: a masked value may be infinite or NaN
      while (see) {
        const int j = __ffs(see) - 1;
        see &= see - 1;
        const float pj = __shfl_sync(0xffffffffu, p, j);
#pragma unroll
        for (int k = 0; k < DK; ++k)
          if (lane + 32 * k < d) o[r][k] = fmaf(pj, vs[j * d + lane + 32 * k], o[r][k]);
      }
    }
  }
  const bool bad = __syncthreads_or(bad_page);
  if (bad && threadIdx.x == 0) gqa_error(a, KDTV_ERR_BAD_PAGE);
#pragma unroll
  for (int r = 0; r < kRowsWarp; ++r) {
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

// Merges the splits of an output row; a warp per row.
template <typename T>
__global__ void __launch_bounds__(256) gqa_simt_combine_kernel(const __grid_constant__ GqaArgs a) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long all = (long long)a.B * a.N * a.H;
  if (row >= all) return;
  const int b = (int)(row / ((long long)a.N * a.H)), i = (int)(row / a.H % a.N);
  int L, n;
  gqa_request(a, b, &L, &n);
  if (i >= n) return;
  const int pieces = (L + n + a.chunk - 1) / a.chunk;
  float m = -INFINITY;
  for (int p = 0; p < pieces; ++p) {
    const float2 ml = a.part_ml[p * all + row];
    if (ml.y < 0.f) return;
    m = fmaxf(m, ml.x);
  }
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int p = 0; p < pieces; ++p) {
    const float2 ml = a.part_ml[p * all + row];
    l += ml.y * gqa_ex2(ml.x - ref);
  }
  for (int e = lane; e < a.d; e += 32) {
    float o = 0.f;
    for (int p = 0; p < pieces; ++p)
      o = fmaf(a.part_o[(p * all + row) * a.d + e], gqa_ex2(a.part_ml[p * all + row].x - ref), o);
    const float x[1] = {o / l};
    store_v<1>(static_cast<T*>(a.out) + row * a.d + e, x);
  }
}

template <typename T, typename C>
int launch_simt_t(const GqaArgs& a, cudaStream_t st) {
  const int dk = (a.d + 31) / 32;
  const size_t smem = sizeof(float) * (kKeys * (a.d + 1) + kKeys * a.d + kRowsCta * a.d);
  auto kern = dk <= 2 ? gqa_simt_kernel<T, C, 2> : dk <= 4 ? gqa_simt_kernel<T, C, 4> : gqa_simt_kernel<T, C, 8>;
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return KDTV_ERR_CUDA;
  const dim3 grid((unsigned)a.splits, (unsigned)((a.N * a.G + kRowsCta - 1) / kRowsCta),
                  (unsigned)(a.B * a.Hkv));
  kern<<<grid, kSimtThreads, smem, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return KDTV_ERR_CUDA;
  if (a.splits > 1) {
    const long long rows = (long long)a.B * a.N * a.H;
    gqa_simt_combine_kernel<T><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return KDTV_ERR_CUDA;
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
  const int sms = device_sm_count() > 0 ? device_sm_count() : 152;
  size_t rows;                                     // partial rows
  if (on_tensor_cores(d)) {
    rows = gqa_tc_workspace(d, sms, a);
    if (!rows) return KDTV_ERR_UNSUPPORTED;
  } else {
    // Splits until the grid holds four CTAs per SM, each of 64 keys or more.
    const long long cap = d->page_size ? (long long)d->max_pages * d->page_size : d->t_stride;
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
