// kdtv_project: a projection that all requests share, with a low-rank adapter
// per request.  Host side, and the CUDA-core path (fp32, and what the tensor
// cores do not take).

#include "kdtv_proj.cuh"
#include "kdtv_ptx.cuh"

#include <math.h>
#include <string.h>

namespace kdtv {
namespace {

constexpr int kThreads = 256;

// s_a A_a x of a request's rows: a CTA has kRows rows of x and kRanks ranks (8 and 4, or 2 and 16 where requests have
// no more rows), its threads go along d_in; their sums meet by shuffles and in shared memory.
constexpr int kJoin = 4;                   // outputs whose last sums a thread makes together

template <typename X, typename T, int kRows, int kRanks>
__global__ void __launch_bounds__(kThreads) proj_low_simt_kernel(const __grid_constant__ ProjArgs a) {
  __shared__ float part[kThreads / 32][kRows * kRanks];
  // proj_few_simt_kernel may start; it waits for this grid at its end.  (The tiles' kernel is launched behind this one:
  // with blocks of this one about, it gave some SMs two blocks and others none, 514 us for 1024 rows, 4096 x 1216, where it
  // takes 302.)
  ptx::grid_dep_launch();
  const int b = blockIdx.y, i0 = blockIdx.x * kRows, r0 = blockIdx.z * kRanks, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = live_rows(a.n_live, b, a.N);
  if (i0 >= n) return;
  const int id = proj_adapter(a, a.adapter[b]);
  if (id < 0) return;
  const float s = a.adapter_scale ? a.adapter_scale[id] : 1.f;
  const X* x = static_cast<const X*>(a.x) + b * a.xs[0] + i0 * a.xs[1];
  const uint8_t* xe = a.x_scale + ((long long)b * a.N + i0) * (a.K / KDTV_GROUP);
  const T* A = static_cast<const T*>(a.A) + ((long long)id * a.R + r0) * a.K;
  float total[kRows][kRanks] = {};
  for (int k0 = 0; k0 < a.K; k0 += kThreads * 32) {      // chains of at most 32 terms, then their sums
    float sum[kRows][kRanks] = {};
#pragma unroll 2
    for (int k = k0 + threadIdx.x; k < min(a.K, k0 + kThreads * 32); k += kThreads) {
      float u[kRows], w[kRanks];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        u[j] = i0 + j < n ? to_f32(x[j * a.xs[1] + k]) : 0.f;
        if constexpr (sizeof(X) == 1)
          if (i0 + j < n) u[j] *= scale_of_byte(xe[(long long)j * (a.K / KDTV_GROUP) + k / KDTV_GROUP]);
      }
#pragma unroll
      for (int r = 0; r < kRanks; ++r) w[r] = r0 + r < a.R ? to_f32(A[(long long)r * a.K + k]) : 0.f;
#pragma unroll
      for (int j = 0; j < kRows; ++j)
#pragma unroll
        for (int r = 0; r < kRanks; ++r) sum[j][r] = fmaf(u[j], w[r], sum[j][r]);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int r = 0; r < kRanks; ++r) total[j][r] += sum[j][r];
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j)
#pragma unroll
    for (int r = 0; r < kRanks; ++r) {
      float v = total[j][r];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) part[warp][j * kRanks + r] = v;
    }
  __syncthreads();
  if (threadIdx.x >= kRows * kRanks) return;
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) v += part[k][threadIdx.x];
  const int i = i0 + threadIdx.x / kRanks, r = r0 + threadIdx.x % kRanks;
  if (i < n && r < a.R) a.low[((long long)b * a.N + i) * a.R + r] = s * v;
}

// y: a CTA has TM rows (of all requests' rows) and TN outputs, kStep elements
// of d_in at a time; its threads are S groups that take alternate steps and
// meet at the end.  A thread has R x 4 sums, rows in fours set apart so that its
// 16-byte reads of shared memory do not conflict; they are taken anew after 128
// terms and added to the totals: no chain of additions is long.
// 128 x 64 with 8 x 4 sums is bound by the fp32 pipe (three 16-byte reads for 32
// multiply-adds, two to an instruction); the smaller tiles are for sizes of which it
// has too few, 16 x 32 with S = 8 for those of few rows.  Where the tiles leave SMs idle, `split` CTAs of
// a cluster share d_in and add their totals up through distributed shared memory,
// in their order, each a part of the tile.
template <typename X, typename T, int TM, int TN, int S, int kStep, int R>
__global__ void __launch_bounds__(kThreads) proj_simt_kernel(const __grid_constant__ ProjArgs a, int split) {
  constexpr int kGroup = kThreads / S, C = R / 4, kRowsOf = TM / C;     // fours of rows, set kRowsOf apart
  static_assert(TM / R * (TN / 4) == kGroup, "R x 4 sums a thread");
  constexpr int kOperands = S * kStep * (TM + 4 + TN + 4), kSums = S * kRowsOf * TN;
  __shared__ __align__(16) float pool[kOperands > kSums ? kOperands : kSums];
  float (*xs)[kStep][TM + 4] = reinterpret_cast<float (*)[kStep][TM + 4]>(pool);
  float (*ws)[kStep][TN + 4] = reinterpret_cast<float (*)[kStep][TN + 4]>(pool + S * kStep * (TM + 4));
  __shared__ long long s_x[TM], s_y[TM];               // offsets of the rows, -1: not live
  __shared__ int s_row[TM], s_id[TM];
  __shared__ int s_any;
  const int g = threadIdx.x / kGroup, t = threadIdx.x % kGroup;
  const long long r0 = (long long)blockIdx.y * TM, rows = (long long)a.B * a.N;
  const int f0 = blockIdx.x * TN;
  if (threadIdx.x == 0) s_any = 0;
  __syncthreads();
  if (threadIdx.x < TM) {
    const long long r = r0 + threadIdx.x;
    long long ox = -1, oy = -1;
    int id = -1;
    if (r < rows) {
      const int b = (int)divide((unsigned)r, a.by_N), i = (int)(r - (long long)b * a.N);
      if (i < live_rows(a.n_live, b, a.N)) {
        id = proj_adapter(a, a.adapter ? a.adapter[b] : -1);
        if (id != -2) {
          ox = b * a.xs[0] + i * a.xs[1];
          oy = b * a.ys[0] + i * a.ys[1];
          s_any = 1;
        }
      }
    }
    s_x[threadIdx.x] = ox;
    s_y[threadIdx.x] = oy;
    s_row[threadIdx.x] = (int)r;
    s_id[threadIdx.x] = id;
  }
  __syncthreads();
  if (!s_any) return;                                  // (the same for all of a cluster)
  const int part = blockIdx.z;
  const int tm = t / (TN / 4) * 4, tn = t % (TN / 4) * 4;
  float2 total[R][2] = {}, sum[R][2] = {};
  const int all_steps = (a.K + kStep - 1) / kStep;
  const int from = (int)((long long)all_steps * part / split), steps = (int)((long long)all_steps * (part + 1) / split);
  const X* x = static_cast<const X*>(a.x);
  const X* W = static_cast<const X*>(a.W);
  int held = 0;
  // A step's elements: kGroup is a multiple of kStep, so a thread stays in its column; the next step's are on their
  // way while this one's are multiplied.
  static_assert(kGroup % kStep == 0, "a thread's column");
  constexpr int kXs = TM * kStep / kGroup, kWs = TN * kStep / kGroup, kDown = kGroup / kStep;
  const int col = t % kStep, row = t / kStep;
  float nx[kXs], nw[kWs];
  auto fetch = [&](int step) {                         // (a group behind the last step gets zeros)
    const int k = step < steps ? step * kStep + col : a.K;
#pragma unroll
    for (int i = 0; i < kXs; ++i) {
      const int m = row + i * kDown;
      const long long o = s_x[m];
      const bool on = o >= 0 && k < a.K;
      nx[i] = on ? to_f32(x[o + k]) : 0.f;
      if constexpr (sizeof(X) == 1)
        if (on) nx[i] *= scale_of_byte(a.x_scale[(long long)s_row[m] * (a.K / KDTV_GROUP) + k / KDTV_GROUP]);
    }
#pragma unroll
    for (int i = 0; i < kWs; ++i) {
      const int f = f0 + row + i * kDown;
      const bool on = f < a.M && k < a.K;
      nw[i] = on ? to_f32(W[(long long)f * a.K + k]) : 0.f;
      if constexpr (sizeof(X) == 1)
        if (on) nw[i] *= scale_of_byte(a.W_scale[(long long)f * (a.K / KDTV_GROUP) + k / KDTV_GROUP]);
    }
  };
  fetch(from + g);
  for (int first = from; first < steps; first += S) {
#pragma unroll
    for (int i = 0; i < kXs; ++i) xs[g][col][row + i * kDown] = nx[i];
#pragma unroll
    for (int i = 0; i < kWs; ++i) ws[g][col][row + i * kDown] = nw[i];
    __syncthreads();
    if (first + S < steps) fetch(first + S + g);
#pragma unroll 8
    for (int k = 0; k < kStep; ++k) {
      float u[R];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float4 p = *reinterpret_cast<const float4*>(&xs[g][k][c * kRowsOf + tm]);
        u[4 * c] = p.x; u[4 * c + 1] = p.y; u[4 * c + 2] = p.z; u[4 * c + 3] = p.w;
      }
      const float4 q = *reinterpret_cast<const float4*>(&ws[g][k][tn]);
      const float2 w[2] = {make_float2(q.x, q.y), make_float2(q.z, q.w)};
#pragma unroll
      for (int p = 0; p < R; ++p)
#pragma unroll
        for (int e = 0; e < 2; ++e) sum[p][e] = ptx::fma2(make_float2(u[p], u[p]), w[e], sum[p][e]);
    }
    if (++held == 128 / kStep || first + S >= steps) {
      held = 0;
#pragma unroll
      for (int p = 0; p < R; ++p)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          total[p][e] = ptx::add2(total[p][e], sum[p][e]);
          sum[p][e] = make_float2(0.f, 0.f);
        }
    }
    __syncthreads();
  }
  // Block of rows by block: the groups' totals, in their order, then the cluster's, of which a CTA finishes rows part,
  // part + split, ..
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (c > 0) {                                       // (the last block's are read)
      if (split > 1) ptx::cluster_sync();
      else __syncthreads();
    }
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int e = 0; e < 2; ++e) *reinterpret_cast<float2*>(pool + (g * kRowsOf + tm + p) * TN + tn + 2 * e) = total[4 * c + p][e];
    __syncthreads();
    if constexpr (S > 1) {
      for (int e = threadIdx.x; e < kRowsOf * TN; e += kThreads) {
        float v = pool[e];
#pragma unroll
        for (int s = 1; s < S; ++s) v += pool[s * kRowsOf * TN + e];
        pool[e] = v;
      }
      __syncthreads();
    }
    if (split > 1) ptx::cluster_sync();
    const int own = kRowsOf / split * TN;              // (kRowsOf is a multiple of 16)
    for (int e0 = threadIdx.x; e0 < own; e0 += kJoin * kThreads) {
      // kJoin outputs, whose look-ups are under way together
      float v[kJoin] = {}, d[kJoin] = {};
      long long to[kJoin];
      const T* Bm[kJoin];
      const float* low[kJoin];
      bool with[kJoin], any = false;
#pragma unroll
      for (int j = 0; j < kJoin; ++j) {
        const int e = min(e0 + j * kThreads, own - 1), at = (e / TN * split + part) * TN + e % TN;
        const int m = c * kRowsOf + at / TN, f = f0 + at % TN, id = s_id[m];
        to[j] = e0 + j * kThreads < own && s_y[m] >= 0 && f < a.M ? s_y[m] + f : -1;
        with[j] = to[j] >= 0 && id >= 0;
        any |= with[j];
        Bm[j] = static_cast<const T*>(a.Bm) + (with[j] ? ((long long)id * a.M + f) * a.R : 0);
        low[j] = a.low + (with[j] ? (long long)s_row[m] * a.R : 0);
        if (split > 1) {
#pragma unroll 4
          for (int k = 0; k < split; ++k) {
            float u;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u) : "r"(ptx::mapa(ptx::smem_u32(pool + at), k)) : "memory");
            v[j] += u;
          }
        } else {
          v[j] = pool[at];
        }
      }
      if (any) {
#pragma unroll 4
        for (int r = 0; r < a.R; ++r)
#pragma unroll
          for (int j = 0; j < kJoin; ++j) d[j] = fmaf(low[j][r], to_f32(Bm[j][r]), d[j]);
      }
#pragma unroll
      for (int j = 0; j < kJoin; ++j)
        if (to[j] >= 0) {
          const float one[1] = {with[j] ? v[j] + d[j] : v[j]};
          store_v<1>(static_cast<T*>(a.y) + to[j], one);
        }
    }
  }
  if (split > 1) ptx::cluster_sync();                  // (the others have read this CTA's sums)
}

// y of few rows: the weights go from global memory to registers once per RT rows.  A warp has F outputs, its
// lanes go along d_in, V neighbours at a time and U such loads of each output under way together; `slices` warps
// share d_in.  The rows' elements come from L1, where a block's warps share them.  A lane's sums are
// taken anew after at most 128 terms, as above.  One row is bound by DRAM (8192 x 10240: 64 us, 5300 GB/s), more by L1.
// (16 elements a lane and step: 73 us for one row, 78 for four where 8 take 71; eight rows and two outputs a warp: 157
// for eight rows where two passes of four take 101; two outputs and four rows: 111 for four.)
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* p, const uint8_t* scale, long long at, float* x) {
  float v[V];
  if constexpr (sizeof(T) == 1 && V == 8) {
    const uint2 w = *reinterpret_cast<const uint2*>(p + at);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 two = widen2(((k < 2 ? w.x : w.y) >> (16 * (k & 1))) & 0xffffu);
      v[2 * k] = two.x;
      v[2 * k + 1] = two.y;
    }
  } else {
    load_v<V>(p + at, v);
  }
  const float f = sizeof(T) == 1 ? scale_of_byte(scale[at / KDTV_GROUP]) : 1.f;   // (rows are whole groups)
#pragma unroll
  for (int k = 0; k < V; ++k) x[k] = sizeof(T) == 1 ? v[k] * f : v[k];
}

template <typename X, typename T, int V, int F, int RT>
__global__ void __launch_bounds__(kThreads) proj_few_simt_kernel(const __grid_constant__ ProjArgs a, int slices) {
  constexpr int E = 8, U = E / V;                  // a lane's elements of a step
  __shared__ long long s_x[RT], s_y[RT];
  __shared__ int s_row[RT], s_id[RT];
  __shared__ float red[kThreads / 32][F * RT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slice = warp % slices;
  const int f0 = (blockIdx.y * (kThreads / 32 / slices) + warp / slices) * F;
  const long long r0 = (long long)blockIdx.x * RT, rows = (long long)a.B * a.N;
  if (threadIdx.x < 32) {
    const long long r = r0 + lane;
    long long ox = -1;
    int id = -1;
    if (lane < RT && r < rows) {
      const int b = (int)divide((unsigned)r, a.by_N), i = (int)(r - (long long)b * a.N);
      if (i < live_rows(a.n_live, b, a.N)) {
        id = proj_adapter(a, a.adapter ? a.adapter[b] : -1);
        if (id != -2) ox = b * a.xs[0] + i * a.xs[1];
      }
      if (ox >= 0) s_y[lane] = b * a.ys[0] + i * a.ys[1];
    }
    const unsigned live = __ballot_sync(0xffffffffu, ox >= 0);
    // (rows that are not live read another's elements, for nothing)
    const int other = live ? __ffs(live) - 1 : 0;
    const long long its = __shfl_sync(0xffffffffu, ox, other);
    if (lane < RT) {
      s_x[lane] = ox >= 0 ? ox : its;
      s_row[lane] = (int)(ox >= 0 ? r : r0 + other);
      s_id[lane] = ox >= 0 ? id : -2;
    }
  }
  __syncthreads();
  if (s_x[0] < 0) {                                      // no row is live
    ptx::grid_dep_wait();
    return;
  }
  const X* x[RT];
  const uint8_t* xe[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    x[r] = static_cast<const X*>(a.x) + s_x[r];
    xe[r] = a.x_scale + (long long)s_row[r] * (a.K / KDTV_GROUP);
  }
  const int all = a.K / V, from = (int)((long long)all * slice / slices), end = (int)((long long)all * (slice + 1) / slices);
  float total[F][RT] = {};
  float2 sum[F][RT] = {};
  auto flush = [&]() {
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        total[f][r] += sum[f][r].x + sum[f][r].y;
        sum[f][r] = make_float2(0.f, 0.f);
      }
  };
  int held = 0;
#pragma unroll 1
  for (int i0 = from + lane; i0 < end; i0 += 32 * U) {
    float w[F][E];
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int k = 0; k < V; ++k) w[f][u * V + k] = 0.f;
        if (f0 + f < a.M && i0 + 32 * u < end)
          load_row<X, V>(static_cast<const X*>(a.W), a.W_scale, (long long)(f0 + f) * a.K + (long long)(i0 + 32 * u) * V, &w[f][u * V]);
      }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float v[E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int k = 0; k < V; ++k) v[u * V + k] = 0.f;
        if (i0 + 32 * u < end) load_row<X, V>(x[r], xe[r], (long long)(i0 + 32 * u) * V, &v[u * V]);
      }
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int e = 0; e < E; e += 2)
          sum[f][r] = ptx::fma2(make_float2(v[e], v[e + 1]), make_float2(w[f][e], w[f][e + 1]), sum[f][r]);
    }
    if (++held == 256 / E) {
      held = 0;
      flush();
    }
  }
  flush();
  float mine = 0.f;                                      // lane f RT + r keeps that sum
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float v = total[f][r];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == f * RT + r) mine = v;
    }
  if (slices > 1) {
    if (lane < F * RT) red[warp][lane] = mine;
    __syncthreads();
    if (slice > 0) {
      ptx::grid_dep_wait();
      return;
    }
    if (lane < F * RT)
      for (int s = 1; s < slices; ++s) mine += red[warp + s][lane];
  }
  ptx::grid_dep_wait();                                  // A x of all rows, where there are adapters
  const int f = f0 + lane / RT, r = lane % RT;
  if (lane >= F * RT || f >= a.M || s_id[r] == -2) return;
  if (s_id[r] >= 0) {
    const T* Bm = static_cast<const T*>(a.Bm) + ((long long)s_id[r] * a.M + f) * a.R;
    const float* low = a.low + (long long)s_row[r] * a.R;
    float d = 0.f;
    for (int k = 0; k < a.R; ++k) d = fmaf(low[k], to_f32(Bm[k]), d);
    mine += d;
  }
  const float one[1] = {mine};
  store_v<1>(static_cast<T*>(a.y) + s_y[r] + f, one);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int kFew = 4, kFewOut = 4;
bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Warps that share d_in: as many as an SM holds, if their parts are two steps' at least.  (One row, 8192 x 10240: half as
// many warps 76 us, these 64, twice as many 61; eight rows 105, 101, 109.)
int few_slices(const ProjArgs& a, int sms) {
  int slices = 1;
  while (slices < 8 && (long long)(a.M + kFewOut - 1) / kFewOut * slices < 64ll * sms && a.K / (2 * slices) >= 512) slices *= 2;
  return slices;
}

template <typename X, typename T>
int launch_few(const ProjArgs& a, long long rows, int sms, cudaStream_t st) {
  auto go = [&](auto kern, int rt) {
    const int slices = few_slices(a, sms), outputs = kThreads / 32 / slices * kFewOut;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + rt - 1) / rt), (unsigned)((a.M + outputs - 1) / outputs));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.adapter ? 1 : 0;                  // beside the first kernel, where there is one
    return cudaLaunchKernelEx(&cfg, kern, a, slices) == cudaSuccess ? KDTV_OK : KDTV_ERR_CUDA;
  };
  constexpr int V = sizeof(X) == 4 ? 4 : 8;
  const bool vec = a.K % 8 == 0 && aligned(a.x) && aligned(a.W) && a.xs[0] % V == 0 && a.xs[1] % V == 0;
  if (rows == 1) return vec ? go(proj_few_simt_kernel<X, T, V, kFewOut, 1>, 1) : go(proj_few_simt_kernel<X, T, 1, kFewOut, 1>, 1);
  return vec ? go(proj_few_simt_kernel<X, T, V, kFewOut, kFew>, kFew) : go(proj_few_simt_kernel<X, T, 1, kFewOut, kFew>, kFew);
}

template <typename X, typename T>
int launch_simt(const ProjArgs& a, int sms, cudaStream_t st) {
  if (a.adapter && a.N <= 2)
    proj_low_simt_kernel<X, T, 2, 16><<<dim3(1, (unsigned)a.B, (unsigned)((a.R + 15) / 16)), kThreads, 0, st>>>(a);
  else if (a.adapter)
    proj_low_simt_kernel<X, T, 8, 4><<<dim3((unsigned)((a.N + 7) / 8), (unsigned)a.B, (unsigned)((a.R + 3) / 4)), kThreads, 0, st>>>(a);
  const long long rows = (long long)a.B * a.N;
  if (cudaGetLastError() != cudaSuccess) return KDTV_ERR_CUDA;
  // The tile, and how many CTAs share d_in (four steps each at least), with the least time in cycles by this reckoning:
  // the SM with the most CTAs does its products at the tile's share of the fp32 rate (measured: 55, 43 and 28 %), a step
  // takes some 500 at least, a CTA as much besides, and joining a cluster 3000.  Without tiles four rows take 7 weights a
  // cycle of each SM, 4.5 where all of a block's warps share d_in and none the rows, and four blocks 1000 besides.
  // (Measured with 8192 x 10240 and 4, 8, 12, 16, 24 rows: 71, 101, 139, 178, 261 us, the tiles 154 to 159 and 280; 4096 x
  // 4096: 21, 31, 44, 57, 83, the tiles 41 to 43 and 61; 1001 x 515, 16 and 32 rows: 7.5 and 8.2, the tiles 14 and 23).
  struct Tile {
    int tm, tn, step, groups, percent;
  };
  const Tile tiles[3] = {{128, 64, 16, 1, 55}, {64, 64, 32, 1, 43}, {16, 32, 16, 8, 28}};
  int best = -1, split = 1;
  const int slices = few_slices(a, sms);
  const double fours = (double)((rows + kFew - 1) / kFew), blocks = fours * ((a.M + 32 / slices - 1) / (32 / slices));
  double least = 2500.0 + fours * a.M * a.K / ((slices == 8 ? 4.5 : 7.0) * sms) + blocks / (4.0 * sms) * 1000.0;
  for (int k = 0; k < 3; ++k) {
    const Tile& e = tiles[k];
    const long long down = (rows + e.tm - 1) / e.tm, n = down * ((a.M + e.tn - 1) / e.tn);
    if (down > 65535) continue;
    for (int s = 1; s <= 8; s *= 2) {
      if (s > 1 && a.K / s < 4 * e.step * e.groups) break;
      const int usable = s >= 4 && n * s <= 2 * sms ? sms * 8 / 9 : sms;     // (larger clusters leave SMs out)
      const double per = (double)((n * s + usable - 1) / usable), depth = (double)a.K / s;
      const double work = per * e.tm * e.tn * depth / (1.28 * e.percent), steps = depth / (e.step * e.groups) * 500.0;
      const double time = (work > steps ? work : steps) + per * 500.0 + (s > 1 ? 3000.0 : 0.0);
      if (time < least) {
        least = time;
        best = k;
        split = s;
      }
    }
  }
  auto go = [&](auto kern, int tm, int tn) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.M + tn - 1) / tn), (unsigned)((rows + tm - 1) / tm), (unsigned)split);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {1, 1, (unsigned)split};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, split) == cudaSuccess ? KDTV_OK : KDTV_ERR_CUDA;
  };
  if (best < 0) return launch_few<X, T>(a, rows, sms, st);
  if (best == 0) return go(proj_simt_kernel<X, T, 128, 64, 1, 16, 8>, 128, 64);
  if (best == 1) return go(proj_simt_kernel<X, T, 64, 64, 1, 32, 4>, 64, 64);
  return go(proj_simt_kernel<X, T, 16, 32, 8, 16, 4>, 16, 32);
}

int check_dims(const kdtv_project_dims* d) {
  if (!d) return KDTV_ERR_INVALID_ARG;
  if (d->B <= 0 || d->N <= 0 || d->d_in <= 0 || d->d_out <= 0 || d->adapters < 0) return KDTV_ERR_INVALID_ARG;
  if (d->dtype != KDTV_F32 && d->dtype != KDTV_BF16 && d->dtype != KDTV_BF16_FP8KV) return KDTV_ERR_INVALID_ARG;
  if (d->adapters > 0 && d->rank <= 0) return KDTV_ERR_INVALID_ARG;
  if (d->dtype == KDTV_BF16_FP8KV && d->d_in % KDTV_GROUP) return KDTV_ERR_INVALID_ARG;
  if (d->adapters > KDTV_MAX_ADAPTERS || (d->adapters > 0 && d->rank > 256)) return KDTV_ERR_UNSUPPORTED;
  if (d->B > 65535 || d->d_in > (1 << 20) || d->d_out > (1 << 20) || (long long)d->B * d->N > 64ll * 65535)
    return KDTV_ERR_UNSUPPORTED;                           // grid rows
  return KDTV_OK;
}

int sm_count() { return device_sm_count() > 0 ? device_sm_count() : 152; }

// For either path: which one runs depends on addresses too.
size_t workspace_of(const kdtv_project_dims* d) {
  ProjArgs a;
  memset(&a, 0, sizeof(a));
  const size_t low = (size_t)d->B * d->N * (d->adapters > 0 ? d->rank : 0) * sizeof(float);
  const size_t tc = proj_tc_sizes(d, sm_count(), &a) ? proj_tc_workspace(a, sm_count()) : 0;
  return align256(low > tc ? low : tc) + 256;
}

// Rows that TMA can read: strides (of what has more than one element) multiples of 16 bytes, not 0, below 2^40.
bool tma_rows(const kdtv_project_dims* d, const ProjArgs& a) {
  if (d->dtype == KDTV_BF16_FP8KV) return true;          // contiguous
  auto fits = [](long long s) { return s > 0 && s % 8 == 0 && s < (1ll << 39); };
  return (d->N == 1 || fits(a.xs[1])) && (d->B == 1 || fits(a.xs[0]));
}

}  // namespace
}  // namespace kdtv

using namespace kdtv;

extern "C" size_t kdtv_project_workspace_size(const kdtv_project_dims* d) {
  return check_dims(d) == KDTV_OK ? workspace_of(d) : 0;
}

extern "C" int kdtv_project_launches_per_call(const kdtv_project_dims* d) {
  if (check_dims(d) != KDTV_OK) return -1;
  ProjArgs a;
  memset(&a, 0, sizeof(a));
  return proj_tc_sizes(d, sm_count(), &a) ? proj_tc_launches(a) : 1 + (d->adapters > 0);
}

extern "C" int kdtv_project(const kdtv_project_dims* d, const void* x, const uint8_t* x_scale,
                            const void* W, const uint8_t* W_scale, const void* A, const void* Bm,
                            const float* adapter_scale, const int32_t* adapter, const int32_t* n_live,
                            void* y, unsigned int* status, cudaStream_t stream) {
  const int rc = check_dims(d);
  if (rc != KDTV_OK) return rc;
  if (!x || !W || !y || !status || y == x || y == W) return KDTV_ERR_INVALID_ARG;
  const bool one_byte = d->dtype == KDTV_BF16_FP8KV;
  if (one_byte != (x_scale != nullptr) || one_byte != (W_scale != nullptr)) return KDTV_ERR_INVALID_ARG;
  if ((A != nullptr) != (Bm != nullptr) || (adapter && !A) || (A && d->adapters == 0)) return KDTV_ERR_INVALID_ARG;
  // (strides of dimensions of one element mean nothing, here and below)
  if (one_byte && (d->x_stride[0] || d->x_stride[1]) &&
      ((d->B > 1 && d->x_stride[0] != (int64_t)d->N * d->d_in) || (d->N > 1 && d->x_stride[1] != d->d_in)))
    return KDTV_ERR_INVALID_ARG;
  if ((d->y_stride[0] || d->y_stride[1]) && ((d->B > 1 && !d->y_stride[0]) || (d->N > 1 && !d->y_stride[1])))
    return KDTV_ERR_INVALID_ARG;                            // rows over one another
  if (!d->workspace || (reinterpret_cast<uintptr_t>(d->workspace) & 255u) || d->workspace_bytes < workspace_of(d))
    return KDTV_ERR_INVALID_ARG;
  ProjArgs a;
  memset(&a, 0, sizeof(a));
  a.B = d->B; a.N = d->N; a.K = d->d_in; a.M = d->d_out; a.R = d->adapters > 0 ? d->rank : 0;
  a.adapters = d->adapters; a.dtype = d->dtype;
  a.x = x; a.W = W; a.A = A; a.Bm = Bm; a.x_scale = x_scale; a.W_scale = W_scale;
  a.adapter_scale = adapter_scale; a.adapter = adapter; a.n_live = n_live;
  a.y = y; a.status = status;
  auto strides = [&](const int64_t (&in)[2], long long width, long long (&out)[2]) {
    const bool given = in[0] || in[1];
    out[0] = d->B > 1 ? (given ? in[0] : d->N * width) : 0;
    out[1] = d->N > 1 ? (given ? in[1] : width) : 0;
  };
  strides(d->x_stride, d->d_in, a.xs);
  strides(d->y_stride, d->d_out, a.ys);
  a.by_N = divisor((unsigned)d->N);
  a.low = static_cast<float*>(d->workspace);
  const int sms = sm_count();
  if (aligned(x) && aligned(W) && aligned(A) && aligned(Bm) && tma_rows(d, a) && proj_tc_sizes(d, sms, &a))
    return launch_proj_tc(a, sms, d->flags & KDTV_FLAG_TEST_STALL, stream);
  if (d->dtype == KDTV_F32) return launch_simt<float, float>(a, sms, stream);
  if (d->dtype == KDTV_BF16) return launch_simt<__nv_bfloat16, __nv_bfloat16>(a, sms, stream);
  return launch_simt<__nv_fp8_e4m3, __nv_bfloat16>(a, sms, stream);
}
