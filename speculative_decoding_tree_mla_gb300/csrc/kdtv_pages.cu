// kdtv_pages_resize: block tables and slots of a paged cache from the
// requests' lengths, on the GPU.

#include "kdtv_rope.cuh"
#include "kdtv_ptx.cuh"

#include <limits.h>
#include <string.h>

namespace kdtv {
namespace {

constexpr int kPageThreads = 1024;
constexpr int kMaxCluster = 8;

struct PageArgs {
  int B, N, page_size, max_pages, num_pages;
  const int32_t *prefix_len, *n_live;
  int32_t *free_pages, *free_count, *n_pages, *page_table;
  int64_t* slots;
  unsigned int* status;
  Divisor by_page, by_N;
};

__device__ __forceinline__ void page_error(const PageArgs& a, unsigned int code) { atomicCAS(a.status, 0u, code); }

// Index of the first entry of the ascending incl[0 .. n) that is above v; v < incl[n - 1].
__device__ __forceinline__ int first_above(const int* incl, int n, int v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (incl[mid] > v) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Inclusive sums of v[0 .. n) and w[0 .. n), in place, by the block (a thread
// has a run of neighbours).
__device__ __forceinline__ void scan2(int* v, int* w, int n) {
  __shared__ int2 part[32];
  const int per = (n + kPageThreads - 1) / kPageThreads;
  const int lo = min((int)threadIdx.x * per, n), hi = min(lo + per, n);
  int2 s = make_int2(0, 0);
  for (int i = lo; i < hi; ++i) {
    s.x += v[i];
    s.y += w[i];
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 incl = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
    if (lane >= o) {
      incl.x += x;
      incl.y += y;
    }
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int2 p = part[lane];
    const int2 own = p;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, p.x, o), y = __shfl_up_sync(0xffffffffu, p.y, o);
      if (lane >= o) {
        p.x += x;
        p.y += y;
      }
    }
    part[lane] = make_int2(p.x - own.x, p.y - own.y);
  }
  __syncthreads();
  int x = part[warp].x + incl.x - s.x, y = part[warp].y + incl.y - s.y;
  for (int i = lo; i < hi; ++i) {
    v[i] = x += v[i];
    w[i] = y += w[i];
  }
  __syncthreads();
}

// Slot of row i of request b, whose pages are those of `page_at`.
template <typename F>
__device__ __forceinline__ int64_t slot_of(const PageArgs& a, int L, int n, int pages, int i, F page_at) {
  if (i >= n || L < 0 || pages < 0 || pages > a.max_pages || (long long)L + n > (long long)pages * a.page_size) return -1;
  const int t = L + i, p = (int)divide(t, a.by_page), id = page_at(p);
  return id < 0 || id >= a.num_pages ? -1 : (int64_t)id * a.page_size + (t - p * a.page_size);
}

// One cluster of CTAs.  Each scans all requests by itself (they are few, and
// their lengths are in L2), so that the CTAs share nothing but barriers:
// what all of them read (counts, the free list's length, page ids that go
// back) is read before the first one, what goes back is on the stack before
// the second, behind which pages are taken, and behind the third all know
// whether an id that was taken is no page's.  What goes back, or is taken, is
// spread by entries, which find their requests by bisection in the sums, so
// that one request with many pages is spread like many with one.
// Latency bound: trips to L2, a scan and barriers (64 requests with 8 rows each: 4.5 us, one CTA; 512 prompts of up
// to 6000 rows in pages of 16: 11 us to take 96000 pages and 20 to give them back, eight CTAs).
__global__ void __launch_bounds__(kPageThreads) pages_resize_kernel(const __grid_constant__ PageArgs a, int ctas) {
  extern __shared__ __align__(16) int ps[];
  int *give = ps, *take = give + a.B, *want = take + a.B, *have = want + a.B;
  uint32_t* bad = reinterpret_cast<uint32_t*>(have + a.B);       // one bit a request
  __shared__ int s_wrong;                              // the first of the entries that are taken whose id is no page's
  const int rank = ctas > 1 ? (int)ptx::cluster_ctarank() : 0, tid = threadIdx.x;
  const int all = ctas * kPageThreads, me = rank * kPageThreads + tid;
  for (int i = tid; i < (a.B + 31) / 32; i += kPageThreads) bad[i] = 0u;
  if (tid == 0) s_wrong = INT_MAX;
  const int count = *a.free_count;
  const bool usable = count >= 0 && count <= a.num_pages;
  for (int b = tid; b < a.B; b += kPageThreads) {
    const int L = a.prefix_len[b], n = live_rows(a.n_live, b, a.N), h = a.n_pages[b];
    const long long rows = (long long)L + n;
    int w = h;
    if (L < 0 || rows > (long long)a.max_pages * a.page_size) {
      if (rank == 0) page_error(a, KDTV_ERR_BAD_PREFIX);
    } else if (h < 0 || h > a.max_pages || !usable) {
      if (rank == 0) page_error(a, KDTV_ERR_BAD_PAGE);
    } else {
      w = (int)divide((unsigned)(rows + a.page_size - 1), a.by_page);
    }
    want[b] = w;
    have[b] = h;
    give[b] = max(h - w, 0);
    take[b] = max(w - h, 0);
  }
  __syncthreads();
  if (ctas > 1) ptx::cluster_sync();                   // every CTA's bits and s_wrong are set up
  // Pages that go back must be pages: each CTA looks at its share of the requests.
  for (int b = rank * (kPageThreads / 32) + (tid >> 5); b < a.B; b += ctas * (kPageThreads / 32)) {
    const int32_t* row = a.page_table + (long long)b * a.max_pages;
    bool wrong = false;
    if (give[b])
#pragma unroll 8
      for (int p = want[b] + (tid & 31); p < have[b]; p += 32) wrong |= row[p] < 0 || row[p] >= a.num_pages;
    if (__any_sync(0xffffffffu, wrong) && (tid & 31) == 0) {
      page_error(a, KDTV_ERR_BAD_PAGE);
      const uint32_t at = ptx::smem_u32(&bad[b >> 5]);
      for (int c = 0; c < ctas; ++c)
        asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;"
                     :: "r"(ctas > 1 ? ptx::mapa(at, c) : at), "r"(1u << (b & 31)) : "memory");
    }
  }
  if (ctas > 1) ptx::cluster_sync();
  else __syncthreads();
  for (int b = tid; b < a.B; b += kPageThreads)
    if ((bad[b >> 5] >> (b & 31)) & 1u) {
      give[b] = 0;
      want[b] = have[b];
    }
  __syncthreads();
  scan2(give, take, a.B);
  int given = give[a.B - 1];
  // More pages than there are: counts or tables are wrong, and nothing moves.
  const bool over = usable && (long long)count + given > a.num_pages;
  const int top = over ? count : count + given;
  if (over && rank == 0 && tid == 0) page_error(a, KDTV_ERR_BAD_PAGE);
  if (over) given = 0;
  // Who gets pages: the sums ascend, so those that the stack suffices for come first.
  int grant = a.B;                                     // requests from here on get none
  if (over) grant = 0;
  else if (take[a.B - 1] > top) grant = first_above(take, a.B, top);
  const int taken = grant ? take[grant - 1] : 0;
  if (!over && taken != take[a.B - 1] && rank == 0 && tid == 0) page_error(a, KDTV_ERR_NO_PAGES);
  // What request b holds now.
  auto pages_of = [&](int b) { return over ? have[b] : want[b] > have[b] && b >= grant ? have[b] : want[b]; };
  for (int b = me; b < a.B; b += all) {
    const int p = pages_of(b);
    if (p != have[b]) a.n_pages[b] = p;
  }
  if (me == 0 && usable) *a.free_count = top - taken;
  // A warp takes runs of 32 kBatch entries, all of them under way together.  Requests with many pages each: an
  // entry's request is found from the one 32 entries before; with few, by bisection each time.
  constexpr int kBatch = 8;
  const bool few = (long long)given + taken < 64ll * a.B;
  // (a run that begins behind the last entry may begin behind 2^31 too)
  const unsigned lane = tid & 31, run0 = (me >> 5) * 32 * kBatch, runs = all * kBatch;
  if (given) {
    for (unsigned e0 = run0; e0 < (unsigned)given; e0 += runs) {
      int32_t* entry[kBatch];
      int id[kBatch], b = 0;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int k = (int)(given - 1 - (e0 + 32 * i + lane));       // from the last request's last page on
        entry[i] = nullptr;
        if (k < 0) continue;
        if (i == 0 || few) b = first_above(give, a.B, k);
        else
          while (b > 0 && give[b - 1] > k) --b;
        entry[i] = a.page_table + (long long)b * a.max_pages + want[b] + k - (b ? give[b - 1] : 0);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) id[i] = entry[i] ? *entry[i] : 0;
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (entry[i]) {
          a.free_pages[count + e0 + 32 * i + lane] = id[i];
          *entry[i] = -1;
        }
    }
    if (taken) {                                       // (it may be among those that are taken)
      __threadfence();
      if (ctas > 1) ptx::cluster_sync();
      else __syncthreads();
    }
  }
  // The k-th page that is taken, from the top of the stack down.
  auto page_taken = [&](int k) { return *reinterpret_cast<volatile int32_t*>(a.free_pages + (top - 1 - k)); };
  auto entry_taken = [&](int b, int k) { return a.page_table + (long long)b * a.max_pages + have[b] + k - (b ? take[b - 1] : 0); };
  int wrong = INT_MAX;
  for (unsigned k0 = run0; k0 < (unsigned)taken; k0 += runs) {
    int id[kBatch], b = 0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) id[i] = k0 + 32 * i + lane < (unsigned)taken ? page_taken(k0 + 32 * i + lane) : 0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (k0 + 32 * i + lane >= (unsigned)taken) continue;
      const int k = (int)(k0 + 32 * i + lane);
      if (i == 0 || few) b = first_above(take, a.B, k);
      else
        while (take[b] <= k) ++b;
      if (id[i] < 0 || id[i] >= a.num_pages) wrong = min(wrong, k);
      *entry_taken(b, k) = id[i];
    }
  }
  // An id that is no page's: the request that would get it, and those behind it, get none after all.  (The stack still holds
  // what was taken.)
  if (taken) {
    if (wrong != INT_MAX) {
      const uint32_t at = ptx::smem_u32(&s_wrong);
      for (int c = 0; c < ctas; ++c)
        asm volatile("red.relaxed.cluster.shared::cluster.min.s32 [%0], %1;" :: "r"(ctas > 1 ? ptx::mapa(at, c) : at), "r"(wrong) : "memory");
      asm volatile("fence.acq_rel.cluster;" ::: "memory");
    }
    __syncwarp();
    // (relaxed: the tables' stores need not be done; ordered 34.4 us a pass for the 512 prompts, so 33.7)
    if (ctas > 1) ptx::cluster_sync_relaxed();
    else __syncthreads();
    if (s_wrong != INT_MAX) {
      if (ctas > 1) ptx::cluster_sync();               // the stores that are taken back are done
      else __syncthreads();
      const int first = first_above(take, a.B, s_wrong), left = first ? take[first - 1] : 0;
      for (unsigned k = left + me; k < (unsigned)taken; k += all) *entry_taken(first_above(take, a.B, k), k) = -1;
      for (int b = first + me; b < grant; b += all)
        if (want[b] > have[b]) a.n_pages[b] = have[b];
      if (me == 0) {
        *a.free_count = top - left;
        page_error(a, KDTV_ERR_BAD_PAGE);
      }
      grant = first;
    }
  }
  if (a.slots)
    for (long long k = me; k < (long long)a.B * a.N; k += all) {
      const int b = (int)divide((unsigned)k, a.by_N), i = (int)(k - (long long)b * a.N);
      a.slots[k] = slot_of(a, a.prefix_len[b], live_rows(a.n_live, b, a.N), pages_of(b), i, [&](int p) {
        return p >= have[b] ? page_taken(p - have[b] + (b ? take[b - 1] : 0)) : a.page_table[(long long)b * a.max_pages + p];
      });
    }
}

// The slots of many rows, behind the tables.
constexpr int kSlotRows = 8;
__global__ void __launch_bounds__(256) page_slots_kernel(const __grid_constant__ PageArgs a) {
  ptx::grid_dep_wait();
  const int b = blockIdx.y, L = a.prefix_len[b], n = live_rows(a.n_live, b, a.N), pages = a.n_pages[b];
  const int32_t* row = a.page_table + (long long)b * a.max_pages;
  int64_t* out = a.slots + (long long)b * a.N;
  // (the look-ups of a thread's rows are under way together)
  int64_t slot[kSlotRows];
  const int i0 = blockIdx.x * (256 * kSlotRows) + threadIdx.x;
#pragma unroll
  for (int k = 0; k < kSlotRows; ++k) slot[k] = slot_of(a, L, n, pages, i0 + 256 * k, [&](int p) { return row[p]; });
#pragma unroll
  for (int k = 0; k < kSlotRows; ++k)
    if (i0 + 256 * k < a.N) out[i0 + 256 * k] = slot[k];
}

}  // namespace
}  // namespace kdtv

using namespace kdtv;

extern "C" int kdtv_pages_resize(const kdtv_pages_dims* d, const int32_t* prefix_len,
                                 const int32_t* n_live, int32_t* free_pages, int32_t* free_count,
                                 int32_t* n_pages, int32_t* page_table, int64_t* slots,
                                 unsigned int* status, cudaStream_t stream) {
  if (!d || !prefix_len || !free_pages || !free_count || !n_pages || !page_table || !status) return KDTV_ERR_INVALID_ARG;
  if (d->B <= 0 || d->N < 0 || d->page_size <= 0 || d->max_pages <= 0 || d->num_pages <= 0) return KDTV_ERR_INVALID_ARG;
  if ((long long)d->max_pages * d->page_size > (1ll << 30)) return KDTV_ERR_INVALID_ARG;
  if (d->B > KDTV_MAX_POOL_REQUESTS || (long long)d->B * d->N > (1ll << 30) ||
      (long long)d->B * d->max_pages >= (1ll << 31))          // 32-bit sums
    return KDTV_ERR_UNSUPPORTED;
  PageArgs a;
  memset(&a, 0, sizeof(a));
  a.B = d->B; a.N = d->N; a.page_size = d->page_size; a.max_pages = d->max_pages; a.num_pages = d->num_pages;
  a.prefix_len = prefix_len; a.n_live = n_live;
  a.free_pages = free_pages; a.free_count = free_count; a.n_pages = n_pages; a.page_table = page_table;
  a.status = status;
  a.by_page = divisor((unsigned)d->page_size);
  a.by_N = divisor((unsigned)(d->N > 0 ? d->N : 1));
  // A second kernel writes the slots of more rows than the cluster writes in the time that its launch
  // takes.
  const long long rows = (long long)d->B * d->N;
  const bool apart = slots && rows > 32768;
  a.slots = apart || rows == 0 ? nullptr : slots;
  const int ctas = rows <= 4096 && d->B <= 256 ? 1 : kMaxCluster;
  const size_t smem = (size_t)d->B * 16 + (d->B + 31) / 32 * 4;
  if (allow_smem(pages_resize_kernel, smem) != cudaSuccess) return KDTV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPageThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)ctas, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, pages_resize_kernel, a, ctas) != cudaSuccess) return KDTV_ERR_CUDA;
  if (apart) {
    a.slots = slots;
    const unsigned blocks = (unsigned)((d->N + 256 * kSlotRows - 1) / (256 * kSlotRows));
    if (launch_ex(page_slots_kernel, dim3(blocks, (unsigned)d->B), dim3(256), 0, stream, true, a) != cudaSuccess)
      return KDTV_ERR_CUDA;
  }
  return KDTV_OK;
}
