// d2f_page_map kernels: the block table, slot map and append list of a batch of
// requests from their lengths, with pages off the device free list.
//
// Source: "D2F: 확산 언어 모델이 KV 캐시를 얻고 자기회귀 모델보다 2.5배 빨라지는
// 방법", §운영 관점 (a paged cache; a page holds one block of one sequence).
//
// Pages are handed out in (request, block) order, so everything follows from two
// running sums over the requests: of their tokens (row_start) and of their pages.
// Every CTA that fills the maps forms the sums itself (a few thousand additions)
// and then finds a row's or a page's request by bisection in shared memory.
//
// Measured: 16 requests (512 rows at most) 7.0 us, 1024 requests with 2 million rows
// 18.4 us, of which the 17 MB of the slot map would take 3: two launches, each a chain of
// dependent loads and barriers (7 us for the plan), and some 300 instructions per four
// rows (bisection, one division a request). Every CTA planning for itself, in one launch,
// took as long.
#include "d2f_internal.cuh"

namespace d2f {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kOneCtaRows = 16384;  // slots + 4 per list entry

__device__ __forceinline__ longlong2 warp_scan(longlong2 v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v.x, o);
    const long long y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) {
      v.x += x;
      v.y += y;
    }
  }
  return v;
}

// Exclusive running sum over the CTA's threads of (x, y), and the totals.
__device__ longlong2 block_scan(longlong2 v, longlong2 *warp_sum, longlong2 &total) {
  static_assert(kWarps == 32, "one lane per warp");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const longlong2 inc = warp_scan(v, lane);
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  const longlong2 all = warp_scan(warp_sum[lane], lane);
  const int before = warp > 0 ? warp - 1 : 0;
  const long long bx = __shfl_sync(0xffffffffu, all.x, before);
  const long long by = __shfl_sync(0xffffffffu, all.y, before);
  total.x = __shfl_sync(0xffffffffu, all.x, 31);
  total.y = __shfl_sync(0xffffffffu, all.y, 31);
  __syncthreads();
  return make_longlong2((warp > 0 ? bx : 0) + inc.x - v.x, (warp > 0 ? by : 0) + inc.y - v.y);
}

// Largest i of [0, n) with start[i] <= x (start ascending, start[0] <= x).
__device__ __forceinline__ int find(const int *start, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Phase kPlan decides the admission and writes the per-request results; phase kFill
// writes the maps from those results (which may have replaced the inputs in place);
// kBoth does the two in one CTA.
constexpr int kPlan = 1, kFill = 2, kBoth = 3;

template <int PHASE>
__global__ void __launch_bounds__(kThreads) page_map_kernel(const PageMapArgs a) {
  extern __shared__ int sm[];
  int *row0 = sm;                  // [batch]: first packed row of each request
  int *page0 = row0 + a.batch;     // [batch]: pages handed out before the request
  int *ctxp = page0 + a.batch;     // [batch]: cached pages before, -1: not admitted
  __shared__ longlong2 warp_sum[kWarps];
  __shared__ int bad_s;
  const int tid = threadIdx.x, B = a.block_size, batch = a.batch;
  if (PHASE == kPlan) grid_launch_dependents();  // (the fill waits for this grid's end)
  grid_dependency_wait();
  const int per = (batch + kThreads - 1) / kThreads;  // consecutive requests of a thread
  const int b0 = min(tid * per, batch), b1 = min(b0 + per, batch);
  int n_pages = 0, n_rows = 0, free0 = 0;  // (0: an inconsistent state, empty maps)

  if (PHASE & kPlan) {
    free0 = *a.free_count;
    if (tid == 0) bad_s = free0 < 0;
    __syncthreads();
    longlong2 sum = make_longlong2(0, 0);  // tokens, pages
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
      const int nn = a.num_new[b], c = a.ctx_len[b];
      if (nn < 0 || c < 0 || (nn > 0 && c % B != 0)) {
        bad = true;
        continue;
      }
      const long long need = ((long long)nn + B - 1) / B;
      const bool fits = c / B + need <= a.max_pages_per_seq && (long long)c + nn <= 0x7fffffffLL;
      sum.x += nn;
      sum.y += fits ? need : 0;
    }
    if (bad) bad_s = 1;
    longlong2 total;
    longlong2 at = block_scan(sum, warp_sum, total);
    const bool refused = bad_s || total.x > a.capacity;  // an inconsistent state
    if (refused) {
      for (int b = b0; b < b1; ++b) {
        a.row_start[b] = 0;
        a.admitted[b] = 0;
        if (a.fresh) a.ctx_out[b] = a.ctx_len[b];
      }
      if (tid == 0) {
        set_err(a.err, D2F_ERR_INVALID_ARG);
        a.row_start[batch] = 0;
        *a.n_append = -1;
        if (a.fresh) *a.free_out = free0;
      }
    } else {
      n_rows = (int)total.x;
    }
    const long long most = min(free0, a.max_append);
    // requests are admitted while the running sum of pages fits
    long long mine = 0, given = 0;
    for (int b = b0; b < b1 && !refused; ++b) {
      const int nn = a.num_new[b], c = a.ctx_len[b];
      const long long need = ((long long)nn + B - 1) / B;
      const bool fits = c / B + need <= a.max_pages_per_seq && (long long)c + nn <= 0x7fffffffLL;
      const bool ok = fits && at.y + mine + need <= most;
      if (PHASE & kFill) {
        row0[b] = (int)at.x;
        page0[b] = (int)min(at.y + mine, (long long)0x7fffffff);
        ctxp[b] = ok ? c / B : -1;
      }
      if (fits) mine += need;
      if (ok) given += need;
      else set_err(a.err, D2F_ERR_NO_PAGE);
      a.row_start[b] = (int)at.x;
      a.admitted[b] = ok;
      a.ctx_out[b] = ok ? c + nn : c;
      at.x += nn;
    }
    block_scan(make_longlong2(given, 0), warp_sum, total);
    n_pages = (int)total.x;
    if (tid == 0 && !refused) {
      a.row_start[batch] = n_rows;
      *a.n_append = n_pages;
      *a.free_out = free0 - n_pages;
    }
  } else if (*a.n_append >= 0) {
    // the plan's results: admission, starts and the context after it
    longlong2 sum = make_longlong2(0, 0);
    for (int b = b0; b < b1; ++b)
      if (a.admitted[b]) sum.y += (a.num_new[b] + (long long)B - 1) / B;
    longlong2 total;
    long long p = block_scan(sum, warp_sum, total).y;
    for (int b = b0; b < b1; ++b) {
      const bool ok = a.admitted[b];
      const int nn = a.num_new[b];
      row0[b] = a.row_start[b];
      page0[b] = (int)p;
      ctxp[b] = ok ? (a.ctx_out[b] - nn) / B : -1;
      if (ok) p += (nn + (long long)B - 1) / B;
    }
    n_pages = *a.n_append;
    n_rows = a.row_start[batch];
    free0 = *a.free_out + n_pages;
  }
  if (!(PHASE & kFill)) return;
  __syncthreads();

  const int64_t first = (int64_t)blockIdx.x * kThreads + tid, step = (int64_t)gridDim.x * kThreads;
  // the list, and the table's new entries. Requests without pages share a start, so
  // the last request whose start is <= p is the one that owns page p.
  for (int64_t p = first; p < a.max_append; p += step) {
    int src = -1, dst = -1, rows = 0;
    if (p < n_pages) {
      const int b = find(page0, batch, (int)p);
      const int i = (int)p - page0[b];
      dst = a.free_pages[free0 - 1 - p];
      src = row0[b] + i * B;
      rows = min(B, a.num_new[b] - i * B);
      a.page_table[(int64_t)b * a.max_pages_per_seq + ctxp[b] + i] = dst;
    }
    a.app_src[p] = src;
    a.app_dst[p] = dst;
    a.app_rows[p] = rows;
  }
  // slots, four rows a thread: one search, then a walk (a row's request and page are
  // mostly its predecessor's)
  for (int64_t q = first; 4 * q < a.capacity; q += step) {
    const int r0 = (int)(4 * q), r1 = min(r0 + 4, a.capacity);
    int64_t slot[4];
    int b = r0 < n_rows ? find(row0, batch, r0) : 0;
    int next = 0, o = 0;      // end of the request's rows; offset in the page
    const int *page = nullptr;  // the request's page of this row on the list
    int64_t base = -1;        // page * B, -1: a refused request
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + j;
      slot[j] = -1;
      if (r >= n_rows) continue;
      const bool turn = r >= next;  // another request (the first row's is known)
      if (turn) {
        if (j == 0) next = b + 1 < batch ? row0[b + 1] : n_rows;
        while (r >= next) {
          ++b;
          next = b + 1 < batch ? row0[b + 1] : n_rows;
        }
        const int t = r - row0[b];
        page = a.free_pages + (free0 - 1 - page0[b] - t / B);
        o = t % B;
      } else if (++o == B) {
        o = 0;
        --page;
      }
      if (turn || o == 0) base = ctxp[b] < 0 ? -1 : (int64_t)*page * B;
      if (base >= 0) slot[j] = base + o;
    }
    if (r1 - r0 == 4 && (reinterpret_cast<uintptr_t>(a.slot) & 15) == 0) {
      reinterpret_cast<longlong2 *>(a.slot + r0)[0] = make_longlong2(slot[0], slot[1]);
      reinterpret_cast<longlong2 *>(a.slot + r0)[1] = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (r0 + j < r1) a.slot[r0 + j] = slot[j];
    }
  }
}

constexpr size_t smem_bytes(int batch) { return (size_t)batch * 3 * sizeof(int); }

template <int PHASE>
cudaError_t launch_phase(const PageMapArgs &a, unsigned grid, size_t smem, cudaStream_t s) {
  if (smem > 48 * 1024) {
    // the largest batch's bytes, not this one's: another thread may be about to launch with
    // more than this call needs
    const cudaError_t e = cudaFuncSetAttribute(
        page_map_kernel<PHASE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        (int)smem_bytes(kPageMapMaxBatch));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, page_map_kernel<PHASE>, a);
}

}  // namespace

cudaError_t launch_page_map(const PageMapArgs &a, cudaStream_t s) {
  const size_t smem = smem_bytes(a.batch);
  // One CTA does it all up to some ten thousand rows; beyond, a second launch fills the
  // maps on every SM.
  if ((long long)a.capacity + 4LL * a.max_append <= kOneCtaRows)
    return launch_phase<kBoth>(a, 1, smem, s);
  const cudaError_t e = launch_phase<kPlan>(a, 1, 0, s);
  if (e != cudaSuccess) return e;
  const long long work = max((long long)a.capacity / 4, (long long)a.max_append);
  const unsigned grid = (unsigned)min(2LL * max(1, num_sms_current_device()),
                                      (work + kThreads - 1) / kThreads);
  return launch_phase<kFill>(a, grid, smem, s);
}

}  // namespace d2f
