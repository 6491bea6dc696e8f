// Block tables and slot maps of a paged cache from request lengths, and the
// return of finished requests' pages.
//
// With L_b tokens held, n_b to append and pages of P tokens, request b takes
// a_b = ceil((L_b + n_b) / P) - ceil(L_b / P) new pages from the top of a stack of
// free pages; which ones follows from the exclusive scan of a over the
// requests, and row t of the appended tokens from the exclusive scan of n.
// So every output element is a function of the two scans: each CTA scans all
// requests itself (B <= 4096: four elements a thread, in shared memory), then
// the warps of all CTAs share the new pages and the token rows in contiguous
// runs, finding a run's first request by binary search and walking on from
// there, 32 elements a step (a grid stride would walk past many requests
// between two elements of a thread).
//
// Bound: latency (a launch, one round trip for the lengths, one for the page
// ids, one for the stores); the largest calls write about a megabyte.  One
// CTA for a decode step; a cluster of eight when more than kOneCtaItems elements are
// written.  A cluster rather than a plain grid because the lengths may be
// updated in place: its barrier orders every CTA's reads before rank 0's
// writes without a second launch or a counter that outlives the call.
#include <cooperative_groups.h>

#include "seer_device.cuh"
#include "seer_internal.h"

namespace seer {
namespace {

constexpr int kThreads = 1024;
constexpr int kPer = kMaxDecodeB / kThreads;   // requests per thread in the scan
constexpr int kCluster = 8;

// Exclusive scan of two per-thread values over the CTA (totals in *ta, *tb).
__device__ __forceinline__ void scan2(long long& a, long long& b, long long* ta, long long* tb, long long (*ws)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ia = a, ib = b;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long xa = __shfl_up_sync(0xffffffffu, ia, off), xb = __shfl_up_sync(0xffffffffu, ib, off);
    if (lane >= off) {
      ia += xa;
      ib += xb;
    }
  }
  if (lane == 31) {
    ws[warp][0] = ia;
    ws[warp][1] = ib;
  }
  __syncthreads();
  if (warp == 0) {
    long long xa = ws[lane][0], xb = ws[lane][1];   // kThreads / 32 == 32 warps
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long ya = __shfl_up_sync(0xffffffffu, xa, off), yb = __shfl_up_sync(0xffffffffu, xb, off);
      if (lane >= off) {
        xa += ya;
        xb += yb;
      }
    }
    ws[lane][0] = xa;
    ws[lane][1] = xb;
  }
  __syncthreads();
  const long long ba = warp ? ws[warp - 1][0] : 0, bb = warp ? ws[warp - 1][1] : 0;
  *ta = ws[31][0];
  *tb = ws[31][1];
  a = ba + ia - a;
  b = bb + ib - b;
}

// Last request r in [0, n) with first[r] <= x (first non-decreasing, first[0] = 0 <= x).
__device__ __forceinline__ int row_of(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Elements [lo, hi) of n that this warp handles: equal runs over all warps, whole steps of 32.
__device__ __forceinline__ void warp_run(int n, int* lo, int* hi) {
  const int warps = gridDim.x * (kThreads / 32), w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int run = ((n - 1) / (warps * 32) + 1) * 32;   // n >= 1
  const long long at = (long long)w * run;
  *lo = (int)(at < n ? at : n);
  *hi = n - *lo < run ? n : *lo + run;
}

__device__ __forceinline__ int div_up(int x, int page) { return x / page + (x % page != 0 ? 1 : 0); }

// The requests of this thread in the scan: kPer consecutive ones.  Returns false (to the whole CTA)
// when a length is out of range.  Fills, in shared memory, the length of every request and the
// scans of its appended tokens (plan only) and of its pages.
template <bool PLAN>
__device__ __forceinline__ bool scan_requests(const PageParams& p, int* len, int* tok, int* pag, int* total_tok,
                                              int* total_pag, int* free_count, long long (*ws)[2]) {
  const int F = *p.free_count;
  int L[kPer], n[kPer], own[kPer];
  bool bad = F < 0 || F > p.num_pages;
  long long st = 0, sp = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int b = threadIdx.x * kPer + j;
    L[j] = n[j] = 0;
    if (b < p.B) {
      L[j] = p.seqlens[b];
      n[j] = p.per_request[b];   // plan: tokens to append; release: finished flag
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    own[j] = 0;
    if (PLAN) {
      const long long room = (long long)p.width * p.page;
      const bool ok = L[j] >= 0 && n[j] >= 0 && (long long)L[j] + n[j] <= room;
      bad |= !ok;
      if (ok) {
        own[j] = div_up(L[j] + n[j], p.page) - div_up(L[j], p.page);
        st += n[j];
        sp += own[j];
      }
    } else if (n[j] != 0) {
      const bool ok = L[j] >= 0 && L[j] <= (long long)p.width * p.page;
      bad |= !ok;
      if (ok) {
        own[j] = div_up(L[j], p.page);
        sp += own[j];
      }
    }
  }
  long long tt, tp;
  scan2(st, sp, &tt, &tp, ws);
  if (PLAN) bad |= tt > p.max_tokens || tp > F;
  else bad |= tp > p.num_pages - (long long)F;
  // totals below 2^31 from here on (max_tokens and num_pages are); on a bad call nothing below is used
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int b = threadIdx.x * kPer + j;
    if (b < p.B) {
      len[b] = L[j];
      if (PLAN) {
        tok[b] = (int)st;
        st += n[j];
      }
      pag[b] = (int)sp;
      sp += own[j];
    }
  }
  *total_tok = (int)tt;
  *total_pag = (int)tp;
  *free_count = F;
  return __syncthreads_or(bad) == 0;
}

__global__ void __launch_bounds__(kThreads) page_plan_kernel(const PageParams p) {
  extern __shared__ int sm[];
  __shared__ long long ws[32][2];
  int *len = sm, *tok = sm + p.B, *pag = sm + 2 * p.B;
  const int B = p.B, page = p.page, pages = p.num_pages;
  const int gt = blockIdx.x * kThreads + threadIdx.x, gn = gridDim.x * kThreads;
  pdl_wait();
  pdl_trigger();
  int T, A, F;
  const bool ok = scan_requests<true>(p, len, tok, pag, &T, &A, &F, ws);
  if (gridDim.x > 1) cooperative_groups::this_cluster().sync();   // every CTA has read what rank 0 now writes
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < B; b += kThreads) {
      // bounded: requests in range sum to at most max_tokens
      const int n = ok ? (b + 1 < B ? tok[b + 1] : T) - tok[b] : 0;
      p.seqlens_out[b] = len[b] + n;
      p.cu_tokens[b] = ok ? tok[b] : 0;
    }
    if (threadIdx.x == 0) {
      p.cu_tokens[B] = ok ? T : 0;
      *p.free_count_out = ok ? F - A : F;
      if (!ok) report(p.err, SEER_DEVERR_COUNT);
    }
  }
  if (!ok) T = A = 0;
  const int lane = threadIdx.x & 31;
  int lo, hi;
  // new pages: element i is page i - A_b of request b
  if (A > 0) {
    warp_run(A, &lo, &hi);
    int b = lo + lane < hi ? row_of(pag, B, lo + lane) : 0;
    for (int i = lo + lane; i < hi; i += 32) {
      while (b + 1 < B && pag[b + 1] <= i) ++b;
      int id = p.free_list[F - 1 - i];
      if (id < 0 || id >= pages) {
        report(p.err, SEER_DEVERR_PAGE_INDEX);
        id = -1;
      }
      p.block_table[(size_t)b * p.width + div_up(len[b], page) + (i - pag[b])] = id;
    }
  }
  // appended tokens; a page that is new in this call is read from the stack, not from the table
  if (T > 0) {
    warp_run(T, &lo, &hi);
    int b = lo + lane < hi ? row_of(tok, B, lo + lane) : 0;
    for (int t = lo + lane; t < hi; t += 32) {
      while (b + 1 < B && tok[b + 1] <= t) ++b;
      const int L = len[b], pos = L + (t - tok[b]);
      const int at = pos / page, own = div_up(L, page);
      const int id = at < own ? p.block_table[(size_t)b * p.width + at] : p.free_list[F - 1 - (pag[b] + at - own)];
      const bool good = id >= 0 && id < pages;
      if (!good) report(p.err, SEER_DEVERR_PAGE_INDEX);
      p.slot_map[t] = good ? id * page + (pos - at * page) : -1;
      p.positions[t] = pos;
    }
  }
  for (int t = T + gt; t < p.max_tokens; t += gn) {
    p.slot_map[t] = -1;
    p.positions[t] = 0;
  }
}

__global__ void __launch_bounds__(kThreads) page_release_kernel(const PageParams p) {
  extern __shared__ int sm[];
  __shared__ long long ws[32][2];
  int *len = sm, *pag = sm + p.B;
  const int B = p.B;
  pdl_wait();
  pdl_trigger();
  int T, A, F;
  const bool ok = scan_requests<false>(p, len, nullptr, pag, &T, &A, &F, ws);
  if (gridDim.x > 1) cooperative_groups::this_cluster().sync();   // every CTA has read what rank 0 now writes
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < B; b += kThreads)
      p.seqlens_out[b] = ok && p.per_request[b] != 0 ? 0 : len[b];
    if (threadIdx.x == 0) {
      *p.free_count_out = ok ? F + A : F;
      if (!ok) report(p.err, SEER_DEVERR_COUNT);
    }
  }
  if (!ok || A == 0) return;
  int lo, hi;
  warp_run(A, &lo, &hi);
  const int first = lo + (threadIdx.x & 31);
  int b = first < hi ? row_of(pag, B, first) : 0;
  for (int i = first; i < hi; i += 32) {
    while (b + 1 < B && pag[b + 1] <= i) ++b;
    int id = p.block_table[(size_t)b * p.width + (i - pag[b])];
    if (id < 0 || id >= p.num_pages) {
      report(p.err, SEER_DEVERR_PAGE_INDEX);
      id = -1;
    }
    p.free_out[F + i] = id;
  }
}

std::atomic<uint64_t> g_limit[2];

cudaError_t launch(void (*kern)(const PageParams), const PageParams& p, int ctas, size_t smem, std::atomic<uint64_t>& done,
                   cudaStream_t s) {
  cudaError_t e = ensure_smem_limit(kern, 3 * kMaxDecodeB * (int)sizeof(int), done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// Elements written by one CTA before eight share them.
constexpr int kOneCtaItems = 4 * kThreads;

}  // namespace

cudaError_t launch_page_plan(const PageParams& p, cudaStream_t s) {
  return launch(page_plan_kernel, p, p.max_tokens > kOneCtaItems ? kCluster : 1, 3 * (size_t)p.B * sizeof(int),
                g_limit[0], s);
}

cudaError_t launch_page_release(const PageParams& p, cudaStream_t s) {
  // the host does not know how many pages come back; the pool bounds it
  const int64_t most = (int64_t)p.B * p.width;
  return launch(page_release_kernel, p, (most < p.num_pages ? most : p.num_pages) > kOneCtaItems ? kCluster : 1,
                2 * (size_t)p.B * sizeof(int), g_limit[1], s);
}

}  // namespace seer
