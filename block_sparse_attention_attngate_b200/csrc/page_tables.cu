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
// ids, one for the stores) for a decode step; integer instructions for the
// largest calls (a megabyte of slots), so divisions by the page size are a
// multiplication (14 us -> 7.3 us for 131072 tokens of 1024 requests) and the work is shared
// by up to kMaxCtas CTAs.  When the lengths or the count are updated in place, all reads of them have to
// come before rank 0's writes: then a cluster of eight, whose barrier orders them without a second launch
// or a counter that outlives the call.  Small calls run one CTA of kSmall threads (a barrier of 32 warps costs more
// than their work: 5.7 us -> 3.7 us).
#include <cooperative_groups.h>

#include <algorithm>

#include "seer_device.cuh"
#include "seer_internal.h"

namespace seer {
namespace {

constexpr int kPer = 4;       // requests per thread in the scan
constexpr int kSmall = 128, kLarge = kMaxDecodeB / kPer;   // threads of a CTA
constexpr int kCluster = 8, kMaxCtas = 64;
constexpr int kBatch = 8;   // page ids a thread has on their way at once

// Exclusive scan of two per-thread values over the CTA (totals in *ta, *tb).
template <int THREADS>
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
    long long xa = lane < THREADS / 32 ? ws[lane][0] : 0, xb = lane < THREADS / 32 ? ws[lane][1] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long ya = __shfl_up_sync(0xffffffffu, xa, off), yb = __shfl_up_sync(0xffffffffu, xb, off);
      if (lane >= off) {
        xa += ya;
        xb += yb;
      }
    }
    if (lane < THREADS / 32) {
      ws[lane][0] = xa;
      ws[lane][1] = xb;
    }
  }
  __syncthreads();
  const long long ba = warp ? ws[warp - 1][0] : 0, bb = warp ? ws[warp - 1][1] : 0;
  *ta = ws[THREADS / 32 - 1][0];
  *tb = ws[THREADS / 32 - 1][1];
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
template <int THREADS>
__device__ __forceinline__ void warp_run(int n, int* lo, int* hi) {
  const int warps = gridDim.x * (THREADS / 32), w = blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
  const int run = ((n - 1) / (warps * 32) + 1) * 32;   // n >= 1
  const long long at = (long long)w * run;
  *lo = (int)(at < n ? at : n);
  *hi = n - *lo < run ? n : *lo + run;
}

// x / page for 0 <= x < 2^31, and rounded up
__device__ __forceinline__ int div(const PageParams& p, int x) {
  return p.by_page.div(x);
}
__device__ __forceinline__ int div_up(const PageParams& p, int x) {
  const int q = div(p, x);
  return q + (x - q * p.page != 0 ? 1 : 0);
}

// The requests of this thread in the scan: kPer consecutive ones.  Returns false (to the whole CTA)
// when a length is out of range.  Fills, in shared memory, the length of every request and the
// scans of its appended tokens (plan only) and of its pages.
template <bool PLAN, int THREADS>
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
      const long long room = min((long long)p.width * p.page, (long long)INT32_MAX);
      const bool ok = L[j] >= 0 && n[j] >= 0 && (long long)L[j] + n[j] <= room;
      bad |= !ok;
      if (ok) {
        own[j] = div_up(p, L[j] + n[j]) - div_up(p, L[j]);
        st += n[j];
        sp += own[j];
      }
    } else if (n[j] != 0) {
      const bool ok = L[j] >= 0 && L[j] <= (long long)p.width * p.page;
      bad |= !ok;
      if (ok) {
        own[j] = div_up(p, L[j]);
        sp += own[j];
      }
    }
  }
  long long tt, tp;
  scan2<THREADS>(st, sp, &tt, &tp, ws);
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

template <int THREADS>
__global__ void __launch_bounds__(THREADS) page_plan_kernel(const PageParams p) {
  extern __shared__ int sm[];
  __shared__ long long ws[32][2];
  int *len = sm, *tok = sm + p.B, *pag = sm + 2 * p.B;
  const int B = p.B, page = p.page, pages = p.num_pages;
  const int gt = blockIdx.x * THREADS + threadIdx.x, gn = gridDim.x * THREADS;
  pdl_wait();
  pdl_trigger();
  int T, A, F;
  const bool ok = scan_requests<true, THREADS>(p, len, tok, pag, &T, &A, &F, ws);
  if (p.in_place && gridDim.x > 1) cooperative_groups::this_cluster().sync();   // every CTA has read what rank 0 now writes
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < B; b += THREADS) {
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
    warp_run<THREADS>(A, &lo, &hi);
    int b = lo + lane < hi ? row_of(pag, B, lo + lane) : 0;
    for (int i0 = lo + lane; i0 < hi; i0 += 32 * kBatch) {
      int id[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) id[k] = i0 + 32 * k < hi ? p.free_list[F - 1 - (i0 + 32 * k)] : 0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + 32 * k;
        if (i >= hi) break;
        while (b + 1 < B && pag[b + 1] <= i) ++b;
        const bool good = id[k] >= 0 && id[k] < pages;
        if (!good) report(p.err, SEER_DEVERR_PAGE_INDEX);
        p.block_table[(size_t)b * p.width + div_up(p, len[b]) + (i - pag[b])] = good ? id[k] : -1;
      }
    }
  }
  // appended tokens; a page that is new in this call is read from the stack, not from the table
  if (T > 0) {
    warp_run<THREADS>(T, &lo, &hi);
    int b = lo + lane < hi ? row_of(tok, B, lo + lane) : 0;
    for (int t0 = lo + lane; t0 < hi; t0 += 32 * kBatch) {
      int id[kBatch], pos[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int t = t0 + 32 * k;
        id[k] = pos[k] = 0;
        if (t < hi) {
          while (b + 1 < B && tok[b + 1] <= t) ++b;
          pos[k] = len[b] + (t - tok[b]);
          const int at = div(p, pos[k]), own = div_up(p, len[b]);
          id[k] = *(at < own ? p.block_table + (size_t)b * p.width + at : p.free_list + (F - 1 - (pag[b] + at - own)));
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int t = t0 + 32 * k;
        if (t >= hi) break;
        const bool good = id[k] >= 0 && id[k] < pages;
        if (!good) report(p.err, SEER_DEVERR_PAGE_INDEX);
        p.slot_map[t] = good ? id[k] * page + (pos[k] - div(p, pos[k]) * page) : -1;
        p.positions[t] = pos[k];
      }
    }
  }
  for (int t = T + gt; t < p.max_tokens; t += gn) {
    p.slot_map[t] = -1;
    p.positions[t] = 0;
  }
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) page_release_kernel(const PageParams p) {
  extern __shared__ int sm[];
  __shared__ long long ws[32][2];
  int *len = sm, *pag = sm + p.B;
  const int B = p.B;
  pdl_wait();
  pdl_trigger();
  int T, A, F;
  const bool ok = scan_requests<false, THREADS>(p, len, nullptr, pag, &T, &A, &F, ws);
  if (p.in_place && gridDim.x > 1) cooperative_groups::this_cluster().sync();   // every CTA has read what rank 0 now writes
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < B; b += THREADS)
      p.seqlens_out[b] = ok && p.per_request[b] != 0 ? 0 : len[b];
    if (threadIdx.x == 0) {
      *p.free_count_out = ok ? F + A : F;
      if (!ok) report(p.err, SEER_DEVERR_COUNT);
    }
  }
  if (!ok || A == 0) return;
  int lo, hi;
  warp_run<THREADS>(A, &lo, &hi);
  const int first = lo + (threadIdx.x & 31);
  int b = first < hi ? row_of(pag, B, first) : 0;
  for (int i0 = first; i0 < hi; i0 += 32 * kBatch) {
    int id[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + 32 * k;
      id[k] = 0;
      if (i < hi) {
        while (b + 1 < B && pag[b + 1] <= i) ++b;
        id[k] = p.block_table[(size_t)b * p.width + (i - pag[b])];
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (i0 + 32 * k >= hi) break;
      const bool good = id[k] >= 0 && id[k] < p.num_pages;
      if (!good) report(p.err, SEER_DEVERR_PAGE_INDEX);
      p.free_out[F + i0 + 32 * k] = good ? id[k] : -1;
    }
  }
}

std::atomic<uint64_t> g_limit[2];

// arrays: of p.B ints in shared memory; items: elements to write, at most
cudaError_t launch(void (*small)(const PageParams), void (*large)(const PageParams), PageParams p, int arrays,
                   int64_t items, std::atomic<uint64_t>& done, cudaStream_t s) {
  p.by_page = divisor(p.page);
  p.in_place = p.seqlens == p.seqlens_out || p.free_count == p.free_count_out || p.per_request == p.seqlens_out;
  const bool one = p.B <= kSmall * kPer && items <= 8 * kSmall;
  int ctas = 1;
  if (!one && items > 4 * kLarge)
    ctas = p.in_place ? kCluster : (int)std::min<int64_t>(kMaxCtas, (items + 2 * kLarge - 1) / (2 * kLarge));
  cudaError_t e = ensure_smem_limit(large, 3 * kMaxDecodeB * (int)sizeof(int), done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(one ? kSmall : kLarge);
  cfg.dynamicSmemBytes = (size_t)arrays * p.B * sizeof(int);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.in_place && ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, one ? small : large, p);
}

}  // namespace

cudaError_t launch_page_plan(const PageParams& p, cudaStream_t s) {
  return launch(page_plan_kernel<kSmall>, page_plan_kernel<kLarge>, p, 3, p.max_tokens, g_limit[0], s);
}

cudaError_t launch_page_release(const PageParams& p, cudaStream_t s) {
  // the host does not know how many pages come back; the pool bounds it
  return launch(page_release_kernel<kSmall>, page_release_kernel<kLarge>, p, 2,
                std::min<int64_t>((int64_t)p.B * p.width, p.num_pages), g_limit[1], s);
}

}  // namespace seer
