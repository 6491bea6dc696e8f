// Attention of one new token per sequence over its whole cache, split over the
// cache's length and joined.
//
// For query head i of KV head h and tokens t in [lo_b, hi_b):
//   s_t = scale q_i . K_t,   out = sum_t exp(s_t) V_t / sum_t exp(s_t)
// by the running maximum m, sum l and output o (log2 domain, fp32):
//   m' = max(m, max s),  o' = o 2^(m - m') + sum 2^(s - m') V,  l' likewise,
// and pieces (m_i, l_i, o_i) of one row join by the same rule.
//
// Bound: HBM -- every key and value is read once; three products of g heads a key, 15 % of what the warp-level tensor
// instructions sustain (measured with inputs that change from call to call, against the copy bandwidth: 4 x 65536
// tokens, 8 KV heads of 128, four query heads each, pages of 64, bf16: 167 to 171 us, 96 to 98 %; 16 sequences of 8000 to 32000
// tokens, five heads, token-major pages of 16, fp16: 204 to 209 us, 93 to 95 %; 8 x 32768 tokens, 4 KV heads of 128, 16 heads each:
// 101 us, 81 %; one sequence of 2048 tokens, one KV head: 8.6 us, all of it latency: lengths, page ids, rows, the merge, the join's
// two round trips).  Rows of some hundred tokens are two to three times as long as their bytes: 8 x 1000 tokens 16.4 us (floor 5.0),
// 64 x 300 25 us (12.0), one row of 32768 beside 63 of 20 51 us (21.3).
//
// The figures of the choices below are of graphs that repeat one call, with the weights of one rounding (below); inputs under
// 126 MB then lie in L2, and a call with others takes 10 to 15 % more.
//
// Split.  The rows' (sequence, KV head) tokens in units of kDenseUnit are one long axis; equal ranges of it are the work
// of as many teams, one wave.  A team's warps take its steps of 4 KB of keys and 4 KB of values in turn, each through a ring
// of shared-memory slots that it fills itself (cp.async, kSlots - 1 slots ahead, on across the ends of rows).  No
// warp waits for another but at the end of a row.  cp.async of 16-byte chunks takes any page
// size and stride: tokens that are out of range or on a bad page are filled
// with zeros and masked, whatever lies there.
// A team is a CTA when the rows are long (its warps merge their parts of a row in shared memory, so that a row leaves few
// pieces: one row of 65536 tokens took 59 us with a piece from every warp, 15 us with one from every CTA), and a single warp
// when they are short (a merge costs 1.5 us: 64 sequences of up to 600 tokens 64 us with CTAs, 24 us with warps).  A row
// counts kPad units on top of its own, about what a merge costs, so that ranges of many short rows beside few long ones take
// alike.
// Twelve warps with three slots: the computation of a step is long (0.7 us), so its warps have to be many, and
// more bytes in flight than the 96 KB an SM of this choice measured slower (12 x 4 slots: 185 us against 168, 8 x 6: 182).
//
// Products.  Both are taken transposed so that 16 tokens (or 16 channels) fill the
// long side of the 16x8x16 instruction and the group's heads the short one (eight a
// tile; two tiles above eight): S^T = K Q^T with K as it lies, then O^T = V^T P^T,
// with V^T from transposing loads and P^T from the scores' registers by one
// 8x8 register transpose each.  A lane then holds the same two heads' columns in S, m, l and O.
//
// A row that lies in one range is finished there; the pieces of the others go to
// the workspace in register order, and the join kernel merges them.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "seer_device.cuh"
#include "seer_internal.h"

namespace seer {
namespace {

constexpr int kWarps = 12, kSlots = 3;   // of a CTA, of a warp's ring
constexpr int kThreads = kWarps * 32;
// Rows an SM from which on teams are single warps whatever the lengths.  A long row among so many then lies in hundreds of ranges,
// which the join takes one after another: 128 sequences of 20 tokens, one of them 20000, 8 KV heads of 128: 73 us, floor 14.
constexpr int kTeamRows = 6;
constexpr int kTeamUnits = 24;     // units of the mean token's row from which on teams are CTAs (1000 tokens: 22 us against 29)
constexpr int kPad = 6;
constexpr int kMinUnits = 4, kMinUnitsTeam = 8;   // of a range, about (warps: 64 short sequences 24 us, 31 us with eight)
// While the mean row, padding included, is no longer than this there are as many ranges as rows, if there are teams for them: equally
// long rows then lie in one range each and need no join, which takes 2.4 us (100 tokens: 6.5 us against 8.8).  Ranges are equal,
// so rows of different lengths are still cut where the ranges end.
constexpr int kWholeUnits = 24;
constexpr int kSlotBytes = 4096;   // keys or values of one step
constexpr int kMaskSteps = 4;      // steps whose masks are kept: more than are in the ring
static_assert(kMaskSteps > (kSlots + 1) / 2, "a mask outlives its step");
constexpr int kJoinWarps = 32, kNarrowWarps = 8;
constexpr int kWideRows = 8;       // rows up to which a join takes a CTA for each

template <int D>
constexpr int step_tokens() { return kSlotBytes / (2 * D); }   // 16 (d = 128) or 32 (d = 64)

// d = 128: a row is 256 bytes, which L2 may fetch at once; d = 64: the next 128 bytes may be another head's.
template <int D>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  if constexpr (D == 128)
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, __nv_bfloat16) {
  mma_bf16_16816(d, a0, a1, a2, a3, b0, b1);
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A weight meets V as two numbers of the cache's type, its leading bits (cut, not rounded, so that the rest is not negative)
// and the rest, each with a product of its own: 2^-15 (bf16) or 2^-21 (fp16) of it is lost.  One rounding loses up to 2^-8 or
// 2^-11, as much as the output's own, and left the outputs a quarter to a third further from their 64-bit values.  The rest is
// kept above zero: a value that is infinite and seen then gives infinity, not 0 x infinity (while its weight's leading bits are
// not 0: fp16 down to 2^-38 of the largest).
// fp16 has few exponents: its weights are 2^kLift times theirs (2^14 for the row's largest), with the sum, so that they
// keep those bits down to 2^-18 of the largest and are good to 2^-37 of it below (unlifted, all below 2^-25 are lost, however
// many they are).
template <typename T>
constexpr int kLift = std::is_same<T, __half>::value ? 14 : 0;

__device__ __forceinline__ void split2(float a, float b, uint32_t& lead, uint32_t& rest, __nv_bfloat16) {
  const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
  lead = __byte_perm(x, y, 0x7632);
  rest = pack_bf16(fmaxf(a - __uint_as_float(x & 0xffff0000u), 1e-36f), fmaxf(b - __uint_as_float(y & 0xffff0000u), 1e-36f));
}
__device__ __forceinline__ void split2(float a, float b, uint32_t& lead, uint32_t& rest, __half) {
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(lead) : "f"(b), "f"(a));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lead));
  const __half2 r = __floats2half2_rn(fmaxf(a - x.x, 0x1p-24f), fmaxf(b - x.y, 0x1p-24f));
  rest = *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint16_t round1(float a, __nv_bfloat16) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(a));
}
__device__ __forceinline__ uint16_t round1(float a, __half) { return __half_as_ushort(__float2half_rn(a)); }

// Tokens [lo, hi) that sequence b's new token sees.
__device__ __forceinline__ void token_range(const DenseParams& p, int len, int* lo, int* hi) {
  const int n = min(max(len, 0), p.cap);
  *hi = n;
  *lo = p.window > 0 ? max(n - p.window, 0) : 0;
}
__device__ __forceinline__ int units_of(const DenseParams& p, int len) {
  int lo, hi;
  token_range(p, len, &lo, &hi);
  return (hi - lo + kDenseUnit - 1) / kDenseUnit;
}

// A range's part of one row: tokens [t0, t1) of sequence b, KV head h.
struct Part {
  int b, h;
  int first, units;   // of the row's tokens, on the axis (its padding lies before them)
  int t0, t1;
};

__device__ __forceinline__ void clip(const DenseParams& p, const int* len, int u0, int u1, Part* r) {
  int lo, hi;
  token_range(p, len[r->b], &lo, &hi);
  const int skip = max(u0 - r->first, 0), left = max(u1 - r->first, 0);
  r->t0 = lo + skip * kDenseUnit;
  r->t1 = left >= r->units ? hi : lo + left * kDenseUnit;
}

// The part of the row that unit u0 < Hkv * pre[B] belongs to; empty when the range ends in the row's padding.  For whole warps.
__device__ __forceinline__ void first_part(const DenseParams& p, const int* pre, const int* len, int u0, int u1, Part* r) {
  // the last sequence that starts at or before u0 (a sequence without units shares its successor's start)
  int b = 0;
  if (p.B <= 32) {
    const int lane = threadIdx.x & 31;
    b = __popc(__ballot_sync(0xffffffffu, lane < p.B && pre[min(lane, p.B)] * p.Hkv <= u0)) - 1;
  } else {
    for (int hi = p.B; hi - b > 1;) {
      const int mid = (b + hi) >> 1;
      if (pre[mid] * p.Hkv <= u0) b = mid;
      else hi = mid;
    }
  }
  const int span = pre[b + 1] - pre[b];
  r->b = b;
  r->units = span - p.pad;
  r->h = (int)((uint32_t)(u0 - pre[b] * p.Hkv) / (uint32_t)span);
  r->first = pre[b] * p.Hkv + r->h * span + p.pad;
  clip(p, len, u0, u1, r);
}

// The range's next part; false at its end.
__device__ __forceinline__ bool next_part(const DenseParams& p, const int* pre, const int* len, int u0, int u1, Part* r) {
  r->first += r->units + p.pad;
  if (r->first >= u1) return false;
  if (++r->h == p.Hkv) {
    r->h = 0;
    do ++r->b;
    while (pre[r->b + 1] == pre[r->b]);   // ends: first < u1 <= the axis' length
    r->units = pre[r->b + 1] - pre[r->b] - p.pad;
  }
  clip(p, len, u0, u1, r);
  return true;
}

// Element offset of token t of sequence b and whether it is readable (t inside the cache).
__device__ __forceinline__ bool locate(const DenseParams& p, const KvPlain& kv, int page_id, int b, int t, int h,
                                       int64_t* off) {
  if (kv.paged) {
    const bool ok = page_id >= 0 && page_id < kv.num_pages;
    *off = ok ? page_id * kv.stride_b + h * kv.stride_h + (int64_t)(t - p.by_page.div(t) * p.page) * kv.stride_t : 0;
    return ok;
  }
  *off = b * kv.stride_b + h * kv.stride_h + t * kv.stride_t;
  return true;
}

// Output and log-sum-exp of one head's channels 16 k + quad and + 8 from its sums (log2 domain).
template <typename T, int D>
__device__ __forceinline__ void finish(const DenseParams& p, size_t row0, int head, int k, int quad, float2 o, float m, float l) {
  if (head >= p.g) return;
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  uint16_t* out = p.out + (row0 + head) * D + k * 16 + quad;
  out[0] = round1(o.x * inv, T());
  out[8] = round1(o.y * inv, T());
  if (p.lse && k == 0 && quad == 0)
    p.lse[row0 + head] = l == 0.f ? -INFINITY : (m + (log2f(l) - kLift<T>)) * 0.6931471805599453f;
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) dense_decode_kernel(const __grid_constant__ DenseParams p) {
  constexpr int TS = step_tokens<D>();
  constexpr int MT = TS / 16;        // token tiles a step
  constexpr int KS = D / 16;         // channel steps
  constexpr int CPR = D / 8;         // 16-byte chunks a row
  constexpr int RPI = 32 / CPR;      // rows a warp-wide copy covers
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t masks[kWarps][kMaskSteps];
  __shared__ int scan_ws[kWarps];
  __shared__ float squares_ws[kWarps];
  constexpr int kSets = NT == 1 ? 2 : 1;   // shared memory is full with two of 16 heads
  __shared__ float2 parts_ml[kSets][kWarps][NT * 8];   // the warps' maxima and sums
  constexpr int kRing = kWarps * kSlots * kSlotBytes, kParts = kWarps * KS * 512;
  float4* parts_o = reinterpret_cast<float4*>(smem + kRing);          // the warps' outputs of one head tile
  int* pre = reinterpret_cast<int*>(smem + kRing + kParts);            // [B + 1]
  int* len = pre + p.B + 1;                                            // [B]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane >> 2, c2 = 2 * (lane & 3);   // row of a tile, first of the lane's two columns

  pdl_wait();
  pdl_trigger();

  // exclusive scan of the sequences' units, a row's padding with them
  int total = 0, filled = 0;   // units of one KV head's rows, rows with tokens
  float sq = 0.f;              // squares of the rows' own units
  auto row_units = [&](int b, int* L) {
    *L = b < p.B ? p.seqlens[b] : 0;
    if (*L > p.cap && blockIdx.x == 0) report(p.err, SEER_DEVERR_COUNT);
    const int n = units_of(p, *L);
    return n > 0 ? n + p.pad : 0;
  };
  auto squares = [&](int n) {
    float x = n > 0 ? (float)(n - p.pad) : 0.f;
    x *= x;
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
  };
  auto warp_scan = [&](int x) {   // inclusive
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    return x;
  };
  if (p.B <= 32) {   // every warp for itself: all write the same
    int L;
    const int n = row_units(lane, &L), inc = warp_scan(n);
    if (lane < p.B) {
      pre[lane] = inc - n;
      len[lane] = L;
    }
    total = __shfl_sync(0xffffffffu, inc, 31);
    filled = __popc(__ballot_sync(0xffffffffu, n > 0));
    sq = squares(n);
    if (lane == 0) pre[p.B] = total;
    __syncwarp();
  } else {
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      int L;
      const int n = row_units(b, &L), inc = warp_scan(n);
      const float x = squares(n);
      if (lane == 31) {
        scan_ws[warp] = inc;
        squares_ws[warp] = x;
      }
      filled += __syncthreads_count(n > 0);
      int before = 0, all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? scan_ws[w] : 0;
        all += scan_ws[w];
        sq += squares_ws[w];
      }
      if (b < p.B) {
        pre[b] = total + before + inc - n;
        len[b] = L;
      }
      total += all;
      __syncthreads();
    }
    if (threadIdx.x == 0) pre[p.B] = total;
    __syncthreads();
  }

  const int W = gridDim.x * kWarps, gw = blockIdx.x * kWarps + warp;
  const int axis = total * p.Hkv;   // units of all rows
  // CTAs when every row can have one, or when the mean token's row is long
  const bool wide = p.pad > 0 && (filled * p.Hkv <= (int)gridDim.x || sq >= (float)kTeamUnits * (total - filled * p.pad));
  const int S = wide ? kWarps : 1;  // warps of a team
  // rows without a token
  for (int r = gw; r < p.B * p.Hkv; r += W) {
    const int b = r / p.Hkv, h = r - b * p.Hkv;
    if (pre[b + 1] != pre[b]) continue;
    uint16_t* o = p.out + ((size_t)b * p.Hq + (size_t)h * p.g) * D;
    for (int i = lane; i < p.g * D; i += 32) o[i] = 0;
    if (p.lse)
      for (int i = lane; i < p.g; i += 32) p.lse[(size_t)b * p.Hq + h * p.g + i] = -INFINITY;
    if (p.by_row && lane == 0) p.join[r] = make_int4(0, 0, 0, 0);
  }

  const uint32_t ring = smem_u32(smem) + warp * kSlots * kSlotBytes;
  const int team = wide ? blockIdx.x : gw;
  const int rows = filled * p.Hkv;
  int G = (axis + (wide ? kMinUnitsTeam : kMinUnits) - 1) / (wide ? kMinUnitsTeam : kMinUnits);   // ranges
  if (wide) G = axis <= kWholeUnits * rows ? rows : max(G, rows);
  G = min(G, wide ? (int)gridDim.x : W);
  int4 entry = make_int4(0, 0, 0, 0);
  // ranges of base units, the first `extra` of them one more
  const int base = G ? (int)((uint32_t)axis / (uint32_t)G) : 0, extra = axis - base * G;
  int u0 = 0, u1 = 0;
  Part rd, nx;     // being computed; of the next request (whose page ids are on their way)
  rd.t0 = rd.t1 = 0;
  if (team < G) {
    u0 = team * base + min(team, extra);
    u1 = u0 + base + (team < extra ? 1 : 0);
    first_part(p, pre, len, u0, u1, &rd);
  }
  if (rd.t0 < rd.t1) {
    nx = rd;
    int rj = wide ? warp : 0, nj = rj;   // this warp's next step of the part
    bool nx_ok = true, values = false;   // the next request is of a step's keys, or of the values beside the last keys
    auto settle = [&]() {   // to the part that holds step nj
      while (nx_ok && nx.t0 + nj * TS >= nx.t1) {
        nj -= (nx.t1 - nx.t0 + TS - 1) / TS;
        nx_ok = next_part(p, pre, len, u0, u1, &nx);
      }
    };
    settle();
    int id_k = 0, id_v = 0, nstep = 0;
    uint32_t fill = ring;                // slot of the next request
    int64_t off_v = 0;                   // values of the last requested keys, one token a lane
    uint32_t valid = 0;
    auto fetch_ids = [&]() {   // page ids of nx's tokens, one token a lane
      const int t = nx.t0 + nj * TS + lane;
      if (lane < TS && t < nx.t1) {
        const int page = p.by_page.div(t);
        if (p.k.paged) id_k = p.k.block_table[(int64_t)nx.b * p.k.max_pages + page];
        if (p.v.paged) id_v = p.v.block_table[(int64_t)nx.b * p.v.max_pages + page];
      }
    };
    const int ch = lane % CPR;
    auto copy = [&](const uint16_t* data, int64_t off) {
#pragma unroll
      for (int i = 0; i < TS / RPI; ++i) {
        const int r = i * RPI + lane / CPR;
        const int64_t a = __shfl_sync(0xffffffffu, off, r);
        cp_async16<D>(fill + r * (2 * D) + ((ch ^ (r & 7)) << 4), data + a + ch * 8, (valid >> r) & 1);
      }
    };
    auto request = [&]() {   // fill the next slot: a step's keys, then its values, in turn
      if (values) {
        copy(p.v.data, off_v);
        values = false;
      } else if (nx_ok) {
        const int t = nx.t0 + nj * TS + lane;
        int64_t off_k = 0;
        off_v = 0;
        bool good = lane < TS && t < nx.t1;
        if (good) {
          const bool gk = locate(p, p.k, id_k, nx.b, t, nx.h, &off_k);
          const bool gv = locate(p, p.v, id_v, nx.b, t, nx.h, &off_v);
          good = gk && gv;
          if (!good) report(p.err, SEER_DEVERR_PAGE_INDEX);
        }
        valid = __ballot_sync(0xffffffffu, good);
        if (lane == 0) masks[warp][nstep % kMaskSteps] = valid;
        ++nstep;
        copy(p.k.data, off_k);
        values = true;
        nj += S;
        settle();
        if (nx_ok) fetch_ids();
      }
      cp_commit();   // one group a slot, empty behind the range's end
      fill = fill == ring + (kSlots - 1) * kSlotBytes ? ring : fill + kSlotBytes;
    };
    if (nx_ok) fetch_ids();
#pragma unroll
    for (int s = 0; s < kSlots - 1; ++s) request();

    uint32_t q[NT][KS][2];
    float o[NT][KS][4], m[NT][2], l[NT][2];
    int step = 0;
    uint32_t take = ring;   // slot of the next keys or values to compute with
    int parity = 0;
    do {   // parts of the range
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int head = n * 8 + quad;
        const uint16_t* src = p.q + ((size_t)rd.b * p.Hq + (size_t)rd.h * p.g + head) * D + c2;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          q[n][k][0] = head < p.g ? *reinterpret_cast<const uint32_t*>(src + k * 16) : 0u;
          q[n][k][1] = head < p.g ? *reinterpret_cast<const uint32_t*>(src + k * 16 + 8) : 0u;
          o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
        }
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
      }
      for (; rd.t0 + rj * TS < rd.t1; rj += S) {
        // the next slot has arrived for every lane, and every lane is done with the one before, which is filled again
        auto next_slot = [&]() {
          cp_wait<kSlots - 2>();
          __syncwarp();
          request();
          const uint32_t at = take;
          take = take == ring + (kSlots - 1) * kSlotBytes ? ring : take + kSlotBytes;
          return at;
        };
        const uint32_t kb = next_slot();
        const uint32_t mask = masks[warp][step % kMaskSteps];

        // S^T = K Q^T
        float s[MT][NT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          float s2[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][n][j] = s2[n][j] = 0.f;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const int r = i * 16 + (lane & 15), ch = 2 * k + (lane >> 4);
            uint32_t a0, a1, a2, a3;
            ldsm_x4(kb + r * (2 * D) + ((ch ^ (r & 7)) << 4), a0, a1, a2, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma(k & 1 ? s2[n] : s[i][n], a0, a1, a2, a3, q[n][k][0], q[n][k][1], T());
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][n][j] = (s[i][n][j] + s2[n][j]) * p.scale_log2;
        }
        if (mask != (TS == 32 ? 0xffffffffu : (1u << (TS & 31)) - 1)) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (!((mask >> (i * 16 + quad + (j >> 1) * 8)) & 1)) s[i][n][j] = -INFINITY;
        }

        // running maximum, probabilities
        uint32_t pt[MT][NT][2], pr[MT][NT][2];   // leading bits, the rest
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float mx[2], al[2];
          bool up = false;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = fmaxf(s[0][n][j], s[0][n][j + 2]);
#pragma unroll
            for (int i = 1; i < MT; ++i) x = fmaxf(x, fmaxf(s[i][n][j], s[i][n][j + 2]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            mx[j] = fmaxf(m[n][j], x);
            up |= mx[j] > m[n][j];
          }
          if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              al[j] = m[n][j] == -INFINITY ? 0.f : exp2f(m[n][j] - mx[j]);
              m[n][j] = mx[j];
              l[n][j] *= al[j];
            }
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[n][k][j] *= al[j & 1];
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            float e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float ref = m[n][j & 1] == -INFINITY ? 0.f : m[n][j & 1] - kLift<T>;   // nothing seen yet: 2^-inf = 0
              e[j] = exp2f(s[i][n][j] - ref);
              l[n][j & 1] += e[j];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              split2(e[2 * j], e[2 * j + 1], pt[i][n][j], pr[i][n][j], T());
              pt[i][n][j] = transpose8x8(pt[i][n][j]);
              pr[i][n][j] = transpose8x8(pr[i][n][j]);
            }
          }
        }

        // O^T += V^T P^T, two channel steps at a time: the two products of one do not wait for each other
        const uint32_t vb = next_slot();
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            const int r = i * 16 + (lane & 7) + ((lane >> 4) << 3);
            uint32_t a[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int ch = 2 * (k + u) + ((lane >> 3) & 1);
              ldsm_x4_trans(vb + r * (2 * D) + ((ch ^ (r & 7)) << 4), a[u][0], a[u][1], a[u][2], a[u][3]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
              for (int u = 0; u < 2; ++u) mma(o[n][k + u], a[u][0], a[u][1], a[u][2], a[u][3], pt[i][n][0], pt[i][n][1], T());
#pragma unroll
              for (int u = 0; u < 2; ++u) mma(o[n][k + u], a[u][0], a[u][1], a[u][2], a[u][3], pr[i][n][0], pr[i][n][1], T());
            }
          }

        ++step;
      }
      rj -= (rd.t1 - rd.t0 + TS - 1) / TS;

      // the range's part of the row is done
      const bool head_in = rd.first >= u0, tail_in = rd.first + rd.units <= u1, whole = head_in && tail_in;
      const size_t row0 = (size_t)rd.b * p.Hq + (size_t)rd.h * p.g;
      const int slot = 2 * team + (head_in ? 1 : 0);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 4);
          l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 8);
          l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 16);
        }
      if (wide) {
        // The warps' parts: to the common maximum, then added up by all threads.  With two sets of maxima the next
        // row's may be written while these are read; with one, the warps wait for the readers.
        if (quad == 0)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            parts_ml[parity][warp][n * 8 + c2] = make_float2(m[n][0], l[n][0]);
            parts_ml[parity][warp][n * 8 + c2 + 1] = make_float2(m[n][1], l[n][1]);
          }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          __syncthreads();   // the maxima are there (n = 0); the tile before has been added up
          float f[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, parts_ml[parity][w][n * 8 + c2 + j].x);
            f[j] = m[n][j] == -INFINITY ? 0.f : exp2f(m[n][j] - top);
          }
#pragma unroll
          for (int k = 0; k < KS; ++k)
            parts_o[(warp * KS + k) * 32 + lane] =
                make_float4(o[n][k][0] * f[0], o[n][k][1] * f[1], o[n][k][2] * f[0], o[n][k][3] * f[1]);
          __syncthreads();
          if (threadIdx.x < KS * 32) {
            const int k = threadIdx.x >> 5;
            float4 x = parts_o[threadIdx.x];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
              const float4 y = parts_o[w * KS * 32 + threadIdx.x];
              x.x += y.x;
              x.y += y.y;
              x.z += y.z;
              x.w += y.w;
            }
            float mm[2], ll[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              mm[j] = -INFINITY;
              ll[j] = 0.f;
#pragma unroll
              for (int w = 0; w < kWarps; ++w) mm[j] = fmaxf(mm[j], parts_ml[parity][w][n * 8 + c2 + j].x);
#pragma unroll
              for (int w = 0; w < kWarps; ++w) {
                const float2 ml = parts_ml[parity][w][n * 8 + c2 + j];
                ll[j] += ml.x == -INFINITY ? ml.y : ml.y * exp2f(ml.x - mm[j]);   // 0, or NaN kept
              }
            }
            if (whole) {
              finish<T, D>(p, row0, n * 8 + c2, k, quad, make_float2(x.x, x.z), mm[0], ll[0]);
              finish<T, D>(p, row0, n * 8 + c2 + 1, k, quad, make_float2(x.y, x.w), mm[1], ll[1]);
            } else {
              p.o_part[((size_t)slot * NT * KS + n * KS + k) * 32 + lane] = x;
              if (k == 0 && quad == 0) p.ml_part[(size_t)slot * NT * 4 + n * 4 + lane] = make_float4(mm[0], ll[0], mm[1], ll[1]);
            }
          }
        }
        if (kSets == 2) parity ^= 1;
        else __syncthreads();
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            if (whole) {
              finish<T, D>(p, row0, n * 8 + c2, k, quad, make_float2(o[n][k][0], o[n][k][2]), m[n][0], l[n][0]);
              finish<T, D>(p, row0, n * 8 + c2 + 1, k, quad, make_float2(o[n][k][1], o[n][k][3]), m[n][1], l[n][1]);
            } else {
              p.o_part[((size_t)slot * NT * KS + n * KS + k) * 32 + lane] =
                  make_float4(o[n][k][0], o[n][k][1], o[n][k][2], o[n][k][3]);
            }
          }
          if (!whole && quad == 0)
            p.ml_part[(size_t)slot * NT * 4 + n * 4 + lane] = make_float4(m[n][0], l[n][0], m[n][1], l[n][1]);
        }
      }
      if (head_in && lane == 0 && (!wide || warp == 0)) {
        // last range of the row: the one that holds its last unit
        const int at = rd.first + rd.units - 1, big = extra * (base + 1);
        const int last = whole ? team : (at < big ? at / (base + 1) : extra + (at - big) / base);
        const int4 e = make_int4(rd.b * p.Hkv + rd.h, last - team + 1, team, 0);
        if (p.by_row) p.join[e.x] = e;
        else if (!whole) entry = e;
      }
    } while (next_part(p, pre, len, u0, u1, &rd));
    cp_wait<0>();
  }
  if (!p.by_row && lane == 0) p.join[gw] = entry;   // more rows than warps: teams are warps
}

// Joins the rows that lie in several ranges, 16 channels x 8 heads of one at a time.  WIDE (few rows, so many pieces): a CTA
// each, whose warps take the pieces in turn, before warp w merges what all warps' lanes w hold.  Else a warp each.
template <typename T, int D, int NT, bool WIDE>
__global__ void __launch_bounds__((WIDE ? kJoinWarps : kNarrowWarps) * 32)
    dense_join_kernel(const __grid_constant__ DenseParams p, int entries) {
  constexpr int KS = D / 16, kAhead = 5;   // pieces requested at once
  __shared__ float4 so[WIDE ? kJoinWarps : 1][33], sml[WIDE ? kJoinWarps : 1][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = WIDE ? blockIdx.x : blockIdx.x * kNarrowWarps + warp;
  const int at = item / (NT * KS), nk = item - at * (NT * KS);
  const int n = nk / KS, k = nk - n * KS;
  pdl_wait();
  pdl_trigger();
  if (at >= entries) return;
  const int4 e = p.join[at];
  if (e.y < 2) return;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  auto weight = [](float m, float top) { return m == -INFINITY ? 0.f : exp2f(m - top); };
  constexpr int kStep = WIDE ? kJoinWarps : 1;
  for (int i0 = WIDE ? warp : 0; i0 < e.y; i0 += kStep * kAhead) {
    float4 x[kAhead], ml[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * kStep;
      x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      ml[u] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
      if (i < e.y) {
        const size_t slot = 2 * (size_t)(e.z + i) + (i == 0 ? 1 : 0);
        x[u] = p.o_part[(slot * NT * KS + nk) * 32 + lane];
        ml[u] = p.ml_part[slot * NT * 4 + n * 4 + (lane & 3)];
      }
    }
    float t0 = m0, t1 = m1;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      t0 = fmaxf(t0, ml[u].x);
      t1 = fmaxf(t1, ml[u].z);
    }
    const float a0 = weight(m0, t0), a1 = weight(m1, t1);
    o = make_float4(o.x * a0, o.y * a1, o.z * a0, o.w * a1);
    l0 *= a0;
    l1 *= a1;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const float w0 = weight(ml[u].x, t0), w1 = weight(ml[u].z, t1);
      o.x += x[u].x * w0;
      o.y += x[u].y * w1;
      o.z += x[u].z * w0;
      o.w += x[u].w * w1;
      l0 += ml[u].y * (ml[u].x == -INFINITY ? 1.f : w0);   // without weight it is 0, or NaN that has to stay
      l1 += ml[u].w * (ml[u].z == -INFINITY ? 1.f : w1);
    }
    m0 = t0;
    m1 = t1;
  }
  const int b = e.x / p.Hkv, h = e.x - b * p.Hkv;
  const size_t row0 = (size_t)b * p.Hq + (size_t)h * p.g;
  if constexpr (WIDE) {
    so[warp][lane] = o;
    sml[warp][lane] = make_float4(m0, l0, m1, l1);
    __syncthreads();
#pragma unroll
    for (int col = warp; col < 32; col += kJoinWarps) {
      const bool there = lane < kJoinWarps;
      const float4 x = so[there ? lane : 0][col], ml = sml[there ? lane : 0][col];
      float top[2] = {ml.x, ml.z};
#pragma unroll
      for (int off = 16; off; off >>= 1) {
        top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], off));
        top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], off));
      }
      const float w0 = weight(ml.x, top[0]), w1 = weight(ml.z, top[1]);
      float v[6] = {x.x * w0, x.y * w1, x.z * w0, x.w * w1, ml.y * (ml.x == -INFINITY ? 1.f : w0),
                    ml.w * (ml.z == -INFINITY ? 1.f : w1)};
#pragma unroll
      for (int i = 0; i < 6; ++i) {
        if (!there) v[i] = 0.f;
#pragma unroll
        for (int off = kJoinWarps / 2; off; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
      }
      const int head = n * 8 + 2 * (col & 3);
      if (lane == 0) finish<T, D>(p, row0, head, k, col >> 2, make_float2(v[0], v[2]), top[0], v[4]);
      if (lane == 1) finish<T, D>(p, row0, head + 1, k, col >> 2, make_float2(v[1], v[3]), top[1], v[5]);
    }
  } else {
    const int quad = lane >> 2, head = n * 8 + 2 * (lane & 3);
    finish<T, D>(p, row0, head, k, quad, make_float2(o.x, o.z), m0, l0);
    finish<T, D>(p, row0, head + 1, k, quad, make_float2(o.y, o.w), m1, l1);
  }
}

std::atomic<uint64_t> g_limit[8];

template <typename T, int D, int NT>
cudaError_t run(DenseParams p, int ctas, cudaStream_t s) {
  constexpr int fixed = kWarps * (kSlots * kSlotBytes + (D / 16) * 512);
  constexpr int which = (std::is_same<T, __half>::value ? 4 : 0) + (D == 128 ? 2 : 0) + NT - 1;
  cudaError_t e = ensure_smem_limit(dense_decode_kernel<T, D, NT>, fixed + (2 * kMaxDecodeB + 1) * (int)sizeof(int),
                                    g_limit[which]);
  if (e != cudaSuccess) return e;
  const int rows = p.B * p.Hkv;
  p.by_row = rows <= dense_ranges(ctas);
  p.pad = rows < kTeamRows * ctas ? kPad : 0;
  const size_t smem = fixed + (2 * (size_t)p.B + 1) * sizeof(int);
  e = launch_pdl(dense_decode_kernel<T, D, NT>, dim3(ctas), dim3(kThreads), smem, s, p);
  if (e != cudaSuccess) return e;
  const int entries = p.by_row ? rows : dense_ranges(ctas), items = entries * NT * (D / 16);
  if (rows <= kWideRows)
    return launch_pdl(dense_join_kernel<T, D, NT, true>, dim3(items), dim3(kJoinWarps * 32), 0, s, p, entries);
  return launch_pdl(dense_join_kernel<T, D, NT, false>, dim3((items + kNarrowWarps - 1) / kNarrowWarps),
                    dim3(kNarrowWarps * 32), 0, s, p, entries);
}

template <typename T>
cudaError_t run_type(const DenseParams& p, int D, int ctas, cudaStream_t s) {
  if (D == 64) return p.g <= 8 ? run<T, 64, 1>(p, ctas, s) : run<T, 64, 2>(p, ctas, s);
  return p.g <= 8 ? run<T, 128, 1>(p, ctas, s) : run<T, 128, 2>(p, ctas, s);
}

}  // namespace

int dense_ranges(int ctas) { return ctas * kWarps; }

cudaError_t launch_dense_decode(const DenseParams& p, int D, int dtype, int ctas, cudaStream_t s) {
  return dtype == SEER_BF16 ? run_type<__nv_bfloat16>(p, D, ctas, s) : run_type<__half>(p, D, ctas, s);
}

}  // namespace seer
