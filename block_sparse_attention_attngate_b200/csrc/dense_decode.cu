// Attention of one new token per sequence over its whole cache, split over the
// cache's length and joined.
//
// For query head i of KV head h and tokens t in [lo_b, hi_b):
//   s_t = scale q_i . K_t,   out = sum_t exp(s_t) V_t / sum_t exp(s_t)
// by the running maximum m, sum l and output o (log2 domain, fp32):
//   m' = max(m, max s),  o' = o 2^(m - m') + sum 2^(s - m') V,  l' likewise,
// and pieces (m_i, l_i, o_i) of one row join by the same rule.
//
// Bound: HBM -- every key and value is read once; 4 g flops a byte pair at most, a
// tenth of what the warp-level tensor instructions sustain.
//
// Split.  The sequences' tokens in steps of kDenseUnit are one long axis; G
// ranges of it, times the KV heads, are the work of as many independent warps
// (one wave, eight to an SM).  A warp walks its range through a ring of
// shared-memory stages that it fills itself (cp.async, kStages - 1 stages
// ahead), so the loads never stop at the end of a sequence and no warp waits for
// another: there is no barrier past the prologue.  The KV heads of a range run
// at the same time on neighbouring SMs, so a token-major cache's rows are read
// whole within a short time.  cp.async of 16-byte chunks takes any page size
// and stride: tokens that are out of range or on a bad page are filled
// with zeros and masked, whatever lies there.
//
// Products.  Both are taken transposed so that 16 tokens (or 16 channels) fill the
// long side of the 16x8x16 instruction and the group's heads the short one (eight a
// tile; two tiles above eight): S^T = K Q^T with K as it lies, then O^T = V^T P^T,
// with V^T from transposing loads and P^T from the scores' registers by one
// 8x8 register transpose each.  A lane then holds the same two heads' columns in S, m, l and O.
//
// A row that lies in one range is finished there; the pieces of the others go to
// the workspace in register order, and the join kernel (one warp per eight or
// fewer pieces, sixteen warps a CTA) merges them.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "seer_device.cuh"
#include "seer_internal.h"

namespace seer {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kStageBytes = 4096;          // K (or V) of one stage
constexpr int kJoinWarps = 16;

template <int D>
constexpr int stage_tokens() { return kStageBytes / (2 * D); }   // 16 (d = 128) or 32 (d = 64)

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
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
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) { return pack_bf16(a, b); }
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
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

// Position of a warp in its range: the stage of sequence b that starts at token t.
struct Cursor {
  int b, t, end;   // end: first token of the sequence that is not this range's
  int lo;          // first token of the sequence that is seen
};

// Move to the first token of unit u (u < total) of a range that ends at unit u1.
__device__ __forceinline__ void seek(const DenseParams& p, const int* pre, const int* len, int b, int u, int u1,
                                     Cursor* c) {
  int lo, hi;
  token_range(p, len[b], &lo, &hi);
  c->b = b;
  c->lo = lo;
  c->t = lo + (u - pre[b]) * kDenseUnit;
  const int last = u1 - pre[b];   // units of this sequence up to the range's end
  c->end = pre[b + 1] <= u1 ? hi : lo + last * kDenseUnit;
}

// Next stage of TS tokens; at a sequence's end the next one that is not empty.  False at the range's end.
template <int TS>
__device__ __forceinline__ bool advance(const DenseParams& p, const int* pre, const int* len, int u1, Cursor* c) {
  c->t += TS;
  if (c->t < c->end) return true;
  int b = c->b + 1;
  if (pre[b] >= u1) return false;
  while (pre[b + 1] == pre[b]) ++b;   // ends: pre[b] < u1 <= total
  seek(p, pre, len, b, pre[b], u1, c);
  return true;
}

// Element offset of token t of sequence b and whether it is readable (t inside the cache).
__device__ __forceinline__ bool locate(const DenseParams& p, const KvPlain& kv, int page_id, int b, int t, int h,
                                       int64_t* off) {
  if (kv.paged) {
    const bool ok = page_id >= 0 && page_id < kv.num_pages;
    *off = ok ? page_id * kv.stride_b + h * kv.stride_h + (int64_t)(t % p.page) * kv.stride_t : 0;
    return ok;
  }
  *off = b * kv.stride_b + h * kv.stride_h + t * kv.stride_t;
  return true;
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) dense_decode_kernel(const __grid_constant__ DenseParams p) {
  constexpr int TS = stage_tokens<D>();
  constexpr int MT = TS / 16;        // token tiles a stage
  constexpr int KS = D / 16;         // channel steps
  constexpr int CPR = D / 8;         // 16-byte chunks a row
  constexpr int RPI = 32 / CPR;      // rows a warp-wide copy covers
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t masks[kWarps][kStages];
  __shared__ int scan_ws[kWarps];
  int* pre = reinterpret_cast<int*>(smem + (size_t)kWarps * kStages * 2 * kStageBytes);   // [B + 1]
  int* len = pre + p.B + 1;                                                              // [B]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane >> 2, c2 = 2 * (lane & 3);   // row of a tile, first of the lane's two columns

  pdl_wait();
  pdl_trigger();

  // exclusive scan of the sequences' units
  int total = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const int L = b < p.B ? p.seqlens[b] : 0;
    const int n = b < p.B ? units_of(p, L) : 0;
    if (L > p.cap && blockIdx.x == 0) report(p.err, SEER_DEVERR_COUNT);
    int inc = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += x;
    }
    if (lane == 31) scan_ws[warp] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      before += w < warp ? scan_ws[w] : 0;
      all += scan_ws[w];
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

  const int W = gridDim.x * kWarps;
  const int gw = warp * gridDim.x + blockIdx.x;     // neighbouring work on neighbouring SMs
  const int slots = max(W, p.Hkv);
  const int G = min(max(W / p.Hkv, 1), total);
  // rows without a token
  for (int r = gw; r < p.B * p.Hkv; r += W) {
    const int b = r / p.Hkv, h = r - b * p.Hkv;
    if (pre[b + 1] != pre[b]) continue;
    uint16_t* o = p.out + ((size_t)b * p.Hq + (size_t)h * p.g) * D;
    for (int i = lane; i < p.g * D; i += 32) o[i] = 0;
    if (p.lse)
      for (int i = lane; i < p.g; i += 32) p.lse[(size_t)b * p.Hq + h * p.g + i] = __int_as_float(0xff800000);
    if (p.by_row && lane == 0) p.join[r] = make_int4(0, 0, 0, 0);
  }

  const uint32_t ring = smem_u32(smem) + warp * kStages * 2 * kStageBytes;
  for (int v = gw; v < slots; v += W) {
    int4 entry = make_int4(0, 0, 0, 0);
    if (v < G * p.Hkv) {
      const int grp = v / p.Hkv, h = v - grp * p.Hkv;
      const int u0 = (int)((int64_t)grp * total / G), u1 = (int)((int64_t)(grp + 1) * total / G);
      // first sequence: the last one with pre[b] <= u0 (a sequence without units shares its successor's value)
      int b0 = 0;
      for (int hi = p.B; hi - b0 > 1;) {
        const int mid = (b0 + hi) >> 1;
        if (pre[mid] <= u0) b0 = mid;
        else hi = mid;
      }
      Cursor rd, ld, nx;   // being computed; being requested; whose page ids are on their way
      seek(p, pre, len, b0, u0, u1, &rd);
      nx = rd;
      bool nx_ok = true;
      int id_k = 0, id_v = 0;
      auto fetch_ids = [&]() {   // page ids of nx's tokens, one token a lane
        const int t = nx.t + lane;
        if (lane < TS && t < nx.end) {
          if (p.k.paged) id_k = p.k.block_table[(int64_t)nx.b * p.k.max_pages + t / p.page];
          if (p.v.paged) id_v = p.v.block_table[(int64_t)nx.b * p.v.max_pages + t / p.page];
        }
      };
      auto request = [&](int stage) {   // fill a stage with nx's tokens and move nx on
        if (nx_ok) {
          ld = nx;
          const int t = ld.t + lane;
          int64_t ok_ = 0, ov_ = 0;
          bool good = lane < TS && t < ld.end;
          if (good) {
            const bool gk = locate(p, p.k, id_k, ld.b, t, h, &ok_);
            const bool gv = locate(p, p.v, id_v, ld.b, t, h, &ov_);
            good = gk && gv;
            if (!good) report(p.err, SEER_DEVERR_PAGE_INDEX);
          }
          const uint32_t m = __ballot_sync(0xffffffffu, good);
          if (lane == 0) masks[warp][stage] = m;
          nx_ok = advance<TS>(p, pre, len, u1, &nx);
          if (nx_ok) fetch_ids();
          const uint32_t base = ring + stage * 2 * kStageBytes;
          const int ch = lane % CPR;
#pragma unroll
          for (int i = 0; i < TS / RPI; ++i) {
            const int r = i * RPI + lane / CPR;
            const int64_t a = __shfl_sync(0xffffffffu, ok_, r);
            cp_async16(base + r * (2 * D) + ((ch ^ (r & 7)) << 4), p.k.data + a + ch * 8, (m >> r) & 1);
          }
#pragma unroll
          for (int i = 0; i < TS / RPI; ++i) {
            const int r = i * RPI + lane / CPR;
            const int64_t a = __shfl_sync(0xffffffffu, ov_, r);
            cp_async16(base + kStageBytes + r * (2 * D) + ((ch ^ (r & 7)) << 4), p.v.data + a + ch * 8, (m >> r) & 1);
          }
        }
        cp_commit();   // one group a stage, empty behind the range's end
      };
      fetch_ids();
#pragma unroll
      for (int s = 0; s < kStages - 1; ++s) request(s);

      uint32_t q[NT][KS][2];
      float o[NT][KS][4], m[NT][2], l[NT][2];
      int stage = 0;
      bool fresh = true;   // rd stands at the first stage of a sequence's part
      bool more = true;
      while (more) {
        if (fresh) {
          fresh = false;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int head = n * 8 + quad;
            const uint16_t* src = p.q + ((size_t)rd.b * p.Hq + (size_t)h * p.g + head) * D + c2;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              q[n][k][0] = head < p.g ? *reinterpret_cast<const uint32_t*>(src + k * 16) : 0u;
              q[n][k][1] = head < p.g ? *reinterpret_cast<const uint32_t*>(src + k * 16 + 8) : 0u;
              o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
            }
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
          }
        }
        cp_wait<kStages - 2>();
        __syncwarp();   // the stage is there for every lane, and every lane is done with the one before
        request(stage == 0 ? kStages - 1 : stage - 1);
        const uint32_t kb = ring + stage * 2 * kStageBytes, vb = kb + kStageBytes;
        const uint32_t mask = masks[warp][stage];

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
        uint32_t pt[MT][NT][2];
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
              const float ref = m[n][j & 1] == -INFINITY ? 0.f : m[n][j & 1];   // nothing seen yet: 2^-inf = 0
              e[j] = exp2f(s[i][n][j] - ref);
              l[n][j & 1] += e[j];
            }
            pt[i][n][0] = transpose8x8(pack2(e[0], e[1], T()));
            pt[i][n][1] = transpose8x8(pack2(e[2], e[3], T()));
          }
        }

        // O^T += V^T P^T
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const int r = i * 16 + (lane & 7) + ((lane >> 4) << 3), ch = 2 * k + ((lane >> 3) & 1);
            uint32_t a0, a1, a2, a3;
            ldsm_x4_trans(vb + r * (2 * D) + ((ch ^ (r & 7)) << 4), a0, a1, a2, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma(o[n][k], a0, a1, a2, a3, pt[i][n][0], pt[i][n][1], T());
          }

        stage = stage + 1 == kStages ? 0 : stage + 1;
        const Cursor was = rd;
        more = advance<TS>(p, pre, len, u1, &rd);
        if (more && rd.b == was.b) continue;
        fresh = true;

        // the range's part of sequence was.b is done
        const bool head_in = pre[was.b] >= u0, tail_in = pre[was.b + 1] <= u1;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 4);
            l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 8);
            l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 16);
          }
        if (head_in && tail_in) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int head = n * 8 + c2 + j;
              if (head >= p.g) continue;
              const size_t row = (size_t)was.b * p.Hq + (size_t)h * p.g + head;
              const float inv = l[n][j] == 0.f ? 0.f : 1.0f / l[n][j];
#pragma unroll
              for (int k = 0; k < KS; ++k) {
                p.out[row * D + k * 16 + quad] = round1(o[n][k][j] * inv, T());
                p.out[row * D + k * 16 + quad + 8] = round1(o[n][k][j + 2] * inv, T());
              }
              if (p.lse && quad == 0) p.lse[row] = l[n][j] == 0.f ? -INFINITY : (m[n][j] + log2f(l[n][j])) * 0.6931471805599453f;
            }
          if (p.by_row && lane == 0) p.join[was.b * p.Hkv + h] = make_int4(0, 1, 0, 0);
        } else {
          const int slot = 2 * v + (head_in ? 1 : 0);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < KS; ++k)
              p.o_part[((size_t)slot * NT * KS + n * KS + k) * 32 + lane] =
                  make_float4(o[n][k][0], o[n][k][1], o[n][k][2], o[n][k][3]);
            if (quad == 0)
              p.ml_part[(size_t)slot * NT * 4 + n * 4 + lane] = make_float4(m[n][0], l[n][0], m[n][1], l[n][1]);
          }
          if (head_in) {
            // last range of the sequence: the one that holds its last unit
            const int last = (int)((((int64_t)pre[was.b + 1]) * G - 1) / total);
            entry = make_int4(was.b * p.Hkv + h, last - grp + 1, grp, 0);
            if (p.by_row && lane == 0) p.join[was.b * p.Hkv + h] = entry;
          }
        }
      }
      cp_wait<0>();
      __syncwarp();   // the ring is free for the next range
    }
    if (!p.by_row && lane == 0) p.join[v] = entry;
  }
}

// One CTA per row that lies in several ranges (x) and 16 channels x 8 heads of it (y): its warps take the
// pieces in turn, then warp 0 merges the warps.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kJoinWarps * 32) dense_join_kernel(const __grid_constant__ DenseParams p) {
  constexpr int KS = D / 16;
  __shared__ float4 so[kJoinWarps][32], sml[kJoinWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = blockIdx.y / KS, k = blockIdx.y - n * KS;
  pdl_wait();
  pdl_trigger();
  const int4 e = p.join[blockIdx.x];
  if (e.y < 2) return;
  const int b = e.x / p.Hkv, h = e.x - b * p.Hkv;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  auto merge = [&](const float4& x, const float4& ml) {
    const float n0 = fmaxf(m0, ml.x), n1 = fmaxf(m1, ml.z);
    const float a0 = m0 == -INFINITY ? 0.f : exp2f(m0 - n0), a1 = m1 == -INFINITY ? 0.f : exp2f(m1 - n1);
    const float w0 = ml.x == -INFINITY ? 0.f : exp2f(ml.x - n0), w1 = ml.z == -INFINITY ? 0.f : exp2f(ml.z - n1);
    o.x = o.x * a0 + x.x * w0;
    o.y = o.y * a1 + x.y * w1;
    o.z = o.z * a0 + x.z * w0;
    o.w = o.w * a1 + x.w * w1;
    l0 = l0 * a0 + ml.y * w0;
    l1 = l1 * a1 + ml.w * w1;
    m0 = n0;
    m1 = n1;
  };
#pragma unroll 4
  for (int i = warp; i < e.y; i += kJoinWarps) {
    const size_t slot = 2 * ((size_t)(e.z + i) * p.Hkv + h) + (i == 0 ? 1 : 0);
    merge(p.o_part[(slot * NT * KS + n * KS + k) * 32 + lane], p.ml_part[slot * NT * 4 + n * 4 + (lane & 3)]);
  }
  so[warp][lane] = o;
  sml[warp][lane] = make_float4(m0, l0, m1, l1);
  __syncthreads();
  if (warp != 0) return;
  const int used = min(kJoinWarps, e.y);
  for (int w = 1; w < used; ++w) merge(so[w][lane], sml[w][lane]);
  const int quad = lane >> 2, head = n * 8 + 2 * (lane & 3);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (head + j >= p.g) continue;
    const size_t row = (size_t)b * p.Hq + (size_t)h * p.g + head + j;
    const float l = j ? l1 : l0, mm = j ? m1 : m0, inv = l == 0.f ? 0.f : 1.0f / l;
    p.out[row * D + k * 16 + quad] = round1((j ? o.y : o.x) * inv, T());
    p.out[row * D + k * 16 + quad + 8] = round1((j ? o.w : o.z) * inv, T());
    if (p.lse && k == 0 && quad == 0) p.lse[row] = l == 0.f ? -INFINITY : (mm + log2f(l)) * 0.6931471805599453f;
  }
}

std::atomic<uint64_t> g_limit[8];

template <typename T, int D, int NT>
cudaError_t run(const DenseParams& p, int ctas, cudaStream_t s) {
  constexpr int ring = kWarps * kStages * 2 * kStageBytes;
  constexpr int which = (std::is_same<T, __half>::value ? 4 : 0) + (D == 128 ? 2 : 0) + NT - 1;
  cudaError_t e = ensure_smem_limit(dense_decode_kernel<T, D, NT>, ring + (2 * kMaxDecodeB + 1) * (int)sizeof(int),
                                    g_limit[which]);
  if (e != cudaSuccess) return e;
  const size_t smem = ring + (2 * (size_t)p.B + 1) * sizeof(int);
  if ((e = launch_pdl(dense_decode_kernel<T, D, NT>, dim3(ctas), dim3(kThreads), smem, s, p)) != cudaSuccess) return e;
  const int rows = p.by_row ? p.B * p.Hkv : dense_ranges(ctas, p.Hkv);
  return launch_pdl(dense_join_kernel<T, D, NT>, dim3(rows, NT * (D / 16)), dim3(kJoinWarps * 32), 0, s, p);
}

template <typename T>
cudaError_t run_type(const DenseParams& p, int D, int ctas, cudaStream_t s) {
  if (D == 64) return p.g <= 8 ? run<T, 64, 1>(p, ctas, s) : run<T, 64, 2>(p, ctas, s);
  return p.g <= 8 ? run<T, 128, 1>(p, ctas, s) : run<T, 128, 2>(p, ctas, s);
}

}  // namespace

int dense_ranges(int ctas, int Hkv) { return std::max(ctas * kWarps, Hkv); }

cudaError_t launch_dense_decode(const DenseParams& p, int D, int dtype, int ctas, cudaStream_t s) {
  return dtype == SEER_BF16 ? run_type<__nv_bfloat16>(p, D, ctas, s) : run_type<__half>(p, D, ctas, s);
}

}  // namespace seer
