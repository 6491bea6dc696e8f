// RMS norm of every query and key head, position rotation and cache write in
// one pass, and the backward pass.
//
// Forward, per row (token t, head h), fp32 throughout, one rounding per output:
//   y = x * w / sqrt(mean(x^2) + eps),   z = R(position) y
// with R rotating channel pairs (i, i + rope_dim / 2) by position * theta_i.
// y is what the gate and the compression cache read, z what the attention
// reads; keys go to their cache slot as z, values are copied beside them.
// Backward, with r = 1 / sqrt(mean(x^2) + eps):
//   dy = R^T dz + dy',   dx = r (w dy) - x r^3 mean(w dy x),   dw = sum dy x r
//
// Bound: HBM -- every input is read once and every output written once; the
// angles (fp64 products reduced modulo 2 pi, as in the gate) are computed once
// per token and CTA, not per head.
//
// Layout.  D / 16 lanes share a row, two 8-channel chunks (16 bytes in 16-bit types) each:
// lane l of a row takes chunks l and l + rope_dim / 16 while those are
// rotated, so both halves of its pairs are its own and the rotation needs no exchange; the
// rest of the lanes take the unrotated chunks two by two.  At full rotation a
// row's lanes then read 128 contiguous bytes per load.  Because a lane writes
// exactly the elements it has read, every output may be its input's rows.
//
// A CTA takes a tile of tokens of one kind (query, key or value heads): about
// rows_per_cta rows, so the three kinds' CTAs cost alike.
#include "seer_device.cuh"
#include "seer_internal.h"

#include <cuda_fp16.h>

#include <algorithm>

namespace seer {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Chunk {   // eight channels as stored
  uint4 v[sizeof(T) == 4 ? 2 : 1];
};

template <typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T* p) {
  Chunk<T> c;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(c.v) / 16); ++i) c.v[i] = reinterpret_cast<const uint4*>(p)[i];
  return c;
}

template <typename T>
__device__ __forceinline__ void store_chunk(T* p, const Chunk<T>& c) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(c.v) / 16); ++i) reinterpret_cast<uint4*>(p)[i] = c.v[i];
}

__device__ __forceinline__ void unpack(const Chunk<float>& c, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(c.v[i].x);
    f[4 * i + 1] = __uint_as_float(c.v[i].y);
    f[4 * i + 2] = __uint_as_float(c.v[i].z);
    f[4 * i + 3] = __uint_as_float(c.v[i].w);
  }
}
__device__ __forceinline__ void unpack(const Chunk<__nv_bfloat16>& c, float (&f)[8]) {
  const uint32_t w[4] = {c.v[0].x, c.v[0].y, c.v[0].z, c.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void unpack(const Chunk<__half>& c, float (&f)[8]) {
  const uint32_t w[4] = {c.v[0].x, c.v[0].y, c.v[0].z, c.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) { return pack_bf16(a, b); }
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ Chunk<T> pack(const float (&f)[8]) {
  Chunk<T> c;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      c.v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                          __float_as_uint(f[4 * i + 3]));
  } else {
    c.v[0] = make_uint4(pack2(f[0], f[1], T()), pack2(f[2], f[3], T()), pack2(f[4], f[5], T()),
                        pack2(f[6], f[7], T()));
  }
  return c;
}

// The two chunks of lane l (channel offsets) and whether they are a rotated pair.
template <int D>
__device__ __forceinline__ bool lane_chunks(int l, int rope_dim, int* c0, int* c1) {
  const int rh = rope_dim >> 4;   // chunks in half of the rotated channels
  const bool rot = l < rh;
  *c0 = 8 * (rot ? l : 2 * rh + 2 * (l - rh));
  *c1 = rot ? *c0 + 8 * rh : *c0 + 8;
  return rot;
}

template <typename T>
__device__ __forceinline__ T* row_at(const Rows& r, int t, int h) {
  return static_cast<T*>(r.data) + (int64_t)t * r.stride_t + (int64_t)h * r.stride_h;
}

// cos / sin of the tile's tokens and frequencies: cs[t][i], i < rope_dim / 2.
__device__ __forceinline__ void tile_angles(const NormParams& p, int t0, int nt, float2* cs) {
  const int half = p.rope_dim >> 1;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    float c, s;
    rope_cos_sin((double)p.positions[t0 + t] * p.theta[f], c, s);
    cs[t * kMaxHalfGate + f] = make_float2(c, s);
  }
}

// (a, b) -> (a c - b s, b c + a s), or with the opposite angle
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float2* cs, float sign) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float4 w = *reinterpret_cast<const float4*>(cs + i);   // cos, sin, cos, sin
    const float s0 = sign * w.y, s1 = sign * w.w;
    const float a0 = a[i], a1 = a[i + 1];
    a[i] = a0 * w.x - b[i] * s0;
    b[i] = b[i] * w.x + a0 * s0;
    a[i + 1] = a1 * w.z - b[i + 1] * s1;
    b[i + 1] = b[i + 1] * w.z + a1 * s1;
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = 1; off < LPR; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

__device__ __forceinline__ int kind_of(const NormParams& p, int cta) {
  int k = 0;
  while (k < 2 && cta >= p.kind[k].cta0 + p.kind[k].ctas) ++k;
  return k;
}

__device__ __forceinline__ int live_rows(const NormParams& p) {
  return p.live ? min(max(*p.live, 0), p.T) : p.T;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormParams p) {
  constexpr int LPR = D / 16, RPP = kThreads / LPR;   // lanes per row, rows per pass
  __shared__ __align__(16) float2 cs[kNormMaxTile * kMaxHalfGate];
  const int which = kind_of(p, blockIdx.x);
  const NormKind& kd = p.kind[which];
  const int t0 = (blockIdx.x - kd.cta0) * kd.tile;
  pdl_wait();
  pdl_trigger();
  const int nt = min(kd.tile, live_rows(p) - t0);
  if (nt <= 0) return;
  const int rows = nt * kd.heads;
  const int sub = threadIdx.x / LPR, l = threadIdx.x & (LPR - 1);
  int c0, c1;
  const bool rot = lane_chunks<D>(l, p.rope_dim, &c0, &c1) && which < 2;

  Chunk<T> n0 = {}, n1 = {};
  int nti = 0, nh = 0;
  auto fetch = [&](int r) {   // the row's chunks, requested one pass ahead
    if (r < rows) {
      nti = r / kd.heads;
      nh = r - nti * kd.heads;
      const T* x = row_at<T>(kd.x, t0 + nti, nh);
      n0 = load_chunk(x + c0);
      n1 = load_chunk(x + c1);
    }
  };
  fetch(sub);
  if (which < 2) tile_angles(p, t0, nt, cs);
  __syncthreads();

  for (int r0 = 0; r0 < rows; r0 += RPP) {   // uniform over the CTA: the row sums are warp-wide
    const bool mine = r0 + sub < rows;
    const Chunk<T> x0 = n0, x1 = n1;
    const int ti = nti, h = nh;
    fetch(r0 + RPP + sub);
    T* dst = nullptr;   // this row's place in the cache
    if (kd.cache.data != nullptr && mine) {
      const int slot = p.slot_map[t0 + ti];
      if (slot >= 0 && slot < p.slots) {
        const int page = slot / p.page_size;
        dst = static_cast<T*>(kd.cache.data) + page * kd.cache.stride_page + h * kd.cache.stride_h +
              (int64_t)(slot - page * p.page_size) * kd.cache.stride_t;
      } else if (slot != -1 && l == 0) {
        report(p.err, SEER_DEVERR_PAGE_INDEX);
      }
    }
    if (which == 2) {   // values: the cache copy only
      if (dst) {
        store_chunk(dst + c0, x0);
        store_chunk(dst + c1, x1);
      }
      continue;
    }
    float a[8], b[8];
    unpack(x0, a);
    unpack(x1, b);
    if (kd.weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += a[i] * a[i] + b[i] * b[i];
      const float rs = rsqrtf(row_sum<LPR>(ss) * (1.0f / D) + p.eps);
      float wa[8], wb[8];
      unpack(load_chunk(static_cast<const T*>(kd.weight) + c0), wa);
      unpack(load_chunk(static_cast<const T*>(kd.weight) + c1), wb);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= rs * wa[i];
        b[i] *= rs * wb[i];
      }
    }
    if (!mine) continue;
    if (kd.nope.data) {
      T* y = row_at<T>(kd.nope, t0 + ti, h);
      store_chunk(y + c0, pack<T>(a));
      store_chunk(y + c1, pack<T>(b));
    }
    if (rot) rotate(a, b, cs + ti * kMaxHalfGate + c0, 1.f);
    const Chunk<T> z0 = pack<T>(a), z1 = pack<T>(b);
    if (kd.out.data) {
      T* z = row_at<T>(kd.out, t0 + ti, h);
      store_chunk(z + c0, z0);
      store_chunk(z + c1, z1);
    }
    if (dst) {
      store_chunk(dst + c0, z0);
      store_chunk(dst + c1, z1);
    }
  }
}

// Backward: each CTA walks its kind's tiles with a stride, holding the weight gradient of its
// 16 channels per lane in registers; at the end the CTA's sum goes to its row of the workspace.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_backward_kernel(const __grid_constant__ NormParams p) {
  constexpr int LPR = D / 16, RPP = kThreads / LPR;
  __shared__ __align__(16) float2 cs[kNormMaxTile * kMaxHalfGate];
  __shared__ float red[kThreads / 32][D];
  const int which = kind_of(p, blockIdx.x);
  const NormKind& kd = p.kind[which];
  const int sub = threadIdx.x / LPR, l = threadIdx.x & (LPR - 1);
  int c0, c1;
  const bool rot = lane_chunks<D>(l, p.rope_dim, &c0, &c1);
  float dw0[8] = {}, dw1[8] = {};
  pdl_wait();
  pdl_trigger();
  const int live = live_rows(p);
  for (int tile = blockIdx.x - kd.cta0; tile < kd.tiles; tile += kd.ctas) {
    const int t0 = tile * kd.tile, nt = min(kd.tile, live - t0);
    if (nt <= 0) break;
    const int rows = nt * kd.heads;
    __syncthreads();   // the previous tile's angles have been used
    tile_angles(p, t0, nt, cs);
    __syncthreads();
    for (int r0 = 0; r0 < rows; r0 += RPP) {
      const int r = r0 + sub;
      const bool mine = r < rows;
      const int ti = mine ? r / kd.heads : 0, h = mine ? r - ti * kd.heads : 0;
      float a[8] = {}, b[8] = {}, xa[8] = {}, xb[8] = {};
      if (mine) {
        Chunk<T> g0 = {}, g1 = {}, y0 = {}, y1 = {}, x0 = {}, x1 = {};
        if (kd.weight) {
          const T* x = row_at<T>(kd.x, t0 + ti, h);
          x0 = load_chunk(x + c0);
          x1 = load_chunk(x + c1);
        }
        if (kd.out.data) {
          const T* g = row_at<T>(kd.out, t0 + ti, h);
          g0 = load_chunk(g + c0);
          g1 = load_chunk(g + c1);
        }
        if (kd.nope.data) {
          const T* g = row_at<T>(kd.nope, t0 + ti, h);
          y0 = load_chunk(g + c0);
          y1 = load_chunk(g + c1);
        }
        unpack(g0, a);
        unpack(g1, b);
        if (rot) rotate(a, b, cs + ti * kMaxHalfGate + c0, -1.f);
        if (kd.nope.data) {
          float ya[8], yb[8];
          unpack(y0, ya);
          unpack(y1, yb);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            a[i] += ya[i];
            b[i] += yb[i];
          }
        }
        unpack(x0, xa);
        unpack(x1, xb);
      }
      if (kd.weight) {
        float wa[8], wb[8];
        unpack(load_chunk(static_cast<const T*>(kd.weight) + c0), wa);
        unpack(load_chunk(static_cast<const T*>(kd.weight) + c1), wb);
        float ss = 0.f, sd = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss += xa[i] * xa[i] + xb[i] * xb[i];
          sd += xa[i] * (a[i] * wa[i]) + xb[i] * (b[i] * wb[i]);
        }
        const float rs = rsqrtf(row_sum<LPR>(ss) * (1.0f / D) + p.eps);
        const float k = row_sum<LPR>(sd) * (1.0f / D) * rs * rs;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw0[i] += a[i] * (xa[i] * rs);
          dw1[i] += b[i] * (xb[i] * rs);
          a[i] = rs * (a[i] * wa[i] - xa[i] * k);
          b[i] = rs * (b[i] * wb[i] - xb[i] * k);
        }
      }
      if (mine) {
        T* dx = row_at<T>(kd.dx, t0 + ti, h);
        store_chunk(dx + c0, pack<T>(a));
        store_chunk(dx + c1, pack<T>(b));
      }
    }
  }
  if (!kd.weight) return;
  // lanes with the same channels, then the CTA's warps, in a fixed order
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) {
      dw0[i] += __shfl_xor_sync(0xffffffffu, dw0[i], off);
      dw1[i] += __shfl_xor_sync(0xffffffffu, dw1[i], off);
    }
  }
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) < LPR) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      red[warp][c0 + i] = dw0[i];
      red[warp][c1 + i] = dw1[i];
    }
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += red[w][threadIdx.x];
    p.partial[(size_t)blockIdx.x * D + threadIdx.x] = s;
  }
}

// Sum of a kind's partial weight gradients, in a fixed order: CTA 0 the query's, CTA 1 the key's.
constexpr int kReduceThreads = 1024;
template <int D>
__global__ void __launch_bounds__(kReduceThreads) norm_weight_kernel(const __grid_constant__ NormParams p) {
  constexpr int NG = kReduceThreads / D;
  __shared__ float red[NG][D];
  const NormKind& kd = p.kind[blockIdx.x];
  const int c = threadIdx.x & (D - 1), g = threadIdx.x / D;
  pdl_wait();
  pdl_trigger();
  if (!kd.dw) return;
  float s = 0.f;
#pragma unroll 8
  for (int i = g; i < kd.ctas; i += NG) s += p.partial[(size_t)(kd.cta0 + i) * D + c];
  red[g][c] = s;
  __syncthreads();
  if (g == 0) {
#pragma unroll
    for (int i = 1; i < NG; ++i) s += red[i][c];
    kd.dw[c] = s;
  }
}

// Tokens per CTA and CTAs of each kind: about `target` rows a CTA; `most` > 0 bounds the CTAs
// (persistent form), shared out by rows.
int plan_kinds(NormParams& p, int target, int most) {
  int64_t all = 0;
  int grid = 0;
  for (NormKind& k : p.kind)
    if (k.ctas) all += k.heads;
  for (NormKind& k : p.kind) {
    k.cta0 = grid;
    if (!k.ctas) continue;
    k.tile = std::min(std::max(target / k.heads, 1), kNormMaxTile);
    k.tiles = (p.T + k.tile - 1) / k.tile;
    k.ctas = k.tiles;
    if (most > 0) k.ctas = (int)std::max<int64_t>(1, std::min<int64_t>(k.tiles, (int64_t)most * k.heads / all));
    grid += k.ctas;
  }
  return grid;
}

// Rows per pass of one CTA, and passes per CTA: one while that leaves SMs idle, four (so that the
// angles and the launch are shared by more rows) once there are enough rows.
int target_rows(const NormParams& p, int D, int sms) {
  int64_t heads = 0;
  for (const NormKind& k : p.kind)
    if (k.ctas) heads += k.heads;
  const int pass = kThreads / (D / 16);
  return heads * p.T > (int64_t)16 * sms * pass ? 4 * pass : pass;
}

template <typename T, int D>
cudaError_t forward(NormParams p, int sms, cudaStream_t s) {
  const int grid = plan_kinds(p, target_rows(p, D, sms), 0);
  return launch_pdl(norm_rope_kernel<T, D>, dim3(grid), dim3(kThreads), 0, s, p);
}

template <typename T, int D>
cudaError_t backward(NormParams p, int sms, cudaStream_t s) {
  const int grid = plan_kinds(p, target_rows(p, D, sms), std::min(3 * sms, kNormPartials - 2));
  cudaError_t e = launch_pdl(norm_rope_backward_kernel<T, D>, dim3(grid), dim3(kThreads), 0, s, p);
  if (e != cudaSuccess || !(p.kind[0].dw || p.kind[1].dw)) return e;
  return launch_pdl(norm_weight_kernel<D>, dim3(2), dim3(kReduceThreads), 0, s, p);
}

}  // namespace

#define SEER_NORM_DISPATCH(fn)                                               \
  if (D == 64) {                                                             \
    if (dtype == SEER_BF16) return fn<__nv_bfloat16, 64>(p, sms, s);         \
    if (dtype == SEER_FP16) return fn<__half, 64>(p, sms, s);                \
    return fn<float, 64>(p, sms, s);                                         \
  }                                                                          \
  if (dtype == SEER_BF16) return fn<__nv_bfloat16, 128>(p, sms, s);          \
  if (dtype == SEER_FP16) return fn<__half, 128>(p, sms, s);                 \
  return fn<float, 128>(p, sms, s);

cudaError_t launch_norm_rope(const NormParams& p, int D, int dtype, int sms, cudaStream_t s) {
  SEER_NORM_DISPATCH(forward)
}
cudaError_t launch_norm_rope_backward(const NormParams& p, int D, int dtype, int sms, cudaStream_t s) {
  SEER_NORM_DISPATCH(backward)
}

}  // namespace seer
