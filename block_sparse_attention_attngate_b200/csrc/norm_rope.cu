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
// Bound: HBM -- every input is read once and every output written once.  Measured (inputs that change from call to call,
// against the copy bandwidth): 8192 tokens of 32 + 8 heads of 128, rotated and plain outputs and both caches in bf16, 49 to
// 50 us, 87 to 89 %; the gradients of the same rows 49 to 51 us, 75 to 79 %, with those of the un-rotated rows 77 us, 67 %; 4096
// tokens in fp32 33 us, 78 %, their gradients 75 us, 51 % (two stages in the ring: a pass waits for the newest request); 2049
// tokens of 40 + 8 heads in fp16, half rotated, 13.1 us, 59 % (9.9 us where the inputs lie in L2).  The arithmetic is close
// behind the memory in the gradients, so it is done two channels at a time (f32x2 instructions: 50 us, 53 without) and addresses
// are stepped.
//
// Layout.  D / 16 lanes share a row, two 8-channel chunks (16 bytes in 16-bit types) each:
// lane l of a row takes chunks l and l + rope_dim / 16 while those are
// rotated, so both halves of its pairs are its own and the rotation needs no exchange; the
// rest of the lanes take the unrotated chunks two by two.  At full rotation a
// row's lanes then read 128 contiguous bytes per load.  Because a lane writes
// exactly the elements it has read, every output may be its input's rows.
//
// Work.  A CTA works on one kind of row (query, key, value), so that all it needs to know of the kind is uniform.
// A pass is 32 / (D / 16) heads of one token.  Warps are independent.  A token's angles (fp64 products, whole
// turns taken off) are computed by the warp's lanes while the token's first rows are on their way, exchanged
// through the warp's own shared memory and kept in registers for all its heads.
// Forward, a warp takes up to kUnitPasses passes of one token and ends; its first rows, position, slot and the live count are
// all requested at once.  Backward, it takes kRunPasses passes of the list of all tokens' passes, and keeps
// some in flight through a ring in shared memory (cp.async; every lane reads back what it has requested itself, so no
// lane waits for another).  (Staying CTAs with equal shares measured 10-20 % slower in both directions: some SMs get less
// of the memory's bandwidth than others, and the rest wait for them at the end.)
#include "seer_device.cuh"
#include "seer_internal.h"

#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

namespace seer {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kForwardCtas = 5, kBackwardCtas = 4;   // per SM, at least
constexpr int kUnitPasses = 8, kRunPasses = 8;       // of a warp, forward and backward

// ---------------------------------------------------------------- two channels at a time
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 sub2(F2 a, F2 b) {
  F2 r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// ---------------------------------------------------------------- chunks of eight channels
template <typename T>
struct Chunk {   // as stored
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

__device__ __forceinline__ F2 unpack2(uint32_t w, __nv_bfloat16) { return f2(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ F2 unpack2(uint32_t w, __half) {
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return f2(x.x, x.y);
}
template <typename T>
__device__ __forceinline__ void unpack(const Chunk<T>& c, F2 (&f)[4]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[2 * i] = f2(__uint_as_float(c.v[i].x), __uint_as_float(c.v[i].y));
      f[2 * i + 1] = f2(__uint_as_float(c.v[i].z), __uint_as_float(c.v[i].w));
    }
  } else {
    f[0] = unpack2(c.v[0].x, T());
    f[1] = unpack2(c.v[0].y, T());
    f[2] = unpack2(c.v[0].z, T());
    f[3] = unpack2(c.v[0].w, T());
  }
}

__device__ __forceinline__ uint32_t pack2(float2 a, __nv_bfloat16) { return pack_bf16(a.x, a.y); }
__device__ __forceinline__ uint32_t pack2(float2 a, __half) {
  const __half2 h = __floats2half2_rn(a.x, a.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ Chunk<T> pack(const F2 (&f)[4]) {
  Chunk<T> c;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 x = split(f[2 * i]), y = split(f[2 * i + 1]);
      c.v[i] = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y));
    }
  } else {
    c.v[0] = make_uint4(pack2(split(f[0]), T()), pack2(split(f[1]), T()), pack2(split(f[2]), T()),
                        pack2(split(f[3]), T()));
  }
  return c;
}

// The two chunks of lane l (channel offsets) and whether they are a rotated pair.
__device__ __forceinline__ bool lane_chunks(int l, int rope_dim, int* c0, int* c1) {
  const int rh = rope_dim >> 4;   // chunks in half of the rotated channels
  const bool rot = l < rh;
  *c0 = 8 * (rot ? l : 2 * rh + 2 * (l - rh));
  *c1 = rot ? *c0 + 8 * rh : *c0 + 8;
  return rot;
}

// (a, b) -> (a c - b s, b c + a s), or by the opposite angle
template <bool BACK>
__device__ __forceinline__ void rotate(F2 (&a)[4], F2 (&b)[4], const F2 (&c)[4], const F2 (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const F2 x = a[i], y = b[i];
    a[i] = BACK ? fma2(x, c[i], mul2(y, s[i])) : sub2(mul2(x, c[i]), mul2(y, s[i]));
    b[i] = BACK ? sub2(mul2(y, c[i]), mul2(x, s[i])) : fma2(y, c[i], mul2(x, s[i]));
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = 1; off < LPR; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

__device__ __forceinline__ int live_rows(const NormParams& p) {
  return p.live ? min(max(*p.live, 0), p.T) : p.T;
}

// Angles of a token, given to each rotated lane as its eight frequencies' cos and sin.
__device__ __forceinline__ void token_angles(const NormParams& p, int pos, int c0, bool rot, float* cs, F2 (&c)[4],
                                             F2 (&s)[4]) {
  const int half = p.rope_dim >> 1;
  for (int i = threadIdx.x & 31; i < half; i += 32) {
    double turns;   // by its generic address: an indexed constant load would serve the lanes one after another
    asm("ld.f64 %0, [%1];" : "=d"(turns) : "l"(&p.turns[i]));
    turns *= pos;
    float x, y;
    sincospif((float)(2.0 * (turns - rint(turns))), &y, &x);   // the whole turns go in 64 bits, exactly
    cs[i] = x;
    cs[kMaxHalfGate + i] = y;
  }
  __syncwarp();
  if (rot) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(cs + c0 + 4 * i);
      const float4 y = *reinterpret_cast<const float4*>(cs + kMaxHalfGate + c0 + 4 * i);
      c[2 * i] = f2(x.x, x.y);
      c[2 * i + 1] = f2(x.z, x.w);
      s[2 * i] = f2(y.x, y.y);
      s[2 * i + 1] = f2(y.z, y.w);
    }
  }
  __syncwarp();   // the next token's angles may go there
}

template <typename T>
__device__ __forceinline__ T* lane_row(const Rows& r, int t, int h, int c0) {
  return static_cast<T*>(r.data) + (int64_t)t * r.stride_t + (int64_t)h * r.stride_h + c0;
}

// This CTA's kind.
__device__ __forceinline__ int cta_kind(const NormParams& p) {
  int k = 0;
  while (k < 2 && blockIdx.x >= p.kind[k].cta0 + p.kind[k].ctas) ++k;
  return k;
}

// passes requested at once (more spill registers: three 50.0 us, four 50.6 against 48.4 for 8192 tokens; two in fp32 53 against
// 45 for 4096)
template <typename T>
constexpr int kForwardBatch = sizeof(T) == 4 ? 1 : 2;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kForwardCtas) norm_rope_kernel(const __grid_constant__ NormParams p) {
  constexpr int LPR = D / 16, RPP = 32 / LPR;   // lanes per row, rows per pass
  constexpr int B = kForwardBatch<T>;
  __shared__ __align__(16) float angles[kWarps][2 * kMaxHalfGate];
  const int which = cta_kind(p);
  const NormKind& kd = p.kind[which];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR, l = lane & (LPR - 1);
  const int unit = (blockIdx.x - kd.cta0) * (kWarps) + warp;
  const int t = unit / kd.units, j = (unit - t * kd.units) * kd.per_unit;
  if (t >= p.T) return;
  int c0, c1;
  const bool rot = lane_chunks(l, p.rope_dim, &c0, &c1);
  const int gap = c1 - c0;
  const int n = min(kd.per_unit, kd.passes - j);
  const int h = j * RPP + sub;
  int room = kd.heads - h;   // rows h, h + RPP, .. while room > 0
  const T* src = lane_row<T>(kd.x, t, h, c0);
  pdl_wait();
  pdl_trigger();
  Chunk<T> x0[B], x1[B];
  auto load = [&]() {
#pragma unroll
    for (int u = 0; u < B; ++u) {
      x0[u] = x1[u] = Chunk<T>{};
      if (room > u * RPP) {
        x0[u] = load_chunk(src);
        x1[u] = load_chunk(src + gap);
      }
      src += RPP * kd.x.stride_h;
    }
  };
  load();
  const int live = live_rows(p);
  const bool turn = which < 2 && p.rope_dim > 0;
  const int pos = turn ? p.positions[t] : 0;
  const int slot = kd.cache.data ? p.slot_map[t] : -1;
  Chunk<T> w0 = {}, w1 = {};
  if (kd.weight) {
    w0 = load_chunk(static_cast<const T*>(kd.weight) + c0);
    w1 = load_chunk(static_cast<const T*>(kd.weight) + c1);
  }
  if (t >= live) return;
  F2 c[4], s[4];
  if (turn) token_angles(p, pos, c0, rot, angles[warp], c, s);
  T* cache = nullptr;   // the row's place in the cache
  if (kd.cache.data) {
    if (slot >= 0 && slot < p.slots) {
      const int page = slot / p.page_size;
      cache = static_cast<T*>(kd.cache.data) + page * kd.cache.stride_page + h * kd.cache.stride_h +
              (int64_t)(slot - page * p.page_size) * kd.cache.stride_t + c0;
    } else if (slot != -1 && lane == 0) {
      report(p.err, SEER_DEVERR_PAGE_INDEX);
    }
  }
  T* out = lane_row<T>(kd.out, t, h, c0);
  T* nope = lane_row<T>(kd.nope, t, h, c0);
  for (int i = 0; i < n; i += B) {
#pragma unroll
    for (int u = 0; u < B; ++u) {
      if (i + u >= n) break;
      const bool mine = room > 0;
      if (which == 2) {   // values: the cache copy only
        if (cache && mine) {
          store_chunk(cache, x0[u]);
          store_chunk(cache + gap, x1[u]);
        }
      } else {
        F2 a[4], b[4];
        unpack(x0[u], a);
        unpack(x1[u], b);
        if (kd.weight) {
          F2 qa = mul2(a[0], a[0]), qb = mul2(b[0], b[0]);
#pragma unroll
          for (int e = 1; e < 4; ++e) {
            qa = fma2(a[e], a[e], qa);
            qb = fma2(b[e], b[e], qb);
          }
          const float2 qs = split(add2(qa, qb));
          const float rs = rsqrtf(row_sum<LPR>(qs.x + qs.y) * (1.0f / D) + p.eps);
          const F2 r2 = f2(rs, rs);
          F2 wa[4], wb[4];
          unpack(w0, wa);
          unpack(w1, wb);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = mul2(a[e], mul2(r2, wa[e]));
            b[e] = mul2(b[e], mul2(r2, wb[e]));
          }
        }
        if (mine) {
          if (kd.nope.data) {
            store_chunk(nope, pack<T>(a));
            store_chunk(nope + gap, pack<T>(b));
          }
          if (rot) rotate<false>(a, b, c, s);
          const Chunk<T> z0 = pack<T>(a), z1 = pack<T>(b);
          if (kd.out.data) {
            store_chunk(out, z0);
            store_chunk(out + gap, z1);
          }
          if (cache) {
            store_chunk(cache, z0);
            store_chunk(cache + gap, z1);
          }
        }
        out += RPP * kd.out.stride_h;
        nope += RPP * kd.nope.stride_h;
      }
      cache += cache ? RPP * kd.cache.stride_h : 0;
      room -= RPP;
    }
    if (i + B < n) load();
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}

// A ring of STAGES passes of N arrays' chunks (x, gradient of the rotated rows, of the un-rotated ones), a
// lane's 16 bytes beside its neighbours'.
template <typename T, int N, int STAGES>
struct Ring {
  static constexpr int kHalf = (int)sizeof(Chunk<T>) / 16;   // pieces of a chunk
  static constexpr int kStage = N * 2 * kHalf * 512, kBytes = STAGES * kStage;   // per warp
  static __device__ __forceinline__ void request(uint32_t at, int array, const char* lo, int gap) {
#pragma unroll
    for (int i = 0; i < 2 * kHalf; ++i)
      cp_async16(at + (array * 2 * kHalf + i) * 512, lo + (i < kHalf ? 0 : gap) + i % kHalf * 16);
  }
  static __device__ __forceinline__ void read(uint32_t at, int array, Chunk<T>* x0, Chunk<T>* x1) {
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      x0->v[i] = lds16(at + (array * 2 * kHalf + i) * 512);
      x1->v[i] = lds16(at + (array * 2 * kHalf + kHalf + i) * 512);
    }
  }
};
template <typename T>
constexpr int backward_stages() { return sizeof(T) == 4 ? 2 : 4; }

// Backward: the weight gradient of a lane's 16 channels stays in registers over the warp's passes; at the end the lanes
// and warps of the CTA are added up in a fixed order and go to the CTA's row of the workspace.  These sums are fp32, as
// sine and cosine are (of angles reduced in fp64): chains are short (8 passes for most sizes, 32 lanes, up to 32 CTAs a thread), and
// fp32 gradients come out 2e-7 from their 64-bit values, where sums and angles in 64 bits leave 8e-8.
// Y: whether the un-rotated rows have a gradient.
template <typename T, int D, bool Y>
__global__ void __launch_bounds__(kThreads, kBackwardCtas) norm_rope_backward_kernel(const __grid_constant__ NormParams p) {
  constexpr int LPR = D / 16, RPP = 32 / LPR;
  constexpr int STAGES = backward_stages<T>();
  using R = Ring<T, Y ? 3 : 2, STAGES>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float angles[kWarps][2 * kMaxHalfGate];
  const int which = cta_kind(p);
  const NormKind& kd = p.kind[which];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR, l = lane & (LPR - 1);
  const uint32_t ring = smem_u32(smem) + warp * R::kBytes + lane * 16;
  int c0, c1;
  const bool rot = lane_chunks(l, p.rope_dim, &c0, &c1);
  const int gap = (c1 - c0) * (int)sizeof(T);
  pdl_wait();
  pdl_trigger();
  const int live = live_rows(p);
  const int total = live * kd.passes;
  const int64_t first = ((int64_t)(blockIdx.x - kd.cta0) * kWarps + warp) * kd.run;   // of the list of all passes
  int left = (int)min((int64_t)kd.run, total - first);
  F2 dw0[4] = {}, dw1[4] = {};
  if (left > 0) {
    int t = (int)first / kd.passes, j = (int)first - t * kd.passes;
    const bool turn = kd.out.data && p.rope_dim > 0;
    int npos = turn ? p.positions[t] : 0;   // of the next token
    int ahead = left, rt = t, rj = j;       // passes to request, and where
    const char *sx, *sz, *sy;
    auto place = [&]() {
      sx = reinterpret_cast<const char*>(lane_row<T>(kd.x, rt, rj * RPP + sub, c0));
      sz = reinterpret_cast<const char*>(lane_row<T>(kd.out, rt, rj * RPP + sub, c0));
      sy = reinterpret_cast<const char*>(lane_row<T>(kd.nope, rt, rj * RPP + sub, c0));
    };
    place();
    auto request = [&](uint32_t at) {
      if (ahead > 0) {
        if (rj * RPP + sub < kd.heads) {   // rows that are not there stay unread
          if (kd.weight) R::request(at, 0, sx, gap);
          if (kd.out.data) R::request(at, 1, sz, gap);
          if (Y && kd.nope.data) R::request(at, 2, sy, gap);
        }
        --ahead;
        if (++rj == kd.passes) {
          rj = 0;
          ++rt;
          place();
        } else {
          sx += RPP * (int)sizeof(T) * kd.x.stride_h;
          sz += RPP * (int)sizeof(T) * kd.out.stride_h;
          if (Y) sy += RPP * (int)sizeof(T) * kd.nope.stride_h;
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) request(ring + s * R::kStage);
    Chunk<T> w0 = {}, w1 = {};
    if (kd.weight) {
      w0 = load_chunk(static_cast<const T*>(kd.weight) + c0);
      w1 = load_chunk(static_cast<const T*>(kd.weight) + c1);
    }
    uint32_t at = ring, prev = ring + (STAGES - 1) * R::kStage;
    F2 c[4], s[4];
    while (left > 0) {
      const int n = min(kd.passes - j, left);
      if (turn) {
        const int pos = npos;
        if (t + 1 < live) npos = p.positions[t + 1];
        token_angles(p, pos, c0, rot, angles[warp], c, s);
      }
      int room = kd.heads - j * RPP - sub;
      T* out = lane_row<T>(kd.dx, t, j * RPP + sub, c0);
      for (int i = 0; i < n; ++i) {
        cp_wait<STAGES - 2>();
        const bool mine = room > 0;
        // a row that is not there reads whatever lies in the ring: it meets no other row and is not stored
        Chunk<T> x0, x1, z0 = {}, z1 = {}, y0, y1;
        R::read(at, 0, &x0, &x1);
        if (kd.out.data) R::read(at, 1, &z0, &z1);
        if (Y && kd.nope.data) R::read(at, 2, &y0, &y1);
        request(prev);
        prev = at;
        at = at == ring + (STAGES - 1) * R::kStage ? ring : at + R::kStage;
        F2 a[4], b[4];
        unpack(z0, a);
        unpack(z1, b);
        if (rot && turn) rotate<true>(a, b, c, s);
        if (Y && kd.nope.data) {
          F2 ya[4], yb[4];
          unpack(y0, ya);
          unpack(y1, yb);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = add2(a[e], ya[e]);
            b[e] = add2(b[e], yb[e]);
          }
        }
        if (kd.weight) {
          F2 wa[4], wb[4], xa[4], xb[4], ga[4], gb[4];   // ga: dy x
          unpack(x0, xa);
          unpack(x1, xb);
          unpack(w0, wa);
          unpack(w1, wb);
          F2 qa = mul2(xa[0], xa[0]), qb = mul2(xb[0], xb[0]);
          ga[0] = mul2(a[0], xa[0]);
          gb[0] = mul2(b[0], xb[0]);
          F2 da = mul2(ga[0], wa[0]), db = mul2(gb[0], wb[0]);
#pragma unroll
          for (int e = 1; e < 4; ++e) {
            qa = fma2(xa[e], xa[e], qa);
            qb = fma2(xb[e], xb[e], qb);
            ga[e] = mul2(a[e], xa[e]);
            gb[e] = mul2(b[e], xb[e]);
            da = fma2(ga[e], wa[e], da);
            db = fma2(gb[e], wb[e], db);
          }
          const float2 qs = split(add2(qa, qb)), ds = split(add2(da, db));
          const float rs = rsqrtf(row_sum<LPR>(qs.x + qs.y) * (1.0f / D) + p.eps);
          const float k = row_sum<LPR>(ds.x + ds.y) * (-1.0f / D) * rs * rs;
          const F2 r2 = f2(rs, rs), k2 = f2(k, k);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (mine) {
              dw0[e] = fma2(ga[e], r2, dw0[e]);
              dw1[e] = fma2(gb[e], r2, dw1[e]);
            }
            a[e] = mul2(r2, fma2(xa[e], k2, mul2(a[e], wa[e])));
            b[e] = mul2(r2, fma2(xb[e], k2, mul2(b[e], wb[e])));
          }
        }
        if (mine) {
          store_chunk(out, pack<T>(a));
          store_chunk(out + (c1 - c0), pack<T>(b));
        }
        out += RPP * kd.dx.stride_h;
        room -= RPP;
      }
      left -= n;
      j = 0;
      ++t;
    }
  }
  if (!kd.weight) return;
  cp_wait<0>();
  __syncwarp();   // the ring's memory is free
  static_assert(R::kBytes >= RPP * D * 4, "a warp's sums fit its ring");
  auto sums = [&](int w) { return reinterpret_cast<float*>(smem + w / RPP * R::kBytes) + w % RPP * D; };
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const float2 x = split(dw0[e]), x2 = split(dw0[e + 1]), y = split(dw1[e]), y2 = split(dw1[e + 1]);
    *reinterpret_cast<float4*>(sums(warp * RPP + sub) + c0 + 2 * e) = make_float4(x.x, x.y, x2.x, x2.y);
    *reinterpret_cast<float4*>(sums(warp * RPP + sub) + c1 + 2 * e) = make_float4(y.x, y.y, y2.x, y2.y);
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps * RPP; ++w) x += sums(w)[threadIdx.x];
    p.partial[(size_t)blockIdx.x * D + threadIdx.x] = x;
  }
}

// Sums of the CTAs' partial weight gradients in a fixed order: eight channels of one kind a CTA, 128 threads each.
struct WeightSums {
  const float* partial;
  float* dw[2];   // null: absent
  int cta0[2], ctas[2];
};
template <int D>
__global__ void __launch_bounds__(1024) norm_weight_kernel(const __grid_constant__ WeightSums p) {
  __shared__ float red[32][8];
  const int k = blockIdx.x / (D / 8), c = blockIdx.x % (D / 8) * 8 + (threadIdx.x & 7), g = threadIdx.x >> 3;
  pdl_wait();
  pdl_trigger();
  if (!p.dw[k]) return;
  float s = 0.f;
#pragma unroll 8
  for (int i = g; i < p.ctas[k]; i += 128) s += p.partial[(size_t)(p.cta0[k] + i) * D + c];
  s += __shfl_xor_sync(0xffffffffu, s, 8);
  s += __shfl_xor_sync(0xffffffffu, s, 16);
  if ((threadIdx.x & 31) < 8) red[threadIdx.x >> 5][threadIdx.x & 7] = s;
  __syncthreads();
  if (threadIdx.x < 8) {
#pragma unroll
    for (int w = 1; w < 32; ++w) s += red[w][threadIdx.x];
    p.dw[k][c] = s;
  }
}

// Passes a warp takes: `most`, fewer while that leaves warps of the machine idle.
int64_t warp_passes(const NormParams& p, int rpp, int64_t warps, int64_t most) {
  int64_t passes = 0;
  for (const NormKind& k : p.kind)
    if (k.used) passes += (int64_t)p.T * ((k.heads + rpp - 1) / rpp);
  return std::min(most, std::max<int64_t>(1, passes / warps));
}

template <typename T, int D>
cudaError_t forward(NormParams p, int sms, cudaStream_t s) {
  constexpr int rpp = 512 / D;
  const int64_t most = warp_passes(p, rpp, (int64_t)sms * kForwardCtas * kWarps, kUnitPasses);
  int grid = 0;
  for (NormKind& k : p.kind) {
    k.cta0 = grid;
    k.ctas = 0;
    if (!k.used) continue;
    k.passes = (k.heads + rpp - 1) / rpp;
    k.units = (int)((k.passes + most - 1) / most);
    k.per_unit = (k.passes + k.units - 1) / k.units;
    k.ctas = (int)(((int64_t)p.T * k.units + kWarps - 1) / kWarps);
    grid += k.ctas;
  }
  return launch_pdl(norm_rope_kernel<T, D>, dim3(grid), dim3(kThreads), 0, s, p);
}

std::atomic<uint64_t> g_limit[12];

template <typename T, int D, bool Y>
cudaError_t backward_of(NormParams p, int sms, cudaStream_t s) {
  constexpr int rpp = 512 / D, smem = kWarps * Ring<T, Y ? 3 : 2, backward_stages<T>()>::kBytes;
  constexpr int which = (Y ? 6 : 0) + (D == 128 ? 3 : 0) + (sizeof(T) == 4 ? 2 : std::is_same<T, __half>::value ? 1 : 0);
  cudaError_t e = ensure_smem_limit(norm_rope_backward_kernel<T, D, Y>, smem, g_limit[which]);
  if (e != cudaSuccess) return e;
  const int64_t run = warp_passes(p, rpp, (int64_t)sms * kBackwardCtas * kWarps, kRunPasses);
  constexpr int64_t rows = (int64_t)kNormPartials / 2 * kWarps;   // warps of a kind, at most
  int grid = 0;
  for (NormKind& k : p.kind) {
    k.cta0 = grid;
    k.ctas = 0;
    if (!k.used) continue;
    k.passes = (k.heads + rpp - 1) / rpp;
    const int64_t all = (int64_t)p.T * k.passes;
    k.run = (int)std::max(run, (all + rows - 1) / rows);
    k.ctas = (int)((all + (int64_t)k.run * kWarps - 1) / ((int64_t)k.run * kWarps));
    grid += k.ctas;
  }
  e = launch_pdl(norm_rope_backward_kernel<T, D, Y>, dim3(grid), dim3(kThreads), smem, s, p);
  if (e != cudaSuccess || !(p.kind[0].dw || p.kind[1].dw)) return e;
  WeightSums w = {p.partial};
  for (int k = 0; k < 2; ++k) {
    w.dw[k] = p.kind[k].dw;
    w.cta0[k] = p.kind[k].cta0;
    w.ctas[k] = p.kind[k].ctas;
  }
  return launch_pdl(norm_weight_kernel<D>, dim3(2 * (D / 8)), dim3(1024), 0, s, w);
}

template <typename T, int D>
cudaError_t backward(const NormParams& p, int sms, cudaStream_t s) {
  return p.kind[0].nope.data || p.kind[1].nope.data ? backward_of<T, D, true>(p, sms, s) : backward_of<T, D, false>(p, sms, s);
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
