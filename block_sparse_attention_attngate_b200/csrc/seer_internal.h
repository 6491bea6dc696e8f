// Internal launch interface between the C ABI layer (seer_api.cu) and the
// kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "seer.h"

namespace seer {

// Launch `kern` on `s` with programmatic stream serialization (see pdl_wait /
// pdl_trigger in seer_device.cuh).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
}

// Raise a kernel's dynamic shared-memory limit once per device (a host-side
// attribute call, kept out of CUDA-graph capture after the first use).
template <typename Kernel>
cudaError_t ensure_smem_limit(Kernel kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}


// ~1 s at 2 GHz: a wait that runs this long means a copy never landed (the default bound).
constexpr long long kWaitLimitCycles = 2000000000LL;
constexpr int kMaxGroup = 8;        // query heads per KV head
constexpr int kMaxBlocksRow = 8192; // max_blocks limit (selection keeps a row in shared memory)
constexpr int kMaxDecodeB = 4096;   // decode keeps the sequence lengths in shared memory
constexpr int kMaxDecodeBH = 4096;  // balanced decode keeps the list-length prefix in shared memory

// Where a K/V tile lives, for kernels that read it with plain loads.
struct KvPlain {
  const uint16_t* data;
  int64_t stride_b, stride_h, stride_t;   // elements
  const int32_t* block_table;             // paged only
  int32_t max_pages;
  int64_t num_pages;
  int64_t num_tokens;                     // contiguous only: token capacity
  int32_t paged;
};

// ---------------------------------------------------------------- kcomp update
constexpr int kMaxHalfGate = 64;    // d_gate / 2 rotation frequencies

struct KcompParams {
  double theta[kMaxHalfGate];   // base^(-2i/d_gate), computed on the host in fp64
  KvPlain k;
  const int32_t* seqlens;
  const int32_t* valid;
  int32_t* valid_out;
  const uint16_t* w_k;     // [Hkv, DG, 3D]
  uint16_t* kcomp;         // [B, Hkv, NB, DG]
  int32_t B, Hkv, NB;
  float rope_base;
  int32_t* err;
};
cudaError_t launch_kcomp_update(const KcompParams& p, int D, int BLK, int DG, int grid_x,
                                cudaStream_t s);

// ---------------------------------------------------------------- cache from running block statistics
struct AppendParams {
  double theta[kMaxHalfGate];   // base^(-2i/d_gate), computed on the host in fp64
  const uint16_t* k_new;   // [B, Hkv, D] pre-RoPE key of token seqlens[b]-1 (append)
  KvPlain k;               // pre-RoPE key cache (state init)
  const int32_t* seqlens;
  int32_t* valid;          // [B, Hkv] fill counts, read and advanced
  float* state;            // [B, Hkv, 3, D] running max / min / sum of the current block
  const uint16_t* w_k;     // [Hkv, DG, 3D]
  uint16_t* kcomp;         // [B, Hkv, NB, DG]
  int32_t B, Hkv, NB;
  int32_t* err;
};
cudaError_t launch_kcomp_append(const AppendParams& p, int D, int BLK, int DG, cudaStream_t s);
cudaError_t launch_kcomp_state_init(const AppendParams& p, int D, int BLK, cudaStream_t s);

// ---------------------------------------------------------------- prefill attention + block target
struct PrefillParams {
  const uint16_t* q;       // [B, Hq, T, D]
  uint16_t* o;             // [B, Hq, T, D]
  float* lse;              // [B, Hq, T] or null
  float* gt;               // [B, Hkv, T, NB]
  float* rmax;             // workspace [B, Hq, NB, T]: each row's tile maxima (log2 domain)
  float* rnorm;            // workspace [B, Hq, T]: each row's final m + log2(l) (tcgen05 path)
  const int32_t* seqlens;  // [B]
  int32_t k_perm[3], v_perm[3];
  int32_t B, Hq, Hkv, g, NB, T;
  int32_t kcap;            // tokens the K and V caches hold per sequence
  float scale_log2;
  int32_t* err;
};
cudaError_t launch_prefill_gt(const CUtensorMap& tk, const CUtensorMap& tv, const PrefillParams& p, int D, int BLK,
                              int max_len, cudaStream_t s);
// The same forward on tcgen05 / TMEM (prefill_tc.cu): head_dim 128, groups of 1, 2, 4 or 8.
bool prefill_tc_supported(int D, int BLK, int g);
// One persistent CTA per SM (sms = the device's SM count), items of 128 rows heaviest first.
cudaError_t launch_prefill_tc(const CUtensorMap& tk, const CUtensorMap& tv, const PrefillParams& p, int D, int BLK,
                              int max_len, int sms, cudaStream_t s);

// ---------------------------------------------------------------- gate score
struct GateParams {
  double theta[kMaxHalfGate];   // base^(-2i/d_gate), computed on the host in fp64
  const uint16_t* q;       // [B, Hq, D]
  const uint16_t* w_q;     // [Hkv, DG, g*D]
  const uint16_t* kcomp;   // [B, Hkv, NB, DG]
  const int32_t* seqlens;
  float* logits;           // [B, Hkv, NB]
  float* q_gate;           // [B, Hkv, DG] or null
  int32_t B, Hq, Hkv, g, NB, BLK;
  float rope_base;
};
cudaError_t launch_gate_score(const GateParams& p, int D, int DG, cudaStream_t s);

// ---------------------------------------------------------------- select
struct SelectParams {
  const float* logits;     // [B, Hkv, NB]
  const int32_t* seqlens;
  int32_t* idx;            // [B, Hkv, cap]
  int32_t* cnt;            // [B, Hkv]
  int32_t B, Hkv, NB, BLK, cap;
  int32_t mode;            // 0 top-k, 1 threshold, 2 top-p
  int32_t kblocks;         // top-k
  double tau;              // threshold / top-p mass
};
cudaError_t launch_select(const SelectParams& p, cudaStream_t s);

// ---------------------------------------------------------------- fused plan (cache update + gate + select)
struct PlanParams {
  KcompParams k;
  GateParams g;
  SelectParams s;
  int32_t update_cache;   // run the cache update first
};
cudaError_t launch_plan(const PlanParams& p, int D, int BLK, int DG, cudaStream_t s);

// ---------------------------------------------------------------- sparse decode
struct DecodeParams {
  const uint16_t* q;        // [B, Hq, D]
  const int32_t* idx;       // [B, Hkv, cap]
  const int32_t* cnt;       // [B, Hkv]
  const int32_t* seqlens;   // [B]
  const int32_t* k_table;   // paged block tables (may be equal)
  const int32_t* v_table;
  int32_t k_maxp, v_maxp;
  int64_t k_pages, v_pages;
  int32_t k_paged, v_paged;
  int32_t k_perm[3], v_perm[3];   // TMA dim (1..3) that holds token / head / batch-or-page
  int32_t B, Hq, Hkv, g;
  int32_t flat;             // 0: (split, kv head, batch) grid; one-wave ranges over 1: the concatenated
                            // lists (balanced), 2: every list padded to its capacity (capacity schedule)
  int32_t cap, ns, per_split;
  float scale_log2;         // softmax scale * log2(e)
  float* o_part;            // [B, Hq, ns, D]
  float* lse_part;          // [B, Hq, ns]
  int32_t* counters;        // [B, Hkv] split-arrival counters (zero between calls)
  uint16_t* out;            // [B, Hq, D] bf16
  float* lse_out;           // [B, Hq] or null
  int32_t* err;
  int32_t* ready;           // fused step: [B, Hkv] per-row list-ready flags (zero between calls); else null
  long long wait_limit;     // bound of every copy / hand-off wait, in SM cycles
  int32_t starve;           // debug: the producer issues no copy (every first wait runs out); 0 in use
};
cudaError_t launch_sparse_decode(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p,
                                 int D, int BLK, int grid_flat, cudaStream_t s);
int decode_ctas_per_sm(int D, int BLK);

// ---------------------------------------------------------------- fused decode step (plan + decode)
struct StepParams {
  DecodeParams d;   // capacity schedule (flat == 2), d.ready set
  PlanParams pl;
};
// Grid of the fused step on the current device: 2 x the co-resident clusters of two, at most one
// CTA per SM; 0 when the shape has no fused kernel or its shared memory does not fit.
int step_grid(int D, int BLK, int DG, int g, int NB, int mode, int B, int BH);
cudaError_t launch_decode_step(const CUtensorMap& tk, const CUtensorMap& tv, const StepParams& p, int D, int BLK,
                               int DG, int grid, cudaStream_t s);

// seer_sparse_decode in two stages: every argument check and the launch set-up (tensor maps,
// parameters), which enqueues nothing, then the launch itself.
struct DecodeLaunch {
  CUtensorMap tk, tv;
  DecodeParams p;
  int D, BLK, ctas;
  size_t need;   // workspace bytes the launch uses
};
seer_status prepare_sparse_decode(const seer_dims_t* dims, const void* q, const seer_kv_t* k, const seer_kv_t* v,
                                  const int32_t* block_idx, const int32_t* block_cnt, const int32_t* seqlens,
                                  int32_t capacity, int32_t num_split, void* workspace, size_t workspace_bytes,
                                  void* out, float* lse_out, int32_t* err_word, DecodeLaunch* launch);
seer_status launch_prepared_decode(const DecodeLaunch& launch, cudaStream_t s);

// ---------------------------------------------------------------- decode ground truth
struct TruthParams {
  const uint16_t* q;        // [B, Hq, D]
  const int32_t* seqlens;   // [B]
  const int32_t* k_table;   // paged block table or null
  int32_t k_maxp;
  int64_t k_pages;
  int32_t k_paged;
  int32_t k_perm[3];
  int32_t B, Hq, Hkv, g, NB, nchunk;
  int32_t nitems;           // B * Hkv * nchunk work items
  float scale_log2;         // softmax scale * log2(e)
  float* scores;            // [B, Hkv, NB]
  float* log_scores;        // [B, Hkv, NB] or null
  float* bmax;              // workspace [B*Hkv, NB, 8]: per head, the block's score maximum (log2 domain)
  float* part;              // workspace [B*Hkv, nchunk, 8, 2]: per head, the chunk's (max, sum of exp2)
  int32_t* counters;        // workspace [B*Hkv] (zero between calls)
  int32_t* err;
};
cudaError_t launch_gate_truth(const CUtensorMap& tk, const TruthParams& p, int D, int BLK, int sms, cudaStream_t s);
int truth_chunk_blocks();

// ---------------------------------------------------------------- division by a number known at the launch
// x / d = mulhi(x, magic) >> shift for 0 <= x < 2^31 and d >= 2: with s = ceil(log2 d) and
// magic = ceil(2^(31 + s) / d) < 2^32, the excess magic d - 2^(31 + s) is below d <= 2^s, so x times it is below
// 2^(31 + s) and the quotient's floor is exact.  mulhi takes 32 of the 31 + s bits.
struct Divisor {
  int32_t d;
  uint32_t magic;
  int32_t shift;
#ifdef __CUDACC__
  __device__ __forceinline__ int div(int x) const { return d == 1 ? x : (int)(__umulhi((uint32_t)x, magic) >> shift); }
#endif
};
inline Divisor divisor(int32_t d) {   // d >= 1
  int s = 0;
  while (((int64_t)1 << s) < d) ++s;
  return {d, d < 2 ? 0u : (uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d), s - 1};
}

// ---------------------------------------------------------------- page tables
struct PageParams {
  const int32_t* seqlens;       // [B]
  const int32_t* per_request;   // [B] plan: tokens to append; release: finished flags
  int32_t* block_table;         // [B, width]
  const int32_t* free_list;     // [num_pages] stack (plan reads it)
  int32_t* free_out;            // [num_pages] the same stack (release pushes)
  const int32_t* free_count;
  int32_t* seqlens_out;         // may be seqlens
  int32_t* free_count_out;      // may be free_count
  int32_t* cu_tokens;           // [B + 1]
  int32_t* slot_map;            // [max_tokens]
  int32_t* positions;           // [max_tokens]
  int32_t B, page, num_pages, width, max_tokens;
  int32_t* err;
  Divisor by_page;              // set by the launch, as the next
  int32_t in_place;
};
cudaError_t launch_page_plan(const PageParams& p, cudaStream_t s);
cudaError_t launch_page_release(const PageParams& p, cudaStream_t s);

// ---------------------------------------------------------------- per-head norm + rotation (+ cache write)
struct Rows {
  void* data;
  int64_t stride_t, stride_h;   // elements
};
struct Pool {
  void* data;
  int64_t stride_page, stride_h, stride_t;   // elements
};
// One kind of row (query, key or value heads) of a norm + rotation launch.
struct NormKind {
  Rows x;             // input rows; data null: absent (values: the cache copy's source)
  Rows out, nope;     // forward: rotated / un-rotated outputs (null: absent); backward: their gradients
  Rows dx;            // backward: gradient of x (null: the kind is absent)
  Pool cache;         // forward: rows of slot_map (null: absent)
  const void* weight; // [D] or null (no norm)
  float* dw;          // backward: [D] or null
  int32_t heads;
  int32_t used;       // whether the kind has anything to do
  // set by the launch: passes of a token's heads, units of a token, passes of a unit, passes of a warp (backward), the kind's CTAs
  int32_t passes, units, per_unit, run, cta0, ctas;
};
struct NormParams {
  double turns[kMaxHalfGate];   // base^(-2i / rope_dim) / 2 pi, i < rope_dim / 2
  NormKind kind[3];             // query, key, value (values: cache copy only)
  const int32_t* positions;
  const int32_t* slot_map;
  const int32_t* live;          // device row count or null
  int32_t T, rope_dim, page_size;
  int32_t slots;                // token slots of the pools
  float eps;
  float* partial;               // backward workspace [kNormPartials][D]
  int32_t* err;
};
constexpr int kNormPartials = 8192;   // CTAs of the backward pass, at most
cudaError_t launch_norm_rope(const NormParams& p, int D, int dtype, int sms, cudaStream_t s);
cudaError_t launch_norm_rope_backward(const NormParams& p, int D, int dtype, int sms, cudaStream_t s);

// ---------------------------------------------------------------- dense one-token attention
struct DenseParams {
  const uint16_t* q;            // [B, Hq, D]
  uint16_t* out;                // [B, Hq, D]
  float* lse;                   // [B, Hq] or null
  KvPlain k, v;
  const int32_t* seqlens;       // [B]
  int32_t B, Hq, Hkv, g, window, page;
  int32_t cap;                  // tokens the caches hold per sequence
  float scale_log2;             // softmax scale * log2(e)
  int4* join;                   // [entries] {row b * Hkv + h, pieces, first range, 0}; fewer than 2 pieces: nothing to join
  float4* ml_part;              // [2 * ranges][NT * 4] {m, l, m, l} of a lane's two heads (log2 domain)
  float4* o_part;               // [2 * ranges][NT * d / 16][32] register order
  int32_t* err;
  int32_t by_row;               // join entries are indexed by row, else by range; set by the launch, as the next
  int32_t pad;                  // units a row counts on top of its own
  Divisor by_page;
};
constexpr int kDenseMaxGroup = 16;
constexpr int kDenseUnit = 32;  // tokens per scheduling unit
int dense_ranges(int ctas);     // ranges of a launch, at most
cudaError_t launch_dense_decode(const DenseParams& p, int D, int dtype, int ctas, cudaStream_t s);

// Record `msg` as the text seer_last_error() returns on this thread; returns `status`.
int set_last_error(int status, const char* msg);

}  // namespace seer
