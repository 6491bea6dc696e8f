// C ABI of libseer (declared in include/seer.h): argument validation, TMA
// descriptor encoding (cached), launch-shape choices and kernel launches.
// Nothing here allocates device memory or synchronises the host.
#include <cstdint>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <string>

#include "seer.h"
#include "seer_internal.h"

namespace {

thread_local std::string g_err;

seer_status fail(seer_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_err = buf;
  return st;
}

seer_status cuda_fail(cudaError_t e, const char* what) {
  return fail(SEER_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

seer_status check_dims(const seer_dims_t* d) {
  if (!d) return fail(SEER_ERR_INVALID_ARG, "dims is NULL");
  if (d->batch < 1 || d->num_q_heads < 1 || d->num_kv_heads < 1)
    return fail(SEER_ERR_INVALID_ARG, "batch, num_q_heads and num_kv_heads must be >= 1");
  if (d->num_q_heads % d->num_kv_heads != 0)
    return fail(SEER_ERR_INVALID_ARG, "num_q_heads (%d) is not a multiple of num_kv_heads (%d)",
                d->num_q_heads, d->num_kv_heads);
  const int g = d->num_q_heads / d->num_kv_heads;
  if (g > seer::kMaxGroup) return fail(SEER_ERR_UNSUPPORTED, "group size %d > %d", g, seer::kMaxGroup);
  if (d->head_dim != 64 && d->head_dim != 128)
    return fail(SEER_ERR_UNSUPPORTED, "head_dim %d not in {64, 128}", d->head_dim);
  if (d->gate_dim != 64 && d->gate_dim != 128)
    return fail(SEER_ERR_UNSUPPORTED, "gate_dim %d not in {64, 128}", d->gate_dim);
  if (d->block_size != 64 && d->block_size != 128)
    return fail(SEER_ERR_UNSUPPORTED, "block_size %d not in {64, 128}", d->block_size);
  if (d->max_blocks < 1 || d->max_blocks > seer::kMaxBlocksRow)
    return fail(SEER_ERR_UNSUPPORTED, "max_blocks %d not in [1, %d]", d->max_blocks, seer::kMaxBlocksRow);
  if (!(d->rope_base > 0.f) || !isfinite(d->rope_base)) return fail(SEER_ERR_INVALID_ARG, "rope_base must be > 0");
  if (!(d->softmax_scale >= 0.f) || !isfinite(d->softmax_scale))
    return fail(SEER_ERR_INVALID_ARG, "softmax_scale must be >= 0 (0 = 1/sqrt(head_dim))");
  return SEER_OK;
}

seer_status check_kv(const seer_dims_t* d, const seer_kv_t* kv, const char* name) {
  if (!kv) return fail(SEER_ERR_INVALID_ARG, "%s descriptor is NULL", name);
  if (!kv->data) return fail(SEER_ERR_INVALID_ARG, "%s data is NULL", name);
  if (!aligned16(kv->data)) return fail(SEER_ERR_INVALID_ARG, "%s data is not 16-byte aligned", name);
  if (kv->layout != SEER_KV_CONTIGUOUS && kv->layout != SEER_KV_PAGED)
    return fail(SEER_ERR_INVALID_ARG, "%s layout %d unknown", name, kv->layout);
  const int64_t D = d->head_dim;
  if (kv->stride_t < D || kv->stride_h < 1 || kv->stride_b < 1)
    return fail(SEER_ERR_INVALID_ARG, "%s strides (b=%lld h=%lld t=%lld) invalid for head_dim %lld", name,
                (long long)kv->stride_b, (long long)kv->stride_h, (long long)kv->stride_t, (long long)D);
  if ((kv->stride_t % 8) || (kv->stride_h % 8) || (kv->stride_b % 8))
    return fail(SEER_ERR_INVALID_ARG, "%s strides must be multiples of 8 elements (16 bytes)", name);
  if (kv->layout == SEER_KV_CONTIGUOUS) {
    if (kv->num_tokens < 1) return fail(SEER_ERR_INVALID_ARG, "%s num_tokens must be >= 1", name);
  } else {
    if (!kv->block_table) return fail(SEER_ERR_INVALID_ARG, "%s block_table is NULL (paged layout)", name);
    if (kv->num_pages < 1 || kv->max_pages_per_seq < 1)
      return fail(SEER_ERR_INVALID_ARG, "%s num_pages and max_pages_per_seq must be >= 1", name);
    if (kv->num_pages > INT32_MAX) return fail(SEER_ERR_UNSUPPORTED, "%s num_pages above 2^31", name);
  }
  return SEER_OK;
}

// ------------------------------------------------------------------ device facts (cached per device)
struct DevFacts {
  int sms = 0;
  int occ[2][2] = {{0, 0}, {0, 0}};  // decode CTAs/SM by [D==128][BLK==128]
};
std::mutex g_mu;
DevFacts g_dev[64];

seer_status device_facts(int* dev_out, DevFacts** f) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= 64) return fail(SEER_ERR_UNSUPPORTED, "device ordinal %d", dev);
  std::lock_guard<std::mutex> lk(g_mu);
  DevFacts& df = g_dev[dev];
  if (df.sms == 0) {
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
    df.sms = sms;
  }
  *dev_out = dev;
  *f = &df;
  return SEER_OK;
}

int decode_occ(DevFacts* df, int D, int BLK) {
  int& o = df->occ[D == 128][BLK == 128];
  if (o == 0) {
    std::lock_guard<std::mutex> lk(g_mu);
    if (o == 0) o = seer::decode_ctas_per_sm(D, BLK);
  }
  return o;
}

// ------------------------------------------------------------------ TMA descriptors
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;
std::once_flag g_encode_once;
cudaError_t g_encode_err = cudaSuccess;

seer_status encoder(EncodeTiledFn* fn) {
  std::call_once(g_encode_once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    g_encode_err = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
    if (g_encode_err == cudaSuccess && q != cudaDriverEntryPointSuccess) g_encode_err = cudaErrorNotSupported;
    if (g_encode_err == cudaSuccess) g_encode = reinterpret_cast<EncodeTiledFn>(p);
  });
  if (!g_encode) return cuda_fail(g_encode_err == cudaSuccess ? cudaErrorNotSupported : g_encode_err,
                                  "resolving cuTensorMapEncodeTiled");
  *fn = g_encode;
  return SEER_OK;
}

struct MapKey {
  const void* data;
  int64_t ext[3], str[3];
  int D, BLK;
  bool operator==(const MapKey& o) const {
    if (data != o.data || D != o.D || BLK != o.BLK) return false;
    for (int i = 0; i < 3; ++i)
      if (ext[i] != o.ext[i] || str[i] != o.str[i]) return false;
    return true;
  }
};
struct MapEntry {
  MapKey key;
  CUtensorMap map;
  int perm[3];
  bool used = false;
};
constexpr int kMapCache = 128;
MapEntry g_maps[kMapCache];
int g_map_next = 0;

// Describe a K/V cache as a 4-D tensor (channel, then token / head / batch-or-page
// sorted by stride), box = 64 channels x BLK tokens, 128-byte swizzle.
seer_status tensor_map(const seer_dims_t* d, const seer_kv_t* kv, const char* name, CUtensorMap* out,
                       int perm[3]) {
  MapKey key;
  key.data = kv->data;
  key.D = d->head_dim;
  key.BLK = d->block_size;
  const bool paged = kv->layout == SEER_KV_PAGED;
  key.ext[0] = paged ? d->block_size : kv->num_tokens;  // role 0: token
  key.ext[1] = d->num_kv_heads;                          // role 1: head
  key.ext[2] = paged ? kv->num_pages : d->batch;         // role 2: batch or page
  key.str[0] = kv->stride_t;
  key.str[1] = kv->stride_h;
  key.str[2] = kv->stride_b;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    for (int i = 0; i < kMapCache; ++i) {
      if (g_maps[i].used && g_maps[i].key == key) {
        *out = g_maps[i].map;
        for (int r = 0; r < 3; ++r) perm[r] = g_maps[i].perm[r];
        return SEER_OK;
      }
    }
  }
  EncodeTiledFn enc;
  seer_status st = encoder(&enc);
  if (st != SEER_OK) return st;
  // order roles by stride (stable): TMA dims 1..3
  int order[3] = {0, 1, 2};
  for (int i = 1; i < 3; ++i)
    for (int j = i; j > 0 && key.str[order[j]] < key.str[order[j - 1]]; --j) {
      int t = order[j];
      order[j] = order[j - 1];
      order[j - 1] = t;
    }
  cuuint64_t gdim[4], gstr[3];
  cuuint32_t box[4], estr[4] = {1, 1, 1, 1};
  gdim[0] = (cuuint64_t)d->head_dim;
  box[0] = 64;
  for (int i = 0; i < 3; ++i) {
    const int role = order[i];
    perm[role] = i;
    if (key.ext[role] < 1 || key.ext[role] > (int64_t(1) << 32))
      return fail(SEER_ERR_INVALID_ARG, "%s extent out of range for a TMA descriptor", name);
    gdim[i + 1] = (cuuint64_t)key.ext[role];
    gstr[i] = (cuuint64_t)key.str[role] * 2;
    if (gstr[i] >= (cuuint64_t(1) << 40)) return fail(SEER_ERR_INVALID_ARG, "%s stride too large for TMA", name);
    box[i + 1] = role == 0 ? (cuuint32_t)d->block_size : 1u;
  }
  CUtensorMap map;
  CUresult r = enc(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(kv->data), gdim, gstr, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SEER_ERR_INVALID_ARG, "%s: cuTensorMapEncodeTiled failed (%d)", name, (int)r);
  {
    std::lock_guard<std::mutex> lk(g_mu);
    MapEntry& e = g_maps[g_map_next];
    g_map_next = (g_map_next + 1) % kMapCache;
    e.key = key;
    e.map = map;
    for (int i = 0; i < 3; ++i) e.perm[i] = perm[i];
    e.used = true;
  }
  *out = map;
  return SEER_OK;
}

void rope_thetas(const seer_dims_t* d, double* theta) {
  const int half = d->gate_dim / 2;
  for (int i = 0; i < half; ++i) theta[i] = pow((double)d->rope_base, -2.0 * i / d->gate_dim);
}

seer_status select_args(const seer_dims_t* dims, int32_t mode, int32_t token_budget, float tau, int32_t capacity,
                        int32_t* kblocks) {
  if (mode != SEER_SELECT_TOPK && mode != SEER_SELECT_THRESHOLD && mode != SEER_SELECT_TOPP)
    return fail(SEER_ERR_INVALID_ARG, "unknown selection mode %d", mode);
  if (capacity < 1) return fail(SEER_ERR_INVALID_ARG, "capacity must be >= 1");
  *kblocks = 0;
  if (mode == SEER_SELECT_TOPK) {
    if (token_budget < 0) return fail(SEER_ERR_INVALID_ARG, "token_budget must be >= 0");
    int32_t k = (int32_t)(((int64_t)token_budget + dims->block_size - 1) / dims->block_size);
    if (k > dims->max_blocks) k = dims->max_blocks;
    if (capacity < k + 1 && capacity < dims->max_blocks)
      return fail(SEER_ERR_CAPACITY, "capacity %d < k+1 = %d (top-k plus the partial block)", capacity, k + 1);
    *kblocks = k;
  } else {
    if (!isfinite(tau)) return fail(SEER_ERR_INVALID_ARG, "tau must be finite");
    if (capacity < dims->max_blocks)
      return fail(SEER_ERR_CAPACITY, "capacity %d < max_blocks %d (threshold / top-p may select every block)",
                  capacity, dims->max_blocks);
  }
  return SEER_OK;
}

seer::KvPlain plain(const seer_kv_t* kv) {
  seer::KvPlain k;
  k.data = static_cast<const uint16_t*>(kv->data);
  k.stride_b = kv->stride_b;
  k.stride_h = kv->stride_h;
  k.stride_t = kv->stride_t;
  k.paged = kv->layout == SEER_KV_PAGED;
  k.block_table = kv->block_table;
  k.max_pages = kv->max_pages_per_seq;
  k.num_pages = kv->num_pages;
  k.num_tokens = kv->num_tokens;
  return k;
}

int32_t auto_split(const seer_dims_t* d, int32_t capacity, DevFacts* df) {
  const int64_t units = (int64_t)d->batch * d->num_kv_heads;
  const int64_t slots = (int64_t)df->sms * decode_occ(df, d->head_dim, d->block_size);
  int64_t ns = slots / units;                       // fill one wave, never spill into a second
  ns = ns < 1 ? 1 : ns;
  const int64_t max_ns = (capacity + 1) / 2;        // at least two list slots per split
  if (ns > max_ns) ns = max_ns;
  return (int32_t)(ns < 1 ? 1 : ns);
}

// CTAs of the balanced (num_split == 0) schedule: one per SM slot.
int flat_grid(const seer_dims_t* d, DevFacts* df) { return df->sms * decode_occ(df, d->head_dim, d->block_size); }

// Workspace: split-arrival counters [B*Hkv] int32 (zero before the first call, left zero) |
// lse partials [slots][g] | o partials [slots][g][d].  Balanced schedule: 2 partial slots per
// CTA (a CTA's first and last segment are the only ones that can belong to a (b, h) split
// across CTAs).  Grid schedule: num_split slots per (b, h).
size_t ws_layout(const seer_dims_t* d, int32_t ns, int flat_ctas, size_t* off_lse, size_t* off_o) {
  // ns <= 0: one of the one-wave schedules (balanced or capacity), 2 slots per CTA
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t g = (size_t)(d->num_q_heads / d->num_kv_heads);
  const size_t bh = (size_t)d->batch * d->num_kv_heads;
  const size_t slots = ns <= 0 ? 2 * (size_t)flat_ctas : bh * ns;
  const size_t rec = up(bh * 4);
  const size_t lse = up(slots * g * 4);
  const size_t o = slots * g * d->head_dim * 4;
  *off_lse = rec;
  *off_o = rec + lse;
  return ns == 1 ? 0 : rec + lse + o;
}

}  // namespace

int seer::set_last_error(int status, const char* msg) {
  g_err = msg ? msg : "";
  return status;
}

extern "C" {

const char* seer_last_error(void) { return g_err.c_str(); }

const char* seer_version(void) { return "libseer 0.1 (sm_100a)"; }

// process-wide bound and debug switch of the sparse decode's waits, read at each launch
namespace {
std::atomic<long long> g_wait_limit{seer::kWaitLimitCycles};
std::atomic<int32_t> g_debug{0};
}  // namespace

seer_status seer_set_wait_limit(int64_t cycles) {
  if (cycles == 0) cycles = seer::kWaitLimitCycles;
  if (cycles < SEER_WAIT_LIMIT_MIN || cycles > SEER_WAIT_LIMIT_MAX)
    return fail(SEER_ERR_INVALID_ARG, "wait limit %lld cycles outside [%lld, %lld] (0 = the default)",
                (long long)cycles, (long long)SEER_WAIT_LIMIT_MIN, (long long)SEER_WAIT_LIMIT_MAX);
  g_wait_limit.store(cycles);
  return SEER_OK;
}

int64_t seer_get_wait_limit(void) { return g_wait_limit.load(); }

seer_status seer_set_debug_flags(int32_t flags) {
  if (flags & ~SEER_DEBUG_STARVE_COPIES) return fail(SEER_ERR_INVALID_ARG, "unknown debug flags 0x%x", flags);
  g_debug.store(flags);
  return SEER_OK;
}

seer_status seer_kcomp_update(const seer_dims_t* dims, const seer_kv_t* k_nope, const int32_t* seqlens,
                              int32_t* valid_blocks, const void* w_k, void* kcomp, void* stream) {
  seer_status st = check_dims(dims);
  if (st != SEER_OK) return st;
  if ((st = check_kv(dims, k_nope, "k_nope")) != SEER_OK) return st;
  if (!seqlens || !valid_blocks || !w_k || !kcomp) return fail(SEER_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned16(w_k) || !aligned16(kcomp)) return fail(SEER_ERR_INVALID_ARG, "w_k / kcomp not 16-byte aligned");
  int dev;
  DevFacts* df;
  if ((st = device_facts(&dev, &df)) != SEER_OK) return st;
  seer::KcompParams p;
  rope_thetas(dims, p.theta);
  p.k = plain(k_nope);
  p.seqlens = seqlens;
  p.valid = valid_blocks;
  p.valid_out = valid_blocks;
  p.w_k = static_cast<const uint16_t*>(w_k);
  p.kcomp = static_cast<uint16_t*>(kcomp);
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.NB = dims->max_blocks;
  p.rope_base = dims->rope_base;
  p.err = nullptr;
  const int units = dims->batch * dims->num_kv_heads;
  int gx = (2 * df->sms + units - 1) / units;
  const int groups = (dims->max_blocks + 7) / 8;
  gx = gx < 1 ? 1 : (gx > groups ? groups : gx);
  cudaError_t e = seer::launch_kcomp_update(p, dims->head_dim, dims->block_size, dims->gate_dim, gx,
                                            static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kcomp_update launch");
  return SEER_OK;
}

size_t seer_prefill_gt_workspace_bytes(const seer_dims_t* dims, int32_t max_len) {
  if (check_dims(dims) != SEER_OK || max_len < 1) return 0;
  return (size_t)dims->batch * dims->num_q_heads * (dims->max_blocks + (size_t)1) * (size_t)max_len * sizeof(float);
}

seer_status seer_prefill_gt(const seer_dims_t* dims, const void* q, int32_t max_len, const seer_kv_t* k,
                            const seer_kv_t* v, const int32_t* seqlens, void* out, float* lse_out, float* gt,
                            void* workspace, size_t workspace_bytes, int32_t* err_word, void* stream) {
  seer_status st = check_dims(dims);
  if (st != SEER_OK) return st;
  if ((st = check_kv(dims, k, "k")) != SEER_OK) return st;
  if ((st = check_kv(dims, v, "v")) != SEER_OK) return st;
  if (k->layout != SEER_KV_CONTIGUOUS || v->layout != SEER_KV_CONTIGUOUS)
    return fail(SEER_ERR_UNSUPPORTED, "prefill attention takes contiguous K/V caches");
  if (!q || !seqlens || !out || !gt || !workspace) return fail(SEER_ERR_INVALID_ARG, "NULL pointer argument");
  if (max_len < 1) return fail(SEER_ERR_INVALID_ARG, "max_len must be >= 1");
  if ((int64_t)dims->max_blocks * dims->block_size < max_len)
    return fail(SEER_ERR_INVALID_ARG, "max_blocks * block_size < max_len");
  if (!aligned16(q) || !aligned16(out) || !aligned16(gt) || !aligned16(workspace) || (lse_out && !aligned16(lse_out)))
    return fail(SEER_ERR_INVALID_ARG, "pointer not 16-byte aligned");
  const size_t need = seer_prefill_gt_workspace_bytes(dims, max_len);
  if (workspace_bytes < need)
    return fail(SEER_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed", workspace_bytes, need);
  int dev;
  DevFacts* df;
  if ((st = device_facts(&dev, &df)) != SEER_OK) return st;
  CUtensorMap tk, tv;
  seer::PrefillParams p{};
  if ((st = tensor_map(dims, k, "k", &tk, p.k_perm)) != SEER_OK) return st;
  if ((st = tensor_map(dims, v, "v", &tv, p.v_perm)) != SEER_OK) return st;
  p.q = static_cast<const uint16_t*>(q);
  p.o = static_cast<uint16_t*>(out);
  p.lse = lse_out;
  p.gt = gt;
  p.rmax = static_cast<float*>(workspace);
  p.rnorm = p.rmax + (size_t)dims->batch * dims->num_q_heads * dims->max_blocks * (size_t)max_len;
  p.seqlens = seqlens;
  p.B = dims->batch;
  p.Hq = dims->num_q_heads;
  p.Hkv = dims->num_kv_heads;
  p.g = dims->num_q_heads / dims->num_kv_heads;
  p.NB = dims->max_blocks;
  p.T = max_len;
  const int64_t cap = k->num_tokens < v->num_tokens ? k->num_tokens : v->num_tokens;
  p.kcap = cap > max_len ? max_len : (int32_t)cap;
  const float scale = dims->softmax_scale > 0.f ? dims->softmax_scale : 1.0f / sqrtf((float)dims->head_dim);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.err = err_word;
  // the tcgen05 / TMEM kernel where it takes the shape, the warp-level mma kernel otherwise
  cudaError_t e = seer::prefill_tc_supported(dims->head_dim, dims->block_size, p.g)
                      ? seer::launch_prefill_tc(tk, tv, p, dims->head_dim, dims->block_size, max_len, df->sms,
                                                static_cast<cudaStream_t>(stream))
                      : seer::launch_prefill_gt(tk, tv, p, dims->head_dim, dims->block_size, max_len,
                                                static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "prefill_gt launch");
  return SEER_OK;
}

size_t seer_kcomp_state_bytes(const seer_dims_t* dims) {
  if (check_dims(dims) != SEER_OK) return 0;
  return (size_t)dims->batch * dims->num_kv_heads * 3 * dims->head_dim * sizeof(float);
}

seer_status seer_kcomp_append(const seer_dims_t* dims, const void* k_new, const int32_t* seqlens, float* state,
                              int32_t* valid_blocks, const void* w_k, void* kcomp, int32_t* err_word,
                              void* stream) {
  seer_status st = check_dims(dims);
  if (st != SEER_OK) return st;
  if (!k_new || !seqlens || !state || !valid_blocks || !w_k || !kcomp)
    return fail(SEER_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned16(k_new) || !aligned16(state) || !aligned16(w_k) || !aligned16(kcomp))
    return fail(SEER_ERR_INVALID_ARG, "k_new / state / w_k / kcomp not 16-byte aligned");
  seer::AppendParams p{};
  rope_thetas(dims, p.theta);
  p.k_new = static_cast<const uint16_t*>(k_new);
  p.seqlens = seqlens;
  p.valid = valid_blocks;
  p.state = state;
  p.w_k = static_cast<const uint16_t*>(w_k);
  p.kcomp = static_cast<uint16_t*>(kcomp);
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.NB = dims->max_blocks;
  p.err = err_word;
  cudaError_t e = seer::launch_kcomp_append(p, dims->head_dim, dims->block_size, dims->gate_dim,
                                            static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kcomp_append launch");
  return SEER_OK;
}

seer_status seer_kcomp_state_init(const seer_dims_t* dims, const seer_kv_t* k_nope, const int32_t* seqlens,
                                  float* state, int32_t* err_word, void* stream) {
  seer_status st = check_dims(dims);
  if (st != SEER_OK) return st;
  if ((st = check_kv(dims, k_nope, "k_nope")) != SEER_OK) return st;
  if (!seqlens || !state) return fail(SEER_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned16(state)) return fail(SEER_ERR_INVALID_ARG, "state not 16-byte aligned");
  seer::AppendParams p{};
  p.k = plain(k_nope);
  p.seqlens = seqlens;
  p.state = state;
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.NB = dims->max_blocks;
  p.err = err_word;
  cudaError_t e = seer::launch_kcomp_state_init(p, dims->head_dim, dims->block_size,
                                                static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kcomp_state_init launch");
  return SEER_OK;
}

seer_status seer_gate_score(const seer_dims_t* dims, const void* q_nope, const void* w_q, const void* kcomp,
                            const int32_t* seqlens, float* logits, float* q_gate_out, void* stream) {
  seer_status st = check_dims(dims);
  if (st != SEER_OK) return st;
  if (!q_nope || !w_q || !kcomp || !seqlens || !logits) return fail(SEER_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned16(q_nope) || !aligned16(w_q) || !aligned16(kcomp) || !aligned16(logits) ||
      (q_gate_out && !aligned16(q_gate_out)))
    return fail(SEER_ERR_INVALID_ARG, "pointer not 16-byte aligned");
  seer::GateParams p;
  rope_thetas(dims, p.theta);
  p.q = static_cast<const uint16_t*>(q_nope);
  p.w_q = static_cast<const uint16_t*>(w_q);
  p.kcomp = static_cast<const uint16_t*>(kcomp);
  p.seqlens = seqlens;
  p.logits = logits;
  p.q_gate = q_gate_out;
  p.B = dims->batch;
  p.Hq = dims->num_q_heads;
  p.Hkv = dims->num_kv_heads;
  p.g = dims->num_q_heads / dims->num_kv_heads;
  p.NB = dims->max_blocks;
  p.BLK = dims->block_size;
  p.rope_base = dims->rope_base;
  cudaError_t e = seer::launch_gate_score(p, dims->head_dim, dims->gate_dim, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gate_score launch");
  return SEER_OK;
}

seer_status seer_select_blocks(const seer_dims_t* dims, const float* logits, const int32_t* seqlens, int32_t mode,
                               int32_t token_budget, float tau, int32_t* block_idx, int32_t* block_cnt,
                               int32_t capacity, void* stream) {
  seer_status st = check_dims(dims);
  if (st != SEER_OK) return st;
  if (!logits || !seqlens || !block_idx || !block_cnt) return fail(SEER_ERR_INVALID_ARG, "NULL pointer argument");
  int32_t kblocks = 0;
  if ((st = select_args(dims, mode, token_budget, tau, capacity, &kblocks)) != SEER_OK) return st;
  seer::SelectParams p;
  p.logits = logits;
  p.seqlens = seqlens;
  p.idx = block_idx;
  p.cnt = block_cnt;
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.NB = dims->max_blocks;
  p.BLK = dims->block_size;
  p.cap = capacity;
  p.mode = mode;
  p.kblocks = kblocks;
  p.tau = (double)tau;
  cudaError_t e = seer::launch_select(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "select_blocks launch");
  return SEER_OK;
}

}  // extern "C"

namespace {

// Argument checks and kernel parameters of seer_decode_plan (shared with seer_decode_step).
seer_status plan_params(const seer_dims_t* dims, const seer_kv_t* k_nope, const int32_t* seqlens,
                        int32_t* valid_blocks, const void* w_k, void* kcomp, const void* q_nope, const void* w_q,
                        float* logits_out, float* q_gate_out, int32_t mode, int32_t token_budget, float tau,
                        int32_t* block_idx, int32_t* block_cnt, int32_t capacity, seer::PlanParams* pp) {
  seer_status st = check_dims(dims);
  if (st != SEER_OK) return st;
  if (!seqlens || !kcomp || !q_nope || !w_q || !block_idx || !block_cnt)
    return fail(SEER_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned16(kcomp) || !aligned16(q_nope) || !aligned16(w_q) || (logits_out && !aligned16(logits_out)) ||
      (q_gate_out && !aligned16(q_gate_out)))
    return fail(SEER_ERR_INVALID_ARG, "pointer not 16-byte aligned");
  const bool update = valid_blocks != nullptr;
  if (update) {
    if ((st = check_kv(dims, k_nope, "k_nope")) != SEER_OK) return st;
    if (!w_k || !aligned16(w_k)) return fail(SEER_ERR_INVALID_ARG, "w_k is NULL or not 16-byte aligned");
  }
  int32_t kblocks = 0;
  if ((st = select_args(dims, mode, token_budget, tau, capacity, &kblocks)) != SEER_OK) return st;
  seer::PlanParams& p = *pp;
  p.update_cache = update;
  rope_thetas(dims, p.k.theta);
  if (update) p.k.k = plain(k_nope);
  else memset(&p.k.k, 0, sizeof(p.k.k));
  p.k.seqlens = seqlens;
  p.k.valid = valid_blocks;
  p.k.valid_out = valid_blocks;
  p.k.w_k = static_cast<const uint16_t*>(w_k);
  p.k.kcomp = static_cast<uint16_t*>(kcomp);
  p.k.B = dims->batch;
  p.k.Hkv = dims->num_kv_heads;
  p.k.NB = dims->max_blocks;
  p.k.rope_base = dims->rope_base;
  p.k.err = nullptr;
  rope_thetas(dims, p.g.theta);
  p.g.q = static_cast<const uint16_t*>(q_nope);
  p.g.w_q = static_cast<const uint16_t*>(w_q);
  p.g.kcomp = static_cast<const uint16_t*>(kcomp);
  p.g.seqlens = seqlens;
  p.g.logits = logits_out;
  p.g.q_gate = q_gate_out;
  p.g.B = dims->batch;
  p.g.Hq = dims->num_q_heads;
  p.g.Hkv = dims->num_kv_heads;
  p.g.g = dims->num_q_heads / dims->num_kv_heads;
  p.g.NB = dims->max_blocks;
  p.g.BLK = dims->block_size;
  p.g.rope_base = dims->rope_base;
  p.s.logits = nullptr;
  p.s.seqlens = seqlens;
  p.s.idx = block_idx;
  p.s.cnt = block_cnt;
  p.s.B = dims->batch;
  p.s.Hkv = dims->num_kv_heads;
  p.s.NB = dims->max_blocks;
  p.s.BLK = dims->block_size;
  p.s.cap = capacity;
  p.s.mode = mode;
  p.s.kblocks = kblocks;
  p.s.tau = (double)tau;
  return SEER_OK;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

extern "C" {

seer_status seer_decode_plan(const seer_dims_t* dims, const seer_kv_t* k_nope, const int32_t* seqlens,
                             int32_t* valid_blocks, const void* w_k, void* kcomp, const void* q_nope,
                             const void* w_q, float* logits_out, float* q_gate_out, int32_t mode,
                             int32_t token_budget, float tau, int32_t* block_idx, int32_t* block_cnt,
                             int32_t capacity, void* stream) {
  seer::PlanParams p;
  const seer_status st = plan_params(dims, k_nope, seqlens, valid_blocks, w_k, kcomp, q_nope, w_q, logits_out,
                                     q_gate_out, mode, token_budget, tau, block_idx, block_cnt, capacity, &p);
  if (st != SEER_OK) return st;
  cudaError_t e = seer::launch_plan(p, dims->head_dim, dims->block_size, dims->gate_dim, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "decode_plan launch");
  return SEER_OK;
}

size_t seer_decode_step_workspace_bytes(const seer_dims_t* dims, int32_t capacity) {
  if (check_dims(dims) != SEER_OK || capacity < 1) return 0;
  return up256((size_t)dims->batch * dims->num_kv_heads * 4) + seer_sparse_decode_workspace_bytes(dims, capacity, -1);
}

int32_t seer_decode_step_supported(const seer_dims_t* dims, int32_t mode, int32_t capacity) {
  if (check_dims(dims) != SEER_OK || capacity < 1) return 0;
  if ((int64_t)dims->batch * dims->num_kv_heads > seer::kMaxDecodeBH) return 0;
  if ((int64_t)dims->batch * dims->num_kv_heads * capacity >= (int64_t)1 << 30) return 0;
  const int bh = dims->batch * dims->num_kv_heads;
  return seer::step_grid(dims->head_dim, dims->block_size, dims->gate_dim, dims->num_q_heads / dims->num_kv_heads,
                         dims->max_blocks, mode, dims->batch, bh) > 0;
}

seer_status seer_decode_step(const seer_dims_t* dims, const seer_kv_t* k_nope, const int32_t* seqlens,
                             int32_t* valid_blocks, const void* w_k, void* kcomp, const void* q_nope,
                             const void* w_q, float* logits_out, float* q_gate_out, int32_t mode,
                             int32_t token_budget, float tau, int32_t* block_idx, int32_t* block_cnt,
                             int32_t capacity, const void* q, const seer_kv_t* k, const seer_kv_t* v,
                             void* workspace, size_t workspace_bytes, void* out, float* lse_out,
                             int32_t* err_word, void* stream) {
  seer::StepParams sp;
  seer_status st = plan_params(dims, k_nope, seqlens, valid_blocks, w_k, kcomp, q_nope, w_q, logits_out, q_gate_out,
                               mode, token_budget, tau, block_idx, block_cnt, capacity, &sp.pl);
  if (st != SEER_OK) return st;
  if (!workspace || !aligned16(workspace)) return fail(SEER_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
  const size_t flags = up256((size_t)dims->batch * dims->num_kv_heads * 4);
  const size_t need = seer_decode_step_workspace_bytes(dims, capacity);
  if (workspace_bytes < need)
    return fail(SEER_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed", workspace_bytes, need);
  const int bh = dims->batch * dims->num_kv_heads;
  const int grid = (int64_t)bh * capacity >= (int64_t)1 << 30
                       ? 0
                       : seer::step_grid(dims->head_dim, dims->block_size, dims->gate_dim,
                                         dims->num_q_heads / dims->num_kv_heads, dims->max_blocks, mode, dims->batch, bh);
  if (grid <= 0)
    return fail(SEER_ERR_UNSUPPORTED, "no fused step for this shape (shared memory or cluster residency); call "
                                      "seer_decode_plan and seer_sparse_decode instead");
  seer::DecodeLaunch L;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  st = seer::prepare_sparse_decode(dims, q, k, v, block_idx, block_cnt, seqlens, capacity, -1, ws + flags,
                                   workspace_bytes - flags, out, lse_out, err_word, &L);
  if (st != SEER_OK) return st;
  if (L.ctas < grid) return fail(SEER_ERR_UNSUPPORTED, "fused step grid %d above the decode's %d", grid, L.ctas);
  sp.d = L.p;
  sp.d.ready = reinterpret_cast<int32_t*>(ws);
  sp.d.starve = 0;   // the debug switch covers the two-launch decode only
  sp.pl.k.err = err_word;
  cudaError_t e = seer::launch_decode_step(L.tk, L.tv, sp, dims->head_dim, dims->block_size, dims->gate_dim, grid,
                                           static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "decode_step launch");
  return SEER_OK;
}

int32_t seer_sparse_decode_auto_split(const seer_dims_t* dims, int32_t capacity) {
  if (check_dims(dims) != SEER_OK || capacity < 1) return 1;
  int dev;
  DevFacts* df;
  if (device_facts(&dev, &df) != SEER_OK) return 1;
  return auto_split(dims, capacity, df);
}

size_t seer_sparse_decode_workspace_bytes(const seer_dims_t* dims, int32_t capacity, int32_t num_split) {
  if (check_dims(dims) != SEER_OK || capacity < 1 || num_split < -1) return 0;
  const int32_t ns = num_split > capacity ? capacity : num_split;
  int ctas = 0;
  if (ns <= 0) {
    int dev;
    DevFacts* df;
    if (device_facts(&dev, &df) != SEER_OK) return 0;
    ctas = flat_grid(dims, df);
  }
  size_t a, b;
  return ws_layout(dims, ns, ctas, &a, &b);
}

}  // extern "C"

namespace seer {

seer_status prepare_sparse_decode(const seer_dims_t* dims, const void* q, const seer_kv_t* k, const seer_kv_t* v,
                                  const int32_t* block_idx, const int32_t* block_cnt, const int32_t* seqlens,
                                  int32_t capacity, int32_t num_split, void* workspace, size_t workspace_bytes,
                                  void* out, float* lse_out, int32_t* err_word, DecodeLaunch* L) {
  seer_status st = check_dims(dims);
  if (st != SEER_OK) return st;
  if ((st = check_kv(dims, k, "k")) != SEER_OK) return st;
  if ((st = check_kv(dims, v, "v")) != SEER_OK) return st;
  if (!q || !block_idx || !block_cnt || !seqlens || !out) return fail(SEER_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned16(q) || !aligned16(out)) return fail(SEER_ERR_INVALID_ARG, "q / out not 16-byte aligned");
  if (capacity < 1) return fail(SEER_ERR_INVALID_ARG, "capacity must be >= 1");
  if (num_split < -1) return fail(SEER_ERR_INVALID_ARG, "num_split must be >= -1");
  int dev;
  DevFacts* df;
  if ((st = device_facts(&dev, &df)) != SEER_OK) return st;
  if (dims->batch > seer::kMaxDecodeB) return fail(SEER_ERR_UNSUPPORTED, "batch %d > %d", dims->batch, seer::kMaxDecodeB);
  int32_t ns = num_split > capacity ? capacity : num_split;
  if (ns <= 0 && dims->batch * dims->num_kv_heads > seer::kMaxDecodeBH)
    return fail(SEER_ERR_UNSUPPORTED, "one-wave schedules need batch*num_kv_heads <= %d; pass num_split >= 1",
                seer::kMaxDecodeBH);
  if (ns <= 0 && (int64_t)dims->batch * dims->num_kv_heads * capacity >= (int64_t)1 << 30)
    return fail(SEER_ERR_UNSUPPORTED, "one-wave schedules need batch*num_kv_heads*capacity < 2^30");
  const int ctas = ns <= 0 ? flat_grid(dims, df) : 0;
  size_t off_lse, off_o;
  const size_t need = ws_layout(dims, ns, ctas, &off_lse, &off_o);
  if (need > 0) {
    if (!workspace) return fail(SEER_ERR_INVALID_ARG, "workspace is NULL (num_split %d needs %zu bytes)", ns, need);
    if (workspace_bytes < need)
      return fail(SEER_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed for num_split %d", workspace_bytes, need, ns);
    if (!aligned16(workspace)) return fail(SEER_ERR_INVALID_ARG, "workspace not 16-byte aligned");
  }
  DecodeParams& p = L->p;
  if ((st = tensor_map(dims, k, "k", &L->tk, p.k_perm)) != SEER_OK) return st;
  if ((st = tensor_map(dims, v, "v", &L->tv, p.v_perm)) != SEER_OK) return st;
  p.q = static_cast<const uint16_t*>(q);
  p.idx = block_idx;
  p.cnt = block_cnt;
  p.seqlens = seqlens;
  p.k_paged = k->layout == SEER_KV_PAGED;
  p.v_paged = v->layout == SEER_KV_PAGED;
  p.k_table = k->block_table;
  p.v_table = v->block_table;
  p.k_maxp = k->max_pages_per_seq;
  p.v_maxp = v->max_pages_per_seq;
  p.k_pages = k->num_pages;
  p.v_pages = v->num_pages;
  p.B = dims->batch;
  p.Hq = dims->num_q_heads;
  p.Hkv = dims->num_kv_heads;
  p.g = dims->num_q_heads / dims->num_kv_heads;
  p.cap = capacity;
  p.flat = ns == 0 ? 1 : (ns == -1 ? 2 : 0);
  p.ns = ns > 0 ? ns : 0;
  p.per_split = ns > 0 ? (capacity + ns - 1) / ns : capacity;
  const float scale = dims->softmax_scale > 0.f ? dims->softmax_scale : 1.0f / sqrtf((float)dims->head_dim);
  p.scale_log2 = scale * 1.4426950408889634f;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.counters = need ? reinterpret_cast<int32_t*>(ws) : nullptr;
  p.lse_part = need ? reinterpret_cast<float*>(ws + off_lse) : nullptr;
  p.o_part = need ? reinterpret_cast<float*>(ws + off_o) : nullptr;
  p.out = static_cast<uint16_t*>(out);
  p.lse_out = lse_out;
  p.err = err_word;
  p.ready = nullptr;
  p.wait_limit = g_wait_limit.load();
  p.starve = (g_debug.load() & SEER_DEBUG_STARVE_COPIES) ? 1 : 0;
  L->D = dims->head_dim;
  L->BLK = dims->block_size;
  L->ctas = ctas;
  L->need = need;
  return SEER_OK;
}

// Capacity schedule with short shares (at most this many list positions per CTA): the grid is cut
// to a whole multiple of the row count, so every row splits at the same points and no CTA carries a
// segment flush in mid-stream (measured: 90 %- and 95 %-sparse rows 1-5 % of the copy peak faster);
// with longer shares every SM's bandwidth counts for more (the 50 %-sparse and dense rows lose 6-9 %
// with the cut).  The workspace stays sized for the full grid.
constexpr int kShortShare = 28;

int decode_grid(const DecodeParams& p, int ctas) {
  const long long bh = (long long)p.B * p.Hkv;
  if (p.flat != 2 || bh > ctas) return ctas;
  const int whole = (int)(ctas / bh * bh);
  return bh * p.cap <= (long long)kShortShare * whole ? whole : ctas;
}

seer_status launch_prepared_decode(const DecodeLaunch& L, cudaStream_t s) {
  cudaError_t e = launch_sparse_decode(L.tk, L.tv, L.p, L.D, L.BLK, decode_grid(L.p, L.ctas), s);
  if (e != cudaSuccess) return cuda_fail(e, "sparse_decode launch");
  return SEER_OK;
}

}  // namespace seer

extern "C" {

seer_status seer_sparse_decode(const seer_dims_t* dims, const void* q, const seer_kv_t* k, const seer_kv_t* v,
                               const int32_t* block_idx, const int32_t* block_cnt, const int32_t* seqlens,
                               int32_t capacity, int32_t num_split, void* workspace, size_t workspace_bytes,
                               void* out, float* lse_out, int32_t* err_word, void* stream) {
  seer::DecodeLaunch L;
  const seer_status st = seer::prepare_sparse_decode(dims, q, k, v, block_idx, block_cnt, seqlens, capacity, num_split,
                                                     workspace, workspace_bytes, out, lse_out, err_word, &L);
  if (st != SEER_OK) return st;
  return seer::launch_prepared_decode(L, static_cast<cudaStream_t>(stream));
}

// ---------------------------------------------------------------- decode ground truth

namespace {
// counters [BH] | per-chunk (max, sum) [BH][nchunk][8][2] | block maxima [BH][NB][8] (8 = the largest group)
size_t truth_layout(const seer_dims_t* d, int* nchunk, size_t* off_part, size_t* off_bmax) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t bh = (size_t)d->batch * d->num_kv_heads;
  const int nc = (d->max_blocks + seer::truth_chunk_blocks() - 1) / seer::truth_chunk_blocks();
  const size_t w = seer::kMaxGroup;
  *nchunk = nc;
  *off_part = up(bh * 4);
  *off_bmax = *off_part + up(bh * nc * w * 2 * 4);
  return *off_bmax + bh * d->max_blocks * w * 4;
}
}  // namespace

size_t seer_gate_truth_workspace_bytes(const seer_dims_t* dims) {
  if (check_dims(dims) != SEER_OK) return 0;
  int nc;
  size_t a, b;
  return truth_layout(dims, &nc, &a, &b);
}

seer_status seer_gate_truth(const seer_dims_t* dims, const void* q, const seer_kv_t* k, const int32_t* seqlens,
                            float* scores, float* log_scores, void* workspace, size_t workspace_bytes,
                            int32_t* err_word, void* stream) {
  seer_status st = check_dims(dims);
  if (st != SEER_OK) return st;
  if ((st = check_kv(dims, k, "k")) != SEER_OK) return st;
  if (!q || !seqlens || !scores || !workspace) return fail(SEER_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned16(q) || !aligned16(scores) || (log_scores && !aligned16(log_scores)) || !aligned16(workspace))
    return fail(SEER_ERR_INVALID_ARG, "pointer not 16-byte aligned");
  int nc;
  size_t off_part, off_bmax;
  const size_t need = truth_layout(dims, &nc, &off_part, &off_bmax);
  if (workspace_bytes < need)
    return fail(SEER_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed", workspace_bytes, need);
  int dev;
  DevFacts* df;
  if ((st = device_facts(&dev, &df)) != SEER_OK) return st;
  CUtensorMap tk;
  seer::TruthParams p;
  if ((st = tensor_map(dims, k, "k", &tk, p.k_perm)) != SEER_OK) return st;
  p.q = static_cast<const uint16_t*>(q);
  p.seqlens = seqlens;
  p.k_paged = k->layout == SEER_KV_PAGED;
  p.k_table = k->block_table;
  p.k_maxp = k->max_pages_per_seq;
  p.k_pages = k->num_pages;
  p.B = dims->batch;
  p.Hq = dims->num_q_heads;
  p.Hkv = dims->num_kv_heads;
  p.g = dims->num_q_heads / dims->num_kv_heads;
  p.NB = dims->max_blocks;
  p.nchunk = nc;
  p.nitems = dims->batch * dims->num_kv_heads * nc;
  const float scale = dims->softmax_scale > 0.f ? dims->softmax_scale : 1.0f / sqrtf((float)dims->head_dim);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.scores = scores;
  p.log_scores = log_scores;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.counters = reinterpret_cast<int32_t*>(ws);
  p.part = reinterpret_cast<float*>(ws + off_part);
  p.bmax = reinterpret_cast<float*>(ws + off_bmax);
  p.err = err_word;
  cudaError_t e = seer::launch_gate_truth(tk, p, dims->head_dim, dims->block_size, df->sms,
                                          static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gate_truth launch");
  return SEER_OK;
}

}  // extern "C"

extern "C" {

// ---------------------------------------------------------------- page tables

namespace {

// The page kernels count in 32 bits and step past the last element by up to a grid's threads (64 x 1024) before they stop.
constexpr int32_t kMaxPageItems = INT32_MAX - (1 << 17) + 1;   // 2^31 - 2^17

seer_status check_pages(int32_t batch, int32_t page_size, int32_t num_pages, int32_t max_pages_per_seq) {
  if (batch < 1 || page_size < 1 || num_pages < 1 || max_pages_per_seq < 1)
    return fail(SEER_ERR_INVALID_ARG, "batch, page_size, num_pages and max_pages_per_seq must be >= 1");
  if (batch > seer::kMaxDecodeB) return fail(SEER_ERR_UNSUPPORTED, "batch %d > %d", batch, seer::kMaxDecodeB);
  if ((int64_t)num_pages * page_size > INT32_MAX)
    return fail(SEER_ERR_UNSUPPORTED, "num_pages * page_size must be below 2^31");
  if (num_pages > kMaxPageItems) return fail(SEER_ERR_UNSUPPORTED, "num_pages %d above 2^31 - 2^17", num_pages);
  return SEER_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

seer_status seer_page_plan(int32_t batch, int32_t page_size, int32_t num_pages, int32_t max_pages_per_seq,
                           int32_t max_tokens, const int32_t* seqlens, const int32_t* new_tokens,
                           int32_t* block_table, const int32_t* free_list, const int32_t* free_count,
                           int32_t* seqlens_out, int32_t* free_count_out, int32_t* cu_tokens, int32_t* slot_map,
                           int32_t* positions, int32_t* err_word, void* stream) {
  seer_status st = check_pages(batch, page_size, num_pages, max_pages_per_seq);
  if (st != SEER_OK) return st;
  if (max_tokens < 1) return fail(SEER_ERR_INVALID_ARG, "max_tokens must be >= 1");
  if (max_tokens > kMaxPageItems) return fail(SEER_ERR_UNSUPPORTED, "max_tokens %d above 2^31 - 2^17", max_tokens);
  const void* const ptrs[] = {seqlens,     new_tokens,     block_table, free_list, free_count,
                              seqlens_out, free_count_out, cu_tokens,   slot_map,  positions};
  for (const void* p : ptrs) {
    if (!p) return fail(SEER_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned4(p)) return fail(SEER_ERR_INVALID_ARG, "pointer not 4-byte aligned");
  }
  seer::PageParams p{};
  p.seqlens = seqlens;
  p.per_request = new_tokens;
  p.block_table = block_table;
  p.free_list = free_list;
  p.free_count = free_count;
  p.seqlens_out = seqlens_out;
  p.free_count_out = free_count_out;
  p.cu_tokens = cu_tokens;
  p.slot_map = slot_map;
  p.positions = positions;
  p.B = batch;
  p.page = page_size;
  p.num_pages = num_pages;
  p.width = max_pages_per_seq;
  p.max_tokens = max_tokens;
  p.err = err_word;
  cudaError_t e = seer::launch_page_plan(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "page_plan launch");
  return SEER_OK;
}

seer_status seer_page_release(int32_t batch, int32_t page_size, int32_t num_pages, int32_t max_pages_per_seq,
                              const int32_t* seqlens, const int32_t* finished, const int32_t* block_table,
                              int32_t* free_list, const int32_t* free_count, int32_t* seqlens_out,
                              int32_t* free_count_out, int32_t* err_word, void* stream) {
  seer_status st = check_pages(batch, page_size, num_pages, max_pages_per_seq);
  if (st != SEER_OK) return st;
  const void* const ptrs[] = {seqlens, finished, block_table, free_list, free_count, seqlens_out, free_count_out};
  for (const void* p : ptrs) {
    if (!p) return fail(SEER_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned4(p)) return fail(SEER_ERR_INVALID_ARG, "pointer not 4-byte aligned");
  }
  seer::PageParams p{};
  p.seqlens = seqlens;
  p.per_request = finished;
  p.block_table = const_cast<int32_t*>(block_table);   // read only by the release kernel
  p.free_out = free_list;
  p.free_count = free_count;
  p.seqlens_out = seqlens_out;
  p.free_count_out = free_count_out;
  p.B = batch;
  p.page = page_size;
  p.num_pages = num_pages;
  p.width = max_pages_per_seq;
  p.err = err_word;
  cudaError_t e = seer::launch_page_release(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "page_release launch");
  return SEER_OK;
}

// ---------------------------------------------------------------- per-head norm + rotation

namespace {


seer_status check_qk(const seer_qk_t* s) {
  if (!s) return fail(SEER_ERR_INVALID_ARG, "shape is NULL");
  if (s->num_tokens < 0 || s->num_q_heads < 1 || s->num_kv_heads < 1)
    return fail(SEER_ERR_INVALID_ARG, "num_tokens must be >= 0, num_q_heads and num_kv_heads >= 1");
  if (s->num_q_heads > 65536 || s->num_kv_heads > 65536) return fail(SEER_ERR_UNSUPPORTED, "more than 65536 heads");
  if ((int64_t)s->num_tokens * (s->num_q_heads + 2 * s->num_kv_heads) >= (int64_t)1 << 31)
    return fail(SEER_ERR_UNSUPPORTED, "num_tokens * (num_q_heads + 2 * num_kv_heads) must be below 2^31");
  if (s->head_dim != 64 && s->head_dim != 128)
    return fail(SEER_ERR_UNSUPPORTED, "head_dim %d not in {64, 128}", s->head_dim);
  if (s->rope_dim < 0 || s->rope_dim > s->head_dim || s->rope_dim % 16)
    return fail(SEER_ERR_UNSUPPORTED, "rope_dim %d is not a multiple of 16 in [0, head_dim]", s->rope_dim);
  if (s->dtype != SEER_BF16 && s->dtype != SEER_FP16 && s->dtype != SEER_FP32)
    return fail(SEER_ERR_UNSUPPORTED, "dtype %d unknown", s->dtype);
  if (!(s->rope_base > 0.f) || !isfinite(s->rope_base)) return fail(SEER_ERR_INVALID_ARG, "rope_base must be > 0");
  if (!(s->eps >= 0.f) || !isfinite(s->eps)) return fail(SEER_ERR_INVALID_ARG, "eps must be >= 0");
  return SEER_OK;
}

bool has(const seer_rows_t* r) { return r && r->data; }

// Rows (or a pool's strides) that the kernel reads or writes 16 bytes at a time.
seer_status check_rows(const seer_qk_t* s, const seer_rows_t* r, const char* name, seer::Rows* out) {
  *out = seer::Rows{};
  if (!has(r)) return SEER_OK;
  const int64_t unit = s->dtype == SEER_FP32 ? 4 : 8;
  if (!aligned16(r->data)) return fail(SEER_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  if (r->stride_t < 0 || r->stride_h < 0 || r->stride_t % unit || r->stride_h % unit)
    return fail(SEER_ERR_INVALID_ARG, "%s strides (t=%lld h=%lld) must be non-negative multiples of 16 bytes", name,
                (long long)r->stride_t, (long long)r->stride_h);
  out->data = r->data;
  out->stride_t = r->stride_t;
  out->stride_h = r->stride_h;
  return SEER_OK;
}

// Rows that are written: distinct (t, h) must be distinct memory.
seer_status check_written(const seer_qk_t* s, const seer_rows_t* r, int heads, const char* name, seer::Rows* out) {
  const seer_status st = check_rows(s, r, name, out);
  if (st != SEER_OK || !has(r)) return st;
  const int64_t T = s->num_tokens, D = s->head_dim;
  const bool token_major = (heads == 1 || r->stride_h >= D) && (T <= 1 || r->stride_t >= (heads - 1) * r->stride_h + D);
  const bool head_major = (T <= 1 || r->stride_t >= D) && (heads == 1 || r->stride_h >= (T - 1) * r->stride_t + D);
  if (T > 0 && !token_major && !head_major)
    return fail(SEER_ERR_INVALID_ARG, "%s is written but its rows overlap (strides t=%lld h=%lld)", name,
                (long long)r->stride_t, (long long)r->stride_h);
  return SEER_OK;
}

seer_status check_pool(const seer_qk_t* s, const seer_pool_t* c, const char* name, seer::Pool* out) {
  *out = seer::Pool{};
  if (!c || !c->data) return SEER_OK;
  if (s->dtype == SEER_FP32) return fail(SEER_ERR_UNSUPPORTED, "%s: caches are bf16 or fp16", name);
  if (!aligned16(c->data)) return fail(SEER_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  if (c->stride_page < 1 || c->stride_h < 1 || c->stride_t < s->head_dim || c->stride_page % 8 || c->stride_h % 8 ||
      c->stride_t % 8)
    return fail(SEER_ERR_INVALID_ARG, "%s strides must be positive multiples of 8 elements, stride_t >= head_dim", name);
  if (c->num_pages < 1 || c->page_size < 1) return fail(SEER_ERR_INVALID_ARG, "%s num_pages and page_size must be >= 1", name);
  if (c->num_pages > INT32_MAX / c->page_size)
    return fail(SEER_ERR_UNSUPPORTED, "%s num_pages * page_size must be below 2^31", name);
  out->data = c->data;
  out->stride_page = c->stride_page;
  out->stride_h = c->stride_h;
  out->stride_t = c->stride_t;
  return SEER_OK;
}

// Frequencies of (base, rope_dim) in turns per position; the thread's last set is kept, since 64 powers cost
// more than the launch.
void rope_frequencies(float base, int rope_dim, double* turns) {
  static thread_local struct {
    float base = 0.f;
    int dim = 0;
    double turns[seer::kMaxHalfGate];
  } last;
  constexpr double kTwoPi = 6.283185307179586;
  if (last.base != base || last.dim != rope_dim) {
    for (int i = 0; i < rope_dim / 2; ++i) last.turns[i] = pow((double)base, -2.0 * i / rope_dim) / kTwoPi;
    last.base = base;
    last.dim = rope_dim;
  }
  memcpy(turns, last.turns, rope_dim / 2 * sizeof(double));
}

void norm_common(const seer_qk_t* s, seer::NormParams* p) {
  rope_frequencies(s->rope_base, s->rope_dim, p->turns);
  p->T = s->num_tokens;
  p->rope_dim = s->rope_dim;
  p->eps = s->eps;
  p->kind[0].heads = s->num_q_heads;
  p->kind[1].heads = p->kind[2].heads = s->num_kv_heads;
}

}  // namespace

seer_status seer_qk_norm_rope(const seer_qk_t* shape, const seer_rows_t* q, const seer_rows_t* k,
                              const seer_rows_t* v, const void* q_weight, const void* k_weight,
                              const int32_t* positions, const seer_rows_t* q_out, const seer_rows_t* k_out,
                              const seer_rows_t* q_nope, const seer_rows_t* k_nope, const seer_pool_t* k_cache,
                              const seer_pool_t* v_cache, const int32_t* slot_map, const int32_t* live_tokens,
                              int32_t* err_word, void* stream) {
  seer_status st = check_qk(shape);
  if (st != SEER_OK) return st;
  if (shape->num_tokens == 0) return SEER_OK;
  seer::NormParams p{};
  norm_common(shape, &p);
  const int Hq = shape->num_q_heads, H = shape->num_kv_heads;
  if ((st = check_rows(shape, q, "q", &p.kind[0].x)) != SEER_OK) return st;
  if ((st = check_rows(shape, k, "k", &p.kind[1].x)) != SEER_OK) return st;
  if ((st = check_rows(shape, v, "v", &p.kind[2].x)) != SEER_OK) return st;
  if ((st = check_written(shape, q_out, Hq, "q_out", &p.kind[0].out)) != SEER_OK) return st;
  if ((st = check_written(shape, k_out, H, "k_out", &p.kind[1].out)) != SEER_OK) return st;
  if ((st = check_written(shape, q_nope, Hq, "q_nope", &p.kind[0].nope)) != SEER_OK) return st;
  if ((st = check_written(shape, k_nope, H, "k_nope", &p.kind[1].nope)) != SEER_OK) return st;
  if ((st = check_pool(shape, k_cache, "k_cache", &p.kind[1].cache)) != SEER_OK) return st;
  if ((st = check_pool(shape, v_cache, "v_cache", &p.kind[2].cache)) != SEER_OK) return st;
  p.kind[0].used = has(q_out) || has(q_nope);
  p.kind[1].used = has(k_out) || has(k_nope) || p.kind[1].cache.data;
  p.kind[2].used = p.kind[2].cache.data != nullptr;
  if (!p.kind[0].used && !p.kind[1].used && !p.kind[2].used) return fail(SEER_ERR_INVALID_ARG, "no output");
  const char* const names[3] = {"q", "k", "v"};
  for (int i = 0; i < 3; ++i)
    if (p.kind[i].used && !p.kind[i].x.data) return fail(SEER_ERR_INVALID_ARG, "%s is NULL but an output of it is not", names[i]);
  const void* const outs[] = {p.kind[0].out.data, p.kind[1].out.data, p.kind[0].nope.data, p.kind[1].nope.data,
                              p.kind[1].cache.data, p.kind[2].cache.data};
  for (int i = 0; i < 6; ++i)
    for (int j = 0; j < i; ++j)
      if (outs[i] && outs[i] == outs[j]) return fail(SEER_ERR_INVALID_ARG, "two outputs share their memory");
  if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight)))
    return fail(SEER_ERR_INVALID_ARG, "norm weight not 16-byte aligned");
  p.kind[0].weight = q_weight;
  p.kind[1].weight = k_weight;
  if (shape->rope_dim > 0 && !positions) return fail(SEER_ERR_INVALID_ARG, "positions is NULL");
  if (p.kind[1].cache.data || p.kind[2].cache.data) {
    if (!slot_map) return fail(SEER_ERR_INVALID_ARG, "slot_map is NULL but a cache is given");
    const seer_pool_t* a = p.kind[1].cache.data ? k_cache : v_cache;
    const seer_pool_t* b = p.kind[2].cache.data ? v_cache : k_cache;
    if (a->page_size != b->page_size || a->num_pages != b->num_pages)
      return fail(SEER_ERR_INVALID_ARG, "k_cache and v_cache differ in page_size or num_pages");
    p.page_size = a->page_size;
    p.slots = (int32_t)(a->num_pages * a->page_size);
  }
  p.positions = positions;
  p.slot_map = slot_map;
  p.live = live_tokens;
  p.err = err_word;
  int dev;
  DevFacts* df;
  if ((st = device_facts(&dev, &df)) != SEER_OK) return st;
  cudaError_t e = seer::launch_norm_rope(p, shape->head_dim, shape->dtype, df->sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "qk_norm_rope launch");
  return SEER_OK;
}

size_t seer_qk_norm_rope_workspace_bytes(int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return (size_t)seer::kNormPartials * head_dim * sizeof(float);
}

seer_status seer_qk_norm_rope_backward(const seer_qk_t* shape, const seer_rows_t* dq_out, const seer_rows_t* dk_out,
                                       const seer_rows_t* dq_nope, const seer_rows_t* dk_nope, const seer_rows_t* q,
                                       const seer_rows_t* k, const void* q_weight, const void* k_weight,
                                       const int32_t* positions, const seer_rows_t* dq, const seer_rows_t* dk,
                                       float* dq_weight, float* dk_weight, const int32_t* live_tokens,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  seer_status st = check_qk(shape);
  if (st != SEER_OK) return st;
  if (shape->num_tokens == 0) {   // no rows: the weight gradients are zero
    for (float* dw : {dq_weight, dk_weight}) {
      if (!dw) continue;
      cudaError_t e = cudaMemsetAsync(dw, 0, shape->head_dim * sizeof(float), static_cast<cudaStream_t>(stream));
      if (e != cudaSuccess) return cuda_fail(e, "qk_norm_rope_backward memset");
    }
    return SEER_OK;
  }
  seer::NormParams p{};
  norm_common(shape, &p);
  struct Side {
    const seer_rows_t *z, *y, *x, *dx;
    const void* w;
    float* dw;
    const char* names[4];
  };
  const Side sides[2] = {{dq_out, dq_nope, q, dq, q_weight, dq_weight, {"dq_out", "dq_nope", "q", "dq"}},
                         {dk_out, dk_nope, k, dk, k_weight, dk_weight, {"dk_out", "dk_nope", "k", "dk"}}};
  for (int i = 0; i < 2; ++i) {
    const Side& s = sides[i];
    seer::NormKind& kd = p.kind[i];
    if ((st = check_rows(shape, s.z, s.names[0], &kd.out)) != SEER_OK) return st;
    if ((st = check_rows(shape, s.y, s.names[1], &kd.nope)) != SEER_OK) return st;
    if ((st = check_rows(shape, s.x, s.names[2], &kd.x)) != SEER_OK) return st;
    if ((st = check_written(shape, s.dx, kd.heads, s.names[3], &kd.dx)) != SEER_OK) return st;
    kd.used = kd.dx.data != nullptr;
    if (!kd.used) {
      if (s.w || s.dw) return fail(SEER_ERR_INVALID_ARG, "%s is NULL but its norm weight or gradient is not", s.names[3]);
      continue;
    }
    if (!kd.out.data && !kd.nope.data)
      return fail(SEER_ERR_INVALID_ARG, "%s needs %s or %s", s.names[3], s.names[0], s.names[1]);
    if (s.w && !kd.x.data) return fail(SEER_ERR_INVALID_ARG, "%s is NULL", s.names[2]);
    if (!s.w != !s.dw) return fail(SEER_ERR_INVALID_ARG, "a norm weight and its gradient go together");
    if (s.w && !aligned16(s.w)) return fail(SEER_ERR_INVALID_ARG, "norm weight not 16-byte aligned");
    if (s.dw && !aligned4(s.dw)) return fail(SEER_ERR_INVALID_ARG, "weight gradient not 4-byte aligned");
    kd.weight = s.w;
    kd.dw = s.dw;
    if (shape->rope_dim > 0 && kd.out.data && !positions) return fail(SEER_ERR_INVALID_ARG, "positions is NULL");
  }
  if (!p.kind[0].used && !p.kind[1].used) return fail(SEER_ERR_INVALID_ARG, "no output");
  if (p.kind[0].dx.data == p.kind[1].dx.data || (dq_weight && dq_weight == dk_weight))
    return fail(SEER_ERR_INVALID_ARG, "two outputs share their memory");
  if (dq_weight || dk_weight) {
    const size_t need = seer_qk_norm_rope_workspace_bytes(shape->head_dim);
    if (!workspace || !aligned16(workspace)) return fail(SEER_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
    if (workspace_bytes < need)
      return fail(SEER_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed", workspace_bytes, need);
  }
  p.positions = positions;
  p.live = live_tokens;
  p.partial = static_cast<float*>(workspace);
  int dev;
  DevFacts* df;
  if ((st = device_facts(&dev, &df)) != SEER_OK) return st;
  cudaError_t e =
      seer::launch_norm_rope_backward(p, shape->head_dim, shape->dtype, df->sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "qk_norm_rope_backward launch");
  return SEER_OK;
}

// ---------------------------------------------------------------- dense one-token attention

namespace {

seer_status check_dense(const seer_dense_t* s) {
  if (!s) return fail(SEER_ERR_INVALID_ARG, "shape is NULL");
  if (s->batch < 1 || s->num_q_heads < 1 || s->num_kv_heads < 1)
    return fail(SEER_ERR_INVALID_ARG, "batch, num_q_heads and num_kv_heads must be >= 1");
  if (s->num_q_heads % s->num_kv_heads != 0)
    return fail(SEER_ERR_INVALID_ARG, "num_q_heads (%d) is not a multiple of num_kv_heads (%d)", s->num_q_heads,
                s->num_kv_heads);
  if (s->num_q_heads / s->num_kv_heads > seer::kDenseMaxGroup)
    return fail(SEER_ERR_UNSUPPORTED, "group size %d > %d", s->num_q_heads / s->num_kv_heads, seer::kDenseMaxGroup);
  if (s->head_dim != 64 && s->head_dim != 128)
    return fail(SEER_ERR_UNSUPPORTED, "head_dim %d not in {64, 128}", s->head_dim);
  if (s->dtype != SEER_BF16 && s->dtype != SEER_FP16) return fail(SEER_ERR_UNSUPPORTED, "dtype %d not bf16 or fp16", s->dtype);
  if (s->batch > seer::kMaxDecodeB) return fail(SEER_ERR_UNSUPPORTED, "batch %d > %d", s->batch, seer::kMaxDecodeB);
  if ((int64_t)s->batch * s->num_kv_heads >= (int64_t)1 << 24)
    return fail(SEER_ERR_UNSUPPORTED, "batch * num_kv_heads must be below 2^24");
  if (s->window < 0) return fail(SEER_ERR_INVALID_ARG, "window must be >= 0 (0 = all tokens)");
  if (!(s->softmax_scale >= 0.f) || !isfinite(s->softmax_scale))
    return fail(SEER_ERR_INVALID_ARG, "softmax_scale must be >= 0 (0 = 1/sqrt(head_dim))");
  return SEER_OK;
}

// join entries | {m, l} of the pieces | outputs of the pieces (two pieces a range: its first and last sequence)
size_t dense_layout(const seer_dense_t* s, int ctas, size_t* off_ml, size_t* off_o) {
  const size_t ranges = seer::dense_ranges(ctas);
  const size_t tiles = s->num_q_heads / s->num_kv_heads > 8 ? 2 : 1;   // of eight heads
  *off_ml = up256(ranges * sizeof(int4));
  *off_o = *off_ml + up256(2 * ranges * tiles * 4 * sizeof(float4));
  return *off_o + 2 * ranges * tiles * 8 * s->head_dim * sizeof(float);
}

// Tokens a sequence can have in the cache.
int64_t kv_capacity(const seer_dense_t* s, const seer_kv_t* kv) {
  return kv->layout == SEER_KV_PAGED ? (int64_t)kv->max_pages_per_seq * s->page_size : kv->num_tokens;
}

}  // namespace

size_t seer_dense_decode_workspace_bytes(const seer_dense_t* shape) {
  if (check_dense(shape) != SEER_OK) return 0;
  int dev;
  DevFacts* df;
  if (device_facts(&dev, &df) != SEER_OK) return 0;
  size_t a, b;
  return dense_layout(shape, df->sms, &a, &b);
}

seer_status seer_dense_decode(const seer_dense_t* shape, const void* q, const seer_kv_t* k, const seer_kv_t* v,
                              const int32_t* seqlens, void* out, float* lse_out, void* workspace,
                              size_t workspace_bytes, int32_t* err_word, void* stream) {
  seer_status st = check_dense(shape);
  if (st != SEER_OK) return st;
  seer_dims_t dims{};   // of check_kv: the row width is all it looks at
  dims.head_dim = shape->head_dim;
  if ((st = check_kv(&dims, k, "k")) != SEER_OK) return st;
  if ((st = check_kv(&dims, v, "v")) != SEER_OK) return st;
  if (!q || !seqlens || !out || !workspace) return fail(SEER_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || !aligned4(lse_out))
    return fail(SEER_ERR_INVALID_ARG, "pointer not aligned (16 bytes; lse 4 bytes)");
  const bool paged = k->layout == SEER_KV_PAGED || v->layout == SEER_KV_PAGED;
  if (paged && shape->page_size < 1) return fail(SEER_ERR_INVALID_ARG, "page_size must be >= 1");
  const int64_t cap = std::min(kv_capacity(shape, k), kv_capacity(shape, v));
  if (cap >= (int64_t)1 << 30 || cap / 32 + 8 >= ((int64_t)1 << 30) / shape->batch / shape->num_kv_heads)
    return fail(SEER_ERR_UNSUPPORTED, "cache capacity and batch * num_kv_heads * (capacity / 32 + 8) must be below 2^30");
  int dev;
  DevFacts* df;
  if ((st = device_facts(&dev, &df)) != SEER_OK) return st;
  size_t off_ml, off_o;
  const size_t need = dense_layout(shape, df->sms, &off_ml, &off_o);
  if (workspace_bytes < need)
    return fail(SEER_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed", workspace_bytes, need);
  seer::DenseParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse_out;
  p.k = plain(k);
  p.v = plain(v);
  p.seqlens = seqlens;
  p.B = shape->batch;
  p.Hq = shape->num_q_heads;
  p.Hkv = shape->num_kv_heads;
  p.g = shape->num_q_heads / shape->num_kv_heads;
  p.window = shape->window;
  p.page = paged ? shape->page_size : 1;
  p.by_page = seer::divisor(p.page);
  p.cap = (int32_t)cap;
  const float scale = shape->softmax_scale > 0.f ? shape->softmax_scale : 1.0f / sqrtf((float)shape->head_dim);
  p.scale_log2 = scale * 1.4426950408889634f;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.join = reinterpret_cast<int4*>(ws);
  p.ml_part = reinterpret_cast<float4*>(ws + off_ml);
  p.o_part = reinterpret_cast<float4*>(ws + off_o);
  p.err = err_word;
  cudaError_t e = seer::launch_dense_decode(p, shape->head_dim, shape->dtype, df->sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dense_decode launch");
  return SEER_OK;
}

}  // extern "C"
