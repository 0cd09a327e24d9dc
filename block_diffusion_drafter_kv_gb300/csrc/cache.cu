// C ABI of the target's paged cache (declared in include/dflash.h): the handle, its argument
// checks, workspace layout and tensor maps. The kernels are in append.cu and paged_attn.cu.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "dflash.h"
#include "internal.h"
#include "target.h"

using namespace dfl;

namespace {

size_t up256(size_t v) { return (v + 255) / 256 * 256; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct CacheLayout {
  size_t err, prefix, part, total;
};

CacheLayout layout_of(const dflash_cache_config& c) {
  CacheLayout L{};
  L.err = 0;
  L.prefix = 256;
  L.part = L.prefix + up256((std::min<size_t>(c.max_batch, kAttnMaxBatch) + 1) * 4);
  const size_t rows = paged_attn_rows(c.n_heads / c.n_kv_heads * c.max_block);
  L.total = L.part + up256(2 * kPagedMaxCtas * rows * (c.head_dim + 2) * 4);
  return L;
}

// One layer's pool [rows][nkv][d]: boxes of 64 positions x 1 head x 64 dims (128 bytes).
bool encode(PFN_cuTensorMapEncodeTiled_v12000 fn, CUtensorMap* m, void* base, const dflash_cache_config& c) {
  const cuuint64_t d = c.head_dim, nkv = c.n_kv_heads;
  const cuuint64_t dims[3] = {d, nkv, static_cast<cuuint64_t>(c.n_pages) * kPagePos};
  const cuuint64_t strides[2] = {d * 2, nkv * d * 2};
  const cuuint32_t box[3] = {64, 1, kPagePos};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(m, c.dtype == DFLASH_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims,
            strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

struct dflash_cache {
  dflash_cache_config cfg{};
  int device = 0;
  int n_sms = 0;
  bool bound = false;
  uint8_t* k_pool = nullptr;
  uint8_t* v_pool = nullptr;
  const int* page_table = nullptr;
  int* len = nullptr;
  const float* rope_cos = nullptr;
  const float* rope_sin = nullptr;
  uint8_t* ws = nullptr;
  CacheLayout L{};
  std::vector<CUtensorMap> kmap, vmap;

  size_t layer_bytes() const {
    return static_cast<size_t>(cfg.n_pages) * kPagePos * cfg.n_kv_heads * cfg.head_dim * 2;
  }
  int* err() const { return reinterpret_cast<int*>(ws + L.err); }
};

extern "C" {

int dflash_cache_config_check(const dflash_cache_config* c) {
  if (!c) return DFLASH_E_INVAL;
  const bool ok =
      c->n_layers >= 1 && c->n_layers <= 1024 && c->n_kv_heads >= 1 && c->n_kv_heads <= 1024 && c->n_heads >= c->n_kv_heads &&
      c->n_heads % c->n_kv_heads == 0 && c->max_block >= 1 && c->max_block <= 16 &&
      static_cast<long long>(c->n_heads / c->n_kv_heads) * c->max_block <= 128 && (c->head_dim == 64 || c->head_dim == 128) &&
      (c->dtype == DFLASH_F16 || c->dtype == DFLASH_BF16) && c->n_pages >= 1 &&
      static_cast<long long>(c->n_pages) * kPagePos < (1LL << 31) && c->pages_per_seq >= 1 &&
      static_cast<long long>(c->pages_per_seq) * kPagePos < (1LL << 31) && c->max_batch >= 1 &&
      c->max_batch <= kMaxBatch && static_cast<long long>(c->max_batch) * c->pages_per_seq < (1LL << 31) &&
      c->rope_dim >= 0 && c->rope_dim <= c->head_dim && c->rope_dim % 16 == 0 &&
      (c->rope_interleaved == 0 || c->rope_interleaved == 1) && (c->rope_dim == 0 || c->rope_positions >= 1) &&
      c->scale >= 0.f && c->scale <= 1e38f;
  return ok ? DFLASH_OK : DFLASH_E_CONFIG;
}

size_t dflash_cache_workspace_size(const dflash_cache_config* c) {
  return dflash_cache_config_check(c) == DFLASH_OK ? layout_of(*c).total : 0;
}

int dflash_cache_create(const dflash_cache_config* cfg, dflash_cache** out) {
  if (!cfg || !out) return DFLASH_E_INVAL;
  if (const int r = dflash_cache_config_check(cfg)) return r;
  dflash_cache* c = new (std::nothrow) dflash_cache();
  if (!c) return DFLASH_E_CAPACITY;
  c->cfg = *cfg;
  if (c->cfg.scale == 0.f) c->cfg.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(cfg->head_dim)));
  try {
    c->kmap.resize(cfg->n_layers);
    c->vmap.resize(cfg->n_layers);
  } catch (const std::bad_alloc&) {
    delete c;
    return DFLASH_E_CAPACITY;
  }
  if (cudaGetDevice(&c->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&c->n_sms, cudaDevAttrMultiProcessorCount, c->device) != cudaSuccess ||
      paged_attn_set_attributes() != 0) {
    delete c;
    return DFLASH_E_CUDA;
  }
  *out = c;
  return DFLASH_OK;
}

int dflash_cache_destroy(dflash_cache* c) {
  if (!c) return DFLASH_E_INVAL;
  delete c;
  return DFLASH_OK;
}

int dflash_cache_bind(dflash_cache* c, void* k_pool, void* v_pool, const int32_t* page_table, int32_t* len,
                      const float* rope_cos, const float* rope_sin, void* workspace, size_t workspace_bytes) {
  if (!c || !k_pool || !v_pool || !page_table || !len || !workspace) return DFLASH_E_INVAL;
  if (c->cfg.rope_dim > 0 && (!rope_cos || !rope_sin)) return DFLASH_E_INVAL;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(page_table, 4) || !aligned(len, 4) || !aligned(rope_cos, 16) ||
      !aligned(rope_sin, 16) || !aligned(workspace, 256))
    return DFLASH_E_INVAL;
  const CacheLayout L = layout_of(c->cfg);
  if (workspace_bytes < L.total) return DFLASH_E_CAPACITY;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return DFLASH_E_CUDA;
  const auto encoder = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  const DeviceGuard on(c->device);
  if (!on.ok()) return DFLASH_E_CUDA;
  c->bound = false;
  c->k_pool = static_cast<uint8_t*>(k_pool);
  c->v_pool = static_cast<uint8_t*>(v_pool);
  for (int l = 0; l < c->cfg.n_layers; ++l)
    if (!encode(encoder, &c->kmap[l], c->k_pool + l * c->layer_bytes(), c->cfg) ||
        !encode(encoder, &c->vmap[l], c->v_pool + l * c->layer_bytes(), c->cfg))
      return DFLASH_E_CUDA;
  if (cudaMemset(workspace, 0, L.total) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return DFLASH_E_CUDA;
  c->page_table = page_table;
  c->len = len;
  c->rope_cos = rope_cos;
  c->rope_sin = rope_sin;
  c->ws = static_cast<uint8_t*>(workspace);
  c->L = L;
  c->bound = true;
  return DFLASH_OK;
}

int dflash_cache_append(dflash_cache* c, int32_t layer, const void* q, const void* k, const void* v, int32_t x_dtype,
                        int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t* slots, int32_t batch,
                        int32_t rows_per_seq, void* q_out, void* stream) {
  if (!c) return DFLASH_E_INVAL;
  if (!c->bound) return DFLASH_E_STATE;
  const auto& f = c->cfg;
  if (layer < 0 || layer >= f.n_layers || !k || !v || !slots || !q != !q_out || batch < 1 || rows_per_seq < 1)
    return DFLASH_E_INVAL;
  if (x_dtype != DFLASH_F16 && x_dtype != DFLASH_BF16) return DFLASH_E_INVAL;
  // rows are read 16 bytes at a time, and must not overlap one another
  const int64_t kv = static_cast<int64_t>(f.n_kv_heads) * f.head_dim, qd = static_cast<int64_t>(f.n_heads) * f.head_dim;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(slots, 4) ||
      (q && (q_stride < qd || q_stride % 8)) || k_stride < kv || k_stride % 8 || v_stride < kv || v_stride % 8)
    return DFLASH_E_INVAL;
  const long long rows = static_cast<long long>(batch) * rows_per_seq;
  if (batch > f.max_batch || rows >= (1LL << 31)) return DFLASH_E_CAPACITY;
  const DeviceGuard on(c->device);
  if (!on.ok()) return DFLASH_E_CUDA;
  AppendParams P{};
  P.q = q;
  P.k = k;
  P.v = v;
  P.q_stride = q_stride;
  P.k_stride = k_stride;
  P.v_stride = v_stride;
  P.slots = slots;
  P.len = c->len;
  P.cos = c->rope_cos;
  P.sin = c->rope_sin;
  P.q_out = q_out;
  P.k_pool = c->k_pool + layer * c->layer_bytes();
  P.v_pool = c->v_pool + layer * c->layer_bytes();
  P.err = c->err();
  P.rows = rows;
  P.rows_per_seq = rows_per_seq;
  P.nq = f.n_heads;
  P.nkv = f.n_kv_heads;
  P.d = f.head_dim;
  P.rope_dim = f.rope_dim;
  P.interleaved = f.rope_interleaved;
  P.positions = f.rope_positions;
  P.pool_rows = f.n_pages * kPagePos;
  return launch_append(P, x_dtype, f.dtype, static_cast<cudaStream_t>(stream)) == 0 ? DFLASH_OK : DFLASH_E_CUDA;
}

int dflash_cache_attend(dflash_cache* c, int32_t layer, const void* q, const int32_t* n_new, int32_t batch,
                        int32_t rows_per_seq, void* out, void* stream) {
  if (!c) return DFLASH_E_INVAL;
  if (!c->bound) return DFLASH_E_STATE;
  const auto& f = c->cfg;
  if (layer < 0 || layer >= f.n_layers || !q || !n_new || !out || batch < 1 || rows_per_seq < 1) return DFLASH_E_INVAL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(n_new, 4)) return DFLASH_E_INVAL;
  if (batch > f.max_batch || rows_per_seq > f.max_block) return DFLASH_E_CAPACITY;
  const DeviceGuard on(c->device);
  if (!on.ok()) return DFLASH_E_CUDA;
  PagedAttnParams P{};
  P.kmap = c->kmap[layer];
  P.vmap = c->vmap[layer];
  P.err = c->err();
  P.prefix = reinterpret_cast<int*>(c->ws + c->L.prefix);
  P.part = reinterpret_cast<float*>(c->ws + c->L.part);
  P.rows_per_seq = rows_per_seq;
  P.nq = f.n_heads;
  P.nkv = f.n_kv_heads;
  P.d = f.head_dim;
  P.n_pages = f.n_pages;
  P.pages_per_seq = f.pages_per_seq;
  P.group = f.n_heads / f.n_kv_heads;
  P.group_inv = 1.f / static_cast<float>(P.group);
  P.rows = P.group * rows_per_seq;
  P.scale_log2 = static_cast<float>(1.4426950408889634 * f.scale);
  P.wait_ns = kDefaultWaitLimitNs;
  const size_t seq_bytes = static_cast<size_t>(rows_per_seq) * f.n_heads * f.head_dim * 2;
  for (int s = 0; s < batch; s += kAttnMaxBatch) {
    P.q = static_cast<const uint8_t*>(q) + s * seq_bytes;
    P.out = static_cast<uint8_t*>(out) + s * seq_bytes;
    P.len = c->len + s;
    P.n_new = n_new + s;
    P.page_table = c->page_table + static_cast<size_t>(s) * f.pages_per_seq;
    P.batch = std::min(batch - s, kAttnMaxBatch);
    if (launch_paged_attn(P, f.dtype == DFLASH_BF16, std::min(c->n_sms, kPagedMaxCtas), static_cast<cudaStream_t>(stream)) != 0)
      return DFLASH_E_CUDA;
  }
  return DFLASH_OK;
}

int dflash_cache_read_error(dflash_cache* c, int32_t* flags, int32_t clear, void* stream) {
  if (!c || !flags) return DFLASH_E_INVAL;
  if (!c->bound) return DFLASH_E_STATE;
  const DeviceGuard on(c->device);
  if (!on.ok()) return DFLASH_E_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t v = 0;
  if (cudaMemcpyAsync(&v, c->err(), 4, cudaMemcpyDeviceToHost, st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
    return DFLASH_E_CUDA;
  *flags = v;
  if (clear && (cudaMemsetAsync(c->err(), 0, 4, st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess))
    return DFLASH_E_CUDA;
  return DFLASH_OK;
}

}  // extern "C"
