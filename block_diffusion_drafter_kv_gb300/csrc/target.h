// Internal interfaces of the target-side operators (page pool, rotary append, paged
// attention, log probabilities) between their kernels and the C ABI glue.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dflash.h"

namespace dfl {

constexpr int kPagePos = 64;          // positions per page, and keys per attention tile
constexpr int kMaxBatch = 8192;       // sequences of a pool and of a cache (a pool call keeps five integers each in shared memory)
constexpr int kAttnMaxBatch = 1024;   // sequences of an attention launch (three integers each beside its rings)
constexpr int kMaxExtra = 32;         // PagedAttnParams::extra at most
constexpr int kPagedMaxCtas = 256;    // attention partial slots are sized for this many CTAs
constexpr int kSharedMaxCtas = 320;   // with a shared prefix, of up to two a SM

// Makes a handle's device current for a call, and the caller's again afterwards.
class DeviceGuard {
 public:
  explicit DeviceGuard(int device) {
    ok_ = cudaGetDevice(&before_) == cudaSuccess;
    if (ok_ && before_ != device) ok_ = changed_ = cudaSetDevice(device) == cudaSuccess;
  }
  ~DeviceGuard() {
    if (changed_) cudaSetDevice(before_);
  }
  bool ok() const { return ok_; }

 private:
  int before_ = 0;
  bool ok_ = false, changed_ = false;
};

// ---------------------------------------------------------------- rotary append
struct AppendParams {
  const void* q;  // null: keys and values only
  const void* k;
  const void* v;
  long long q_stride, k_stride, v_stride;  // elements from one row to the next
  const int* slots;
  const int* len;
  const float* cos;  // [positions][rope_dim / 2]
  const float* sin;
  void* q_out;
  void* k_pool;  // this layer's
  void* v_pool;
  uint8_t* scales;        // this layer's, of an 8-bit cache
  const int* prefix_len;  // positions before those that len counts, or null
  int* err;
  long long rows;
  int rows_per_seq, nq, nkv, d, rope_dim, interleaved, positions;
  int pool_rows;
};
// pool_dtype: DFLASH_F16, DFLASH_BF16, or an 8-bit cache's, whose q_out is of the type it names
int launch_append(const AppendParams& p, int x_dtype, int pool_dtype, cudaStream_t stream);

// ---------------------------------------------------------------- rows of the cache, dense
struct ReadParams {
  const uint8_t* k_pool;  // this layer's
  const uint8_t* v_pool;
  const uint8_t* scales;
  const int* page_table;
  const int* first;
  const int* count;
  void* k_out;
  void* v_out;
  int* err;
  int batch, rows_per_seq, nkv, d, n_pages, pages_per_seq;
};
int launch_cache_read(const ReadParams& p, int pool_dtype, int out_dtype, int n_sms, cudaStream_t stream);

// ---------------------------------------------------------------- paged attention
struct PagedAttnParams {
  CUtensorMap kmap;  // this layer's pool: {d, nkv, n_pages * 64}, box {64, 1, 64}, 128-byte swizzle
  CUtensorMap vmap;
  const void* q;     // [batch * rows_per_seq][nq][d]
  void* out;         // the same shape
  const int* len;
  const int* n_new;
  const int* page_table;
  int* err;
  int* prefix;       // [batch + 1] key tiles per head before each sequence, written by the first kernel for the second
  float* part;       // [2 * CTAs] slots of rows * d outputs, then (max, sum) per row
  int batch, rows_per_seq, nq, nkv, d, n_pages, pages_per_seq;
  int rows;          // (nq / nkv) * rows_per_seq
  int group;         // nq / nkv
  float group_inv;   // its inverse
  float scale_log2;  // scale * log2(e)
  unsigned long long wait_ns;
  const uint8_t* k_pool;   // this layer's
  const uint8_t* v_pool;
  const uint8_t* scales;   // of an 8-bit cache
  // A prefix that all sequences share (null: none). The list of tiles then has batch entries for the
  // sequences' own positions and n_pre for the prefix, pre_rows new rows of the batch each.
  const int* prefix_len;
  const int* prefix_table; // its row of the page table
  int n_pre, pre_rows;
  int slot_rows;           // rows of a partial slot
  int strands;             // ranges of the list that a CTA takes
  int extra;               // tiles that the list counts behind each pair for a segment's start and end
  float* state;            // [2: own, prefix][batch * rows_per_seq][nq] rows of d outputs, then of (max, sum)
};
// With a shared prefix: chooses pre_rows, n_pre, slot_rows and strands; at most shared_batch() sequences.
int launch_paged_attn_shared(PagedAttnParams p, int dtype, int n_ctas, cudaStream_t stream);
int launch_shared_join(const PagedAttnParams& p, bool bf16, int n_ctas, cudaStream_t stream);
int shared_batch();
int paged_attn8_rows(int rows);     // as paged_attn_rows, of the kernel for 8-bit caches
int paged_attn8_strands(int rows);  // and its ranges a CTA
int paged_attn8_extra(int rows);    // and what a list counts behind each pair
int paged_attn8_set_attributes();
int launch_paged_attn8(const PagedAttnParams& p, bool bf16, int n_ctas, cudaStream_t stream);
int launch_paged_attn_join(const PagedAttnParams& p, bool bf16, int n_ctas, cudaStream_t stream);
int paged_attn_rows(int rows);  // rows of a partial slot: `rows` rounded up to what a kernel variant holds
int paged_attn_set_attributes();
int launch_paged_attn(const PagedAttnParams& p, bool bf16, int n_ctas, cudaStream_t stream);
// The first kernel's tcgen05 form, for more than 16 rows; called by the above.
int paged_attn_tc_set_attributes();
int launch_paged_attn_tc(const PagedAttnParams& p, bool bf16, int n_ctas, cudaStream_t stream);

// ---------------------------------------------------------------- log probabilities
constexpr int kLpMaxTop = 32;
constexpr int kLpMaxCtas = 512;
constexpr int kLpSlotWords = 68;   // (max, sum, weighted sum, pad) then 32 keys of 64 bits
struct LogprobParams {
  const void* logits;
  long long row_stride;
  const int* tokens;
  float scale;        // log2(e) / temperature
  float inv_temp;     // 1 / temperature
  int V, rows, n_top;
  int units;          // 4 KB units of a row (set by the launcher)
  float* logprob;
  float* entropy;
  int* top_ids;
  float* top_logprobs;
  float* part;        // [2 * kLpMaxCtas][kLpSlotWords]: each CTA's part of its first and of its last row
  int* row_cnt;       // [kLpMaxCtas] arrivals at the row that a CTA ends with, zero between launches
  int* err;
  unsigned long long wait_ns;  // limit of every wait in the kernel
};
int logprob_set_attributes();
int launch_logprobs(LogprobParams p, int dtype, int n_sms, cudaStream_t stream);

}  // namespace dfl
