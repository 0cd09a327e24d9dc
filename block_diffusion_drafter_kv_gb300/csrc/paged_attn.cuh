// Shared by the two kernels of the attention over a paged cache (mma.sync and tcgen05) and the
// join of their parts: the cut of the list of tiles, softmax states, types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "math.cuh"
#include "ptx.cuh"
#include "target.h"

namespace dfl {

namespace {

constexpr int kKeys = kPagePos;  // keys per tile

// Two values as the cache's 16-bit type, the first in the low half.
template <bool BF16>
DEV uint32_t pack2(float lo, float hi) {
  if (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <bool BF16>
DEV float2 unpack2(uint32_t u) {
  if (BF16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
// Whether one of the two 16-bit values is infinite or NaN.
template <bool BF16>
DEV bool non_finite2(uint32_t u) {
  constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
  return (u & kExp) == kExp || ((u >> 16) & kExp) == kExp;
}

// What a state (max, sum) weighs against the maximum of all of them: nothing where it has seen no
// key, and NaN as it is where all it has seen were NaN.
DEV float weight_of(float2 ml, float top) {
  if (ml.x == -INFINITY) return ml.y == 0.f ? 0.f : 1.f;
  return ex2(ml.x - top);
}

// Sequence s's rows of this call: 0 where its lengths are out of range.
DEV int rows_of(const PagedAttnParams& P, int s, int& len, bool& bad) {
  len = __ldcg(P.len + s);
  const int n = __ldcg(P.n_new + s);
  bad = len < 0 || n < 0 || n > P.rows_per_seq ||
        static_cast<long long>(len) + n > static_cast<long long>(P.pages_per_seq) * kPagePos;
  return bad ? 0 : n;
}

// With up to 32 sequences, one a lane: the tiles per head of those before the lane's, and with its own.
DEV int scan_tiles(int n, int len, int extra, int lane, int& upto) {
  const int mine = n > 0 ? (len + n + kKeys - 1) / kKeys + extra : 0;
  upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  return upto - mine;
}

// The lengths of the call in shared memory, and the tiles per head before each sequence: with more
// sequences each thread a run of them, then a scan over the block's THREADS threads, and CTA 0
// leaves the prefix for the join.
template <int THREADS>
DEV void count_tiles(const PagedAttnParams& P, int* s_pre, int* s_len, int* s_new, int* s_warp) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (P.batch <= 32) {  // a sequence a lane, in every warp for itself: the same values, and no barrier
    int len = 0, upto = 0;
    bool bad = false;
    const int n = lane < P.batch ? rows_of(P, lane, len, bad) : 0;
    if (bad && blockIdx.x == 0 && warp == 0) raise_flag(P.err, kDevCapacity);
    const int before = scan_tiles(n, len, P.extra, lane, upto);
    if (lane < P.batch) {
      s_len[lane] = len;
      s_new[lane] = n;
      s_pre[lane] = before;
    }
    if (lane == P.batch - 1) s_pre[P.batch] = upto;
    __syncwarp();
    return;
  }
  const int per = (P.batch + THREADS - 1) / THREADS;
  const int s0 = min(tid * per, P.batch), s1 = min(s0 + per, P.batch);
  int mine = 0;
  for (int s = s0; s < s1; ++s) {
    int len;
    bool bad;
    const int n = rows_of(P, s, len, bad);
    if (bad && blockIdx.x == 0) raise_flag(P.err, kDevCapacity);
    s_len[s] = len;
    s_new[s] = n;
    s_pre[s + 1] = n > 0 ? (len + n + kKeys - 1) / kKeys + P.extra : 0;
    mine += s_pre[s + 1];
  }
  int v = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  int before = v - mine;
  for (int w = 0; w < warp; ++w) before += s_warp[w];
  for (int s = s0; s < s1; ++s) {
    before += s_pre[s + 1];
    s_pre[s + 1] = before;
  }
  if (tid == 0) s_pre[0] = 0;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int s = tid; s <= P.batch; s += THREADS) P.prefix[s] = s_pre[s];
}

// With a shared prefix the list has the sequences' own positions first (entries 0 .. batch - 1), then the
// prefix once for every pre_rows new rows of the batch. An entry of the prefix is as one whose rows all stand at its
// last position: s_len is that, s_new its new rows (of several sequences).
// entry_tiles: what the list counts of entry e for each head.
DEV int entry_tiles(const PagedAttnParams& P, int e, int before, bool none, int& len, int& n, bool& bad) {
  len = before - 1;
  int keys = before;
  bad = false;
  if (e < P.batch) {
    n = rows_of(P, e, len, bad);
    keys = len + n;
  } else {
    n = min(P.pre_rows, P.batch * P.rows_per_seq - (e - P.batch) * P.pre_rows);
  }
  if (none) n = 0;
  return n > 0 && keys > 0 ? (keys + kKeys - 1) / kKeys + P.extra : 0;
}
DEV bool no_prefix(const PagedAttnParams& P, int before) {
  return before < 0 || before > static_cast<long long>(P.pages_per_seq) * kPagePos;
}
template <int THREADS>
DEV void count_entries(const PagedAttnParams& P, int* s_pre, int* s_len, int* s_new, int* s_warp) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int entries = P.batch + P.n_pre, before = __ldcg(P.prefix_len);
  const bool none = no_prefix(P, before);
  if (none && blockIdx.x == 0 && tid == 0) raise_flag(P.err, kDevCapacity);
  const int per = (entries + THREADS - 1) / THREADS;
  const int e0 = min(tid * per, entries), e1 = min(e0 + per, entries);
  int mine = 0;
  for (int e = e0; e < e1; ++e) {
    int len, n;
    bool bad;
    s_pre[e + 1] = entry_tiles(P, e, before, none, len, n, bad);
    if (bad && blockIdx.x == 0) raise_flag(P.err, kDevCapacity);
    s_len[e] = len;
    s_new[e] = n;
    mine += s_pre[e + 1];
  }
  int v = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  int sum = v - mine;
  for (int w = 0; w < warp; ++w) sum += s_warp[w];
  for (int e = e0; e < e1; ++e) {
    sum += s_pre[e + 1];
    s_pre[e + 1] = sum;
  }
  if (tid == 0) s_pre[0] = 0;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = tid; e <= entries; e += THREADS) P.prefix[e] = s_pre[e];
}
// Of an entry: its first row among the batch's new rows, its pages, and where a row of its outputs goes in `state`.
template <bool SHARED>
DEV int first_row(const PagedAttnParams& P, int e) { return !SHARED || e < P.batch ? e * P.rows_per_seq : (e - P.batch) * P.pre_rows; }
// Whether row `row` of the batch's buffers is one of this call's new rows.
DEV bool row_is_new(const PagedAttnParams& P, const int* s_new, int row) {
  const int s = row / P.rows_per_seq;
  return row - s * P.rows_per_seq < s_new[s];
}
template <bool SHARED>
DEV const int* pages_of(const PagedAttnParams& P, int e) {
  return !SHARED || e < P.batch ? P.page_table + static_cast<size_t>(e) * P.pages_per_seq : P.prefix_table;
}
DEV size_t state_row(const PagedAttnParams& P, int e, int row, int head) {
  return (static_cast<size_t>(e < P.batch ? 0 : P.batch * P.rows_per_seq) + row) * P.nq + head;
}
DEV float2* state_sums(const PagedAttnParams& P) {
  return reinterpret_cast<float2*>(P.state + 2 * static_cast<size_t>(P.batch) * P.rows_per_seq * P.nq * P.d);
}

// How many ranges the list of T tiles is cut into, for n_ctas CTAs of `strands` ranges each: no empty one, and
// no more than one a CTA where they would be shorter than two tiles.
DEV int n_ranges(long long T, int n_ctas, int strands) {
  const long long n = n_ctas;
  return static_cast<int>(min(T, strands == 1 ? n : min(n * strands, max(n, (T + 1) >> 1))));
}

// The new row that row x < 256 of a problem belongs to, x / group: (x + 1/2) / group is 1 / 512 or more
// from the next integers, far more than a product of floats is off.
DEV int new_row(const PagedAttnParams& P, int x) { return static_cast<int>((static_cast<float>(x) + 0.5f) * P.group_inv); }

// List position u: sequence s, KV head g, tile t of the pair's nt (or behind them, where a list counts more).
struct Place {
  int s, g, t, nt;
};
DEV Place locate(const int* s_pre, int batch, int nkv, long long u, int extra = 0) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<long long>(nkv) * s_pre[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  Place p;
  p.s = lo;
  p.nt = s_pre[lo + 1] - s_pre[lo];
  const long long rest = u - static_cast<long long>(nkv) * s_pre[lo];
  p.g = static_cast<int>(quotient(rest, p.nt));
  p.t = static_cast<int>(rest - static_cast<long long>(p.g) * p.nt);
  p.nt -= extra;
  return p;
}

__device__ __noinline__ void wait_long(uint64_t* bar, uint32_t parity, volatile int* abort, int* err, unsigned long long limit_ns) {
  if (*abort) return;
  if (!mbar_wait(bar, parity, limit_ns)) {
    *abort = 1;
    raise_flag(err, kDevTimeout);
  }
}

}  // namespace

}  // namespace dfl
