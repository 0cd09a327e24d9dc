// Log probabilities of given tokens, the entropy of their distributions and the most likely
// alternatives, in one pass over the logits.
//
// With c = log2(e) / T, M = max z, d = c (z - M), S = sum 2^d, W = sum 2^d d:
//   log p(token) = (z_token - M) / T - ln 2 log2 S,  H = ln 2 (log2 S - W / S)
// (M, S, W) of two parts join by rescaling the smaller max's: W' = 2^e (W + e S), e = c (M - M').
// The difference z - M is taken before the scaling: a row of nothing but the type's lowest
// value stays a uniform one.
// The bound is reading the logits. A row is cut into chunks where there are few rows; the
// CTA that arrives last at a row joins its parts in chunk order (no waiting, no dependence
// on timing).
//
// The n_top largest: every warp keeps the best of what it has read as a sorted list of 64-bit
// keys, one per lane, (order-preserving bits of the logit, ~index): ties go to the lowest
// index and all keys differ. What keeps this off the streaming path is a threshold that the
// warps share: each publishes the ceil(n_top / 8)-th largest value it has seen, and the least
// of the eight bounds the n_top-th largest of the CTA from below. It starts from one sort of
// the lane maxima of the first batch, so that a few dozen values of a chunk of thousands
// reach a list. Values come one at a time by insertion, or many at once (sorted inputs, long
// runs of equal values) by sorting and merging 32, so that no order of the logits costs
// more than a small multiple of another.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "target.h"

namespace dfl {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;
using Key = unsigned long long;

DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Order-preserving bits of a logit: NaN above all, -0 as +0.
DEV uint32_t order_bits(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
DEV float from_order_bits(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
DEV Key make_key(uint32_t ord, int index) { return (static_cast<Key>(ord) << 32) | (0xffffffffu - static_cast<uint32_t>(index)); }

// One compare-exchange step of a bitonic network over the lanes, larger values to lower lanes
// where `up` is false.
template <typename V>
DEV V exchange(V v, int mask, bool up) {
  const V w = __shfl_xor_sync(kAll, v, mask);
  const bool lower = (threadIdx.x & mask) == 0;
  return (lower != up) == (v > w) ? v : w;
}
// The lanes' values in descending order.
template <typename V>
DEV V sort_desc(V v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int step = size / 2; step >= 1; step >>= 1) v = exchange(v, step, size < 32 && (lane & size) != 0);
  return v;
}
// The 32 largest of two descending lists.
DEV Key merge_desc(Key a, Key b) {
  const Key r = __shfl_sync(kAll, b, 31 - (threadIdx.x & 31));
  Key v = a > r ? a : r;
#pragma unroll
  for (int step = 16; step >= 1; step >>= 1) v = exchange(v, step, false);
  return v;
}

struct Part {
  float M, S, W;
};
DEV Part join(const Part& a, const Part& b, float c) {
  Part r;
  r.M = fmaxf(a.M, b.M);
  const float base = r.M == -INFINITY ? 0.f : r.M;
  // a part without mass has M = -inf, S = W = 0; its shift must not become 0 * inf
  const float da = a.M == -INFINITY ? 0.f : (a.M - base) * c, db = b.M == -INFINITY ? 0.f : (b.M - base) * c;
  const float ea = ex2(da), eb = ex2(db);
  r.S = ea * a.S + eb * b.S;
  r.W = ea * (a.W + fmaxf(da, -200.f) * a.S) + eb * (b.W + fmaxf(db, -200.f) * b.S);
  return r;
}
DEV Part shfl_xor(const Part& p, int mask) {
  return {__shfl_xor_sync(kAll, p.M, mask), __shfl_xor_sync(kAll, p.S, mask), __shfl_xor_sync(kAll, p.W, mask)};
}

template <typename T>
DEV float widen(T v);
template <>
DEV float widen<float>(float v) {
  return v;
}
template <>
DEV float widen<__half>(__half v) {
  return __half2float(v);
}
template <>
DEV float widen<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

// Lists of the CTA's warps into warp 0's, the chunk's or row's best.
DEV Key merge_warps(Key list, Key (*s_list)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int half = kWarps / 2; half >= 1; half >>= 1) {
    if (warp >= half && warp < 2 * half) s_list[warp][lane] = list;
    __syncthreads();
    if (warp < half) list = merge_desc(list, s_list[warp + half][lane]);
  }
  return list;
}
DEV Part merge_parts(Part p, Part* s_part, float c) {  // every thread's part into every thread of warp 0
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) p = join(p, shfl_xor(p, o), c);
  if (lane == 0) s_part[warp] = p;
  __syncthreads();
  p = s_part[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) p = join(p, s_part[w], c);
  return p;
}

template <typename T>
DEV void write_row(const LogprobParams& P, int row, const T* z, int token, const Part& p, Key list) {
  constexpr float kLn2 = 0.6931471805599453f;
  const int lane = threadIdx.x & 31;
  const bool empty = p.S == 0.f;  // no finite logit
  const float base = p.M == -INFINITY ? 0.f : p.M, ls = log2f(p.S);
  if (lane == 0) {
    if (P.logprob) {
      P.logprob[row] = empty ? -INFINITY : (widen(z[token]) - base) * P.inv_temp - kLn2 * ls;
    }
    P.entropy[row] = empty ? 0.f : kLn2 * (ls - p.W / p.S);
  }
  if (lane < P.n_top) {
    const size_t at = static_cast<size_t>(row) * P.n_top + lane;
    const float x = from_order_bits(static_cast<uint32_t>(list >> 32));
    P.top_ids[at] = static_cast<int>(0xffffffffu - static_cast<uint32_t>(list));
    P.top_logprobs[at] = empty ? -INFINITY : (x - base) * P.inv_temp - kLn2 * ls;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobParams P) {
  constexpr int VE = 16 / sizeof(T);      // logits per 16-byte load
  constexpr int U = sizeof(T) == 4 ? 4 : 2;  // loads per thread and batch
  constexpr int NV = VE * U;              // 16 logits per thread and batch
  __shared__ Key s_list[kWarps][32];
  __shared__ Part s_part[kWarps];
  __shared__ volatile uint32_t s_thr[kWarps];
  __shared__ int s_last;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / P.chunks, chunk = blockIdx.x - row * P.chunks;
  const int V = P.V, k = P.n_top;
  const int token = P.tokens ? __ldcg(P.tokens + row) : 0;
  if (token < 0 || token >= V) {  // a row without a token
    if (chunk == 0) {
      if (tid == 0) {
        if (token != -1) raise_flag(P.err, kDevToken);
        if (P.logprob) P.logprob[row] = 0.f;
        P.entropy[row] = 0.f;
      }
      if (tid < k) {
        P.top_ids[static_cast<size_t>(row) * k + tid] = -1;
        P.top_logprobs[static_cast<size_t>(row) * k + tid] = 0.f;
      }
    }
    return;
  }
  const T* z = static_cast<const T*>(P.logits) + row * P.row_stride;
  // 16-byte words from the one that holds the row's first logit: word w holds logits
  // w * VE - skew .. + VE, of which those in [0, V) are the row's
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
  const uint4* words = reinterpret_cast<const uint4*>(z - skew);
  const int n_words = (V + skew + VE - 1) / VE;
  const int per = (n_words + P.chunks - 1) / P.chunks;
  const int w0 = min(chunk * per, n_words), w1 = min(w0 + per, n_words);
  const float c = P.scale;
  const int m = (k + kWarps - 1) / kWarps;  // a warp's share of the n_top largest
  Part p = {-INFINITY, 0.f, 0.f};
  Key list = 0;
  if (k > 0 && lane == 0) s_thr[warp] = 0;
  __syncthreads();

  auto load = [&](int base, uint4 (&q)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int w = base + u * kThreads + tid;
      if (w > 0 && w < w1 && w + 1 < n_words) {
        q[u] = __ldcs(words + w);
      } else {
        // the row's first and last word by single logits, what is not the row's as -inf
        T e[VE];
#pragma unroll
        for (int x = 0; x < VE; ++x) {
          const int at = w * VE - skew + x;
          e[x] = w < w1 && at >= 0 && at < V ? __ldcs(z + at) : static_cast<T>(-INFINITY);
        }
        q[u] = *reinterpret_cast<const uint4*>(e);
      }
    }
  };
  bool first = true;
  uint4 next[U];
  if (w0 < w1) load(w0, next);
  for (int base = w0; base < w1; base += U * kThreads) {
    float x[NV];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const T* e = reinterpret_cast<const T*>(&next[u]);
#pragma unroll
      for (int y = 0; y < VE; ++y) x[u * VE + y] = widen(e[y]);
    }
    if (base + U * kThreads < w1) load(base + U * kThreads, next);
    float top = x[0];
#pragma unroll
    for (int y = 1; y < NV; ++y) top = fmaxf(top, x[y]);
    if (top > p.M) p = join(p, Part{top, 0.f, 0.f}, c);
    const float b = p.M == -INFINITY ? 0.f : p.M;
    float ps = 0.f, pw = 0.f;
#pragma unroll
    for (int y = 0; y < NV; ++y) {
      const float d = (x[y] - b) * c, e = ex2(d);
      ps += e;
      pw = fmaf(e, fmaxf(d, -200.f), pw);  // a masked logit: 0 * -200
    }
    p.S += ps;
    p.W += pw;
    if (k > 0) {
      // the logit's index of x[u * VE + y] is (base + u * kThreads + tid) * VE - skew + y
      uint32_t best = 0;
#pragma unroll
      for (int y = 0; y < NV; ++y) best = max(best, order_bits(x[y]));
      uint32_t thr;
      if (first) {
        const uint32_t sorted = sort_desc(best);
        if (lane == m - 1) s_thr[warp] = sorted;
        __syncthreads();
        first = false;
      }
      thr = __reduce_min_sync(kAll, s_thr[lane & (kWarps - 1)]);
      if (__any_sync(kAll, best >= thr)) {
        Key kth = __shfl_sync(kAll, list, k - 1);
#pragma unroll
        for (int y = 0; y < NV; ++y) {
          const int at = (base + (y / VE) * kThreads + tid) * VE - skew + y % VE;
          const uint32_t ord = order_bits(x[y]);
          const Key key = make_key(ord, at);
          const bool cand = ord >= thr && key > kth && at >= 0 && at < V && at < w1 * VE - skew;
          unsigned votes = __ballot_sync(kAll, cand);
          if (votes == 0) continue;
          if (__popc(votes) <= 6) {
            while (votes) {
              const int from = __ffs(votes) - 1;
              votes &= votes - 1;
              const Key in = __shfl_sync(kAll, key, from);
              const Key above = __shfl_up_sync(kAll, list, 1);
              const bool keep = list > in;
              const bool above_keep = lane == 0 || above > in;
              list = keep ? list : above_keep ? in : above;
            }
          } else {
            list = merge_desc(list, sort_desc(cand ? key : 0));
          }
          kth = __shfl_sync(kAll, list, k - 1);
        }
        const uint32_t mine = static_cast<uint32_t>(list >> 32);
        if (lane == m - 1 && mine > s_thr[warp]) s_thr[warp] = mine;
        __syncwarp();
      }
    }
  }
  if (k > 0) list = merge_warps(list, s_list);
  p = merge_parts(p, s_part, c);
  if (P.chunks == 1) {
    if (warp == 0) write_row(P, row, z, token, p, list);
    return;
  }
  float* slot = P.part + static_cast<size_t>(blockIdx.x) * kLpSlotWords;
  if (warp == 0) {
    if (lane == 0) __stcg(reinterpret_cast<float4*>(slot), make_float4(p.M, p.S, p.W, 0.f));
    if (lane < k) __stcg(reinterpret_cast<Key*>(slot + 4) + lane, list);
    __threadfence();
    __syncwarp();
    if (lane == 0) {
      const int before = atomicAdd(P.row_cnt + row, 1);
      s_last = before == P.chunks - 1;
      if (s_last) P.row_cnt[row] = 0;
    }
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // the row's chunks in order: (max, sums) by threads, lists by warps
  const float* parts = P.part + static_cast<size_t>(row) * P.chunks * kLpSlotWords;
  p = {-INFINITY, 0.f, 0.f};
  for (int i = tid; i < P.chunks; i += kThreads) {
    const float4 q = __ldcg(reinterpret_cast<const float4*>(parts + static_cast<size_t>(i) * kLpSlotWords));
    p = join(p, Part{q.x, q.y, q.z}, c);
  }
  if (k > 0) {
    list = 0;
    for (int i = warp; i < P.chunks; i += kWarps) {
      const Key* other = reinterpret_cast<const Key*>(parts + static_cast<size_t>(i) * kLpSlotWords + 4);
      list = merge_desc(list, lane < k ? __ldcg(other + lane) : 0);
    }
    list = merge_warps(list, s_list);
  }
  __syncthreads();  // s_part of the first use has been read
  p = merge_parts(p, s_part, c);
  if (warp == 0) write_row(P, row, z, token, p, list);
}

}  // namespace

// Chunks per row: enough CTAs to fill the GPU eight times over (so that the last wave's
// remainder is small), chunks of 16 KB of logits at least, and no more parts than the
// workspace holds; rows that need no cutting are not cut.
int logprob_chunks(int rows, int vocab, int elem_bytes, int n_sms) {
  const long long bytes = static_cast<long long>(vocab) * elem_bytes;
  long long chunks = (8LL * n_sms + rows - 1) / rows;
  chunks = chunks < bytes / 16384 ? chunks : bytes / 16384;
  if (chunks < 1) chunks = 1;
  if (chunks > 256) chunks = 256;
  if (chunks > 1 && rows * chunks > kLpSlots) chunks = kLpSlots / rows;
  return chunks < 1 ? 1 : static_cast<int>(chunks);
}

int launch_logprobs(const LogprobParams& p, int dtype, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * p.chunks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (dtype == DFLASH_F32) e = cudaLaunchKernelEx(&cfg, logprobs_kernel<float>, p);
  else if (dtype == DFLASH_F16) e = cudaLaunchKernelEx(&cfg, logprobs_kernel<__half>, p);
  else e = cudaLaunchKernelEx(&cfg, logprobs_kernel<__nv_bfloat16>, p);
  return static_cast<int>(e);
}

}  // namespace dfl
