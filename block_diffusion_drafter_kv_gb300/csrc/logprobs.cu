// Log probabilities of given tokens, the entropy of their distributions and the most likely
// alternatives, in one pass over the logits.
//
// With c = log2(e) / T, a base B near c max z, d = c z - B, S = sum 2^d, W = sum 2^d d:
//   log p(token) = (z_token - max z) / T - ln 2 (log2 S - (c max z - B)),  H = ln 2 (log2 S - W / S)
// hold for any B. B is c max z rounded, and d one fused multiply-add, so that only 2^d rounds;
// sums of two bases join by 2^(B - B'): W' = 2^e (W + e S), e = B - B'. Where c max z is past 2^30
// (masks of the type's lowest value, tiny temperatures) d is c (z - max z), which cannot
// overflow, and every base involved stands for its exact c max z.
//
// Bound: reading the logits, once, at 2 or 4 bytes each.
// Split. The rows that have a token, in units of 4 KB of logits, form one list that is cut evenly
// over persistent CTAs: rows without a token cost nothing, no wave is left half full, few rows are
// split over all SMs, and a CTA has at most two rows that it shares with others. Those join in CTA
// order in the CTA that arrives last at the row, which does not depend on who that is; a row
// inside one range never leaves its CTA. (Chunks of 64 KB taken from a counter, each joined through
// global memory, took 129 us for 289 rows of 151936 fp32 against 46 then: fence, counter and parts
// are microseconds of latency, too many for 1.4 us of copying.)
// In a CTA a producer warp keeps a ring of 16 KB stages full by bulk copies across rows, and
// eight consumer warps share each stage. Two CTAs per SM with six stages where alternatives are
// wanted (registers), three with four where they are not (more warps for the arithmetic of 16-bit
// logits): 40.7 us and 45.1 us, 28.9 us and 27.2 us for the cases below.
//
// The n_top largest: every warp keeps the best of what it has read as a sorted list of 64-bit
// keys, one per lane, (order-preserving bits of the logit, ~index): ties go to the lowest
// index and all keys differ. What keeps this off the streaming path is a threshold: n_top values of
// the row are not below it, so that few values are candidates. A row starts with one from the first
// stage's lane maxima; then a warp of its own takes the n_top-th largest of all 256 lane maxima
// while they change (each warp raising it for itself, from four maxima a warp: 44.4 us against 40.7).
// Candidates wait in a buffer until 32 can be sorted and merged into the list at once: sorted
// logits, where every value is a candidate, take the same path.
//
// Measured: 289 of 512 rows of 151936 fp32, n_top 5, 41 us (63% of the copy rate; 32.8 us without
// alternatives, 62 us with 32: a row's first stages have many candidates); 1000 rows of 50257 bf16 without
// alternatives 27.7 us (53%: 3.7 us of it are the sums, 3 the join of cut rows at the end), with 5 of them
// 55 us (27%: a row is six stages long, and most of it is its start);
// 16 rows, n_top 20, 13.6 us, a chain of latencies: token list, first copy, sums, sort, join.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "math.cuh"
#include "ptx.cuh"
#include "target.h"

namespace dfl {

namespace {

constexpr int kWarps = 8;                    // consumer warps
constexpr int kConsumers = 32 * kWarps;
constexpr int kUnitWords = kConsumers;       // 16-byte words of a unit: one per consumer thread
constexpr int kStageUnits = 4;
constexpr int kStageWords = kStageUnits * kUnitWords;
// CTAs of an SM, and stages of 16 KB of each one's ring
template <bool TOP>
struct Shape {
  static constexpr int kCtasPerSm = TOP ? 2 : 3, kStages = TOP ? 6 : 4;
  static constexpr int kThreads = kConsumers + (TOP ? 64 : 32);  // and the producer, and the threshold's warp
};
// Rows of a call whose tokens are looked through before the list is cut: every CTA looks through all of
// them, a few to a thread. Calls of more rows cut a list of all rows, and a CTA walks past those without a
// token: 1107 of 2048 rows of 151936 fp32, n_top 5, 192 us (52% of the copy rate).
constexpr int kListed = 1024;
constexpr unsigned kAll = 0xffffffffu;
using Key = unsigned long long;

// NaN if one of them is.
DEV float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
DEV float warp_max_nan(float x) {
  float y;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
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
// The lanes' values in descending order. This and the functions below that are not inlined run a
// few times per chunk: inlined at each use they made the loop's code miss the instruction cache.
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
__device__ __noinline__ Key merge_lists(Key a, Key b) { return merge_desc(a, b); }
// Eight lists in shared memory into one.
__device__ __noinline__ Key merge_eight(const Key (*lists)[32]) {
  const int lane = threadIdx.x & 31;
  Key l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) l[i] = lists[i][lane];
#pragma unroll
  for (int h = 4; h >= 1; h >>= 1)
#pragma unroll
    for (int i = 0; i < h; ++i) l[i] = merge_desc(l[i], l[i + h]);
  return l[0];
}
DEV float widen1(float v) { return v; }
DEV float widen1(__half v) { return __half2float(v); }
DEV float widen1(__nv_bfloat16 v) { return __bfloat162float(v); }
// A warp's best values: a sorted list, one key per lane, and keys that wait for it until there
// are enough of them to sort.
constexpr int kWaiting = 96;
__device__ __noinline__ Key sort_into(Key list, const Key* waiting, int count) {  // count <= 32
  const int lane = threadIdx.x & 31;
  return merge_desc(list, sort_desc(lane < count ? waiting[lane] : 0));
}

// Sums relative to the maximum M.
struct Part {
  float M, S, W;
};
struct Scale {
  float c;
  float floor;  // kFloor / 16 of the logits' type
  // whether sums on the base of M can be taken by fused multiply-adds over raised logits: what is
  // raised to kFloor weighs 2^-240 at most there, 0 in fp32 (not so at high temperatures)
  DEV bool fast(float M) const { return fabsf(M * c) < 1073741824.f && M > floor && c < 1e8f && c * -floor > 16.f; }
  // log2 of the factor between sums on base `from` and sums on base `to` >= from
  DEV float shift(float from, float to) const {
    return fast(from) && fast(to) ? __fmul_rn(from, c) - __fmul_rn(to, c) : (from - to) * c;
  }
  // c z - B, the base B of M
  DEV float residual(float M) const { return fast(M) ? fmaf(M, c, -__fmul_rn(M, c)) : 0.f; }
  DEV Part join(const Part& a, const Part& b) const {
    Part r;
    r.M = fmaxf(a.M, b.M);
    // a part without mass has M = -inf and S = W = 0: its shift must not become 0 * inf
    const float da = a.M == -INFINITY ? 0.f : shift(a.M, r.M), db = b.M == -INFINITY ? 0.f : shift(b.M, r.M);
    const float ea = ex2(da), eb = ex2(db);
    r.S = ea * a.S + eb * b.S;
    r.W = ea * (a.W + fmaxf(da, -200.f) * a.S) + eb * (b.W + fmaxf(db, -200.f) * b.S);
    return r;
  }
};

// A 16-byte word of logits: their maximum (NaN if one is), and their values as fp32 with what
// lies below kFloor raised to it: d of a masked logit is then finite, and 2^d d is 0.
template <typename T>
struct Word;
template <>
struct Word<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kMinusInf = 0xff800000u;
  static constexpr float kFloor = -1e30f;
  DEV static void widen(const uint4& q, float* x) {
    x[0] = __uint_as_float(q.x), x[1] = __uint_as_float(q.y), x[2] = __uint_as_float(q.z), x[3] = __uint_as_float(q.w);
  }
  DEV static float top(const uint4& q) {
    return max_nan(max_nan(__uint_as_float(q.x), __uint_as_float(q.y)), max_nan(__uint_as_float(q.z), __uint_as_float(q.w)));
  }
  DEV static uint4 raised(uint4 q) {
    q.x = __float_as_uint(fmaxf(__uint_as_float(q.x), kFloor)), q.y = __float_as_uint(fmaxf(__uint_as_float(q.y), kFloor));
    q.z = __float_as_uint(fmaxf(__uint_as_float(q.z), kFloor)), q.w = __float_as_uint(fmaxf(__uint_as_float(q.w), kFloor));
    return q;
  }
};
template <typename H2>
struct Word16 {
  DEV static H2 as2(uint32_t u) { return *reinterpret_cast<const H2*>(&u); }
  DEV static uint32_t bits(H2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
  DEV static H2 top2(const uint4& q) { return __hmax2_nan(__hmax2_nan(as2(q.x), as2(q.y)), __hmax2_nan(as2(q.z), as2(q.w))); }
  DEV static uint4 raised(const uint4& q, H2 floor) {
    return {bits(__hmax2(as2(q.x), floor)), bits(__hmax2(as2(q.y), floor)), bits(__hmax2(as2(q.z), floor)), bits(__hmax2(as2(q.w), floor))};
  }
};
template <>
struct Word<__nv_bfloat16> : Word16<__nv_bfloat162> {
  static constexpr int N = 8;
  static constexpr uint32_t kMinusInf = 0xff80ff80u;
  static constexpr float kFloor = -1e30f;
  DEV static void widen(const uint4& q, float* x) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(u[i] << 16), x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
  DEV static float top(const uint4& q) {
    const float2 f = __bfloat1622float2(top2(q));
    return max_nan(f.x, f.y);
  }
  DEV static uint4 raised(const uint4& q) { return Word16::raised(q, __float2bfloat162_rn(kFloor)); }
};
template <>
struct Word<__half> : Word16<__half2> {
  static constexpr int N = 8;
  static constexpr uint32_t kMinusInf = 0xfc00fc00u;
  static constexpr float kFloor = -65504.f;
  DEV static void widen(const uint4& q, float* x) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  DEV static float top(const uint4& q) {
    const float2 f = __half22float2(top2(q));
    return max_nan(f.x, f.y);
  }
  DEV static uint4 raised(const uint4& q) { return Word16::raised(q, __float2half2_rn(kFloor)); }
};

// Candidates of a warp, the values not below `floor` of the lanes in `votes`: their NW words of a
// lane are read again by the whole warp, an element each. Lane 0's words start at `vals` and lie
// `stride` apart there and in the row, from `index` on; elements from `limit` on do not count.
// (A chain of latencies on the streaming path: the lanes' numbers go through shared memory, and two
// rounds of loads and votes are in flight together. Compact, too: a ballot for each of the words'
// elements in registers is fewer steps, but so much code that it waits for its instructions, 49 us
// against 41.)
struct Noted {
  Key list;
  int waiting;  // keys that wait now
};
template <typename T, int NW>
__device__ __noinline__ Noted note_candidates(Noted to, Key* waiting, uint8_t* lanes, unsigned votes, float floor, const T* vals,
                                              int stride, int index, int limit) {
  constexpr int VE = 16 / sizeof(T), N = NW * VE;  // elements of a lane: 32 or 16
  const int lane = threadIdx.x & 31, sub = lane % N;
  const unsigned below = (1u << lane) - 1;
  if (votes >> lane & 1) lanes[__popc(votes & below)] = static_cast<uint8_t>(lane);
  __syncwarp();
  const int total = __popc(votes);
#pragma unroll 1
  for (int done = 0; done < total; done += 2 * (32 / N)) {
    float x[2];
    int at[2];
    unsigned in[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int who = done + i * (32 / N) + lane / N;
      const int off = (who < total ? lanes[who] : 0) * VE + sub / VE * stride + sub % VE;
      at[i] = who < total && index + off < limit ? index + off : -1;
      x[i] = widen1(vals[off]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) in[i] = __ballot_sync(kAll, at[i] >= 0 && !(x[i] < floor));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (in[i] >> lane & 1) waiting[to.waiting + __popc(in[i] & below)] = make_key(order_bits(x[i]), at[i]);
      to.waiting += __popc(in[i]);
    }
    __syncwarp();
    while (to.waiting >= 32) {  // (at most 31 + 64)
      to.waiting -= 32;
      to.list = sort_into(to.list, waiting + to.waiting, 32);
      __syncwarp();
    }
  }
  return to;
}

// A row's words of 16 bytes: `lead` logits before the first whole aligned word, `words` whole
// ones, the rest behind them.
template <typename T>
struct RowWords {
  const T* z;
  int lead, words;
  DEV RowWords(const LogprobParams& P, int row) {
    constexpr int N = Word<T>::N;
    z = static_cast<const T*>(P.logits) + row * P.row_stride;
    lead = min(P.V, static_cast<int>((N - (reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T)) % N));
    words = (P.V - lead) / N;
  }
};

DEV int add_acq_rel(int* p, int v) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

template <int STAGES, bool TOP>
struct SharedOf {
  uint4 ring[STAGES][kStageWords];
  static constexpr int kLists = TOP ? kWarps : 1;
  Key waiting[kLists][kWaiting];
  Key list[kLists][32];         // the warps' results of a segment
  Part part[kWarps];
  uint64_t full[STAGES], empty[STAGES], ready, taken;
  // by segment mod 2, since a warp can be one segment ahead of another:
  uint8_t lanes[kLists][32];
  uint32_t best[2][kLists][32];      // each lane's largest value
  uint4 tops[2][kWarps];             // the four largest of each warp after its first stage
  unsigned long long thr;            // (segment + 1, bits of a value that no candidate of it lies below)
  volatile uint32_t started;         // the last segment of which all warps have stored their first `best`
  volatile uint32_t events;          // stores to `best` so far
  volatile int done;
  float z_token[2];                  // the token's logit, of the row this CTA begins with, of the row it ends with
  volatile int abort;
  volatile int last[2];         // whether this CTA arrived last at the row it begins with, at the row it ends with
  int warp_rows[kWarps + 2];
  uint16_t rows[2];             // [min(rows, kListed)] the rows that have a token
};

// The threshold that a segment starts with: the k-th largest of the four largest lane maxima of
// each warp, which the warps leave before a barrier and each looks at behind it.
template <typename Shared>
__device__ __noinline__ void publish_tops(Shared& sh, int par, uint32_t best) {
  static_assert(kLpMaxTop == 4 * kWarps, "four of each warp make the longest list");
  const int lane = threadIdx.x & 31;
  uint32_t t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = __reduce_max_sync(kAll, best);
    if (lane == __ffs(__ballot_sync(kAll, best == t[i])) - 1) best = 0;
  }
  if (lane == 0) sh.tops[par][threadIdx.x >> 5] = make_uint4(t[0], t[1], t[2], t[3]);
  __syncwarp();
}
template <typename Shared>
__device__ __noinline__ uint32_t first_threshold(const Shared& sh, int par, int k) {
  const int lane = threadIdx.x & 31;
  const uint32_t mine = reinterpret_cast<const uint32_t*>(sh.tops[par])[lane];
  int above = 0;  // values before this one in descending order
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const uint32_t v = __shfl_sync(kAll, mine, i);
    above += v > mine || (v == mine && i < lane);
  }
  return __shfl_sync(kAll, mine, __ffs(__ballot_sync(kAll, above == k - 1)) - 1);
}
// The k-th largest of the 256 lane maxima of the segment that runs, again and again while they change:
// k values of the row are not below it. (Maxima that change meanwhile only grow. A segment's name goes
// with its threshold, so that one that is late for it is not taken for the next.)
template <typename Shared>
DEV void keep_threshold(Shared& sh, int k) {
  const int lane = threadIdx.x & 31;
  uint32_t seen = 0;
  while (true) {
    const uint32_t events = __shfl_sync(kAll, sh.events, 0);
    if (__any_sync(kAll, sh.done != 0)) return;
    if (events == seen) {
      __nanosleep(100);
      continue;
    }
    seen = events;
    const uint32_t seg = __shfl_sync(kAll, sh.started, 0);
    __threadfence_block();
    uint32_t v[kWarps], top = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v[w] = *const_cast<volatile uint32_t*>(&sh.best[seg & 1][w][lane]);
#pragma unroll 1
    for (int i = 0; i < k; ++i) {
      uint32_t mine = v[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mine = max(mine, v[w]);
      top = __reduce_max_sync(kAll, mine);
      bool drop = lane == __ffs(__ballot_sync(kAll, mine == top)) - 1;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (drop && v[w] == top) v[w] = 0, drop = false;
    }
    if (lane == 0) atomicMax(&sh.thr, static_cast<Key>(seg + 1) << 32 | top);
  }
}

__device__ __noinline__ void wait_long(uint64_t* bar, uint32_t parity, volatile int* abort, int* err, unsigned long long limit_ns) {
  if (*abort) return;
  if (!mbar_wait(bar, parity, limit_ns)) {
    *abort = 1;
    raise_flag(err, kDevTimeout);
  }
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(Shape<TOP>::kThreads, Shape<TOP>::kCtasPerSm) logprobs_kernel(const LogprobParams P) {
  using Shared = SharedOf<Shape<TOP>::kStages, TOP>;
  constexpr int kStages = Shape<TOP>::kStages, kThreads = Shape<TOP>::kThreads;
  constexpr int VE = Word<T>::N;
  constexpr float kLn2 = 0.6931471805599453f;
  extern __shared__ uint8_t smem_raw[];
  Shared& sh = *reinterpret_cast<Shared*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int V = P.V, k = TOP ? P.n_top : 0;
  const bool listed = P.rows <= kListed;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kWarps);
    }
    mbar_init(&sh.ready, kWarps);
    mbar_init(&sh.taken, 1);
    sh.abort = sh.last[0] = sh.last[1] = 0;
    sh.thr = 0;
    sh.started = sh.events = 0;
    sh.done = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  // Every wait is bounded: past the limit the flag is set and every role leaves its loop.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_try_wait(bar, parity)) wait_long(bar, parity, &sh.abort, P.err, P.wait_ns);
  };
  // The rows to read. Rows without a token get their values from CTA 0, or in calls of more rows
  // than are looked through from the CTA that walks past them.
  auto no_token = [&](int row, int token) {  // one thread
    if (token != -1) raise_flag(P.err, kDevToken);
    if (P.logprob) P.logprob[row] = 0.f;
    P.entropy[row] = 0.f;
    for (int i = 0; i < k; ++i) {
      P.top_ids[static_cast<size_t>(row) * k + i] = -1;
      P.top_logprobs[static_cast<size_t>(row) * k + i] = 0.f;
    }
  };
  auto has_token = [&](int token) { return token >= 0 && token < V; };
  int n_rows = P.rows;
  if (listed && P.tokens) {
    // each thread a run of rows, all its loads in flight, then a scan over the threads
    constexpr int kRun = (kListed + kThreads - 1) / kThreads;
    const int run = (P.rows + kThreads - 1) / kThreads;
    int token[kRun];
    uint32_t in = 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int row = tid * run + i;
      token[i] = i < run && row < P.rows ? __ldcg(P.tokens + row) : -1;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int row = tid * run + i;
      if (has_token(token[i])) in |= 1u << i;
      else if (blockIdx.x == 0 && i < run && row < P.rows) no_token(row, token[i]);
    }
    int upto = __popc(in);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) sh.warp_rows[warp] = upto;
    __syncthreads();
    int at = upto - __popc(in);
    n_rows = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += sh.warp_rows[w];
      n_rows += sh.warp_rows[w];
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i)
      if (in >> i & 1) sh.rows[at++] = static_cast<uint16_t>(tid * run + i);
    __syncthreads();
  }
  const int per_row = P.units;  // units of a row
  const long long U = static_cast<long long>(n_rows) * per_row;
  // at most one CTA for every two stages of a row; where rows go to eight or more CTAs each, to the same number
  int G = static_cast<int>(min(static_cast<long long>(gridDim.x), static_cast<long long>(n_rows) * ((per_row + 2 * kStageUnits - 1) / (2 * kStageUnits))));
  if (n_rows > 0 && G / 8 >= n_rows) G -= G % n_rows;
  const int cta = blockIdx.x;
  if (cta >= G) return;
  const long long U0 = range_begin(cta, U, G), U1 = range_begin(cta + 1, U, G);
  // The walk of both roles: the rows of this range from rank r0 on (the first from its unit u00),
  // with their first and last unit in the range: no division past the first.
  const int r0 = static_cast<int>(quotient(U0, per_row)), u00 = static_cast<int>(U0 - static_cast<long long>(r0) * per_row);
  auto row_of = [&](int rank) { return listed && P.tokens ? static_cast<int>(sh.rows[rank]) : rank; };
  auto token_of = [&](int row) { return P.tokens ? __ldcg(P.tokens + row) : 0; };

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer warp
    if (lane != 0) return;
    const uint64_t pol = policy_evict_first();
    int n = 0;  // stages issued
    int rank = r0, u0 = u00;
    for (long long left = U1 - U0; left > 0 && !sh.abort; ++rank, u0 = 0) {
      const int u1 = static_cast<int>(min(static_cast<long long>(per_row), u0 + left)), row = row_of(rank);
      left -= u1 - u0;
      if (!listed && P.tokens) {
        const int token = token_of(row);
        if (!has_token(token)) {
          if (u0 == 0) no_token(row, token);
          continue;
        }
      }
      const RowWords<T> rw(P, row);
      const int end = min(u1 * kUnitWords, rw.words);
      for (int w = u0 * kUnitWords; w < end && !sh.abort; w += kStageWords) {
        const int st = n % kStages, words = min(kStageWords, end - w);
        if (n >= kStages) wait(&sh.empty[st], (n / kStages - 1) & 1);
        if (sh.abort) break;
        mbar_arrive_expect_tx(&sh.full[st], words * 16);
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
                smem_u32(sh.ring[st])),
            "l"(reinterpret_cast<uint64_t>(rw.z + rw.lead + static_cast<size_t>(w) * VE)), "r"(words * 16),
            "r"(smem_u32(&sh.full[st])), "l"(pol)
            : "memory");
        ++n;
      }
    }
    if (sh.abort)  // the copies still in flight land before the CTA leaves
      for (int i = max(0, n - kStages); i < n; ++i) mbar_wait(&sh.full[i % kStages], (i / kStages) & 1, P.wait_ns);
    return;
  }

  if (TOP && warp == kWarps + 1) {
    // ------------------------------------------------------------ the threshold's warp
    keep_threshold(sh, k);
    return;
  }

  // -------------------------------------------------------------- consumer warps
  const Scale sc = {P.scale, Word<T>::kFloor / 16};
  float M = -INFINITY;                       // the warp's, the same in every lane
  float2 S2 = {0.f, 0.f}, W2 = {0.f, 0.f};   // the thread's
  Key list = 0;
  int waiting = 0;                           // keys that are not in the list yet
  uint32_t best = 0;                         // the lane's largest value in the segment
  uint32_t thr = 0;                          // the threshold as last read
  bool fresh = true;
  int seg_no = 0;

  auto rebase = [&](float wtop) {  // onto a larger maximum
    if (wtop <= M) return;
    if (wtop == wtop) {
      const float e = M == -INFINITY ? 0.f : sc.shift(M, wtop);
      const float f = ex2(e), ec = fmaxf(e, -200.f);
      W2 = {f * (W2.x + ec * S2.x), f * (W2.y + ec * S2.y)};
      S2 = {f * S2.x, f * S2.y};
      M = wtop;
    } else {
      S2.x = W2.x = wtop;  // a NaN spoils the row's sums
    }
  };
  // NW words of each thread. The warp's words start at `vals` and lie a unit apart there and in the
  // row, from `index` on; elements from `limit` on are filled up with -inf and do not count.
  auto take = [&](auto& q, auto nw_const, const T* vals, int index, int limit) {
    constexpr int NW = decltype(nw_const)::value;
    float top = Word<T>::top(q[0]);
#pragma unroll
    for (int w = 1; w < NW; ++w) top = max_nan(top, Word<T>::top(q[w]));
    if (__any_sync(kAll, !(top <= M))) rebase(warp_max_nan(top));
    if (sc.fast(M)) {
      const float B = __fmul_rn(M, sc.c);
      const float2 c2 = {sc.c, sc.c}, b2 = {-B, -B};
      float2 s2 = {0.f, 0.f}, w2 = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        float x[VE];
        Word<T>::widen(Word<T>::raised(q[w]), x);
#pragma unroll
        for (int y = 0; y < VE; y += 2) {
          const float2 d = fma2(float2{x[y], x[y + 1]}, c2, b2);
          const float2 e = {ex2(d.x), ex2(d.y)};
          s2 = add2(s2, e);
          w2 = fma2(e, d, w2);
        }
      }
      S2 = add2(S2, s2);
      W2 = add2(W2, w2);
    } else if (M > -INFINITY) {  // (nothing but -inf so far: nothing to add)
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        float x[VE];
        Word<T>::widen(q[w], x);
#pragma unroll
        for (int y = 0; y < VE; ++y) {
          const float d = (x[y] - M) * sc.c, e = ex2(d);
          S2.x += e;
          W2.x = fmaf(e, fmaxf(d, -200.f), W2.x);  // a masked logit: 0 * -200
        }
      }
    }
    if (TOP) {
      best = max(best, order_bits(top));
      if (fresh) {
        sh.best[seg_no & 1][warp][lane] = best;
        publish_tops(sh, seg_no & 1, best);
        named_bar_sync(1, kConsumers);
        if (tid == 0) sh.started = seg_no;
        thr = first_threshold(sh, seg_no & 1, k);
        fresh = false;
      }
      const float thr_f = from_order_bits(thr);
      const unsigned votes = __ballot_sync(kAll, !(top < thr_f));
      if (votes) {
        const Noted to = note_candidates<T, NW>({list, waiting}, sh.waiting[warp], sh.lanes[warp], votes, thr_f, vals, kUnitWords * VE, index, limit);
        list = to.list, waiting = to.waiting;
        sh.best[seg_no & 1][warp][lane] = best;
        __syncwarp();
        if (lane == 0) atomicAdd(const_cast<uint32_t*>(&sh.events), 1u);
      }
    }
  };
  // The parts of the first `lanes` lanes into one, in all lanes; what the others up to the next power
  // of two hold has no mass.
  auto join_lanes = [&](Part p, int lanes) {
#pragma unroll 1
    for (int o = 1; o < min(lanes, 32); o <<= 1)
      p = sc.join(p, Part{__shfl_xor_sync(kAll, p.M, o), __shfl_xor_sync(kAll, p.S, o), __shfl_xor_sync(kAll, p.W, o)});
    return Part{__shfl_sync(kAll, p.M, 0), __shfl_sync(kAll, p.S, 0), __shfl_sync(kAll, p.W, 0)};
  };
  auto write_row = [&](int row, float z_token, const Part& p) {  // one warp; its list is the row's, lane 0 has the token's logit
    const bool empty = p.S == 0.f;  // every logit -inf
    const float top = p.M == -INFINITY ? 0.f : p.M;
    const float ls = kLn2 * (log2f(p.S) - (p.M == -INFINITY ? 0.f : sc.residual(p.M)));
    if (lane == 0) {
      if (P.logprob) P.logprob[row] = empty ? -INFINITY : (z_token - top) * P.inv_temp - ls;
      P.entropy[row] = empty ? 0.f : max_nan(kLn2 * (log2f(p.S) - p.W / p.S), 0.f);  // (rounding could leave -1e-7)
    }
    if (lane < k) {
      const size_t to = static_cast<size_t>(row) * k + lane;
      P.top_ids[to] = static_cast<int>(0xffffffffu - static_cast<uint32_t>(list));
      P.top_logprobs[to] = empty ? -INFINITY : (from_order_bits(static_cast<uint32_t>(list >> 32)) - top) * P.inv_temp - ls;
    }
  };
  // a CTA's part of the row that it begins with (0), or of the row that it ends with (1); a row's
  // counter is that of the first CTA that has a part of it
  auto slot_of = [&](int c, int which) { return P.part + (2 * static_cast<size_t>(c) + which) * kLpSlotWords; };

  int n = 0;  // stages taken
  int rank = r0, u0 = u00;
  for (long long left = U1 - U0; left > 0; ++rank, u0 = 0) {
    const int u1 = static_cast<int>(min(static_cast<long long>(per_row), u0 + left)), row = row_of(rank);
    left -= u1 - u0;
    if (!listed && P.tokens && !has_token(token_of(row))) continue;
    const RowWords<T> rw(P, row);
    // the logits outside whole words, before and behind them, one to a lane of warp 0: loaded now,
    // taken at the segment's end
    int edge = -1;
    if (warp == 0 && lane < VE) edge = u0 == 0 && lane < rw.lead ? lane : -1;
    else if (warp == 0 && lane < 2 * VE) edge = rw.lead + rw.words * VE + lane - VE;
    if (edge >= V || (lane >= VE && u1 < per_row)) edge = -1;
    const float edge_x = edge >= 0 ? widen1(rw.z[edge]) : -INFINITY;
    const int finisher = seg_no % kWarps;
    float z_token = 0.f;  // asked for now, used at the segment's end
    if (warp == finisher && lane == 0 && P.logprob) z_token = widen1(rw.z[token_of(row)]);
    const int end = min(u1 * kUnitWords, rw.words);
    for (int w0 = u0 * kUnitWords; w0 < end; w0 += kStageWords, ++n) {
      const int st = n % kStages, words = min(kStageWords, end - w0);
      if (TOP && !fresh) {
        const Key now = *const_cast<volatile Key*>(&sh.thr);
        if (static_cast<uint32_t>(now >> 32) == static_cast<uint32_t>(seg_no) + 1) thr = max(thr, static_cast<uint32_t>(now));
      }
      wait(&sh.full[st], (n / kStages) & 1);
      __syncwarp();
      constexpr int L = kStageUnits;  // words of a thread at a time
      uint4* ring = sh.ring[st] + tid;
      if (words < kStageWords) {  // the thread's words that the stage lacks
        constexpr uint32_t f = Word<T>::kMinusInf;
#pragma unroll
        for (int i = 0; i < L; ++i)
          if (i * kUnitWords + tid >= words) ring[i * kUnitWords] = uint4{f, f, f, f};
        fence_async_shared();  // the next copy into them comes after
      }
      uint4 q[L];
#pragma unroll
      for (int i = 0; i < L; ++i) q[i] = ring[i * kUnitWords];
      take(q, std::integral_constant<int, L>(), reinterpret_cast<const T*>(sh.ring[st] + warp * 32),
           rw.lead + (w0 + warp * 32) * VE, rw.lead + end * VE);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[st]);
    }
    // ---- the segment's end
    if (TOP && fresh) named_bar_sync(1, kConsumers);  // a segment without a whole word
    if (__any_sync(kAll, edge >= 0)) {
      rebase(warp_max_nan(edge_x));
      if (M > -INFINITY) {
        const float d = sc.fast(M) ? fmaf(fmaxf(edge_x, Word<T>::kFloor), sc.c, -__fmul_rn(M, sc.c)) : (edge_x - M) * sc.c;
        const float e = ex2(d);
        S2.x += e;
        W2.x = fmaf(e, fmaxf(d, -200.f), W2.x);
      }
      if (TOP) {
        if (fresh) thr = 0;
        const bool in = edge >= 0 && order_bits(edge_x) >= thr;
        const unsigned votes = __ballot_sync(kAll, in);
        if (in) sh.waiting[warp][waiting + __popc(votes & ((1u << lane) - 1))] = make_key(order_bits(edge_x), edge);
        waiting += __popc(votes);  // at most 31 + 16
        __syncwarp();
        if (waiting >= 32) {
          waiting -= 32;
          list = sort_into(list, sh.waiting[warp] + waiting, 32);
          __syncwarp();
        }
      }
    }
    if (TOP) {
      list = sort_into(list, sh.waiting[warp], waiting);
      waiting = 0;
    }
    float S = S2.x + S2.y, W = W2.x + W2.y;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      S += __shfl_xor_sync(kAll, S, o);
      W += __shfl_xor_sync(kAll, W, o);
    }
    // The warps hand their results to one of them, another for each segment, and go on.
    if (seg_no >= 1) wait(&sh.taken, (seg_no - 1) & 1);
    __syncwarp();
    if (lane == 0) sh.part[warp] = {M, S, W};
    if (TOP) sh.list[warp][lane] = list;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.ready);
    M = -INFINITY;
    S2 = W2 = {0.f, 0.f};
    fresh = true;
    best = 0;
    const uint32_t round = seg_no++;
    if (warp == finisher) {
      const bool whole = u0 == 0 && u1 == per_row;
      const long long base = static_cast<long long>(rank) * per_row;
      int c0 = 0, c1 = 0;
      if (!whole) c0 = cta_of(base, U, G), c1 = cta_of(base + per_row - 1, U, G);
      wait(&sh.ready, round & 1);
      __syncwarp();
      if (TOP) list = merge_eight(sh.list);
      const Part p = join_lanes(sh.part[lane & (kWarps - 1)], kWarps);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.taken);
      if (whole) {
        write_row(row, z_token, p);
      } else {
        float* slot = slot_of(cta, base > U0);
        if (lane == 0) __stcg(reinterpret_cast<float4*>(slot), make_float4(p.M, p.S, p.W, 0.f));
        if (lane < k) __stcg(reinterpret_cast<Key*>(slot + 4) + lane, list);
        __syncwarp();
        // releases the warp's part, and acquires the others' for the CTA (by way of the barrier below)
        if (lane == 0 && add_acq_rel(P.row_cnt + c0, 1) == c1 - c0) {
          P.row_cnt[c0] = 0;
          sh.last[base > U0] = 1;
          sh.z_token[base > U0] = z_token;
        }
      }
    }
    list = 0;
  }
  // ---- the rows that this CTA shares with others and was the last to arrive at, by all warps
  named_bar_sync(1, kConsumers);
  if (tid == 0) sh.done = 1;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (!sh.last[which]) continue;
    const int rank = which == 0 ? r0 : static_cast<int>(quotient(U1 - 1, per_row)), row = row_of(rank);
    const long long base = static_cast<long long>(rank) * per_row;
    const int c0 = cta_of(base, U, G), c1 = cta_of(base + per_row - 1, U, G);
    // the row is the first of every CTA that has a part of it but perhaps c0
    const int c0_which = range_begin(c0, U, G) < base;
    if (TOP) {
      list = 0;
#pragma unroll 1
      for (int c = c0 + warp; c <= c1; c += 4 * kWarps) {
        Key other[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int from = c + i * kWarps;
          other[i] = from <= c1 && lane < k ? __ldcg(reinterpret_cast<const Key*>(slot_of(from, from == c0 ? c0_which : 0) + 4) + lane) : 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i * kWarps <= c1) list = merge_lists(list, other[i]);
      }
      sh.list[warp][lane] = list;
      named_bar_sync(1, kConsumers);
    }
    if (warp == 0) {
      if (TOP) list = merge_eight(sh.list);
      Part p = {-INFINITY, 0.f, 0.f};
      for (int c = c0 + lane; c <= c1; c += 32) {
        const float4 q = __ldcg(reinterpret_cast<const float4*>(slot_of(c, c == c0 ? c0_which : 0)));
        p = c - c0 < 32 ? Part{q.x, q.y, q.z} : sc.join(p, Part{q.x, q.y, q.z});
      }
      p = join_lanes(p, c1 - c0 + 1);
      write_row(row, sh.z_token[which], p);
    }
    if (TOP) named_bar_sync(1, kConsumers);  // the lists' buffer is the other row's
  }
}

template <bool TOP>
int smem_bytes(int rows) {
  using Shared = SharedOf<Shape<TOP>::kStages, TOP>;
  static_assert(sizeof(Shared) + 128 + 2 * kListed + 1024 <= 233472 / Shape<TOP>::kCtasPerSm, "shared memory of an SM");
  return static_cast<int>(sizeof(Shared)) + 128 + 2 * rows;
}

template <typename T, bool TOP>
cudaError_t launch(const LogprobParams& p, int n_sms, cudaStream_t stream) {
  const long long stages = (static_cast<long long>(p.rows) * p.units + kStageUnits - 1) / kStageUnits;
  const int most = std::min(Shape<TOP>::kCtasPerSm * n_sms, kLpMaxCtas);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(stages, most)));
  cfg.blockDim = dim3(Shape<TOP>::kThreads);
  cfg.dynamicSmemBytes = smem_bytes<TOP>(p.rows <= kListed ? p.rows : 0);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, TOP>, p);
}

template <typename T, bool TOP>
cudaError_t set_attr() {
  return cudaFuncSetAttribute(logprobs_kernel<T, TOP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<TOP>(kListed));
}

}  // namespace

int logprob_set_attributes() {
  const cudaError_t e[] = {set_attr<float, false>(),  set_attr<float, true>(),         set_attr<__half, false>(),
                           set_attr<__half, true>(),  set_attr<__nv_bfloat16, false>(), set_attr<__nv_bfloat16, true>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return static_cast<int>(x);
  return 0;
}

int launch_logprobs(LogprobParams p, int dtype, int n_sms, cudaStream_t stream) {
  const long long bytes = static_cast<long long>(p.V) * (dtype == DFLASH_F32 ? 4 : 2);
  p.units = static_cast<int>((bytes + 16 * kUnitWords - 1) / (16 * kUnitWords));
  const bool top = p.n_top > 0;
  cudaError_t e;
  if (dtype == DFLASH_F32) e = top ? launch<float, true>(p, n_sms, stream) : launch<float, false>(p, n_sms, stream);
  else if (dtype == DFLASH_F16) e = top ? launch<__half, true>(p, n_sms, stream) : launch<__half, false>(p, n_sms, stream);
  else e = top ? launch<__nv_bfloat16, true>(p, n_sms, stream) : launch<__nv_bfloat16, false>(p, n_sms, stream);
  return static_cast<int>(e);
}

}  // namespace dfl
