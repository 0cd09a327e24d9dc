// The page pool of a paged cache: pages handed out and taken back on the GPU, and the cache
// rows (slots) of the positions they make room for.
//
// The mathematics is a prefix sum over the sequences: with add_s pages wanted by sequence s
// and A_s their exclusive prefix sum, new page number i of the call is entry n_free - 1 - i
// of the free list, and belongs to the last s with A_s <= i. Every CTA computes the prefix
// sum for itself (a few hundred integers, cheaper than a second launch or a grid barrier)
// and takes its share of the new table entries and of the slots. Slots of a page that this
// same call hands out are read from the free list, not from the table, so that no CTA waits
// for another's writes; the held counts and the length of the list, which every CTA reads,
// are written by the CTA that arrives last.
//
// Bound: latency (a few hundred bytes to read, 4 bytes a new row to write): lengths, prefix sum,
// list, slots, and with more than one CTA the counter. Measured, reserve and release together: 32
// blocks of 16 rows 6.8 us, 256 prompts of up to 2048 rows (2 MB of slots) 11.1 us.
#include "ptx.cuh"
#include "target.h"

namespace dfl {

namespace {

constexpr int kThreads = 256;

struct PageParams {
  dflash_page_pool p;
  const int* len;
  const int* n_new;  // reserve only
  int* slots;        // reserve only; null: none wanted
  int batch, rows_per_seq;
  int wide;          // slots is 16-byte aligned
};

// Exclusive prefix sum of `mine` over the block's threads; `total` gets the sum.
DEV long long block_scan(long long mine, long long* warp_sum, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long v = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    all += warp_sum[w];
  }
  total = all;
  return before + v - mine;
}

// The last sequence whose first page number is at most i (s_off is non-decreasing).
DEV int owner_of(const int* s_off, int batch, int i) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_off[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Pages that a sequence wants beyond those it holds; -1 where its lengths are out of range.
DEV int pages_wanted(const PageParams& P, int len, int n, int held) {
  if (len < 0 || n < 0 || n > P.rows_per_seq || held < 0 || held > P.p.pages_per_seq) return -1;
  const long long need = (static_cast<long long>(len) + n + kPagePos - 1) / kPagePos;
  if (need > P.p.pages_per_seq) return -1;
  return need > held ? static_cast<int>(need) - held : 0;
}

__global__ void __launch_bounds__(kThreads) pages_reserve_kernel(const PageParams P) {
  extern __shared__ int s_off[];    // [batch] number of the sequence's first new page
  int* s_new = s_off + P.batch;     // [batch] its new pages; -1: refused
  int* s_held = s_new + P.batch;    // [batch] the pages it holds
  int* s_len = s_held + P.batch;    // [batch]
  int* s_rows = s_len + P.batch;    // [batch] its new rows, 0 if it is refused
  __shared__ long long warp_sum[kThreads / 32];
  __shared__ int s_total, s_last;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, batch = P.batch;
  const int n_free = min(max(__ldcg(P.p.state), 0), P.p.n_pages);
  for (int s = tid; s < batch; s += kThreads) {
    s_held[s] = __ldcg(P.p.held + s);
    s_len[s] = __ldcg(P.len + s);
    s_rows[s] = __ldcg(P.n_new + s);
  }
  if (tid == 0) s_total = 0;
  __syncthreads();
  // each thread a run of neighbouring sequences
  const int per = (batch + kThreads - 1) / kThreads;
  const int s0 = min(tid * per, batch), s1 = min(s0 + per, batch);
  long long mine = 0;
  for (int s = s0; s < s1; ++s) {
    const int w = pages_wanted(P, s_len[s], s_rows[s], s_held[s]);
    s_new[s] = w;
    mine += max(w, 0);
  }
  long long total;
  long long off = block_scan(mine, warp_sum, total);
  int served = 0;
  bool refused = false;
  for (int s = s0; s < s1; ++s) {
    const int w = s_new[s];
    // the sequences that get pages are those whose prefix fits: a run from the front
    s_off[s] = static_cast<int>(min(off, static_cast<long long>(n_free)));
    if (w > 0) {
      off += w;
      if (off > n_free) s_new[s] = -1;
      else served = static_cast<int>(off);
    }
    if (s_new[s] < 0) {
      refused = true;
      s_rows[s] = 0;
    }
  }
  if (refused && blockIdx.x == 0) raise_flag(P.p.state + 2, kDevCapacity);
  if (served) atomicMax(&s_total, served);
  __syncthreads();
  const int N = s_total;
  // owner_of() never names a refused sequence: the first of them starts at N, the rest later.
  const int* newest = P.p.free_list + n_free - 1;  // page number i of the call is newest[-i]
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  const long long me = static_cast<long long>(blockIdx.x) * kThreads + tid;
  for (long long i = me; i < N; i += stride) {
    const int s = owner_of(s_off, batch, static_cast<int>(i));
    const int j = s_held[s] + static_cast<int>(i) - s_off[s];
    P.p.page_table[static_cast<size_t>(s) * P.p.pages_per_seq + j] = __ldcg(newest - i);
  }
  if (P.slots) {
    auto page_of = [&](int s, int j) {
      return j < s_held[s] ? __ldcg(P.p.page_table + static_cast<size_t>(s) * P.p.pages_per_seq + j)
                           : __ldcg(newest - (s_off[s] + j - s_held[s]));
    };
    const uint32_t rows = static_cast<uint32_t>(batch) * P.rows_per_seq;  // < 2^31
    const uint32_t quads = (rows + 3) / 4;
    for (uint32_t q = static_cast<uint32_t>(me); q < quads; q += static_cast<uint32_t>(stride)) {
      int s = static_cast<int>(4 * q / P.rows_per_seq), r = static_cast<int>(4 * q - static_cast<uint32_t>(s) * P.rows_per_seq);
      int slot[4], j = -1, page = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        slot[e] = -1;
        if (s < batch && r < s_rows[s]) {
          const int pos = s_len[s] + r;
          if (pos / kPagePos != j) page = page_of(s, j = pos / kPagePos);
          slot[e] = page * kPagePos + pos % kPagePos;
        }
        if (++r == P.rows_per_seq) r = 0, ++s, j = -1;
      }
      if (P.wide && 4 * q + 3 < rows) {
        *reinterpret_cast<int4*>(P.slots + 4 * static_cast<size_t>(q)) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * q + e < rows) P.slots[4 * static_cast<size_t>(q) + e] = slot[e];
      }
    }
  }
  __syncthreads();
  // every CTA has read the held counts and the list's length before the last one writes them
  if (tid == 0) {
    s_last = 1;
    if (gridDim.x > 1) {
      __threadfence();
      s_last = atomicAdd(P.p.state + 1, 1) == static_cast<int>(gridDim.x) - 1;
      __threadfence();
    }
  }
  __syncthreads();
  if (!s_last) return;
  for (int s = s0; s < s1; ++s)
    if (s_new[s] > 0) P.p.held[s] = s_held[s] + s_new[s];
  if (tid == 0) {
    P.p.state[0] = n_free - N;
    P.p.state[1] = 0;
  }
}

__global__ void __launch_bounds__(kThreads) pages_release_kernel(const PageParams P) {
  extern __shared__ int s_off[];   // [batch] number of the sequence's first released page
  int* s_drop = s_off + P.batch;   // [batch] pages it releases
  int* s_held = s_drop + P.batch;  // [batch] pages it holds
  __shared__ long long warp_sum[kThreads / 32];
  __shared__ int s_last;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, batch = P.batch;
  const int n_free = min(max(__ldcg(P.p.state), 0), P.p.n_pages);
  bool bad = false;
  for (int s = tid; s < batch; s += kThreads) {
    const int len = __ldcg(P.len + s), held = __ldcg(P.p.held + s);
    const int keep = len / kPagePos + (len % kPagePos != 0);
    const bool ok = len >= 0 && held >= 0 && held <= P.p.pages_per_seq;
    bad |= !ok;
    s_drop[s] = ok && held > keep ? held - keep : 0;
    s_held[s] = held;
  }
  __syncthreads();
  const int per = (batch + kThreads - 1) / kThreads;
  const int s0 = min(tid * per, batch), s1 = min(s0 + per, batch);
  long long mine = 0;
  for (int s = s0; s < s1; ++s) mine += s_drop[s];
  long long total;
  long long off = block_scan(mine, warp_sum, total);
  // held counts and a list that do not add up to the pool: nothing is released
  const bool broken = total > P.p.n_pages - n_free;
  if ((bad || (broken && tid == 0)) && blockIdx.x == 0) raise_flag(P.p.state + 2, kDevCapacity);
  for (int s = s0; s < s1; ++s) {
    s_off[s] = static_cast<int>(off);
    off += s_drop[s];
  }
  __syncthreads();
  const int R = broken ? 0 : static_cast<int>(total);
  const int stride = gridDim.x * kThreads;
  for (int i = blockIdx.x * kThreads + tid; i < R; i += stride) {
    const int s = owner_of(s_off, batch, i);
    const int j = s_held[s] - s_drop[s] + i - s_off[s];
    int* entry = P.p.page_table + static_cast<size_t>(s) * P.p.pages_per_seq + j;
    const int page = __ldcg(entry);
    *entry = -1;
    P.p.free_list[n_free + R - 1 - i] = page;
  }
  __syncthreads();
  if (tid == 0) {
    s_last = 1;
    if (gridDim.x > 1) {
      __threadfence();
      s_last = atomicAdd(P.p.state + 1, 1) == static_cast<int>(gridDim.x) - 1;
      __threadfence();
    }
  }
  __syncthreads();
  if (!s_last) return;
  for (int s = s0; s < s1 && !broken; ++s)
    if (s_drop[s] > 0) P.p.held[s] = s_held[s] - s_drop[s];
  if (tid == 0) {
    P.p.state[0] = n_free + R;
    P.p.state[1] = 0;
  }
}

__global__ void __launch_bounds__(kThreads) pages_init_kernel(const dflash_page_pool p) {
  pdl_wait();
  pdl_launch_dependents();
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  const long long me = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long entries = static_cast<long long>(p.max_batch) * p.pages_per_seq;
  for (long long i = me; i < p.n_pages; i += stride) p.free_list[i] = p.n_pages - 1 - static_cast<int>(i);
  for (long long i = me; i < entries; i += stride) p.page_table[i] = -1;
  for (long long i = me; i < p.max_batch; i += stride) p.held[i] = 0;
  if (me < 4) p.state[me] = me == 0 ? p.n_pages : 0;
}

bool pool_ok(const dflash_page_pool* p) {
  auto at4 = [](const void* q) { return q && (reinterpret_cast<uintptr_t>(q) & 3) == 0; };
  return p && p->n_pages >= 1 && static_cast<long long>(p->n_pages) * kPagePos < (1LL << 31) && p->pages_per_seq >= 1 &&
         static_cast<long long>(p->pages_per_seq) * kPagePos < (1LL << 31) && p->max_batch >= 1 &&
         p->max_batch <= kMaxBatch && at4(p->page_table) && at4(p->held) && at4(p->free_list) && at4(p->state);
}

// ints: the kernel's integers in shared memory for each of `batch` sequences.
template <typename K, typename A>
int launch(K kernel, long long items, int ints, int batch, const A& arg, void* stream) {
  cudaLaunchConfig_t cfg = {};
  // a thread per item up to 512 CTAs (each repeats the prefix sum), then more items a thread
  const long long ctas = (items + kThreads - 1) / kThreads;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas < 1 ? 1 : ctas > 512 ? 512 : ctas));
  const size_t smem = sizeof(int) * ints * batch;
  // With the static part past the 48 KB that need no asking. The limit belongs to the kernel, not to the
  // call: always the same one, so that host threads with pools of their own cannot lower each other's.
  if (smem > 40 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(sizeof(int)) * ints * kMaxBatch) != cudaSuccess)
    return DFLASH_E_CUDA;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, arg) == cudaSuccess ? DFLASH_OK : DFLASH_E_CUDA;
}

bool at4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

}  // namespace

}  // namespace dfl

extern "C" int dflash_pages_init(const dflash_page_pool* p, void* stream) {
  if (!dfl::pool_ok(p)) return DFLASH_E_INVAL;
  const long long entries = static_cast<long long>(p->max_batch) * p->pages_per_seq;
  return dfl::launch(dfl::pages_init_kernel, entries > p->n_pages ? entries : p->n_pages, 0, 0, *p, stream);
}

extern "C" int dflash_pages_reserve(const dflash_page_pool* p, const int32_t* len, const int32_t* n_new, int32_t batch,
                                    int32_t rows_per_seq, int32_t* slots, void* stream) {
  if (!dfl::pool_ok(p) || !len || !n_new || !dfl::at4(len) || !dfl::at4(n_new) || !dfl::at4(slots) || batch < 1 ||
      rows_per_seq < 1)
    return DFLASH_E_INVAL;
  if (batch > p->max_batch || static_cast<long long>(batch) * rows_per_seq >= (1LL << 31)) return DFLASH_E_CAPACITY;
  dfl::PageParams P{};
  P.p = *p;
  P.len = len;
  P.n_new = n_new;
  P.slots = slots;
  P.batch = batch;
  P.rows_per_seq = rows_per_seq;
  P.wide = (reinterpret_cast<uintptr_t>(slots) & 15) == 0;
  // four slots a thread; without slots, a thread for about every page
  const long long rows = static_cast<long long>(batch) * rows_per_seq;
  return dfl::launch(dfl::pages_reserve_kernel, slots ? (rows + 3) / 4 : rows / dfl::kPagePos + batch,
                     5, batch, P, stream);
}

extern "C" int dflash_pages_release(const dflash_page_pool* p, const int32_t* len, int32_t batch, void* stream) {
  if (!dfl::pool_ok(p) || !len || !dfl::at4(len) || batch < 1) return DFLASH_E_INVAL;
  if (batch > p->max_batch) return DFLASH_E_CAPACITY;
  dfl::PageParams P{};
  P.p = *p;
  P.len = len;
  P.batch = batch;
  // at most the pool's pages come back, and at most what the sequences can hold
  const long long most = static_cast<long long>(batch) * p->pages_per_seq;
  return dfl::launch(dfl::pages_release_kernel, (most < p->n_pages ? most : p->n_pages) / 2, 3, batch, P,
                     stream);
}
