// Attention with a prefix that all sequences of a batch share: the list of tiles of paged_attn.cu with the
// prefix's tiles behind the sequences' own, once for every pre_rows of the batch's new rows. Of those rows one
// product takes all query heads of a KV head, so that the prefix is read once for 64 or 128 rows
// instead of once a sequence. Own positions and prefix run in the same launch of the kernels for blocks
// (paged_attn_tc.cu, paged_attn8.cu), whose list is cut evenly whatever the two take; this file has the
// join of a row's parts, of both.
//
// Bound: the prefix's products (4 d operations a key and query row) once there are some hundred rows, else bytes.
// In 16 bits a product of 128 rows and 64 keys is 512 cycles of the tensor cores in a chain of 1900 (S, softmax, P by one
// warpgroup), so two CTAs share a SM: 1030 cycles a tile. Measured (32 query heads on 8 KV heads, d 128): 32 sequences behind 4096
// positions, one token 31 us (every sequence reading the prefix itself: 93 us); 16 behind 8190, blocks of 16 60 us (98 us);
// 64 behind 8192, blocks of 16 194 us (368 us), 697 TFLOP/s; 8 behind 131072, blocks of 16 293 us (626 us). In 8 bits 42 us (32 behind
// 8192, one token) and 107 us (16 behind 8190, blocks of 16). A sequence with more than half of an entry's rows has the entry for
// itself: in 8 bits (64 rows, or 128 for sequences of more than 64) one of more than 32 is no faster than without a prefix to share.
#include "paged_attn.cuh"

namespace dfl {

namespace {

constexpr int kJoinHeads = 8;  // query heads of a CTA, a warp each (16 x 8190, blocks of 16: 63.6 us; with 32 heads 65.7, half a wave of the CTAs idle)

// One CTA a row and 8 query heads: which ranges the row's own positions and its prefix lie in, a lane for each KV
// head and both (the divisions took most of the time when every warp made its own), then a warp a head: weights
// 2^(m - M) / sum 2^(m - M) l over the parts of its own positions, then of the prefix, each in the order of the ranges.
template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kJoinHeads) shared_join_kernel(const __grid_constant__ PagedAttnParams P, int n_ctas) {
  __shared__ int s_c0[2][kJoinHeads], s_c1[2][kJoinHeads], s_slot0[2][kJoinHeads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x, head0 = blockIdx.y * kJoinHeads, head = head0 + warp;
  const int s = row / P.rows_per_seq, r = row - s * P.rows_per_seq, g0 = head0 / P.group, tile = row / P.pre_rows;
  // With an entry a lane the list is known before the first kernel ends (it let this one start once all before it had
  // finished), and the ranges are worked out meanwhile.
  const int entries = P.batch + P.n_pre;
  if (entries > 32) pdl_wait();
  const int before = __ldcg(P.prefix_len);
  int len;
  bool bad;
  const bool there = r < rows_of(P, s, len, bad) && !no_prefix(P, before);  // the same for the whole CTA
  if (there && warp < 2) {
    const int e = warp == 0 ? s : P.batch + tile, g = g0 + lane;
    int p0, all, list;
    if (entries <= 32) {
      int l, n;
      const int mine = lane < entries ? entry_tiles(P, lane, before, false, l, n, bad) : 0;
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      p0 = __shfl_sync(0xffffffffu, upto - mine, e), all = __shfl_sync(0xffffffffu, mine, e), list = __shfl_sync(0xffffffffu, upto, 31);
    } else {
      p0 = __ldcg(P.prefix + e), all = __ldcg(P.prefix + e + 1) - p0, list = __ldcg(P.prefix + entries);
    }
    const int nt = all - P.extra;
    int c0 = 0, c1 = -1, slot0 = 0;
    if (nt > 0 && g < P.nkv) {
      const long long T = static_cast<long long>(P.nkv) * list;
      const int G = n_ranges(T, n_ctas, P.strands);
      const long long base = static_cast<long long>(P.nkv) * p0 + static_cast<long long>(g) * all;
      c0 = cta_of(base, T, G), c1 = cta_of(base + nt - 1, T, G);
      slot0 = 2 * c0 + (range_begin(c0, T, G) < base);  // c0's, of the others it is the first
    }
    if (lane < kJoinHeads) s_c0[warp][lane] = c0, s_c1[warp][lane] = c1, s_slot0[warp][lane] = slot0;
  }
  if (entries <= 32) pdl_wait();
  pdl_launch_dependents();
  if (!there) return;
  __syncthreads();
  if (head >= P.nq) return;
  const int g = head / P.group;
  const size_t slot_floats = static_cast<size_t>(P.slot_rows) * (D + 2);
  constexpr int E = D / 32, kAhead = 4;
  float acc[E] = {}, M = -INFINITY, den = 0.f;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int c0 = s_c0[which][g - g0], c1 = s_c1[which][g - g0], slot0 = s_slot0[which][g - g0];
    if (c1 < c0) continue;
    const int at = (which == 0 ? r : row - tile * P.pre_rows) * P.group + head - g * P.group;  // the row in its entry
    const bool whole = c0 == c1;
    const size_t state = state_row(P, which == 0 ? s : P.batch, row, head);
    auto slot_of = [&](int c) { return P.part + static_cast<size_t>(c == c0 ? slot0 : 2 * c) * slot_floats; };
#pragma unroll 1
    for (int b = c0; b <= c1; b += 32) {
      const int cnt = min(32, c1 - b + 1);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < cnt)
        ml = __ldcg(whole ? state_sums(P) + state
                          : reinterpret_cast<const float2*>(slot_of(b + lane) + static_cast<size_t>(P.slot_rows) * D) + at);
      float v[kAhead][E];
      auto load = [&](int k0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (k0 + k >= cnt) break;
          const float* src = (whole ? P.state + state * D : slot_of(b + k0 + k) + static_cast<size_t>(at) * D) + lane * E;
          if (E == 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
            v[k][0] = x.x, v[k][1] = x.y, v[k][E - 2] = x.z, v[k][E - 1] = x.w;
          } else {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
            v[k][0] = x.x, v[k][1] = x.y;
          }
        }
      };
      load(0);
      float top = ml.x;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = fmaxf(top, M);
      // what the parts so far weigh now: nothing where they have seen no key, as they are where all was NaN
      const float was = weight_of(make_float2(M, den), top);
      M = top;
      den = was == 0.f ? 0.f : den * was;
#pragma unroll
      for (int x = 0; x < E; ++x) acc[x] = was == 0.f ? 0.f : acc[x] * was;
      const float w = weight_of(ml, M), wl = w == 0.f ? 0.f : w * ml.y;
#pragma unroll 1
      for (int k0 = 0; k0 < cnt; k0 += kAhead) {
        if (k0 > 0) load(k0);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (k0 + k >= cnt) break;
          const float wk = __shfl_sync(0xffffffffu, w, k0 + k);
          den += __shfl_sync(0xffffffffu, wl, k0 + k);
#pragma unroll
          for (int x = 0; x < E; ++x) acc[x] = wk == 0.f ? acc[x] : fmaf(wk, v[k][x], acc[x]);
        }
      }
    }
  }
  const float inv = den > 0.f ? 1.f / den : (den == 0.f ? 0.f : den);
  uint16_t* dst = static_cast<uint16_t*>(P.out) + (static_cast<size_t>(row) * P.nq + head) * D + lane * E;
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(acc[0] * inv, acc[1] * inv), pack2<BF16>(acc[E - 2] * inv, acc[E - 1] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack2<BF16>(acc[0] * inv, acc[1] * inv);
}

template <int D, bool BF16>
int launch_join(const PagedAttnParams& p, int n_ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.batch * p.rows_per_seq, (p.nq + kJoinHeads - 1) / kJoinHeads);
  cfg.blockDim = dim3(32 * (p.nq < kJoinHeads ? (p.nq > 1 ? p.nq : 2) : kJoinHeads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, shared_join_kernel<D, BF16>, p, n_ctas));
}

}  // namespace

int launch_shared_join(const PagedAttnParams& p, bool bf16, int n_ctas, cudaStream_t stream) {
  if (p.d == 128) return bf16 ? launch_join<128, true>(p, n_ctas, stream) : launch_join<128, false>(p, n_ctas, stream);
  return bf16 ? launch_join<64, true>(p, n_ctas, stream) : launch_join<64, false>(p, n_ctas, stream);
}

// Sequences of a launch: their own entries and the prefix's, no more than these, leave room for two CTAs a SM.
int shared_batch() { return kAttnMaxBatch / 4; }

int launch_paged_attn_shared(PagedAttnParams p, int dtype, int n_ctas, cudaStream_t stream) {
  const bool bits8 = dtype == DFLASH_E4M3_F16 || dtype == DFLASH_E4M3_BF16, bf16 = dtype == DFLASH_BF16 || dtype == DFLASH_E4M3_BF16;
  // Rows of an entry: all of the batch where they are few, else as many as a product takes, and at least a sequence's own
  // (group * rows_per_seq <= 128: there are no more entries of the prefix than sequences).
  const long long all = static_cast<long long>(p.batch) * p.rows_per_seq * p.group;
  const int most = bits8 ? (p.rows <= 64 ? 64 : 128) : 128;
  const int rows = static_cast<int>(all < most ? all : most);
  p.slot_rows = bits8 ? paged_attn8_rows(rows) : rows <= 64 ? 64 : 128;
  p.strands = bits8 ? paged_attn8_strands(rows) : 1;
  p.pre_rows = p.slot_rows / p.group;
  p.n_pre = (p.batch * p.rows_per_seq + p.pre_rows - 1) / p.pre_rows;
  if (bits8) {
    p.extra = paged_attn8_extra(p.rows);
    return launch_paged_attn8(p, bf16, n_ctas, stream);
  }
  if (p.slot_rows == 128) n_ctas = 2 * n_ctas < kSharedMaxCtas ? 2 * n_ctas : kSharedMaxCtas;  // two CTAs a SM
  // With 4, 5, 6 and 8 tiles: one token of 32 sequences behind 4096 positions 32.0, 32.2, 33.3 and 34.3 us, blocks of 16 of 64
  // behind 8192 244, 224, 213 and 198 us, of 16 behind 8190 75, 69, 65 and 66 us (10: 68).
  p.extra = p.rows <= 16 ? 5 : 8;
  const int e = launch_paged_attn_tc(p, bf16, n_ctas, stream);
  return e != 0 ? e : launch_shared_join(p, bf16, n_ctas, stream);
}

}  // namespace dfl
