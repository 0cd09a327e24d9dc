// Causal attention of a few new rows per sequence over a paged K/V cache: one new token
// (decoding) or a block of up to 16 (verification).
//
//   out[s][r][h] = sum_j p_j V_j / sum_j p_j,  p_j = exp(scale q.K_j - m),  j = 0 .. len[s] + r
//
// The query heads that share a KV head and the sequence's new rows are the M rows of one
// problem (row r * group + head in group), so every K and V byte is read once for all of
// them. Bound: the K/V bytes, 4 d per key and KV head.
//
// Split. The 64-key tiles (pages) of all (sequence, KV head) pairs form one list, cut evenly
// over the CTAs (one per SM), which balances ragged lengths and splits a long cache when
// there are few sequences. A pair inside one range is finished there; of a pair that a cut
// divides each CTA leaves its unnormalised output with the rows' (max, sum), and a second
// small kernel joins those in CTA order: the result does not depend on timing, and no
// counter has to be kept between calls.
//
// CTA (up to 16 rows; more rows: paged_attn_tc.cu). One producer warp walks the range: page ids a
// warp-load at a time, K/V tiles by TMA into a ring of shared-memory stages, each segment's q
// rows by bulk copies. Of the four compute warps two take one half each of every second tile, with
// a softmax state of their own, so that warps meet only where a segment ends. S = q K^T and
// O += P V are mma.sync m16n8k16 with fp32 accumulation: the rows are few (4 in ordinary
// grouped decoding), so a 128-row tcgen05 tile would be mostly padding, while the loads bound
// the kernel: 4 rows over 4 sequences of 32768 keys take 86 us (0.92 of the measured copy rate), 32
// ragged sequences of 512 to 8192 keys 93 to 94 us (0.89 to 0.90). One sequence of 2048 takes 8.7 us:
// two launches, lengths, page ids, q, K/V, softmax, parts, one latency after another. With d 64 a tile is
// half the bytes for the same steps of the warps: 59 us (0.66), 68 us (0.61), 7.9 us.
#include "paged_attn.cuh"

namespace dfl {

namespace {

constexpr int kStep = 32;  // keys per warp step

template <bool TRANS>
DEV void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <bool BF16>
DEV void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte address of element (key, dim) in a staged tile: d / 64 boxes of 64 keys x 128 bytes,
// written by TMA with the 128-byte swizzle (16-byte chunk c of row r lands at c ^ (r & 7)).
DEV uint32_t tile_addr(uint32_t base, int key, int dim) {
  return base + (dim >> 6) * (kKeys * 128) + key * 128 + ((((dim & 63) >> 3) ^ (key & 7)) << 4) + (dim & 7) * 2;
}

DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

constexpr int kRowsFew = 16;  // rows of a problem that this kernel takes
constexpr int KG = 4;         // key groups: compute warps

template <int D>
struct Layout {
  static constexpr int STAGES = D == 128 ? 4 : 8;
  static constexpr int kThreads = 32 * (KG + 1);
  static constexpr int kRows = kRowsFew;
  static constexpr int kTileBytes = kKeys * D * 2;          // one operand
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kQStride = D * 2 + 16;               // bytes; the pad keeps ldmatrix free of conflicts
  static constexpr int kQBufs = 2;
  static constexpr int kQOff = STAGES * kStageBytes;
  static constexpr int kXOff = kQOff + kQBufs * kRows * kQStride;
  static constexpr int kMlOff = kXOff + KG * kRows * D * 4;
  static constexpr int kBarOff = kMlOff + KG * kRows * 8;   // full, empty [STAGES]; q full, q empty [kQBufs]
  static constexpr int kMetaOff = kBarOff + (2 * STAGES + 2 * kQBufs) * 8;
  static constexpr int kPreOff = kMetaOff + (STAGES + 4) * 4;  // stage valid flags, abort flag, scan scratch
  static constexpr int smem(int batch) { return 1024 + kPreOff + 64 + (3 * batch + 1) * 4; }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(Layout<D>::kThreads, 1) paged_attn_kernel(const __grid_constant__ PagedAttnParams P) {
  using L = Layout<D>;
  constexpr int STAGES = L::STAGES;
  // A stage has to serve the same two key groups every time: a group that skipped a phase of a
  // stage's barrier could take the phase before it for its own.
  static_assert(STAGES % 2 == 0, "stages of alternating tiles");
  constexpr int NT = D / 8;  // 8-dim column tiles of the output
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float4* s_x = reinterpret_cast<float4*>(smem + L::kXOff);
  float2* s_ml = reinterpret_cast<float2*>(smem + L::kMlOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* empty = full + STAGES;
  uint64_t* qfull = empty + STAGES;
  uint64_t* qempty = qfull + L::kQBufs;
  volatile int* s_valid = reinterpret_cast<volatile int*>(smem + L::kMetaOff);
  volatile int* s_abort = s_valid + STAGES;
  int* s_warp = reinterpret_cast<int*>(smem + L::kPreOff);
  int* s_pre = s_warp + 16;        // [batch + 1]
  int* s_len = s_pre + P.batch + 1;  // [batch]
  int* s_new = s_len + P.batch;      // [batch] rows of this call
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);  // the two key groups that take it
    }
    for (int i = 0; i < L::kQBufs; ++i) {
      mbar_init(&qfull[i], 1);
      mbar_init(&qempty[i], KG);
    }
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&P.kmap);
    tma_prefetch_desc(&P.vmap);
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();

  count_tiles<L::kThreads>(P, s_pre, s_len, s_new, s_warp);
  const int batch = P.batch, nkv = P.nkv, grp = P.group;
  const long long T = static_cast<long long>(nkv) * s_pre[batch];
  const int G = static_cast<int>(min(static_cast<long long>(gridDim.x), T));
  const int cta = blockIdx.x;
  if (cta >= G) return;
  const long long T0 = range_begin(cta, T, G), T1 = range_begin(cta + 1, T, G);
  // Every wait is bounded: past the limit the flag is set, later waits pass at once and the
  // CTA walks to its end without results.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_try_wait(bar, parity)) wait_long(bar, parity, s_abort, P.err, P.wait_ns);
  };

  if (warp == KG) {
    // ------------------------------------------------------------ producer warp
    // K/V are read once per call: streamed through L2, unless all of it (16 MB, one eighth of L2) can stay
    // there until it is read again. Three caches in turn, one row (us), kept and streamed: 1 x 2048 (8.4
    // MB each) 8.7 and 9.1, 1 x 3900 (16.0 MB) 9.6 and 10.4, 8 x 2048 (67 MB) 18.8 and 18.2.
    const uint64_t pol = T * L::kStageBytes > (16ll << 20) ? policy_evict_first() : policy_evict_last();
    int i = 0, seg_no = 0;
    int q_issued = 0, kv_issued = 0;  // of the segments and tiles walked so far
    for (long long u = T0; u < T1; ++seg_no) {
      const Place at = locate(s_pre, batch, nkv, u);
      const int s = at.s, g = at.g, t0 = at.t, nt = at.nt;
      const int seg = static_cast<int>(min(T1 - u, static_cast<long long>(nt - t0)));
      const int n = s_new[s];
      const int qb = seg_no % L::kQBufs;
      // page ids, one a lane: the next 32, asked for before q's copies
      auto ids = [&](int b0) { return b0 + lane < seg ? __ldcg(P.page_table + static_cast<size_t>(s) * P.pages_per_seq + t0 + b0 + lane) : 0; };
      int page = ids(0);
      if (seg_no >= L::kQBufs) wait(&qempty[qb], (seg_no / L::kQBufs - 1) & 1);
      if (__all_sync(0xffffffffu, !*s_abort)) {
        q_issued = seg_no + 1;
        if (lane == 0) mbar_arrive_expect_tx(&qfull[qb], n * grp * D * 2);
        __syncwarp();
        const uint32_t qdst = smem_u32(smem + L::kQOff + qb * L::kRows * L::kQStride);
        const uint16_t* q = static_cast<const uint16_t*>(P.q);
        for (int m = lane; m < n * grp; m += 32) {
          const int r = new_row(P, m), hh = m - r * grp;
          bulk_load(qdst + m * L::kQStride,
                    q + ((static_cast<size_t>(s) * P.rows_per_seq + r) * P.nq + static_cast<size_t>(g) * grp + hh) * D,
                    D * 2, &qfull[qb]);
        }
      }
      for (int b0 = 0; b0 < seg; b0 += 32) {
        if (b0 > 0) page = ids(b0);
        if (page < 0 || page >= P.n_pages) {
          raise_flag(P.err, kDevCapacity);
          page = -1;
        }
        const int cnt = min(32, seg - b0);
        for (int k = 0; k < cnt; ++k, ++i) {
          const int pg = __shfl_sync(0xffffffffu, page, k);
          const int st = i % STAGES;
          if (lane == 0) {
            if (i >= STAGES) wait(&empty[st], (i / STAGES - 1) & 1);
            if (!*s_abort) {
              kv_issued = i + 1;
              s_valid[st] = pg >= 0;
              if (pg >= 0) {
                uint8_t* kd = smem + st * L::kStageBytes;
                mbar_arrive_expect_tx(&full[st], L::kStageBytes);
#pragma unroll
                for (int b = 0; b < D / 64; ++b)
                  tma_load_3d(kd + b * kKeys * 128, &P.kmap, &full[st], b * 64, g, pg * kKeys, pol);
#pragma unroll
                for (int b = 0; b < D / 64; ++b)
                  tma_load_3d(kd + L::kTileBytes + b * kKeys * 128, &P.vmap, &full[st], b * 64, g, pg * kKeys, pol);
              } else {
                mbar_arrive(&full[st]);
              }
            }
          }
          __syncwarp();
        }
      }
      u += seg;
    }
    // after an abandoned wait: the copies still in flight land before the CTA leaves
    if (lane == 0 && *s_abort) {
      for (int k = max(0, kv_issued - STAGES); k < kv_issued; ++k) mbar_wait(&full[k % STAGES], (k / STAGES) & 1, P.wait_ns);
      for (int k = max(0, q_issued - L::kQBufs); k < q_issued; ++k)
        mbar_wait(&qfull[k % L::kQBufs], (k / L::kQBufs) & 1, P.wait_ns);
    }
    return;
  }

  // -------------------------------------------------------------- compute warps
  const int kg = warp;
  const int r0 = lane >> 2, kq = (lane & 3) * 2, mi = lane >> 3;
  int i = 0, seg_no = 0;
  for (long long u = T0; u < T1; ++seg_no) {
    const Place at = locate(s_pre, batch, nkv, u);
    const int s = at.s, g = at.g, t0 = at.t, nt = at.nt;
    const int seg = static_cast<int>(min(T1 - u, static_cast<long long>(nt - t0)));
    const int len = s_len[s], n_new = s_new[s];
    const int nk = len + n_new;
    int lim[2];  // last key each of the thread's rows may see
#pragma unroll
    for (int h = 0; h < 2; ++h) lim[h] = len + new_row(P, h * 8 + r0);
    const int qb = seg_no % L::kQBufs;
    wait(&qfull[qb], (seg_no / L::kQBufs) & 1);
    __syncwarp();
    uint32_t qa[D / 16][4];
    {
      const uint32_t qbase = smem_u32(smem + L::kQOff + qb * L::kRows * L::kQStride) + (lane & 15) * L::kQStride + (lane >> 4) * 16;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) ldsm4<false>(qbase + kk * 32, qa[kk]);
    }
    float o[NT][4], m_[2] = {-INFINITY, -INFINITY}, l_[2] = {0.f, 0.f};
#pragma unroll
    for (int nt2 = 0; nt2 < NT; ++nt2) o[nt2][0] = o[nt2][1] = o[nt2][2] = o[nt2][3] = 0.f;
    for (int j = 0; j < seg; ++j, ++i) {
      if ((i & 1) != kg >> 1) continue;  // the other two key groups' tile
      const int st = i % STAGES;
      wait(&full[st], (i / STAGES) & 1);
      const uint32_t kb = smem_u32(smem + st * L::kStageBytes), vb = kb + L::kTileBytes;
      // the whole warp takes the tile or skips it: the steps below are collective
      if (__all_sync(0xffffffffu, s_valid[st] != 0 && !*s_abort)) {
        const int half = kg & 1;
        const int key0 = (t0 + j) * kKeys + half * kStep;  // position of the step's first key
        if (key0 < nk) {
          const bool edge = key0 + kStep - 1 > len;  // some row may not see some key
          float sc[4][4];
#pragma unroll
          for (int n8 = 0; n8 < 4; ++n8) sc[n8][0] = sc[n8][1] = sc[n8][2] = sc[n8][3] = 0.f;
          // matrices 0..3: keys 0-7 dims lo, keys 0-7 dims hi, keys 8-15 dims lo, keys 8-15 dims hi
          const int kkey = half * kStep + (mi >> 1) * 8 + (lane & 7);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
            for (int n16 = 0; n16 < 2; ++n16) {
              uint32_t b[4];
              ldsm4<false>(tile_addr(kb, kkey + n16 * 16, kk * 16 + (mi & 1) * 8), b);
              mma16816<BF16>(sc[2 * n16], qa[kk], b[0], b[1]);
              mma16816<BF16>(sc[2 * n16 + 1], qa[kk], b[2], b[3]);
            }
          }
          // Online softmax in log2 units. The reference of a row moves only where a score passes
          // it by more than 8 (a weight is then at most 256, as exact in 16 bits as near 1), so that
          // the outputs are rarely rescaled.
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int n8 = 0; n8 < 4; ++n8)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              // (rounded here, not in one step with the base below: the maximum is of rounded scores)
              float v = __fmul_rn(sc[n8][c], P.scale_log2);
              if (edge && key0 + n8 * 8 + kq + (c & 1) > lim[c >> 1]) v = -INFINITY;
              sc[n8][c] = v;
              mx[c >> 1] = fmaxf(mx[c >> 1], v);
            }
          if (__any_sync(0xffffffffu, mx[0] > m_[0] + 8.f || mx[1] > m_[1] + 8.f)) {
            float corr[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
              mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
              const float mnew = fmaxf(m_[h], mx[h]);
              corr[h] = ex2(m_[h] - (mnew == -INFINITY ? 0.f : mnew));
              m_[h] = mnew;
              l_[h] *= corr[h];
            }
#pragma unroll
            for (int nt2 = 0; nt2 < NT; ++nt2) {
              o[nt2][0] *= corr[0];
              o[nt2][1] *= corr[0];
              o[nt2][2] *= corr[1];
              o[nt2][3] *= corr[1];
            }
          }
          const float base[2] = {m_[0] == -INFINITY ? 0.f : m_[0], m_[1] == -INFINITY ? 0.f : m_[1]};
          float ls[2] = {0.f, 0.f};
#pragma unroll
          for (int n8 = 0; n8 < 4; ++n8)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float p = ex2(sc[n8][c] - base[c >> 1]);
              sc[n8][c] = p;
              ls[c >> 1] += p;
            }
          l_[0] += ls[0];
          l_[1] += ls[1];
          // the probabilities in the cache's type for the tensor cores, at most half a step of it
          // from their fp32 values; their sum keeps fp32
          uint32_t pa[2][4];
#pragma unroll
          for (int k16 = 0; k16 < 2; ++k16) {
            pa[k16][0] = pack2<BF16>(sc[2 * k16][0], sc[2 * k16][1]);
            pa[k16][1] = pack2<BF16>(sc[2 * k16][2], sc[2 * k16][3]);
            pa[k16][2] = pack2<BF16>(sc[2 * k16 + 1][0], sc[2 * k16 + 1][1]);
            pa[k16][3] = pack2<BF16>(sc[2 * k16 + 1][2], sc[2 * k16 + 1][3]);
          }
          // O += P V. Matrices 0..3: keys 0-7 dims lo, keys 8-15 dims lo, keys 0-7 dims hi, keys 8-15 dims hi
          const int vkey = half * kStep + (mi & 1) * 8 + (lane & 7);
          if (!edge) {
#pragma unroll
            for (int k16 = 0; k16 < 2; ++k16)
#pragma unroll
              for (int dp = 0; dp < D / 16; ++dp) {
                uint32_t b[4];
                ldsm4<true>(tile_addr(vb, vkey + k16 * 16, dp * 16 + (mi >> 1) * 8), b);
                mma16816<BF16>(o[2 * dp], pa[k16], b[0], b[1]);
                mma16816<BF16>(o[2 * dp + 1], pa[k16], b[2], b[3]);
              }
          } else {
            // What lies behind the last key may be anything (0 * NaN is NaN): cleared. A key
            // that is in the cache but hidden from some row may be infinite or NaN: then the
            // step's products are taken one key at a time, for the rows that see it.
            uint32_t keep[2][2];
#pragma unroll
            for (int k16 = 0; k16 < 2; ++k16)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int key = key0 + k16 * 16 + h * 8 + kq;
                keep[k16][h] = (key < nk ? 0xffffu : 0u) | (key + 1 < nk ? 0xffff0000u : 0u);
              }
            bool odd = false;
            if (n_new > 1) {
#pragma unroll
              for (int k16 = 0; k16 < 2; ++k16)
#pragma unroll 1
                for (int dp = 0; dp < D / 16; ++dp) {
                  uint32_t b[4];
                  ldsm4<true>(tile_addr(vb, vkey + k16 * 16, dp * 16 + (mi >> 1) * 8), b);
#pragma unroll
                  for (int x = 0; x < 4; ++x) odd |= non_finite2<BF16>(b[x] & keep[k16][x & 1]);
                }
              odd = __any_sync(0xffffffffu, odd);
            }
            if (!odd) {
#pragma unroll
              for (int k16 = 0; k16 < 2; ++k16)
#pragma unroll
                for (int dp = 0; dp < D / 16; ++dp) {
                  uint32_t b[4];
                  ldsm4<true>(tile_addr(vb, vkey + k16 * 16, dp * 16 + (mi >> 1) * 8), b);
#pragma unroll
                  for (int x = 0; x < 4; ++x) b[x] &= keep[k16][x & 1];
                  mma16816<BF16>(o[2 * dp], pa[k16], b[0], b[1]);
                  mma16816<BF16>(o[2 * dp + 1], pa[k16], b[2], b[3]);
                }
            } else {
#pragma unroll 1
              for (int x = 0; x < kStep && key0 + x < nk; ++x) {
                float mine[2];  // the weights that this lane may hold of key x, by row
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float v = 0.f;
#pragma unroll
                  for (int n8 = 0; n8 < 4; ++n8)
                    if (x >> 3 == n8) v = x & 1 ? sc[n8][2 * h + 1] : sc[n8][2 * h];
                  mine[h] = v;
                }
                const int from = (lane & ~3) + ((x & 7) >> 1);
                const float p0 = __shfl_sync(0xffffffffu, mine[0], from), p1 = __shfl_sync(0xffffffffu, mine[1], from);
                const bool see0 = key0 + x <= lim[0], see1 = key0 + x <= lim[1];
#pragma unroll
                for (int nt2 = 0; nt2 < NT; ++nt2) {
                  uint32_t raw;
                  asm volatile("ld.shared.b32 %0, [%1];"
                               : "=r"(raw)
                               : "r"(tile_addr(vb, half * kStep + x, nt2 * 8 + kq))
                               : "memory");
                  const float2 v = unpack2<BF16>(raw);
                  if (see0) o[nt2][0] += p0 * v.x, o[nt2][1] += p0 * v.y;
                  if (see1) o[nt2][2] += p1 * v.x, o[nt2][3] += p1 * v.y;
                }
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&qempty[qb]);
    // row sums over the four lanes of a row
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l_[h] += __shfl_xor_sync(0xffffffffu, l_[h], 1);
      l_[h] += __shfl_xor_sync(0xffffffffu, l_[h], 2);
    }
    // ---- the key groups' states into one: o = sum_k 2^(m_k - M) o_k, l alike
    // (max, sum) of every row and group first, then the outputs, in fragment order
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if ((lane & 3) == 0) s_ml[kg * L::kRows + h * 8 + r0] = make_float2(m_[h], l_[h]);
#pragma unroll
    for (int nt2 = 0; nt2 < NT; ++nt2)
      s_x[(kg * NT + nt2) * 32 + lane] = make_float4(o[nt2][0], o[nt2][1], o[nt2][2], o[nt2][3]);
    named_bar_sync(1, 32 * KG);
    float M[2], den[2], w[KG][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = h * 8 + r0;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int k = 0; k < KG; ++k) top = fmaxf(top, s_ml[k * L::kRows + row].x);
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        const float2 ml = s_ml[k * L::kRows + row];
        w[k][h] = weight_of(ml, top);
        sum += w[k][h] == 0.f ? 0.f : w[k][h] * ml.y;
      }
      M[h] = top;
      den[h] = sum;
    }
    const bool whole = t0 == 0 && seg == nt;
    // finished rows to the output, a cut pair's to this CTA's slot
    float* slot = P.part + (2 * static_cast<size_t>(cta) + (seg_no == 0 ? 0 : 1)) * static_cast<size_t>(L::kRows) * (D + 2);
    uint16_t* dst[2];
    bool there[2];
    float inv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = h * 8 + r0, r = new_row(P, row), hh = row - r * grp;
      there[h] = row < n_new * grp;
      inv[h] = den[h] > 0.f ? 1.f / den[h] : (den[h] == 0.f ? 0.f : den[h]);
      dst[h] = static_cast<uint16_t*>(P.out) + ((static_cast<size_t>(s) * P.rows_per_seq + r) * P.nq + static_cast<size_t>(g) * grp + hh) * D;
    }
    auto put = [&](int nt2, const float (&v)[4]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!there[h]) continue;
        if (whole)
          *reinterpret_cast<uint32_t*>(dst[h] + nt2 * 8 + kq) = pack2<BF16>(v[2 * h] * inv[h], v[2 * h + 1] * inv[h]);
        else
          __stcg(reinterpret_cast<float2*>(slot + static_cast<size_t>(h * 8 + r0) * D + nt2 * 8 + kq),
                 make_float2(v[2 * h], v[2 * h + 1]));
      }
    };
    // each key group finishes its share of the columns
#pragma unroll
    for (int n4 = 0; n4 < NT / KG; ++n4) {
      const int nt2 = kg * (NT / KG) + n4;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        const float4 x = s_x[(k * NT + nt2) * 32 + lane];
        v[0] += w[k][0] * x.x;
        v[1] += w[k][0] * x.y;
        v[2] += w[k][1] * x.z;
        v[3] += w[k][1] * x.w;
      }
      put(nt2, v);
    }
    if (kg == 0 && !whole && (lane & 3) == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        __stcg(reinterpret_cast<float2*>(slot + static_cast<size_t>(L::kRows) * D) + h * 8 + r0, make_float2(M[h], den[h]));
    }
    named_bar_sync(1, 32 * KG);  // the exchange buffers are the next segment's
    u += seg;
  }
}

// ---------------------------------------------------------------- the join of cut pairs
// One warp per (pair, row): weights 2^(m_c - M) / sum_c 2^(m_c - M) l_c over the CTAs whose
// ranges the pair lies in, in CTA order.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) paged_attn_join_kernel(const __grid_constant__ PagedAttnParams P, int n_ctas, int slot_rows) {
  const int pair = blockIdx.x, s = pair / P.nkv, g = pair - s * P.nkv;
  const int lane = threadIdx.x & 31;
  const int grp = P.group;
  const int row = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  // The tiles before the pair, and its own. What the lengths say is known before the first kernel ends
  // (it let this one start once all before it had finished): with a sequence a lane, from them.
  int p0, p1, all, n_new;
  if (P.batch <= 32) {
    int len = 0, upto;
    bool bad;
    const int n = lane < P.batch ? rows_of(P, lane, len, bad) : 0;
    const int before = scan_tiles(n, len, P.extra, lane, upto);
    n_new = __shfl_sync(0xffffffffu, n, s);
    p0 = __shfl_sync(0xffffffffu, before, s);
    p1 = __shfl_sync(0xffffffffu, upto, s);
    all = __shfl_sync(0xffffffffu, upto, 31);
  } else {
    pdl_wait();
    p0 = __ldcg(P.prefix + s), p1 = __ldcg(P.prefix + s + 1), all = __ldcg(P.prefix + P.batch);
    n_new = __ldcg(P.n_new + s);
  }
  const long long T = static_cast<long long>(P.nkv) * all;
  const int nt = p1 - p0 - P.extra;
  const bool cut = nt > 0 && row < n_new * grp;
  long long base = 0;
  int G = 1, c0 = 0, c1 = 0, c0_second = 0;
  if (cut) {
    G = n_ranges(T, n_ctas, P.strands);
    base = static_cast<long long>(P.nkv) * p0 + static_cast<long long>(g) * (p1 - p0);
    c0 = cta_of(base, T, G), c1 = cta_of(base + nt - 1, T, G);
    // The pair is the first segment of every CTA whose range starts with it or inside it: of all but
    // perhaps c0. (Asking each range's start, a 64-bit division, took most of this kernel's time.)
    c0_second = range_begin(c0, T, G) < base;
  }
  if (P.batch <= 32) pdl_wait();
  pdl_launch_dependents();
  if (c0 == c1) return;
  const size_t slot_floats = static_cast<size_t>(slot_rows) * (D + 2);
  auto slot_of = [&](int c) { return P.part + (2 * static_cast<size_t>(c) + (c == c0 ? c0_second : 0)) * slot_floats; };
  constexpr int E = D / 32;  // columns of a lane
  constexpr int kAhead = 8;  // parts whose loads are in flight together
  float acc[E] = {};
  float M = -INFINITY, den = 0.f;
  for (int b = c0; b <= c1; b += 32) {
    const int cnt = min(32, c1 - b + 1);
    float v[kAhead][E];
    auto load = [&](int k0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (k0 + k >= cnt) break;
        const float* src = slot_of(b + k0 + k) + static_cast<size_t>(row) * D + lane * E;
        if (E == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
          v[k][0] = x.x, v[k][1] = x.y, v[k][E - 2] = x.z, v[k][E - 1] = x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
          v[k][0] = x.x, v[k][1] = x.y;
        }
      }
    };
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < cnt) ml = __ldcg(reinterpret_cast<const float2*>(slot_of(b + lane) + static_cast<size_t>(slot_rows) * D) + row);
    load(0);
    float top = ml.x;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(top, M);
    const float before = M == -INFINITY ? 0.f : ex2(M - top);  // what the parts so far weigh now
    M = top;
    den *= before;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= before;
    const float w = weight_of(ml, M), wl = w == 0.f ? 0.f : w * ml.y;
    for (int k0 = 0; k0 < cnt; k0 += kAhead) {
      if (k0 > 0) load(k0);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (k0 + k >= cnt) break;
        const float wk = __shfl_sync(0xffffffffu, w, k0 + k);
        den += __shfl_sync(0xffffffffu, wl, k0 + k);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += wk * v[k][e];
      }
    }
  }
  const float inv = den > 0.f ? 1.f / den : (den == 0.f ? 0.f : den);
  const int r = new_row(P, row), hh = row - r * grp;
  uint16_t* dst = static_cast<uint16_t*>(P.out) +
                  ((static_cast<size_t>(s) * P.rows_per_seq + r) * P.nq + static_cast<size_t>(g) * grp + hh) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = pack2<BF16>(acc[e] * inv, acc[e + 1] * inv);
}

template <int D, bool BF16>
int set_attr() {
  static_assert(Layout<D>::smem(kAttnMaxBatch) <= 232448, "shared memory of a CTA");
  return static_cast<int>(cudaFuncSetAttribute(paged_attn_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Layout<D>::smem(kAttnMaxBatch)));
}

template <int D, bool BF16>
int launch(const PagedAttnParams& p, int n_ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_ctas);
  cfg.blockDim = dim3(Layout<D>::kThreads);
  cfg.dynamicSmemBytes = Layout<D>::smem(p.batch);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Up to the 16 rows of an mma.sync tile here, more on tcgen05. Measured (bf16, d 128, 32 query heads on
  // 8 KV heads, us):
  //   rows  1 x 2048  32 x 1000  4 x 32768       1 x 2048  32 x 1000  4 x 32768
  //      4       8.7       27.6       85.6  here     11.1       29.1       86.2  tcgen05
  //      8      10.8       29.1       86.0  here     13.4       31.3       88.5  tcgen05
  //     16      11.1       30.3       86.0  here     14.3       32.8       89.8  tcgen05
  //     20                                           14.6       34.3       90.5  tcgen05
  const int e = p.rows <= kRowsFew ? static_cast<int>(cudaLaunchKernelEx(&cfg, paged_attn_kernel<D, BF16>, p))
                                   : launch_paged_attn_tc(p, BF16, n_ctas, stream);
  return e != 0 ? e : launch_paged_attn_join(p, BF16, n_ctas, stream);
}

template <int D, bool BF16>
int launch_join(const PagedAttnParams& p, int n_ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.batch * p.nkv, (p.rows + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, paged_attn_join_kernel<D, BF16>, p, n_ctas, p.slot_rows));
}

}  // namespace

int paged_attn_rows(int rows) { return rows <= kRowsFew ? kRowsFew : rows <= 64 ? 64 : 128; }

int paged_attn_set_attributes() {
  const int e[] = {set_attr<64, false>(), set_attr<64, true>(), set_attr<128, false>(), set_attr<128, true>(),
                   paged_attn_tc_set_attributes()};
  for (int x : e)
    if (x != 0) return x;
  return 0;
}

int launch_paged_attn_join(const PagedAttnParams& p, bool bf16, int n_ctas, cudaStream_t stream) {
  if (p.d == 128) return bf16 ? launch_join<128, true>(p, n_ctas, stream) : launch_join<128, false>(p, n_ctas, stream);
  return bf16 ? launch_join<64, true>(p, n_ctas, stream) : launch_join<64, false>(p, n_ctas, stream);
}

int launch_paged_attn(const PagedAttnParams& p, bool bf16, int n_ctas, cudaStream_t stream) {
  if (p.batch < 1 || p.batch > kAttnMaxBatch || n_ctas < 1 || n_ctas > kPagedMaxCtas || p.rows > 128)
    return static_cast<int>(cudaErrorInvalidValue);
  if (p.d == 128) return bf16 ? launch<128, true>(p, n_ctas, stream) : launch<128, false>(p, n_ctas, stream);
  return bf16 ? launch<64, true>(p, n_ctas, stream) : launch<64, false>(p, n_ctas, stream);
}

}  // namespace dfl
