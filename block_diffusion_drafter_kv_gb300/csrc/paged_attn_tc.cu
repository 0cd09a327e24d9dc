// The attention over a paged cache on the tcgen05 tensor cores, for problems of more than 16
// rows (a block to verify times the query heads of a KV head), whose mma.sync form was bound by
// its fragments' trips through ldmatrix. The same list of tiles, cut and parts as in
// paged_attn.cu, whose join follows.
//
// Bound: the K/V bytes. A step takes two tiles (128 keys) where the rows are at most 64: S = Q K^T
// is one M = 128, N = 128 product with the rows twice in Q, once for each tile, so that all
// 128 lanes of the softmax have a row of 64 scores; P keeps zeros where a row's other tile is, and
// O += P V (M = 128, K = 128 keys) adds up two states per row, which meet at the segment's
// end. With 65 to 128 rows a step is one tile. Measured (bf16, 32 query heads on 8 KV heads, 4
// sequences of 32768, d 128): 90 us with 20 rows, 97 with 64 (81% of the copy rate), 119 with 128;
// against a two-tile step's 2750 cycles of HBM time (64 KB) issuing its products takes 1250 and its
// softmax 1100, overlapped between steps, so that it waits for copies; a one-tile step (1400 cycles of
// HBM time) waits for the chain of its products and softmax (1700), d 64 likewise (75 us with 64 rows, 53%).
// Short caches (128 sequences of 500: 117 us with 64 rows, 38%, 168 us with 128 rows, 29%) are bound by the
// segments' ends: q, output.
//
//   S   two TMEM buffers of N columns: the next step's Q K^T runs under this one's softmax
//   Q, P  in TMEM too, as the products' A operands: with them in shared memory (64 KB) the rings
//       held two steps instead of three, and a step waited for its copies (104 us against 99 then
//       at 4 sequences of 32768, 64 rows)
//   O   TMEM, kept over the segment. A row's reference moves only where a score passes it by more
//       than 8 binary orders; that row of O is then rescaled in TMEM between two products
//   K, V  rings of their own: a K stage is free after its Q K^T, a V stage after its P V
// The next segment's q is fetched while a segment ends (the producer has asked for it in L2
// when it began the segment's copies), so that its first product runs under the output.
// Warps 0-3: softmax and output, a row per thread; warp 4: MMA issuer; warp 5: producer. Every
// wait is bounded; past the limit the later ones pass at once and the softmax warps walk to
// the end without results, so that none of their barriers and collective steps is missed.
//
// Keys that are hidden: weights 0. What lies behind a sequence's last key is cleared in the V
// stage before the product, and so is a dropped page (0 * NaN is NaN). The new rows' own keys, of
// which some rows see some, may hold infinities or NaN: if one does, those keys of the step leave
// the product (V cleared, weight 0), their values and the rows' scores are kept, and they are added
// row by row at the segment's end.
#include "paged_attn.cuh"

namespace dfl {

namespace {

// ---------------------------------------------------------------- tensor memory, descriptors
// D[tmem] (+)= A[tmem] * B[smem]: A is a row per lane, two 16-bit values to a column.
DEV void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// kind::f16: fp32 accumulator, both operands fp16 or both bf16, A K-major, B K-major or MN-major.
constexpr uint32_t idesc_f32(bool bf16, int M, int N, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// An MN-major operand in 128-byte rows of 64 consecutive MN elements, one row per K index, 8 rows
// to a 1024-byte swizzle atom; the next 64 MN elements lie `mn_stride` bytes further on.
DEV uint64_t desc_mn_sw128(uint32_t saddr, uint32_t mn_stride) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((mn_stride >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// Byte offset of 16-byte chunk `ch` of row `r` in a 128-byte-swizzled box.
DEV uint32_t sw128(int r, int ch) { return static_cast<uint32_t>(r * 128 + ((ch ^ (r & 7)) << 4)); }

DEV void tmem_load16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
DEV void tmem_store16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Whether a phase is complete, without the suspension that a try_wait may take: for a thread that
// watches several barriers.
DEV bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
DEV void tmem_wait_loads() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
DEV void tmem_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

constexpr int kLanes = 128;          // rows of the products
constexpr int kTcThreads = 192;
constexpr float kMove = 8.f;         // log2 growth of a row's maximum that moves its reference
constexpr int kNewKeys = 16;         // new rows' keys at most

// D: head dim; H: tiles a step takes (2: at most 64 rows; 1: at most 128).
template <int D, int H>
struct TcLayout {
  static constexpr int kRows = kLanes / H;                 // rows of a problem
  static constexpr int kN = 64 * H;                        // keys of a step
  static constexpr int kTile = kKeys * 128;                // one 64-dim box of one tile
  static constexpr int kBox = H * kTile;                   // of a step's tiles
  static constexpr int kOperand = D / 64 * kBox;           // K, or V, of a step
  static constexpr int kSlots = D == 128 ? (H == 2 ? 3 : 6) : (H == 2 ? 6 : 8);  // of each ring
  static constexpr int kK = 0;
  static constexpr int kV = kK + kSlots * kOperand;
  static constexpr int kZ = kV + kSlots * kOperand;        // values of new keys that left the products
  static constexpr int kZs = kZ + kNewKeys * D * 2;        // their scores [128][16]
  static constexpr int kX = kZs + kLanes * kNewKeys * 4;   // outputs that meet at a segment's end: two rounds of 16 columns
  static constexpr int kMl = kX + (H == 2 ? 8192 : 0);     // and their (max, sum)
  static constexpr int kBar = kMl + kLanes * 8;
  static constexpr int kBars = 4 * kSlots + 2 + 2 + 4;     // K full, empty; V full, empty; S ready, free [2]; P, PV, Q, done
  static constexpr int kFlags = kBar + kBars * 8;          // [0] abort, [1] TMEM base, [2..3] odd values, [4..19] valid tiles of steps
  static constexpr int kWarpSums = kFlags + 80;
  static constexpr int kPre = kWarpSums + 32;
  static constexpr int smem(int batch) { return 1024 + kPre + (3 * batch + 1) * 4; }
  static constexpr uint32_t kS = 0, kO = 256, kQ = 384, kP = 448;  // TMEM columns: S buffers at 0 and kN
};

template <int D, bool BF16, int H>
__global__ void __launch_bounds__(kTcThreads, 1) paged_attn_tc_kernel(const __grid_constant__ PagedAttnParams P) {
  using L = TcLayout<D, H>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* kempty = kfull + L::kSlots;
  uint64_t* vfull = kempty + L::kSlots;
  uint64_t* vempty = vfull + L::kSlots;
  uint64_t* sready = vempty + L::kSlots;
  uint64_t* sfree = sready + 2;
  uint64_t* pready = sfree + 2;
  uint64_t* pvdone = pready + 1;
  uint64_t* qready = pvdone + 1;
  uint64_t* mdone = qready + 1;
  volatile int* flag = reinterpret_cast<volatile int*>(smem + L::kFlags);
  volatile int* s_odd = flag + 2;    // a new key of the step holds an infinity or NaN; by step mod 2
  volatile int* s_valid = flag + 4;  // bit h: tile h of the step is there; by step mod 16, more than the rings hold
  int* s_warp = reinterpret_cast<int*>(smem + L::kWarpSums);
  int* s_pre = reinterpret_cast<int*>(smem + L::kPre);
  int* s_len = s_pre + P.batch + 1;
  int* s_new = s_len + P.batch;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t WL = P.wait_ns;

  if (tid == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(&kfull[i], 1);
      mbar_init(&kempty[i], 1);
      mbar_init(&vfull[i], 1);
      mbar_init(&vempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sready[i], 1);
      mbar_init(&sfree[i], kLanes);
    }
    mbar_init(pready, kLanes);
    mbar_init(pvdone, 1);
    mbar_init(qready, kLanes);
    mbar_init(mdone, 1);
    flag[0] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&P.kmap);
    tma_prefetch_desc(&P.vmap);
  }
  pdl_wait();
  pdl_launch_dependents();
  count_tiles<kTcThreads>(P, s_pre, s_len, s_new, s_warp);
  const int batch = P.batch, nkv = P.nkv, grp = P.group;
  const long long T = static_cast<long long>(nkv) * s_pre[batch];
  const int G = static_cast<int>(min(static_cast<long long>(gridDim.x), T));
  const int cta = blockIdx.x;
  if (cta >= G) return;  // the whole CTA, before it holds any tensor memory
  if (warp == 4) tmem_alloc(reinterpret_cast<uint32_t*>(smem + L::kFlags + 4), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(flag[1]);
  const long long T0 = range_begin(cta, T, G), T1 = range_begin(cta + 1, T, G);

  // The walk of every role: steps of up to H tiles of the segments of [T0, T1).
  struct Walk {
    long long u;
    int left;    // tiles of the segment that are left
    Place at;    // of the next tile
  };
  auto begin_segment = [&](Walk& w) {
    w.at = locate(s_pre, batch, nkv, w.u);
    w.left = static_cast<int>(min(T1 - w.u, static_cast<long long>(w.at.nt - w.at.t)));
  };

  if (warp == 5) {
    // ------------------------------------------------------------------ producer
    const uint64_t pol = T * (D * 256) > (16ll << 20) ? policy_evict_first() : policy_evict_last();
    int i = 0;       // step
    bool go = true;  // the same in every lane
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      bool ok = go && !flag[0];
      if (ok && lane == 0 && !mbar_wait(bar, parity, WL)) {
        raise_flag(P.err, kDevTimeout);
        flag[0] = 1;
        ok = false;
      }
      go = __all_sync(0xffffffffu, ok);
    };
    Walk w{T0, 0, {}};
    int ids = -1;           // page ids of the segment's next tiles, one a lane
    int id0 = 0;            // lane that has the next one
    while (w.u < T1 && go) {
      if (w.left == 0) {
        begin_segment(w);
        id0 = 32;
        if (lane < s_new[w.at.s])  // the segment's q, a new row a lane
          bulk_prefetch_l2(static_cast<const uint16_t*>(P.q) +
                               ((static_cast<size_t>(w.at.s) * P.rows_per_seq + lane) * P.nq + static_cast<size_t>(w.at.g) * grp) * D,
                           grp * D * 2);
      }
      int page[2] = {-1, -1};
      const int cnt = min(H, w.left);
      for (int h = 0; h < cnt; ++h) {
        if (id0 == 32) {
          ids = -1;
          if (lane < w.left - h) {
            ids = __ldcg(P.page_table + static_cast<size_t>(w.at.s) * P.pages_per_seq + w.at.t + h + lane);
            if (ids < 0 || ids >= P.n_pages) {
              raise_flag(P.err, kDevCapacity);
              ids = -1;
            }
          }
          id0 = 0;
        }
        page[h] = __shfl_sync(0xffffffffu, ids, id0++);
      }
      const int st = i % L::kSlots;
      const uint32_t bytes = ((page[0] >= 0) + (page[1] >= 0)) * D * 128;  // of K, and of V
      uint8_t* kd = smem + L::kK + st * L::kOperand;
      uint8_t* vd = smem + L::kV + st * L::kOperand;
      if (i >= L::kSlots) wait(&kempty[st], (i / L::kSlots - 1) & 1);
      if (!go) break;
      if (lane == 0) {
        s_valid[i & 15] = (page[0] >= 0) | (page[1] >= 0) << 1;
        if (bytes) mbar_arrive_expect_tx(&kfull[st], bytes);
        else mbar_arrive(&kfull[st]);
#pragma unroll
        for (int h = 0; h < H; ++h)
          if (page[h] >= 0)
#pragma unroll
            for (int b = 0; b < D / 64; ++b)
              tma_load_3d(kd + b * L::kBox + h * L::kTile, &P.kmap, &kfull[st], b * 64, w.at.g, page[h] * kKeys, pol);
      }
      __syncwarp();
      if (i >= L::kSlots) wait(&vempty[st], (i / L::kSlots - 1) & 1);
      if (!go) {
        // K's copy of this step is in flight and V's is not: its slot's barrier never completes
        if (lane == 0) mbar_wait(&kfull[st], (i / L::kSlots) & 1, WL);
        break;
      }
#pragma unroll
      for (int h = 0; h < H; ++h)
        if (page[h] < 0) {  // no such tile: its values are cleared
          for (int k = lane; k < D / 64 * kKeys * 8; k += 32)
            *reinterpret_cast<uint4*>(vd + k / (kKeys * 8) * L::kBox + h * L::kTile + k % (kKeys * 8) * 16) = uint4{0, 0, 0, 0};
        }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        if (bytes) mbar_arrive_expect_tx(&vfull[st], bytes);
        else mbar_arrive(&vfull[st]);
#pragma unroll
        for (int h = 0; h < H; ++h)
          if (page[h] >= 0)
#pragma unroll
            for (int b = 0; b < D / 64; ++b)
              tma_load_3d(vd + b * L::kBox + h * L::kTile, &P.vmap, &vfull[st], b * 64, w.at.g, page[h] * kKeys, pol);
      }
      __syncwarp();
      ++i;
      w.u += cnt;
      w.left -= cnt;
      w.at.t += cnt;
    }
    // every copy issued has landed before the CTA leaves
    if (lane == 0)
      for (int k = max(0, i - L::kSlots); k < i; ++k) {
        mbar_wait(&kfull[k % L::kSlots], (k / L::kSlots) & 1, WL);
        mbar_wait(&vfull[k % L::kSlots], (k / L::kSlots) & 1, WL);
      }
    __syncwarp();
  } else if (warp == 4) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t kQk = idesc_f32(BF16, kLanes, L::kN, false), kPv = idesc_f32(BF16, kLanes, D, true);
      auto qk = [&](int i) {  // S[i & 1] = Q K^T
        const int st = i % L::kSlots;
        tc_fence_after();
        // one descriptor and constant steps of its address field: building each one took longer
        // than the product it describes
        const uint64_t k0 = smem_desc_k_sw128(smem_u32(smem + L::kK + st * L::kOperand));
        const uint32_t d = tmem + L::kS + (i & 1) * L::kN;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ts(d, tmem + L::kQ + kk * 8, k0 + (((kk >> 2) * L::kBox + (kk & 3) * 32) >> 4), kQk, kk > 0 ? 1u : 0u);
        tc_commit(&sready[i & 1]);
        tc_commit(&kempty[st]);
      };
      auto pv = [&](int i, bool first) {  // O (+)= P V
        const int st = i % L::kSlots;
        tc_fence_after();
        const uint64_t v0 = desc_mn_sw128(smem_u32(smem + L::kV + st * L::kOperand), L::kBox);
#pragma unroll
        for (int kk = 0; kk < L::kN / 16; ++kk)
          mma_ts(tmem + L::kO, tmem + L::kP + kk * 8, v0 + (kk * 2048 >> 4), kPv, (kk > 0 || !first) ? 1u : 0u);
        tc_commit(pvdone);
        tc_commit(&vempty[st]);
      };
      // Whichever product's inputs are ready goes next, so that neither waits behind the other's.
      Walk w{T0, 0, {}};
      int nqk = 0, npv = 0, segs = 0;
      bool first_of[4] = {};
      uint64_t idle_since = 0;
      uint32_t spins = 0;
      bool start = true;
      while (w.u < T1 || npv < nqk) {
        bool moved = false;
        if (w.u < T1 && nqk <= npv + 2) {
          if (w.left == 0) {
            begin_segment(w);
            start = true;
          }
          if (mbar_test(&kfull[nqk % L::kSlots], (nqk / L::kSlots) & 1) &&
              (nqk < 2 || mbar_test(&sfree[nqk & 1], ((nqk >> 1) - 1) & 1)) && (!start || mbar_test(qready, segs & 1))) {
            qk(nqk);
            first_of[nqk & 3] = start;
            segs += start;
            start = false;
            const int cnt = min(H, w.left);
            w.u += cnt;
            w.left -= cnt;
            ++nqk;
            moved = true;
          }
        }
        if (npv < nqk && mbar_test(pready, npv & 1) && mbar_test(&vfull[npv % L::kSlots], (npv / L::kSlots) & 1)) {
          pv(npv, first_of[npv & 3]);
          ++npv;
          moved = true;
        }
        // (reading the timer takes some 600 cycles: only where nothing has moved for a while)
        if (moved) {
          spins = 0;
        } else if ((++spins & 1023u) == 0) {
          const uint64_t now = globaltimer_ns();
          if (spins == 1024) idle_since = now;
          if (flag[0] || now - idle_since > WL) {
            if (!flag[0]) raise_flag(P.err, kDevTimeout);
            flag[0] = 1;
            break;
          }
        }
      }
      tc_commit(mdone);
      if (!mbar_wait(mdone, 0, WL)) raise_flag(P.err, kDevTimeout);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax and output
    const int hh = H == 2 ? tid >> 6 : 0;        // which of the step's tiles the thread's row takes
    const int row = H == 2 ? tid & 63 : tid;     // row of the problem
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t orow = tmem + lanes + L::kO;
    float* s_z = reinterpret_cast<float*>(smem + L::kZs) + tid * kNewKeys;
    float2* s_ml = reinterpret_cast<float2*>(smem + L::kMl);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!mbar_try_wait(bar, parity)) wait_long(bar, parity, flag, P.err, WL);
      __syncwarp();
    };
    // a segment's row of q; rows that are not there are zero
    uint4 qrow[D / 8];
    auto load_q = [&](const Place& p) {
      const int r = new_row(P, row);
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(P.q) +
          ((static_cast<size_t>(p.s) * P.rows_per_seq + r) * P.nq + p.g * grp + row - r * grp) * D);
      const bool there = row < s_new[p.s] * grp;
#pragma unroll
      for (int ch = 0; ch < D / 8; ++ch) qrow[ch] = there ? __ldcg(src + ch) : make_uint4(0, 0, 0, 0);
    };
    auto store_q = [&]() {  // once the products with the q before it are done
      __syncwarp();
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t u[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 v = qrow[c * 4 + k];
          u[4 * k] = v.x, u[4 * k + 1] = v.y, u[4 * k + 2] = v.z, u[4 * k + 3] = v.w;
        }
        tmem_store16(tmem + lanes + L::kQ + c * 16, u);
      }
      tmem_wait_stores();
      tc_fence_before();
      mbar_arrive(qready);
    };
    if (H == 2) {  // the weights of the other tile's keys stay zero
      const uint32_t zero[16] = {};
      tmem_store16(tmem + lanes + L::kP + (1 - hh) * 32, zero);
      tmem_store16(tmem + lanes + L::kP + (1 - hh) * 32 + 16, zero);
    }
    int i = 0, seg_no = 0;
    Walk w{T0, 0, {}};
    begin_segment(w);
    load_q(w.at);
    store_q();
    for (; w.u < T1; ++seg_no) {
      const int s = w.at.s, g = w.at.g, t0 = w.at.t;
      const bool whole = t0 == 0 && w.left == w.at.nt;
      const int len = s_len[s], n_new = s_new[s], nk = len + n_new;
      const int r = new_row(P, row), head = g * grp + row - r * grp;
      const bool there = row < n_new * grp;
      const int lim = len + r;  // last key the row may see
      float m = -INFINITY, l = 0.f;
      uint32_t kept = 0;  // new keys whose values are added at the end
      bool first = true, huge = false;
      for (; w.left > 0; ++i, first = false) {
        const int cnt = min(H, w.left), t = w.at.t + hh;
        w.u += cnt;
        w.left -= cnt;
        w.at.t += cnt;
        wait(&sready[i & 1], (i >> 1) & 1);
        tc_fence_after();
        float sc[64];
        {
          uint32_t u[4][16];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_load16(tmem + lanes + L::kS + (i & 1) * L::kN + hh * 64 + c * 16, u[c]);
          tmem_wait_loads();
#pragma unroll
          for (int k = 0; k < 64; ++k) sc[k] = __uint_as_float(u[k >> 4][k & 15]);
        }
        tc_fence_before();
        mbar_arrive(&sfree[i & 1]);
        const bool valid = s_valid[i & 15] >> hh & 1;
        const int key0 = t * kKeys;
        const bool edge = (w.at.t * kKeys) > len + 1;  // some row may not see some key of the step (the same for all threads)
        if (!valid || edge) {
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (!valid || key0 + k > lim) sc[k] = -INFINITY;
        }
        // one warp to a scheduler: four chains, not one
        float top[4] = {sc[0], sc[1], sc[2], sc[3]};
#pragma unroll
        for (int k = 4; k < 64; ++k) top[k & 3] = fmaxf(top[k & 3], sc[k]);
        // (a rounded product: wherever it is used, it is the same number)
        const float mx = __fmul_rn(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), P.scale_log2);
        const bool need = mx > m + kMove;
        if (__any_sync(0xffffffffu, need)) {
          const float corr = need && !first ? ex2(m - mx) : 1.f;
          if (!first) {  // that row of O in TMEM, once the products so far are done
            wait(pvdone, (i - 1) & 1);
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t u[16];
              tmem_load16(orow + c * 16, u);
              tmem_wait_loads();
#pragma unroll
              for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * corr);
              tmem_store16(orow + c * 16, u);
            }
            tmem_wait_stores();
            tc_fence_before();
          }
          if (need) {
            l *= corr;
            m = mx;
          }
          huge = __any_sync(0xffffffffu, fabsf(m) > 1048576.f && fabsf(m) < INFINITY);
        }
        if (edge) {
          // The step's V rows behind the last key are cleared; new keys are looked through, a key
          // a thread (with two tiles every thread has one, with one the first 64).
          const int vk = H == 2 ? tid & 63 : tid;  // key in the thread's tile
          const int vkey = key0 + vk;
          const bool mine = vk < kKeys && valid;
          uint8_t* vrow = smem + L::kV + (i % L::kSlots) * L::kOperand + hh * L::kTile;
          wait(&vfull[i % L::kSlots], (i / L::kSlots) & 1);
          if (tid == 0) s_odd[i & 1] = 0;
          named_bar_sync(2, kLanes);
          if (mine && vkey >= len && vkey < nk && n_new > 1) {
            bool odd = false;
#pragma unroll 4
            for (int ch = 0; ch < D / 8; ++ch) {
              const uint4 v = *reinterpret_cast<const uint4*>(vrow + (ch >> 3) * L::kBox + sw128(vk, ch & 7));
              odd |= non_finite2<BF16>(v.x) || non_finite2<BF16>(v.y) || non_finite2<BF16>(v.z) || non_finite2<BF16>(v.w);
            }
            if (odd) s_odd[i & 1] = 1;
          }
          named_bar_sync(2, kLanes);
          const bool odd = s_odd[i & 1] != 0;
          if (mine && (vkey >= nk || (odd && vkey >= len))) {
#pragma unroll 4
            for (int ch = 0; ch < D / 8; ++ch) {
              uint4* at = reinterpret_cast<uint4*>(vrow + (ch >> 3) * L::kBox + sw128(vk, ch & 7));
              if (vkey < nk) *reinterpret_cast<uint4*>(smem + L::kZ + (vkey - len) * (D * 2) + ch * 16) = *at;
              *at = make_uint4(0, 0, 0, 0);
            }
          }
          if (odd && valid) {  // (a tile of another CTA's has its new keys looked after there)
            const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int k = 0; k < 64; ++k) {
              const int key = key0 + k;
              if (key < len || key >= nk) continue;
              // The rounded product for the sum here and for the weight at the segment's end: a product
              // fused with the subtraction would differ from it by the product's rounding.
              const float z = __fmul_rn(sc[k], P.scale_log2);
              s_z[key - len] = z;
              kept |= 1u << (key - len);
              l += ex2(z - base);
              sc[k] = -INFINITY;
            }
          }
        }
        {
          const float base = m == -INFINITY ? 0.f : m;
          // One rounding of score times scale less base. Past 2^20 the base's own rounding would show
          // in it (a weight of 2^32 at scores of 2^30): there the product is rounded as the base was.
          if (huge)
#pragma unroll
            for (int k = 0; k < 64; ++k) sc[k] *= P.scale_log2;
          const float scale = huge ? 1.f : P.scale_log2;
          const float2 scale2 = {scale, scale}, base2 = {-base, -base};
          float2 ls[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
          for (int k = 0; k < 64; k += 2) {
            const float2 x = fma2(float2{sc[k], sc[k + 1]}, scale2, base2);
            sc[k] = ex2(x.x);
            sc[k + 1] = ex2(x.y);
            ls[k >> 1 & 1] = add2(ls[k >> 1 & 1], float2{sc[k], sc[k + 1]});
          }
          ls[0] = add2(ls[0], ls[1]);
          l += ls[0].x + ls[0].y;
        }
        // P, once the previous step's product has read it
        if (i > 0) wait(pvdone, (i - 1) & 1);
        __syncwarp();
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t u[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) u[k] = pack2<BF16>(sc[32 * c + 2 * k], sc[32 * c + 2 * k + 1]);
          tmem_store16(tmem + lanes + L::kP + hh * 32 + c * 16, u);
        }
        tmem_wait_stores();
        fence_async_shared();  // (cleared values)
        tc_fence_before();
        mbar_arrive(pready);
      }
      // the next segment's q: every score of this one has been read
      const bool more = w.u < T1;
      if (more) {
        begin_segment(w);
        load_q(w.at);
        store_q();
      }
      wait(pvdone, (i - 1) & 1);
      tc_fence_after();
      // ---- the row's state out: with two tiles a step its two halves meet through P's buffer
      float M = m, w_own = 1.f, den = l;
      s_ml[tid] = make_float2(m, l);
      named_bar_sync(1, kLanes);
      if (H == 2) {
        const float2 a = s_ml[row], b = s_ml[row + 64];
        M = fmaxf(a.x, b.x);
        const float wa = weight_of(a, M), wb = weight_of(b, M);
        den = (wa == 0.f ? 0.f : wa * a.y) + (wb == 0.f ? 0.f : wb * b.y);
        w_own = hh == 0 ? wa : wb;
      }
      auto load_o = [&](int c, float (&o)[16]) {  // 16 columns of the thread's row, with the new keys that left the products
        uint32_t u[16];
        __syncwarp();
        tmem_load16(orow + c * 16, u);
        tmem_wait_loads();
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = __uint_as_float(u[k]);
        for (uint32_t rest = kept; rest; rest &= rest - 1) {
          const int z = __ffs(rest) - 1;
          if (len + z > lim) continue;
          const float p = ex2(s_z[z] - (m == -INFINITY ? 0.f : m));
          const uint32_t* v = reinterpret_cast<const uint32_t*>(smem + L::kZ + z * (D * 2) + c * 32);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 f = unpack2<BF16>(v[k]);
            o[2 * k] += p * f.x;
            o[2 * k + 1] += p * f.y;
          }
        }
      };
      const float inv = den > 0.f ? 1.f / den : (den == 0.f ? 0.f : den);
      float* slot = P.part + (2 * static_cast<size_t>(cta) + (seg_no == 0 ? 0 : 1)) * static_cast<size_t>(L::kRows) * (D + 2);
      uint16_t* dst = static_cast<uint16_t*>(P.out) + ((static_cast<size_t>(s) * P.rows_per_seq + r) * P.nq + head) * D;
      auto put = [&](int c, const float (&o)[16]) {
        if (!there) return;
        if (whole) {
          uint4 v[2];
          uint32_t* b = reinterpret_cast<uint32_t*>(v);
#pragma unroll
          for (int k = 0; k < 8; ++k) b[k] = pack2<BF16>(o[2 * k] * inv, o[2 * k + 1] * inv);
          *reinterpret_cast<uint4*>(dst + c * 16) = v[0];
          *reinterpret_cast<uint4*>(dst + c * 16 + 8) = v[1];
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            __stcg(reinterpret_cast<float4*>(slot + static_cast<size_t>(row) * D + c * 16 + 4 * q),
                   make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]));
        }
      };
      if (H == 2) {
        // each half of the rows' threads finishes half of the columns, 16 a round, with the other's from shared memory
        float4* xch = reinterpret_cast<float4*>(smem + L::kX);  // [2 halves][4][64 rows]
        const float w_other = weight_of(s_ml[tid ^ 64], M);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          const int own = hh * (D / 32) + c, other = (1 - hh) * (D / 32) + c;
          float o[16];
          load_o(other, o);
#pragma unroll
          for (int q = 0; q < 4; ++q) xch[(hh * 4 + q) * 64 + row] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          load_o(own, o);
          named_bar_sync(1, kLanes);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 x = xch[((1 - hh) * 4 + q) * 64 + row];
            o[4 * q] = o[4 * q] * w_own + x.x * w_other;
            o[4 * q + 1] = o[4 * q + 1] * w_own + x.y * w_other;
            o[4 * q + 2] = o[4 * q + 2] * w_own + x.z * w_other;
            o[4 * q + 3] = o[4 * q + 3] * w_own + x.w * w_other;
          }
          put(own, o);
          named_bar_sync(1, kLanes);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          float o[16];
          load_o(c, o);
          put(c, o);
        }
      }
      if (hh == 0 && there && !whole)
        __stcg(reinterpret_cast<float2*>(slot + static_cast<size_t>(L::kRows) * D) + row, make_float2(M, den));
      tc_fence_before();
      named_bar_sync(1, kLanes);  // the exchange buffers are the next segment's
    }
  }

  // ---- every product has completed (the issuer waited for them) before the tensor memory goes
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool BF16, int H>
int set_tc_attr() {
  static_assert(TcLayout<D, H>::smem(kAttnMaxBatch) <= 232448, "shared memory of a CTA");
  return static_cast<int>(cudaFuncSetAttribute(paged_attn_tc_kernel<D, BF16, H>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               TcLayout<D, H>::smem(kAttnMaxBatch)));
}
template <int D, bool BF16, int H>
int launch_tc(const PagedAttnParams& p, int n_ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_ctas);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = TcLayout<D, H>::smem(p.batch);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, paged_attn_tc_kernel<D, BF16, H>, p));
}

}  // namespace

int paged_attn_tc_set_attributes() {
  const int e[] = {set_tc_attr<64, false, 1>(),  set_tc_attr<64, false, 2>(),  set_tc_attr<64, true, 1>(),  set_tc_attr<64, true, 2>(),
                   set_tc_attr<128, false, 1>(), set_tc_attr<128, false, 2>(), set_tc_attr<128, true, 1>(), set_tc_attr<128, true, 2>()};
  for (int x : e)
    if (x != 0) return x;
  return 0;
}

int launch_paged_attn_tc(const PagedAttnParams& p, bool bf16, int n_ctas, cudaStream_t stream) {
  const bool two = p.rows <= 64;
  if (p.d == 128) {
    if (bf16) return two ? launch_tc<128, true, 2>(p, n_ctas, stream) : launch_tc<128, true, 1>(p, n_ctas, stream);
    return two ? launch_tc<128, false, 2>(p, n_ctas, stream) : launch_tc<128, false, 1>(p, n_ctas, stream);
  }
  if (bf16) return two ? launch_tc<64, true, 2>(p, n_ctas, stream) : launch_tc<64, true, 1>(p, n_ctas, stream);
  return two ? launch_tc<64, false, 2>(p, n_ctas, stream) : launch_tc<64, false, 1>(p, n_ctas, stream);
}

}  // namespace dfl
