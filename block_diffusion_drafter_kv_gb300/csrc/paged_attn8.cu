// Causal attention of new rows over an 8-bit paged cache, on the fp8 tensor cores: the same list of
// tiles, cut and parts as in paged_attn.cu, whose join follows.
//
//   out = sum_j w_j V_j / sum_j p_j,  p_j = 2^(s_j - m),  w_j = p_j 2^ev_j,  s_j = scale_log2 2^ek_j q . K_j
//
// with K_j, V_j the stored e4m3 values and ek_j, ev_j their rows' exponents. Bound: the cache's bytes,
// 2 (d + 1) per key and KV head.
//
// The cache's bytes go from memory to the tensor cores as they are. Both products are taken with the
// cache as the M operand, so that a step's cost goes with the rows there are, not with 128 of them:
//   S^T = K Q^T   M = 128 keys (two tiles), N = rows;   K as loaded, K-major
//   O^T += V^T P^T   M = dims, N = rows, K = 128 keys;  V as loaded, MN-major
// What multiplies the cache is e4m3 too, split so that little is lost:
//   q   a row is scaled by a power of two to a largest magnitude in [128, 256) and taken apart into
//       2 (bf16) or 3 (fp16) numbers of 4 significant bits: exact, but for what lies below 2^-10
//       of e4m3's scale there, 2^-17 of the row's largest value. Their products add up in one accumulator.
//   w   as fp16, then 2 (bf16) or 3 (fp16) e4m3 numbers, each 32 times the rest of the one before; an
//       accumulator each, N = pieces x rows.
// A thread of the softmax has one key and all rows: the key's scales are its own two numbers, and so is
// the first row that may see the key. The weights' reference m' is set to the maximum of s_j + ev_j over a step less 4, and
// moved up where a w_j passes 256; p_j is w_j 2^-ev_j (|ev_j| <= 40: no overflow).
//   small w  The last piece ends at 2^-15 (2^-20), whatever the largest weight is. One key far above thousands of others, as a
//       context's first often is, would leave their sum out: 9% of an output at 18 binary orders and 28000 keys, when
//       references only rose. So one step in 8 is looked at, and a row that had too few weights of 8 or more gets a lower
//       reference: O and the sums grow, up to 40 orders. Where a reference is set the sum is 16 at least, a step with a weight of
//       8 adds 8, and a look stands for 8 x 128 weights of 2^-15 each at most: of a row's weights at most 3/8 x 1024 x 2^-15 (2^-20)
//       of the sum of its steps' largest is lost, however long the range, and a sixth of that behind one key far above all.
//       Of 4 x 32768 keys, 64 rows: 82 us without the looks, 87 with them (89 and 99 where scores spread twice as far); 128
//       rows 164 and 198, whose threads have no registers left for it.
//
// Measured (32 query heads on 8 KV heads, d 128; in brackets the 16-bit cache): 32 ragged sequences of 512 to 8192
// keys, one token, 52 to 56 us, 75 to 81% of the copy rate (94); 4 sequences of 32768, one token, 51 us, 79% (89; with d 64 36 us,
// 55%), with blocks of 16 (64 rows) 87 us, 46% (97), with 128 rows 198 us (119). Few rows are bound by memory, one row of 128 bytes
// a position and head, and by the starts and ends of the ranges. From 64 rows on it is the softmax: a step of
// 128 keys is 6500 warp instructions (some 300 in each of 16 warps, half of them whatever its rows, the rest the issuer's
// polling), 58% of what the SM can issue, in a chain of some 2700 cycles, against 1400 cycles of HBM time. (Choices below that name 83
// and 126 us were measured while references only rose.)
//
// CTA: one per SM; four softmax groups of 128 threads, a key of the step each. Of at most 16 rows each group is a
// strand of its own: a range of the list, a producer warp, stages, accumulators, so that one's start and end
// of a segment run under the others' steps. Of more rows two or four groups make a strand, some of its rows
// each. Of a strand that is one group the first warp issues the products: the next S as soon as the scores of
// this one are in registers, O once the weights are written. (One warp that issued for four strands noticed what
// was ready some 1200 cycles late.) Larger strands have a warp for that. Every wait is bounded; past the limit
// the later ones pass at once and the CTA walks to its end without results.
#include "paged_attn.cuh"
#include "quant.cuh"

namespace dfl {

namespace {

constexpr int kStepKeys = 128;
constexpr float kNone = 3e38f;      // the negative of a reference where no key has been seen
constexpr float kHeadroom = 4.f;    // a reference is set so many binary orders below the largest score,
constexpr float kMost = 256.f;      // moves up where a weight passes this,
constexpr int kLook = 8;            // and down where, of one step in so many, more had no weight of 8
constexpr int kGain = 2;            // than so many times those that had one,
constexpr int kCredit = 4;          // and this more behind a move up by less than 2^12 (where scores spread, the next steps are lower again)
constexpr float kDeepest = 40.f;    // no further than this below its highest in a segment (what is lost then is nothing)
constexpr float kRest = 32.f;       // a weight's pieces: the rest of one, at most 8, goes into the next times this

// ---------------------------------------------------------------- descriptors
DEV void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// fp32 accumulator, both operands e4m3, each K-major or MN-major.
constexpr uint32_t idesc_f8(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// An operand in rows of W bytes (32, 64 or 128, the width of its swizzle), 8 rows to an atom. K-major: a row an M
// or N index, atoms 8 W apart. MN-major: a row a K index, the next W indices of M or N `mn_stride` bytes on.
template <int W>
DEV uint64_t desc_rows(uint32_t saddr, uint32_t mn_stride) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((mn_stride >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(8 * W >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(W == 128 ? 2 : W == 64 ? 4 : 6) << 61;
  return d;
}
// Byte offset of 16-byte chunk `ch` of row `r` of such an operand.
template <int W>
DEV uint32_t chunk_at(int r, int ch) {
  return static_cast<uint32_t>(r * W + ((ch ^ (W == 128 ? r & 7 : W == 64 ? (r >> 1) & 3 : (r >> 2) & 1)) << 4));
}

DEV void load16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
DEV void store16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
DEV void load4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
}
DEV void wait_loads() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
DEV void wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
DEV bool test_wait(uint64_t* bar, uint32_t parity) {
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
// A barrier of `n` threads that tells each of them whether one had `v`.
DEV bool named_bar_any(int id, int n, bool v) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(v ? 1u : 0u), "r"(id), "r"(n)
      : "memory");
  return any != 0;
}
DEV void named_bar_arrive(int id, int n) { asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }
DEV float warp_max(float x) {  // NaN left out
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
DEV uint32_t half2_to_e4m3x2(__half2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&v)));
  return r;
}
DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
DEV bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
DEV float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&d))
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return d;
}
DEV bool has_nan8(uint32_t v) { return (((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0; }

// Sums of 16 values over the warp: lane L gets that of value L / 2.
DEV float reduce16(float (&v)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 8; h >= 1; h >>= 1) {
    const bool up = lane & (2 * h);
#pragma unroll
    for (int k = 0; k < h; ++k) {
      const float keep = up ? v[k + h] : v[k], send = up ? v[k] : v[k + h];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * h);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// D: head dim; R: rows of a problem that the buffers hold (16, 32, 64, 128); PH: strands of a CTA, each with a range of
// the list, accumulators and 4 / PH of the softmax groups (4: at most 16 rows; 2: at most 32 rows; 1).
template <int D, int R, int PH, bool BF16>
struct Layout8 {
  static constexpr int kPieces = BF16 ? 2 : 3;              // of q, and of the weights
  static constexpr int RT = R == 16 ? 16 : R * PH / 4;      // rows of a softmax thread
  // A product's time hardly goes with N up to a hundred, and every product reads its 128 rows of A again: pieces of q side
  // by side, in columns of their own, as far as tensor memory holds them (the rest add up in the last of them). 64 rows:
  // 83.3 us with two columns a score, 84.9 with one.
  static constexpr int ST = R <= 32 ? kPieces : R == 64 ? 2 : 1;
  static constexpr int kPW = R > 16 ? R : BF16 ? 32 : 64;   // bytes of a key's row of weights: a piece, or with 16 rows all pieces
  static constexpr int kPiece = R > 16 ? kStepKeys * R : 16;     // from a weight's piece to the next
  static constexpr int kPBuf = R > 16 ? kPieces * kPiece : kStepKeys * kPW;
  static constexpr int kOCols = R > 16 ? kPieces * R : kPW;
  static constexpr int NB = PH > 1 ? PH : R == 128 && !BF16 ? 1 : 2;  // buffers of S and P, taken by the steps in turn
  static constexpr int NS = NB / PH;                        // of a strand
  static constexpr bool kIssuer = PH < 4;                   // a warp for the products
  static constexpr int kThreads = 512 + 32 * PH * (kIssuer ? 2 : 1);
  static constexpr int kOperand = kStepKeys * D;            // K, or V, of a step
  static constexpr int STAGES = D == 64 ? (R == 128 ? 6 : 8) : R == 128 ? 3 : 4;
  static constexpr int SP = STAGES / PH;                    // of a strand
  static constexpr int kQPiece = R * D;
  static constexpr int kK = 0;
  static constexpr int kV = kK + STAGES * kOperand;
  static constexpr int kP = kV + STAGES * kOperand;
  static constexpr int kQ = kP + NB * kPBuf;
  static constexpr int kSc = kQ + PH * kPieces * kQPiece;   // [PH][2 SP] scales of a step: two tiles' 128 bytes
  static constexpr int kBase = kSc + 2 * STAGES * 256;      // [PH][R] references, negative
  static constexpr int kGain = kBase + PH * R * 4;          // [PH][R] 1 / the power of two that q was scaled by
  static constexpr int kCorr = kGain + PH * R * 4;          // [PH][R] factors of a moved reference
  static constexpr int kTop = kCorr + PH * R * 4;           // [4 groups][4 warps][RT] warps' maxima; sums at the end
  static constexpr int kHigh = kTop + 4 * 4 * RT * 4;       // [PH][R] references, negative, where they were highest
  static constexpr int kLeft = kHigh + PH * R * 4;          // [PH][R] what is left of kCredit
  static constexpr int kMl = kLeft + PH * R * 4;            // [PH][R] (max, sum)
  static constexpr int kRow = kMl + PH * R * 8;             // [PH][R] where a row's output goes, in rows of D
  static constexpr int kBar = kRow + PH * R * 4;
  static constexpr int kBars = 6 * SP + 4 * NS + 2;         // of a strand: K full, empty, V full, empty [SP]; scales full [2 SP]; S ready, PV done, S free, P ready [NS]; Q; all done
  static constexpr int kFlags = kBar + PH * kBars * 8;      // [0] abort, [1] TMEM base, then [PH][16] steps: 1, 2: tiles that are there, 4: a segment's first, 8: the last
  static constexpr int kWarpSums = kFlags + 16 + PH * 64;
  static constexpr int kPre = kWarpSums + 128;
  static constexpr int smem(int batch) { return 1024 + kPre + (3 * batch + 1) * 4; }
  static constexpr uint32_t tS(int b) { return b * ST * R; }     // TMEM columns
  static constexpr uint32_t tO(int ph) { return NB * ST * R + ph * kOCols; }
  static_assert(NB * ST * R + PH * kOCols <= 512, "tensor memory");
  static_assert(kThreads <= 32 * 32 && 4 * RT / PH <= R, "groups");
};

template <int D, int R, int PH, bool BF16, bool SHARED>
__global__ void __launch_bounds__(Layout8<D, R, PH, BF16>::kThreads, 1) paged_attn8_kernel(const __grid_constant__ PagedAttnParams P) {
  using L = Layout8<D, R, PH, BF16>;
  constexpr int NS = L::NS, SP = L::SP, PC = L::kPieces;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* flag = reinterpret_cast<volatile int*>(smem + L::kFlags);
  int* s_warp = reinterpret_cast<int*>(smem + L::kWarpSums);
  int* s_pre = reinterpret_cast<int*>(smem + L::kPre);
  const int entries = SHARED ? P.batch + P.n_pre : P.batch;
  int* s_len = s_pre + entries + 1;
  int* s_new = s_len + entries;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t WL = P.wait_ns;

  if (tid == 0) {
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
    for (int i = 0; i < PH * L::kBars; ++i) {
      const int k = i % L::kBars - 6 * SP - 2 * NS;  // from S free on
      mbar_init(&bars[i], k >= 0 && k <= 2 * NS ? 512 / PH : 1);
    }
    flag[0] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&P.kmap);
    tma_prefetch_desc(&P.vmap);
  }
  pdl_wait();
  pdl_launch_dependents();
  if constexpr (SHARED) count_entries<L::kThreads>(P, s_pre, s_len, s_new, s_warp);
  else count_tiles<L::kThreads>(P, s_pre, s_len, s_new, s_warp);
  const int nkv = P.nkv, grp = P.group;
  const long long T = static_cast<long long>(nkv) * s_pre[entries];
  const int G = n_ranges(T, gridDim.x, PH);
  const int cta = blockIdx.x;
  if (cta >= G) return;  // the whole CTA, before it holds any tensor memory
  if (warp == 16) tmem_alloc(reinterpret_cast<uint32_t*>(smem + L::kFlags + 4), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(flag[1]);

  // The thread's strand, and its walk: steps of up to two tiles of the segments of its range.
  const int g = tid >> 7;                                     // softmax group
  const int ph = warp < 16 ? g & (PH - 1) : (warp - 16) % PH;
  const int range = ph * static_cast<int>(gridDim.x) + cta;
  const long long end = range < G ? range_begin(range + 1, T, G) : 0;
  long long u = range < G ? range_begin(range, T, G) : 0;     // the next tile
  Place at{};
  int left = 0, began = 0;                                    // tiles of the segment that are left; whether the range begins behind a pair's tiles
  auto begin_segment = [&] {
    at = locate(s_pre, entries, nkv, u, P.extra);
    left = static_cast<int>(min(end - u, static_cast<long long>(at.nt - at.t)));
  };
  auto advance = [&](int cnt) {
    u += cnt;
    left -= cnt;
    at.t += cnt;
    if (at.t == at.nt) u = min(end, u + P.extra);
  };
  if (P.extra > 0 && u < end) {
    const Place p = locate(s_pre, entries, nkv, u, P.extra);
    if (p.t >= p.nt) u = min(end, u + p.nt + P.extra - p.t), began = 1;
  }
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + L::kBar) + ph * L::kBars;
  uint64_t* kempty = kfull + SP;
  uint64_t* vfull = kempty + SP;
  uint64_t* vempty = vfull + SP;
  uint64_t* scfull = vempty + SP;
  uint64_t* sready = scfull + 2 * SP;
  uint64_t* pvdone = sready + NS;
  uint64_t* sfree = pvdone + NS;
  uint64_t* pready = sfree + NS;
  uint64_t* qready = pready + NS;
  uint64_t* mdone = qready + 1;
  volatile int* s_step = flag + 4 + ph * 16;  // by step mod 16, more than a ring holds
  uint8_t* kring = smem + L::kK + ph * SP * L::kOperand;
  uint8_t* vring = smem + L::kV + ph * SP * L::kOperand;
  uint8_t* scring = smem + L::kSc + ph * 2 * SP * 256;  // twice as long: a step's scales are read after K's stage may go on

  // The products of step n, by one lane; the whole warp is here, so that descriptors are built in uniform registers.
  constexpr uint32_t kQkAll = idesc_f8(128, L::ST * R, false, false), kQkOne = idesc_f8(128, R, false, false);
  auto qk = [&](int n) {  // S^T = K Q^T
    const uint64_t k0 = desc_rows<D>(smem_u32(kring) + n % SP * L::kOperand, 16), q0 = desc_rows<D>(smem_u32(smem + L::kQ) + ph * PC * L::kQPiece, 16);
    const uint32_t d = tmem + L::tS(ph * NS + n % NS);
    tc_fence_after();
    if (elect_one()) {
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) mma_f8(d, k0 + (kk * 32 >> 4), q0 + (kk * 32 >> 4), kQkAll, kk > 0 ? 1u : 0u);
#pragma unroll
      for (int p = L::ST; p < PC; ++p)
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          mma_f8(d + (L::ST - 1) * R, k0 + (kk * 32 >> 4), q0 + ((p * L::kQPiece + kk * 32) >> 4), kQkOne, 1u);
      tc_commit(&sready[n % NS]);
      tc_commit(&kempty[n % SP]);
    }
    __syncwarp();
  };
  auto pv = [&](int n, bool first) {  // O^T (+)= V^T P^T. With 64 dims the upper half of M is the same dims again, unused.
    const uint64_t v0 = desc_rows<D>(smem_u32(vring) + n % SP * L::kOperand, 0);
    const uint64_t p0 = desc_rows<L::kPW>(smem_u32(smem + L::kP) + (ph * NS + n % NS) * L::kPBuf, L::kPiece);
    const uint32_t d = tmem + L::tO(ph), keep = first ? 0u : 1u;
    constexpr int N1 = L::kOCols <= 256 ? L::kOCols : 256, N2 = L::kOCols - N1;
    constexpr uint32_t kPv1 = idesc_f8(128, N1, true, true);
    tc_fence_after();
    if (elect_one()) {
#pragma unroll
      for (int kk = 0; kk < kStepKeys / 32; ++kk) {
        mma_f8(d, v0 + (kk * 32 * D >> 4), p0 + (kk * 32 * L::kPW >> 4), kPv1, kk > 0 ? 1u : keep);
        if constexpr (N2 > 0) {
          constexpr uint32_t kPv2 = idesc_f8(128, N2, true, true);
          mma_f8(d + N1, v0 + (kk * 32 * D >> 4), p0 + ((N1 / R * L::kPiece + kk * 32 * R) >> 4), kPv2, kk > 0 ? 1u : keep);
        }
      }
      tc_commit(&pvdone[n % NS]);
      tc_commit(&vempty[n % SP]);
    }
    __syncwarp();
  };

  if (warp >= 16 && warp < 16 + PH) {
    // ------------------------------------------------------------------ producer
    const uint64_t pol = T * (2 * kKeys * D) > (16ll << 20) ? policy_evict_first() : policy_evict_last();
    int n = 0, kn = 0, vn = 0;  // step; copies of K and of V issued
    bool go = true;             // the same in every lane
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      bool ok = !flag[0];
      if (ok && lane == 0 && !mbar_wait(bar, parity, WL)) {
        raise_flag(P.err, kDevTimeout);
        flag[0] = 1;
        ok = false;
      }
      go = __all_sync(0xffffffffu, ok);
    };
    int ids = -1, id0 = 32;  // page ids of the segment's next tiles, one a lane; the lane that has the next one
    while (u < end && go) {
      const bool start = left == 0;
      if (start) {
        begin_segment();
        id0 = 32;
        for (int r = lane; r < s_new[at.s]; r += 32)  // the segment's q, a new row a lane
          bulk_prefetch_l2(static_cast<const uint16_t*>(P.q) +
                               ((static_cast<size_t>(first_row<SHARED>(P, at.s)) + r) * P.nq + static_cast<size_t>(at.g) * grp) * D,
                           grp * D * 2);
      }
      int page[2] = {-1, -1};
      const int cnt = min(2, left);
      for (int h = 0; h < cnt; ++h) {
        if (id0 == 32) {
          ids = -1;
          if (lane < left - h) {
            ids = __ldcg(pages_of<SHARED>(P, at.s) + at.t + h + lane);
            if (ids < 0 || ids >= P.n_pages) {
              raise_flag(P.err, kDevCapacity);
              ids = -1;
            }
          }
          id0 = 0;
        }
        page[h] = __shfl_sync(0xffffffffu, ids, id0++);
      }
      const int st = n % SP, sc = n % (2 * SP), valid = (page[0] >= 0) | (page[1] >= 0) << 1, tiles = (valid & 1) + (valid >> 1);
      if (n >= SP) wait(&kempty[st], (n / SP - 1) & 1);
      if (!go) break;
      if (lane == 0) {
        s_step[n & 15] = valid | (start ? 4 : 0) | (u + cnt + (at.t + cnt == at.nt ? P.extra : 0) >= end ? 8 : 0);
        if (tiles) {
          mbar_arrive_expect_tx(&scfull[sc], tiles * 2 * kKeys);
          mbar_arrive_expect_tx(&kfull[st], tiles * kKeys * D);
        } else {
          mbar_arrive(&scfull[sc]);
          mbar_arrive(&kfull[st]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (page[h] >= 0) {
            tma_load_3d(kring + st * L::kOperand + h * kKeys * D, &P.kmap, &kfull[st], 0, at.g, page[h] * kKeys, pol);
            bulk_load(scring + sc * 256 + h * 128, P.scales + (static_cast<size_t>(page[h]) * nkv + at.g) * 128, 128, &scfull[sc]);
          }
      }
      __syncwarp();
      kn = n + 1;
      if (n >= SP) wait(&vempty[st], (n / SP - 1) & 1);
      if (!go) break;
      if (lane == 0) {
        if (tiles) mbar_arrive_expect_tx(&vfull[st], tiles * kKeys * D);
        else mbar_arrive(&vfull[st]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (page[h] >= 0) tma_load_3d(vring + st * L::kOperand + h * kKeys * D, &P.vmap, &vfull[st], 0, at.g, page[h] * kKeys, pol);
      }
      __syncwarp();
      vn = ++n;
      advance(cnt);
    }
    // every copy issued has landed before the CTA leaves
    if (lane == 0) {
      for (int k = max(0, kn - SP); k < kn; ++k) mbar_wait(&kfull[k % SP], (k / SP) & 1, WL);
      for (int k = max(0, kn - 2 * SP); k < kn; ++k) mbar_wait(&scfull[k % (2 * SP)], (k / (2 * SP)) & 1, WL);
      for (int k = max(0, vn - SP); k < vn; ++k) mbar_wait(&vfull[k % SP], (k / SP) & 1, WL);
    }
    __syncwarp();
  } else if (warp >= 16) {
    // ------------------------------------------------------------------ issuer: whichever product's inputs are ready goes next
    auto ready = [](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, test_wait(bar, parity)) != 0; };
    int nqk = 0, npv = 0, segs = 0;  // products issued, segments begun
    uint32_t starts = 0;             // by step mod 32: whether it begins a segment, whose O is new
    bool open = u < end;             // steps to come
    uint64_t idle_since = 0;
    uint32_t spins = 0;
    while (open || npv < nqk) {
      bool moved = false;
      if (open && nqk < npv + 2 * NS && ready(&kfull[nqk % SP], (nqk / SP) & 1)) {
        const int info = s_step[nqk & 15];
        if ((nqk < NS || ready(&sfree[nqk % NS], (nqk / NS - 1) & 1)) && (!(info & 4) || ready(qready, segs & 1))) {
          qk(nqk);
          starts = (starts & ~(1u << (nqk & 31))) | static_cast<uint32_t>(info >> 2 & 1) << (nqk & 31);
          segs += info >> 2 & 1;
          ++nqk;
          if (info & 8) open = false;
          moved = true;
        }
      }
      if (npv < nqk && ready(&pready[npv % NS], (npv / NS) & 1) && ready(&vfull[npv % SP], (npv / SP) & 1)) {
        pv(npv, starts >> (npv & 31) & 1);
        ++npv;
        moved = true;
      }
      // (reading the timer takes some 600 cycles: only where nothing has moved for a while)
      if (moved) {
        spins = 0;
      } else if ((++spins & 1023u) == 0) {
        const uint64_t now = __shfl_sync(0xffffffffu, globaltimer_ns(), 0);
        if (spins == 1024) idle_since = now;
        if (__any_sync(0xffffffffu, flag[0] != 0) || now - idle_since > WL) {
          if (lane == 0 && !flag[0]) raise_flag(P.err, kDevTimeout);
          flag[0] = 1;
          break;
        }
      }
    }
    if (elect_one()) {
      tc_commit(mdone);
      if (!mbar_wait(mdone, 0, WL)) raise_flag(P.err, kDevTimeout);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax, products and output
    const int j = tid & 127, gw = warp & 3, row0 = g / PH * L::RT;  // key of the step, warp of the group, first row
    const int sid = g / PH * 128 + j;                        // thread of the strand
    const bool issues = !L::kIssuer && gw == 0;              // the products
    constexpr int RT = L::RT, kStrand = 512 / PH;
    const uint32_t lanes = static_cast<uint32_t>(gw * 32) << 16;
    float* s_base = reinterpret_cast<float*>(smem + L::kBase) + ph * R + row0;
    float* s_gain = reinterpret_cast<float*>(smem + L::kGain) + ph * R;
    float* s_corr = reinterpret_cast<float*>(smem + L::kCorr) + ph * R + row0;
    float* s_top = reinterpret_cast<float*>(smem + L::kTop) + g * 4 * RT;
    float* s_high = reinterpret_cast<float*>(smem + L::kHigh) + ph * R + row0;
    int* s_left = reinterpret_cast<int*>(smem + L::kLeft) + ph * R + row0;
    float2* s_ml = reinterpret_cast<float2*>(smem + L::kMl) + ph * R;
    uint32_t* s_row = reinterpret_cast<uint32_t*>(smem + L::kRow) + ph * R;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!mbar_try_wait(bar, parity)) wait_long(bar, parity, flag, P.err, WL);
      __syncwarp();
    };
    // a segment's q, taken apart; rows up to the next multiple of 16 that are not there are zero, and so are those of a
    // prefix's entry that are not of this call: what lies there must not move the references of the rows beside them
    auto put_q = [&] {
      constexpr int kParts = D / 16;  // threads of a row
      const int live = s_new[at.s] * grp, rows = (live + 15) & ~15;
      for (int item = sid; item < rows * kParts; item += kStrand) {
        const int row = item / kParts, part = item % kParts;
        uint4 in[2] = {};
        const int r = new_row(P, row);
        if (row < live && (!SHARED || at.s < P.batch || row_is_new(P, s_new, first_row<SHARED>(P, at.s) + r))) {
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const uint16_t*>(P.q) +
              ((static_cast<size_t>(first_row<SHARED>(P, at.s)) + r) * P.nq + static_cast<size_t>(at.g) * grp + row - r * grp) * D + part * 16);
          in[0] = __ldcg(src), in[1] = __ldcg(src + 1);
        }
        const uint32_t* u = reinterpret_cast<const uint32_t*>(in);
        float x[16];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 v = unpack2<BF16>(u[k]);
          x[2 * k] = v.x, x[2 * k + 1] = v.y;
          top = max(top, max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu));
        }
#pragma unroll
        for (int o = 1; o < kParts; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const bool fine = top < 0x7f800000u;
        const int e = max(static_cast<int>(top >> 23) - 127, -119);
        const float f = fine ? exponent_value(7 - e) : 0.f;
        if (part == 0) s_gain[row] = fine ? exponent_value(e - 7) : __uint_as_float(0x7fc00000u);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = fine ? x[k] * f : 0.f;
#pragma unroll
        for (int p2 = 0; p2 < PC; ++p2) {
          uint32_t out[4] = {0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t b = to_e4m3x2(x[2 * k], x[2 * k + 1]);
            out[k >> 1] |= b << ((k & 1) * 16);
            const float2 v = __half22float2(from_e4m3x2(b));
            x[2 * k] -= v.x, x[2 * k + 1] -= v.y;
          }
          *reinterpret_cast<uint4*>(smem + L::kQ + (ph * PC + p2) * L::kQPiece + chunk_at<D>(row, part)) = make_uint4(out[0], out[1], out[2], out[3]);
        }
      }
      fence_async_shared();
      if (L::kIssuer) mbar_arrive(qready);
    };

    float2 l2[RT / 2];  // the key's part of every row's sum
    int n = 0, seg_no = began;  // step
    if (u < end) {
      begin_segment();
      put_q();
      if (j < RT) s_base[j] = s_high[j] = kNone, s_left[j] = 0;
      named_bar_sync(6 + ph, kStrand);
    }
    for (; u < end; ++seg_no) {
      const int s = at.s, kvh = at.g;
      const bool whole = at.t == 0 && left == at.nt;
      const bool pre = SHARED && s >= P.batch;
      const int len = s_len[s], n_new = pre ? 1 : s_new[s], nk = len + n_new;
      const int live = s_new[s] * grp;
      const int last = live > row0 ? min(RT / 16, (live - row0 + 15) / 16) - 1 : -1;  // of the group's 16 rows at a time
#pragma unroll
      for (int k = 0; k < RT / 2; ++k) l2[k] = {0.f, 0.f};
      const int n0 = n, n1 = n + ((left + 1) >> 1);  // the segment's steps
      if (issues)
        for (int k = n0; k < min(n1, n0 + NS); ++k) {
          wait(&kfull[k % SP], (k / SP) & 1);
          qk(k);
        }
      for (; n < n1; ++n) {
        const int t = at.t, cnt = min(2, left);
        advance(cnt);
        const int st = n % SP, b = n % NS;
        wait(&scfull[n % (2 * SP)], (n / (2 * SP)) & 1);
        const uint8_t* sc = scring + n % (2 * SP) * 256 + (j >> 6) * 128 + (j & 63);
        const uint32_t kb = sc[0], vb = sc[64];
        const int valid = s_step[n & 15] & 3;
        // Some row may not see some key of the step: by the walk alone, and so the same for all threads whatever a wait that
        // ran out has left in s_step. Barriers go by this.
        const bool ends = cnt < 2 || (t + 2) * kKeys > len + 1;
        const bool edge = ends || valid != 3;
        int rmin = 0;  // the first row that sees the thread's key
        bool nan = false;
        if (edge) {
          // Values that no row sees are cleared (0 * NaN is NaN); a key that some rows see and that has a NaN
          // among its values becomes one of zeros whose scale is NaN.
          uint4* vrow = reinterpret_cast<uint4*>(vring + st * L::kOperand + j * D);
          // Eight neighbours at eight places of 128 bytes (128 sequences of 500, blocks of 16: 126 us, 132 without); with 128 rows a
          // thread has no registers left for it (180 us against 165 at 4 sequences of 32768).
          auto bank = [&](int ch) { return R == 128 ? ch : (ch + (j >> (D == 64))) & (D / 16 - 1); };
          // (a barrier tells phases apart by parity: only after the stage's last values are spent may the next be asked for)
          if (n >= NS) wait(&pvdone[b], (n / NS - 1) & 1);
          wait(&vfull[st], (n / SP) & 1);
          const int key = t * kKeys + j;
          const bool alive = (valid >> (j >> 6) & 1) && key < nk;
          rmin = (!alive ? R : key <= len ? 0 : (key - len) * grp) - row0;
          bool clear = !alive;
          if (ends && alive && key >= len && n_new > 1) {
#pragma unroll 4
            for (int ch = 0; ch < D / 16; ++ch) {
              const uint4 v = vrow[bank(ch)];
              nan |= has_nan8(v.x) || has_nan8(v.y) || has_nan8(v.z) || has_nan8(v.w);
            }
            clear = nan;
          }
          // (all groups of the step have looked; where only a page is missing none looks, and each thread clears what is its own)
          if (PH < 4 && ends) named_bar_sync(6 + ph, kStrand);
          if (clear && g < PH)
#pragma unroll
            for (int ch = 0; ch < D / 16; ++ch) vrow[bank(ch)] = make_uint4(0, 0, 0, 0);
        }
        // the scales of the thread's key
        const float f = P.scale_log2 * scale_value(kb);
        const float ev = vb == kScaleNan || nan ? __uint_as_float(0x7fc00000u) : static_cast<float>(static_cast<int>(vb) - kScaleBias);
        const float inv_v = scale_value(254u - min(vb, 253u));
        wait(&sready[b], (n / NS) & 1);
        tc_fence_after();
        const float2 f2 = {f, f}, ev2 = {ev, ev}, inv2 = {inv_v, inv_v};
        bool later = false;  // the next S, where its K is not there yet
        auto scores_read = [&] {  // by the group: the next S may come into their place
          if (L::kIssuer) {
            mbar_arrive(&sfree[b]);
          } else if (issues && n + NS < n1) {
            later = !__all_sync(0xffffffffu, test_wait(&kfull[(n + NS) % SP], ((n + NS) / SP) & 1));
            if (!later) qk(n + NS);
          }
        };
        if (last < 0) scores_read();
#pragma unroll
        for (int c = 0; c < RT / 16; ++c) {  // 16 rows at a time
          if (c > last) break;
          float2 x[8];
          auto scores = [&] {  // s_j + ev_j; what a row does not see is -inf
            uint32_t sraw[L::ST][16];
#pragma unroll
            for (int p = 0; p < L::ST; ++p) load16(tmem + lanes + L::tS(ph * NS + b) + row0 + c * 16 + p * R, sraw[p]);
            wait_loads();
            tc_fence_before();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              x[k] = {__uint_as_float(sraw[0][2 * k]), __uint_as_float(sraw[0][2 * k + 1])};
#pragma unroll
              for (int p = 1; p < L::ST; ++p) x[k] = add2(x[k], float2{__uint_as_float(sraw[p][2 * k]), __uint_as_float(sraw[p][2 * k + 1])});
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 gain = reinterpret_cast<const float4*>(s_gain + row0)[c * 4 + k];
              x[2 * k] = fma2(x[2 * k], mul2(float2{gain.x, gain.y}, f2), ev2);
              x[2 * k + 1] = fma2(x[2 * k + 1], mul2(float2{gain.z, gain.w}, f2), ev2);
            }
            if (edge)
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                if (c * 16 + 2 * k < rmin) x[k].x = -INFINITY;
                if (c * 16 + 2 * k + 1 < rmin) x[k].y = -INFINITY;
              }
          };
          __half2 h[8], top = __float2half2_rn(0.f);
          auto weights = [&] {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 base = reinterpret_cast<const float4*>(s_base)[c * 4 + k];
              const float2 d0 = add2(x[2 * k], float2{base.x, base.y}), d1 = add2(x[2 * k + 1], float2{base.z, base.w});
              x[2 * k] = {ex2(d0.x), ex2(d0.y)};
              x[2 * k + 1] = {ex2(d1.x), ex2(d1.y)};
              h[2 * k] = __floats2half2_rn(x[2 * k].x, x[2 * k].y);
              h[2 * k + 1] = __floats2half2_rn(x[2 * k + 1].x, x[2 * k + 1].y);
              top = __hmax2(top, __hmax2(h[2 * k], h[2 * k + 1]));
            }
          };
          scores();
          const bool look = (n - n0) % kLook == kLook / 2 && !ends;  // (by the walk alone)
          bool move = n == n0 || look;
          if (!move) {
            weights();
            move = named_bar_any(2 + g, 128, __hgt(__hmax(__low2half(top), __high2half(top)), __float2half_rn(kMost)));
            if (move) scores();
            else if (c == last) scores_read();
          }
          if (move) {
            // ---- references that may move: the rows' maxima over the group, then O and the sums. (Few instructions: most
            // steps do not come here, and those that do wait for each of them to be fetched.)
            float mine = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float most = warp_max(k & 1 ? x[k / 2].y : x[k / 2].x);
              if (lane == k) mine = most;
            }
            if (lane < 16) s_top[gw * RT + c * 16 + lane] = mine;
            named_bar_sync(2 + g, 128);
            if (c == last) scores_read();
            bool moved = false;
            if (j < 16) {
              const float* tops = s_top + c * 16 + j;
              const float most = fmaxf(fmaxf(tops[0], tops[RT]), fmaxf(tops[2 * RT], tops[3 * RT]));
              const float old = s_base[c * 16 + j], high = s_high[c * 16 + j], over = most + old;  // log2 of the largest weight
              const bool up = over > (look ? 8.f : kHeadroom);  // (a look alone moves none that kMost lets be)
              bool down = false;
              if (look) {
                const int rest = s_left[c * 16 + j] + (over >= 3.f ? kGain : -1);
                s_left[c * 16 + j] = rest;
                // (not where no key has been seen, nor where there is no such row)
                down = rest < 0 && over < 3.f && most > -INFINITY && old < high + kDeepest && row0 + c * 16 + j < live;
              }
              moved = up || down;
              s_corr[c * 16 + j] = 1.f;
              if (moved) {
                const float now = up ? kHeadroom - most : fminf(kHeadroom - most, high + kDeepest);
                s_corr[c * 16 + j] = ex2(now - old);
                s_base[c * 16 + j] = now;
                s_high[c * 16 + j] = fminf(high, now);
                s_left[c * 16 + j] = up && over <= 16.f ? kCredit : 0;
              }
            }
            moved = named_bar_any(2 + g, 128, moved);
            if (moved) {
#pragma unroll
              for (int k = 0; k < 8; ++k) l2[c * 8 + k].x *= s_corr[c * 16 + 2 * k], l2[c * 8 + k].y *= s_corr[c * 16 + 2 * k + 1];
            }
            if (moved && n > n0) {
              wait(&pvdone[(n - 1) % NS], ((n - 1) / NS) & 1);
              tc_fence_after();
#pragma unroll 1
              for (int p = 0; p < PC; ++p) {
                const uint32_t to = tmem + lanes + L::tO(ph) + p * R + row0 + c * 16;
                uint32_t u[16];
                __syncwarp();
                load16(to, u);
                wait_loads();
#pragma unroll
                for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * s_corr[c * 16 + k]);
                store16(to, u);
              }
              wait_stores();
            }
            weights();
          }
          if (c == 0 && n >= NS) wait(&pvdone[b], (n / NS - 1) & 1);  // the last product from the buffer
          uint8_t* to = smem + L::kP + (ph * NS + b) * L::kPBuf;
#pragma unroll
          for (int k = 0; k < 8; ++k) l2[c * 8 + k] = fma2(x[k], inv2, l2[c * 8 + k]);
#pragma unroll
          for (int p = 0; p < PC; ++p) {
            uint32_t out[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t b0 = half2_to_e4m3x2(h[2 * k]), b1 = half2_to_e4m3x2(h[2 * k + 1]);
              out[k] = b0 | b1 << 16;
              if (p + 1 < PC) {
                h[2 * k] = __hmul2(__hsub2(h[2 * k], from_e4m3x2(b0)), __float2half2_rn(kRest));
                h[2 * k + 1] = __hmul2(__hsub2(h[2 * k + 1], from_e4m3x2(b1)), __float2half2_rn(kRest));
              }
            }
            *reinterpret_cast<uint4*>(to + (R > 16 ? p * L::kPiece + chunk_at<R>(j, row0 / 16 + c) : chunk_at<L::kPW>(j, p))) = make_uint4(out[0], out[1], out[2], out[3]);
          }
        }
        // (a group without rows must not be a step ahead of the others at P's barrier either)
        if (last < 0 && n >= NS) wait(&pvdone[b], (n / NS - 1) & 1);
        fence_async_shared();
        tc_fence_before();
        if (L::kIssuer) {
          mbar_arrive(&pready[b]);
        } else if (issues) {
          named_bar_sync(10 + ph, kStrand);
          wait(&vfull[st], (n / SP) & 1);
          pv(n, n == n0);
          if (later) {
            wait(&kfull[(n + NS) % SP], ((n + NS) / SP) & 1);
            qk(n + NS);
          }
        } else {
          named_bar_arrive(10 + ph, kStrand);
        }
      }
      // ---- the segment's end. Every score of it has been read once the strand's groups are here: q is the next one's.
#pragma unroll
      for (int c = 0; c < RT / 16; ++c) {
        if (row0 + c * 16 >= live) break;
        float v[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[2 * k] = l2[c * 8 + k].x, v[2 * k + 1] = l2[c * 8 + k].y;
        const float sum = reduce16(v);
        if ((lane & 1) == 0) s_top[gw * RT + c * 16 + (lane >> 1)] = sum;
      }
      named_bar_sync(6 + ph, kStrand);
      if (u < end) {
        begin_segment();
        put_q();
      }
      // its rows' (max, sum), or for finished outputs (max, 1 / sum), and where they go: among the outputs, in `state`, in a slot
      if (j < RT) {
        const float base = s_base[j], den = (s_top[j] + s_top[RT + j]) + (s_top[2 * RT + j] + s_top[3 * RT + j]);
        const int row = row0 + j, r = new_row(P, row), head = kvh * grp + row - r * grp;
        float2 ml = make_float2(base == kNone ? -INFINITY : -base, den);
        s_row[row] = !whole ? row : static_cast<uint32_t>(SHARED ? state_row(P, s, first_row<SHARED>(P, s) + r, head)
                                                                   : (static_cast<size_t>(s) * P.rows_per_seq + r) * P.nq + head);
        if (SHARED && whole && row < live) __stcg(state_sums(P) + s_row[row], ml);
        if (!SHARED && whole) ml.y = den > 0.f ? 1.f / den : (den == 0.f ? 0.f : den);
        s_ml[row] = ml;
        s_base[j] = s_high[j] = kNone, s_left[j] = 0;
      }
      wait(&pvdone[(n - 1) % NS], ((n - 1) / NS) & 1);
      named_bar_sync(6 + ph, kStrand);
      tc_fence_after();
      float* slot = P.part + (2 * static_cast<size_t>(range) + (seg_no == 0 ? 0 : 1)) * static_cast<size_t>(P.slot_rows) * (D + 2);
      if (gw * 32 < D) {  // a dim a lane, four rows at a time, in turn by the groups
        const int dim = gw * 32 + lane;
        float* to = (SHARED && whole ? P.state : slot) + dim;
        uint16_t* out = static_cast<uint16_t*>(P.out) + dim;
#pragma unroll 1
        for (int r4 = g / PH * 4; r4 < live; r4 += 16 / PH) {
          uint32_t u[PC][4];
          __syncwarp();
#pragma unroll
          for (int p = 0; p < PC; ++p) load4(tmem + lanes + L::tO(ph) + p * R + r4, u[p]);
          wait_loads();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float o = 0.f;
#pragma unroll
            for (int p = PC - 1; p >= 0; --p) o = fmaf(o, 1.f / kRest, __uint_as_float(u[p][q]));
            const size_t at_row = static_cast<size_t>(s_row[r4 + q]) * D;
            if (r4 + q >= live) break;
            if (!SHARED && whole) out[at_row] = static_cast<uint16_t>(pack2<BF16>(o * s_ml[r4 + q].y, 0.f));
            else __stcg(to + at_row, o);
          }
        }
      }
      if (sid < live && !whole) __stcg(reinterpret_cast<float2*>(slot + static_cast<size_t>(P.slot_rows) * D) + sid, s_ml[sid]);
      tc_fence_before();
      named_bar_sync(6 + ph, kStrand);  // the accumulators and sums are the next segment's
    }
    if (issues && elect_one()) {  // every product has completed before the CTA leaves
      tc_commit(mdone);
      if (!mbar_wait(mdone, 0, WL)) raise_flag(P.err, kDevTimeout);
    }
    __syncwarp();
  }

  // ---- every product has completed (the issuing warps waited for them) before the tensor memory goes
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int R, int PH, bool BF16, bool SHARED>
int set_attr() {
  using L = Layout8<D, R, PH, BF16>;
  static_assert(L::smem(kAttnMaxBatch) <= 232448, "shared memory of a CTA");
  return static_cast<int>(cudaFuncSetAttribute(paged_attn8_kernel<D, R, PH, BF16, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               L::smem(kAttnMaxBatch)));
}
template <int D, bool BF16, bool SHARED>
int set_attrs() {
  const int e[] = {set_attr<D, 16, 4, BF16, SHARED>(), set_attr<D, 32, 2, BF16, SHARED>(), set_attr<D, 64, 1, BF16, SHARED>(),
                   set_attr<D, 128, 1, BF16, SHARED>()};
  for (int x : e)
    if (x != 0) return x;
  return 0;
}
template <int D, int R, int PH, bool BF16, bool SHARED>
int launch(const PagedAttnParams& p, int n_ctas, cudaStream_t stream) {
  using L = Layout8<D, R, PH, BF16>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_ctas);
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::smem(p.batch + p.n_pre);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, paged_attn8_kernel<D, R, PH, BF16, SHARED>, p));
}
template <int D, bool BF16, bool SHARED>
int launch_slots(const PagedAttnParams& p, int n_ctas, cudaStream_t stream) {
  if (p.slot_rows <= 16) return launch<D, 16, 4, BF16, SHARED>(p, n_ctas, stream);
  if (p.slot_rows <= 32) return launch<D, 32, 2, BF16, SHARED>(p, n_ctas, stream);
  return p.slot_rows <= 64 ? launch<D, 64, 1, BF16, SHARED>(p, n_ctas, stream) : launch<D, 128, 1, BF16, SHARED>(p, n_ctas, stream);
}
template <int D, bool BF16>
int launch_rows(const PagedAttnParams& p, int n_ctas, cudaStream_t stream) {
  return p.prefix_len ? launch_slots<D, BF16, true>(p, n_ctas, stream) : launch_slots<D, BF16, false>(p, n_ctas, stream);
}

}  // namespace

int paged_attn8_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }
// Strands: 4 and 1 measured at 4 rows, 32 ragged sequences: 57 and 84 us; 2 and 1 at 20 rows, 4 x 32768: 55 and 70 us; 2 and 1
// at 64 rows: 119 (32 rows a thread: two passes, spills) and 83 us.
int paged_attn8_strands(int rows) { return rows <= 16 ? 4 : rows <= 32 ? 2 : 1; }
// A segment's start and end cost about as much as so many tiles (q in, the first references, O out: 7000 to 17000
// cycles). With and without: 32 ragged sequences, one token 57 and 60 us, blocks of 16 111 and 154 us; a prefix of 8190 shared by
// 16 sequences' blocks 105 and 292 us. (8 + rows / 4: 58, 111 and 108.)
int paged_attn8_extra(int rows) { return 6 + rows / 8; }
static_assert(6 + 128 / 8 <= kMaxExtra, "tiles that a list counts behind a pair");

int paged_attn8_set_attributes() {
  const int e[] = {set_attrs<64, false, false>(), set_attrs<64, true, false>(), set_attrs<128, false, false>(), set_attrs<128, true, false>(),
                   set_attrs<64, false, true>(),  set_attrs<64, true, true>(),  set_attrs<128, false, true>(),  set_attrs<128, true, true>()};
  for (int x : e)
    if (x != 0) return x;
  return 0;
}

int launch_paged_attn8(const PagedAttnParams& p, bool bf16, int n_ctas, cudaStream_t stream) {
  if (p.batch < 1 || p.batch + p.n_pre > kAttnMaxBatch || n_ctas < 1 || n_ctas > kPagedMaxCtas || p.rows > 128)
    return static_cast<int>(cudaErrorInvalidValue);
  int e;
  if (p.d == 128) e = bf16 ? launch_rows<128, true>(p, n_ctas, stream) : launch_rows<128, false>(p, n_ctas, stream);
  else e = bf16 ? launch_rows<64, true>(p, n_ctas, stream) : launch_rows<64, false>(p, n_ctas, stream);
  if (e != 0) return e;
  return p.prefix_len ? launch_shared_join(p, bf16, n_ctas, stream) : launch_paged_attn_join(p, bf16, n_ctas, stream);
}

}  // namespace dfl
