// Attention of new rows over a paged cache of 16 or 8 bits, with or without a prefix that all
// sequences share: one CTA per row and query head, a key per lane for the scores, a few dims per
// lane for the values, fp32 throughout.
#include <type_traits>

#include "paged_attn.cuh"
#include "quant.cuh"

namespace dfl {

namespace {

constexpr int kRowWarps = 8;

template <typename X>
DEV float2 pair_at(const uint8_t* row, int i, float f) {  // values 2i and 2i + 1
  if (sizeof(X) == 1) {
    const float2 x = __half22float2(from_e4m3x2(reinterpret_cast<const uint16_t*>(row)[i]));
    return make_float2(x.x * f, x.y * f);
  }
  return unpack2<std::is_same<X, __nv_bfloat16>::value>(reinterpret_cast<const uint32_t*>(row)[i]);
}

template <typename X, bool BF16, int D>
__global__ void __launch_bounds__(32 * kRowWarps) attn_rows_kernel(const __grid_constant__ PagedAttnParams P) {
  constexpr int E = D / 32;
  __shared__ float s_q[D], s_o[kRowWarps][D];
  __shared__ float2 s_ml[kRowWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x, head = blockIdx.y, s = row / P.rows_per_seq, r = row - s * P.rows_per_seq, g = head / P.group;
  int len;
  bool bad;
  const int n = rows_of(P, s, len, bad);
  const int before = P.prefix_len ? __ldcg(P.prefix_len) : 0;
  if (before < 0 || before > static_cast<long long>(P.pages_per_seq) * kPagePos) bad = true;
  if (bad && tid == 0) raise_flag(P.err, kDevCapacity);
  if (bad || r >= n) return;
  for (int i = tid; i < D / 2; i += blockDim.x) {
    const float2 v = unpack2<BF16>(static_cast<const uint32_t*>(P.q)[(static_cast<size_t>(row) * P.nq + head) * (D / 2) + i]);
    s_q[2 * i] = v.x, s_q[2 * i + 1] = v.y;
  }
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[E] = {};
  const int own = len + r + 1;
  for (int part = 0; part < 2; ++part) {
    const int keys = part == 0 ? before : own;
    const int* table = part == 0 ? P.prefix_table : P.page_table + static_cast<size_t>(s) * P.pages_per_seq;
    for (int k0 = warp * 32; k0 < keys; k0 += 32 * kRowWarps) {
      const int page = __ldcg(table + k0 / kPagePos);
      if (page < 0 || page >= P.n_pages) {
        if (lane == 0) raise_flag(P.err, kDevCapacity);
        continue;
      }
      const int slot0 = page * kPagePos + k0 % kPagePos, cnt = min(32, keys - k0);
      float z = -INFINITY, vs = 0.f;
      if (lane < cnt) {
        const int slot = slot0 + lane;
        float ks = 1.f;
        if (sizeof(X) == 1) {
          ks = scale_value(P.scales[scale_index(slot, P.nkv, g, 0)]);
          vs = scale_value(P.scales[scale_index(slot, P.nkv, g, 1)]);
        }
        const uint8_t* k = P.k_pool + (static_cast<size_t>(slot) * P.nkv + g) * D * sizeof(X);
        float dot = 0.f;
        for (int i = 0; i < D / 2; ++i) {
          const float2 x = pair_at<X>(k, i, 1.f);
          dot += s_q[2 * i] * x.x;
          dot += s_q[2 * i + 1] * x.y;
        }
        z = dot * ks * P.scale_log2;
      }
      float top = z;
      for (int x = 16; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn, corr = ex2(m - base);
      m = mn;
      const float p = lane < cnt ? ex2(z - base) : 0.f;
      float sum = p;
      for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l = l * corr + sum;
      for (int e = 0; e < E; ++e) o[e] *= corr;
      for (int j = 0; j < cnt; ++j) {
        const float pj = __shfl_sync(0xffffffffu, p, j), f = __shfl_sync(0xffffffffu, vs, j);
        const uint8_t* v = P.v_pool + (static_cast<size_t>(slot0 + j) * P.nkv + g) * D * sizeof(X);
        for (int e = 0; e < E; e += 2) {
          const float2 x = pair_at<X>(v, lane * (E / 2) + e / 2, f);
          o[e] += pj * x.x;
          o[e + 1] += pj * x.y;
        }
      }
    }
  }
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  if (lane == 0) s_ml[warp] = make_float2(m, l);
  __syncthreads();
  float top = -INFINITY, den = 0.f;
  for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, s_ml[w].x);
  for (int w = 0; w < kRowWarps; ++w) {
    const float f = weight_of(s_ml[w], top);
    den += f == 0.f ? 0.f : f * s_ml[w].y;
  }
  const float inv = den > 0.f ? 1.f / den : (den == 0.f ? 0.f : den);
  for (int i = tid; i < D / 2; i += blockDim.x) {
    float x = 0.f, y = 0.f;
    for (int w = 0; w < kRowWarps; ++w) {
      const float f = weight_of(s_ml[w], top);
      if (f != 0.f) x += f * s_o[w][2 * i], y += f * s_o[w][2 * i + 1];
    }
    static_cast<uint32_t*>(P.out)[(static_cast<size_t>(row) * P.nq + head) * (D / 2) + i] = pack2<BF16>(x * inv, y * inv);
  }
}

template <typename X, bool BF16>
int launch(const PagedAttnParams& p, cudaStream_t stream) {
  const dim3 grid(p.batch * p.rows_per_seq, p.nq);
  if (p.d == 128) attn_rows_kernel<X, BF16, 128><<<grid, 32 * kRowWarps, 0, stream>>>(p);
  else attn_rows_kernel<X, BF16, 64><<<grid, 32 * kRowWarps, 0, stream>>>(p);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_paged_attn_rows(const PagedAttnParams& p, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case DFLASH_F16: return launch<__half, false>(p, stream);
    case DFLASH_BF16: return launch<__nv_bfloat16, true>(p, stream);
    case DFLASH_E4M3_F16: return launch<uint8_t, false>(p, stream);
    default: return launch<uint8_t, true>(p, stream);
  }
}

}  // namespace dfl
