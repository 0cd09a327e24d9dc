// Rows of a paged cache, dense: positions first[s] .. first[s] + count[s] of every sequence, from 16
// or 8 bits, to fp16 or bf16. Bound: memory, each row read once and written once.
//
// A thread takes 16 values of a row's K and the same of its V: 16 or 32 bytes in, 32 out.
#include "quant.cuh"

namespace dfl {

namespace {

constexpr int kReadThreads = 256;

template <typename Y>
DEV uint32_t pack(float lo, float hi);
template <>
DEV uint32_t pack<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
DEV uint32_t pack<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
DEV float2 widen(__half, uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
DEV float2 widen(__nv_bfloat16, uint32_t u) { return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u)); }

// X: uint8_t for an 8-bit cache.
template <typename X, typename Y>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const ReadParams P) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr bool kBits8 = sizeof(X) == 1;
  const int per_row = P.nkv * (P.d / 16);
  const long long items = static_cast<long long>(P.batch) * P.rows_per_seq * per_row;
  for (long long i = blockIdx.x * static_cast<long long>(kReadThreads) + threadIdx.x; i < items; i += static_cast<long long>(gridDim.x) * kReadThreads) {
    const long long row = i / per_row;
    const int part = static_cast<int>(i - row * per_row);
    const int s = static_cast<int>(row / P.rows_per_seq), r = static_cast<int>(row - static_cast<long long>(s) * P.rows_per_seq);
    const int first = __ldcg(P.first + s), count = __ldcg(P.count + s);
    if (first < 0 || count < 0 || count > P.rows_per_seq ||
        static_cast<long long>(first) + count > static_cast<long long>(P.pages_per_seq) * kPagePos) {
      if (r == 0 && part == 0) raise_flag(P.err, kDevCapacity);
      continue;
    }
    if (r >= count) continue;
    const int pos = first + r;
    const int page = __ldcg(P.page_table + static_cast<size_t>(s) * P.pages_per_seq + pos / kPagePos);
    if (page < 0 || page >= P.n_pages) {
      if (part == 0) raise_flag(P.err, kDevCapacity);
      continue;
    }
    const int slot = page * kPagePos + pos % kPagePos;
    const size_t at = static_cast<size_t>(slot) * P.nkv * P.d + part * 16, to = static_cast<size_t>(row) * P.nkv * P.d + part * 16;
    const int head = part / (P.d / 16);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const X* src = reinterpret_cast<const X*>(which == 0 ? P.k_pool : P.v_pool) + at;
      uint32_t out[8];
      if constexpr (kBits8) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src));
        const float f = scale_value(__ldg(P.scales + scale_index(slot, P.nkv, head, which)));
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 x = __half22float2(from_e4m3x2(u[k >> 1] >> ((k & 1) * 16)));
          out[k] = pack<Y>(x.x * f, x.y * f);
        }
      } else {
        const uint4 v[2] = {__ldcs(reinterpret_cast<const uint4*>(src)), __ldcs(reinterpret_cast<const uint4*>(src) + 1)};
        const uint32_t u[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 x = widen(X{}, u[k]);
          out[k] = pack<Y>(x.x, x.y);
        }
      }
      uint4* dst = reinterpret_cast<uint4*>(static_cast<Y*>(which == 0 ? P.k_out : P.v_out) + to);
      dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
      dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
  }
}

template <typename X, typename Y>
int launch(const ReadParams& p, int n_sms, cudaStream_t stream) {
  const long long items = static_cast<long long>(p.batch) * p.rows_per_seq * p.nkv * (p.d / 16);
  const long long blocks = (items + kReadThreads - 1) / kReadThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < 8ll * n_sms ? blocks : 8ll * n_sms));
  cfg.blockDim = dim3(kReadThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, cache_read_kernel<X, Y>, p));
}

template <typename Y>
int launch_from(const ReadParams& p, int pool_dtype, int n_sms, cudaStream_t stream) {
  if (pool_dtype == DFLASH_F16) return launch<__half, Y>(p, n_sms, stream);
  if (pool_dtype == DFLASH_BF16) return launch<__nv_bfloat16, Y>(p, n_sms, stream);
  return launch<uint8_t, Y>(p, n_sms, stream);
}

}  // namespace

int launch_cache_read(const ReadParams& p, int pool_dtype, int out_dtype, int n_sms, cudaStream_t stream) {
  return out_dtype == DFLASH_F16 ? launch_from<__half>(p, pool_dtype, n_sms, stream)
                                 : launch_from<__nv_bfloat16>(p, pool_dtype, n_sms, stream);
}

}  // namespace dfl
