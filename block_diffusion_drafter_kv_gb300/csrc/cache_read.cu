// Rows of a paged cache, dense: positions first[s] .. first[s] + count[s] of every sequence, from 16
// or 8 bits, to fp16 or bf16. Bound: memory, each row read once and written once.
//
// A warp takes a row of positions x heads (or several, where they are short): the length and page are looked up
// once for it, then each lane has 8 values of K and of V at a time, 8 or 16 bytes in and 16 out each, with four such
// pairs under way. Measured: 8 sequences of up to 8192 positions, 8 heads of 128 in 8 bits 54 us (91% of the copy rate), in 16 bits
// 67 us (97%); 64 of 1024, 8 heads of 64 in 8 bits 29 us (72%). (A thread for every 16 values, which looks its row up by
// itself: 75, 91 and 35 us.)
#include <type_traits>

#include "quant.cuh"

namespace dfl {

namespace {

constexpr int kReadThreads = 256;
constexpr int kAhead = 4;

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

// X: uint8_t for an 8-bit cache. Lengths, page ids and scales by ordinary loads: the kernel before may still write them when
// this one starts, so they are not read-only for as long as it runs.
template <typename X, typename Y>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const ReadParams P) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr bool kBits8 = sizeof(X) == 1;
  using Word = std::conditional_t<kBits8, uint2, uint4>;  // a lane's 8 values
  const int lane = threadIdx.x & 31;
  const int width = P.nkv * P.d / 8, heads_step = P.d / 8;  // lanes' worth of a row, of a head
  const int per_warp = width < 32 ? 32 / width : 1;         // rows of a warp
  const int sub = width < 32 ? lane / width : 0, at0 = width < 32 ? lane - sub * width : lane;
  const int rows = P.batch * P.rows_per_seq;  // (less than 2^31)
  const int warps = gridDim.x * (kReadThreads / 32), warp = blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5);
  if (sub >= per_warp) return;
  for (long long row0 = static_cast<long long>(warp) * per_warp + sub; row0 < rows; row0 += static_cast<long long>(warps) * per_warp) {
    const int row = static_cast<int>(row0), s = row / P.rows_per_seq, r = row - s * P.rows_per_seq;
    const int first = P.first[s], count = P.count[s];
    if (first < 0 || count < 0 || count > P.rows_per_seq ||
        static_cast<long long>(first) + count > static_cast<long long>(P.pages_per_seq) * kPagePos) {
      if (r == 0 && at0 == 0) raise_flag(P.err, kDevCapacity);
      continue;
    }
    if (r >= count) continue;
    const int pos = first + r;
    const int page = P.page_table[static_cast<size_t>(s) * P.pages_per_seq + pos / kPagePos];
    if (page < 0 || page >= P.n_pages) {
      if (at0 == 0) raise_flag(P.err, kDevCapacity);
      continue;
    }
    const int slot = page * kPagePos + pos % kPagePos;
    const size_t from = static_cast<size_t>(slot) * P.nkv * P.d, to = static_cast<size_t>(row) * P.nkv * P.d;
    for (int at = at0; at < width; at += 32 * kAhead) {
      Word in[kAhead][2];
      uint32_t scale[kAhead][2];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          const int x = at + 32 * k;
          if (x >= width) break;
          in[k][which] = __ldcs(reinterpret_cast<const Word*>(reinterpret_cast<const X*>(which == 0 ? P.k_pool : P.v_pool) + from + x * 8));
          if (kBits8) scale[k][which] = P.scales[scale_index(slot, P.nkv, x / heads_step, which)];
        }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          const int x = at + 32 * k;
          if (x >= width) break;
          uint32_t out[4];
          const uint32_t* u = reinterpret_cast<const uint32_t*>(&in[k][which]);
          if constexpr (kBits8) {
            const float f = scale_value(scale[k][which]);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float2 v = __half22float2(from_e4m3x2(u[y >> 1] >> ((y & 1) * 16)));
              out[y] = pack<Y>(v.x * f, v.y * f);
            }
          } else {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float2 v = widen(X{}, u[y]);
              out[y] = pack<Y>(v.x, v.y);
            }
          }
          *reinterpret_cast<uint4*>(static_cast<Y*>(which == 0 ? P.k_out : P.v_out) + to + x * 8) = make_uint4(out[0], out[1], out[2], out[3]);
        }
      if (width < 32) break;  // (a row that shares its warp is done)
    }
  }
}

template <typename X, typename Y>
int launch(const ReadParams& p, int n_sms, cudaStream_t stream) {
  const int width = p.nkv * p.d / 8, per_cta = kReadThreads / 32 * (width < 32 ? 32 / width : 1);
  const long long blocks = (static_cast<long long>(p.batch) * p.rows_per_seq + per_cta - 1) / per_cta;
  cudaLaunchConfig_t cfg = {};
  // Wide rows: as good as one a warp, so that new warps' loads run under the others' stores; short ones, whose look-ups
  // count, several. 8 x 8192 rows of 1024 values in 8 bits: 54 us against 57; 64 x 1024 of 512 values: 31.6 against 29.5.
  const long long most = (width > 64 ? 64ll : 8ll) * n_sms;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most));
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
