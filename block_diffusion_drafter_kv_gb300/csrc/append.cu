// Rotary positions on a step's new q and k rows, and k and v into the paged cache, in one
// pass: every value is read once and written once, so the bound is memory bandwidth
// (2 bytes in, 2 bytes out per value; the rotary tables come from L2).
//
// A thread owns 16 dims of a head that are closed under the rotation: [8i, 8i + 8) and its
// partners rope_dim / 2 further on (half layout), or the eight pairs of [16i, 16i + 16)
// (interleaved), or 16 plain dims past rope_dim. Its eight angles are the same for every
// head of the row, so it keeps their cos and sin in registers and walks the row's heads. A CTA a
// row: many rows fill the SMs with small CTAs, whose loads overlap each other's latency.
//
// Measured (bf16, 32 query heads on 8 KV heads, d 128): a prompt of 8191 rows 33.0 us, 90% of the
// copy rate (102.8 MB read, as much written, most of it still in L2 at the end); 32 blocks of 16
// rows 4.1 us and one row 2.1 us, a launch and the latencies slot, tables, values.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "quant.cuh"

namespace dfl {

namespace {

template <typename T>
DEV float to_f32(T v);
template <>
DEV float to_f32<__half>(__half v) {
  return __half2float(v);
}
template <>
DEV float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <typename T>
DEV T from_f32(float v);
template <>
DEV __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}
template <>
DEV __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

constexpr int kThreads = 128;

// One CTA per row. blockDim covers d / 16 items of kThreads / (d / 16) heads at a time.
template <typename X, typename Y>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams P) {
  pdl_wait();
  pdl_launch_dependents();
  const long long row = blockIdx.x;
  const int slot = __ldcg(P.slots + row);
  const int s = static_cast<int>(row / P.rows_per_seq);
  const int before = P.prefix_len ? __ldcg(P.prefix_len) : 0;
  const long long pos = static_cast<long long>(__ldcg(P.len + s)) + (row - static_cast<long long>(s) * P.rows_per_seq) + before;
  if (slot == -1) return;
  if (slot < 0 || slot >= P.pool_rows || before < 0 || (P.rope_dim > 0 && (pos < 0 || pos >= P.positions))) {
    if (threadIdx.x == 0) raise_flag(P.err, kDevCapacity);
    return;
  }
  const int items = P.d / 16;  // 4 or 8
  const int item = threadIdx.x % items, h0 = threadIdx.x / items, step = kThreads / items;
  const bool turn = item * 16 < P.rope_dim;
  const int half = P.rope_dim / 2;
  // the two runs of eight dims
  const int d0 = turn && !P.interleaved ? 8 * item : 16 * item;
  const int d1 = turn && !P.interleaved ? d0 + half : d0 + 8;
  float cs[8], sn[8];
  if (turn) {
    const float4* c4 = reinterpret_cast<const float4*>(P.cos + pos * half + 8 * item);
    const float4* s4 = reinterpret_cast<const float4*>(P.sin + pos * half + 8 * item);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 c = __ldg(c4 + i), t = __ldg(s4 + i);
      cs[4 * i] = c.x, cs[4 * i + 1] = c.y, cs[4 * i + 2] = c.z, cs[4 * i + 3] = c.w;
      sn[4 * i] = t.x, sn[4 * i + 1] = t.y, sn[4 * i + 2] = t.z, sn[4 * i + 3] = t.w;
    }
  }
  const int nq = P.q ? P.nq : 0, heads = nq + 2 * P.nkv;
  for (int h = h0; h < heads; h += step) {
    const X* src;
    Y* dst;
    bool rot = turn;
    if (h < nq) {
      src = static_cast<const X*>(P.q) + row * P.q_stride + static_cast<size_t>(h) * P.d;
      dst = static_cast<Y*>(P.q_out) + (static_cast<size_t>(row) * P.nq + h) * P.d;
    } else if (h < nq + P.nkv) {
      src = static_cast<const X*>(P.k) + row * P.k_stride + static_cast<size_t>(h - nq) * P.d;
      dst = static_cast<Y*>(P.k_pool) + (static_cast<size_t>(slot) * P.nkv + (h - nq)) * P.d;
    } else {
      src = static_cast<const X*>(P.v) + row * P.v_stride + static_cast<size_t>(h - nq - P.nkv) * P.d;
      dst = static_cast<Y*>(P.v_pool) + (static_cast<size_t>(slot) * P.nkv + (h - nq - P.nkv)) * P.d;
      rot = false;
    }
    uint4 in[2] = {__ldcs(reinterpret_cast<const uint4*>(src + d0)), __ldcs(reinterpret_cast<const uint4*>(src + d1))};
    const X* x = reinterpret_cast<const X*>(in);
    uint4 out[2];
    Y* y = reinterpret_cast<Y*>(out);
    if (rot) {
      auto pair = [&](int i0, int i1, int e) {
        const float a = to_f32(x[i0]), b = to_f32(x[i1]);
        y[i0] = from_f32<Y>(a * cs[e] - b * sn[e]);
        y[i1] = from_f32<Y>(b * cs[e] + a * sn[e]);
      };
      if (P.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) pair(2 * e, 2 * e + 1, e);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) pair(e, e + 8, e);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = from_f32<Y>(to_f32(x[e]));
    }
    *reinterpret_cast<uint4*>(dst + d0) = out[0];
    *reinterpret_cast<uint4*>(dst + d1) = out[1];
  }
}

// The same for an 8-bit cache: q as above, K and V rows in e4m3 with a scale byte. The threads of a head
// (4 or 8 neighbouring lanes) join their largest magnitude. The rotation's products and sums are
// rounded one by one, not fused: a value next to a rounding border of e4m3 or of the scale then goes the
// way that plain fp32 arithmetic takes it.
//
// Measured (32 query heads on 8 KV heads, d 128): a prompt of 8191 rows 33.8 us, 82% of the copy rate, with 64
// threads a row; 35.4 us with 128, 48 us with 256: a small CTA has its passes' loads, joins and stores one
// after another, and more rows at a time hide them.
constexpr int kThreads8 = 64;

template <typename X, typename Y>
__global__ void __launch_bounds__(kThreads8) append8_kernel(const AppendParams P) {
  pdl_wait();
  pdl_launch_dependents();
  const long long row = blockIdx.x;
  const int slot = __ldcg(P.slots + row);
  const int s = static_cast<int>(row / P.rows_per_seq);
  const int before = P.prefix_len ? __ldcg(P.prefix_len) : 0;
  const long long pos = static_cast<long long>(__ldcg(P.len + s)) + (row - static_cast<long long>(s) * P.rows_per_seq) + before;
  if (slot == -1) return;
  if (slot < 0 || slot >= P.pool_rows || before < 0 || (P.rope_dim > 0 && (pos < 0 || pos >= P.positions))) {
    if (threadIdx.x == 0) raise_flag(P.err, kDevCapacity);
    return;
  }
  const int items = P.d / 16;  // 4 or 8
  const int item = threadIdx.x % items, h0 = threadIdx.x / items, step = kThreads8 / items;
  const bool turn = item * 16 < P.rope_dim;
  const int half = P.rope_dim / 2;
  const int d0 = turn && !P.interleaved ? 8 * item : 16 * item;
  const int d1 = turn && !P.interleaved ? d0 + half : d0 + 8;
  float cs[8], sn[8];
  if (turn) {
    const float4* c4 = reinterpret_cast<const float4*>(P.cos + pos * half + 8 * item);
    const float4* s4 = reinterpret_cast<const float4*>(P.sin + pos * half + 8 * item);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 c = __ldg(c4 + i), t = __ldg(s4 + i);
      cs[4 * i] = c.x, cs[4 * i + 1] = c.y, cs[4 * i + 2] = c.z, cs[4 * i + 3] = c.w;
      sn[4 * i] = t.x, sn[4 * i + 1] = t.y, sn[4 * i + 2] = t.z, sn[4 * i + 3] = t.w;
    }
  }
  const int nq = P.q ? P.nq : 0, heads = nq + 2 * P.nkv;
  // (the lanes of a warp walk together, past the last head too: the maxima are joined by shuffles; the next heads'
  // values are asked for before these are worked on)
  auto load = [&](int base, uint4 (&to)[2]) {
    const int h = min(base + h0, heads - 1), which = h < nq ? -1 : h < nq + P.nkv ? 0 : 1, kv = h - nq - (which == 1 ? P.nkv : 0);
    const X* src = which < 0 ? static_cast<const X*>(P.q) + row * P.q_stride + static_cast<size_t>(h) * P.d
                             : static_cast<const X*>(which == 0 ? P.k : P.v) + row * (which == 0 ? P.k_stride : P.v_stride) +
                                   static_cast<size_t>(kv) * P.d;
    to[0] = __ldcs(reinterpret_cast<const uint4*>(src + d0)), to[1] = __ldcs(reinterpret_cast<const uint4*>(src + d1));
  };
  uint4 in[2], next[2];
  load(0, next);
  for (int base = 0; base < heads; base += step) {
    const int h = min(base + h0, heads - 1);
    const bool there = base + h0 < heads;
    const int which = h < nq ? -1 : h < nq + P.nkv ? 0 : 1, kv = h - nq - (which == 1 ? P.nkv : 0);
    in[0] = next[0], in[1] = next[1];
    if (base + step < heads) load(base + step, next);
    const X* x = reinterpret_cast<const X*>(in);
    float y[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = to_f32(x[e]);
    if (turn && which != 1) {
      auto pair = [&](float& a, float& b, int e) {
        const float u = __fsub_rn(__fmul_rn(a, cs[e]), __fmul_rn(b, sn[e]));
        b = __fadd_rn(__fmul_rn(b, cs[e]), __fmul_rn(a, sn[e]));
        a = u;
      };
      if (P.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) pair(y[2 * e], y[2 * e + 1], e);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) pair(y[e], y[e + 8], e);
      }
    }
    uint32_t top = 0;  // the bits of a magnitude are ordered as it is, infinities and NaN above all others
    if (__any_sync(0xffffffffu, which >= 0)) {
#pragma unroll
      for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
      for (int o = 1; o < items; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (!there) continue;
    if (which < 0) {
      Y* dst = static_cast<Y*>(P.q_out) + (static_cast<size_t>(row) * P.nq + h) * P.d;
      uint4 out[2];
      Y* o = reinterpret_cast<Y*>(out);
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = from_f32<Y>(y[e]);
      *reinterpret_cast<uint4*>(dst + d0) = out[0];
      *reinterpret_cast<uint4*>(dst + d1) = out[1];
      continue;
    }
    const int byte = scale_byte(top);
    uint32_t out[4] = {0, 0, 0, 0};
    if (byte != kScaleNan) {
      const float f = exponent_value(kScaleBias - byte);
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e >> 1] |= to_e4m3x2(y[2 * e] * f, y[2 * e + 1] * f) << ((e & 1) * 16);
    }
    uint8_t* dst = static_cast<uint8_t*>(which == 0 ? P.k_pool : P.v_pool) + (static_cast<size_t>(slot) * P.nkv + kv) * P.d;
    *reinterpret_cast<uint2*>(dst + d0) = make_uint2(out[0], out[1]);
    *reinterpret_cast<uint2*>(dst + d1) = make_uint2(out[2], out[3]);
    if (item == 0) P.scales[scale_index(slot, P.nkv, kv, which)] = static_cast<uint8_t>(byte);
  }
}

}  // namespace

int launch_append(const AppendParams& p, int x_dtype, int pool_dtype, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool xh = x_dtype == DFLASH_F16, yh = pool_dtype == DFLASH_F16 || pool_dtype == DFLASH_E4M3_F16;
  cudaError_t e;
  if (pool_dtype == DFLASH_E4M3_F16 || pool_dtype == DFLASH_E4M3_BF16) {
    cfg.blockDim = dim3(kThreads8);
    if (xh && yh) e = cudaLaunchKernelEx(&cfg, append8_kernel<__half, __half>, p);
    else if (xh) e = cudaLaunchKernelEx(&cfg, append8_kernel<__half, __nv_bfloat16>, p);
    else if (yh) e = cudaLaunchKernelEx(&cfg, append8_kernel<__nv_bfloat16, __half>, p);
    else e = cudaLaunchKernelEx(&cfg, append8_kernel<__nv_bfloat16, __nv_bfloat16>, p);
  } else if (xh && yh) e = cudaLaunchKernelEx(&cfg, append_kernel<__half, __half>, p);
  else if (xh) e = cudaLaunchKernelEx(&cfg, append_kernel<__half, __nv_bfloat16>, p);
  else if (yh) e = cudaLaunchKernelEx(&cfg, append_kernel<__nv_bfloat16, __half>, p);
  else e = cudaLaunchKernelEx(&cfg, append_kernel<__nv_bfloat16, __nv_bfloat16>, p);
  return static_cast<int>(e);
}

}  // namespace dfl
