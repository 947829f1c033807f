// The block-scaled FP8 form of a shared block and of activations, and the
// theta forward over the two.
//
// Encoding: E4M3 codes with one power-of-two scale (E8M0: exponent + 127) per
// block of 128 -- 128 x 128 of W0, one token x 128 columns of X. The scale is
// the least 2^e that brings the block's largest finite magnitude to 448 (the
// largest E4M3 value) or below; a block of zeros takes scale 1. E4M3 is a
// floating-point format, so the scale only places the block in its exponent
// range: a power of two loses no significand bits, divides exactly, and is
// what the tensor cores' block-scaled MMA applies by itself. A code is
// x * 2^-e rounded to nearest even; a value that is not finite becomes the
// NaN code and does not count for the scale, so it stays visible in every
// result it enters instead of turning into 448 * 2^e.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace theta {

namespace {

constexpr int kBlock = kFp8Block;
constexpr int kThreads = 256;
constexpr float kMaxFinite = 3.402823466e38f;

// The E8M0 byte of a block whose largest finite magnitude is amax: with
// amax = 1.f * 2^(E - 127), 448 * 2^e = 1.75 * 2^(e + 8), so e + 127 = E - 8,
// plus one when the significand is above 1.75; at least 0 (2^-127).
__device__ __forceinline__ int scale_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0) return 127;
  const int b = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(b, 0);
}

// 2^(127 - byte), the reciprocal of the scale (byte <= 247: always normal).
__device__ __forceinline__ float inverse_scale(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

__device__ __forceinline__ float scaled(float x, float inv) {
  return fabsf(x) <= kMaxFinite ? x * inv : __uint_as_float(0x7fffffffu);
}

// E4M3 codes of four values, the first in the low byte. A NaN gives 0x7f.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// 8 values as loaded (16 bytes of bf16, 32 of fp32), kept packed so that a
// thread can hold many of them in flight.
//   abs_max   the largest magnitude, NaN ignored, infinities not
//   encode    the codes of x * inv, for values without infinities
// The encoders are bound by instructions as much as by HBM, so bf16 is worked
// on in pairs: the maximum, and the product with a power of two, which is
// exact in bf16 (results below its smallest normal number encode to 0 either
// way).
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16> {
  __nv_bfloat162 v[4];
  __device__ __forceinline__ void load(const bf16* p) {
    *reinterpret_cast<uint4*>(v) = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void zero() { *reinterpret_cast<uint4*>(v) = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const { unpack(*reinterpret_cast<const uint4*>(v), f); }
  static __device__ __forceinline__ __nv_bfloat162 max_init() { return __floats2bfloat162_rn(0.f, 0.f); }
  __device__ __forceinline__ void abs_max(__nv_bfloat162& m) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) m = __hmax2(m, __habs2(v[q]));
  }
  static __device__ __forceinline__ float max_value(const __nv_bfloat162& m) {
    return fmaxf(__low2float(m), __high2float(m));
  }
  __device__ __forceinline__ uint2 encode(float inv) const {
    const __nv_bfloat162 k = __float2bfloat162_rn(inv);
    float f[8];
    uint4 s;
    uint32_t* w = reinterpret_cast<uint32_t*>(&s);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __nv_bfloat162 y = __hmul2_rn(v[q], k);
      w[q] = *reinterpret_cast<const uint32_t*>(&y);
    }
    unpack(s, f);
    return make_uint2(encode4(f[0], f[1], f[2], f[3]), encode4(f[4], f[5], f[6], f[7]));
  }
};
template <>
struct Raw8<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v[e];
  }
  static __device__ __forceinline__ float max_init() { return 0.f; }
  __device__ __forceinline__ void abs_max(float& m) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
  }
  static __device__ __forceinline__ float max_value(float m) { return m; }
  __device__ __forceinline__ uint2 encode(float inv) const {
    return make_uint2(encode4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                      encode4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
  }
};

// The rare form, for a block that holds an infinity: magnitudes and codes
// value by value.
template <typename T>
__device__ __noinline__ float finite_abs_max(const Raw8<T>& r, float mx) {
  float f[8];
  r.get(f);
#pragma unroll
  for (int e = 0; e < 8; ++e) mx = fabsf(f[e]) <= kMaxFinite ? fmaxf(mx, fabsf(f[e])) : mx;
  return mx;
}
template <typename T>
__device__ __noinline__ uint2 encode_checked(const Raw8<T>& r, float inv) {
  float v[8];
  r.get(v);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = scaled(v[e], inv);
  return make_uint2(encode4(v[0], v[1], v[2], v[3]), encode4(v[4], v[5], v[6], v[7]));
}

// The largest magnitude of the CTA's values: `mx` reduced over its threads.
__device__ __forceinline__ float cta_max(float mx, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = mx;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) mx = fmaxf(mx, red[i]);
  return mx;
}

// One CTA per 128 x 128 block of W0: a thread holds 8 vectors of 8 values
// (rows t / 16 + 16 j), so the block is read once, with all its loads in
// flight, and written from registers. [21504, 5376]: 53 us in bf16, 86 in fp32,
// 6.6 and 6.7 TB/s, the rate of a plain copy.
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2)
fp8_quantize_kernel(const T* __restrict__ W, int64_t O, int64_t I, uint8_t* __restrict__ codes,
                    uint8_t* __restrict__ scales) {
  __shared__ float red[2][kThreads / 32];
  pdl_enter(W);
  const int64_t nb = ceil_div(I, kBlock);
  const int64_t bo = blockIdx.x / nb, bi = blockIdx.x % nb;
  const int64_t r0 = bo * kBlock + threadIdx.x / 16, col = bi * kBlock + (threadIdx.x % 16) * 8;
  const int rows = col < I ? (int)max((int64_t)0, min((int64_t)8, ceil_div(O - r0, 16))) : 0;  // of this thread
  const T* src = W + r0 * I + col;
  Raw8<T> raw[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j < rows)
      raw[j].load(src + j * 16 * I);
    else
      raw[j].zero();
  }
  auto m = Raw8<T>::max_init();
#pragma unroll
  for (int j = 0; j < 8; ++j) raw[j].abs_max(m);
  float mx = cta_max(Raw8<T>::max_value(m), red[0]);
  const bool rare = mx > kMaxFinite;
  if (rare) {
    mx = 0.f;
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
      Raw8<T> x;  // read again: indexing raw[] here would put it in local memory
      x.zero();
      if (j < rows) x.load(src + j * 16 * I);
      mx = finite_abs_max(x, mx);
    }
    mx = cta_max(mx, red[1]);
  }
  const int byte = scale_byte(mx);
  const float inv = inverse_scale(byte);
  uint8_t* dst = codes + r0 * I + col;
  if (!rare) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < rows) *reinterpret_cast<uint2*>(dst + j * 16 * I) = raw[j].encode(inv);
  } else {
#pragma unroll 1
    for (int j = 0; j < rows; ++j) {
      Raw8<T> x;
      x.load(src + j * 16 * I);
      *reinterpret_cast<uint2*>(dst + j * 16 * I) = encode_checked(x, inv);
    }
  }
  if (threadIdx.x == 0) scales[bo * nb + bi] = (uint8_t)byte;
}

// The largest magnitudes of two blocks over 16 lanes: for bf16 both in the
// halves of one word.
__device__ __forceinline__ void group_max(const Raw8<bf16>& a, const Raw8<bf16>& b, float& ma, float& mb) {
  __nv_bfloat162 x = Raw8<bf16>::max_init(), y = x;
  a.abs_max(x);
  b.abs_max(y);
  __nv_bfloat162 m = __hmax2(__lows2bfloat162(x, y), __highs2bfloat162(x, y));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = __hmax2(m, __shfl_xor_sync(0xffffffffu, m, o));
  ma = __low2float(m);
  mb = __high2float(m);
}
__device__ __forceinline__ void group_max(const Raw8<float>& a, const Raw8<float>& b, float& ma, float& mb) {
  ma = mb = 0.f;
  a.abs_max(ma);
  b.abs_max(mb);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, o));
    mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
  }
}

// 16 lanes per block of 128 columns of one token, kRowBlocks consecutive
// blocks of the token in flight per lane. A CTA's 16 groups of lanes take up to
// 16 tokens (1 << row_bits) side by side, so that a block's scales, which lie
// token by token, leave as runs of bytes: with all 16 groups on one token they
// were single bytes, a sector each. [2048, 21504]: 25.8 us in bf16, 5.1 TB/s,
// 74% of the issue slots used, and 47 in fp32, 4.7 TB/s; one token of 5376 1.5
// us (2.9 with eight blocks a lane, which bf16 rows did not gain from either:
// 29.6).
constexpr int kRowBlocks = 2;
template <typename T>
__global__ void __launch_bounds__(kThreads) fp8_quantize_rows_kernel(const T* __restrict__ X, int64_t M, int64_t I,
                                                                     int row_bits, uint8_t* __restrict__ codes,
                                                                     uint8_t* __restrict__ scales) {
  __shared__ uint8_t bytes[kRowBlocks][kThreads / 16];
  pdl_enter(X);
  const uint32_t nb = (uint32_t)ceil_div(I, kBlock), units = (nb + kRowBlocks - 1) / kRowBlocks;
  const uint32_t group = threadIdx.x / 16, col_bits = 4 - row_bits;
  // CTAs walk the columns of a band of tokens first
  const uint32_t across = (units + (1u << col_bits) - 1) >> col_bits;
  const uint32_t band = blockIdx.x / across;
  const uint32_t m = (band << row_bits) + (group & ((1u << row_bits) - 1));
  const uint32_t b0 = (((blockIdx.x - band * across) << col_bits) + (group >> row_bits)) * kRowBlocks;
  const int lane = threadIdx.x % 16;
  const int64_t at = (int64_t)m * I + (int64_t)b0 * kBlock + lane * 8;
  // this lane's vectors inside the row
  const int live = m < M && b0 < nb ? (int)max((int64_t)0, min((int64_t)kRowBlocks,
                                                     ceil_div(I - (int64_t)b0 * kBlock - lane * 8, kBlock)))
                         : 0;
  Raw8<T> raw[kRowBlocks];
#pragma unroll
  for (int j = 0; j < kRowBlocks; ++j) {
    if (j < live)
      raw[j].load(X + at + j * kBlock);
    else
      raw[j].zero();
  }
  float top[kRowBlocks];
  group_max(raw[0], raw[1], top[0], top[1]);
#pragma unroll
  for (int j = 0; j < kRowBlocks; ++j) {
    float mx = top[j];
    const bool rare = mx > kMaxFinite;  // the same in the block's 16 lanes
    if (__any_sync(0xffffffffu, rare)) {
      float fm = finite_abs_max(raw[j], 0.f);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) fm = fmaxf(fm, __shfl_xor_sync(0xffffffffu, fm, o));
      mx = fm;
    }
    const int byte = scale_byte(mx);
    const float inv = inverse_scale(byte);
    if (j < live) {
      *reinterpret_cast<uint2*>(codes + at + j * kBlock) = rare ? encode_checked(raw[j], inv) : raw[j].encode(inv);
    }
    if (lane == 0) bytes[j][group] = (uint8_t)byte;
  }
  __syncthreads();
  if (threadIdx.x < kRowBlocks * 16) {
    // the thread of (block, group): tokens of a block are consecutive threads
    const uint32_t j = threadIdx.x / 16, g = threadIdx.x % 16;
    const int64_t token = ((int64_t)band << row_bits) + (g & ((1u << row_bits) - 1));
    const uint32_t b = (((blockIdx.x - band * across) << col_bits) + (g >> row_bits)) * kRowBlocks + j;
    if (token < M && b < nb) scales[(int64_t)b * M + token] = bytes[j][g];
  }
}

}  // namespace

cudaError_t launch_fp8_quantize(const LaunchCtx& c, theta_dtype dt, const void* W, int64_t O, int64_t I, void* codes,
                                void* scales) {
  const dim3 grid((unsigned)(ceil_div(O, kBlock) * ceil_div(I, kBlock)));
  auto* q = static_cast<uint8_t*>(codes);
  auto* e = static_cast<uint8_t*>(scales);
  return dt == THETA_BF16 ? launch_pdl(fp8_quantize_kernel<bf16>, grid, dim3(kThreads), 0, c.stream, 1,
                                       static_cast<const bf16*>(W), O, I, q, e)
                          : launch_pdl(fp8_quantize_kernel<float>, grid, dim3(kThreads), 0, c.stream, 1,
                                       static_cast<const float*>(W), O, I, q, e);
}

cudaError_t launch_fp8_quantize_rows(const LaunchCtx& c, theta_dtype dt, const void* X, int64_t M, int64_t I,
                                     void* codes, void* scales) {
  const int row_bits = M >= 16 ? 4 : M >= 8 ? 3 : M >= 4 ? 2 : M >= 2 ? 1 : 0;
  const int64_t units = ceil_div(ceil_div(I, kBlock), kRowBlocks);
  const dim3 grid((unsigned)(ceil_div(M, (int64_t)1 << row_bits) * ceil_div(units, (int64_t)16 >> row_bits)));
  auto* q = static_cast<uint8_t*>(codes);
  auto* e = static_cast<uint8_t*>(scales);
  return dt == THETA_BF16 ? launch_pdl(fp8_quantize_rows_kernel<bf16>, grid, dim3(kThreads), 0, c.stream, 1,
                                       static_cast<const bf16*>(X), M, I, row_bits, q, e)
                          : launch_pdl(fp8_quantize_rows_kernel<float>, grid, dim3(kThreads), 0, c.stream, 1,
                                       static_cast<const float*>(X), M, I, row_bits, q, e);
}

}  // namespace theta
