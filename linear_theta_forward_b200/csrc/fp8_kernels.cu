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

__device__ __forceinline__ float finite_abs_max(float mx, float x) {
  const float a = fabsf(x);
  return a <= kMaxFinite ? fmaxf(mx, a) : mx;
}

__device__ __forceinline__ float scaled(float x, float inv) {
  return fabsf(x) <= kMaxFinite ? x * inv : __uint_as_float(0x7fffffffu);
}

// E4M3 codes of four values, the first in the low byte.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ uint2 encode8(const float (&f)[8], float inv) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = scaled(f[e], inv);
  return make_uint2(encode4(v[0], v[1], v[2], v[3]), encode4(v[4], v[5], v[6], v[7]));
}

// 8 values as loaded (16 bytes of bf16, 32 of fp32), kept packed so that a
// thread can hold many of them in flight.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const { unpack(v, f); }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};

// One CTA per 128 x 128 block of W0: a thread holds 8 vectors of 8 values
// (rows t / 16 + 16 j), so the block is read once, with all its loads in
// flight, and written from registers.
template <typename T>
__global__ void __launch_bounds__(kThreads) fp8_quantize_kernel(const T* __restrict__ W, int64_t O, int64_t I,
                                                                uint8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
  __shared__ float red[kThreads / 32];
  pdl_enter(W);
  const int64_t nb = ceil_div(I, kBlock);
  const int64_t bo = blockIdx.x / nb, bi = blockIdx.x % nb;
  const int64_t r0 = bo * kBlock + threadIdx.x / 16, col = bi * kBlock + (threadIdx.x % 16) * 8;
  Raw8<T> raw[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (r0 + 16 * j < O && col < I)
      raw[j].load(W + (r0 + 16 * j) * I + col);
    else
      raw[j].zero();
  }
  float mx = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float f[8];
    raw[j].get(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = finite_abs_max(mx, f[e]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = mx;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) mx = fmaxf(mx, red[i]);
  const int byte = scale_byte(mx);
  const float inv = inverse_scale(byte);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (r0 + 16 * j >= O || col >= I) continue;
    float f[8];
    raw[j].get(f);
    *reinterpret_cast<uint2*>(codes + (r0 + 16 * j) * I + col) = encode8(f, inv);
  }
  if (threadIdx.x == 0) scales[bo * nb + bi] = (uint8_t)byte;
}

// 16 lanes per block of 128 columns of one token, kRowBlocks consecutive
// blocks of the token in flight per lane.
constexpr int kRowBlocks = 4;
template <typename T>
__global__ void __launch_bounds__(kThreads) fp8_quantize_rows_kernel(const T* __restrict__ X, int64_t M, int64_t I,
                                                                     uint8_t* __restrict__ codes,
                                                                     uint8_t* __restrict__ scales) {
  pdl_enter(X);
  const int64_t nb = ceil_div(I, kBlock), units = ceil_div(nb, kRowBlocks);
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 16) + threadIdx.x / 16;
  const int64_t m = unit / units, b0 = unit % units * kRowBlocks;
  const bool live = m < M;
  const int lane = threadIdx.x % 16;
  Raw8<T> raw[kRowBlocks];
#pragma unroll
  for (int j = 0; j < kRowBlocks; ++j) {
    const int64_t col = (b0 + j) * kBlock + lane * 8;
    if (live && col < I)
      raw[j].load(X + m * I + col);
    else
      raw[j].zero();
  }
#pragma unroll
  for (int j = 0; j < kRowBlocks; ++j) {
    const int64_t col = (b0 + j) * kBlock + lane * 8;
    float f[8];
    raw[j].get(f);
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = finite_abs_max(mx, f[e]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const int byte = scale_byte(mx);
    if (live && col < I) {
      *reinterpret_cast<uint2*>(codes + m * I + col) = encode8(f, inverse_scale(byte));
      if (lane == 0) scales[(b0 + j) * M + m] = (uint8_t)byte;
    }
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
  const int64_t units = M * ceil_div(ceil_div(I, kBlock), kRowBlocks);
  const dim3 grid((unsigned)ceil_div(units, kThreads / 16));
  auto* q = static_cast<uint8_t*>(codes);
  auto* e = static_cast<uint8_t*>(scales);
  return dt == THETA_BF16 ? launch_pdl(fp8_quantize_rows_kernel<bf16>, grid, dim3(kThreads), 0, c.stream, 1,
                                       static_cast<const bf16*>(X), M, I, q, e)
                          : launch_pdl(fp8_quantize_rows_kernel<float>, grid, dim3(kThreads), 0, c.stream, 1,
                                       static_cast<const float*>(X), M, I, q, e);
}

size_t forward_fp8_workspace_bytes(int64_t M, int r) { return forward_fp8_umma_workspace_bytes(M, r); }

int launch_forward_fp8(const LaunchCtx& c, const void* X, const void* xq, const void* xs, const void* wq,
                       const void* ws, const float* s, const void* U, const void* V, int64_t M, int64_t O, int64_t I,
                       int r, void* Y, void* work, cudaError_t* ce) {
  return launch_forward_fp8_umma(c, X, xq, xs, wq, ws, s, U, V, M, O, I, r, Y, work, ce);
}

}  // namespace theta
