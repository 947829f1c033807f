// Per-head RMS norm of queries and keys with the position rotation, the step
// between the q and k projections and attention:
//   h = x / sqrt(mean(x^2) + eps) * (w + offset)        for each head of D values
//   y_a = h_a cos t - h_b sin t,  y_b = h_b cos t + h_a sin t
// over the pairs (a, b) of the head's first `rotary` values, t = position *
// inv_freq[pair]; the other values are only normed.
//
// The bound is HBM (each value read once, written once; a few operations an
// element). A group of G lanes owns a head, a lane one or more vectors of 8
// values. With r = 1 / sqrt(...) one number per head, a value's result is
//   y = r (x A + p B),   p the pair's other value,
//   A = (w + offset) cos t,   B = -/+ (w_p + offset) sin t,
// and A, B depend on the token and the value's place only, so a lane forms
// them once and keeps them in registers over all the heads it walks.
//
// Angles: t in turns, position * inv_freq / 2 pi in fp64 with whole turns
// taken off before rounding to fp32, so that positions in the millions keep
// their full precision; the block computes one sine and cosine per pair and
// token, shared by its heads.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace theta {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDim = 1024;

struct HeadArgs {
  HeadSide side[2];  // queries, keys
  const int64_t* pos;
  const float* inv_freq;
  int D, rotary;
  int aligned;  // half-split pairs whose halves are whole 8-value vectors
  float offset, eps;
  int per_block;  // heads (queries then keys) of one block
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    unpack(*reinterpret_cast<const uint4*>(p), f);
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = pack(f, (uint4*)nullptr);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// G lanes a head, VPL vectors of 8 values a lane.
template <typename T, int G, int VPL, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) heads_kernel(const __grid_constant__ HeadArgs a) {
  __shared__ float cs[kMaxDim / 2], sn[kMaxDim / 2];
  const int64_t* pos = a.pos;
  const float* freq = a.inv_freq;
  pdl_enter(pos, freq);
  const int64_t m = blockIdx.x;
  const int half = a.rotary / 2;
  if (half > 0) {
    const double turns0 = (double)pos[m] * 0.15915494309189535;  // position / 2 pi
    for (int i = threadIdx.x; i < half; i += kThreads) {
      // the nearest quarter turn k and what is left of it, exact in fp64; the
      // remainder is at most an eighth of a turn, so its fp32 rounding is
      // below 2^-25 of a radian
      const double t4 = 4.0 * (turns0 * (double)freq[i]);
      const double k = rint(t4);
      float s, co;
      sincospif(0.5f * (float)(t4 - k), &s, &co);
      const int quarter = (int)((long long)k & 3);
      const float c1 = quarter & 1 ? -s : co, s1 = quarter & 1 ? co : s;
      cs[i] = quarter & 2 ? -c1 : c1;
      sn[i] = quarter & 2 ? -s1 : s1;
    }
    __syncthreads();
  }
  constexpr int kGroups = kThreads / G;  // heads a block works on at once
  const int grp = threadIdx.x / G, lane = threadIdx.x % G;
  const unsigned mask = G == 32 ? 0xffffffffu : ((1u << G) - 1u) << (threadIdx.x % 32 / G * G);
  const int D = a.D;
  int h = (int)blockIdx.y * a.per_block;
  const int h_end = min(h + a.per_block, a.side[0].heads + a.side[1].heads);
  for (int w = 0; w < 2; ++w) {
    // this block's heads of this side
    const int base = w == 0 ? 0 : a.side[0].heads;
    const int lo = max(h, base), hi = min(h_end, base + a.side[w].heads);
    if (lo >= hi) continue;
    const T* x0 = static_cast<const T*>(a.side[w].x) + m * a.side[w].ld;
    T* y0 = static_cast<T*>(a.side[w].y) + m * a.side[w].ld_out;
    const T* wt = static_cast<const T*>(a.side[w].weight);
    after_wait(x0), after_wait(wt);
    float A[VPL][8], B[VPL][8];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int i0 = (lane + v * G) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = i0 + e;
        A[v][e] = B[v][e] = 0.f;
        if (i >= D) continue;
        const float wi = wt ? to_f32(wt[i]) + a.offset : 1.f;
        if (i < a.rotary) {
          const bool second = INTERLEAVED ? (i & 1) : i >= half;
          const int pair = INTERLEAVED ? i / 2 : second ? i - half : i;
          const int j = INTERLEAVED ? i ^ 1 : second ? i - half : i + half;
          const float wj = wt ? to_f32(wt[j]) + a.offset : 1.f;
          A[v][e] = wi * cs[pair];
          B[v][e] = second ? wj * sn[pair] : -wj * sn[pair];
        } else {
          A[v][e] = wi;
        }
      }
    }
    for (int hh = lo + grp; hh < hi; hh += kGroups) {
      const T* x = x0 + (int64_t)(hh - base) * D;
      float f[VPL][8], p[VPL][8];
      float ss = 0.f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const int i0 = (lane + v * G) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[v][e] = p[v][e] = 0.f;
        if (i0 < D) {
          load8(x + i0, f[v]);
          if constexpr (INTERLEAVED) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (i0 + e < a.rotary) p[v][e] = f[v][e ^ 1];
          } else if (a.aligned) {
            if (i0 < a.rotary) load8(x + (i0 < half ? i0 + half : i0 - half), p[v]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int i = i0 + e;
              if (i < a.rotary) p[v][e] = to_f32(x[i < half ? i + half : i - half]);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(f[v][e], f[v][e], ss);
      }
      // every lane of the group has read the head before any lane writes it
      // (the outputs may be the inputs): the shuffles order them
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      __syncwarp(mask);
      const float r = rsqrtf(ss / (float)D + a.eps);
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const int i0 = (lane + v * G) * 8;
        if (i0 >= D) continue;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = r * fmaf(f[v][e], A[v][e], p[v][e] * B[v][e]);
        store8(y0 + (int64_t)(hh - base) * D + i0, y);
      }
    }
  }
}

template <typename T, int G, int VPL>
cudaError_t launch_heads(const LaunchCtx& c, const HeadArgs& a, int64_t M, bool interleaved) {
  const int heads = a.side[0].heads + a.side[1].heads;
  HeadArgs b = a;
  // few tokens: one pass of heads a block, so that the heads spread over the GPU
  b.per_block = M < 2 * (int64_t)c.num_sms ? std::min(heads, kThreads / G) : heads;
  const dim3 grid((unsigned)M, (unsigned)ceil_div(heads, b.per_block));
  return interleaved
             ? launch_pdl(heads_kernel<T, G, VPL, true>, grid, dim3(kThreads), 0, c.stream, 1, b)
             : launch_pdl(heads_kernel<T, G, VPL, false>, grid, dim3(kThreads), 0, c.stream, 1, b);
}

template <typename T>
cudaError_t launch_dim(const LaunchCtx& c, const HeadArgs& a, int64_t M, bool interleaved) {
  if (a.D <= 64) return launch_heads<T, 8, 1>(c, a, M, interleaved);
  if (a.D <= 128) return launch_heads<T, 16, 1>(c, a, M, interleaved);
  if (a.D <= 256) return launch_heads<T, 32, 1>(c, a, M, interleaved);
  if (a.D <= 512) return launch_heads<T, 32, 2>(c, a, M, interleaved);
  return launch_heads<T, 32, 4>(c, a, M, interleaved);
}

}  // namespace

int heads_max_dim() { return kMaxDim; }

cudaError_t launch_qk_norm_rope(const LaunchCtx& c, theta_dtype dt, const HeadSide& q, const HeadSide& k, int64_t M,
                                int head_dim, float offset, float eps, const int64_t* positions,
                                const float* inv_freq, int rotary, bool interleaved) {
  HeadArgs a = {};
  a.side[0] = q;
  a.side[1] = k;
  a.pos = positions;
  a.inv_freq = inv_freq;
  a.D = head_dim;
  a.rotary = rotary;
  a.aligned = rotary % 16 == 0;
  a.offset = offset;
  a.eps = eps;
  return dt == THETA_BF16 ? launch_dim<bf16>(c, a, M, interleaved) : launch_dim<float>(c, a, M, interleaved);
}

}  // namespace theta
