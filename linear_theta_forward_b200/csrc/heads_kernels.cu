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
//
// Measured: 8192 tokens of 32 + 8 heads of 256 in bf16 67 us, 5.0 TB/s (0.76
// of the copy rate); loads in flight and issue slots bound it, not the angles
// (1 us of it). One token 3.4 us.
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace theta {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDim = 1024;

// How a value finds its pair's other value: halves of whole 8-value vectors,
// neighbours, or halves that cut a vector.
enum Pairing { HALVES = 0, NEIGHBOURS = 1, ODD_HALVES = 2 };

struct HeadArgs {
  HeadSide side[2];  // queries, keys
  const int64_t* pos;
  const float* inv_freq;
  int64_t M;
  int D, rotary;
  float offset, eps;
  int warps;      // warps per token: a block works on kWarps / warps tokens at a time
  int per_block;  // heads (queries then keys) of a token that one block takes
};

// 8 values as loaded: 16 bytes of bf16, 32 of fp32.
template <typename T>
struct Raw8 {
  static constexpr int kWords = 2 * sizeof(T);
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    if constexpr (sizeof(T) == 4) {
      const uint4 b = reinterpret_cast<const uint4*>(p)[1];
      w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (sizeof(T) == 2) {
      unpack(make_uint4(w[0], w[1], w[2], w[3]), f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
  }
};

// Pairs of fp32 in one register pair: two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ void split2(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
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

template <typename T>
__device__ __forceinline__ void weights8(const T* w, int i, float offset, float (&f)[8]) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 1.f;
    return;
  }
  Raw8<T> r;
  r.load(w + i);
  r.get(f);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] += offset;
}

// Sine and cosine of the token's angle of pair i. The angle in turns, whole
// and quarter turns taken off exactly in fp64; what is left is at most an
// eighth of a turn, so its fp32 rounding is below 2^-25 of a radian.
__device__ __forceinline__ void angle(double turns, float freq, float* c, float* s) {
  const double t4 = 4.0 * (turns * (double)freq);
  const double k = rint(t4);
  float s0, c0;
  sincospif(0.5f * (float)(t4 - k), &s0, &c0);
  const int quarter = (int)((long long)k & 3);
  const float c1 = quarter & 1 ? -s0 : c0, s1 = quarter & 1 ? c0 : s0;
  *c = quarter & 2 ? -c1 : c1;
  *s = quarter & 2 ? -s1 : s1;
}

// Whether a lane loads its next round of heads while it works on one. The
// round's registers pay where as many blocks fit an SM with them (65536 /
// (256 threads x registers)). us without and with, 32 + 8 heads of 256 and
// 512, 16 + 4 of 1024, 4096 tokens in bf16 and 2048 in fp32 unless noted:
//   three blocks still, D = 256 bf16   70.2, 67.2 (8192 tokens)
//   two still, D = 512 bf16            halves 84.1, 75.4
//   one either way, D = 1024           halves 114, 112 and 82.8, 82.2 (fp32), neighbours 81.8, 73.7 (fp32)
//   one instead of two, D = 512 fp32   halves 66.5, 78.8, neighbours 63.2, 68.9
//   one instead of two, D = 1024 bf16  neighbours 84.8, 94.7
// Halves that cut a vector load the partner value by value and are bound by
// that, at 124 registers and more: D = 256 81.3, 85.5 (4096 tokens of fp32)
// and 109, 107 (8192 of bf16), D = 512 138, 150 and 107, 111, D = 1024 in fp32
// 121, 126; only in bf16 at D = 1024, one head a lane at a time, 254, 178.
template <typename T, int VPL, int PAIRING>
constexpr bool fetches_ahead() {
  if (PAIRING == ODD_HALVES) return VPL == 4 && sizeof(T) == 2;
  if (VPL == 2) return sizeof(T) == 2;
  if (VPL == 4) return sizeof(T) == 4 || PAIRING == HALVES;
  return true;
}

// G lanes a head, VPL vectors of 8 values a lane.
template <typename T, int G, int VPL, int PAIRING>
__global__ void __launch_bounds__(kThreads) heads_kernel(const __grid_constant__ HeadArgs a) {
  extern __shared__ float table[];  // two buffers of [tokens][cos, sin][rotary / 2]
  constexpr bool kFetchAhead = fetches_ahead<T, VPL, PAIRING>();
  // a partner's vector that another lane holds is loaded with the head's own,
  // unless those were loaded a round ago: it is in L1 then
  constexpr bool kPartners = PAIRING == HALVES && VPL > 1 && !kFetchAhead;
  // heads a lane loads at once (D = 256, 8192 tokens of bf16, a round ahead:
  // 67.2 us; 69.8 and 74.0 with 2 and 4)
  constexpr int kAhead = VPL == 1 ? (kFetchAhead ? 3 : 4) : VPL == 2 ? 2 : 1;
  const int64_t* pos = a.pos;
  const float* freq = a.inv_freq;
  pdl_enter(pos, freq);
  const int D = a.D, rotary = a.rotary, half = rotary / 2;
  const float inv_d = 1.f / (float)D;
  const int tokens = kWarps / a.warps;                     // of a block at a time
  const int mine = threadIdx.x / 32 / a.warps;             // this warp's among them
  const int groups = a.warps * (32 / G);                   // heads of a token worked on at once
  const int grp = threadIdx.x % (32 * a.warps) / G, lane = threadIdx.x % G;
  const unsigned mask = G == 32 ? 0xffffffffu : ((1u << G) - 1u) << (threadIdx.x % 32 / G * G);
  const int h_lo = (int)blockIdx.y * a.per_block, h_hi = min(h_lo + a.per_block, a.side[0].heads + a.side[1].heads);
  int buf = 0;
  for (int64_t m0 = (int64_t)blockIdx.x * tokens; m0 < a.M; m0 += (int64_t)gridDim.x * tokens, buf ^= 1) {
    float* tab = table + buf * tokens * rotary;
    if (half > 0) {
      for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int t = i / half, p = i - t * half;
        const int64_t m = min(m0 + t, a.M - 1);
        angle((double)pos[m] * 0.15915494309189535, freq[p], &tab[t * rotary + p], &tab[t * rotary + half + p]);
      }
      // one barrier a round: the buffer written next round was last read the
      // round before this barrier
      __syncthreads();
    }
    const int64_t m = m0 + mine;
    if (m >= a.M) continue;
    const float* cs = tab + mine * rotary;
    const float* sn = cs + half;
    for (int w = 0; w < 2; ++w) {
      // this block's heads of this side
      const int base = w == 0 ? 0 : a.side[0].heads;
      const int lo = max(h_lo, base), hi = min(h_hi, base + a.side[w].heads);
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
        for (int e = 0; e < 8; ++e) A[v][e] = B[v][e] = 0.f;
        if (i0 >= D) continue;
        weights8(wt, i0, a.offset, A[v]);
        if constexpr (PAIRING == HALVES) {
          if (i0 < rotary) {
            const bool second = i0 >= half;
            const int p0 = second ? i0 - half : i0;
            weights8(wt, second ? p0 : i0 + half, a.offset, B[v]);
#pragma unroll
            for (int e = 0; e < 8; e += 4) {  // 16-byte aligned: rotary is a multiple of 16
              const float4 c4 = *reinterpret_cast<const float4*>(cs + p0 + e);
              const float4 s4 = *reinterpret_cast<const float4*>(sn + p0 + e);
              const float sg = second ? 1.f : -1.f;
              A[v][e] *= c4.x, A[v][e + 1] *= c4.y, A[v][e + 2] *= c4.z, A[v][e + 3] *= c4.w;
              B[v][e] *= sg * s4.x, B[v][e + 1] *= sg * s4.y, B[v][e + 2] *= sg * s4.z, B[v][e + 3] *= sg * s4.w;
            }
          }
        } else if constexpr (PAIRING == NEIGHBOURS) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            if (i0 + e < rotary) {
              const float c = cs[i0 / 2 + e / 2], s = sn[i0 / 2 + e / 2], w0 = A[v][e], w1 = A[v][e + 1];
              A[v][e] = w0 * c, B[v][e] = -w1 * s;
              A[v][e + 1] = w1 * c, B[v][e + 1] = w0 * s;
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int i = i0 + e;
            if (i < rotary) {
              const bool second = i >= half;
              const int p = second ? i - half : i, j = second ? p : i + half;
              const float wj = wt ? to_f32(wt[j]) + a.offset : 1.f;
              A[v][e] *= cs[p];
              B[v][e] = second ? wj * sn[p] : -wj * sn[p];
            }
          }
        }
      }
      uint64_t A2[VPL][4], B2[VPL][4];
#pragma unroll
      for (int v = 0; v < VPL; ++v)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          A2[v][q] = pair2(A[v][2 * q], A[v][2 * q + 1]);
          B2[v][q] = pair2(B[v][2 * q], B[v][2 * q + 1]);
        }
      Raw8<T> raw[kAhead][VPL], ahead[kFetchAhead ? kAhead : 1][VPL], other[kPartners ? kAhead : 1][VPL];
      auto fetch = [&](auto& into, int h0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const T* x = x0 + (int64_t)(h0 + u * groups - base) * D;
#pragma unroll
          for (int v = 0; v < VPL; ++v) {
            const int i0 = (lane + v * G) * 8;
            into[u][v].zero();
            if (i0 < D && h0 + u * groups < hi) into[u][v].load(x + i0);
            if constexpr (kPartners) {
              other[u][v].zero();
              if (i0 < rotary && h0 + u * groups < hi) other[u][v].load(x + (i0 < half ? i0 + half : i0 - half));
            }
          }
        }
      };
      if constexpr (kFetchAhead) fetch(ahead, lo + grp);
      for (int h0 = lo + grp; h0 < hi; h0 += kAhead * groups) {
        if constexpr (kFetchAhead) {
#pragma unroll
          for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int v = 0; v < VPL; ++v) raw[u][v] = ahead[u][v];
          fetch(ahead, h0 + kAhead * groups);
        } else {
          fetch(raw, h0);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (h0 + u * groups >= hi) break;
          const int64_t at = (int64_t)(h0 + u * groups - base) * D;
          float f[VPL][8], p[VPL][8];
          uint64_t sum = 0;
#pragma unroll
          for (int v = 0; v < VPL; ++v) {
            const int i0 = (lane + v * G) * 8;
            raw[u][v].get(f[v]);
            if constexpr (PAIRING == HALVES && VPL == 1) {
              // the other half's vector is another lane's
              const int from = i0 >= rotary ? lane : i0 < half ? lane + half / 8 : lane - half / 8;
              Raw8<T> o;
#pragma unroll
              for (int q = 0; q < Raw8<T>::kWords; ++q) o.w[q] = __shfl_sync(mask, raw[u][v].w[q], from, G);
              if (i0 >= rotary) o.zero();
              o.get(p[v]);
            } else if constexpr (kPartners) {
              other[u][v].get(p[v]);
            } else if constexpr (PAIRING == HALVES) {
              // in L1: the same head's vectors, loaded by this group of lanes
              Raw8<T> o;
              o.zero();
              if (i0 < rotary) o.load(x0 + at + (i0 < half ? i0 + half : i0 - half));
              o.get(p[v]);
            } else if constexpr (PAIRING == NEIGHBOURS) {
#pragma unroll
              for (int e = 0; e < 8; ++e) p[v][e] = i0 + e < rotary ? f[v][e ^ 1] : 0.f;
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int i = i0 + e;
                p[v][e] = i < rotary ? to_f32(x0[at + (i < half ? i + half : i - half)]) : 0.f;
              }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint64_t x2 = pair2(f[v][2 * q], f[v][2 * q + 1]);
              sum = fma2(x2, x2, sum);
            }
          }
          float ss, odd;
          split2(sum, ss, odd);
          ss += odd;
#pragma unroll
          for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
          // every lane of the group has read the head before any lane writes
          // it (the outputs may be the inputs)
          __syncwarp(mask);
          const float r = rsqrtf(ss * inv_d + a.eps);
          const uint64_t r2 = pair2(r, r);
#pragma unroll
          for (int v = 0; v < VPL; ++v) {
            const int i0 = (lane + v * G) * 8;
            if (i0 >= D) continue;
            float y[8];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              split2(mul2(r2, fma2(pair2(f[v][2 * q], f[v][2 * q + 1]), A2[v][q],
                                   mul2(pair2(p[v][2 * q], p[v][2 * q + 1]), B2[v][q]))),
                     y[2 * q], y[2 * q + 1]);
            store8(y0 + at + i0, y);
          }
        }
      }
    }
  }
}

template <typename T, int G, int VPL, int PAIRING>
cudaError_t launch_heads(const LaunchCtx& c, HeadArgs a) {
  auto kern = heads_kernel<T, G, VPL, PAIRING>;
  static int resident[kMaxContexts] = {};
  int per_sm;
  {
    std::lock_guard<std::mutex> lk(setup_mutex());
    int& slot = resident[c.slot];
    if (!slot && (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&slot, kern, kThreads, 4 * kMaxDim) != cudaSuccess ||
                  slot < 1))
      slot = 1;
    per_sm = slot;
  }
  const int heads = a.side[0].heads + a.side[1].heads;
  // Few tokens: a block a token and pass of heads, so that the heads spread
  // over the GPU. Many: two warps a token, which share its angles and factors
  // over more heads, in one wave of blocks. us, few and many, at 148, 222, 295
  // and 296 tokens (148 SMs): 32 + 8 heads of 256 in bf16 6.0, 7.9; 8.1, 7.9;
  // 10.3, 7.9; 10.3, 7.9; 4 + 1 heads of 256 3.4, 3.9; 3.8, 3.9; 4.3, 3.9; 4.3,
  // 3.9; 32 + 8 heads of 512 in fp32 11.2, 16.1; 16.2, 19.4; 20.8, 20.4; 20.9,
  // 20.5.
  const bool few = a.M < 2 * (int64_t)c.num_sms;
  a.warps = few ? kWarps : 2;
  a.per_block = few ? std::min(heads, kThreads / G) : heads;
  const int tokens = kWarps / a.warps;
  const int64_t blocks = ceil_div(a.M, tokens);
  const dim3 grid((unsigned)(few ? blocks : std::min<int64_t>(blocks, (int64_t)c.num_sms * per_sm)),
                  (unsigned)ceil_div(heads, a.per_block));
  return launch_pdl(kern, grid, dim3(kThreads), (size_t)2 * tokens * a.rotary * sizeof(float), c.stream, 1, a);
}

template <typename T, int G, int VPL>
cudaError_t launch_pairing(const LaunchCtx& c, const HeadArgs& a, bool interleaved) {
  if (interleaved) return launch_heads<T, G, VPL, NEIGHBOURS>(c, a);
  return a.rotary % 16 == 0 ? launch_heads<T, G, VPL, HALVES>(c, a) : launch_heads<T, G, VPL, ODD_HALVES>(c, a);
}

template <typename T>
cudaError_t launch_dim(const LaunchCtx& c, const HeadArgs& a, bool interleaved) {
  if (a.D <= 64) return launch_pairing<T, 8, 1>(c, a, interleaved);
  if (a.D <= 128) return launch_pairing<T, 16, 1>(c, a, interleaved);
  if (a.D <= 256) return launch_pairing<T, 32, 1>(c, a, interleaved);
  if (a.D <= 512) return launch_pairing<T, 32, 2>(c, a, interleaved);
  return launch_pairing<T, 32, 4>(c, a, interleaved);
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
  a.M = M;
  a.D = head_dim;
  a.rotary = rotary;
  a.offset = offset;
  a.eps = eps;
  return dt == THETA_BF16 ? launch_dim<bf16>(c, a, interleaved) : launch_dim<float>(c, a, interleaved);
}

}  // namespace theta
