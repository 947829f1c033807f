// The block-scaled FP8 theta forward on tensor cores (sm_100a):
//   Y[m, o] = s[o] * D1[o, m] + D2[o, m]
//   D1 = sum over blocks b of 128 columns of 2^(ew + ex) Wq[o, b] . Xq[m, b]
//   D2 = U . (T_hi + T_lo)^T,  T = X . V
// D1 runs on kind::mxf8f6f4: E4M3 operands, and for each row of A and of B a
// power-of-two scale per 32 values of K that the tensor core applies itself.
// Here all four 32-wide steps of a 128-wide K block use one scale, so a word
// of four scale bytes in tensor memory serves four K blocks (512 columns): a
// "scale group", selected byte by byte in the instruction descriptor. D2 is
// the bf16 rank term of the bf16 forward, in its own accumulator.
//
// As in the bf16 forward, W0 rows are the MMA's M side (128 rows are exactly
// one block of scales, so a tile's A scales are one byte per K block), tokens
// its N side, and s is a per-thread factor in the epilogue.
//
// Roles of a CTA's warps:
//   warp 0       TMA producer (one lane): 128 x 128 bytes of W0 codes and the
//                tile's token codes per stage, 128-byte swizzle
//   warp 1       tensor-memory allocation; MMA issuer (one lane)
//   scales       bytes from global memory packed into words. One-SM tiles: warps
//                2-5 write them to tensor memory (tcgen05.st), each its 32-lane
//                quarter, a ring of groups ahead of the MMAs. CTA pairs: warps 2
//                and 3 write them to shared memory, and the MMA issuer copies a
//                group to tensor memory (tcgen05.cp) in order with its MMAs
//   epilogue     the same warps 2-5 after the last group (one-SM tiles); warps
//                4-11 of their own in the persistent CTA-pair kernel
// Waits are bounded as everywhere in the library.
//
// Measured (device time, rank 64 on [21504, 5376]): 1 token 24.4 us (4.9 TB/s,
// HBM and the T = X.V launch in front), 64 tokens 28.5, 2048 tokens 245 us (1.96
// PFLOP/s at the power cap, where the SM clock is 1.35 GHz; 214 us alone).
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "umma_host.cuh"
#include "umma_ptx.cuh"

namespace theta {

namespace {

constexpr int kBM = 128;
constexpr int kBK = 128;               // bytes of K per stage: 128 codes, or 64 bf16 of the rank term
constexpr int kRankBK = 64;
constexpr int kABytes = kBM * 128;
constexpr int kGroup = 4;              // K blocks per scale word
constexpr int kPitch = 132;            // fp32 pitch of the split-K partial tiles (16-byte rows)

struct Args {
  int rows;   // O
  int cols;   // M tokens
  int kb1;    // K blocks of 128 codes
  int kb2;    // rank blocks of 64 (0: none)
  int splits;
  const uint8_t* xs;  // [kb1, cols]
  const uint8_t* ws;  // [ceil(rows / 128), kb1]
  const float* s;
  bf16* out;
  int early_start;  // launched right after this call's T = X.V kernel
  const float* t_parts;  // few tokens: [nparts, cols, r] partial sums of T = X.V
  const bf16* U;
  int nparts, r;
  int tile_tokens;  // CTA pairs: tokens of a tile, a multiple of 16, at most kPairN
  unsigned* err;
};

// The scale words of N rows for K blocks [kb, kb + 4): bytes at p[row + block *
// pitch]. Blocks and rows past the end repeat the last one -- their scales
// meet no MMA, or only columns that are never stored -- so that every load is
// unconditional and all of them are in flight together.
template <int N>
__device__ __forceinline__ void scale_words(const uint8_t* p, int64_t pitch, int row, int last_row, int kb, int last_kb,
                                            uint32_t (&w)[N]) {
  uint32_t byte[N][kGroup];
#pragma unroll
  for (int j = 0; j < kGroup; ++j) {
    const uint8_t* q = p + (int64_t)min(kb + j, last_kb) * pitch;
#pragma unroll
    for (int c = 0; c < N; ++c) byte[c][j] = q[min(row + 32 * c, last_row)];
  }
#pragma unroll
  for (int c = 0; c < N; ++c)
    w[c] = __byte_perm(byte[c][0] | (byte[c][1] << 8), byte[c][2] | (byte[c][3] << 8), 0x5410);
}

// ------------------------------------------------------------ one-SM tiles
constexpr int kThreads = 192;

// One or two tokens (FEW): T = X.V comes as fp32 partial sums from a CUDA-core
// kernel, and the rank term is a dot product of at most 256 values per row in
// the epilogue -- shorter than a tensor-core T and two more accumulations (one
// token of [6912, 1152], rank 32: 5.1 us without a rank term, 7.9 us with T
// on tensor cores).
constexpr int kFewTokens = 2;
constexpr int kMaxRank = 256;

template <int BN>
struct Cfg {
  static constexpr int kBBytes = BN * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 4;
  static constexpr int kRing = 4;                          // scale groups in tensor memory
  static constexpr int kSfbCols = BN <= 32 ? 1 : BN / 32;  // columns of token scales
  static constexpr int kSf = 2 * BN;                       // first scale column (after D1, D2); 8 per group
  static constexpr int kTmemNeed = kSf + 8 * kRing;
  static constexpr int kTmemCols = kTmemNeed <= 64 ? 64 : kTmemNeed <= 128 ? 128 : kTmemNeed <= 256 ? 256 : 512;
  static_assert(kTmemNeed <= 512 && kSfbCols <= 4 && BN <= 64, "accumulators and scales must fit in tensor memory");
  static_assert(BN * kPitch * 4 <= kStages * kStageBytes, "partial tile must fit in the stage ring");
  static constexpr int kSmemBytes = kStages * kStageBytes + 1024 /*align*/ + 256 /*barriers*/;
};

template <int BN, bool FEW>
__global__ void __launch_bounds__(kThreads)
fp8_tile_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmTh,
                const __grid_constant__ CUtensorMap tmTl, const __grid_constant__ Args args) {
  using C = Cfg<BN>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * C::kStageBytes);
  uint64_t* empty = full + S;
  uint64_t* sf_full = empty + S;
  uint64_t* sf_empty = sf_full + C::kRing;
  uint64_t* accum = sf_empty + C::kRing;
  uint64_t* drain = accum + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int split = args.splits > 1 ? (int)ptx::cluster_ctarank() : 0;
  const int n_tile = blockIdx.x / args.splits;
  const int m_tile = blockIdx.y;
  const int kb_begin = (int)((int64_t)split * args.kb1 / args.splits);
  const int kb_end = (int)((int64_t)(split + 1) * args.kb1 / args.splits);
  const bool has_d2 = args.kb2 > 0 && split == 0;
  const int n1 = kb_end - kb_begin;
  const int total = n1 + (has_d2 ? 2 * args.kb2 : 0);

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::kRing; ++i) {
      ptx::mbar_init(&sf_full[i], 4);  // one arrival per scale warp
      ptx::mbar_init(&sf_empty[i], 1);
    }
    ptx::mbar_init(accum, 1);
    ptx::mbar_init(drain, 1);
    *abort_flag = prior_timeout(args.err);
    ptx::fence_mbarrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, C::kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // programmatic dependent launch as in the bf16 forward: right after its own
  // T = X.V kernel (which has seen all earlier work complete) the codes,
  // scales and s are streamed at once, and only the loads of T wait
  const bool early = args.early_start;
  if (!early) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  auto give_up = [&]() {
    record_timeout(args.err);
    *abort_flag = 1;
  };

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------- producer
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmX);
    int issued = 0;
    for (int i = 0; i < total; ++i) {
      const int st = i % S;
      if (!ptx::mbar_wait(&empty[st], ((uint32_t)(i / S) & 1u) ^ 1u, abort_flag)) {
        give_up();
        break;
      }
      uint8_t* a = smem + st * C::kStageBytes;
      uint8_t* b = a + kABytes;
      ptx::mbar_arrive_expect_tx(&full[st], C::kStageBytes);
      if (i < n1) {
        ptx::tma_load_2d(a, &tmW, &full[st], (kb_begin + i) * kBK, m_tile * kBM);
        ptx::tma_load_2d(b, &tmX, &full[st], (kb_begin + i) * kBK, n_tile * BN);
      } else {
        const int j = i - n1;
        if (early && j == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
        const int jx = (j % args.kb2) * kRankBK;
        ptx::tma_load_2d(a, &tmU, &full[st], jx, m_tile * kBM);
        ptx::tma_load_2d(b, j < args.kb2 ? &tmTh : &tmTl, &full[st], jx, n_tile * BN);
      }
      ++issued;
    }
    // drain: wait for the last armed phase of every stage (all loads landed)
    for (int st = 0; st < S && st < issued; ++st) {
      const int last = st + ((issued - 1 - st) / S) * S;
      if (!ptx::mbar_wait(&full[st], (uint32_t)(last / S) & 1u, abort_flag)) {
        int never = 0;
        ptx::mbar_wait(&full[st], (uint32_t)(last / S) & 1u, &never);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    // The whole warp walks the loop, so that addresses and descriptors stay in
    // uniform registers, and one lane issues.
    const bool issuer = ptx::elect_one();
    const uint64_t desc0 = ptx::sdesc_sw128(ptx::smem_u32(smem), 16, 1024);
    int done = 0, st = 0, ring = 0;
    uint32_t ph = 0, ring_ph = 0;
    for (int i = 0; i < total; ++i) {
      const int byte = i % kGroup;
      bool ok = ptx::mbar_wait(&full[st], ph, abort_flag);
      if (ok && i < n1 && byte == 0) ok = ptx::mbar_wait(&sf_full[ring], ring_ph, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        give_up();
        break;
      }
      ptx::tc_fence_after();
      const uint64_t ad = desc0 + (uint64_t)(st * (C::kStageBytes / 16));
      const uint64_t bd = ad + kABytes / 16;
      if (i < n1) {
        const uint32_t sf = tmem + (uint32_t)(C::kSf + 8 * ring);
        const uint32_t idesc = ptx::idesc_mxf8(kBM, BN, byte);
        if (issuer) {
#pragma unroll
          for (int kk = 0; kk < kBK / 32; ++kk)
            ptx::umma_mxf8<false>(tmem, ad + 2 * kk, bd + 2 * kk, idesc, sf, sf + 4, (i > 0 || kk > 0) ? 1u : 0u);
          if (byte == kGroup - 1) ptx::umma_commit(&sf_empty[ring]);
          ptx::umma_commit(&empty[st]);
        }
        if (byte == kGroup - 1 && ++ring == C::kRing) ring = 0, ring_ph ^= 1u;
      } else if (issuer) {
        constexpr uint32_t idesc = ptx::idesc_bf16(kBM, BN, 0);
#pragma unroll
        for (int kk = 0; kk < kRankBK / 16; ++kk)
          ptx::umma_bf16(tmem + BN, ad + 2 * kk, bd + 2 * kk, idesc, (i > n1 || kk > 0) ? 1u : 0u);
        ptx::umma_commit(&empty[st]);
      }
      __syncwarp();
      if (++st == S) st = 0, ph ^= 1u;
      ++done;
    }
    if (done == total) {
      if (issuer) ptx::umma_commit(accum);
    } else if (done > 0) {
      // aborted: the issued MMAs finish before tensor memory is freed
      if (issuer) ptx::umma_commit(drain);
      __syncwarp();
      int never = 0;
      ptx::mbar_wait(drain, 0, &never);
    }
  } else if (warp >= 2) {
    // ---------------------------------------------------------- scales
    const int quarter = warp & 3;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint8_t* wsp = args.ws + (int64_t)m_tile * args.kb1;
    const int groups = (n1 + kGroup - 1) / kGroup;
    for (int g = 0; g < groups; ++g) {
      const int ring = g % C::kRing, kb = kb_begin + g * kGroup;
      uint32_t wa[1], wb[C::kSfbCols];
      scale_words(wsp, 1, 0, 0, kb, kb_end - 1, wa);
      scale_words(args.xs, args.cols, n_tile * BN + lane, args.cols - 1, kb, kb_end - 1, wb);
      bool ok = g < C::kRing || ptx::mbar_wait(&sf_empty[ring], (uint32_t)(g / C::kRing - 1) & 1u, abort_flag);
      if (!ok) give_up();
      if (!__all_sync(0xffffffffu, ok)) break;
      ptx::tc_fence_after();
      const uint32_t sf = tmem + lanes + (uint32_t)(C::kSf + 8 * ring);
      ptx::tmem_st4(sf, wa[0], wa[0], wa[0], wa[0]);
#pragma unroll
      for (int c = 0; c < C::kSfbCols; ++c) ptx::tmem_st1(sf + 4 + c, wb[c]);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sf_full[ring]);
    }
    // ---------------------------------------------------------- epilogue
    const int row = quarter * 32 + lane;  // accumulator row = tensor-memory lane
    const uint32_t taddr = tmem + lanes;
    if (early) asm volatile("griddepcontrol.wait;" ::: "memory");
    float rank_term[kFewTokens] = {};
    if constexpr (FEW) {
      if (split == 0 && args.r > 0) {
        __shared__ float t_sum[kFewTokens * kMaxRank];  // [token][r]
        const int n = args.cols * args.r;
        for (int i = threadIdx.x - 64; i < n; i += 128) {
          float t = 0.f;
#pragma unroll 8
          for (int p = 0; p < args.nparts; ++p) t += args.t_parts[p * n + i];
          t_sum[i] = t;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (m_tile * kBM + row < args.rows) {
          const uint4* u = reinterpret_cast<const uint4*>(args.U + (int64_t)(m_tile * kBM + row) * args.r);
#pragma unroll 4
          for (int j = 0; j < args.r / 8; ++j) {
            float f[8];
            unpack(u[j], f);
#pragma unroll
            for (int m = 0; m < kFewTokens; ++m)
              if (m < args.cols)
#pragma unroll
                for (int e = 0; e < 8; ++e) rank_term[m] = fmaf(f[e], t_sum[m * args.r + 8 * j + e], rank_term[m]);
          }
        }
      }
    }
    bool ok = ptx::mbar_wait(accum, 0, abort_flag);
    if (!ok) give_up();
    ok = __all_sync(0xffffffffu, ok);  // tcgen05.ld below is warp-collective
    ptx::tc_fence_after();
    const int grow = m_tile * kBM + row;
    const int col0 = n_tile * BN;
    const int ncols = min(BN, args.cols - col0);
    const float so = grow < args.rows ? args.s[grow] : 0.f;
    float* part = reinterpret_cast<float*>(smem);
    if (ok) {
      for (int c0 = 0; c0 < ncols; c0 += 16) {
        float d1[16], d2[16];
        ptx::tmem_ld16(taddr + c0, d1);
        if (has_d2) ptx::tmem_ld16(taddr + BN + c0, d2);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float v = has_d2 ? fmaf(so, d1[e], d2[e]) : so * d1[e];
          if constexpr (FEW) {
            if (e >= kFewTokens) break;
            v = fmaf(so, d1[e], rank_term[e]);
          }
          const int m = col0 + c0 + e;
          if (args.splits > 1)
            part[(c0 + e) * kPitch + row] = v;
          else if (grow < args.rows && m < args.cols)
            args.out[(int64_t)m * args.rows + grow] = __float2bfloat16_rn(v);
        }
      }
    }
  }

  // ------------------------------------------------------------ split-K sum
  __syncwarp();
  if (args.splits > 1) {
    ptx::cluster_sync();  // every CTA of the cluster has staged its partial tile
    if (!*abort_flag) {
      const int col0 = n_tile * BN;
      // four rows at a time: O is a multiple of 8, so they are all inside or all outside
      const int E = min(BN, args.cols - col0) * (kBM / 4);
      const int e0 = (int)((int64_t)split * E / args.splits), e1 = (int)((int64_t)(split + 1) * E / args.splits);
      const uint32_t part_addr = ptx::smem_u32(smem);
#pragma unroll 2
      for (int e = e0 + threadIdx.x; e < e1; e += kThreads) {
        const int c = e / (kBM / 4), rr = e % (kBM / 4) * 4;
        const int grow = m_tile * kBM + rr;
        if (grow >= args.rows) continue;
        const float4 v = ptx::cluster_sum4(part_addr + (uint32_t)((c * kPitch + rr) * 4), args.splits);
        *reinterpret_cast<uint2*>(args.out + (int64_t)(col0 + c) * args.rows + grow) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      }
    }
    ptx::cluster_sync();  // no CTA leaves while a peer still reads its tile
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) ptx::tmem_dealloc(tmem, C::kTmemCols);
}

// ------------------------------------------------------------ CTA-pair tiles
// 256 rows x up to 240 tokens (tile_tokens, the tokens spread evenly over the
// fewest tiles) per pair of SMs (cta_group::2), persistent. Each
// CTA stages 128 rows of W0 codes and half of the tile's tokens per K block
// and holds its 128 rows of both accumulators. 240 tokens, not 256: D1 and D2
// take 2 x 240 columns of tensor memory and the scales of two groups the
// other 32. A's scales are each CTA's own rows', B's those of all the tile's
// tokens, in both CTAs.
constexpr int kPairN = 240;
constexpr int kPairHalf = kPairN / 2;
constexpr int kPairStages = 5;
constexpr int kPairBBytes = kPairHalf * 128;
constexpr int kPairStageBytes = kABytes + kPairBBytes;
constexpr int kPairOutBytes = kBM * kPairN * 2;
constexpr int kPairSf = 2 * kPairN;  // scale columns: 16 per group, two groups
constexpr int kPairRing = 4;         // scale groups in shared memory
constexpr int kPairSfBytes = 3 * 512;  // of a group: the CTA's 128 rows, then 256 tokens
constexpr int kPairSmemBytes =
    kPairStages * kPairStageBytes + kPairOutBytes + kPairRing * kPairSfBytes + 1024 /*align*/ + 256 /*barriers*/;
constexpr int kPairEpiWarps = 8;
constexpr int kPairEpi = 32 * kPairEpiWarps;
constexpr int kPairThreads = 128 + kPairEpi;
constexpr uint16_t kPairMask = 0x3;
static_assert(kPairSf + 2 * 16 <= 512, "accumulators and scales must fit in tensor memory");
// The copy of group g + 2 to tensor memory overwrites group g's scales, so group
// g's MMAs must be done by then. Between two groups of a tile: g + 1 is full, so
// the stage of g + 2's first block lies kGroup + 1 blocks behind g's last, and
// its load waited for the MMAs kPairStages blocks back. A group may be short only
// as a tile's last one; behind it the issuer waits for the tile's accumulators
// to have been read (tmem_free), which all of the tile's MMAs precede. A tile
// that did not wait there (two accumulators in turn) would need a wait of its own.
static_assert(kPairStages <= kGroup + 1, "a scale group's columns must be free when they are written again");
static_assert(kPairBBytes % 1024 == 0, "swizzled tiles start on 1024-byte boundaries");

__global__ void __launch_bounds__(kPairThreads, 1)
fp8_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmTh,
                const __grid_constant__ CUtensorMap tmTl, const __grid_constant__ CUtensorMap tmY,
                const __grid_constant__ Args args) {
  constexpr int S = kPairStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  bf16* sOut = reinterpret_cast<bf16*>(smem + S * kPairStageBytes);
  uint8_t* sScale = smem + S * kPairStageBytes + kPairOutBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sScale + kPairRing * kPairSfBytes);
  uint64_t* empty = full + S;
  uint64_t* sf_full = empty + S;
  uint64_t* sf_empty = sf_full + kPairRing;
  uint64_t* accum = sf_empty + kPairRing;
  uint64_t* tmem_free = accum + 1;
  uint64_t* drain = tmem_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t cta = ptx::cluster_ctarank();  // 0 issues the MMAs
  const int cluster = blockIdx.x / 2, n_clusters = gridDim.x / 2;
  const int width = args.tile_tokens;
  const int n_tiles = (args.cols + width - 1) / width;
  const int tiles = n_tiles * ((args.rows + 2 * kBM - 1) / (2 * kBM));
  const bool has_d2 = args.kb2 > 0;
  const int n1 = args.kb1;
  const int per_tile = n1 + (has_d2 ? 2 * args.kb2 : 0);
  const int groups = (n1 + kGroup - 1) / kGroup;
  // tokens of a tile's MMA: the last tile's rounded up to a multiple of 16
  auto tile_n = [&](int tile) { return min(width, (args.cols - (tile % n_tiles) * width + 15) / 16 * 16); };
  const uint32_t stage_bytes = kABytes + width / 2 * 128;  // that a CTA loads per stage

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kPairRing; ++i) {
      ptx::mbar_init(&sf_full[i], 2);  // one arrival per CTA
      ptx::mbar_init(&sf_empty[i], 1);
    }
    ptx::mbar_init(accum, 1);
    ptx::mbar_init(tmem_free, 2 * kPairEpiWarps);  // one arrival per epilogue warp of both CTAs
    ptx::mbar_init(drain, 1);
    *abort_flag = prior_timeout(args.err);
    ptx::fence_mbarrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(tmem_slot, 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();  // both CTAs' barriers exist before either signals the other's
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const bool early = args.early_start;
  if (!early) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  auto give_up = [&]() {
    record_timeout(args.err);
    *abort_flag = 1;
  };

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------- producer (both CTAs)
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmX);
    const uint32_t full0 = ptx::mapa(ptx::smem_u32(full), 0);  // the MMA CTA's full barriers
    bool waited = !early, stop = false;
    int g = 0;  // stage items issued, over all tiles
    for (int tile = cluster; tile < tiles && !stop; tile += n_clusters) {
      const int row0 = (tile / n_tiles) * (2 * kBM) + (int)cta * kBM;
      const int tok0 = (tile % n_tiles) * width + (int)cta * (tile_n(tile) / 2);
      for (int i = 0; i < per_tile; ++i, ++g) {
        const int st = g % S;
        if (!ptx::mbar_wait(&empty[st], ((uint32_t)(g / S) & 1u) ^ 1u, abort_flag)) {
          give_up();
          stop = true;
          break;
        }
        uint8_t* a = smem + st * kPairStageBytes;
        uint8_t* b = a + kABytes;
        const uint32_t bar = full0 + (uint32_t)(st * 8);
        if (cta == 0) ptx::mbar_arrive_expect_tx(&full[st], 2 * stage_bytes);  // both CTAs' loads
        if (i < n1) {
          ptx::tma_load_2d_pair(a, &tmW, bar, i * kBK, row0);
          ptx::tma_load_2d_pair(b, &tmX, bar, i * kBK, tok0);
        } else {
          const int j = i - n1;
          if (!waited) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            waited = true;
          }
          const int jx = (j % args.kb2) * kRankBK;
          ptx::tma_load_2d_pair(a, &tmU, bar, jx, row0);
          ptx::tma_load_2d_pair(b, j < args.kb2 ? &tmTh : &tmTl, bar, jx, tok0);
        }
      }
    }
    // drain: a stage's last MMAs complete after its last loads landed, and
    // their commit reaches empty[] in both CTAs. After an abort, loads in
    // flight land within microseconds: a bounded tenth of a second for them
    for (int st = 0; st < S && st < g; ++st) {
      const int last = st + ((g - 1 - st) / S) * S;
      if (!ptx::mbar_wait(&empty[st], (uint32_t)(last / S) & 1u, abort_flag)) {
        int never = 0;
        ptx::mbar_wait(&empty[st], (uint32_t)(last / S) & 1u, &never, 100000000ull);
      }
    }
  } else if (warp == 1 && cta == 0) {
    // ---------------------------------------------------------- MMA issuer (even CTA)
    // The whole warp walks the loop, so that addresses and descriptors stay in
    // uniform registers, and one lane issues (one lane walking it alone spent
    // 830 cycles a K block on the four MMAs' operands, their time being 480).
    const bool issuer = ptx::elect_one();
    const uint64_t desc0 = ptx::sdesc_sw128(ptx::smem_u32(smem), 16, 1024);
    bool stop = false, any = false;
    const uint64_t sf_desc0 = ptx::sdesc_rows16(ptx::smem_u32(sScale));
    int st = 0, ring = 0;
    uint32_t ph = 0, ring_ph = 0, free_ph = 1;
    for (int tile = cluster; tile < tiles && !stop; tile += n_clusters) {
      // the epilogues of both CTAs have read the previous tile's accumulators
      // (its last scale groups are done with too)
      bool ok = !any || ptx::mbar_wait(tmem_free, free_ph, abort_flag);
      free_ph ^= 1u;
      const int N = tile_n(tile);
      const uint32_t idesc1 = ptx::idesc_mxf8(2 * kBM, N, 0), idesc2 = ptx::idesc_bf16(2 * kBM, N, 0);
      for (int i = 0; i < per_tile; ++i) {
        const int byte = i % kGroup;
        ok = ok && ptx::mbar_wait(&full[st], ph, abort_flag);
        if (ok && i < n1 && byte == 0) ok = ptx::mbar_wait(&sf_full[ring], ring_ph, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {
          give_up();
          stop = true;
          break;
        }
        ptx::tc_fence_after();
        const uint64_t ad = desc0 + (uint64_t)(st * (kPairStageBytes / 16));
        const uint64_t bd = ad + kABytes / 16;
        if (i < n1) {
          const bool last = byte == kGroup - 1 || i == n1 - 1;  // of its scale group
          const uint32_t sf = tmem + (uint32_t)(kPairSf + 16 * (ring & 1));
          const uint32_t idesc = idesc1 | ((uint32_t)byte << 4) | ((uint32_t)byte << 29);
          if (issuer) {
            if (byte == 0) {
              const uint64_t sd = sf_desc0 + (uint64_t)(ring * (kPairSfBytes / 16));
#pragma unroll
              for (int q = 0; q < 3; ++q) ptx::tmem_cp_scales_pair(sf + 4 * q, sd + 32 * q);
            }
#pragma unroll
            for (int kk = 0; kk < kBK / 32; ++kk)
              ptx::umma_mxf8<true>(tmem, ad + 2 * kk, bd + 2 * kk, idesc, sf, sf + 4, (i > 0 || kk > 0) ? 1u : 0u);
            if (last) ptx::umma_commit_pair(&sf_empty[ring], kPairMask);
            ptx::umma_commit_pair(&empty[st], kPairMask);
          }
          if (last && ++ring == kPairRing) ring = 0, ring_ph ^= 1u;
        } else if (issuer) {
#pragma unroll
          for (int kk = 0; kk < kRankBK / 16; ++kk)
            ptx::umma_bf16_pair(tmem + (uint32_t)kPairN, ad + 2 * kk, bd + 2 * kk, idesc2,
                                (i > n1 || kk > 0) ? 1u : 0u);
          ptx::umma_commit_pair(&empty[st], kPairMask);
        }
        __syncwarp();
        any = true;
        if (++st == S) st = 0, ph ^= 1u;
      }
      if (!stop && issuer) ptx::umma_commit_pair(accum, kPairMask);
      __syncwarp();
    }
    if (stop && any) {
      // aborted: the issued MMAs finish before tensor memory is released
      if (issuer) ptx::umma_commit_pair(drain, 0x1);
      __syncwarp();
      int never = 0;
      ptx::mbar_wait(drain, 0, &never);
    }
  } else if (warp == 2 || warp == 3) {
    // ---------------------------------------------------------- scales (both CTAs)
    // Groups in turn between the two warps: lane l writes the words of rows l,
    // 32 + l, 64 + l and 96 + l, 16 bytes for the W0 rows (all alike) and twice
    // 16 for the tokens.
    const uint32_t full_bar = ptx::mapa(ptx::smem_u32(sf_full), 0);
    const int row_blocks = (args.rows + kBM - 1) / kBM;
    bool ok = true;
    int sg = 0;
    for (int tile = cluster; tile < tiles && ok; tile += n_clusters) {
      // the odd CTA's rows may all be past O: its scales are then not used
      const int rb = min((tile / n_tiles) * 2 + (int)cta, row_blocks - 1);
      const uint8_t* wsp = args.ws + (int64_t)rb * args.kb1;
      const int tok = (tile % n_tiles) * width + lane;
      for (int q = 0; q < groups; ++q, ++sg) {
        if ((sg & 1) != (warp & 1)) continue;
        const int ring = sg % kPairRing, kb = q * kGroup;
        uint32_t wa[1], wb[8];
        scale_words(wsp, 1, 0, 0, kb, n1 - 1, wa);
        scale_words(args.xs, args.cols, tok, args.cols - 1, kb, n1 - 1, wb);
        ok = sg < kPairRing || ptx::mbar_wait(&sf_empty[ring], (uint32_t)(sg / kPairRing - 1) & 1u, abort_flag);
        if (!ok) give_up();
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint4* dst = reinterpret_cast<uint4*>(sScale + ring * kPairSfBytes) + lane;
        dst[0] = make_uint4(wa[0], wa[0], wa[0], wa[0]);
        dst[32] = make_uint4(wb[0], wb[1], wb[2], wb[3]);
        dst[64] = make_uint4(wb[4], wb[5], wb[6], wb[7]);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(full_bar + (uint32_t)(ring * 8));
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------- epilogue (both CTAs)
    // The tile is rounded to bf16 in registers and tensor memory handed back
    // before anything is written to shared memory: the MMAs wait for the
    // tensor-memory reads alone.
    const int quarter = warp & 3;         // a warp reads lanes 32 * (warp % 4) ...
    const int part = (warp - 4) / 4;      // ... and columns 128 * part ...
    const int row = quarter * 32 + lane;  // accumulator row = tensor-memory lane
    const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(part * 128);
    const bool storer = threadIdx.x == 128;  // issues the TMA stores of the tile
    const uint32_t free_bar = ptx::mapa(ptx::smem_u32(tmem_free), 0);
    if (early) asm volatile("griddepcontrol.wait;" ::: "memory");
    bool ok = true;
    int j = 0;
    for (int tile = cluster; tile < tiles; tile += n_clusters, ++j) {
      const int row0 = (tile / n_tiles) * (2 * kBM) + (int)cta * kBM;
      const int col0 = (tile % n_tiles) * width;
      const int ncols = min(width, args.cols - col0) - part * 128;  // of this warp's columns
      const int grow = row0 + row;
      const float so = grow < args.rows ? args.s[grow] : 0.f;
      const bool got = __all_sync(0xffffffffu, ptx::mbar_wait(accum, (uint32_t)j & 1u, abort_flag));
      uint32_t y[64];
      if (got) {
        ptx::tc_fence_after();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float d1[32], d2[32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // columns past the tile's tokens are not read
            if (32 * q + 16 * h < ncols) {
              ptx::tmem_ld16(taddr + 32 * q + 16 * h, *reinterpret_cast<float(*)[16]>(d1 + 16 * h));
              if (has_d2)
                ptx::tmem_ld16(taddr + kPairN + 32 * q + 16 * h, *reinterpret_cast<float(*)[16]>(d2 + 16 * h));
            }
          }
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            y[16 * q + e] = has_d2 ? pack_bf16x2(fmaf(so, d1[2 * e], d2[2 * e]), fmaf(so, d1[2 * e + 1], d2[2 * e + 1]))
                                   : pack_bf16x2(so * d1[2 * e], so * d1[2 * e + 1]);
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(free_bar);
      }
      if (storer) ptx::bulk_wait_read();  // the previous tile's store has read sOut
      // one decision for all epilogue warps: the barriers need every one of them
      ok = ptx::bar_red_and(1, kPairEpi, got);
      if (!ok) break;
      uint16_t* dst = reinterpret_cast<uint16_t*>(sOut) + part * 128 * kBM + row;
#pragma unroll
      for (int e = 0; e < 64; ++e) {
        if (2 * e < ncols) {
          dst[2 * e * kBM] = (uint16_t)y[e];
          dst[(2 * e + 1) * kBM] = (uint16_t)(y[e] >> 16);
        }
      }
      ptx::fence_proxy_async_smem();
      asm volatile("bar.sync 1, %0;" ::"n"(kPairEpi) : "memory");
      if (storer && row0 < args.rows) {
        // rows past O and tokens past M fall outside Y and are not written
        ptx::tma_store_2d(&tmY, sOut, row0, col0);
        ptx::bulk_commit();
      }
    }
    if (!ok && !*abort_flag) give_up();
    if (storer) ptx::bulk_wait_all();
  }

  __syncwarp();
  ptx::tc_fence_before();
  ptx::cluster_sync();  // both epilogues have read their accumulators; every MMA has completed
  if (warp == 1) ptx::tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------------ host side
struct Maps {
  CUtensorMap w, x, u, th, tl;
};

// K splits of the one-SM tiles: while every SM still gets at most one CTA and
// each split keeps 8 K blocks; below that the sum over the cluster costs more
// than the shorter walk saves. us with 1, 2, 4 and 8 splits (* this rule's):
//     1 token of  [6912, 1152]     6.9*  7.9   8.1  14.5     9 blocks
//   128 tokens of [1152, 6912]    23.1  15.9  11.7* 14.5    54 blocks
//     1 token of  [21504, 5376]   24.2* 30.3  33.8  54.8   168 tiles
//    16 tokens of [8192, 5376]    19.1  14.8* 14.4  21.0    64 tiles
//    16 tokens of [5376, 8192]    25.2  17.3* 15.2  14.8    42 tiles
//    16 tokens of [5376, 21504]   56.5  34.0* 25.9  25.4    42 tiles, 168 blocks
// The last two are where it stops early: a power of two leaves 84 CTAs, and
// behind a long walk a second CTA of an SM would pay.
int tile_splits(const LaunchCtx& c, int64_t m_tiles, int64_t n_tiles, int kb) {
  int s = 1;
  if (c.policy != THETA_POLICY_THROUGHPUT)
    while (s < 8 && m_tiles * n_tiles * 2 * s <= c.num_sms && kb / (2 * s) >= 8) s *= 2;
  return s;
}

template <int BN, bool FEW = false>
cudaError_t launch_tile(const LaunchCtx& c, const Maps& mp, Args args) {
  using C = Cfg<BN>;
  auto kern = fp8_tile_kernel<BN, FEW>;
  static KernelInfo info[kMaxContexts];
  cudaError_t e = prepare_kernel(&info[c.slot], c.device, kern, kThreads, C::kSmemBytes, C::kTmemCols, true);
  if (e != cudaSuccess) return e;
  const int m_tiles = (int)ceil_div(args.rows, kBM), n_tiles = (int)ceil_div(args.cols, BN);
  args.splits = tile_splits(c, m_tiles, n_tiles, args.kb1);
  return launch_pdl(kern, dim3((unsigned)(n_tiles * args.splits), (unsigned)m_tiles), dim3(kThreads), C::kSmemBytes,
                    c.stream, args.splits, mp.w, mp.x, mp.u, mp.th, mp.tl, args);
}

cudaError_t launch_pair(const LaunchCtx& c, const Maps& mp, const Args& args, const CUtensorMap& mY) {
  static KernelInfo info[kMaxContexts];
  cudaError_t e =
      prepare_kernel(&info[c.slot], c.device, fp8_pair_kernel, kPairThreads, kPairSmemBytes, 512, false);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ceil_div(args.rows, 2 * kBM) * ceil_div(args.cols, args.tile_tokens);
  const int64_t clusters = tiles < c.num_sms / 2 ? tiles : c.num_sms / 2;  // one CTA per SM
  return launch_pdl(fp8_pair_kernel, dim3((unsigned)(2 * clusters)), dim3(kPairThreads), kPairSmemBytes, c.stream, 2,
                    mp.w, mp.x, mp.u, mp.th, mp.tl, mY, args);
}

}  // namespace

// Slices of I in the partial sums of T = X.V: about 84 rows of V each, up to 64.
constexpr int kXvParts = 64;
constexpr int kXvRows = 84;

// Bytes of one part of T, the offset of the low one.
static size_t t_part_bytes(int64_t M, int r) { return ((size_t)M * r * 2 + 255) / 256 * 256; }

// T's high and low parts, or its partial sums, whichever the call takes. The
// partial sums of one or two tokens are larger than the parts of a few more,
// so every size covers them: a buffer sized for a batch serves smaller ones.
size_t forward_fp8_workspace_bytes(int64_t M, int r) {
  const size_t sums = (size_t)kXvParts * std::min<int64_t>(M, kFewTokens) * r * sizeof(float);
  return std::max(2 * t_part_bytes(M, r), sums);
}

int launch_forward_fp8(const LaunchCtx& c, const void* X, const void* xq, const void* xs, const void* wq,
                       const void* ws, const float* s, const void* U, const void* V, int64_t M, int64_t O, int64_t I,
                       int r, void* Y, void* work, cudaError_t* ce) {
  *ce = cudaSuccess;
  int st;
  bf16* t_hi = static_cast<bf16*>(work);
  bf16* t_lo = nullptr;
  const bool few = M <= kFewTokens;
  const int nparts = (int)std::min<int64_t>(kXvParts, ceil_div(I, kXvRows));
  if (few && r > 0) {
    *ce = launch_xv_parts(c, X, V, M, I, r, nparts, static_cast<float*>(work));
    if (*ce != cudaSuccess) return THETA_ERR_CUDA;
  } else if (r > 0) {
    t_lo = reinterpret_cast<bf16*>(static_cast<uint8_t*>(work) + t_part_bytes(M, r));
    if ((st = launch_xv_umma(c, X, V, M, I, r, t_hi, t_lo, ce))) return st;
  }
  const int width = (int)(ceil_div(ceil_div(M, ceil_div(M, kPairN)), 16) * 16);  // tokens of a pair's tile
  // 64 tokens a tile at most on one SM: wider tiles leave SMs without work (128
  // tokens of [1152, 6912], K split 4 ways: 11.7 us, 14.5 with 128)
  const int BN = M <= 16 ? 16 : M <= 32 ? 32 : 64;
  // More than 64 tokens: CTA pairs, which load less per product, unless the
  // one-SM tiles are so few that they split K. us, one-SM and pairs (* this
  // rule's): 2048 tokens of [21504, 5376] 416, 245*; 128 of it 44.7, 39.9*; 333
  // of [2056, 1168] 12.7, 12.3*; 256 of [5376, 8192] 30.2, 28.0*; 100 of [1152,
  // 6912] 11.6*, 22.5. It asks for a split that the tiles could take on SMs of
  // their own; with one they cannot, 128 tokens of [8192, 5376] take 19.4 (2
  // ways), 21.7*, of [5376, 8192] 21.5, 27.6*, of [5376, 21504] 40.1, 57.6*.
  const bool pair = M > 64 && tile_splits(c, ceil_div(O, kBM), ceil_div(M, 64), (int)ceil_div(I, kBK)) == 1;
  const int box = pair ? width / 2 : BN;  // tokens per box
  Maps mp;
  if ((st = make_map_box(&mp.w, wq, O, I, kBM, kBK, CU_TENSOR_MAP_SWIZZLE_128B, ce, 1))) return st;
  if ((st = make_map_box(&mp.x, xq, M, I, box, kBK, CU_TENSOR_MAP_SWIZZLE_128B, ce, 1))) return st;
  mp.u = mp.w;
  mp.th = mp.tl = mp.x;
  if (r > 0 && !few) {
    if ((st = make_map_box(&mp.u, U, O, r, kBM, kRankBK, CU_TENSOR_MAP_SWIZZLE_128B, ce))) return st;
    if ((st = make_map_box(&mp.th, t_hi, M, r, box, kRankBK, CU_TENSOR_MAP_SWIZZLE_128B, ce))) return st;
    if ((st = make_map_box(&mp.tl, t_lo, M, r, box, kRankBK, CU_TENSOR_MAP_SWIZZLE_128B, ce))) return st;
  }
  Args a = {};
  a.rows = (int)O;
  a.cols = (int)M;
  a.kb1 = (int)ceil_div(I, kBK);
  a.kb2 = few ? 0 : (int)ceil_div(r, kRankBK);
  a.splits = 1;
  a.xs = static_cast<const uint8_t*>(xs);
  a.ws = static_cast<const uint8_t*>(ws);
  a.t_parts = static_cast<const float*>(work);
  a.U = static_cast<const bf16*>(U);
  a.nparts = nparts;
  a.r = r;
  a.s = s;
  a.out = static_cast<bf16*>(Y);
  a.early_start = r > 0;
  a.tile_tokens = width;
  a.err = c.err;
  if (pair) {
    CUtensorMap mY;
    if ((st = make_map_box(&mY, Y, M, O, width, kBM, CU_TENSOR_MAP_SWIZZLE_NONE, ce))) return st;
    *ce = launch_pair(c, mp, a, mY);
  } else {
    switch (BN) {
      case 16: *ce = few ? launch_tile<16, true>(c, mp, a) : launch_tile<16>(c, mp, a); break;
      case 32: *ce = launch_tile<32>(c, mp, a); break;
      default: *ce = launch_tile<64>(c, mp, a); break;
    }
  }
  return *ce == cudaSuccess ? THETA_OK : THETA_ERR_CUDA;
}

}  // namespace theta
