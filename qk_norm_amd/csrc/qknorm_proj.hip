// The QKV projection with per-head QK-Norm in its epilogue (gfx950).
//
// qkv[t, n] = sum_k x[t, k] * w[n, k] (x is [T, K], w the projection weight
// [N, K], both K-contiguous: the "NT" product), accumulated in fp32 by MFMA;
// before the result is ever rounded, each Q head and each K head of a row is
// RMS-normalised over its head_dim values and multiplied by its gamma, and
// the V columns are stored as they are.  One pass instead of a projection
// that writes qkv and a normalisation that reads and writes it again.
//
// Tiling: a block of 512 threads (4 x 2 waves, two per SIMD) owns a 256 x 256
// output tile; each wave a 64 x 128 slab of 4 x 8 v_mfma_f32_16x16x32_bf16
// blocks (v_mfma_f32_16x16x32_f16 for fp16, the same layout).  K advances 64
// at a time through a ring of LDS stages (two for these tiles, three or four
// for the smaller ones) filled straight from global memory (buffer loads
// into LDS, no staging registers), with the operand rows XOR-swizzled so that
// fragment reads hit distinct banks.  Where 256 x 256 tiles would leave a
// round of the chip's CUs half empty, the last columns go to 256 x 128 tiles
// of the same launch.  Tiles are ordered so the blocks
// each XCD holds at once share operand panels in its L2.  Because tile widths
// are multiples of head_dim (or one head spans a tile's two column waves)
// and tiles start at multiples of it, a tile holds whole heads, and the
// epilogue normalises them in registers without leaving the block.  The
// MFMAs take the weight's fragment as their first operand, so a lane's
// accumulators are four consecutive columns of one token: one lane swap
// then gives each lane eight consecutive outputs, stored as one 16-byte
// write straight from registers.
//
// Fewer tokens take narrower launches of the same kernel (128-row tiles one
// head wide up to 512 tokens, or on to 1024 while they fit one round of the
// CUs; 64-row tiles from 1 token to 256).  With a workspace, up to 64 tokens
// take two other kernels instead: the weight split over many more blocks
// into fp32 partials, then one block per head adding them and normalising
// (qkv_proj_split_kernel, qkv_proj_split_finish_kernel).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "qknorm_launch.hpp"
#include "qknorm_proj_tiles.hpp"

namespace qknorm {

bool proj_shape_ok(const ProjArgs& a) {
  // buffer offsets inside one tile's rows stay below 2^31
  const uint64_t es = 2;
  return (uint64_t)kBM * a.ldx * es < (UINT64_C(1) << 31) &&
         (uint64_t)kBN * a.ldw * es < (UINT64_C(1) << 31) &&
         (uint64_t)kBM * a.ld * es < (UINT64_C(1) << 31) && a.hidden % 64 == 0 &&
         // the tiles (full or half-width) are numbered in one grid
         // dimension, whose size in threads must fit 32 bits
         (uint64_t)((a.T + kBM - 1) / kBM) *
                 (uint64_t)(((a.hq + 2 * a.hkv) * a.head_dim + GeoH::BN - 1) / GeoH::BN) *
                 (uint64_t)kThreads <
             (UINT64_C(1) << 32) &&
         (a.head_dim == 64 || a.head_dim == 128 || a.head_dim == 256);
}

// Where the half-width tail starts: the column n_split (a multiple of 256)
// that minimises the estimated time in rounds of the chip's CUs, a full tile
// costing 1 and a half-width tile kHalfCost; n_split = N means no tail.
// Head dims above 128 never split (a half-width tile would cut a head).
uint32_t proj_split_column(uint32_t T, uint32_t N, uint32_t head_dim, int cus) {
#ifndef QKNORM_PROJ_HALF_COST
#define QKNORM_PROJ_HALF_COST 0.6
#endif
  constexpr double kHalfCost = QKNORM_PROJ_HALF_COST;
  const uint64_t m_tiles = (T + kBM - 1) / kBM;
  const uint64_t c = cus > 0 ? (uint64_t)cus : 1;
  auto rounds = [&](uint64_t n) { return (double)((n + c - 1) / c); };
  const uint64_t all = m_tiles * ((N + kBN - 1) / kBN);
  uint32_t best = N;
  double best_cost = rounds(all);
  if (!kSplit || head_dim > (uint32_t)GeoH::BN) return best;
  for (uint32_t n1 = 0; n1 < N; n1 += kBN) {
    const uint64_t full = m_tiles * (n1 / kBN);
    const uint64_t half = m_tiles * ((N - n1 + GeoH::BN - 1) / GeoH::BN);
    const double cost = rounds(full) + kHalfCost * rounds(half);
    if (cost < best_cost - 1e-9) { best_cost = cost; best = n1; }
  }
  return best;
}

// The kernel arguments of one call (both kernels take them).
static ProjKArgs kernel_args(const ProjArgs& a) {
  ProjKArgs k;
  k.x = (const uint8_t*)a.x;
  k.w = (const uint8_t*)a.w;
  k.out = (uint8_t*)a.qkv;
  k.gamma_q = (const uint8_t*)a.gamma_q;
  k.gamma_k = (const uint8_t*)a.gamma_k;
  k.ld_bytes = (uint64_t)a.ld * 2;
  k.ldx_bytes = (uint32_t)(a.ldx * 2);
  k.ldw_bytes = (uint32_t)(a.ldw * 2);
  k.T = (uint32_t)a.T;
  k.K = (uint32_t)a.hidden;
  k.N = (uint32_t)((a.hq + 2 * a.hkv) * a.head_dim);
  k.hq = (uint32_t)a.hq;
  k.hkv = (uint32_t)a.hkv;
  k.norm = (uint32_t)((a.flags & 1) == 0);
  k.eps = a.eps;
  k.inv_d = 1.0f / (float)a.head_dim;
  k.x_scale = k.w_scale = nullptr;
  return k;
}

// One launch of geometry G (G256 for head_dim 256), every block a full tile.
template <class G, class G256>
static hipError_t launch_qkv_proj_tiles(const ProjArgs& a, hipStream_t s) {
  const uint32_t N = (uint32_t)((a.hq + 2 * a.hkv) * a.head_dim);
  const uint32_t m_tiles = (uint32_t)((a.T + G::BM - 1) / G::BM);
  const uint32_t bn = a.head_dim == 256 ? G256::BN : G::BN;
  const uint32_t tiles = m_tiles * ((N + bn - 1) / bn);
  auto kern = a.dtype == kF16
                  ? (a.head_dim == 64    ? qkv_proj_kernel<G, G, kF16, kF16, 64>
                     : a.head_dim == 128 ? qkv_proj_kernel<G, G, kF16, kF16, 128>
                                         : qkv_proj_kernel<G256, G256, kF16, kF16, 256>)
                  : (a.head_dim == 64    ? qkv_proj_kernel<G, G, kBF16, kBF16, 64>
                     : a.head_dim == 128 ? qkv_proj_kernel<G, G, kBF16, kBF16, 128>
                                         : qkv_proj_kernel<G256, G256, kBF16, kBF16, 256>);
  const int lds = (a.head_dim == 256 ? G256::kStagesBytes : G::kStagesBytes) +
                  (kGammaFloats + kHalfFloats) * 4;
  static_assert(G::kStagesBytes + (kGammaFloats + kHalfFloats) * 4 <= 160 * 1024 &&
                    G256::kStagesBytes + (kGammaFloats + kHalfFloats) * 4 <= 160 * 1024,
                "the stages fit a CU's 160 KiB of LDS");
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(tiles), dim3(G::kThreads), lds, s, kernel_args(a), tiles, N);
  return hipGetLastError();
}

// The split geometry for a token count: KS slices of K, blocks of 16 * JB
// columns, TB blocks of 16 tokens.  Up to 8 tokens 16 columns by 4 slices
// (1536 blocks for the Qwen3-8B layer; with the norm kernel 12.1 us per
// call at T = 1 and 14.8 us at T = 8, against 12.2 and 14.9 us with 8
// slices); from 9 tokens 32 columns, which halves the activation fragments
// loaded per weight fragment (17.2 against 18.5 us at T = 16).  From 17
// tokens two or four token blocks share each weight fragment; K slices
// measured with the weight rotating through 6 copies: 8 slices 17.0, 18.0
// and 19.9 us at 17, 24 and 32 tokens (4 slices 17.6, 18.7, 19.8; 16 slices
// 18.2, 20.0, 21.9); 4 slices 23.4 and 25.8 us at 48 and 64 tokens (8
// slices 24.0 and 27.3; 2 slices 26.7 and 30.1).
#ifndef QKNORM_PROJ_SPLIT_KS32
#define QKNORM_PROJ_SPLIT_KS32 8   // K slices for 17 to 32 tokens
#endif
#ifndef QKNORM_PROJ_SPLIT_KS64
#define QKNORM_PROJ_SPLIT_KS64 4   // K slices for 33 to 64 tokens
#endif
struct SplitGeo {
  uint32_t ks, jb, tb;
};
static SplitGeo split_geo(int64_t T) {
  if (T <= 8) return SplitGeo{4, 1, 1};
  if (T <= 16) return SplitGeo{8, 2, 1};
  if (T <= 32) return SplitGeo{QKNORM_PROJ_SPLIT_KS32, 2, 2};
  return SplitGeo{QKNORM_PROJ_SPLIT_KS64, 2, 4};
}

int64_t proj_workspace_bytes(int64_t T, int64_t N) {
  if (T <= 0 || T > kProjSplitMaxT || N <= 0) return 0;
  const int64_t b = (int64_t)split_geo(T).ks * T * N * 4;
  return (b + 255) & ~(int64_t)255;
}

typedef void (*SplitKernel)(ProjKArgs, float*);
typedef void (*FinishKernel)(ProjKArgs, const float*);

template <int DT, int D>
static void split_kernels(const SplitGeo& g, SplitKernel* k1, FinishKernel* k2) {
  constexpr int S32 = QKNORM_PROJ_SPLIT_KS32, S64 = QKNORM_PROJ_SPLIT_KS64;
  if (g.tb == 1 && g.jb == 1) {
    *k1 = qkv_proj_split_kernel<DT, D, 4, 1, 1, 8>;
    *k2 = qkv_proj_split_finish_kernel<DT, DT, D, 4>;
  } else if (g.tb == 1) {
    *k1 = qkv_proj_split_kernel<DT, D, 8, 2, 1, 4>;
    *k2 = qkv_proj_split_finish_kernel<DT, DT, D, 8>;
  } else if (g.tb == 2) {
    *k1 = qkv_proj_split_kernel<DT, D, S32, 2, 2, 4>;
    *k2 = qkv_proj_split_finish_kernel<DT, DT, D, S32>;
  } else {
    *k1 = qkv_proj_split_kernel<DT, D, S64, 2, 4, 4>;
    *k2 = qkv_proj_split_finish_kernel<DT, DT, D, S64>;
  }
}

template <int DT>
static void split_kernels_dt(int head_dim, const SplitGeo& g, SplitKernel* k1, FinishKernel* k2) {
  if (head_dim == 64) split_kernels<DT, 64>(g, k1, k2);
  else if (head_dim == 128) split_kernels<DT, 128>(g, k1, k2);
  else split_kernels<DT, 256>(g, k1, k2);
}

hipError_t launch_qkv_proj_split(const ProjArgs& a, void* workspace, hipStream_t s) {
  const SplitGeo g = split_geo(a.T);
  const uint32_t N = (uint32_t)((a.hq + 2 * a.hkv) * a.head_dim);
  SplitKernel k1;
  FinishKernel k2;
  if (a.dtype == kF16) split_kernels_dt<kF16>(a.head_dim, g, &k1, &k2);
  else split_kernels_dt<kBF16>(a.head_dim, g, &k1, &k2);
  const ProjKArgs k = kernel_args(a);
  float* part = static_cast<float*>(workspace);
  hipLaunchKernelGGL(k1, dim3(N / (16 * g.jb) * g.ks), dim3(256), 0, s, k, part);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k2, dim3(N / (uint32_t)a.head_dim, (uint32_t)(a.T + 15) / 16), dim3(256), 0, s, k,
                     (const float*)part);
  return hipGetLastError();
}

// The split projection's partials for callers that cannot allocate a
// workspace: one array per GPU, held from the library's load until the
// process ends.  Host code never passes the array's name to a kernel (on the
// host it names a stand-in, not device memory); the device address comes
// from hipGetSymbolAddress, looked up once per device with that device
// current and kept per device.  Every such call on one GPU shares the array,
// so calls that can overlap on one GPU (different streams) race.  Nothing in
// it needs clearing between calls: the first kernel writes every partial the
// second one reads.
static __device__ __align__(256) uint8_t scratch[kProjScratchBytes];

static std::mutex g_scratch_mu;
static std::atomic<void*> g_scratch_ptr[kMaxScratchDevices];

hipError_t proj_scratch(void** ptr) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxScratchDevices) return hipErrorInvalidDevice;
  void* p = g_scratch_ptr[dev].load(std::memory_order_acquire);
  if (p == nullptr) {
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    p = g_scratch_ptr[dev].load(std::memory_order_relaxed);
    if (p == nullptr) {
      e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
      if (e != hipSuccess || p == nullptr) return e != hipSuccess ? e : hipErrorInvalidSymbol;
      g_scratch_ptr[dev].store(p, std::memory_order_release);
    }
  }
  *ptr = p;
  return hipSuccess;
}

hipError_t launch_qkv_proj(const ProjArgs& a, hipStream_t s, int cus) {
  if (a.T <= QKNORM_PROJ_SMALL_T) return launch_qkv_proj_tiles<GeoS, GeoS256>(a, s);
  const uint32_t N = (uint32_t)((a.hq + 2 * a.hkv) * a.head_dim);
  // 128-row tiles up to 512 tokens, and up to 1024 while they fit one round
  // of the chip's CUs (on a Qwen3-8B layer up to 640 tokens: 36 against 43 us
  // for the 256-row launch at 513 tokens, 60 against 52 us at 768, where a
  // second round would hold 32 tiles)
  const uint64_t bn_m = a.head_dim == 256 ? GeoM256::BN : GeoM::BN;
  const uint64_t m_tiles_m = (uint64_t)(a.T + GeoM::BM - 1) / GeoM::BM;
  if (a.T <= QKNORM_PROJ_MID_T ||
      (a.T <= 2 * QKNORM_PROJ_MID_T && m_tiles_m * ((N + bn_m - 1) / bn_m) <= (uint64_t)(cus > 0 ? cus : 1)))
    return launch_qkv_proj_tiles<GeoM, GeoM256>(a, s);
  const uint32_t T = (uint32_t)a.T;
  const uint32_t n_split = proj_split_column(T, N, (uint32_t)a.head_dim, cus);
  const uint32_t m_tiles = (T + kBM - 1) / kBM;
  const uint32_t n_full = m_tiles * ((n_split + kBN - 1) / kBN);
  const uint32_t n_half = n_split < N ? m_tiles * ((N - n_split + GeoH::BN - 1) / GeoH::BN) : 0;
  auto pick = [&](auto k64, auto k128, auto k256) {
    return a.head_dim == 64 ? k64 : (a.head_dim == 128 ? k128 : k256);
  };
  auto kern = a.dtype == kF16
                  ? pick(qkv_proj_kernel<GeoF, GeoH, kF16, kF16, 64>, qkv_proj_kernel<GeoF, GeoH, kF16, kF16, 128>,
                         qkv_proj_kernel<GeoF, GeoH, kF16, kF16, 256>)
                  : pick(qkv_proj_kernel<GeoF, GeoH, kBF16, kBF16, 64>, qkv_proj_kernel<GeoF, GeoH, kBF16, kBF16, 128>,
                         qkv_proj_kernel<GeoF, GeoH, kBF16, kBF16, 256>);
  // more than the default 64 KiB of dynamic LDS (gfx950 has 160 KiB per CU);
  // a host-side attribute, set on every call (no shared state between threads)
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kLdsBytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(n_full + n_half), dim3(kThreads), kLdsBytes, s, kernel_args(a), n_full,
                     n_split);
  return hipGetLastError();
}

}  // namespace qknorm
