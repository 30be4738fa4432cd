// The QKV projection on 8-bit integers, QK-Norm in its epilogue (gfx950).
//
//   qkv[t, n] = (sum_k xq[t, k] * wq[n, k]) * w_scale[n] * x_scale[t]
//
// with xq and wq int8, the sum exact in int32 (v_mfma_i32_16x16x64_i8: twice
// the products of the 16-bit MFMA in the same time from the same bytes), then
// each Q and K head normalised as in the 16-bit projection.  The tiles, their
// LDS stages and the split over K for few tokens are the 16-bit kernels' with
// K counted in bytes; the scales wait in LDS and meet the sums in the
// epilogue.  Integer partial sums are exact in any order, so the split over K
// adds nothing to the rounding.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qknorm_launch.hpp"
#include "qknorm_proj_tiles.hpp"

namespace qknorm {

namespace {

constexpr int kTables = (kGammaFloats + kHalfFloats + kScaleFloats) * 4;

ProjKArgs w8a8_args(const W8a8Args& q) {
  const ProjArgs& a = q.p;
  ProjKArgs k;
  k.x = (const uint8_t*)a.x;
  k.w = (const uint8_t*)a.w;
  k.out = (uint8_t*)a.qkv;
  k.gamma_q = (const uint8_t*)a.gamma_q;
  k.gamma_k = (const uint8_t*)a.gamma_k;
  k.ld_bytes = (uint64_t)a.ld * 2;
  k.ldx_bytes = (uint32_t)a.ldx;
  k.ldw_bytes = (uint32_t)a.ldw;
  k.T = (uint32_t)a.T;
  k.K = (uint32_t)(a.hidden / 2);
  k.N = (uint32_t)((a.hq + 2 * a.hkv) * a.head_dim);
  k.hq = (uint32_t)a.hq;
  k.hkv = (uint32_t)a.hkv;
  k.norm = (uint32_t)((a.flags & 1) == 0);
  k.eps = a.eps;
  k.inv_d = 1.0f / (float)a.head_dim;
  k.x_scale = q.x_scale;
  k.w_scale = q.w_scale;
  return k;
}

// One launch: n_full blocks of GF over columns [0, n_split), the rest GH.
template <class GF, class GH, int DT, int D>
hipError_t tiles(const W8a8Args& q, uint32_t n_full, uint32_t n_half, uint32_t n_split, hipStream_t s) {
  constexpr int kLds = (GF::kStagesBytes > GH::kStagesBytes ? GF::kStagesBytes : GH::kStagesBytes) + kTables;
  static_assert(kLds <= 160 * 1024, "the stages fit a CU's 160 KiB of LDS");
  auto kern = qkv_proj_kernel<GF, GH, kI8, DT, D>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(n_full + n_half), dim3(GF::kThreads), kLds, s, w8a8_args(q), n_full, n_split);
  return hipGetLastError();
}

template <class G, int DT, int D>
hipError_t one_shape(const W8a8Args& q, hipStream_t s) {
  const uint32_t T = (uint32_t)q.p.T, N = (uint32_t)((q.p.hq + 2 * q.p.hkv) * D);
  return tiles<G, G, DT, D>(q, (T + G::BM - 1) / G::BM * ((N + G::BN - 1) / G::BN), 0, N, s);
}

// Tile shapes: 64 or 128 rows one head wide (256 columns for head_dim 256),
// or the 256-row tiles.  The shape is the one whose rounds of the chip's CUs
// are estimated to take the least time, in units of a round of 64-row tiles;
// a round of each on a Qwen3-8B layer (hidden 4096): 64 rows 15.2 us, 128
// rows 19.2, 256 x 128 26.4, 256 x 256 48.5.  By the 16-bit projection's token
// ranges instead: 11.5 against 9.1 us for 333 tokens by 1728 columns of a
// hidden size of 2048, 17.0 against 12.8 for 1500 by 2560.
//
// What bounds a K step of the smaller tiles is the LDS: 64 rows read 80 KiB
// of fragments and take in 24 KiB, 830 cycles at 128 bytes a cycle of the 900
// measured.  Three to six stages, K steps of 256 bytes, and four waves of
// twice the rows (fewer fragment reads, but one wave a SIMD) measured the
// same or slower.  The 256 x 256 tiles need the LDS and the matrix cores for
// 2048 cycles each of the 3300 that a step takes.
// (head_dim 256: 64 x 256 22.0 us, 128 x 256 26.6, 256 x 256 43.5.)
constexpr double kCostM = 1.27, kCostH = 1.75;
constexpr double cost_full(int d) { return d == 256 ? 1.9 : 3.2; }

template <int DT, int D>
hipError_t by_tokens(const W8a8Args& q, hipStream_t s, int cus) {
  typedef typename std::conditional<D == 256, GeoS256, GeoS>::type S;
  typedef typename std::conditional<D == 256, GeoM256, GeoM>::type M;
  const ProjArgs& a = q.p;
  const uint32_t T = (uint32_t)a.T, N = (uint32_t)((a.hq + 2 * a.hkv) * D);
  const uint64_t c = cus > 0 ? (uint64_t)cus : 1;
  auto rounds = [&](uint64_t tiles) { return (double)((tiles + c - 1) / c); };
  auto count = [&](uint32_t bm, uint32_t bn) { return (uint64_t)((T + bm - 1) / bm) * ((N + bn - 1) / bn); };
  const uint32_t n_split = proj_split_column(T, N, D, cus), m_tiles = (T + kBM - 1) / kBM;
  const uint32_t n_full = m_tiles * ((n_split + kBN - 1) / kBN);
  const uint32_t n_half = n_split < N ? m_tiles * ((N - n_split + GeoH::BN - 1) / GeoH::BN) : 0;
  const double cost_s = rounds(count(S::BM, S::BN)), cost_m = kCostM * rounds(count(M::BM, M::BN));
  const double cost_f = cost_full(D) * rounds(n_full) + kCostH * rounds(n_half);
  if (cost_s <= cost_m && cost_s <= cost_f) return one_shape<S, DT, D>(q, s);
  if (cost_m <= cost_f) return one_shape<M, DT, D>(q, s);
  return tiles<GeoF, GeoH, DT, D>(q, n_full, n_half, n_split, s);
}

// The split form: four slices of K by 32 columns for every token count, one,
// two or four 16-token blocks a weight fragment.  On the Qwen3-8B layer 8.2
// us at 1 token, 8.7 at 8, 9.9 at 16, 11.4 at 32 and 14.8 at 64 (the 16-bit
// kernel's slices and columns: 8.2, 9.1, 10.5, 12.1, 14.8; two slices: 8.3,
// 9.3, 11.1, 13.2, 16.9; 16 columns from 17 tokens: 13.6 and 19.9).  Of the
// 8.2 us the weight's 25 MB take 4.1 at 6.2 TB/s and the second launch 1.8.
constexpr int kSlices = 4;

template <int DT, int D, int TB>
hipError_t split(const W8a8Args& q, void* workspace, hipStream_t s) {
  const uint32_t N = (uint32_t)((q.p.hq + 2 * q.p.hkv) * D);
  const ProjKArgs k = w8a8_args(q);
  float* part = static_cast<float*>(workspace);
  hipLaunchKernelGGL((qkv_proj_split_kernel<kI8, D, kSlices, 2, TB, 4>), dim3(N / 32 * kSlices), dim3(256), 0, s, k, part);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((qkv_proj_split_finish_kernel<kI8, DT, D, kSlices>), dim3(N / D, (uint32_t)(q.p.T + 15) / 16),
                     dim3(256), 0, s, k, (const float*)part);
  return hipGetLastError();
}

template <int DT, int D>
hipError_t split_by_tokens(const W8a8Args& q, void* w, hipStream_t s) {
  if (q.p.T <= 16) return split<DT, D, 1>(q, w, s);
  if (q.p.T <= 32) return split<DT, D, 2>(q, w, s);
  return split<DT, D, 4>(q, w, s);
}

template <template <int, int> class F, class... A>
hipError_t by_type(const W8a8Args& q, A... args) {
  const bool h = q.p.dtype == kF16;
  if (q.p.head_dim == 64) return h ? F<kF16, 64>::go(q, args...) : F<kBF16, 64>::go(q, args...);
  if (q.p.head_dim == 128) return h ? F<kF16, 128>::go(q, args...) : F<kBF16, 128>::go(q, args...);
  return h ? F<kF16, 256>::go(q, args...) : F<kBF16, 256>::go(q, args...);
}
template <int DT, int D>
struct Tiles {
  static hipError_t go(const W8a8Args& q, hipStream_t s, int cus) { return by_tokens<DT, D>(q, s, cus); }
};
template <int DT, int D>
struct Split {
  static hipError_t go(const W8a8Args& q, void* w, hipStream_t s) { return split_by_tokens<DT, D>(q, w, s); }
};

}  // namespace

bool w8a8_shape_ok(const ProjArgs& a) {
  // as for 16-bit operands, with x and w one byte a value; no int32 sum of
  // hidden products of int8 values (at most 2^14 each) overflows
  ProjArgs b = a;
  b.ldx = (a.ldx + 1) / 2;
  b.ldw = (a.ldw + 1) / 2;
  return a.hidden < 131072 && proj_shape_ok(b);
}

int64_t w8a8_workspace_bytes(int64_t T, int64_t N) {
  if (T <= 0 || T > kProjSplitMaxT || N <= 0) return 0;
  return (kSlices * T * N * 4 + 255) & ~(int64_t)255;
}

hipError_t launch_w8a8(const W8a8Args& q, void* workspace, hipStream_t s, int cus) {
  if (workspace != nullptr) return by_type<Split>(q, workspace, s);
  return by_type<Tiles>(q, s, cus);
}

}  // namespace qknorm
