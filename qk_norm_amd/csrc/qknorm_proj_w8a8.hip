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

template <int DT, int D>
hipError_t by_tokens(const W8a8Args& q, hipStream_t s, int cus) {
  typedef typename std::conditional<D == 256, GeoS256, GeoS>::type S;
  typedef typename std::conditional<D == 256, GeoM256, GeoM>::type M;
  const ProjArgs& a = q.p;
  if (a.T <= QKNORM_PROJ_SMALL_T) return one_shape<S, DT, D>(q, s);
  const uint32_t T = (uint32_t)a.T, N = (uint32_t)((a.hq + 2 * a.hkv) * D);
  const uint64_t tiles_m = (uint64_t)((T + M::BM - 1) / M::BM) * ((N + M::BN - 1) / M::BN);
  if (a.T <= QKNORM_PROJ_MID_T || (a.T <= 2 * QKNORM_PROJ_MID_T && tiles_m <= (uint64_t)(cus > 0 ? cus : 1)))
    return one_shape<M, DT, D>(q, s);
  const uint32_t n_split = proj_split_column(T, N, D, cus), m_tiles = (T + kBM - 1) / kBM;
  const uint32_t n_full = m_tiles * ((n_split + kBN - 1) / kBN);
  const uint32_t n_half = n_split < N ? m_tiles * ((N - n_split + GeoH::BN - 1) / GeoH::BN) : 0;
  return tiles<GeoF, GeoH, DT, D>(q, n_full, n_half, n_split, s);
}

template <int DT, int D, int KS, int JB, int TB, int PF>
hipError_t split(const W8a8Args& q, void* workspace, hipStream_t s) {
  const uint32_t N = (uint32_t)((q.p.hq + 2 * q.p.hkv) * D);
  const ProjKArgs k = w8a8_args(q);
  float* part = static_cast<float*>(workspace);
  hipLaunchKernelGGL((qkv_proj_split_kernel<kI8, D, KS, JB, TB, PF>), dim3(N / (16 * JB) * KS), dim3(256), 0, s, k, part);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((qkv_proj_split_finish_kernel<kI8, DT, D, KS>), dim3(N / D, (uint32_t)(q.p.T + 15) / 16), dim3(256),
                     0, s, k, (const float*)part);
  return hipGetLastError();
}

template <int DT, int D>
hipError_t split_by_tokens(const W8a8Args& q, void* w, hipStream_t s) {
  if (q.p.T <= 8) return split<DT, D, 4, 1, 1, 8>(q, w, s);
  if (q.p.T <= 16) return split<DT, D, 8, 2, 1, 4>(q, w, s);
  if (q.p.T <= 32) return split<DT, D, 8, 2, 2, 4>(q, w, s);
  return split<DT, D, 4, 2, 4, 4>(q, w, s);
}

// K slices of a token count (as above), for the workspace's size.
int64_t slices(int64_t T) { return T <= 8 ? 4 : (T <= 32 ? 8 : 4); }

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
  return (slices(T) * T * N * 4 + 255) & ~(int64_t)255;
}

hipError_t launch_w8a8(const W8a8Args& q, void* workspace, hipStream_t s, int cus) {
  if (workspace != nullptr) return by_type<Split>(q, workspace, s);
  return by_type<Tiles>(q, s, cus);
}

}  // namespace qknorm
