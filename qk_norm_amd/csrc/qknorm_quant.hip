// Rows to 8-bit integers with one scale a row (gfx950).
//
//   amax = max_j |x_j|,  scale = amax / 127,  q_j = rne(127 * x_j / amax)
//
// The row is read once and held in registers between the maximum and the
// quotients (rows past 16384 values are read twice).  Bound by memory: 3
// bytes a value.
//
// The quotient decides between neighbouring integers, and x = amax / 2 lies
// exactly halfway (63.5), so it is rounded correctly rather than taken as a
// product with a reciprocal: y = (127 x) * rcp(amax) and one residual step
// y += (127 x - y amax) * rcp(amax).  127 x has at most 18 significant bits
// and the residual is exact in one fma, so a quotient that is exactly halfway
// comes out exactly halfway; any other is at least 2^-20 (relative) away from
// one, and y is within 2^-23.  Adding 1.5 * 2^23 rounds to nearest even and
// leaves the integer in the low byte.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qknorm_device.hpp"
#include "qknorm_launch.hpp"

namespace qknorm {

namespace {

// Rows are read through the caches (the kernel before has just written them) and
// the integers stored with `nt`: 8192 rows of 4096 in 16.5 us, 6.1 TB/s; with
// `nt sc1` loads and stores, as the norms have them, 19.3.
constexpr int kRowStore = 2;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Magnitudes order like their bits, NaN above infinity above the finite, so
// the maximum is one of unsigned halves.
__device__ __forceinline__ uint32_t max_abs2(uint32_t v, uint32_t m) {
  const uint32_t a = v & 0x7FFF7FFFu;
  const u16x2 r = __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, m));
  return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t w = __shfl_xor(v, o);
    v = v > w ? v : w;
  }
  return v;
}

// What the row's largest magnitude (its 16 bits) says: the factor of x, the
// divisor and its reciprocal (rows past 2^64 are scaled down by 2^64 first,
// where 127 x would overflow), and the stored scale.  Below 2^-100 the row is
// zeros with scale 0; a row with an infinity or a NaN is zeros with scale NaN.
struct RowScale {
  float mul, div, rcp, scale;
  bool zero;
};

template <int DT>
__device__ __forceinline__ RowScale row_scale(uint32_t bits) {
  constexpr uint32_t kInf = DT == kBF16 ? 0x7F80u : 0x7C00u;
  float a;
  if constexpr (DT == kBF16) {
    a = __uint_as_float(bits << 16);
  } else {
    const uint16_t h = (uint16_t)bits;
    a = (float)__builtin_bit_cast(_Float16, h);
  }
  RowScale s;
  const bool bad = bits >= kInf, tiny = a < 0x1p-100f;
  s.zero = bad || tiny;
  s.scale = bad ? __builtin_nanf("") : (tiny ? 0.f : a / 127.f);
  const float down = a >= 0x1p64f ? 0x1p-64f : 1.f;
  s.mul = s.zero ? 0.f : 127.f * down;
  s.div = s.zero ? 1.f : a * down;
  s.rcp = __builtin_amdgcn_rcpf(s.div);
  return s;
}

template <int DT>
__device__ __forceinline__ u32x2 quantise8(u32x4 v, const RowScale& s) {
  float f[8];
  unpack<DT>(v, f);
  uint32_t b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = f[e] * s.mul;
    float y = x * s.rcp;
    y = __builtin_fmaf(__builtin_fmaf(-y, s.div, x), s.rcp, y);
    // (an infinity or a NaN in a row of scale NaN gives NaN here)
    b[e] = __float_as_uint(y + 12582912.f);
  }
  u32x2 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x0C0C0400u);
    o[i] = s.zero ? 0u : (lo | (hi << 16));
  }
  return o;
}

// WPR waves a row (1 or 4), V vectors of 8 values a lane; KEEP: the row fits
// 512 * WPR * V values and stays in registers.
template <int DT, int WPR, int V, bool KEEP>
__global__ __launch_bounds__(256) void quant_rows_kernel(const uint8_t* __restrict__ x, uint64_t ldx_bytes,
                                                         uint8_t* __restrict__ q, uint64_t ldq,
                                                         float* __restrict__ scale, uint32_t T, uint32_t n) {
  constexpr uint32_t kRows = 4 / WPR;
  __shared__ uint32_t part[4];
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t row = blockIdx.x * kRows + wave / WPR;
  const bool live = row < T;                      // (whole rows: the barrier below is WPR = 4's only)
  if (WPR == 1 && !live) return;
  const Rsrc rx = make_rsrc(x + (uint64_t)row * ldx_bytes, (uint64_t)n * 2);
  const Rsrc rq = make_rsrc(q + (uint64_t)row * ldq, (uint64_t)n);
  const uint32_t first = (WPR == 1 ? lane : threadIdx.x), step = 64 * WPR;   // in vectors
  u32x4 v[V];
  uint32_t m = 0;
  if constexpr (KEEP) {
    // vectors past the row's end read zeros
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = cached_load(rx, (first + i * step) * 16);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = max_abs2(v[i][e], m);
  } else {
    for (uint32_t b = first; b < n / 8; b += V * step) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = cached_load(rx, (b + i * step) * 16);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max_abs2(v[i][e], m);
    }
  }
  m = (m & 0xFFFFu) > (m >> 16) ? (m & 0xFFFFu) : (m >> 16);
  m = wave_max_u32(m);
  if constexpr (WPR == 4) {
    if (lane == 0) part[wave] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) m = m > part[i] ? m : part[i];
  }
  const RowScale s = row_scale<DT>(m);
  if (first == 0) scale[row] = s.scale;
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      __builtin_amdgcn_raw_buffer_store_b64(quantise8<DT>(v[i], s), rq, (first + i * step) * 8, 0, kRowStore);
  } else {
    for (uint32_t b = first; b < n / 8; b += V * step) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = cached_load(rx, (b + i * step) * 16);
#pragma unroll
      for (int i = 0; i < V; ++i)
        __builtin_amdgcn_raw_buffer_store_b64(quantise8<DT>(v[i], s), rq, (b + i * step) * 8, 0, kRowStore);
    }
  }
}

template <int DT>
hipError_t launch(const QuantArgs& a, hipStream_t s) {
  const uint32_t T = (uint32_t)a.T, n = (uint32_t)a.n;
  auto go = [&](auto kern, uint32_t rows) {
    hipLaunchKernelGGL(kern, dim3((T + rows - 1) / rows), dim3(256), 0, s, (const uint8_t*)a.x, (uint64_t)a.ldx * 2,
                       (uint8_t*)a.q, (uint64_t)a.ldq, a.scale, T, n);
    return hipGetLastError();
  };
  if (n <= 512) return go(quant_rows_kernel<DT, 1, 1, true>, 4);
  if (n <= 2048) return go(quant_rows_kernel<DT, 1, 4, true>, 4);
  if (n <= 4096) return go(quant_rows_kernel<DT, 4, 2, true>, 1);
  if (n <= 8192) return go(quant_rows_kernel<DT, 4, 4, true>, 1);
  if (n <= 16384) return go(quant_rows_kernel<DT, 4, 8, true>, 1);
  return go(quant_rows_kernel<DT, 4, 4, false>, 1);
}

}  // namespace

hipError_t launch_quant_rows(const QuantArgs& a, hipStream_t s) {
  return a.dtype == kF16 ? launch<kF16>(a, s) : launch<kBF16>(a, s);
}

}  // namespace qknorm
