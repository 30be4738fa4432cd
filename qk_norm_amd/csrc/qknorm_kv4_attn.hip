// Attention of fused rows' Q over the paged 4-bit KV cache (gfx950).
//
//   o_t = sum_j p_tj V_j,  p_tj = exp(c q_t.K_j - m_t) / l_t  over the visible j
//
// in one pass over the cache with the running maximum m and sum l of each
// row.  K_j = sk_j * (codes of K_j): the matrix products take the codes alone
// (exact in bf16 and fp16; one conversion instruction makes two of them) and
// the scale multiplies the score.  Likewise the weight of V_j's codes is
// p_tj * sv_j.
//
// One wave takes a page (64 tokens) of one KV head against 16 * QT rows: the
// rows of a sequence's new tokens times the query heads that share the KV
// head.  Scores are computed transposed, S = K Q^T (16 x 16 x 32 MFMA, 16
// tokens by 16 rows), with tile j's row 4g + r holding token 16g + 4j + r:
// lane group g then has the 16 tokens 16g .. 16g+15 of its row, which are the
// weights that the second product, O^T = V^T P, wants of it as its second
// operand, so the weights never leave their lane.  V codes lie dim pair by dim pair, so
// a lane's 16 tokens of a pair are one 16-byte load.
//
// The weights are rounded to fp16 for that product, in both types: 11 bits
// against the 8 that a bf16 output keeps.  p is at most 2^8 (the maximum is
// kept until a row exceeds it by more than 8 powers of two) and sv is taken
// relative to the largest seen by the wave, so the products stay in fp16's
// range whatever V's magnitude.  Statistics and accumulators are fp32.
//
// Where there are few rows the pages of a sequence are split over blocks.
// How many ways is decided on the GPU from the lengths there (they may change
// between replays of a captured graph): every block works out the same plan.
// A block's waves take its pages in turn and are joined through LDS; the
// splits of a sequence leave fp32 partials in the workspace, which a second
// launch joins in split order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qknorm_device.hpp"
#include "qknorm_kv4.hpp"
#include "qknorm_launch.hpp"

namespace qknorm {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;        // powers of two a score may exceed the kept maximum by

template <int DT>
struct AttnElem;
template <>
struct AttnElem<kBF16> {
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  // eight codes to eight values, in order
  static __device__ __forceinline__ u32x4 codes(uint32_t w) {
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.f, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.f, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.f, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.f, 3))};
  }
};
template <>
struct AttnElem<kF16> {
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ u32x4 codes(uint32_t w) {
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, 3))};
  }
};

template <int DT>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (DT == kBF16) {
    const bf16x2 h = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, h);
  } else {
    const f16x2 h = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, h);
  }
}

// Over the four lanes of a row (l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float row_max(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float row_sum(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// ------------------------------------------------------------------ plan --

// A sequence as the kernels see it: its rows [start, start + rows) clamped to
// the T rows there are, its length to the page table's width.
struct Seq {
  uint32_t start, rows, len;
};

__device__ __forceinline__ Seq load_seq(const Kv4AttnK& a, uint32_t b) {
  Seq s;
  int64_t st = b, en = (int64_t)b + 1;
  if (a.starts != nullptr) {
    st = a.starts[b];
    en = a.starts[b + 1];
  }
  st = st < 0 ? 0 : (st > a.T ? a.T : st);
  en = en < st ? st : (en > a.T ? a.T : en);
  const int64_t most = (int64_t)a.max_pages * kKv4Tokens;
  int64_t n = a.lens[b];
  n = n < 0 ? 0 : (n > most ? most : n);
  s.start = (uint32_t)st;
  s.rows = (uint32_t)(en - st);
  s.len = a.pages > 0 ? (uint32_t)n : 0;
  return s;
}

// Row tiles of a sequence, and the most pages that one of them sees.
__device__ __forceinline__ uint32_t seq_tiles(const Kv4AttnK& a, const Seq& s, uint32_t rt) {
  return (uint32_t)(((uint64_t)s.rows * a.group + rt - 1) / rt);
}
__device__ __forceinline__ uint32_t seq_pages(const Kv4AttnK& a, const Seq& s) {
  uint32_t p = (s.len + kKv4Tokens - 1) / kKv4Tokens;
  if (a.window) {
    const uint64_t w = ((uint64_t)a.window + s.rows) / kKv4Tokens + 2;
    if (w < p) p = (uint32_t)w;
  }
  return p;
}
__device__ __forceinline__ uint32_t seq_splits(uint32_t pages, uint32_t chunk) {
  return pages <= chunk ? 1 : (pages + chunk - 1) / chunk;
}

__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t* red) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

// Fills items[0..B] and slots[0..B] with the running counts of work items
// and of partial slots (items of sequences that are split), and returns the
// pages a split takes.
__device__ __forceinline__ uint32_t make_plan(const Kv4AttnK& a, uint32_t rt, uint32_t* items, uint32_t* slots,
                                              uint32_t* red) {
  const uint32_t tid = threadIdx.x, lane = tid & 63;
  uint64_t mine = 0;
  for (uint32_t b = tid; b < a.B; b += 256) {
    const Seq s = load_seq(a, b);
    mine += (uint64_t)seq_tiles(a, s, rt) * seq_pages(a, s) * a.hkv;
  }
  // the total in units of 256 pages, rounded up per thread, fits 32 bits
  const uint32_t units = block_sum((uint32_t)((mine + 255) / 256), red);
  uint64_t chunk = ((uint64_t)units * 256 + a.target - 1) / a.target;
  if (chunk < a.min_chunk) chunk = a.min_chunk;
  uint32_t base_i = 0, base_s = 0;
  for (uint32_t b0 = 0; b0 < a.B; b0 += 256) {
    const uint32_t b = b0 + tid;
    uint32_t ni = 0, ns = 0;
    if (b < a.B) {
      const Seq s = load_seq(a, b);
      const uint32_t sp = seq_splits(seq_pages(a, s), (uint32_t)chunk);
      ni = seq_tiles(a, s, rt) * a.hkv * sp;
      ns = sp > 1 ? ni : 0;
    }
    uint32_t xi = ni, xs = ns;                       // inclusive scan over the wave
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t ui = __shfl_up(xi, o), us = __shfl_up(xs, o);
      if (lane >= (uint32_t)o) { xi += ui; xs += us; }
    }
    __syncthreads();
    if (lane == 63) { red[tid >> 6] = xi; red[4 + (tid >> 6)] = xs; }
    __syncthreads();
    uint32_t pi = base_i, ps = base_s;
    for (uint32_t w = 0; w < (tid >> 6); ++w) { pi += red[w]; ps += red[4 + w]; }
    if (b < a.B) { items[b] = pi + xi - ni; slots[b] = ps + xs - ns; }
    base_i += red[0] + red[1] + red[2] + red[3];
    base_s += red[4] + red[5] + red[6] + red[7];
  }
  if (tid == 0) { items[a.B] = base_i; slots[a.B] = base_s; }
  __syncthreads();
  return (uint32_t)chunk;
}

// The largest b with items[b] <= i (items[0] = 0 <= i < items[B]).
__device__ __forceinline__ uint32_t find(const uint32_t* items, uint32_t B, uint32_t i) {
  uint32_t lo = 0, hi = B;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (items[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------- main kernel --

// What a wave holds of one page of one head, as loaded.
template <int D>
struct PageRegs {
  static constexpr int KD = D / 32;
  uint32_t k[4][KD];       // tile j: the lane's token, its KD dwords of codes
  u32x4 v[D / 32];         // dim pair 16*jj + l%16: 16 tokens
  u32x4 ks[2], vs[2];      // scales of the lane's 16 tokens
};

template <int D>
__device__ __forceinline__ void load_page(PageRegs<D>& p, const uint8_t* __restrict__ base, uint32_t m, uint32_t g) {
  constexpr int KD = D / 32;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t tok = 16 * (m / 4) + 4 * j + m % 4;
    const uint8_t* q = base + tok * (D / 2) + g * (D / 8);
    if constexpr (KD == 2) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const u32x2 x = *reinterpret_cast<const u32x2*>(q);
      p.k[j][0] = x[0];
      p.k[j][1] = x[1];
    } else {
#pragma unroll
      for (int i = 0; i < KD / 4; ++i) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(q + 16 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) p.k[j][4 * i + e] = x[e];
      }
    }
  }
#pragma unroll
  for (int jj = 0; jj < D / 32; ++jj)
    p.v[jj] = *reinterpret_cast<const u32x4*>(base + 32 * D + (16 * jj + m) * 64 + 16 * g);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    p.ks[i] = *reinterpret_cast<const u32x4*>(base + 64 * D + 32 * g + 16 * i);
    p.vs[i] = *reinterpret_cast<const u32x4*>(base + 64 * D + 128 + 32 * g + 16 * i);
  }
}

// The wave's running state over its pages.
template <int D, int QT>
struct State {
  f32x4 acc[QT][D / 32][2];      // O^T: dim pairs 16*jj + 4g + r, low and high dim
  float m[QT], l[QT];            // of row l%16 (l: this lane's tokens)
  float vref;                    // the largest V scale seen
};

template <int DT, int D, int QT, bool MASKED>
__device__ __forceinline__ void use_page(const PageRegs<D>& p, const u32x4 (&qf)[QT][D / 32], State<D, QT>& st,
                                         float scale2, uint32_t g, uint32_t tok0, const uint32_t (&lo)[QT],
                                         const uint32_t (&hi)[QT]) {
  constexpr int KD = D / 32;
  f32x4 s[QT][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int t = 0; t < QT; ++t) s[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KD; ++i) {
      const u32x4 kf = AttnElem<DT>::codes(p.k[j][i]);
#pragma unroll
      for (int t = 0; t < QT; ++t) s[t][j] = AttnElem<DT>::mfma(kf, qf[t][i], s[t][j]);
    }
  }
  // scales of token 16g + 4j + r: word 2j + r/2 of the lane's eight
  float kc[4][4], vc[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t kw = p.ks[j / 2][2 * (j % 2) + r / 2], vw = p.vs[j / 2][2 * (j % 2) + r / 2];
      kc[j][r] = __uint_as_float(r % 2 ? kw & 0xFFFF0000u : kw << 16) * scale2;
      vc[j][r] = __uint_as_float(r % 2 ? vw & 0xFFFF0000u : vw << 16);
      if constexpr (MASKED) {
        // tokens that no row sees may hold anything
        const uint32_t tok = tok0 + 16 * g + 4 * j + r;
        bool seen = false;
#pragma unroll
        for (int t = 0; t < QT; ++t) seen = seen || (tok >= lo[t] && tok < hi[t]);
        if (!seen) vc[j][r] = 0.f;
      }
    }
  float vmax = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) vmax = __builtin_fmaxf(vmax, vc[j][r]);
  vmax = row_max(vmax);
  if constexpr (MASKED) {
    // rows see different tokens, so the largest scale is taken over the wave
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) vmax = __builtin_fmaxf(vmax, __shfl_xor(vmax, o));
  }
  float top[QT];
  bool grow = false;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    float x = -INFINITY;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float y = s[t][j][r] * kc[j][r];
        if constexpr (MASKED) {
          const uint32_t tok = tok0 + 16 * g + 4 * j + r;
          if (!(tok >= lo[t] && tok < hi[t])) y = -INFINITY;
        }
        s[t][j][r] = y;
        x = __builtin_fmaxf(x, y);
      }
    top[t] = row_max(x);
    grow = grow || top[t] > st.m[t] + kLazy;
  }
  if (__builtin_amdgcn_ballot_w64(grow || vmax > st.vref) != 0) {
    const float vnew = __builtin_fmaxf(vmax, st.vref);
    const float vscale = st.vref / vnew;             // vref starts above zero
    st.vref = vnew;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const float mn = __builtin_fmaxf(st.m[t], top[t]);
      const float f = mn == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(st.m[t] - mn);
      st.m[t] = mn;
      st.l[t] *= f;
      const float fa = f * vscale;
#pragma unroll
      for (int jj = 0; jj < D / 32; ++jj)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r) st.acc[t][jj][h][r] *= fa;
    }
  }
  const float vinv = __builtin_amdgcn_rcpf(st.vref);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) vc[j][r] *= vinv;
  u32x4 w[QT][2];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const float m = st.m[t] == -INFINITY ? 0.f : st.m[t];
    float l = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float p0 = __builtin_amdgcn_exp2f(s[t][2 * u][r] - m), p1 = __builtin_amdgcn_exp2f(s[t][2 * u + 1][r] - m);
        l += p0 + p1;
        float w0 = p0 * vc[2 * u][r], w1 = p1 * vc[2 * u + 1][r];
        if constexpr (MASKED) {
          // a hidden token's scale may be NaN
          if (s[t][2 * u][r] == -INFINITY) w0 = 0.f;
          if (s[t][2 * u + 1][r] == -INFINITY) w1 = 0.f;
        }
        w[t][u][r] = pack16<kF16>(w0, w1);           // tokens 8u + r and 8u + 4 + r of the group
      }
    st.l[t] += l;
  }
#pragma unroll
  for (int jj = 0; jj < D / 32; ++jj)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // low codes of tokens 8u + x and 8u + 4 + x side by side, then the high ones
      const uint32_t a = p.v[jj][2 * u], b = p.v[jj][2 * u + 1];
      const uint32_t dl = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
      const uint32_t dh = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
      const u32x4 vl = AttnElem<kF16>::codes(dl), vh = AttnElem<kF16>::codes(dh);
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        st.acc[t][jj][0] = AttnElem<kF16>::mfma(vl, w[t][u], st.acc[t][jj][0]);
        st.acc[t][jj][1] = AttnElem<kF16>::mfma(vh, w[t][u], st.acc[t][jj][1]);
      }
    }
}

// LDS: the plan's counts (2 * (B + 1)), eight words of reductions, then the
// waves' m and l ([4][RT] each) and one wave's output ([RT][D + 4]).
template <int DT, int D, int QT>
__global__ __launch_bounds__(256) void kv4_attn_kernel(Kv4AttnK a) {
  constexpr uint32_t RT = 16 * QT;
  constexpr int kPitch = D + 4;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  float* const sm = reinterpret_cast<float*>(smem);
  float* const sl = sm + 4 * RT;
  float* const so = sl + 4 * RT;
  uint32_t* const red = reinterpret_cast<uint32_t*>(so + RT * kPitch);
  uint32_t* const items = red + 8;
  uint32_t* const slots = items + a.B + 1;
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const uint32_t m16 = lane % 16, g = lane / 16;

  const uint32_t chunk = make_plan(a, RT, items, slots, red);
  if (blockIdx.x == 0) {                              // for the launch that joins the splits
    for (uint32_t b = tid; b <= a.B; b += 256) a.plan[1 + b] = slots[b];
    if (tid == 0) a.plan[0] = chunk;
  }
  const uint32_t total = items[a.B];
  for (uint32_t item = blockIdx.x; item < total; item += gridDim.x) {
    const uint32_t b = uniform(find(items, a.B, item));
    const Seq sq = load_seq(a, b);
    const uint32_t tiles = seq_tiles(a, sq, RT), splits = seq_splits(seq_pages(a, sq), chunk);
    const uint32_t in = item - items[b];
    const uint32_t tile = in % tiles, head = in / tiles % a.hkv, split = in / (tiles * a.hkv);
    const uint32_t nrows = sq.rows * a.group;
    const uint32_t r0 = tile * RT, r1 = r0 + RT < nrows ? r0 + RT : nrows;
    if (r0 >= nrows) continue;                        // (row offsets out of order)
    // the tokens that row r of the tile sees: [lo, hi)
    const uint32_t L = sq.len, n = sq.rows;
    auto row_hi = [&](uint32_t r) {
      const int64_t h = (int64_t)L - n + r / a.group + 1;
      return (uint32_t)(h < 0 ? 0 : h);
    };
    auto row_lo = [&](uint32_t hi) { return a.window && hi > a.window ? hi - a.window : 0u; };
    const uint32_t hi_first = row_hi(r0), hi_last = row_hi(r1 - 1);
    const uint32_t lo_first = row_lo(hi_first), lo_last = row_lo(hi_last);
    uint32_t p0 = lo_first / kKv4Tokens, p1 = (hi_last + kKv4Tokens - 1) / kKv4Tokens;
    const uint32_t per = (p1 - p0 + splits - 1) / splits;
    p0 = p0 + split * per;
    p1 = p0 + per < p1 ? p0 + per : p1;

    u32x4 qf[QT][D / 32];
    uint32_t lo[QT], hi[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      uint32_t r = r0 + t * 16 + m16;
      r = r < r1 ? r : r1 - 1;                        // rows past the end repeat the last and are not stored
      const uint8_t* q = a.q + (uint64_t)(sq.start + r / a.group) * a.ldq_bytes +
                         ((uint64_t)head * a.group + r % a.group) * D * 2 + g * (D / 4) * 2;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) qf[t][i] = load16(q + 16 * i);
      hi[t] = row_hi(r);
      lo[t] = row_lo(hi[t]);
    }

    State<D, QT> st;
    st.vref = 0x1p-126f;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      st.m[t] = -INFINITY;
      st.l[t] = 0.f;
#pragma unroll
      for (int jj = 0; jj < D / 32; ++jj) st.acc[t][jj][0] = st.acc[t][jj][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const int32_t* const table = a.table + (uint64_t)b * a.table_stride;
    const uint64_t head_off = (uint64_t)head * kv4_head_bytes(D);
    for (uint32_t pg = p0 + wave; pg < p1; pg += 4) {
      const int32_t id = (int32_t)uniform((uint32_t)table[pg]);
      if (id < 0 || id >= a.pages) continue;          // a page that is not there hides its tokens
      PageRegs<D> p;
      load_page<D>(p, a.cache + (uint64_t)id * a.page_stride + head_off, m16, g);
      const uint32_t tok0 = pg * kKv4Tokens;
      if (tok0 >= lo_last && tok0 + kKv4Tokens <= hi_first)
        use_page<DT, D, QT, false>(p, qf, st, a.scale2, g, tok0, lo, hi);
      else
        use_page<DT, D, QT, true>(p, qf, st, a.scale2, g, tok0, lo, hi);
    }

    // join the four waves
    __syncthreads();
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const float l = row_sum(st.l[t]);
      if (g == 0) {
        sm[wave * RT + t * 16 + m16] = st.m[t];
        sl[wave * RT + t * 16 + m16] = l;
      }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) M = __builtin_fmaxf(M, sm[w * RT + t * 16 + m16]);
      const float f = st.m[t] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(st.m[t] - M) * st.vref;
#pragma unroll
      for (int jj = 0; jj < D / 32; ++jj)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r) st.acc[t][jj][h][r] *= f;
    }
    for (uint32_t w = 0; w < 4; ++w) {                // in wave order
      if (wave == w) {
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
          for (int jj = 0; jj < D / 32; ++jj)
#pragma unroll
            for (int r = 0; r < 4; r += 2) {
              float* o = so + (t * 16 + m16) * kPitch + 32 * jj + 8 * g + 2 * r;
              f32x4 x = {st.acc[t][jj][0][r], st.acc[t][jj][1][r], st.acc[t][jj][0][r + 1], st.acc[t][jj][1][r + 1]};
              if (w != 0) x += *reinterpret_cast<const f32x4*>(o);
              *reinterpret_cast<f32x4*>(o) = x;
            }
      }
      __syncthreads();
    }
    // RT rows, D / 8 threads a row
    const bool whole = splits == 1;
    const uint32_t slot = slots[b] + in;
    for (uint32_t i = tid; i < RT * (D / 8); i += 256) {
      const uint32_t rr = i / (D / 8), c = i % (D / 8) * 8, r = r0 + rr;
      if (r >= r1) continue;
      float M = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) M = __builtin_fmaxf(M, sm[w * RT + rr]);
      const float mm = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < 4; ++w) l += sl[w * RT + rr] * __builtin_amdgcn_exp2f(sm[w * RT + rr] - mm);
      const f32x4 x0 = *reinterpret_cast<const f32x4*>(so + rr * kPitch + c);
      const f32x4 x1 = *reinterpret_cast<const f32x4*>(so + rr * kPitch + c + 4);
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const uint64_t row = sq.start + r / a.group;
        const uint32_t hd = head * a.group + r % a.group;
        const u32x4 o = {pack16<DT>(x0[0] * inv, x0[1] * inv), pack16<DT>(x0[2] * inv, x0[3] * inv),
                         pack16<DT>(x1[0] * inv, x1[1] * inv), pack16<DT>(x1[2] * inv, x1[3] * inv)};
        *reinterpret_cast<u32x4*>(a.out + row * a.ldo_bytes + ((uint64_t)hd * D + c) * 2) = o;
        if (c == 0 && a.lse) a.lse[row * a.hq + hd] = l == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(l)) * kLn2;
      } else if (slot < a.max_slots) {                // (always, for row offsets in order)
        float* o = a.part + ((uint64_t)slot * RT + rr) * D + c;
        *reinterpret_cast<f32x4*>(o) = x0;
        *reinterpret_cast<f32x4*>(o + 4) = x1;
        if (c == 0) {
          a.stat[((uint64_t)slot * RT + rr) * 2] = M;
          a.stat[((uint64_t)slot * RT + rr) * 2 + 1] = l;
        }
      }
    }
    __syncthreads();
  }
}

// Joins the splits: one group of D / 4 threads per row and head, the
// partials in split order.  Rows whose sequence was not split are done.
template <int DT, int D, int QT>
__global__ __launch_bounds__(256) void kv4_attn_join_kernel(Kv4AttnK a) {
  constexpr uint32_t RT = 16 * QT, TP = D / 4, kRows = 256 / TP;
  const uint32_t tid = threadIdx.x, c = tid % TP * 4;
  const uint64_t id = (uint64_t)blockIdx.x * kRows + tid / TP;
  const uint64_t row = id / a.hq;
  const uint32_t hd = (uint32_t)(id % a.hq);
  if (row >= (uint64_t)a.T) return;
  uint32_t b = (uint32_t)row;
  if (a.starts != nullptr) {
    // the last sequence that starts at or before the row
    uint32_t lo = 0, hi = a.B;
    if ((int64_t)a.starts[0] > (int64_t)row) return;
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) / 2;
      if ((int64_t)a.starts[mid] <= (int64_t)row) lo = mid; else hi = mid;
    }
    b = lo;
  }
  if (b >= a.B) return;
  const Seq sq = load_seq(a, b);
  if (row < sq.start || row >= (uint64_t)sq.start + sq.rows) return;
  const uint32_t chunk = a.plan[0], slot0 = a.plan[1 + b];
  const uint32_t splits = seq_splits(seq_pages(a, sq), chunk);
  if (splits == 1) return;
  const uint32_t tiles = seq_tiles(a, sq, RT);
  const uint32_t head = hd / a.group, r = ((uint32_t)row - sq.start) * a.group + hd % a.group;
  const uint32_t step = tiles * a.hkv;
  const uint64_t first = slot0 + (uint64_t)head * tiles + r / RT;
  if (first + (uint64_t)(splits - 1) * step >= a.max_slots) return;
  float M = -INFINITY;
  for (uint32_t s = 0; s < splits; ++s) M = __builtin_fmaxf(M, a.stat[((first + (uint64_t)s * step) * RT + r % RT) * 2]);
  const float mm = M == -INFINITY ? 0.f : M;
  float l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  for (uint32_t s = 0; s < splits; ++s) {
    const uint64_t at = (first + (uint64_t)s * step) * RT + r % RT;
    const float f = __builtin_amdgcn_exp2f(a.stat[at * 2] - mm);
    l += a.stat[at * 2 + 1] * f;
    o += *reinterpret_cast<const f32x4*>(a.part + at * D + c) * f;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 v = {pack16<DT>(o[0] * inv, o[1] * inv), pack16<DT>(o[2] * inv, o[3] * inv)};
  *reinterpret_cast<u32x2*>(a.out + row * a.ldo_bytes + ((uint64_t)hd * D + c) * 2) = v;
  if (c == 0 && a.lse) a.lse[row * a.hq + hd] = l == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(l)) * kLn2;
}

// ------------------------------------------------------------------- host --

// Blocks of the launch, and the work items that the plan aims at.
constexpr uint32_t kBlocks = 512, kTarget = 1024;
constexpr uint32_t kMinChunk = 4;                     // pages: one a wave

// 16-row tiles a wave: as many as an average sequence fills, up to two.
int row_tiles(int64_t T, int64_t B, int64_t group) {
  const int64_t rows = B > 0 ? (T * group + B - 1) / B : 0;
  return rows <= 16 ? 1 : 2;
}

// No more slots than this hold partials: items of a split sequence take at
// least half a chunk each, and a chunk is at least 1 / kTarget of the work.
int64_t most_slots(int64_t T, int64_t B, int64_t max_pages, int64_t hkv, int64_t group, int qt) {
  const int64_t rt = 16 * qt;
  // row tiles of all sequences, at most; each at most max_pages chunks of one
  const __int128 tiles = ((__int128)T * group) / rt + (B < T ? B : T);
  const __int128 all = tiles * hkv * (max_pages / kMinChunk + 1);
  const int64_t cap = 2 * kTarget;
  return all < cap ? (int64_t)all : cap;
}

int64_t plan_bytes(int64_t B) { return ((B + 2) * 4 + 255) & ~(int64_t)255; }

template <int DT, int D, int QT>
hipError_t launch(const Kv4AttnK& k, hipStream_t s) {
  constexpr uint32_t RT = 16 * QT;
  const int lds = (int)((8 * RT + RT * (D + 4) + 8 + 2 * (k.B + 1)) * 4);
  auto kern = kv4_attn_kernel<DT, D, QT>;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(kBlocks), dim3(256), lds, s, k);
  e = hipGetLastError();
  if (e != hipSuccess || k.max_pages <= (int64_t)kMinChunk) return e;      // (nothing can be split)
  constexpr uint32_t kRows = 256 / (D / 4);
  const uint64_t blocks = ((uint64_t)k.T * k.hq + kRows - 1) / kRows;
  hipLaunchKernelGGL((kv4_attn_join_kernel<DT, D, QT>), dim3((uint32_t)blocks), dim3(256), 0, s, k);
  return hipGetLastError();
}

template <int DT, int D>
hipError_t launch_qt(const Kv4AttnK& k, int qt, hipStream_t s) {
  return qt == 1 ? launch<DT, D, 1>(k, s) : launch<DT, D, 2>(k, s);
}

}  // namespace

int64_t kv4_attn_workspace_bytes(int64_t T, int64_t B, int64_t max_pages, int32_t hq, int32_t hkv, int32_t head_dim) {
  if (T <= 0 || B <= 0 || hq == 0) return 0;
  const int64_t group = hq / hkv;
  const int qt = row_tiles(T, B, group);
  const int64_t rows = most_slots(T, B, max_pages, hkv, group, qt) * 16 * qt;
  return plan_bytes(B) + rows * 8 + rows * head_dim * 4;
}

hipError_t launch_kv4_attn(const Kv4AttnArgs& a, hipStream_t s) {
  Kv4AttnK k;
  const int64_t group = a.hq / a.hkv;
  const int qt = row_tiles(a.T, a.B, group);
  const int64_t rows = most_slots(a.T, a.B, a.max_pages, a.hkv, group, qt) * 16 * qt;
  k.q = (const uint8_t*)a.q;
  k.ldq_bytes = (uint64_t)a.ldq * 2;
  k.cache = (const uint8_t*)a.cache;
  k.pages = a.pages;
  k.page_stride = (uint64_t)a.page_stride;
  k.table = a.table;
  k.table_stride = (uint64_t)a.table_stride;
  k.max_pages = (uint32_t)a.max_pages;
  k.lens = a.lens;
  k.starts = a.starts;
  k.out = (uint8_t*)a.out;
  k.ldo_bytes = (uint64_t)a.ldo * 2;
  k.lse = a.lse;
  k.T = a.T;
  k.B = (uint32_t)a.B;
  k.hq = (uint32_t)a.hq;
  k.hkv = (uint32_t)a.hkv;
  k.group = (uint32_t)group;
  k.window = (uint32_t)a.window;
  k.scale2 = a.scale * kLog2e;
  k.target = kTarget;
  k.min_chunk = kMinChunk;
  k.max_slots = (uint32_t)(rows / (16 * qt));
  uint8_t* w = static_cast<uint8_t*>(a.workspace);
  k.plan = reinterpret_cast<uint32_t*>(w);
  k.stat = reinterpret_cast<float*>(w + plan_bytes(a.B));
  k.part = reinterpret_cast<float*>(w + plan_bytes(a.B) + rows * 8);
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    return a.dtype == kF16 ? launch_qt<kF16, D>(k, qt, s) : launch_qt<kBF16, D>(k, qt, s);
  };
  if (a.head_dim == 64) return pick(IntC<64>{});
  if (a.head_dim == 128) return pick(IntC<128>{});
  return pick(IntC<256>{});
}

}  // namespace qknorm
