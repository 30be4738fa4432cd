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
// operand, so the weights never leave their lane.  V codes lie dim pair by dim
// pair, so a lane's 16 tokens of a pair are one 16-byte load.
//
// The weights are rounded to fp16 for that product, in both types: 11 bits
// against the 8 that a bf16 output keeps.  They stay in fp16's range whatever
// V's magnitude (struct State).  The maximum is kept until a row exceeds it by
// more than 8 powers of two.  Statistics and accumulators are fp32.
//
// Work is counted in page visits: one page of one head for one tile of rows,
// and a few more for each tile and head (a unit), for starting and ending it.
// The plan is made on the GPU from the lengths there (they may change between
// replays of a captured graph), the same by every block.
// Where there are few units, all visits laid end to end are cut into equal
// runs, one a wave, whatever sequences and heads they fall in: a wave
// then takes the end of one unit's pages, some whole units, and the start of
// another's, so that it leaves at most two partial results, in the workspace,
// which a second launch joins in page order.  Where there are many, each is one
// wave's.  Waves share nothing but the plan.  Short sequences and most prompts
// take a block a unit instead, whose waves share its pages and join in LDS, in
// one launch (block_waves).
// Not kept: runs cut by the pages that each causal tile really sees, instead of
// taking a sequence's tiles as alike (202 us against 181 for four chunks of 512
// rows over 4096 tokens, since fewer cuts then fall on a unit's end); a block
// converting each page into LDS once for 128 rows (182 us against 176); pages of one row tile through LDS, K two
// ahead (102.7 against 102.9 us for four sequences of 131071 tokens, 33.0
// against 31.6 for a ragged batch of 64).
//
// What bounds it.  One row tile a sequence: memory.  Four sequences of 131071
// tokens and 8 KV heads, 554 MB, take 91 us in this kernel, 6.1 TB/s, and 5 less
// with the softmax and the scores left out.  64 sequences of 1024 tokens, 71 MB:
// 19 us, of which the plan and the first loads take 5.  Two row tiles: vector
// instructions, issued in about 70 % of the time (some 500 a page of 32 rows,
// beside 64 matrix products that take 30 %): four prompts' 512 rows each over
// 4096 tokens 171 us in runs with their join, 161 in blocks, 800 TFLOP/s.
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
constexpr int kLazyV = 4;           // and a V scale the kept exponent
constexpr float kNoScore = -1e30f;  // a partial result's maximum if it has no visible score

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

// The larger of two numbers that are no NaN, as the middle one of three with
// infinity: one instruction, where fmaxf makes operands quiet first if it cannot
// see where they come from.  (An infinity that the compiler knows, it would
// turn back into fmaxf: four prompts' 512 rows each 172 against 170 us.)
__device__ __forceinline__ float max_of(uint32_t a, uint32_t b) {
  uint32_t top = 0x7F800000u;
  asm("" : "+s"(top));
  return __builtin_amdgcn_fmed3f(__uint_as_float(a), __uint_as_float(b), __uint_as_float(top));
}
// Over the four lanes of a row (l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float row_max(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = max_of(r[0], r[1]);
  auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return max_of(q[0], q[1]);
}
__device__ __forceinline__ float row_sum(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// The kernel's arguments, read again from where the launch put them.  The
// kernels have many, and what is read before a loop is kept through it: read
// this way where they are needed, they do not take the loop's scalar registers.
__device__ __forceinline__ Kv4AttnK launch_args() {
  typedef const __attribute__((address_space(4))) Kv4AttnK* Ptr;
  Ptr p = (Ptr)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const Kv4AttnK*)p;
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
    // (a tile's own rows span at most the sequence's)
    const uint64_t w = ((uint64_t)a.window + s.rows) / kKv4Tokens + 2;
    if (w < p) p = (uint32_t)w;
  }
  return p > 0 ? p : 1;                               // (a tile that sees nothing still gives zeros)
}
// Fills visits[0..B] and units[0..B] with the running counts of page visits
// and of units (a row tile of one head).
__device__ __forceinline__ void make_plan(const Kv4AttnK& a, uint32_t rt, uint32_t* visits, uint32_t* units,
                                          uint32_t* red) {
  const uint32_t tid = threadIdx.x, lane = tid & 63;
  uint32_t base_v = 0, base_u = 0;
  for (uint32_t b0 = 0; b0 < a.B; b0 += 256) {
    const uint32_t b = b0 + tid;
    uint32_t nv = 0, nu = 0;
    if (b < a.B) {
      const Seq s = load_seq(a, b);
      nu = seq_tiles(a, s, rt) * a.hkv;
      nv = nu * (seq_pages(a, s) + a.unit_cost);
    }
    uint32_t xv = nv, xu = nu;                       // inclusive scan over the wave
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t uv = __shfl_up(xv, o), uu = __shfl_up(xu, o);
      if (lane >= (uint32_t)o) { xv += uv; xu += uu; }
    }
    if (b0 != 0) __syncthreads();
    if (lane == 63) { red[tid >> 6] = xv; red[4 + (tid >> 6)] = xu; }
    __syncthreads();
    uint32_t pv = base_v, pu = base_u;
    for (uint32_t w = 0; w < (tid >> 6); ++w) { pv += red[w]; pu += red[4 + w]; }
    if (b < a.B) { visits[b] = pv + xv - nv; units[b] = pu + xu - nu; }
    base_v += red[0] + red[1] + red[2] + red[3];
    base_u += red[4] + red[5] + red[6] + red[7];
  }
  if (tid == 0) { visits[a.B] = base_v; units[a.B] = base_u; }
  __syncthreads();
}

// Page visits a wave takes, or 0 where each unit is one wave's: where there
// are two units a wave or more.  At least two, and one where the work is
// single row tiles over up to 40 visits each: then a wave a page and the more
// partials to join are still faster (a sequence of 1000 tokens 9.3 against 9.9
// us; of 8192 tokens 15.5 against 13.7, before the join took eight at a time).
__device__ __forceinline__ uint32_t run_length(const Kv4AttnK& a, uint32_t rt, uint32_t visits, uint32_t units) {
  if (units >= 2 * a.workers) return 0;
  const uint32_t per = visits / a.workers + (visits % a.workers != 0);
  const uint32_t least = rt == 16 && visits <= 40 * units ? 1 : 2;
  return per > least ? per : least;
}

// The largest b with count[b] <= i (count[0] = 0 <= i < count[B]).
__device__ __forceinline__ uint32_t find(const uint32_t* count, uint32_t B, uint32_t i) {
  uint32_t lo = 0, hi = B;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (count[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// ----------------------------------------------------------------- softmax --

// A wave's running state over its pages.  With m a row's kept maximum (in
// powers of two) and 2^e the size of the V scales, weights are taken relative to
// 2^M, M = m + e: the exponential then makes what the second product wants,
// exp2(s - M) * sv, of order one whatever V's magnitude, in fp16's range.
// l sums exp2(s - M).  Scores are taken relative to M as they are made (one
// multiply-add with the K scale), so that the exponential's argument costs
// nothing more unless M changes.  e stays within +-60, where no fp32 sum can leave its
// range; V scales beyond that are multiplied by 2^-rem.
template <int D, int QT>
struct State {
  f32x4 acc[QT][D / 32][2];      // O^T: dim pairs 16*jj + 4g + r, low and high dim
  float M[QT], l[QT];            // of row l%16 (l: this lane's tokens)
  float least[QT];               // 0, or -infinity (and M 0) before the row's first visible score
  int size;                      // e + rem (wave-uniform)
};

__device__ __forceinline__ int kept_exponent(int size) { return size < -60 ? -60 : (size > 60 ? 60 : size); }
__device__ __forceinline__ float power_of_two(int e) { return __builtin_amdgcn_ldexpf(1.f, e); }

template <int D, int QT>
__device__ __forceinline__ void clear(State<D, QT>& st) {
  st.size = -200;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    st.M[t] = st.l[t] = 0.f;
    st.least[t] = -INFINITY;
#pragma unroll
    for (int jj = 0; jj < D / 32; ++jj) st.acc[t][jj][0] = st.acc[t][jj][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
}

// A page's part in the running maximum and sum, from its scores s relative to
// M (tile j's row 4g + r: token 16g + 4j + r of the page, which begins at token tok0) and
// its V scales vc, and its weights w for the second product (tokens 8u + r and
// 8u + 4 + r of the lane's group).  `full`: every row sees all of the page;
// else what a row [lo, hi) does not see is taken out, whatever it holds.
template <int D, int QT>
__device__ __forceinline__ void weigh(f32x4 (&s)[QT][4], float (&vc)[4][4], State<D, QT>& st, bool full, uint32_t g,
                                      uint32_t tok0, const uint32_t (&lo)[QT], const uint32_t (&hi)[QT],
                                      u32x4 (&w)[QT][2]) {
  // bit 4j + r of a row's mask: whether it sees the lane's token 4j + r.  As
  // bits the 32 answers take two registers, not 32 pairs of scalar ones.
  uint32_t sees[QT] = {};
  auto keep = [](uint32_t mask, int k) { return (uint32_t)__builtin_amdgcn_sbfe((int)mask, k, 1); };   // all ones or none
  if (!full) {
    uint32_t any = 0;
    const int first = (int)(tok0 + 16 * g);
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const int a = (int)lo[t] - first, b = (int)hi[t] - first;
      const uint32_t below = (1u << (a < 0 ? 0 : (a > 16 ? 16 : a))) - 1, until = (1u << (b < 0 ? 0 : (b > 16 ? 16 : b))) - 1;
      sees[t] = until & ~below;
      any |= sees[t];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          const uint32_t k = keep(sees[t], 4 * j + r);
          s[t][j][r] = __uint_as_float((__float_as_uint(s[t][j][r]) & k) | (0xFF800000u & ~k));
        }
        vc[j][r] = __uint_as_float(__float_as_uint(vc[j][r]) & keep(any, 4 * j + r));
      }
  }
  float vmax = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) vmax = __builtin_fmaxf(vmax, vc[j][r]);
  vmax = row_max(vmax);
  if (!full) {
    // rows see different tokens, so the largest scale is taken over the wave
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) vmax = __builtin_fmaxf(vmax, __shfl_xor(vmax, o));
  }
  const uint32_t vbits = uniform(__float_as_uint(vmax));
  const int vsize = vbits == 0 ? -200 : (int)(vbits >> 23) - 126;      // vmax < 2^vsize
  const float e = (float)kept_exponent(st.size);
  float top[QT];
  bool grow = false;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    float x = -INFINITY;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) x = __builtin_fmaxf(x, s[t][j][r]);
    top[t] = row_max(x);
    grow = grow || top[t] + e > st.least[t] + kLazy;
  }
  if (vsize > st.size + kLazyV || __builtin_amdgcn_ballot_w64(grow) != 0) {
    const int size = vsize > st.size ? vsize : st.size, en = kept_exponent(size);
    const float back = power_of_two((st.size - kept_exponent(st.size)) - (size - en));
    st.size = size;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      // the new M less the old one; a row without a visible score keeps 0
      const float to = __builtin_fmaxf(st.least[t] - e, top[t]) + (float)en;
      const float by = to == -INFINITY ? 0.f : to;
      // (a row's first: nothing to scale, and 2^-by may be beyond fp32)
      const float f = __builtin_fminf(__builtin_amdgcn_exp2f(-by), 1.f), fa = f * back;
      if (top[t] > -INFINITY) st.least[t] = 0.f;
      st.M[t] += by;
      st.l[t] *= f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[t][j][r] -= by;
#pragma unroll
      for (int jj = 0; jj < D / 32; ++jj)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r) st.acc[t][jj][h][r] *= fa;
    }
  }
  if (st.size != kept_exponent(st.size)) {
    const float f = power_of_two(kept_exponent(st.size) - st.size);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) vc[j][r] *= f;
  }
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    float l = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = __builtin_amdgcn_exp2f(s[t][j][r]);
        l += x;
        s[t][j][r] = x * vc[j][r];
      }
    st.l[t] += l;
  }
  if (!full) {
    // (a hidden token's scale may be NaN)
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[t][j][r] = __uint_as_float(__float_as_uint(s[t][j][r]) & keep(sees[t], 4 * j + r));
  }
#pragma unroll
  for (int t = 0; t < QT; ++t)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) w[t][u][r] = pack16<kF16>(s[t][2 * u][r], s[t][2 * u + 1][r]);
}

// The tokens that row r (new token r / group of n, whose last is the cache's
// token L - 1) sees: [row_lo, row_hi).
__device__ __forceinline__ uint32_t row_hi(const Kv4AttnK& a, const Seq& sq, uint32_t r) {
  const int64_t h = (int64_t)sq.len - sq.rows + r / a.group + 1;
  return (uint32_t)(h < 0 ? 0 : h);
}
__device__ __forceinline__ uint32_t row_lo(const Kv4AttnK& a, uint32_t hi) {
  return a.window && hi > a.window ? hi - a.window : 0u;
}

// The end of a unit for one wave: rows first .. first + 16*QT - 1 (those
// before `last`), which are rows `at` and on of the tile; to the output where
// the unit is whole, else to the slot's RT rows.  (No store has a scalar
// offset: after a 16-byte store with one, the compiler lets the next
// instruction overwrite the stored registers, and gfx950 then stored the new
// values of the last lanes.)
template <int DT, int D, int QT, int RT>
__device__ __forceinline__ void store_rows(const Seq& sq, State<D, QT>& st, uint32_t head, uint32_t first,
                                           uint32_t last, uint32_t at, bool whole, uint32_t slot) {
  const Kv4AttnK a = launch_args();
  const uint32_t lane = threadIdx.x & 63, m16 = lane % 16, g = lane / 16;
  // (offsets from the wave's first row: below 2^31, rows being 32 MiB apart at most)
  const Rsrc ro = make_rsrc(a.out + (uint64_t)(sq.start + first / a.group) * a.ldo_bytes, 0xFFFFFFFFu);
  const Rsrc rp = make_rsrc(a.part + ((uint64_t)slot * RT + at) * D, 16 * QT * D * 4);
  const float back = power_of_two(st.size - kept_exponent(st.size));
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const uint32_t r = first + t * 16 + m16;
    const float l = row_sum(st.l[t]);
    if (r >= last) continue;
    const float f = whole ? (l == 0.f ? 0.f : back / l) : back;
    const uint32_t hd = head * a.group + r % a.group;
    const uint32_t ro_at = (r / a.group - first / a.group) * (uint32_t)a.ldo_bytes + hd * D * 2;
#pragma unroll
    for (int jj = 0; jj < D / 32; ++jj) {
      // dims 32*jj + 8g .. + 7
      const f32x4 (&o)[2] = st.acc[t][jj];
      if (whole) {
        const u32x4 v = {pack16<DT>(o[0][0] * f, o[1][0] * f), pack16<DT>(o[0][1] * f, o[1][1] * f),
                         pack16<DT>(o[0][2] * f, o[1][2] * f), pack16<DT>(o[0][3] * f, o[1][3] * f)};
        __builtin_amdgcn_raw_buffer_store_b128(v, ro, ro_at + g * 16 + jj * 64, 0, 0);
      } else {
        const f32x4 x = f32x4{o[0][0], o[1][0], o[0][1], o[1][1]} * f, y = f32x4{o[0][2], o[1][2], o[0][3], o[1][3]} * f;
        const uint32_t to = m16 * D * 4 + g * 32 + t * 16 * D * 4 + jj * 128;
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), rp, to, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), rp, to + 16, 0, 0);
      }
    }
    if (g == 0) {
      if (!whole) {
        const uint64_t i = (uint64_t)slot * RT + at + t * 16 + m16;
        a.stat[i * 2] = st.least[t] == 0.f ? st.M[t] : kNoScore;
        a.stat[i * 2 + 1] = l;
      } else if (a.lse) {
        a.lse[(uint64_t)(sq.start + r / a.group) * a.hq + hd] = l == 0.f ? -INFINITY : (st.M[t] + __builtin_amdgcn_logf(l)) * kLn2;
      }
    }
  }
}

// The end of a unit for the W waves of a block: their maxima and sums, then
// their values 64 dims at a time, through LDS (kJoinBytes); the sums over the
// waves in their order.
constexpr int kJoinPitch = 68;                        // floats a row of 64 dims
template <int QT, int W>
constexpr int kJoinBytes = (W * 16 * QT * (2 + kJoinPitch) + 16 * QT) * 4;

template <int DT, int D, int QT, int W>
__device__ __forceinline__ void join_waves(const Seq& sq, State<D, QT>& st, uint32_t head, uint32_t first,
                                           uint32_t last, float* smem) {
  constexpr uint32_t R = 16 * QT;
  const Kv4AttnK a = launch_args();
  const uint32_t tid = threadIdx.x, lane = tid & 63, m16 = lane % 16, g = lane / 16, wave = uniform(tid >> 6);
  float* const sm = smem;
  float* const sl = sm + W * R;
  float* const sinv = sl + W * R;
  float* const so = sinv + R;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const float l = row_sum(st.l[t]);
    if (g == 0) {
      sm[wave * R + t * 16 + m16] = st.least[t] == 0.f ? st.M[t] : kNoScore;
      sl[wave * R + t * 16 + m16] = l;
    }
  }
  __syncthreads();
  const float back = power_of_two(st.size - kept_exponent(st.size));
  float f[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    float top = sm[t * 16 + m16], l = 0.f;
#pragma unroll
    for (int w = 1; w < W; ++w) top = __builtin_fmaxf(top, sm[w * R + t * 16 + m16]);
#pragma unroll
    for (int w = 0; w < W; ++w) l += sl[w * R + t * 16 + m16] * __builtin_amdgcn_exp2f(sm[w * R + t * 16 + m16] - top);
    f[t] = back * __builtin_amdgcn_exp2f((st.least[t] == 0.f ? st.M[t] : kNoScore) - top);
    const uint32_t r = first + t * 16 + m16;
    if (wave == 0 && g == 0) {
      sinv[t * 16 + m16] = l == 0.f ? 0.f : 1.f / l;
      if (a.lse && r < last)
        a.lse[(uint64_t)(sq.start + r / a.group) * a.hq + head * a.group + r % a.group] =
            l == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(l)) * kLn2;
    }
  }
#pragma unroll
  for (int h = 0; h < D / 64; ++h) {
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // dims 32*jj + 8g .. + 7
        const f32x4 (&o)[2] = st.acc[t][2 * h + i];
        float* to = so + (wave * R + t * 16 + m16) * kJoinPitch + 32 * i + 8 * g;
        *reinterpret_cast<f32x4*>(to) = f32x4{o[0][0], o[1][0], o[0][1], o[1][1]} * f[t];
        *reinterpret_cast<f32x4*>(to + 4) = f32x4{o[0][2], o[1][2], o[0][3], o[1][3]} * f[t];
      }
    __syncthreads();
#pragma unroll
    for (uint32_t i = tid; i < R * 32; i += 64 * W) {
      const uint32_t m = i / 32, r = first + m, d = 2 * (i % 32);
      if (r >= last) continue;
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        x += so[(w * R + m) * kJoinPitch + d];
        y += so[(w * R + m) * kJoinPitch + d + 1];
      }
      const float inv = sinv[m];
      *reinterpret_cast<uint32_t*>(a.out + (uint64_t)(sq.start + r / a.group) * a.ldo_bytes +
                                   ((uint64_t)(head * a.group + r % a.group) * D + 64 * h + d) * 2) =
          pack16<DT>(x * inv, y * inv);
    }
    __syncthreads();
  }
}

// A sequence's page numbers, read with scalar loads (uniform addresses): as
// vector loads, which return in order, the wait for a number would be a wait
// for every page in flight.
typedef const __attribute__((address_space(4))) int32_t* PageTable;
__device__ __forceinline__ PageTable page_table(const Kv4AttnK& a, uint32_t b) {
  const uint64_t at = (uint64_t)(a.table + (uint64_t)b * a.table_stride);
  return (PageTable)(((uint64_t)uniform((uint32_t)(at >> 32)) << 32) | uniform((uint32_t)at));
}

// The Q rows of a wave as the products' second operands, and the tokens that
// each sees.
template <int D, int QT>
__device__ __forceinline__ void load_q(const Kv4AttnK& a, const Seq& sq, uint32_t head, uint32_t first, uint32_t last,
                                       u32x4 (&qf)[QT][D / 32], uint32_t (&lo)[QT], uint32_t (&hi)[QT]) {
  const uint32_t lane = threadIdx.x & 63, m16 = lane % 16, g = lane / 16;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    uint32_t r = first + t * 16 + m16;
    r = r < last ? r : last - 1;                      // rows past the end repeat the last and are not stored
    const uint8_t* q = a.q + (uint64_t)(sq.start + r / a.group) * a.ldq_bytes +
                       ((uint64_t)head * a.group + r % a.group) * D * 2 + g * (D / 4) * 2;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) qf[t][i] = load16(q + 16 * i);
    hi[t] = row_hi(a, sq, r);
    lo[t] = row_lo(a, hi[t]);
  }
}

// Inclusive sum over the wave's lanes (row shifts, then the row totals passed on).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t scan_step(uint32_t v) {
  return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v = scan_step<0x111, 0xF>(v);                       // row_shr 1, 2, 4, 8
  v = scan_step<0x112, 0xF>(v);
  v = scan_step<0x114, 0xF>(v);
  v = scan_step<0x118, 0xF>(v);
  v = scan_step<0x142, 0xA>(v);                       // row_bcast 15 into rows 1 and 3
  return scan_step<0x143, 0xC>(v);                    // row_bcast 31 into rows 2 and 3
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, uint32_t lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, (int)lane);
}

// Calls f(sequence, its number, row tile, head, first page, pages, whole,
// slot) for every piece of work of one wave out of a.workers, rt rows a tile;
// `smem` holds 8 words and the plan's counts.  Block 0 leaves the plan for the
// launch that joins.  UNITS: whole units, one after another (a worker is a
// block then, and every wave of it makes the same calls).
template <bool UNITS, class F>
__device__ __forceinline__ void walk(uint32_t rt, uint32_t worker, uint32_t* smem, F f) {
  const Kv4AttnK a = launch_args();
  uint32_t* const red = smem;
  uint32_t* const visits = red + 8;
  uint32_t* const units = visits + a.B + 1;
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  // up to 64 sequences each wave keeps the plan in its lanes, else the block keeps it in LDS
  const bool in_lanes = a.B <= 64;
  Seq mine = {0, 0, 0};
  uint32_t my_visits = 0, my_units = 0, all_visits, all_units;      // (counts before the lane's sequence)
  if (in_lanes) {
    uint32_t nu = 0, nv = 0;
    if (lane < a.B) {
      mine = load_seq(a, lane);
      nu = seq_tiles(a, mine, rt) * a.hkv;
      nv = nu * (seq_pages(a, mine) + a.unit_cost);
    }
    const uint32_t xv = wave_scan(nv), xu = wave_scan(nu);
    my_visits = lane < a.B ? xv - nv : 0xFFFFFFFFu;
    my_units = lane < a.B ? xu - nu : 0xFFFFFFFFu;
    all_visits = lane_value(xv, 63);
    all_units = lane_value(xu, 63);
  } else {
    make_plan(a, rt, visits, units, red);
    all_visits = uniform(visits[a.B]);
    all_units = uniform(units[a.B]);
  }
  const uint32_t run = UNITS ? 0 : run_length(a, rt, all_visits, all_units);
  if (!UNITS && blockIdx.x == 0) {                              // for the launch that joins
    if (in_lanes) {
      if (wave == 0 && lane < a.B) a.plan[1 + lane] = my_visits;
    } else {
      for (uint32_t b = threadIdx.x; b < a.B; b += 256) a.plan[1 + b] = visits[b];
    }
    if (threadIdx.x == 0) a.plan[0] = run;
  }
  const uint32_t total = run ? all_visits : all_units;
  uint32_t pos = run ? worker * run : worker;
  const uint32_t end = run ? (total - (pos < total ? pos : total) < run ? total : pos + run) : total;
  while (pos < end) {
    const Kv4AttnK a = launch_args();
    const uint32_t* const visits = smem + 8;
    const uint32_t* const units = visits + a.B + 1;
    uint32_t b, u;
    Seq sq;
    if (a.B <= 64) {
      // the last lane whose count before it is at most pos (lane 0's is 0)
      const uint32_t before = run ? my_visits : my_units;
      const uint64_t at = __builtin_amdgcn_ballot_w64(before <= pos) | 1;
      b = 63 - (uint32_t)__builtin_clzll(at);
      sq.start = lane_value(mine.start, b);
      sq.rows = lane_value(mine.rows, b);
      sq.len = lane_value(mine.len, b);
      u = pos - lane_value(before, b);
    } else {
      const uint32_t* const count = run ? visits : units;
      b = uniform(find(count, a.B, pos));
      sq = load_seq(a, b);
      u = pos - uniform(count[b]);
    }
    const uint32_t tiles = seq_tiles(a, sq, rt), pages = seq_pages(a, sq);
    if (tiles == 0) break;                            // (row offsets out of order can make the counts wrap)
    uint32_t off = 0, seg = pages;
    if (run) {
      // a unit is a.unit_cost visits and then its pages
      const uint32_t unit = pages + a.unit_cost, in = u % unit;
      u = u / unit;
      const uint32_t take = unit - in < end - pos ? unit - in : end - pos;
      off = in > a.unit_cost ? in - a.unit_cost : 0;
      seg = in + take > a.unit_cost ? in + take - a.unit_cost - off : 0;
      pos += take;
      if (seg == 0) break;                            // (the run ends before the unit's first page)
    } else {
      pos += a.workers;
    }
    // heads vary fastest, and the tiles that see the most pages come first;
    // of a wave's units one at most began in an earlier run, and one ends in a later
    const uint32_t head = u % a.hkv, t = u / a.hkv;
    f(sq, b, tiles - 1 - (t < tiles ? t : tiles - 1), head, off, seg, seg == pages, 2 * worker + (off == 0));
  }
}

// ------------------------------------------------------------- main kernel --

// What the registers of the kernel for D dims and QT row tiles allow, without
// spills.  More waves hide more of the memory's latency and of the steps
// from one unit to the next.
constexpr int waves_per_simd(int d, int qt) {
  return d * qt <= 64 ? 4 : (d * qt <= 128 && qt == 1 ? 3 : (d * qt <= 256 ? 2 : 1));
}

// What a wave holds of one page of one head, as loaded: K of tile j's lanes'
// tokens (KD dwords of codes each) and the K scales of the lane group's 16
// tokens; V of dim pairs 16*jj + l%16 for those tokens, and their scales.
template <int D>
struct PageK {
  uint32_t k[4][D / 32];
  u32x4 s[2];
};
template <int D>
struct PageV {
  u32x4 v[D / 32];
  u32x4 s[2];
};

// A page of one head is one buffer (wave-uniform), so that a lane keeps three
// offsets for all its loads (what is the same for all lanes goes in the scalar offset).
template <int D, int kPagePolicy>
__device__ __forceinline__ void load_k(PageK<D>& p, Rsrc page, uint32_t m, uint32_t g) {
  constexpr int KD = D / 32;
  const uint32_t at = (16 * (m / 4) + m % 4) * (D / 2) + g * (D / 8);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (KD == 2) {
      const auto x = __builtin_amdgcn_raw_buffer_load_b64(page, at, 4 * j * (D / 2), kPagePolicy);
      p.k[j][0] = x[0];
      p.k[j][1] = x[1];
    } else {
#pragma unroll
      for (int i = 0; i < KD / 4; ++i) {
        const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(page, at, 4 * j * (D / 2) + 16 * i, kPagePolicy);
#pragma unroll
        for (int e = 0; e < 4; ++e) p.k[j][4 * i + e] = x[e];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) p.s[i] = __builtin_amdgcn_raw_buffer_load_b128(page, 32 * g, 64 * D + 16 * i, kPagePolicy);
}

template <int D, int kPagePolicy>
__device__ __forceinline__ void load_v(PageV<D>& p, Rsrc page, uint32_t m, uint32_t g) {
#pragma unroll
  for (int jj = 0; jj < D / 32; ++jj)
    p.v[jj] = __builtin_amdgcn_raw_buffer_load_b128(page, 64 * m + 16 * g, 32 * D + 1024 * jj, kPagePolicy);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    p.s[i] = __builtin_amdgcn_raw_buffer_load_b128(page, 32 * g, 64 * D + 128 + 16 * i, kPagePolicy);
}

// Scores of a page (tile j's row 4g + r: token 16g + 4j + r), in powers of two.
template <int DT, int D, int QT>
__device__ __forceinline__ void score_page(const PageK<D>& p, const u32x4 (&qf)[QT][D / 32], float scale2,
                                           const float (&M)[QT], f32x4 (&s)[QT][4]) {
  constexpr int KD = D / 32;
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
  // the scale of token 16g + 4j + r: half r%2 of word 2j + r/2 of the lane's eight
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t w = p.s[j / 2][2 * (j % 2) + r / 2];
      const float k = __uint_as_float(r % 2 ? w & 0xFFFF0000u : w << 16) * scale2;
#pragma unroll
      for (int t = 0; t < QT; ++t) s[t][j][r] = __builtin_fmaf(s[t][j][r], k, -M[t]);
    }
}

template <int D, int QT>
__device__ __forceinline__ void add_page(const PageV<D>& p, const u32x4 (&w)[QT][2], State<D, QT>& st) {
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

// One unit's pages [off, off + seg): the results where that is all of them,
// else a partial result in `slot`.  W > 1: all of its pages, by the W waves of
// a block, which join their results in `smem`.
template <int DT, int D, int QT, int W>
__device__ __forceinline__ void run_unit(const Seq& sq, uint32_t b, uint32_t tile, uint32_t head, uint32_t off,
                                         uint32_t seg, bool whole, uint32_t slot, float* smem) {
  constexpr uint32_t RT = 16 * QT;
  const Kv4AttnK a = launch_args();
  // One row tile a sequence reads its pages once: streamed (nt), 10 % faster than
  // through the caches (four caches of 131071 tokens: 104 against 115 us).
  // Several share them (four prompts' 512 rows each: 98 us, streamed 110).
  constexpr int kPolicy = QT == 1 ? 2 : 0;
  const uint32_t lane = threadIdx.x & 63, m16 = lane % 16, g = lane / 16;
  const uint32_t nrows = sq.rows * a.group;
  const uint32_t r0 = tile * RT, r1 = r0 + RT < nrows ? r0 + RT : nrows;
  if (r0 >= nrows) return;                            // (row offsets out of order)
  const uint32_t hi_first = row_hi(a, sq, r0), hi_last = row_hi(a, sq, r1 - 1);
  const uint32_t lo_first = row_lo(a, hi_first), lo_last = row_lo(a, hi_last);
  uint32_t p0 = lo_first / kKv4Tokens, p1 = (hi_last + kKv4Tokens - 1) / kKv4Tokens;
  if constexpr (W > 1) {
    const uint32_t n = p1 > p0 ? p1 - p0 : 0, w = uniform(threadIdx.x >> 6);
    p1 = p0 + n * (w + 1) / W;
    p0 += n * w / W;
  } else {
    p0 += off;
    p1 = seg < p1 - (p0 < p1 ? p0 : p1) ? p0 + seg : p1;
  }

  State<D, QT> st;
  clear(st);
  // The next page's K is asked for as soon as this page's has been used, and
  // its V likewise, so about a page a wave is in flight at all times without
  // a second set of registers.  A page that is not there is read as page 0
  // and counted as past every row's tokens.
  const PageTable table = page_table(a, b);
  const uint8_t* const cache = a.cache + (uint64_t)head * kv4_head_bytes(D);
  auto page_id = [&](uint32_t pg) { return table[pg < p1 ? pg : p1 - 1]; };
  auto there = [&](int32_t id) { return id >= 0 && id < a.pages; };
  auto base = [&](int32_t id) {
    return make_rsrc(cache + (uint64_t)(there(id) ? id : 0) * a.page_stride, kv4_head_bytes(D));
  };
  uint32_t pg = p0;
  if (pg < p1) {
    u32x4 qf[QT][D / 32];
    uint32_t lo[QT], hi[QT];
    load_q<D, QT>(a, sq, head, r0, r1, qf, lo, hi);
    PageK<D> pk;
    PageV<D> pv;
    int32_t id = page_id(pg), next = page_id(pg + 1);
    load_k<D, kPolicy>(pk, base(id), m16, g);
    load_v<D, kPolicy>(pv, base(id), m16, g);
    for (;;) {
      const bool more = pg + 1 < p1;
      const uint32_t tok0 = there(id) ? pg * kKv4Tokens : 0x7FFFFF00u;
      const Rsrc nb = base(next);
      const int32_t after = page_id(pg + 2);
      f32x4 s[QT][4];
      u32x4 w[QT][2];
      score_page<DT, D, QT>(pk, qf, a.scale2, st.M, s);
      if (more) load_k<D, kPolicy>(pk, nb, m16, g);
      float vc[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t x = pv.s[j / 2][2 * (j % 2) + r / 2];
          vc[j][r] = __uint_as_float(r % 2 ? x & 0xFFFF0000u : x << 16);
        }
      weigh<D, QT>(s, vc, st, tok0 >= lo_last && tok0 + kKv4Tokens <= hi_first, g, tok0, lo, hi, w);
      add_page<D, QT>(pv, w, st);
      if (!more) break;
      load_v<D, kPolicy>(pv, nb, m16, g);
      ++pg;
      id = next;
      next = after;
    }
  }

  if constexpr (W > 1)
    join_waves<DT, D, QT, W>(sq, st, head, r0, r1, smem);
  else
    store_rows<DT, D, QT, RT>(sq, st, head, r0, r1, 0, whole, slot);
}

template <int DT, int D, int QT>
__global__ __launch_bounds__(256, waves_per_simd(D, QT)) void kv4_attn_kernel(Kv4AttnK) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  walk<false>(16 * QT, blockIdx.x * 4 + uniform(threadIdx.x >> 6), reinterpret_cast<uint32_t*>(smem),
              [&](const Seq& sq, uint32_t b, uint32_t tile, uint32_t head, uint32_t off, uint32_t seg, bool whole,
                  uint32_t slot) { run_unit<DT, D, QT, 1>(sq, b, tile, head, off, seg, whole, slot, nullptr); });
}

// A block a unit, its pages shared by W waves, one launch.
template <int DT, int D, int QT, int W>
__global__ __launch_bounds__(64 * W, D * QT <= 64 ? 3 : (W > 4 ? 2 : waves_per_simd(D, QT))) void kv4_attn_block_kernel(Kv4AttnK) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  float* const join = reinterpret_cast<float*>(smem);
  walk<true>(16 * QT, blockIdx.x, reinterpret_cast<uint32_t*>(smem + kJoinBytes<QT, W>),
             [&](const Seq& sq, uint32_t b, uint32_t tile, uint32_t head, uint32_t off, uint32_t seg, bool whole,
                 uint32_t slot) { run_unit<DT, D, QT, W>(sq, b, tile, head, off, seg, whole, slot, join); });
}

// Joins the partial results of units that several waves shared, in page
// order.  D / 4 threads hold a row and head; WIDE: the other groups of its
// block take every so many-th of its partials (few rows, many partials
// each), else rows of their own.  Every partial's statistics and values are
// asked for together and joined by a running maximum, so that a row waits for
// memory once for its place in the plan and once for its partials.
constexpr uint32_t kJoinSeqs = 256;                    // (a thread each)

template <int DT, int D, int RT_, bool WIDE>
__global__ __launch_bounds__(256) void kv4_attn_join_kernel(Kv4AttnK a) {
  constexpr uint32_t RT = RT_, TP = D / 4, G = 256 / TP, U = 8;
  __shared__ float sm[G], sl[G];
  __shared__ __attribute__((aligned(16))) f32x4 so[G][TP];
  const uint32_t tid = threadIdx.x, col = tid % TP, grp = tid / TP;
  // where rows are told by offsets: a row's sequence is looked for in LDS, not by
  // loads that wait for one another
  __shared__ Seq seqs[kJoinSeqs];
  __shared__ uint32_t visits[kJoinSeqs];
  const bool staged = a.starts != nullptr && a.B <= kJoinSeqs;
  const uint32_t run = a.plan[0];
  if (staged) {
    if (tid < a.B) {
      seqs[tid] = load_seq(a, tid);
      visits[tid] = a.plan[1 + tid];
    }
    __syncthreads();
  }
  const uint64_t total = (uint64_t)a.T * a.hq, step = (uint64_t)gridDim.x * (WIDE ? 1 : G);
  for (uint64_t id = WIDE ? blockIdx.x : (uint64_t)blockIdx.x * G + grp; id < total; id += step) {
    const uint32_t row = (uint32_t)(id / a.hq), hd = (uint32_t)(id % a.hq);
    uint32_t b = row;
    if (a.starts != nullptr) {
      // the last sequence that starts at or before the row
      uint32_t lo = 0, hi = a.B;
      if (run == 0) continue;
      while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        const bool at = staged ? seqs[mid].start <= row : a.starts[mid] <= (int64_t)row;
        if (at) lo = mid; else hi = mid;
      }
      b = lo;
    }
    const Seq sq = staged ? seqs[b] : load_seq(a, b);
    const uint32_t before = staged ? visits[b] : a.plan[1 + b];
    if (run == 0 || row < sq.start || row - sq.start >= sq.rows) continue;
    const uint32_t tiles = seq_tiles(a, sq, RT), pages = seq_pages(a, sq);
    const uint32_t r = (row - sq.start) * a.group + hd % a.group;
    const uint32_t first = before + ((tiles - 1 - r / RT) * a.hkv + hd / a.group) * (pages + a.unit_cost) + a.unit_cost;
    const uint32_t i0 = first / run, i1 = (first + pages - 1) / run;
    if (i0 >= i1 || i1 >= a.workers) continue;        // one wave's: done (or row offsets out of order)
    float M = kNoScore, l = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    constexpr uint32_t stride = WIDE ? G : 1;
    for (uint32_t i = i0 + (WIDE ? grp : 0); i <= i1; i += U * stride) {
      float pm[U], pl[U];
      f32x4 po[U];
#pragma unroll
      for (uint32_t k = 0; k < U; ++k) {
        // wave j's partial: its second where the unit's pages begin in it, else its first
        const uint32_t j = i + k * stride <= i1 ? i + k * stride : i1;
        const uint64_t at = (uint64_t)(2 * j + (j == i0)) * RT + r % RT;
        pm[k] = a.stat[at * 2];
        pl[k] = a.stat[at * 2 + 1];
        po[k] = *reinterpret_cast<const f32x4*>(a.part + at * D + 4 * col);
      }
      float mn = M;
#pragma unroll
      for (uint32_t k = 0; k < U; ++k) mn = __builtin_fmaxf(mn, pm[k]);
      const float f = __builtin_amdgcn_exp2f(M - mn);
      M = mn;
      l *= f;
      o *= f;
#pragma unroll
      for (uint32_t k = 0; k < U; ++k) {
        if (i + k * stride > i1) continue;
        const float e = __builtin_amdgcn_exp2f(pm[k] - M);
        l += pl[k] * e;
        o += po[k] * e;
      }
    }
    if constexpr (WIDE) {
      if (col == 0) { sm[grp] = M; sl[grp] = l; }
      so[grp][col] = o;
      __syncthreads();
      if (grp == 0) {
        float mn = M;
#pragma unroll
        for (uint32_t k = 1; k < G; ++k) mn = __builtin_fmaxf(mn, sm[k]);
        l = 0.f;
        o = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (uint32_t k = 0; k < G; ++k) {
          const float e = __builtin_amdgcn_exp2f(sm[k] - mn);
          l += sl[k] * e;
          o += so[k][col] * e;
        }
        M = mn;
      }
      __syncthreads();
      if (grp != 0) continue;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 v = {pack16<DT>(o[0] * inv, o[1] * inv), pack16<DT>(o[2] * inv, o[3] * inv)};
    *reinterpret_cast<u32x2*>(a.out + (uint64_t)row * a.ldo_bytes + ((uint64_t)hd * D + 4 * col) * 2) = v;
    if (col == 0 && a.lse) a.lse[(uint64_t)row * a.hq + hd] = l == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(l)) * kLn2;
  }
}

// ------------------------------------------------------------------- host --

constexpr uint32_t kSimds = 1024;                      // four to each of 256 CUs
// LDS of walk()'s plan.
inline int plan_lds(uint32_t B) { return (8 + 2 * ((int)B + 1)) * 4; }

constexpr uint32_t kJoinBlocks = 2048;
// Rows and heads up to this: a block each (attn over one sequence of 1000 tokens
// 9.2 us; 2048 of them, 64 sequences of 256 tokens: 13.4 us by groups of D / 4
// threads, 16.5 a block each).
constexpr uint64_t kWideRows = 1024;

template <int DT, int D, int RT>
hipError_t launch_join(const Kv4AttnK& k, hipStream_t s) {
  const uint64_t rows = (uint64_t)k.T * k.hq;
  if (rows <= kWideRows) {
    hipLaunchKernelGGL((kv4_attn_join_kernel<DT, D, RT, true>), dim3((uint32_t)rows), dim3(256), 0, s, k);
  } else {
    const uint64_t blocks = (rows + 1024 / D - 1) / (1024 / D);
    hipLaunchKernelGGL((kv4_attn_join_kernel<DT, D, RT, false>), dim3(blocks < kJoinBlocks ? (uint32_t)blocks : kJoinBlocks),
                       dim3(256), 0, s, k);
  }
  return hipGetLastError();
}
template <int DT, int D, int QT, int W>
hipError_t launch_blocks(const Kv4AttnK& k, hipStream_t s) {
  const int lds = kJoinBytes<QT, W> + plan_lds(k.B);
  hipLaunchKernelGGL((kv4_attn_block_kernel<DT, D, QT, W>), dim3(k.workers), dim3(64 * W), lds, s, k);
  return hipGetLastError();
}
template <int DT, int D, int QT>
hipError_t launch(const Kv4AttnK& k, int block, hipStream_t s) {
  if (block == 4) return launch_blocks<DT, D, QT, 4>(k, s);
  if constexpr (QT == 2)
    if (block == 1) return launch_blocks<DT, D, QT, 1>(k, s);
  if constexpr (QT == 1)
    if (block == 8) return launch_blocks<DT, D, QT, 8>(k, s);
  hipLaunchKernelGGL((kv4_attn_kernel<DT, D, QT>), dim3(k.workers / 4), dim3(256), plan_lds(k.B), s, k);
  const hipError_t e = hipGetLastError();
  // (a unit of one page is one wave's)
  if (e != hipSuccess || k.max_pages <= 1) return e;
  return launch_join<DT, D, 16 * QT>(k, s);
}

// Waves of a block a unit, or 0 for equal runs over all waves and a second
// launch.  Blocks need no second launch and no partial results in memory, but
// leave waves idle where units are few, or their lengths unlike; so they are
// taken up to a number of pages (of the longest sequence there could be) that
// grows with the units (the most there could be).  32 KV-sharing query heads
// over 8, us by runs / by blocks: one token for one sequence of 1000 tokens 9.2 /
// 8.5 (2000 tokens: 9.6 / 12.7), for 16 of 1000 13.7 / 9.6, for 64 of 500 19.3 /
// 11.0, for 64 of up to 2000 19.5 / 19.9, for 64 of up to 8192 31.4 / 62; chunks of
// 512 rows over 4096 tokens, four: 171 / 162, over up to 5000 81.5 / 66; 256 rows
// over 4000 39.6 / 31.7; 64 rows over 4000 24.8 / 31.0.  Where
// units of two tiles outnumber the waves that the chip holds, a wave each, given
// out by the hardware as others end (whole units in runs / blocks of four / of
// one: eight prompts of 1000 tokens 169 / 188 / 113, one of 4096 198 / 191 / 167;
// four of 300 36 / 27 / 17; but chunks over up to 5000, with as many units as
// waves, 81.5 / 66 / 137).
int block_waves(int tile, int64_t units, int64_t pages, int64_t workers) {
  if (tile == 16) {
    const int64_t most = units / 10 < 16 ? 16 : (units / 10 > 32 ? 32 : units / 10);
    if (pages > most) return 0;
    // (16 of 1000 with four waves 10.7, 64 of 500 with eight 14.4)
    return pages > 4 && units <= 384 ? 8 : 4;
  }
  if (units >= 2 * workers || (units >= workers * 5 / 4 && pages <= 512) || (units >= workers / 2 && pages <= 8)) return 1;
  return pages <= (units / 4 > 128 ? 128 : units / 4) ? 4 : 0;
}

// How a call is run: rows a tile, and how many waves take runs of page
// visits: as many as the chip holds, fewer where the sequences, each as long as
// its table, would not fill them.
struct Shape {
  int tile;
  uint32_t workers;
  uint32_t unit_cost;          // page visits that starting and ending a unit counts as
  int block;                   // or a block of so many waves for each unit (else 0)
  uint32_t blocks;             // and the most units there can be
};

Shape shape_of(int64_t T, int64_t B, int64_t max_pages, int64_t window, int64_t hkv, int64_t group, int d) {
  // One 16-row tile a wave where an average sequence has no more, else two,
  // which convert a page's codes once for both.  (Four, one wave a SIMD: 265 us against
  // 176 for four chunks of 512 rows over 4096 tokens.)
  Shape s;
  s.tile = (T * group + B - 1) / B <= 16 ? 16 : 32;
  s.workers = kSimds * waves_per_simd(d, s.tile / 16);
  s.unit_cost = s.tile == 16 ? 6 : 3;
  const int64_t tiles = T * group / s.tile + (B < T ? B : T);
  const int64_t most = (tiles * hkv * ((max_pages > 0 ? max_pages : 1) + s.unit_cost) + 4) & ~(int64_t)3;
  if (most < (int64_t)s.workers) s.workers = (uint32_t)most;
  int64_t pages = max_pages;
  if (window > 0 && (window + T) / kKv4Tokens + 2 < pages) pages = (window + T) / kKv4Tokens + 2;
  // (up to 64 sequences: the plan is kept in lanes; one page: one wave's anyway)
  s.blocks = (uint32_t)(tiles * hkv);
  s.block = pages > 1 && B <= 64 ? block_waves(s.tile, tiles * hkv, pages, kSimds * waves_per_simd(d, s.tile / 16)) : 0;
  return s;
}

int64_t plan_bytes(int64_t B) { return ((B + 2) * 4 + 255) & ~(int64_t)255; }

}  // namespace

int64_t kv4_attn_workspace_bytes(int64_t T, int64_t B, int64_t max_pages, int32_t hq, int32_t hkv, int32_t head_dim) {
  if (T <= 0 || B <= 0 || hq == 0) return 0;
  // (the window is not known here: what the form that needs it takes)
  const Shape h = shape_of(T, B, max_pages, 0, hkv, hq / hkv, head_dim);
  const int64_t rows = (int64_t)2 * h.workers * h.tile;
  return plan_bytes(B) + rows * 8 + rows * head_dim * 4;
}

hipError_t launch_kv4_attn(const Kv4AttnArgs& a, hipStream_t s) {
  Kv4AttnK k;
  const int64_t group = a.hq / a.hkv;
  const Shape h = shape_of(a.T, a.B, a.max_pages, a.window, a.hkv, group, a.head_dim);
  k.workers = h.block ? h.blocks : h.workers;
  k.unit_cost = h.unit_cost;
  const int64_t rows = (int64_t)2 * h.workers * h.tile;
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
  uint8_t* w = static_cast<uint8_t*>(a.workspace);
  k.plan = reinterpret_cast<uint32_t*>(w);
  k.stat = reinterpret_cast<float*>(w + plan_bytes(a.B));
  k.part = reinterpret_cast<float*>(w + plan_bytes(a.B) + rows * 8);
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (h.tile == 16) return a.dtype == kF16 ? launch<kF16, D, 1>(k, h.block, s) : launch<kBF16, D, 1>(k, h.block, s);
    return a.dtype == kF16 ? launch<kF16, D, 2>(k, h.block, s) : launch<kBF16, D, 2>(k, h.block, s);
  };
  if (a.head_dim == 64) return pick(IntC<64>{});
  if (a.head_dim == 128) return pick(IntC<128>{});
  return pick(IntC<256>{});
}

}  // namespace qknorm
