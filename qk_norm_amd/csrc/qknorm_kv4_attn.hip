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
// against the 8 that a bf16 output keeps.  They stay in fp16's range whatever
// V's magnitude (struct State).  The maximum is kept until a row exceeds it by
// more than 8 powers of two.  Statistics and accumulators are fp32.
//
// Work is counted in page visits: one page of one head for one tile of rows,
// and a few more for each tile and head (a unit), for starting and ending it.  The plan is made on the GPU from the lengths there (they
// may change between replays of a captured graph), the same by every block.
// Where there are few units, all visits laid end to end are cut into equal
// runs, one a wave, whatever sequences and heads they fall in: a wave
// then takes the end of one unit's pages, some whole units, and the start of
// another's, so that it leaves at most two partial results, in the workspace,
// which a second launch joins in page order.  Where there are many, each is one
// wave's.  Waves share nothing but the plan.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qknorm_kv4_attn.hpp"

namespace qknorm {

namespace {

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
                                           f32x4 (&s)[QT][4]) {
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
      for (int t = 0; t < QT; ++t) s[t][j][r] *= k;
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
// else a partial result in `slot`.
template <int DT, int D, int QT>
__device__ __forceinline__ void run_unit(const Seq& sq, uint32_t b, uint32_t tile, uint32_t head,
                                         uint32_t off, uint32_t seg, bool whole, uint32_t slot) {
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
  p0 += off;
  p1 = seg < p1 - (p0 < p1 ? p0 : p1) ? p0 + seg : p1;

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
      score_page<DT, D, QT>(pk, qf, a.scale2, s);
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

  store_rows<DT, D, QT, RT>(sq, st, head, r0, r1, 0, whole, slot);
}

template <int DT, int D, int QT>
__global__ __launch_bounds__(256, waves_per_simd(D, QT)) void kv4_attn_kernel(Kv4AttnK) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  walk(16 * QT, blockIdx.x * 4 + uniform(threadIdx.x >> 6), reinterpret_cast<uint32_t*>(smem),
       [&](const Seq& sq, uint32_t b, uint32_t tile, uint32_t head, uint32_t off, uint32_t seg, bool whole, uint32_t slot) {
         run_unit<DT, D, QT>(sq, b, tile, head, off, seg, whole, slot);
       });
}

// ------------------------------------------------------------------- host --

constexpr uint32_t kSimds = 1024;                      // four to each of 256 CUs
constexpr int kMaxLds = 160 * 1024;
#ifndef UC_R
#define UC_R 1
#define UC_2 3
#endif
#ifndef QKNORM_ATTN_ROWS
#define QKNORM_ATTN_ROWS 64
#endif

template <int DT, int D, int QT>
hipError_t launch(const Kv4AttnK& k, hipStream_t s) {
  hipLaunchKernelGGL((kv4_attn_kernel<DT, D, QT>), dim3(k.workers / 4), dim3(256), plan_lds(k.B), s, k);
  const hipError_t e = hipGetLastError();
  // (a unit of one page is one wave's)
  if (e != hipSuccess || k.max_pages <= 1) return e;
  return launch_join<DT, D, 16 * QT>(k, s);
}

// How a call is run: rows a tile (16 or 32 a wave, or 128 a block), and how
// many waves or blocks take runs of page visits: as many as the chip holds,
// fewer where the sequences, each as long as its table, would not fill them.
struct Shape {
  int tile;
  uint32_t workers;
  uint32_t unit_cost;          // page visits that starting and ending a unit counts as
};

Shape shape_of(int64_t T, int64_t B, int64_t max_pages, int64_t hkv, int64_t group, int d) {
  // what an average sequence fills; the block's tile from more than two waves' rows
  const int64_t rows = (T * group + B - 1) / B;
  Shape s;
  if (rows > QKNORM_ATTN_ROWS && kv4_attn_rows_lds(d, B) <= kMaxLds) {
    s.tile = kv4_attn_rows_tile();
    s.workers = kv4_attn_rows_workers(d);
    s.unit_cost = UC_R;
  } else {
    s.tile = rows <= 16 ? 16 : 32;
    s.workers = kSimds * waves_per_simd(d, s.tile / 16);
    s.unit_cost = s.tile == 16 ? 6 : UC_2;
  }
  const int64_t tiles = T * group / s.tile + (B < T ? B : T);
  const int64_t most = (tiles * hkv * ((max_pages > 0 ? max_pages : 1) + s.unit_cost) / kMinRun + 4) & ~(int64_t)3;
  if (most < (int64_t)s.workers) s.workers = (uint32_t)most;
  return s;
}

int64_t plan_bytes(int64_t B) { return ((B + 2) * 4 + 255) & ~(int64_t)255; }

}  // namespace

int64_t kv4_attn_workspace_bytes(int64_t T, int64_t B, int64_t max_pages, int32_t hq, int32_t hkv, int32_t head_dim) {
  if (T <= 0 || B <= 0 || hq == 0) return 0;
  const Shape h = shape_of(T, B, max_pages, hkv, hq / hkv, head_dim);
  const int64_t rows = (int64_t)2 * h.workers * h.tile;
  return plan_bytes(B) + rows * 8 + rows * head_dim * 4;
}

hipError_t launch_kv4_attn(const Kv4AttnArgs& a, hipStream_t s) {
  Kv4AttnK k;
  const int64_t group = a.hq / a.hkv;
  const Shape h = shape_of(a.T, a.B, a.max_pages, a.hkv, group, a.head_dim);
  k.workers = h.workers;
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
  if (h.tile > 32) return launch_kv4_attn_rows(k, a.head_dim, a.dtype, s);
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (h.tile == 16) return a.dtype == kF16 ? launch<kF16, D, 1>(k, s) : launch<kBF16, D, 1>(k, s);
    return a.dtype == kF16 ? launch<kF16, D, 2>(k, s) : launch<kBF16, D, 2>(k, s);
  };
  if (a.head_dim == 64) return pick(IntC<64>{});
  if (a.head_dim == 128) return pick(IntC<128>{});
  return pick(IntC<256>{});
}

}  // namespace qknorm
