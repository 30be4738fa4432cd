// Attention of many rows a sequence (prompt chunks) over the paged 4-bit KV
// cache (gfx950): the arithmetic of qknorm_kv4_attn.hip with a page's codes
// converted once for a block.
//
// A block of four waves takes 128 rows of one KV head, a wave 32 of them.
// Each page's codes are converted by the block into LDS, in the order that
// the matrix products read their first operands (a fragment of 16 x 32
// values is 64 lanes' 16 bytes in a row, so every read and write is
// contiguous), and its scales beside them; then each wave runs the page
// against its rows.  There are two page buffers: while one is used the next
// page's codes, already in registers, are converted into the other, with one
// barrier a page.  Two blocks fit a CU (64 KiB of buffers each at head_dim
// 128), so one converts or waits while the other computes.
//
// What bounds it is vector instructions: a wave's page takes about 200 for the
// softmax of its 32 rows (32 of them exponentials, at a quarter of the rate)
// and 50 for its share of the conversions beside 64 matrix products, 1.9 k
// cycles against the products' 1.0 k.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qknorm_kv4_attn.hpp"

namespace qknorm {

namespace {

constexpr int kWaves = 4, kQT = 2, kRows = kWaves * 16 * kQT;

// One page in LDS: K fragments (tile j, step i), V fragments (dim pairs
// 16*jj, step u, low or high dim), K scales times the softmax's factor, V scales.
template <int D>
struct RowsLds {
  static constexpr int kK = 64 * D * 2, kV = 64 * D * 2, kPage = kK + kV + 2 * 64 * 4;
  static constexpr int kBytes = 2 * kPage;
};

// A thread's share of a page as loaded: K of its lane's token in tile `wave`,
// V of its lane's dim pair in row group(s) of its wave, one scale.
template <int D>
struct RawPage {
  uint32_t k[D / 32];
  u32x4 v[D <= 128 ? 1 : 2];
  uint32_t s;
};

template <int D>
__device__ __forceinline__ void load_raw(RawPage<D>& p, Rsrc page, uint32_t wave, uint32_t lane) {
  const uint32_t m = lane % 16, g = lane / 16;
  const uint32_t at = (16 * (m / 4) + m % 4) * (D / 2) + g * (D / 8), row = 4 * wave * (D / 2);
  if constexpr (D == 64) {
    const auto x = __builtin_amdgcn_raw_buffer_load_b64(page, at, row, 0);
    p.k[0] = x[0];
    p.k[1] = x[1];
    // half of a pair's 16 tokens: wave = 2 * jj + u
    const auto y = __builtin_amdgcn_raw_buffer_load_b64(page, 64 * m + 16 * g, 32 * D + (wave / 2) * 1024 + (wave % 2) * 8, 0);
    p.v[0][0] = y[0];
    p.v[0][1] = y[1];
  } else {
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(page, at, row + 16 * i, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) p.k[4 * i + e] = x[e];
      p.v[i] = __builtin_amdgcn_raw_buffer_load_b128(page, 64 * m + 16 * g, 32 * D + (wave * (D / 128) + i) * 1024, 0);
    }
  }
  // wave 0 takes the K scales, wave 1 the V scales
  p.s = wave < 2 ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(page, 2 * lane, 64 * D + 128 * wave, 0) : 0u;
}

template <int DT, int D>
__device__ __forceinline__ void put_page(const RawPage<D>& p, uint8_t* lds, float scale2, uint32_t wave, uint32_t lane) {
  constexpr int KD = D / 32;
#pragma unroll
  for (int i = 0; i < KD; ++i)
    *reinterpret_cast<u32x4*>(lds + ((wave * KD + i) * 64 + lane) * 16) = AttnElem<DT>::codes(p.k[i]);
  uint8_t* const v = lds + RowsLds<D>::kK;
  // low codes of tokens x and 4 + x side by side, then the high ones
  auto put = [&](uint32_t a, uint32_t b, uint32_t frag) {
    const uint32_t dl = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
    const uint32_t dh = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
    *reinterpret_cast<u32x4*>(v + (frag * 128 + lane) * 16) = AttnElem<kF16>::codes(dl);
    *reinterpret_cast<u32x4*>(v + (frag * 128 + 64 + lane) * 16) = AttnElem<kF16>::codes(dh);
  };
  if constexpr (D == 64) {
    put(p.v[0][0], p.v[0][1], wave);
  } else {
#pragma unroll
    for (int i = 0; i < D / 128; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) put(p.v[i][2 * u], p.v[i][2 * u + 1], (wave * (D / 128) + i) * 2 + u);
  }
  if (wave < 2) {
    float* const s = reinterpret_cast<float*>(lds + RowsLds<D>::kK + RowsLds<D>::kV);
    const float x = __uint_as_float(p.s << 16);
    s[64 * wave + lane] = wave == 0 ? x * scale2 : x;
  }
}

// LDS writes before it are seen after it; loads in flight stay in flight.
__device__ __forceinline__ void page_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <int DT, int D>
__device__ __forceinline__ void use_page(const uint8_t* lds, const u32x4 (&qf)[kQT][D / 32], State<D, kQT>& st, bool full,
                                         uint32_t lane, uint32_t tok0, const uint32_t (&lo)[kQT], const uint32_t (&hi)[kQT]) {
  constexpr int KD = D / 32;
  const uint32_t g = lane / 16;
  const float* const scales = reinterpret_cast<const float*>(lds + RowsLds<D>::kK + RowsLds<D>::kV);
  f32x4 s[kQT][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int t = 0; t < kQT; ++t) s[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KD; ++i) {
      const u32x4 kf = load16(lds + ((j * KD + i) * 64 + lane) * 16);
#pragma unroll
      for (int t = 0; t < kQT; ++t) s[t][j] = AttnElem<DT>::mfma(kf, qf[t][i], s[t][j]);
    }
    const f32x4 k = *reinterpret_cast<const f32x4*>(scales + 16 * g + 4 * j);
#pragma unroll
    for (int t = 0; t < kQT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) s[t][j][r] *= k[r];
  }
  float vc[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(scales + 64 + 16 * g + 4 * j);
#pragma unroll
    for (int r = 0; r < 4; ++r) vc[j][r] = v[r];
  }
  u32x4 w[kQT][2];
  weigh<D, kQT>(s, vc, st, full, g, tok0, lo, hi, w);
  const uint8_t* const v = lds + RowsLds<D>::kK;
#pragma unroll
  for (int jj = 0; jj < D / 32; ++jj)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 vf = load16(v + (((jj * 2 + u) * 2 + h) * 64 + lane) * 16);
#pragma unroll
        for (int t = 0; t < kQT; ++t) st.acc[t][jj][h] = AttnElem<kF16>::mfma(vf, w[t][u], st.acc[t][jj][h]);
      }
}

template <int DT, int D>
__device__ __forceinline__ void run_rows(uint8_t* lds, const Seq& sq, uint32_t b, uint32_t tile,
                                         uint32_t head, uint32_t off, uint32_t seg, bool whole, uint32_t slot) {
  const Kv4AttnK a = launch_args();
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t nrows = sq.rows * a.group;
  const uint32_t r0 = tile * kRows, r1 = r0 + kRows < nrows ? r0 + kRows : nrows;
  if (r0 >= nrows) return;                            // (row offsets out of order; the same for the whole block)
  // the block's pages
  uint32_t p0 = row_lo(a, row_hi(a, sq, r0)) / kKv4Tokens, p1 = (row_hi(a, sq, r1 - 1) + kKv4Tokens - 1) / kKv4Tokens;
  p0 += off;
  p1 = seg < p1 - (p0 < p1 ? p0 : p1) ? p0 + seg : p1;
  // the wave's rows (a wave past the end helps with the pages)
  const uint32_t w0 = r0 + wave * 16 * kQT;
  const bool mine = w0 < r1;
  const uint32_t first = mine ? w0 : r1 - 1, last = first + 16 * kQT < r1 ? first + 16 * kQT : r1;
  const uint32_t hi_first = row_hi(a, sq, first), hi_last = row_hi(a, sq, last - 1);
  const uint32_t lo_first = row_lo(a, hi_first), lo_last = row_lo(a, hi_last);
  State<D, kQT> st;
  clear(st);

  const PageTable table = page_table(a, b);
  const uint8_t* const cache = a.cache + (uint64_t)head * kv4_head_bytes(D);
  auto page_id = [&](uint32_t pg) { return table[pg < p1 ? pg : p1 - 1]; };
  auto there = [&](int32_t id) { return id >= 0 && id < a.pages; };
  // a page that is not there is read as page 0 and skipped
  auto base = [&](int32_t id) {
    return make_rsrc(cache + (uint64_t)(there(id) ? id : 0) * a.page_stride, kv4_head_bytes(D));
  };
  if (p0 < p1) {
    u32x4 qf[kQT][D / 32];
    uint32_t lo[kQT], hi[kQT];
    load_q<D, kQT>(a, sq, head, first, last, qf, lo, hi);
    RawPage<D> raw;
    int32_t id = page_id(p0), next = page_id(p0 + 1);
    load_raw<D>(raw, base(id), wave, lane);
    put_page<DT, D>(raw, lds, a.scale2, wave, lane);
    if (p0 + 1 < p1) load_raw<D>(raw, base(next), wave, lane);
    for (uint32_t pg = p0;; ++pg) {
      uint8_t* const now = lds + ((pg - p0) & 1) * RowsLds<D>::kPage;
      uint8_t* const other = lds + ((pg - p0 + 1) & 1) * RowsLds<D>::kPage;
      const int32_t after = page_id(pg + 2);
      page_barrier();                                 // page pg is in LDS, and page pg - 1 has been used
      const uint32_t tok0 = pg * kKv4Tokens;
      if (mine && there(id) && tok0 < hi_last && tok0 + kKv4Tokens > lo_first)
        use_page<DT, D>(now, qf, st, tok0 >= lo_last && tok0 + kKv4Tokens <= hi_first, lane, tok0, lo, hi);
      if (pg + 1 >= p1) break;
      put_page<DT, D>(raw, other, a.scale2, wave, lane);
      if (pg + 2 < p1) load_raw<D>(raw, base(after), wave, lane);
      id = next;
      next = after;
    }
    page_barrier();                                   // the buffers are free for the next unit
  }
  if (mine) store_rows<DT, D, kQT, kRows>(sq, st, head, first, last, wave * 16 * kQT, whole, slot);
}

// Two blocks a CU; at head_dim 256 (twice the buffers and accumulators) one.
constexpr int rows_blocks_per_cu(int d) { return d <= 128 ? 2 : 1; }

template <int DT, int D>
__global__ __launch_bounds__(256, rows_blocks_per_cu(D)) void kv4_attn_rows_kernel(Kv4AttnK) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  walk(kRows, blockIdx.x, reinterpret_cast<uint32_t*>(smem + RowsLds<D>::kBytes),
       [&](const Seq& sq, uint32_t b, uint32_t tile, uint32_t head, uint32_t off, uint32_t seg, bool whole, uint32_t slot) {
         run_rows<DT, D>(smem, sq, b, tile, head, off, seg, whole, slot);
       });
}

template <int DT, int D>
hipError_t launch(const Kv4AttnK& k, hipStream_t s) {
  const int lds = RowsLds<D>::kBytes + plan_lds(k.B);
  auto kern = kv4_attn_rows_kernel<DT, D>;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(k.workers), dim3(256), lds, s, k);
  e = hipGetLastError();
  if (e != hipSuccess || k.max_pages <= 1) return e;
  return launch_join<DT, D, kRows>(k, s);
}

}  // namespace

int kv4_attn_rows_tile() { return kRows; }

int64_t kv4_attn_rows_lds(int head_dim, int64_t B) {
  const int pages = head_dim == 64 ? RowsLds<64>::kBytes : (head_dim == 128 ? RowsLds<128>::kBytes : RowsLds<256>::kBytes);
  return pages + plan_lds((uint32_t)B);
}

uint32_t kv4_attn_rows_workers(int head_dim) { return 256u * rows_blocks_per_cu(head_dim); }

hipError_t launch_kv4_attn_rows(const Kv4AttnK& k, int head_dim, int dtype, hipStream_t s) {
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    return dtype == kF16 ? launch<kF16, D>(k, s) : launch<kBF16, D>(k, s);
  };
  if (head_dim == 64) return pick(IntC<64>{});
  if (head_dim == 128) return pick(IntC<128>{});
  return pick(IntC<256>{});
}

}  // namespace qknorm
