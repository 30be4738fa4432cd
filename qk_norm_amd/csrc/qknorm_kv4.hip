// A paged KV cache in 4 bits: writing it from fused rows and reading it back
// (gfx950).  The attention over it is in qknorm_kv4_attn.hip.
//
// Each head vector x of D values is stored as D four-bit floats (a sign, two
// exponent bits, one fraction bit: 0, .5, 1, 1.5, 2, 3, 4, 6) and one bf16
// scale:
//   s = bf16(amax / 6),   code_j = round(x_j / s), halfway to the even code,
// beyond 6 to 6.  One scale per vector (not per 32 values) is what lets the
// attention apply it to a score or a weight, once per token, instead of to
// every value.
//
// The quotients are rounded correctly before the hardware conversion rounds
// them to codes (one residual step, exact where the quotient is representable,
// which every halfway point is), so the codes are those of the exact
// quotients: amax / 6 and x / s with 8- or 11-bit operands are never nearer
// than 2^-16 (relative) to a halfway point without being on it.
//
// A page of one head holds 64 tokens (64*D + 256 bytes): K codes token by
// token, V codes dim pair by dim pair (the order each lane of the attention's
// matrix products reads them in), then the K and the V scales.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qknorm_device.hpp"
#include "qknorm_kv4.hpp"
#include "qknorm_launch.hpp"

namespace qknorm {

namespace {

template <int DT>
__device__ __forceinline__ float widen16(uint32_t bits) {
  if constexpr (DT == kBF16) {
    return __uint_as_float(bits << 16);
  } else {
    const uint16_t h = (uint16_t)bits;
    return (float)__builtin_bit_cast(_Float16, h);
  }
}

__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const uint32_t w = __shfl_xor(v, o);
    v = v > w ? v : w;
  }
  return v;
}

// W consecutive dwords (aligned to 4 * W bytes, 16 at most).
template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&v)[W]) {
  if constexpr (W == 2) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 x = *reinterpret_cast<const u32x2*>(p);
    v[0] = x[0];
    v[1] = x[1];
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const u32x4 x = load16(p + 16 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * i + e] = x[e];
    }
  }
}
template <int W>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t (&v)[W]) {
  if constexpr (W == 2) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    *reinterpret_cast<u32x2*>(p) = u32x2{v[0], v[1]};
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i)
      __builtin_nontemporal_store(u32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]}, reinterpret_cast<u32x4*>(p + 16 * i));
  }
}

// The code of `slot`'s page and place, or false where it names none.
__device__ __forceinline__ bool slot_place(int64_t slot, int64_t pages, uint64_t page_stride, uint32_t head,
                                           uint32_t head_bytes, uint64_t* base, uint32_t* tok) {
  if (slot < 0 || slot >= pages * kKv4Tokens) return false;
  *base = (uint64_t)(slot / kKv4Tokens) * page_stride + (uint64_t)head * head_bytes;
  *tok = (uint32_t)(slot % kKv4Tokens);
  return true;
}

// A block takes TOK rows of one head's K (`which` 0) or V (1), sixteen
// threads a head vector, D / 16 values each.  K codes go straight out (D / 2
// consecutive bytes a token).  V codes pass through LDS, so that the lanes
// of a wave hold consecutive tokens of one dim pair: rows with consecutive
// slots then store runs of bytes.
template <int DT, int D, int TOK>
__global__ __launch_bounds__(256) void kv4_append_kernel(Kv4AppendK a) {
  constexpr int E = D / 16, W = E / 2, kRowB = D / 2 + 4;       // values and dwords a thread; LDS pitch
  constexpr uint32_t kGroups = 256 / TOK, kSteps = (D / 8 + kGroups - 1) / kGroups;
  __shared__ __attribute__((aligned(16))) uint8_t lds[TOK * kRowB];
  // the blocks of the same rows follow each other, so that a row's heads are read together
  const uint32_t tid = threadIdx.x, part = tid % 16, hv = blockIdx.x % (2 * a.hkv);
  const uint32_t which = hv / a.hkv, head = hv % a.hkv, row0 = blockIdx.x / (2 * a.hkv) * TOK;
  uint32_t v[TOK / 16][W];
  int64_t slot[TOK / 16];
  const uint64_t col = (uint64_t)(a.hq + (which ? a.hkv : 0) + head) * D * 2 + part * E * 2;
#pragma unroll
  for (int i = 0; i < TOK / 16; ++i) {
    const uint32_t r = row0 + i * 16 + tid / 16;
    slot[i] = -1;
    if (r < a.T) {
      slot[i] = a.slots[r];
      load_words<W>(a.qkv + (uint64_t)r * a.ld_bytes + col, v[i]);
    } else {
#pragma unroll
      for (int w = 0; w < W; ++w) v[i][w] = 0;
    }
  }
  constexpr uint32_t kInf = DT == kBF16 ? 0x7F80u : 0x7C00u;
#pragma unroll
  for (int i = 0; i < TOK / 16; ++i) {
    uint32_t m = 0;                                  // magnitudes order like their bits
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint32_t lo = v[i][w] & 0x7FFFu, hi = (v[i][w] >> 16) & 0x7FFFu;
      m = m > lo ? m : lo;
      m = m > hi ? m : hi;
    }
    m = row16_max_u32(m);
    const float amax = widen16<DT>(m);
    const bool bad = m >= kInf;                      // an infinity or a NaN: scale NaN, codes 0
    const bool none = bad || amax < 0x1p-100f;       // tiny: scale 0, codes 0
    const __bf16 sb = (__bf16)(amax / 6.f);
    const uint32_t sbits = bad ? 0x7FC0u : (none ? 0u : (uint32_t)__builtin_bit_cast(uint16_t, sb));
    const float s = none ? 1.f : __uint_as_float(sbits << 16), r = __builtin_amdgcn_rcpf(s);
    uint32_t code[(E + 7) / 8];
#pragma unroll
    for (int d = 0; d < (E + 7) / 8; ++d) code[d] = 0;
    auto quotient = [&](uint32_t bits) {
      const float x = widen16<DT>(bits);
      const float y = x * r;
      return __builtin_fmaf(__builtin_fmaf(-y, s, x), r, y);
    };
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float y0 = quotient(v[i][w] & 0xFFFFu), y1 = quotient(v[i][w] >> 16);
      uint32_t& c = code[w / 4];
      switch (w % 4) {                               // (the byte is an immediate)
        case 0: c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y0, y1, 1.f, 0); break;
        case 1: c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y0, y1, 1.f, 1); break;
        case 2: c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y0, y1, 1.f, 2); break;
        default: c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y0, y1, 1.f, 3); break;
      }
    }
    if (none) {
#pragma unroll
      for (int d = 0; d < (E + 7) / 8; ++d) code[d] = 0;
    }
    uint64_t base = 0;
    uint32_t tok = 0;
    const bool live = slot_place(slot[i], a.pages, a.page_stride, head, kv4_head_bytes(D), &base, &tok);
    if (live && part == 0)
      *reinterpret_cast<uint16_t*>(a.cache + base + 64 * D + which * 128 + tok * 2) = (uint16_t)sbits;
    if (which == 0) {
      if (live) {
        uint8_t* p = a.cache + base + tok * (D / 2) + part * (E / 2);
        if constexpr (E == 4) *reinterpret_cast<uint16_t*>(p) = (uint16_t)code[0];
        else {
#pragma unroll
          for (int d = 0; d < E / 8; ++d) reinterpret_cast<uint32_t*>(p)[d] = code[d];
        }
      }
    } else {
      uint8_t* p = lds + (i * 16 + tid / 16) * kRowB + part * (E / 2);
      if constexpr (E == 4) *reinterpret_cast<uint16_t*>(p) = (uint16_t)code[0];
      else {
#pragma unroll
        for (int d = 0; d < E / 8; ++d) reinterpret_cast<uint32_t*>(p)[d] = code[d];
      }
    }
  }
  if (which == 0) return;
  __syncthreads();
  // TOK consecutive threads hold TOK rows; each takes every (256/TOK)-th dword of its row
  const uint32_t t = tid % TOK, r = row0 + t;
  if (r >= a.T) return;
  uint64_t base = 0;
  uint32_t tok = 0;
  if (!slot_place(a.slots[r], a.pages, a.page_stride, head, kv4_head_bytes(D), &base, &tok)) return;
  uint8_t* out = a.cache + base + 32 * D + tok;
#pragma unroll
  for (uint32_t k = 0; k < kSteps; ++k) {
    const uint32_t d = tid / TOK + k * kGroups;
    if (kSteps * kGroups > D / 8 && d >= D / 8) break;
    const uint32_t c = *reinterpret_cast<const uint32_t*>(lds + t * kRowB + d * 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) out[(uint64_t)(d * 4 + e) * kKv4Tokens] = (uint8_t)(c >> (8 * e));
  }
}

// The way back: code * scale in fp32, rounded once to the output's type.
// The same blocks and threads as the append's; V passes through LDS the other way.
template <int DT, int D, int TOK>
__global__ __launch_bounds__(256) void kv4_gather_kernel(Kv4GatherK a) {
  constexpr int E = D / 16, W = E / 2, kRowB = D / 2 + 4, ES = IoTraits<DT>::kBytes, N = TOK / 16;
  constexpr uint32_t kGroups = 256 / TOK, kSteps = (D / 8 + kGroups - 1) / kGroups;
  __shared__ __attribute__((aligned(16))) uint8_t lds[TOK * kRowB];
  // the blocks of the same rows follow each other, so that a row's heads are read together
  const uint32_t tid = threadIdx.x, part = tid % 16, hv = blockIdx.x % (2 * a.hkv);
  const uint32_t which = hv / a.hkv, head = hv % a.hkv, row0 = blockIdx.x / (2 * a.hkv) * TOK;
  if (a.pages == 0) return;
  // every place first, then every load, so that they are in flight together
  // (a row without a place reads the cache's first and stores nothing)
  uint64_t base[N];
  uint32_t tok[N];
  bool live[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t r = row0 + i * 16 + tid / 16;
    base[i] = tok[i] = 0;
    live[i] = slot_place(r < a.T ? a.slots[r] : -1, a.pages, a.page_stride, head, kv4_head_bytes(D), &base[i], &tok[i]);
  }
  uint32_t sbits[N], code[N][(W + 3) / 4];
#pragma unroll
  for (int i = 0; i < N; ++i)
    sbits[i] = *reinterpret_cast<const uint16_t*>(a.cache + base[i] + 64 * D + which * 128 + tok[i] * 2);
  auto codes = [&](const uint8_t* c, uint32_t (&out)[(W + 3) / 4]) {
    if constexpr (E == 4) out[0] = *reinterpret_cast<const uint16_t*>(c);
    else {
#pragma unroll
      for (int d = 0; d < W / 4; ++d) out[d] = reinterpret_cast<const uint32_t*>(c)[d];
    }
  };
  if (which == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) codes(a.cache + base[i] + tok[i] * (D / 2) + part * (E / 2), code[i]);
  } else {
    const uint32_t t = tid % TOK, r = row0 + t;
    uint64_t vbase = 0;
    uint32_t vtok = 0;
    slot_place(r < a.T ? a.slots[r] : -1, a.pages, a.page_stride, head, kv4_head_bytes(D), &vbase, &vtok);
    const uint8_t* in = a.cache + vbase + 32 * D + vtok;
    uint32_t c[kSteps];
#pragma unroll
    for (uint32_t k = 0; k < kSteps; ++k) {
      const uint32_t d = tid / TOK + k * kGroups;
      c[k] = 0;
      if (kSteps * kGroups > D / 8 && d >= D / 8) break;
#pragma unroll
      for (int e = 0; e < 4; ++e) c[k] |= (uint32_t)in[(uint64_t)(d * 4 + e) * kKv4Tokens] << (8 * e);
    }
#pragma unroll
    for (uint32_t k = 0; k < kSteps; ++k) {
      const uint32_t d = tid / TOK + k * kGroups;
      if (kSteps * kGroups > D / 8 && d >= D / 8) break;
      *reinterpret_cast<uint32_t*>(lds + t * kRowB + d * 4) = c[k];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) codes(lds + (i * 16 + tid / 16) * kRowB + part * (E / 2), code[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!live[i]) continue;
    const uint32_t r = row0 + i * 16 + tid / 16;
    const float s = __uint_as_float(sbits[i] << 16);
    uint8_t* out = which ? a.v + (uint64_t)r * a.ldv_bytes : a.k + (uint64_t)r * a.ldk_bytes;
    out += ((uint64_t)head * D + part * E) * ES;
    uint32_t word[E * ES / 4];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const f16x2 h = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code[i][w / 4] >> (8 * (w % 4)), 1.f, 0);
      const float x = (float)h[0] * s, y = (float)h[1] * s;
      if constexpr (DT == kF32) {
        word[2 * w] = __float_as_uint(x);
        word[2 * w + 1] = __float_as_uint(y);
      } else if constexpr (DT == kBF16) {
        const bf16x2 o = {(__bf16)x, (__bf16)y};
        word[w] = __builtin_bit_cast(uint32_t, o);
      } else {
        const f16x2 o = {(_Float16)x, (_Float16)y};
        word[w] = __builtin_bit_cast(uint32_t, o);
      }
    }
    store_words<E * ES / 4>(out, word);
  }
}

constexpr uint32_t kFewRows = 4096;

template <int DT, int D>
hipError_t append(const Kv4AppendK& k, hipStream_t s) {
  // 64 rows a block make V's runs of bytes longer; 16 fill the CUs sooner: 1500
  // rows of 8 heads in and out 7.7 us against 9.0, 8192 rows 23.3 against 21.3
  if (k.T <= kFewRows) {
    hipLaunchKernelGGL((kv4_append_kernel<DT, D, 16>), dim3((k.T + 15) / 16 * k.hkv * 2), dim3(256), 0, s, k);
  } else {
    hipLaunchKernelGGL((kv4_append_kernel<DT, D, 64>), dim3((k.T + 63) / 64 * k.hkv * 2), dim3(256), 0, s, k);
  }
  return hipGetLastError();
}

template <int DT, int D>
hipError_t gather(const Kv4GatherK& k, hipStream_t s) {
  if (k.T <= kFewRows) {
    hipLaunchKernelGGL((kv4_gather_kernel<DT, D, 16>), dim3((k.T + 15) / 16 * k.hkv * 2), dim3(256), 0, s, k);
  } else {
    hipLaunchKernelGGL((kv4_gather_kernel<DT, D, 64>), dim3((k.T + 63) / 64 * k.hkv * 2), dim3(256), 0, s, k);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_append(const Kv4AppendArgs& a, hipStream_t s) {
  Kv4AppendK k;
  k.qkv = (const uint8_t*)a.qkv;
  k.ld_bytes = (uint64_t)a.ld * 2;
  k.cache = (uint8_t*)a.cache;
  k.pages = a.pages;
  k.page_stride = (uint64_t)a.page_stride;
  k.slots = a.slots;
  k.T = (uint32_t)a.T;
  k.hq = (uint32_t)a.hq;
  k.hkv = (uint32_t)a.hkv;
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    return a.dtype == kF16 ? append<kF16, D>(k, s) : append<kBF16, D>(k, s);
  };
  if (a.head_dim == 64) return pick(IntC<64>{});
  if (a.head_dim == 128) return pick(IntC<128>{});
  return pick(IntC<256>{});
}

hipError_t launch_kv4_gather(const Kv4GatherArgs& a, hipStream_t s) {
  Kv4GatherK k;
  k.cache = (const uint8_t*)a.cache;
  k.pages = a.pages;
  k.page_stride = (uint64_t)a.page_stride;
  k.slots = a.slots;
  k.k = (uint8_t*)a.k;
  k.v = (uint8_t*)a.v;
  const uint64_t es = a.dtype == kF32 ? 4 : 2;
  k.ldk_bytes = (uint64_t)a.ldk * es;
  k.ldv_bytes = (uint64_t)a.ldv * es;
  k.T = (uint32_t)a.T;
  k.hkv = (uint32_t)a.hkv;
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (a.dtype == kF32) return gather<kF32, D>(k, s);
    return a.dtype == kF16 ? gather<kF16, D>(k, s) : gather<kBF16, D>(k, s);
  };
  if (a.head_dim == 64) return pick(IntC<64>{});
  if (a.head_dim == 128) return pick(IntC<128>{});
  return pick(IntC<256>{});
}

}  // namespace qknorm
