// The 4-bit KV cache's page layout and the kernels' arguments.
#pragma once

#include <stdint.h>

namespace qknorm {

// Tokens a page, and the bytes one KV head takes of it: K codes (token t,
// byte j: dims 2j low, 2j+1 high) at t*D/2 + j; V codes (dims 2j, 2j+1 of
// token t) at 32*D + 64*j + t; K scales (bf16) at 64*D + 2t; V scales at
// 64*D + 128 + 2t.
constexpr int kKv4Tokens = 64;
constexpr uint32_t kv4_head_bytes(uint32_t head_dim) { return 64 * head_dim + 256; }

template <int V>
struct IntC {
  static constexpr int value = V;
};

struct Kv4AppendK {
  const uint8_t* qkv;
  uint8_t* cache;
  const int64_t* slots;
  int64_t pages;
  uint64_t ld_bytes, page_stride;
  uint32_t T, hq, hkv;
};

struct Kv4GatherK {
  const uint8_t* cache;
  const int64_t* slots;
  uint8_t* k;
  uint8_t* v;
  int64_t pages;
  uint64_t page_stride, ldk_bytes, ldv_bytes;
  uint32_t T, hkv;
};

struct Kv4AttnK {
  const uint8_t* q;
  const uint8_t* cache;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* starts;       // or null: one row a sequence
  uint8_t* out;
  float* lse;                  // or null
  uint32_t* plan;              // page visits a wave, then the count of them before each sequence
  float* stat;                 // [slot][row]: maximum (log2) and sum; two slots a wave
  float* part;                 // [slot][row][D]
  int64_t pages, T;
  uint64_t ldq_bytes, ldo_bytes, page_stride, table_stride;
  uint32_t max_pages, B, hq, hkv, group, window, workers, unit_cost;
  float scale2;
};

}  // namespace qknorm
