// Internal interface between the C-ABI front end and the kernel launchers.
// Arguments reaching these functions have already been validated on the host.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qknorm {

struct PerHeadArgs {
  void* qkv;
  int64_t T, ld;
  int32_t hq, hkv, head_dim;
  const void* gamma_q;
  const void* gamma_k;
  float eps;
  int32_t dtype;
};

struct LayerwiseArgs {
  void* qkv;
  int64_t T, ld, wq, wk;
  const void* gamma_q;
  const void* gamma_k;
  float eps;
  int32_t nshards, dtype;
};

struct PartialArgs {
  const void* qkv;
  int64_t T, ld, wq, wk;
  int32_t nshards;
  float* part_q;
  float* part_k;
  int32_t dtype;
};

struct ApplyArgs {
  void* qkv;
  int64_t T, ld, wq, wk;
  const float* part_q;
  const float* part_k;
  int32_t nparts;
  int64_t norm_wq, norm_wk;
  const void* gamma_q;
  const void* gamma_k;
  float eps;
  int32_t dtype;
};

struct ProjArgs {
  const void* x;
  int64_t ldx;
  const void* w;
  int64_t ldw;
  void* qkv;
  int64_t ld, T, hidden;
  int32_t hq, hkv, head_dim;
  const void* gamma_q;
  const void* gamma_k;
  float eps;
  int32_t flags;
  int32_t dtype;       // kBF16 or kF16: x, w, gamma and qkv share it
};

// The projection on 8-bit integers: `p` with x and w int8 and the output's dtype.
struct W8a8Args {
  ProjArgs p;
  const float* x_scale;
  const float* w_scale;
};

struct QuantArgs {
  const void* x;
  int64_t ldx;
  void* q;
  int64_t ldq;
  float* scale;
  int64_t T, n;
  int32_t dtype;
};

struct Kv4AppendArgs {
  const void* qkv;
  int64_t ld, T;
  int32_t hq, hkv, head_dim;
  void* cache;
  int64_t pages, page_stride;  // page_stride in bytes
  const int64_t* slots;
  int32_t dtype;
};

struct Kv4GatherArgs {
  const void* cache;
  int64_t pages, page_stride;
  const int64_t* slots;
  int64_t T;
  int32_t hkv, head_dim;
  void* k;
  int64_t ldk;
  void* v;
  int64_t ldv;
  int32_t dtype;
};

struct Kv4AttnArgs {
  const void* q;
  int64_t ldq, T;
  const void* cache;
  int64_t pages, page_stride;
  const int32_t* table;
  int64_t table_stride, max_pages;
  const int32_t* lens;
  const int32_t* starts;
  int64_t B;
  void* out;
  int64_t ldo;
  float* lse;
  int32_t hq, hkv, head_dim, window;
  float scale;
  int32_t dtype;
  void* workspace;
};

// Whether every per-head trip's buffer span stays below 2^31 bytes.
bool per_head_span_ok(const PerHeadArgs& a);
// Whether the projection kernel takes this shape (tile offsets, K step, head_dim).
bool proj_shape_ok(const ProjArgs& a);

// `cus` is the compute-unit count of the current device (grid sizing).
hipError_t launch_per_head(const PerHeadArgs& a, hipStream_t s, int cus);
hipError_t launch_layerwise(const LayerwiseArgs& a, hipStream_t s, int cus);
hipError_t launch_partial_sumsq(const PartialArgs& a, hipStream_t s, int cus);
hipError_t launch_apply_scalar(const ApplyArgs& a, hipStream_t s, int cus);
hipError_t launch_qkv_proj(const ProjArgs& a, hipStream_t s, int cus);

// The column where the half-width tiles start (the whole width: none do).
uint32_t proj_split_column(uint32_t T, uint32_t N, uint32_t head_dim, int cus);

// The 8-bit projection: whether it takes this shape, the workspace of its
// split form (0 where T is outside 1..kProjSplitMaxT), and its launch (the
// split form where a workspace is given, which T must then be in range for).
bool w8a8_shape_ok(const ProjArgs& a);
int64_t w8a8_workspace_bytes(int64_t T, int64_t N);
hipError_t launch_w8a8(const W8a8Args& a, void* workspace, hipStream_t s, int cus);

hipError_t launch_quant_rows(const QuantArgs& a, hipStream_t s);
hipError_t launch_kv4_append(const Kv4AppendArgs& a, hipStream_t s);
hipError_t launch_kv4_gather(const Kv4GatherArgs& a, hipStream_t s);
hipError_t launch_kv4_attn(const Kv4AttnArgs& a, hipStream_t s);
// Workspace of the attention's plan and of its splits' partials.
int64_t kv4_attn_workspace_bytes(int64_t T, int64_t B, int64_t max_pages, int32_t hq, int32_t hkv,
                                 int32_t head_dim);

// Token counts up to this take the split projection when the caller gives a
// workspace (or the library's own scratch); larger ones take the tiles.
constexpr int64_t kProjSplitMaxT = 64;
// Bytes of fp32 partials the split projection needs for T tokens and N
// output columns (0 where T is outside 1..kProjSplitMaxT).
int64_t proj_workspace_bytes(int64_t T, int64_t N);
// The split projection: partial sums into `workspace`, then one block per
// head adds them and normalises (two launches on `s`).
hipError_t launch_qkv_proj_split(const ProjArgs& a, void* workspace, hipStream_t s);

// The library's own scratch for the split projection (one array per GPU):
// its size, and its device address on the current device (looked up once per
// device).  Devices numbered kMaxScratchDevices or higher are not served.
constexpr int64_t kProjScratchBytes = INT64_C(8) << 20;
constexpr int kMaxScratchDevices = 64;
hipError_t proj_scratch(void** ptr);

}  // namespace qknorm
