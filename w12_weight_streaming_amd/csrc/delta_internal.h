// Host-side launch interface of the recurrent layers' kernels
// (delta_append.hip, delta_rule.hip, delta_commit.hip) and of the norms
// (norm.hip), and the device helpers they share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_internal.h"

namespace w12 {

// The recurrent layers' arrays (w12.h) with every size in elements.
struct DeltaArgs {
  float* state;
  uint16_t* conv;
  uint16_t* raw;
  uint16_t* kv;
  float* gates;
  float* delta;
  int layers, slots, step_rows, key_heads, value_heads, key_dim, value_dim, width;
  int channels;  // 2 key_heads key_dim + value_heads value_dim
  int kv_width;  // key_heads key_dim + value_heads value_dim
};

struct DeltaAppendArgs {
  DeltaArgs c;
  StepArgs st;
  int layer;
  const void* qkv;
  int64_t qkv_stride;
  const void* ba;
  int64_t ba_stride;
  int f32;
  const float* conv_weight;
  const float* conv_bias;  // null: none
  const float* a_log;
  const float* dt_bias;
  uint16_t* q;
};

struct DeltaRuleArgs {
  DeltaArgs c;
  StepArgs st;
  int layer;
  const uint16_t* q;
  float scale;
  int keep;
  uint16_t* out;
};

struct DeltaCommitArgs {
  DeltaArgs c;
  StepArgs st;
  const int32_t* accept_len;
  const int32_t* path;  // null: the first accept_len + 1 rows
  int32_t* kept;
};

struct NormArgs {
  int64_t rows;
  int groups, width;
  const void* y;  // null: h alone
  int y_f32;
  int64_t y_stride;
  const float* post_weight;
  const void* gate;
  int gate_f32;
  int64_t gate_stride;
  float scale;
  void* h;
  int h_f32;
  const float* weight;
  float eps;
  uint16_t* out;
};

hipError_t launch_delta_append(const DeltaAppendArgs& a, hipStream_t s);
hipError_t launch_delta_rule(const DeltaRuleArgs& a, hipStream_t s);
hipError_t launch_delta_chain(const DeltaRuleArgs& a, hipStream_t s);  // parent null
hipError_t launch_delta_commit(const DeltaCommitArgs& a, hipStream_t s);
hipError_t launch_norm(const NormArgs& a, hipStream_t s);

#ifdef __HIPCC__
__device__ __forceinline__ float bf16_to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Two values as bf16, rounded to nearest even (one instruction).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16_2 __attribute__((ext_vector_type(2)));
  const bf16_2 p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}
// z / (1 + e^-z): the reciprocal is off by one step, and 0 from z = -87.3 down,
// where it would be denormal (the value is below 1.1e-36).
__device__ __forceinline__ float silu(float z) { return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

__device__ __forceinline__ size_t state_at(const DeltaArgs& c, int layer, int slot, int head) {
  return (((size_t)layer * c.slots + slot) * c.value_heads + head) * ((size_t)c.key_dim * c.value_dim);
}
__device__ __forceinline__ size_t conv_at(const DeltaArgs& c, int layer, int slot, int back_row) {
  return (((size_t)layer * c.slots + slot) * (c.width - 1) + back_row) * (size_t)c.channels;
}
__device__ __forceinline__ size_t raw_at(const DeltaArgs& c, int layer, int row) {
  return ((size_t)layer * c.step_rows + row) * (size_t)c.channels;
}
__device__ __forceinline__ size_t kv_at(const DeltaArgs& c, int layer, int row) {
  return ((size_t)layer * c.step_rows + row) * (size_t)c.kv_width;
}
__device__ __forceinline__ size_t gate_at(const DeltaArgs& c, int layer, int row, int beta, int head) {
  return (((size_t)layer * c.step_rows + row) * 2 + beta) * (size_t)c.value_heads + head;
}
__device__ __forceinline__ size_t delta_at(const DeltaArgs& c, int layer, int row, int head) {
  return (((size_t)layer * c.step_rows + row) * c.value_heads + head) * (size_t)c.value_dim;
}

// Sequence s (the same for all lanes) of a step: ok is false where its offsets
// or its slot are outside their arrays. In scalar registers, so that addresses are too.
struct RowsView {
  int row0, rows, slot;
  bool ok;
};
__device__ __forceinline__ RowsView rows_view(const DeltaArgs& c, const StepArgs& st, int s) {
  RowsView v;
  const int b0 = __builtin_amdgcn_readfirstlane(st.row_off[s]), b1 = __builtin_amdgcn_readfirstlane(st.row_off[s + 1]);
  v.ok = b0 >= 0 && b0 <= b1 && b1 <= st.total;
  v.row0 = v.ok ? b0 : 0;
  v.rows = v.ok ? b1 - b0 : 0;
  v.slot = st.slot ? __builtin_amdgcn_readfirstlane(st.slot[s]) : s;
  if (v.slot < 0 || v.slot >= c.slots) {
    v.ok = false;
    v.slot = 0;
  }
  return v;
}

// A log decay in 64 bits, for sums whose differences stay sums: e^-1e4 is 0 in
// either type, and minus infinity would leave no difference. NaN stays NaN.
__device__ __forceinline__ double log_decay(float g) { return g < -1e4f ? -1e4 : (double)g; }

// The window behind a sequence's committed rows when `n` more join them, the
// j-th of them row `row(j)` of the step: channels [c0, c1) of it, a channel by
// one thread (it reads the old window before it writes).
template <typename Row>
__device__ __forceinline__ void advance_window(const DeltaArgs& c, int layer, int slot, int n, int c0, int c1, Row row) {
  const int w = c.width - 1;
  for (int ch = c0 + threadIdx.x; ch < c1; ch += blockDim.x) {
    uint16_t x[3];
    for (int i = 0; i < w; ++i) {
      const int at = n + i;  // of the old window's w rows, then the n new ones
      x[i] = at < w ? c.conv[conv_at(c, layer, slot, at) + ch] : c.raw[raw_at(c, layer, row(at - w)) + ch];
    }
    for (int i = 0; i < w; ++i) c.conv[conv_at(c, layer, slot, i) + ch] = x[i];
  }
}
#endif

}  // namespace w12
