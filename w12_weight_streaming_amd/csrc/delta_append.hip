// Inputs of a recurrent layer's rows (gfx950): the short causal convolution
// along each row's root path, SiLU, normalised query and key heads, and the
// decay and strength of every value head.
//
// Each input is read once by its own row and up to three times more, from the
// caches, by the rows behind it; outputs are written once. Bound by latency at
// few rows (the row's sequence, then its parents, then their inputs): 32 rows of
// 10240 channels 5.5 us. 512 fp32 rows 15.5 us for 42 MB (2.7 TB/s).
#include "delta_internal.h"
#include "w12_device.h"

namespace w12 {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;  // neighbouring channels a thread
constexpr int kWaves = kThreads / 64;
constexpr float kHeadEps = 1e-6f;

// 8 inputs of a row, rounded to bf16 as they are staged: the convolution is of
// what later steps will find in the window, however rows are grouped into steps.
__device__ __forceinline__ uint4 load_bf16x8(const void* p, int f32, size_t at) {
  if (!f32) return *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
  const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
  const float4 a = f[0], b = f[1];
  const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = bf16_pair(x[2 * i], x[2 * i + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Where a row's inputs come from. tap[t]: the row of the step t above it, or
// (below 0) the window's entry -1 - tap.
template <int W>
struct Place {
  int tap[W];
  int slot, state;  // state 0: a row; 1: of a sequence that is refused; 2: of none
};

// By one wave, in as few dependent loads as there are: sequences 64 at a time,
// then the sequence's parents.
template <int W>
__device__ __forceinline__ Place<W> place_of(const DeltaAppendArgs& a, int row) {
  const int lane = threadIdx.x & 63;
  Place<W> p;
  p.state = 2;
  p.slot = 0;
#pragma unroll
  for (int t = 0; t < W; ++t) p.tap[t] = 0;
  int seq = -1, row0 = 0, rows = 0, slot = 0;
  bool none = false;
  for (int j0 = 0; j0 < a.st.num_seq && seq < 0; j0 += 64) {
    const int j = min(j0 + lane, a.st.num_seq - 1);
    const int b0 = a.st.row_off[j], b1 = a.st.row_off[j + 1], sl = a.st.slot ? a.st.slot[j] : j;
    const bool in = j0 + lane < a.st.num_seq && b0 >= 0 && b1 <= a.st.total;
    const unsigned long long got = __ballot(in && b0 <= row && row < b1);
    if (!got) continue;
    const int at = __builtin_ctzll(got);
    seq = j0 + at;
    row0 = __shfl(b0, at);
    rows = __shfl(b1, at) - row0;
    slot = __shfl(sl, at);
    none = __any(in && lane < at && b0 < b1 && b0 < row0 + rows && b1 > row0);
    for (int i = lane; i < j0; i += 64) none = none || rows_meet(a.st.row_off, a.st.total, i, row0, rows);
  }
  if (seq < 0 || __any(none)) return p;
  bool bad = slot < 0 || slot >= a.c.slots;
  int mine = lane - 1;  // the parent of the sequence's row `lane`
  if (a.st.parent)
    for (int i = lane; i < rows; i += 64) {
      const int up = a.st.parent[row0 + i];
      bad = bad || (i == 0 ? up != -1 : (up < 0 || up >= i));
      if (i == lane) mine = up;
    }
  p.state = __any(bad) ? 1 : 0;
  if (p.state) return p;
  p.slot = slot;
  int at = row - row0;
#pragma unroll
  for (int t = 0; t < W; ++t) {
    p.tap[t] = at >= 0 ? row0 + at : -W - at;  // -1: the newest entry, W - 2
    const int near = __shfl(mine, at & 63);
    at = at <= 0 || !a.st.parent ? at - 1 : at < 64 ? near : a.st.parent[row0 + at];
  }
  return p;
}

// One workgroup per Rows rows and 2048 of their channels; a thread takes 8
// neighbouring ones, so a head is 8 or 16 neighbouring lanes of one wave, and
// keeps their weights for all rows. The last column of workgroups makes the gates.
template <int W, int Rows>
__global__ __launch_bounds__(kThreads) void delta_append_kernel(DeltaAppendArgs a) {
  __shared__ Place<W> s_place[Rows];
  const int tid = threadIdx.x, row0 = blockIdx.x * Rows;
  const int hk = a.c.key_heads, hv = a.c.value_heads, kd = a.c.key_dim;
  const bool gates = blockIdx.y + 1 == gridDim.y;
  const int at = (blockIdx.y * kThreads + tid) * kPer;
  const bool on = !gates && at < a.c.channels;
  float w[kPer * W], bias[kPer];
  uint4 own[Rows];  // the rows' own inputs: known before their places are
#pragma unroll
  for (int r = 0; r < Rows; ++r)
    own[r] = on ? load_bf16x8(a.qkv, a.f32, (size_t)min(row0 + r, a.st.total - 1) * a.qkv_stride + at) : make_uint4(0, 0, 0, 0);
  if (on) {
    const float4* p = reinterpret_cast<const float4*>(a.conv_weight + (size_t)at * W);
#pragma unroll
    for (int i = 0; i < kPer * W / 4; ++i) {
      const float4 x = p[i];
      w[4 * i] = x.x;
      w[4 * i + 1] = x.y;
      w[4 * i + 2] = x.z;
      w[4 * i + 3] = x.w;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) bias[i] = a.conv_bias ? a.conv_bias[at + i] : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < kPer * W; ++i) w[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) bias[i] = 0.0f;
  }
  for (int r = tid >> 6; r < Rows; r += kWaves)
    if (row0 + r < a.st.total) {
      const Place<W> p = place_of<W>(a, row0 + r);
      if ((tid & 63) == 0) s_place[r] = p;
    }
  __syncthreads();
  if (gates) {
    for (int e = tid; e < Rows * hv; e += kThreads) {
      const int r = e / hv, h = e - r * hv, row = row0 + r;
      if (row >= a.st.total || s_place[r].state != 0) continue;
      const size_t b0 = (size_t)row * a.ba_stride + h;
      float b, x;
      if (a.f32) {
        b = static_cast<const float*>(a.ba)[b0];
        x = static_cast<const float*>(a.ba)[b0 + hv];
      } else {
        b = bf16_to_f32(static_cast<const uint16_t*>(a.ba)[b0]);
        x = bf16_to_f32(static_cast<const uint16_t*>(a.ba)[b0 + hv]);
      }
      x += a.dt_bias[h];
      // log(1 + e^x) without overflow; e^-|x| <= 1
      const float soft = fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x)));
      a.c.gates[gate_at(a.c, a.layer, row, 0, h)] = x != x ? x : -expf(a.a_log[h]) * soft;
      const float e1 = expf(-fabsf(b));  // not past fp32's range on either side
      a.c.gates[gate_at(a.c, a.layer, row, 1, h)] = b != b ? b : (b < 0 ? e1 : 1.0f) / (1.0f + e1);
    }
    return;
  }
  uint4 x[W];
#pragma unroll
  for (int t = 0; t < W; ++t) x[t] = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int r = 0; r < Rows; ++r) {
    const int row = row0 + r;
    if (row >= a.st.total) return;
    const Place<W> p = s_place[r];
    if (p.state == 2) continue;  // a row of no sequence stays as it is
    const bool mine = on && p.state == 0;
    bool follows = r > 0 && s_place[max(r - 1, 0)].state == 0 && p.slot == s_place[max(r - 1, 0)].slot;
#pragma unroll
    for (int t = 1; t < W; ++t) follows = follows && p.tap[t] == s_place[max(r - 1, 0)].tap[t - 1];
    if (follows) {  // the row before is its parent, and has its other inputs
#pragma unroll
      for (int t = W - 1; t > 0; --t) x[t] = x[t - 1];
    } else if (mine) {
#pragma unroll
      for (int t = 1; t < W; ++t)
        x[t] = p.tap[t] >= 0 ? load_bf16x8(a.qkv, a.f32, (size_t)p.tap[t] * a.qkv_stride + at)
                             : *reinterpret_cast<const uint4*>(a.c.conv + conv_at(a.c, a.layer, p.slot, -1 - p.tap[t]) + at);
    }
    x[0] = own[r];
    float y[kPer], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) y[i] = bias[i];
#pragma unroll
    for (int t = 0; t < W; ++t) {
      const uint32_t u[4] = {x[t].x, x[t].y, x[t].z, x[t].w};
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        y[i] += w[i * W + W - 1 - t] * ((i & 1) ? __uint_as_float(u[i >> 1] & 0xFFFF0000u) : __uint_as_float(u[i >> 1] << 16));
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      y[i] = silu(y[i]);
      sum += y[i] * y[i];
    }
    if (at < 2 * hk * kd) {  // whole heads: channels and kd are multiples of 64
      for (int m = 1; m < kd / kPer; m <<= 1) sum += __shfl_xor(sum, m);
      const float f = 1.0f / sqrtf(sum + kHeadEps);
#pragma unroll
      for (int i = 0; i < kPer; ++i) y[i] *= f;
    }
    if (!on) continue;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = bf16_pair(y[2 * i], y[2 * i + 1]);
    if (!mine) o[0] = o[1] = o[2] = o[3] = 0x7FC07FC0u;  // reported through the queries: NaN
    const uint4 out = make_uint4(o[0], o[1], o[2], o[3]);
    if (at < hk * kd) *reinterpret_cast<uint4*>(a.q + (size_t)row * hk * kd + at) = out;
    if (!mine) continue;
    if (at >= hk * kd) *reinterpret_cast<uint4*>(a.c.kv + kv_at(a.c, a.layer, row) + at - hk * kd) = out;
    *reinterpret_cast<uint4*>(a.c.raw + raw_at(a.c, a.layer, row) + at) = x[0];
  }
}

// Rows a workgroup: one leaves more of them to hide each other's waits, four read
// the weights and hand on chains' inputs for four: 128 rows 7.1 us against 8.3,
// 256 rows 10.8 against 9.9, 512 fp32 rows 22 against 15.5.
template <int W>
void launch(const DeltaAppendArgs& a, hipStream_t s) {
  const int parts = (a.c.channels + kThreads * kPer - 1) / (kThreads * kPer) + 1;
  if (a.st.total <= 128)
    delta_append_kernel<W, 1><<<dim3(a.st.total, parts), kThreads, 0, s>>>(a);
  else
    delta_append_kernel<W, 4><<<dim3((a.st.total + 3) / 4, parts), kThreads, 0, s>>>(a);
}

}  // namespace

hipError_t launch_delta_append(const DeltaAppendArgs& a, hipStream_t s) {
  if (a.c.width == 2)
    launch<2>(a, s);
  else if (a.c.width == 3)
    launch<3>(a, s);
  else
    launch<4>(a, s);
  return hipGetLastError();
}

}  // namespace w12
