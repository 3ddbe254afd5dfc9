// Inputs of a recurrent layer's rows (gfx950): the short causal convolution
// along each row's root path, SiLU, normalised query and key heads, and the
// decay and strength of every value head.
#include "delta_internal.h"
#include "w12_device.h"

namespace w12 {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;  // neighbouring channels a thread
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
  for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16_rne(x[2 * i]) | ((uint32_t)f32_to_bf16_rne(x[2 * i + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One workgroup per row and 2048 of its channels; a thread takes 8
// neighbouring ones, so a head is 8 or 16 neighbouring lanes of one wave.
__global__ __launch_bounds__(kThreads) void delta_append_kernel(DeltaAppendArgs a) {
  __shared__ int s_seq, s_bad;
  const int tid = threadIdx.x, row = blockIdx.x;
  if (tid == 0) {
    s_seq = a.st.num_seq;
    s_bad = 0;
  }
  __syncthreads();
  for (int s = tid; s < a.st.num_seq; s += kThreads)
    if (rows_meet(a.st.row_off, a.st.total, s, row, 1)) atomicMin(&s_seq, s);
  __syncthreads();
  const int s = s_seq;
  if (s >= a.st.num_seq) return;  // a row of no sequence stays as it is
  const RowsView v = rows_view(a.c, a.st, s);
  int bad = v.ok ? 0 : 1;
  const int r = row - v.row0;
  for (int j = tid; j < s; j += kThreads)
    if (rows_meet(a.st.row_off, a.st.total, j, v.row0, v.rows)) bad |= 2;
  if (a.st.parent) {
    for (int i = tid; i < v.rows; i += kThreads) {
      const int p = a.st.parent[v.row0 + i];
      if (i == 0 ? p != -1 : (p < 0 || p >= i)) bad |= 1;
    }
  }
  if (bad) atomicOr(&s_bad, bad);
  __syncthreads();
  bad = s_bad;
  if (bad & 2) return;
  const int hk = a.c.key_heads, hv = a.c.value_heads, kd = a.c.key_dim;
  const int at = (blockIdx.y * kThreads + tid) * kPer;
  if (blockIdx.y == 0 && tid < hv && !bad) {
    const size_t b0 = (size_t)row * a.ba_stride + tid;
    float b, x;
    if (a.f32) {
      b = static_cast<const float*>(a.ba)[b0];
      x = static_cast<const float*>(a.ba)[b0 + hv];
    } else {
      b = bf16_to_f32(static_cast<const uint16_t*>(a.ba)[b0]);
      x = bf16_to_f32(static_cast<const uint16_t*>(a.ba)[b0 + hv]);
    }
    x += a.dt_bias[tid];
    // log(1 + e^x) without overflow; e^-|x| <= 1
    const float soft = fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x)));
    a.c.gates[gate_at(a.c, a.layer, row, 0, tid)] = x != x ? x : -expf(a.a_log[tid]) * soft;
    const float e = expf(-fabsf(b));  // not past fp32's range on either side
    a.c.gates[gate_at(a.c, a.layer, row, 1, tid)] = b != b ? b : (b < 0 ? e : 1.0f) / (1.0f + e);
  }
  const int qk = 2 * hk * kd;
  const bool on = at < a.c.channels, mine = on && !bad;
  float y[kPer];
  uint4 x0 = make_uint4(0, 0, 0, 0);
  if (mine) {
    x0 = load_bf16x8(a.qkv, a.f32, (size_t)row * a.qkv_stride + at);
#pragma unroll
    for (int i = 0; i < kPer; ++i) y[i] = a.conv_bias ? a.conv_bias[at + i] : 0.0f;
    const int w = a.c.width;
    int p = r;  // the tap's row in its tree; below 0: the window's entries, the newest at -1
    for (int t = 0; t < w; ++t) {
      uint4 x = x0;
      if (t > 0) {
        p = p > 0 ? (a.st.parent ? a.st.parent[v.row0 + p] : p - 1) : p - 1;
        x = p >= 0 ? load_bf16x8(a.qkv, a.f32, (size_t)(v.row0 + p) * a.qkv_stride + at)
                   : *reinterpret_cast<const uint4*>(a.c.conv + conv_at(a.c, a.layer, v.slot, w - 1 + p) + at);
      }
      const uint32_t u[4] = {x.x, x.y, x.z, x.w};
      const float* cw = a.conv_weight + (size_t)at * w + (w - 1 - t);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        y[i] += cw[i * w] * ((i & 1) ? __uint_as_float(u[i >> 1] & 0xFFFF0000u) : __uint_as_float(u[i >> 1] << 16));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) y[i] = 0.0f;
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    y[i] = y[i] / (1.0f + __expf(-y[i]));
    sum += y[i] * y[i];
  }
  if (at < qk) {  // whole heads: channels and kd are multiples of 64
    for (int m = 1; m < kd / kPer; m <<= 1) sum += __shfl_xor(sum, m);
    const float f = 1.0f / sqrtf(sum + kHeadEps);
#pragma unroll
    for (int i = 0; i < kPer; ++i) y[i] *= f;
  }
  if (!on) return;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = f32_to_bf16_rne(y[2 * i]) | ((uint32_t)f32_to_bf16_rne(y[2 * i + 1]) << 16);
  if (bad) o[0] = o[1] = o[2] = o[3] = 0x7FC07FC0u;  // reported through the queries: NaN
  const uint4 out = make_uint4(o[0], o[1], o[2], o[3]);
  if (at < hk * kd) *reinterpret_cast<uint4*>(a.q + (size_t)row * hk * kd + at) = out;
  if (bad) return;
  if (at >= hk * kd) *reinterpret_cast<uint4*>(a.c.kv + kv_at(a.c, a.layer, row) + at - hk * kd) = out;
  *reinterpret_cast<uint4*>(a.c.raw + raw_at(a.c, a.layer, row) + at) = x0;
}

}  // namespace

hipError_t launch_delta_append(const DeltaAppendArgs& a, hipStream_t s) {
  const int parts = (a.c.channels + kThreads * kPer - 1) / (kThreads * kPer);
  delta_append_kernel<<<dim3(a.st.total, parts), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace w12
