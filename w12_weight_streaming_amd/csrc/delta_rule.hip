// The gated delta rule over a step's rows (gfx950).
#include "delta_internal.h"
#include "w12_device.h"

namespace w12 {
namespace {

constexpr int kThreads = 256;

// One workgroup per sequence and value head, a thread per value dim. Chains
// run the recurrence on a state column in registers; rows of a tree each sum
// over their ancestors, whose deltas the same thread wrote.
template <int KD>
__global__ __launch_bounds__(kThreads) void delta_rule_kernel(DeltaRuleArgs a) {
  __shared__ float s_k[KD], s_q[KD];
  __shared__ int s_bad;
  const int tid = threadIdx.x, head = blockIdx.x, s = blockIdx.y, vd = a.c.value_dim;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  const RowsView v = rows_view(a.c, a.st, s);
  int bad = v.ok ? 0 : 1;
  for (int j = tid; j < s; j += kThreads) {
    if (rows_meet(a.st.row_off, a.st.total, j, v.row0, v.rows)) bad |= 2;
    if (a.keep && a.st.slot && a.st.slot[j] == v.slot) bad |= 1;
  }
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
  const int hv = a.c.value_heads, key = head / (hv / a.c.key_heads);
  const size_t kat = (size_t)key * KD, vat = (size_t)a.c.key_heads * KD + (size_t)head * vd;
  if (bad) {
    for (int i = 0; i < v.rows; ++i)
      if (tid < vd) a.out[((size_t)(v.row0 + i) * hv + head) * vd + tid] = 0x7FC0;
    return;
  }
  float* state = a.c.state + state_at(a.c, a.layer, v.slot, head);
  float S[KD];
  if (tid < vd)
#pragma unroll
    for (int i = 0; i < KD; ++i) S[i] = state[i * vd + tid];
  for (int i = 0; i < v.rows; ++i) {
    const int row = v.row0 + i;
    const uint16_t* kv = a.c.kv + kv_at(a.c, a.layer, row);
    __syncthreads();
    if (tid < KD) {
      s_k[tid] = bf16_to_f32(kv[kat + tid]);
      s_q[tid] = bf16_to_f32(a.q[((size_t)row * a.c.key_heads + key) * KD + tid]);
    }
    __syncthreads();
    if (tid >= vd) continue;
    const float beta = a.c.gates[gate_at(a.c, a.layer, row, 1, head)];
    const float val = bf16_to_f32(kv[vat + tid]);
    float x = 0, o = 0, d;
    if (!a.st.parent) {
      const float f = expf(a.c.gates[gate_at(a.c, a.layer, row, 0, head)]);
#pragma unroll
      for (int k = 0; k < KD; ++k) {
        S[k] *= f;
        x += S[k] * s_k[k];
      }
      d = beta * (val - x);
#pragma unroll
      for (int k = 0; k < KD; ++k) {
        S[k] += s_k[k] * d;
        o += S[k] * s_q[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < KD; ++k) {
        x += S[k] * s_k[k];
        o += S[k] * s_q[k];
      }
      // up the path: `sum` is what decays lie between the ancestor and this row
      double sum = 0;
      float xa = 0, oa = 0, self = 0;
      int p = i;
      while (true) {
        const int up = a.st.parent[v.row0 + p];
        sum += log_decay(a.c.gates[gate_at(a.c, a.layer, v.row0 + p, 0, head)]);
        if (up < 0) break;
        const uint16_t* kj = a.c.kv + kv_at(a.c, a.layer, v.row0 + up) + kat;
        float kk = 0, kq = 0;
        for (int k = 0; k < KD; ++k) {
          const float y = bf16_to_f32(kj[k]);
          kk += y * s_k[k];
          kq += y * s_q[k];
        }
        const float w = expf((float)sum) * a.c.delta[delta_at(a.c, a.layer, v.row0 + up, head) + tid];
        xa += kk * w;
        oa += kq * w;
        p = up;
      }
      for (int k = 0; k < KD; ++k) self += s_k[k] * s_q[k];
      const float f = (float)exp(sum);
      d = beta * (val - f * x - xa);
      o = f * o + oa + self * d;
    }
    if (!a.keep) a.c.delta[delta_at(a.c, a.layer, row, head) + tid] = d;
    a.out[((size_t)row * hv + head) * vd + tid] = f32_to_bf16_rne(a.scale * o);
  }
  if (!a.keep || v.rows == 0) return;
  if (tid < vd)
#pragma unroll
    for (int i = 0; i < KD; ++i) state[i * vd + tid] = S[i];
  const int share = (a.c.channels + gridDim.x - 1) / gridDim.x;
  advance_window(a.c, a.layer, v.slot, v.rows, head * share, min(a.c.channels, (head + 1) * share),
                 [&](int j) { return v.row0 + j; });
}

}  // namespace

hipError_t launch_delta_rule(const DeltaRuleArgs& a, hipStream_t s) {
  const dim3 grid(a.c.value_heads, a.st.num_seq);
  if (a.c.key_dim == 64)
    delta_rule_kernel<64><<<grid, kThreads, 0, s>>>(a);
  else
    delta_rule_kernel<128><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace w12
