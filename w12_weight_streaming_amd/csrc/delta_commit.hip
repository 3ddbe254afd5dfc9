// Commit of a recurrent layer's accepted rows (gfx950), all layers at once.
//
// A row's delta depends on its ancestors alone, so the deltas that the pass
// computed for an accepted path are those of a replay, and the state behind it is
//   S e^G_n + sum_j k_j (e^(G_n - G_j) delta_j)^T,
// one pass over the state with no product that depends on another.
#include "delta_internal.h"
#include "w12_device.h"

namespace w12 {
namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void delta_commit_kernel(DeltaCommitArgs a) {
  __shared__ int s_row[kStepRows];
  __shared__ double s_sum[kStepRows];
  __shared__ int s_bad;
  const int tid = threadIdx.x, head = blockIdx.x, s = blockIdx.y, layer = blockIdx.z;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  const RowsView v = rows_view(a.c, a.st, s);
  const int acc = a.accept_len[s], n = v.ok ? acc + 1 : 0;
  int bad = (!v.ok || acc < -1 || acc >= v.rows) ? 1 : 0;
  for (int j = tid; j < s; j += kThreads) {
    if ((a.st.slot ? a.st.slot[j] : j) == v.slot) bad = 1;
    if (rows_meet(a.st.row_off, a.st.total, j, v.row0, v.rows)) bad = 1;
  }
  if (!bad) {
    for (int j = tid; j < n; j += kThreads) {
      int p = j;
      if (a.path) {
        p = a.path[v.row0 + j];
        if (j == 0 ? p != 0 : (p <= a.path[v.row0 + j - 1] || p >= v.rows)) bad = 1;
      }
      s_row[j] = v.row0 + p;
    }
  }
  if (bad) atomicOr(&s_bad, 1);
  __syncthreads();
  bad = s_bad;
  if (tid == 0 && head == 0 && layer == 0) a.kept[s] = bad ? -1 : n;
  if (bad || n == 0) return;
  if (tid == 0) {
    double sum = 0;
    for (int j = 0; j < n; ++j) s_sum[j] = sum += log_decay(a.c.gates[gate_at(a.c, layer, s_row[j], 0, head)]);
  }
  __syncthreads();
  const int kd = a.c.key_dim, vd = a.c.value_dim;
  const int key = head / (a.c.value_heads / a.c.key_heads);
  float* state = a.c.state + state_at(a.c, layer, v.slot, head);
  const float keep = (float)exp(s_sum[n - 1]);
  for (int e = tid; e < kd * vd; e += kThreads) {
    const int k = e / vd, d = e - k * vd;
    float x = keep * state[e];
    for (int j = 0; j < n; ++j) {
      const float w = expf((float)(s_sum[n - 1] - s_sum[j]));
      x += bf16_to_f32(a.c.kv[kv_at(a.c, layer, s_row[j]) + key * kd + k]) *
           (w * a.c.delta[delta_at(a.c, layer, s_row[j], head) + d]);
    }
    state[e] = x;
  }
  const int share = (a.c.channels + gridDim.x - 1) / gridDim.x;
  advance_window(a.c, layer, v.slot, n, head * share, min(a.c.channels, (head + 1) * share),
                 [&](int j) { return s_row[j]; });
}

}  // namespace

hipError_t launch_delta_commit(const DeltaCommitArgs& a, hipStream_t s) {
  delta_commit_kernel<<<dim3(a.c.value_heads, a.st.num_seq, a.c.layers), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace w12
