// Commit of a recurrent layer's accepted rows (gfx950), all layers at once.
//
// A row's delta depends on its ancestors alone, so the deltas that the pass
// computed for an accepted path are those of a replay, and the state behind it is
//   S e^G_n + sum_j k_j (e^(G_n - G_j) delta_j)^T,
// one pass over the state with no product that depends on another. Bound by
// the state's bytes, read and written once: a workgroup holds one head's state
// in registers and adds 32 rows at a time on the matrix cores (most paths are
// one turn), keys as they are (bf16), weighted deltas in three bf16 pieces. 48
// layers of 48 heads of 128 x 128, one sequence: 64 us for 313 MB of states,
// windows and rows (4.9 TB/s); 12 layers of 24 sequences 330 us for 1.87 GB (5.7
// TB/s, where 4 GiB rewritten in place past the caches reach 5.9). With the
// states' traffic through the caches 77 and 389.
#include "delta_mfma.h"

namespace w12 {
namespace {

constexpr int kThreads = 256;
constexpr int kTurn = 32;             // rows a turn
constexpr int kStride = kTurn + 8;    // of a key dim's rows in LDS: 8-byte reads meet no bank twice

// A wave owns NC * 16 of the head's value dims, the lane NC neighbouring ones.
template <int KD, int NC>
__global__ __launch_bounds__(kThreads, 4) void delta_commit_kernel(DeltaCommitArgs a) {
  constexpr int KT = KD / 16, VD = 64 * NC;
  __shared__ alignas(16) uint16_t s_k[KD * kStride];
  __shared__ int s_row[kStepRows];
  __shared__ float s_part[kTurn];
  __shared__ float s_keep;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int head = blockIdx.x, seq = blockIdx.y, layer = blockIdx.z;
  const RowsView v = rows_view(a.c, a.st, seq);
  const int acc = a.accept_len[seq];
  float* state = a.c.state + state_at(a.c, layer, v.slot, head);
  f32x4 S[KT][NC];
  load_state<KT, VD, NC>(state, wave * 16 * NC, S);
  const int n = v.ok ? acc + 1 : 0;
  int bad = (!v.ok || acc < -1 || acc >= v.rows) ? 1 : 0;
  for (int j = tid; j < seq; j += kThreads) {
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
  bad = __syncthreads_or(bad);
  if (tid == 0 && head == 0 && layer == 0) a.kept[seq] = bad ? -1 : n;
  if (bad || n == 0) return;
  const int share = (a.c.channels + gridDim.x - 1) / gridDim.x;
  advance_window(a.c, layer, v.slot, n, head * share, min(a.c.channels, (head + 1) * share),
                 [&](int j) { return s_row[j]; });

  const int key = head / (a.c.value_heads / a.c.key_heads);
  for (int j0 = 0; j0 < n; j0 += kTurn) {
    const int m = min(kTurn, n - j0);
    f32x4 d[2][NC];
    {
      const int lane = thread_now() & 63, at = (wave * 16 + (lane & 15)) * NC;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * i + 4 * (lane >> 4) + r;
          const float* p = a.c.delta + delta_at(a.c, layer, s_row[j0 + min(j, m - 1)], head) + at;
#pragma unroll
          for (int c = 0; c < NC; ++c) d[i][c][r] = j < m ? p[c] : 0.0f;
        }
    }
    if (j0 > 0) __syncthreads();
    for (int e = thread_now(); e < (kTurn / 2) * (KD / 8); e += kThreads) {
      const int r = (e % (kTurn / 2)) * 2, c = (e / (kTurn / 2)) * 8;
      uint4 x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        x[i] = r + i < m ? *reinterpret_cast<const uint4*>(a.c.kv + kv_at(a.c, layer, s_row[j0 + r + i]) + (size_t)key * KD + c)
                         : make_uint4(0, 0, 0, 0);
      store_turned(s_k + c * kStride + r, kStride, x[0], x[1]);
    }
    if (const int lane = thread_now(); lane < kTurn) {  // decays to the turn's end, summed along the path in 64 bits
      double sum = lane < m ? log_decay(a.c.gates[gate_at(a.c, layer, s_row[j0 + lane], 0, head)]) : 0.0;
#pragma unroll
      for (int step = 1; step < kTurn; step <<= 1) {
        const double up = __shfl_up(sum, step);
        if (lane >= step) sum += up;
      }
      const double end = __shfl(sum, kTurn - 1);
      s_part[lane] = expf((float)(end - sum));
      if (lane == 0) s_keep = expf((float)end);
    }
    __syncthreads();
    const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4;
    const float keep = s_keep;
    uint4 piece[NC][3];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) d[i][c][r] *= s_part[16 * i + 4 * g + r];
      split3(d[0][c], d[1][c], piece[c][0], piece[c][1], piece[c][2]);
    }
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const uint4 f = fragment(s_k + (16 * t + col) * kStride + 4 * g);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
f32x4 add = {0, 0, 0, 0};
#pragma unroll
        for (int p = 2; p >= 0; --p) add = mfma_bf16(f, piece[c][p], add);
        join_state(S[t][c], keep, add);
        asm volatile("" : "+v"(S[t][c]));  // keeps its place among the products: else 157 registers and 354 us for 12 x 24
      }
    }
  }
  store_state<KT, VD, NC>(state, wave * 16 * NC, S);
}

}  // namespace

hipError_t launch_delta_commit(const DeltaCommitArgs& a, hipStream_t s) {
  const dim3 grid(a.c.value_heads, a.st.num_seq, a.c.layers);
  if (a.c.key_dim == 64)
    a.c.value_dim == 64 ? delta_commit_kernel<64, 1><<<grid, kThreads, 0, s>>>(a) : delta_commit_kernel<64, 2><<<grid, kThreads, 0, s>>>(a);
  else
    a.c.value_dim == 64 ? delta_commit_kernel<128, 1><<<grid, kThreads, 0, s>>>(a) : delta_commit_kernel<128, 2><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace w12
