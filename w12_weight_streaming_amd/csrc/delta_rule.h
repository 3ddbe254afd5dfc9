// What the delta rule's kernels share (gfx950): the state in registers, the
// look at a sequence, a sequence of one row.
#pragma once

#include "delta_mfma.h"

namespace w12 {

// A kept sequence's window, shared out among the workgroups of its heads.
__device__ __forceinline__ void keep_window(const DeltaRuleArgs& a, const RowsView& v) {
  const int share = (a.c.channels + gridDim.x - 1) / gridDim.x;
  advance_window(a.c, a.layer, v.slot, v.rows, blockIdx.x * share, min(a.c.channels, (int)(blockIdx.x + 1) * share),
                 [&](int j) { return v.row0 + j; });
}

// What a wave looks at to tell whether its sequence is one, the first 64 of
// each: read before the state, whose loads a later one would have to wait for.
struct Look {
  int first, end, slot, parent;
};
__device__ __forceinline__ Look look(const DeltaRuleArgs& a, const RowsView& v) {
  const int lane = thread_now() & 63, j = min(lane, a.st.num_seq - 1);
  Look l;
  l.first = a.st.row_off[j];
  l.end = a.st.row_off[j + 1];
  l.slot = a.st.slot ? a.st.slot[j] : j;
  l.parent = a.st.parent ? a.st.parent[v.row0 + min(lane, v.rows - 1)] : lane - 1;
  return l;
}
// By one wave: 1 if the sequence is refused, 2 if it has no rows.
__device__ __forceinline__ int refused(const DeltaRuleArgs& a, const RowsView& v, int seq, const Look& l) {
  const int lane = thread_now() & 63, last = v.row0 + v.rows;
  bool none = lane < seq && l.first >= 0 && l.end <= a.st.total && l.first < l.end && l.first < last && l.end > v.row0;
  bool bad = !v.ok || (a.keep && lane < seq && l.slot == v.slot) ||
             (lane < v.rows && (lane == 0 ? l.parent != -1 : (l.parent < 0 || l.parent >= lane)));
  for (int j = lane + 64; j < seq; j += 64) {
    none = none || rows_meet(a.st.row_off, a.st.total, j, v.row0, v.rows);
    bad = bad || (a.keep && (a.st.slot ? a.st.slot[j] : j) == v.slot);
  }
  if (a.st.parent)
    for (int i = lane + 64; i < v.rows; i += 64) {
      const int p = a.st.parent[v.row0 + i];
      bad = bad || p < 0 || p >= i;
    }
  return __any(none) ? 2 : __any(bad) ? 1 : 0;
}

// A refused sequence's outputs, `wide` value dims of a head from v0.
__device__ __forceinline__ void no_numbers(const DeltaRuleArgs& a, const RowsView& v, int head, int vd, int v0, int wide) {
  for (int e = thread_now(); e < v.rows * wide; e += blockDim.x)
    a.out[((size_t)(v.row0 + e / wide) * a.c.value_heads + head) * vd + v0 + e % wide] = 0x7FC0;
}

// A sequence's rows one after another (plain decoding: one), each wave by itself
// and without LDS: the products with its columns in fp32, summed over the four
// lanes of a column. Rows follow each other (a tree has one row here).
template <int KD, int VD, int NC>
__device__ __forceinline__ void rows_in_turn(const DeltaRuleArgs& a, const RowsView& v, int seq, int head, int key, int vw,
                                             float* state, const Look& seen, f32x4 (&S)[KD / 16][NC]) {
  constexpr int KT = KD / 16;
  const int lane = thread_now() & 63, g = lane >> 4, v0 = vw + (lane & 15) * NC;
  const int bad = refused(a, v, seq, seen);
  for (int i = 0; i < v.rows; ++i) {
    const int row = v.row0 + i;
    const uint16_t* kp = a.c.kv + kv_at(a.c, a.layer, row) + (key * KD + 4 * g);
    const uint16_t* qp = a.q + ((size_t)row * a.c.key_heads + key) * KD + 4 * g;
    uint2 k[KT], q[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      k[t] = *reinterpret_cast<const uint2*>(kp + 16 * t);
      q[t] = *reinterpret_cast<const uint2*>(qp + 16 * t);
    }
    const uint16_t* vp = a.c.kv + kv_at(a.c, a.layer, row) + (a.c.key_heads * KD + head * VD) + v0;
    const uint32_t val = NC == 2 ? *reinterpret_cast<const uint32_t*>(vp) : *vp;
    const float gate = a.c.gates[gate_at(a.c, a.layer, row, 0, head)], beta = a.c.gates[gate_at(a.c, a.layer, row, 1, head)];
    uint16_t* out = a.out + ((size_t)row * a.c.value_heads + head) * VD + v0;
    if (bad) {
      if (bad == 1 && g == 0)
#pragma unroll
        for (int c = 0; c < NC; ++c) out[c] = 0x7FC0;
      continue;
    }
    const auto at = [](const uint2& x, int r) {
      const uint32_t w = r < 2 ? x.x : x.y;
      return r & 1 ? __uint_as_float(w & 0xFFFF0000u) : __uint_as_float(w << 16);
    };
    float x[NC], o[NC], kq = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) x[c] = o[c] = 0;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float kk = at(k[t], r), qq = at(q[t], r);
        kq += kk * qq;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          x[c] += S[t][c][r] * kk;
          o[c] += S[t][c][r] * qq;
        }
      }
#pragma unroll
    for (int m = 16; m < 64; m <<= 1) {
      kq += __shfl_xor(kq, m);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        x[c] += __shfl_xor(x[c], m);
        o[c] += __shfl_xor(o[c], m);
      }
    }
    const float f = expf(gate);
    float d[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      d[c] = beta * (__uint_as_float(c ? val & 0xFFFF0000u : val << 16) - f * x[c]);
      o[c] = a.scale * (f * o[c] + kq * d[c]);
    }
    if (g == 0) {
      const uint32_t w = bf16_pair(o[0], o[NC - 1]);
      if constexpr (NC == 2)
        *reinterpret_cast<uint32_t*>(out) = w;
      else
        *out = (uint16_t)w;
      if (!a.keep) {
        float* p = a.c.delta + delta_at(a.c, a.layer, row, head) + v0;
#pragma unroll
        for (int c = 0; c < NC; ++c) p[c] = d[c];
      }
    }
    if (a.keep || i + 1 < v.rows) {
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < NC; ++c) S[t][c][r] = f * S[t][c][r] + at(k[t], r) * d[c];
    }
  }
  if (!a.keep || bad) return;
  store_state<KT, VD, NC>(state, vw, S);
  keep_window(a, v);
}

}  // namespace w12
