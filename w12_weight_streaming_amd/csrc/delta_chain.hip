// The gated delta rule over long chains (gfx950): prompts, and the rows of long
// drafts. The mathematics and the layouts are delta_rule.hip's; rows go through
// in blocks of 32, one state to the next.
//
// What a block needs before its state is known (its rows in LDS, its tiles of L
// and D (q . k), the inverses of the diagonal ones) is made by four waves
// for the next block, while the others take this block from the old state to
// the new one, 16 value dims a wave: the two fill each other's waits. Blocks of
// 32 rows rather than 64 let both halves of the buffers fit (82 KB), and leave
// two steps of the triangular system. 512 rows of 16 key and 48 value heads of
// 128 x 128: 46 us, 2.9 a block, of which the takers' products with the state take
// 1.2 and the system, the new state and the outputs 1.6 (the way from state to
// state bounds it, not a rate: the rule's own 6 operations a row and entry of the
// state are 2.4 GFLOP, at 53 TFLOP/s). Makers need at most 2.2 of it.
#include "delta_rule.h"

namespace w12 {
namespace {

constexpr int kMakers = 4;  // waves
constexpr int R = 32;

template <int KD>
struct Block {
  static constexpr int KS = KD + 8, TS = R + 8;  // rows 4 banks (of 64) further each: 8-byte reads meet none twice
  alignas(16) uint16_t q[R * KS];
  alignas(16) uint16_t k[R * KS];
  alignas(16) uint16_t t[KD * TS];  // k with rows innermost
  f32x4 low[3][64];   // tiles (0, 0), (1, 1), (1, 0) of -L, and
  f32x4 see[3][64];   // of D (q . k)
  f32x4 inv[2][64];   // (I + L)^-1 of the diagonal ones
};
template <int KD>
struct Shared {
  Block<KD> block[2];
  // by the sequence's row; rows past the end decay by nothing and have no strength
  alignas(16) double sum[kStepRows];     // of g from the block's first row
  alignas(16) float beta[kStepRows], grow[kStepRows], part[kStepRows];  // beta, e^G_i, e^(G_n - G_i)
  uint32_t odd[kStepRows / R], odd_q[kStepRows / R];  // rows of each block, and queries, that hold no numbers
  int bad;
};

// Two neighbouring rows' 8 keys and 8 queries of one thread.
struct Rows {
  uint4 k[2], q[2];
};

// kv: the key head's values of the sequence's first row; rows past the end
// stand for the last one (a branch would wait for the loads).
template <int KD>
__device__ __forceinline__ void fetch(const uint16_t* kv, int kv_step, const uint16_t* q, int q_step, int first, int last, int tid, Rows& x) {
  const int c = min(tid / (R / 2), KD / 8 - 1) * 8, r = first + (tid % (R / 2)) * 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = min(r + i, last);
    x.k[i] = *reinterpret_cast<const uint4*>(behind(kv, 2 * (__umul24(at, kv_step) + c)));
    x.q[i] = *reinterpret_cast<const uint4*>(behind(q, 2 * (__umul24(at, q_step) + c)));
  }
}

template <int KD>
__device__ __forceinline__ void stage(Shared<KD>& s, int b, int n, int tid, Rows& x) {
  using B = Block<KD>;
  B& o = s.block[b & 1];
  const int c = (tid / (R / 2)) * 8, r = (tid % (R / 2)) * 2;
  if (c >= KD) return;
  if (n < R) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (r + i >= n) x.k[i] = x.q[i] = make_uint4(0, 0, 0, 0);
  }
  if (is_odd(odd_sum(x.k[0]) | odd_sum(x.k[1]) | odd_sum(x.q[0]) | odd_sum(x.q[1]))) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (is_odd(odd_sum(x.k[i]))) {
        atomicOr(&s.odd[b], 1u << (r + i));
        x.k[i] = make_uint4(0, 0, 0, 0);
      }
      if (is_odd(odd_sum(x.q[i]))) {
        atomicOr(&s.odd_q[b], 1u << (r + i));
        x.q[i] = make_uint4(0, 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    *reinterpret_cast<uint4*>(o.k + (r + i) * B::KS + c) = x.k[i];
    *reinterpret_cast<uint4*>(o.q + (r + i) * B::KS + c) = x.q[i];
  }
  store_turned(o.t + c * B::TS + r, B::TS, x.k[0], x.k[1]);
}

// Decays and strengths of all rows, 64 a wave: sums along each block.
template <int KD>
__device__ __forceinline__ void gates(const DeltaRuleArgs& a, Shared<KD>& s, const RowsView& v, int head, int blocks, int wave) {
  for (int i0 = wave * 64; i0 < blocks * R; i0 += kMakers * 64) {
    const int lane = thread_now() & 63, i = i0 + lane, row = lane & (R - 1);
    float gate = 0.0f, beta = 0.0f;
    if (i < v.rows) {
      gate = a.c.gates[gate_at(a.c, a.layer, v.row0 + i, 0, head)];
      beta = a.c.gates[gate_at(a.c, a.layer, v.row0 + i, 1, head)];
      if (!(gate <= 3.4e38f) || odd32(beta)) {
        atomicOr(&s.odd[i / R], 1u << row);
        gate = beta = 0.0f;
      }
    }
    double sum = log_decay(gate);
#pragma unroll
    for (int step = 1; step < R; step <<= 1) {
      const double up = __shfl_up(sum, step, R);
      if (row >= step) sum += up;
    }
    const double end = __shfl(sum, R - 1, R);
    s.sum[i] = sum;  // i < 512: 64 divides it
    s.beta[i] = beta;
    s.grow[i] = expf((float)sum);
    s.part[i] = expf((float)(end - sum));
  }
}

// Tile u of a block: 0, 1 diagonal, 2 the lower one.
template <int KD>
__device__ __forceinline__ void tile(const Shared<KD>& s, Block<KD>& o, int first, bool of_low, int u) {
  using B = Block<KD>;
  const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4, bi = u ? 1 : 0, bj = u & 1;
  const double* sj = s.sum + first + 16 * bj + 4 * g;
  const double gi = s.sum[first + 16 * bi + col];
  float f[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) f[r] = (float)(gi - sj[r]);
  const float beta = -s.beta[first + 16 * bi + col];
  f32x4 x = pair_tile<KD>((of_low ? o.k : o.q) + 16 * bi * B::KS, o.k + 16 * bj * B::KS, B::KS, lane);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int over = u == 2 ? 1 : col - (4 * g + r);  // how far row i lies behind row j
    // (__expf: off by about |f| 2^-23 of itself, as much as f's own rounding to fp32)
    x[r] = (of_low ? over > 0 : over >= 0) ? (of_low ? beta * x[r] : x[r]) * __expf(f[r]) : 0.0f;
  }
  (of_low ? o.low : o.see)[u][lane] = x;
}

template <int KD, int VD, int kTakers>
__global__ __launch_bounds__(64 * (kMakers + kTakers)) __attribute__((amdgpu_waves_per_eu(2, 2))) void delta_chain_kernel(DeltaRuleArgs a) {
  using B = Block<KD>;
  constexpr int KT = KD / 16, slabs = VD / (16 * kTakers);
  __shared__ Shared<KD> s;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hv = a.c.value_heads, head = blockIdx.x / slabs, key = head / (hv / a.c.key_heads), seq = blockIdx.y;
  const int v_slab = (blockIdx.x - head * slabs) * (16 * kTakers);
  const RowsView v = rows_view(a.c, a.st, seq);
  if (v.rows == 0) return;
  const int blocks = (v.rows + R - 1) / R;
  if (tid < kStepRows / R) s.odd[tid] = s.odd_q[tid] = 0;
  if (wave == 0) {
    const int bad = refused(a, v, seq, look(a, v));
    if ((thread_now() & 63) == 0) s.bad = bad;
  }
  bool before = false;  // a block holds a row that is no number
  const uint16_t* kv = a.c.kv + kv_at(a.c, a.layer, v.row0);
  float* state = a.c.state + state_at(a.c, a.layer, v.slot, head);
  // The makers' turn b + 1 goes with the others' turn b: rows are staged while
  // the block before meets its state, tiles are made while it makes the next.
  if (wave >= kTakers) {
    const int mw = wave - kTakers;
    const uint16_t *keys = kv + key * KD, *queries = a.q + ((size_t)v.row0 * a.c.key_heads + key) * KD;
    Rows x;
    fetch<KD>(keys, a.c.kv_width, queries, a.c.key_heads * KD, 0, v.rows - 1, thread_now() - 64 * kTakers, x);
    __syncthreads();
    if (s.bad) {
      if (!(s.bad & 2)) no_numbers(a, v, head, VD, v_slab, 16 * kTakers);
      return;
    }
    gates<KD>(a, s, v, head, blocks, mw);
    for (int b = 0; b <= blocks; ++b) {
      if (b < blocks) {
        const int me = thread_now() - 64 * kTakers;
        stage<KD>(s, b, v.rows - b * R, me, x);
        fetch<KD>(keys, a.c.kv_width, queries, a.c.key_heads * KD, (b + 1) * R, v.rows - 1, me, x);
      }
      __syncthreads();
      if (b < blocks) {
        B& o = s.block[b & 1];
        if (mw < 2) {
          tile<KD>(s, o, b * R, true, mw);
          wave_lds_sync();
          invert<true>(o.low[mw], o.inv[mw], 16);
        } else {  // the lower tile of L and of D (q . k), then the diagonal ones of the latter
          tile<KD>(s, o, b * R, mw == 2, 2);
          tile<KD>(s, o, b * R, false, mw - 2);
        }
      }
      __syncthreads();
    }
  } else {
    const int vw = v_slab + wave * 16;
    f32x4 S[KT][1];
    load_state<KT, VD, 1>(state, vw, S);
    const uint16_t* values = kv + (a.c.key_heads * KD + head * VD + vw);
    uint32_t val[2][4];  // a block's values
    const auto fetch_values = [&](int first) {
      const int lane = thread_now() & 63;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          val[m][r] = *behind(values, 2 * (__umul24(min(first + 16 * m + 4 * (lane >> 4) + r, v.rows - 1), a.c.kv_width) + (lane & 15)));
    };
    fetch_values(0);
    __syncthreads();
    if (s.bad) {
      if (!(s.bad & 2)) no_numbers(a, v, head, VD, v_slab, 16 * kTakers);
      return;
    }
    __syncthreads();
    __syncthreads();
    for (int b = 0; b < blocks; ++b) {
      B& o = s.block[b & 1];
      const int n = min(R, v.rows - b * R);
      const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4;
      f32x4 rhs[2], acc[2];
      // products with the old state
      {
        uint4 fk[2][KT / 2], fq[2][KT / 2];
#pragma unroll
        for (int t = 0; t < KT / 2; ++t)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            fk[m][t] = fragment(o.k + (16 * m + col) * B::KS + 32 * t + 4 * g);
            fq[m][t] = fragment(o.q + (16 * m + col) * B::KS + 32 * t + 4 * g);
          }
        f32x4 w[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) w[m] = acc[m] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < KT / 2; ++t) {
          uint4 piece[3];
          split3(S[2 * t][0], S[2 * t + 1][0], piece[0], piece[1], piece[2]);
#pragma unroll
          for (int p = 2; p >= 0; --p)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              w[m] = mfma_bf16(fk[m][t], piece[p], w[m]);
              acc[m] = mfma_bf16(fq[m][t], piece[p], acc[m]);
            }
        }
        uint32_t sums = 0;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) sums |= odd_sum(val[m][r]);
        if (is_odd(sums)) {
          uint32_t odd = 0;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (is_odd(odd_sum(val[m][r]))) {
                const int i = 16 * m + 4 * g + r;
                if (i < n) odd |= 1u << i;
                val[m][r] = 0;
              }
          if (odd) atomicOr(&s.odd[b], odd);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int i = b * R + 16 * m + 4 * g;
          const f32x4 grow = *reinterpret_cast<const f32x4*>(s.grow + i), beta = *reinterpret_cast<const f32x4*>(s.beta + i);
#pragma unroll
          for (int r = 0; r < 4; ++r) {  // rows past the end have no strength
            rhs[m][r] = beta[r] * (__uint_as_float(val[m][r] << 16) - grow[r] * w[m][r]);
            acc[m][r] *= grow[r];
          }
        }
        fetch_values((b + 1) * R);
      }
      __syncthreads();
      // the triangular system, the state behind the block, the outputs
      const f32x4 inv0 = o.inv[0][lane], inv1 = o.inv[1][lane], low2 = o.low[2][lane];
      const f32x4 see0 = o.see[0][lane], see1 = o.see[1][lane], see2 = o.see[2][lane];
      uint4 ft[KT];
#pragma unroll
      for (int t = 0; t < KT; ++t) ft[t] = fragment(o.t + (16 * t + col) * B::TS + 4 * g);
      const f32x4 zero = {0, 0, 0, 0};
      const f32x4 d0 = mfma_f32(inv0, rhs[0], zero);
      const f32x4 d1 = mfma_f32(inv1, mfma_f32(low2, d0, rhs[1]), zero);
      acc[0] = mfma_f32(see0, d0, acc[0]);
      acc[1] = mfma_f32(see2, d0, acc[1]);
      if (a.keep || b + 1 < blocks) {
        const f32x4 p0 = *reinterpret_cast<const f32x4*>(s.part + b * R + 4 * g), p1 = *reinterpret_cast<const f32x4*>(s.part + b * R + 16 + 4 * g);
        uint4 piece[3];
        split3(p0 * d0, p1 * d1, piece[0], piece[1], piece[2]);
        const float keep = s.grow[b * R + R - 1];  // rows past the end decay by nothing
        f32x4 add[KT];
#pragma unroll
        for (int t = 0; t < KT; ++t) add[t] = mfma_bf16(ft[t], piece[2], zero);
#pragma unroll
        for (int p = 1; p >= 0; --p)
#pragma unroll
          for (int t = 0; t < KT; ++t) add[t] = mfma_bf16(ft[t], piece[p], add[t]);
#pragma unroll
        for (int t = 0; t < KT; ++t) join_state(S[t][0], keep, add[t]);
      }
      acc[1] = mfma_f32(see1, d1, acc[1]);
      const uint32_t odd = s.odd[b], odd_q = s.odd_q[b];
      const int row0 = v.row0 + b * R;
      uint16_t* outs = a.out + ((size_t)row0 * hv + head) * VD + vw;
      float* deltas = a.c.delta + delta_at(a.c, a.layer, row0, head) + vw;
      const uint32_t step = hv * VD, at0 = 4 * g * step + col;
      if (n == R && !before && !(odd | odd_q)) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t at = at0 + (16 * m + r) * step;
            *behind(outs, 2 * at) = (uint16_t)bf16_pair(a.scale * acc[m][r], 0.0f);
            if (!a.keep) *behind(deltas, 4 * at) = m ? d1[r] : d0[r];
          }
      } else {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = 16 * m + 4 * g + r;
            if (i < n) {
              const bool no = before || (odd & ((2u << i) - 1));
              const uint32_t at = at0 + (16 * m + r) * step;
              outs[at] = no || ((odd_q >> i) & 1) ? 0x7FC0 : (uint16_t)bf16_pair(a.scale * acc[m][r], 0.0f);
              if (!a.keep) deltas[at] = no ? __builtin_nanf("") : m ? d1[r] : d0[r];
            }
          }
      }
      before = before || odd;
      __syncthreads();
    }
    if (a.keep) {
      if (before) {
#pragma unroll
        for (int t = 0; t < KT; ++t) S[t][0] = f32x4{__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};
      }
      store_state<KT, VD, 1>(state, vw, S);
    }
  }
  if (a.keep) keep_window(a, v);
}

template <int KD, int VD, int kTakers>
void go(const DeltaRuleArgs& a, hipStream_t s) {
  delta_chain_kernel<KD, VD, kTakers><<<dim3(a.c.value_heads * (VD / (16 * kTakers)), a.st.num_seq), 64 * (kMakers + kTakers), 0, s>>>(a);
}
template <int KD, int VD>
hipError_t launch(const DeltaRuleArgs& a, hipStream_t s) {
  // two takers where that leaves a CU for each workgroup, as fewer waves share a
  // SIMD: 1 x 512 rows 46 us against 50, 1 x 32 8.5 against 9.0; 2 x 256 50 against
  // 31, 2 x 64 20.3 against 12.5
  if (a.c.value_heads * (VD / 32) * a.st.num_seq <= 256)
    go<KD, VD, 2>(a, s);
  else
    go<KD, VD, 4>(a, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_chain(const DeltaRuleArgs& a, hipStream_t s) {
  if (a.c.key_dim == 64) return a.c.value_dim == 64 ? launch<64, 64>(a, s) : launch<64, 128>(a, s);
  return a.c.value_dim == 64 ? launch<128, 64>(a, s) : launch<128, 128>(a, s);
}

}  // namespace w12
