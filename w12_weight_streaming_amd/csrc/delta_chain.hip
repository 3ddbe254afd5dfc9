// The gated delta rule over long chains (gfx950): prompts, and the rows of long
// drafts. The mathematics and the layouts are delta_rule.hip's; rows go through
// in blocks of 32, one state to the next.
//
// What a block needs before its state is known (its rows in LDS, its tiles of L
// and D (q . k), the inverses of the diagonal ones) is made by four waves
// for the next block, while four others take this block from the old state to
// the new one: a workgroup has one wave of each kind on every SIMD, and the
// one fills the other's waits. Blocks of 32 rows rather than 64 let both halves
// of the buffers fit (69 KB), and leave two steps of the triangular system.
#include "delta_rule.h"

namespace w12 {
namespace {

constexpr int kWaves = 4;  // of each kind
constexpr int kThreads = 128 * kWaves;
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
  double sum[R];      // of g from the block's first row
  float beta[R], grow[R], part[R];  // beta, e^G_i, e^(G_n - G_i)
};
template <int KD>
struct Shared {
  Block<KD> block[2];
  uint32_t odd[kStepRows / R], odd_q[kStepRows / R];  // rows of each block, and queries, that hold no numbers
  int bad;
};

// Two neighbouring rows' 8 keys and 8 queries of one thread.
struct Rows {
  uint4 k[2], q[2];
  float gate, beta;
};

template <int KD>
__device__ __forceinline__ void fetch(const DeltaRuleArgs& a, const RowsView& v, int b, int head, int key, int tid, Rows& x) {
  const int last = v.rows - 1, first = b * R;  // rows past the end stand for the last one: no branch, which would wait for the loads
  const int c = min(tid / (R / 2), KD / 8 - 1) * 8, r = (tid % (R / 2)) * 2;
  const uint16_t* kp = a.c.kv + kv_at(a.c, a.layer, v.row0) + (key * KD + c);
  const uint16_t* qp = a.q + ((size_t)v.row0 * a.c.key_heads + key) * KD + c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t at = min(first + r + i, last);
    x.k[i] = *reinterpret_cast<const uint4*>(kp + at * a.c.kv_width);
    x.q[i] = *reinterpret_cast<const uint4*>(qp + at * (a.c.key_heads * KD));
  }
  const float* gp = a.c.gates + gate_at(a.c, a.layer, v.row0, 0, head) + (uint32_t)min(first + (tid & (R - 1)), last) * (2 * a.c.value_heads);
  x.gate = gp[0];
  x.beta = gp[a.c.value_heads];
}

template <int KD>
__device__ __forceinline__ void stage(Shared<KD>& s, const RowsView& v, int b, int tid, Rows& x) {
  using B = Block<KD>;
  B& o = s.block[b & 1];
  const int n = min(R, v.rows - b * R);
  const int c = (tid / (R / 2)) * 8, r = (tid % (R / 2)) * 2;
  if (c < KD) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool no = odd8(x.k[i]), no_q = odd8(x.q[i]);
      if (no && r + i < n) atomicOr(&s.odd[b], 1u << (r + i));
      if (no_q && r + i < n) atomicOr(&s.odd_q[b], 1u << (r + i));
      if (no || r + i >= n) x.k[i] = make_uint4(0, 0, 0, 0);
      if (no_q || r + i >= n) x.q[i] = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(o.k + (r + i) * B::KS + c) = x.k[i];
      *reinterpret_cast<uint4*>(o.q + (r + i) * B::KS + c) = x.q[i];
    }
    store_turned(o.t + c * B::TS + r, B::TS, x.k[0], x.k[1]);
  }
  if (tid < 64) {  // one wave; rows past n decay by nothing
    const bool no = !(x.gate <= 3.4e38f) || odd32(x.beta);
    if (no && tid < n) atomicOr(&s.odd[b], 1u << tid);
    const float gate = no || tid >= n ? 0.0f : x.gate, beta = no || tid >= n ? 0.0f : x.beta;
    double sum = log_decay(gate);
#pragma unroll
    for (int step = 1; step < R; step <<= 1) {
      const double up = __shfl_up(sum, step);
      if (tid >= step) sum += up;
    }
    const double end = __shfl(sum, R - 1);
    if (tid < R) {
      o.sum[tid] = sum;
      o.beta[tid] = beta;
      o.grow[tid] = expf((float)sum);
      o.part[tid] = expf((float)(end - sum));
    }
  }
}

// Tile u of a block: 0, 1 diagonal, 2 the lower one.
template <int KD>
__device__ __forceinline__ void tile(Block<KD>& o, bool of_low, int u) {
  using B = Block<KD>;
  const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4, bi = u ? 1 : 0, bj = u & 1;
  f32x4 x = pair_tile<KD>((of_low ? o.k : o.q) + 16 * bi * B::KS, o.k + 16 * bj * B::KS, B::KS, lane);
  const int i = 16 * bi + col;
  const double gi = o.sum[i];
  const float f = of_low ? -o.beta[i] : 1.0f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int j = 16 * bj + 4 * g + r;
    x[r] = (of_low ? j < i : j <= i) ? f * __expf((float)(gi - o.sum[j])) * x[r] : 0.0f;
  }
  (of_low ? o.low : o.see)[u][lane] = x;
}

template <int KD, int VD>
__global__ __launch_bounds__(kThreads, 2) void delta_chain_kernel(DeltaRuleArgs a) {
  using B = Block<KD>;
  constexpr int KT = KD / 16, slabs = VD / (16 * kWaves);
  __shared__ Shared<KD> s;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hv = a.c.value_heads, head = blockIdx.x / slabs, key = head / (hv / a.c.key_heads), seq = blockIdx.y;
  const int v_slab = (blockIdx.x - head * slabs) * (16 * kWaves), vw = v_slab + (wave & (kWaves - 1)) * 16;
  const RowsView v = rows_view(a.c, a.st, seq);
  if (v.rows == 0) return;
  const bool maker = wave >= kWaves;  // of the next block
  const int blocks = (v.rows + R - 1) / R;
  float* state = a.c.state + state_at(a.c, a.layer, v.slot, head);
  const uint16_t* values = a.c.kv + kv_at(a.c, a.layer, v.row0) + (a.c.key_heads * KD + head * VD);
  if (tid < kStepRows / R) s.odd[tid] = s.odd_q[tid] = 0;
  if (wave == 0) {
    const int bad = refused(a, v, seq, true);
    if ((thread_now() & 63) == 0) s.bad = bad;
  }
  bool before = false;  // a block holds a row that is no number
  // Each turn of either loop has two barriers: the makers' block b + 1 is staged,
  // then made; the others' block b meets the old state, then makes the new one.
  if (maker) {
    Rows x;
    fetch<KD>(a, v, 0, head, key, thread_now() - 64 * kWaves, x);
    __syncthreads();
    if (s.bad) {
      if (!(s.bad & 2)) no_numbers(a, v, head, VD, v_slab, 16 * kWaves);
      return;
    }
    for (int b = 0; b <= blocks; ++b) {
      if (b < blocks) {
        const int me = thread_now() - 64 * kWaves;
        stage<KD>(s, v, b, me, x);
        fetch<KD>(a, v, min(b + 1, blocks - 1), head, key, me, x);
      }
      __syncthreads();
      if (b < blocks) {
        B& o = s.block[b & 1];
        const int u = wave - kWaves;
        if (u < 2) {
          tile<KD>(o, true, u);
          wave_lds_sync();
          invert(o.low[u], o.inv[u], min(R, v.rows - b * R) - 16 * u);
        } else {
          tile<KD>(o, u == 2, 2);
          tile<KD>(o, false, u - 2);
          if (u == 3) tile<KD>(o, false, 2);
        }
      }
      __syncthreads();
    }
  } else {
    f32x4 S[KT][1];
    load_state<KT, VD, 1>(state, vw, S);
    const uint16_t* values = a.c.kv + kv_at(a.c, a.layer, v.row0) + (a.c.key_heads * KD + head * VD);
    uint16_t val[2][4];  // a block's values
    const auto fetch_values = [&](int b) {
      const int lane = thread_now() & 63;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          val[m][r] = values[(uint32_t)min(b * R + 16 * m + 4 * (lane >> 4) + r, v.rows - 1) * a.c.kv_width + vw + (lane & 15)];
    };
    fetch_values(0);
    __syncthreads();
    if (s.bad) {
      if (!(s.bad & 2)) no_numbers(a, v, head, VD, v_slab, 16 * kWaves);
      return;
    }
    __syncthreads();
    __syncthreads();
    for (int b = 0; b < blocks; ++b) {
      B& o = s.block[b & 1];
      const int n = min(R, v.rows - b * R);
      f32x4 rhs[2], acc[2];
      {  // products with the old state
        const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4;
        f32x4 w[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) w[m] = acc[m] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < KT; t += 2) {
          uint4 piece[3];
          split3(S[t][0], S[t + 1][0], piece[0], piece[1], piece[2]);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint4 fk = fragment(o.k + (16 * m + col) * B::KS + 16 * t + 4 * g);
            const uint4 fq = fragment(o.q + (16 * m + col) * B::KS + 16 * t + 4 * g);
#pragma unroll
            for (int p = 2; p >= 0; --p) {
              w[m] = mfma_bf16(fk, piece[p], w[m]);
              acc[m] = mfma_bf16(fq, piece[p], acc[m]);
            }
          }
        }
        uint32_t odd = 0;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = 16 * m + 4 * g + r;
            uint32_t y = val[m][r];
            const bool no = odd16(y);
            if (no && i < n) odd |= 1u << i;
            y = no || i >= n ? 0 : y << 16;
            const float grow = o.grow[i];
            rhs[m][r] = o.beta[i] * (__uint_as_float(y) - grow * w[m][r]);
            acc[m][r] *= grow;
          }
        if (odd) atomicOr(&s.odd[b], odd);
        fetch_values(min(b + 1, blocks - 1));
      }
      __syncthreads();
      {  // the triangular system, the state behind the block, the outputs
        const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4, v0 = vw + col;
        const f32x4 zero = {0, 0, 0, 0};
        const f32x4 d0 = mfma_f32(o.inv[0][lane], rhs[0], zero);
        const f32x4 d1 = mfma_f32(o.inv[1][lane], mfma_f32(o.low[2][lane], d0, rhs[1]), zero);
        if (a.keep || b + 1 < blocks) {
          uint4 piece[3];
          f32x4 y[2];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            y[0][r] = o.part[4 * g + r] * d0[r];
            y[1][r] = o.part[16 + 4 * g + r] * d1[r];
          }
          split3(y[0], y[1], piece[0], piece[1], piece[2]);
          const float keep = o.grow[R - 1];  // rows past n decay by nothing
#pragma unroll
          for (int t = 0; t < KT; ++t) {
            const uint4 f = fragment(o.t + (16 * t + col) * B::TS + 4 * g);
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][0][r] *= keep;
#pragma unroll
            for (int p = 2; p >= 0; --p) S[t][0] = mfma_bf16(f, piece[p], S[t][0]);
          }
        }
        acc[0] = mfma_f32(o.see[0][lane], d0, acc[0]);
        acc[1] = mfma_f32(o.see[1][lane], d1, mfma_f32(o.see[2][lane], d0, acc[1]));
        const uint32_t odd = s.odd[b], odd_q = s.odd_q[b];
        const int row0 = v.row0 + b * R;
        uint16_t* outs = a.out + ((size_t)row0 * hv + head) * VD;
        float* deltas = a.c.delta + delta_at(a.c, a.layer, row0, head);
        const uint32_t step = hv * VD, at0 = 4 * g * step + v0;
        if (n == R && !before && !(odd | odd_q)) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint32_t at = at0 + (16 * m + r) * step;
              outs[at] = (uint16_t)bf16_pair(a.scale * acc[m][r], 0.0f);
              if (!a.keep) deltas[at] = m ? d1[r] : d0[r];
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
      }
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

}  // namespace

hipError_t launch_delta_chain(const DeltaRuleArgs& a, hipStream_t s) {
  const dim3 grid(a.c.value_heads * (a.c.value_dim / (16 * kWaves)), a.st.num_seq);
  if (a.c.key_dim == 64)
    a.c.value_dim == 64 ? delta_chain_kernel<64, 64><<<grid, kThreads, 0, s>>>(a) : delta_chain_kernel<64, 128><<<grid, kThreads, 0, s>>>(a);
  else
    a.c.value_dim == 64 ? delta_chain_kernel<128, 64><<<grid, kThreads, 0, s>>>(a) : delta_chain_kernel<128, 128><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace w12
