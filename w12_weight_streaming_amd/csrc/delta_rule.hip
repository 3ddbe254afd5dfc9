// The gated delta rule over a step's rows (gfx950).
//
// Along a row's root path S <- e^g S; delta = beta (v - S^T k); S <- S + k
// delta^T; out = scale S^T q. With S0 the state before a block of rows, G_i the
// sum of g over row i's path within reach, and D_ij = e^(G_i - G_j) where j lies
// on i's path, the rows of a block answer a triangular system at once:
//   (I + L) delta = rhs,  rhs_i = beta_i (v_i - e^G_i S0^T k_i),
//   L_ij = beta_i D_ij (k_i . k_j), j before i,
//   out_i = scale (e^G_i S0^T q_i + sum_j D_ij (q_i . k_j) delta_j).
// Parents come before their children, so L is lower triangular for trees as
// for chains; the mask alone differs. Chains go from block to block by the
// state behind the block, S0 <- e^G_n S0 + sum_j k_j (e^(G_n - G_j) delta_j)^T;
// rows of a tree have no such state in common, and add what the rows of
// earlier blocks on their path contribute, from the deltas those left.
//
// Value dims are independent of each other: a wave owns NC times 16 of them,
// and holds its columns of S0 in registers, in the layout in which the matrix
// core leaves a result (lane l: column l % 16, rows 4 (l / 16) + r). That is
// also an operand's layout when the other operand takes its depth in the same
// order, so states, deltas and products pass from one product into the next
// without leaving the registers.
//
// Precision: q and k are bf16 and enter as they are. A state or delta (fp32)
// enters a bf16 product as three bf16 pieces, each the top of what the one
// before left, which hold all its 24 bits; products of two fp32 factors (L and
// D (q . k) with deltas) run on the fp32 matrix core. Sums of g are held in 64 bits.
#include "delta_mfma.h"

namespace w12 {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;

// An infinity or NaN among 8 bf16 values.
__device__ __forceinline__ bool odd16(uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; }
__device__ __forceinline__ bool odd8(const uint4& x) { return odd16(x.x) || odd16(x.y) || odd16(x.z) || odd16(x.w); }
__device__ __forceinline__ bool odd32(float x) { return !(fabsf(x) <= 3.4e38f); }

template <int KD, int RT>
struct Shared {
  static constexpr int R = 16 * RT;
  static constexpr int KS = KD + 16;                // row of q and k: 8 rows of 8-byte reads meet no bank twice
  static constexpr int TS = RT == 1 ? 16 : R + 16;  // the same for a key dim's rows
  alignas(16) uint16_t q[R * KS];
  alignas(16) uint16_t k[R * KS];
  // chains: k with rows innermost; trees: the rows of an earlier block
  alignas(16) uint16_t t[KD * TS > R * KS ? KD * TS : R * KS];
  f32x4 low[RT * RT][64];   // tiles of -L, and
  f32x4 see[RT * RT][64];   // of D (q . k): lane (g, i) holds row i, columns 4 g + r
  f32x4 far_low[RT * RT][64], far_see[RT * RT][64];  // the same against an earlier block of a tree
  f32x4 inv[RT][64];        // (I + L)^-1 of the diagonal tiles
  double sum[kStepRows];                // of g from the state (chains: the block) to the row
  unsigned long long in[kStepRows];     // the row's path within its block, itself included
  int leave[kStepRows];                 // the row above that, in an earlier block, or below 0
  unsigned long long odd[kStepRows / R];  // rows of each block that hold no numbers; of a tree's earlier blocks, those behind such rows too
  unsigned long long odd_q;             // queries of the block that are no numbers
  unsigned long long cross[R];          // the path's rows in an earlier block
  int next[R];                          // where the path leaves that block
  int behind[R];                        // a row on the path in an earlier block holds no number
  float beta[R], grow[R], part[R];      // beta, e^G_i, e^(G_n - G_j)
  int bad;
};

// Rows of q and k (k from an earlier block: q null) into LDS, rows past `n` zero. A row with an infinity or
// NaN is marked, and zeros stand in for it: its outputs are set apart from the products.
template <int KD, int RT, bool KT>
__device__ __forceinline__ void load_rows(const DeltaRuleArgs& a, Shared<KD, RT>& s, int row0, int n, int key, uint16_t* kdst,
                                          unsigned long long* odd) {
  using Sh = Shared<KD, RT>;
  constexpr int kPairs = Sh::R / 2, kChunks = KD / 8;
  for (int e = thread_now(); e < kPairs * kChunks; e += kThreads) {
    const int r = (e % kPairs) * 2, c = (e / kPairs) * 8;
    uint4 x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[i] = make_uint4(0, 0, 0, 0);
      if (r + i < n) {
        x[i] = *reinterpret_cast<const uint4*>(a.c.kv + kv_at(a.c, a.layer, row0 + r + i) + (size_t)key * KD + c);
        if (odd8(x[i])) {
          atomicOr(odd, 1ull << (r + i));
          x[i] = make_uint4(0, 0, 0, 0);
        }
      }
      *reinterpret_cast<uint4*>(kdst + (r + i) * Sh::KS + c) = x[i];
    }
    if constexpr (KT) store_turned(s.t + c * Sh::TS + r, Sh::TS, x[0], x[1]);
  }
}
template <int KD, int RT>
__device__ __forceinline__ void load_queries(const DeltaRuleArgs& a, Shared<KD, RT>& s, int row0, int n, int key) {
  using Sh = Shared<KD, RT>;
  constexpr int kChunks = KD / 8;
  for (int e = thread_now(); e < Sh::R * kChunks; e += kThreads) {
    const int r = e / kChunks, c = (e % kChunks) * 8;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r < n) {
      x = *reinterpret_cast<const uint4*>(a.q + ((size_t)(row0 + r) * a.c.key_heads + key) * KD + c);
      if (odd8(x)) {
        atomicOr(&s.odd_q, 1ull << r);
        x = make_uint4(0, 0, 0, 0);
      }
    }
    *reinterpret_cast<uint4*>(s.q + r * Sh::KS + c) = x;
  }
}

// One tile (row tile bi of `x`, row tile bj of `k`) of x . k, transposed: lane (g, i) holds row i, columns 4 g + r.
template <int KD, int RT>
__device__ __forceinline__ f32x4 pair_tile(const uint16_t* x, const uint16_t* k, int bi, int bj) {
  constexpr int KS = Shared<KD, RT>::KS;
  const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4;
  f32x4 acc = {0, 0, 0, 0};
#pragma unroll
  for (int t = 0; t < KD / 32; ++t)
    acc = mfma_bf16(fragment(k + (16 * bj + col) * KS + 32 * t + 4 * g), fragment(x + (16 * bi + col) * KS + 32 * t + 4 * g), acc);
  return acc;
}

// (I + L)^-1 of a diagonal tile from -L, a column per lane of the first 16, forward substitution.
__device__ __forceinline__ void invert(const f32x4* low, f32x4* inv, int n) {
  const int lane = thread_now() & 63, c = lane & 15;
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float y = i == c ? 1.0f : 0.0f;
    if (i < n)  // the same for all lanes
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (4 * g < i) {
        const f32x4 l = low[g * 16 + i];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (4 * g + r < i) y += l[r] * x[4 * g + r];
      }
    }
    x[i] = y;
    if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // all rows of L at once would take 160 registers
  }
  if (lane < 16) {
    float* o = reinterpret_cast<float*>(inv);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[((c >> 2) * 16 + i) * 4 + (c & 3)] = x[i];
  }
}

template <int KD, int VD, int RT, int NC>
__global__ __launch_bounds__(kThreads, RT == 1 ? 4 : RT == 2 ? 2 : 1) void delta_rule_kernel(DeltaRuleArgs a) {
  using Sh = Shared<KD, RT>;
  constexpr int R = Sh::R, KS = Sh::KS, TS = Sh::TS, KT = KD / 16;
  __shared__ Sh s;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hv = a.c.value_heads;
  constexpr int slabs = VD / (kWaves * 16 * NC);
  const int head = blockIdx.x / slabs, key = head / (hv / a.c.key_heads), seq = blockIdx.y;
  const int vw = (blockIdx.x - head * slabs) * (kWaves * 16 * NC) + wave * (16 * NC);  // the wave's first value dim
  const RowsView v = rows_view(a.c, a.st, seq);
  if (v.rows == 0) return;
  if (tid < kStepRows / R) s.odd[tid] = 0;
  if (tid == 0) s.odd_q = 0, s.bad = 0;

  // addresses: a uniform part, and the lane's in 32 bits
  float* state = a.c.state + state_at(a.c, a.layer, v.slot, head);
  const auto state_place = [&]() {
    const int lane = thread_now() & 63;
    return (uint32_t)(4 * (lane >> 4) * VD + vw + (lane & 15) * NC);
  };
  f32x4 S[KT][NC];
  const uint32_t at_state = state_place();
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float* p = state + (16 * t + r) * VD + at_state;
      if constexpr (NC == 2) {
        const float2 x = *reinterpret_cast<const float2*>(p);
        S[t][0][r] = x.x;
        S[t][1][r] = x.y;
      } else {
        S[t][0][r] = *p;
      }
    }
  __syncthreads();
  {  // is the sequence one? 1: NaN, 2: no rows
    int bad = v.ok ? 0 : 1;
    for (int j = tid; j < seq; j += kThreads) {
      if (rows_meet(a.st.row_off, a.st.total, j, v.row0, v.rows)) bad |= 2;
      if (a.keep && a.st.slot && a.st.slot[j] == v.slot) bad |= 1;
    }
    if (a.st.parent)
      for (int i = tid; i < v.rows; i += kThreads) {
        const int p = a.st.parent[v.row0 + i];
        if (i == 0 ? p != -1 : (p < 0 || p >= i)) bad |= 1;
      }
    if (bad) atomicOr(&s.bad, bad);
  }
  const bool chain = !a.st.parent;
  const int blocks = (v.rows + R - 1) / R;
  bool before = false;  // chains: an earlier block holds a row that is no number
  for (int b = 0; b < blocks; ++b) {
    const int row0 = v.row0 + b * R, n = min(R, v.rows - b * R);
    if (b > 0) {
      __syncthreads();
      if (tid == 0) s.odd_q = 0;
      if (!chain && wave == 0) {
        const int lane = thread_now();
        const bool no = lane < R && ((s.in[(b - 1) * R + min(lane, R - 1)] & s.odd[b - 1]) || s.behind[min(lane, R - 1)]);
        const unsigned long long all = __ballot(no);
        if (lane == 0) s.odd[b - 1] = all;
      }
      __syncthreads();
    }
    if (chain)
      load_rows<KD, RT, true>(a, s, row0, n, key, s.k, &s.odd[b]);
    else
      load_rows<KD, RT, false>(a, s, row0, n, key, s.k, &s.odd[b]);
    load_queries<KD, RT>(a, s, row0, n, key);
    // values, in the layout of the products
    f32x4 rhs[RT][NC];
    {
      const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4, v0 = vw + col * NC;
      unsigned long long odd = 0;
      const uint16_t* values = a.c.kv + kv_at(a.c, a.layer, row0) + (a.c.key_heads * KD + head * VD);
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * m + 4 * g + r;
          const uint16_t* p = values + ((uint32_t)min(i, n - 1) * a.c.kv_width + v0);
          uint32_t x = NC == 2 ? *reinterpret_cast<const uint32_t*>(p) : *p;
          if (odd16(x) && i < n) odd |= 1ull << i;
          if (odd16(x) || i >= n) x = 0;
          rhs[m][0][r] = __uint_as_float(x << 16);
          if constexpr (NC == 2) rhs[m][1][r] = __uint_as_float(x & 0xFFFF0000u);
        }
      if (odd) atomicOr(&s.odd[b], odd);
    }
    if (const int lane = thread_now(); lane < R) {  // paths within the block, by doubling; a lane is a row
      float gate = 0, beta = 0;
      int cur = -1, leave = -1;
      if (lane < n) {
        gate = a.c.gates[gate_at(a.c, a.layer, row0 + lane, 0, head)];
        beta = a.c.gates[gate_at(a.c, a.layer, row0 + lane, 1, head)];
        if (!(gate <= 3.4e38f) || odd32(beta)) {
          atomicOr(&s.odd[b], 1ull << lane);
          gate = beta = 0;
        }
        const int i = b * R + lane;
        int p = chain ? (lane > 0 ? i - 1 : -1) : a.st.parent[row0 + lane];
        if (p >= i) p = -1;  // no tree: reported, once every row has been looked at
        cur = p - b * R;
        leave = p;
      }
      double sum = log_decay(gate);
      unsigned long long in = 1ull << lane;
      for (int step = 1; step < R; step <<= 1) {
        const int from = max(cur, 0);
        const double up_sum = __shfl(sum, from);
        const unsigned long long up_in = __shfl(in, from);
        const int up_cur = __shfl(cur, from), up_leave = __shfl(leave, from);
        if (cur >= 0) {
          sum += up_sum;
          in |= up_in;
          cur = up_cur;
          leave = up_leave;
        }
      }
      if (!chain && leave >= 0) sum += s.sum[leave];
      const int at = chain ? lane : b * R + lane;
      s.sum[at] = sum;
      s.in[at] = in;
      s.leave[at] = leave;
      s.next[lane] = leave;
      s.behind[lane] = 0;
      s.beta[lane] = beta;
      const double end = __shfl(sum, n - 1);
      s.grow[lane] = expf((float)sum);
      s.part[lane] = lane < n ? expf((float)(end - sum)) : 0.0f;
    }
    __syncthreads();
    if (s.bad) {
      if (!(s.bad & 2))
        for (int e = thread_now(); e < v.rows * (64 * NC); e += kThreads)
          a.out[((size_t)(v.row0 + e / (64 * NC)) * hv + head) * VD + (vw - wave * (16 * NC)) + e % (64 * NC)] = 0x7FC0;
      return;
    }
    const int base = chain ? 0 : b * R;  // where the block's rows stand in the tables

    // tiles of the block: diagonal ones of L first, each inverted by the wave that made it
    const auto tile = [&](bool of_low, int bi, int bj) {
      f32x4 x = pair_tile<KD, RT>(of_low ? s.k : s.q, s.k, bi, bj);
      const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4;
      const int i = 16 * bi + col;
      const unsigned long long in = s.in[base + i];
      const double gi = s.sum[base + i];
      const float f = of_low ? -s.beta[i] : 1.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * bj + 4 * g + r;
        const bool on = ((in >> j) & 1) && !(of_low && i == j);
        x[r] = on ? f * __expf((float)(gi - s.sum[base + j])) * x[r] : 0.0f;
      }
      (of_low ? s.low : s.see)[bi * RT + bj][lane] = x;
    };
    if (wave < RT) {
      tile(true, wave, wave);
      wave_lds_sync();
      invert(s.low[wave * RT + wave], s.inv[wave], n - 16 * wave);
    }
    {
      int u = RT;
#pragma unroll
      for (int bi = 0; bi < RT; ++bi)
#pragma unroll
        for (int bj = 0; bj <= bi; ++bj) {
          if (bj < bi && (u++ & 3) == wave) tile(true, bi, bj);
          if ((u++ & 3) == wave) tile(false, bi, bj);
        }
    }

    // the rows' products with the old state
    f32x4 acc[RT][NC];
    {
      const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4;
      f32x4 w[RT][NC];
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int c = 0; c < NC; ++c) w[m][c] = acc[m][c] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < KT; t += 2) {
        uint4 piece[NC][3];
#pragma unroll
        for (int c = 0; c < NC; ++c) split3(S[t][c], S[t + 1][c], piece[c][0], piece[c][1], piece[c][2]);
#pragma unroll
        for (int m = 0; m < RT; ++m) {
          const uint4 fk = fragment(s.k + (16 * m + col) * KS + 16 * t + 4 * g);
          const uint4 fq = fragment(s.q + (16 * m + col) * KS + 16 * t + 4 * g);
#pragma unroll
          for (int p = 2; p >= 0; --p)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              w[m][c] = mfma_bf16(fk, piece[c][p], w[m][c]);
              acc[m][c] = mfma_bf16(fq, piece[c][p], acc[m][c]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);  // the pieces of one step at a time
      }
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * m + 4 * g + r;
          const float grow = s.grow[i], beta = s.beta[i];
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            rhs[m][c][r] = beta * (rhs[m][c][r] - grow * w[m][c][r]);
            acc[m][c][r] *= grow;
          }
        }
    }

    // trees: the path's rows in earlier blocks, the nearest first
    if (!chain) {
      for (int e = b - 1; e >= 0; --e) {
        __syncthreads();
        const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4, v0 = vw + col * NC;
        load_rows<KD, RT, false>(a, s, v.row0 + e * R, R, key, s.t, &s.odd[e]);
        if (tid < R) {
          const int p = s.next[tid];
          unsigned long long m = 0;
          if (p >= e * R) {
            m = s.in[p];
            s.next[tid] = s.leave[p];
          }
          s.cross[tid] = m;
          if (m & s.odd[e]) s.behind[tid] = 1;
        }
        __syncthreads();
        for (int u = wave; u < 2 * RT * RT; u += kWaves) {
          const bool of_low = u < RT * RT;
          const int at = of_low ? u : u - RT * RT, bi = at / RT, bj = at - bi * RT, i = 16 * bi + col;
          f32x4 x = pair_tile<KD, RT>(of_low ? s.k : s.q, s.t, bi, bj);
          const unsigned long long in = s.cross[i];
          const double gi = s.sum[base + i];
          const float f = of_low ? -s.beta[i] : 1.0f;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = 16 * bj + 4 * g + r;
            x[r] = (in >> j) & 1 ? f * __expf((float)(gi - s.sum[e * R + j])) * x[r] : 0.0f;
          }
          (of_low ? s.far_low : s.far_see)[at][lane] = x;
        }
        __syncthreads();
        const unsigned long long odd = s.odd[e];
        const float* deltas = a.c.delta + delta_at(a.c, a.layer, v.row0 + e * R, head);  // as this lane wrote them
#pragma unroll
        for (int mj = 0; mj < RT; ++mj) {
          f32x4 d[NC];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = 16 * mj + 4 * g + r;
            const float* p = deltas + ((uint32_t)j * hv * VD + v0);
#pragma unroll
            for (int c = 0; c < NC; ++c) d[c][r] = (odd >> j) & 1 ? 0.0f : p[c];
          }
#pragma unroll
          for (int m = 0; m < RT; ++m)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              rhs[m][c] = mfma_f32(s.far_low[m * RT + mj][lane], d[c], rhs[m][c]);
              acc[m][c] = mfma_f32(s.far_see[m * RT + mj][lane], d[c], acc[m][c]);
            }
        }
      }
    }
    __syncthreads();

    // the triangular system, and the outputs
    const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4, v0 = vw + col * NC;
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        f32x4 d = mfma_f32(s.inv[m][lane], rhs[m][c], f32x4{0, 0, 0, 0});
        rhs[m][c] = d;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          if (i > m) rhs[i][c] = mfma_f32(s.low[i * RT + m][lane], d, rhs[i][c]);
          if (i >= m) acc[i][c] = mfma_f32(s.see[i * RT + m][lane], d, acc[i][c]);
        }
      }
    const unsigned long long odd = s.odd[b], odd_q = s.odd_q;
    uint16_t* outs = a.out + ((size_t)row0 * hv + head) * VD;
    float* deltas = a.c.delta + delta_at(a.c, a.layer, row0, head);
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * m + 4 * g + r;
        if (i < n) {
          const bool no = before || (s.in[base + i] & odd) || (!chain && s.behind[i]);
          const bool no_q = no || ((odd_q >> i) & 1);
          uint16_t o[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) o[c] = no_q ? 0x7FC0 : f32_to_bf16_rne(a.scale * acc[m][c][r]);
          const uint32_t at = (uint32_t)i * hv * VD + v0;
          uint16_t* p = outs + at;
          if constexpr (NC == 2)
            *reinterpret_cast<uint32_t*>(p) = o[0] | ((uint32_t)o[1] << 16);
          else
            *p = o[0];
          if (!a.keep) {
#pragma unroll
            for (int c = 0; c < NC; ++c) deltas[at + c] = no ? __builtin_nanf("") : rhs[m][c][r];
          }
        }
      }
    before = before || (chain && odd);

    // chains: the state behind the block
    if (chain && (a.keep || b + 1 < blocks)) {
      const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4;
      const float keep = s.grow[n - 1];
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[t][c][r] *= keep;
#pragma unroll
      for (int m = 0; m < RT; m += 2) {
        uint4 piece[NC][3];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          f32x4 x[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (m + i < RT)
#pragma unroll
              for (int r = 0; r < 4; ++r) x[i][r] = s.part[16 * (m + i) + 4 * g + r] * rhs[m + i][c][r];
          split3(x[0], x[1], piece[c][0], piece[c][1], piece[c][2]);
        }
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          const uint16_t* p = s.t + (16 * t + col) * TS + 16 * m + 4 * g;
          uint4 f;
          if constexpr (RT == 1) {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            f = make_uint4(x.x, x.y, 0, 0);
          } else {
            f = fragment(p);
          }
#pragma unroll
          for (int q = 2; q >= 0; --q)
#pragma unroll
            for (int c = 0; c < NC; ++c) S[t][c] = mfma_bf16(f, piece[c][q], S[t][c]);
        }
      }
    }
  }
  if (!a.keep) return;
  const uint32_t to_state = state_place();
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float* p = state + (16 * t + r) * VD + to_state;
#pragma unroll
      for (int c = 0; c < NC; ++c) p[c] = before ? __builtin_nanf("") : S[t][c][r];
    }
  const int share = (a.c.channels + gridDim.x - 1) / gridDim.x;
  advance_window(a.c, a.layer, v.slot, v.rows, blockIdx.x * share, min(a.c.channels, (int)(blockIdx.x + 1) * share),
                 [&](int j) { return v.row0 + j; });
}

template <int KD, int VD>
void launch(const DeltaRuleArgs& a, hipStream_t s) {
  const int rows = (a.st.total + a.st.num_seq - 1) / a.st.num_seq;
  const dim3 grid(a.c.value_heads * (VD / 64), a.st.num_seq);
  if (rows <= 16)
    delta_rule_kernel<KD, VD, 1, 1><<<grid, kThreads, 0, s>>>(a);
  else if (rows <= 32)
    delta_rule_kernel<KD, VD, 2, 1><<<grid, kThreads, 0, s>>>(a);
  else
    delta_rule_kernel<KD, VD, 4, 1><<<grid, kThreads, 0, s>>>(a);
}

}  // namespace

hipError_t launch_delta_rule(const DeltaRuleArgs& a, hipStream_t s) {
  if (a.c.key_dim == 64)
    a.c.value_dim == 64 ? launch<64, 64>(a, s) : launch<64, 128>(a, s);
  else
    a.c.value_dim == 64 ? launch<128, 64>(a, s) : launch<128, 128>(a, s);
  return hipGetLastError();
}

}  // namespace w12
